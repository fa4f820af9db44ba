"""Attention of requests that share prefixes: addresses, offsets and neighbours that the documentation allows."""
import pytest
import torch

from tests.test_gpu_shared import check, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dt", [(128, torch.bfloat16), (64, torch.bfloat16), (128, torch.float32), (64, torch.float32)])
def test_a_workspace_at_any_multiple_of_16_bytes(kap, d, dt):
    """Records are stored 32 bytes at a time: the first part of a workspace lies on a multiple of that wherever the workspace
    starts, and the last one ends inside it."""
    s = make([3, 2], [40, 9], [7, 130, 0, 40, 300], [2, 1, 3, 1, 2], d=d, dt=dt)
    n = kap.kap_shared_workspace_size(s["R"], 2, s["hq"], d, s["tq"], 2)
    for off in (0, 16, 32, 48, 128, 240):
        whole = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
        assert whole.data_ptr() % 256 == 0
        out, lse = run(kap, s, ws=whole[off:off + n])
        torch.cuda.synchronize()
        check(s, out, lse)
        assert (whole[:off] == 255).all() and (whole[off + n:] == 255).all(), off
    assert kap.kap_device_error() == 0
