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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("rows", [1, 4, 40])
def test_results_do_not_depend_on_what_ran_before(kap, rows, d):
    """A block of few query rows fills no more than its part of the 128 rows of a product; what an earlier call left in the
    others has no part in the results, not even in a rounding."""
    G = 4 if rows % 4 == 0 else 1
    s = make([1], [0], [152 * 128 * 6 + 37], [rows // G], hkv=1, G=G, d=d)
    # rows in all of both query buffers, of every CTA
    t = make([4], [152 * 16], [3] * 4, [64] * 4, hkv=1, G=1, d=d, seed=1)
    assert s["tq"] * G == rows and t["tq"] == 256
    got = []
    for scale in (0.0, 1e30, -1e30, 1e-3):
        u = {**t, "q": (t["q"].float() * scale).to(torch.bfloat16)}
        run(kap, u)
        got.append(run(kap, s))
    torch.cuda.synchronize()
    check(s, *got[0])
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    assert kap.kap_device_error() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("qo", [[0, 5000, 10, 5100], [0, 90, 40, 5100], [-7, 3, 9, 5100], [0, 10, 20, 6000], [0, 400, 300, 200]])
def test_window_offsets_that_do_not_rise(kap, dt, qo):
    """Rows that no group's records hold are left out and reported, and nothing outside the outputs is written."""
    s = make([1, 2], [9, 40], [7, 130, 0], [1, 1, 1], hkv=1, G=4, d=64, dt=dt)
    s["qo"] = torch.tensor(qo, dtype=torch.int32, device="cuda")
    s["tq"], s["windows"] = 5100, [16, 16, 16]
    s["q"] = torch.randn(5100, 4, 64, device="cuda").to(dt)
    n = kap.kap_shared_workspace_size(3, 1, 4, 64, 5100, 2)
    whole = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
    run(kap, s, ws=whole[256:256 + n])
    torch.cuda.synchronize()
    assert kap.kap_device_error() & 4
    assert (whole[:256] == 255).all() and (whole[256 + n:] == 255).all()
