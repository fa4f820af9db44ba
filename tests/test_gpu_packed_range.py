"""Attention over packed and 16-bit pages at the ends of the range: values of far-apart magnitude in one row, values that
fp32 barely holds."""
import pytest
import torch

from tests.packed_reference import PAGE
from tests.test_gpu_packed_attention import KINDS, Cache

pytestmark = pytest.mark.gpu


def _attend(kap, c, n, q):
    dev = "cuda"
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    pool = kap.PackedPool(kap.KVPool(c.K.to(dev), c.V.to(dev), c.G), c.packed.to(dev))
    out = torch.empty(1, c.G, c.d, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(1, c.G, device=dev)
    ws = kap.workspace(kap.kap_packed_workspace_size(1, 1, c.G, c.d, 1), dev)
    kap.kap_attn_verify_packed(pool, kap.PageMap(c.bt.to(dev), t([n]), t([n])),
                               kap.VerifyPolicy(t([0, 1]), t([n - 1]), 1, 1), q.to(dev), out, lse, ws)
    assert kap.kap_device_error() == 0
    return out, lse


def _params(c):
    nb = c.d // 64
    return c.packed[:, :, 2 * nb * 512:].view(torch.bfloat16).view(c.P4, c.hkv, 2, nb, PAGE, 2)


# log2 of the factors of 16-bit values, packed values, queries and keys; None is a factor of zero. Values are below 2^5
# before, and a sum over 400 tokens takes 2^17 more where a reference lags: 2^105 is within fp32.
@pytest.mark.parametrize("v16,v4,qs,ks", [
    (90, 90, 0, 0), (105, 105, 0, 0), (-90, -90, 0, 0),
    (90, -90, 0, 0), (90, None, 0, 0), (60, -40, 0, 0), (40, None, 0, 0),
    (-90, 90, 0, 0), (None, 90, 0, 0), (None, None, 0, 0), (105, None, 0, 0), (None, 105, 0, 0), (0, 105, 0, 0),
    (0, 0, 90, -90), (0, 0, -90, 90), (90, 90, 90, -90),
])
@pytest.mark.parametrize("kinds", ["mixed", "tail16"])
def test_far_magnitudes(kap, v16, v4, qs, ks, kinds):
    n, f = 400, lambda e: 0.0 if e is None else 2.0 ** e
    c = Cache(kap, [n], 1, 4, 128, KINDS[kinds], seed=5)
    c.K, c.V = c.K * f(ks), torch.nan_to_num(c.V) * f(v16)
    par = _params(c)
    par[:, :, 0] *= f(ks)
    par[:, :, 1] = torch.nan_to_num(par[:, :, 1]) * f(v4)
    q = (c.query(1).float() * f(qs)).to(torch.bfloat16)
    out, lse = _attend(kap, c, n, q)
    for head in range(4):
        c.check(out, lse, q, 0, head, [c.page(int(c.bt[0, i // PAGE]), 0)[i % PAGE] for i in range(n)])
