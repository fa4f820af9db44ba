"""Values that are not finite, at tokens of a verify window: a row that does not see the token keeps its bits, and of a row
that sees it only the dims that the value reaches change."""
import numpy as np
import pytest
import torch

from tests.packed_reference import PAGE
from tests.test_gpu_packed_attention import KINDS, Cache

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")

CASES = [
    # tokens with the window, window, hkv, G, d, kinds, width of the table (129 pages and more are shared out over CTAs)
    (40, 8, 2, 1, 64, "packed", 4),
    (40, 8, 2, 1, 64, "sixteen", 4),
    (75, 4, 1, 4, 128, "packed", 6),       # two column tiles
    (75, 4, 1, 4, 128, "tail16", 6),
    (66, 6, 2, 4, 128, "packed", 6),       # three
    (66, 6, 2, 4, 64, "sixteen", 6),
    (81, 8, 1, 4, 128, "packed", 7),       # four; the window spans two pages
    (81, 8, 1, 4, 128, "tail16", 7),
    (70, 8, 1, 6, 128, "packed", 6),       # two groups of warps
    (70, 8, 1, 6, 128, "tail16", 6),
    (50, 8, 2, 8, 64, "packed", 5),
    (50, 20, 1, 3, 128, "sixteen", 5),     # longer than a page
    (2300, 8, 1, 4, 128, "tail16", 150),
    (2300, 4, 1, 2, 128, "packed", 150),
]
# (scale, lowest) of a group's parameters; of 16-bit pages the values at dims 5, 40 and d - 1
PARAMS = {"nan": (NAN, NAN), "inf": (0.5, INF), "scale": (INF, -1.0)}


def _run(kap, c, n, w, width, q):
    dev = "cuda"
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    bt = torch.full((1, max(width, c.mp)), -1, dtype=torch.int32)
    bt[:, :c.mp] = c.bt
    pool = kap.PackedPool(kap.KVPool(c.K.to(dev), c.V.to(dev), c.hkv * c.G), c.packed.to(dev))
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full(q.shape[:2], 7.0, device=dev)
    ws = kap.workspace(kap.kap_packed_workspace_size(1, c.hkv, c.hkv * c.G, c.d, w), dev)
    kap.kap_attn_verify_packed(pool, kap.PageMap(bt.to(dev), t([n]), t([n])),
                               kap.VerifyPolicy(t([0, w]), t([n - w]), w, w), q, out, lse, ws)
    assert kap.kap_device_error() == 0
    return out.cpu(), lse.cpu()


@pytest.mark.parametrize("kind", list(PARAMS))
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-q{c[1]}-h{c[2]}x{c[3]}-d{c[4]}-{c[5]}")
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(kap, case, kind):
    n, w, hkv, G, d, kinds, width = case
    nb, head = d // 64, hkv - 1
    # tokens of the window (its first is seen by every row) and one before it
    for at in sorted({-17, 0, 1, w // 2, w - 1}):
        c = Cache(kap, [n], hkv, G, d, KINDS[kinds], seed=n + w)
        q = c.query(w).to("cuda")
        pos = n - w + at
        pid, o = int(c.bt[0, pos // PAGE]), pos % PAGE
        hit = torch.zeros(d, dtype=torch.bool)
        got = []
        for bad in (False, True):   # first with zeros in the same places
            if pid < c.P16:
                dims = [5, 40, d - 1]
                vals = [INF, -INF, NAN] if kind != "nan" else [NAN] * 3
                for x, v in zip(dims, vals):
                    c.V[pid, head, o, x] = v if bad else 0.0
                    hit[x] = True
            else:
                par = c.packed[pid - c.P16, head, 2 * nb * 512:].view(torch.bfloat16).view(2, nb, PAGE, 2)
                par[1, nb - 1, o] = torch.tensor(PARAMS[kind] if bad else (0.0, 0.0), dtype=torch.bfloat16)
                hit[64 * (nb - 1):] = True
            got.append(_run(kap, c, n, w, width, q))
        (clean, l0), (out, l1) = got
        assert torch.isfinite(clean).all() and torch.equal(l0, l1), at
        mine = torch.arange(hkv * G) // G == head
        sees = torch.arange(w) >= at
        touched = sees[:, None, None] & mine[None, :, None] & hit[None, None, :]
        assert torch.equal(out[~touched], clean[~touched]), at
        assert not torch.isfinite(out[touched]).any(), at
