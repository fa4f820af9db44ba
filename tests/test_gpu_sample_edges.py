"""Token sampling: rows whose limits meet, equal logits and repeated calls."""
import numpy as np
import pytest
import torch

from tests.test_gpu_sample import check, logits, u_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [2, 9, 90, 310])
def test_flat_rows_under_top_p_and_min_p_repeat(kap, rows):
    """fp32 rows under both limits: the bounds of the border come from sums over all bins, one after the other and ahead of
    a scan. Each row against 64 bits, and 60 calls equal to the bit, alone and with other work beside them."""
    V = 50021 if rows < 300 else 20011
    lg = logits(rows, V, torch.float32, rows, scale=1.3, lift=False)
    kw = dict(T=0.9 + 0.1 * (np.arange(rows) % 3), p=0.4 + 0.13 * (np.arange(rows) % 4), mp=1e-3)
    u = u_of(rows, 1)
    want = check(kap, lg, u, **kw)
    as_ = lambda v, dt=torch.float32: torch.as_tensor(np.broadcast_to(np.asarray(v), (rows,)).copy()).to(dt).cuda()  # noqa: E731
    args = dict(temperature=as_(kw["T"]), top_p=as_(kw["p"]), min_p=as_(kw["mp"]))
    uc, side, busy = as_(u), torch.cuda.Stream(), torch.randn(1 << 24, device="cuda")
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        tok, lp, kept = (torch.empty(rows, dtype=t, device="cuda") for t in (torch.int32, torch.float32, torch.int32))
        if i % 2:
            with torch.cuda.stream(side):
                busy.mul_(1.0)
        kap.kap_sample_tokens(lg, uc, tok, logprob=lp, kept=kept, **args)
        got.append((tok, lp, kept))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert (a.cpu().numpy() == b).all()
    assert kap.kap_device_error() == 0
