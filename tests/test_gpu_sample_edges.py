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


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [3, 900, 5003, 40000])
def test_min_p_above_one_keeps_the_first_token_alone(kap, V, dt):
    """No weight reaches it, and the first token is always kept: the lowest id of equal largest logits. At one, all of them."""
    lg = logits(5, V, dt, V, lift=False)
    lg[1] = 0.25
    lg[2, V // 2:] = lg[2].max() + 1.0
    lg[3, [0, V - 1]] = 30.0
    lg[4, :V - 2] = -float("inf")
    for mp in (1.0, 1.0000001, 1.5, 5.0, float("inf")):
        for kw in ({}, dict(p=0.5), dict(k=2), dict(k=2, p=0.3, T=0.6), dict(k=V - 1), dict(T=3.0)):
            for u in (0.0, 0.99999994):
                tok, lp, kept = check(kap, lg, np.full(5, u), mp=mp, **kw)
                if mp > 1.0:
                    assert (kept == 1).all() and (lp == 0.0).all() and (tok == lg.float().argmax(1).cpu().numpy()).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("low", [-1e9, -3.38e38])
def test_temperatures_at_which_masked_logits_weigh_as_much(kap, dt, low):
    """At temperatures past 1e38 a mask of a finite value takes nothing from a token's weight."""
    rows, V = 4, 10958
    lg = logits(rows, V, dt, 4, lift=False)
    lg[:, torch.arange(V) % 97 != 0] = low
    for T in (float("inf"), 3e38, 1e31):
        for kw in (dict(p=0.43), dict(p=0.9, mp=1e-6), dict(p=0.004, k=9000), dict(mp=0.3)):
            check(kap, lg, u_of(rows, 3), T=T, **kw)
