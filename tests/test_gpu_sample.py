"""Token sampling against 64 bits: the token and the number of kept tokens exactly, whatever limits it."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def plain(x, T=1.0, k=0, p=1.0, mp=0.0, u=0.5):
    """{(token, number kept): log probability} of what may come out of one row, in 64 bits. Weights are
    held to 2^-45 of the largest, so a border within V 2^-44 of a sum may fall either way (none of that counts on rows
    whose sums are exact)."""
    x = x.astype(np.float64) + 0.0
    V = len(x)
    ids = np.lexsort((np.arange(V), np.isnan(x), np.where(np.isnan(x), np.inf, -x)))
    m = x[ids[0]]
    if np.isnan(x).any() or not np.isfinite(m):
        return {(int(ids[0]), 0): np.nan}
    if not T > 0:
        return {(int(ids[0]), 1): 0.0}
    with np.errstate(under="ignore", over="ignore"):
        w = np.where(np.isneginf(x), 0.0, np.exp((np.where(np.isneginf(x), m, x) - m) / T))[ids]
    finite = ~np.isneginf(x[ids])
    n = int(finite.sum())
    slack = V * 2.0 ** -44
    if mp > 0:
        n = min(n, max(1, int((w[:n] >= mp).sum())))
    if 0 < k < n:
        n = k
    ns = {n}
    if p < 1:
        c = np.cumsum(w[:n])
        ns = {max(1, int(np.searchsorted(c, p * c[-1] + e)) + 1) for e in (-slack, 0.0, slack)}
        ns = {min(z, n) for z in ns}
    may = {}
    u = 0.0 if np.isnan(u) else min(max(u, 0.0), 0.99999994)
    for z in ns:
        keep = np.sort(ids[:z])
        wk = np.zeros(V)
        wk[ids[:z]] = w[:z]
        c = np.cumsum(wk[keep])
        for e in (-slack, 0.0, slack):
            j = min(int(np.searchsorted(c, u * c[-1] + e, side="right")), z - 1)
            t = int(keep[j])
            may[t, z] = (x[t] - m) / T - np.log(c[-1])
    return may


def call(kap, lg, u, T=None, k=None, p=None, mp=None):
    rows = lg.shape[0]
    tok = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((rows,), 7.0, device="cuda")
    kept = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    as_ = lambda v, dt: None if v is None else torch.as_tensor(np.broadcast_to(np.asarray(v), (rows,)).copy()).to(dt).cuda()  # noqa: E731
    kap.kap_sample_tokens(lg, as_(u, torch.float32), tok, temperature=as_(T, torch.float32), top_k=as_(k, torch.int32),
                          top_p=as_(p, torch.float32), min_p=as_(mp, torch.float32), logprob=lp, kept=kept)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), lp.cpu().numpy(), kept.cpu().numpy()


def check(kap, lg, u, T=None, k=None, p=None, mp=None):
    rows, V = lg.shape
    tok, lp, kept = call(kap, lg, u, T, k, p, mp)
    x = lg.float().cpu().numpy()
    at = lambda v, r, dt, off: off if v is None else float(dt(np.broadcast_to(np.asarray(v), (rows,))[r]))  # noqa: E731
    for r in range(rows):
        may = plain(x[r], at(T, r, np.float32, 1.0), int(at(k, r, np.int32, 0)), at(p, r, np.float32, 1.0),
                    at(mp, r, np.float32, 0.0), at(u, r, np.float32, 0.5))
        assert (int(tok[r]), int(kept[r])) in may, (r, tok[r], kept[r], may)
        l = may[int(tok[r]), int(kept[r])]
        # one rounding to fp32, and sums that are off by V 2^-44 of a sum of at least 1
        assert np.isnan(l) == np.isnan(lp[r]) and not abs(lp[r] - l) > 2.0 ** -23 * abs(l) + V * 2.0 ** -43, (r, lp[r], l)
    return tok, lp, kept


def logits(rows, V, dt, seed, scale=2.5, lift=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, V, generator=g) * scale
    if lift:
        x[::2, torch.randint(0, V, (5,), generator=g)] += 9.0
    return x.to(dt).cuda()


def u_of(rows, seed=0):
    return np.random.default_rng(seed).integers(0, 1 << 24, rows).astype(np.float32) * np.float32(2.0 ** -24)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4097, 32000, 128256])
@pytest.mark.parametrize("kw", [dict(), dict(k=5), dict(p=0.9), dict(mp=0.02), dict(k=300, p=0.7, mp=0.001),
                                dict(k=20000), dict(p=0.999), dict(T=0.3, p=0.5), dict(T=3.0, k=4000, p=0.99)],
                         ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()) or "none")
def test_limits(kap, V, dt, kw):
    rows = 6
    check(kap, logits(rows, V, dt, V), u_of(rows, V), **kw)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 3, 9, 40, 160, 700])
def test_row_counts_and_settings_a_row(kap, rows, dt):
    """From a cluster of 16 CTAs a row to a CTA a row, each row with settings of its own."""
    V = 5003
    r = np.arange(rows)
    check(kap, logits(rows, V, dt, rows), u_of(rows), T=np.where(r % 7 == 3, 0.0, 0.5 + 0.25 * (r % 5)),
          k=np.where(r % 3 == 0, 0, 10 * r + 1), p=np.where(r % 4 == 0, 1.0, 0.2 + 0.15 * (r % 5)),
          mp=np.where(r % 5 == 0, 0.05, 0.0))


@pytest.mark.parametrize("rows", [2, 90, 310])
@pytest.mark.parametrize("steps", [0, 256, 3])
def test_top_p_of_flat_rows(kap, rows, steps):
    """Borders that tens of thousands of fp32 logits lie above: all different, in runs of tens of equal ones, and in runs that
    are longer than any list of candidates."""
    V = 50021 if rows < 300 else 20011
    lg = logits(rows, V, torch.float32, rows, scale=1.5, lift=False)
    if steps:
        lg = (lg * steps).round() / steps
    r = np.arange(rows)
    check(kap, lg, u_of(rows, steps), T=0.8 + 0.2 * (r % 4), p=np.where(r % 5 == 4, 0.0001, 0.3 + 0.23 * (r % 4)),
          mp=np.where(r % 3 == 1, 1e-3, 0.0), k=np.where(r % 7 == 6, V - 1, 0))
    assert kap.kap_device_error() == 0


@pytest.mark.parametrize("T", [1.0, 0.7, 1.3])
def test_borders_that_a_weights_last_bits_decide(kap, T):
    """Two tokens of weights 1 and w whose share 1 / (1 + w) lies 2^-37 to 2^-33 from a value of top_p. A weight is right to
    2^-38 of itself and a unit of 2^-44, so the share to w / (1 + w)^2 of 2^-38 and a unit, less than 2^-39: every row falls
    on its own side."""
    rng = np.random.default_rng(int(10 * T))
    T = float(np.float32(T))
    x = rng.uniform(0.05, 12.0, (1 << 20, 2)).astype(np.float32)
    x.sort(axis=1)
    share = 1.0 / (1.0 + np.exp((x[:, 0].astype(np.float64) - x[:, 1]) / T))
    p = share.astype(np.float32)
    off = np.abs(p - share)
    at = np.flatnonzero((off > 2.0 ** -37) & (off < 2.0 ** -33) & (p < 1))[:2000]
    assert len(at) > 100
    lg = torch.from_numpy(x[at]).cuda()
    _, _, kept = call(kap, lg, 0.0, T=T, p=p[at])
    assert (kept == np.where(share[at] >= p[at], 1, 2)).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_temperatures_past_any_use(kap, dt):
    """Weights that are all the same, and a step apart, under limits that flat rows meet."""
    rows, V = 6, 5003
    check(kap, logits(rows, V, dt, 2, lift=False), u_of(rows), T=np.array([np.inf, 1e30, 1e6, 1e38, 300.0, 1e-30]),
          p=np.array([0.5, 0.5, 0.9, 0.001, 0.99, 0.9]))


def test_a_rows_result_does_not_depend_on_the_batch(kap):
    """The same rows alone (a cluster each) and in a large batch (a CTA each): equal to the bit."""
    lg = logits(8, 128256, torch.float32, 3)
    u = u_of(8)
    one = call(kap, lg, u, T=0.9, p=0.95)
    many = call(kap, lg.repeat(80, 1), np.tile(u, 80), T=0.9, p=0.95)
    for a, b in zip(one, many):
        assert (np.tile(a, 80) == b).all()


@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 0), (5, 3), (61, 7), (8, 1)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_strides_and_alignment(kap, dt, pad, shift):
    rows, V = 5, 1777
    flat = torch.full((rows * (V + pad) + shift + 8,), 50.0, dtype=dt, device="cuda")   # the gaps would win
    lg = flat[shift:shift + rows * (V + pad)].view(rows, V + pad)[:, :V]
    lg.copy_(logits(rows, V, dt, 1))
    check(kap, lg, u_of(rows), k=50, p=0.9)
    check(kap, lg, u_of(rows, 1))


def test_ties(kap):
    """Equal logits: top-k keeps the lowest ids, top-p as many as its share, and a draw counts in id order."""
    V = 1000
    x = torch.zeros(12, V)
    x[2:4, 5::7] = 1.0
    x[4:6] = -3.5
    x[6:8, 500:] = -float("inf")
    x[8:10, ::2] = 2.0 ** -20
    x[10:, 1:] = -0.0
    for dt in (torch.bfloat16, torch.float32):
        lg = x.to(dt).cuda()
        for kw in (dict(k=3), dict(k=143), dict(k=200), dict(p=0.5), dict(p=0.1), dict(k=77, p=0.5), dict(k=150, p=0.99), {}):
            for u in (0.0, 0.4999, 0.75, 0.99999994):
                check(kap, lg, np.full(12, u), **kw)
    big = torch.zeros(2, 128256, dtype=torch.bfloat16, device="cuda")
    check(kap, big, np.array([0.3, 0.9]), p=0.25)
    check(kap, big, np.array([0.3, 0.9]), k=100000, p=0.25)


def test_ends_of_the_random_number(kap):
    lg = logits(6, 3000, torch.float32, 5)
    lg[1, :10] = -float("inf")
    for u in (0.0, 2.0 ** -24, 0.5, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, float("nan"), float("inf"), 1e-42):
        check(kap, lg, np.full(6, u))
        check(kap, lg, np.full(6, u), k=7, p=0.8)


def test_settings_out_of_range(kap):
    lg = logits(4, 2000, torch.bfloat16, 6)
    u = u_of(4)
    for kw in (dict(k=-3), dict(k=2 ** 31 - 1), dict(p=0.0), dict(p=-1.0), dict(p=2.0), dict(mp=1.0), dict(mp=5.0),
               dict(mp=-1.0), dict(T=-1.0), dict(T=0.0, k=5, p=0.1), dict(T=1e-3, p=0.9), dict(T=1e-30), dict(T=1e3, p=0.5),
               dict(T=1e30, k=700)):
        check(kap, lg, u, **kw)
    # NaN settings count as off, a NaN temperature as none above 0
    nan = float("nan")
    a = call(kap, lg, u, T=0.7)
    b = call(kap, lg, u, T=0.7, p=nan, mp=nan)
    assert all((x == y).all() for x, y in zip(a, b))
    assert (call(kap, lg, u, T=nan)[0] == call(kap, lg, u, T=0.0)[0]).all()


def test_rows_without_a_distribution(kap):
    V = 300
    x = torch.randn(6, V, generator=torch.Generator().manual_seed(0))
    x[0, 17] = float("nan")
    x[1, 40], x[1, 20] = float("inf"), float("inf")
    x[2] = -float("inf")
    x[3] = float("nan")
    x[4] = float("nan")
    x[4, 9] = -float("inf")
    x[5, :-1] = -float("inf")
    for dt in (torch.bfloat16, torch.float32):
        for kw in ({}, dict(k=3, p=0.5), dict(T=0.0), dict(mp=0.1)):
            tok, lp, kept = check(kap, x.to(dt).cuda(), np.full(6, 0.7), **kw)
            assert tok[1] == 20 and tok[2] == 0 and tok[3] == 0 and tok[4] == 9 and tok[5] == V - 1
            assert kept.tolist()[:5] == [0] * 5 and kept[5] == 1 and lp[5] == 0.0


def test_logits_over_the_whole_range(kap):
    g = torch.Generator().manual_seed(2)
    for dt in (torch.bfloat16, torch.float32):
        x = torch.randn(8, 4000, generator=g)
        x[0] *= 1e30
        x[1] *= 1e-30
        x[2] *= 1e-42
        x[3] += 1e6
        x[4] = 3.0e38 * torch.sign(x[4])
        x[5] = 1.0 + x[5] * 2.0 ** -22
        x[6, 100:] -= 200.0
        x[7] = -1e5 + 3 * x[7]
        for kw in ({}, dict(k=900), dict(p=0.6), dict(k=2000, p=0.9, mp=1e-3), dict(T=1e5, p=0.3)):
            check(kap, x.to(dt).cuda(), u_of(8, 4), **kw)


def test_vocabularies_past_the_usual(kap):
    lg = logits(2, 1 << 20, torch.bfloat16, 8)
    check(kap, lg, u_of(2), p=0.9)
    check(kap, lg, u_of(2), k=70000)


def test_captured_and_on_another_stream(kap):
    lg, u = logits(20, 32000, torch.bfloat16, 9), torch.from_numpy(u_of(20)).cuda()
    tok = torch.zeros(20, dtype=torch.int32, device="cuda")
    p = torch.full((20,), 0.9, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kap.kap_sample_tokens(lg, u, tok, top_p=p, stream=st)
    st.synchronize()
    want = tok.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kap.kap_sample_tokens(lg, u, tok, top_p=p)
    tok.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(tok, want) and kap.kap_device_error() == 0


def test_the_share_of_draws_is_the_share_of_weight(kap):
    """A million random numbers over 4 tokens: counts within 6 deviations of their shares."""
    n = 1 << 20
    lg = torch.tensor([[0.0, 1.0, -1.0, 2.0]]).cuda().expand(n, 4).contiguous()
    u = torch.rand(n, generator=torch.Generator().manual_seed(1)).cuda()
    tok = torch.empty(n, dtype=torch.int32, device="cuda")
    kap.kap_sample_tokens(lg, u, tok)
    share = torch.softmax(lg[0].double(), 0).cpu()
    got = torch.bincount(tok.long(), minlength=4).cpu().double()
    assert ((got - n * share).abs() <= 6 * torch.sqrt(n * share * (1 - share))).all()


def test_refusals(kap):
    lg, f = logits(3, 100, torch.bfloat16, 0), torch.zeros(3, device="cuda")
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        kap.kap_sample_tokens(lg.half(), f, i)
    with pytest.raises(TypeError):
        kap.kap_sample_tokens(lg, f, f)
    with pytest.raises(TypeError):
        kap.kap_sample_tokens(lg, f, i, top_k=f)
    with pytest.raises(ValueError):
        kap.kap_sample_tokens(lg, f[:2], i)
    with pytest.raises(ValueError):
        kap.kap_sample_tokens(lg.t().contiguous().t(), f, i)
    with pytest.raises(ValueError):
        kap.kap_sample_tokens(lg, f.cpu(), i)
    with pytest.raises(kap.KapError):
        kap.kap_sample_tokens(torch.zeros(1, (1 << 24) + 8, dtype=torch.bfloat16, device="cuda"), f[:1], i[:1])
    kap.kap_sample_tokens(lg[:0], f[:0], i[:0])
