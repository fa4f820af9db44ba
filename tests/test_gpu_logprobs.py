"""Log probabilities of given tokens, entropy, rank and best alternatives against 64 bits; ids and ranks exactly."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def order(x):
    """Token ids of a row by (logit descending, lower id first, NaN last)."""
    x = x.astype(np.float64)
    key = np.where(np.isnan(x), np.inf, -x)           # ascending
    return np.lexsort((np.arange(len(x)), np.isnan(x), key))


def plain(x, tok, top):
    x = x.astype(np.float64)
    V = len(x)
    ids = order(x)
    rank = int(np.where(ids == tok)[0][0]) if 0 <= tok < V else V
    m = x.max()
    if not np.isfinite(m) or np.isnan(x).any():
        lp = np.full(V, np.nan)
        ent = np.nan
    else:
        lp = (x - m) - np.log(np.exp(x - m).sum())   # m + log(...) would lose the logarithm next to a huge m
        p = np.exp(lp[np.isfinite(lp)])
        ent = -(p * lp[np.isfinite(lp)]).sum()
    return (lp[tok] if 0 <= tok < V else -np.inf), ent, rank, ids[:top], lp[ids[:top]]


def run(kap, lg, tok, top, entropy=True, rank=True, ws=None):
    rows, V = lg.shape
    f = dict(dtype=torch.float32, device="cuda")
    i = dict(dtype=torch.int32, device="cuda")
    lp, ent, rk = torch.full((rows,), 7.0, **f), torch.full((rows,), 7.0, **f), torch.full((rows,), -7, **i)
    ids, tlp = torch.full((rows, top), -7, **i), torch.full((rows, top), 7.0, **f)
    ws = kap.workspace(kap.kap_logprobs_workspace_size(rows, V), "cuda") if ws is None else ws
    kap.kap_token_logprobs(lg, tok, lp, ws, entropy=ent if entropy else None, rank=rk if rank else None,
                           top_ids=ids if top else None, top_logprobs=tlp if top else None)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (lp, ent, rk, ids, tlp)]


def check(lg, tok, top, got, rows=None):
    """Sums of V terms in fp32: a lane adds at most V / 256 + 64 of them in a row, each rounding 2^-24, and each
    exponential is off by 2^-22 and by the rounding of its argument, d * 2^-23 for a logit d below the maximum, which
    weighs d e^-d <= 0.37 of it. The entropy's sum has the same errors on sum p |log p|."""
    x = lg.float().cpu().numpy()
    lp, ent, rank, ids, tlp = got
    V = x.shape[1]
    t = tok.cpu().numpy()
    rel = (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -21
    for r in range(x.shape[0]) if rows is None else rows:
        wl, we, wr, wi, wt = plain(x[r], int(t[r]), top)
        near = lambda a, b, tol: (np.isnan(a) and np.isnan(b)) or a == b or abs(a - b) <= tol  # noqa: E731
        assert near(lp[r], wl, rel + 2.0 ** -22 * abs(wl) if np.isfinite(wl) else 0), (r, lp[r], wl)
        assert near(ent[r], we, (rel + 2.0 ** -22) * (1 + abs(we))), (r, ent[r], we)
        assert rank[r] == wr, (r, rank[r], wr)
        assert ids[r].tolist() == wi.tolist(), r
        for a, b in zip(tlp[r], wt):
            assert near(a, b, rel + 2.0 ** -22 * abs(b) if np.isfinite(b) else 0), (r, a, b)


def logits(rows, V, dt, seed, pad=0, off=0, scale=2.5):
    g = torch.Generator().manual_seed(seed)
    full = (scale * torch.randn(rows, V + pad + off, generator=g)).to(dt)
    return full.to("cuda")[:, off:off + V], torch.randint(0, V, (rows,), generator=g, dtype=torch.int32).to("cuda")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,V,top,pad,off", [
    (1, 1, 1, 0, 0), (3, 2, 2, 0, 0), (5, 31, 5, 0, 0), (4, 513, 32, 0, 0), (7, 1000, 20, 8, 0), (2, 4097, 3, 0, 0),
    (3, 5000, 5, 3, 1), (9, 32000, 20, 1, 3), (2, 50257, 1, 0, 0), (1, 128256, 32, 0, 0), (20, 128256, 5, 0, 0),
    (700, 600, 4, 0, 0), (1300, 2050, 0, 5, 7),
])
def test_against_64_bits(kap, dt, rows, V, top, pad, off):
    lg, tok = logits(rows, V, dt, V + rows, pad, off)
    got = run(kap, lg, tok, top)
    check(lg, tok, top, got, rows=range(0, rows, max(1, rows // 12)))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [40, 3000, 70000])
def test_hard_rows(kap, dt, V):
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(dt).min
    lg, tok = logits(18, V, dt, 5)
    lg = lg.clone()
    lg[0] = 0.0                              # all equal
    lg[1] = -inf                             # nothing left by the mask
    lg[2, : V // 2] = -inf                   # half masked
    lg[3] = low                              # the type's lowest value throughout: equal logits
    lg[4, 1:] = low                          # masked with the lowest value, one left
    lg[5, 1:] = -inf
    lg[6, V // 3] = nan
    lg[7, V // 3] = inf
    lg[8] = torch.arange(V, device="cuda").to(dt)       # ascending (with ties in bf16)
    lg[9] = -torch.arange(V, device="cuda").to(dt)      # descending
    lg[10] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0).to(dt)   # zeros of both signs are equal
    lg[11] = lg[11] * 1000                   # large logits
    lg[12] = lg[12] + 10000
    lg[13] = nan
    lg[14, ::3] = nan
    lg[15] = torch.finfo(dt).max             # the largest finite value throughout
    lg[16, :-1] = -inf                       # only the last token
    lg[17, 5] = low
    tok[0], tok[4], tok[5], tok[6] = V - 1, 3, 0, V // 3
    tok[14], tok[2], tok[17] = 3, 1, 5
    got = run(kap, lg, tok, min(32, V))
    check(lg, tok, min(32, V), got)


def test_tokens_outside_and_optional_outputs(kap):
    lg, tok = logits(4, 777, torch.float32, 1)
    tok[0], tok[1], tok[2] = -1, 777, 1 << 30
    got = run(kap, lg, tok, 3)
    check(lg, tok, 3, got)
    bare = run(kap, lg, tok, 0, entropy=False, rank=False)
    assert np.array_equal(bare[0], got[0]) and (bare[1] == 7).all() and (bare[2] == -7).all()


def test_no_rows(kap):
    lg = torch.empty(0, 100, device="cuda")
    z = torch.empty(0, dtype=torch.int32, device="cuda")
    kap.kap_token_logprobs(lg, z, torch.empty(0, device="cuda"), kap.workspace(1, "cuda"))


def test_same_bits_again_in_graphs_and_on_streams(kap):
    """Split rows are joined in a fixed order: repeats, replays and concurrent streams give the same bits."""
    a, ta = logits(3, 128256, torch.bfloat16, 3)
    b, tb = logits(3, 128256, torch.bfloat16, 4)
    ref = [run(kap, a, ta, 20), run(kap, b, tb, 20)]
    size = kap.kap_logprobs_workspace_size(3, 128256)
    ws = kap.workspace(size, "cuda")
    for _ in range(3):
        for (x, t), want in zip(((a, ta), (b, tb)), ref):
            for g, w in zip(run(kap, x, t, 20, ws=ws), want):
                assert np.array_equal(g, w)
    f, i = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    outs = [(torch.empty(3, **f), torch.empty(3, **f), torch.empty(3, **i), torch.empty(3, 20, **i),
             torch.empty(3, 20, **f), kap.workspace(size, "cuda")) for _ in range(2)]
    x, t = a.clone(), ta.clone()
    g = torch.cuda.CUDAGraph()
    o = outs[0]
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        kap.kap_token_logprobs(x, t, o[0], o[5], entropy=o[1], rank=o[2], top_ids=o[3], top_logprobs=o[4])
    for src, st, want in ((b, tb, ref[1]), (a, ta, ref[0])):
        x.copy_(src)
        t.copy_(st)
        g.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(y.cpu().numpy(), w) for y, w in zip(o, want))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        for s, (src, st), o in zip(streams, ((a, ta), (b, tb)), outs):
            kap.kap_token_logprobs(src, st, o[0], o[5], entropy=o[1], rank=o[2], top_ids=o[3], top_logprobs=o[4],
                                   stream=s)
    torch.cuda.synchronize()
    for o, want in zip(outs, ref):
        assert all(np.array_equal(y.cpu().numpy(), w) for y, w in zip(o, want))


def test_binding_refusals(kap):
    lg, tok = logits(2, 64, torch.float32, 1)
    lp = torch.empty(2, device="cuda")
    ws = kap.workspace(kap.kap_logprobs_workspace_size(2, 64), "cuda")
    call = lambda lg=lg, tok=tok, lp=lp, ws=ws, **kw: kap.kap_token_logprobs(lg, tok, lp, ws, **kw)  # noqa: E731
    call()
    for bad in (dict(lg=lg.half()), dict(lg=lg.cpu())):
        with pytest.raises(TypeError):
            call(**bad)
    i = dict(dtype=torch.int32, device="cuda")
    for bad in (dict(lg=lg.t()), dict(lg=lg[:1].expand(2, 64)), dict(tok=tok.long()), dict(lp=lp[:1]),
                dict(rank=torch.empty(2, device="cuda")), dict(top_ids=torch.empty(2, 3, **i)),
                dict(top_ids=torch.empty(2, 3, **i), top_logprobs=torch.empty(2, 4, device="cuda")), dict(ws=ws.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    for n, status in ((33, -1), (40, -1)):
        with pytest.raises(kap.KapError) as e:
            call(top_ids=torch.empty(2, n, **i), top_logprobs=torch.empty(2, n, device="cuda"))
        assert e.value.status == status
    with pytest.raises(kap.KapError) as e:
        call(ws=ws[:4])
    assert e.value.status == -3
