"""Attention of requests that share prefixes, against 64 bits and against kap_attn_verify."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
PAGE = 16


def make(members, prefix, suffix, windows, hkv=2, G=4, d=128, dt=torch.bfloat16, seed=0, spare=4):
    """members[g] requests in group g over prefix[g] pages; suffix[r] tokens of its own before request r's window of
    windows[r]. The pool has NaN pages that nothing names, and NaN past each request's end."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    R = sum(members)
    first = [sum(members[:i]) for i in range(len(members) + 1)]
    of = [k for k, n in enumerate(members) for _ in range(n)]
    starts = [prefix[of[r]] * PAGE + suffix[r] for r in range(R)]
    ends = [s + w for s, w in zip(starts, windows)]
    pages = [(e + PAGE - 1) // PAGE for e in ends]
    P = sum(prefix) + sum(pages[r] - prefix[of[r]] for r in range(R)) + spare
    ids = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    K = torch.full((P, hkv, PAGE, d), float("nan"), dtype=dt, device="cuda")
    V = K.clone()
    bt = torch.full((R, max(pages) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for k in range(len(members)):
        head = ids[at:at + prefix[k]]
        at += prefix[k]
        for r in range(first[k], first[k + 1]):
            bt[r, :prefix[k]] = head
            bt[r, prefix[k]:pages[r]] = ids[at:at + pages[r] - prefix[k]]
            at += pages[r] - prefix[k]
    for r in range(R):
        n = ends[r]
        page = bt[r, :pages[r]].long()
        k = torch.randn(pages[r] * PAGE, hkv, d, generator=g, device="cuda").to(dt)
        v = (0.5 * torch.randn(pages[r] * PAGE, hkv, d, generator=g, device="cuda")).to(dt)
        k[n:], v[n:] = float("nan"), float("nan")
        lo = 0 if r in first else prefix[of[r]]     # the prefix is written once
        K[page[lo:]] = k.view(-1, PAGE, hkv, d).transpose(1, 2)[lo:]
        V[page[lo:]] = v.view(-1, PAGE, hkv, d).transpose(1, 2)[lo:]
    i32 = dict(dtype=torch.int32, device="cuda")
    qo = torch.zeros(R + 1, **i32)
    qo[1:] = torch.tensor(windows, **i32).cumsum(0)
    tq = sum(windows)
    return dict(K=K, V=V, bt=bt, starts=starts, windows=windows, qo=qo, start=torch.tensor(starts, **i32),
                go=torch.tensor(first, **i32), pp=torch.tensor(prefix, **i32), G=G, hq=hkv * G, R=R, tq=tq,
                q=(1.5 * torch.randn(tq, hkv * G, d, generator=g, device="cuda")).to(dt))


def run(kap, s, ws=None, stream=None, groups=True):
    hkv, d = s["K"].shape[1], s["K"].shape[3]
    out = torch.full(s["q"].shape, 7.0, dtype=s["q"].dtype, device="cuda")
    lse = torch.full((s["tq"], s["hq"]), 7.0, device="cuda")
    go, pp = (s["go"], s["pp"]) if groups else (s["go"][:1], s["pp"][:0])
    if ws is None:   # whatever the workspace holds
        ws = torch.full((kap.kap_shared_workspace_size(s["R"], hkv, s["hq"], d, s["tq"], pp.numel()),), 255,
                        dtype=torch.uint8, device="cuda")
    kap.kap_attn_verify_shared(kap.KVPool(s["K"], s["V"], s["hq"]), kap.PageMap(s["bt"], s["start"]),
                               kap.VerifyPolicy(s["qo"], s["start"], max(s["windows"]), s["tq"]),
                               kap.PrefixGroups(go, pp), s["q"], out, lse, ws, stream=stream)
    return out, lse


def check(s, out, lse, hide=None):
    """Each row against 64 bits. A score is a sum of d products in fp32: off by d 2^-24 of sum |q k| / sqrt(d) at most, call
    it e; a weight is then off by 2 e (and 2^-21 for its exponential) relative, and over a bf16 pool by a rounding of 2^-8;
    sums of n terms in fp32 by n 2^-24, joined records included; the output has one rounding of its own."""
    dt, d, G = s["q"].dtype, s["q"].shape[2], s["G"]
    t = 0
    for r in range(s["R"]):
        for i in range(s["windows"][r]):
            n = s["starts"][r] + i + 1
            see = torch.arange(n, device="cuda")
            if hide is not None:
                see = see[~hide(r, see)]
            page = s["bt"][r].long()[see // PAGE]
            if len(see) == 0:
                assert (out[t] == 0).all() and torch.isneginf(lse[t]).all()
                t += 1
                continue
            k, v = s["K"][page, :, see % PAGE].double(), s["V"][page, :, see % PAGE].double()    # [n][hkv][d]
            q = s["q"][t].double().view(-1, G, d)
            x = torch.einsum("hgd,nhd->hgn", q, k) / math.sqrt(d)
            e = d * 2.0 ** -24 * torch.einsum("hgd,nhd->hgn", q.abs(), k.abs()).amax(-1) / math.sqrt(d)
            l = torch.logsumexp(x, -1)
            p = torch.exp(x - l[..., None])
            o = torch.einsum("hgn,nhd->hgd", p, v)
            mass = torch.einsum("hgn,nhd->hgd", p, v.abs())
            rel = 4 * e + 2.0 ** -20 + n * 2.0 ** -24 + (2.0 ** -8 if dt is torch.bfloat16 else 0.0)
            tol = rel[..., None] * (mass + o.abs()) + torch.finfo(dt).eps / 2 * o.abs()
            err = (out[t].double().view_as(o) - o).abs()
            assert (err <= tol).all(), (r, i, (err - tol).max())
            lerr = (lse[t].double().view_as(l) - l).abs()
            assert (lerr <= 2 * e + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -22 * l.abs()).all(), (r, i, lerr.max())
            t += 1


SHAPES = [
    ([1], [0], [0], [1]),                                        # one token of one request sees itself
    ([2], [1], [0, 0], [1, 1]),                                  # the window starts at the prefix's end
    ([2], [3], [5, 40], [1, 2]),
    ([3], [9], [0, 129, 300], [4, 1, 3]),                        # tiles that end inside
    ([1, 1, 1], [4, 8, 0], [3, 0, 7], [1, 2, 1]),                # groups of one
    ([4, 1, 6], [20, 3, 0], [7, 130, 0, 128, 10, 1, 2, 3, 250, 5, 6], [2, 1, 3, 1, 2, 1, 1, 4, 1, 2, 1]),
    ([40], [17], [13 * (i % 5) for i in range(40)], [1 + i % 3 for i in range(40)]),     # several blocks of rows
    ([9, 25], [70, 33], [11 * (i % 4) for i in range(34)], [2] * 34),
]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_against_64_bits(kap, shape, d, dt):
    s = make(*SHAPES[shape], d=d, dt=dt, seed=shape)
    out, lse = run(kap, s)
    torch.cuda.synchronize()
    check(s, out, lse)
    assert kap.kap_device_error() == 0


@pytest.mark.parametrize("hkv,G", [(1, 1), (1, 8), (3, 2), (8, 3), (4, 5), (2, 7)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_head_layouts(kap, hkv, G, dt):
    s = make([5, 3], [12, 4], [0, 9, 100, 17, 33, 2, 150, 64], [1, 3, 2, 1, 1, 2, 3, 1], hkv=hkv, G=G, dt=dt)
    out, lse = run(kap, s)
    torch.cuda.synchronize()
    check(s, out, lse)
    assert kap.kap_device_error() == 0


def test_widest_windows(kap):
    """64 query columns: windows of 64 rows of one head and of 8 rows of 8."""
    for G, n in ((1, 64), (8, 8)):
        s = make([3], [10], [5, 0, 77], [n, n - 1, n], G=G)
        out, lse = run(kap, s)
        torch.cuda.synchronize()
        check(s, out, lse)


@pytest.mark.parametrize("d,dt", [(128, torch.bfloat16), (64, torch.bfloat16), (128, torch.float32)])
def test_requests_without_rows(kap, d, dt):
    """Windows of no rows: first, last, between others, a group's first request, and all of a group's."""
    s = make([3, 2, 2, 1, 2], [12, 9, 3, 0, 5], [7, 0, 30, 129, 4, 0, 5, 60, 1, 2], [0, 1, 2, 0, 0, 3, 0, 1, 1, 0], d=d, dt=dt)
    out, lse = run(kap, s)
    torch.cuda.synchronize()
    check(s, out, lse)
    assert kap.kap_device_error() == 0


def test_two_streams_at_once(kap):
    """Calls with a workspace each, in flight together on two streams."""
    a, b = make([9], [200], [60] * 9, [2] * 9), make([3, 5], [40, 300], [30] * 8, [1] * 8, d=64, seed=1)
    ws = [kap.workspace(kap.kap_shared_workspace_size(s["R"], 2, s["hq"], s["K"].shape[3], s["tq"], s["pp"].numel()), "cuda")
          for s in (a, b)]
    want = [run(kap, s) for s in (a, b)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(24):
        with torch.cuda.stream(streams[i % 2]):
            got.append(run(kap, (a, b)[i % 2], ws=ws[i % 2], stream=streams[i % 2]))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    assert kap.kap_device_error() == 0


def test_long_prefix_split_over_all_ctas(kap):
    s = make([6], [2048], [3, 200, 0, 31, 640, 16], [1] * 6, hkv=1, G=8)
    out, lse = run(kap, s)
    torch.cuda.synchronize()
    check(s, out, lse)


def test_same_results_as_without_sharing(kap):
    """The groups only say how the work is shared out: results agree up to rounding with those without groups and with
    kap_attn_verify's. Both sides are off by no more than check() allows; here twice a bf16 rounding of values of size
    about 1 (the sums' errors are far below)."""
    s = make([7, 5], [40, 9], [3 * i for i in range(12)], [1 + i % 4 for i in range(12)])
    a, la = run(kap, s)
    b, lb = run(kap, s, groups=False)
    torch.cuda.synchronize()
    check(s, b, lb)
    pool = kap.KVPool(torch.nan_to_num(s["K"]), torch.nan_to_num(s["V"]), s["hq"])
    ws = kap.workspace(kap.kap_verify_workspace_size(s["R"], 2, 8, 128, 4), "cuda")
    o, l = torch.empty_like(a), torch.empty_like(la)
    kap.kap_attn_verify(pool, kap.PageMap(s["bt"], s["start"], s["start"]), kap.VerifyPolicy(s["qo"], s["start"], 4, s["tq"]),
                        s["q"], o, l, ws)
    torch.cuda.synchronize()
    for x, lx in ((b, lb), (o, l)):
        assert (a.float() - x.float()).abs().max() <= 4 * 2.0 ** -8 and (la - lx).abs().max() <= 1e-4
    assert kap.kap_device_error() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(kap, dt):
    s = make([3], [9], [20, 7, 0], [4, 3, 2], dt=dt)
    page, off = s["bt"][0].long(), s["starts"][0] + 2      # the third window token of request 0
    s["V"][page[off // PAGE], :, off % PAGE] = float("inf")
    off1 = s["starts"][1] - 3                              # a token of request 1's own context
    s["V"][s["bt"][1].long()[off1 // PAGE], 0, off1 % PAGE, 5] = float("nan")
    out, lse = run(kap, s)
    torch.cuda.synchronize()
    fin = torch.isfinite(out).all(dim=-1)                  # [tq][hq]
    assert fin[:2].all() and not fin[2:4].any() and torch.isfinite(lse).all()
    assert not fin[4:7, :4].any() and fin[4:7, 4:].all() and fin[7:].all()
    bad = torch.isnan(out[4:7, :4])
    assert bad[..., 5].all() and not bad[..., :5].any() and not bad[..., 6:].any()
    s["V"][page[off // PAGE], :, off % PAGE] = 0.0
    s["V"][s["bt"][1].long()[off1 // PAGE], 0, off1 % PAGE, 5] = 0.0
    out, lse = run(kap, s)
    torch.cuda.synchronize()
    check(s, out, lse)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_pages_outside_the_pool_are_skipped(kap, dt):
    s = make([4, 2], [20, 5], [30, 5, 260, 0, 40, 8], [2, 1, 1, 1, 2, 1], dt=dt)
    bad = {(0, 3): -1, (2, 25): s["K"].shape[0], (2, 27): 2 ** 31 - 1, (4, 6): -5}
    for r in range(4):
        s["bt"][r, 3] = -1                                 # a shared page
    for (r, j), v in bad.items():
        s["bt"][r, j] = v
    out, lse = run(kap, s)
    torch.cuda.synchronize()
    hidden = lambda r, t: torch.tensor([(x // PAGE == 3 and r < 4) or (r, x // PAGE) in bad for x in t.tolist()],  # noqa: E731
                                       dtype=torch.bool, device="cuda")
    check(s, out, lse, hide=hidden)
    assert kap.kap_device_error() == 1
    # a row that sees nothing at all
    s = make([2], [2], [0, 16], [1, 1], dt=dt)
    s["bt"][:] = -1
    out, lse = run(kap, s)
    torch.cuda.synchronize()
    check(s, out, lse, hide=lambda r, t: torch.ones(len(t), dtype=torch.bool, device="cuda"))
    assert kap.kap_device_error() == 1


def test_contexts_past_the_table(kap):
    """A length that runs past the table's columns: what the table names is attended to, the rest reported."""
    s = make([2], [4], [10, 20], [1, 1])
    s["bt"] = s["bt"][:, :5].contiguous()
    s["start"] = torch.tensor([4 * PAGE + 10, 2 ** 31 - 100], dtype=torch.int32, device="cuda")
    s["bt"][1, 4] = s["bt"][0, 4]
    kv = s["bt"][0, 4].long()
    s["K"][kv], s["V"][kv] = torch.nan_to_num(s["K"][kv]), torch.nan_to_num(s["V"][kv])
    out, lse = run(kap, s)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    assert kap.kap_device_error() == 1


def test_a_window_inside_the_shared_pages(kap):
    """A request whose window starts before its group's shared pages end sees no more than its own positions."""
    s = make([3], [10], [0, 30, 5], [1, 2, 2])
    s["starts"][1] = 70
    s["start"][1] = 70
    out, lse = run(kap, s)
    torch.cuda.synchronize()
    check(s, out, lse)
    assert kap.kap_device_error() == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_outside_the_windows_are_left_as_they_are(kap, d, dt):
    """A batch padded to a fixed number of rows, ahead of the first window and behind the last one."""
    s = make([3, 2], [20, 9], [7, 130, 0, 40, 300], [2, 1, 3, 1, 2], d=d, dt=dt)
    want, wlse = run(kap, s)
    before, behind = 2, 60
    q = torch.cat([torch.randn(before, *s["q"].shape[1:], device="cuda").to(dt), s["q"],
                   torch.randn(behind, *s["q"].shape[1:], device="cuda").to(dt)])
    out, lse = torch.full_like(q, 5.0), torch.full(q.shape[:2], 6.0, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    qo = torch.tensor([0, 2, 3, 6, 7, 9], **i32) + before
    start = torch.tensor(s["starts"], **i32)
    hkv = s["K"].shape[1]
    ws = kap.workspace(kap.kap_shared_workspace_size(5, hkv, q.shape[1], d, q.shape[0], 2), "cuda")
    kap.kap_attn_verify_shared(kap.KVPool(s["K"], s["V"], q.shape[1]), kap.PageMap(s["bt"], start),
                               kap.VerifyPolicy(qo, start, 3, q.shape[0]), kap.PrefixGroups(s["go"], s["pp"]), q, out, lse, ws)
    torch.cuda.synchronize()
    assert torch.equal(out[before:before + 9], want) and torch.equal(lse[before:before + 9], wlse)
    for a, b in ((0, before), (before + 9, before + 9 + behind)):
        assert (out[a:b] == 5.0).all() and (lse[a:b] == 6.0).all()
    assert kap.kap_device_error() == 0


def test_offsets_that_do_not_cover_the_requests(kap):
    for off in ([0, 3, 5], [1, 3, 6], [0, 4, 2], [0, 9, 6], [-4, 3, 6]):
        s = make([3, 3], [4, 5], [1] * 6, [1] * 6)
        s["go"] = torch.tensor(off, dtype=torch.int32, device="cuda")
        run(kap, s)
        assert kap.kap_device_error() & 4, off


def test_more_groups_and_requests_than_threads(kap):
    n = 700
    s = make([1 + g % 3 for g in range(n)], [1 + g % 2 for g in range(n)], [5 * (i % 3) for i in range(sum(1 + g % 3 for g in range(n)))],
             [1] * sum(1 + g % 3 for g in range(n)), hkv=1, G=2, d=64)
    out, lse = run(kap, s)
    torch.cuda.synchronize()
    check(s, out, lse)
    n = 1100
    s = make([2] * n, [1] * n, [0] * (2 * n), [1] * (2 * n), hkv=1, G=1, d=64)
    out, lse = run(kap, s)
    torch.cuda.synchronize()
    check(s, out, lse)
    assert kap.kap_device_error() == 0


def test_one_workspace_for_calls_in_turn_and_captured(kap):
    a = make([5], [30], [9] * 5, [2] * 5)
    b = make([2, 3], [7, 60], [0, 5, 90, 1, 2], [1, 1, 2, 3, 1], hkv=1, G=6, d=64)
    ws = kap.workspace(max(kap.kap_shared_workspace_size(s["R"], s["K"].shape[1], s["hq"], s["K"].shape[3], s["tq"],
                                                         s["pp"].numel()) for s in (a, b)), "cuda")
    first = [run(kap, s, ws) for s in (a, b, a, b)]
    torch.cuda.synchronize()
    for x, y in zip(first[:2], first[2:]):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    check(a, *first[0])
    check(b, *first[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = run(kap, a, ws)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0][0]) and torch.equal(lse, first[0][1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        out, lse = run(kap, b, ws, stream=st)
    st.synchronize()
    assert torch.equal(out, first[1][0])


def test_refusals(kap):
    s = make([2], [2], [1, 1], [1, 1])
    run(kap, s)
    with pytest.raises(kap.KapError):
        run(kap, s, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    for name, bad in (("q", s["q"].float()), ("bt", s["bt"].long()), ("pp", s["pp"].long())):
        with pytest.raises(TypeError):
            run(kap, {**s, name: bad})
    for name, bad in (("go", s["go"][:1]), ("q", s["q"][:, :4]), ("start", s["start"][:1]), ("qo", s["qo"].cpu())):
        with pytest.raises(ValueError):
            run(kap, {**s, name: bad})
    with pytest.raises(kap.KapError):
        run(kap, {**s, "windows": [65, 1]})      # more than 64 query columns
    torch.cuda.synchronize()
    assert kap.kap_device_error() == 0
