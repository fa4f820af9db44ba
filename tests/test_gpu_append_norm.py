"""The append with norms of queries and keys and several position axes, against 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
PAGE = 16


def reference(x, w, eps, pos, axis, inv):
    """Rows [T][heads][d] in 64 bits: norm (where w is given), then pairs (i, i + d/2) turned."""
    y = x.double()
    half = y.shape[-1] // 2
    if w is not None:
        y = y / torch.sqrt((y * y).mean(dim=-1, keepdim=True) + eps) * w.double()
    live = (axis >= 0) & (axis < pos.shape[0])
    angle = pos.double()[axis.clamp(0, pos.shape[0] - 1).long()].T * inv.double()    # [T][d/2]
    angle = torch.where(live, angle, 0.0)[:, None]
    a, b = y[..., :half], y[..., half:]
    out = torch.cat([a * torch.cos(angle) - b * torch.sin(angle), a * torch.sin(angle) + b * torch.cos(angle)], dim=-1)
    return out, torch.sqrt(a * a + b * b).repeat(1, 1, 2)


def near(got, want, size):
    """A pair's results are off by one rounding into the type, and by less than 2^-20 of its length: the sum of d squares in
    fp32 (2^-19 of it at most, so half of that on its root, for 128 terms 19 additions deep: 19 * 2^-25), rsqrtf 2^-22,
    three products, and a sine and a cosine within 2^-22 of an angle that is right to 2^-23."""
    tol = torch.finfo(got.dtype).eps / 2 * want.abs() + 2.0 ** -20 * size
    assert ((got.double() - want).abs() <= tol).all(), ((got.double() - want).abs() - tol).max()


def make(T, hkv, G, d, dt, axes, seed=0, extra=0, start=100):
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq = hkv * G
    qkv = torch.randn(T, hq + 2 * hkv + extra, d, generator=g, device="cuda").to(dt)
    P = T // PAGE + 3
    return dict(qkv=qkv, q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:hq + 2 * hkv],
                slots=torch.randperm(P * PAGE, generator=g, device="cuda")[:T].contiguous(),
                pos=start + torch.randint(0, 1 + 3 * T, (axes, T), generator=g, device="cuda", dtype=torch.int32),
                inv=torch.tensor([10000.0 ** (-2 * i / d) for i in range(d // 2)], device="cuda"),
                wq=0.5 + torch.rand(d, generator=g, device="cuda"), wk=0.5 + torch.rand(d, generator=g, device="cuda"),
                K=torch.full((P, hkv, PAGE, d), 7.0, dtype=dt, device="cuda"),
                V=torch.full((P, hkv, PAGE, d), 7.0, dtype=dt, device="cuda"), hq=hq)


def check(kap, s, axis=None, wq=None, wk=None, eps=1e-6, in_place=False, q=True, stream=None):
    hkv, d = s["K"].shape[1], s["K"].shape[3]
    T = s["k"].shape[0]
    ax = axis if axis is not None else torch.zeros(d // 2, dtype=torch.int32, device="cuda")
    want_q, size_q = reference(s["q"], wq, eps, s["pos"], ax, s["inv"])
    want_k, size_k = reference(s["k"], wk, eps, s["pos"], ax, s["inv"])
    v = s["v"].clone()
    out = None
    if q:
        out = s["q"] if in_place else torch.full((T, s["hq"], d), 9.0, dtype=s["K"].dtype, device="cuda")
    kap.kap_append_kv_norm(kap.KVPool(s["K"], s["V"], s["hq"]), s["k"], s["v"], s["q"] if q else None, out, s["pos"],
                           s["slots"], s["inv"], q_weight=wq, k_weight=wk, eps=eps, freq_axis=axis, stream=stream)
    torch.cuda.synchronize()
    if q:
        near(out, want_q, size_q)
    live = (s["slots"] >= 0) & (s["slots"] < s["K"].shape[0] * PAGE)
    page, off = s["slots"][live] // PAGE, s["slots"][live] % PAGE
    near(s["K"][page, :, off], want_k[live], size_k[live])
    assert torch.equal(s["V"][page, :, off], v[live])
    rest = torch.ones(s["K"].shape[0] * PAGE, dtype=torch.bool, device="cuda")
    rest[s["slots"][live]] = False
    for t in (s["K"], s["V"]):   # every other slot is as it was
        assert (t.transpose(1, 2).reshape(-1, hkv, d)[rest] == 7.0).all()
    return out


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,hkv,G", [(1, 1, 1), (3, 2, 3), (17, 8, 4), (200, 3, 8), (700, 8, 5), (2500, 1, 1)])
def test_against_64_bits(kap, T, hkv, G, d, dt):
    s = make(T, hkv, G, d, dt, 3, seed=T)
    axis = kap.rope_freq_axis(d, [d // 2 - 2 * (d // 8), d // 8, d // 8], interleaved=True, device="cuda")
    check(kap, s, axis, s["wq"], s["wk"])
    assert kap.kap_device_error() == 0


@pytest.mark.parametrize("wq,wk", [(True, False), (False, True), (False, False)])
def test_one_norm_or_none(kap, wq, wk):
    s = make(33, 2, 4, 128, torch.bfloat16, 1)
    check(kap, s, None, s["wq"] if wq else None, s["wk"] if wk else None, eps=0.3)


def test_positions_far_out_and_below_zero(kap):
    """Angles of positions up to 2^31 - 1 and below 0, at a frequency of a turn and more a position too."""
    s = make(64, 2, 2, 128, torch.float32, 2)
    s["pos"][0] = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 2 ** 24 + 1] * 16, dtype=torch.int32, device="cuda")
    s["pos"][1] = 131072 + torch.arange(64, device="cuda", dtype=torch.int32)
    s["inv"][0], s["inv"][1] = 9.5, 1.0
    # 64-bit angles lose 2^31 * 9.5 * 2^-53 of a radian: 2^-18.7, the reference's own; so the far ones are formed from
    # the remainder by whole turns in extended precision
    inv = s["inv"].cpu().numpy().astype(np.longdouble)
    axis = (torch.arange(64, device="cuda", dtype=torch.int32) % 2).contiguous()
    p = s["pos"].cpu().numpy().astype(np.longdouble)[axis.cpu().numpy()].T     # [T][d/2]
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    ang = np.fmod(p * inv, two_pi).astype(np.float64)
    out = torch.empty(64, 4, 128, device="cuda")
    kap.kap_append_kv_norm(kap.KVPool(s["K"], s["V"], 4), s["k"], s["v"], s["q"], out, s["pos"], s["slots"], s["inv"],
                           freq_axis=axis)
    a, b = s["q"][..., :64].double(), s["q"][..., 64:].double()
    c, sn = (torch.from_numpy(f(ang)).cuda()[:, None] for f in (np.cos, np.sin))
    want = torch.cat([a * c - b * sn, a * sn + b * c], dim=-1)
    size = torch.sqrt(a * a + b * b).repeat(1, 1, 2)
    # a turn's fraction is held to 2^31 * 2^-53 of a turn (2^-19 rad) beside the bound above; where the host's extended
    # type is a 64-bit one (or has 64 bits of mantissa) its own remainder is off by no more
    assert ((out.double() - want).abs() <= (2.0 ** -20 + 2.0 ** -17) * size + 2.0 ** -24 * want.abs()).all()


def test_pairs_of_no_axis_keep_their_values(kap):
    s = make(20, 2, 2, 64, torch.bfloat16, 2)
    axis = torch.tensor([-1, 2, 0, 1] * 8, dtype=torch.int32, device="cuda")
    check(kap, s, axis, s["wq"], s["wk"])
    s = make(20, 2, 2, 64, torch.bfloat16, 2, seed=1)
    out = check(kap, s, torch.full((32,), -1, dtype=torch.int32, device="cuda"))
    assert torch.equal(out, s["q"])


def test_skipped_and_foreign_slots(kap):
    s = make(100, 2, 4, 128, torch.bfloat16, 1)
    s["slots"][::3] = -1
    s["slots"][7] = s["K"].shape[0] * PAGE
    s["slots"][8] = 2 ** 40
    check(kap, s, None, s["wq"], s["wk"])
    assert kap.kap_device_error() == 1
    assert kap.kap_device_error() == 0


def test_in_place_and_without_queries(kap):
    s = make(50, 2, 4, 128, torch.bfloat16, 1)
    rest = s["qkv"][:, 8:].clone()
    check(kap, s, None, s["wq"], s["wk"], in_place=True)
    assert torch.equal(s["qkv"][:, 8:], rest)
    s = make(50, 2, 4, 64, torch.float32, 1)
    check(kap, s, None, s["wq"], s["wk"], q=False)


def test_rows_that_are_zero_or_not_finite(kap):
    s = make(16, 1, 1, 64, torch.float32, 1)
    s["q"][0] = 0.0
    s["q"][1, 0, 5] = float("inf")
    s["q"][2, 0, 5] = float("nan")
    out = torch.empty(16, 1, 64, device="cuda")
    kap.kap_append_kv_norm(kap.KVPool(s["K"], s["V"], 1), s["k"], s["v"], s["q"], out, s["pos"], s["slots"], s["inv"],
                           q_weight=s["wq"], k_weight=s["wk"])
    assert (out[0] == 0).all() and torch.isnan(out[1, 0, 5]) and torch.isnan(out[2]).all() and torch.isfinite(out[3:]).all()


def test_strided_steps_match_the_packed_ones(kap):
    """tok_stride: the slots and positions of one step of a cycle's [R][horizon]."""
    s = make(6, 2, 2, 64, torch.bfloat16, 1)
    pos, slots = torch.zeros(24, dtype=torch.int32, device="cuda"), torch.full((24,), -1, device="cuda")
    pos[2::4], slots[2::4] = s["pos"][0], s["slots"]
    K2, V2 = s["K"].clone(), s["V"].clone()
    out = check(kap, s, None, s["wq"], s["wk"])
    o2 = torch.empty_like(out)
    kap.kap_append_kv_norm(kap.KVPool(K2, V2, 4), s["k"], s["v"], s["q"], o2, pos[2:], slots[2:], s["inv"],
                           q_weight=s["wq"], k_weight=s["wk"], num_tokens=6, tok_stride=4)
    torch.cuda.synchronize()
    assert torch.equal(out, o2) and torch.equal(K2, s["K"]) and torch.equal(V2, s["V"])


def test_without_norms_near_zero_it_is_the_plain_append(kap):
    """At positions whose fp32 angle is exact both appends turn by the same angle; their sines and cosines differ by the
    two functions' errors, 2^-22 of a pair's length, and one rounding."""
    s = make(40, 2, 4, 128, torch.float32, 1)
    s["inv"] = 2.0 ** -torch.arange(64, device="cuda").float()
    out = torch.empty(40, 8, 128, device="cuda")
    kap.kap_append_kv_norm(kap.KVPool(s["K"], s["V"], 8), s["k"], s["v"], s["q"], out, s["pos"], s["slots"], s["inv"])
    K2, V2, q2 = torch.full_like(s["K"], 7.0), torch.full_like(s["V"], 7.0), s["q"].contiguous()
    kap.kap_append_kv(kap.KVPool(K2, V2, 8), s["k"].contiguous(), s["v"].contiguous(), q2, s["pos"][0].contiguous(),
                      s["slots"], s["inv"])
    size = torch.sqrt(s["q"][..., :64] ** 2 + s["q"][..., 64:] ** 2).repeat(1, 1, 2)
    assert ((out - q2).abs() <= 2.0 ** -20 * size).all() and torch.equal(s["V"], V2)


def test_captured_and_on_another_stream(kap):
    s = make(90, 2, 4, 128, torch.bfloat16, 1)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    want = check(kap, s, None, s["wq"], s["wk"], stream=st)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kap.kap_append_kv_norm(kap.KVPool(s["K"], s["V"], 8), s["k"], s["v"], s["q"], out, s["pos"], s["slots"], s["inv"],
                               q_weight=s["wq"], k_weight=s["wk"])
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_refusals(kap):
    s = make(10, 2, 2, 64, torch.bfloat16, 1, extra=1)
    pool = kap.KVPool(s["K"], s["V"], 4)
    out = torch.empty(10, 4, 64, dtype=torch.bfloat16, device="cuda")
    call = lambda **kw: kap.kap_append_kv_norm(**{**dict(pool=pool, k_new=s["k"], v_new=s["v"], q=s["q"], q_out=out,  # noqa: E731
                                                         pos=s["pos"], slots=s["slots"], inv_freq=s["inv"]), **kw})
    call()
    for bad in (dict(k_new=s["k"].float()), dict(slots=s["slots"].int()), dict(pos=s["pos"].long()),
                dict(q_weight=s["wq"].half()), dict(freq_axis=torch.zeros(32, dtype=torch.int64, device="cuda"))):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(k_new=s["k"][:, :1]), dict(q=None), dict(pos=s["pos"][:, :9]), dict(slots=s["slots"][:9]),
                dict(inv_freq=s["inv"][:31]), dict(q=s["q"].transpose(0, 1)), dict(v_new=s["v"].cpu()),
                dict(q_weight=s["wq"][:63]), dict(q=s["q"].transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**bad)
    flat = torch.zeros(10 * 260, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(pos=torch.zeros(9, 10, dtype=torch.int32, device="cuda")),
                dict(q=flat.as_strided((10, 4, 64), (260, 64, 1))),        # tokens 520 bytes apart
                dict(q=torch.zeros(10 * 256 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(10, 4, 64))):
        with pytest.raises(kap.KapError):
            call(**bad)
    call(k_new=s["k"][:0], v_new=s["v"][:0], q=s["q"][:0], q_out=out[:0])   # no tokens: nothing to do
    assert kap.kap_device_error() == 0
