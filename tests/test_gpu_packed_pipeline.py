"""The pipeline over a packed cache in its other forms: a view shared by the KV heads, span selections, the side flow."""
import pytest
import torch

from tests.packed_reference import PAGE
from tests.test_gpu_packed_flow import Server, _close

pytestmark = pytest.mark.gpu


def _randn(s, *n):
    return torch.randn(*n, generator=s.g, device="cuda").to(torch.bfloat16)


def _ready(kap, lens, hkv, G, d, seed, room):
    """A server whose full prompt pages are packed and whose tables have `room` more tokens a request."""
    s = Server(kap, lens, hkv, G, d, seed=seed)
    committed = s.len.clone()
    R = len(lens)
    s.grow(torch.full((R,), room, dtype=torch.int32, device="cuda"), R * room)
    s.pack_full_prompt_pages()
    return s, committed


@pytest.mark.parametrize("form", ["shared", "spans"])
def test_cycle_with_one_view_for_all_heads(kap, form):
    lens, hkv, G, d, steps = [90, 260], 2, 3, 64, 2
    R, Hq = len(lens), hkv * G
    s, committed = _ready(kap, lens, hkv, G, d, 21, steps)
    n_q = torch.full((R,), steps, dtype=torch.int32, device="cuda")
    pol = kap.AccessPolicy(1, 1, 3, False, 12)
    kw = {}
    if form == "spans":   # (first token, length): one of request 0, two of request 1
        kw = dict(spans=torch.tensor([[20, 20], [100, 30], [180, 5]], dtype=torch.int32, device="cuda"),
                  span_offsets=torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda"))
    cyc = kap.DecodeCycle(s.pool, s.bt, s.ctx, committed, steps, n_q, s.inv, policy=pol, packed=s.packed, **kw)
    qp, kp, vp = _randn(s, steps, R, Hq, d), _randn(s, steps, R, hkv, d), _randn(s, steps, R, hkv, d)
    cyc.plan(_randn(s, R, Hq, d))
    for i in range(steps):
        cyc.propose_step(i, qp[i], kp[i], vp[i])   # rotates qp[i] in place
    torch.cuda.synchronize()
    assert kap.kap_device_error() == 0
    sel, ns = cyc.sel_ids.cpu().numpy(), cyc.n_sel.cpu().numpy()
    assert sel.shape[1] == 1 and (ns > 0).all()
    if form == "spans":
        assert {1, 2} <= set(sel[0, 0, :ns[0, 0]].tolist()) and {6, 7, 8, 11} <= set(sel[1, 0, :ns[1, 0]].tolist())
    i = steps - 1
    for r in range(R):
        pages = set(sel[r, 0, :ns[r, 0]].tolist())
        for head in range(Hq):
            toks = [s.token(r, head // G, t) for t in range(lens[r] + i + 1) if t >= lens[r] or t // PAGE in pages]
            _close(cyc.o_prop[i, r, head], cyc.lse_prop[i, r, head], qp[i, r, head], toks, d)


@pytest.mark.parametrize("graph", [False, True])
def test_side_flow_equals_the_layers_in_turn(kap, graph):
    lens, hkv, G, d, layers = [300, 120], 2, 4, 128, 3
    R, Hq = len(lens), hkv * G
    pol = kap.AccessPolicy(1, 1, 4, True, 6)

    def build():
        cycles, args = [], []
        for l in range(layers):
            s, committed = _ready(kap, lens, hkv, G, d, 30 + l, 1)
            one = torch.ones(R, dtype=torch.int32, device="cuda")
            cycles.append(kap.DecodeCycle(s.pool, s.bt, s.ctx, committed, 1, one, s.inv, policy=pol, packed=s.packed))
            args.append((_randn(s, R, Hq, d), _randn(s, R, Hq, d), _randn(s, R, hkv, d), _randn(s, R, hkv, d)))
        return kap.SideFlowDecode(cycles), [list(a) for a in zip(*args)]

    ref, args = build()
    ref.step(*args, overlap=False)
    flow, args = build()
    raw = [q.clone() for q in args[1]]
    flow.step(*args)
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            flow.step(*args)
        for _ in range(2):
            for q, x in zip(args[1], raw):   # a step rotates its queries in place
                q.copy_(x)
            for c in flow.cycles:
                c.o_prop.zero_()
            g.replay()
            torch.cuda.synchronize()
    assert kap.kap_device_error() == 0
    for a, b in zip(flow.cycles, ref.cycles):
        assert torch.equal(a.sel_ids, b.sel_ids) and torch.equal(a.view.block_table, b.view.block_table)
        assert torch.equal(a.o_prop, b.o_prop) and torch.equal(a.lse_prop, b.lse_prop)
        assert torch.isfinite(a.o_prop.float()).all()
