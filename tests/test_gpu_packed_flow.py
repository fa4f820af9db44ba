"""The packed cache as a server uses it: tables from lengths, prompt appended, routed, packed, decoded, verified and
scored, each step's result against 64 bits or against the call it stands beside."""
import numpy as np
import pytest
import torch

from tests.packed_reference import PAGE, attend, chunk_values, tolerances

pytestmark = pytest.mark.gpu


class Server:
    """Requests of the given prompt lengths on pages that the table calls hand out; prompts appended and summarised."""

    def __init__(self, kap, lens, hkv, G, d, seed, spare=40):
        self.kap, self.hkv, self.G, self.d, self.lens = kap, hkv, G, d, lens
        dev = "cuda"
        i32 = dict(dtype=torch.int32, device=dev)
        R = len(lens)
        g = torch.Generator(device=dev).manual_seed(seed)
        need = sum(-(-n // PAGE) for n in lens)
        self.P16, self.P4 = need + spare, need
        self.mp = max(-(-n // PAGE) for n in lens) + 3
        K = torch.full((self.P16, hkv, PAGE, d), float("nan"), dtype=torch.bfloat16, device=dev)
        self.ks = torch.zeros(self.P16 + self.P4, hkv, d, device=dev)
        self.pool = kap.KVPool(K, K.clone(), hkv * G, self.ks[:self.P16])
        self.packed = kap.PackedPool(self.pool, torch.zeros(self.P4, hkv, kap.kap_packed_chunk_bytes(d), dtype=torch.uint8,
                                                            device=dev), self.ks)
        self.bt = torch.full((R, self.mp), -1, **i32)
        self.stack = torch.randperm(self.P16, generator=g, device=dev).to(torch.int32)
        self.count = torch.tensor([self.P16], **i32)
        self.len = torch.zeros(R, **i32)
        self.inv = kap.rope_inv_freq(d, 1.0e4, dev)
        slots, pos = self.grow(torch.tensor(lens, **i32), sum(lens))
        T = sum(lens)
        self.k_new = torch.randn(T, hkv, d, generator=g, device=dev).to(torch.bfloat16)
        self.v_new = torch.randn(T, hkv, d, generator=g, device=dev).to(torch.bfloat16)
        kap.kap_append_kv(self.pool, self.k_new, self.v_new, None, pos, slots, self.inv)
        self.ctx = torch.tensor(lens, **i32)
        kap.kap_build_summaries(self.pool, kap.PageMap(self.bt, self.ctx, self.len))
        self.g = g

    def grow(self, new, T):
        kap, dev = self.kap, "cuda"
        i32 = dict(dtype=torch.int32, device=dev)
        R = self.bt.shape[0]
        count, length, ok = torch.zeros(1, **i32), torch.zeros(R, **i32), torch.zeros(R, **i32)
        off, slots = torch.zeros(R + 1, **i32), torch.zeros(T, dtype=torch.int64, device=dev)
        pos = torch.zeros(T, **i32)
        kap.kap_extend_tables(self.bt, self.len, new, self.stack, self.count, count, off, slots, pos, length, ok)
        self.count, self.len = count, length
        assert ok.all()
        return slots, pos

    def pack_full_prompt_pages(self):
        """Packs every full prompt page and gives its 16-bit page back to the stack."""
        full = torch.arange(self.mp, device="cuda")[None] < (self.ctx // PAGE)[:, None]
        src = self.bt[full].contiguous()
        dst = torch.arange(len(src), dtype=torch.int32, device="cuda") + self.packed.first_packed
        self.kap.kap_pack_pages(self.packed, src, dst)
        self.bt[full] = dst
        n = int(self.count)
        self.stack[n:n + len(src)] = src
        self.count = self.count + len(src)
        # the given-back pages hold nothing any more
        self.pool.k_pages[src.long()] = float("nan")
        self.pool.v_pages[src.long()] = float("nan")

    def token(self, r, h, t):
        pid = int(self.bt[r, t // PAGE])
        o = t % PAGE
        if pid < self.P16:
            k = self.pool.k_pages[pid, h, o].double().cpu().numpy()
            v = self.pool.v_pages[pid, h, o].double().cpu().numpy()
            return k, v, np.zeros(self.d), np.abs(k), np.abs(v)
        val, sc, lo = self.values(pid, h)
        return val[0, o], val[1, o], sc[1, o], sc[0, o] + lo[0, o], sc[1, o] + lo[1, o]

    def values(self, pid, h, cache={}):
        key = (id(self), pid, h)
        if key not in cache:
            cache[key] = chunk_values(self.packed.packed[pid - self.P16, h].cpu().numpy(), self.d)
        return cache[key]


def _close(o, lse, q, tokens, d):
    w, l, pv, pvc, s = attend(q.double().cpu().numpy(), tokens, d)
    to, tl = tolerances(d, len(tokens), l, pv, pvc, s)
    got = o.double().cpu().numpy()
    assert (np.abs(got - w) <= to + 2.0 ** -8 * np.abs(w)).all()
    assert abs(float(lse) - l) <= tl


@pytest.mark.parametrize("lens,hkv,G,d", [([70, 33, 256], 2, 4, 128), ([500, 16], 1, 5, 64)])
def test_cycle_over_a_packed_prompt(kap, lens, hkv, G, d):
    s = Server(kap, lens, hkv, G, d, seed=len(lens))
    R, Hq, dev = len(lens), hkv * G, "cuda"
    k_prop, nq = 2, 3
    pol = kap.AccessPolicy(1, 1, 3, True, 5)
    q = lambda *n: torch.randn(*n, generator=s.g, device=dev).to(torch.bfloat16)  # noqa: E731
    q_route = q(R, Hq, d)
    # the tables get the pages that the window will write; the committed length stays
    committed = s.len.clone()
    s.grow(torch.full((R,), nq, dtype=torch.int32, device=dev), R * nq)
    n_q = torch.full((R,), nq, dtype=torch.int32, device=dev)
    plain = kap.DecodeCycle(s.pool, s.bt.clone(), s.ctx, committed, k_prop, n_q, s.inv, policy=pol)
    plain.plan(q_route)
    s.pack_full_prompt_pages()
    cyc = kap.DecodeCycle(s.pool, s.bt, s.ctx, committed, k_prop, n_q, s.inv, policy=pol, packed=s.packed)
    qp, kp, vp = q(k_prop, R, Hq, d), q(k_prop, R, hkv, d), q(k_prop, R, hkv, d)
    qv, kv, vv = q(R * nq, Hq, d), q(R * nq, hkv, d), q(R * nq, hkv, d)
    cyc.plan(q_route)
    # the summaries moved with the pages: routing chooses as it did over the 16-bit pages
    assert torch.equal(cyc.sel_ids, plain.sel_ids) and torch.equal(cyc.n_sel, plain.n_sel)
    for i in range(k_prop):
        cyc.propose_step(i, qp[i], kp[i], vp[i])
        torch.cuda.synchronize()
        sel, ns = cyc.sel_ids.cpu().numpy(), cyc.n_sel.cpu().numpy()
        for r in range(R):
            for head in (0, Hq - 1):
                h = head // G
                pages = set(sel[r, h, :ns[r, h]].tolist())
                toks = [s.token(r, h, t) for t in range(lens[r] + i + 1) if t >= lens[r] or t // PAGE in pages]
                _close(cyc.o_prop[i, r, head], cyc.lse_prop[i, r, head], qp[i, r, head], toks, d)
    cyc.verify(qv, kv, vv)
    torch.cuda.synchronize()
    assert kap.kap_device_error() == 0
    for r in range(R):
        for head in (0, Hq // 2):
            for i in range(nq):
                toks = [s.token(r, head // G, t) for t in range(lens[r] + i + 1)]
                _close(cyc.o_ver[r * nq + i, head], cyc.lse_ver[r * nq + i, head], qv[r * nq + i, head], toks, d)
    # the verifier's logits: ranks and acceptance agree, log probabilities against 64 bits
    V = 3001
    logits = cyc.o_ver.float().flatten(1) @ torch.randn(Hq * d, V, generator=s.g, device=dev) * 0.05
    tok = logits.topk(4, dim=-1).indices[torch.arange(R * nq), torch.arange(R * nq) % 4].to(torch.int32)
    window = torch.roll(tok, 1)    # window token j + 1 is judged by row j
    f = dict(dtype=torch.float32, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    lp, rank = torch.empty(R * nq, **f), torch.empty(R * nq, **i32)
    kap.kap_token_logprobs(logits, tok, lp, kap.workspace(kap.kap_logprobs_workspace_size(R * nq, V), dev), rank=rank)
    acc, car = torch.zeros(R, **i32), torch.zeros(R, **i32)
    kap.kap_accept_commit(logits, cyc.q_offsets, window.contiguous(), 3, acc, car,
                          kap.workspace(kap.kap_accept_workspace_size(R, R * nq, V), dev))
    ranks = rank.cpu().view(R, nq)
    for r in range(R):
        m = 0
        while m < nq - 1 and int(ranks[r, m]) < 3:
            m += 1
        assert m == int(acc[r])
    ref = torch.log_softmax(logits.double(), dim=-1).gather(1, tok.long()[:, None])[:, 0]
    assert ((lp.double() - ref).abs() <= (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * ref.abs()).all()


def test_loop_over_a_packed_prompt_in_a_graph(kap):
    """DecodeLoop over a packed prompt: eager steps, and the same steps captured and replayed."""
    lens, hkv, G, d, steps = [90, 300], 2, 4, 128, 4
    s = Server(kap, lens, hkv, G, d, seed=3)
    R, Hq, dev = 2, 8, "cuda"
    committed = s.len.clone()
    s.grow(torch.full((R,), steps, dtype=torch.int32, device=dev), R * steps)
    s.pack_full_prompt_pages()
    q = lambda *n: torch.randn(*n, generator=s.g, device=dev).to(torch.bfloat16)  # noqa: E731
    qr, qp, kn, vn = q(steps, R, Hq, d), q(steps, R, Hq, d), q(steps, R, hkv, d), q(steps, R, hkv, d)
    pol = kap.AccessPolicy(1, 1, 4, True, 6)

    def run(loop, qq):
        for t in range(steps):
            loop.plan(qr[t])
            loop.propose_step(0, qq[t], kn[t], vn[t])
            loop.advance()

    loop = kap.DecodeLoop(s.pool, s.bt, s.ctx, committed, steps, s.inv, pol, packed=s.packed)
    mine = qp.clone()
    run(loop, mine)
    torch.cuda.synchronize()
    assert kap.kap_device_error() == 0
    t = steps - 1
    sel, ns = loop.sel_ids.cpu().numpy(), loop.n_sel.cpu().numpy()
    for r in range(R):
        for head in (0, 5):
            h = head // G
            pages = set(sel[r, h, :ns[r, h]].tolist())
            toks = [s.token(r, h, x) for x in range(lens[r] + t + 1) if x >= lens[r] or x // PAGE in pages]
            _close(loop.o[t, r, head], loop.lse[t, r, head], mine[t, r, head], toks, d)
    other = kap.DecodeLoop(s.pool, s.bt, s.ctx, committed, steps, s.inv, pol, packed=s.packed)
    buf = qp.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(other, buf)
    for _ in range(2):
        buf.copy_(qp)
        other.o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(other.o, loop.o) and torch.equal(other.lse, loop.lse)


def test_pipeline_refusals(kap):
    s = Server(kap, [40], 1, 2, 64, seed=1)
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    pol = kap.AccessPolicy(1, 1, 1, True, 3)
    other = kap.KVPool(s.pool.k_pages, s.pool.v_pages, 2, s.pool.k_summary)
    for kw in (dict(pool=other), dict(pool=s.pool, workspace_pages=(10, 2))):
        pool = kw.pop("pool")
        with pytest.raises(ValueError):
            kap.DecodeCycle(pool, s.bt, s.ctx, s.len, 1, one, s.inv, policy=pol, packed=s.packed, **kw)
    with pytest.raises(ValueError):
        kap.DecodeLoop(other, s.bt, s.ctx, s.len, 2, s.inv, pol, packed=s.packed)
