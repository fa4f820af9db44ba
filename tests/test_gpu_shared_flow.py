"""The append with norms and position axes, attention over shared prefixes and sampling as one decoding batch, with the page
tables, and within DecodeCycle."""
import pytest
import torch

from tests.test_gpu_append_norm import near, reference
from tests.test_gpu_sample import plain
from tests.test_gpu_shared import check

pytestmark = pytest.mark.gpu
PAGE = 16


class Batch:
    """R requests on two documents with pictures: tables, a pool, a small model of one layer."""

    def __init__(self, kap, members=(4, 3), doc_pages=(9, 6), hkv=2, G=4, d=64, vocab=900, dt=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.kap, self.hkv, self.hq, self.d, self.dt, self.vocab = kap, hkv, hkv * G, d, dt, vocab
        R = self.R = sum(members)
        self.first = [0, members[0], R]
        i32 = dict(dtype=torch.int32, device="cuda")
        P, mp = sum(doc_pages) + 4 * R + 3, max(doc_pages) + 5
        ids = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
        self.K = torch.full((P, hkv, PAGE, d), float("nan"), dtype=dt, device="cuda")
        self.V = self.K.clone()
        self.pool = kap.KVPool(self.K, self.V, self.hq, torch.zeros(P, hkv, d, device="cuda"))
        self.bt = torch.full((R, mp), -1, **i32)
        self.len = torch.zeros(R, **i32)
        self.embed, self.W = rnd(vocab, 96), rnd(96, (self.hq + 2 * hkv) * d) * 0.1
        self.head = rnd(self.hq * d, vocab) * 0.4
        self.inv = kap.rope_inv_freq(d, 5e5, "cuda")
        self.axis = kap.rope_freq_axis(d, [d // 2 - 2 * (d // 8), d // 8, d // 8], True, "cuda")
        self.wq, self.wk = 0.5 + torch.rand(d, generator=g, device="cuda"), 0.5 + torch.rand(d, generator=g, device="cuda")
        self.groups = kap.PrefixGroups(torch.tensor(self.first, **i32), torch.tensor(doc_pages, **i32))
        at = 0
        self.offset = torch.zeros(R, **i32)     # rope position less logical position of the text after the pictures
        for k, n in enumerate(doc_pages):
            pages, T = ids[at:at + n], n * PAGE
            at += n
            self.bt[self.first[k]:self.first[k + 1], :n] = pages
            self.len[self.first[k]:self.first[k + 1]] = T
            # text, then a picture of 8 x 6 patches, then text from the picture's largest position on
            pos = torch.arange(T, device="cuda").repeat(3, 1)
            i = torch.arange(48, device="cuda")
            pos[0, 20:68], pos[1, 20:68], pos[2, 20:68] = 20, 20 + i // 6, 20 + i % 6
            pos[:, 68:] -= 40
            self.offset[self.first[k]:self.first[k + 1]] = -40
            slots = (pages.long()[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()
            self.append(torch.randint(0, vocab, (T,), generator=g, device="cuda"), pos.to(torch.int32), slots)
        self.free = ids[at:].contiguous()
        self.count = torch.tensor([self.free.numel()], **i32)
        self.g = g

    def project(self, tokens):
        y = (self.embed[tokens.long()] @ self.W).to(self.dt).view(len(tokens), -1, self.d)
        return y[:, :self.hq], y[:, self.hq:self.hq + self.hkv], y[:, self.hq + self.hkv:]

    def append(self, tokens, pos, slots):
        """Appends and checks what was written; the rotated queries."""
        q, k, v = self.project(tokens)
        out = torch.empty(q.shape, dtype=self.dt, device="cuda")
        self.kap.kap_append_kv_norm(self.pool, k, v, q, out, pos.contiguous(), slots, self.inv, self.wq, self.wk, 1e-6,
                                    self.axis)
        torch.cuda.synchronize()
        near(out, *reference(q, self.wq, 1e-6, pos, self.axis, self.inv))
        near(self.K[slots // PAGE, :, slots % PAGE], *reference(k, self.wk, 1e-6, pos, self.axis, self.inv))
        assert torch.equal(self.V[slots // PAGE, :, slots % PAGE], v)
        return out


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_decoding_on_shared_documents(kap, dt):
    b = Batch(kap, dt=dt)
    R, i32 = b.R, dict(dtype=torch.int32, device="cuda")
    tokens = torch.arange(R, **i32)
    ws = kap.workspace(kap.kap_shared_workspace_size(R, b.hkv, b.hq, b.d, R, 2), "cuda")
    off = torch.arange(R + 1, **i32)
    temp = torch.tensor([0.0, 0.7, 1.0, 1.3, 0.7, 1.0, 1.0], device="cuda")
    top_k = torch.tensor([0, 40, 0, 0, 5, 0, 0], **i32)
    top_p = torch.tensor([1.0, 0.9, 0.8, 1.0, 1.0, 0.95, 1.0], device="cuda")
    min_p = torch.tensor([0.0, 0.0, 0.0, 0.02, 0.0, 0.01, 0.0], device="cuda")
    for step in range(20):
        slots, pos = torch.full((R,), -1, device="cuda"), torch.zeros(R, **i32)
        new_len, granted, count2 = torch.zeros(R, **i32), torch.zeros(R, **i32), torch.zeros(1, **i32)
        start = b.len
        kap.kap_extend_tables(b.bt, start, torch.ones(R, **i32), b.free, b.count, count2, torch.zeros(R + 1, **i32), slots,
                              pos, new_len, granted)
        torch.cuda.synchronize()
        assert granted.all()
        q = b.append(tokens, (pos + b.offset).repeat(3, 1), slots)
        out, lse = torch.empty_like(q), torch.empty(R, b.hq, device="cuda")
        kap.kap_attn_verify_shared(b.pool, kap.PageMap(b.bt, start), kap.VerifyPolicy(off, start, 1, R), b.groups, q, out,
                                   lse, ws)
        torch.cuda.synchronize()
        check(dict(K=b.K, V=b.V, bt=b.bt, q=q, G=b.hq // b.hkv, R=R, starts=start.tolist(), windows=[1] * R), out, lse)
        logits = (out.float().view(R, -1) @ b.head).to(dt)
        u = torch.rand(R, generator=b.g, device="cuda")
        tok, lp, kept = torch.empty(R, **i32), torch.empty(R, device="cuda"), torch.empty(R, **i32)
        kap.kap_sample_tokens(logits, u, tok, temp, top_k, top_p, min_p, lp, kept)
        torch.cuda.synchronize()
        for r in range(R):
            may = plain(logits[r].float().cpu().numpy(), float(temp[r]), int(top_k[r]), float(top_p[r]), float(min_p[r]),
                        float(u[r]))
            assert (int(tok[r]), int(kept[r])) in may, (step, r)
        tokens, b.len, b.count = tok, new_len, count2
    assert kap.kap_device_error() == 0


def _cycle(kap, b, n_q, **kw):
    pol = kap.AccessPolicy(1, 1, 3, True, 8)
    return kap.DecodeCycle(b.pool, b.bt, b.len, b.len, 2, torch.tensor(n_q), b.inv, policy=pol, **kw)


@pytest.mark.parametrize("n_q", [[2] * 7, [3, 1, 2, 3, 3, 1, 2]])
def test_cycle_with_norms_offsets_and_groups(kap, n_q):
    """The cycle's steps against the calls that make it up, and its verification with groups against that without."""
    def batch():
        b = Batch(kap, d=128)
        for r in range(b.R):     # room for the window's tokens
            n = int(b.len[r]) // PAGE
            b.bt[r, n] = b.free[2 * r]
        return b
    res = []
    for groups in (True, False):
        b = batch()
        g = torch.Generator(device="cuda").manual_seed(5)
        tq = sum(n_q)
        proj = lambda n: [x.contiguous() for x in b.project(torch.randint(0, b.vocab, (n,), generator=g, device="cuda"))]  # noqa: E731
        kap.kap_build_summaries(b.pool, kap.PageMap(b.bt, b.len, b.len))
        cyc = _cycle(kap, b, n_q, norm=kap.QKNorm(b.wq, b.wk), rope_offset=b.offset, groups=b.groups if groups else None)
        assert not cyc.fused and cyc.launches_per_cycle() == 2 + (0 if len(set(n_q)) == 1 else 1) + 4 + 2 + int(groups)
        steps, win = [proj(b.R) for _ in range(2)], proj(tq)
        qs, qw = [s[0].clone() for s in steps], win[0].clone()
        cyc.run(steps[0][0].clone(), qs, [s[1] for s in steps], [s[2] for s in steps], qw, win[1], win[2])
        torch.cuda.synchronize()
        assert torch.isfinite(cyc.o_prop).all()
        # the appends: step i at position length + i, the window from the length on, all 40 positions behind
        r_of = torch.repeat_interleave(torch.arange(b.R, device="cuda"), torch.tensor(n_q, device="cuda"))
        i_of = torch.cat([torch.arange(n, device="cuda") for n in n_q])
        pos = (b.len[r_of] + i_of).to(torch.int32)
        none = torch.zeros(b.d // 2, dtype=torch.int32, device="cuda")
        near(qw, *reference(win[0], b.wq, 1e-6, (pos - 40)[None], none, b.inv))
        near(qs[1], *reference(steps[1][0], b.wq, 1e-6, (b.len + 1 - 40)[None], none, b.inv))
        slot = b.bt[r_of, (pos // PAGE).long()].long() * PAGE + pos % PAGE
        near(b.K[slot // PAGE, :, slot % PAGE], *reference(win[1], b.wk, 1e-6, (pos - 40)[None], none, b.inv))
        if groups:
            check(dict(K=b.K, V=b.V, bt=b.bt, q=qw, G=4, R=b.R, starts=b.len.tolist(), windows=n_q), cyc.o_ver, cyc.lse_ver)
        res.append((cyc.o_prop.clone(), cyc.o_ver.float(), cyc.lse_ver.clone()))
    assert torch.equal(res[0][0], res[1][0])
    # both verifications are within check()'s bound of 64 bits: a few bf16 roundings of values of size about 1
    assert (res[0][1] - res[1][1]).abs().max() <= 4 * 2.0 ** -8 and (res[0][2] - res[1][2]).abs().max() <= 1e-3
    assert kap.kap_device_error() == 0


def test_cycle_captured(kap):
    b = Batch(kap, d=128)
    for r in range(b.R):
        b.bt[r, int(b.len[r]) // PAGE] = b.free[2 * r]
    kap.kap_build_summaries(b.pool, kap.PageMap(b.bt, b.len, b.len))
    cyc = _cycle(kap, b, [2] * b.R, norm=kap.QKNorm(b.wq, b.wk), rope_offset=b.offset, groups=b.groups)
    q, k, v = [x.contiguous() for x in b.project(torch.arange(2 * b.R, device="cuda"))]
    raw, step = q.clone(), [x[:b.R].clone() for x in (q, k, v)]

    def run():
        q.copy_(raw)
        cyc.plan(step[0])
        cyc.verify(q, k, v)
    run()
    torch.cuda.synchronize()
    want = cyc.o_ver.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    cyc.o_ver.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cyc.o_ver, want)


def test_cycle_refusals(kap):
    b = Batch(kap)
    with pytest.raises(ValueError):
        _cycle(kap, b, [2] * 7, rope_offset=b.offset.long())
    with pytest.raises(ValueError):
        _cycle(kap, b, [2] * 7, rope_offset=b.offset[:3])
    packed = kap.PackedPool(b.pool, torch.zeros(2, b.hkv, kap.kap_packed_chunk_bytes(64), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        _cycle(kap, b, [2] * 7, packed=packed, groups=b.groups)
