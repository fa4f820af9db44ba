"""Measured cases of the 4-bit page cache, the token log-probabilities and the page-table step.

Every case is one pass through one operator, either in its plain form (`own` false: elementary torch operations in
32 bits, 64 where 32 lose what matters) or through the library's calls (`own` true).

The packed page format both forms read: the chunk of one (page, KV head) holds, for nb = head_dim / 64 blocks of 64
dims, K codes [nb][16 tokens][32 bytes], V codes alike, K parameters [nb][16 tokens][2] bf16 (scale, lowest value) and
V parameters alike. Byte b of a token's block holds dim 2b in its low and dim 2b + 1 in its high four bits; a code c
stands for lowest + scale * c. Physical pages below the 16-bit pool's size are 16-bit pages, the others packed ones.
"""
import math

import torch

own = False

PAGE = 16


def _kap():
    import selected_kv_sparse_gb300 as kap
    kap.load()
    return kap


# ------------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # the pages that three requests fill in one decode step, packed and read back
        dict(name="pack 3 pages", op="pack", pages=3, hkv=8, d=128),
        # one 32768-token prompt, packed after its prefill and read back
        dict(name="pack a 32K prompt", op="pack", pages=2048, hkv=8, d=128),
        # a decode step of one request with a 128-token budget per head
        dict(name="propose 1 x 8 pages", op="propose", R=1, hkv=8, G=4, d=128, ctx=40960, gen=3, sel=8, shared=False,
             ragged=False),
        # the Llama-3-8B-shaped proposal step: 4 requests, 128 pages of 2048 per head
        dict(name="propose 4 x 128 pages", op="propose", R=4, hkv=8, G=4, d=128, ctx=32768, gen=4, sel=128,
             shared=False, ragged=False),
        # short ragged prompts, heads of 64 dims, a window of 4
        dict(name="verify 2 x 1000 d64", op="verify", R=2, hkv=2, G=4, d=64, ctx=1000, gen=0, nq=4, ragged=True),
        # decode over the whole cache, 8 requests of 40960 tokens, one token each
        dict(name="decode 8 x 40960", op="verify", R=8, hkv=8, G=4, d=128, ctx=40960, gen=20, nq=1, ragged=False),
        # the Llama-3-8B-shaped verification window
        dict(name="verify 4 x 32768 q4", op="verify", R=4, hkv=8, G=4, d=128, ctx=32768, gen=0, nq=4, ragged=False),
        # the long-context window: 5 query heads a KV head, 8 rows
        dict(name="verify 1 x 131072 q8", op="verify", R=1, hkv=8, G=5, d=128, ctx=131072, gen=0, nq=8, ragged=False),
        # the rows of four verify windows of 5
        dict(name="logprobs 20 rows f32", op="logprobs", rows=20, vocab=128256, bf16=False, top=5, pad=0),
        # log probabilities of a prompt's tokens, with the 20 best alternatives of each
        dict(name="logprobs 2048 rows bf16", op="logprobs", rows=2048, vocab=128256, bf16=True, top=20, pad=0),
        # one decode step of 32 requests
        dict(name="tables 32 x 1", op="tables", R=32, new=1, long=0, ctx=32768, free=64),
        # a step of 1024 requests, a few of them with long new prompts
        dict(name="tables 1024 mixed", op="tables", R=1024, new=8, long=8192, ctx=4096, free=40000),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pack", "propose", "verify", "logprobs", "tables"])
    if op == "pack":
        return dict(op=op, pages=_log(rng, 1, 2000), hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]))
    if op == "propose":
        return dict(op=op, R=_log(rng, 1, 32), hkv=rng.choice([1, 2, 4, 8]), G=rng.randint(1, 8),
                    d=rng.choice([64, 128]), ctx=_log(rng, 20, 40000), gen=rng.randint(1, 40), sel=_log(rng, 1, 300),
                    shared=rng.random() < 0.3, ragged=rng.random() < 0.7)
    if op == "verify":
        G = rng.randint(1, 8)
        R = _log(rng, 1, 24)
        return dict(op=op, R=R, hkv=rng.choice([1, 2, 4, 8]), G=G, d=rng.choice([64, 128]),
                    ctx=_log(rng, 1, 200000 // R), gen=rng.randint(0, 40), nq=rng.randint(1, min(16, 64 // G)),
                    ragged=rng.random() < 0.7)
    if op == "logprobs":
        return dict(op=op, rows=_log(rng, 1, 1000), vocab=_log(rng, 40, 128256), bf16=rng.random() < 0.6,
                    top=rng.choice([0, 1, 3, 5, 20, 32]), pad=rng.choice([0, 0, 1, 8, 61]))
    return dict(op=op, R=_log(rng, 1, 1024), new=rng.randint(1, 40), long=rng.choice([0, 0, _log(rng, 16, 8000)]),
                ctx=_log(rng, 1, 32768), free=_log(rng, 4, 40000))


# ---------------------------------------------------------------------------------------------------- sizes of a case
def _lens(c):
    """Prompt lengths: equal, or falling to 40% and off the page boundaries."""
    if not c["ragged"]:
        return [c["ctx"]] * c["R"]
    return [max(1, int(c["ctx"] * (1.0 - 0.6 * r / c["R"])) - 5 * (r % 3)) for r in range(c["R"])]


def _windows(c):
    return [c["nq"] if not c["ragged"] else 1 + (c["nq"] - 1 + 3 * r) % c["nq"] for r in range(c["R"])]


def _chunk(d):
    return d // 64 * (2 * PAGE * 32 + 2 * PAGE * 4)


def _table_new(c):
    """New tokens of each request: mostly up to `new`, every eleventh none, every 64th a prompt of about `long`."""
    return [0 if r % 11 == 7 else (c["long"] - r % 50 if c["long"] and r % 64 == 5 and c["long"] > 50
                                   else 1 + (r * 7) % c["new"]) for r in range(c["R"])]


def work(c):
    if c["op"] == "pack":   # both directions: 16-bit pages read and written, packed chunks written and read
        n = c["pages"] * c["hkv"]
        return dict(bytes=2.0 * n * (2 * PAGE * c["d"] * 2 + _chunk(c["d"])), flops=n * 2 * PAGE * c["d"] * 8.0)
    if c["op"] == "propose":
        b = f = 0.0
        for L in _lens(c):
            packed = min(c["sel"], L // PAGE)
            tail = (L + c["gen"] + PAGE - 1) // PAGE - L // PAGE
            b += c["hkv"] * (packed * _chunk(c["d"]) + tail * 2 * PAGE * c["d"] * 2 + 8 * (packed + tail))
            f += c["hkv"] * c["G"] * (packed * PAGE + c["gen"]) * c["d"] * 4.0
        b += c["R"] * c["hkv"] * c["G"] * (c["d"] * 4 + 4)
        return dict(bytes=b, flops=f)
    if c["op"] == "verify":
        b = f = 0.0
        for L, n in zip(_lens(c), _windows(c)):
            end = L + c["gen"] + n
            packed = L // PAGE
            b += c["hkv"] * (packed * _chunk(c["d"]) + (end - packed * PAGE) * 2 * c["d"] * 2)
            b += 4 * ((end + PAGE - 1) // PAGE) + n * c["hkv"] * c["G"] * (c["d"] * 4 + 4)
            f += c["hkv"] * c["G"] * n * (end - n / 2) * c["d"] * 4.0
        return dict(bytes=b, flops=f)
    if c["op"] == "logprobs":
        n = c["rows"] * c["vocab"]
        return dict(bytes=n * (2.0 if c["bf16"] else 4.0) + c["rows"] * (16 + 8 * c["top"]), flops=n * 6.0)
    new = _table_new(c)
    return dict(bytes=sum(new) * 12.0 + c["R"] * 28.0 + sum(new) / PAGE * 8, flops=sum(new) * 4.0)


# ------------------------------------------------------------------------------------------------------------ inputs
def _perm(n, g):
    return torch.randperm(n, generator=g, device="cuda")


def _packed(n, hkv, d, g):
    """Packed chunks as a cache of normal keys and values holds them: codes around the middle, each (token, block)
    with its own scale and lowest value, values at half the keys' size."""
    nb = d // 64
    a = torch.randint(0, 256, (n, hkv, 2, nb, PAGE, 32), generator=g, device="cuda", dtype=torch.uint8)
    b = torch.randint(0, 256, (n, hkv, 2, nb, PAGE, 32), generator=g, device="cuda", dtype=torch.uint8)
    codes = ((((a & 15) + (b & 15)) >> 1) | ((((a >> 4) + (b >> 4)) >> 1) << 4)).reshape(n, hkv, -1)
    s = 0.32 * torch.exp(0.25 * torch.randn(n, hkv, 2, nb, PAGE, generator=g, device="cuda"))
    s[:, :, 1] *= 0.5
    lo = -s * (7.5 + 0.5 * torch.randn(n, hkv, 2, nb, PAGE, generator=g, device="cuda"))
    par = torch.stack([s, lo], dim=-1).to(torch.bfloat16).reshape(n, hkv, -1)
    return torch.cat([codes, par.view(torch.uint8)], dim=-1).contiguous()


def _cache(c, g, window):
    """A cache whose full prompt pages are packed and whose other pages (a partial prompt page, generated tokens, the
    window) are 16-bit ones, with shuffled page ids in both pools."""
    lens = _lens(c)
    ends = [L + c["gen"] + n for L, n in zip(lens, window)]
    n4 = [L // PAGE for L in lens]
    n16 = [(e + PAGE - 1) // PAGE - p for e, p in zip(ends, n4)]
    P16, P4 = max(1, sum(n16)), max(1, sum(n4))
    K = torch.randn(P16, c["hkv"], PAGE, c["d"], generator=g, device="cuda").to(torch.bfloat16)
    V = (0.5 * torch.randn(P16, c["hkv"], PAGE, c["d"], generator=g, device="cuda")).to(torch.bfloat16)
    packed = _packed(P4, c["hkv"], c["d"], g)
    p16, p4 = _perm(P16, g).to(torch.int32), _perm(P4, g).to(torch.int32) + P16
    mp = max(a + b for a, b in zip(n4, n16))
    bt = torch.full((c["R"], mp), -1, dtype=torch.int32, device="cuda")
    o16 = o4 = 0
    for r in range(c["R"]):
        bt[r, :n4[r]] = p4[o4:o4 + n4[r]]
        bt[r, n4[r]:n4[r] + n16[r]] = p16[o16:o16 + n16[r]]
        o4, o16 = o4 + n4[r], o16 + n16[r]
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(K=K, V=V, packed=packed, bt=bt, ctx=torch.tensor(lens, **i32), P16=P16, n4=n4, ends=ends, case=c)


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=c, op=c["op"])
    i32 = dict(dtype=torch.int32, device="cuda")
    if c["op"] == "pack":
        n, hkv, d = c["pages"], c["hkv"], c["d"]
        K = torch.empty(2 * n, hkv, PAGE, d, dtype=torch.bfloat16, device="cuda")
        V = torch.empty_like(K)
        # keys with a few large channels, as rotary keys have, and their own offset a channel
        ch = 1.0 + 3.0 * (torch.rand(hkv, 1, d, generator=g, device="cuda") > 0.95)
        off = 0.5 * torch.randn(hkv, 1, d, generator=g, device="cuda")
        K[:n] = (torch.randn(n, hkv, PAGE, d, generator=g, device="cuda") * ch + off).to(torch.bfloat16)
        V[:n] = (0.5 * torch.randn(n, hkv, PAGE, d, generator=g, device="cuda")).to(torch.bfloat16)
        s.update(K=K, V=V, src=_perm(n, g).to(torch.int32), dst=(_perm(n, g) + 2 * n).to(torch.int32),
                 back=torch.arange(n, 2 * n, **i32), packed=torch.zeros(n, hkv, _chunk(d), dtype=torch.uint8,
                                                                        device="cuda"))
        if own:
            kap = _kap()
            s["pool"] = kap.PackedPool(kap.KVPool(K, V, hkv), s["packed"])
        return s
    if c["op"] == "propose":
        s.update(_cache(c, g, [0] * c["R"]))
        rows = 1 if c["shared"] else c["hkv"]
        R, N = c["R"], torch.tensor(s["n4"], device="cuda")
        nsel = torch.clamp(N, max=c["sel"])
        mp = s["bt"].shape[1]
        ntail = torch.tensor([(e + PAGE - 1) // PAGE for e in s["ends"]], device="cuda") - N
        cap = int(nsel.max()) + int(ntail.max()) + 1
        score = torch.rand(R, rows, mp, generator=g, device="cuda")
        score[torch.arange(mp, device="cuda")[None, None] .expand(R, rows, mp) >= N[:, None, None]] = 2.0
        first = score.argsort(dim=-1)[:, :, :cap]   # the full prompt pages in random order, then the others
        if first.shape[2] < cap:
            first = torch.cat([first, first.new_zeros(R, rows, cap - first.shape[2])], dim=2)
        i = torch.arange(cap, device="cuda")[None, None]
        sel = torch.where(i < nsel[:, None, None], first, mp).sort(dim=-1).values
        lp = torch.where(i < nsel[:, None, None], sel, (N - nsel)[:, None, None] + i)
        used = i < (nsel + ntail)[:, None, None]
        lp = torch.where(used, lp, 0)
        vbt = torch.where(used, s["bt"][torch.arange(R, device="cuda")[:, None, None], lp.clamp(max=mp - 1)], 0)
        s.update(lp=lp.to(torch.int32).contiguous(), vbt=vbt.to(torch.int32).contiguous(),
                 nent=(nsel + ntail)[:, None].expand(R, rows).to(torch.int32).contiguous(),
                 nsel=nsel[:, None].expand(R, rows).to(torch.int32).contiguous(),
                 seq=torch.tensor(s["ends"], **i32), rows=rows, cap=cap,
                 q=torch.randn(R, c["hkv"] * c["G"], c["d"], generator=g, device="cuda").to(torch.bfloat16))
        tq = R
    elif c["op"] == "verify":
        w = _windows(c)
        s.update(_cache(c, g, w))
        off = torch.zeros(c["R"] + 1, **i32)
        off[1:] = torch.tensor(w, **i32).cumsum(0)
        tq = sum(w)
        s.update(windows=w, off=off, start=s["ctx"] + c["gen"], seq=torch.tensor(s["ends"], **i32),
                 q=torch.randn(tq, c["hkv"] * c["G"], c["d"], generator=g, device="cuda").to(torch.bfloat16))
    elif c["op"] == "logprobs":
        rows, V, pad = c["rows"], c["vocab"], c["pad"]
        lg = torch.empty(rows, V + pad, dtype=torch.bfloat16 if c["bf16"] else torch.float32, device="cuda")
        lg.normal_(0.0, 2.5, generator=g)
        tok = torch.randint(0, V, (rows,), generator=g, device="cuda")
        r = torch.arange(rows, device="cuda")
        # the given token is often a likely one; every fourth row is decoded under a mask that keeps half the tokens
        lift = torch.randn(rows, generator=g, device="cuda") * 3.0 + 8.0
        lg[r, tok] = lift.to(lg.dtype)
        masked = torch.rand(-(-rows // 4), V, generator=g, device="cuda") < 0.5
        masked[:, 0] = False
        part = lg[::4, :V]
        part[masked] = float("-inf")
        s.update(logits=lg[:, :V], tok=tok.to(torch.int32))
        if own:
            kap = _kap()
            f = dict(dtype=torch.float32, device="cuda")
            s.update(logprob=torch.empty(rows, **f), entropy=torch.empty(rows, **f), rank=torch.empty(rows, **i32),
                     top_ids=torch.empty(rows, c["top"], **i32), top_lp=torch.empty(rows, c["top"], **f),
                     ws=kap.workspace(kap.kap_logprobs_workspace_size(rows, V), "cuda"))
        return s
    else:
        R = c["R"]
        seq = (torch.rand(R, generator=g, device="cuda") * c["ctx"]).to(torch.int32)
        new = torch.tensor(_table_new(c), **i32)
        gone = ((torch.arange(R, device="cuda") % 11 == 7) & (torch.rand(R, generator=g, device="cuda") < 0.7))
        have = (c["ctx"] + PAGE - 1) // PAGE
        mp = have + (max(_table_new(c)) + PAGE - 1) // PAGE + 1
        ids = _perm(R * have + c["free"], g).to(torch.int32)
        bt = torch.full((R, mp), -1, **i32)
        bt[:, :have] = ids[:R * have].view(R, have)
        j = torch.arange(mp, device="cuda")[None]
        bt[j >= ((seq + PAGE - 1) // PAGE)[:, None]] = -1
        stack = torch.full((R * have + c["free"],), -1, **i32)
        stack[:c["free"]] = ids[R * have:]
        T = sum(_table_new(c))
        s.update(bt=bt, seq=seq, new=new, gone=gone.to(torch.int32), stack=stack,
                 count=torch.tensor([c["free"]], **i32), T=T,
                 out=dict(count1=torch.empty(1, **i32), count2=torch.empty(1, **i32), seq1=torch.empty(R, **i32),
                          seq2=torch.empty(R, **i32), off=torch.empty(R + 1, **i32), granted=torch.empty(R, **i32),
                          slots=torch.empty(T, dtype=torch.int64, device="cuda"), pos=torch.empty(T, **i32)))
        return s
    # buffers that a user's program keeps for attention
    hq = c["hkv"] * c["G"]
    if own:
        kap = _kap()
        s["out"] = torch.empty(tq, hq, c["d"], dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(tq, hq, dtype=torch.float32, device="cuda")
        nq = 1 if c["op"] == "propose" else max(s["windows"])
        s["pool"] = kap.PackedPool(kap.KVPool(s["K"], s["V"], hq), s["packed"])
        s["map"] = kap.PageMap(s["bt"], s["ctx"], s["seq"])
        s["ws"] = kap.workspace(kap.kap_packed_workspace_size(c["R"], c["hkv"], hq, c["d"], nq), "cuda")
        if c["op"] == "propose":
            s["view"] = kap.View(s["rows"], s["cap"], s["vbt"], s["lp"], s["nent"], s["nsel"])
        else:
            s["policy"] = kap.VerifyPolicy(s["off"], s["start"], nq, tq)
    return s


# ------------------------------------------------------------------------------------------------------- plain forms
def _pages(chunk, d):
    """Keys and values [...][16][d] (fp32) that packed chunks [...][bytes] stand for."""
    nb = d // 64
    n = nb * PAGE * 32
    lead = chunk.shape[:-1]
    codes = chunk[..., :2 * n].reshape(*lead, 2, nb, PAGE, 32)
    par = chunk[..., 2 * n:].contiguous().view(torch.bfloat16).reshape(*lead, 2, nb, PAGE, 2).float()
    c = torch.stack([codes & 15, codes >> 4], dim=-1).reshape(*lead, 2, nb, PAGE, 64).float()
    v = par[..., 1:] + par[..., :1] * c
    v = v.transpose(-3, -2).reshape(*lead, 2, PAGE, d)
    return v[..., 0, :, :], v[..., 1, :, :]


def _gather(s, ids, heads):
    """Keys and values [..., 16, d] of (page id, head), from whichever pool the id names."""
    P16 = s["P16"]
    kp, vp = _pages(s["packed"][(ids - P16).clamp(min=0), heads], s["case"]["d"])
    low = ids.clamp(min=0, max=P16 - 1)
    is4 = (ids >= P16)[..., None, None]
    return torch.where(is4, kp, s["K"][low, heads].float()), torch.where(is4, vp, s["V"][low, heads].float())


def _attend(q, k, v, see):
    """q [..., M, d], k, v [..., T, d], see [..., M, T]: outputs and log-sum-exps; a hidden token counts for nothing."""
    x = (q @ k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    x = x.masked_fill(~see, float("-inf"))
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - m)
    n = p.sum(dim=-1, keepdim=True)
    return (p @ v) / n, (m + torch.log(n))[..., 0]


def _plain_propose(s):
    c = s["case"]
    R, hkv, G, d, cap = c["R"], c["hkv"], c["G"], c["d"], s["cap"]
    ids = s["vbt"].long().expand(R, hkv, cap)
    lp = s["lp"].long().expand(R, hkv, cap)
    k, v = _gather(s, ids, torch.arange(hkv, device="cuda")[None, :, None])
    i = torch.arange(cap, device="cuda")
    pos = lp[..., None] * PAGE + torch.arange(PAGE, device="cuda")
    see = (i < s["nent"][..., None])[..., None] & (pos < s["seq"][:, None, None, None])
    see = see & ((i < s["nsel"][..., None])[..., None] | (pos >= s["ctx"][:, None, None, None]))
    q = s["q"].float().view(R, hkv, G, d)
    o, l = _attend(q, k.flatten(2, 3), v.flatten(2, 3), see.flatten(2)[:, :, None, :])
    return o.reshape(R, hkv * G, d).to(torch.bfloat16), l.reshape(R, hkv * G)


def _plain_verify(s):
    c = s["case"]
    R, hkv, G, d = c["R"], c["hkv"], c["G"], c["d"]
    nq, mp, tq = max(s["windows"]), s["bt"].shape[1], s["q"].shape[0]
    ids = s["bt"].long()[:, None, :].expand(R, hkv, mp)
    k, v = _gather(s, ids, torch.arange(hkv, device="cuda")[None, :, None])
    t = torch.arange(tq, device="cuda")
    r = torch.searchsorted(s["off"].long(), t, right=True) - 1
    i = t - s["off"].long()[r]
    q = torch.zeros(R, nq, hkv, G, d, device="cuda")
    q[r, i] = s["q"].float().view(tq, hkv, G, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(R, hkv, G * nq, d)
    pos = torch.arange(mp * PAGE, device="cuda")
    see = pos[None, None] <= (s["start"].long()[:, None] + torch.arange(nq, device="cuda"))[..., None]
    see = see[:, None, None].expand(R, hkv, G, nq, mp * PAGE).reshape(R, hkv, G * nq, mp * PAGE)
    o, l = _attend(q, k.flatten(2, 3), v.flatten(2, 3), see)
    o = o.view(R, hkv, G, nq, d).permute(0, 3, 1, 2, 4)[r, i]
    l = l.view(R, hkv, G, nq).permute(0, 3, 1, 2)[r, i]
    return o.reshape(tq, hkv * G, d).to(torch.bfloat16), l.reshape(tq, hkv * G)


def _through_codes(x):
    """The values [n][hkv][16][d] that 4-bit groups of 64 dims give back, in 64 bits up to the last rounding."""
    n, hkv, _, d = x.shape
    x = x.double().view(n, hkv, PAGE, d // 64, 64)
    lo = x.amin(dim=-1, keepdim=True)
    want = (x.amax(dim=-1, keepdim=True) - lo) / 15.0
    bits = want.float().view(torch.int32) & -65536      # the bf16 at or just below, then up where that is too small
    s = bits.view(torch.float32)
    s = torch.where(s.double() < want, (bits + 65536).view(torch.float32), s).double()
    code = torch.where(s > 0, torch.round((x - lo) / torch.where(s > 0, s, 1.0)), 0.0)
    return (lo + s * code).view(n, hkv, PAGE, d).to(torch.bfloat16)


def _plain_logprobs(s):
    x = s["logits"].float()
    rows, V = x.shape
    tok = s["tok"].long()[:, None]
    m = x.amax(dim=-1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(dim=-1, keepdim=True)
    lse = m + torch.log(z)
    lp = torch.where(torch.isinf(x), 0.0, x - lse)
    entropy = -(e / z * lp).sum(dim=-1)
    # one whole number a token that sorts as (logit, then lower id): the bits of the float, made monotone
    b = (x + 0.0).view(torch.int32)
    key = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long() * (1 << 32) + (V - 1 - torch.arange(V, device="cuda"))
    rank = (key > key.gather(1, tok)).sum(dim=-1).to(torch.int32)
    best = torch.topk(key, s["case"]["top"], dim=-1).values
    ids = V - 1 - (best & 0xFFFFFFFF)
    return (x.gather(1, tok) - lse)[:, 0], entropy, rank, ids.to(torch.int32), x.gather(1, ids) - lse


def _plain_tables(s):
    bt, seq, new, gone, count = s["bt"].clone(), s["seq"].long(), s["new"].long(), s["gone"].long(), s["count"].long()
    R, mp = bt.shape
    stack = s["stack"].clone()
    dev = dict(device="cuda")
    # the gone requests' pages go on the free stack, in request and then in page order
    pages = (seq + PAGE - 1) // PAGE
    back = pages * gone
    at = count + back.cumsum(0) - back
    j = torch.arange(mp, **dev)[None]
    put = j < back[:, None]
    put_at = torch.where(put, at[:, None] + j, stack.shape[0])
    wide = torch.cat([stack, stack.new_zeros(1)])
    wide[put_at.flatten()] = torch.where(put, bt, 0).flatten()
    stack = wide[:-1]
    count1 = count + back.sum()
    seq1 = seq * (1 - gone)
    # the others' new pages come from its top, in request order
    old = (seq1 + PAGE - 1) // PAGE
    need = (seq1 + new + PAGE - 1) // PAGE - old
    first = need.cumsum(0) - need
    granted = (need == 0) | (first + need <= count1)
    take = (j >= old[:, None]) & (j < (old + need)[:, None]) & granted[:, None]
    src = (count1 - 1 - first)[:, None] - (j - old[:, None])
    bt = torch.where(take, stack[src.clamp(0, stack.shape[0] - 1)], bt)
    off = torch.cat([torch.zeros(1, dtype=torch.long, **dev), new.cumsum(0)])
    t = torch.arange(s["T"], **dev)
    r = torch.searchsorted(off, t, right=True) - 1
    pos = seq1[r] + t - off[r]
    slot = torch.where(granted[r], bt[r, pos // PAGE].long() * PAGE + pos % PAGE, -1)
    count2 = count1 - (need * granted).sum()
    i32 = torch.int32
    return (bt, stack, count2.to(i32), (seq1 + new * granted).to(i32), off.to(i32), granted.to(i32), slot, pos.to(i32))


# ----------------------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if op == "pack":
        n = s["case"]["pages"]
        if own:
            kap = _kap()
            kap.kap_pack_pages(s["pool"], s["src"], s["dst"])
            kap.kap_unpack_pages(s["pool"], s["dst"], s["back"])
            return s["K"][n:], s["V"][n:]
        return _through_codes(s["K"][s["src"].long()]), _through_codes(s["V"][s["src"].long()])
    if op == "propose":
        if own:
            _kap().kap_attn_propose_packed(s["pool"], s["map"], s["view"], s["q"], s["out"], s["lse"], s["ws"])
            return s["out"], s["lse"]
        return _plain_propose(s)
    if op == "verify":
        if own:
            _kap().kap_attn_verify_packed(s["pool"], s["map"], s["policy"], s["q"], s["out"], s["lse"], s["ws"])
            return s["out"], s["lse"]
        return _plain_verify(s)
    if op == "logprobs":
        if own:
            _kap().kap_token_logprobs(s["logits"], s["tok"], s["logprob"], s["ws"], entropy=s["entropy"],
                                      rank=s["rank"], top_ids=s["top_ids"], top_logprobs=s["top_lp"])
            return s["logprob"], s["entropy"], s["rank"], s["top_ids"], s["top_lp"]
        return _plain_logprobs(s)
    if own:
        kap, o = _kap(), s["out"]
        kap.kap_release_tables(s["bt"], s["seq"], s["gone"], s["stack"], s["count"], o["count1"], o["seq1"])
        kap.kap_extend_tables(s["bt"], o["seq1"], s["new"], s["stack"], o["count1"], o["count2"], o["off"],
                              o["slots"], o["pos"], o["seq2"], o["granted"])
        return s["bt"], s["stack"], o["count2"], o["seq2"], o["off"], o["granted"], o["slots"], o["pos"]
    return _plain_tables(s)


# ------------------------------------------------------------------------------------------------------ in 64 bits
def _words(chunk, d, which, block):
    """The 64-bit values [n][16][64] of one block of packed chunks [n][bytes]: K for which = 0, V for 1."""
    nb = d // 64
    at = (which * nb + block) * 512
    byte = chunk[:, at:at + 512].reshape(-1, 16, 32).to(torch.int64)
    p = 2 * nb * 512 + (which * nb + block) * 64
    pair = chunk[:, p:p + 64].reshape(-1, 16, 2, 2).to(torch.int64)
    f = ((pair[..., 0] | pair[..., 1] << 8) << 16).to(torch.int32).view(torch.float32).double()
    out = torch.empty(chunk.shape[0], 16, 64, dtype=torch.float64, device=chunk.device)
    out[:, :, 0::2] = f[..., 1:] + f[..., :1] * (byte % 16)
    out[:, :, 1::2] = f[..., 1:] + f[..., :1] * (byte // 16)
    return out


def _exact_rows(s, ids, h, which):
    """The 64-bit keys or values [len(ids) * 16][d] of one head of a list of pages."""
    d, P16 = s["case"]["d"], s["P16"]
    out = torch.empty(len(ids), PAGE, d, dtype=torch.float64, device="cuda")
    four = ids >= P16
    ch = s["packed"][ids[four] - P16, h]
    for b in range(d // 64):
        out[four, :, 64 * b:64 * b + 64] = _words(ch, d, which, b)
    out[~four] = (s["V"] if which else s["K"])[ids[~four], h].double()
    return out.view(-1, d)


def _exact_head(q, k, v, see):
    """One query [d] over the tokens that `see` keeps."""
    k, v = k[see], v[see]
    x = (k * q).sum(dim=1) / math.sqrt(len(q))
    lse = torch.logsumexp(x, dim=0)
    return (torch.exp(x - lse)[:, None] * v).sum(dim=0), lse


def exact(c, seed):
    op = c["op"]
    s = prepare(c, seed)
    if op == "pack":
        res = []
        for x in (s["K"], s["V"]):
            y = x[s["src"].long()].double().reshape(-1, 64)
            lo, hi = y.min(dim=1).values, y.max(dim=1).values
            e = torch.frexp((hi - lo) / 15.0).exponent   # the smallest number of 8 bits that is not below range / 15
            ulp = (e.long() - 8 + 1023 << 52).view(torch.float64)   # two to the power e - 8, exactly
            sc = torch.ceil((hi - lo) / 15.0 / ulp) * ulp
            code = ((y - lo[:, None]) / torch.where(sc > 0, sc, torch.ones_like(sc))[:, None]).round()
            res.append((lo[:, None] + sc[:, None] * code).view(c["pages"], c["hkv"], PAGE, c["d"]))
        return tuple(res)
    if op in ("propose", "verify"):
        R, hkv, G, d = c["R"], c["hkv"], c["G"], c["d"]
        w = [1] * R if op == "propose" else s["windows"]
        o = torch.empty(sum(w), hkv * G, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(sum(w), hkv * G, dtype=torch.float64, device="cuda")
        t0 = 0
        for r in range(R):
            for h in range(hkv):
                if op == "propose":
                    row = h if s["rows"] > 1 else 0
                    n, ns = int(s["nent"][r, row]), int(s["nsel"][r, row])
                    ids, lp = s["vbt"][r, row, :n].long(), s["lp"][r, row, :n].long()
                    pos = (lp[:, None] * PAGE + torch.arange(PAGE, device="cuda")).flatten()
                    chosen = (torch.arange(n, device="cuda") < ns)[:, None].expand(n, PAGE).flatten()
                    base = chosen | (pos >= int(s["ctx"][r]))
                    last = int(s["seq"][r]) - 1
                else:
                    end = s["ends"][r]
                    ids = s["bt"][r, :(end + PAGE - 1) // PAGE].long()
                    pos = torch.arange(len(ids) * PAGE, device="cuda")
                    base = pos >= 0
                    last = int(s["start"][r])
                k, v = _exact_rows(s, ids, h, 0), _exact_rows(s, ids, h, 1)
                for i in range(w[r]):
                    for a in range(h * G, h * G + G):
                        o[t0 + i, a], lse[t0 + i, a] = _exact_head(s["q"][t0 + i, a].double(), k, v,
                                                                   base & (pos <= last + i))
            t0 += w[r]
        return o, lse
    if op == "logprobs":
        lp, ent, top = [], [], []
        for r in range(c["rows"]):
            x = s["logits"][r].double()
            y = x - torch.logsumexp(x, dim=0)
            lp.append(y[int(s["tok"][r])])
            z = y[torch.isfinite(y)]
            ent.append(-(torch.exp(z) * z).sum())
            top.append(torch.topk(y, c["top"]).values)   # values alone: the ids of equal ones do not matter here
        return torch.stack(lp), torch.stack(ent), None, None, torch.stack(top)
    return None
