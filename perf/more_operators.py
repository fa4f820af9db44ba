"""Measured cases of the normalising KV append with several position axes, of attention over a prefix that requests share,
and of token sampling.

Every case is one pass through one operator, either in its plain form (`own` false: elementary torch operations in
32 bits, 64 where 32 lose what matters: angles of far positions, sums that a border is compared with) or through the
library's calls (`own` true).

append: rows of queries and keys [T][heads][d], views of one fused projection, are divided by the root of their mean
square (plus eps) and multiplied by a weight a dim where weights are given, and rotated in pairs (i, i + d/2) by
pos[axis(i)] * inv_freq[i]; keys and values go to their cache slots (slot -1: nowhere), queries to their own buffer.
shared: causal windows over paged caches whose requests come in groups; the tables of a group's requests begin with the
same pages.
sample: of a row of logits x at temperature T, the tokens of weight w = exp((x - max) / T) that are among the top_k first
(logit descending, lower id first) and weigh min_p or more; of these the shortest run from the first that holds top_p of
their weight; of these the first in id order whose running sum passes u times their sum. T = 0 takes the first token.
"""
import math
import random

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
        # one decode step of 4 requests: 32 query and 8 KV heads, norms of both, text positions
        dict(name="append 4 tokens", op="append", T=4, hkv=8, G=4, d=128, bf16=True, axes=1, norm=True, start=32768,
             skip=False),
        # the windows of 64 requests with 5 tokens each, positions of three axes in turn, a padded batch
        dict(name="append 320 tokens 3 axes", op="append", T=320, hkv=8, G=5, d=128, bf16=True, axes=3, norm=True,
             start=40960, skip=True),
        # a small fp32 model's prompt chunk, rotation without norms
        dict(name="append 1000 tokens f32 d64", op="append", T=1000, hkv=2, G=4, d=64, bf16=False, axes=1, norm=False,
             start=0, skip=True),
        # a prompt of text and images
        dict(name="append 16384 tokens 3 axes", op="append", T=16384, hkv=8, G=4, d=128, bf16=True, axes=3, norm=True,
             start=0, skip=False),
        # two answers sampled from one short prompt, heads of 64 dims
        dict(name="shared 2 x 1000 d64", op="shared", R=2, groups=1, hkv=2, G=4, d=64, prefix=1000, suffix=100, nq=1,
             bf16=True, ragged=True),
        # 32 questions on one 32768-token document, one decode step
        dict(name="shared 32 x 32768", op="shared", R=32, groups=1, hkv=8, G=4, d=128, prefix=32768, suffix=512, nq=1,
             bf16=True, ragged=True),
        # 64 requests on five documents, verification windows of up to 5
        dict(name="shared 64 in 5 groups q5", op="shared", R=64, groups=5, hkv=8, G=4, d=128, prefix=16384, suffix=700,
             nq=5, bf16=True, ragged=True),
        # windows of 8 over one 131072-token document, 5 query heads a KV head
        dict(name="shared 8 x 131072 q8", op="shared", R=8, groups=1, hkv=8, G=5, d=128, prefix=131072, suffix=256, nq=8,
             bf16=True, ragged=False),
        # the next tokens of 4 requests
        dict(name="sample 4 rows", op="sample", rows=4, vocab=128256, bf16=True, pad=0, top_k=50, top_p=0.9, min_p=0.0,
             mixed=False),
        # the rows of 16 windows of 5 whose requests each have settings of their own
        dict(name="sample 80 rows f32 mixed", op="sample", rows=80, vocab=128256, bf16=False, pad=0, top_k=40, top_p=0.95,
             min_p=0.05, mixed=True),
        # a small vocabulary, padded rows, no limits
        dict(name="sample 300 rows of 32000", op="sample", rows=300, vocab=32000, bf16=True, pad=61, top_k=0, top_p=1.0,
             min_p=0.0, mixed=False),
        # a large batch under top-p alone
        dict(name="sample 2048 rows top-p", op="sample", rows=2048, vocab=128256, bf16=True, pad=0, top_k=0, top_p=0.9,
             min_p=0.0, mixed=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "shared", "sample"])
    if op == "append":
        hkv, G, d, bf16 = rng.choice([1, 2, 4, 8]), rng.randint(1, 8), rng.choice([64, 128]), rng.random() < 0.7
        most = 400000000 // (hkv * (2 * G + 4) * d * (2 if bf16 else 4))
        return dict(op=op, T=_log(rng, 1, min(16384, most)), hkv=hkv, G=G, d=d, bf16=bf16,
                    axes=rng.choice([1, 1, 2, 3, 4]), norm=rng.random() < 0.7,
                    start=rng.choice([0, _log(rng, 1, 2000000)]), skip=rng.random() < 0.4)
    if op == "shared":
        bf16 = rng.random() < 0.85
        G = rng.randint(1, 8)
        R = _log(rng, 1, 64 if bf16 else 8)
        groups = rng.choice([1, 1, rng.randint(1, R)])
        return dict(op=op, R=R, groups=groups, hkv=rng.choice([1, 2, 4, 8]), G=G, d=rng.choice([64, 128]),
                    prefix=_log(rng, 1, (100000 if bf16 else 4000) // groups), suffix=rng.choice([0, _log(rng, 1, 1500)]),
                    nq=rng.choice([1, 1, rng.randint(1, min(8, 64 // G))]), bf16=bf16, ragged=rng.random() < 0.7)
    return dict(op=op, rows=_log(rng, 1, 1000), vocab=_log(rng, 40, 128256), bf16=rng.random() < 0.6,
                pad=rng.choice([0, 0, 1, 8, 61]), top_k=rng.choice([0, 1, 20, 50, _log(rng, 1, 2000)]),
                top_p=rng.choice([1.0, rng.uniform(0.3, 0.98)]), min_p=rng.choice([0.0, 0.0, rng.uniform(0.01, 0.3)]),
                mixed=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------------- sizes of a case
def _groups(c):
    """The first request of each group and R: uneven shares of the requests, one at least."""
    R, n = c["R"], c["groups"]
    if not c["ragged"]:
        return [g * R // n for g in range(n + 1)]
    w = [1 + (5 * g + 2) % 7 for g in range(n)]
    off, spare = [0], R - n
    for g in range(n):
        off.append(off[-1] + 1 + spare * w[g] // sum(w))
    return off[:-1] + [R]


def _prefixes(c):
    """Shared pages of each group (the last group's prefix is the shortest)."""
    return [max(0, int(c["prefix"] * (1.0 - (0.5 * g / c["groups"] if c["ragged"] else 0.0)))) // PAGE
            for g in range(c["groups"])]


def _starts(c):
    """Tokens that each request holds before its window: its group's prefix and a suffix of its own."""
    off, pre = _groups(c), _prefixes(c)
    res = []
    for g in range(c["groups"]):
        for r in range(off[g], off[g + 1]):
            own_part = c["suffix"] if not c["ragged"] else c["suffix"] * ((7 * r + 3) % 11) // 10
            res.append(pre[g] * PAGE + own_part)
    return res


def _windows(c):
    return [c["nq"] if not c["ragged"] else 1 + (c["nq"] - 1 + 3 * r) % c["nq"] for r in range(c["R"])]


def work(c):
    if c["op"] == "append":
        n = c["T"] * c["hkv"] * c["d"] * (2 if c["bf16"] else 4)
        return dict(bytes=n * (2.0 * c["G"] + 4.0) + c["T"] * (4.0 * c["axes"] + 8.0),
                    flops=c["T"] * c["hkv"] * (c["G"] + 1) * c["d"] * 8.0)
    if c["op"] == "shared":
        es, hq = (2 if c["bf16"] else 4), c["hkv"] * c["G"]
        starts, w, off, pre = _starts(c), _windows(c), _groups(c), _prefixes(c)
        b = sum(pre) * PAGE * c["hkv"] * c["d"] * 2.0 * es
        f = 0.0
        for g in range(c["groups"]):
            for r in range(off[g], off[g + 1]):
                b += (starts[r] + w[r] - pre[g] * PAGE) * c["hkv"] * c["d"] * 2.0 * es
                b += w[r] * hq * (c["d"] * 2.0 * es + 4.0) + 4.0 * (starts[r] + w[r]) / PAGE
                f += hq * w[r] * (starts[r] + (w[r] + 1) / 2.0) * c["d"] * 4.0
        return dict(bytes=b, flops=f)
    n = c["rows"] * c["vocab"]
    return dict(bytes=n * (2.0 if c["bf16"] else 4.0) + c["rows"] * 32.0, flops=n * 6.0)


# ------------------------------------------------------------------------------------------------------------ inputs
def _positions(c, seed):
    """Position ids [axes][T]: text counts on all axes alike, a picture's patches hold one time and count rows and
    columns (and a fourth axis a patch's layer), and the text after it goes on from the largest."""
    rng = random.Random(seed)
    rows = [[] for _ in range(c["axes"])]
    at = c["start"]
    while len(rows[0]) < c["T"]:
        n = rng.randint(1, 400)
        for x in rows:
            x.extend(range(at, at + n))
        at += n
        if c["axes"] > 1:
            h, w = rng.randint(2, 40), rng.randint(2, 40)
            for k, x in enumerate(rows):
                x.extend(at + ((i // w, i // w, i % w, i % 7)[k] if k else 0) for i in range(h * w))
            at += max(h, w)
    return torch.tensor([x[:c["T"]] for x in rows], dtype=torch.int32, device="cuda")


def _axis_of(c):
    """The axis of each of the d/2 pairs, dealt out in turn, with the last pairs left to the first axis."""
    half, n = c["d"] // 2, c["axes"]
    k = half // n - (1 if n > 1 else 0)
    return [i % n if i % n and i < n * k else 0 for i in range(half)]


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case=c, op=c["op"])
    i32 = dict(dtype=torch.int32, device="cuda")
    f32 = dict(dtype=torch.float32, device="cuda")
    if c["op"] == "append":
        T, hkv, d = c["T"], c["hkv"], c["d"]
        hq = hkv * c["G"]
        dt = torch.bfloat16 if c["bf16"] else torch.float32
        ch = 1.0 + 3.0 * (torch.rand(hq + 2 * hkv, d, generator=g, device="cuda") > 0.95)
        qkv = (torch.randn(T, hq + 2 * hkv, d, generator=g, device="cuda") * ch).to(dt)   # one projection's output
        P = (T + PAGE - 1) // PAGE + 1
        slots = torch.randperm(P * PAGE, generator=g, device="cuda")[:T].contiguous()
        if c["skip"]:   # a padded batch: every seventh token is nobody's
            slots[6::7] = -1
        inv = torch.tensor([float(5.0e5 ** (-2.0 * i / d)) for i in range(d // 2)], **f32)
        s.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], slots=slots, inv=inv,
                 pos=_positions(c, seed), axis=torch.tensor(_axis_of(c), **i32),
                 K=torch.zeros(P, hkv, PAGE, d, dtype=dt, device="cuda"),
                 V=torch.zeros(P, hkv, PAGE, d, dtype=dt, device="cuda"),
                 wq=0.2 + torch.rand(d, generator=g, **f32) * 1.6, wk=0.2 + torch.rand(d, generator=g, **f32) * 1.6)
        if own:
            s["q_out"] = torch.empty(T, hq, d, dtype=dt, device="cuda")
            s["pool"] = _kap().KVPool(s["K"], s["V"], hq)
        return s
    if c["op"] == "shared":
        R, hkv, d = c["R"], c["hkv"], c["d"]
        hq = hkv * c["G"]
        dt = torch.bfloat16 if c["bf16"] else torch.float32
        off, pre, starts, w = _groups(c), _prefixes(c), _starts(c), _windows(c)
        ends = [a + b for a, b in zip(starts, w)]
        pages = [(e + PAGE - 1) // PAGE for e in ends]
        mp = max(pages)
        P = sum(pre) + sum(pages[r] - pre[k] for k in range(c["groups"]) for r in range(off[k], off[k + 1]))
        ids = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
        bt = torch.full((R, mp), -1, **i32)
        at = 0
        for k in range(c["groups"]):
            head = ids[at:at + pre[k]]
            at += pre[k]
            for r in range(off[k], off[k + 1]):
                bt[r, :pre[k]] = head
                bt[r, pre[k]:pages[r]] = ids[at:at + pages[r] - pre[k]]
                at += pages[r] - pre[k]
        qo = torch.zeros(R + 1, **i32)
        qo[1:] = torch.tensor(w, **i32).cumsum(0)
        s.update(K=torch.randn(P, hkv, PAGE, d, generator=g, device="cuda").to(dt),
                 V=(0.5 * torch.randn(P, hkv, PAGE, d, generator=g, device="cuda")).to(dt), bt=bt, starts=starts,
                 windows=w, qo=qo, start=torch.tensor(starts, **i32), group=torch.tensor(off, **i32),
                 prefix=torch.tensor(pre, **i32),
                 q=(1.5 * torch.randn(sum(w), hq, d, generator=g, device="cuda")).to(dt))
        if own:
            kap = _kap()
            s["out"] = torch.empty(sum(w), hq, d, dtype=dt, device="cuda")
            s["lse"] = torch.empty(sum(w), hq, **f32)
            s["pool"] = kap.KVPool(s["K"], s["V"], hq)
            s["map"] = kap.PageMap(bt, s["start"])
            s["policy"] = kap.VerifyPolicy(qo, s["start"], max(w), sum(w))
            s["groups"] = kap.PrefixGroups(s["group"], s["prefix"])
            s["ws"] = kap.workspace(kap.kap_shared_workspace_size(R, hkv, hq, d, sum(w), c["groups"]), "cuda")
        return s
    rows, V = c["rows"], c["vocab"]
    lg = torch.empty(rows, V + c["pad"], dtype=torch.bfloat16 if c["bf16"] else torch.float32, device="cuda")
    # two rows in three are sure of a few tokens, the others spread over many; every fourth row is decoded under a mask
    lg.normal_(0.0, 1.0, generator=g)
    lg[::3] *= 2.5
    r = torch.arange(rows, device="cuda")
    for _ in range(8):
        t = torch.randint(0, V, (rows,), generator=g, device="cuda")
        lift = torch.randn(rows, generator=g, device="cuda") * 2.0 + torch.where(r % 3 == 0, 6.0, 14.0)
        lg[r, t] = lift.to(lg.dtype)
    masked = torch.rand(-(-rows // 4), V, generator=g, device="cuda") < 0.5
    masked[:, 0] = False
    lg[::4, :V][masked] = float("-inf")
    pick = torch.rand(4, rows, generator=g, device="cuda")
    temp = torch.where(r % 16 == 5, 0.0, 0.6 + 0.1 * torch.floor(pick[0] * 7.0))
    on = pick[1:] < 0.5 if c["mixed"] else torch.ones(3, rows, dtype=torch.bool, device="cuda")
    s.update(logits=lg[:, :V], temp=temp, top_k=torch.where(on[0], c["top_k"], 0).to(torch.int32),
             top_p=torch.where(on[1], c["top_p"], 1.0).float(), min_p=torch.where(on[2], c["min_p"], 0.0).float(),
             u=torch.rand(rows, generator=g, **f32))
    if own:
        s.update(token=torch.empty(rows, **i32), logprob=torch.empty(rows, **f32), kept=torch.empty(rows, **i32))
    return s


# ------------------------------------------------------------------------------------------------------- plain forms
def _plain_append(s):
    c = s["case"]
    half = c["d"] // 2
    pos = s["pos"][s["axis"].long()].T.double()                       # [T][d/2]
    angle = pos * s["inv"].double()
    cs, sn = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turned(x, w):
        x = x.float()
        if c["norm"]:
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + 1e-6) * w
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * cs - b * sn, a * sn + b * cs], dim=-1).to(s["K"].dtype)

    live = s["slots"] >= 0
    page, at = s["slots"][live] // PAGE, s["slots"][live] % PAGE
    s["K"][page, :, at] = turned(s["k"], s["wk"])[live]
    s["V"][page, :, at] = s["v"][live]
    return turned(s["q"], s["wq"]), s["K"], s["V"]


def _plain_shared(s):
    c = s["case"]
    hkv, G, d = c["hkv"], c["G"], c["d"]
    outs, lses, t0 = [], [], 0
    for r in range(c["R"]):
        n, start = s["windows"][r], s["starts"][r]
        ids = s["bt"][r, :(start + n + PAGE - 1) // PAGE].long()
        k = s["K"][ids].float().transpose(0, 1).reshape(hkv, 1, -1, d)      # [hkv][1][tokens][d]
        v = s["V"][ids].float().transpose(0, 1).reshape(hkv, 1, -1, d)
        q = s["q"][t0:t0 + n].float().view(n, hkv, G, d).permute(1, 2, 0, 3)    # [hkv][G][n][d]
        x = (q @ k.transpose(-1, -2)) / math.sqrt(d)
        see = torch.arange(k.shape[2], device="cuda") <= start + torch.arange(n, device="cuda")[:, None]
        x = x.masked_fill(~see, float("-inf"))
        m = x.amax(dim=-1, keepdim=True)
        p = torch.exp(x - m)
        z = p.sum(dim=-1, keepdim=True)
        outs.append(((p @ v) / z).permute(2, 0, 1, 3).reshape(n, hkv * G, d))
        lses.append((m + torch.log(z))[..., 0].permute(2, 0, 1).reshape(n, hkv * G))
        t0 += n
    return torch.cat(outs).to(s["K"].dtype), torch.cat(lses)


def _plain_sample(s):
    V = s["case"]["vocab"]
    tokens, logprobs, kepts = [], [], []
    for a in range(0, s["logits"].shape[0], 256):
        e = a + 256
        x = s["logits"][a:e].double() + 0.0
        temp, k = s["temp"][a:e, None].double(), s["top_k"][a:e, None]
        xs, order = torch.sort(x, dim=-1, descending=True, stable=True)
        w = torch.exp((xs - xs[:, :1]) / torch.where(temp > 0, temp, 1.0))
        rank = torch.arange(V, device="cuda")
        k = torch.where((k > 0) & (k < V), k, V)
        k = torch.where(temp > 0, k, 1)
        keep = (rank < k) & (w >= s["min_p"][a:e, None].double()) & ~torch.isinf(xs)
        w = torch.where(keep, w, 0.0)
        before = torch.cumsum(w, dim=-1) - w
        p = s["top_p"][a:e, None].double()
        keep = keep & ((before < p * w.sum(dim=-1, keepdim=True)) | (p >= 1.0) | (rank == 0))
        w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))     # in id order
        c = torch.cumsum(w, dim=-1)
        t = ((c > s["u"][a:e, None].double() * c[:, -1:]) & (w > 0)).to(torch.int8).argmax(dim=-1)
        tokens.append(t.to(torch.int32))
        logprobs.append(torch.log(w.gather(1, t[:, None]) / c[:, -1:])[:, 0].float())
        kepts.append(keep.sum(dim=-1).to(torch.int32))
    return torch.cat(tokens), torch.cat(logprobs), torch.cat(kepts)


# ----------------------------------------------------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if not own:
        return {"append": _plain_append, "shared": _plain_shared, "sample": _plain_sample}[s["op"]](s)
    kap = _kap()
    if s["op"] == "append":
        norm = dict(q_weight=s["wq"], k_weight=s["wk"], eps=1e-6) if c["norm"] else {}
        kap.kap_append_kv_norm(s["pool"], s["k"], s["v"], s["q"], s["q_out"], s["pos"], s["slots"], s["inv"],
                               freq_axis=s["axis"] if c["axes"] > 1 else None, **norm)
        return s["q_out"], s["K"], s["V"]
    if s["op"] == "shared":
        kap.kap_attn_verify_shared(s["pool"], s["map"], s["policy"], s["groups"], s["q"], s["out"], s["lse"], s["ws"])
        return s["out"], s["lse"]
    kap.kap_sample_tokens(s["logits"], s["u"], s["token"], temperature=s["temp"], top_k=s["top_k"], top_p=s["top_p"],
                          min_p=s["min_p"], logprob=s["logprob"], kept=s["kept"])
    return s["token"], s["logprob"], s["kept"]


# --------------------------------------------------------------------------------------------------------- in 64 bits
def _exact_rotated(rows, weight, pos, axis, inv, norm):
    """One token's rows [heads][d] after norm and rotation, as complex numbers: a pair (i, i + d/2) is one of them."""
    x = rows.double()
    half = x.shape[-1] // 2
    if norm:
        x = weight.double() * x / torch.sqrt(x.square().sum(dim=-1, keepdim=True) / (2 * half) + 1e-6)
    z = torch.complex(x[..., :half], x[..., half:])
    phase = pos.double().gather(-1, axis.expand(pos.shape[0], half)) * inv.double()
    z = z * torch.polar(torch.ones_like(phase), phase)[:, None, :]
    return torch.cat([z.real, z.imag], dim=-1)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "append":
        axis = s["axis"].long()[None]
        args = (s["pos"].T.contiguous(), axis, s["inv"], c["norm"])
        q = _exact_rotated(s["q"], s["wq"], *args)
        k = _exact_rotated(s["k"], s["wk"], *args)
        P, hkv, d = s["K"].shape[0], c["hkv"], c["d"]
        K = torch.zeros(P * PAGE + 1, hkv, d, dtype=torch.float64, device="cuda")
        Vv = torch.zeros_like(K)
        to = torch.where(s["slots"] < 0, P * PAGE, s["slots"])   # skipped tokens fall into a row that is cut off
        K[to], Vv[to] = k, s["v"].double()
        return q, *(x[:-1].view(P, PAGE, hkv, d).transpose(1, 2).contiguous() for x in (K, Vv))
    if c["op"] == "shared":
        tq, hq, d, G = sum(s["windows"]), c["hkv"] * c["G"], c["d"], c["G"]
        out = torch.empty(tq, hq, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(tq, hq, dtype=torch.float64, device="cuda")
        row = 0
        for r in range(c["R"]):
            for i in range(s["windows"][r]):
                n = s["starts"][r] + i + 1          # every token this row sees, and none after it
                ids = s["bt"][r, :(n + PAGE - 1) // PAGE].long()
                for h in range(c["hkv"]):
                    k = s["K"][ids, h].double().view(-1, d)[:n]
                    x = (s["q"][row, h * G:h * G + G].double() @ k.T) / math.sqrt(d)
                    l = torch.logsumexp(x, dim=1)
                    lse[row, h * G:h * G + G] = l
                    out[row, h * G:h * G + G] = torch.exp(x - l[:, None]) @ s["V"][ids, h].double().view(-1, d)[:n]
                row += 1
        return out, lse
    tok, lp, kept = [], [], []
    for r in range(c["rows"]):
        x = s["logits"][r].double()
        best = x.max()
        T, k, u = float(s["temp"][r]), int(s["top_k"][r]), float(s["u"][r])
        if not T > 0:
            tok.append(torch.argmax(x))
            lp.append(x.new_zeros(()))
            kept.append(torch.ones((), dtype=torch.long, device="cuda"))
            continue
        ids = torch.nonzero(x > float("-inf"))[:, 0]               # ascending, as every list below
        w = torch.exp((x[ids] - best) / T)
        heavy = w >= float(s["min_p"][r])
        ids, w = ids[heavy], w[heavy]
        if 0 < k < len(ids):
            first = torch.argsort(x[ids], descending=True, stable=True)[:k]
            first = torch.sort(first).values
            ids, w = ids[first], w[first]
        if float(s["top_p"][r]) < 1.0:
            down = torch.argsort(x[ids], descending=True, stable=True)
            sums = torch.cumsum(w[down], dim=0)
            n = torch.searchsorted(sums, float(s["top_p"][r]) * sums[-1:]) + 1
            run_ = torch.sort(down[:int(n)]).values
            ids, w = ids[run_], w[run_]
        sums = torch.cumsum(w, dim=0)
        j = int(torch.searchsorted(sums, u * sums[-1:], right=True).clamp(max=len(ids) - 1))
        tok.append(ids[j])
        lp.append(torch.log(w[j]) - torch.log(sums[-1]))
        kept.append(torch.full((), len(ids), device="cuda"))
    return torch.stack(tok).to(torch.int32), torch.stack(lp), torch.stack(kept).to(torch.int32)
