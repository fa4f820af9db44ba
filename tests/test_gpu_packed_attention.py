"""Attention over a pool with packed pages (proposal over a view, windows over the whole table) against 64 bits."""
import numpy as np
import pytest
import torch

from tests.packed_reference import PAGE, attend, chunk_values, random_chunks, tolerances

pytestmark = pytest.mark.gpu


class Cache:
    """Requests of the given token counts on pages of both kinds: page kinds by `kinds(r, j)` ('4' or '16'). Rows of no
    request hold NaN, in 16-bit pages and in the parameters of packed ones."""

    def __init__(self, kap, lens, hkv, G, d, kinds, seed=0, spare=2):
        self.kap, self.lens, self.hkv, self.G, self.d = kap, lens, hkv, G, d
        g = torch.Generator().manual_seed(seed)
        self.g = g
        npg = [(n + PAGE - 1) // PAGE for n in lens]
        kind = [[kinds(r, j) for j in range(n)] for r, n in enumerate(npg)]
        n4 = sum(k == "4" for row in kind for k in row)
        n16 = sum(k == "16" for row in kind for k in row)
        self.P16, self.P4 = n16 + spare, n4 + spare
        K = torch.randn(self.P16, hkv, PAGE, d, generator=g)
        V = torch.randn(self.P16, hkv, PAGE, d, generator=g)
        self.K, self.V = K.to(torch.bfloat16), V.to(torch.bfloat16)
        self.packed = random_chunks(self.P4, hkv, d, g)
        i16, i4 = iter(torch.randperm(self.P16, generator=g).tolist()), iter(torch.randperm(self.P4, generator=g).tolist())
        self.mp = max(1, max(npg)) + 1
        self.bt = torch.full((len(lens), self.mp), -1, dtype=torch.int32)
        nb = d // 64
        par = self.packed[:, :, 2 * nb * 512:].view(torch.bfloat16).view(self.P4, hkv, 2, nb, PAGE, 2)
        for r, n in enumerate(lens):
            for j, k in enumerate(kind[r]):
                pid = next(i16) if k == "16" else next(i4)
                used = min(PAGE, n - j * PAGE)
                if k == "16":
                    self.K[pid, :, used:] = float("nan")
                    self.V[pid, :, used:] = float("nan")
                else:
                    par[pid, :, :, :, used:] = float("nan")
                self.bt[r, j] = pid if k == "16" else self.P16 + pid
        for pid in i16:   # pages of no request
            self.K[pid] = float("nan")
            self.V[pid] = float("nan")
        dev = "cuda"
        self.pool = kap.PackedPool(kap.KVPool(self.K.to(dev), self.V.to(dev), hkv * G), self.packed.to(dev))
        self.vals = {}

    def page(self, pid, h):
        """Rows of a page for attend(): [(k, v, scale * code of v, |k| bound, |v| bound)] x 16."""
        if (pid, h) not in self.vals:
            d = self.d
            if pid < self.P16:
                k, v = self.K[pid, h].double().numpy(), self.V[pid, h].double().numpy()
                self.vals[pid, h] = [(k[t], v[t], np.zeros(d), np.abs(k[t]), np.abs(v[t])) for t in range(PAGE)]
            else:
                val, sc, lo = chunk_values(self.packed[pid - self.P16, h].numpy(), d)
                self.vals[pid, h] = [(val[0, t], val[1, t], sc[1, t], sc[0, t] + lo[0, t], sc[1, t] + lo[1, t])
                                     for t in range(PAGE)]
        return self.vals[pid, h]

    def query(self, rows, scale=1.0):
        return (scale * torch.randn(rows, self.hkv * self.G, self.d, generator=self.g)).to(torch.bfloat16)

    def check(self, out, lse, q, row, head, tokens):
        d = self.d
        o, l, pv, pvc, s = attend(q[row, head].double().numpy(), tokens, d)
        got, gl = out[row, head].double().cpu().numpy(), float(lse[row, head])
        if not tokens:
            assert (got == 0).all() and gl == -np.inf, (row, head)
            return
        to, tl = tolerances(d, len(tokens), l, pv, pvc, s)
        assert np.isfinite(got).all(), (row, head)
        over = np.abs(got - o) - (to + 2.0 ** -8 * np.abs(o))
        assert over.max() <= 0, (row, head, over.max(), np.abs(got - o).max())
        assert abs(gl - l) <= tl, (row, head, gl, l, tl)


KINDS = {
    "packed": lambda r, j: "4",
    "tail16": lambda r, j: "4" if j < 3 else "16",
    "sixteen": lambda r, j: "16",
    "mixed": lambda r, j: "4" if (j * 7 + r * 3) % 5 < 3 else "16",
}

VERIFY = [
    # lens (tokens with the window), windows, hkv, G, d, kinds
    ([1], [1], 1, 1, 64, "packed"),
    ([1, 2, 16, 17], [1, 2, 1, 3], 2, 4, 128, "packed"),
    ([1, 2, 16, 17], [1, 2, 1, 3], 2, 4, 128, "sixteen"),
    ([15, 16, 33, 300], [1, 1, 1, 1], 2, 8, 128, "mixed"),
    ([200, 31], [4, 8], 2, 4, 64, "tail16"),
    ([500, 64, 65], [5, 1, 12], 1, 5, 128, "mixed"),
    ([130, 250], [21, 8], 1, 3, 64, "mixed"),
    ([260], [64], 2, 1, 128, "mixed"),
    ([700], [8], 1, 8, 128, "packed"),
    ([90, 0, 40], [3, 0, 2], 2, 7, 128, "mixed"),     # a request without a window
    ([1000, 33], [16, 1], 8, 2, 64, "mixed"),
    ([4000], [2], 2, 6, 128, "tail16"),
]


@pytest.mark.parametrize("case", VERIFY, ids=lambda c: f"{'_'.join(map(str, c[0]))}-q{max(c[1])}-h{c[2]}x{c[3]}-d{c[4]}-{c[5]}")
def test_windows_over_the_whole_table(kap, case):
    lens, win, hkv, G, d, kinds = case
    c = Cache(kap, lens, hkv, G, d, KINDS[kinds], seed=len(lens) + hkv)
    dev = "cuda"
    q = c.query(sum(win))
    off = torch.tensor([0] + list(np.cumsum(win)), dtype=torch.int32)
    start = torch.tensor([n - w for n, w in zip(lens, win)], dtype=torch.int32)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    pmap = kap.PageMap(c.bt.to(dev), ln, ln)
    vp = kap.VerifyPolicy(off.to(dev), start.to(dev), max(win), sum(win))
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=dev)
    lse = torch.full(q.shape[:2], float("nan"), device=dev)
    ws = kap.workspace(kap.kap_packed_workspace_size(len(lens), hkv, hkv * G, d, max(win)), dev)
    for _ in range(2):   # the counters are left at zero
        out.fill_(float("nan"))
        kap.kap_attn_verify_packed(c.pool, pmap, vp, q.to(dev), out, lse, ws)
        assert kap.kap_device_error() == 0
    for r, (n, w) in enumerate(zip(lens, win)):
        for i in range(w):
            for head in range(0, hkv * G, max(1, hkv * G // 5)):
                h = head // G
                toks = [c.page(int(c.bt[r, t // PAGE]), h)[t % PAGE] for t in range(n - w + i + 1)]
                c.check(out, lse, q, int(off[r]) + i, head, toks)


PROPOSE = [
    # prompt lengths, generated, pages selected, hkv, G, d, shared, kinds
    ([1], 1, 1, 1, 1, 64, False, "packed"),
    ([33, 16, 200], 2, 3, 2, 4, 128, False, "tail16"),
    ([33, 16, 200], 19, 5, 2, 4, 128, True, "mixed"),
    ([400, 70], 1, 20, 2, 5, 64, False, "mixed"),
    ([1000], 3, 60, 8, 1, 128, False, "packed"),
    ([300, 8, 90, 31], 40, 4, 1, 8, 128, True, "mixed"),
    ([128], 1, 8, 4, 3, 128, False, "sixteen"),
    ([2000], 5, 100, 1, 7, 64, True, "mixed"),
]


@pytest.mark.parametrize("case", PROPOSE, ids=lambda c: f"{'_'.join(map(str, c[0]))}-g{c[1]}-s{c[2]}-h{c[3]}x{c[4]}-d{c[5]}-{c[6]}-{c[7]}")
def test_proposal_over_a_view(kap, case):
    ctx, gen, nsel, hkv, G, d, shared, kinds = case
    lens = [n + gen for n in ctx]
    c = Cache(kap, lens, hkv, G, d, KINDS[kinds], seed=gen)
    dev = "cuda"
    rows = 1 if shared else hkv
    R = len(ctx)
    cap = nsel + (gen + PAGE - 1) // PAGE + 2
    i32 = dict(dtype=torch.int32)
    vbt, lp = torch.zeros(R, rows, cap, **i32), torch.zeros(R, rows, cap, **i32)
    nent, ns = torch.zeros(R, rows, **i32), torch.zeros(R, rows, **i32)
    ent = {}
    for r, n in enumerate(ctx):
        N = (n + PAGE - 1) // PAGE
        for v in range(rows):
            sel = sorted(torch.randperm(N, generator=c.g)[:nsel].tolist())
            tail = [j for j in range(n // PAGE, (lens[r] + PAGE - 1) // PAGE) if j not in sel]
            pages = sel + tail
            ent[r, v] = [(j, i < len(sel)) for i, j in enumerate(pages)]
            lp[r, v, :len(pages)] = torch.tensor(pages, **i32)
            vbt[r, v, :len(pages)] = c.bt[r, pages]
            vbt[r, v, len(pages):] = 1 << 28     # never read
            nent[r, v], ns[r, v] = len(pages), len(sel)
    q = c.query(R, scale=0.7)
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device=dev)
    lse = torch.full(q.shape[:2], float("nan"), device=dev)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    pmap = kap.PageMap(c.bt.to(dev), t(ctx), t(lens))
    view = kap.View(rows, cap, vbt.to(dev), lp.to(dev), nent.to(dev), ns.to(dev))
    ws = kap.workspace(kap.kap_packed_workspace_size(R, hkv, hkv * G, d), dev)
    for _ in range(2):
        out.fill_(float("nan"))
        kap.kap_attn_propose_packed(c.pool, pmap, view, q.to(dev), out, lse, ws)
        assert kap.kap_device_error() == 0
    for r in range(R):
        for head in range(0, hkv * G, max(1, hkv * G // 6)):
            h = head // G
            toks = [c.page(int(c.bt[r, j]), h)[o] for j, chosen in ent[r, 0 if shared else h] for o in range(PAGE)
                    if j * PAGE + o < lens[r] and (chosen or j * PAGE + o >= ctx[r])]
            c.check(out, lse, q, r, head, toks)


SHARED_OUT = [
    # tables wider than a CTA's own rows: lens, windows, hkv, G, d, kinds, width of the table
    ([2600, 2100, 40], [8, 3, 1], 1, 8, 128, "mixed", 170),
    ([2300], [8], 2, 5, 128, "tail16", 170),
    ([2300, 700], [8, 6], 1, 6, 128, "mixed", 170),
    ([2200], [8], 1, 3, 128, "mixed", 140),
    ([2200, 9], [4, 4], 2, 8, 128, "packed", 140),
    ([2100, 2500], [8, 16], 1, 3, 64, "mixed", 160),
    ([2500], [16], 1, 4, 64, "mixed", 160),
    ([1 + (37 * r) % 60 for r in range(300)], [1] * 300, 1, 2, 64, "mixed", 131),     # more requests than threads
    ([2 + (41 * r) % 50 for r in range(270)], [r % 3 for r in range(270)], 2, 4, 128, "mixed", 131),
]


@pytest.mark.parametrize("case", SHARED_OUT, ids=lambda c: f"R{len(c[0])}-{max(c[0])}-q{max(c[1])}-h{c[2]}x{c[3]}-d{c[4]}-{c[5]}")
def test_rows_shared_out_over_ctas(kap, case):
    lens, win, hkv, G, d, kinds, width = case
    c = Cache(kap, lens, hkv, G, d, KINDS[kinds], seed=len(lens) + G)
    dev, R = "cuda", len(lens)
    bt = torch.full((R, width), -1, dtype=torch.int32)
    bt[:, :min(width, c.mp)] = c.bt[:, :width]
    q = c.query(sum(win) + 3)
    off = torch.tensor([0] + list(np.cumsum(win)), dtype=torch.int32)
    start = torch.tensor([n - w for n, w in zip(lens, win)], dtype=torch.int32)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    vp = kap.VerifyPolicy(off.to(dev), start.to(dev), max(win), sum(win) + 3)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full(q.shape[:2], 7.0, device=dev)
    ws = kap.workspace(kap.kap_packed_workspace_size(R, hkv, hkv * G, d, max(win)), dev)
    for _ in range(2):
        kap.kap_attn_verify_packed(c.pool, kap.PageMap(bt.to(dev), ln, ln), vp, q.to(dev), out, lse, ws)
        assert kap.kap_device_error() == 0
    assert (out[sum(win):] == 7.0).all() and (lse[sum(win):] == 7.0).all()   # rows behind the last window stay
    for r in range(0, R, max(1, R // 12)):
        for i in sorted({0, win[r] - 1} if win[r] else set()):
            for head in sorted({0, hkv * G - 1}):
                toks = [c.page(int(c.bt[r, t // PAGE]), head // G)[t % PAGE] for t in range(lens[r] - win[r] + i + 1)]
                c.check(out, lse, q, int(off[r]) + i, head, toks)


def test_views_shared_out_over_ctas(kap):
    """More view rows than threads, in a view wider than a CTA's own rows; some hold nothing."""
    hkv, G, d, R, cap = 2, 3, 128, 150, 140
    lens = [(29 * r) % 90 for r in range(R)]
    c = Cache(kap, lens, hkv, G, d, KINDS["mixed"], seed=8)
    dev = "cuda"
    i32 = dict(dtype=torch.int32)
    vbt, lp = torch.zeros(R, hkv, cap, **i32), torch.zeros(R, hkv, cap, **i32)
    n = torch.tensor([[(x + PAGE - 1) // PAGE] * hkv for x in lens], **i32)
    for r in range(R):
        k = int(n[r, 0])
        vbt[r, :, :k] = c.bt[r, :k]
        lp[r, :, :k] = torch.arange(k, **i32)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    q = c.query(R)
    out, lse = torch.empty(q.shape, dtype=torch.bfloat16, device=dev), torch.empty(q.shape[:2], device=dev)
    ws = kap.workspace(kap.kap_packed_workspace_size(R, hkv, hkv * G, d), dev)
    kap.kap_attn_propose_packed(c.pool, kap.PageMap(c.bt.to(dev), t(lens), t(lens)),
                                kap.View(hkv, cap, vbt.to(dev), lp.to(dev), n.to(dev), n.to(dev)), q.to(dev), out, lse, ws)
    assert kap.kap_device_error() == 4   # the rows that hold nothing
    for r in list(range(0, R, 13)) + [r for r in range(R) if lens[r] == 0]:
        for head in (0, 5):
            c.check(out, lse, q, r, head, [c.page(int(c.bt[r, x // PAGE]), head // G)[x % PAGE] for x in range(lens[r])])


def test_value_scales_far_apart(kap):
    """Tokens with a value scale 2^13 of the others' and nearly all of the weight, after and before large ones."""
    dev = "cuda"
    for order in (0, 1):
        n = 320
        c = Cache(kap, [n], 1, 2, 128, KINDS["packed"], seed=11)
        q = c.query(1)
        heavy = [3, 4] if order else [15, 16]
        for j in range(n // PAGE):
            pid = int(c.bt[0, j]) - c.P16
            par = c.packed[pid, 0, 2048:].view(torch.bfloat16).view(2, 2, PAGE, 2)
            if j in heavy:
                par[1] *= 2.0 ** -13
                par[0, :, :, 0] *= 0.0                  # keys along the query: all codes stand for the lowest value
                par[0, :, :, 1] = 2.0 * q[0, 0].float().sign().view(2, 64)[:, :1].to(torch.bfloat16)
        c.pool = kap.PackedPool(kap.KVPool(c.K.to(dev), c.V.to(dev), 2), c.packed.to(dev))
        t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        out, lse = torch.empty(1, 2, 128, dtype=torch.bfloat16, device=dev), torch.empty(1, 2, device=dev)
        ws = kap.workspace(kap.kap_packed_workspace_size(1, 1, 2, 128, 1), dev)
        kap.kap_attn_verify_packed(c.pool, kap.PageMap(c.bt.to(dev), t([n]), t([n])),
                                   kap.VerifyPolicy(t([0, 1]), t([n - 1]), 1, 1), q.to(dev), out, lse, ws)
        for head in range(2):
            c.check(out, lse, q, 0, head, [c.page(int(c.bt[0, i // PAGE]), 0)[i % PAGE] for i in range(n)])


def test_large_and_small_magnitudes(kap):
    """Keys, values and queries far from 1: sums stay in range and keep their bits."""
    dev = "cuda"
    for qs, ks, vs in ((2.0 ** 12, 2.0 ** -12, 2.0 ** 20), (2.0 ** -30, 2.0 ** 30, 2.0 ** -20), (0.0, 1.0, 1.0),
                       (2.0 ** 60, 2.0 ** -60, 2.0 ** 60)):
        c = Cache(kap, [400], 1, 4, 128, KINDS["mixed"], seed=5)
        c.K, c.V = c.K * ks, c.V * vs
        par = c.packed[:, :, 2048:].view(torch.bfloat16).view(c.P4, 1, 2, 2, PAGE, 2)
        par[:, :, 0] *= ks
        par[:, :, 1] *= vs
        c.pool = kap.PackedPool(kap.KVPool(c.K.to(dev), c.V.to(dev), 4), c.packed.to(dev))
        q = (c.query(1).float() * qs).to(torch.bfloat16)
        t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        out, lse = torch.empty(1, 4, 128, dtype=torch.bfloat16, device=dev), torch.empty(1, 4, device=dev)
        ws = kap.workspace(kap.kap_packed_workspace_size(1, 1, 4, 128, 1), dev)
        kap.kap_attn_verify_packed(c.pool, kap.PageMap(c.bt.to(dev), t([400]), t([400])),
                                   kap.VerifyPolicy(t([0, 1]), t([399]), 1, 1), q.to(dev), out, lse, ws)
        for head in range(4):
            c.check(out, lse, q, 0, head, [c.page(int(c.bt[0, i // PAGE]), 0)[i % PAGE] for i in range(400)])


def test_growing_logits(kap):
    """Logits that rise page by page over hundreds: the running maximum is renewed again and again."""
    dev = "cuda"
    n = 640
    c = Cache(kap, [n], 1, 2, 64, KINDS["mixed"], seed=9)
    for j in range(n // PAGE):
        pid = int(c.bt[0, j])
        if pid < c.P16:
            c.K[pid] *= 0.5 * j
        else:
            c.packed[pid - c.P16, :, 1024:].view(torch.bfloat16).view(1, 2, 1, PAGE, 2)[:, 0] *= 0.5 * j
    c.pool = kap.PackedPool(kap.KVPool(c.K.to(dev), c.V.to(dev), 2), c.packed.to(dev))
    q = c.query(1)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    out, lse = torch.empty(1, 2, 64, dtype=torch.bfloat16, device=dev), torch.empty(1, 2, device=dev)
    ws = kap.workspace(kap.kap_packed_workspace_size(1, 1, 2, 64, 1), dev)
    kap.kap_attn_verify_packed(c.pool, kap.PageMap(c.bt.to(dev), t([n]), t([n])),
                               kap.VerifyPolicy(t([0, 1]), t([n - 1]), 1, 1), q.to(dev), out, lse, ws)
    for head in range(2):
        c.check(out, lse, q, 0, head, [c.page(int(c.bt[0, i // PAGE]), 0)[i % PAGE] for i in range(n)])


def test_empty_rows_and_bad_pages(kap):
    dev = "cuda"
    c = Cache(kap, [40, 40], 2, 2, 64, KINDS["mixed"], seed=2)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    q = c.query(2)
    out, lse = torch.empty(2, 4, 64, dtype=torch.bfloat16, device=dev), torch.empty(2, 4, device=dev)
    ws = kap.workspace(kap.kap_packed_workspace_size(2, 2, 4, 64), dev)
    # request 0 holds nothing, request 1 sees its 40 tokens
    view = kap.View(1, 4, torch.zeros(2, 1, 4, dtype=torch.int32, device=dev),
                    torch.zeros(2, 1, 4, dtype=torch.int32, device=dev), t([[0], [3]]), t([[0], [3]]))
    view.block_table[1, 0, :3] = c.bt[1, :3].to(dev)
    view.logical_page[1, 0, :3] = t([0, 1, 2])
    kap.kap_attn_propose_packed(c.pool, kap.PageMap(c.bt.to(dev), t([0, 40]), t([0, 40])), view, q.to(dev), out, lse, ws)
    assert kap.kap_device_error() == 4
    for head in range(4):
        c.check(out, lse, q, 0, head, [])
        c.check(out, lse, q, 1, head, [c.page(int(c.bt[1, i // PAGE]), head // 2)[i % PAGE] for i in range(40)])
    # a view entry past both pools, one below zero: skipped, error bit 1, the rest is as without them
    bt = c.bt.clone()
    bt[0, 1], bt[1, 0] = c.P16 + c.P4, -7
    vp = kap.VerifyPolicy(t([0, 1, 2]), t([39, 39]), 1, 2)
    kap.kap_attn_verify_packed(c.pool, kap.PageMap(bt.to(dev), t([40, 40]), t([40, 40])), vp, q.to(dev), out, lse, ws)
    assert kap.kap_device_error() == 1
    for r, skip in ((0, 1), (1, 0)):
        for head in range(4):
            c.check(out, lse, q, r, head, [c.page(int(c.bt[r, i // PAGE]), head // 2)[i % PAGE] for i in range(40)
                                           if i // PAGE != skip])
    # a table shorter than the positions: what it holds is read
    bt = c.bt[:, :2].contiguous()
    kap.kap_attn_verify_packed(c.pool, kap.PageMap(bt.to(dev), t([40, 40]), t([40, 40])), vp, q.to(dev), out, lse, ws)
    assert kap.kap_device_error() == 1
    c.check(out, lse, q, 0, 0, [c.page(int(c.bt[0, i // PAGE]), 0)[i % PAGE] for i in range(32)])


def test_nan_parameters_of_visible_tokens_show(kap):
    dev = "cuda"
    c = Cache(kap, [64], 1, 2, 64, KINDS["packed"], seed=2)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    pid = int(c.bt[0, 1]) - c.P16
    c.pool.packed[pid, 0, 1024 + 64 + 4 * 3:1024 + 64 + 4 * 3 + 4] = 0xFF   # value parameters of token 3 of page 1
    q = c.query(1)
    out, lse = torch.empty(1, 2, 64, dtype=torch.bfloat16, device=dev), torch.empty(1, 2, device=dev)
    ws = kap.workspace(kap.kap_packed_workspace_size(1, 1, 2, 64), dev)
    kap.kap_attn_verify_packed(c.pool, kap.PageMap(c.bt.to(dev), t([64]), t([64])),
                               kap.VerifyPolicy(t([0, 1]), t([63]), 1, 1), q.to(dev), out, lse, ws)
    assert torch.isnan(out).all() and torch.isfinite(lse).all()


def test_graphs_and_streams(kap):
    """The same numbers from a captured graph replayed on new inputs, and from two streams at once."""
    dev = "cuda"
    c = Cache(kap, [3000, 700], 2, 4, 128, KINDS["mixed"], seed=4)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    pmap = kap.PageMap(c.bt.to(dev), t([3000, 700]), t([3000, 700]))
    vp = kap.VerifyPolicy(t([0, 3, 4]), t([2997, 699]), 3, 4)
    q1, q2 = c.query(4).to(dev), c.query(4).to(dev)
    size = kap.kap_packed_workspace_size(2, 2, 8, 128, 3)
    new = lambda: (torch.empty(4, 8, 128, dtype=torch.bfloat16, device=dev), torch.empty(4, 8, device=dev),  # noqa: E731
                   kap.workspace(size, dev))
    eager = []
    for q in (q1, q2):
        o, l, ws = new()
        kap.kap_attn_verify_packed(c.pool, pmap, vp, q, o, l, ws)
        eager.append((o, l))
    torch.cuda.synchronize()
    o, l, ws = new()
    q = q1.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kap.kap_attn_verify_packed(c.pool, pmap, vp, q, o, l, ws)
        kap.kap_attn_verify_packed(c.pool, pmap, vp, q, o, l, ws)
    for x, ref in ((q2, eager[1]), (q1, eager[0]), (q2, eager[1])):
        q.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ref[0]) and torch.equal(l, ref[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    res = [new() for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x, (o, l, ws) in zip(streams, (q1, q2), res):
            kap.kap_attn_verify_packed(c.pool, pmap, vp, x, o, l, ws, stream=s)
    torch.cuda.synchronize()
    for (o, l, _), ref in zip(res, eager):
        assert torch.equal(o, ref[0]) and torch.equal(l, ref[1])


def test_binding_refusals(kap):
    dev = "cuda"
    c = Cache(kap, [64], 1, 2, 64, KINDS["packed"], seed=2)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    pmap = kap.PageMap(c.bt.to(dev), t([64]), t([64]))
    vp = kap.VerifyPolicy(t([0, 1]), t([63]), 1, 1)
    q = c.query(1).to(dev)
    out, lse = torch.empty_like(q), torch.empty(1, 2, device=dev)
    ws = kap.workspace(kap.kap_packed_workspace_size(1, 1, 2, 64), dev)
    call = lambda q=q, out=out, lse=lse, ws=ws, vp=vp: kap.kap_attn_verify_packed(c.pool, pmap, vp, q, out, lse, ws)  # noqa: E731
    call()
    for bad in (dict(q=q.float()), dict(lse=lse.double())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(q=q[:, :1].contiguous()), dict(out=out.cpu()), dict(lse=lse[:, :1]),
                dict(vp=kap.VerifyPolicy(t([0, 1, 1]), t([63]), 1, 1))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(kap.KapError) as e:
        call(ws=ws[:16])
    assert e.value.status == -3
    with pytest.raises(kap.KapError) as e:   # G * max_q = 66
        call(vp=kap.VerifyPolicy(t([0, 1]), t([63]), 33, 1))
    assert e.value.status == -5
