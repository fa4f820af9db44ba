"""One workspace, sized for the largest call and zero-filled once, taken by calls of other sizes in turn: the bits are
those of a workspace of the call's own."""
import pytest
import torch

from tests.test_gpu_packed_attention import KINDS, Cache

pytestmark = pytest.mark.gpu


class Windows:
    """Verify windows of w rows over R requests of n tokens."""

    def __init__(self, kap, R, n, w, hkv, G, d, seed):
        dev = "cuda"
        t = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        c = Cache(kap, [n - 5 * r % 40 for r in range(R)], hkv, G, d, KINDS["mixed"], seed=seed)
        self.kap, self.pool = kap, c.pool
        self.pmap = kap.PageMap(c.bt.to(dev), t(c.lens), t(c.lens))
        self.vp = kap.VerifyPolicy(t([w * r for r in range(R + 1)]), t([x - w for x in c.lens]), w, R * w)
        self.q = c.query(R * w).to(dev)
        self.size = kap.kap_packed_workspace_size(R, hkv, hkv * G, d, w)

    def run(self, ws):
        out = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:2], float("nan"), device="cuda")
        self.kap.kap_attn_verify_packed(self.pool, self.pmap, self.vp, self.q, out, lse, ws)
        return out, lse


class Logprobs:
    def __init__(self, kap, rows, V, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        self.kap, self.rows = kap, rows
        self.x = torch.randn(rows, V, generator=g).to(dtype).cuda()
        self.tok = torch.randint(V, (rows,), generator=g, dtype=torch.int32).cuda()
        self.size = kap.kap_logprobs_workspace_size(rows, V)

    def run(self, ws):
        lp, ent = torch.full((self.rows,), float("nan"), device="cuda"), torch.full((self.rows,), float("nan"), device="cuda")
        rank = torch.full((self.rows,), -7, dtype=torch.int32, device="cuda")
        ids, tlp = torch.full((self.rows, 5), -7, dtype=torch.int32, device="cuda"), torch.full((self.rows, 5), 7.0, device="cuda")
        self.kap.kap_token_logprobs(self.x, self.tok, lp, ws, entropy=ent, rank=rank, top_ids=ids, top_logprobs=tlp)
        return lp, ent, rank, ids, tlp


def in_turn(kap, calls, order):
    fresh = [c.run(kap.workspace(c.size, "cuda")) for c in calls]
    ws = kap.workspace(max(c.size for c in calls), "cuda")
    got = [(i, calls[i].run(ws)) for i in order]
    torch.cuda.synchronize()
    assert kap.kap_device_error() == 0
    for n, (i, tensors) in enumerate(got):
        for a, b in zip(tensors, fresh[i]):
            assert not a.isnan().any() and torch.equal(a, b), (n, i)


@pytest.mark.parametrize("order", [(0, 1, 2, 3), (3, 2, 1, 0), (0, 2, 0, 1, 3, 1)])
def test_attention_calls_of_several_sizes(kap, order):
    # tables of more than 128 pages, so that rows are shared out over CTAs
    calls = [Windows(kap, 1, 6000, 1, 8, 4, 64, 1), Windows(kap, 24, 2600, 1, 8, 4, 64, 2),
             Windows(kap, 2, 3000, 8, 2, 4, 128, 3), Windows(kap, 11, 2300, 2, 8, 2, 128, 4)]
    in_turn(kap, calls, order)


@pytest.mark.parametrize("order", [(0, 1, 2, 3), (3, 2, 1, 0), (0, 2, 0, 1, 3, 1)])
def test_logprob_calls_of_several_sizes(kap, order):
    # fewer than 512 rows: a row is shared out over CTAs
    calls = [Logprobs(kap, 4, 128256, torch.float32, 1), Logprobs(kap, 130, 50257, torch.bfloat16, 2),
             Logprobs(kap, 511, 32000, torch.bfloat16, 3), Logprobs(kap, 600, 4096, torch.float32, 4)]
    in_turn(kap, calls, order)
