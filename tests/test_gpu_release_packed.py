"""Pages of both kinds given back: 16-bit ids to one stack, packed ids to another, in request and then page order; and a
server's step with them, until the freed pages hold other requests."""
import numpy as np
import pytest
import torch

from tests.packed_reference import PAGE, chunk_values
from tests.test_gpu_packed_flow import Server, _close

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def plain(bt, seq, gone, P16, P4, s16, n16, s4, n4):
    s16, s4, out, err = s16.copy(), s4.copy(), seq.copy(), 0
    for r in range(len(seq)):
        if not gone[r]:
            continue
        for j in range(-(-int(seq[r]) // PAGE)):
            pid = int(bt[r, j])
            if 0 <= pid < P16:
                if n16 < len(s16):
                    s16[n16] = pid
                    n16 += 1
                else:
                    err |= 2
            elif P16 <= pid < P16 + P4:
                if n4 < len(s4):
                    s4[n4] = pid
                    n4 += 1
                else:
                    err |= 2
            else:
                err |= 1
        out[r] = 0
    return s16, n16, s4, n4, out, err


def _pool(kap, P16, P4):
    k = torch.zeros(P16, 1, PAGE, 64, dtype=torch.bfloat16, device="cuda")
    return kap.PackedPool(kap.KVPool(k, k, 1), torch.zeros(P4, 1, 1152, dtype=torch.uint8, device="cuda"))


def _release(kap, pool, bt, seq, gone, s16, n16, s4, n4):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to("cuda")  # noqa: E731
    t16, t4 = d(s16), d(s4)
    c16, c4, out = torch.full((1,), -9, **I32), torch.full((1,), -9, **I32), torch.full((len(seq),), -9, **I32)
    kap.kap_release_tables(d(bt), d(seq), d(gone), t16, torch.tensor([n16], **I32), c16, out, pool=pool, free_packed=t4,
                           packed_count=torch.tensor([n4], **I32), packed_count_out=c4)
    torch.cuda.synchronize()
    return t16.cpu().numpy(), int(c16), t4.cpu().numpy(), int(c4), out.cpu().numpy(), kap.kap_device_error()


@pytest.mark.parametrize("R,mp,share,bad", [
    (1, 1, 1.0, 0), (1, 1, 0.0, 0), (3, 700, 0.9, 0), (2, 5000, 0.97, 0), (33, 9, 0.5, 0), (40, 60, 0.8, 25),
    (2047, 4, 0.3, 0), (2049, 5, 0.6, 7), (5000, 3, 1.0, 0),
])
def test_pages_go_back_by_kind(kap, R, mp, share, bad):
    rng = np.random.default_rng(R + mp)
    P16, P4 = R * mp + 20, R * mp + 30
    bt = np.where(rng.random((R, mp)) < share, P16 + rng.permutation(P4)[:R * mp].reshape(R, mp),
                  rng.permutation(P16)[:R * mp].reshape(R, mp)).astype(np.int32)
    seq = rng.integers(0, mp * PAGE + 1, R).astype(np.int32)
    seq[0] = mp * PAGE
    gone = (rng.random(R) < 0.6).astype(np.int32) * 3
    gone[0] = 1
    for _ in range(bad):   # ids of neither pool
        bt[rng.integers(R), rng.integers(mp)] = rng.choice([-1, -2 ** 31, P16 + P4, 2 ** 31 - 1])
    s16, s4 = np.full(P16, -5, np.int32), np.full(P4, -6, np.int32)
    s16[:7], s4[:3] = np.arange(7), P16 + np.arange(3)
    got = _release(kap, _pool(kap, P16, P4), bt, seq, gone, s16, 7, s4, 3)
    for a, b in zip(got, plain(bt, seq, gone, P16, P4, s16, 7, s4, 3)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("room16,room4", [(5, 100), (100, 4), (0, 0)])
def test_stacks_that_are_too_small(kap, room16, room4):
    P16, P4 = 200, 200
    rng = np.random.default_rng(1)
    bt = np.concatenate([rng.permutation(400)]).astype(np.int32).reshape(8, 50)
    seq = np.full(8, 50 * PAGE, np.int32)
    gone = np.array([1, 0, 1, 0, 0, 1, 0, 0], np.int32)
    s16, s4 = np.full(room16, -5, np.int32), np.full(room4, -6, np.int32)
    got = _release(kap, _pool(kap, P16, P4), bt, seq, gone, s16, 0, s4, 0)
    for a, b in zip(got, plain(bt, seq, gone, P16, P4, s16, 0, s4, 0)):
        assert np.array_equal(a, b)


def test_counts_and_lengths_out_of_range(kap):
    P16, P4 = 10, 10
    bt = np.arange(12, dtype=np.int32).reshape(2, 6) + 4     # 4 .. 9 16-bit, 10 .. 15 packed
    s16, s4 = np.full(12, -5, np.int32), np.full(12, -6, np.int32)
    # a negative count is 0, one past the capacity the capacity; a negative length holds nothing, a long one the row
    got = _release(kap, _pool(kap, P16, P4), bt, np.array([-3, 500], np.int32), [1, 1], s16, -2, s4, 99)
    assert got[5] == 4 | 2
    assert got[1] == 0 and got[3] == 12 and got[4].tolist() == [0, 0] and (got[2] == -6).all()
    got = _release(kap, _pool(kap, P16, P4), bt, np.array([500, 7], np.int32), [1, 0], s16, -2, s4, 3)
    assert got[5] == 4
    assert got[0][:6].tolist() == [4, 5, 6, 7, 8, 9] and got[1] == 6 and got[3] == 3 and got[4].tolist() == [0, 7]


def test_binding_refusals(kap):
    pool = _pool(kap, 4, 4)
    z = lambda n=1: torch.zeros(n, **I32)  # noqa: E731
    a = dict(block_table=torch.zeros(2, 3, **I32), seq_len=z(2), released=z(2), free_pages=z(4), free_count=z(),
             free_count_out=z(), seq_len_out=z(2), pool=pool, free_packed=z(4), packed_count=z(), packed_count_out=z())
    kap.kap_release_tables(**a)
    for name in ("free_packed", "packed_count", "packed_count_out", "pool"):
        with pytest.raises(ValueError):
            kap.kap_release_tables(**{**a, name: None})
    for bad in (dict(packed_count=z(2)), dict(free_packed=z(4).cpu()), dict(packed_count_out=z(3))):
        with pytest.raises(ValueError):
            kap.kap_release_tables(**{**a, **bad})
    with pytest.raises(TypeError):
        kap.kap_release_tables(**{**a, "free_packed": z(4).long()})
    for bad in (dict(packed_count_out=a["packed_count"]), dict(packed_count_out=a["free_count_out"]),
                dict(free_packed=a["free_pages"]), dict(seq_len_out=a["seq_len"])):
        with pytest.raises(kap.KapError) as e:
            kap.kap_release_tables(**{**a, **bad})
        assert e.value.status == -1


def _step(s, new, T):
    """Slots of T more tokens, which are appended with fresh keys and values."""
    slots, pos = s.grow(torch.tensor(new, **I32), T)
    k = torch.randn(T, s.hkv, s.d, generator=s.g, device="cuda").to(torch.bfloat16)
    v = torch.randn(T, s.hkv, s.d, generator=s.g, device="cuda").to(torch.bfloat16)
    s.kap.kap_append_kv(s.pool, k, v, None, pos, slots, s.inv)
    return slots, v


def _check(s, n, hkv, G, d):
    """Attention of each request's last token over its n[r] tokens, page by page from the tables."""
    kap, R = s.kap, len(n)
    t = lambda x: torch.tensor(x, **I32)  # noqa: E731
    q = torch.randn(R, hkv * G, d, generator=s.g, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(R, hkv * G, device="cuda")
    ws = kap.workspace(kap.kap_packed_workspace_size(R, hkv, hkv * G, d), "cuda")
    kap.kap_attn_verify_packed(s.packed, kap.PageMap(s.bt, s.ctx, s.len),
                               kap.VerifyPolicy(t(list(range(R + 1))), t([x - 1 for x in n]), 1, R), q, out, lse, ws)
    torch.cuda.synchronize()
    assert kap.kap_device_error() == 0
    for r in range(R):
        for head in (0, hkv * G - 1):
            _close(out[r, head], lse[r, head], q[r, head], [s.token(r, head // G, i) for i in range(n[r])], d)


def test_released_pages_hold_other_requests(kap):
    """Extend, append, pack; then release a packed request, extend, append, pack again and attend: new tokens lie on 16-bit
    pages, packings take the packed pages that came back, and both requests read what they wrote."""
    hkv, G, d = 2, 4, 128
    s = Server(kap, [70, 200], hkv, G, d, seed=12, spare=4)
    s.pack_full_prompt_pages()
    P16, P4 = s.P16, s.P4
    s.values = lambda pid, h: chunk_values(s.packed.packed[pid - P16, h].cpu().numpy(), d)   # pages change hands: none kept
    _check(s, [70, 200], hkv, G, d)
    used4 = int((s.bt >= P16).sum())
    free4 = torch.full((P4,), -1, **I32)
    free4[:P4 - used4] = torch.arange(P16 + used4, P16 + P4, **I32)
    c4 = torch.tensor([P4 - used4], **I32)
    gone_ids = s.bt[1, :-(-200 // PAGE)].tolist()
    count, length, c4_out = torch.zeros(1, **I32), torch.zeros(2, **I32), torch.zeros(1, **I32)
    kap.kap_release_tables(s.bt, s.len, torch.tensor([0, 1], **I32), s.stack, s.count, count, length, pool=s.packed,
                           free_packed=free4, packed_count=c4, packed_count_out=c4_out)
    torch.cuda.synchronize()
    assert kap.kap_device_error() == 0
    n4 = sum(p >= P16 for p in gone_ids)
    assert int(c4_out) == int(c4) + n4 and free4[int(c4):int(c4_out)].tolist() == [p for p in gone_ids if p >= P16]
    assert int(count) == int(s.count) + len(gone_ids) - n4
    s.count, s.len = count, length
    s.bt[1] = -1
    # the freed request's slot takes a prompt of another length, the other request goes on
    slots, _ = _step(s, [9, 150], 159)
    assert kap.kap_device_error() == 0 and int(slots.max()) < P16 * PAGE and int(slots.min()) >= 0
    _check(s, [79, 150], hkv, G, d)
    # the new prompt's full pages go to packed pages off the stack that came back
    src = s.bt[1, :150 // PAGE].contiguous()
    top = int(c4_out)
    dst = free4[top - len(src):top].contiguous()
    kap.kap_pack_pages(s.packed, src, dst)
    s.bt[1, :150 // PAGE] = dst
    _check(s, [79, 150], hkv, G, d)
