"""Packing 16-bit pages into 4-bit ones and back, against exact arithmetic: codes and parameters bit for bit."""
import numpy as np
import pytest
import torch

from tests.packed_reference import PAGE, chunk_parts, chunk_values, pack_group

pytestmark = pytest.mark.gpu


def _pools(kap, P16, P4, hkv, d, fill=None, summaries=False):
    dev = "cuda"
    g = torch.Generator().manual_seed(7)
    K = torch.randn(P16, hkv, PAGE, d, generator=g).to(torch.bfloat16)
    V = (0.3 * torch.randn(P16, hkv, PAGE, d, generator=g) + 0.1).to(torch.bfloat16)
    if fill is not None:
        fill(K, V)
    packed = torch.full((P4, hkv, kap.kap_packed_chunk_bytes(d)), 0xAB, dtype=torch.uint8, device=dev)
    ks = torch.randn(P16 + P4, hkv, d, generator=g).to(dev) if summaries else None
    pool = kap.PackedPool(kap.KVPool(K.to(dev), V.to(dev), hkv), packed, ks)
    return pool, K, V


def _hard_rows(K, V):
    """Groups on which a careless rounding shows."""
    d = K.shape[3]
    bf = lambda x: torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)  # noqa: E731
    K[0, 0, 0] = 0.0                                             # all zero
    K[0, 0, 1] = -1.5                                            # constant
    K[0, 0, 2] = 0.0
    K[0, 0, 2, 5] = 15.0                                         # scale exactly 1, everything else on the lowest
    K[0, 0, 3, :64] = bf([0.5 * (i % 31) for i in range(64)])    # every second value on a border between two codes
    K[0, 0, 4] = bf(1.0) * 2.0 ** -130                           # subnormal, constant
    K[0, 0, 5] = (torch.arange(d) % 16).float().to(torch.bfloat16) * 2.0 ** -133   # subnormal codes
    K[0, 0, 6, ::2] = bf(3.0e38)
    K[0, 0, 6, 1::2] = bf(-3.0e38)                               # a range past fp32's largest number
    K[0, 0, 7, 3] = float("inf")
    K[0, 0, 8, 3] = float("nan")
    K[0, 0, 9, 3] = float("-inf")
    # lowest -15/16 and highest 15/16: the middle border is 0; values far below lowest's last bit decide it by sign
    K[0, 0, 10] = 0.0
    K[0, 0, 10, 0], K[0, 0, 10, 1] = -0.9375, 0.9375
    K[0, 0, 10, 2], K[0, 0, 10, 3] = 2.0 ** -30, -(2.0 ** -30)
    K[0, 0, 11] = -0.0
    K[0, 0, 11, ::3] = 0.0                                       # zeros of both signs
    K[0, 0, 12, :] = bf(2.0) ** -100
    K[0, 0, 12, 7] = bf(15.0) * 2.0 ** -97                       # tiny scale
    V[0, 0, 0, :] = bf(1.0e38)
    V[0, 0, 0, 1] = bf(-1.0e38)                                  # large but finite
    V[0, 0, 1, :64] = bf([1.0 + i / 128 for i in range(64)])     # small range on a large offset


@pytest.mark.parametrize("d,hkv", [(64, 1), (128, 3), (128, 8)])
def test_codes_are_exact(kap, d, hkv):
    P16, P4 = 5, 6
    pool, K, V = _pools(kap, P16, P4, hkv, d, fill=_hard_rows)
    src, dst = [0, 3, 4], [P16 + 5, P16 + 0, P16 + 2]
    i32 = dict(dtype=torch.int32, device="cuda")
    kap.kap_pack_pages(pool, torch.tensor(src, **i32), torch.tensor(dst, **i32))
    torch.cuda.synchronize()
    assert kap.kap_device_error() == 0
    got = pool.packed.cpu().numpy()
    for a, b in zip(src, dst):
        for h in range(hkv):
            codes, s, lo = chunk_parts(got[b - P16, h], d)
            for t, X in enumerate((K, V)):
                rows = X[a, h].float().numpy()
                for tok in range(PAGE if (a, h) == (0, 0) else 3):
                    for blk in range(d // 64):
                        ref = pack_group(rows[tok, 64 * blk:64 * blk + 64])
                        if ref is None:
                            assert np.isnan(s[t, tok, blk]) and np.isnan(lo[t, tok, blk])
                            continue
                        at = (a, h, t, tok, blk)
                        assert (s[t, tok, blk], lo[t, tok, blk]) == ref[:2], at
                        assert codes[t, tok, 64 * blk:64 * blk + 64].tolist() == ref[2], at
    # packed pages that were not named keep their bytes
    for j in (1, 3, 4):
        assert (got[j] == 0xAB).all()


@pytest.mark.parametrize("d,hkv,n", [(64, 2, 1), (128, 2, 9), (128, 8, 70)])
def test_round_trip_and_summaries(kap, d, hkv, n):
    P16, P4 = 2 * n, n
    pool, K, V = _pools(kap, P16, P4, hkv, d, summaries=True)
    ks0 = pool.k_summary.clone()
    g = torch.Generator().manual_seed(3)
    i32 = dict(dtype=torch.int32, device="cuda")
    src = torch.randperm(n, generator=g)
    dst = torch.randperm(n, generator=g) + P16
    kap.kap_pack_pages(pool, src.to(**i32), dst.to(**i32))
    kap.kap_unpack_pages(pool, dst.to(**i32), (src + n).to(**i32))
    torch.cuda.synchronize()
    assert kap.kap_device_error() == 0
    packed = pool.packed.cpu().numpy()
    back = [pool.pool.k_pages.cpu(), pool.pool.v_pages.cpu()]
    for i in range(0, n, max(1, n // 5)):
        for h in range(hkv):
            want, _, _ = chunk_values(packed[int(dst[i]) - P16, h], d)
            for t, X in enumerate((K, V)):
                w = torch.from_numpy(want[t])
                # one fp32 rounding, then half a bf16 step
                got = back[t][n + int(src[i]), h].double()
                assert ((got - w).abs() <= w.abs() * (2.0 ** -8 + 2.0 ** -24)).all()
                # half a scale is the most that a value moves (and half a bf16 step in reading it back)
                _, s, _ = chunk_parts(packed[int(dst[i]) - P16, h], d)
                half = torch.from_numpy(np.repeat(s[t].astype(np.float64), 64, axis=1)) * 0.5
                assert ((w - X[int(src[i]), h].double()).abs() <= half * (1 + 2.0 ** -40)).all()
    assert torch.equal(back[0][:n], K[:n]) and torch.equal(back[1][:n], V[:n])   # sources stay
    ks = pool.k_summary
    d_dev, s_dev = dst.to("cuda"), src.to("cuda")
    assert torch.equal(ks[d_dev], ks0[s_dev]) and torch.equal(ks[s_dev + n], ks0[s_dev])


def test_ids_outside_their_pool_are_skipped(kap):
    P16, P4, hkv, d = 4, 3, 2, 64
    pool, K, V = _pools(kap, P16, P4, hkv, d)
    i32 = dict(dtype=torch.int32, device="cuda")
    # a source that is packed, a destination that is 16-bit, ids past both ends; the third pair is sound
    kap.kap_pack_pages(pool, torch.tensor([4, 0, 1, -1, 2], **i32), torch.tensor([5, 3, 4, 6, 7], **i32))
    assert kap.kap_device_error() == 1
    got = pool.packed.cpu()
    assert (got[1:] == 0xAB).all() and not (got[0] == 0xAB).all()
    kap.kap_unpack_pages(pool, torch.tensor([0, 4, 7, 4], **i32), torch.tensor([1, 4, 2, -1], **i32))
    assert kap.kap_device_error() == 1
    assert torch.equal(pool.pool.k_pages.cpu(), K) and torch.equal(pool.pool.v_pages.cpu(), V)


def test_no_pages_is_no_work(kap):
    pool, K, _ = _pools(kap, 2, 1, 1, 64)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    kap.kap_pack_pages(pool, e, e)
    kap.kap_unpack_pages(pool, e, e)
    assert kap.kap_device_error() == 0 and (pool.packed.cpu() == 0xAB).all()


def test_binding_refusals(kap):
    pool, _, _ = _pools(kap, 2, 1, 1, 64)
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        kap.kap_pack_pages(pool, i.long(), i)
    with pytest.raises(ValueError):
        kap.kap_pack_pages(pool, i, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        kap.kap_pack_pages(pool, i.cpu(), i.cpu())
    with pytest.raises(ValueError):
        kap.kap_pack_pages(kap.PackedPool(pool.pool, pool.packed[:, :, :-1].contiguous()), i, i)
    f32 = kap.KVPool(pool.pool.k_pages.float(), pool.pool.v_pages.float(), 1)
    with pytest.raises(TypeError):
        kap.kap_pack_pages(kap.PackedPool(f32, pool.packed), i, i)
    with pytest.raises(ValueError):
        kap.kap_pack_pages(kap.PackedPool(pool.pool, pool.packed, torch.zeros(2, 1, 64, device="cuda")), i, i)
    with pytest.raises(ValueError):
        pool.routing()
