"""Host-side checks of the packed-page, log-probability and table calls: documented codes before any CUDA call.

Placeholder addresses, never dereferenced when the checks work; run only where no kernel can launch."""
import ctypes

import pytest
import torch

cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host checks run where no kernel can launch")
KAP_OK, KAP_EINVAL, KAP_ESHAPE, KAP_ECAPACITY, KAP_EUNSUPPORTED = 0, -1, -2, -3, -5
ADDR = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10004)
Z = ctypes.c_size_t


@pytest.fixture(scope="module")
def abi():
    from selected_kv_sparse_gb300 import build as kbuild
    kbuild.build()
    import selected_kv_sparse_gb300._binding as b
    return b, b.load()


def _pool(b, P=8, P4=4, hkv=2, hq=8, d=64, dtype=0, packed=0x10000):
    return b._Packed(b._Pool(P, 16, hkv, hq, d, dtype, 0x10000, 0x10000, None), P4, packed)


def _map(b, R=2, mp=4):
    return b._Map(R, mp, 0x10000, 0x10000, 0x10000)


def test_struct_matches_the_header(tmp_path):
    import os
    import shutil
    import subprocess
    from selected_kv_sparse_gb300 import _binding as b
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kap.h"\nint main(void) { printf("%zu %zu %zu %zu", '
                   "sizeof(kap_packed_pool), offsetof(kap_packed_pool, pool), offsetof(kap_packed_pool, num_packed), "
                   "offsetof(kap_packed_pool, packed)); return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(b._Packed), b._Packed.pool.offset, b._Packed.num_packed.offset, b._Packed.packed.offset]


def test_sizes(abi):
    _, lib = abi
    assert [lib.kap_packed_chunk_bytes(d) for d in (64, 128, 96, 0, -64)] == [1152, 2304, 0, 0, 0]
    assert lib.kap_packed_workspace_size(4, 8, 32, 128, 4) > 0 and lib.kap_packed_workspace_size(0, 8, 32, 128, 4) == 0
    assert lib.kap_logprobs_workspace_size(3, 100) > 0 and lib.kap_logprobs_workspace_size(0, 100) == 0


@cpu_only
def test_packed_pool_is_checked(abi):
    b, lib = abi
    for fn in (lib.kap_pack_pages, lib.kap_unpack_pages):
        call = lambda p, src=ADDR, dst=ADDR, n=1: fn(ctypes.byref(p), src, dst, n, None)  # noqa: E731
        assert fn(None, ADDR, ADDR, 1, None) == KAP_EINVAL
        assert call(_pool(b, dtype=1)) == KAP_EUNSUPPORTED            # an fp32 pool
        assert call(_pool(b, d=96)) == KAP_EUNSUPPORTED
        assert call(_pool(b, packed=None)) == KAP_EINVAL
        assert call(_pool(b, packed=0x10008)) == KAP_EINVAL           # not 16-byte aligned
        assert call(_pool(b, P4=-1)) == KAP_EINVAL
        assert call(_pool(b, P=1 << 20, P4=1 << 26)) == KAP_EUNSUPPORTED   # more slots than 31 bits
        assert call(_pool(b), src=None) == KAP_EINVAL
        assert call(_pool(b), n=-1) == KAP_EINVAL
        assert call(_pool(b), n=0, src=None, dst=None) == KAP_OK


@cpu_only
def test_attention_is_checked(abi):
    b, lib = abi
    size = lib.kap_packed_workspace_size(2, 2, 8, 64, 1)
    view = lambda rows=2, cap=4: b._View(rows, cap, 0x10000, 0x10000, 0x10000, 0x10000, 0)  # noqa: E731

    def propose(pool=None, m=None, v=None, q=ADDR, out=ADDR, lse=ADDR, ws=ADDR, n=size):
        return lib.kap_attn_propose_packed(ctypes.byref(pool or _pool(b)), ctypes.byref(m or _map(b)),
                                           ctypes.byref(v or view()), q, out, lse, ws, Z(n), None)

    for bad in (dict(q=None), dict(out=None), dict(lse=None), dict(ws=None), dict(q=ODD), dict(out=ODD), dict(ws=ODD),
                dict(v=view(cap=0)), dict(m=_map(b, R=0))):
        assert propose(**bad) == KAP_EINVAL, bad
    assert propose(v=view(rows=3)) == KAP_ESHAPE
    assert propose(n=size - 1) == KAP_ECAPACITY
    assert propose(pool=_pool(b, dtype=1)) == KAP_EUNSUPPORTED
    assert propose(pool=_pool(b, hq=18)) == KAP_EUNSUPPORTED          # G = 9

    size2 = lib.kap_packed_workspace_size(2, 2, 8, 64, 16)

    def verify(max_q=16, total=3, off=0x10000, start=0x10000, n=size2, **kw):
        pool, q, out = kw.get("pool", _pool(b)), kw.get("q", ADDR), kw.get("out", ADDR)
        return lib.kap_attn_verify_packed(ctypes.byref(pool), ctypes.byref(_map(b)),
                                          ctypes.byref(b._Verify(max_q, total, off, start)), q, out, ADDR, ADDR, Z(n),
                                          None)

    assert verify(max_q=17) == KAP_EUNSUPPORTED                       # G * max_q = 68
    assert verify(max_q=1 << 30) == KAP_EUNSUPPORTED
    assert verify(max_q=0) == KAP_EINVAL and verify(total=-1) == KAP_EINVAL
    assert verify(off=None) == KAP_EINVAL and verify(start=None) == KAP_EINVAL and verify(q=ODD) == KAP_EINVAL
    assert verify(n=size2 - 1) == KAP_ECAPACITY
    assert verify(total=0) == KAP_OK


@cpu_only
def test_logprobs_are_checked(abi):
    _, lib = abi
    size = lib.kap_logprobs_workspace_size(2, 100)

    def call(lg=ADDR, dt=1, V=100, stride=100, rows=2, tok=ADDR, top=3, lp=ADDR, ids=ADDR, tlp=ADDR, ws=ADDR, n=size):
        return lib.kap_token_logprobs(lg, dt, V, ctypes.c_int64(stride), rows, tok, top, lp, None, None, ids, tlp, ws,
                                      Z(n), None)

    for bad in (dict(lg=None), dict(tok=None), dict(lp=None), dict(ws=None), dict(ids=None), dict(tlp=None),
                dict(V=0), dict(rows=-1), dict(stride=99), dict(top=-1), dict(top=33), dict(V=2, stride=2, top=3),
                dict(lg=ctypes.c_void_p(0x10002)), dict(dt=0, lg=ctypes.c_void_p(0x10001)), dict(ws=ODD)):
        assert call(**bad) == KAP_EINVAL, bad
    assert call(dt=2) == KAP_EUNSUPPORTED
    assert call(V=(1 << 24) + 1, stride=1 << 25) == KAP_EUNSUPPORTED
    assert call(n=size - 1) == KAP_ECAPACITY
    assert call(rows=0, lg=None, tok=None) == KAP_OK


@cpu_only
def test_tables_are_checked(abi):
    _, lib = abi
    B = ctypes.c_void_p(0x20000)

    def extend(R=2, mp=3, bt=ADDR, seq=ADDR, new=ADDR, free=ADDR, cap=4, cnt=ADDR, cnt2=B, off=ADDR, slot=ADDR,
               pos=ADDR, T=5, seq2=B, ok=ADDR):
        return lib.kap_extend_tables(R, mp, bt, seq, new, free, cap, cnt, cnt2, off, slot, pos, T, seq2, ok, None)

    for name in ("bt", "seq", "new", "free", "cnt", "cnt2", "off", "slot", "pos", "seq2", "ok"):
        assert extend(**{name: None}) == KAP_EINVAL, name
    for bad in (dict(R=0), dict(mp=0), dict(cap=-1), dict(T=-1), dict(seq2=ADDR), dict(cnt2=ADDR)):
        assert extend(**bad) == KAP_EINVAL, bad
    assert extend(mp=(1 << 26) + 1) == KAP_EUNSUPPORTED

    def release(R=2, mp=3, bt=ADDR, seq=ADDR, gone=ADDR, free=ADDR, cap=4, cnt=ADDR, cnt2=B, seq2=B):
        return lib.kap_release_tables(R, mp, bt, seq, gone, free, cap, cnt, cnt2, seq2, None)

    for name in ("bt", "seq", "gone", "free", "cnt", "cnt2", "seq2"):
        assert release(**{name: None}) == KAP_EINVAL, name
    for bad in (dict(R=0), dict(mp=0), dict(cap=-1), dict(seq2=ADDR), dict(cnt2=ADDR)):
        assert release(**bad) == KAP_EINVAL, bad
    assert release(mp=(1 << 26) + 1) == KAP_EUNSUPPORTED
