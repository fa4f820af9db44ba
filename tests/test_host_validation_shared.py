"""Host-side checks of the normalising append, the attention over shared prefixes and the sampling: documented codes before any
CUDA call, struct layouts, and the pairs' axes.

Placeholder addresses, never dereferenced when the checks work; refusals run only where no kernel can launch."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host checks run where no kernel can launch")
KAP_OK, KAP_EINVAL, KAP_ESHAPE, KAP_ECAPACITY, KAP_EUNSUPPORTED = 0, -1, -2, -3, -5
A, ODD = 0x10000, 0x10004


@pytest.fixture(scope="module")
def abi():
    from selected_kv_sparse_gb300 import build as kbuild
    kbuild.build()
    import selected_kv_sparse_gb300._binding as b
    return b, b.load()


def test_structs_match_the_header(tmp_path):
    from selected_kv_sparse_gb300 import _binding as b
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    mirrors = {"kap_prefix_groups": b._Groups, "kap_norm_append": b._NormAppend}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "kap.h"', "int main(void) {"]
    for c, py in mirrors.items():
        lines.append(f'  printf("{c} size %zu\\n", sizeof({c}));')
        lines += [f'  printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([cc, "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in out if x.strip()}
    for c, py in mirrors.items():
        assert got[(c, "size")] == ctypes.sizeof(py)
        for f, _ in py._fields_:
            assert got[(c, f)] == getattr(py, f).offset, (c, f)


def test_axes_of_the_pairs(abi):
    b, _ = abi
    f = lambda d, sec, inter=False: b.rope_freq_axis(d, sec, inter).tolist()  # noqa: E731
    assert f(8, [4]) == [0] * 4
    assert f(16, [2, 3, 3]) == [0, 0, 1, 1, 1, 2, 2, 2]
    assert f(16, [4, 2, 2], True) == [0, 1, 2, 0, 1, 2, 0, 0]
    got = f(128, [24, 20, 20], True)
    assert got == [i % 3 if i % 3 and i < 60 else 0 for i in range(64)]
    assert [got.count(a) for a in range(3)] == [24, 20, 20]
    assert f(16, [0, 8]) == [1] * 8
    for bad in ((16, [2, 3, 2], False), (16, [9, -1], False), (15, [7], False), (0, [0], False), (16, [], False),
                (16, [1] * 8 + [0], False), (16, [2, 3, 3], True), (16, [0, 8], True)):
        with pytest.raises(b.KapError):
            b.rope_freq_axis(*bad)


def test_sizes(abi):
    _, lib = abi
    size = lib.kap_shared_workspace_size
    assert size(4, 8, 32, 128, 4, 1) > 0 and size(4, 8, 32, 128, 64, 1) > size(4, 8, 32, 128, 4, 1)
    for bad in ((0, 8, 32, 128, 4, 1), (4, 0, 32, 128, 4, 1), (4, 8, 32, 128, -1, 1), (4, 8, 32, 128, 4, -1)):
        assert size(*bad) == 0


def _pool(b, P=8, hkv=2, hq=8, d=64, dtype=0, k=A):
    return b._Pool(P, 16, hkv, hq, d, dtype, k, A, None)


@cpu_only
def test_append_is_checked(abi):
    b, lib = abi
    good = dict(k_new=A, v_new=A, q=A, q_out=A, k_stride=128, v_stride=128, q_stride=512, q_out_stride=512, q_weight=None,
                k_weight=None, eps=1e-6, num_axes=1, pos=A, axis_stride=4, freq_axis=None, slots=A, inv_freq=A, num_tokens=4,
                tok_stride=1)
    call = lambda pool=None, **kw: lib.kap_append_kv_norm(ctypes.byref(pool or _pool(b)),  # noqa: E731
                                                          ctypes.byref(b._NormAppend(**{**good, **kw})), None)
    assert lib.kap_append_kv_norm(None, None, None) == KAP_EINVAL
    assert lib.kap_append_kv_norm(ctypes.byref(_pool(b)), None, None) == KAP_EINVAL
    for name in ("k_new", "v_new", "q_out", "pos", "slots", "inv_freq"):
        assert call(**{name: None}) == KAP_EINVAL, name
    for name in ("k_new", "v_new", "q", "q_out"):
        assert call(**{name: ODD}) == KAP_EINVAL, name
    for bad in (dict(num_tokens=-1), dict(num_axes=0), dict(num_axes=9), dict(tok_stride=0), dict(axis_stride=-1),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(k_stride=127), dict(k_stride=64),
                dict(v_stride=132), dict(q_stride=511), dict(q_out_stride=504), dict(q_stride=520)):
        assert call(**bad) == KAP_EINVAL, bad
    assert call(pool=_pool(b, d=96)) == KAP_EUNSUPPORTED
    assert call(pool=_pool(b, hq=18)) == KAP_EUNSUPPORTED
    assert call(pool=_pool(b, k=ODD)) == KAP_EINVAL
    assert call(num_tokens=0, k_new=None, q=None) == KAP_OK


@cpu_only
def test_shared_attention_is_checked(abi):
    b, lib = abi
    size = lib.kap_shared_workspace_size(2, 2, 8, 64, 3, 1)

    def call(pool=None, m=None, v=None, g=None, q=A, out=A, lse=A, ws=A, n=size):
        m = m or b._Map(2, 4, A, A, None)
        v = v or b._Verify(2, 3, A, A)
        g = g or b._Groups(1, A, A)
        return lib.kap_attn_verify_shared(ctypes.byref(pool or _pool(b)), ctypes.byref(m), ctypes.byref(v), ctypes.byref(g),
                                          q, out, lse, ws, n, None)
    assert lib.kap_attn_verify_shared(None, None, None, None, A, A, A, A, size, None) == KAP_EINVAL
    for bad in (dict(q=None), dict(out=None), dict(lse=None), dict(ws=None), dict(q=ODD), dict(out=ODD), dict(ws=ODD),
                dict(v=b._Verify(0, 3, A, A)), dict(v=b._Verify(2, -1, A, A)), dict(v=b._Verify(2, 3, None, A)),
                dict(v=b._Verify(2, 3, A, None)), dict(g=b._Groups(-1, A, A)), dict(g=b._Groups(1, None, A)),
                dict(g=b._Groups(1, A, None)), dict(m=b._Map(0, 4, A, A, None)), dict(m=b._Map(2, 4, None, A, None))):
        assert call(**bad) == KAP_EINVAL, bad
    assert call(v=b._Verify(17, 17, A, A)) == KAP_EUNSUPPORTED                # 68 query columns
    assert call(m=b._Map(2, (1 << 26) + 1, A, A, None)) == KAP_EUNSUPPORTED
    assert call(g=b._Groups((1 << 20) + 1, A, A)) == KAP_EUNSUPPORTED
    assert call(v=b._Verify(2, 1 << 30, A, A)) == KAP_EUNSUPPORTED            # more query rows than 31 bits
    assert call(n=size - 1) == KAP_ECAPACITY
    assert call(v=b._Verify(2, 0, A, A), q=None, out=None, lse=None, ws=None, n=1 << 30) == KAP_OK
    assert call(v=b._Verify(2, 0, A, A), n=0) in (KAP_OK, KAP_ECAPACITY)


@cpu_only
def test_shared_attention_over_no_rows_needs_no_workspace(abi):
    b, lib = abi
    pool, m, g = _pool(b), b._Map(2, 4, A, A, None), b._Groups(1, A, A)
    call = lambda v, ws, n: lib.kap_attn_verify_shared(ctypes.byref(pool), ctypes.byref(m), ctypes.byref(v),  # noqa: E731
                                                       ctypes.byref(g), None, None, None, ws, n, None)
    for v in (b._Verify(2, 0, A, A), b._Verify(2, 0, None, None)):
        for ws, n in ((A, 0), (None, 0), (ODD, 1 << 30)):
            assert call(v, ws, n) == KAP_OK
    g = b._Groups(1, None, A)
    assert call(b._Verify(2, 0, A, A), A, 0) == KAP_EINVAL
    g = b._Groups((1 << 20) + 1, A, A)
    assert call(b._Verify(2, 0, A, A), A, 0) == KAP_EUNSUPPORTED


@cpu_only
def test_sampling_is_checked(abi):
    _, lib = abi
    call = lambda lg=A, dt=0, V=100, st=100, rows=3, u=A, tok=A: lib.kap_sample_tokens(  # noqa: E731
        lg, dt, V, st, rows, u, None, None, None, None, tok, None, None, None)
    assert call(dt=2) == KAP_EUNSUPPORTED and call(V=(1 << 24) + 1, st=1 << 25) == KAP_EUNSUPPORTED
    assert call(rows=(1 << 26) + 1) == KAP_EUNSUPPORTED
    for bad in (dict(V=0), dict(V=-1), dict(st=99), dict(rows=-1), dict(lg=None), dict(u=None), dict(tok=None), dict(lg=A + 1),
                dict(lg=A + 2, dt=1)):
        assert call(**bad) == KAP_EINVAL, bad
    assert call(rows=0, lg=None, u=None, tok=None) == KAP_OK
