"""Host-side checks of the release over both kinds of page: documented codes before any CUDA call.

Placeholder addresses, never dereferenced when the checks work; run only where no kernel can launch."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host checks run where no kernel can launch")
KAP_EINVAL, KAP_EUNSUPPORTED = -1, -5
NAMES = ("R", "mp", "bt", "seq", "gone", "P16", "free", "cap", "cnt", "cnt2", "P4", "free4", "cap4", "cnt4", "cnt42", "seq2")
SOUND = dict(R=2, mp=3, bt=0x10000, seq=0x20000, gone=0x30000, P16=8, free=0x40000, cap=8, cnt=0x50000, cnt2=0x60000, P4=4,
             free4=0x70000, cap4=4, cnt4=0x80000, cnt42=0x90000, seq2=0xA0000)


@pytest.fixture(scope="module")
def release():
    from selected_kv_sparse_gb300 import build as kbuild
    kbuild.build()
    import selected_kv_sparse_gb300._binding as b
    lib = b.load()

    def call(**kw):
        a = {**SOUND, **kw}
        return lib.kap_release_tables_packed(*[a[n] for n in NAMES], None)
    return call


def test_null_and_negative_arguments(release):
    for name in ("bt", "seq", "gone", "free", "cnt", "cnt2", "free4", "cnt4", "cnt42", "seq2"):
        assert release(**{name: None}) == KAP_EINVAL, name
    for bad in (dict(R=0), dict(mp=0), dict(cap=-1), dict(cap4=-1), dict(P16=-1), dict(P4=-1)):
        assert release(**bad) == KAP_EINVAL, bad


def test_sizes_past_the_limits(release):
    assert release(mp=(1 << 26) + 1) == KAP_EUNSUPPORTED
    assert release(P16=1 << 30, P4=1 << 30) == KAP_EUNSUPPORTED


def test_aliased_arrays(release):
    for bad in (dict(seq2=SOUND["seq"]), dict(cnt2=SOUND["cnt"]), dict(cnt42=SOUND["cnt4"]), dict(cnt42=SOUND["cnt2"]),
                dict(cnt42=SOUND["cnt"]), dict(cnt2=SOUND["cnt4"]), dict(free4=SOUND["free"])):
        assert release(**bad) == KAP_EINVAL, bad
