"""What the calls of drafted tokens refuse, without a GPU: the checks fire
before any CUDA call."""
import ctypes

import pytest

from variable_length_batching_gb300 import build as nt_build, nt

FAKE, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002)         # never dereferenced
INVALID, UNSUPPORTED, OVERFLOW = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    nt_build.build()
    return nt.lib()


def _pages(**kw):
    a = dict(k=0x1000, v=0x1000, n_pages=8, page_size=16, H_kv=2, d=64, dtype=1)
    a.update(kw)
    return ctypes.byref(nt.nt_kv_pages(*a.values()))


def test_tree_attn(lib):
    def run(pages=None, **kw):
        a = dict(q=FAKE, stride=256, T=6, H=4, cu=FAKE, B=2, max_new=8, table=FAKE, max_pages=4, lengths=FAKE, bits=FAKE,
                 scale=0.125, o=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 30)
        a.update(kw)
        return lib.nt_paged_tree_attn(pages or _pages(), *a.values(), None)
    for bad in (dict(T=-1), dict(B=-1), dict(H=0), dict(H=3), dict(max_new=-1), dict(max_pages=-1), dict(q=None),
                dict(stride=255), dict(stride=248), dict(cu=None), dict(B=0), dict(lengths=None), dict(o=None),
                dict(ws=None), dict(ws_bytes=1 << 10), dict(scale=0.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(table=None), dict(bits=ctypes.c_void_p(0x1004)), dict(cu=ODD),
                dict(lengths=ODD), dict(lse=ODD), dict(o=ctypes.c_void_p(0x1008)), dict(table=ODD),
                dict(pages=_pages(k=None)), dict(pages=_pages(page_size=0)), dict(pages=_pages(dtype=5))):
        assert run(**bad) == INVALID, bad
    assert run(max_new=257) == UNSUPPORTED and run(pages=_pages(d=48)) == UNSUPPORTED
    assert run(max_pages=(1 << 20) + 1) == UNSUPPORTED
    assert run(T=1 << 31) == OVERFLOW and run(B=(1 << 30) + 1) == OVERFLOW
    assert run(T=1 << 30, H=65536, max_pages=1 << 10, stride=1 << 22) == OVERFLOW
    assert run(T=0) == 0 and run(T=0, q=None, cu=None, B=0, lengths=None, o=None, ws=None, ws_bytes=0) == 0
    assert lib.nt_paged_tree_attn(None, FAKE, 256, 6, 4, FAKE, 2, 8, FAKE, 4, FAKE, None, 0.125, FAKE, None, FAKE, 1 << 30,
                                  None) == INVALID


def test_tree_attn_workspace(lib):
    f = nt.nt_paged_tree_attn_workspace_bytes
    for H, Hk, d, n in ((0, 1, 64, 4), (3, 2, 64, 4), (4, 2, 48, 4), (4, 2, 64, 257), (4, 2, 64, -1), (4, 0, 64, 1)):
        assert f(H, Hk, d, n) == 0
    for d in (32, 64, 128):
        assert 0 < f(32, 8, d, 256) <= 137 << 20


def test_resize(lib):
    def run(**kw):
        a = dict(new=FAKE, B=2, page=16, table=FAKE, max_pages=4, lengths=FAKE, free=FAKE, n_pages=8, n_free=FAKE, cu=FAKE,
                 pos0=FAKE, slots=FAKE, T=4, lacking=FAKE)
        a.update(kw)
        return lib.nt_paged_resize(*a.values(), None)
    for bad in (dict(B=-1), dict(page=0), dict(page=65537), dict(max_pages=-1), dict(n_pages=-1), dict(T=-1), dict(new=None),
                dict(table=None), dict(lengths=None), dict(free=None), dict(n_free=None), dict(cu=None), dict(pos0=None),
                dict(slots=None), dict(lacking=None), dict(new=ODD), dict(table=ODD), dict(lengths=ODD), dict(free=ODD),
                dict(n_free=ODD), dict(cu=ODD), dict(pos0=ODD), dict(lacking=ODD), dict(slots=ctypes.c_void_p(0x1004))):
        assert run(**bad) == INVALID, bad
    assert run(T=1 << 31) == OVERFLOW and run(B=(1 << 30) + 1) == OVERFLOW


def test_draft_tree(lib):
    def run(**kw):
        a = dict(parents=FAKE, cu=FAKE, B=2, T=4, max_new=8, pos0=None, bits=FAKE, positions=None)
        a.update(kw)
        return lib.nt_draft_tree(*a.values(), None)
    for bad in (dict(parents=None), dict(cu=None), dict(B=-1), dict(B=0), dict(T=-1), dict(max_new=0), dict(bits=None),
                dict(parents=ODD), dict(cu=ODD), dict(pos0=ODD), dict(positions=ODD), dict(bits=ctypes.c_void_p(0x1004))):
        assert run(**bad) == INVALID, bad
    assert run(max_new=257) == UNSUPPORTED and run(T=1 << 31) == OVERFLOW and run(B=(1 << 30) + 1) == OVERFLOW
    assert run(T=0, parents=None, bits=None) == 0 and run(T=0, B=0, cu=None, parents=None, bits=None) == 0


def test_keep_and_write_slots(lib):
    def keep(pages=None, **kw):
        a = dict(kept=FAKE, K=4, cu=FAKE, B=2, table=FAKE, max_pages=4, pos0=FAKE)
        a.update(kw)
        return lib.nt_paged_keep(pages or _pages(), *a.values(), None)
    for bad in (dict(kept=None), dict(K=-1), dict(cu=None), dict(B=0), dict(B=-1), dict(table=None), dict(max_pages=-1),
                dict(pos0=None), dict(kept=ODD), dict(cu=ODD), dict(pos0=ODD), dict(pages=_pages(v=None))):
        assert keep(**bad) == INVALID, bad
    assert keep(K=1 << 31) == OVERFLOW and keep(B=(1 << 30) + 1) == OVERFLOW and keep(pages=_pages(d=4)) == UNSUPPORTED
    assert keep(K=0) == 0 and keep(K=0, kept=None, cu=None, B=0, pos0=None) == 0

    def write(pages=None, **kw):
        a = dict(k=FAKE, ks=128, v=FAKE, vs=128, T=4, slots=FAKE)
        a.update(kw)
        return lib.nt_paged_write_slots(pages or _pages(), *a.values(), None)
    for bad in (dict(k=None), dict(v=None), dict(ks=120), dict(vs=127), dict(T=-1), dict(slots=None),
                dict(slots=ctypes.c_void_p(0x1004)), dict(k=ctypes.c_void_p(0x1008))):
        assert write(**bad) == INVALID, bad
    assert write(T=1 << 31) == OVERFLOW and write(T=0, k=None, v=None, slots=None) == 0
