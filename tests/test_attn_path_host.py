"""Host side of the attention-path operators, without a GPU: the frequency
table against the definition, and the refusals of every entry point (they
fire before any CUDA call)."""
import ctypes
import math

import pytest
import torch

from _attn_path import inv_freq
from variable_length_batching_gb300 import build as nt_build, nt

FAKE, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)     # never dereferenced: the checks fire first
OK, INVALID, UNSUPPORTED, OVERFLOW = 0, 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def lib():
    nt_build.build()
    return nt.lib()


@pytest.mark.parametrize("rot,kw", [
    (2, {}), (64, {}), (128, dict(base=1e6)), (64, dict(scaling="linear", factor=4.0)),
    (64, dict(scaling="ntk", factor=8.0, base=5e5)), (2, dict(scaling="ntk", factor=8.0)),
    (128, dict(scaling="bands", factor=4.0, original_len=8192.0)),
    (128, dict(scaling="bands", factor=8.0, original_len=8192.0, low=1.0, high=4.0, base=5e5)),
])
def test_turns(rot, kw):
    """The table's fractions of a turn equal the definition's to fp64's
    precision (pow and the products are off by a few steps of 2^-53) and to
    the table's unit: a fraction held in 64 bits is cut at 2^-64."""
    t = nt.nt_rope_turns(rot, **kw)
    want = inv_freq(rot, **kw) / (2 * math.pi)
    got = torch.tensor([(int(x) % (1 << 64)) / 2.0 ** 64 for x in t], dtype=torch.float64)
    assert t.dtype == torch.int64 and t.numel() == rot // 2
    assert bool(((got - want).abs() <= 32 * 2.0 ** -53 * want + 2.0 ** -64).all())


def test_turns_wrap_above_a_turn():
    """A frequency above a turn per position keeps its fraction."""
    t = nt.nt_rope_turns(2, scaling="linear", factor=1.0 / (2 * math.pi * 3.25))
    assert abs((int(t[0]) % (1 << 64)) / 2.0 ** 64 - 0.25) < 1e-14


@pytest.mark.parametrize("args", [
    (0, 1e4, 0, 1, 0, 1, 32), (3, 1e4, 0, 1, 0, 1, 32), (70000, 1e4, 0, 1, 0, 1, 32), (64, 0.0, 0, 1, 0, 1, 32),
    (64, math.inf, 0, 1, 0, 1, 32), (64, math.nan, 0, 1, 0, 1, 32), (64, 1e4, 4, 1, 0, 1, 32),
    (64, 1e4, -1, 1, 0, 1, 32), (64, 1e4, 1, 0.0, 0, 1, 32), (64, 1e4, 2, -1.0, 0, 1, 32),
    (64, 1e4, 1, math.nan, 0, 1, 32), (64, 1e4, 3, 2.0, 0, 1, 32), (64, 1e4, 3, 2.0, 8192, 4, 4),
    (64, 1e4, 3, 2.0, 8192, math.nan, 4), (64, 1e4, 3, 2.0, math.inf, 1, 4),
])
def test_turns_refusals(lib, args):
    out = (ctypes.c_uint64 * 40000)()
    assert lib.nt_rope_turns(*args, out) == INVALID
    assert lib.nt_rope_turns(64, 1e4, 0, 1.0, 0.0, 1.0, 32.0, None) == INVALID


def _rope(lib, **kw):
    a = dict(dtype=1, q=FAKE, qs=256, k=FAKE, ks=256, T=10, Hq=4, Hk=4, d=64, qg=None, kg=None, eps=1e-6, cu=FAKE,
             B=2, p0=None, pos=None, turns=FAKE, rot=64, inter=0, scale=1.0, qo=FAKE, qos=256, ko=FAKE, kos=256)
    a.update(kw)
    return lib.nt_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), OVERFLOW), (dict(Hq=-1), INVALID),
    (dict(d=0), INVALID), (dict(d=72), UNSUPPORTED), (dict(d=272, rot=0, qs=2048), UNSUPPORTED),
    (dict(rot=80), INVALID), (dict(rot=24), UNSUPPORTED), (dict(rot=-16), INVALID), (dict(inter=2), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(q=None), INVALID),
    (dict(ko=None), INVALID), (dict(q=ODD), INVALID), (dict(k=ODD), INVALID), (dict(qo=ODD), INVALID),
    (dict(qs=255), INVALID), (dict(qs=260), INVALID), (dict(ks=248), INVALID), (dict(kos=0), INVALID),
    (dict(turns=None), INVALID), (dict(turns=ctypes.c_void_p(0x1004)), INVALID), (dict(cu=None), INVALID),
    (dict(B=0), INVALID), (dict(B=-1), INVALID), (dict(pos=FAKE), INVALID), (dict(cu=None, p0=FAKE, pos=FAKE), INVALID),
    (dict(qg=ODD), INVALID), (dict(qos=512), INVALID), (dict(cu=ctypes.c_void_p(0x1002)), INVALID),
    (dict(T=0, q=None, k=None, qo=None, ko=None, cu=None, B=0), OK),
    (dict(Hq=0, Hk=0, q=None, k=None, qo=None, ko=None), OK),
])
def test_rope_refusals(lib, kw, status):
    assert _rope(lib, **kw) == status


def _rope_bwd(lib, **kw):
    a = dict(dtype=1, uq=FAKE, uqs=256, uk=FAKE, uks=256, q=FAKE, qs=256, k=FAKE, ks=256, T=10, Hq=4, Hk=4, d=64,
             qg=FAKE, kg=FAKE, eps=1e-6, cu=FAKE, B=2, p0=None, pos=None, turns=FAKE, rot=64, inter=0, scale=1.0,
             dq=FAKE, dqs=256, dk=FAKE, dks=256, dqg=FAKE, dkg=FAKE, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return lib.nt_qk_norm_rope_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(uq=None), INVALID), (dict(dk=None), INVALID),
    (dict(dqg=None), INVALID), (dict(kg=None), INVALID), (dict(ws=None), INVALID), (dict(wsb=16), INVALID),
    (dict(ws=ODD), INVALID), (dict(dqs=512), INVALID), (dict(d=72), UNSUPPORTED), (dict(rot=24), UNSUPPORTED),
    (dict(T=1 << 31), OVERFLOW),
])
def test_rope_bwd_refusals(lib, kw, status):
    assert _rope_bwd(lib, **kw) == status


def _pages(**kw):
    p = nt.nt_kv_pages(0x1000, 0x1000, 8, 16, 2, 64, 1)
    for name, v in kw.items():
        setattr(p, name, v)
    return p


BAD_PAGES = [(dict(dtype=3), INVALID), (dict(n_pages=-1), INVALID), (dict(page_size=0), INVALID),
             (dict(page_size=65537), INVALID), (dict(H_kv=0), INVALID), (dict(d=0), INVALID),
             (dict(d=12), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=0x1008), INVALID),
             (dict(n_pages=2**31 - 1, H_kv=2), OVERFLOW)]


@pytest.mark.parametrize("kw,status", BAD_PAGES)
def test_pages_refusals(lib, kw, status):
    p = ctypes.byref(_pages(**kw))
    one = (ctypes.c_int32 * 1)(0)
    two = (ctypes.c_int32 * 1)(1)
    assert lib.nt_paged_copy(p, one, two, 1, None) == status
    assert lib.nt_paged_write(p, FAKE, 128, FAKE, 128, 1, FAKE, 1, None, FAKE, 4, None) == status
    assert lib.nt_paged_attn(p, FAKE, 256, 1, 4, FAKE, 4, FAKE, 0.125, FAKE, None, FAKE, 1 << 30, None) == status
    assert lib.nt_paged_copy(None, one, two, 1, None) == INVALID


def test_copy_refusals(lib):
    p = ctypes.byref(_pages())
    arr = lambda *v: (ctypes.c_int32 * len(v))(*v)
    cp = lambda s, d, n=None: lib.nt_paged_copy(p, arr(*s), arr(*d), len(s) if n is None else n, None)
    assert cp([0], [8]) == INVALID           # outside the pool
    assert cp([-1], [0]) == INVALID
    assert cp([0, 1], [2, 2]) == INVALID     # written twice
    assert cp([0, 2], [2, 3]) == INVALID     # read and written
    assert cp([1], [1]) == INVALID
    assert cp([0], [1], -1) == INVALID
    assert lib.nt_paged_copy(p, arr(*range(9)), arr(*range(9)), 9, None) == INVALID      # more copies than pages
    assert lib.nt_paged_copy(p, None, arr(1), 1, None) == INVALID
    assert lib.nt_paged_copy(p, None, None, 0, None) == OK


def test_write_refusals(lib):
    def wr(k=FAKE, ks=128, v=FAKE, vs=128, T=3, cu=FAKE, B=1, p0=None, table=FAKE, mp=4):
        return lib.nt_paged_write(ctypes.byref(_pages()), k, ks, v, vs, T, cu, B, p0, table, mp, None)
    assert wr(T=-1) == INVALID and wr(B=-1) == INVALID and wr(T=1 << 31) == OVERFLOW
    assert wr(k=None) == INVALID and wr(v=ODD) == INVALID and wr(ks=120) == INVALID and wr(vs=132) == INVALID
    assert wr(cu=None) == INVALID and wr(B=0) == INVALID and wr(table=None) == INVALID and wr(mp=-1) == INVALID
    assert wr(p0=ctypes.c_void_p(0x1002)) == INVALID and wr(table=ctypes.c_void_p(0x1001)) == INVALID
    assert wr(T=0, k=None, v=None, cu=None, B=0, table=None) == OK


def test_attn_refusals(lib):
    need = nt.nt_paged_attn_workspace_bytes(4, 2, 64)

    def at(pages=None, q=FAKE, qs=256, B=1, H=4, table=FAKE, mp=4, lens=FAKE, scale=0.125, o=FAKE, lse=None, ws=FAKE,
           wsb=need):
        return lib.nt_paged_attn(ctypes.byref(pages or _pages()), q, qs, B, H, table, mp, lens, scale, o, lse, ws, wsb,
                                 None)
    assert at(B=-1) == INVALID and at(H=0) == INVALID and at(H=3) == INVALID
    assert at(pages=_pages(d=48), qs=192) == UNSUPPORTED
    for s in (0.0, -1.0, math.nan, math.inf):
        assert at(scale=s) == INVALID
    assert at(q=None) == INVALID and at(q=ODD) == INVALID and at(qs=248) == INVALID and at(qs=260) == INVALID
    assert at(table=None) == INVALID and at(mp=-1) == INVALID and at(lens=None) == INVALID and at(o=None) == INVALID
    assert at(o=ODD) == INVALID and at(ws=None) == INVALID and at(ws=ODD) == INVALID and at(wsb=need - 1) == INVALID
    assert at(lse=ctypes.c_void_p(0x1002)) == INVALID and at(lens=ctypes.c_void_p(0x1002)) == INVALID
    assert at(B=0, q=None, table=None, lens=None, o=None, ws=None, wsb=0) == OK
    assert lib.nt_paged_attn_workspace_bytes(4, 3, 64) == 0 and lib.nt_paged_attn_workspace_bytes(4, 2, 48) == 0


def test_limits_of_segments_and_of_a_batch(lib):
    """Counts the kernels' indexes could not hold."""
    far = (1 << 30) + 1
    assert _rope(lib, B=far) == OVERFLOW and _rope_bwd(lib, B=far) == OVERFLOW
    p = ctypes.byref(_pages())
    assert lib.nt_paged_write(p, FAKE, 128, FAKE, 128, 1, FAKE, far, None, FAKE, 4, None) == OVERFLOW
    attn = lambda B, pages: lib.nt_paged_attn(p, FAKE, 256, B, 4, FAKE, pages, FAKE, 0.125, FAKE, None, FAKE, 1 << 30,
                                              None)
    assert attn(far, 0) == OVERFLOW
    odd = ctypes.byref(_pages(page_size=12))
    assert lib.nt_paged_attn(odd, FAKE, 256, 1, 4, FAKE, (1 << 24) // 12 + 1, FAKE, 0.125, FAKE, None, FAKE, 1 << 30,
                             None) == UNSUPPORTED
    assert attn(1 << 30, 1 << 8) == OVERFLOW           # 2^30 * 2^8 pages of 16 * 4 heads


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    q = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        nt.nt_qk_norm_rope(q, q, nt.nt_rope_turns(64), positions=torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        nt.nt_qk_norm_rope(None, None, None)
    with pytest.raises(ValueError):
        nt.nt_qk_norm_rope(q, q[:3], None)
    with pytest.raises(ValueError):
        nt.nt_qk_norm_rope(q, q, None, positions=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        nt.nt_qk_norm_rope(q, q, None, q_gamma=torch.ones(32))
    with pytest.raises(ValueError):
        nt.nt_rope_turns(64, scaling="other")
    with pytest.raises(ValueError):
        nt.KVPages(torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 16, 64))
    with pytest.raises(ValueError):
        nt.KVPages(torch.zeros(2, 1, 16, 64), torch.zeros(3, 1, 16, 64))
