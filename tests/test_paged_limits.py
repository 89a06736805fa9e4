"""Limits of paged attention's longest tables, without a GPU: what one SM
would add up in turn, and wait for, is refused before any CUDA call."""
import ctypes

import pytest

from variable_length_batching_gb300 import build as nt_build, nt

FAKE = ctypes.c_void_p(0x1000)          # never dereferenced: the checks fire first
UNSUPPORTED, OVERFLOW = 2, 3


@pytest.fixture(scope="module")
def lib():
    nt_build.build()
    return nt.lib()


@pytest.mark.parametrize("B,H,Hk,page,max_pages", [
    (152, 1, 1, 64, (1 << 28) // 64),               # an SM to each of 152 contexts of 2^28
    (129, 1, 1, 16, (1 << 24) // 16 + 1),
    (1, 8, 8, 8, (1 << 28) // 8 + 1),               # eight key heads
    (1, 64, 1, 8, (1 << 28) // 8 + 1),              # one, read once for every eight of its queries
    (2, 1, 1, 65536, 1 << 15),
])
def test_long_tables_of_many_items(lib, B, H, Hk, page, max_pages):
    p = nt.nt_kv_pages(0x1000, 0x1000, 8, page, Hk, 64, 1)
    assert lib.nt_paged_attn(ctypes.byref(p), FAKE, 64 * H, B, H, FAKE, max_pages, FAKE, 0.125, FAKE, None, FAKE, 1 << 30,
                             None) == UNSUPPORTED
    assert b"2^31" in lib.nt_last_error()


def test_named_kernels_refusals(lib):
    """What a kernel does not take, and kernels there are not."""
    def run(kernel, cluster=0, page=16, max_pages=4, n_pages=8, **kw):
        p = nt.nt_kv_pages(0x1000, 0x1000, n_pages, page, 2, 64, 1)
        a = dict(B=1, H=4, scale=0.125)
        a.update(kw)
        return lib.nt_selftest_paged_attn(kernel, cluster, ctypes.byref(p), FAKE, 256, a["B"], a["H"], FAKE, max_pages, FAKE,
                                          a["scale"], FAKE, None, FAKE, 1 << 30, None)
    for kernel, cluster in ((-1, 0), (3, 0), (0, 1), (2, 4), (1, -1), (1, 13)):
        assert run(kernel, cluster) == 1
    assert run(0, max_pages=65) == UNSUPPORTED and run(0, n_pages=0) == UNSUPPORTED
    assert run(2, page=12) == UNSUPPORTED and run(2, n_pages=0) == UNSUPPORTED
    for kernel in range(3):
        assert run(kernel, scale=0.0) == 1 and run(kernel, H=3) == 1 and run(kernel, B=-1) == 1
        assert run(kernel, B=0) == 0
