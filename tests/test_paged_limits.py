"""Sizes of the paged 4-bit cache's calls that are refused on the host, before 32-bit arithmetic could overflow.

Every call here is refused: those whose sizes are fine by a workspace of 0
bytes, which is looked at last.
"""
import ctypes as C

import pytest

import block_diffusion_speculative_dfl_gb300 as dfl

FAKE = 1 << 20   # an aligned stand-in address; refused calls never reach the device
SHAPE, WORKSPACE = 2, 4


def pool(num_pages=10, page=16, Hkv=1, hd=64):
    return dfl.Kv4Pool(FAKE, num_pages * 18 * hd * (page // 16) * Hkv, 1, num_pages, page, Hkv, hd, 0, 0)


@pytest.mark.parametrize("B,Hq,Hkv,rc", [
    (64, 1024, 1, WORKSPACE), (64, 1025, 1, SHAPE), (2, 2 ** 30, 1, SHAPE), (64, 2 ** 26, 1, SHAPE),
    (1, 65536, 1, WORKSPACE), (1, 65537, 1, SHAPE), (65, 1, 1, SHAPE)])
def test_query_rows_of_a_head(B, Hq, Hkv, rc):
    pages = dfl.Pages(FAKE, FAKE, FAKE, 2, 4)
    got = dfl.load().dfl_kv4_attn(C.byref(pool(Hkv=Hkv)), 0, C.byref(pages), FAKE, FAKE, FAKE, B, Hq, FAKE, FAKE, 0, None)
    assert got == rc
    if B <= 64:
        need = dfl.workspace_size(dfl.DFL_OP_KV4_ATTN, N=2, B=B, Hq=Hq, Hkv=Hkv, hd=64)
        assert (need > 0) == (rc == WORKSPACE)


@pytest.mark.parametrize("max_pages,rc", [(1 << 15, SHAPE), ((1 << 15) - 1, WORKSPACE)])
def test_entries_of_the_tables(max_pages, rc):
    lib, p, pages = dfl.load(), pool(), dfl.Pages(FAKE, FAKE, FAKE, 1 << 16, max_pages)
    for f in (lib.dfl_pages_reserve, lib.dfl_pages_remap, lib.dfl_pages_compact):
        assert f(C.byref(p), C.byref(pages), FAKE, FAKE, FAKE, 0, None) == rc


def test_heads_of_a_pool():
    p = dfl.Kv4Pool(FAKE, 1 << 50, 1, 1, 16, 1 << 25, 64, 0, 0)
    pages = dfl.Pages(FAKE, FAKE, FAKE, 2, 4)
    assert dfl.load().dfl_kv4_append(C.byref(p), 0, C.byref(pages), FAKE, FAKE, 1, FAKE, FAKE, None) == SHAPE


@pytest.mark.parametrize("N,max_pages,rc", [(1000, 1 << 15, WORKSPACE), (1 << 15, 1 << 15, SHAPE), (1 << 25, 1, WORKSPACE),
                                            (1 << 29, 1, SHAPE)])
def test_units_of_work(N, max_pages, rc):
    pages = dfl.Pages(FAKE, FAKE, FAKE, N, max_pages)
    got = dfl.load().dfl_kv4_attn(C.byref(pool(Hkv=8)), 0, C.byref(pages), FAKE, FAKE, FAKE, 1, 8, FAKE, FAKE, 0, None)
    assert got == rc
