"""More sizes and structs that the paged 4-bit cache's calls settle on the host, without a GPU."""
import ctypes as C

import pytest

import block_diffusion_speculative_dfl_gb300 as dfl

FAKE = 1 << 20   # an aligned stand-in address; refused calls never reach the device
SHAPE, WORKSPACE = 2, 4


@pytest.mark.parametrize("page,max_pages,rc", [
    (1024, (1 << 21) - 8, WORKSPACE), (1024, (1 << 21) - 7, SHAPE), (1024, (1 << 21) - 1, SHAPE),
    (16, (1 << 27) - 512, WORKSPACE), (16, (1 << 27) - 511, SHAPE)])
@pytest.mark.parametrize("B,Hq", [(1, 1), (4, 4), (16, 4), (64, 2)])
def test_positions_of_attention_keep_to_32_bits(page, max_pages, rc, B, Hq):
    # positions are looked up as much as 4,096 tokens ahead of a sequence's last
    pool = dfl.Kv4Pool(FAKE, 10 * 18 * 64 * (page // 16), 1, 10, page, 1, 64, 0, 0)
    pages = dfl.Pages(FAKE, FAKE, FAKE, 1, max_pages)
    got = dfl.load().dfl_kv4_attn(C.byref(pool), 0, C.byref(pages), FAKE, FAKE, FAKE, B, Hq, FAKE, FAKE, 0, None)
    assert got == rc
