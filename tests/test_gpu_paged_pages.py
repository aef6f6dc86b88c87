"""Page operations of the paged 4-bit cache on tables that are not in order, and on many small pages (GPU)."""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_dfl_gb300 as dfl
from gpu_util import host
from oracle import kv4_oracle as ko
from test_gpu_paged import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.build()
    dfl.load()
    torch.cuda.set_device(0)
    yield
    assert dfl.dfl_get_device_error() == 0


@pytest.mark.parametrize("entry", [-1, 40, 1 << 30, -(1 << 31)])
@pytest.mark.parametrize("N", [4, 1500])   # 1500: more sequences than the planning block has threads
def test_no_room_is_given_behind_a_last_page_that_is_none(entry, N):
    c = dfl.PagedCache(1, 40, 16, 1, 64, N, 4)
    length = np.zeros(N, int)
    length[:4] = [20, 20, 16, 20]
    c.reserve(i32(length))
    c.table[1, 1] = c.table[2, 0] = c.table[3, 1] = entry
    before, new = c.book.clone(), np.zeros(N, int)
    new[:4] = [1, 30, 5, 0]
    start = host(c.reserve(i32(new)))
    assert dfl.dfl_get_device_error() == 1
    # 1: behind a bad page.  2: its last page is full, the next one is its own.  3: nothing asked for.
    assert start[:4].tolist() == [20, -1, 16, 20] and (start[4:] == 0).all()
    want = before.clone()
    table, ln, ref = want[:4 * N].view(N, 4), want[4 * N:5 * N], want[5 * N:]
    ln[0], ln[2], table[2, 1], ref[7] = 21, 21, 7, 1   # pages 0 to 6 are taken
    assert torch.equal(c.book, want)


@pytest.mark.parametrize("N,layers,Hkv,hd,page", [
    (56, 1, 1, 64, 16), (57, 1, 1, 64, 16), (8, 7, 1, 64, 16), (9, 7, 1, 64, 16), (200, 1, 1, 64, 16), (32, 7, 1, 64, 16),
    (4, 7, 1, 64, 32), (5, 7, 1, 64, 32), (14, 2, 1, 128, 16), (15, 2, 1, 128, 16), (3, 3, 5, 64, 16), (2, 1, 7, 128, 32),
    (3, 1, 8, 128, 16), (4, 1, 8, 128, 16)])
@pytest.mark.parametrize("share", ["all", "some"])
def test_shared_last_pages_are_copied_on_both_sides_of_the_rule(N, layers, Hkv, hd, page, share):
    # up to 64 KB of last pages in all are the planning block's
    rng = np.random.default_rng(N + layers)
    num = 4 * N + 5
    c = dfl.PagedCache(layers, num, page, Hkv, hd, N, 3)
    c.data.random_(0, 256)
    b = ko.PageBook(host(c.table), host(c.len), host(c.ref), page)
    data = c.data.clone()

    def reserve(new):
        start, copies = b.reserve(new)
        assert np.array_equal(host(c.reserve(i32(new))), start)
        for s, d in copies:
            data[:, d] = data[:, s]
        assert torch.equal(c.data, data)
        assert np.array_equal(host(c.table), b.table) and np.array_equal(host(c.ref), b.ref)
        return len(copies)

    first = np.full(N, page - 1)
    reserve(first)
    parent = np.zeros(N, int) if share == "all" else np.arange(N) // 2 * 2
    c.remap(i32(parent))
    b.remap(parent)
    assert reserve(rng.integers(1, page, N)) == (N if share == "all" else N // 2 * 2)
    assert reserve(rng.integers(0, 2, N)) == 0
