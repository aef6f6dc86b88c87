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


def test_shapes_of_before_the_paged_cache_end_before_its_field():
    # the old struct lies at the end of a mapping; behind it an unreadable page of memory
    import mmap
    libc, old = C.CDLL(None, use_errno=True), dfl._lib.Shape.pages.offset
    libc.mprotect.argtypes = [C.c_void_p, C.c_size_t, C.c_int]
    m = mmap.mmap(-1, 2 * mmap.PAGESIZE)
    base = C.addressof(C.c_char.from_buffer(m))
    sizes = dict(N=2, C=64, B=16, d=256, Hq=4, Hkv=2, hd=64, D=2, L=3, V=1000, K=4, G=15, row0=1, dtype=1, F=512, R=8)
    s = dfl._lib.Shape(**sizes)
    C.memmove(base + mmap.PAGESIZE - old, C.addressof(s), old)
    f = dfl.load().dfl_workspace_size
    at = C.cast(base + mmap.PAGESIZE - old, C.POINTER(dfl._lib.Shape))
    try:
        assert libc.mprotect(base + mmap.PAGESIZE, mmap.PAGESIZE, 0) == 0
        got = [f(op, at) for op in list(range(1, 14))]
    finally:
        libc.mprotect(base + mmap.PAGESIZE, mmap.PAGESIZE, mmap.PROT_READ | mmap.PROT_WRITE)
    assert got == [dfl.workspace_size(op, **sizes) for op in range(1, 14)] and all(got)


@pytest.mark.parametrize("op", range(1, 18))
def test_a_negative_count_of_pages_matters_to_its_ops_only(op):
    sizes = dict(N=2, C=64, B=16, d=256, Hq=4, Hkv=2, hd=64, D=2, L=3, V=1000, K=4, G=15, row0=1, dtype=1, F=512, R=8)
    paged = op in (dfl.DFL_OP_PAGES_RESERVE, dfl.DFL_OP_PAGES_REMAP, dfl.DFL_OP_PAGES_COMPACT, dfl.DFL_OP_DRAFT_STEP_PAGED)
    assert (dfl.workspace_size(op, pages=-1, **sizes) == 0) == paged
    assert dfl.workspace_size(op, pages=9, **sizes) > 0


def _paged_step(F=0, sample=None, vlog=False, accept_rule=0, d=256, L=3, V=1000):
    lib = dfl._lib
    layers = (lib.LayerWeights * 2)()
    for w in layers:
        for n, _ in lib.LayerWeights._fields_:
            setattr(w, n, FAKE)
    a = lib.StepArgs()
    a.N, a.C, a.B, a.d, a.Hq, a.Hkv, a.hd, a.D, a.L, a.V, a.dtype, a.F = 2, 64, 16, d, 4, 2, 64, 2, L, V, 1, F
    a.eps, a.h_layer_stride, a.accept_rule = 1e-6, 2 * 64 * d, accept_rule
    for n in ("H", "mix_logits", "mix_gain", "blk_gain", "final_gain", "W_lm", "Xb0", "Xb", "draft", "ffn_gain", "samples",
              "scores", "selected", "accept_len", "bonus"):
        setattr(a, n, FAKE)
    a.layers = layers
    sp = dfl._lib.SampleParams(*sample) if sample else None
    if sp is not None:
        a.sample = C.pointer(sp)
    if vlog:
        a.vlog = FAKE
    pool = dfl.Kv4Pool(FAKE, 8 * dfl.dfl_kv4_page_bytes(32, 2, 64), 2, 8, 32, 2, 64, 0, 0)
    ctx = dfl.PagedCtx(pool=C.pointer(pool), pages=dfl.Pages(FAKE, FAKE, FAKE, 2, 2), R=8, n_new=FAKE, start=FAKE)
    return dfl.load().dfl_draft_step_paged(C.byref(a), C.byref(ctx), FAKE, 0, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(), WORKSPACE), (dict(F=128), WORKSPACE), (dict(F=72), SHAPE),                      # the feed-forward's K blocks
    (dict(d=5120), WORKSPACE), (dict(d=5152), SHAPE), (dict(d=8192), SHAPE),                 # the mix's and the norm's rows
    (dict(sample=(4, 1.0, 1)), WORKSPACE), (dict(sample=(0, 1.0, 1)), 1), (dict(sample=(65, 1.0, 1)), 1),
    (dict(sample=(4, 0.0, 1)), 1), (dict(sample=(4, float("nan"), 1)), 1), (dict(sample=(4, -1.0, 1)), 1),
    (dict(sample=(4, 1.0, 1), V=6398 * 256), WORKSPACE), (dict(sample=(4, 1.0, 1), V=6400 * 256), SHAPE),
    (dict(sample=(4, 1.0, 1), vlog=True, accept_rule=2), WORKSPACE)])
def test_a_paged_step_that_is_refused_has_launched_nothing(kw, rc):
    # a workspace of 0 bytes is looked at last, before the reservation of pages, the first launch
    assert _paged_step(**kw) == rc
