"""The paged 4-bit cache without a GPU: pins of its oracle, refusals decided on the host, workspace sizes."""
import ctypes as C
import itertools

import numpy as np
import pytest

import block_diffusion_speculative_dfl_gb300 as dfl
from oracle import kv4_oracle as ko

FAKE = 1 << 20   # an aligned stand-in address; refused calls never reach the device


# ------------------------------------------------------------ oracle pins --

def test_number_tables():
    assert ko.E4M3[1] == 2.0 ** -9 and ko.E4M3[8] == 2.0 ** -6 and ko.E4M3[-1] == 448 and len(ko.E4M3) == 127
    assert np.all(np.diff(ko.E4M3) > 0) and np.all(np.diff(ko.E2M1) > 0)


def test_rounding_goes_to_the_nearest_and_ties_to_even_codes():
    y = np.linspace(0, 7, 1401)
    c = ko.nearest_code(y, ko.E2M1)
    d = np.abs(y[:, None] - ko.E2M1)
    assert np.array_equal(np.abs(y - ko.E2M1[c]), d.min(1))
    for border, code in ((0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (9.0, 7)):
        assert ko.nearest_code(border, ko.E2M1) == code
    assert ko.E4M3[ko.nearest_code(1.0 + 1 / 16, ko.E4M3)] == 1.0 and ko.E4M3[ko.nearest_code(1e4, ko.E4M3)] == 448


def test_values_of_known_groups():
    x = np.zeros((3, 16))
    x[0] = [0, 1, 2, 3, 4, 6, -6, -1, 0.5, 0.25, 0.26, -0.75, 5.0, 5.1, 2.5, 3.5]   # max 6: scale 1
    x[1, 3] = np.inf
    x[2, 0] = 1e-9                                                                  # below the smallest scale
    v = ko.kv4_values(x, 0)
    assert v[0].tolist() == [0, 1, 2, 3, 4, 6, -6, -1, 0.5, 0, 0.5, -1, 4, 6, 2, 4]
    assert np.isnan(v[1]).all() and (v[2] == 0).all()
    assert np.array_equal(ko.kv4_values(x[0] * 8, 3), 8 * v[0])


def test_attention_of_equal_scores_averages():
    rng = np.random.default_rng(0)
    kc, vc, vb = np.zeros((5, 1, 64)), rng.standard_normal((5, 1, 64)), rng.standard_normal((2, 1, 64))
    O, _, _, _ = ko.paged_attn(rng.standard_normal((2, 3, 64)), kc, vc, np.zeros((2, 1, 64)), vb)
    want = np.concatenate([vc, vb])[:, 0].mean(0)
    assert np.allclose(O, want, atol=1e-14)


def test_page_book_by_hand():
    b = ko.PageBook(np.full((3, 4), -1), np.zeros(3, np.int32), np.zeros(6, np.int32), 16)
    start, copies = b.reserve([20, 16, 0])
    assert b.table[0, :2].tolist() == [0, 1] and b.table[1, 0] == 2 and start.tolist() == [0, 0, 0] and not copies
    b.remap([0, 1, 0])                       # sequence 2 forks sequence 0
    assert b.ref.tolist() == [2, 2, 1, 0, 0, 0] and b.len.tolist() == [20, 16, 20]
    start, copies = b.reserve([1, 0, 0])     # writing the shared last page copies it
    assert copies == [(1, 3)] and b.table[0, 1] == 3 and b.ref.tolist() == [2, 1, 1, 1, 0, 0]
    start, copies = b.reserve([60, 1, 1])    # three pages of two left: refused, and what comes after it too
    assert start.tolist() == [-1, -1, 20] and b.len.tolist() == [21, 16, 21]
    b.remap([-1, 1, 2], [-1, 3, -1])
    assert b.ref.tolist() == [1, 1, 1, 0, 0, 0] and b.len.tolist() == [0, 3, 21]
    b.remap([-1, -1, 2])
    m, live, moves = b.compact()
    assert live == 2 and moves == [] and m.tolist() == [0, 1, -1, -1, -1, -1]


# -------------------------------------------------------------- refusals --

def _pool(**kw):
    f = dict(data=FAKE, layer_stride=8 * dfl.dfl_kv4_page_bytes(32, 2, 64), layers=3, num_pages=8, page=32, Hkv=2, hd=64,
             k_exp=0, v_exp=0)
    f.update(kw)
    return dfl.Kv4Pool(**f)


def _pages(**kw):
    f = dict(table=FAKE, len=FAKE, ref=FAKE, N=4, max_pages=5)
    f.update(kw)
    return dfl.Pages(**f)


WS = dict(ws=FAKE, ws_bytes=1 << 30)


def _append(pool, pages, layer=0, start=FAKE, n_new=FAKE, R=7, K=FAKE, V=FAKE, fn="dfl_kv4_append"):
    return getattr(dfl.load(), fn)(C.byref(pool), layer, C.byref(pages), start, n_new, R, K, V, None)


def _read(pool, pages, **kw):
    return _append(pool, pages, fn="dfl_kv4_read", **kw)


def _attn(pool, pages, layer=0, Q=FAKE, Kb=FAKE, Vb=FAKE, B=2, Hq=4, O=FAKE, ws=FAKE, ws_bytes=1 << 30):
    return dfl.load().dfl_kv4_attn(C.byref(pool), layer, C.byref(pages), Q, Kb, Vb, B, Hq, O, ws, ws_bytes, None)


def _reserve(pool, pages, n_new=FAKE, start=FAKE, ws=FAKE, ws_bytes=1 << 30):
    return dfl.load().dfl_pages_reserve(C.byref(pool), C.byref(pages), n_new, start, ws, ws_bytes, None)


def _remap(pool, pages, parent=FAKE, keep=None, ws=FAKE, ws_bytes=1 << 30):
    return dfl.load().dfl_pages_remap(C.byref(pool), C.byref(pages), parent, keep, ws, ws_bytes, None)


def _compact(pool, pages, map_=FAKE, live=FAKE, ws=FAKE, ws_bytes=1 << 30):
    return dfl.load().dfl_pages_compact(C.byref(pool), C.byref(pages), map_, live, ws, ws_bytes, None)


CALLS = [_append, _read, _attn, _reserve, _remap, _compact]
INVALID, SHAPE, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("field,value,code", [
    ("data", None, INVALID), ("layers", 0, INVALID), ("num_pages", 0, INVALID), ("Hkv", 0, INVALID),
    ("page", 24, SHAPE), ("page", 2048, SHAPE), ("hd", 96, SHAPE), ("hd", 0, INVALID), ("k_exp", 61, INVALID),
    ("v_exp", -61, INVALID), ("layer_stride", 8 * 2 * 2 * 18 * 64 - 16, INVALID), ("data", FAKE + 8, MISALIGNED),
    ("layer_stride", 8 * 2 * 2 * 18 * 64 + 8, MISALIGNED)])
def test_pools_are_refused(call, field, value, code):
    assert call(_pool(**{field: value}), _pages()) == code


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("field,value,code", [
    ("table", None, INVALID), ("len", None, INVALID), ("N", 0, INVALID), ("max_pages", 0, INVALID),
    ("table", FAKE + 2, MISALIGNED), ("len", FAKE + 1, MISALIGNED), ("max_pages", 1 << 26, SHAPE)])
def test_tables_are_refused(call, field, value, code):
    assert call(_pool(), _pages(**{field: value})) == code


@pytest.mark.parametrize("call,kw,code", [
    (_append, dict(layer=3), INVALID), (_append, dict(layer=-1), INVALID), (_append, dict(start=None), INVALID),
    (_append, dict(n_new=None), INVALID), (_append, dict(K=None), INVALID), (_append, dict(V=None), INVALID),
    (_append, dict(R=0), INVALID), (_append, dict(K=FAKE + 8), MISALIGNED), (_append, dict(R=1 << 30), SHAPE),
    (_append, dict(start=FAKE + 2), MISALIGNED), (_read, dict(V=FAKE + 4), MISALIGNED), (_read, dict(K=None), INVALID),
    (_attn, dict(layer=3), INVALID), (_attn, dict(Q=None), INVALID), (_attn, dict(Kb=None), INVALID),
    (_attn, dict(Vb=None), INVALID), (_attn, dict(O=None), INVALID), (_attn, dict(ws=None), INVALID),
    (_attn, dict(B=0), INVALID), (_attn, dict(B=65), SHAPE), (_attn, dict(Hq=3), INVALID), (_attn, dict(Hq=0), INVALID),
    (_attn, dict(Q=FAKE + 8), MISALIGNED), (_attn, dict(ws=FAKE + 8), MISALIGNED), (_attn, dict(ws_bytes=16), WORKSPACE),
    (_reserve, dict(n_new=None), INVALID), (_reserve, dict(start=None), INVALID), (_reserve, dict(ws=None), INVALID),
    (_reserve, dict(ws_bytes=100), WORKSPACE), (_reserve, dict(n_new=FAKE + 2), MISALIGNED),
    (_remap, dict(parent=None), INVALID), (_remap, dict(keep=FAKE + 2), MISALIGNED), (_remap, dict(ws_bytes=10), WORKSPACE),
    (_remap, dict(ws=FAKE + 8), MISALIGNED), (_compact, dict(map_=None), INVALID), (_compact, dict(live=None), INVALID),
    (_compact, dict(ws_bytes=10), WORKSPACE), (_compact, dict(map_=FAKE + 2), MISALIGNED)])
def test_arguments_are_refused(call, kw, code):
    assert call(_pool(), _pages(), **kw) == code


@pytest.mark.parametrize("call", [_reserve, _remap, _compact])
def test_page_operations_need_the_counts(call):
    assert call(_pool(), _pages(ref=None)) == INVALID


def test_too_many_cells_are_refused():
    n = 1 << 27
    p = _pool(num_pages=n, Hkv=8, layer_stride=n * dfl.dfl_kv4_page_bytes(32, 8, 64))
    assert _append(p, _pages()) == SHAPE


def test_page_bytes():
    for page, hkv, hd in itertools.product((16, 48, 64, 1024), (1, 8), (64, 128)):
        assert dfl.dfl_kv4_page_bytes(page, hkv, hd) == page * hkv * 2 * (hd // 2 + hd // 16)
    assert dfl.dfl_kv4_page_bytes(17, 1, 64) == dfl.dfl_kv4_page_bytes(0, 1, 64) == dfl.dfl_kv4_page_bytes(16, 1, 80) == 0


def test_workspace_sizes():
    w = dfl.workspace_size
    assert w(dfl.DFL_OP_KV4_ATTN, N=3, B=2, Hq=4, Hkv=2, hd=64, dtype=1) > 0
    assert w(dfl.DFL_OP_KV4_ATTN, N=3, B=2, Hq=3, Hkv=2, hd=64, dtype=1) == 0
    assert w(dfl.DFL_OP_PAGES_RESERVE, N=3, pages=100) >= (100 + 5 * 3) * 4
    assert w(dfl.DFL_OP_PAGES_REMAP, N=3, pages=100) >= 3 * 101 * 4
    assert w(dfl.DFL_OP_PAGES_COMPACT, pages=100) >= 2 * 100 * 4
    assert w(dfl.DFL_OP_PAGES_RESERVE, N=0, pages=100) == w(dfl.DFL_OP_PAGES_COMPACT, pages=-1) == 0
    shape = dict(N=2, C=64, B=16, d=256, Hq=4, Hkv=2, hd=64, D=2, L=3, V=1000, G=15, row0=1, dtype=1, R=8)
    assert w(dfl.DFL_OP_DRAFT_STEP_PAGED, pages=9, **shape) > 0
    assert w(dfl.DFL_OP_DRAFT_STEP_PAGED, pages=0, **shape) == 0
    assert w(dfl.DFL_OP_DRAFT_STEP_PAGED, pages=9, **dict(shape, dtype=0)) == 0


def _step_args(dtype=1):
    lib = dfl._lib
    layers = (lib.LayerWeights * 2)()
    for w in layers:
        for n, _ in lib.LayerWeights._fields_[:6]:
            setattr(w, n, FAKE)
    a = lib.StepArgs()
    a.N, a.C, a.B, a.d, a.Hq, a.Hkv, a.hd, a.D, a.L, a.V, a.dtype = 2, 64, 16, 256, 4, 2, 64, 2, 3, 1000, dtype
    a.eps, a.h_layer_stride = 1e-6, 2 * 64 * 256
    for n in ("H", "mix_logits", "mix_gain", "blk_gain", "final_gain", "W_lm", "Xb0", "Xb", "draft"):
        setattr(a, n, FAKE)
    a.layers = layers
    return a, layers


def test_paged_steps_are_refused_on_the_host():
    pool = _pool()

    def call(args=None, ws_bytes=1 << 32, pool=pool, pages=None, **kw):
        a = args or _step_args()[0]
        f = dict(R=8, n_new=FAKE, start=FAKE)
        f.update(kw)
        ctx = dfl.PagedCtx(pool=C.pointer(pool) if pool else None, pages=pages or _pages(N=2, max_pages=2), **f)
        return dfl.load().dfl_draft_step_paged(C.byref(a), C.byref(ctx), FAKE, ws_bytes, None)

    assert call(ws_bytes=1 << 10) == WORKSPACE
    assert call(args=_step_args(dtype=0)[0]) == SHAPE
    assert call(R=0) == INVALID and call(n_new=None) == INVALID and call(start=None) == INVALID
    assert call(pool=None) == INVALID
    assert call(pool=_pool(layers=1)) == INVALID                       # fewer layers than the drafter
    assert call(pool=_pool(hd=128, layer_stride=1 << 20)) == INVALID   # another head dim
    assert call(pages=_pages(N=3, max_pages=2)) == INVALID             # another batch
    assert call(pages=_pages(N=2, max_pages=3)) == INVALID             # 96 tokens in 64 rotary positions
    assert call(pages=_pages(N=2, max_pages=2, ref=None)) == INVALID
    assert call(start=FAKE + 2) == MISALIGNED
    assert dfl.load().dfl_draft_step_paged(C.byref(_step_args()[0]), None, FAKE, 1 << 30, None) == INVALID
    b = _step_args()[0]
    b.B = 65
    assert call(args=b) == SHAPE
