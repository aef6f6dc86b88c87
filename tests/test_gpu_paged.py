"""The paged 4-bit context cache on the GPU against its fp64 oracle.

Values written and read back, page numbers, counts and moved bytes are exact.
Attention's bound counts its roundings: the output (bf16, half a step 2^-8 of
the value), the softmax weights (fp16, 2^-11, of the cached keys and bf16,
2^-8, of the block's own), the scores and exponentials in fp32 (2^-18 of the
weight, times 1 + the largest score, covers hd = 128 products, the base-2
exponential's 2^-22 and a query's fp16 form), and weights below fp16's normal
range (2^-32 a key of the largest value).
"""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_dfl_gb300 as dfl
from dfl_synth import Workload
from gpu_util import assert_bf16_close, host
from oracle import kv4_oracle as ko

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.build()
    dfl.load()
    torch.cuda.set_device(0)
    yield
    assert dfl.dfl_get_device_error() == 0


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def bf16(rng, shape, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)) * scale).to(torch.bfloat16).cuda()


def make_cache(rng, N, lens, page, Hkv, hd, layers=1, extra=0, spare=3, **kw):
    """A cache whose sequences hold scattered pages for lens[n] + extra tokens (ref set, len = lens)."""
    used = [-(-(int(l) + extra) // page) for l in lens]
    total = sum(used) + spare
    c = dfl.PagedCache(layers, total, page, Hkv, hd, N, max(1, max(used)), **kw)
    ids = rng.permutation(total)
    table, at = np.full((N, c.max_pages), -1), 0
    for n, u in enumerate(used):
        table[n, :u] = ids[at:at + u]
        at += u
    ref = np.zeros(total)
    ref[ids[:at]] = 1
    c.table.copy_(i32(table))
    c.len.copy_(i32(lens))
    c.ref.copy_(i32(ref))
    return c


def fill(rng, c, layer, lens, scale=1.0):
    """Random rows at positions 0 .. lens[n]-1; returns K, V bf16 on the host as fp64 [N][T][Hkv][hd]."""
    T = max(1, int(max(lens)))
    K, V = bf16(rng, (c.N, T, c.Hkv, c.hd), scale), bf16(rng, (c.N, T, c.Hkv, c.hd), scale)
    c.append(layer, K, V, i32(np.zeros(c.N)), i32(lens))
    return host(K).astype(np.float64), host(V).astype(np.float64)


# ------------------------------------------------------------ append, read --

@pytest.mark.parametrize("hd,page,Hkv,N,R,e", [
    (128, 64, 8, 3, 16, 0), (64, 16, 1, 1, 1, 0), (64, 32, 2, 5, 33, 1), (128, 48, 3, 4, 130, -2), (128, 16, 2, 2, 17, 5),
    (64, 1024, 2, 2, 9, 0)])
def test_rows_come_back_as_the_values_they_stand_for(hd, page, Hkv, N, R, e):
    rng = np.random.default_rng(hd + page + R)
    start = rng.integers(0, 70, N)
    cnt = rng.integers(0, R + 1, N)
    cnt[0] = R
    c = make_cache(rng, N, start, page, Hkv, hd, extra=R, layers=2, k_exp=e, v_exp=-e)
    before = c.data.clone()
    K, V = bf16(rng, (N, R, Hkv, hd), 2.0 ** e), bf16(rng, (N, R, Hkv, hd), 3.0)
    c.append(1, K, V, i32(start), i32(cnt))
    oK, oV = torch.full_like(K, 7.0), torch.full_like(V, 7.0)
    c.read(1, i32(start), i32(cnt), oK, oV)
    assert torch.equal(c.data[0], before[0])   # the other layer
    for x, o, ex in ((K, oK, e), (V, oV, -e)):
        want = ko.kv4_values(host(x), ex)
        for n in range(N):
            assert np.array_equal(host(o)[n, :cnt[n]], want[n, :cnt[n]])
            assert (host(o)[n, cnt[n]:] == 7.0).all()


@pytest.mark.parametrize("hd", [64, 128])
def test_values_on_borders_and_out_of_range(hd):
    # every border times several scales, zeros, the ends of bf16's range, infinities and NaN
    base = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, 0.0])
    rows = [base * f for f in (1.0, 2.0, 0.4375, 2.0 ** -9, 2.0 ** -11, 448.0, 3e38 / 6, 1e-38)]
    rows += [np.zeros(16), np.r_[np.inf, base[1:]], np.r_[base[:15], np.nan], np.r_[-np.inf, base[1:]]]
    x = np.zeros((1, len(rows), 1, hd), np.float32)
    for r, v in enumerate(rows):
        for g in range(hd // 16):
            x[0, r, 0, 16 * g:16 * g + 16] = v if g % 2 == 0 else base
    X = torch.from_numpy(x).to(torch.bfloat16).cuda()
    rng = np.random.default_rng(1)
    for e in (0, 3, -60, 60):
        c = make_cache(rng, 1, [0], 16, 1, hd, extra=len(rows), k_exp=e, v_exp=e)
        oK, oV = torch.zeros_like(X), torch.zeros_like(X)
        c.append(0, X, X, i32([0]), i32([len(rows)]))
        c.read(0, i32([0]), i32([len(rows)]), oK, oV)
        want = ko.kv4_values(host(X), e)
        assert np.array_equal(host(oK), want, equal_nan=True) and np.array_equal(host(oV), want, equal_nan=True)


def test_single_tokens_into_a_partly_filled_cell():
    rng = np.random.default_rng(3)
    c = make_cache(rng, 2, [0, 0], 16, 2, 128, extra=40)
    K, V = bf16(rng, (2, 40, 2, 128)), bf16(rng, (2, 40, 2, 128))
    for i in range(40):
        c.append(0, K[:, i:i + 1].contiguous(), V[:, i:i + 1].contiguous(), i32([i, i]), i32([1, i % 2]))
    oK, oV = torch.zeros_like(K), torch.zeros_like(V)
    c.read(0, i32([0, 0]), i32([40, 40]), oK, oV)
    want = ko.kv4_values(host(K), 0)
    assert np.array_equal(host(oK)[0], want[0])
    assert np.array_equal(host(oK)[1, 1::2], want[1, 1::2]) and (host(oK)[1, 0::2] == 0).all()


# ---------------------------------------------------------------- attention --

def check_attn(O, q, kc, vc, kb, vb, name=""):
    ref, Ac, Ab, smax = ko.paged_attn(q, kc, vc, kb, vb)
    keys = kc.shape[0] + kb.shape[0]
    vmax = max(np.abs(vc).max(initial=0), np.abs(vb).max(initial=0))
    tol = 2.0 ** -8 * np.abs(ref) + 1.01 * (2.0 ** -11 * Ac + 2.0 ** -8 * Ab) + \
        2.0 ** -18 * (1 + smax) * (Ac + Ab) + keys * 2.0 ** -32 * vmax + 1e-30
    err = np.abs(O - ref)
    assert (err <= tol).all(), (name, float((err / tol).max()), float(err.max()))


def run_attn(rng, c, lens, B, Hq, kscale=1.0, qscale=1.0, layer=0):
    K, V = fill(rng, c, layer, lens, kscale)
    Q = bf16(rng, (c.N, B, Hq, c.hd), qscale)
    Kb, Vb = bf16(rng, (c.N, B, c.Hkv, c.hd), kscale), bf16(rng, (c.N, B, c.Hkv, c.hd), kscale)
    O = c.attn(layer, Q, Kb, Vb)
    return K, V, Q, Kb, Vb, O


def check_all(c, K, V, Q, Kb, Vb, O, lens, k_exp=0, v_exp=0):
    K, V = ko.kv4_values(K, k_exp), ko.kv4_values(V, v_exp)
    Q, Kb, Vb, O = (host(x).astype(np.float64) for x in (Q, Kb, Vb, O))
    for n, l in enumerate(lens):
        check_attn(O[n], Q[n], K[n, :l], V[n, :l], Kb[n], Vb[n], f"sequence {n}")


@pytest.mark.parametrize("B,Hq,Hkv,hd,page,lens", [
    (1, 1, 1, 128, 16, [0]),                          # nothing cached: the token itself
    (1, 4, 1, 64, 16, [1]),
    (1, 8, 2, 128, 64, [15, 16, 17, 63, 64, 65, 0]),  # around cells, units and pages
    (1, 32, 8, 128, 16, [517]),
    (1, 3, 1, 64, 48, [1000, 0, 47, 48, 49]),
    (16, 8, 2, 128, 64, [129, 2, 300]),
    (16, 4, 4, 64, 32, [77, 640]),
    (5, 6, 2, 128, 32, [33, 95, 96]),                 # 15 rows: a row tile with one empty row
    (17, 3, 3, 64, 16, [31, 200]),
    (33, 8, 2, 128, 64, [100, 65]),
    (64, 2, 2, 64, 128, [130, 0]),                    # the largest block
    (64, 16, 2, 128, 16, [50]),                       # 512 rows of one head
    (8, 64, 8, 64, 32, [2000, 3, 1111]),
])
def test_attention_of_every_shape(B, Hq, Hkv, hd, page, lens):
    rng = np.random.default_rng(B * 1000 + Hq + hd + page)
    c = make_cache(rng, len(lens), lens, page, Hkv, hd)
    c.data.random_(0, 256)   # rows past a length and free pages hold anything, NaN scales among it
    out = run_attn(rng, c, lens, B, Hq)
    check_all(c, *out, lens)


@pytest.mark.parametrize("B,Hq,Hkv,hd", [(1, 8, 2, 128), (1, 8, 1, 64), (16, 4, 2, 128)])
def test_long_contexts_split_over_the_gpu(B, Hq, Hkv, hd):
    rng = np.random.default_rng(B + hd)
    lens = [40000, 1, 9999]
    c = make_cache(rng, 3, lens, 64, Hkv, hd)
    out = run_attn(rng, c, lens, B, Hq)
    check_all(c, *out, lens)


def test_many_short_sequences():
    rng = np.random.default_rng(11)
    lens = rng.integers(0, 40, 700)
    c = make_cache(rng, 700, lens, 16, 2, 64)
    out = run_attn(rng, c, lens, 1, 4)
    check_all(c, *out, lens)


@pytest.mark.parametrize("k_exp,v_exp,kscale,qscale", [(3, 3, 8.0, 1.0), (-4, -4, 2.0 ** -4, 16.0), (0, 0, 30.0, 10.0),
                                                       (0, 0, 1.0, 1e-6), (0, 0, 1.0, 3e4)])
def test_scales_of_keys_and_queries(k_exp, v_exp, kscale, qscale):
    # sharp and flat softmaxes, queries outside fp16's range, exponents of the pool
    rng = np.random.default_rng(7)
    lens = [333, 70]
    c = make_cache(rng, 2, lens, 32, 2, 128, k_exp=k_exp, v_exp=v_exp)
    out = run_attn(rng, c, lens, 3, 4, kscale, qscale)
    check_all(c, *out, lens, k_exp, v_exp)


def test_growing_maxima_rescale():
    # keys sorted by their score: every cell raises the running maximum
    rng = np.random.default_rng(5)
    lens, hd = [700], 64
    c = make_cache(rng, 1, lens, 16, 1, hd)
    K = torch.zeros((1, 700, 1, hd)).to(torch.bfloat16).cuda()
    K[0, :, 0, 0] = torch.linspace(-6, 6, 700).to(torch.bfloat16).cuda()
    V = bf16(rng, (1, 700, 1, hd))
    c.append(0, K, V, i32([0]), i32(lens))
    Q = torch.full((1, 1, 2, hd), 0.0).to(torch.bfloat16).cuda()
    Q[0, 0, 0, 0], Q[0, 0, 1, 0] = 200.0, -200.0
    Kb, Vb = bf16(rng, (1, 1, 1, hd)), bf16(rng, (1, 1, 1, hd))
    O = c.attn(0, Q, Kb, Vb)
    check_all(c, host(K).astype(np.float64), host(V).astype(np.float64), Q, Kb, Vb, O, lens)


def test_one_heavy_key_and_a_long_tail():
    # 60000 keys of weight 2^-15 each beside one: the tail carries most of the sum
    rng = np.random.default_rng(9)
    T, hd = 60000, 64
    c = make_cache(rng, 1, [T], 64, 1, hd)
    K = torch.zeros((1, T, 1, hd), dtype=torch.bfloat16, device="cuda")
    K[0, 123, 0, 0] = 6.0
    V = bf16(rng, (1, T, 1, hd)) + 1.0
    c.append(0, K, V, i32([0]), i32([T]))
    Q = torch.zeros((1, 1, 1, hd), dtype=torch.bfloat16, device="cuda")
    Q[..., 0] = 15 * 0.6931 * 8 / 6
    Kb = torch.zeros((1, 1, 1, hd), dtype=torch.bfloat16, device="cuda")
    O = c.attn(0, Q, Kb, bf16(rng, (1, 1, 1, hd)) * 0)
    check_all(c, host(K).astype(np.float64), host(V).astype(np.float64), Q, Kb, torch.zeros_like(Kb), O, [T])


def test_nan_in_a_held_row_shows_and_past_the_length_does_not():
    rng = np.random.default_rng(2)
    lens = [50, 50, 50]
    c = make_cache(rng, 3, lens, 16, 1, 128, extra=14)
    K, V = bf16(rng, (3, 64, 1, 128)), bf16(rng, (3, 64, 1, 128))
    K[0, 50:] = float("nan")
    V[0, 50:] = float("inf")
    K[1, 20, 0, 5] = float("nan")
    V[2, 49, 0, 0] = float("inf")
    c.append(0, K, V, i32([0] * 3), i32([64] * 3))
    Q, Kb, Vb = bf16(rng, (3, 2, 1, 128)), bf16(rng, (3, 2, 1, 128)), bf16(rng, (3, 2, 1, 128))
    O = host(c.attn(0, Q, Kb, Vb))
    kd, vd = ko.kv4_values(host(K), 0), ko.kv4_values(host(V), 0)
    check_attn(O[0], host(Q)[0], kd[0, :50], vd[0, :50], host(Kb)[0], host(Vb)[0])
    assert np.isnan(O[1]).all()
    assert np.isnan(O[2, :, :, :16]).all() and np.isfinite(O[2, :, :, 16:]).all()   # one group of values


def test_lengths_and_pages_out_of_range_are_reported():
    rng = np.random.default_rng(4)
    lens = [40, 40, 40]
    c = make_cache(rng, 3, lens, 16, 1, 64)
    out = run_attn(rng, c, lens, 1, 2)
    check_all(c, *out, lens)
    K, V, Q, Kb, Vb, O = out
    c.table[1, 1] = c.num_pages + 5    # read as page 0
    c.len[2] = 1 << 30                 # read as the table's capacity
    O2 = c.attn(0, Q, Kb, Vb)
    assert dfl.dfl_get_device_error() == 1
    assert torch.equal(O2[0], O[0])
    one = torch.zeros((3, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    before = c.data.clone()
    c.append(0, one, one, i32([0, 20, 0]), i32([0, 1, 2]))       # a page, a count out of range
    assert dfl.dfl_get_device_error() == 1 and torch.equal(c.data, before)
    c.append(0, one, one, i32([c.max_pages * 16, -1, 0]), i32([1, 1, 0]))
    assert dfl.dfl_get_device_error() == 1 and torch.equal(c.data, before)
    c.append(0, one, one, i32([-1, -1, -1]), i32([1, 1, 1]))     # skipped, not an error
    assert dfl.dfl_get_device_error() == 0 and torch.equal(c.data, before)


def test_results_repeat_and_do_not_depend_on_pages_or_stream():
    rng = np.random.default_rng(6)
    lens = [3000, 500, 77, 1500]
    c = make_cache(rng, 4, lens, 32, 2, 128)
    K, V, Q, Kb, Vb, O = run_attn(rng, c, lens, 4, 8)
    O = O.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        O2 = c.attn(0, Q, Kb, Vb)
    side.synchronize()
    assert torch.equal(O, O2)
    c2 = make_cache(rng, 4, lens, 64, 2, 128)
    k = torch.from_numpy(K).to(torch.bfloat16).cuda()
    v = torch.from_numpy(V).to(torch.bfloat16).cuda()
    c2.append(0, k, v, i32([0] * 4), i32(lens))
    assert torch.equal(c2.attn(0, Q, Kb, Vb), O)


# --------------------------------------------------------- page operations --

def check_book(c, b):
    assert np.array_equal(host(c.table), b.table)
    assert np.array_equal(host(c.len), b.len)
    assert np.array_equal(host(c.ref), b.ref)


@pytest.mark.parametrize("N,num_pages,page,max_pages,layers", [(1, 5, 16, 4, 1), (7, 40, 16, 12, 3), (40, 1500, 32, 90, 2),
                                                               (1100, 3001, 16, 6, 1)])
def test_page_operations_against_lists(N, num_pages, page, max_pages, layers):
    rng = np.random.default_rng(N)
    c = dfl.PagedCache(layers, num_pages, page, 1, 64, N, max_pages)
    c.data.random_(0, 256)
    b = ko.PageBook(host(c.table), host(c.len), host(c.ref), page)
    data = host(c.data).copy()
    cap = max_pages * page
    for step in range(12):
        m = rng.integers(0, max(2, cap // 3), N)
        m[rng.random(N) < 0.3] = 0
        m = np.minimum(m, cap - b.len)
        start = host(c.reserve(i32(m)))
        want, copies = b.reserve(m)
        for s, d in copies:
            data[:, d] = data[:, s]
        assert np.array_equal(start, want)
        check_book(c, b)
        assert np.array_equal(host(c.data), data)
        parent = np.where(rng.random(N) < 0.6, np.arange(N), rng.integers(-1, N, N))
        keep = None if step % 3 == 0 else np.where(rng.random(N) < 0.5, -1, rng.integers(0, cap + 5, N))
        c.remap(i32(parent), None if keep is None else i32(keep))
        b.remap(parent, keep)
        check_book(c, b)
        if step % 2:
            mp, live = c.compact()
            want, n_live, moves = b.compact()
            for s, d in moves:
                data[:, d] = data[:, s]
            assert np.array_equal(host(mp), want) and int(live) == n_live
            check_book(c, b)
            assert np.array_equal(host(c.data), data)
    assert dfl.dfl_get_device_error() == 0


def test_a_large_pool():
    # more pages than one pass of the planning block covers
    rng = np.random.default_rng(0)
    num, N = 70001, 3
    c = dfl.PagedCache(1, num, 16, 1, 64, N, 30000)
    ref = (rng.random(num) < 0.7).astype(np.int32)
    c.ref.copy_(i32(ref))
    b = ko.PageBook(host(c.table), host(c.len), ref, 16)
    m = [16 * 9000 - 3, 5, 16 * 11000]
    assert np.array_equal(host(c.reserve(i32(m))), b.reserve(m)[0])
    check_book(c, b)
    data = torch.randint(0, 256, c.data.shape, dtype=torch.uint8, device="cuda")
    c.data.copy_(data)
    mp, live = c.compact()
    want, n_live, moves = b.compact()
    s, d = (torch.tensor(x, device="cuda") for x in zip(*moves))
    data[:, d] = data[:, s]
    assert np.array_equal(host(mp), want) and int(live) == n_live and torch.equal(c.data, data)
    check_book(c, b)


def test_counts_of_other_holders_survive():
    c = dfl.PagedCache(1, 8, 16, 1, 64, 2, 4)
    c.reserve(i32([20, 0]))
    c.ref[1] += 1                       # a holder outside the table
    c.remap(i32([-1, 1]))
    assert host(c.ref).tolist() == [0, 1, 0, 0, 0, 0, 0, 0]
    mp, live = c.compact()
    assert host(c.ref).tolist() == [1, 0, 0, 0, 0, 0, 0, 0] and host(mp).tolist() == [-1, 0] + [-1] * 6
    assert int(live) == 1


def test_page_arguments_out_of_range_are_reported():
    c = dfl.PagedCache(1, 8, 16, 1, 64, 3, 2)
    s = c.reserve(i32([33, -1, 5]))     # past the table, negative, fine
    assert host(s).tolist() == [-1, -1, 0] and host(c.len).tolist() == [0, 0, 5]
    assert dfl.dfl_get_device_error() == 1
    c.remap(i32([2, 7, 2]))             # a parent that is no sequence: the row stays
    assert host(c.len).tolist() == [5, 0, 5] and host(c.ref)[0] == 2
    assert dfl.dfl_get_device_error() == 1


# ------------------------------------------------------- the run of a server --

def _serve(c, rng, steps, check, graph=False):
    """Reserve, append, attend, roll back, fork, compact, against lists of rows per sequence."""
    N, Hkv, hd, B, Hq = c.N, c.Hkv, c.hd, 3, 2 * c.Hkv
    rows = [np.zeros((0, Hkv, hd)) for _ in range(N)], [np.zeros((0, Hkv, hd)) for _ in range(N)]
    cap, R = c.max_pages * c.page, 24
    for step in range(steps):
        m = np.minimum(rng.integers(0, R + 1, N), [cap - len(r) for r in rows[0]])
        K, V = bf16(rng, (N, R, Hkv, hd)), bf16(rng, (N, R, Hkv, hd))
        start, n_new = c.reserve(i32(m)), i32(m)
        for l in range(c.layers):
            c.append(l, K, V, start, n_new)
        s = host(start)
        for n in range(N):
            if s[n] >= 0:
                for r, x in zip(rows, (K, V)):
                    r[n] = np.concatenate([r[n], ko.kv4_values(host(x)[n, :m[n]], 0)])
        Q, Kb, Vb = bf16(rng, (N, B, Hq, hd)), bf16(rng, (N, B, Hkv, hd)), bf16(rng, (N, B, Hkv, hd))
        O = host(c.attn(step % c.layers, Q, Kb, Vb))
        for n in range(N):
            check_attn(O[n], host(Q)[n], rows[0][n], rows[1][n], host(Kb)[n], host(Vb)[n], f"step {step} sequence {n}")
        parent = np.where(rng.random(N) < 0.7, np.arange(N), rng.integers(-1, N, N))
        keep = np.array([max(0, len(rows[0][p]) - int(rng.integers(0, 9))) if p >= 0 else 0 for p in parent])
        c.remap(i32(parent), i32(keep))
        for r in rows:
            r[:] = [r[p][:k] if p >= 0 else r[0][:0] for p, k in zip(parent, keep)]
        if step % 3 == 2:
            c.compact()
    assert host(c.len).tolist() == [len(r) for r in rows[0]]


@pytest.mark.parametrize("hd,page", [(64, 16), (128, 32)])
def test_serving_run(hd, page):
    c = dfl.PagedCache(2, 6 * 160 // page, page, 2, hd, 6, 160 // page)
    _serve(c, np.random.default_rng(hd), 9, None)
    assert dfl.dfl_get_device_error() == 0


def test_captured_run_replays():
    rng = np.random.default_rng(8)
    N, Hkv, hd, R, B = 4, 2, 128, 8, 4
    c = dfl.PagedCache(1, 64, 16, Hkv, hd, N, 16)
    K, V, n_new = bf16(rng, (N, R, Hkv, hd)), bf16(rng, (N, R, Hkv, hd)), i32([8, 3, 0, 5])
    Q, Kb, Vb = bf16(rng, (N, B, 4, hd)), bf16(rng, (N, B, Hkv, hd)), bf16(rng, (N, B, Hkv, hd))
    parent, O = i32([1, 1, 2, 3]), torch.empty_like(Q)

    def step():
        start = c.reserve(n_new)
        c.append(0, K, V, start, n_new)
        c.attn(0, Q, Kb, Vb, out=O)
        c.remap(parent)
        c.compact()

    def reset():
        c.book.zero_()
        c.table.fill_(-1)

    step()
    torch.cuda.synchronize()
    reset()
    eager = []
    for _ in range(4):
        step()
        eager.append((O.clone(), c.book.clone()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    reset()
    for o, book in eager:
        g.replay()
        assert torch.equal(O, o) and torch.equal(c.book, book)


# -------------------------------------------------------------- draft step --

def _models(hd, Hq, Hkv, B, page, num_pages, C=128, N=3, F=0):
    from dfl_synth import (gen_block_init, gen_ffn_gains, gen_gains, gen_layer_weights, gen_lm_head, gen_mix_logits)
    w = Workload("paged", N=N, d=256, Hq=Hq, Hkv=Hkv, hd=hd, D=2, L=3, B=B, C=C, V=1500, dtype="bf16", seed=31, R=24, F=F)
    shape = dfl.DraftShape(N=N, d=w.d, Hq=Hq, Hkv=Hkv, hd=hd, D=2, L=3, B=B, C=C, V=w.V, dtype="bf16", F=F)
    g_mix, g_blk, g_fin = gen_gains(w)
    layers = [gen_layer_weights(w, l) for l in range(2)]
    W_lm = torch.from_numpy(gen_lm_head(w, as_bits=True).view(np.int16)).view(torch.bfloat16)
    args = (gen_mix_logits(w), g_mix, g_blk, g_fin, layers, W_lm)
    kw = dict(ffn_gain=gen_ffn_gains(w)) if F else {}
    return (w, dfl.CachedDraftModel(shape, 24, *args, **kw),
            dfl.PagedDraftModel(shape, 24, num_pages, *args, page=page, **kw),
            torch.from_numpy(gen_block_init(w)).cuda())


@pytest.mark.parametrize("hd,Hq,Hkv,B,page,F", [(64, 4, 2, 8, 16, 0), (128, 8, 2, 16, 32, 512), (128, 2, 1, 2, 64, 0)])
def test_paged_step_against_the_contiguous_cache(hd, Hq, Hkv, B, page, F):
    """The pages hold exactly the 4-bit values of the rows that the bf16 cache holds; over those values both steps agree."""
    w, m16, m4, X0 = _models(hd, Hq, Hkv, B, page, 60, F=F)
    rng = np.random.default_rng(hd)
    for n_new in ([24, 5, 0], [7, 24, 24], [24, 1, 13]):
        H = bf16(rng, (w.L, w.N * 24, w.d))
        m16.step(H, X0, i32(n_new))
        m4.step(H, X0, i32(n_new))
    lens = host(m4.cache.len)
    assert lens.tolist() == host(m16.ctx_len).tolist() == [55, 30, 37]
    for l in range(w.D):
        K, V = (torch.zeros((w.N, w.C, Hkv, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        m4.cache.read(l, i32([0, 0, 0]), m4.cache.len, K, V)
        for got, cache in ((K, m16.K_cache), (V, m16.V_cache)):
            for n in range(w.N):
                assert np.array_equal(host(got)[n, :lens[n]], ko.kv4_values(host(cache[l, n, :lens[n]]), 0))
        m16.K_cache[l].copy_(K)
        m16.V_cache[l].copy_(V)
    H = bf16(rng, (w.L, w.N * 24, w.d))
    for m in (m16, m4):
        m.want_logits()
        m.step(H, X0, i32([0, 0, 0]))
    assert_bf16_close(host(m4.Xb) - host(X0), host(m16.Xb) - host(X0), "Xb")
    assert_bf16_close(host(m4.logits), host(m16.logits), "logits")
    assert np.array_equal(host(m4.draft), host(m4.logits).reshape(w.N, B - 1, -1).argmax(-1))


def test_paged_step_without_room_and_through_a_fork():
    w, _, m, X0 = _models(64, 4, 2, 8, 16, 4)      # 4 pages in all
    rng = np.random.default_rng(1)
    H = bf16(rng, (w.L, w.N * 24, w.d))
    m.step(H, X0, i32([20, 24, 3]))                # two pages, two pages, none left
    assert host(m.cache.start).tolist() == [0, 0, -1] and host(m.cache.len).tolist() == [20, 24, 0]
    assert np.isfinite(host(m.Xb)).all()
    m.cache.remap(i32([0, -1, 0]))                 # the first forks into the third, the second ends
    m.step(H, X0, i32([2, 0, 2]))                  # both copy the shared last page
    assert host(m.cache.start).tolist() == [20, 0, 20] and host(m.cache.len).tolist() == [22, 0, 22]
    K, V = (torch.zeros((3, 32, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.cache.read(1, i32([0, 0, 0]), m.cache.len, K, V)
    assert torch.equal(K[0, :20], K[2, :20]) and not torch.equal(K[0, 20:22], K[2, 20:22])
    assert dfl.dfl_get_device_error() == 0


def test_paged_step_from_host_and_in_a_graph():
    w, _, m, X0 = _models(128, 8, 2, 16, 32, 60)
    rng = np.random.default_rng(2)
    H, n_new = bf16(rng, (w.L, w.N * 24, w.d)), i32([24, 9, 1])
    out, _ = m.step_from_host(H.cpu().pin_memory(), X0.cpu().pin_memory(), n_new.cpu().pin_memory())
    xb, draft = m.Xb.clone(), m.draft.clone()
    assert torch.equal(out["draft"], draft.cpu()) and out["start"].tolist() == [0, 0, 0]
    m.cache.remap(i32([-1, -1, -1]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.step(H, X0, n_new)
    for _ in range(2):
        m.Xb.zero_()
        g.replay()
        assert torch.equal(m.Xb, xb) and torch.equal(m.draft, draft)
        m.cache.remap(i32([-1, -1, -1]))


def test_arguments_of_the_python_calls_are_checked():
    c = dfl.PagedCache(1, 8, 16, 2, 64, 2, 4)
    t = lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")
    K = t(2, 3, 2, 64)
    for bad in (lambda: c.append(0, K.float(), K, c.len, c.len), lambda: c.append(0, K, t(2, 4, 2, 64), c.len, c.len),
                lambda: c.append(0, t(2, 3, 4, 64)[:, :, ::2], K, c.len, c.len), lambda: c.reserve(c.len.long()),
                lambda: c.reserve(c.len[:1]), lambda: c.attn(0, t(2, 1, 4, 64), t(2, 2, 2, 64), t(2, 1, 2, 64)),
                lambda: c.attn(0, t(1, 1, 4, 64), t(2, 1, 2, 64), t(2, 1, 2, 64)), lambda: c.remap(c.len.cpu()),
                lambda: dfl.PagedCache(1, 8, 20, 2, 64, 2, 4), lambda: dfl.PagedCache(1, 0, 16, 2, 64, 2, 4)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dfl.DflError):
        c.append(1, K, K, c.len, c.len)
