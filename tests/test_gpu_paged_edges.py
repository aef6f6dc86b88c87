"""The paged 4-bit context cache where its calls can go wrong (GPU).

Every count of query rows around the kernels' tiles, lengths around cells,
units and halves of units, lines of work that are cut and that are not, guard
bands around what the calls write, pools past 2^31 bytes, the block's own rows
past fp16's range, infinities and NaN, and calls of two caches on two streams.

Attention's bound: bf16 output (2^-8 of the value), fp16 weights (2^-11), fp32
scores and exponentials (2^-18 of the weight times 1 + the largest score: 128
products, the base-2 exponential's 2^-22, a query's fp16 form), weights below
fp16's normal range (2^-32 a key of the largest value), and the block's own
rows in fp16 units of the pool's power of two (2^-25 of a unit each).
"""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_dfl_gb300 as dfl
from gpu_util import host
from oracle import kv4_oracle as ko
from test_gpu_guard_bands import Guarded
from test_gpu_paged import bf16, fill, i32, make_cache, run_attn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.build()
    dfl.load()
    torch.cuda.set_device(0)
    yield
    assert dfl.dfl_get_device_error() == 0


def check(c, K, V, Q, Kb, Vb, O, lens, k_exp=0, v_exp=0, which=None):
    K, V = ko.kv4_values(K, k_exp), ko.kv4_values(V, v_exp)
    Q, Kb, Vb, O = (host(x).astype(np.float64) for x in (Q, Kb, Vb, O))
    for n in range(len(lens)) if which is None else which:
        kb = np.clip(Kb[n], -65504 * 2.0 ** k_exp, 65504 * 2.0 ** k_exp)
        vb = np.clip(Vb[n], -65504 * 2.0 ** v_exp, 65504 * 2.0 ** v_exp)
        ref, Ac, Ab, smax = ko.paged_attn(Q[n], K[n, :lens[n]], V[n, :lens[n]], kb, vb)
        vmax = max(np.abs(V[n, :lens[n]]).max(initial=0), np.abs(vb).max())
        tol = 2.0 ** -8 * np.abs(ref) + (1.01 * 2.0 ** -11 + 2.0 ** -18 * (1 + smax)) * (Ac + Ab) + \
            (lens[n] + kb.shape[0]) * 2.0 ** -32 * vmax + 2.0 ** (v_exp - 25) + 1e-30
        err = np.abs(O[n] - ref)
        assert (err <= tol).all(), (n, lens[n], float((err / tol).max()))


EDGES = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 160, 191, 192, 193, 255, 256, 257]


@pytest.mark.parametrize("B,Hq,Hkv", [
    (1, 2, 2), (2, 4, 1), (3, 6, 2), (16, 1, 1),     # 1, 8, 9 and 16 rows of a head
    (17, 1, 1), (1, 32, 1), (9, 14, 2), (16, 8, 2),  # 17, 32, 63 and 64
    (13, 10, 2), (1, 71, 1), (64, 2, 1),             # 65, 71 and 128
    (43, 3, 1), (64, 5, 1)])                         # 129 and 320
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_around_every_edge(B, Hq, Hkv, hd):
    rng = np.random.default_rng(B * 100 + Hq + hd)
    c = make_cache(rng, len(EDGES), EDGES, 48, Hkv, hd)
    c.data.random_(0, 256)   # what lies past a length is anything, NaN scales among it
    check(c, *run_attn(rng, c, EDGES, B, Hq), EDGES)


@pytest.mark.parametrize("B,Hq,Hkv,hd,lens", [
    (16, 32, 8, 128, [200] * 38),                    # as many triples as ranges
    (16, 32, 8, 128, [200] * 39),                    # one more sequence: the line is cut
    (16, 32, 8, 128, [70] * 20 + [3000]),            # a long one among short ones
    (16, 16, 4, 64, [1] * 100),
    (8, 64, 8, 64, [20000, 5]),
    (1, 32, 8, 128, [100] * 76),                     # single tokens: 608 triples of equal length
    (1, 32, 8, 128, [100] * 77),
    (1, 8, 1, 128, [2000] + [0] * 150),
    (2, 4, 1, 64, [7] * 1100),                       # more sequences than a block has threads
    (4, 8, 1, 64, [9] * 1100),
])
def test_attention_over_cut_and_uncut_lines(B, Hq, Hkv, hd, lens):
    rng = np.random.default_rng(len(lens) + B)
    c = make_cache(rng, len(lens), lens, 64, Hkv, hd)
    which = sorted({0, 1, len(lens) // 2, len(lens) - 2, len(lens) - 1, int(np.argmax(lens))} & set(range(len(lens))))
    check(c, *run_attn(rng, c, lens, B, Hq), lens, which=which)


@pytest.mark.parametrize("B,Hq", [(16, 4), (16, 8)])
@pytest.mark.parametrize("hd", [64, 128])
def test_maxima_that_grow_fall_and_jump(B, Hq, hd):
    # keys sorted by their score, rows that see them rise and fall by much or little, and one key far above the rest
    rng = np.random.default_rng(hd + Hq)
    T, lens = 1500, [1500, 700]
    c = make_cache(rng, 2, lens, 16, 1, hd)
    K = torch.zeros((2, T, 1, hd), dtype=torch.bfloat16, device="cuda")
    K[0, :, 0, 0] = torch.linspace(-6, 6, T).to(torch.bfloat16).cuda()
    K[1, :, 0, 0] = (torch.rand(T, device="cuda") * 0.2).to(torch.bfloat16)
    K[1, 333, 0, 0], K[1, 600, 0, 0] = 6.0, -6.0
    V = bf16(rng, (2, T, 1, hd))
    c.append(0, K, V, i32([0, 0]), i32(lens))
    Q = torch.zeros((2, B, Hq, hd), dtype=torch.bfloat16, device="cuda")
    Q[..., 0] = torch.tensor([200.0, -200.0, 30.0, -30.0, 6.0, -6.0, 1.0, 0.0], device="cuda").repeat(B * Hq // 8).view(B, Hq)
    Kb, Vb = bf16(rng, (2, B, 1, hd)), bf16(rng, (2, B, 1, hd))
    O = c.attn(0, Q, Kb, Vb)
    check(c, host(K).astype(np.float64), host(V).astype(np.float64), Q, Kb, Vb, O, lens)


@pytest.mark.parametrize("B,Hq", [(3, 2), (16, 8)])
@pytest.mark.parametrize("hd", [64, 128])
def test_own_rows_past_fp16_and_below_it(B, Hq, hd):
    rng = np.random.default_rng(hd + B)
    for e in (0, 4, -6):
        lens = [20, 0]
        c = make_cache(rng, 2, lens, 16, 2, hd, k_exp=e, v_exp=e)
        K, V = fill(rng, c, 0, lens, 2.0 ** e)
        Q, Kb, Vb = bf16(rng, (2, B, Hq, hd)), bf16(rng, (2, B, 2, hd), 2.0 ** e), bf16(rng, (2, B, 2, hd), 2.0 ** e)
        Q[..., 0], Kb[:, 0, 0, 0] = 2.0 ** -17 * 2.0 ** -e, 3e5 * 2.0 ** e
        Vb[:, 0, 0, 1], Vb[:, 1, 0, 1], Vb[:, 0, 1, 2], Vb[:, 2, 1, :] = 1e9, -1e9, 3e38, 2.0 ** (e - 20)
        check(c, K, V, Q, Kb, Vb, c.attn(0, Q, Kb, Vb), lens, e, e)


@pytest.mark.parametrize("B,Hq", [(3, 2), (16, 8)])
def test_infinities_and_nan_of_own_rows_show(B, Hq):
    rng = np.random.default_rng(B)
    lens = [200, 200, 200, 200]
    c = make_cache(rng, 4, lens, 16, 2, 128)
    K, V, Q, Kb, Vb, O = run_attn(rng, c, lens, B, Hq)
    inf, nan = float("inf"), float("nan")
    Kb[0, 0, 0, 5], Vb[1, 2, 1, 7], Vb[2, 0, 0, 0] = nan, -inf, nan
    O2 = host(c.attn(0, Q, Kb, Vb))
    G, O = Hq // 2, host(O)
    assert np.isnan(O2[0, :, :G]).all() and np.array_equal(O2[0, :, G:], O[0, :, G:])
    assert (O2[1, :, G:, 7] == -inf).all() and np.isnan(O2[2, :, :G, 0]).all()
    for n, h, d in ((1, slice(G, None), 7), (2, slice(0, G), 0)):
        keep = np.arange(128) != d
        assert np.array_equal(O2[n, :, h][..., keep], O[n, :, h][..., keep])
    assert np.array_equal(O2[3], O[3])


@pytest.mark.parametrize("B,Hq", [(16, 8), (64, 4)])
def test_pages_and_lengths_out_of_range_with_many_rows(B, Hq):
    rng = np.random.default_rng(4)
    lens = [400, 400, 400]
    c = make_cache(rng, 3, lens, 16, 2, 64)
    K, V, Q, Kb, Vb, O = run_attn(rng, c, lens, B, Hq)
    O = O.clone()
    c.table[1, 1], c.table[1, 7] = c.num_pages, -1   # read as page 0
    c.len[2] = -5                                    # read as no token
    O2 = c.attn(0, Q, Kb, Vb)
    assert dfl.dfl_get_device_error() == 1
    assert torch.equal(O2[0], O[0])
    check(c, K, V, Q, Kb, Vb, O2, [400, 400, 0], which=[2])


def _guarded(c):
    """The cache's pool and tables between guard bands."""
    g = {k: Guarded(tuple(x.shape), x.dtype, x) for k, x in (("data", c.data), ("table", c.table), ("len", c.len),
                                                            ("ref", c.ref))}
    pool = dfl._lib.Kv4Pool(g["data"].t.data_ptr(), c.num_pages * c.page_bytes, c.layers, c.num_pages, c.page, c.Hkv, c.hd,
                            0, 0)
    pages = dfl._lib.Pages(g["table"].t.data_ptr(), g["len"].t.data_ptr(), g["ref"].t.data_ptr(), c.N, c.max_pages)
    return g, pool, pages


@pytest.mark.parametrize("B,Hq,Hkv,hd,N", [(1, 6, 2, 128, 5), (3, 9, 3, 64, 40), (16, 8, 2, 128, 5), (13, 10, 2, 64, 40),
                                           (40, 6, 2, 128, 3)])
def test_attention_writes_only_its_output_and_workspace(B, Hq, Hkv, hd, N):
    rng = np.random.default_rng(N + B)
    lens = rng.integers(0, 700, N)
    c = make_cache(rng, N, lens, 32, Hkv, hd)
    K, V, Q, Kb, Vb, O = run_attn(rng, c, lens, B, Hq)
    g, pool, pages = _guarded(c)
    need = dfl.workspace_size(dfl.DFL_OP_KV4_ATTN, N=N, B=B, Hq=Hq, Hkv=Hkv, hd=hd)
    ws, out = Guarded((max(need, 16),), torch.uint8), Guarded(tuple(O.shape), torch.bfloat16)
    for byte in (0xFF, 0x00):   # nothing is read from the scratch that the call has not written
        ws.t.fill_(byte)
        out.t.zero_()
        dfl.dfl_kv4_attn(pool, 0, pages, Q, Kb, Vb, B, Hq, out.t, ws.t, need)
        assert torch.equal(out.t, O)
    for k, x in list(g.items()) + [("workspace", ws), ("out", out)]:
        x.check(k)
    assert all(torch.equal(g[k].t, getattr(c, k)) for k in g)


@pytest.mark.parametrize("Hkv,hd,page,R", [(3, 64, 16, 7), (40, 128, 32, 3), (2, 128, 16, 50), (1, 64, 1024, 1)])
def test_append_and_read_write_only_the_rows(Hkv, hd, page, R):
    # 40 heads of 128: a row has more groups than a block threads
    rng = np.random.default_rng(Hkv)
    N = 4
    start, cnt = np.array([0, 5, -1, 30]), np.array([R, R // 2, R, R])
    c = make_cache(rng, N, np.maximum(start, 0), page, Hkv, hd, extra=R)
    c.data.random_(0, 256)
    g, pool, pages = _guarded(c)
    K, V = bf16(rng, (N, R, Hkv, hd)), bf16(rng, (N, R, Hkv, hd))
    dfl.dfl_kv4_append(pool, 0, pages, i32(start), i32(cnt), R, K, V)
    oK, oV = Guarded(tuple(K.shape), torch.bfloat16), Guarded(tuple(K.shape), torch.bfloat16)
    oK.t.fill_(3.0)
    oV.t.fill_(3.0)
    dfl.dfl_kv4_read(pool, 0, pages, i32(start), i32(cnt), R, oK.t, oV.t)
    for x, o in ((K, oK), (V, oV)):
        want = ko.kv4_values(host(x), 0)
        for n in range(N):
            m = cnt[n] if start[n] >= 0 else 0
            assert np.array_equal(host(o.t)[n, :m], want[n, :m]) and (host(o.t)[n, m:] == 3.0).all()
    for k, x in list(g.items()) + [("K", oK), ("V", oV)]:
        x.check(k)
    # bytes of the pool that differ: at most those of the written rows
    rows = sum(int(m) for s, m in zip(start, cnt) if s >= 0)
    assert int((g["data"].t != c.data).sum()) <= rows * Hkv * 18 * hd // 16


@pytest.mark.parametrize("N,page,num_pages,max_pages", [(5, 16, 60, 9), (1500, 16, 4000, 5), (40, 32, 9000, 200)])
def test_page_operations_write_only_theirs(N, page, num_pages, max_pages):
    # 1500 sequences: more than the planning block has threads; 40 * 180 pages: more than it keeps in shared memory
    rng = np.random.default_rng(N)
    c = dfl.PagedCache(2, num_pages, page, 1, 64, N, max_pages)
    c.data.random_(0, 256)
    g, pool, pages = _guarded(c)
    b = ko.PageBook(host(c.table), host(c.len), host(c.ref), page)
    data = g["data"].t.clone()
    cap = max_pages * page

    def ws_of(op, **shape):
        need = dfl.workspace_size(op, **shape)
        return Guarded((max(need, 16),), torch.uint8), need

    def same():
        assert np.array_equal(host(g["table"].t), b.table) and np.array_equal(host(g["len"].t), b.len)
        assert np.array_equal(host(g["ref"].t), b.ref)
        for k, x in g.items():
            x.check(k)

    for big in (0.9, 0.05, 0.05):
        new = np.minimum(rng.integers(0, max(2, int(cap * big)), N), cap - b.len)
        start = Guarded((N,), torch.int32)
        ws, need = ws_of(dfl.DFL_OP_PAGES_RESERVE, N=N, pages=num_pages)
        dfl.dfl_pages_reserve(pool, pages, i32(new), start.t, ws.t, need)
        want, copies = b.reserve(new)
        assert np.array_equal(host(start.t), want)
        for s, d in copies:
            data[:, d] = data[:, s]
        assert torch.equal(g["data"].t, data)
        ws.check("reserve workspace")
        start.check("start")
        same()
        parent, keep = rng.integers(-1, N, N), rng.integers(-1, cap + 1, N)
        ws, need = ws_of(dfl.DFL_OP_PAGES_REMAP, N=N, pages=max_pages)
        dfl.dfl_pages_remap(pool, pages, i32(parent), i32(keep), ws.t, need)
        b.remap(parent, keep)
        ws.check("remap workspace")
        same()
        mp, live = Guarded((num_pages,), torch.int32), Guarded((1,), torch.int32)
        ws, need = ws_of(dfl.DFL_OP_PAGES_COMPACT, pages=num_pages)
        dfl.dfl_pages_compact(pool, pages, mp.t, live.t, ws.t, need)
        want, n_live, moves = b.compact()
        for s, d in moves:
            data[:, d] = data[:, s]
        assert np.array_equal(host(mp.t), want) and int(live.t) == n_live
        assert torch.equal(g["data"].t, data)
        ws.check("compact workspace")
        mp.check("map")
        live.check("live")
        same()


@pytest.mark.parametrize("N,Hkv,layers", [(1, 1, 1), (6, 2, 3), (28, 2, 2), (29, 2, 2), (200, 1, 1)])
def test_shared_last_pages_are_copied(N, Hkv, layers):
    # pages of 4,608 bytes with two heads: 28 sequences in two layers are the most that the planning block copies itself
    rng = np.random.default_rng(N)
    page, num = 32, 4 * N + 5
    c = dfl.PagedCache(layers, num, page, Hkv, 64, N, 3)
    c.data.random_(0, 256)
    b = ko.PageBook(host(c.table), host(c.len), host(c.ref), page)
    data = c.data.clone()
    first = np.zeros(N, int)
    first[0] = 40
    for new in (first, None, rng.integers(0, 20, N), rng.integers(0, 20, N)):
        if new is None:   # everyone forks sequence 0
            c.remap(i32(np.zeros(N)))
            b.remap(np.zeros(N, int))
            continue
        new = np.minimum(new, 96 - b.len)
        start, copies = b.reserve(new)
        assert np.array_equal(host(c.reserve(i32(new))), start)
        for s, d in copies:
            data[:, d] = data[:, s]
        assert torch.equal(c.data, data)
        assert np.array_equal(host(c.table), b.table) and np.array_equal(host(c.ref), b.ref)


@pytest.mark.parametrize("N,max_pages", [(1, 1), (3, 7), (9, 33), (4096, 1), (8, 512), (8, 513), (700, 600)])
def test_remap_of_tables_of_every_size(N, max_pages):
    # up to 4,096 entries are one block's
    rng = np.random.default_rng(N)
    page, num = 16, 5000
    c = dfl.PagedCache(1, num, page, 1, 64, N, max_pages)
    length = rng.integers(0, max_pages * page + 1, N)
    table = rng.integers(0, num, (N, max_pages))
    table[np.arange(max_pages)[None] * page >= length[:, None]] = -1
    ref = np.bincount(table[table >= 0], minlength=num)
    for x, v in ((c.table, table), (c.len, length), (c.ref, ref)):
        x.copy_(i32(v))
    b = ko.PageBook(table, length, ref, page)
    for i in range(3):
        parent, keep = rng.integers(-1, N, N), rng.integers(-1, max_pages * page + 9, N)
        if i == 1:
            parent[0] = N   # no sequence: the row stays
        c.remap(i32(parent), None if i == 2 else i32(keep))
        if i == 1:
            assert dfl.dfl_get_device_error() == 1
            parent[0], keep[0] = 0, -1
        b.remap(parent, None if i == 2 else keep)
        assert np.array_equal(host(c.table), b.table) and np.array_equal(host(c.len), b.len)
        assert np.array_equal(host(c.ref), b.ref)


@pytest.mark.parametrize("B,Hq", [(1, 16), (16, 16)])
def test_a_pool_past_2_31_bytes(B, Hq):
    rng = np.random.default_rng(B)
    page, Hkv, hd, num, lens = 64, 4, 128, 65000, [900, 130]
    c = dfl.PagedCache(2, num, page, Hkv, hd, 2, 20)    # 36,864 bytes a page, 2.4e9 a layer
    table = np.full((2, 20), -1)
    table[0, :15], table[1, :3] = num - 1 - np.arange(15), num - 40 + np.arange(3)
    c.table.copy_(i32(table))
    c.len.copy_(i32(lens))
    for layer in (0, 1):
        out = run_attn(rng, c, lens, B, Hq, layer=layer)
        check(c, *out, lens)
        K, V = out[:2]
        oK, oV = (torch.zeros(K.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        c.read(layer, i32([0, 0]), i32(lens), oK, oV)
        assert np.array_equal(host(oK)[0], ko.kv4_values(K, 0)[0]) and np.array_equal(host(oV)[0], ko.kv4_values(V, 0)[0])
    # copies and moves up there: sequence 1 forks into its shared last page, then all moves to the low end
    c.ref.copy_(i32(np.bincount(table[table >= 0], minlength=num)))
    c.ref[num - 38] += 1
    c.ref[:num - 60] = 1
    before = c.data[:, table[1, 2]].clone()
    start = c.reserve(i32([0, 1]))
    t = host(c.table)
    assert host(start).tolist() == lens and t[1, 2] == num - 60
    assert torch.equal(c.data[:, num - 60], before)
    c.ref[:num - 60] = 0
    first = c.data[:, num - 15].clone()
    mp, live = c.compact()
    assert int(live) == 15 + 3 + 1 and torch.equal(c.data[:, int(mp[num - 15])], first)


def test_rows_past_2_31_elements():
    # one sequence of 4.2 million tokens in a single call: K alone is 4.3 GB
    R, Hkv, hd, page = 4_200_000, 8, 64, 1024
    c = dfl.PagedCache(1, R // page + 1, page, Hkv, hd, 1, R // page + 1)
    c.table.copy_(torch.arange(c.num_pages, dtype=torch.int32, device="cuda")[None])
    K = torch.zeros((1, R, Hkv, hd), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    tail = torch.randn((1, 1000, Hkv, hd), device="cuda", generator=gen).to(torch.bfloat16)
    K[:, -1000:] = tail
    c.append(0, K, K, i32([0]), i32([R]))
    oK, oV = torch.ones_like(K), torch.ones_like(K)
    c.read(0, i32([0]), i32([R]), oK, oV)
    want = ko.kv4_values(host(tail), 0)
    for o in (oK, oV):
        assert np.array_equal(host(o[:, -1000:]), want) and not bool(o[:, :-1000].any())


@pytest.mark.parametrize("B,Hq", [(1, 8), (16, 8)])
def test_two_caches_on_two_streams(B, Hq):
    rng = np.random.default_rng(B)
    lens = [[3000, 10, 500], [77, 4000, 1]]
    caches = [make_cache(rng, 3, l, 32, 2, 128) for l in lens]
    args = [run_attn(rng, c, l, B, Hq) for c, l in zip(caches, lens)]
    want = [a[-1].clone() for a in args]
    streams = [torch.cuda.Stream() for _ in caches]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (c, a, s) in enumerate(zip(caches, args, streams)):
            with torch.cuda.stream(s):
                got[i].append(c.attn(0, *a[2:5]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)


@pytest.mark.parametrize("B,Hq", [(1, 8), (16, 8)])
def test_a_captured_call_follows_the_lengths(B, Hq):
    rng = np.random.default_rng(B)
    lens = [3000, 40, 1200]
    c = make_cache(rng, 3, lens, 32, 2, 128)
    K, V, Q, Kb, Vb, _ = run_attn(rng, c, lens, B, Hq)
    out, g = torch.empty_like(Q), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attn(0, Q, Kb, Vb, out=out)
    for l in ([3000, 40, 1200], [0, 0, 0], [1, 33, 1199], [40, 40, 40], [2999, 0, 7]):
        c.len.copy_(i32(l))
        g.replay()
        check(c, K, V, Q, Kb, Vb, out, l)
        assert torch.equal(out, c.attn(0, Q, Kb, Vb))


def test_streams_given_by_handle_or_object():
    rng = np.random.default_rng(1)
    c = make_cache(rng, 1, [50], 16, 1, 64)
    K, V, Q, Kb, Vb, O = run_attn(rng, c, [50], 1, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for how in (s, s.cuda_stream):
        out = torch.zeros_like(O)
        torch.cuda.synchronize()
        c.attn(0, Q, Kb, Vb, out=out, stream=how)
        s.synchronize()
        assert torch.equal(out, O)


def test_parity_cases_pass_under_the_bounds_checked_build():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    from block_diffusion_speculative_dfl_gb300._build import build
    build(checked=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_paged.py", __file__, "-m", "gpu", "-q", "-x", "-p",
                        "no:cacheprovider", "-k", "not bounds_checked and not past_2_31"], cwd=root,
                       env=dict(os.environ, DFL_CHECKED_BUILD="1"), capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and " failed" not in r.stdout
