"""Drafted-token trees on the GPU against the fp64 oracle.

Ids, trees, paths and cached values are exact.  Log probabilities: with y =
z log2(e) / T never rounded, what is left is log2(e) / T itself (half a step,
2^-24 of a logp's distance), the base-2 exponentials (2^-22 each), exponents
rounded to 2^-24 of themselves (2^-24 |d| 2^d: under 2^-24 of a sum), the sums:
at most `adds` of a thread's elements in turn and 16 levels above them (2^-24
each), and the roundings of the result (2^-24 of it, log2 2^-22).  The entropy is
a weighted mean of |d| of at most H + 8 (a reference trails its row's maximum by
2^8 at most) less a logarithm, with the same relative errors.
Attention's bound is test_gpu_paged.py's, over the keys that a row sees.
"""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_dfl_gb300 as dfl
from gpu_util import host
from oracle import kv4_oracle as ko
from oracle import tree_oracle as to
from test_gpu_paged import bf16, fill, i32, make_cache

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.build()
    dfl.load()
    torch.cuda.set_device(0)
    yield
    assert dfl.dfl_get_device_error() == 0


# ------------------------------------------------------- log probabilities --

def adds(V, per_vector):
    return -(-(-(-V // per_vector) + 1) // 256) * per_vector


def check_logprobs(logits, ids, K, T, rows=None):
    """One call against the oracle, row by row (all, or those given)."""
    got = dfl.token_logprobs(logits, ids, top=K, T=T)
    lp, top, tl = (host(x).reshape(-1, x.shape[-1]) for x in (got.logp, got.top_ids, got.top_logp))
    H = host(got.entropy).reshape(-1)
    V = logits.shape[-1]
    z, ids = host(logits).reshape(-1, V), host(ids).reshape(lp.shape)
    n = adds(V, 8 if logits.dtype is torch.bfloat16 else 4)
    for r in range(len(z)) if rows is None else rows:
        w_lp, w_H, w_top, w_tl = to.token_logprobs(z[r], ids[r].tolist(), K, float(np.float32(T)))
        assert np.array_equal(top[r], w_top), r
        for g, w, scale in ((lp[r], w_lp, 1 + np.abs(w_lp)), (tl[r], w_tl, 1 + np.abs(w_tl)), (H[r:r + 1], np.array([w_H]), w_H + 9)):
            with np.errstate(over="ignore"):
                w = np.where(np.isfinite(w.astype(np.float32)), w, w.astype(np.float32))   # beyond fp32's range: -inf
            off = np.isfinite(w)
            assert np.array_equal(g[~off], w[~off], equal_nan=True), (r, g, w)
            tol = ((n + 32) * 2.0 ** -24 + 2.0 ** -21) * (scale if np.ndim(scale) == 0 else scale[off])
            assert (np.abs(g[off] - w[off]) <= tol).all(), (r, g, w)
    return got


def logits_of(rng, rows, V, dtype, scale=3.0, pad=0, shift=0):
    """[rows, V] in a wider buffer whose other elements are NaN, `shift` elements (a multiple of 16 bytes) into it."""
    buf = torch.full((rows * (V + pad) + shift,), float("nan"), dtype=dtype, device="cuda")
    out = buf[shift:].view(rows, V + pad)[:, :V]
    out.copy_(torch.from_numpy(rng.standard_normal((rows, V)).astype(np.float32) * scale))
    return out


def some_ids(rng, rows, V, M):
    ids = rng.integers(0, V, (rows, M))
    return i32(ids)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,pad,M,K,T", [
    (1, 1, 0, 1, 1, 1.0), (3, 2, 1, 2, 4, 0.7), (9, 7, 0, 1, 3, 1.0), (5, 8, 3, 1, 8, 1.0), (17, 9, 0, 3, 9, 2.0),
    (33, 100, 5, 2, 64, 1.5), (40, 257, 0, 1, 7, 1.0), (16, 1000, 1, 4, 5, 0.25), (700, 2047, 2, 1, 1, 1.0),
    (4, 4099, 0, 1, 33, 1.0), (2, 33000, 7, 2, 64, 3.0), (3, 151936, 0, 1, 8, 1.0), (1, 201087, 0, 300, 5, 1.0)])
def test_logprobs_of_all_sizes(dtype, rows, V, pad, M, K, T):
    rng = np.random.default_rng(V + rows + K)
    check_logprobs(logits_of(rng, rows, V, dtype, pad=pad, shift=16 if pad else 0), some_ids(rng, rows, V, M), K, T,
                   None if rows < 100 else range(0, rows, 97))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,rows", [(50, 3), (5000, 700), (70001, 3), (151936, 1)])
@pytest.mark.parametrize("order", ["constant", "up", "down", "steps", "two", "last", "first"])
def test_ties_and_sorted_rows(dtype, V, rows, order):
    # equal logits go to the lowest id; rows in order make every later element a candidate
    rng = np.random.default_rng(V)
    at = np.arange(V)
    z = {"constant": np.full(V, 2.5), "up": at / V * 8, "down": -at / V * 8, "steps": at % 5 * 1.0, "two": np.where(at < V // 2, 1.0, 1.5),
         "last": (at == V - 1) * 4.0, "first": (at == 0) * 4.0}[order]
    logits = torch.from_numpy(np.tile(z, (rows, 1)).astype(np.float32)).to(dtype).cuda()
    for K in (1, 12, 64):
        check_logprobs(logits, some_ids(rng, rows, V, 2), K, 1.0, [0, rows - 1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [300, 40001])
def test_masked_and_unusual_rows(dtype, V):
    rng = np.random.default_rng(V)
    low = float(torch.finfo(dtype).min)
    z = logits_of(rng, 16, V, dtype, pad=3)
    keep = torch.from_numpy(rng.permutation(V)[:5].copy()).cuda()
    for r, fill_with in ((1, -INF), (2, low)):
        masked = torch.full((V,), fill_with, dtype=dtype, device="cuda")
        masked[keep] = z[r, keep]
        z[r] = masked
    z[3] = -INF                       # nothing left
    z[4] = -INF
    z[4, V // 2] = -7.0               # one token left
    z[5] = low                        # all masked by the lowest number: alike
    z[6] = low
    z[6, 17] = -INF
    z[7, 5], z[8, 5] = float("nan"), INF
    z[9] *= 1e30                      # products with log2(e) / T beyond any reference
    z[10] = z[10].abs() * -1e36
    z[11] = 0.0
    z[11, ::2] = -0.0                 # one value
    z[12, V - 1] = float("nan")
    z[13] += 3e4
    z[14] = z[14] * 1e-30
    ids = some_ids(rng, 16, V, 4)
    ids[:, 2], ids[:, 3] = -1, V      # no tokens
    ids[1, 0] = int(keep[0])
    for T in (1.0, 0.3, 1e-6, 1e6):
        check_logprobs(z, ids, 12, T)


def test_leading_dims_strides_and_optional_outputs():
    rng = np.random.default_rng(1)
    z = torch.from_numpy(rng.standard_normal((4, 6, 3, 1000)).astype(np.float32)).cuda()
    ids = i32(rng.integers(0, 900, (4, 6, 3, 2)))
    check_logprobs(z, ids, 4, 1.0)
    part = z[:, :, :, :900]           # rows 1000 apart
    check_logprobs(part, ids, 4, 1.0)
    every = dfl.token_logprobs(z[:, 1:2, 2], ids[:, 1:2, 2].contiguous(), top=3)   # one stride over two dims
    assert every.logp.shape == (4, 1, 2) and every.entropy.shape == (4, 1) and every.top_ids.shape == (4, 1, 3)
    whole = dfl.token_logprobs(z, ids, top=3)
    assert torch.equal(every.top_logp, whole.top_logp[:, 1:2, 2]) and torch.equal(every.logp, whole.logp[:, 1:2, 2])
    only = dfl.token_logprobs(z, entropy=False, top=2)
    assert only.logp is None and only.entropy is None and torch.equal(only.top_ids, whole.top_ids[..., :2])
    none = dfl.token_logprobs(z, ids)
    assert none.top_ids.shape == (4, 6, 3, 0) and torch.equal(none.logp, whole.logp) and torch.equal(none.entropy, whole.entropy)
    empty = dfl.token_logprobs(z[:0], top=2)
    assert empty.top_ids.shape == (0, 6, 3, 2) and empty.entropy.shape == (0, 6, 3)
    for bad in (z.transpose(2, 3), z[:, ::2, :2], z.half(), z.double()):
        with pytest.raises(ValueError):
            dfl.token_logprobs(bad)
    for bad in (ids.long(), ids[:, :5], ids.transpose(0, 1), ids[0]):
        with pytest.raises(ValueError):
            dfl.token_logprobs(z, bad)
    with pytest.raises(ValueError):
        dfl.token_logprobs(z, top=65)
    with pytest.raises(dfl.DflError):
        dfl.token_logprobs(z, T=0.0)
    flat = torch.zeros(4097, device="cuda")
    with pytest.raises(dfl.DflError):
        dfl.token_logprobs(flat[1:])  # not on a 16-byte boundary


def test_rows_past_2_31_elements():
    rng = np.random.default_rng(3)
    V, stride = 1000, (1 << 31) + 8
    buf = torch.zeros(2 * stride, dtype=torch.bfloat16, device="cuda")
    z = buf.view(2, stride)[:, :V]
    z.copy_(torch.from_numpy(rng.standard_normal((2, V)).astype(np.float32)))
    check_logprobs(z, some_ids(rng, 2, V, 2), 5, 1.0)


def test_logprobs_write_their_rows_only_and_repeat():
    rng = np.random.default_rng(2)
    rows, V, M, K = 37, 5003, 3, 6
    z, ids = logits_of(rng, rows, V, torch.float32, pad=1), some_ids(rng, rows, V, M)
    sizes = (rows * M, rows, rows * K, rows * K)
    runs = []
    for _ in range(2):
        bufs = [torch.full((n + 64,), 77, dtype=d, device="cuda") for n, d in zip(sizes, (torch.float32, torch.float32, torch.int32, torch.float32))]
        at = [b[32:] for b in bufs]
        dfl.dfl_token_logprobs(z, dfl.DFL_F32, rows, V, V + 1, 1.0, ids, M, at[0], at[1], K, at[2], at[3])
        for b, n in zip(bufs, sizes):
            assert (b[:32] == 77).all() and (b[32 + n:] == 77).all()
        runs.append([b[32:32 + n].clone() for b, n in zip(bufs, sizes)])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    got = dfl.token_logprobs(z, ids, top=K)
    assert torch.equal(got.logp.flatten(), runs[0][0]) and torch.equal(got.top_ids.flatten(), runs[0][2])


# ------------------------------------------------------------------- trees --

def check_tree(tree, anchor, ids, lp):
    N, B = tree.N, tree.B
    got = {k: host(getattr(tree, k)) for k in ("token", "parent", "depth", "mask", "count")}
    for n in range(N):
        token, parent, depth = to.draft_tree(anchor[n], ids[n], lp[n], B)
        c, rest = len(token), B - len(token)
        assert got["count"][n] == c
        assert got["token"][n].tolist() == token + [-1] * rest and got["parent"][n].tolist() == parent + [-2] * rest
        assert got["depth"][n].tolist() == depth + [0] * rest
        want = np.array(to.tree_mask(parent) + [0] * rest, np.uint64).view(np.int64)
        assert np.array_equal(got["mask"][n], want)


@pytest.mark.parametrize("N,G,K,B", [(1, 1, 1, 1), (2, 1, 1, 2), (3, 1, 9, 6), (1, 15, 4, 16), (5, 40, 1, 33), (4, 70, 3, 64),
                                     (3, 5, 64, 64), (2, 100, 100, 64), (300, 32, 8, 64), (2, 2, 2, 64), (7, 9, 5, 32)])
@pytest.mark.parametrize("kind", ["usual", "flat", "sure", "grid"])
def test_trees_of_all_sizes(N, G, K, B, kind):
    rng = np.random.default_rng(N + G + K + B)
    scale = {"usual": 3.0, "flat": 0.1, "sure": 30.0, "grid": 1.0}[kind]
    lp = -np.sort(rng.exponential(scale, (N, G, K)), -1).astype(np.float32)
    if kind == "grid":     # many equal scores
        lp = np.round(lp)
    if kind == "sure":     # the first alternative has all of it, to fp32
        lp[:, :, 0] = -0.0
    ids, anchor = rng.integers(0, 200000, (N, G, K)).astype(np.int32), rng.integers(0, 200000, N)
    tree = dfl.DraftTree(N, B)
    assert tree.build(i32(anchor), i32(ids), torch.from_numpy(lp).cuda()) is tree
    check_tree(tree, anchor, ids, lp)
    tree.build(i32(anchor), i32(ids), torch.from_numpy(lp).cuda())   # over an older tree
    check_tree(tree, anchor, ids, lp)


def test_alternatives_that_are_none_end_a_trees_branches():
    rng = np.random.default_rng(4)
    N, G, K, B = 8, 6, 4, 40
    lp = -np.sort(rng.exponential(1.0, (N, G, K)), -1).astype(np.float32)
    ids = rng.integers(0, 1000, (N, G, K)).astype(np.int32)
    lp[0, :, 2:] = -INF
    lp[1, 3] = -INF
    lp[2, 0] = -INF          # nothing behind the anchor
    lp[3, 1, 1] = np.nan
    lp[4, 0, 0] = np.nan
    lp[5] = -1e38            # sums past fp32
    lp[6, 2] = INF
    lp[7] = 0.25             # a little above 0, as rounding leaves them
    tree = dfl.DraftTree(N, B).build(i32(np.arange(N)), i32(ids), torch.from_numpy(lp).cuda())
    check_tree(tree, np.arange(N), ids, lp)
    assert host(tree.count)[[2, 4]].tolist() == [1, 1]


def test_alternatives_far_out_count_as_1024():
    lp = np.array([[[-1.0, -1500.0, -3000.0]], [[-1.0, -1500.0, -3000.0]]], np.float32).repeat(2, 1)
    lp[0, 1], ids = [-0.5, -900.0, -1100.0], np.arange(12).reshape(2, 2, 3)
    tree = dfl.DraftTree(2, 13).build(i32([0, 0]), i32(ids), torch.from_numpy(lp).cuda())
    check_tree(tree, [0, 0], ids, np.maximum(lp, -1024.0))


def random_tree(rng, B, count):
    parent = [-1] + [int(rng.integers(0, i)) if rng.random() < 0.5 else i - 1 for i in range(1, count)]
    return parent + [-2] * (B - count)


@pytest.mark.parametrize("N,B", [(1, 1), (2, 2), (5, 16), (3, 33), (301, 64)])
def test_acceptance_along_trees(N, B):
    rng = np.random.default_rng(N + B)
    tree, parent = dfl.DraftTree(N, B), np.zeros((N, B), np.int32)
    token, target = rng.integers(0, 3, (N, B)).astype(np.int32), rng.integers(0, 3, (N, B)).astype(np.int32)
    for n in range(N):
        parent[n] = random_tree(rng, B, int(rng.integers(1, B + 1)))
    token[parent == -2] = -1
    tree.token.copy_(i32(token))
    tree.parent.copy_(i32(parent))
    path, length, bonus = tree.accept(i32(target))
    for n in range(N):
        w_path, w_bonus = to.tree_accept(token[n], parent[n], target[n])
        assert host(path)[n].tolist() == w_path + [-1] * (B - len(w_path))
        assert (int(length[n]), int(tree.n_rows[n]), int(bonus[n])) == (len(w_path) - 1, len(w_path), w_bonus)


def test_a_tree_without_branches_accepts_as_the_greedy_rule():
    rng = np.random.default_rng(5)
    N, B = 40, 16
    draft, target = rng.integers(0, 2, (N, B - 1)), rng.integers(0, 2, (N, B))
    tree = dfl.DraftTree(N, B)
    tree.token[:, 1:] = i32(draft)
    tree.parent.copy_(i32(np.tile(np.arange(B) - 1, (N, 1))))
    tree.accept(i32(target))
    a, b = i32(np.zeros(N)), i32(np.zeros(N))
    dfl.dfl_greedy_accept(i32(draft), i32(target), N, B - 1, a, b)
    assert torch.equal(a, tree.accept_len) and torch.equal(b, tree.bonus)


def test_chosen_rows_are_appended_in_their_order():
    rng = np.random.default_rng(6)
    c = make_cache(rng, 3, [5, 0, 17], 16, 2, 64, extra=20)
    K, V = bf16(rng, (3, 9, 2, 64)), bf16(rng, (3, 9, 2, 64))
    rows = np.array([[0, 3, 8, 3, -1, 0, 0, 0, 0], [8, 7, 6, 5, 4, 3, 2, 1, 0], [4, -1, 9, 2, 0, 0, 0, 0, 0]])
    n_new, start = [4, 9, 0], i32([5, 0, 17])
    c.append(0, K, V, start, i32(n_new), rows=i32(rows))
    oK, oV = torch.zeros_like(K), torch.zeros_like(V)
    c.read(0, start, i32(n_new), oK, oV)
    for x, o in ((K, oK), (V, oV)):
        want = ko.kv4_values(host(x), 0)
        for n in range(3):
            assert np.array_equal(host(o)[n, :n_new[n]], want[n, rows[n, :n_new[n]]])
    assert dfl.dfl_get_device_error() == 0
    # an entry that is no row writes nothing, alone
    before = c.data.clone()
    c.append(0, K, V, start, i32([0, 0, 3]), rows=i32(rows))
    assert dfl.dfl_get_device_error() == 1
    c.read(0, i32([0, 0, 17]), i32([0, 0, 1]), oK, oV)
    assert np.array_equal(host(oK)[2, 0], ko.kv4_values(host(K), 0)[2, 4])
    c.data.copy_(before)
    with pytest.raises(ValueError):
        c.append(0, K, V, start, i32(n_new), rows=i32(rows[:, :8]))


# --------------------------------------------------------------- attention --

# query rows to a K/V head: 1, 2, 8, 12, 16 (warp products), 34, 64, 96, 128, 256 (tensor memory)
HEADS = [(1, 2, 2, 64), (1, 8, 1, 128), (4, 4, 2, 64), (3, 8, 2, 128), (16, 2, 2, 128), (16, 1, 1, 64), (17, 4, 2, 64),
         (16, 8, 2, 128), (16, 8, 2, 64), (32, 3, 1, 64), (32, 8, 2, 128), (64, 4, 2, 64), (64, 4, 1, 128)]
LENS = [[0], [1, 0, 300], [517], [128, 64, 127, 63, 65, 129], [40] * 30, [3000, 5]]
SEEN = [("tree", 0, 0), ("tree", 40, 3), ("tree", 5, 0), ("tree", 1, 70), ("tree", 128, 4), ("tree", 4000, 0), ("block", 64, 0),
        ("block", 130, 20), ("block", 2, 1), ("any", 30, 10)]


def own_masks(rng, kind, N, B):
    """Masks [N][B] (Python ints): random trees with rows missing, any bits at all, or None for a block."""
    if kind == "block":
        return None
    if kind == "any":
        return [[int(rng.integers(0, 1 << 62)) & ((1 << B) - 1) if rng.random() < 0.9 else 0 for _ in range(B)] for _ in range(N)]
    return [to.tree_mask(random_tree(rng, B, B if n % 2 == 0 else int(rng.integers(1, B + 1)))) for n in range(N)]


def mask_tensor(mask):
    return None if mask is None else torch.from_numpy(np.array(mask, np.uint64).view(np.int64)).cuda()


def check_attn(c, K, V, lens, Q, Kb, Vb, mask, window, sinks, O, seqs=None):
    Kd, Vd = ko.kv4_values(K, c.pool.k_exp), ko.kv4_values(V, c.pool.v_exp)
    q, kb, vb, got = (host(x).astype(np.float64) for x in (Q, Kb, Vb, O))
    B = q.shape[1]
    for n in range(c.N) if seqs is None else seqs:
        l = int(lens[n])
        see = to.sees(l, B, mask[n] if mask is not None else None, window, sinks)
        ref, A, smax = to.masked_attn(q[n], Kd[n, :l], Vd[n, :l], kb[n], vb[n], see)
        vmax = max(np.abs(Vd[n, :l]).max(initial=0), np.abs(vb[n]).max())
        tol = 2.0 ** -8 * np.abs(ref) + (1.01 * 2.0 ** -11 + 2.0 ** -18 * (1 + smax)) * A + (l + B) * 2.0 ** -32 * vmax + 2.0 ** -25
        err = np.abs(got[n] - ref)
        assert (err <= tol).all(), (n, float(np.nanmax(err / tol)), int((~(err <= tol)).sum()))
        blank = ~see.any(1)
        assert (got[n][blank] == 0).all()


@pytest.mark.parametrize("B,Hq,Hkv,hd", HEADS)
@pytest.mark.parametrize("kind,window,sinks", SEEN)
def test_masked_attention_over_the_cache(B, Hq, Hkv, hd, kind, window, sinks):
    rng = np.random.default_rng(B + Hq + hd + window)
    for i, lens in enumerate(LENS):
        page = (16, 48, 64)[i % 3]
        c = make_cache(rng, len(lens), lens, page, Hkv, hd, k_exp=i % 2, v_exp=-(i % 2))
        K, V = fill(rng, c, 0, lens)
        N = c.N
        mask = own_masks(rng, kind, N, B)
        Q, Kb, Vb = bf16(rng, (N, B, Hq, hd)), bf16(rng, (N, B, Hkv, hd)), bf16(rng, (N, B, Hkv, hd))
        O = c.attn(0, Q, Kb, Vb, mask=mask_tensor(mask), window=window, sinks=sinks)
        check_attn(c, K, V, lens, Q, Kb, Vb, mask, window, sinks, O, None if N < 8 else [0, 1, N - 1])


@pytest.mark.parametrize("B,Hq,Hkv,hd", [(1, 4, 1, 64), (8, 2, 1, 128), (16, 4, 1, 128), (16, 8, 1, 64)])
def test_every_window_around_the_units_borders(B, Hq, Hkv, hd):
    rng = np.random.default_rng(hd)
    lens = [384, 321, 256, 192, 129, 128, 127, 63]
    c = make_cache(rng, len(lens), lens, 16, Hkv, hd)
    K, V = fill(rng, c, 0, lens)
    mask = own_masks(rng, "tree", c.N, B)
    Q, Kb, Vb = bf16(rng, (c.N, B, Hq, hd)), bf16(rng, (c.N, B, Hkv, hd)), bf16(rng, (c.N, B, Hkv, hd))
    for window in (1, 2, 15, 16, 17, 48, 63, 64, 65, 66, 127, 128, 129, 130, 191, 193, 255, 257, 320, 383, 384, 385, 400):
        for sinks in (0, 1, 16, 65, 128, 1000):
            O = c.attn(0, Q, Kb, Vb, mask=mask_tensor(mask), window=window, sinks=sinks)
            check_attn(c, K, V, lens, Q, Kb, Vb, mask, window, sinks, O)


@pytest.mark.parametrize("B,Hq,Hkv,hd", HEADS)
def test_rows_that_see_everything_see_what_unmasked_ones_do(B, Hq, Hkv, hd):
    # the line is cut elsewhere, so partials are summed in another order: both within the bound, and the masked forms alike
    rng = np.random.default_rng(hd + B)
    lens = [700, 33, 0, 2000]
    c = make_cache(rng, 4, lens, 32, Hkv, hd)
    K, V = fill(rng, c, 0, lens)
    Q, Kb, Vb = bf16(rng, (4, B, Hq, hd)), bf16(rng, (4, B, Hkv, hd)), bf16(rng, (4, B, Hkv, hd))
    plain = c.attn(0, Q, Kb, Vb)
    ones = [[(1 << B) - 1] * B] * 4
    every = mask_tensor(ones)
    O = c.attn(0, Q, Kb, Vb, mask=every)
    check_attn(c, K, V, lens, Q, Kb, Vb, ones, 0, 0, O)
    check_attn(c, K, V, lens, Q, Kb, Vb, ones, 0, 0, plain)
    assert torch.equal(c.attn(0, Q, Kb, Vb, mask=torch.full_like(every, -1)), O)   # bits from B on count for nothing
    assert torch.equal(c.attn(0, Q, Kb, Vb, mask=every, window=2 ** 31 - 1), O)
    assert torch.equal(c.attn(0, Q, Kb, Vb, window=2065, sinks=1), O)
    assert torch.equal(c.attn(0, Q, Kb, Vb, sinks=5), plain)


@pytest.mark.parametrize("B,Hq,Hkv,hd", HEADS)
@pytest.mark.parametrize("lens", [[90, 0, 700], [90, 0, 150] * 54])   # triples cut and joined; whole ones
def test_unseen_own_rows_touch_nothing(B, Hq, Hkv, hd, lens):
    # infinities and NaN in rows that are none, and in branches that a row does not see
    rng = np.random.default_rng(hd + B)
    N = len(lens)
    c = make_cache(rng, N, lens, 32, Hkv, hd)
    K, V = fill(rng, c, 0, lens)
    mask = [to.tree_mask(random_tree(rng, B, max(1, B - 2 * (n % 3)))) for n in range(N)]
    Q, Kb, Vb = bf16(rng, (N, B, Hq, hd)), bf16(rng, (N, B, Hkv, hd)), bf16(rng, (N, B, Hkv, hd))
    m = mask_tensor(mask)
    clean = c.attn(0, Q, Kb, Vb, mask=m)
    check_attn(c, K, V, lens, Q, Kb, Vb, mask, 0, 0, clean, [0, 1, 2])
    for n in range(N):
        for b in range(B):
            if mask[n][b] == 0:   # no row: whatever was in memory
                Q[n, b], Kb[n, b], Vb[n, b] = float("nan"), float("nan"), float("nan")
                Vb[n, b, :, ::3], Kb[n, b, :, 1::3] = INF, -INF
    assert torch.equal(c.attn(0, Q, Kb, Vb, mask=m), clean)
    if B < 3:
        return
    bad = B // 2                 # a row of the first tree, seen by itself and what hangs on it
    Vb[0, bad, 0, 3], Vb[0, bad, 0, hd - 1], Vb[0, bad, Hkv - 1, 8] = INF, float("nan"), -INF
    O, want = host(c.attn(0, Q, Kb, Vb, mask=m)), host(clean).copy()
    G = Hq // Hkv
    for b in range(B):
        if mask[0][b] >> bad & 1:
            want[0, b, (Hkv - 1) * G:, 8] = -INF
            want[0, b, :G, 3], want[0, b, :G, hd - 1] = INF, np.nan
            if Hkv == 1:
                want[0, b, :G, 8] = -INF
    assert np.array_equal(O, want, equal_nan=True)
    Kb[0, bad] = float("nan")    # a key that is NaN: the scores of the rows that see it, whole heads
    O = host(c.attn(0, Q, Kb, Vb, mask=m))
    for b in range(B):
        if mask[0][b] >> bad & 1:
            assert np.isnan(O[0, b]).all()
        else:
            assert np.array_equal(O[0, b], want[0, b])
    assert np.array_equal(O[1:], want[1:])


@pytest.mark.parametrize("B,Hq,Hkv,hd", HEADS)
@pytest.mark.parametrize("window,sinks", [(70, 5), (200, 0), (33, 40)])
@pytest.mark.parametrize("lens", [[600, 333], [600, 333] * 80])   # triples cut and joined; whole ones
def test_cached_tokens_outside_a_rows_window_touch_nothing(B, Hq, Hkv, hd, window, sinks, lens):
    rng = np.random.default_rng(hd + B)
    N = len(lens)
    c = make_cache(rng, N, lens, 32, Hkv, hd)
    Kc, Vc = (bf16(rng, (N, 600, Hkv, hd)) for _ in range(2))
    zero = i32(np.zeros(N))
    Q, Kb, Vb = bf16(rng, (N, B, Hq, hd)), bf16(rng, (N, B, Hkv, hd)), bf16(rng, (N, B, Hkv, hd))
    mask = [to.tree_mask([-1] + list(range(B - 1)))] * N    # one path: every depth
    m = mask_tensor(mask)
    c.append(0, Kc, Vc, zero, i32(lens))
    clean = host(c.attn(0, Q, Kb, Vb, mask=m, window=window, sinks=sinks))
    bad = Vc.clone()
    for n, l in enumerate(lens):
        bad[n, sinks:l - window + 1] = float("nan")         # seen by no row
    c.append(0, Kc, bad, zero, i32(lens))
    assert np.array_equal(host(c.attn(0, Q, Kb, Vb, mask=m, window=window, sinks=sinks)), clean)
    deep = min(B // 2, window - 2)
    at = [l - window + 1 + deep for l in lens]              # seen by the rows of that depth and less
    want = clean.copy()
    G = Hq // Hkv
    for n in range(N):
        bad[n, at[n], 0, hd - 16] = float("nan")            # its group of 16 dims reads back as NaN
        for b in range(B):
            if b <= deep:
                want[n, b, :G, hd - 16:] = np.nan
    c.append(0, Kc, bad, zero, i32(lens))
    O = host(c.attn(0, Q, Kb, Vb, mask=m, window=window, sinks=sinks))
    assert np.array_equal(O, want, equal_nan=True)
    if sinks:                                               # a sink: all rows see it
        bad[:, sinks - 1, 0, 0] = float("nan")
        c.append(0, Kc, bad, zero, i32(lens))
        O = host(c.attn(0, Q, Kb, Vb, mask=m, window=window, sinks=sinks))
        want[:, :, :G, :16] = np.nan
        assert np.array_equal(O, want, equal_nan=True)


@pytest.mark.parametrize("B,Hq,Hkv,hd", [(1, 8, 1, 128), (8, 2, 1, 64), (16, 4, 1, 128), (32, 4, 1, 64)])
def test_windows_deep_in_a_long_cache(B, Hq, Hkv, hd):
    # 130,000 tokens of one sequence: its last tokens and its first, nothing between is read
    rng = np.random.default_rng(7)
    l = 130001
    c = make_cache(rng, 2, [l, 3], 128, Hkv, hd)
    tail, sinks, window = 700, 9, 600
    Kt, Vt = bf16(rng, (2, tail, Hkv, hd)), bf16(rng, (2, tail, Hkv, hd))
    c.data.fill_(0x7F)           # NaN scales wherever nothing is written
    c.append(0, Kt, Vt, i32([0, 0]), i32([sinks, 3]))
    K0, V0 = host(Kt).astype(np.float64), host(Vt).astype(np.float64)
    c.append(0, Kt, Vt, i32([l - tail, 0]), i32([tail, 0]))
    Kd, Vd = np.zeros((2, l, Hkv, hd)), np.zeros((2, l, Hkv, hd))
    for x, y in ((Kd, K0), (Vd, V0)):
        x[:, l - tail:] = y
        x[:, :sinks] = y[:, :sinks]
    Q, Kb, Vb = bf16(rng, (2, B, Hq, hd)), bf16(rng, (2, B, Hkv, hd)), bf16(rng, (2, B, Hkv, hd))
    mask = own_masks(rng, "tree", 2, B)
    O = c.attn(0, Q, Kb, Vb, mask=mask_tensor(mask), window=window, sinks=sinks)
    check_attn(c, Kd, Vd, [l, 3], Q, Kb, Vb, mask, window, sinks, O)


# --------------------------------------------------------------- all of it --

def serve(c, tree, z, Q, Kb, Vb, target, anchor):
    """One step of a tree: alternatives, tree, attention of a full and of a windowed layer, acceptance, accepted rows."""
    lp = dfl.token_logprobs(z, top=6, T=1.3, entropy=False)
    tree.build(anchor, lp.top_ids, lp.top_logp)
    full = c.attn(0, Q, Kb, Vb, mask=tree.mask)
    win = c.attn(1, Q, Kb, Vb, mask=tree.mask, window=50, sinks=4)
    tree.accept(target)
    start = c.reserve(tree.n_rows)
    for layer in range(2):
        c.append(layer, Kb, Vb, start, tree.n_rows, rows=tree.path)
    return full, win


def serving_state(seed):
    rng = np.random.default_rng(seed)
    N, B, Hq, Hkv, hd, G, V = 5, 16, 8, 2, 64, 15, 4000
    lens = [100, 0, 37, 260, 64]
    c = dfl.PagedCache(2, 60, 16, Hkv, hd, N, 24)
    total = i32(np.zeros(N))
    total.copy_(i32(lens))
    c.reserve(total)
    K, V_ = bf16(rng, (N, 260, Hkv, hd)), bf16(rng, (N, 260, Hkv, hd))
    for layer in range(2):
        c.append(layer, K, V_, i32(np.zeros(N)), i32(lens))
    z = torch.from_numpy(rng.standard_normal((N, G, V)).astype(np.float32) * 3).cuda()
    Q, Kb, Vb = bf16(rng, (N, B, Hq, hd)), bf16(rng, (N, B, Hkv, hd)), bf16(rng, (N, B, Hkv, hd))
    return c, dfl.DraftTree(N, B), z, Q, Kb, Vb, i32(rng.integers(0, V, (N, B))), i32(rng.integers(0, V, N)), K, V_, lens


def test_a_serving_run_of_all_calls():
    c, tree, z, Q, Kb, Vb, target, anchor, K, V, lens = serving_state(11)
    lp = dfl.token_logprobs(z, top=6, T=1.3)
    tree.build(anchor, lp.top_ids, lp.top_logp)
    check_tree(tree, host(anchor), host(lp.top_ids), host(lp.top_logp))
    for n in range(c.N):       # targets that agree for n rows: each row's first child
        cur = 0
        for _ in range(n):
            kids = (tree.parent[n] == cur).nonzero().flatten()
            if kids.numel() == 0:
                break
            target[n, cur] = tree.token[n, int(kids[0])]
            cur = int(kids[0])
    full, win = serve(c, tree, z, Q, Kb, Vb, target, anchor)
    mask = [[int(x) for x in row] for row in host(tree.mask).view(np.uint64)]
    Kh, Vh = host(K).astype(np.float64), host(V).astype(np.float64)
    check_attn(c, Kh, Vh, lens, Q, Kb, Vb, mask, 0, 0, full)
    check_attn(c, Kh, Vh, lens, Q, Kb, Vb, mask, 50, 4, win)
    n_rows = host(tree.n_rows)
    assert host(c.len).tolist() == [l + int(m) for l, m in zip(lens, n_rows)] and n_rows.max() > 1
    oK, oV = torch.zeros_like(Kb), torch.zeros_like(Vb)
    c.read(1, i32(lens), tree.n_rows, oK, oV)
    for n in range(c.N):
        want = ko.kv4_values(host(Kb)[n], 0)[host(tree.path)[n, :n_rows[n]]]
        assert np.array_equal(host(oK)[n, :n_rows[n]], want)


def test_a_captured_step_replays_with_new_inputs():
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        c, tree, z, Q, Kb, Vb, target, anchor, *_ = serving_state(12)
        book, data = c.book.clone(), c.data.clone()
        serve(c, tree, z, Q, Kb, Vb, target, anchor)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        full, win = serve(c, tree, z, Q, Kb, Vb, target, anchor)
    other = serving_state(13)
    for x, y in zip((z, Q, Kb, Vb, target, anchor), other[2:8]):
        x.copy_(y)
    c.book.copy_(book)
    c.data.copy_(data)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (full, win, tree.path, tree.mask, c.book, c.data)]
    c.book.copy_(book)
    c.data.copy_(data)
    f2, w2 = serve(c, tree, z, Q, Kb, Vb, target, anchor)
    for a, b in zip(got, (f2, w2, tree.path, tree.mask, c.book, c.data)):
        assert torch.equal(a, b)


def test_calls_on_another_stream_and_two_at_once():
    c, tree, z, Q, Kb, Vb, target, anchor, *_ = serving_state(14)
    c2, tree2, *rest = serving_state(15)
    z2, Q2, Kb2, Vb2, target2, anchor2 = rest[:6]
    want = [x.clone() for x in serve(c, tree, z, Q, Kb, Vb, target, anchor)] + [tree.path.clone()]
    want2 = [x.clone() for x in serve(c2, tree2, z2, Q2, Kb2, Vb2, target2, anchor2)] + [tree2.path.clone()]
    c, tree, *_ = serving_state(14)
    c2, tree2, *_ = serving_state(15)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        got = list(serve(c, tree, z, Q, Kb, Vb, target, anchor)) + [tree.path]
    with torch.cuda.stream(s2):
        got2 = list(serve(c2, tree2, z2, Q2, Kb2, Vb2, target2, anchor2)) + [tree2.path]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want + want2, got + got2))
    lp = dfl.token_logprobs(z, top=3, stream=s1)   # a stream that is not current
    s1.synchronize()
    assert torch.equal(lp.top_ids, dfl.token_logprobs(z, top=3).top_ids)


def test_a_draft_model_builds_trees_of_its_step():
    from dfl_synth import Workload, gen_block_init, gen_gains, gen_hidden, gen_layer_weights, gen_lm_head, gen_mix_logits
    w = Workload(name="tree", N=3, d=256, Hq=4, Hkv=2, hd=64, D=1, L=2, B=8, C=32, V=1000, dtype="bf16", seed=5, geom_p=0.3)
    g_mix, g_blk, g_fin = gen_gains(w)
    s = dfl.DraftShape(N=3, d=256, Hq=4, Hkv=2, hd=64, D=1, L=2, B=8, C=32, V=1000)
    model = dfl.DraftModel(s, gen_mix_logits(w), g_mix, g_blk, g_fin, [gen_layer_weights(w, 0)], gen_lm_head(w))
    H = torch.from_numpy(gen_hidden(w)).to(torch.bfloat16).cuda()
    Xb0 = torch.from_numpy(gen_block_init(w)).float().cuda()
    tree, anchor = dfl.DraftTree(3, 12), i32([1, 2, 3])
    model.step(H, Xb0)
    with pytest.raises(ValueError):
        model.tree(tree, anchor)
    model.want_logits()
    model.step(H, Xb0)
    assert model.tree(tree, anchor, top=5, T=0.9) is tree
    lp = dfl.token_logprobs(model.logits, top=5, T=0.9)
    check_tree(tree, [1, 2, 3], host(lp.top_ids).reshape(3, 7, 5), host(lp.top_logp).reshape(3, 7, 5))
    assert torch.equal(lp.top_ids[:, 0].view(3, 7), model.draft)


# ------------------------------------------------- shapes of several paths --

@pytest.mark.parametrize("rows,V,dtype,K", [(1, 151936, torch.bfloat16, 8), (3, 60001, torch.float32, 64), (100, 40000, torch.float32, 3),
                                            (1300, 9000, torch.bfloat16, 32), (2000, 500, torch.float32, 33), (1217, 8192, torch.float32, 5)])
def test_rows_by_warps_ctas_and_clusters_replay_from_a_graph(rows, V, dtype, K):
    rng = np.random.default_rng(rows)
    z, ids = logits_of(rng, rows, V, dtype, pad=3), some_ids(rng, rows, V, 2)
    some = sorted({0, rows // 2, rows - 1})
    check_logprobs(z, ids, K, 0.8, some)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = dfl.token_logprobs(z, ids, top=K, T=0.8)
    z.copy_(z.flip(0))
    g.replay()
    torch.cuda.synchronize()
    again = dfl.token_logprobs(z, ids, top=K, T=0.8)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("N,B,Hq,Hkv,hd,window,sinks", [(40, 1, 64, 8, 64, 128, 4), (40, 1, 64, 8, 64, 129, 64), (19, 2, 32, 8, 128, 64, 0),
                                                        (30, 16, 32, 4, 128, 128, 3), (30, 16, 32, 4, 64, 500, 3), (20, 16, 16, 4, 128, 600, 0)])
def test_windows_whose_triples_are_always_whole(N, B, Hq, Hkv, hd, window, sinks):
    # nothing is joined: lengths from none to long ones
    rng = np.random.default_rng(N + window)
    lens = rng.permutation(np.r_[[0, 1, window - 1, window, window + 1], rng.integers(0, 1000, N - 5)])
    c = make_cache(rng, N, lens, 64, Hkv, hd)
    K, V = fill(rng, c, 0, lens)
    Q, Kb, Vb = bf16(rng, (N, B, Hq, hd)), bf16(rng, (N, B, Hkv, hd)), bf16(rng, (N, B, Hkv, hd))
    for kind in ("block", "tree"):
        mask = own_masks(rng, kind, N, B)
        out = torch.full_like(Q, 7.0)
        c.attn(0, Q, Kb, Vb, out=out, mask=mask_tensor(mask), window=window, sinks=sinks)
        check_attn(c, K, V, lens, Q, Kb, Vb, mask, window, sinks, out, np.argsort(lens)[::N // 9])


@pytest.mark.parametrize("hd,Hq", [(128, 32), (64, 64), (128, 64)])
def test_many_ragged_trees_cut_anywhere(hd, Hq):
    rng = np.random.default_rng(hd + Hq)
    N, B, Hkv = 90, 16, 8
    lens = rng.integers(0, 700, N)
    c = make_cache(rng, N, lens, 48, Hkv, hd)
    K, V = fill(rng, c, 0, lens)
    mask = own_masks(rng, "tree", N, B)
    Q, Kb, Vb = bf16(rng, (N, B, Hq, hd)), bf16(rng, (N, B, Hkv, hd)), bf16(rng, (N, B, Hkv, hd))
    O = c.attn(0, Q, Kb, Vb, mask=mask_tensor(mask))
    check_attn(c, K, V, lens, Q, Kb, Vb, mask, 0, 0, O, [0, 1, 44, 71, 89])
    assert torch.equal(O, c.attn(0, Q, Kb, Vb, mask=mask_tensor(mask)))


def test_these_cases_pass_under_the_bounds_checked_build():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    from block_diffusion_speculative_dfl_gb300._build import build
    build(checked=True)
    r = subprocess.run([sys.executable, "-m", "pytest", __file__, "-m", "gpu", "-q", "-x", "-p", "no:cacheprovider", "-k",
                        "(all_sizes and not 151936 and not 201087) or unusual or acceptance or chosen or unseen or serving or ragged"],
                       cwd=root,
                       env=dict(os.environ, DFL_CHECKED_BUILD="1"), capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and " failed" not in r.stdout


def test_calls_refuse_tensors_of_the_wrong_kind():
    rng = np.random.default_rng(1)
    c = make_cache(rng, 2, [5, 9], 16, 2, 64)
    Q, Kb, Vb = bf16(rng, (2, 4, 4, 64)), bf16(rng, (2, 4, 2, 64)), bf16(rng, (2, 4, 2, 64))
    m = torch.ones((2, 4), dtype=torch.int64, device="cuda")
    for bad in (m.int(), m[:, :3], m.cpu(), m.t(), m[:1]):
        with pytest.raises(ValueError):
            c.attn(0, Q, Kb, Vb, mask=bad)
    for kw in (dict(window=-1), dict(sinks=-1), dict(window=5, sinks=-2)):
        with pytest.raises(dfl.DflError):
            c.attn(0, Q, Kb, Vb, mask=m, **kw)
    t = dfl.DraftTree(2, 4)
    anchor, ids, lp = i32([1, 2]), torch.zeros((2, 3, 2), dtype=torch.int32, device="cuda"), torch.zeros((2, 3, 2), device="cuda")
    t.build(anchor, ids, lp)
    for bad in ((anchor[:1], ids, lp), (anchor.long(), ids, lp), (anchor, ids.long(), lp), (anchor, ids, lp.double()), (anchor, ids[:, :2], lp),
                (anchor, ids[0], lp[0]), (anchor.cpu(), ids, lp), (anchor, ids[:, :0], lp[:, :0])):
        with pytest.raises(ValueError):
            t.build(*bad)
    for bad in (i32(np.zeros((2, 3))), torch.zeros((2, 4), device="cuda"), i32(np.zeros((4, 2))).t()):
        with pytest.raises(ValueError):
            t.accept(bad)
