"""Drafted-token trees without a GPU: the oracle's pins, and what the calls refuse on the host."""
import ctypes as C
import itertools

import numpy as np
import pytest
import torch

import block_diffusion_speculative_dfl_gb300 as dfl
from oracle import tree_oracle as to

FAKE = 1 << 20   # an aligned stand-in address; refused calls never reach the device
ARG, SHAPE, ALIGN, WORKSPACE, NO_DEVICE = 1, 2, 3, 4, 7


# ------------------------------------------------------------------ oracle --

def test_logprobs_of_worked_rows():
    # weights 1, 2, 4, 1 of 8: H = 1.75 bits
    lp, H, top, tl = to.token_logprobs(np.log([1.0, 2, 4, 1]), [2, 0, 9, -1], 3, 1.0)
    assert np.allclose(lp[:2], np.log([0.5, 0.125])) and (lp[2:] == -np.inf).all() and abs(H - 1.75 * np.log(2)) < 1e-14
    assert top.tolist() == [2, 1, 0] and np.allclose(tl, np.log([0.5, 0.25, 0.125]))
    # temperature 2 takes square roots of the weights
    lp, _, _, _ = to.token_logprobs(np.log([1.0, 4, 16]), [0, 1, 2], 0, 2.0)
    assert np.allclose(lp, np.log([1 / 7, 2 / 7, 4 / 7]))
    lp, H, top, tl = to.token_logprobs([0.0, -np.inf, 0.0], [0, 1], 3, 1.0)
    assert np.allclose(lp[0], -np.log(2)) and lp[1] == -np.inf and abs(H - np.log(2)) < 1e-15
    assert top.tolist() == [0, 2, -1] and tl[2] == -np.inf
    for bad in ([np.nan, 1.0], [np.inf, 1.0], [-np.inf, -np.inf]):
        lp, H, top, _ = to.token_logprobs(bad, [1], 2, 1.0)
        assert np.isnan(lp).all() and np.isnan(H)


def test_a_tree_holds_the_most_probable_prefixes():
    rng = np.random.default_rng(3)
    G, K, B = 4, 3, 14
    lp = np.sort(np.log(rng.dirichlet(np.ones(5), G)))[:, ::-1][:, :K]
    ids = rng.permutation(100)[:G * K].reshape(G, K)
    token, parent, depth = to.draft_tree(7, ids, lp, B)
    got = {tuple(token[j] for j in reversed(to.ancestors(parent, i)) if j) for i in range(1, B)}
    every = {}
    for d in range(1, G + 1):
        for ranks in itertools.product(range(K), repeat=d):
            every[tuple(int(ids[g][k]) for g, k in enumerate(ranks))] = sum(lp[g][k] for g, k in enumerate(ranks))
    best = sorted(every, key=every.get, reverse=True)[:B - 1]
    assert got == set(best) and token[0] == 7 and parent[0] == -1
    assert [len(to.ancestors(parent, i)) - 1 for i in range(B)] == depth
    # equal scores: the lowest parent first, then the better rank
    t, p, d = to.draft_tree(0, [[1, 2], [3, 4]], np.zeros((2, 2)), 7)
    assert p == [-1, 0, 0, 1, 1, 2, 2] and t == [0, 1, 2, 3, 4, 3, 4]
    # nothing behind infinities or NaN
    assert to.draft_tree(0, [[1, 2]], [[-1.0, -np.inf]], 9)[0] == [0, 1]
    assert to.draft_tree(0, [[1, 2]], [[np.nan, -1.0]], 9)[0] == [0]
    assert to.draft_tree(0, [[1, 2]], [[np.inf, -1.0]], 9)[0] == [0]


def test_what_rows_see():
    parent = [-1, 0, 0, 1, -2]
    mask = to.tree_mask(parent)
    assert mask == [1, 3, 5, 11, 0]
    see = to.sees(3, 5, mask, 0, 0)
    assert see[:4, :3].all() and not see[4].any()
    assert see[3].tolist() == [True] * 3 + [True, True, False, True, False]
    # positions 3, 4, 4, 5; a window of 2 sees q and q - 1, and token 0 as a sink
    see = to.sees(3, 5, mask, 2, 1)
    assert see[0].tolist() == [True, False, True, True, False, False, False, False]
    assert see[1].tolist() == [True, False, False, True, True, False, False, False]
    assert see[3].tolist() == [True, False, False, False, True, False, True, False]
    # a block without a mask: row i at position len + i, later rows visible
    see = to.sees(2, 3, None, 2, 0)
    assert see.tolist() == [[False, True, True, True, True], [False, False, True, True, True], [False, False, False, True, True]]


def test_acceptance_walks_along_the_targets_tokens():
    token, parent = [9, 1, 2, 3, 3], [-1, 0, 0, 1, 2]
    assert to.tree_accept(token, parent, [2, 0, 3, 0, 5]) == ([0, 2, 4], 5)
    assert to.tree_accept(token, parent, [1, 4, 3, 0, 5]) == ([0, 1], 4)
    assert to.tree_accept(token, parent, [8, 4, 3, 0, 5]) == ([0], 8)
    assert to.tree_accept([9, 1, 1], [-1, 0, 0], [1, 7, 8]) == ([0, 1], 7)   # two alike: the lower row


def test_masked_attention_without_a_mask_is_attention():
    from oracle import kv4_oracle as ko
    rng = np.random.default_rng(0)
    q, kc, vc, kb, vb = (rng.standard_normal(s) for s in ((3, 4, 8), (5, 2, 8), (5, 2, 8), (3, 2, 8), (3, 2, 8)))
    want = ko.paged_attn(q, kc, vc, kb, vb)[0]
    assert np.allclose(to.masked_attn(q, kc, vc, kb, vb, np.ones((3, 8), bool))[0], want)
    see = np.ones((3, 8), bool)
    see[1] = False
    see[2, 2:] = False
    O = to.masked_attn(q, kc, vc, kb, vb, see)[0]
    assert (O[1] == 0).all() and np.allclose(O[0], want[0])
    assert np.allclose(O[2], ko.paged_attn(q[2:], kc[:2], vc[:2], kb[:0], vb[:0])[0][0])


# ---------------------------------------------------------------- refusals --

def no_device():
    code = C.c_int32(0)
    return dfl.load().dfl_get_device_error(None, C.byref(code)) == NO_DEVICE


needs_no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="stand-in addresses must not reach a launch")


def lp_args(**kw):
    a = dict(logits=FAKE, dt=1, rows=3, V=100, stride=104, T=1.0, ids=FAKE, M=2, logp=FAKE, entropy=FAKE, K=4, top_ids=FAKE,
             top_logp=FAKE)
    a.update(kw)
    return dfl.load().dfl_token_logprobs(*a.values(), None)


@needs_no_device
@pytest.mark.parametrize("kw,rc", [
    (dict(), NO_DEVICE), (dict(ids=None, M=0, logp=None), NO_DEVICE), (dict(entropy=None), NO_DEVICE),
    (dict(K=0, top_ids=None, top_logp=None), NO_DEVICE), (dict(K=64), NO_DEVICE), (dict(dt=0), NO_DEVICE),
    (dict(T=1e-6), NO_DEVICE), (dict(T=1e6), NO_DEVICE), (dict(stride=100), NO_DEVICE), (dict(logp=FAKE + 4), NO_DEVICE),
    (dict(logits=None), ARG), (dict(dt=2), ARG), (dict(rows=0), ARG), (dict(V=0), ARG), (dict(stride=99), ARG),
    (dict(T=0.0), ARG), (dict(T=-1.0), ARG), (dict(T=float("nan")), ARG), (dict(T=float("inf")), ARG), (dict(T=1e-7), ARG),
    (dict(M=-1), ARG), (dict(K=-1), ARG), (dict(K=65), ARG), (dict(ids=None), ARG), (dict(logp=None), ARG),
    (dict(top_ids=None), ARG), (dict(top_logp=None), ARG), (dict(M=0, K=0, entropy=None), ARG),
    (dict(rows=1 << 31), SHAPE), (dict(V=(1 << 30) + 1, stride=1 << 31), SHAPE), (dict(stride=(1 << 40) + 1), SHAPE),
    (dict(logits=FAKE + 8), ALIGN), (dict(ids=FAKE + 2), ALIGN), (dict(logp=FAKE + 2), ALIGN), (dict(entropy=FAKE + 1), ALIGN),
    (dict(top_ids=FAKE + 2), ALIGN), (dict(top_logp=FAKE + 2), ALIGN)])
def test_token_logprobs_refuses_on_the_host(kw, rc):
    assert lp_args(**kw) == rc


TREE = ("anchor", "top_ids", "top_logp", "N", "G", "K", "B", "token", "parent", "depth", "mask", "count")
ACCEPT = ("token", "parent", "target", "N", "B", "path", "accept_len", "n_rows", "bonus")


@needs_no_device
@pytest.mark.parametrize("fn,names", [("dfl_draft_tree", TREE), ("dfl_tree_accept", ACCEPT)])
def test_tree_calls_refuse_on_the_host(fn, names):
    f = getattr(dfl.load(), fn)
    ok = {n: FAKE for n in names} | {"N": 2, "B": 64} | ({"G": 3, "K": 5} if "G" in names else {})
    call = lambda **kw: f(*(ok | kw).values(), None)
    assert call() == NO_DEVICE and call(B=1) == NO_DEVICE
    for n in names:
        if n in ("N", "G", "K", "B"):
            assert call(**{n: 0}) == ARG and call(**{n: -1}) == ARG
        else:
            assert call(**{n: None}) == (NO_DEVICE if n == "n_rows" else ARG)
            assert call(**{n: FAKE + 2}) == ALIGN
    assert call(B=65) == SHAPE
    if "G" in names:
        assert call(mask=FAKE + 4) == ALIGN and call(G=1 << 16, K=1 << 15) == SHAPE


POOL = dict(page=32, Hkv=2, hd=64)


def pool_pages():
    pool = dfl.Kv4Pool(FAKE, 8 * dfl.dfl_kv4_page_bytes(32, 2, 64), 1, 8, 32, 2, 64, 0, 0)
    return pool, dfl.Pages(FAKE, FAKE, FAKE, 2, 4)


@needs_no_device
def test_masked_attention_refuses_on_the_host():
    pool, pages = pool_pages()
    need = dfl.workspace_size(dfl.DFL_OP_KV4_ATTN, N=2, B=5, Hq=4, Hkv=2, hd=64)
    ok = dict(pool=C.byref(pool), layer=0, pages=C.byref(pages), Q=FAKE, Kb=FAKE, Vb=FAKE, B=5, Hq=4, mask=FAKE, window=7,
              sinks=2, O=FAKE, ws=FAKE, ws_bytes=need)
    call = lambda **kw: dfl.load().dfl_kv4_attn_masked(*(ok | kw).values(), None)
    for kw in (dict(), dict(mask=None), dict(window=0), dict(window=0, mask=None), dict(window=(1 << 31) - 1, sinks=(1 << 31) - 1),
               dict(mask=FAKE + 8)):
        assert call(**kw) == NO_DEVICE, kw
    for n in ("pool", "pages", "Q", "Kb", "Vb", "O", "ws"):
        assert call(**{n: None}) == ARG, n
    for n in ("Q", "Kb", "Vb", "O", "ws"):
        assert call(**{n: FAKE + 8}) == ALIGN, n
    assert call(mask=FAKE + 4) == ALIGN
    for kw in (dict(window=-1), dict(sinks=-1), dict(B=0), dict(Hq=3), dict(layer=1)):
        assert call(**kw) == ARG, kw
    assert call(B=65) == SHAPE and call(ws_bytes=need - 1) == WORKSPACE


@needs_no_device
def test_append_of_chosen_rows_refuses_on_the_host():
    pool, pages = pool_pages()
    ok = dict(pool=C.byref(pool), layer=0, pages=C.byref(pages), start=FAKE, n_new=FAKE, rows=FAKE, R=3, K=FAKE, V=FAKE)
    call = lambda **kw: dfl.load().dfl_kv4_append_rows(*(ok | kw).values(), None)
    assert call() == NO_DEVICE
    for n in ("pool", "pages", "start", "n_new", "rows", "K", "V"):
        assert call(**{n: None}) == ARG, n
    for n in ("start", "n_new", "rows"):
        assert call(**{n: FAKE + 2}) == ALIGN, n
    assert call(K=FAKE + 8) == ALIGN and call(V=FAKE + 8) == ALIGN and call(R=0) == ARG


def test_python_calls_refuse_tensors_of_the_wrong_kind():
    with pytest.raises(ValueError):
        dfl.token_logprobs(torch.zeros(3, 10))           # not on a GPU
    for N, B in ((0, 4), (2, 0), (2, 65)):
        with pytest.raises(ValueError):
            dfl.DraftTree(N, B, device="cpu")
    t = dfl.DraftTree(2, 5, device="cpu")
    with pytest.raises(ValueError):
        t.build(torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, 4, dtype=torch.int32), torch.zeros(2, 3, 4))
    with pytest.raises(ValueError):
        t.accept(torch.zeros(2, 5, dtype=torch.int32))


@pytest.mark.parametrize("name,kernels", [("logprobs.cu", 1), ("tree.cu", 2)])
def test_the_bounds_checked_build_covers_every_kernel(name, kernels):
    import os
    from test_checked_build_sources import CSRC, functions
    fs = functions(os.path.join(CSRC, name))
    found = [n for n, body in fs.items() if "__global__" in body]
    assert len(found) == kernels == open(os.path.join(CSRC, name)).read().count("__global__ void")
    assert all("DFL_IN_BOUNDS" in fs[n] for n in found)
