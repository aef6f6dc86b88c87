"""Forms of the paged draft step: attention to the rows of the same step, sampling, the fusion, fewer rows than room (GPU).

The cached step, which test_gpu_cached.py compares with the fp64 oracle, is the
reference over the values that the pages hold (they are exact in bf16).
"""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_dfl_gb300 as dfl
from dfl_synth import (Workload, gen_block_init, gen_fc_weights, gen_ffn_gains, gen_gains, gen_layer_weights, gen_lm_head,
                       gen_mix_logits)
from gpu_util import assert_bf16_close, check_samples, host
from oracle import kv4_oracle as ko
from test_gpu_paged import bf16, i32

pytestmark = pytest.mark.gpu
R_MAX = 24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.build()
    dfl.load()
    torch.cuda.set_device(0)
    yield
    assert dfl.dfl_get_device_error() == 0


def workload(hd=64, Hq=4, Hkv=2, B=8, C=128, N=3, F=0, fc=0, K=0):
    return Workload("pagedstep", N=N, d=256, Hq=Hq, Hkv=Hkv, hd=hd, D=2, L=3, B=B, C=C, V=1500, dtype="bf16", seed=37,
                    R=R_MAX, F=F, fc=fc, K=K, T=1.5, philox_seed=0x5EEDD1F5)


def model(cls, w, *extra, **kw):
    shape = dfl.DraftShape(N=w.N, d=w.d, Hq=w.Hq, Hkv=w.Hkv, hd=w.hd, D=w.D, L=w.L, B=w.B, C=w.C, V=w.V, dtype="bf16",
                           K=w.K, T=w.T, seed=w.philox_seed, F=w.F, fc=w.fc)
    g_mix, g_blk, g_fin = gen_gains(w)
    W_lm = torch.from_numpy(gen_lm_head(w, as_bits=True).view(np.int16)).view(torch.bfloat16)
    if w.F:
        kw["ffn_gain"] = gen_ffn_gains(w)
    if w.fc:
        kw["W_fc"], kw["fc_gain"] = gen_fc_weights(w)
    return cls(shape, R_MAX, *extra, None if w.fc else gen_mix_logits(w), None if w.fc else g_mix, g_blk, g_fin,
               [gen_layer_weights(w, l) for l in range(w.D)], W_lm, **kw)


def pages_into(m4, m16, w):
    """The cached model's caches become the values that the pages hold."""
    m16.K_cache.zero_()
    m16.V_cache.zero_()
    for l in range(w.D):
        m4.cache.read(l, i32([0] * w.N), m4.cache.len, m16.K_cache[l], m16.V_cache[l])
    m16.ctx_len.copy_(m4.cache.len)


@pytest.mark.parametrize("hd,Hq,Hkv,B,page,F,fc", [(64, 4, 2, 8, 16, 0, 0), (128, 8, 2, 16, 32, 512, 0), (128, 2, 1, 2, 64, 0, 1),
                                                   (64, 8, 2, 16, 16, 0, 1), (128, 4, 4, 8, 48, 256, 1)])
def test_a_step_attends_to_the_rows_it_appends(hd, Hq, Hkv, B, page, F, fc):
    w = workload(hd, Hq, Hkv, B, 144 if page == 48 else 128, F=F, fc=fc)
    m16, m4 = model(dfl.CachedDraftModel, w), model(dfl.PagedDraftModel, w, 30, page=page)
    rng, X0 = np.random.default_rng(hd + B), torch.from_numpy(gen_block_init(w)).cuda()
    for m in (m16, m4):
        m.want_logits()
    want = np.zeros(w.N, int)
    for n_new in ([24, 5, 0], [7, 24, 24], [1, 0, 13], [24, 24, 24]):
        H = bf16(rng, (w.L, w.N * R_MAX, w.d))
        m4.step(H, X0, i32(n_new))
        assert host(m4.cache.start).tolist() == want.tolist()
        want += n_new
        assert host(m4.cache.len).tolist() == want.tolist()
        pages_into(m4, m16, w)
        m16.step(H, X0, i32([0] * w.N))   # the block over those rows, none of them new
        assert_bf16_close(host(m4.Xb) - host(X0), host(m16.Xb) - host(X0), f"Xb after {want}")
        assert_bf16_close(host(m4.logits), host(m16.logits), f"logits after {want}")
        assert np.array_equal(host(m4.draft), host(m4.logits).reshape(w.N, B - 1, -1).argmax(-1))


@pytest.mark.parametrize("fc", [0, 1])
def test_rows_of_a_fused_or_mixed_step_are_the_cached_steps(fc):
    w = workload(hd=128, Hq=8, Hkv=2, B=16, fc=fc)
    m16, m4 = model(dfl.CachedDraftModel, w), model(dfl.PagedDraftModel, w, 30, page=16)
    rng, X0 = np.random.default_rng(fc), torch.from_numpy(gen_block_init(w)).cuda()
    H, n_new = bf16(rng, (w.L, w.N * R_MAX, w.d)), [24, 9, 0]
    m16.step(H, X0, i32(n_new))
    m4.step(H, X0, i32(n_new))
    for l in range(w.D):
        K, V = (torch.zeros((w.N, R_MAX, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        m4.cache.read(l, i32([0] * 3), i32(n_new), K, V)
        for got, cache in ((K, m16.K_cache), (V, m16.V_cache)):
            for n, m in enumerate(n_new):
                assert np.array_equal(host(got)[n, :m], ko.kv4_values(host(cache[l, n, :m]), 0))


@pytest.mark.parametrize("R", [1, 5, 23])
def test_fewer_rows_than_there_is_room_for(R):
    w = workload()
    a, b = model(dfl.PagedDraftModel, w, 30, page=16), model(dfl.PagedDraftModel, w, 30, page=16)
    rng, X0 = np.random.default_rng(R), torch.from_numpy(gen_block_init(w)).cuda()
    for n_new in ([R, 0, (R + 1) // 2], [R, R, R]):
        H = bf16(rng, (w.L, w.N, R, w.d))
        wide = bf16(rng, (w.L, w.N, R_MAX, w.d))   # rows past n_new are not looked at
        wide[:, :, :R] = H
        a.step(H.view(w.L, w.N * R, w.d), X0, i32(n_new), R=R)
        b.step(wide.view(w.L, w.N * R_MAX, w.d), X0, i32(n_new))
        assert torch.equal(a.cache.book, b.cache.book) and torch.equal(a.cache.start, b.cache.start)
        lens = host(a.cache.len)
        for l in range(w.D):
            got = []
            for m in (a, b):
                K, V = (torch.zeros((w.N, 2 * R, w.Hkv, w.hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
                m.cache.read(l, i32([0] * 3), m.cache.len, K, V)
                got.append((K, V))
            assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert_bf16_close(host(a.Xb) - host(X0), host(b.Xb) - host(X0), f"Xb at {lens}")
    for bad in (0, R_MAX + 1):
        with pytest.raises(ValueError):
            a.step(H, X0, i32(n_new), R=bad)


@pytest.mark.parametrize("fc", [0, 1])
@pytest.mark.parametrize("rule", [0, 1, 2])
def test_sampling_and_self_selection(fc, rule):
    # without logits of its own the step lends the feature area to them
    w = workload(hd=128, Hq=8, Hkv=2, B=9, fc=fc, K=6)
    kw = dict(tv=True, accept_rule=rule, accept_seed=77, page=16)
    a, b = model(dfl.PagedDraftModel, w, 30, **kw), model(dfl.PagedDraftModel, w, 30, **kw)
    a.want_logits()
    rng, X0 = np.random.default_rng(rule), torch.from_numpy(gen_block_init(w)).cuda()
    vlog = bf16(rng, (w.N, w.K, w.B, w.V), 2.0)
    for n_new in ([24, 5, 0], [3, 24, 1]):
        H = bf16(rng, (w.L, w.N * R_MAX, w.d))
        for m in (a, b):
            m.step(H, X0, i32(n_new), vlog=vlog)
        z = host(a.logits).reshape(w.N, w.B - 1, w.V).astype(np.float64)
        check_samples(host(a.samples), lambda n, j: z[n, j], w.philox_seed, w.K, w.T,
                      [(n, j) for n in range(w.N) for j in (0, 3, 7)])
        for k in ("samples", "scores", "selected", "accept_len", "bonus", "tv_alpha", "tv_tokens", "draft", "Xb"):
            assert torch.equal(getattr(a, k), getattr(b, k)), k
        assert torch.equal(a.cache.book, b.cache.book)
    assert (host(a.selected) < w.K).all() and (host(a.accept_len) <= w.B - 1).all()
