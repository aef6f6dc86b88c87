"""Attention over the paged 4-bit cache at the ends of the number range (GPU).

The bound where scores are ordinary is test_gpu_paged_edges.py's.
"""
import numpy as np
import pytest
import torch

import block_diffusion_speculative_dfl_gb300 as dfl
from gpu_util import host
from oracle import kv4_oracle as ko
from test_gpu_paged import bf16, fill, i32, make_cache

pytestmark = pytest.mark.gpu

# one head's query rows: 2, 8 and 16 (warp products), 64 and 128 (tensor memory)
ROWS = [(1, 2, 64), (2, 4, 128), (4, 4, 128), (4, 4, 64), (16, 4, 128), (16, 4, 64), (16, 8, 128), (16, 8, 64)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.build()
    dfl.load()
    torch.cuda.set_device(0)
    yield
    assert dfl.dfl_get_device_error() == 0


@pytest.mark.parametrize("B,Hq,hd", ROWS)
@pytest.mark.parametrize("lens", [[400], [2000], [9000, 3], [33] * 40])
def test_own_keys_of_score_minus_infinity_weigh_nothing(B, Hq, hd, lens):
    # with few sequences the line is cut into single units, and the own rows' unit has a range of its own
    rng = np.random.default_rng(B + hd)
    c = make_cache(rng, len(lens), lens, 16, 1, hd)
    K, V = fill(rng, c, 0, lens)
    N = c.N
    Q, Kb, Vb = bf16(rng, (N, B, Hq, hd)), bf16(rng, (N, B, 1, hd)), bf16(rng, (N, B, 1, hd))
    Q[..., 0] = Q[..., 0].abs() + 0.25
    for first in (0, 1):   # all of the own keys, all but one
        Kb[:, first:, 0, 0] = -float("inf")
        Kb[:, :first, 0, 0] = 1.0
        O = host(c.attn(0, Q, Kb, Vb)).astype(np.float64)
        Kd, Vd = ko.kv4_values(K, 0), ko.kv4_values(V, 0)
        q, kb, vb = (host(x).astype(np.float64) for x in (Q, Kb, Vb))
        for n in {0, N // 2, N - 1}:
            l = lens[n]
            ref, Ac, Ab, smax = ko.paged_attn(q[n], Kd[n, :l], Vd[n, :l], kb[n, :first], vb[n, :first])
            vmax = max(np.abs(Vd[n, :l]).max(initial=0), np.abs(vb[n]).max())
            tol = 2.0 ** -8 * np.abs(ref) + (1.01 * 2.0 ** -11 + 2.0 ** -18 * (1 + smax)) * (Ac + Ab) + \
                (l + B) * 2.0 ** -32 * vmax + 2.0 ** -25 + 1e-30
            err = np.abs(O[n] - ref)
            assert (err <= tol).all(), (first, n, float((err / tol).max()))


@pytest.mark.parametrize("B,Hq,hd", ROWS)
def test_rows_without_any_finite_score_are_nan_and_alone(B, Hq, hd):
    # nothing cached and every own score -inf: 0 / 0, in that head only
    rng = np.random.default_rng(B + hd)
    c = make_cache(rng, 2, [0, 0], 16, 2, hd)
    Q, Kb, Vb = bf16(rng, (2, B, 2 * Hq, hd)), bf16(rng, (2, B, 2, hd)), bf16(rng, (2, B, 2, hd))
    Q[..., 0] = 1.0
    Kb[0, :, 0, 0] = -float("inf")
    O = host(c.attn(0, Q, Kb, Vb))
    assert np.isnan(O[0, :, :Hq]).all() and np.isfinite(O[0, :, Hq:]).all() and np.isfinite(O[1]).all()


def _one_hot(c, K, V, Q, Kb, Vb, O, lens):
    """Scores so far apart that every weight but the largest keys' is 0: the mean of their values, rounded once to bf16,
    with the weights' fp16 rounding (2^-11) and fp32's in the sums."""
    Kd, Vd = ko.kv4_values(K, 0), ko.kv4_values(V, 0)
    q, kb, vb, O = (host(x).astype(np.float64) for x in (Q, Kb, Vb, O))
    for n, l in enumerate(lens):
        ref, Ac, Ab, _ = ko.paged_attn(q[n], Kd[n, :l], Vd[n, :l], kb[n], vb[n])
        tol = 2.0 ** -8 * np.abs(ref) + (1.01 * 2.0 ** -11 + 2.0 ** -20) * (Ac + Ab) + 2.0 ** -25
        err = np.abs(O[n] - ref)
        assert (err <= tol).all(), (n, float(np.nanmax(err / tol)), bool(np.isnan(err).any()))


@pytest.mark.parametrize("B,Hq,hd", ROWS)
@pytest.mark.parametrize("power", [20, 23, 26, 29, 33, 40, 90])
def test_scores_of_any_size_give_the_largest_keys_values(B, Hq, hd, power):
    # one dimension carries scores: the codes' steps of 0.5 make gaps of 2^(power - 6) at least
    rng = np.random.default_rng(power + hd + B)
    lens = [700, 1500, 0]
    c = make_cache(rng, 3, lens, 16, 1, hd)
    K, V = torch.zeros((3, 1500, 1, hd)), bf16(rng, (3, 1500, 1, hd))
    K[:, :, 0, 0] = torch.from_numpy(rng.choice([0.5, 1.0, 1.5, 2.0, 3.0, -1.0, -6.0], (3, 1500)))
    K[:, :, 0, 1] = 6.0   # every token's scale is 1
    K[0, 123, 0, 0], K[1, 1400, 0, 0], K[1, 77, 0, 0] = 4.0, 6.0, 6.0
    K = K.to(torch.bfloat16).cuda()
    c.append(0, K, V, i32([0] * 3), i32(lens))
    Q = torch.zeros((3, B, Hq, hd), device="cuda")
    Q[..., 0] = 2.0 ** power * (1 + torch.from_numpy(rng.random((3, B, Hq)).astype(np.float32)).cuda())
    Q[:, :, 1::2] *= -1   # the lowest keys are the largest scores, or all scores are far below zero
    Q = Q.to(torch.bfloat16)
    Kb, Vb = torch.zeros((3, B, 1, hd), dtype=torch.bfloat16, device="cuda"), bf16(rng, (3, B, 1, hd))
    Kb[:, :, 0, 0] = 1.0
    O = c.attn(0, Q, Kb, Vb)
    _one_hot(c, host(K).astype(np.float64), host(V).astype(np.float64), Q, Kb, Vb, O, lens)


@pytest.mark.parametrize("B,Hq,hd", ROWS)
def test_scores_one_fp32_step_apart_stay_in_the_values_hull(B, Hq, hd):
    # tokens after the first 64 score higher by a few steps of fp32 at 2^25 to 2^29: whatever these weigh, no output leaves the values
    rng = np.random.default_rng(hd + B)
    for step, last in ((0.5, 250), (1.0, 250), (2.0, 700), (6.0, 700)):   # whole triples, cut ones
        lens = [64, 128, last]
        c = make_cache(rng, 3, lens, 16, 1, hd)
        K, V = torch.zeros((3, 700, 1, hd)), bf16(rng, (3, 700, 1, hd))
        K[:, :, 0, 0] = 1.0
        K[:, 64:, 0, 16] = step * 2.0 ** -9   # another group, of the smallest scale
        c.append(0, K.to(torch.bfloat16).cuda(), V, i32([0] * 3), i32(lens))
        Kb, Vb = torch.zeros((3, B, 1, hd), dtype=torch.bfloat16, device="cuda"), bf16(rng, (3, B, 1, hd))
        Kb[:, :, 0, 0] = 1.0
        top = max(float(V.abs().max()), float(Vb.abs().max()))
        for power in range(27, 33):
            Q = torch.zeros((3, B, Hq, hd), dtype=torch.bfloat16, device="cuda")
            Q[..., 0], Q[..., 16] = 2.0 ** power * 1.5, 2.0 ** (power - 14) * 1.5
            O = c.attn(0, Q, Kb, Vb).float()
            assert bool(torch.isfinite(O).all()) and float(O.abs().max()) <= top * (1 + 2.0 ** -7), (step, power)


@pytest.mark.parametrize("B,Hq,hd", ROWS)
@pytest.mark.parametrize("q,k_exp", [(1e-36, -60), (1e-38, 0), (1e-38, -30), (2e38, 0), (-3.3e38, -60), (1e38, 60), (0.0, 60)])
def test_queries_at_the_ends_of_bf16(B, Hq, hd, q, k_exp):
    # scores that are all equal (keys of 0), or closer than 2^-20: the mean of the values
    rng = np.random.default_rng(hd + B)
    lens = [300, 37, 1200]
    c = make_cache(rng, 3, lens, 16, 1, hd, k_exp=k_exp)
    tiny = abs(q) < 1e-30
    K, V = bf16(rng, (3, 1200, 1, hd)) * (2.0 ** k_exp if tiny and q else 0), bf16(rng, (3, 1200, 1, hd))
    c.append(0, K, V, i32([0] * 3), i32(lens))
    Q = bf16(rng, (3, B, Hq, hd)) * q if tiny else torch.zeros((3, B, Hq, hd), dtype=torch.bfloat16, device="cuda")
    if not tiny:
        Q[..., 3] = q
    Kb, Vb = torch.zeros((3, B, 1, hd), dtype=torch.bfloat16, device="cuda"), bf16(rng, (3, B, 1, hd))
    O = host(c.attn(0, Q, Kb, Vb)).astype(np.float64)
    Vd, vb = ko.kv4_values(host(V).astype(np.float64), 0), host(Vb).astype(np.float64)
    for n, l in enumerate(lens):
        v = np.concatenate([Vd[n, :l], vb[n]])[:, 0]
        ref, mean_abs = v.mean(0), np.abs(v).mean(0)
        tol = 2.0 ** -8 * np.abs(ref) + (1.01 * 2.0 ** -11 + 2.0 ** -18) * mean_abs + 2.0 ** -25
        assert (np.abs(O[n] - ref) <= tol).all(), n
