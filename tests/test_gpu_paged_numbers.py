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
