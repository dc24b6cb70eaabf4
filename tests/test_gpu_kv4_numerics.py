"""Attention over the 4-bit cache where numbers are far apart, against the float64 oracle."""

import numpy as np
import pytest
import torch

import block_causal_streaming_sa_b200 as sa
from oracle import kv4
from test_gpu_kv4 import BF, HALF, HF, Pair, f64, normal, score_error

pytestmark = pytest.mark.gpu

# P enters the second product as fp16 with the row's largest at 2^10 or above (its half step
# below 2^-14 is 2^-25): relative to the largest, what a rounding of a small P is off by.
P_FLOOR = 2.0 ** -(25 + 10)


@pytest.mark.parametrize("nats,n", [(12.0, 4093), (17.4, 43_200), (20.0, 262_144)])
@pytest.mark.parametrize("T,D,dtype,causal", [(1, 128, BF, False), (8, 64, HF, True),
                                              (24, 128, HF, False), (64, 64, BF, True),
                                              (130, 128, BF, False), (300, 64, HF, True),
                                              (513, 128, HF, True)])
def test_attend_behind_a_row_that_dominates(T, D, dtype, causal, nats, n):
    """The first row's score lies far above all others', which are nearly even, and its V is
    zero: O is what the others have together, each far below the largest probability."""
    p = Pair(1, 1, D, -(-n // 128) * 128, dtype)
    tag = ("sink", T, D, nats)
    K, V = normal((tag, "k"), (1, n, 1, D), dtype, 0.2), normal((tag, "v"), (1, n, 1, D), dtype, 0.2)
    V += 0.5
    K[..., 0] = 0
    K[0, 0, 0], V[0, 0, 0] = 0, 0
    K[0, 0, 0, 0] = nats * D ** 0.5 / 4
    Q = normal((tag, "q"), (1, T, 1, D), dtype)
    Q[..., 0] = 4
    p.gpu.append(K.cuda(), V.cuda())
    p.ref.append(f64(K), f64(V))
    out = torch.empty((1, T, 1, D), dtype=dtype, device="cuda")
    lse = torch.empty((1, 1, T), device="cuda")
    p.gpu.attend(Q.cuda(), causal=causal, out=out, lse=lse, add_weight=True)
    O, L, A, E = p.ref.attend(f64(Q), causal=causal, add_weight=True)
    err = score_error(D, E)
    # as for any attention (p off by e^err, its rounding by half a step, the normalisation, the
    # output's rounding), and small p by P_FLOOR of the largest
    tol = (2 * np.transpose(err, (0, 2, 1))[..., None] + 2.0 ** -11 + 2.0 ** -20) * A \
        + P_FLOOR * np.abs(p.ref.v[0][0]).sum(axis=0) + HALF[dtype] * np.abs(O) + 1e-8
    d = np.abs(f64(out) - O)
    assert np.all(d <= tol), f"off by {(d / np.abs(O)).max():.2e} of O, {(d / tol).max():.2f} of the tolerance"
    assert np.all(np.abs(f64(lse) - L) <= err + 4 * 2.0 ** -24 * np.abs(L))
    p.check_weights(1, float(E.max()))
    assert p.gpu.check() == sa.SA_OK


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,n", [(1, 200), (20, 200), (130, 200), (130, 30_000)])
def test_a_query_that_is_not_finite_has_a_nan_lse(T, n, value):
    """Few and many query rows, whole items and items split over blocks; -inf is for queries
    that see no row, and the other queries' lse stay."""
    p = sa.QuantKVCache(1, 1, 128, -(-n // 128) * 128)
    K = normal(("nlse", n), (1, n, 1, 128), BF).cuda()
    p.append(K, K)
    Q = normal(("nlse", T), (1, T, 2, 128), BF).cuda()
    want, lse = (torch.empty((1, 2, T), device="cuda") for _ in range(2))
    p.attend(Q, lse=want)
    Q[0, 0, 1, 7] = value
    out = p.attend(Q, lse=lse)
    assert torch.isnan(lse[0, 1, 0]) and torch.isnan(out[0, 0, 1].float()).all()
    same = torch.ones((1, 2, T), dtype=torch.bool, device="cuda")
    same[0, 1, 0] = False
    assert torch.equal(lse[same], want[same]) and torch.isfinite(want).all()


@pytest.mark.parametrize("T,causal", [(8, False), (8, True), (24, False), (24, True),
                                      (130, False), (130, True)])
def test_a_nan_query_leaves_nan_weights_that_an_eviction_drops_first(T, causal):
    """Whichever of eight neighbouring queries it is: the rows it sees draw NaN, the others
    what they draw without it, bit for bit; NaN ranks below every number."""
    D, n = 64, 200
    p = Pair(1, 1, D, 256)
    p.append(("nanw", T), n)
    Q = normal(("nanw", T), (1, T, 1, D), BF).cuda()
    p.gpu.weight.zero_()
    p.gpu.attend(Q, causal=causal, add_weight=True)
    want = p.gpu.weight[0, 0, :n].clone()
    assert torch.isfinite(want).all() and (want > 0).all()
    for t in range(T - 8, T):
        q = Q.clone()
        q[0, t, 0, 3] = float("nan")
        p.gpu.weight.zero_()
        p.gpu.attend(q, causal=causal, add_weight=True)
        seen = n - T + t + 1 if causal else n
        w = p.gpu.weight[0, 0, :n]
        assert torch.isnan(w[:seen]).all(), t
        assert torch.equal(w[seen:], want[seen:]), t
    if causal:  # the last query sees every row: take the first of the eight
        q = Q.clone()
        q[0, T - 8] = float("nan")
        p.gpu.weight.zero_()
        p.gpu.attend(q, causal=True, add_weight=True)
        p.gpu.evict(7)
        assert p.gpu.pos[0, 0, :7].tolist() == list(range(n - 7, n))


@pytest.mark.parametrize("T", [1, 20, 130])
def test_a_query_whose_scores_are_all_minus_infinity_draws_nothing(T):
    p = sa.QuantKVCache(1, 1, 64, 128)
    K = torch.zeros((1, 90, 1, 64), dtype=BF, device="cuda")
    K[..., 5] = -6
    p.append(K, K)
    Q = normal(("minus", T), (1, T, 1, 64), BF).cuda()
    Q[0, 0, 0] = 0
    Q[0, 0, 0, 5] = float("inf")  # the keys are 0 elsewhere: no score is NaN
    lse = torch.empty((1, 1, T), device="cuda")
    out = p.attend(Q, lse=lse, add_weight=True)
    assert (out[0, 0] == 0).all() and lse[0, 0, 0] == -float("inf")
    w = p.weight[0, 0, :90].double()
    # the other queries see equal scores: their weight is T - 1 in all, spread evenly
    assert torch.allclose(w, torch.full_like(w, (T - 1) / 90), rtol=1e-5)


def test_rows_that_draw_nothing_from_many_queries_weigh_exactly_zero():
    """Probabilities too small for fp32 add zero, whichever way their exponential is taken,
    and so do the rows that pad the last tile of queries."""
    D, n, T = 128, 300, 131
    p = Pair(1, 1, D, 384)
    K = torch.zeros((1, n, 1, D), dtype=BF)
    K[0, 1:, 0, 0] = -60.0  # scores of 0, and of -4 * 60 * 11.3 = -2715 behind row 0
    p.gpu.append(K.cuda(), K.cuda())
    Q = torch.zeros((1, T, 1, D), dtype=BF)
    Q[..., 0] = 4
    p.gpu.attend(Q.cuda(), scale=11.3, add_weight=True)
    assert (p.gpu.weight[0, 0, 1:n] == 0).all()
    assert abs(float(p.gpu.weight[0, 0, 0]) - T) <= T * 2.0 ** -21


@pytest.mark.parametrize("T", [1, 6, 24, 140])
@pytest.mark.parametrize("D,dtype,qs", [(128, BF, 40.0), (64, HF, 20.0), (128, BF, 2.0 ** -30)])
def test_weights_of_large_and_sharp_scores(T, D, dtype, qs):
    """Keys of very different size: maxima that grow along the rows, probabilities of which
    most vanish, log-sum-exps in the hundreds."""
    p = Pair(1, 2, D, 1024, dtype)
    for i in range(4):
        p.append(("sharpw", T, i, D), 200, scale=0.3 * 3.0 ** i)
    e = p.check_attend(("sharpw", T, D, qs), T, 4, q_scale=qs, add_weight=True)
    p.check_weights(1, e)
    assert p.gpu.check() == sa.SA_OK
