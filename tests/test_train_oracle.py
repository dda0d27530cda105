"""The fp64 gradients of oracle/train_ref.py against central differences of the
forward oracle, and the bounds that the GPU tests use against planted roundings."""
import math

import numpy as np
import pytest

from oracle import sol_ref, train_ref
from tests import anchor_cases


def _problem(N, D, prefix, seed):
    rng = np.random.default_rng(seed)
    Q, K, V, dO = (rng.standard_normal((N, D)) for _ in range(4))
    nb = -(-N // 64)
    sel = rng.random((nb, nb)) < 0.4
    sel[: -(-prefix // 64)] = True
    sel[:, : -(-prefix // 64)] = True
    return rng, Q, K, V, dO, sel


def _loss(Q, K, V, dO, sel, prefix, mode, centroids):
    four = lambda x: x[None, :, None, :]
    if centroids:
        O = sol_ref.sol_forward(four(Q), four(K), four(V), prefix=prefix, mask_override=sel[None, None],
                                log_mass_bias_on=mode == 1, reweight_on=mode == 2)["O"]
    else:
        nb = sel.shape[0]
        z = np.zeros((1, 1, nb, Q.shape[1]))
        O, _ = sol_ref.attention(four(Q), four(K), four(V), sel[None, None], z, z, np.zeros((1, 1, nb)),
                                 1.0 / math.sqrt(Q.shape[1]), 64, 64, centroids=False)
    return float((O[0, :, 0] * dO).sum()), O[0, :, 0]


def _lse(Q, K, kc, off, sel, centroids):
    N, D = Q.shape
    blk = np.arange(N) // 64
    s = 1.0 / math.sqrt(D)
    x = np.where(sel[blk][:, blk], s * Q @ K.T, -np.inf)
    if centroids:
        x = np.concatenate([x, np.where(sel[blk], -np.inf, s * Q @ kc.T + off)], 1)
    m = x.max(1, keepdims=True)
    return (m + np.log(np.exp(x - m).sum(1, keepdims=True)))[:, 0]


def _backward(Q, K, V, dO, sel, prefix, mode, centroids):
    _, O = _loss(Q, K, V, dO, sel, prefix, mode, centroids)
    kc, vc, off = train_ref.centroid_operands(Q, K, V, prefix, mode)
    return train_ref.attention_backward(Q, K, V, dO, O, _lse(Q, K, kc, off, sel, centroids), sel, kc, vc, off, prefix,
                                        mode, centroids)


@pytest.mark.parametrize("N,prefix", [(150, 0), (200, 13), (65, 0), (130, 130), (70, 64)])
@pytest.mark.parametrize("mode,centroids", [(0, True), (1, True), (2, True), (0, False)])
def test_attention_gradient_against_differences(N, prefix, mode, centroids):
    D = 8
    rng, Q, K, V, dO, sel = _problem(N, D, prefix, 3 * N + mode)
    if not centroids:
        sel |= np.eye(sel.shape[0], dtype=bool)
    grads = _backward(Q, K, V, dO, sel, prefix, mode, centroids)
    h = 1e-5
    for x, (g, _) in zip((Q, K, V), grads):
        for _ in range(3):   # along random directions: every element takes part
            u = rng.standard_normal(x.shape)
            x += h * u
            up, _ = _loss(Q, K, V, dO, sel, prefix, mode, centroids)
            x -= 2 * h * u
            down, _ = _loss(Q, K, V, dO, sel, prefix, mode, centroids)
            x += h * u
            # third-derivative error h^2 and a cancellation of 2^-52 |loss| / h
            assert abs((up - down) / (2 * h) - (g * u).sum()) <= 1e-6 * (1 + np.abs(g * u).sum())


def test_bounds_hold_for_rounded_probabilities_and_catch_a_dropped_term():
    D, N = 16, 150
    _, Q, K, V, dO, sel = _problem(N, D, 0, 5)
    sel |= np.eye(sel.shape[0], dtype=bool)
    (dq, bq), _, (dv, bv) = _backward(Q, K, V, dO, sel, 0, 0, False)
    blk = np.arange(N) // 64
    _, O = _loss(Q, K, V, dO, sel, 0, 0, False)
    s = 1.0 / math.sqrt(D)
    kc, vc, off = train_ref.centroid_operands(Q, K, V, 0, 0)
    lse = _lse(Q, K, kc, off, sel, False)
    seen = sel[blk][:, blk]
    p = np.where(seen, np.exp(s * Q @ K.T - np.where(np.isfinite(lse), lse, np.inf)[:, None]), 0.0)
    ds = sol_ref.bf16_round(p * (dO @ V.T - np.where(np.isfinite(lse), (dO * O).sum(1), 0.0)[:, None]))
    assert (np.abs(sol_ref.bf16_round(s * ds @ K) - dq) <= bq).all()
    assert (np.abs(sol_ref.bf16_round(sol_ref.bf16_round(p).T @ dO) - dv) <= bv).all()
    assert (np.abs(s * (ds + 0.05 * p) @ K - dq) > bq).any()      # a wrong delta
    assert (np.abs(1.05 * dv - dv) > bv).any()


@pytest.mark.parametrize("half,interleaved", [(4, False), (2, True), (0, False)])
def test_norm_rope_gradient_against_differences(half, interleaved):
    rng = np.random.default_rng(half)
    x, dz = rng.standard_normal((2, 3, 2, 8)), rng.standard_normal((2, 3, 2, 8))
    w, ang = 1 + 0.1 * rng.standard_normal(8), rng.standard_normal((1, 3, half))
    cos, sin, eps = np.cos(ang), np.sin(ang), 1e-3
    dx, dw, _ = train_ref.norm_rope_backward(x, w, cos, sin, eps, interleaved, dz)
    f = lambda x, w: float((train_ref.norm_rope(x, w, cos, sin, eps, interleaved) * dz).sum())
    h = 1e-5
    for _ in range(4):
        u, v = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
        assert abs((f(x + h * u, w) - f(x - h * u, w)) / (2 * h) - (dx * u).sum()) < 1e-7 * (1 + np.abs(dx * u).sum())
        assert abs((f(x, w + h * v) - f(x, w - h * v)) / (2 * h) - (dw * v).sum()) < 1e-7 * (1 + np.abs(dw * v).sum())


def test_rotation_is_orthogonal_and_pairs_as_named():
    rng = np.random.default_rng(0)
    y, ang = rng.standard_normal((1, 2, 1, 8)), rng.standard_normal((1, 2, 3))
    for inter in (False, True):
        z = train_ref.rotate(y, np.cos(ang), np.sin(ang), inter)
        assert np.allclose(train_ref.rotate(z, np.cos(ang), np.sin(ang), inter, -1.0), y)
        assert np.array_equal(z[..., 6:], y[..., 6:])
        a, b = (2, 3) if inter else (1, 4)
        assert np.allclose(z[0, 1, 0, a] + 1j * z[0, 1, 0, b],
                           (y[0, 1, 0, a] + 1j * y[0, 1, 0, b]) * np.exp(1j * ang[0, 1, 1]))


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("N,D,prefix", anchor_cases.CASES)
def test_bounds_catch_mistakes_in_the_anchor_s_terms(N, D, prefix, mode):
    """On the inputs of the GPU's anchor test every one of these mistakes exceeds the bound twice over."""
    Q, K, V, dO, sel = anchor_cases.inputs(N, D, prefix)
    kc, vc, off = train_ref.centroid_operands(Q, K, V, prefix, mode)
    kc, vc = sol_ref.bf16_round(kc), sol_ref.bf16_round(vc)
    lse = _lse(Q, K, kc, off, sel, True)
    blk, s = np.arange(N) // 64, 1.0 / math.sqrt(D)
    p = np.exp(np.where(sel[blk][:, blk], s * Q @ K.T, -np.inf) - lse[:, None])
    pc = np.exp(np.where(sel[blk], -np.inf, s * Q @ kc.T + off) - lse[:, None])
    O = sol_ref.bf16_round(p @ V + pc @ vc)
    back = lambda tap: train_ref.attention_backward(Q, K, V, dO, O, lse, sel, kc, vc, off, prefix, mode, tap=tap)
    want = back(lambda name, x: x)
    nb = len(sel)
    splits = (nb + 3) // 4 if nb <= 32 else min(8, (nb + 15) // 16)   # query ranges of the centroid pass
    first = (np.arange(N) < 64 * (nb // splits))[:, None]
    plant = {"no da": ("da", lambda x: 0 * x), "da's sign": ("da", lambda x: -x),
             "no gb": ("gb terms", lambda x: 0 * x), "no beta a": ("beta of dk", lambda x: 0 * x)}
    if splits > 1:
        plant["gb of the first range only"] = "gb terms", lambda x: np.where(first, x, 0.0)
    if 0 < prefix < N:
        plant["da on every row"] = "first anchor row", lambda x: 0
    for mistake, (at, f) in plant.items():
        got = back(lambda name, x: f(x) if name == at else x)
        assert max((np.abs(g - w) / b).max() for (g, _), (w, b) in zip(got, want)) >= 2.0, mistake
