"""fp64 gradients of the attention (given lists) and of the norm with rotation.

``attention_backward`` states the gradient of one forward pass: its inputs are
those of the library's entry point (q, k, v, the centroid operands, the saved o
and lse, the incoming gradient), and beside each gradient it returns a bound of
what bf16 probabilities and bf16 outputs may be off, term by term:

  u  = 2^-8   half a bf16 step relative to a value (the rounding of p, of ds and
              of the outputs);
  e1 = D X 2^-24 + 2^-20 with X the largest sum of |logit products| (fp32 sums
              of D products, and the exponential);
  e2 = 2 D 2^-24 (fp32 sums of dp and delta).

A sum of rounded terms is then off by at most (u + e1) times the sum of the
terms' magnitudes, plus e2 times the magnitudes behind the difference dp - delta,
and the stored value by u times itself.  Bounds of sums are carried through the
pooling's gradient linearly.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import sol_ref

U = 2.0 ** -8


def rows_of(N: int, nb: int, j: int):
    return np.arange(64 * j, min(N, 64 * (j + 1)))


def attention_backward(Q, K, V, dO, O, lse, sel, kc, vc, off, prefix=0, mode=0, centroids=True, scale=None,
                       tap=lambda name, x: x):
    """Gradients (and bounds) of one (b, h): Q, K, V, dO, O [N, D]; lse [N]; sel [nb, nb];
    kc, vc [nb, D] and off [nb] the centroid operands as the attention read them.  ``tap`` sees a few
    intermediate values by name and returns what is used instead: tests plant mistakes with it."""
    N, D = Q.shape
    s = 1.0 / math.sqrt(D) if scale is None else scale
    nb = sel.shape[0]
    blk = np.arange(N) // 64
    seen = sel[blk][:, blk]                                        # [N, N]
    x = s * Q @ K.T
    live = np.where(np.isfinite(lse), lse, np.inf)[:, None]        # a row without terms has p = 0
    with np.errstate(over="ignore"):
        p = np.where(seen, np.exp(np.where(seen, x, -np.inf) - live), 0.0)
    dO = np.where(np.isfinite(lse)[:, None], dO, 0.0)
    O = np.where(np.isfinite(lse)[:, None], O, 0.0)
    delta = (dO * O).sum(1, keepdims=True)
    mag = (np.abs(dO) * np.abs(O)).sum(1, keepdims=True)
    ds = p * (dO @ V.T - delta)
    dsm = p * (np.abs(dO) @ np.abs(V).T + mag)
    X = s * float((np.abs(Q) @ np.abs(K).T).max())
    e1, e2 = D * X * 2.0 ** -24 + 2.0 ** -20, 2 * D * 2.0 ** -24
    aQ, aK, adO = np.abs(Q), np.abs(K), np.abs(dO)

    def prod(A, Am, Y):   # a sum of rounded terms A against Y, and its bound
        return A @ Y, (U + e1) * (np.abs(A) @ np.abs(Y)) + e2 * (Am @ np.abs(Y))

    dq, bq = prod(s * ds, s * dsm, K)
    dk, bk = prod(s * ds.T, s * dsm.T, Q)
    dv, bv = prod(p.T, 0 * p.T, dO)
    if centroids:
        seen_c = sel[blk]
        xc = s * Q @ kc.T + off
        with np.errstate(over="ignore"):
            pc = np.where(seen_c, 0.0, np.exp(np.where(seen_c, -np.inf, xc) - live))
        dsc = pc * (dO @ vc.T - delta)
        dscm = pc * (np.abs(dO) @ np.abs(vc).T + mag)
        g, b = prod(s * dsc, s * dscm, kc)
        dq, bq = dq + g, bq + b
        gk, egk = prod(s * dsc.T, s * dscm.T, Q)
        gv, egv = prod(pc.T, 0 * pc.T, dO)
        gb = tap("gb terms", dsc).sum(0)
        egb = e1 * np.abs(dsc).sum(0) + e2 * dscm.sum(0)
        lo = prefix if prefix < N else 0
        a = Q[lo:].mean(0)
        da, eda = np.zeros(D), np.zeros(D)
        for j in range(nb):
            r = rows_of(N, nb, j)
            n = len(r)
            e = s * K[r] @ a
            w = np.exp(e - e.max())
            w /= w.sum()
            if mode == 2:
                h = K[r] @ gk[j] + V[r] @ gv[j] - gb[j] * e
                eh = aK[r] @ egk[j] + np.abs(V[r]) @ egv[j] + egb[j] * np.abs(e)
                eh = eh + e1 * (aK[r] @ np.abs(gk[j]) + np.abs(V[r]) @ np.abs(gv[j]) + abs(gb[j]) * np.abs(e))
                beta = s * w * (h - (w * h).sum())
                eb = s * w * (eh + (w * eh).sum()) + e1 * np.abs(beta)
                al = w
            else:
                al = np.full(n, 1.0 / n)
                beta = s * gb[j] * (w - 1.0 / n) if mode == 1 else np.zeros(n)
                eb = s * (egb[j] + e1 * abs(gb[j])) * np.abs(w - 1.0 / n) + e1 * s * abs(gb[j]) * (w + 1.0 / n) if mode == 1 else np.zeros(n)
            dk[r] += al[:, None] * gk[j] + tap("beta of dk", beta)[:, None] * a
            bk[r] += al[:, None] * (egk[j] + e1 * np.abs(gk[j])) + (eb + e1 * np.abs(beta))[:, None] * np.abs(a)
            dv[r] += al[:, None] * gv[j]
            bv[r] += al[:, None] * (egv[j] + e1 * np.abs(gv[j]))
            da += beta @ K[r]
            eda += (eb + e1 * np.abs(beta)) @ aK[r]
        if mode:
            at = tap("first anchor row", lo)
            dq[at:] += tap("da", da) / (N - at)
            bq[lo:] += eda / (N - lo)
    return [(g, b + U * np.abs(g) + 1e-30) for g, b in ((dq, bq), (dk, bk), (dv, bv))]


def centroid_operands(Q, K, V, prefix, mode):
    """kc, vc [nb, D] and off [nb] of one head in fp64 (no rounding)."""
    N, D = Q.shape
    four = lambda x: x[None, :, None, :]
    n = np.log(sol_ref.block_rows(N, 64).astype(np.float64))
    s = 1.0 / math.sqrt(D)
    kc, vc = sol_ref.pool(four(K), 64)[0, 0], sol_ref.pool(four(V), 64)[0, 0]
    if mode == 0:
        return kc, vc, n
    if mode == 1:
        return kc, vc, n + sol_ref.log_mass_bias(four(Q), four(K), kc[None, None], prefix, s, 64)[0, 0]
    kt, vt, bias = sol_ref.reweighted_summaries(four(Q), four(K), four(V), prefix, s, 64)
    return kt[0, 0], vt[0, 0], n + bias[0, 0]


def rotate(y, cos, sin, interleaved, sign=1.0):
    """The leading 2 * cos.shape[-1] dims of y [B, N, H, D] turned; cos, sin [B or 1, N, half]."""
    half = cos.shape[-1]
    c, sn = cos[:, :, None], sign * sin[:, :, None]
    out = y.copy()
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out[..., a] = y[..., a] * c - y[..., b] * sn
    out[..., b] = y[..., b] * c + y[..., a] * sn
    return out


def norm_rope(x, w, cos, sin, eps, interleaved):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotate(x * r * w, cos, sin, interleaved)


def norm_rope_backward(x, w, cos, sin, eps, interleaved, dz):
    """dx, dw and the sum of magnitudes behind each element of dw."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = rotate(dz, cos, sin, interleaved, -1.0)
    u = g * w
    dx = r * (u - x * r * r * (u * x).mean(-1, keepdims=True))
    ax = (0, 1, 2)
    return dx, (g * x * r).sum(ax), np.abs(g * x * r).sum(ax)
