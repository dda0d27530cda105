"""Inputs on which the anchor's terms of the gradient are far above the roundings.

The centroid modes 1 and 2 send gradients through the anchor (the mean of the query
rows past the prefix): the offset's gradient gb, summed over every query; beta a in dk;
da = sum beta_t k_t over all rows, spread over the anchor's rows.  On centred normal
inputs the anchor is small, and these terms disappear below the rounding of the
others.  Here the queries share a large mean, the keys of a block spread along it (by
a width of the block's own), and dO points along a direction in which the blocks'
values differ, so that ds keeps its sign over many queries; inside a block the values
follow the keys along it (under mode 2 the means' own share cancels).  The lists are
the caller's and leave a share of the blocks to their centroids, whatever the prefix.
"""
import numpy as np

from oracle import sol_ref

# (N, D, prefix): one and several query ranges of the centroid pass, ragged ends, anchors of all rows, of
# those past a prefix, and of all rows again where the prefix is the whole sequence
CASES = [(200, 64, 0), (640, 64, 640), (777, 64, 13), (1000, 128, 100), (1300, 128, 0), (520, 128, 520), (2113, 64, 1500)]


def inputs(N, D, prefix, seed=0):
    """q, k, v, dO [N, D] with bf16 values, and the lists sel [nb, nb]."""
    rng = np.random.default_rng(1000 * seed + N + D + prefix)
    nb = -(-N // 64)
    blk = np.arange(N) // 64
    unit = lambda: (lambda x: x / np.sqrt((x * x).sum()))(rng.standard_normal(D))
    mean, along = unit(), unit()
    q = 0.5 * rng.standard_normal((N, D)) + 0.5 * np.sqrt(D) * mean
    z = rng.standard_normal(N)
    k = 0.5 * rng.standard_normal((N, D)) + (rng.uniform(1.0, 5.0, nb)[blk] * z)[:, None] * mean
    v = 0.5 * rng.standard_normal((N, D)) + (2.0 * rng.standard_normal(nb)[blk] + 2.0 * z)[:, None] * along
    do = 0.1 * rng.standard_normal((N, D)) + along
    sel = rng.random((nb, nb)) < 0.3
    sel[np.arange(nb), rng.integers(0, nb, nb)] = True
    return *(sol_ref.bf16_round(x) for x in (q, k, v, do)), sel
