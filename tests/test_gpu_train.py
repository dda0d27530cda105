"""Gradients on the GPU: sol_attn_bwd and sol_qk_norm_rope(_bwd) against the fp64
formulas of oracle/train_ref.py, element by element.

sol_attn_bwd is given what the forward left (o, lse, lists, centroid operands);
every element of dq, dk, dv has to lie within the bound that attention_backward
derives from the roundings of p, ds and the outputs to bf16 (2^-8 each) and from
fp32 sums.  The norm's outputs are fp32 inside and rounded once: 2^-8 of the
value plus 2^-18 of the magnitudes that it is the sum of (a dozen fp32 steps and
a reciprocal square root of two units in the last place).
"""
import numpy as np
import pytest
import torch

from block_sparse_video_sol_b200 import synth
from oracle import sol_ref, train_ref
from tests import anchor_cases, parity

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


@pytest.fixture(scope="module")
def sol():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from block_sparse_video_sol_b200 import build
    build.build()
    from block_sparse_video_sol_b200 import sol as mod
    return mod


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def inputs(B, N, H, D, seed, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda: torch.randn(B, N, H, D, generator=g, device="cuda")
    topic = torch.randn(B, -(-N // 32), H, D, generator=g, device="cuda").repeat_interleave(32, 1)[:, :N]
    return [(gain * (topic + r())).bfloat16() for _ in range(2)] + [r().bfloat16(), r().bfloat16()]


def check_grads(sol, p, buf, q, k, v, do, grads):
    """dq, dk, dv ([B, N, H, D]) of every head within the derived bounds."""
    _, _, mask = parity.gpu_mask(p, buf)
    w = sol.workspace_views(p, buf.ws)
    cent = p.routing != 1
    worst = 0.0
    for b in range(p.B):
        for h in range(p.H):
            want = train_ref.attention_backward(
                *(f64(x[b, :, h]) for x in (q, k, v, do, buf.o)), f64(buf.lse[b, h]), mask[b, h],
                f64(w["kbar16"][b, h]), f64(w["vbar16"][b, h]), f64(w["cbias"][b, h]), p.prefix_len, p.log_mass_bias,
                cent, p.scale or None)
            for name, got, (g, bound) in zip(("dq", "dk", "dv"), grads, want):
                x = f64(got[b, :, h])
                assert np.isfinite(x).all(), (name, b, h)
                ratio = (np.abs(x - g) / bound).max()
                assert ratio <= 1.0, (name, b, h, ratio, np.unravel_index((np.abs(x - g) / bound).argmax(), g.shape))
                worst = max(worst, ratio)
    return worst


def run(sol, B, N, H, D, seed=0, gain=1.0, **kw):
    q, k, v, do = inputs(B, N, H, D, seed, gain)
    p = sol.make_params(B, N, H, D, **kw)
    buf = sol.alloc_buffers(p, q.device, with_lse=True)
    sol.forward(p, q, k, v, buf)
    g = sol.alloc_grads(p, q.device)
    for t in (g.dq, g.dk, g.dv):
        t.fill_(float("nan"))
    g.ws.fill_(255)   # whatever the workspace held
    sol.backward(p, q, k, v, buf, do, g)
    sol.sol_last_device_status()
    return p, buf, (q, k, v, do), g


ROUTES = [dict(tau=0.5), dict(tau=0.5, log_mass_bias=1), dict(tau=0.5, log_mass_bias=2), dict(topk_ratio=0.3),
          dict(topk_ratio=0.2, compressed=True, log_mass_bias=2)]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N", [1, 5, 63, 64, 65, 128, 129, 200])
@pytest.mark.parametrize("route", range(5))
def test_short_lengths(sol, N, D, route):
    p, buf, (q, k, v, do), g = run(sol, 1, N, 2, D, seed=N, **ROUTES[route])
    check_grads(sol, p, buf, q, k, v, do, (g.dq, g.dk, g.dv))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("route", range(5))
@pytest.mark.parametrize("B,N,H,prefix", [(2, 1000, 3, 100), (1, 777, 2, 13), (1, 2113, 1, 0), (1, 640, 1, 640)])
def test_ragged_lengths_and_prefixes(sol, B, N, H, prefix, route, D):
    p, buf, (q, k, v, do), g = run(sol, B, N, H, D, seed=N, prefix_len=prefix, **ROUTES[route])
    check_grads(sol, p, buf, q, k, v, do, (g.dq, g.dk, g.dv))


@pytest.mark.parametrize("mode", [0, 2])
def test_every_centroid_range_and_long_lists(sol, mode):
    """N = 9,000: 141 blocks, eight query ranges of the centroid pass, several bitmap words."""
    p, buf, (q, k, v, do), g = run(sol, 1, 9000, 1, 128, seed=3, prefix_len=70, log_mass_bias=mode, tau=0.8)
    check_grads(sol, p, buf, q, k, v, do, (g.dq, g.dk, g.dv))


def test_all_blocks_exact_and_no_block_exact(sol):
    p, buf, (q, k, v, do), g = run(sol, 1, 500, 2, 128, tau=-float("inf"))
    check_grads(sol, p, buf, q, k, v, do, (g.dq, g.dk, g.dv))
    p, buf, (q, k, v, do), g = run(sol, 1, 500, 2, 128, tau=50.0)
    assert int(buf.row_ptr[-1]) == 0
    check_grads(sol, p, buf, q, k, v, do, (g.dq, g.dk, g.dv))


def test_large_logits_and_a_scale_of_its_own(sol):
    """Logits of +-100: the softmax is nearly one-hot and the saved normaliser far from zero."""
    p, buf, (q, k, v, do), g = run(sol, 1, 300, 2, 64, seed=9, gain=5.0, scale=0.3, tau=0.3, log_mass_bias=1)
    check_grads(sol, p, buf, q, k, v, do, (g.dq, g.dk, g.dv))


def test_empty_rows_and_repeated_entries(sol):
    """Caller's lists under routing 1: a tile without keys (its o and lse are never written), a tile with one
    empty half, a key block that nobody lists, and an entry listed twice."""
    B, N, H, D = 1, 64 * 6 + 10, 1, 128
    q, k, v, do = inputs(B, N, H, D, 4)
    p = sol.make_params(B, N, H, D, topk_ratio=0.3)
    buf = sol.alloc_buffers(p, q.device, with_lse=True)
    sol.sol_pool(p, q, k, v, buf.ws)
    lists = [[], [], [1, 1, 4], [], [0, 6], [2], [6]]
    buf.row_ptr.copy_(torch.tensor(np.cumsum([0] + [len(x) for x in lists]), dtype=torch.int32))
    flat = torch.tensor(sum(lists, []), dtype=torch.int32, device="cuda")
    buf.col_idx[:len(flat)] = flat
    buf.o.fill_(float("nan"))
    buf.lse.fill_(float("nan"))
    sol.sol_attn_fwd(p, q, k, v, buf.ws, buf.row_ptr, buf.col_idx, buf.o, buf.lse)
    g = sol.alloc_grads(p, q.device)
    sol.backward(p, q, k, v, buf, do, g)
    sol.sol_last_device_status()
    assert (g.dq[:, :128] == 0).all() and (g.dq[:, 192:256] == 0).all()
    for j in (3, 5):
        assert (g.dk[:, 64 * j:64 * (j + 1)] == 0).all() and (g.dv[:, 64 * j:64 * (j + 1)] == 0).all()
    # the oracle's lse of the empty rows: no terms
    rows = torch.zeros(N, dtype=torch.bool)
    rows[:128] = rows[192:256] = True
    buf.lse[:, :, rows] = -float("inf")
    buf.o[:, rows] = 0
    check_grads(sol, p, buf, q, k, v, do, (g.dq, g.dk, g.dv))


def test_bad_list_entry_is_reported_and_skipped(sol):
    p, buf, (q, k, v, do), g = run(sol, 1, 300, 1, 64, topk_ratio=0.4)
    want = [t.clone() for t in (g.dq, g.dk, g.dv)]
    n = int(buf.row_ptr[-1])
    rp, ci = buf.row_ptr.clone(), buf.col_idx.clone()
    rp[-1] += 2
    ci = torch.cat([ci[:n], torch.tensor([5, -1], dtype=torch.int32, device="cuda")])
    sol.sol_attn_bwd(p, q, k, v, buf.ws, rp, ci, buf.o, buf.lse, do, g.dq, g.dk, g.dv, g.ws)
    with pytest.raises(sol.SolError):
        sol.sol_last_device_status()
    assert all(torch.equal(a, b) for a, b in zip(want, (g.dq, g.dk, g.dv)))


def test_strided_views_head_runs_and_repeats_are_bit_identical(sol):
    B, N, H, D = 2, 700, 4, 128
    kw = dict(prefix_len=40, log_mass_bias=2, tau=0.5)
    q, k, v, do = inputs(B, N, H, D, 6)
    p = sol.make_params(B, N, H, D, **kw)
    buf = sol.alloc_buffers(p, "cuda", with_lse=True)
    sol.forward(p, q, k, v, buf)
    g = sol.alloc_grads(p, "cuda")
    sol.backward(p, q, k, v, buf, do, g)
    want = [t.clone() for t in (g.dq, g.dk, g.dv)]
    sol.backward(p, q, k, v, buf, do, g)
    assert all(torch.equal(a, b) for a, b in zip(want, (g.dq, g.dk, g.dv)))

    # views of fused projections in and out; an output gradient with strides of its own
    qkv = torch.stack((q, k, v), 2)
    dqkv = torch.full_like(qkv, float("nan"))
    views, gviews = qkv.unbind(2), dqkv.unbind(2)
    o3, do3 = (torch.empty(B, N, 2, H, D, dtype=q.dtype, device="cuda")[:, :, 1] for _ in range(2))
    o3.copy_(buf.o)
    do3.copy_(do)
    p2 = sol.make_params(B, N, H, D, in_strides=views[0].stride()[:3], out_strides=o3.stride()[:3], **kw)
    sol.sol_attn_bwd(p2, *views, buf.ws, buf.row_ptr, buf.col_idx, o3, buf.lse, do3, *gviews, g.ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, gviews))

    # heads 1 and 2 alone (the other heads' gradients stay as they were)
    sub = sol.make_params(B, N, 2, D, in_strides=q.stride()[:3], out_strides=q.stride()[:3], **kw)
    h12 = [t[:, :, 1:3] for t in (q, k, v)]
    b2 = sol.alloc_buffers(sub, "cuda")
    lse2 = torch.empty(B, 2, N, device="cuda")
    b2.o = torch.empty_like(q)[:, :, 1:3]
    sol.sol_pool(sub, *h12, b2.ws)
    sol.sol_route(sub, b2.ws, b2.row_ptr, b2.col_idx)
    sol.sol_attn_fwd(sub, *h12, b2.ws, b2.row_ptr, b2.col_idx, b2.o, lse2)
    part = [torch.full_like(t, 7.0) for t in want]
    ws2 = torch.empty(sol.sol_attn_bwd_workspace_bytes(sub), dtype=torch.uint8, device="cuda")
    sol.sol_attn_bwd(sub, *h12, b2.ws, b2.row_ptr, b2.col_idx, b2.o, lse2, do[:, :, 1:3], *(t[:, :, 1:3] for t in part), ws2)
    torch.cuda.synchronize()
    for a, b in zip(want, part):
        assert torch.equal(a[:, :, 1:3], b[:, :, 1:3]) and (b[:, :, 0] == 7).all() and (b[:, :, 3] == 7).all()


def test_rows_past_the_last_are_left_alone(sol):
    B, N, H, D = 1, 130, 2, 64
    big = [torch.randn(B, 200, H, D, device="cuda").bfloat16() for _ in range(4)]
    for t in big:
        t[:, N:] = float("nan")
    q, k, v, do = (t[:, :N] for t in big)
    p = sol.make_params(B, N, H, D, tau=0.2)
    buf = sol.alloc_buffers(p, "cuda", with_lse=True)
    sol.forward(p, q, k, v, buf)
    grads = [torch.full_like(t, 3.0) for t in big[:3]]
    g = sol.alloc_grads(p, "cuda")
    sol.sol_attn_bwd(p, q, k, v, buf.ws, buf.row_ptr, buf.col_idx, buf.o, buf.lse, do, *grads, g.ws)
    torch.cuda.synchronize()
    assert all((t[:, N:] == 3).all() for t in grads)
    check_grads(sol, p, buf, q, k, v, do, [t[:, :N] for t in grads])


def test_reblocked_backward(sol):
    w = synth.tiny()
    q, k, v = (parity.to_dev(x) for x in synth.generate(w))
    do = torch.randn_like(q)
    p = sol.make_params(w.B, w.N, w.H, w.D, tau=w.tau)
    rb = sol.alloc_reblock(p, "cuda", with_lse=True)
    sol.forward_reblocked(p, q, k, v, torch.empty_like(q), rb)
    g = sol.alloc_grads(p, "cuda")
    sol.backward_reblocked(p, rb, do, g)
    sol.sol_last_device_status()
    at = rb.perm.long().view(w.B, w.H, w.N)
    # the gradients in the partition's order against the oracle on the permuted rows
    perm = lambda t: torch.stack([t[0, at[0, h], h] for h in range(w.H)], 1)[None]
    bthd = lambda t: t.view(w.B, w.H, w.N, w.D).transpose(1, 2)
    buf = sol.Buffers(rb.buf.ws, rb.buf.row_ptr, rb.buf.col_idx, bthd(rb.buf.o), rb.buf.lse)
    check_grads(sol, p, buf, *(perm(t) for t in (q, k, v, do)), [perm(t) for t in (g.dq, g.dk, g.dv)])


# ---- norm of queries and keys with rotation -------------------------------------------------------
def rope_inputs(B, N, H, D, rot, weights, tables_b, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    q, k = ((r(B, N, H, D) * (1 + 3 * r(1, 1, H, 1).abs())).bfloat16() for _ in range(2))
    w = [None, None] if weights is None else [(1 + 0.2 * r(D)).to(weights) for _ in range(2)]
    ang = 100 * r(tables_b, N, rot // 2) if tables_b else 100 * r(N, rot // 2)
    return q, k, w, ang.cos().contiguous(), ang.sin().contiguous(), r(B, N, H, D).bfloat16(), r(B, N, H, D).bfloat16()


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (64, 0), (128, 128), (128, 48), (128, 16)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,N,H,weights,tables_b", [(1, 1, 56, torch.bfloat16, 0), (8, 1, 5, torch.float32, 8),
                                                    (2, 77, 3, torch.float32, 0), (3, 130, 9, None, 3),
                                                    (1, 1025, 17, torch.bfloat16, 1)])
def test_norm_rope_forward_and_backward(sol, B, N, H, weights, tables_b, inter, D, rot):
    q, k, w, cos, sin, dqo, dko = rope_inputs(B, N, H, D, rot, weights, tables_b, N + rot)
    eps = 1e-5
    p = sol.make_params(B, N, H, D)
    nr = sol.make_norm_rope(*w, cos, sin, eps, interleaved=inter)
    qo, ko, dq, dk = (torch.full_like(q, float("nan")) for _ in range(4))
    dw = [torch.full((D,), float("nan"), device="cuda") for _ in range(2)]
    ws = torch.full((sol.sol_qk_norm_rope_bwd_workspace_bytes(p),), 255, dtype=torch.uint8, device="cuda")
    sol.sol_qk_norm_rope(p, nr, q, k, qo, ko)
    sol.sol_qk_norm_rope_bwd(p, nr, q, k, dqo, dko, dq, dk, *dw, ws)
    torch.cuda.synchronize()
    c, s = (f64(t).reshape(tables_b or 1, N, rot // 2) for t in (cos, sin))
    for x, wt, y, dz, dx, g in ((q, w[0], qo, dqo, dq, dw[0]), (k, w[1], ko, dko, dk, dw[1])):
        wd = np.ones(D) if wt is None else f64(wt)
        want = train_ref.norm_rope(f64(x), wd, c, s, eps, inter)
        size = train_ref.rotate(np.abs(f64(x)) * wd, np.abs(c), -np.abs(s), inter)
        size = np.maximum(size, train_ref.rotate(np.abs(f64(x)) * wd, np.abs(c), np.abs(s), inter))
        size /= np.sqrt((f64(x) ** 2).mean(-1, keepdims=True))
        assert (np.abs(f64(y) - want) <= U * np.abs(want) + 2.0 ** -18 * np.abs(size) + 1e-30).all()
        ex, ew, mag = train_ref.norm_rope_backward(f64(x), wd, c, s, eps, inter, f64(dz))
        r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True))
        big = np.sqrt((f64(dz) ** 2).sum(-1, keepdims=True)) * wd.max() * r * (1 + np.abs(f64(x)) * r)
        assert (np.abs(f64(dx) - ex) <= U * np.abs(ex) + 2.0 ** -18 * big + 1e-30).all()
        # the weight's gradient: chains of at most a few hundred fp32 additions
        assert (np.abs(g.cpu().numpy() - ew) <= 2.0 ** -24 * 600 * mag + 1e-30).all()


@pytest.mark.parametrize("N,H,D", [(4100, 40, 128), (5003, 90, 64), (16500, 3, 128)])
def test_norm_rope_long(sol, N, H, D):
    """Lengths at which a warp takes several whole positions; every row checked in fp64 on the GPU."""
    B, rot = 1, D
    q, k, w, cos, sin, dqo, dko = rope_inputs(B, N, H, D, rot, torch.float32, 0, N)
    p = sol.make_params(B, N, H, D)
    nr = sol.make_norm_rope(*w, cos, sin, 1e-6)
    qo, ko, dq, dk = (torch.full_like(q, float("nan")) for _ in range(4))
    dw = [torch.full((D,), float("nan"), device="cuda") for _ in range(2)]
    ws = torch.full((sol.sol_qk_norm_rope_bwd_workspace_bytes(p),), 255, dtype=torch.uint8, device="cuda")
    sol.sol_qk_norm_rope(p, nr, q, k, qo, ko)
    sol.sol_qk_norm_rope_bwd(p, nr, q, k, dqo, dko, dq, dk, *dw, ws)
    c, s = torch.cat([cos, cos], -1).double()[None, :, None], torch.cat([-sin, sin], -1).double()[None, :, None]
    swap = lambda t: torch.cat([t[..., D // 2:], t[..., :D // 2]], -1)
    for x, wt, y, dz, dx, g in ((q, w[0], qo, dqo, dq, dw[0]), (k, w[1], ko, dko, dk, dw[1])):
        x, z, wt = x.double(), dz.double(), wt.double()
        r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        n = x * r * wt
        want = n * c + swap(n) * s
        size = (n * c).abs() + (swap(n) * s).abs()
        assert ((y.double() - want).abs() <= U * want.abs() + 2.0 ** -18 * size + 1e-30).all()
        gr = z * c - swap(z) * s
        u = gr * wt
        ex = r * (u - x * r * r * (u * x).mean(-1, keepdim=True))
        big = z.norm(dim=-1, keepdim=True) * wt.max() * r * (1 + x.abs() * r)
        assert ((dx.double() - ex).abs() <= U * ex.abs() + 2.0 ** -18 * big + 1e-30).all()
        t = gr * x * r
        # chains of at most N H / 888 + 300 additions
        assert ((g.double() - t.sum((0, 1, 2))).abs() <= 2.0 ** -24 * (N * H / 888 + 300) * t.abs().sum((0, 1, 2))).all()


def test_norm_rope_in_place_strided_and_null_weight_gradients(sol):
    B, N, H, D = 2, 300, 5, 128
    q, k, w, cos, sin, dqo, dko = rope_inputs(B, N, H, D, 128, torch.float32, 0, 1)
    p = sol.make_params(B, N, H, D)
    nr = sol.make_norm_rope(*w, cos, sin)
    qo, ko, dq, dk = (torch.empty_like(q) for _ in range(4))
    dw = [torch.empty(D, device="cuda") for _ in range(2)]
    ws = torch.empty(sol.sol_qk_norm_rope_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    sol.sol_qk_norm_rope(p, nr, q, k, qo, ko)
    sol.sol_qk_norm_rope_bwd(p, nr, q, k, dqo, dko, dq, dk, *dw, ws)
    # in place on the fused projection: v untouched, the same bits
    qkv = torch.stack((q, k, torch.full_like(q, 5.0)), 2)
    qv, kv, vv = qkv.unbind(2)
    pv = sol.make_params(B, N, H, D, in_strides=qv.stride()[:3], out_strides=qv.stride()[:3])
    sol.sol_qk_norm_rope(pv, nr, qv, kv, qv, kv)
    torch.cuda.synchronize()
    assert torch.equal(qv, qo) and torch.equal(kv, ko) and (vv == 5).all()
    # the gradient written over its input, with one weight gradient left out
    keep = torch.full((D,), 9.0, device="cuda")
    a, b = dqo.clone(), dko.clone()
    sol.sol_qk_norm_rope_bwd(p, nr, q, k, a, b, a, b, None, keep, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, dq) and torch.equal(b, dk) and torch.equal(keep, dw[1])
    sol.sol_qk_norm_rope_bwd(p, nr, q, k, dqo, dko, a, b, None, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, dq)
    # an expanded incoming gradient (batch and head strides of zero)
    one = dqo[:1, :, :1]
    pe = sol.make_params(B, N, H, D, out_strides=(0, one.stride(1), 0))
    dense = one.expand(B, N, H, D).contiguous()
    sol.sol_qk_norm_rope_bwd(p, nr, q, k, dense, dense, dq, dk, *dw, ws)
    sol.sol_qk_norm_rope_bwd(pe, nr, q, k, one, one, a, b, None, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, dq) and torch.equal(b, dk)


def test_zero_rows_are_finite(sol):
    p = sol.make_params(1, 4, 1, 64)
    z = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    o, ko, dq, dk = (torch.empty_like(z) for _ in range(4))
    nr = sol.make_norm_rope(None, None)
    ws = torch.empty(sol.sol_qk_norm_rope_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    sol.sol_qk_norm_rope(p, nr, z, z, o, ko)
    sol.sol_qk_norm_rope_bwd(p, nr, z, z, torch.ones_like(z), torch.ones_like(z), dq, dk, None, None, ws)
    torch.cuda.synchronize()
    assert (o == 0).all() and torch.isfinite(dq.float()).all()


def test_calls_from_host_threads_without_a_context(sol):
    """A thread's first CUDA call is the library's: forward and backward, each from a thread of its own."""
    import threading
    q, k, v, do = inputs(1, 300, 2, 128, 8)
    p = sol.make_params(1, 300, 2, 128)
    buf, g = sol.alloc_buffers(p, "cuda", with_lse=True), sol.alloc_grads(p, "cuda")
    sol.forward(p, q, k, v, buf)
    sol.backward(p, q, k, v, buf, do, g)
    torch.cuda.synchronize()
    want = [t.clone() for t in (buf.o, g.dq, g.dk, g.dv)]
    for t in (buf.o, g.dq, g.dk, g.dv):
        t.zero_()
    stream, errors = torch.cuda.current_stream(), []
    torch.cuda.synchronize()

    def call(fn, *a):
        try:
            fn(*a, stream=stream)
        except Exception as e:   # reported by the main thread
            errors.append(e)

    for a in ((sol.sol_attn_fwd, p, q, k, v, buf.ws, buf.row_ptr, buf.col_idx, buf.o, buf.lse),
              (sol.backward, p, q, k, v, buf, do, g)):
        t = threading.Thread(target=call, args=a)
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert all(torch.equal(a, b) for a, b in zip(want, (buf.o, g.dq, g.dk, g.dv)))


def test_expanded_output_gradient(sol):
    """d_o with zero strides (one row for every position and head)."""
    p, buf, (q, k, v, _), g = run(sol, 2, 150, 2, 128, tau=0.5)
    row = torch.randn(128, device="cuda").bfloat16()
    dense = row.expand(2, 150, 2, 128).contiguous()
    want = [t.clone() for t in (sol.backward(p, q, k, v, buf, dense, g).dq, g.dk, g.dv)]
    pe = sol.make_params(2, 150, 2, 128, tau=0.5, out_strides=(0, 0, 0))
    # o has its own strides in this call, so it is given as an expanded row too: delta changes with it
    zero = torch.zeros(128, device="cuda").bfloat16()
    sol.sol_attn_bwd(pe, q, k, v, buf.ws, buf.row_ptr, buf.col_idx, zero, buf.lse, row, g.dq, g.dk, g.dv, g.ws)
    a = [t.clone() for t in (g.dq, g.dk, g.dv)]
    sol.sol_attn_bwd(p, q, k, v, buf.ws, buf.row_ptr, buf.col_idx, torch.zeros_like(q), buf.lse, dense, g.dq, g.dk, g.dv, g.ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, (g.dq, g.dk, g.dv)))
    assert torch.equal(want[2], g.dv)


# ---- together ---------------------------------------------------------------------------------------
def layer(sol, qkv, w, cos, sin, **kw):
    q, k, v = qkv.unbind(2)
    q, k = sol.qk_norm_rope(q, k, *w, cos, sin)
    q.retain_grad()
    k.retain_grad()
    return q, k, sol.differentiable_attention(q, k, v.contiguous(), **kw)


def test_one_training_step_of_a_layer(sol):
    """norm + rotation -> pool -> route -> attention and back: the autograd gradients equal the entry points'
    bit for bit, and both stages' gradients lie within their bounds."""
    B, N, H, D = 1, 600, 2, 128
    kw = dict(tau=0.5, prefix_len=20, log_mass_bias=1)
    q, k, w, cos, sin, do, _ = rope_inputs(B, N, H, D, 128, torch.bfloat16, 0, 2)
    v = torch.randn_like(q)
    qkv = torch.stack((q, k, v), 2).requires_grad_()
    w = [t.requires_grad_() for t in w]
    qn, kn, o = layer(sol, qkv, w, cos, sin, **kw)
    o.backward(do)
    sol.sol_last_device_status()
    p = sol.make_params(B, N, H, D, **kw)
    buf = sol.alloc_buffers(p, "cuda", with_lse=True)
    sol.forward(p, qn.detach(), kn.detach(), v, buf)
    assert torch.equal(buf.o, o)
    g = sol.backward(p, qn.detach(), kn.detach(), v, buf, do, sol.alloc_grads(p, "cuda"))
    assert torch.equal(g.dq, qn.grad) and torch.equal(g.dk, kn.grad) and torch.equal(g.dv, qkv.grad[:, :, 2])
    check_grads(sol, p, buf, qn.detach(), kn.detach(), v, do, (g.dq, g.dk, g.dv))
    c, s = f64(cos)[None], f64(sin)[None]
    for i, (x, wt, dz) in enumerate(((q, w[0], g.dq), (k, w[1], g.dk))):
        ex, ew, mag = train_ref.norm_rope_backward(f64(x), f64(wt), c, s, 1e-6, False, f64(dz))
        got = f64(qkv.grad[:, :, i])
        r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True))
        big = np.sqrt((f64(dz) ** 2).sum(-1, keepdims=True)) * f64(wt).max() * r * (1 + np.abs(f64(x)) * r)
        assert (np.abs(got - ex) <= U * np.abs(ex) + 2.0 ** -18 * big + 1e-30).all()
        assert (np.abs(f64(wt.grad) - ew) <= U * np.abs(ew) + 2.0 ** -24 * 600 * mag + 1e-30).all()
    # a gradient that arrives expanded (o.sum()) and in fp32 arithmetic
    qkv.grad = None
    layer(sol, qkv, w, cos, sin, **kw)[2].sum().backward()
    assert torch.isfinite(qkv.grad.float()).all()


def test_two_layers_share_their_input(sol):
    """Two layers of one fused projection, both backward passes after both forwards: gradients add."""
    B, N, H, D = 1, 200, 2, 64
    q, k, w, cos, sin, do, do2 = rope_inputs(B, N, H, D, 64, torch.float32, 0, 3)
    qkv = torch.stack((q, k, torch.randn_like(q)), 2).requires_grad_()
    outs = []
    for use in ((True, False), (False, True), (True, True)):
        qkv.grad = None
        a = layer(sol, qkv, w, cos, sin, tau=0.3)[2]
        b = layer(sol, qkv, w, cos, sin, topk_ratio=0.5)[2]
        torch.autograd.backward([t for t, u in zip((a, b), use) if u], [d for d, u in zip((do, do2), use) if u])
        outs.append(qkv.grad.float())
    want = outs[0] + outs[1]
    assert ((outs[2] - want).abs() <= U * want.abs() + 1e-30).all()


def test_captured_step_replays_on_new_inputs_and_streams(sol):
    """The whole step captured once on a side stream and replayed; eager calls in between on another stream
    and with buffers of their own give the same bits."""
    B, N, H, D = 1, 900, 2, 128
    kw = dict(tau=0.5, prefix_len=10, log_mass_bias=2)

    def make(seed):
        q, k, w, cos, sin, do, _ = rope_inputs(B, N, H, D, 128, torch.float32, 0, seed)
        return [q, k, torch.randn_like(q), do], w, cos, sin

    def bufs():
        p = sol.make_params(B, N, H, D, **kw)
        return dict(p=p, buf=sol.alloc_buffers(p, "cuda", with_lse=True), g=sol.alloc_grads(p, "cuda"),
                    n=[torch.empty(B, N, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(4)],
                    dw=[torch.empty(D, device="cuda") for _ in range(2)],
                    ws=torch.empty(sol.sol_qk_norm_rope_bwd_workspace_bytes(p), dtype=torch.uint8, device="cuda"))

    def step(x, nr, s):
        q, k, v, do = x
        p, buf, g, n = s["p"], s["buf"], s["g"], s["n"]
        sol.sol_qk_norm_rope(p, nr, q, k, n[0], n[1])
        sol.forward(p, n[0], n[1], v, buf)
        sol.backward(p, n[0], n[1], v, buf, do, g)
        sol.sol_qk_norm_rope_bwd(p, nr, q, k, g.dq, g.dk, n[2], n[3], *s["dw"], s["ws"])

    result = lambda s: [t.clone() for t in (*s["n"], s["g"].dv, *s["dw"])]
    x, w, cos, sin = make(1)
    nr = sol.make_norm_rope(*w, cos, sin)
    s, other = bufs(), bufs()
    step(x, nr, s)
    torch.cuda.synchronize()
    first = result(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(x, nr, s)
    x2 = make(2)[0]
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
        step(x2, nr, other)
        want2 = result(other)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, result(s)))
    for a, b in zip(x, x2):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want2, result(s)))
    sol.sol_last_device_status()


# ---- calls that the documentation allows and that are easy to get wrong ------------------------------
def listed(sol, lists, N, H=1, D=128, seed=4):
    """A forward pass under routing 1 with lists of the caller's own (the same for every head)."""
    q, k, v, do = inputs(1, N, H, D, seed)
    p = sol.make_params(1, N, H, D, topk_ratio=max(0.3, 1.05 * max(map(len, lists)) / len(lists)))
    buf = sol.alloc_buffers(p, q.device, with_lse=True)
    sol.sol_pool(p, q, k, v, buf.ws)
    buf.row_ptr.copy_(torch.tensor(np.cumsum([0] + [len(x) for x in lists] * H), dtype=torch.int32))
    flat = torch.tensor(sum(lists, []) * H, dtype=torch.int32, device="cuda")
    buf.col_idx[:len(flat)] = flat
    sol.sol_attn_fwd(p, q, k, v, buf.ws, buf.row_ptr, buf.col_idx, buf.o, buf.lse)
    return p, buf, [q, k, v, do]


@pytest.mark.parametrize("where", ["q", "k", "v", "do", "lse"])
def test_non_finite_values_go_where_the_formula_takes_them(sol, where):
    """One row of NaN: the rows that the lists tie to it get NaN, every other row keeps its bits, the other
    half of its 128-row tile among them."""
    lists = [[0, 2], [1, 2, 4], [3], [0, 1, 4], [2], [0, 3], [5, 6], [5], [7]]
    N, at = 64 * 8 + 30, 64 * 2 + 17
    p, buf, x = listed(sol, lists, N)
    g = sol.alloc_grads(p, "cuda")
    sol.backward(p, *x[:3], buf, x[3], g)
    clean = [t.clone() for t in (g.dq, g.dk, g.dv)]
    if where == "lse":
        buf.lse[..., at] = float("nan")
    else:
        x["q k v do".split().index(where)][:, at] = float("nan")
    sol.backward(p, *x[:3], buf, x[3], g)
    sol.sol_last_device_status()
    sel = np.zeros((9, 9), bool)
    for i, js in enumerate(lists):
        sel[i, js] = True
    row, block = np.zeros(N, bool), np.arange(N) // 64
    row[at] = True
    asks, asked = sel[:, 2][block], sel[2][block]   # rows whose block lists this one; rows of the blocks that it lists
    none = np.zeros(N, bool)
    want = dict(q=(row, asked, asked), k=(asks, row, row), v=(asks, row, none), do=(row, asked, asked),
                lse=(row, asked, asked))[where]
    for name, t, c, bad in zip(("dq", "dk", "dv"), (g.dq, g.dk, g.dv), clean, want):
        bad = torch.from_numpy(bad).cuda()
        assert torch.isnan(t[0, bad]).all(), name
        assert torch.equal(t[0, ~bad], c[0, ~bad]), name


def test_the_longest_call(sol):
    """N = 65,536 (1,024 blocks, every word of the bitmaps): blocks at both ends and between, each against
    the formulas on the rows that its lists tie it to."""
    N, D = 65536, 64
    rng = np.random.default_rng(5)
    lists = [sorted(set(rng.integers(0, 1024, 5).tolist()) | {1023 - i, (7 * i) % 1024}) for i in range(1024)]
    p, buf, x = listed(sol, lists, N, D=D)
    g = sol.alloc_grads(p, "cuda")
    for t in (g.dq, g.dk, g.dv, g.ws):
        t.fill_(255 if t.dtype == torch.uint8 else float("nan"))
    sol.backward(p, *x[:3], buf, x[3], g)
    sol.sol_last_device_status()
    assert all(torch.isfinite(t).all() for t in (g.dq, g.dk, g.dv))
    host = [f64(t[0, :, 0]) for t in (*x, buf.o)]
    lse = f64(buf.lse[0, 0])

    def part(blocks, sel):
        rows = np.concatenate([np.arange(64 * i, 64 * i + 64) for i in blocks])
        nb = len(blocks)
        return rows, train_ref.attention_backward(*(t[rows] for t in host), lse[rows], sel, np.zeros((nb, D)),
                                                  np.zeros((nb, D)), np.zeros(nb), centroids=False)

    for b in (0, 1, 31, 32, 511, 512, 1022, 1023):
        for grads, blocks in (((g.dq,), sorted({b, *lists[b]})),
                              ((g.dk, g.dv), sorted({b, *(i for i in range(1024) if b in lists[i])}))):
            sel = np.zeros((len(blocks), len(blocks)), bool)
            me = blocks.index(b)
            for i, blk in enumerate(blocks):
                if len(grads) == 1:
                    sel[me, i] = blk in lists[b]
                else:
                    sel[i, me] = b in lists[blk]
            rows, want = part(blocks, sel)
            mine = rows // 64 == b
            for t, (e, bound) in zip(grads, want[:1] if len(grads) == 1 else want[1:]):
                assert (np.abs(f64(t[0, rows[mine], 0]) - e[mine]) <= bound[mine]).all(), (b, len(grads))


def test_the_longest_call_with_centroids(sol):
    """N = 65,536 without any listed block: 1,024 centroid terms a row, the pooled gradients of all rows."""
    N, D = 65536, 64
    p, buf, (q, k, v, do), g = run(sol, 1, N, 1, D, seed=6, tau=50.0)
    assert int(buf.row_ptr[-1]) == 0
    w = sol.workspace_views(p, buf.ws)
    Q, dO, O = (t[0, :, 0].double() for t in (q, do, buf.o))
    kc, vc, off = (w[n][0, 0].double() for n in ("kbar16", "vbar16", "cbias"))
    s, U2 = D ** -0.5, 2.0 ** -24
    prob = torch.exp(s * Q @ kc.T + off - buf.lse[0, 0].double()[:, None])
    delta, mag = (dO * O).sum(1, True), (dO.abs() * O.abs()).sum(1, True)
    ds, dsm = prob * (dO @ vc.T - delta), prob * (dO.abs() @ vc.abs().T + mag)
    e1 = D * float((s * Q.abs() @ kc.abs().T).max()) * U2 + 2.0 ** -20
    e2 = 2 * D * U2

    def near(got, A, Am, Y, n=1):   # as train_ref.attention_backward bounds a sum of rounded terms
        want, bound = A @ Y / n, ((U + 2 * e1) * (A.abs() @ Y.abs()) + e2 * (Am @ Y.abs())) / n
        return ((got - want).abs() <= bound + U * want.abs() + 1e-30).all()

    assert near(g.dq[0, :, 0].double(), s * ds, s * dsm, kc)
    for t, A, Am, Y in ((g.dk, s * ds.T, s * dsm.T, Q), (g.dv, prob.T, 0 * prob.T, dO)):
        rows = t[0, :, 0].view(1024, 64, D)
        assert (rows == rows[:, :1]).all()   # a block's mean: one gradient for its rows
        assert near(rows[:, 0].double(), A, Am, Y, 64)


def test_many_short_sequences(sol):
    """40,000 sequences of 3 rows, 2 heads: each as in a call of its own."""
    B, N, H, D = 40000, 3, 2, 64
    kw = dict(tau=0.5, log_mass_bias=2)
    q, k, v, do = inputs(B, N, H, D, 12)

    def grads(at):
        x = [t[at].contiguous() for t in (q, k, v, do)]
        p = sol.make_params(len(x[0]), N, H, D, **kw)
        buf = sol.alloc_buffers(p, "cuda", with_lse=True)
        sol.sol_pool(p, *x[:3], buf.ws)
        # sol_route takes up to 65,535 heads in all: lists of the caller's, the first head's block exact,
        # the second's by its centroid
        buf.row_ptr.copy_((torch.arange(len(buf.row_ptr)) + 1) // 2)
        buf.col_idx.zero_()
        sol.sol_attn_fwd(p, *x[:3], buf.ws, buf.row_ptr, buf.col_idx, buf.o, buf.lse)
        g = sol.backward(p, *x[:3], buf, x[3], sol.alloc_grads(p, "cuda"))
        sol.sol_last_device_status()
        return torch.stack((g.dq, g.dk, g.dv))

    every = grads(slice(None))
    assert torch.isfinite(every).all() and (every[2] != 0).any(-1).all()
    for at in (slice(0, 3), slice(21844, 21850), slice(39999, 40000)):
        assert torch.equal(every[:, at], grads(at))


def test_calls_at_once_on_two_streams(sol):
    """Calls that overlap, each with buffers of its own, give the bits of calls made alone."""
    N, H, D = 2500, 4, 128
    p = sol.make_params(1, N, H, D, tau=0.7, log_mass_bias=2, prefix_len=70)
    sets = []
    for seed in range(2):
        q, k, v, do = inputs(1, N, H, D, seed)
        buf = sol.alloc_buffers(p, "cuda", with_lse=True)
        sol.forward(p, q, k, v, buf)
        g = sol.backward(p, q, k, v, buf, do, sol.alloc_grads(p, "cuda"))
        sets.append((q, k, v, buf, do, g, [t.clone() for t in (g.dq, g.dk, g.dv)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for q, k, v, buf, do, g, _, s in sets:
            g.dq.zero_(), g.dk.zero_(), g.dv.zero_()
        torch.cuda.synchronize()
        for q, k, v, buf, do, g, _, s in sets:
            for _ in range(3):
                sol.backward(p, q, k, v, buf, do, g, stream=s)
        torch.cuda.synchronize()
        for *_, g, want, s in sets:
            assert all(torch.equal(a, b) for a, b in zip((g.dq, g.dk, g.dv), want))
    sol.sol_last_device_status()


def test_captured_autograd_step_beside_an_eager_graph(sol):
    """Forward and backward captured with leaves of the capture's own, while an eager graph of the same
    tensors is alive and is run afterwards."""
    B, N, H, D = 1, 300, 2, 64
    q, k, w, cos, sin, do, _ = rope_inputs(B, N, H, D, 64, torch.float32, 0, 7)
    qkv = torch.stack((q, k, torch.randn_like(q)), 2).requires_grad_()
    w = [t.requires_grad_() for t in w]

    def step(x, wq, wk):
        a, b, c = x.unbind(2)
        a, b = sol.qk_norm_rope(a, b, wq, wk, cos, sin)
        return sol.differentiable_attention(a, b, c.contiguous(), tau=0.4, log_mass_bias=1)

    o = step(qkv, *w)
    want = torch.autograd.grad(o, (qkv, *w), do, retain_graph=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        leaves = [t.detach().requires_grad_() for t in (qkv, *w)]
        got = torch.autograd.grad(step(*leaves), leaves, do)
    graph.replay()
    o.backward(do)
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, (qkv, *w)):
        assert torch.equal(a, b) and torch.equal(a, c.grad)


def test_reblocked_temporaries_belong_to_the_call_s_stream(sol, monkeypatch):
    """The rows gathered for a call on another stream are not handed out again on the current one while
    that call may still run."""
    w = synth.tiny()
    q, k, v = (parity.to_dev(x) for x in synth.generate(w))
    p = sol.make_params(w.B, w.N, w.H, w.D, tau=w.tau)
    rb = sol.alloc_reblock(p, "cuda", with_lse=True)
    sol.forward_reblocked(p, q, k, v, torch.empty_like(q), rb)
    g = sol.alloc_grads(p, "cuda")
    want = [t.clone() for t in (sol.backward_reblocked(p, rb, q, g).dq, g.dk, g.dv)]
    torch.cuda.synchronize()
    used = []
    gather, scatter = sol.sol_gather_rows, sol.sol_scatter_rows
    monkeypatch.setattr(sol, "sol_gather_rows", lambda p, i, x, y, s=None: (used.append(y.data_ptr()), gather(p, i, x, y, s)))
    monkeypatch.setattr(sol, "sol_scatter_rows", lambda p, i, x, y, s=None: (used.append(x.data_ptr()), scatter(p, i, x, y, s)))
    sol.backward_reblocked(p, rb, q, g, stream=torch.cuda.Stream())
    mine = [torch.empty_like(rb.qp) for _ in range(8)]
    assert len(used) == 4 and not set(used) & {t.data_ptr() for t in mine}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (g.dq, g.dk, g.dv)))


def test_empty_norm_has_zero_weight_gradients(sol):
    p = sol.make_params(2, 0, 4, 128)
    dw = [torch.full((128,), float("nan"), device="cuda") for _ in range(2)]
    x = torch.empty(2, 0, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1, dtype=torch.uint8, device="cuda")
    sol.sol_qk_norm_rope_bwd(p, sol.make_norm_rope(None, None), x, x, x, x, x, x, *dw, ws)
    assert all((t == 0).all() for t in dw)
    x = x.requires_grad_()
    w = torch.ones(128, device="cuda", requires_grad=True)
    sum(t.sum() for t in sol.qk_norm_rope(x, x, w, w)).backward()
    assert (w.grad == 0).all() and x.grad.shape == x.shape


def norm_rope_bwd(sol, q, k, dqo, dko, w, cos=None, sin=None, eps=1e-6, interleaved=False):
    """dq, dk and the two weight gradients of one call, every output NaN before it."""
    B, N, H, D = q.shape
    p = sol.make_params(B, N, H, D)
    nr = sol.make_norm_rope(*w, cos, sin, eps, interleaved=interleaved)
    dq, dk = (torch.full_like(q, float("nan")) for _ in range(2))
    dw = [torch.full((D,), float("nan"), device="cuda") for _ in range(2)]
    ws = torch.full((sol.sol_qk_norm_rope_bwd_workspace_bytes(p),), 255, dtype=torch.uint8, device="cuda")
    sol.sol_qk_norm_rope_bwd(p, nr, q, k, dqo, dko, dq, dk, *dw, ws)
    torch.cuda.synchronize()
    return dq, dk, *dw


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", [1, 3, 9, 17])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_backward_without_eps(sol, D, H, inter):
    """eps = 0 where the heads do not fill a warp's last unit: the lanes past the last head add nothing to the
    weights' gradients."""
    q, k, w, cos, sin, dqo, dko = rope_inputs(2, 37, H, D, 32, torch.float32, 0, 40 + H)
    dq, dk, *dw = norm_rope_bwd(sol, q, k, dqo, dko, w, cos, sin, 0.0, inter)
    c, s = f64(cos)[None], f64(sin)[None]
    for x, wt, dz, dx, g in ((q, w[0], dqo, dq, dw[0]), (k, w[1], dko, dk, dw[1])):
        ex, ew, mag = train_ref.norm_rope_backward(f64(x), f64(wt), c, s, 0.0, inter, f64(dz))
        r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True))
        big = np.sqrt((f64(dz) ** 2).sum(-1, keepdims=True)) * f64(wt).max() * r * (1 + np.abs(f64(x)) * r)
        assert (np.abs(f64(dx) - ex) <= U * np.abs(ex) + 2.0 ** -18 * big + 1e-30).all()
        assert (np.abs(g.cpu().numpy() - ew) <= 2.0 ** -24 * 600 * mag + 1e-30).all()


def grads_of(sol, qkv, w, cos, sin, do, **kw):
    """Gradients of one layer's step with leaves of its own."""
    leaves = [t.detach().clone().requires_grad_() for t in (qkv, *w)]
    _, _, o = layer(sol, leaves[0], leaves[1:], cos, sin, **kw)
    o.backward(do)
    return [t.grad for t in leaves]


@pytest.mark.parametrize("mode", [0, 2])
def test_saved_tensor_hooks_change_nothing(sol, mode):
    """A step whose saved tensors are kept elsewhere, dense, and come back at other addresses: the fused
    projection's views among them.  Bit for bit the plain step's gradients."""
    B, N, H, D = 2, 300, 2, 64
    q, k, w, cos, sin, do, _ = rope_inputs(B, N, H, D, 64, torch.float32, 0, 11)
    qkv = torch.stack((q, k, torch.randn_like(q)), 2)
    kw = dict(tau=0.4, log_mass_bias=mode)
    want = grads_of(sol, qkv, w, cos, sin, do, **kw)
    for hooks in (torch.autograd.graph.save_on_cpu(),
                  torch.autograd.graph.saved_tensors_hooks(lambda t: t, lambda t: t.clone()),
                  torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(memory_format=torch.contiguous_format), lambda t: t)):
        with hooks:
            got = grads_of(sol, qkv, w, cos, sin, do, **kw)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    # recomputed in the backward pass
    from torch.utils.checkpoint import checkpoint
    leaves = [t.detach().clone().requires_grad_() for t in (qkv, *w)]
    step = lambda x, wq, wk: sol.differentiable_attention(*sol.qk_norm_rope(*x.unbind(2)[:2], wq, wk, cos, sin),
                                                          x.unbind(2)[2].contiguous(), **kw)
    checkpoint(step, *leaves, use_reentrant=False).backward(do)
    sol.sol_last_device_status()
    assert all(torch.equal(a, t.grad) for a, t in zip(want, leaves))


@pytest.mark.parametrize("weights", [torch.float32, torch.bfloat16])
def test_weights_renewed_between_the_passes(sol, weights):
    """The weights' storage is released after the forward, its memory overwritten by others, and a new one
    filled before the backward pass, as a trainer with sharded weights does."""
    B, N, H, D = 1, 90, 3, 128
    q, k, w, cos, sin, dqo, dko = rope_inputs(B, N, H, D, 64, weights, 0, 21)
    x = torch.stack((q, k), 2).requires_grad_()
    w = [t.requires_grad_() for t in w]

    def step(between):
        x.grad = w[0].grad = w[1].grad = None
        out = sol.qk_norm_rope(*x.unbind(2), *w, cos, sin)
        between()
        torch.autograd.backward(out, (dqo, dko))
        return [t.grad.clone() for t in (x, *w)]

    def renew():
        torch.cuda.synchronize()
        kept = [t.detach().clone() for t in w]
        for t in w:
            t.untyped_storage().resize_(0)
        other.extend(torch.full((D,), 7.0, dtype=weights, device="cuda") for _ in range(16))
        for t, c in zip(w, kept):
            t.untyped_storage().resize_(D * t.element_size())
            t.data.copy_(c)

    other = []
    want, got = step(lambda: None), step(renew)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_empty_sequence_through_autograd_with_tables(sol):
    x = torch.empty(2, 0, 4, 128, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    w = torch.ones(128, device="cuda", requires_grad=True)
    t = torch.empty(0, 64, device="cuda")
    q, k = sol.qk_norm_rope(x, x, w, w, t, t)
    o = sol.differentiable_attention(q, k, x)
    assert o.shape == x.shape
    o.sum().backward()
    assert (w.grad == 0).all() and x.grad.shape == x.shape


@pytest.mark.parametrize("size", [4e-20, 1e-12, 1e12, 1e17])
def test_norm_rope_of_tiny_and_huge_rows(sol, size):
    """Rows of one size far from 1 without an eps: r^2 alone would overflow (4e-20: r = 2.5e19).  The squares of the
    smallest are subnormal, off by half of 2^-149 each: 2e-7 of r, inside the bound's 2^-18."""
    B, N, H, D = 1, 33, 3, 128
    q, k, w, cos, sin, dqo, dko = rope_inputs(B, N, H, D, 64, torch.float32, 0, 31)
    q, k = ((t.float() / t.float().square().mean(-1, keepdim=True).sqrt() * size).bfloat16() for t in (q, k))
    p = sol.make_params(B, N, H, D)
    nr = sol.make_norm_rope(*w, cos, sin, 0.0)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    sol.sol_qk_norm_rope(p, nr, q, k, qo, ko)
    dq, dk, *dw = norm_rope_bwd(sol, q, k, dqo, dko, w, cos, sin, 0.0)
    c, s = f64(cos)[None], f64(sin)[None]
    for x, wt, y, dz, dx, g in ((q, w[0], qo, dqo, dq, dw[0]), (k, w[1], ko, dko, dk, dw[1])):
        r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True))
        want = train_ref.norm_rope(f64(x), f64(wt), c, s, 0.0, False)
        assert (np.abs(f64(y) - want) <= U * np.abs(want) + 2.0 ** -17 * f64(wt).max() * np.abs(f64(x) * r).max(-1, keepdims=True)).all()
        ex, ew, mag = train_ref.norm_rope_backward(f64(x), f64(wt), c, s, 0.0, False, f64(dz))
        big = np.sqrt((f64(dz) ** 2).sum(-1, keepdims=True)) * f64(wt).max() * r * (1 + np.abs(f64(x)) * r)
        assert (np.abs(f64(dx) - ex) <= U * np.abs(ex) + 2.0 ** -18 * big).all()
        assert (np.abs(g.cpu().numpy() - ew) <= 2.0 ** -24 * 600 * mag).all()


def test_reblocked_backward_of_fused_views(sol):
    """q, k, v as views of the fused projection and a dense d_o: the bits of the dense call."""
    w = synth.tiny()
    q, k, v = (parity.to_dev(x) for x in synth.generate(w))
    do = torch.randn_like(q)
    kw = dict(tau=w.tau, log_mass_bias=2)
    fused = torch.stack((q, k, v), 2).unbind(2)
    out = []
    for x, d in (((q, k, v), do), (fused, do), (fused, torch.stack((do, q), 2)[:, :, 0])):
        p = sol.make_params(w.B, w.N, w.H, w.D, in_strides=x[0].stride()[:3], **kw)
        rb = sol.alloc_reblock(p, "cuda", with_lse=True)
        sol.forward_reblocked(p, *x, torch.empty_like(q), rb)
        g = sol.backward_reblocked(p, rb, d, sol.alloc_grads(p, "cuda"))
        sol.sol_last_device_status()
        out.append((g.dq, g.dk, g.dv))
    for other in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], other))


@pytest.mark.parametrize("mode", [1, 2])
@pytest.mark.parametrize("N,D,prefix", anchor_cases.CASES)
def test_anchor_s_terms(sol, N, D, prefix, mode):
    """Inputs on which the anchor's terms are far above the roundings (a CPU test plants mistakes in them)."""
    heads = [anchor_cases.inputs(N, D, prefix, seed) for seed in range(3)]
    q, k, v, do = (torch.from_numpy(np.stack([h[i] for h in heads], 1)[None]).cuda().bfloat16() for i in range(4))
    p = sol.make_params(1, N, 3, D, prefix_len=prefix, log_mass_bias=mode)
    buf, g = sol.alloc_buffers(p, "cuda", with_lse=True), sol.alloc_grads(p, "cuda")
    sol.sol_pool(p, q, k, v, buf.ws)
    sel = torch.from_numpy(np.concatenate([h[4] for h in heads]))
    buf.row_ptr.copy_(torch.nn.functional.pad(sel.sum(1).cumsum(0), (1, 0)))
    entries = sel.nonzero()[:, 1].int().cuda()
    buf.col_idx[:len(entries)] = entries
    sol.sol_attn_fwd(p, q, k, v, buf.ws, buf.row_ptr, buf.col_idx, buf.o, buf.lse)
    for t in (g.dq, g.dk, g.dv):
        t.fill_(float("nan"))
    g.ws.fill_(255)
    sol.backward(p, q, k, v, buf, do, g)
    sol.sol_last_device_status()
    check_grads(sol, p, buf, q, k, v, do, (g.dq, g.dk, g.dv))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("inter", [False, True])
def test_infinite_values_outside_the_turned_dims(sol, D, inter):
    """An infinity past the turned dims reaches the other dims through the norm alone (with interleaved pairs
    its neighbour becomes NaN too); other rows and the other tensor keep their bits."""
    at = 41
    q, k, w, cos, sin, dqo, dko = rope_inputs(1, 20, 3, D, 32, torch.float32, 0, 51)
    p = sol.make_params(1, 20, 3, D)
    qi, zi = q.clone(), dqo.clone()
    qi[0, 7, 1, at] = float("inf")
    zi[0, 7, 1, at] = float("inf")
    nr = sol.make_norm_rope(*w, cos, sin, interleaved=inter)
    qo, ko = (torch.full_like(q, 3.0) for _ in range(2))
    sol.sol_qk_norm_rope(p, nr, qi, k, qo, ko)
    torch.cuda.synchronize()
    other = torch.arange(D, device="cuda") != at
    if inter:
        other[at - 1] = False
    assert torch.isnan(qo[0, 7, 1, ~other]).all() and (qo[0, 7, 1, other] == 0).all()   # x / infinity
    dq, dk, dwq, dwk = norm_rope_bwd(sol, q, k, zi, dko, w, cos, sin, interleaved=inter)
    clean = norm_rope_bwd(sol, q, k, dqo, dko, w, cos, sin, interleaved=inter)
    assert not torch.isfinite(dwq[~other]).any() and torch.equal(dwq[other], clean[2][other])
    assert torch.equal(dk, clean[1]) and torch.equal(dwk, clean[3])
    if not inter:
        assert torch.isinf(dwq[at]) and torch.isinf(dq[0, 7, 1, other]).all()   # each less x times the mean of u x
    assert not torch.isfinite(dq[0, 7, 1]).any()
    dq[0, 7, 1] = clean[0][0, 7, 1]
    assert torch.equal(dq, clean[0])
