"""Refusals of the training entry points: all synchronous, nothing is launched."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def sol():
    from block_sparse_video_sol_b200 import build
    build.build()
    from block_sparse_video_sol_b200 import sol as mod
    return mod


BIG = 1 << 40


def _bwd(sol, p, ptr=4096, ws_bytes=BIG, bws_bytes=BIG, gs=None, **over):
    names = ["q", "k", "v", "ws", "row_ptr", "col_idx", "o", "lse", "d_o", "dq", "dk", "dv", "bws"]
    a = {n: over.get(n, ptr) for n in names}
    g = None if gs is None else (ctypes.c_int64 * 3)(*gs)
    return sol.lib.sol_attn_bwd(None if p is None else ctypes.byref(p), a["q"], a["k"], a["v"], a["ws"], ws_bytes, a["row_ptr"],
                                a["col_idx"], a["o"], a["lse"], a["d_o"], a["dq"], a["dk"], a["dv"], g, a["bws"], bws_bytes, None)


def _text(sol):
    return sol.lib.sol_last_error_text().decode()


def test_attn_bwd_refusals(sol):
    p = sol.make_params(2, 1000, 4, 128)
    assert _bwd(sol, None) == sol.SOL_ERR_INVALID_ARG
    for name in ("q", "k", "v", "ws", "row_ptr", "col_idx", "o", "lse", "d_o", "dq", "dk", "dv", "bws"):
        assert _bwd(sol, p, **{name: None}) == sol.SOL_ERR_INVALID_ARG and "NULL" in _text(sol), name
    for name in ("q", "k", "v", "o", "d_o", "dq", "dk", "dv"):
        assert _bwd(sol, p, **{name: 4096 + 8}) == sol.SOL_ERR_INVALID_ARG and "aligned" in _text(sol), name
    for name in ("ws", "bws"):
        assert _bwd(sol, p, **{name: 4096 + 128}) == sol.SOL_ERR_INVALID_ARG and "256" in _text(sol), name
    assert _bwd(sol, p, ws_bytes=sol.sol_workspace_bytes(p) - 1) == sol.SOL_ERR_WORKSPACE
    assert _bwd(sol, p, bws_bytes=sol.sol_attn_bwd_workspace_bytes(p) - 1) == sol.SOL_ERR_WORKSPACE
    assert _bwd(sol, sol.make_params(2, 1000, 4, 128, qk_int8=True)) == sol.SOL_ERR_UNSUPPORTED
    assert "INT8" in _text(sol)
    assert sol.sol_attn_bwd_workspace_bytes(sol.make_params(2, 1000, 4, 128, qk_int8=True)) == 0
    assert _bwd(sol, sol.make_params(2, 1000, 4, 96)) == sol.SOL_ERR_UNSUPPORTED
    assert _bwd(sol, sol.make_params(2, 1000, 4, 128, tau=math.nan)) == sol.SOL_ERR_INVALID_ARG
    # an empty problem enqueues nothing, whatever the pointers
    assert _bwd(sol, sol.make_params(0, 1000, 4, 128), ptr=None) == sol.SOL_OK
    assert _bwd(sol, sol.make_params(2, 0, 4, 128), ptr=None) == sol.SOL_OK


@pytest.mark.parametrize("gs,ok", [
    ((512000, 512, 128), True), ((1536000, 1536, 128), True), ((512000, 128, 128000), True), ((1000 * 512 * 3, 1536, 384), True),
    ((0, 512, 128), False), ((512000, 0, 128), False), ((512000, 512, 0), False), ((512000, 512, 120), False),
    ((512000, 504, 128), False), ((511992, 512, 128), False), ((512000, 512, 132), False), ((-512000, 512, 128), False)])
def test_gradient_rows_must_be_distinct(sol, gs, ok):
    p = sol.make_params(2, 1000, 4, 128)
    st = _bwd(sol, p, gs=gs, bws_bytes=1)
    assert st == (sol.SOL_ERR_WORKSPACE if ok else sol.SOL_ERR_INVALID_ARG), _text(sol)


def test_broadcast_inputs_need_gradient_strides_of_their_own(sol):
    p = sol.make_params(2, 1000, 4, 128, in_strides=(0, 512, 128))
    assert _bwd(sol, p, bws_bytes=1) == sol.SOL_ERR_INVALID_ARG and "overlap" in _text(sol)
    assert _bwd(sol, p, gs=(512000, 512, 128), bws_bytes=1) == sol.SOL_ERR_WORKSPACE
    # dims of size one may have any stride
    assert _bwd(sol, sol.make_params(1, 1000, 1, 128, in_strides=(0, 128, 0)), bws_bytes=1) == sol.SOL_ERR_WORKSPACE


def test_attn_bwd_workspace_size(sol):
    for kw, pooled in ((dict(), 0), (dict(log_mass_bias=2), 1), (dict(topk_ratio=0.2), -1)):
        p = sol.make_params(1, 32768, 56, 128, **kw)
        stat = 2 * 56 * 32768 * 4
        plans = 56 * 256 * ((16 + 2 * 16 + 512) + (16 + 512)) * 4
        cent = 0 if pooled < 0 else 8 * 56 * 512 * (2 * 128 + 1) * 4
        rows = 56 * (3 * 32768 + 512 * 128 + 128) * 4 if pooled > 0 else 0
        got = sol.sol_attn_bwd_workspace_bytes(p)
        assert stat + plans + cent + rows <= got <= stat + plans + cent + rows + 16 * 256
    assert sol.sol_attn_bwd_workspace_bytes(sol.make_params(1, 0, 56, 128)) == 0


def _nr(sol, **over):
    f = dict(q_weight=4096, k_weight=4096, weight_type=0, eps=1e-6, rot_dim=64, interleaved=0, cos=4096, sin=4096,
             table_stride_b=0, table_stride_n=32)
    f.update(over)
    return sol.sol_norm_rope(*[f[n] for n, _ in sol.sol_norm_rope._fields_])


def _fwd_nr(sol, p, nr, q=4096, k=4096, qo=8192, ko=8192):
    return sol.lib.sol_qk_norm_rope(ctypes.byref(p), None if nr is None else ctypes.byref(nr), q, k, qo, ko, None)


def _bwd_nr(sol, p, nr, gs=None, ws_bytes=BIG, **over):
    a = {n: over.get(n, 4096) for n in ("q", "k", "dqo", "dko", "dq", "dk", "dqw", "dkw", "ws")}
    g = None if gs is None else (ctypes.c_int64 * 3)(*gs)
    return sol.lib.sol_qk_norm_rope_bwd(ctypes.byref(p), None if nr is None else ctypes.byref(nr), a["q"], a["k"],
                                        a["dqo"], a["dko"], a["dq"], a["dk"], a["dqw"], a["dkw"], g, a["ws"], ws_bytes, None)


@pytest.mark.parametrize("over", [
    dict(weight_type=2), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(rot_dim=8), dict(rot_dim=144),
    dict(rot_dim=-16), dict(interleaved=2), dict(q_weight=4100), dict(k_weight=4104), dict(cos=None), dict(sin=None),
    dict(cos=4100), dict(table_stride_n=30), dict(table_stride_b=-32)])
def test_norm_rope_parameter_refusals(sol, over):
    p = sol.make_params(1, 100, 4, 128)
    assert _fwd_nr(sol, p, _nr(sol, **over)) == sol.SOL_ERR_INVALID_ARG
    assert _text(sol).startswith("sol_qk_norm_rope:")
    assert _bwd_nr(sol, p, _nr(sol, **over)) == sol.SOL_ERR_INVALID_ARG
    assert _text(sol).startswith("sol_qk_norm_rope_bwd:")


def test_norm_rope_refusals(sol):
    p = sol.make_params(1, 100, 4, 128)
    assert _fwd_nr(sol, p, None) == sol.SOL_ERR_INVALID_ARG
    for name in ("q", "k", "qo", "ko"):
        assert _fwd_nr(sol, p, _nr(sol), **{name: None}) == sol.SOL_ERR_INVALID_ARG and "NULL" in _text(sol)
        assert _fwd_nr(sol, p, _nr(sol), **{name: 4104}) == sol.SOL_ERR_INVALID_ARG and "aligned" in _text(sol)
    assert _fwd_nr(sol, sol.make_params(1, 100, 4, 128, out_strides=(51200, 0, 128)), _nr(sol)) == sol.SOL_ERR_INVALID_ARG
    assert _fwd_nr(sol, sol.make_params(1, 100, 4, 96), _nr(sol)) == sol.SOL_ERR_UNSUPPORTED
    assert _fwd_nr(sol, sol.make_params(1, 0, 4, 128), _nr(sol), None, None, None, None) == sol.SOL_OK
    for name in ("q", "k", "dqo", "dko", "dq", "dk", "ws"):
        assert _bwd_nr(sol, p, _nr(sol), **{name: None}) == sol.SOL_ERR_INVALID_ARG and "NULL" in _text(sol)
    for name in ("q", "dqo", "dk", "dqw", "dkw"):
        assert _bwd_nr(sol, p, _nr(sol), **{name: 4104}) == sol.SOL_ERR_INVALID_ARG and "aligned" in _text(sol)
    assert _bwd_nr(sol, p, _nr(sol), gs=(0, 0, 128)) == sol.SOL_ERR_INVALID_ARG
    assert _bwd_nr(sol, p, _nr(sol), ws=4096 + 64) == sol.SOL_ERR_INVALID_ARG
    assert _bwd_nr(sol, p, _nr(sol), ws_bytes=sol.sol_qk_norm_rope_bwd_workspace_bytes(p) - 1) == sol.SOL_ERR_WORKSPACE
    # a norm without tables or weights passes the checks and reaches the next one
    bare = _nr(sol, q_weight=None, k_weight=None, rot_dim=0, cos=None, sin=None)
    assert _bwd_nr(sol, p, bare, ws_bytes=1) == sol.SOL_ERR_WORKSPACE


def test_make_norm_rope(sol):
    w, t = torch.ones(128), torch.zeros(10, 32)
    nr = sol.make_norm_rope(w, w, t, t.clone())
    assert (nr.rot_dim, nr.weight_type, nr.table_stride_n, nr.table_stride_b) == (64, 0, 32, 0)
    assert nr.tensors[0] is w
    nr = sol.make_norm_rope(w.bfloat16(), None, torch.zeros(3, 10, 32), torch.zeros(3, 10, 32), interleaved=True)
    assert (nr.weight_type, nr.interleaved, nr.table_stride_b, nr.k_weight) == (1, 1, 320, None)
    assert sol.make_norm_rope(None, None).rot_dim == 0
    for bad in (lambda: sol.make_norm_rope(w, w.bfloat16()), lambda: sol.make_norm_rope(w.double(), None),
                lambda: sol.make_norm_rope(w, w, t), lambda: sol.make_norm_rope(w, w, t, t.double()),
                lambda: sol.make_norm_rope(w, w, t, t[:, :16]), lambda: sol.make_norm_rope(w, w, t, t, rot_dim=32),
                lambda: sol.make_norm_rope(w, w, t, torch.zeros(32, 10).t()), lambda: sol.make_norm_rope(w, w, rot_dim=16),
                lambda: sol.make_norm_rope(torch.ones(256)[::2], w)):
        with pytest.raises(ValueError):
            bad()


def test_python_refusals(sol):
    q = torch.zeros(1, 64, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sol.differentiable_attention(q, q, q)           # host tensors
    with pytest.raises(ValueError):
        sol.qk_norm_rope(q, q, None, None)
    p = sol.make_params(1, 64, 2, 64)
    buf = sol.alloc_buffers(p, "cpu")
    with pytest.raises(ValueError, match="lse"):
        sol.backward(p, q, q, q, buf, q, sol.alloc_grads(p, "cpu"))


def test_no_gpu_is_an_error(sol):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    p = sol.make_params(1, 100, 4, 128)
    assert _bwd(sol, p) == sol.SOL_ERR_CUDA
    assert _fwd_nr(sol, p, _nr(sol)) == sol.SOL_ERR_CUDA


def test_tables_and_weights_must_cover_the_call(sol):
    w, t = torch.ones(64), torch.zeros(10, 32)
    x = torch.zeros(2, 10, 1, 64, dtype=torch.bfloat16)
    call = lambda p, nr: sol.sol_qk_norm_rope(p, nr, x, x, x, x)
    back = lambda p, nr: sol.sol_qk_norm_rope_bwd(p, nr, x, x, x, x, x, x, None, None, x)
    for p, nr in ((sol.make_params(2, 11, 1, 64), sol.make_norm_rope(w, w, t, t)),                 # a position too many
                  (sol.make_params(2, 10, 1, 128), sol.make_norm_rope(w, w)),                      # longer heads
                  (sol.make_params(3, 10, 1, 64), sol.make_norm_rope(w, w, t.expand(2, 10, 32), t.expand(2, 10, 32)))):
        for f in (call, back):
            with pytest.raises(ValueError, match="cover"):
                f(p, nr)
    with pytest.raises(ValueError):
        sol.make_norm_rope(torch.ones(64), torch.ones(128))
    with pytest.raises(ValueError):
        sol.make_norm_rope(torch.ones(1, 64), None)
    with pytest.raises(ValueError, match="gradient"):
        sol.qk_norm_rope(x, x, w, w, t.requires_grad_(), t.detach())


def test_empty_call_without_weight_gradients_enqueues_nothing(sol):
    p = sol.make_params(1, 0, 4, 128)
    over = dict.fromkeys(("q", "k", "dqo", "dko", "dq", "dk", "dqw", "dkw", "ws"))
    assert _bwd_nr(sol, p, _nr(sol), **over) == sol.SOL_OK


# ---- autograd functions: what the kernels are given in the backward pass -------------------------------
def _host_autograd(sol, monkeypatch):
    """The autograd functions on host tensors, the library's calls replaced by recorders that read what the
    kernels would read: every (b, n, h, d) through the strides of the sol_params, inside the tensor."""
    import contextlib
    seen = {}

    def rows(p, x):
        st = (p.in_stride_b, p.in_stride_n, p.in_stride_h, 1)
        last = sum((n - 1) * s for n, s in zip((p.B, p.N, p.H, p.D), st))
        assert x.storage_offset() + last < x.untyped_storage().nbytes() // x.element_size(), "read out of range"
        return x.as_strided((p.B, p.N, p.H, p.D), st).clone()

    def attn_bwd(p, q, k, v, ws, row_ptr, col_idx, o, lse, d_o, dq, dk, dv, bws, gs):
        seen.update(qkv=[rows(p, x) for x in (q, k, v)], o=o, ws=ws, lse=lse)
        for t in (dq, dk, dv):
            t.zero_()

    def norm_bwd(p, nr, q, k, dqo, dko, dq, dk, dqw, dkw, ws, grad_strides):
        seen.update(qk=[rows(p, x) for x in (q, k)], nr=nr, grad_strides=grad_strides)
        for t in (dq, dk, dqw, dkw):
            if t is not None:
                t.zero_()

    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(sol, "forward", lambda p, q, k, v, buf: [t.zero_() for t in (buf.o, buf.lse, buf.ws, buf.row_ptr, buf.col_idx)])
    monkeypatch.setattr(sol, "sol_qk_norm_rope", lambda p, nr, q, k, qo, ko: (qo.zero_(), ko.zero_()))
    monkeypatch.setattr(sol, "sol_attn_bwd", attn_bwd)
    monkeypatch.setattr(sol, "sol_qk_norm_rope_bwd", norm_bwd)
    return seen


HOOKS = [(lambda t: t, lambda t: t),                                          # none
         (lambda t: t.clone(memory_format=torch.contiguous_format), lambda t: t),   # dense copies, as offloading makes
         (lambda t: t, lambda t: t if t.dim() < 4 else t.transpose(1, 2).contiguous().transpose(1, 2))]


@pytest.mark.parametrize("hooks", HOOKS)
def test_backward_reads_the_saved_tensors_as_they_come_back(sol, monkeypatch, hooks):
    """Views of a fused projection, saved through hooks that give them back with other strides."""
    seen = _host_autograd(sol, monkeypatch)
    B, N, H, D = 2, 100, 3, 64
    qkv = torch.randn(B, N, 3, H, D).bfloat16().requires_grad_()
    q, k, v = qkv.unbind(2)
    p = sol.make_params(B, N, H, D, in_strides=q.stride()[:3])
    with torch.autograd.graph.saved_tensors_hooks(*hooks):
        o = sol._Attention.apply(q, k, v, p)
    o.sum().backward()
    assert all(torch.equal(a, b) for a, b in zip(seen["qkv"], (q, k, v)))
    assert seen["o"].is_contiguous() and seen["lse"].is_contiguous() and seen["ws"].is_contiguous()
    with torch.autograd.graph.saved_tensors_hooks(*hooks):
        qo, ko = sol._QKNormRope.apply(q, k, None, None, None, None, 1e-6, False)
    (qo.sum() + ko.sum()).backward()
    assert all(torch.equal(a, b) for a, b in zip(seen["qk"], (q, k)))


def test_saved_tensors_of_another_kind_are_refused(sol, monkeypatch):
    """Hooks that give back another type, shape or device: an error, not a read through a wrong address."""
    _host_autograd(sol, monkeypatch)
    x = torch.randn(1, 10, 1, 64).bfloat16().requires_grad_()
    p = sol.make_params(1, 10, 1, 64)
    for unpack in (lambda t: t.float(), lambda t: t[:, :5] if t.dim() == 4 else t, lambda t: t.to("meta")):
        with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
            o = sol._Attention.apply(x, x, x, p)
            qo, _ = sol._QKNormRope.apply(x, x, None, None, None, None, 1e-6, False)
        for t in (o, qo):
            with pytest.raises(ValueError, match="saved"):
                t.sum().backward()


def test_backward_takes_weights_and_tables_from_the_saved_tensors(sol, monkeypatch):
    """Weights whose storage is released after the forward and renewed before the backward pass, and weights and
    tables that hooks give back at other addresses: the call has the addresses of what is there now."""
    seen = _host_autograd(sol, monkeypatch)
    B, N, H, D = 1, 10, 2, 64
    x = torch.randn(B, N, H, D).bfloat16().requires_grad_()
    w = [torch.randn(D, requires_grad=True) for _ in range(2)]
    cos, sin = torch.randn(N, 16), torch.randn(N, 16)
    args = lambda: (x, x, *w, cos, sin, 1e-5, True)
    addresses = lambda: [seen["nr"].q_weight, seen["nr"].k_weight, seen["nr"].cos, seen["nr"].sin]

    qo, ko = sol._QKNormRope.apply(*args())
    kept, other = [t.detach().clone() for t in w], []
    for t, c in zip(w, kept):
        t.untyped_storage().resize_(0)
        other.append(torch.empty(D))          # takes the place
        t.untyped_storage().resize_(4 * D)
        t.data.copy_(c)
    (qo.sum() + ko.sum()).backward()
    assert addresses() == [t.data_ptr() for t in (*w, cos, sin)]
    assert abs(seen["nr"].eps - 1e-5) < 1e-11 and seen["nr"].interleaved == 1 and seen["nr"].rot_dim == 32

    # (a copy one element into its storage: made aligned; tables whose rows are not contiguous: made dense)
    def unpack(t):
        if t.dtype != torch.float32:
            return t
        if t.dim() == 2:
            return t.t().contiguous().t()
        return torch.cat((torch.zeros(1), t.detach()))[1:]

    with torch.autograd.graph.saved_tensors_hooks(lambda t: t, unpack):
        qo, ko = sol._QKNormRope.apply(*args())
    (qo.sum() + ko.sum()).backward()
    nr = seen["nr"]
    assert not set(addresses()) & {t.data_ptr() for t in (*w, cos, sin)}
    assert all(a % 16 == 0 for a in addresses()) and nr.table_stride_n == 16
    assert all(torch.equal(a, b) for a, b in zip(nr.tensors, (*w, cos, sin)))


def test_empty_calls_take_empty_tables(sol):
    """Tables of no positions (or of no batch entries) have no address: with B or N = 0 that is a valid call."""
    for B, N, tables in ((2, 0, torch.zeros(0, 32)), (2, 0, torch.zeros(2, 0, 32)), (0, 5, torch.zeros(0, 5, 32))):
        p = sol.make_params(B, N, 4, 128)
        nr = sol.make_norm_rope(None, None, tables, tables.clone())
        assert nr.rot_dim == 64 and not nr.cos
        assert _fwd_nr(sol, p, nr, None, None, None, None) == sol.SOL_OK, _text(sol)
        over = dict.fromkeys(("q", "k", "dqo", "dko", "dq", "dk", "dqw", "dkw", "ws"))
        assert _bwd_nr(sol, p, nr, **over) == sol.SOL_OK, _text(sol)
    full = sol.make_params(2, 5, 4, 128)
    assert _fwd_nr(sol, full, nr) == sol.SOL_ERR_INVALID_ARG and "NULL table" in _text(sol)


@pytest.mark.parametrize("layout", ["dense", "fused", "expanded", "head-major"])
def test_reblocked_gradient_reads_d_o_where_it_lies(sol, monkeypatch, layout):
    """q, k, v are views of a fused projection; the output's gradient has a layout of its own."""
    B, N, H, D = 1, 100, 2, 64
    fused = torch.randn(B, N, 3, H, D).bfloat16()
    q = fused.unbind(2)[0]
    p = sol.make_params(B, N, H, D, in_strides=q.stride()[:3])
    d_o = {"dense": torch.randn(B, N, H, D).bfloat16(), "fused": torch.randn(B, N, 3, H, D).bfloat16()[:, :, 1],
           "expanded": torch.randn(D).bfloat16().expand(B, N, H, D),
           "head-major": torch.randn(B, H, N, D).bfloat16().transpose(1, 2)}[layout]
    seen = []

    def gather(gp, perm, x, xp, stream=None):
        st = (gp.in_stride_b, gp.in_stride_n, gp.in_stride_h, 1)
        last = x.storage_offset() + sum((n - 1) * s for n, s in zip((B, N, H, D), st))
        assert last < x.untyped_storage().nbytes() // 2, "read out of range"
        seen.append(x.as_strided((B, N, H, D), st))

    monkeypatch.setattr(sol, "sol_gather_rows", gather)
    monkeypatch.setattr(sol, "sol_attn_bwd", lambda *a, **k: None)
    monkeypatch.setattr(sol, "sol_scatter_rows", lambda *a, **k: None)
    rb = sol.alloc_reblock(p, "cpu", with_lse=True)
    sol.backward_reblocked(p, rb, d_o, sol.alloc_grads(p, "cpu"))
    assert torch.equal(seen[0], d_o)
    for bad in (d_o.float(), d_o[:, :50], torch.randn(B, N, H, 2 * D).bfloat16()[..., ::2]):
        with pytest.raises(ValueError, match="d_o"):
            sol.backward_reblocked(p, rb, bad, sol.alloc_grads(p, "cpu"))


def test_backward_refuses_a_gradient_that_is_not_laid_out_as_the_output(sol, monkeypatch):
    """o and d_o share p's out_strides: an expanded, transposed or fp32 d_o would be read past its end."""
    B, N, H, D = 1, 64, 2, 64
    x = torch.randn(B, N, H, D).bfloat16()
    p = sol.make_params(B, N, H, D)
    buf, g, calls = sol.alloc_buffers(p, "cpu", with_lse=True), sol.alloc_grads(p, "cpu"), []
    monkeypatch.setattr(sol, "sol_attn_bwd", lambda *a, **k: calls.append(a))
    for bad in (torch.ones(()).bfloat16().expand(B, N, H, D), x.transpose(1, 2), x.float(), x[:, :5],
                torch.zeros(B, H, N, D).bfloat16().transpose(1, 2)):
        with pytest.raises(ValueError, match="d_o"):
            sol.backward(p, x, x, x, buf, bad, g)
    assert not calls
    sol.backward(p, x, x, x, buf, x, g)
    fused = torch.randn(B, N, 2, H, D).bfloat16()[:, :, 1]
    p2 = sol.make_params(B, N, H, D, out_strides=fused.stride()[:3])
    sol.backward(p2, x, x, x, buf, fused, g)
    one = sol.make_params(1, 1, H, D)   # dims of one: any stride
    sol.backward(one, x[:, :1], x[:, :1], x[:, :1], buf, x[:, 3:4], g)
    assert len(calls) == 3


def test_weights_and_tables_without_storage_are_refused(sol):
    """A weight whose storage was released (sharded weights not gathered) has no address: NULL would mean ones."""
    w, t = torch.ones(64), torch.zeros(10, 32)
    empty = [x.clone() for x in (w, t)]
    for x in empty:
        x.untyped_storage().resize_(0)
    for args in ((empty[0], None), (None, empty[0]), (w, w, empty[1], t), (w, w, t, empty[1])):
        with pytest.raises(ValueError, match="storage"):
            sol.make_norm_rope(*args)
    assert sol.make_norm_rope(w, w, torch.zeros(0, 32), torch.zeros(0, 32)).rot_dim == 64   # no positions


def test_saved_tensors_of_another_size_are_refused(sol, monkeypatch):
    _host_autograd(sol, monkeypatch)
    x = torch.randn(1, 100, 1, 64).bfloat16().requires_grad_()
    w, t = torch.randn(64, requires_grad=True), torch.randn(100, 16)
    p = sol.make_params(1, 100, 1, 64)
    short = lambda dims: lambda s: s[..., :1] if s.dim() == dims and s.numel() > 1 else s
    for dims, run in ((1, lambda: sol._Attention.apply(x, x, x, p)), (3, lambda: sol._Attention.apply(x, x, x, p)),
                      (1, lambda: sol._QKNormRope.apply(x, x, w, None, t, t, 1e-6, False)[0]),
                      (2, lambda: sol._QKNormRope.apply(x, x, w, None, t, t, 1e-6, False)[0])):
        with torch.autograd.graph.saved_tensors_hooks(lambda s: s, short(dims)):
            out = run()
        with pytest.raises(ValueError, match="saved"):
            out.sum().backward()


def test_backward_takes_head_major_and_flat_gradients(sol, monkeypatch):
    """Layouts that are the output's although the tensor's shape is not [B, N, H, D]."""
    calls = []
    monkeypatch.setattr(sol, "sol_attn_bwd", lambda *a, **k: calls.append(a))
    for N in (64, 2):   # (N = H: the shapes are alike)
        B, H, D = 2, 2, 64
        p = sol.make_params(B, N, H, D)
        hm = sol.head_major_params(p)
        x = torch.randn(B, N, H, D).bfloat16()
        xh = x.transpose(1, 2).contiguous()
        buf = sol.alloc_buffers(hm, "cpu", with_lse=True, head_major_out=True)
        g = sol.alloc_grads(p, "cpu")
        for d_o in (xh, xh.view(-1), xh.transpose(1, 2)):
            sol.backward(hm, xh, xh, xh, buf, d_o, g)
        flat = sol.alloc_buffers(p, "cpu", with_lse=True)
        for d_o in (x, x.view(B, N, H * D), x.view(-1)):
            sol.backward(p, x, x, x, flat, d_o, g)
        for q, b, d_o in ((p, flat, x.view(-1)[:-8]), (p, flat, x.view(B, N, H * D)[:, :, ::2])):
            with pytest.raises(ValueError, match="d_o"):
                sol.backward(q, x, x, x, b, d_o, g)
    with pytest.raises(ValueError, match="d_o"):   # the output is head-major, d_o is not
        p = sol.make_params(1, 64, 2, 64)
        x = torch.randn(1, 64, 2, 64).bfloat16()
        hm = sol.head_major_params(p)
        sol.backward(hm, x, x, x, sol.alloc_buffers(hm, "cpu", with_lse=True, head_major_out=True), x, sol.alloc_grads(p, "cpu"))
    assert len(calls) == 12


def test_reblocked_gradient_takes_flat_gradients_laid_out_as_the_inputs(sol, monkeypatch):
    B, N, H, D = 1, 100, 2, 64
    x = torch.randn(B, N, H, D).bfloat16()
    seen = []
    monkeypatch.setattr(sol, "sol_gather_rows", lambda gp, perm, t, tp, stream=None: seen.append(
        (t.data_ptr(), gp.in_stride_b, gp.in_stride_n, gp.in_stride_h)))
    monkeypatch.setattr(sol, "sol_attn_bwd", lambda *a, **k: None)
    monkeypatch.setattr(sol, "sol_scatter_rows", lambda *a, **k: None)
    for p, shapes in ((sol.make_params(B, N, H, D), ((B, N, H * D), (-1,))),
                      (sol.head_major_params(sol.make_params(B, N, H, D)), ((B, H, N, D),))):
        rb = sol.alloc_reblock(p, "cpu", with_lse=True)
        for shape in shapes:
            sol.backward_reblocked(p, rb, x.view(shape), sol.alloc_grads(p, "cpu"))
            assert seen.pop() == (x.data_ptr(), p.in_stride_b, p.in_stride_n, p.in_stride_h)
        with pytest.raises(ValueError, match="d_o"):
            sol.backward_reblocked(p, rb, x.view(-1)[:-8], sol.alloc_grads(p, "cpu"))


def test_gradients_of_joined_heads_are_taken_where_they_lie(sol, monkeypatch):
    """d_o as [B, N, H D], a view of something wider (the projection behind the attention takes such rows)."""
    calls, gathers = [], []
    monkeypatch.setattr(sol, "sol_attn_bwd", lambda *a, **k: calls.append(a))
    monkeypatch.setattr(sol, "sol_gather_rows", lambda gp, *a: gathers.append(gp))
    monkeypatch.setattr(sol, "sol_scatter_rows", lambda *a: None)
    B, N, H, D = 2, 30, 2, 64
    x = torch.randn(B, N, H, D).bfloat16()
    wide = torch.randn(B, N, 3 * H * D).bfloat16()[:, :, H * D:2 * H * D]
    st = (N * 3 * H * D, 3 * H * D, D)
    p = sol.make_params(B, N, H, D, in_strides=st, out_strides=st)
    buf, g = sol.alloc_buffers(p, "cpu", with_lse=True), sol.alloc_grads(p, "cpu")
    sol.backward(p, x, x, x, buf, wide, g)
    rb = sol.alloc_reblock(p, "cpu", with_lse=True)
    sol.backward_reblocked(p, rb, wide, g)
    assert len(calls) == 2 and gathers[0].in_stride_n == 3 * H * D
    dense = wide.contiguous()
    for bad_p in (p, sol.head_major_params(p)):   # rows closer together than p says; heads that are not joined
        with pytest.raises(ValueError, match="d_o"):
            sol.backward(bad_p, x, x, x, buf, dense, g)
        with pytest.raises(ValueError, match="d_o"):
            sol.backward_reblocked(bad_p, rb, dense, g)
