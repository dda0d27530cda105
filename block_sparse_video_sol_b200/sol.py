"""Thin ctypes binding of libsol.so (the C ABI declared in include/sol.h).

Argument marshalling only: every step of the forward pass runs in the CUDA
kernels of libsol.so.  Torch tensors supply device memory and the current
stream; nothing here computes.  Importing this module loads the library and
raises if it is missing -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

_LIB_PATH = os.environ.get("SOL_LIB_PATH") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libsol.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libsol.so not built ({_LIB_PATH}); run `python -m block_sparse_video_sol_b200.build`")
lib = ctypes.CDLL(_LIB_PATH)

SOL_OK, SOL_ERR_INVALID_ARG, SOL_ERR_UNSUPPORTED, SOL_ERR_WORKSPACE, SOL_ERR_CUDA, SOL_ERR_TIMEOUT = range(6)

# Every entry point declared in include/sol.h.
EXPORTS = ("sol_workspace_bytes", "sol_workspace_offsets", "sol_workspace_int8_offsets", "sol_col_capacity", "sol_pool", "sol_route", "sol_route_static",
           "sol_attn_fwd", "sol_forward_host", "sol_host_staging_bytes", "sol_last_device_status",
           "sol_status_string", "sol_last_error_text", "sol_debug_drop_arrive",
           "sol_reblock_workspace_bytes", "sol_reblock", "sol_gather_rows", "sol_scatter_rows",
           "sol_attn_bwd_workspace_bytes", "sol_attn_bwd", "sol_qk_norm_rope",
           "sol_qk_norm_rope_bwd_workspace_bytes", "sol_qk_norm_rope_bwd")


class sol_params(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("H", ctypes.c_int32), ("D", ctypes.c_int32),
                ("q_block", ctypes.c_int32), ("k_block", ctypes.c_int32),
                ("tau", ctypes.c_float), ("scale", ctypes.c_float),
                ("prefix_len", ctypes.c_int32), ("log_mass_bias", ctypes.c_int32),
                ("in_stride_b", ctypes.c_int64), ("in_stride_n", ctypes.c_int64), ("in_stride_h", ctypes.c_int64),
                ("out_stride_b", ctypes.c_int64), ("out_stride_n", ctypes.c_int64), ("out_stride_h", ctypes.c_int64),
                ("routing", ctypes.c_int32), ("topk_ratio", ctypes.c_float), ("qk_int8", ctypes.c_int32)]


class sol_norm_rope(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("weight_type", ctypes.c_int32),
                ("eps", ctypes.c_float), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p),
                ("table_stride_b", ctypes.c_int64), ("table_stride_n", ctypes.c_int64)]


_P = ctypes.POINTER(sol_params)
_NR = ctypes.POINTER(sol_norm_rope)
_I64P = ctypes.POINTER(ctypes.c_int64)
_vp = ctypes.c_void_p
lib.sol_workspace_bytes.argtypes = [_P]
lib.sol_workspace_bytes.restype = ctypes.c_size_t
lib.sol_workspace_offsets.argtypes = [_P, ctypes.POINTER(ctypes.c_int64)]
lib.sol_workspace_offsets.restype = ctypes.c_int
lib.sol_workspace_int8_offsets.argtypes = [_P, ctypes.POINTER(ctypes.c_int64)]
lib.sol_workspace_int8_offsets.restype = ctypes.c_int
lib.sol_col_capacity.argtypes = [_P]
lib.sol_col_capacity.restype = ctypes.c_int64
lib.sol_pool.argtypes = [_P, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
lib.sol_pool.restype = ctypes.c_int
lib.sol_route.argtypes = [_P, _vp, ctypes.c_size_t, _vp, _vp, _vp]
lib.sol_route.restype = ctypes.c_int
lib.sol_route_static.argtypes = [_P, _vp, ctypes.c_size_t, _vp, _vp, _vp]
lib.sol_route_static.restype = ctypes.c_int
lib.sol_attn_fwd.argtypes = [_P, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp, _vp, _vp]
lib.sol_attn_fwd.restype = ctypes.c_int
lib.sol_forward_host.argtypes = [_P, _vp, _vp, _vp, _vp, ctypes.c_int32, _vp, ctypes.c_size_t, _vp]
lib.sol_forward_host.restype = ctypes.c_int
lib.sol_host_staging_bytes.argtypes = [_P, ctypes.c_int32]
lib.sol_host_staging_bytes.restype = ctypes.c_size_t
lib.sol_last_device_status.argtypes = [_vp]
lib.sol_last_device_status.restype = ctypes.c_int
lib.sol_status_string.argtypes = [ctypes.c_int]
lib.sol_status_string.restype = ctypes.c_char_p
lib.sol_last_error_text.argtypes = []
lib.sol_last_error_text.restype = ctypes.c_char_p
lib.sol_debug_drop_arrive.argtypes = [ctypes.c_int32]
lib.sol_debug_drop_arrive.restype = ctypes.c_int
lib.sol_reblock_workspace_bytes.argtypes = [_P]
lib.sol_reblock_workspace_bytes.restype = ctypes.c_size_t
lib.sol_reblock.argtypes = [_P, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp]
lib.sol_reblock.restype = ctypes.c_int
lib.sol_gather_rows.argtypes = [_P, _vp, _vp, _vp, _vp]
lib.sol_gather_rows.restype = ctypes.c_int
lib.sol_scatter_rows.argtypes = [_P, _vp, _vp, _vp, _vp]
lib.sol_scatter_rows.restype = ctypes.c_int
lib.sol_attn_bwd_workspace_bytes.argtypes = [_P]
lib.sol_attn_bwd_workspace_bytes.restype = ctypes.c_size_t
lib.sol_attn_bwd.argtypes = [_P, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _I64P,
                             _vp, ctypes.c_size_t, _vp]
lib.sol_attn_bwd.restype = ctypes.c_int
lib.sol_qk_norm_rope.argtypes = [_P, _NR, _vp, _vp, _vp, _vp, _vp]
lib.sol_qk_norm_rope.restype = ctypes.c_int
lib.sol_qk_norm_rope_bwd_workspace_bytes.argtypes = [_P]
lib.sol_qk_norm_rope_bwd_workspace_bytes.restype = ctypes.c_size_t
lib.sol_qk_norm_rope_bwd.argtypes = [_P, _NR, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _I64P, _vp, ctypes.c_size_t, _vp]
lib.sol_qk_norm_rope_bwd.restype = ctypes.c_int


class SolError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        text = lib.sol_last_error_text().decode()
        super().__init__(f"{where}: {lib.sol_status_string(status).decode()} ({text})")


def _check(status: int, where: str):
    if status != SOL_OK:
        raise SolError(status, where)


def make_params(B: int, N: int, H: int, D: int, tau: float = 1.0, prefix_len: int = 0,
                log_mass_bias: int = 0, scale: float = 0.0, in_strides=None, out_strides=None,
                q_block: Optional[int] = None, k_block: int = 64, topk_ratio: Optional[float] = None,
                compressed: bool = False, qk_int8: bool = False) -> sol_params:
    """Fill a sol_params; strides default to contiguous BTHD [B, N, H, D].

    ``log_mass_bias``: 0 (or False) mean-pooled centroids, 1 (or True) plus the
    log-mass bias, 2 anchor-weighted key/value summaries with the bias.
    ``topk_ratio`` selects Top-K routing: the SLA variant (128-row query
    blocks, unselected blocks dropped), or with ``compressed`` the Spark-H3
    configuration (64-row blocks, sink and centroid terms as under threshold
    routing); otherwise threshold routing with ``tau``.
    """
    routing = 0 if topk_ratio is None else (2 if compressed else 1)
    if q_block is None:
        q_block = 128 if routing == 1 else 64
    in_strides = in_strides or (N * H * D, H * D, D)
    out_strides = out_strides or (N * H * D, H * D, D)
    return sol_params(B, N, H, D, q_block, k_block, float(tau), float(scale), prefix_len, int(log_mass_bias),
                      *[int(s) for s in in_strides], *[int(s) for s in out_strides], routing,
                      float(topk_ratio or 0.0), int(bool(qk_int8)))


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    # torch.cuda.current_stream().cuda_stream without the Stream object (0.3 us against 3.2, of a 10 us call)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def sol_workspace_bytes(p: sol_params) -> int:
    return lib.sol_workspace_bytes(ctypes.byref(p))


def sol_workspace_offsets(p: sol_params) -> list:
    out = (ctypes.c_int64 * 8)()
    _check(lib.sol_workspace_offsets(ctypes.byref(p), out), "sol_workspace_offsets")
    return list(out)


def workspace_views(p: sol_params, ws: torch.Tensor) -> dict:
    """Typed views of the pooled quantities inside a workspace (see sol_workspace_offsets)."""
    off = sol_workspace_offsets(p)
    nb = -(-p.N // 64)   # the workspace holds 64-row blocks for Q and K whatever the routing
    mw = -(-nb // 32)
    B, H, D = p.B, p.H, p.D

    def view(i, dtype, shape):
        n = math.prod(shape)
        esz = torch.tensor([], dtype=dtype).element_size()
        return ws[off[i]:off[i] + n * esz].view(dtype).view(*shape)

    return dict(qbar=view(0, torch.float32, (B, H, nb, D)), kbar=view(1, torch.float32, (B, H, nb, D)),
                kbar16=view(2, torch.bfloat16, (B, H, nb, D)), vbar16=view(3, torch.bfloat16, (B, H, nb, D)),
                cbias=view(4, torch.float32, (B, H, nb)), anchor=view(5, torch.float32, (B, H, D)),
                mask=view(6, torch.int32, (B * H * nb, mw)), counts=view(7, torch.int32, (B * H * nb,)))


def int8_views(p: sol_params, ws: torch.Tensor) -> dict:
    """Typed views of the INT8 QK quantities sol_pool leaves in a workspace (qk_int8 = 1)."""
    off = (ctypes.c_int64 * 3)()
    _check(lib.sol_workspace_int8_offsets(ctypes.byref(p), off), "sol_workspace_int8_offsets")
    nb = -(-p.N // 64)
    B, H, N, D = p.B, p.H, p.N, p.D
    return dict(kcode=ws[off[0]:off[0] + B * H * N * D].view(torch.int8).view(B, H, N, D),
                ksig=ws[off[1]:off[1] + B * H * nb * 4].view(torch.float32).view(B, H, nb),
                kmean16=ws[off[2]:off[2] + B * H * nb * D * 2].view(torch.bfloat16).view(B, H, nb, D))


def sol_col_capacity(p: sol_params) -> int:
    return lib.sol_col_capacity(ctypes.byref(p))


def sol_pool(p: sol_params, q, k, v, ws: torch.Tensor, stream=None):
    _check(lib.sol_pool(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(ws), ws.numel() * ws.element_size(),
                        _stream(stream)), "sol_pool")


def sol_route(p: sol_params, ws: torch.Tensor, row_ptr: torch.Tensor, col_idx: torch.Tensor, stream=None):
    _check(lib.sol_route(ctypes.byref(p), _ptr(ws), ws.numel() * ws.element_size(), _ptr(row_ptr), _ptr(col_idx),
                         _stream(stream)), "sol_route")


def sol_route_static(p: sol_params, ws: torch.Tensor, row_ptr: torch.Tensor, col_idx: torch.Tensor,
                     stream=None):
    """Routing without caller scratch (see include/sol.h); ws may hold only the pooled part."""
    _check(lib.sol_route_static(ctypes.byref(p), _ptr(ws), ws.numel() * ws.element_size(), _ptr(row_ptr),
                                _ptr(col_idx), _stream(stream)), "sol_route_static")


def sol_host_staging_bytes(p: sol_params, heads_per_chunk: int = 0) -> int:
    return lib.sol_host_staging_bytes(ctypes.byref(p), heads_per_chunk)


def sol_forward_host(p: sol_params, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                     staging: torch.Tensor, heads_per_chunk: int = 0, stream=None):
    """Whole forward pass on host (CPU) tensors, pipelined over head chunks (see include/sol.h).

    q, k, v, o are CPU bf16 tensors (pinned for copy/compute overlap); staging is a
    CUDA uint8 tensor of at least sol_host_staging_bytes(p, heads_per_chunk) bytes.
    Asynchronous: synchronise the stream before reading o."""
    for t in (q, k, v, o):
        if t.is_cuda:
            raise ValueError("sol_forward_host takes host tensors")
    _check(lib.sol_forward_host(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), heads_per_chunk, _ptr(staging),
                                staging.numel() * staging.element_size(), _stream(stream)), "sol_forward_host")


def sol_attn_fwd(p: sol_params, q, k, v, ws: torch.Tensor, row_ptr: torch.Tensor, col_idx: torch.Tensor,
                 o: torch.Tensor, lse: Optional[torch.Tensor] = None, stream=None):
    _check(lib.sol_attn_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(ws), ws.numel() * ws.element_size(),
                            _ptr(row_ptr), _ptr(col_idx), _ptr(o), _ptr(lse), _stream(stream)), "sol_attn_fwd")


def _strides3(strides):
    return None if strides is None else (ctypes.c_int64 * 3)(*[int(x) for x in strides])


def sol_attn_bwd_workspace_bytes(p: sol_params) -> int:
    return lib.sol_attn_bwd_workspace_bytes(ctypes.byref(p))


def sol_attn_bwd(p: sol_params, q, k, v, ws: torch.Tensor, row_ptr: torch.Tensor, col_idx: torch.Tensor,
                 o: torch.Tensor, lse: torch.Tensor, d_o: torch.Tensor, dq, dk, dv, bws: torch.Tensor,
                 grad_strides=None, stream=None):
    """Gradients of sol_attn_fwd into dq, dk, dv (element strides ``grad_strides`` = (b, n, h), or p's
    in_strides); ws, row_ptr, col_idx, o and lse are the forward's (see include/sol.h)."""
    _check(lib.sol_attn_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(ws), ws.numel() * ws.element_size(),
                            _ptr(row_ptr), _ptr(col_idx), _ptr(o), _ptr(lse), _ptr(d_o), _ptr(dq), _ptr(dk), _ptr(dv),
                            _strides3(grad_strides), _ptr(bws), bws.numel() * bws.element_size(), _stream(stream)),
           "sol_attn_bwd")


def _place(nr: sol_norm_rope, q_weight, k_weight, cos, sin):
    """The addresses of now and the tables' strides into nr, which keeps the tensors alive."""
    nr.tensors = (q_weight, k_weight, cos, sin)
    nr.q_weight, nr.k_weight = _ptr(q_weight), _ptr(k_weight)
    if nr.rot_dim:
        nr.cos, nr.sin = _ptr(cos), _ptr(sin)
        nr.table_stride_n = cos.stride(-2) if cos.shape[-2] > 1 else 0
        nr.table_stride_b = cos.stride(0) if cos.dim() == 3 and cos.shape[0] > 1 else 0
    if ((q_weight is not None and not nr.q_weight) or (k_weight is not None and not nr.k_weight)
            or (nr.rot_dim and cos.numel() and not (nr.cos and nr.sin))):
        raise ValueError("a weight or table has no storage")   # (a NULL weight would mean ones)


def make_norm_rope(q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor],
                   cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   rot_dim: Optional[int] = None, interleaved: bool = False) -> sol_norm_rope:
    """Fill a sol_norm_rope (it keeps the tensors alive, and holds their addresses of now: fill another
    one when a tensor's storage has moved).

    The weights are [D], both fp32 or both bf16 (None: ones).  cos and sin are fp32
    [N, rot_dim/2] or [B, N, rot_dim/2] with equal strides and contiguous rows; without them
    only the norm is applied.  ``rot_dim`` defaults to the tables' width.
    """
    weights = [w for w in (q_weight, k_weight) if w is not None]
    for w in weights:
        if (w.dtype not in (torch.float32, torch.bfloat16) or w.dtype != weights[0].dtype or not w.is_contiguous()
                or w.dim() != 1 or w.shape != weights[0].shape):
            raise ValueError("the weights must be contiguous, of one length, both fp32 or both bf16")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin come together")
    if cos is None:
        if rot_dim:
            raise ValueError("rot_dim needs the cos and sin tables")
        rot_dim = 0
    else:
        if cos.dtype != torch.float32 or sin.dtype != torch.float32 or cos.shape != sin.shape or cos.dim() not in (2, 3):
            raise ValueError("cos and sin must be fp32 tables of one shape, [N, rot_dim/2] or [B, N, rot_dim/2]")
        rot_dim = 2 * cos.shape[-1] if rot_dim is None else rot_dim
        if rot_dim != 2 * cos.shape[-1]:
            raise ValueError(f"rot_dim {rot_dim} needs tables of width {rot_dim // 2}, got {cos.shape[-1]}")
        if cos.numel() and (cos.stride() != sin.stride() or cos.stride(-1) != 1):
            raise ValueError("cos and sin must have identical strides and contiguous rows")
    nr = sol_norm_rope(weight_type=int(bool(weights) and weights[0].dtype == torch.bfloat16), eps=float(eps),
                       rot_dim=int(rot_dim), interleaved=int(bool(interleaved)))
    _place(nr, q_weight, k_weight, cos, sin)
    # what they cover: head dims, positions, batch entries (None: any)
    nr.covers = (weights[0].shape[0] if weights else None, cos.shape[-2] if rot_dim else None,
                 cos.shape[0] if rot_dim and cos.dim() == 3 and cos.shape[0] > 1 else None)
    return nr


def _check_covers(p: sol_params, nr: sol_norm_rope):
    D, N, B = getattr(nr, "covers", (None, None, None))   # a structure filled by hand has none
    if (D is not None and D != p.D) or (N is not None and N < p.N) or (B is not None and B < p.B):
        raise ValueError(f"weights of {D} dims and tables of {B} x {N} positions do not cover B={p.B}, N={p.N}, D={p.D}")


def sol_qk_norm_rope(p: sol_params, nr: sol_norm_rope, q, k, qo, ko, stream=None):
    """RMS norm per head and position rotation of q and k (p's in_strides) into qo and ko (p's out_strides)."""
    _check_covers(p, nr)
    _check(lib.sol_qk_norm_rope(ctypes.byref(p), ctypes.byref(nr), _ptr(q), _ptr(k), _ptr(qo), _ptr(ko),
                                _stream(stream)), "sol_qk_norm_rope")


def sol_qk_norm_rope_bwd_workspace_bytes(p: sol_params) -> int:
    return lib.sol_qk_norm_rope_bwd_workspace_bytes(ctypes.byref(p))


def sol_qk_norm_rope_bwd(p: sol_params, nr: sol_norm_rope, q, k, dqo, dko, dq, dk, dq_weight: Optional[torch.Tensor],
                         dk_weight: Optional[torch.Tensor], ws: torch.Tensor, grad_strides=None, stream=None):
    """Gradient of sol_qk_norm_rope: dqo, dko (p's out_strides) into dq, dk (``grad_strides``, or p's
    in_strides) and the fp32 weight gradients (each may be None)."""
    _check_covers(p, nr)
    _check(lib.sol_qk_norm_rope_bwd(ctypes.byref(p), ctypes.byref(nr), _ptr(q), _ptr(k), _ptr(dqo), _ptr(dko),
                                    _ptr(dq), _ptr(dk), _ptr(dq_weight), _ptr(dk_weight), _strides3(grad_strides),
                                    _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "sol_qk_norm_rope_bwd")


def sol_last_device_status(stream=None):
    _check(lib.sol_last_device_status(_stream(stream)), "device status")


def sol_debug_drop_arrive(step: int):
    """Fault-test library only: withhold the attention's "P ready" arrive of S
    tile `step` in every CTA (-1: none), so that its bounded wait expires; in
    the gradient's passes the "dS ready" arrive of that step."""
    _check(lib.sol_debug_drop_arrive(step), "sol_debug_drop_arrive")


def sol_reblock_workspace_bytes(p: sol_params) -> int:
    return lib.sol_reblock_workspace_bytes(ctypes.byref(p))


def sol_reblock(p: sol_params, q, k, ws: torch.Tensor, perm: torch.Tensor, stream=None):
    _check(lib.sol_reblock(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(ws), ws.numel(), _ptr(perm), _stream(stream)),
           "sol_reblock")


def sol_gather_rows(p: sol_params, perm: torch.Tensor, x, xp: torch.Tensor, stream=None):
    _check(lib.sol_gather_rows(ctypes.byref(p), _ptr(perm), _ptr(x), _ptr(xp), _stream(stream)), "sol_gather_rows")


def sol_scatter_rows(p: sol_params, perm: torch.Tensor, xp: torch.Tensor, x, stream=None):
    _check(lib.sol_scatter_rows(ctypes.byref(p), _ptr(perm), _ptr(xp), _ptr(x), _stream(stream)), "sol_scatter_rows")


def reblock_levels(n_v: int) -> int:
    """Split levels (sol_reblock launches one kernel per level) for n_v partitioned rows."""
    lv, leaves = 0, -(-n_v // 64)
    while leaves > 1:
        leaves, lv = -(-leaves // 2), lv + 1
    return lv


def head_major_params(p: sol_params) -> sol_params:
    """The same problem on head-major [B, H, N, D] copies (inputs and output)."""
    hm = (p.H * p.N * p.D, p.D, p.N * p.D)
    return sol_params(p.B, p.N, p.H, p.D, p.q_block, p.k_block, p.tau, p.scale, p.prefix_len, p.log_mass_bias,
                      *hm, *hm, p.routing, p.topk_ratio, p.qk_int8)


@dataclass
class Buffers:
    """Caller-owned device buffers of one problem shape (allocated by torch)."""
    ws: torch.Tensor
    row_ptr: torch.Tensor
    col_idx: torch.Tensor
    o: torch.Tensor
    lse: Optional[torch.Tensor]


def alloc_buffers(p: sol_params, device, with_lse: bool = False, head_major_out: bool = False) -> Buffers:
    """Workspace, CSR and output of one problem; the output is [B, N, H, D], or
    [B, H, N, D] with ``head_major_out`` (the layout of the reblocked copies)."""
    nqb = -(-p.N // 64)   # CSR rows are 64-row query blocks whatever the routing
    ws = torch.empty(max(1, sol_workspace_bytes(p)), dtype=torch.uint8, device=device)
    row_ptr = torch.empty(p.B * p.H * nqb + 1, dtype=torch.int32, device=device)
    col_idx = torch.empty(max(1, sol_col_capacity(p)), dtype=torch.int32, device=device)
    shape = (p.B, p.H, p.N, p.D) if head_major_out else (p.B, p.N, p.H, p.D)
    o = torch.empty(shape, dtype=torch.bfloat16, device=device)
    lse = torch.empty((p.B, p.H, p.N), dtype=torch.float32, device=device) if with_lse else None
    return Buffers(ws, row_ptr, col_idx, o, lse)


@dataclass
class ReblockBuffers:
    """Caller-owned buffers of a reblocked pass: the partition's workspace and
    order, the head-major row copies and the Sol buffers of the copies (whose
    ``o`` is the head-major output, in the partition's order)."""
    ws: torch.Tensor
    perm: torch.Tensor
    qp: torch.Tensor
    kp: torch.Tensor
    vp: torch.Tensor
    hm: sol_params
    buf: Buffers


def alloc_reblock(p: sol_params, device, with_lse: bool = False) -> ReblockBuffers:
    hm = head_major_params(p)
    ws = torch.empty(max(1, sol_reblock_workspace_bytes(p)), dtype=torch.uint8, device=device)
    perm = torch.empty(max(1, p.B * p.H * p.N), dtype=torch.int32, device=device)
    qp, kp, vp = (torch.empty((p.B, p.H, p.N, p.D), dtype=torch.bfloat16, device=device) for _ in range(3))
    return ReblockBuffers(ws, perm, qp, kp, vp, hm, alloc_buffers(hm, device, with_lse, head_major_out=True))


def forward_reblocked(p: sol_params, q, k, v, o: torch.Tensor, rb: ReblockBuffers, stream=None):
    """Partition, gather q/k/v, pool -> route -> attention on the copies, scatter into ``o``."""
    sol_reblock(p, q, k, rb.ws, rb.perm, stream)
    for x, xp in ((q, rb.qp), (k, rb.kp), (v, rb.vp)):
        sol_gather_rows(p, rb.perm, x, xp, stream)
    forward(rb.hm, rb.qp, rb.kp, rb.vp, rb.buf, stream)
    sol_scatter_rows(p, rb.perm, rb.buf.o, o, stream)
    return o


def forward(p: sol_params, q, k, v, buf: Buffers, stream=None) -> Buffers:
    """Enqueue pool -> route -> attention on one stream; returns ``buf``."""
    sol_pool(p, q, k, v, buf.ws, stream)
    sol_route(p, buf.ws, buf.row_ptr, buf.col_idx, stream)
    sol_attn_fwd(p, q, k, v, buf.ws, buf.row_ptr, buf.col_idx, buf.o, buf.lse, stream)
    return buf


@dataclass
class GradBuffers:
    """Caller-owned buffers of one backward pass: its workspace and the gradients
    (contiguous [B, N, H, D], element strides ``strides``)."""
    ws: torch.Tensor
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor
    strides: tuple


def alloc_grads(p: sol_params, device) -> GradBuffers:
    ws = torch.empty(max(1, sol_attn_bwd_workspace_bytes(p)), dtype=torch.uint8, device=device)
    dq, dk, dv = (torch.empty((p.B, p.N, p.H, p.D), dtype=torch.bfloat16, device=device) for _ in range(3))
    return GradBuffers(ws, dq, dk, dv, (p.N * p.H * p.D, p.H * p.D, p.D))


def _lies(dims, tensor_strides, strides) -> bool:
    return not any(n > 1 and a != b for n, a, b in zip(dims, tensor_strides, strides))


def _lies_by(p: sol_params, t: torch.Tensor, strides) -> bool:
    """Whether a tensor that is not [B, N, H, D] lies as the strides say: rows of joined heads [B, N, H D],
    or any dense one that holds every element they reach."""
    if t.shape == (p.B, p.N, p.H * p.D):
        return (p.H == 1 or strides[2] == p.D) and _lies(t.shape, t.stride(), (strides[0], strides[1], 1))
    return t.is_contiguous() and t.numel() > sum((n - 1) * s for n, s in zip((p.B, p.N, p.H, p.D), strides))


def _like_out(p: sol_params, d_o: torch.Tensor, o: torch.Tensor) -> bool:
    """Whether d_o is laid out by p's out_strides: as [B, N, H, D], as o, or in another shape."""
    dims, want = (p.B, p.N, p.H, p.D), (p.out_stride_b, p.out_stride_n, p.out_stride_h, 1)
    if d_o.shape == dims:
        return d_o.stride() == want or (d_o.shape == o.shape and d_o.stride() == o.stride()) or _lies(dims, d_o.stride(), want)
    return _lies_by(p, d_o, want)


def backward(p: sol_params, q, k, v, buf: Buffers, d_o: torch.Tensor, g: GradBuffers, stream=None) -> GradBuffers:
    """Enqueue the gradient of ``forward`` (buf as it left it, with an lse) for d_o (p's out_strides)."""
    if buf.lse is None:
        raise ValueError("the backward pass needs the forward's lse (alloc_buffers(with_lse=True))")
    if d_o.dtype != torch.bfloat16 or not _like_out(p, d_o, buf.o):
        raise ValueError("d_o must be bf16 and laid out by p's out_strides, as buf.o")
    sol_attn_bwd(p, q, k, v, buf.ws, buf.row_ptr, buf.col_idx, buf.o, buf.lse, d_o, g.dq, g.dk, g.dv, g.ws, g.strides,
                 stream)
    return g


def _with_strides(p: sol_params, q: torch.Tensor) -> sol_params:
    """p for inputs laid out as q."""
    r = sol_params.from_buffer_copy(p)
    r.in_stride_b, r.in_stride_n, r.in_stride_h = q.stride()[:3]
    return r


def backward_reblocked(p: sol_params, rb: ReblockBuffers, d_o: torch.Tensor, g: GradBuffers, stream=None) -> GradBuffers:
    """Gradient of ``forward_reblocked`` (rb as it left it, with an lse) for d_o, a bf16 tensor
    [B, N, H, D] of any strides the kernels take (or one of another shape, laid out as p's
    in_strides): gather it into the partition's order, the backward pass there, scatter the three
    gradients back into ``g`` (g.ws from alloc_grads of the same shape)."""
    if rb.buf.lse is None:
        raise ValueError("the backward pass needs the forward's lse (alloc_reblock(with_lse=True))")
    rows = d_o.shape == (p.B, p.N, p.H, p.D) and d_o.stride(3) == 1
    if d_o.dtype != torch.bfloat16 or (not rows and not _lies_by(p, d_o, (p.in_stride_b, p.in_stride_n, p.in_stride_h, 1))):
        raise ValueError("d_o must be bf16 [B, N, H, D] with contiguous head dim")
    hm = (p.H * p.N * p.D, p.D, p.N * p.D)
    with torch.cuda.stream(stream):   # memory of the stream that uses it
        dop, dqp, dkp, dvp = (torch.empty_like(rb.qp) for _ in range(4))
    sol_gather_rows(_with_strides(p, d_o) if rows else p, rb.perm, d_o, dop, stream)
    sol_attn_bwd(rb.hm, rb.qp, rb.kp, rb.vp, rb.buf.ws, rb.buf.row_ptr, rb.buf.col_idx, rb.buf.o, rb.buf.lse, dop, dqp,
                 dkp, dvp, g.ws, hm, stream)
    to = make_params(p.B, p.N, p.H, p.D, prefix_len=p.prefix_len, out_strides=g.strides)
    for src, dst in ((dqp, g.dq), (dkp, g.dk), (dvp, g.dv)):
        sol_scatter_rows(to, rb.perm, src, dst, stream)
    return g


def _like_output(d_o: torch.Tensor) -> torch.Tensor:
    """An incoming gradient as the kernels read it: bf16, contiguous, 16-byte aligned."""
    return _dense(d_o.to(torch.bfloat16))


def _check_saved(p: sol_params, rows, others, device):
    """Saved tensors as their hooks (offloading, recomputation) give them back: at any address and with any
    strides, but nothing of another kind.  rows are [B, N, H, D] bf16, others (tensor, dtype, elements)."""
    shape = (p.B, p.N, p.H, p.D)
    for t in rows:
        if t.dtype is not torch.bfloat16 or t.shape != shape or t.device != device:
            raise ValueError(f"a saved tensor came back as {t.dtype} {tuple(t.shape)} on {t.device}, "
                             f"not bf16 {shape} on {device}")
    for t, dtype, n in others:
        if t is not None and (t.dtype is not dtype or t.numel() != n or t.device != device):
            raise ValueError(f"a saved tensor came back as {t.numel()} {t.dtype} on {t.device}, not {n} {dtype} on {device}")


def _dense(t: torch.Tensor, align: int = 16) -> torch.Tensor:
    """The tensor contiguous and at an aligned address: itself, or a copy."""
    t = t.contiguous()
    return t if t.data_ptr() % align == 0 else t.clone()


def _laid_out(p: sol_params, tensors):
    """The tensors with one set of strides that the kernels take, as they are or as dense copies, and p for
    these strides."""
    st = tensors[0].stride()
    if st[3] != 1 or (st[0] | st[1] | st[2]) & 7 or any(t.stride() != st or t.data_ptr() & 15 for t in tensors):
        tensors = [t.clone(memory_format=torch.contiguous_format) for t in tensors]
        st = tensors[0].stride()
    if st[:3] != (p.in_stride_b, p.in_stride_n, p.in_stride_h):
        p = _with_strides(p, tensors[0])
    return p, tensors


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, p):
        with torch.cuda.device(q.device):
            buf = alloc_buffers(p, q.device, with_lse=True)
            forward(p, q, k, v, buf)
        ctx.p, ctx.sizes = p, (buf.ws.numel(), buf.row_ptr.numel(), buf.col_idx.numel())
        ctx.save_for_backward(q, k, v, buf.ws, buf.row_ptr, buf.col_idx, buf.o, buf.lse)
        return buf.o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_o):
        q, k, v, ws, row_ptr, col_idx, o, lse = ctx.saved_tensors
        device, n_ws, n_rows, n_cols = d_o.device, *ctx.sizes
        _check_saved(ctx.p, (q, k, v, o), ((ws, torch.uint8, n_ws), (row_ptr, torch.int32, n_rows), (col_idx, torch.int32, n_cols),
                                           (lse, torch.float32, ctx.p.B * ctx.p.H * ctx.p.N)), device)
        with torch.cuda.device(device):
            p, (q, k, v) = _laid_out(ctx.p, (q, k, v))
            g = alloc_grads(p, device)
            sol_attn_bwd(p, q, k, v, _dense(ws, 256), _dense(row_ptr), _dense(col_idx), _dense(o), _dense(lse),
                         _like_output(d_o), g.dq, g.dk, g.dv, g.ws, g.strides)
        return g.dq, g.dk, g.dv, None


def _check_bthd(tensors, what: str):
    for t in tensors:
        if (t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 4 or t.stride(3) != 1
                or t.shape != tensors[0].shape or t.stride() != tensors[0].stride() or t.device != tensors[0].device):
            raise ValueError(f"{what} must be bf16 CUDA tensors [B, N, H, D] on one device with identical shapes and "
                             "strides and contiguous head dim")


def differentiable_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, tau: float = 1.0, prefix_len: int = 0,
                             log_mass_bias: int = 0, scale: float = 0.0, topk_ratio: Optional[float] = None,
                             compressed: bool = False) -> torch.Tensor:
    """``attention`` for autograd: returns o [B, N, H, D], whose backward runs sol_attn_bwd on the
    forward's lists.  The workspace and lists of the call are kept until the backward pass.

    A step with its backward pass can be captured into a graph.  Its leaves must then be new in the
    capture (``q.detach().requires_grad_()``) if an earlier eager graph of them is alive: their
    gradients' accumulation belongs to that graph's stream, which a capture may not wait on."""
    _check_bthd((q, k, v), "q, k, v")
    B, N, H, D = q.shape
    p = make_params(B, N, H, D, tau, prefix_len, log_mass_bias, scale, in_strides=q.stride()[:3],
                    topk_ratio=topk_ratio, compressed=compressed)
    return _Attention.apply(q, k, v, p)


class _QKNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, eps, interleaved):
        B, N, H, D = q.shape
        ctx.p = make_params(B, N, H, D, in_strides=q.stride()[:3])
        nr = make_norm_rope(q_weight, k_weight, cos, sin, eps, interleaved=interleaved)
        ctx.nr, ctx.n_table = sol_norm_rope.from_buffer_copy(nr), 0 if cos is None else cos.numel()   # (not the tensors)
        with torch.cuda.device(q.device):
            qo, ko = (torch.empty((B, N, H, D), dtype=q.dtype, device=q.device) for _ in range(2))
            sol_qk_norm_rope(ctx.p, nr, q, k, qo, ko)
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin)
        return qo, ko

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dqo, dko):
        q, k, *w, cos, sin = ctx.saved_tensors
        device, wdtype = dqo.device, torch.bfloat16 if ctx.nr.weight_type else torch.float32
        _check_saved(ctx.p, (q, k), ((w[0], wdtype, ctx.p.D), (w[1], wdtype, ctx.p.D), (cos, torch.float32, ctx.n_table),
                                     (sin, torch.float32, ctx.n_table)), device)
        with torch.cuda.device(device):
            p, (q, k) = _laid_out(ctx.p, (q, k))
            if cos is not None and (cos.stride() != sin.stride() or cos.stride(-1) != 1 or (cos.data_ptr() | sin.data_ptr()) & 15):
                cos, sin = (t.clone(memory_format=torch.contiguous_format) for t in (cos, sin))
            # addresses of now: a trainer may release the weights' storage after the forward and renew it here
            nr = sol_norm_rope.from_buffer_copy(ctx.nr)
            w = [None if t is None else _dense(t) for t in w]
            _place(nr, *w, cos, sin)
            dq, dk = (torch.empty((p.B, p.N, p.H, p.D), dtype=q.dtype, device=device) for _ in range(2))
            dw = [torch.empty(p.D, device=device) if t is not None and ctx.needs_input_grad[2 + i] else None
                  for i, t in enumerate(w)]
            ws = torch.empty(max(1, sol_qk_norm_rope_bwd_workspace_bytes(p)), dtype=torch.uint8, device=device)
            sol_qk_norm_rope_bwd(p, nr, q, k, _like_output(dqo), _like_output(dko), dq, dk, *dw, ws,
                                 grad_strides=(p.N * p.H * p.D, p.H * p.D, p.D))
        dw = [None if g is None else g.to(t.dtype) for g, t in zip(dw, w)]
        return dq, dk, *dw, None, None, None, None


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor],
                 cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 interleaved: bool = False):
    """RMS norm of every query and key head and the position rotation, for autograd.

    q, k are bf16 CUDA tensors [B, N, H, D] (views of the fused projection allowed); weights and
    tables as for make_norm_rope; the tables have no gradient.  Returns new contiguous (q, k).
    Captured into a graph like ``differentiable_attention``."""
    if any(t is not None and t.requires_grad for t in (cos, sin)):
        raise ValueError("the tables have no gradient: cos and sin must not require one")
    _check_bthd((q, k), "q, k")
    B, N, H, D = q.shape
    for w in (q_weight, k_weight):
        if w is not None and (w.shape != (D,) or w.device != q.device):
            raise ValueError("the weights must have the head dimension's length and q's device")
    if cos is not None and (cos.shape[-2] != N or (cos.dim() == 3 and cos.shape[0] not in (1, B))
                            or cos.device != q.device or sin.device != q.device):
        raise ValueError("the tables must cover q's positions (and batch) on its device")
    return _QKNormRope.apply(q, k, q_weight, k_weight, cos, sin, eps, interleaved)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, tau: float = 1.0, prefix_len: int = 0,
              log_mass_bias: int = 0, scale: float = 0.0, with_lse: bool = False,
              topk_ratio: Optional[float] = None, compressed: bool = False, reblock: bool = False,
              qk_int8: bool = False):
    """Convenience call on BTHD bf16 CUDA tensors (views with unit head-dim stride allowed).

    Returns (o, buffers); the buffers hold row_ptr / col_idx / lse for inspection.  With
    ``reblock`` the rows are first ordered by the adaptive partition (sol_reblock) and the
    buffers are a ReblockBuffers (its ``perm``, and the Sol buffers of the permuted rows;
    ``with_lse`` is not offered there: the LSE would be in the permuted order).
    """
    B, N, H, D = q.shape
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or not t.is_cuda or t.stride(3) != 1 or t.stride() != q.stride():
            raise ValueError("q, k, v must be bf16 CUDA tensors with identical strides and contiguous head dim")
    p = make_params(B, N, H, D, tau, prefix_len, log_mass_bias, scale,
                    in_strides=(q.stride(0), q.stride(1), q.stride(2)), topk_ratio=topk_ratio,
                    compressed=compressed, qk_int8=qk_int8)
    if reblock:
        if with_lse:
            raise ValueError("with_lse is not offered with reblock")
        rb = alloc_reblock(p, q.device)
        o = torch.empty((B, N, H, D), dtype=torch.bfloat16, device=q.device)
        forward_reblocked(p, q, k, v, o, rb)
        return o, rb
    buf = alloc_buffers(p, q.device, with_lse)
    forward(p, q, k, v, buf)
    return buf.o, buf
