"""Python binding of libslra.so (the C ABI in include/slra.h): argument marshalling only.

Every step of the forward pass runs in the library's CUDA kernels; this module only fills the
problem struct, hands device pointers (torch tensors' storage) and the current torch stream to the
C entry points, and raises on a non-zero status.  If the library cannot be loaded the calls raise:
there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass, field
from typing import NamedTuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libslra.so")

OK = 0
ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE_TIMEOUT, ERR_RANGE, \
    ERR_NO_DEVICE, ERR_SCRATCH_LIMIT = range(1, 10)
OUT_F32, OUT_BF16 = 0, 1
BRANCH_SPARSE, BRANCH_LOWRANK, BRANCH_BOTH = 1, 2, 3
DEBUG_UNSATISFIED_WAIT, DEBUG_SERIAL_BRANCHES = 1, 2
ABI_VERSION = 8
DTYPE_BF16, DTYPE_F32, DTYPE_F16 = 0, 1, 2
ACT_RELU, ACT_SILU, ACT_IDENTITY, ACT_TANH = 0, 1, 2, 3
FUSION_SUM, FUSION_GATED = 0, 1
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
QK_NORM_NONE, QK_NORM_HEAD, QK_NORM_TOKEN = 0, 1, 2
ROPE_INTERLEAVED, ROPE_HALVES = 0, 1
ROPE_PER_AXIS, ROPE_SHARED = 0, 1

# Every symbol include/slra.h declares.
EXPORTS = ("slra_abi_version", "slra_status_string", "slra_problem_init", "slra_validate", "slra_keep_count",
           "slra_projection_elems", "slra_workspace_bytes", "slra_attn_fwd", "slra_attn_fwd_ex", "slra_sparse_fwd",
           "slra_lowrank_fwd", "slra_get_device_status", "slra_bwd_workspace_bytes", "slra_attn_bwd",
           "slra_workspace_layout", "slra_host_io_bytes", "slra_host_pipeline_groups",
           "slra_attn_fwd_host",
           "slra_select_blocks", "slra_lowrank_summary", "slra_device_status", "slra_lowrank_summary_noalloc",
           "slra_noalloc_device_status", "slra_attn_fwd_train", "slra_attn_bwd_saved",
           "slra_residual_norm_init", "slra_residual_norm_fwd", "slra_residual_norm_bwd_workspace_bytes",
           "slra_residual_norm_bwd", "slra_qk_rope_init", "slra_qk_rope_fwd", "slra_qk_rope_bwd_workspace_bytes",
           "slra_qk_rope_bwd")


class SlraError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


class _Problem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("T", ctypes.c_int64), ("H", ctypes.c_int64), ("W", ctypes.c_int64),
                ("block", ctypes.c_int64), ("keep_frac", ctypes.c_double), ("rank", ctypes.c_int64),
                ("theta", ctypes.c_double), ("out_dtype", ctypes.c_int32), ("branches", ctypes.c_int32),
                ("pos_offset", ctypes.c_int64 * 3), ("rope_split", ctypes.c_int64 * 3),
                ("wait_timeout_ns", ctypes.c_uint64), ("debug_flags", ctypes.c_uint32),
                ("stage_events", ctypes.c_void_p * 7), ("activation", ctypes.c_int32),
                ("lowrank_norope", ctypes.c_int32), ("proj_separate", ctypes.c_int32),
                ("proj_per_head", ctypes.c_int32), ("fusion", ctypes.c_int32), ("gate_bias", ctypes.c_float),
                ("gate_w", ctypes.c_void_p), ("lowrank_rope_inside", ctypes.c_int32),
                ("q_strides", ctypes.c_int64 * 3), ("k_strides", ctypes.c_int64 * 3),
                ("v_strides", ctypes.c_int64 * 3), ("out_strides", ctypes.c_int64 * 3),
                ("dgate_w", ctypes.c_void_p), ("dgate_b", ctypes.c_void_p)]


class _Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("B", ctypes.c_int64), ("L", ctypes.c_int64),
                ("Hh", ctypes.c_int64), ("D", ctypes.c_int64), ("sB", ctypes.c_int64), ("sL", ctypes.c_int64),
                ("sH", ctypes.c_int64)]


class _Mat(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("D", ctypes.c_int64), ("R", ctypes.c_int64)]


_I32, _I64, _F32, _P = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p


class _ResidualNorm(ctypes.Structure):
    _fields_ = [(n, _I64) for n in ("batch", "tokens", "channels", "groups")] + \
               [(n, _I32) for n in ("norm", "post_norm", "stream_dtype", "block_dtype", "mod_dtype", "weight_dtype")] + \
               [(n, _F32) for n in ("eps", "post_eps", "residual_scale")] + \
               [(n + "_strides", _I64 * 2) for n in ("x", "y", "x_out", "h", "dx", "dy", "gate", "scale", "shift")] + \
               [(n, _P) for n in ("gate", "scale", "shift", "weight", "bias", "post_weight", "dgate", "dscale", "dshift",
                                  "dweight", "dbias", "dpost_weight")]


class _QkRope(ctypes.Structure):
    _fields_ = [(n, _I64) for n in ("batch", "tokens", "heads", "kv_heads", "head_dim", "T", "H", "W", "first_token")] + \
               [("pos_offset", _I64 * 3), ("rope_split", _I64 * 3), ("theta", ctypes.c_double)] + \
               [(n, _I32) for n in ("norm", "rotate", "pairing", "schedule", "x_dtype", "out_dtype", "weight_dtype")] + \
               [("eps", _F32)] + [(n + "_strides", _I64 * 3) for n in ("q", "k", "out_q", "out_k", "dq", "dk")] + \
               [("positions", _P), ("positions_stride", _I64)] + [(n, _P) for n in ("wq", "wk", "dwq", "dwk")]


class _Layout(ctypes.Structure):
    _fields_ = [("total_bytes", ctypes.c_size_t), ("L", ctypes.c_int64), ("nb", ctypes.c_int64),
                ("keep", ctypes.c_int64), ("nsplit", ctypes.c_int64)] + \
               [(n, ctypes.c_size_t) for n in ("status", "rope_table", "qh", "kh", "vh", "qbar", "kbar", "idx",
                                               "tie", "s_part", "z_part", "S", "z")]


_lib = None


def lib():
    """Load libslra.so (raises if it is missing: the CUDA path has no substitute)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m sparse_rank_hybrid_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.slra_abi_version.restype = ctypes.c_int
        if L.slra_abi_version() != ABI_VERSION:  # the structs below mirror this version of include/slra.h
            raise RuntimeError(f"{LIB_PATH} has ABI {L.slra_abi_version()}, this binding expects {ABI_VERSION}")
        missing = [name for name in EXPORTS if not hasattr(L, name)]
        if missing:  # functions were added without a change to what there was
            raise RuntimeError(f"{LIB_PATH} is older than this binding (no {', '.join(missing)}): build it again with "
                               "`python -m sparse_rank_hybrid_b200.build`")
        P, S = ctypes.c_void_p, ctypes.c_size_t
        PP = ctypes.POINTER(_Problem)
        L.slra_abi_version.restype = ctypes.c_int
        L.slra_status_string.restype = ctypes.c_char_p
        L.slra_status_string.argtypes = [ctypes.c_int]
        L.slra_problem_init.argtypes = [PP] + [ctypes.c_int64] * 7 + [ctypes.c_double, ctypes.c_int64]
        L.slra_validate.argtypes = [PP]
        L.slra_keep_count.restype = ctypes.c_int64
        L.slra_keep_count.argtypes = [PP]
        L.slra_projection_elems.restype = ctypes.c_int64
        L.slra_projection_elems.argtypes = [PP]
        L.slra_workspace_layout.argtypes = [PP, ctypes.POINTER(_Layout)]
        L.slra_attn_fwd_ex.argtypes = [PP, P, P, P, P, P, P, S, P]
        PT, PM, I64, C = ctypes.POINTER(_Tensor), ctypes.POINTER(_Mat), ctypes.c_int64, ctypes.c_int
        L.slra_workspace_bytes.restype = S
        L.slra_workspace_bytes.argtypes = [I64] * 7 + [ctypes.c_float, I64]
        L.slra_attn_fwd.argtypes = [PT, PT, PT, PM, C, C, C, C, ctypes.c_float, C, PT, P]
        L.slra_sparse_fwd.argtypes = [PT, PT, PT, C, C, C, C, ctypes.c_float, PT, P, S, P]
        L.slra_lowrank_fwd.argtypes = [PT, PT, PT, PM, C, C, C, C, PT, P, P, P, S, P]
        L.slra_get_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_int32)]
        L.slra_bwd_workspace_bytes.restype = S
        L.slra_bwd_workspace_bytes.argtypes = [PP]
        L.slra_attn_bwd.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, S, P]
        L.slra_attn_bwd_saved.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, S, P]
        L.slra_attn_fwd_train.argtypes = [PP, P, P, P, P, P, P, S, P]
        L.slra_host_io_bytes.restype = S
        L.slra_host_io_bytes.argtypes = [PP]
        L.slra_host_pipeline_groups.restype = ctypes.c_int64
        L.slra_host_pipeline_groups.argtypes = [PP, S, S]
        L.slra_attn_fwd_host.argtypes = [PP, P, P, P, P, P, P, S, P, S, P]
        L.slra_select_blocks.argtypes = [PP, P, P, P, P, S, P]
        L.slra_lowrank_summary.argtypes = [PP, P, P, P, P, S, P]
        L.slra_device_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_int32)]
        L.slra_lowrank_summary_noalloc.argtypes = [PP, P, P, P, P, P, P]
        L.slra_noalloc_device_status.argtypes = [P, ctypes.POINTER(ctypes.c_int32)]
        PN, PR = ctypes.POINTER(_ResidualNorm), ctypes.POINTER(_QkRope)
        L.slra_residual_norm_init.argtypes = [PN, I64, I64, I64]
        L.slra_residual_norm_fwd.argtypes = [PN, P, P, P, P, P]
        L.slra_residual_norm_bwd.argtypes = [PN, P, P, P, P, P, P, P, S, P]
        L.slra_qk_rope_init.argtypes = [PR, I64, I64, I64, I64]
        L.slra_qk_rope_fwd.argtypes = [PR, P, P, P, P, P]
        L.slra_qk_rope_bwd.argtypes = [PR, P, P, P, P, P, P, P, S, P]
        for name, arg in (("slra_residual_norm", PN), ("slra_qk_rope", PR)):
            f = getattr(L, name + "_bwd_workspace_bytes")
            f.restype, f.argtypes = S, [arg]
            for verb in ("_init", "_fwd", "_bwd"):
                getattr(L, name + verb).restype = ctypes.c_int
        for name in ("slra_problem_init", "slra_validate", "slra_workspace_layout", "slra_attn_fwd",
                     "slra_attn_fwd_ex", "slra_sparse_fwd", "slra_lowrank_fwd", "slra_get_device_status",
                     "slra_attn_bwd", "slra_attn_bwd_saved", "slra_attn_fwd_train",
                     "slra_attn_fwd_host", "slra_select_blocks", "slra_lowrank_summary", "slra_device_status",
                     "slra_lowrank_summary_noalloc", "slra_noalloc_device_status"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().slra_status_string(int(s)).decode()


def _check(s: int, where: str):
    if s != OK:
        raise SlraError(s, where)


@dataclass
class Problem:
    batch: int
    heads: int
    head_dim: int
    T: int
    H: int
    W: int
    block: int
    keep_frac: float
    rank: int
    theta: float = 1e4
    out_dtype: int = OUT_F32
    branches: int = BRANCH_BOTH
    pos_offset: tuple = (0, 0, 0)
    rope_split: tuple = (0, 0, 0)
    wait_timeout_ns: int = 2_000_000_000
    debug_flags: int = 0
    stage_events: tuple = (None,) * 7  # raw cudaEvent_t handles (ints) or None, see slra_problem
    activation: int = 0                # ACT_* map of the low-rank features
    lowrank_norope: int = 0            # 1: no RoPE in the low-rank branch
    proj_separate: int = 0             # 1: separate query / key projections Pq, Pk
    proj_per_head: int = 0             # 1: one projection (pair) per head
    fusion: int = 0                    # FUSION_SUM or FUSION_GATED
    gate_bias: float = 0.0             # bg of the gated fusion
    gate_w: object = None              # Wg of the gated fusion: CUDA fp32 tensor [head_dim] (or None)
    lowrank_rope_inside: int = 0       # 1: the low-rank RoPE before the activation
    q_strides: tuple = (0, 0, 0)       # (sB, sL, sH) element strides; all 0 = contiguous [B, L, Hh, D]
    k_strides: tuple = (0, 0, 0)
    v_strides: tuple = (0, 0, 0)
    out_strides: tuple = (0, 0, 0)
    dgate_w: object = None             # backward, gated: output CUDA fp32 tensor [head_dim] (d loss / d Wg)
    dgate_b: object = None             # backward, gated: output CUDA fp32 tensor [1] (d loss / d bg)

    @property
    def L(self) -> int:
        return self.T * self.H * self.W

    @classmethod
    def from_workload(cls, w, **kw) -> "Problem":
        return cls(w.batch, w.heads, w.head_dim, w.T, w.H, w.W, w.block, w.keep_frac, w.rank, **kw)

    def c(self) -> _Problem:
        p = _Problem()
        _check(lib().slra_problem_init(ctypes.byref(p), self.batch, self.heads, self.head_dim, self.T, self.H,
                                       self.W, self.block, float(self.keep_frac), self.rank), "slra_problem_init")
        p.theta = float(self.theta)
        p.out_dtype = int(self.out_dtype)
        p.branches = int(self.branches)
        p.pos_offset[:] = [int(x) for x in self.pos_offset]
        p.rope_split[:] = [int(x) for x in self.rope_split]
        p.wait_timeout_ns = int(self.wait_timeout_ns)
        p.debug_flags = int(self.debug_flags)
        for i, e in enumerate(self.stage_events):
            p.stage_events[i] = e
        p.activation = int(self.activation)
        p.lowrank_norope = int(self.lowrank_norope)
        p.proj_separate = int(self.proj_separate)
        p.proj_per_head = int(self.proj_per_head)
        p.fusion = int(self.fusion)
        p.gate_bias = float(self.gate_bias)
        p.lowrank_rope_inside = int(self.lowrank_rope_inside)
        for name in ("q_strides", "k_strides", "v_strides", "out_strides"):
            getattr(p, name)[:] = [int(x) for x in getattr(self, name)]
        if self.gate_w is not None:
            t = self.gate_w
            torch = _torch()
            if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != (self.head_dim,):
                raise ValueError(f"gate_w: expected a contiguous CUDA fp32 tensor of shape ({self.head_dim},)")
            p.gate_w = int(t.data_ptr())
        for name, n in (("dgate_w", self.head_dim), ("dgate_b", 1)):
            t = getattr(self, name)
            if t is not None:
                torch = _torch()
                if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() or t.numel() != n:
                    raise ValueError(f"{name}: expected a contiguous CUDA fp32 tensor of {n} elements")
                setattr(p, name, int(t.data_ptr()))
        return p

    @property
    def projection_shape(self) -> tuple:
        """Shape of the projection argument A: [D, rank] by default, else
        [1 + proj_separate, proj_per_head ? heads : 1, D, rank] (query projections first)."""
        if not self.proj_separate and not self.proj_per_head:
            return (self.head_dim, self.rank)
        return (1 + int(self.proj_separate), self.heads if self.proj_per_head else 1, self.head_dim, self.rank)


@dataclass
class Layout:
    total_bytes: int
    L: int
    nb: int
    keep: int
    nsplit: int
    offsets: dict = field(default_factory=dict)


def validate(prob: Problem) -> int:
    return int(lib().slra_validate(ctypes.byref(prob.c())))


def keep_count(prob: Problem) -> int:
    return int(lib().slra_keep_count(ctypes.byref(prob.c())))


def projection_elems(prob: Problem) -> int:
    return int(lib().slra_projection_elems(ctypes.byref(prob.c())))


def layout(prob: Problem) -> Layout:
    lay = _Layout()
    _check(lib().slra_workspace_layout(ctypes.byref(prob.c()), ctypes.byref(lay)), "slra_workspace_layout")
    offs = {n: int(getattr(lay, n)) for n, _ in _Layout._fields_[5:]}
    return Layout(int(lay.total_bytes), int(lay.L), int(lay.nb), int(lay.keep), int(lay.nsplit), offs)


# ------------------------------------------------------------------------------- torch helpers
@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


def _ptr(t) -> int:
    return int(t.data_ptr())


def _stream_handle(stream) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def alloc_workspace(prob: Problem, device="cuda"):
    torch = _torch()
    return torch.empty(layout(prob).total_bytes, dtype=torch.uint8, device=device)


def _check_bf16(name, t, shape):
    torch = _torch()
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected contiguous CUDA bf16 tensor of shape {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _row_strides(name, t, shape, dtype):
    """(sB, sL, sH) element strides of a [B, L, Hh, D] CUDA tensor whose last dimension is contiguous;
    (0, 0, 0) when the whole tensor is contiguous."""
    if t.dtype != dtype or not t.is_cuda or tuple(t.shape) != tuple(shape) or t.stride(3) != 1:
        raise ValueError(f"{name}: expected a CUDA {dtype} tensor of shape {tuple(shape)} with a contiguous last "
                         f"dimension, got {t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
    return (0, 0, 0) if t.is_contiguous() else (t.stride(0), t.stride(1), t.stride(2))


def attn_fwd(prob: Problem, q, k, v, A, out=None, workspace=None, stream=None, alloc_workspace_in_library=False):
    """Full forward pass through slra_attn_fwd_ex.  q, k, v: CUDA bf16 [B, L, Hh, D] with a contiguous
    last dimension (any other strides, e.g. views of a fused QKV tensor); A: CUDA bf16 of
    prob.projection_shape.  Returns (out, workspace); out is fp32 or bf16 [B, L, Hh, D] as
    prob.out_dtype (a given out may be strided too).  alloc_workspace_in_library=True passes a NULL
    workspace (the library allocates it on the stream) and returns None for it."""
    import dataclasses
    torch = _torch()
    shp = (prob.batch, prob.L, prob.heads, prob.head_dim)
    odt = torch.float32 if prob.out_dtype == OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty(shp, dtype=odt, device=q.device)
    strides = {f"{n}_strides": _row_strides(n, t, shp, dt) for n, t, dt in
               (("q", q, torch.bfloat16), ("k", k, torch.bfloat16), ("v", v, torch.bfloat16), ("out", out, odt))}
    if prob.branches & BRANCH_LOWRANK or A is not None:
        _check_bf16("A", A, prob.projection_shape)
    p = dataclasses.replace(prob, **strides)
    if workspace is None and not alloc_workspace_in_library:
        workspace = alloc_workspace(p, q.device)
    ws_ptr, ws_n = (0, 0) if workspace is None else (_ptr(workspace), workspace.numel())
    _check(lib().slra_attn_fwd_ex(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), 0 if A is None else _ptr(A),
                                  _ptr(out), ws_ptr or None, ws_n, _stream_handle(stream)), "slra_attn_fwd_ex")
    return out, workspace


def _tensor(t, dtype_code) -> _Tensor:
    """Descriptor of a [B, L, Hh, D] CUDA tensor (strides in elements; the last dimension contiguous)."""
    if t.dim() != 4 or t.stride(3) != 1 or not t.is_cuda:
        raise ValueError("expected a CUDA [B, L, Hh, D] tensor with a contiguous last dimension")
    return _Tensor(_ptr(t), dtype_code, *t.shape, t.stride(0), t.stride(1), t.stride(2))


def _dtype_code(t) -> int:
    torch = _torch()
    return {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}[t.dtype]


def workspace_bytes(batch, heads, head_dim, T, H, W, block, keep_frac, rank) -> int:
    return int(lib().slra_workspace_bytes(batch, heads, head_dim, T, H, W, block, float(keep_frac), rank))


def attn_fwd_tensors(q, k, v, A, T, H, W, block, keep_frac, rank, out, stream=None):
    """slra_attn_fwd: the forward pass from tensor descriptors (strides taken from the tensors), the
    workspace allocated by the library on the stream."""
    a = _Mat(_ptr(A), DTYPE_BF16 if A.dtype == _torch().bfloat16 else DTYPE_F32, A.shape[0], A.shape[1])
    tq, tk, tv, to = (_tensor(t, _dtype_code(t)) for t in (q, k, v, out))
    _check(lib().slra_attn_fwd(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv), ctypes.byref(a), T, H, W,
                               block, float(keep_frac), rank, ctypes.byref(to), _stream_handle(stream)),
           "slra_attn_fwd")
    return out


def sparse_fwd(q, k, v, T, H, W, block, keep_frac, out, workspace=None, stream=None):
    """slra_sparse_fwd: the sparse branch alone into out (workspace None = allocated by the library)."""
    tq, tk, tv, to = (_tensor(t, _dtype_code(t)) for t in (q, k, v, out))
    ws_ptr, ws_n = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel())
    _check(lib().slra_sparse_fwd(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv), T, H, W, block,
                                 float(keep_frac), ctypes.byref(to), ws_ptr, ws_n, _stream_handle(stream)),
           "slra_sparse_fwd")
    return out


def lowrank_fwd(q, k, v, A, T, H, W, rank, out, S=None, z=None, workspace=None, stream=None):
    """slra_lowrank_fwd: the low-rank branch alone into out; S, z (fp32 CUDA) receive the summary."""
    a = _Mat(_ptr(A), DTYPE_BF16, A.shape[0], A.shape[1])
    tq, tk, tv, to = (_tensor(t, _dtype_code(t)) for t in (q, k, v, out))
    ws_ptr, ws_n = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel())
    _check(lib().slra_lowrank_fwd(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv), ctypes.byref(a), T, H, W,
                                  rank, ctypes.byref(to), None if S is None else _ptr(S),
                                  None if z is None else _ptr(z), ws_ptr, ws_n, _stream_handle(stream)),
           "slra_lowrank_fwd")
    return out


def bwd_workspace_bytes(prob: Problem) -> int:
    return int(lib().slra_bwd_workspace_bytes(ctypes.byref(prob.c())))


def attn_fwd_train(prob: Problem, q, k, v, A, out=None, workspace=None, stream=None):
    """Forward pass for training (slra_attn_fwd_train): out as attn_fwd gives it, and the workspace
    (backward-sized, allocated when None) keeps what attn_bwd_saved needs.  Returns (out, workspace)."""
    import dataclasses
    torch = _torch()
    shp = (prob.batch, prob.L, prob.heads, prob.head_dim)
    strides = {f"{n}_strides": _row_strides(n, t, shp, torch.bfloat16) for n, t in (("q", q), ("k", k), ("v", v))}
    p = dataclasses.replace(prob, **strides)
    if A is not None:
        _check_bf16("A", A, prob.projection_shape)
    if out is None:
        out = torch.empty(shp, dtype=torch.float32 if prob.out_dtype == OUT_F32 else torch.bfloat16, device=q.device)
    if workspace is None:
        n = bwd_workspace_bytes(p)
        if n == 0:
            raise SlraError(ERR_UNSUPPORTED, "slra_bwd_workspace_bytes")
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    _check(lib().slra_attn_fwd_train(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), None if A is None else _ptr(A),
                                     _ptr(out), _ptr(workspace), workspace.numel(), _stream_handle(stream)),
           "slra_attn_fwd_train")
    return out, workspace


def attn_bwd_saved(prob: Problem, q, k, v, A, dout, workspace, grads=None, stream=None):
    """Backward pass from attn_fwd_train's workspace (slra_attn_bwd_saved): as attn_bwd, without the
    recompute.  Returns (dq, dk, dv, dA, workspace)."""
    return attn_bwd(prob, q, k, v, A, dout, grads=grads, workspace=workspace, stream=stream, _saved=True)


def attn_bwd(prob: Problem, q, k, v, A, dout, grads=None, workspace=None, stream=None, _saved=False):
    """Backward pass (slra_attn_bwd): gradients of sum(dout * out) for q, k, v (fp32 [B, L, Hh, D]) and the
    projection(s) A (fp32, prob.projection_shape).  dout: contiguous CUDA fp32 [B, L, Hh, D].  q, k, v may be
    strided views.  With the gated fusion, prob.dgate_w and prob.dgate_b receive the gate parameters'
    gradients.  Returns (dq, dk, dv, dA, workspace)."""
    import dataclasses
    torch = _torch()
    shp = (prob.batch, prob.L, prob.heads, prob.head_dim)
    strides = {f"{n}_strides": _row_strides(n, t, shp, torch.bfloat16) for n, t in (("q", q), ("k", k), ("v", v))}
    p = dataclasses.replace(prob, **strides)
    if dout.dtype != torch.float32 or not dout.is_cuda or not dout.is_contiguous() or tuple(dout.shape) != shp:
        raise ValueError(f"dout: expected a contiguous CUDA fp32 tensor of shape {shp}")
    if A is not None:
        _check_bf16("A", A, prob.projection_shape)
    if grads is None:
        grads = tuple(torch.empty(shp, dtype=torch.float32, device=q.device) for _ in range(3)) + \
            (torch.empty(prob.projection_shape, dtype=torch.float32, device=q.device),)
    dq, dk, dv, dA = grads
    if workspace is None:
        n = bwd_workspace_bytes(p)
        if n == 0:
            raise SlraError(ERR_UNSUPPORTED, "slra_bwd_workspace_bytes")
        workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    fn = "slra_attn_bwd_saved" if _saved else "slra_attn_bwd"
    _check(getattr(lib(), fn)(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), None if A is None else _ptr(A),
                              _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dA), _ptr(workspace),
                              workspace.numel(), _stream_handle(stream)), fn)
    return dq, dk, dv, dA, workspace


def get_device_status(stream=None) -> int:
    """Read and clear the device status of the calls whose workspace the library allocated."""
    st = ctypes.c_int32(-1)
    _check(lib().slra_get_device_status(_stream_handle(stream), ctypes.byref(st)), "slra_get_device_status")
    return int(st.value)


def host_io_bytes(prob: Problem) -> int:
    return int(lib().slra_host_io_bytes(ctypes.byref(prob.c())))


def host_pipeline_groups(prob: Problem, io_bytes: int, workspace_bytes: int) -> int:
    """Head groups the host entry point pipelines for these buffer sizes (1: none)."""
    return int(lib().slra_host_pipeline_groups(ctypes.byref(prob.c()), io_bytes, workspace_bytes))


def attn_fwd_host(prob: Problem, q_host, k_host, v_host, A_host, out_host, io, workspace, stream=None):
    """Forward pass on host buffers (pinned CPU tensors): copies in, computes, copies out, synchronizes."""
    if A_host.numel() != projection_elems(prob):
        raise ValueError(f"A_host: expected {projection_elems(prob)} elements, got {A_host.numel()}")
    _check(lib().slra_attn_fwd_host(ctypes.byref(prob.c()), _ptr(q_host), _ptr(k_host), _ptr(v_host),
                                    _ptr(A_host), _ptr(out_host), _ptr(io), io.numel(), _ptr(workspace),
                                    workspace.numel(), _stream_handle(stream)), "slra_attn_fwd_host")
    return out_host


def select_blocks(prob: Problem, q, k, v, workspace=None, stream=None):
    if workspace is None:
        workspace = alloc_workspace(prob, q.device)
    _check(lib().slra_select_blocks(ctypes.byref(prob.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(workspace),
                                    workspace.numel(), _stream_handle(stream)), "slra_select_blocks")
    return workspace


def lowrank_summary(prob: Problem, k, v, A, workspace=None, stream=None):
    _check_bf16("A", A, prob.projection_shape)
    if workspace is None:
        workspace = alloc_workspace(prob, k.device)
    _check(lib().slra_lowrank_summary(ctypes.byref(prob.c()), _ptr(k), _ptr(v), _ptr(A), _ptr(workspace),
                                      workspace.numel(), _stream_handle(stream)), "slra_lowrank_summary")
    return workspace


def lowrank_summary_noalloc(prob: Problem, k, v, A, S, z, stream=None):
    """Low-rank summary into caller tensors S [B*Hh, rank, D] and z [B*Hh, rank] (fp32, CUDA) without
    any allocation: the library's fixed scratch array is used instead of a workspace."""
    _check_bf16("A", A, prob.projection_shape)
    _check(lib().slra_lowrank_summary_noalloc(ctypes.byref(prob.c()), _ptr(k), _ptr(v), _ptr(A), _ptr(S), _ptr(z),
                                              _stream_handle(stream)), "slra_lowrank_summary_noalloc")
    return S, z


def noalloc_device_status(stream=None) -> int:
    """Read and clear the device status of the no-allocation summary on the current device."""
    st = ctypes.c_int32(-1)
    _check(lib().slra_noalloc_device_status(_stream_handle(stream), ctypes.byref(st)), "slra_noalloc_device_status")
    return int(st.value)


def device_status(workspace, stream=None) -> int:
    st = ctypes.c_int32(-1)
    _check(lib().slra_device_status(_ptr(workspace), _stream_handle(stream), ctypes.byref(st)),
           "slra_device_status")
    return int(st.value)


def ws_view(prob: Problem, workspace, name: str):
    """A typed view of one intermediate inside a workspace (see slra_ws_layout)."""
    torch = _torch()
    lay = layout(prob)
    BH, nb, D, R, k = prob.batch * prob.heads, lay.nb, prob.head_dim, prob.rank, lay.keep
    spec = {"qh": (torch.float16, (BH, nb * prob.block, D)), "kh": (torch.float16, (BH, nb * prob.block, D)),
            "vh": (torch.float16, (BH, nb * prob.block, D)), "qbar": (torch.float64, (BH, nb, D)),
            "kbar": (torch.float64, (BH, nb, D)), "idx": (torch.int32, (BH, nb, k)),
            "tie": (torch.uint8, (BH, nb)), "S": (torch.float32, (BH, R, D)), "z": (torch.float32, (BH, R))}
    dt, shape = spec[name]
    off = lay.offsets[name]
    n = 1
    for s in shape:
        n *= s
    nbytes = n * torch.empty(0, dtype=dt).element_size()
    return workspace[off:off + nbytes].view(dt).view(shape)


# ------------------------------------------------------------- operators around the attention
# Single tokens make short calls, so what these functions do on the host is kept small: problems are
# tuples, their C structs are made once, and only what a call changes is set.
@functools.lru_cache(maxsize=None)
def _codes():
    torch = _torch()
    return {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32, torch.float16: DTYPE_F16}


@functools.lru_cache(maxsize=None)
def _types():
    return {code: t for t, code in _codes().items()}


def _code(t) -> int:
    code = _codes().get(t.dtype)
    if code is None:
        raise ValueError(f"expected bf16, fp16 or fp32, got {t.dtype}")
    return code


@functools.lru_cache(maxsize=None)
def _current_stream():
    """device index -> handle of its current stream; the direct query where this torch has one (a fraction of
    the time that making a Stream object takes)."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw if raw is not None else lambda index: torch.cuda.current_stream(index).cuda_stream


def _elsewhere(t, stream):
    """None where t's device is current and `stream` is None; else what makes the device current and the
    stream (None: the device's current one) with it, so that what is allocated inside belongs to it."""
    device = t.device
    if device.type != "cuda":
        raise ValueError(f"expected CUDA tensors, got {device}")
    torch = _torch()
    if stream is None:
        if device.index == torch.cuda.current_device():
            return None
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(stream)


def _rows(c, name, t, shape, dtype, device, field):
    """Checks a tensor (type, where one is given, shape, device, contiguous last dimension), sets its strides
    in the struct's `field` unless it is contiguous, and gives its address."""
    if t.shape != shape or (dtype is not None and t.dtype is not dtype) or t.device != device:
        raise ValueError(f"{name}: expected a {'' if dtype is None else str(dtype) + ' '}tensor of shape {tuple(shape)} on "
                         f"{device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    if not t.is_contiguous():
        st = t.stride()
        # the struct's zeros mean contiguous: an expanded dimension must not reach it
        if (st[-1] != 1 and shape[-1] != 1) or any(s == 0 and n > 1 for s, n in zip(st, shape)):
            raise ValueError(f"{name}: expected a contiguous last dimension and no expanded one, got strides {st}")
        # a dimension of one element gets any valid stride
        getattr(c, field)[:] = [s if n > 1 else 8 for s, n in zip(st[:-1], shape)]
    return t.data_ptr()


def _like(t, shape, dtype):
    """A new contiguous tensor of this shape on t's device, by the quickest of torch's ways."""
    torch = _torch()
    if t.is_contiguous():
        return torch.empty_like(t) if t.dtype is dtype else torch.empty_like(t, dtype=dtype)
    strides, n = [], 1
    for k in reversed(shape):
        strides.append(n)
        n *= k
    return torch.empty_strided(shape, strides[::-1], dtype=dtype, device=t.device)


def _vector(name, t, n, dtype, device):
    if t.shape != (n,) or (dtype is not None and t.dtype is not dtype) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {'' if dtype is None else str(dtype) + ' '}tensor of {n} elements "
                         f"on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _sums_workspace(call, c, workspace, device):
    """The caller's workspace, or one of the size the call needs (a problem that is refused gets a token
    one: the call itself then says why)."""
    torch = _torch()
    if workspace is None:
        return torch.empty_strided((max(call(c), 256),), (1,), dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous() or workspace.dtype is not torch.uint8:
        raise ValueError(f"workspace: expected a contiguous uint8 tensor on {device}")
    return workspace


class ResidualNorm(NamedTuple):
    """Sizes and options of slra_residual_norm (see include/slra.h): x, y, x_out and h are
    [batch, tokens, channels], the modulation vectors [batch, groups, channels].  Types and strides are
    taken from the tensors of each call."""
    batch: int
    tokens: int
    channels: int
    groups: int = 1             # modulation rows of a sample: 1, the number of frames, or tokens
    norm: int = NORM_LAYER      # of h; NORM_NONE: x_out alone
    post_norm: int = NORM_NONE  # of y: NORM_NONE or NORM_RMS
    eps: float = 1e-6
    post_eps: float = 1e-6
    residual_scale: float = 1.0


class ResidualNormGrads(NamedTuple):
    dx: object
    dy: object
    dgate: object
    dscale: object
    dshift: object
    dweight: object
    dbias: object
    dpost_weight: object
    workspace: object


@functools.lru_cache(maxsize=256)
def _residual_norm_template(prob: ResidualNorm):
    c = _ResidualNorm()
    _check(lib().slra_residual_norm_init(ctypes.byref(c), prob.batch, prob.tokens, prob.channels),
           "slra_residual_norm_init")
    c.groups, c.norm, c.post_norm = prob.groups, prob.norm, prob.post_norm
    c.eps, c.post_eps, c.residual_scale = prob.eps, prob.post_eps, prob.residual_scale
    return bytes(c)


def _residual_norm_problem(prob, x, y, h, gate, scale, shift, weight, bias, post_weight):
    """The struct filled from the tensors, the block type (that of y, h or dh, else x's), and the addresses
    of x and y."""
    c = _ResidualNorm.from_buffer_copy(_residual_norm_template(prob))
    device = x.device
    batch, tokens, channels, groups = prob[:4]
    row = (batch, tokens, channels)
    c.stream_dtype = _code(x)
    px = _rows(c, "x", x, row, None, device, "x_strides")
    block = y if y is not None else h if h is not None else x
    c.block_dtype = _code(block)
    py = None if y is None else _rows(c, "y", y, row, None, device, "y_strides")
    mods, dtype = (batch, groups, channels), None
    for name, t in (("gate", gate), ("scale", scale), ("shift", shift)):
        if t is not None:
            if dtype is None:
                dtype = t.dtype
                c.mod_dtype = _code(t)
            st = None if t.is_contiguous() else t.stride()
            if t.shape != mods or t.dtype is not dtype or t.device != device or (st and channels > 1 and st[2] != 1):
                raise ValueError(f"{name}: expected {mods} on {device} with a contiguous last dimension, of one type with "
                                 f"the other modulation vectors, got {t.dtype} {tuple(t.shape)} strides {t.stride()} on "
                                 f"{t.device}")
            setattr(c, name, t.data_ptr())
            if st:
                getattr(c, name + "_strides")[:] = (st[0] if batch > 1 else 0, st[1] if groups > 1 else 0)
    if weight is not None or bias is not None or post_weight is not None:
        dtype = None
        for name, t in (("weight", weight), ("bias", bias), ("post_weight", post_weight)):
            if t is not None:
                setattr(c, name, _vector(name, t, channels, dtype, device))
                if dtype is None:
                    dtype = t.dtype
                    c.weight_dtype = _code(t)
    return c, block.dtype, px, py


def residual_norm_fwd(prob: ResidualNorm, x, y=None, gate=None, scale=None, shift=None, weight=None, bias=None,
                      post_weight=None, x_out=None, h=None, h_dtype=None, stream=None):
    """x_out = residual_scale x + gate post(y) and h = norm(x_out) (1 + scale) + shift in one pass
    (slra_residual_norm_fwd).  x: the residual stream, bf16, fp16 or fp32 [batch, tokens, channels]; y: the
    block's output (None: the norm before the first block); gate, scale, shift: [batch, groups, channels]
    (expanded views broadcast); weight, bias, post_weight: [channels].  h has y's type; without y
    it gets h_dtype (a torch dtype, default x's).  Rows may be strided, x_out may be x and h may be y.
    Returns (x_out, h): x itself where there is no y, None for h with NORM_NONE."""
    row, device = prob[:3], x.device
    if h_dtype is not None:
        block = y if y is not None else h
        if h_dtype not in _codes() or (block is not None and block.dtype is not h_dtype):
            raise ValueError(f"h_dtype: expected {'bf16, fp16 or fp32' if block is None else block.dtype}, got {h_dtype}")
    other = _elsewhere(x, stream)
    if other is not None:
        with other:
            return residual_norm_fwd(prob, x, y, gate, scale, shift, weight, bias, post_weight, x_out, h, h_dtype)
    handle = _current_stream()(x.device.index)
    c, block, px, py = _residual_norm_problem(prob, x, y, h, gate, scale, shift, weight, bias, post_weight)
    if h_dtype is not None and y is None and h is None:
        block = h_dtype
        c.block_dtype = _codes()[h_dtype]
    po = ph = None
    if y is None:
        if x_out is not None:
            raise ValueError("x_out: there is no y to add")
    elif x_out is None:
        x_out = _like(x, row, x.dtype)
        po = x_out.data_ptr()
    else:
        po = _rows(c, "x_out", x_out, row, x.dtype, device, "x_out_strides")
    if prob.norm == NORM_NONE:
        if h is not None:
            raise ValueError("h: the problem has no norm")
    elif h is None:
        h = _like(x if y is None else y, row, block)
        ph = h.data_ptr()
    else:
        ph = _rows(c, "h", h, row, block, device, "h_strides")
    _check(lib().slra_residual_norm_fwd(c, px, py, po, ph, handle), "slra_residual_norm_fwd")
    return (x if y is None else x_out), h


def residual_norm_bwd(prob: ResidualNorm, x, y=None, dh=None, dx_out=None, gate=None, scale=None, shift=None,
                      weight=None, bias=None, post_weight=None, dx=None, dy=None, workspace=None, stream=None):
    """Gradients of sum(dx_out x_out) + sum(dh h) (slra_residual_norm_bwd) from the forward's inputs; dh has
    the block's type, dx_out (the gradient of the stream behind, None: zero) x's.  Every vector that is
    given gets its gradient, in fp32: dgate, dscale, dshift [batch, groups, channels], dweight, dbias,
    dpost_weight [channels].  dx may be dx_out and dy may be dh.  workspace: a uint8 tensor to reuse (None:
    allocated; it comes back in the result).  Returns ResidualNormGrads, None where there is nothing."""
    row, device = prob[:3], x.device
    L = lib()
    other = _elsewhere(x, stream)
    if other is not None:
        with other:
            return residual_norm_bwd(prob, x, y, dh, dx_out, gate, scale, shift, weight, bias, post_weight, dx, dy, workspace)
    handle = _current_stream()(x.device.index)
    c, block, px, py = _residual_norm_problem(prob, x, y, dh, gate, scale, shift, weight, bias, post_weight)
    pdh = None if dh is None else _rows(c, "dh", dh, row, block, device, "h_strides")
    pdo = None if dx_out is None else _rows(c, "dx_out", dx_out, row, x.dtype, device, "x_out_strides")
    if dx is None:
        dx = _like(x, row, x.dtype)
    pdx, pdy = _rows(c, "dx", dx, row, x.dtype, device, "dx_strides"), None
    if y is not None:
        if dy is None:
            dy = _like(y, row, block)
        pdy = _rows(c, "dy", dy, row, block, device, "dy_strides")
    elif dy is not None:
        raise ValueError("dy: there is no y")
    f32, mods, out = _torch().float32, (prob.batch, prob.groups, prob.channels), []
    for name, t in (("dgate", gate), ("dscale", scale), ("dshift", shift), ("dweight", weight), ("dbias", bias),
                    ("dpost_weight", post_weight)):
        g = None
        if t is not None:
            g = _like(t, mods if t.dim() == 3 else mods[2:], f32)
            setattr(c, name, g.data_ptr())
        out.append(g)
    workspace = _sums_workspace(L.slra_residual_norm_bwd_workspace_bytes, c, workspace, device)
    _check(L.slra_residual_norm_bwd(c, px, py, pdo, pdh, pdx, pdy, workspace.data_ptr(), workspace.numel(), handle),
           "slra_residual_norm_bwd")
    return ResidualNormGrads(dx, dy, *out, workspace)


class QkRope(NamedTuple):
    """Sizes and options of slra_qk_rope (see include/slra.h): q is [batch, tokens, heads, head_dim], k the
    same with kv_heads.  Types and strides are taken from the tensors of each call."""
    batch: int
    tokens: int
    heads: int
    head_dim: int
    kv_heads: int = 0                # 0: no k
    grid: tuple = None               # (T, H, W) of the positions (tuples or lists); None: (1, 1, tokens)
    first_token: int = 0             # the grid place of token 0
    pos_offset: tuple = (0, 0, 0)
    rope_split: tuple = (0, 0, 0)    # pairs per axis; all 0: the default split
    theta: float = 1e4
    norm: int = QK_NORM_NONE
    eps: float = 1e-6
    rotate: bool = True
    pairing: int = ROPE_INTERLEAVED
    schedule: int = ROPE_PER_AXIS
    out_dtype: int = None            # of the forward's outputs, DTYPE_*; None: q's


class QkRopeGrads(NamedTuple):
    dq: object
    dk: object
    dwq: object
    dwk: object
    workspace: object


@functools.lru_cache(maxsize=256)
def _qk_rope_template(prob: QkRope):
    c = _QkRope()
    _check(lib().slra_qk_rope_init(ctypes.byref(c), prob.batch, prob.tokens, prob.heads, prob.head_dim),
           "slra_qk_rope_init")
    c.kv_heads, c.first_token, c.theta = prob.kv_heads, prob.first_token, prob.theta
    if prob.grid is not None:
        c.T, c.H, c.W = prob.grid
    c.pos_offset[:] = prob.pos_offset
    c.rope_split[:] = prob.rope_split
    c.norm, c.eps, c.rotate, c.pairing, c.schedule = prob.norm, prob.eps, int(prob.rotate), prob.pairing, prob.schedule
    return bytes(c)


def _qk_rope_problem(prob, q, k, wq, wk, positions):
    """The struct filled from the inputs, and the addresses of q and k."""
    try:
        template = _qk_rope_template(prob)
    except TypeError:  # lists for tuples: the templates are kept by the problem
        template = _qk_rope_template(prob._replace(**{n: tuple(getattr(prob, n)) for n in ("grid", "pos_offset", "rope_split")
                                                      if getattr(prob, n) is not None}))
    c = _QkRope.from_buffer_copy(template)
    device = q.device
    batch, tokens, heads, D, kv_heads = prob[:5]
    if (k is not None) != (kv_heads > 0):
        raise ValueError(f"k: the problem has {kv_heads} key heads")
    c.x_dtype = _code(q)
    pq = _rows(c, "q", q, (batch, tokens, heads, D), None, device, "q_strides")
    pk = None if k is None else _rows(c, "k", k, (batch, tokens, kv_heads, D), q.dtype, device, "k_strides")
    token = prob.norm == QK_NORM_TOKEN
    if wq is not None:
        c.wq = _vector("wq", wq, heads * D if token else D, None, device)
        c.weight_dtype = _code(wq)
    if wk is not None:
        c.wk = _vector("wk", wk, kv_heads * D if token else D, None if wq is None else wq.dtype, device)
        c.weight_dtype = _code(wk)
    if positions is not None:
        n, st = positions.shape[0] if positions.dim() == 3 else 0, positions.stride()
        if positions.shape != (n, tokens, 3) or n not in (1, batch) or positions.dtype is not _torch().int32 or \
                positions.device != device or st[2] != 1 or (tokens > 1 and st[1] != 3):
            raise ValueError(f"positions: expected int32 [1 or {batch}, {tokens}, 3] on {device}, every sample contiguous, "
                             f"got {positions.dtype} {tuple(positions.shape)} strides {st} on {positions.device}")
        c.positions = positions.data_ptr()
        c.positions_stride = st[0] if n > 1 else 0
    return c, pq, pk


def qk_rope_fwd(prob: QkRope, q, k=None, wq=None, wk=None, positions=None, out_q=None, out_k=None, stream=None):
    """QK norm and rotary positions (slra_qk_rope_fwd): q, k bf16, fp16 or fp32 (any strides with a
    contiguous last dimension, e.g. views of a fused QKV tensor); wq, wk: the norm's weights ([head_dim], or
    [heads * head_dim] with QK_NORM_TOKEN); positions: int32 [1 or batch, tokens, 3] in place of the grid.
    out_q may be q and out_k may be k.  Returns (out_q, out_k); out_k is None without k."""
    device, code = q.device, prob.out_dtype
    if code is not None and code not in _types():
        raise ValueError(f"out_dtype: expected DTYPE_BF16, DTYPE_F32 or DTYPE_F16, got {code}")
    other = _elsewhere(q, stream)
    if other is not None:
        with other:
            return qk_rope_fwd(prob, q, k, wq, wk, positions, out_q, out_k)
    handle = _current_stream()(q.device.index)
    c, pq, pk = _qk_rope_problem(prob, q, k, wq, wk, positions)
    dtype = q.dtype if code is None else _types()[code]
    c.out_dtype = c.x_dtype if code is None else code
    shape, po_k = (prob.batch, prob.tokens, prob.heads, prob.head_dim), None
    if out_q is None:
        out_q = _like(q, shape, dtype)
    po_q = _rows(c, "out_q", out_q, shape, dtype, device, "out_q_strides")
    if k is not None:
        shape = (prob.batch, prob.tokens, prob.kv_heads, prob.head_dim)
        if out_k is None:
            out_k = _like(k, shape, dtype)
        po_k = _rows(c, "out_k", out_k, shape, dtype, device, "out_k_strides")
    elif out_k is not None:
        raise ValueError("out_k: there is no k")
    _check(lib().slra_qk_rope_fwd(c, pq, pk, po_q, po_k, handle), "slra_qk_rope_fwd")
    return out_q, out_k


def qk_rope_bwd(prob: QkRope, q, k, dout_q, dout_k=None, wq=None, wk=None, positions=None, dq=None, dk=None,
                workspace=None, stream=None):
    """Gradients of sum(dout_q out_q) + sum(dout_k out_k) (slra_qk_rope_bwd): dq, dk in q's type, and the
    weights' in fp32 where they are given.  dout_q, dout_k: q's type or fp32, any strides.  dq, dk may be
    given (e.g. views of one fused gradient, or dout_q, dout_k themselves where the types agree).
    workspace: as for residual_norm_bwd.  Returns QkRopeGrads, None where there is nothing."""
    f32, device = _torch().float32, q.device
    L = lib()
    if (dout_k is not None) != (prob.kv_heads > 0):
        raise ValueError(f"dout_k: the problem has {prob.kv_heads} key heads")
    other = _elsewhere(q, stream)
    if other is not None:
        with other:
            return qk_rope_bwd(prob, q, k, dout_q, dout_k, wq, wk, positions, dq, dk, workspace)
    handle = _current_stream()(q.device.index)
    c, pq, pk = _qk_rope_problem(prob, q, k, wq, wk, positions)
    c.out_dtype = _code(dout_q)
    shape, dwq, dwk, pgk, pdk = (prob.batch, prob.tokens, prob.heads, prob.head_dim), None, None, None, None
    pgq = _rows(c, "dout_q", dout_q, shape, None, device, "out_q_strides")
    if dq is None:
        dq = _like(q, shape, q.dtype)
    pdq = _rows(c, "dq", dq, shape, q.dtype, device, "dq_strides")
    if k is not None:
        shape = (prob.batch, prob.tokens, prob.kv_heads, prob.head_dim)
        pgk = _rows(c, "dout_k", dout_k, shape, dout_q.dtype, device, "out_k_strides")
        if dk is None:
            dk = _like(k, shape, k.dtype)
        pdk = _rows(c, "dk", dk, shape, q.dtype, device, "dk_strides")
    elif dk is not None:
        raise ValueError("dk: there is no k")
    if wq is not None:
        dwq = _like(wq, wq.shape, f32)
        c.dwq = dwq.data_ptr()
    if wk is not None:
        dwk = _like(wk, wk.shape, f32)
        c.dwk = dwk.data_ptr()
    workspace = _sums_workspace(L.slra_qk_rope_bwd_workspace_bytes, c, workspace, device)
    _check(L.slra_qk_rope_bwd(c, pq, pk, pgq, pgk, pdq, pdk, workspace.data_ptr(), workspace.numel(), handle),
           "slra_qk_rope_bwd")
    return QkRopeGrads(dq, dk, dwq, dwk, workspace)
