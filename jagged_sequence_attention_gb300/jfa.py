"""Thin Python binding of libjfa (include/jfa.h), same entry-point names.

Argument marshalling only: torch tensors are passed as raw device pointers with
the current CUDA stream; every step of the computation runs in the library's
kernels.  The library must have been built (``__graft_entry__.build()`` or
``python -m jagged_sequence_attention_gb300._build``); if it is missing or fails to
load, every call raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libjfa.so")

JFA_OK, JFA_ERR_INVALID_ARG, JFA_ERR_UNSUPPORTED, JFA_ERR_CUDA = 0, 1, 2, 3
JFA_ERR_TIMEOUT, JFA_ERR_DEVICE_BOUNDS, JFA_ERR_PLAN_MISMATCH, JFA_ERR_NO_DEVICE = 4, 5, 6, 7
JFA_ERR_SCRATCH_LIMIT = 8
JFA_STATIC_SCRATCH_BYTES = 64 << 20
JFA_SOFTMAX, JFA_GDPA_GELU_TANH, JFA_GDPA_SILU = 0, 1, 2
JFA_BF16, JFA_F32 = 0, 1
JFA_BIAS_NONE, JFA_BIAS_RELPOS32, JFA_BIAS_DENSE = 0, 1, 2
JFA_ROT_HALF, JFA_ROT_PAIRS = 0, 1
JFA_CACHE_ZERO_BYTES = 32768

MODES = {"softmax": JFA_SOFTMAX, "gelu_tanh": JFA_GDPA_GELU_TANH, "silu": JFA_GDPA_SILU}
DTYPES = {torch.bfloat16: JFA_BF16, torch.float32: JFA_F32}
ROT_KINDS = {"half": JFA_ROT_HALF, "pairs": JFA_ROT_PAIRS}

EXPORTED = ["jfa_plan_create", "jfa_plan_create_ex", "jfa_plan_destroy", "jfa_plan_info", "jfa_fwd", "jfa_bwd_workspace_size",
            "jfa_bwd", "jfa_plan_device_status", "jfa_worklist_size", "jfa_worklist_build",
            "jfa_status_string", "jfa_plan_set_timing", "jfa_plan_kernel_times", "jfa_bwd_static_scratch",
            "jfa_partition_sequences", "jfa_bwd_ex_workspace_size", "jfa_bwd_ex", "jfa_plan_create_shared_kv",
            "jfa_partition_users", "jfa_plan_set_deterministic", "jfa_plan_set_work_item",
            "jfa_cache_create", "jfa_cache_destroy", "jfa_cache_device_status", "jfa_cache_append",
            "jfa_cache_workspace_size", "jfa_cache_fwd", "jfa_cache_create_quantized", "jfa_cache_read",
            "jfa_cache_summarize", "jfa_cache_select_workspace_size", "jfa_cache_select", "jfa_cache_fwd_blocks"]


class JFAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {jfa_status_string(status)} (status {status})")


_lib = None
_calls = None  # the compiled paged-cache calls (csrc/cache_calls.cpp)


def lib():
    """Load libjfa.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libjfa.so is not built ({_LIB_PATH}); run __graft_entry__.build()")
        _lib = load_library(_LIB_PATH)
    return _lib


def _cache_calls():
    """Load the compiled paged-cache calls; raises if they have not been built."""
    global _calls
    if _calls is None:
        L = lib()
        try:
            from . import _cache_calls as m
        except ImportError as e:
            raise RuntimeError(f"the paged cache's compiled calls are not built ({e}); run __graft_entry__.build()") from None
        m.set_calls(*(ctypes.cast(f, ctypes.c_void_p).value
                      for f in (L.jfa_cache_append, L.jfa_cache_fwd, L.jfa_cache_read, L.jfa_cache_summarize,
                                L.jfa_cache_select, L.jfa_cache_fwd_blocks)))
        _calls = m
    return _calls


def load_library(path):
    """A build of the library at `path` (the main one, or a test build) with the C-ABI's
    argument and result types declared."""
    L = ctypes.CDLL(path)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    P = ctypes.POINTER
    L.jfa_plan_create.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, vp, P(vp)]
    L.jfa_plan_create_ex.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, P(vp)]
    L.jfa_plan_create_shared_kv.argtypes = [vp, i32, vp, i32, vp, i32, i32, i32, i32, i32, i32, vp, P(vp)]
    L.jfa_plan_destroy.argtypes = [vp]
    L.jfa_plan_info.argtypes = [vp, P(i64), i32]
    L.jfa_fwd.argtypes = [vp, i32, vp, vp, vp, i32, vp, f32, vp, i32, vp, vp]
    L.jfa_bwd_workspace_size.argtypes = [vp, i32]
    L.jfa_bwd_workspace_size.restype = sz
    L.jfa_bwd.argtypes = [vp, i32, vp, vp, vp, vp, i32, vp, vp, i32, vp, f32, vp, vp, vp, vp, sz, vp]
    L.jfa_bwd_ex_workspace_size.argtypes = [vp, i32, i32]
    L.jfa_bwd_ex_workspace_size.restype = sz
    L.jfa_bwd_ex.argtypes = [vp, i32, vp, vp, vp, vp, i32, vp, vp, i32, vp, f32, vp, vp, vp, vp, vp, sz, vp]
    L.jfa_bwd_static_scratch.argtypes = [vp, i32, vp, vp, vp, vp, i32, vp, vp, i32, vp, f32, vp, vp, vp, vp]
    L.jfa_plan_device_status.argtypes = [vp, vp]
    L.jfa_partition_sequences.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp]
    L.jfa_partition_users.argtypes = [vp, i32, vp, i32, vp, i32, i32, i32, i32, vp, vp]
    L.jfa_worklist_size.argtypes = [vp, vp, i32, i32, i32, i32, i32, P(i64)]
    L.jfa_worklist_build.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, vp]
    L.jfa_plan_set_timing.argtypes = [vp, i32]
    L.jfa_plan_set_deterministic.argtypes = [vp, i32]
    L.jfa_plan_set_work_item.argtypes = [vp, i32, i64, vp]
    L.jfa_plan_kernel_times.argtypes = [vp, vp, vp]
    L.jfa_cache_create.argtypes = [i32, i32, i32, i32, i64, vp, vp, P(i64), P(i64), vp, P(vp)]
    L.jfa_cache_destroy.argtypes = [vp]
    L.jfa_cache_device_status.argtypes = [vp, vp]
    L.jfa_cache_append.argtypes = [vp, i32, i64, vp, vp, vp, i32, vp, i64, vp, i64, vp, i64, i32, vp, i64, vp, i32,
                                   i64, i32, vp]
    L.jfa_cache_workspace_size.argtypes = [vp, i32]
    L.jfa_cache_workspace_size.restype = sz
    L.jfa_cache_fwd.argtypes = [vp, i32, i64, i32, vp, vp, vp, i32, vp, i64, i32, i32, i32, i32, vp, f32, vp, i32, vp,
                                vp, sz, vp]
    L.jfa_cache_create_quantized.argtypes = [i32, i32, i32, i64, vp, vp, P(i64), P(i64), vp, vp, P(i64), P(i64), f32, f32,
                                             vp, P(vp)]
    L.jfa_cache_read.argtypes = [vp, i32, i64, vp, vp, vp, i32, vp, i64, vp, i64, vp]
    L.jfa_cache_summarize.argtypes = [vp, i32, i64, vp, vp, vp, i32, vp, vp]
    L.jfa_cache_select_workspace_size.argtypes = [vp, i64, i32]
    L.jfa_cache_select_workspace_size.restype = sz
    L.jfa_cache_select.argtypes = [vp, i32, i64, i32, vp, vp, vp, i32, vp, vp, i64, i32, i32, i32, i32, vp, vp, sz, vp]
    L.jfa_cache_fwd_blocks.argtypes = [vp, i32, i64, vp, vp, vp, i32, vp, i64, i32, vp, i32, i32, vp, f32, vp, i32, vp,
                                       vp, sz, vp]
    L.jfa_status_string.argtypes = [i32]
    L.jfa_status_string.restype = ctypes.c_char_p
    for name in ("jfa_plan_create", "jfa_plan_create_ex", "jfa_plan_destroy", "jfa_plan_info", "jfa_fwd", "jfa_bwd",
                 "jfa_plan_device_status", "jfa_worklist_size", "jfa_worklist_build", "jfa_plan_set_timing",
                 "jfa_plan_kernel_times", "jfa_bwd_static_scratch", "jfa_partition_sequences", "jfa_bwd_ex",
                 "jfa_plan_create_shared_kv", "jfa_partition_users", "jfa_plan_set_deterministic",
                 "jfa_plan_set_work_item", "jfa_cache_create", "jfa_cache_destroy", "jfa_cache_device_status",
                 "jfa_cache_append", "jfa_cache_fwd", "jfa_cache_create_quantized", "jfa_cache_read",
                 "jfa_cache_summarize", "jfa_cache_select", "jfa_cache_fwd_blocks"):
        getattr(L, name).restype = i32
    return L


def jfa_status_string(status: int) -> str:
    return lib().jfa_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != JFA_OK:
        raise JFAError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    """The tensor's data pointer.  The library reads and writes dense row-major arrays,
    so a tensor with any other strides is refused rather than misread."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise JFAError("tensor layout (must be contiguous)", JFA_ERR_INVALID_ARG)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


class Plan:
    """Owns a jfa_plan handle."""

    def __init__(self, handle, B, H, D, mode, causal, Tq, Tkv):
        self.handle = handle
        self.B, self.H, self.D, self.mode, self.causal = B, H, D, mode, causal
        self.Tq, self.Tkv = Tq, Tkv

    def info(self) -> dict:
        return jfa_plan_info(self)

    def __del__(self):
        try:
            if self.handle is not None and _lib is not None:
                _lib.jfa_plan_destroy(self.handle)
        finally:
            self.handle = None


def _win(window) -> int:
    return -1 if window is None else int(window)


def jfa_plan_create(q_offsets, kv_offsets, H: int, D: int, mode="softmax", causal=False, stream=None,
                    window=None) -> Plan:
    """Offsets: host int32 arrays (or CUDA int32 tensors, copied with a sync).  window: sliding
    window W (query i sees keys i' - W .. i'; needs causal), None for none."""
    m = MODES[mode] if isinstance(mode, str) else int(mode)
    on_dev = isinstance(q_offsets, torch.Tensor) and q_offsets.is_cuda
    if on_dev:
        qo = q_offsets.to(torch.int32).contiguous()
        ko = kv_offsets.to(torch.int32).contiguous()
        qp, kp, B = _ptr(qo), _ptr(ko), qo.numel() - 1
        Tq, Tkv = None, None
    else:
        qo = _i32(q_offsets.cpu() if isinstance(q_offsets, torch.Tensor) else q_offsets)
        ko = _i32(kv_offsets.cpu() if isinstance(kv_offsets, torch.Tensor) else kv_offsets)
        qp, kp, B = qo.ctypes.data_as(ctypes.c_void_p), ko.ctypes.data_as(ctypes.c_void_p), qo.size - 1
        Tq, Tkv = int(qo[-1]), int(ko[-1])
    if (qo.numel() if on_dev else qo.size) != (ko.numel() if on_dev else ko.size):
        raise JFAError("jfa_plan_create", JFA_ERR_INVALID_ARG)
    h = ctypes.c_void_p()
    _check("jfa_plan_create", lib().jfa_plan_create_ex(qp, kp, int(B), int(H), int(D), m, int(bool(causal)),
                                                        _win(window), int(on_dev), _stream(stream), ctypes.byref(h)))
    plan = Plan(h, int(B), int(H), int(D), m, bool(causal), Tq, Tkv)
    plan.window = window
    if Tq is None:
        inf = jfa_plan_info(plan)
        plan.Tq, plan.Tkv = inf["T_q"], inf["T_kv"]
    return plan


def jfa_plan_create_shared_kv(q_offsets, kv_offsets, kv_index, H: int, D: int, mode="softmax", causal=False,
                              stream=None, window=None) -> Plan:
    """Shared key/value plan: query set b attends to the rows of user kv_index[b]
    (kv_offsets over the users).  Host arrays."""
    m = MODES[mode] if isinstance(mode, str) else int(mode)
    qo, ko, ki = _i32(q_offsets), _i32(kv_offsets), _i32(kv_index)
    B, U = qo.size - 1, ko.size - 1
    if ki.size != B:
        raise JFAError("jfa_plan_create_shared_kv", JFA_ERR_INVALID_ARG)
    h = ctypes.c_void_p()
    vp = ctypes.c_void_p
    _check("jfa_plan_create_shared_kv", lib().jfa_plan_create_shared_kv(
        qo.ctypes.data_as(vp), int(B), ko.ctypes.data_as(vp), int(U), ki.ctypes.data_as(vp), int(H), int(D), m,
        int(bool(causal)), _win(window), 0, _stream(stream), ctypes.byref(h)))
    plan = Plan(h, int(B), int(H), int(D), m, bool(causal), int(qo[-1]), int(ko[-1]))
    plan.window = window
    return plan


def jfa_plan_destroy(plan: Plan):
    if plan.handle is not None:
        _check("jfa_plan_destroy", lib().jfa_plan_destroy(plan.handle))
        plan.handle = None


INFO_KEYS = ["T_q", "T_kv", "B", "H", "D", "mode", "causal", "fwd_items", "fwd_grid", "bwd_items", "bwd_grid",
             "num_sms", "dq_items", "dq_grid", "window", "pairs", "users", "merged",
             "fwd_split", "bwd_fused", "bwd_short", "fwd_short"]


def jfa_plan_info(plan: Plan) -> dict:
    buf = (ctypes.c_int64 * len(INFO_KEYS))()
    _check("jfa_plan_info", lib().jfa_plan_info(plan.handle, buf, len(INFO_KEYS)))
    return dict(zip(INFO_KEYS, [int(x) for x in buf]))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in DTYPES:
        raise JFAError("dtype", JFA_ERR_UNSUPPORTED)
    return DTYPES[t.dtype]


def _bias_args(bias, dense=None):
    """(kind, pointer): the bucket table [H, 32], or a dense per-pair bias [H, P]."""
    if dense is not None:
        if bias is not None:
            raise JFAError("bias", JFA_ERR_INVALID_ARG)
        return JFA_BIAS_DENSE, _ptr(dense)
    if bias is None:
        return JFA_BIAS_NONE, None
    return JFA_BIAS_RELPOS32, _ptr(bias)


def jfa_fwd(plan: Plan, Q, K, V, bias=None, scale=None, O=None, lse=None, stream=None, out_dtype=None,
            dense_bias=None):
    """Returns (O, lse); lse is None in GDPA modes.  O is written in out_dtype (default:
    O's dtype if given, else Q's).  bias: the bucket table [H, 32]; dense_bias: a dense
    per-pair bias [H, P] instead."""
    dt = _dtype_code(Q)
    scale = 1.0 / float(plan.D) ** 0.5 if scale is None else float(scale)
    if O is None:
        O = torch.empty(Q.shape, dtype=out_dtype or Q.dtype, device=Q.device)
    if lse is None and plan.mode == JFA_SOFTMAX:
        lse = torch.empty((Q.shape[0], plan.H), dtype=torch.float32, device=Q.device)
    bk, bp = _bias_args(bias, dense_bias)
    _check("jfa_fwd", lib().jfa_fwd(plan.handle, dt, _ptr(Q), _ptr(K), _ptr(V), bk, bp, scale, _ptr(O),
                                    _dtype_code(O), _ptr(lse), _stream(stream)))
    return O, lse


def jfa_bwd_workspace_size(plan: Plan, dtype=torch.bfloat16) -> int:
    return int(lib().jfa_bwd_workspace_size(plan.handle, DTYPES[dtype]))


def jfa_bwd(plan: Plan, Q, K, V, O, dO, lse, bias=None, scale=None, dQ=None, dK=None, dV=None, workspace=None,
            stream=None, dense_bias=None):
    """Returns (dQ, dK, dV)."""
    dt = _dtype_code(Q)
    scale = 1.0 / float(plan.D) ** 0.5 if scale is None else float(scale)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    need = jfa_bwd_workspace_size(plan, Q.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=Q.device)
    bk, bp = _bias_args(bias, dense_bias)
    _check("jfa_bwd", lib().jfa_bwd(plan.handle, dt, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _dtype_code(O), _ptr(dO),
                                    _ptr(lse), bk, bp, scale, _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream)))
    return dQ, dK, dV


def jfa_bwd_ex_workspace_size(plan: Plan, dtype=torch.bfloat16, bias_grad=True, dense=False) -> int:
    kind = (JFA_BIAS_DENSE if dense else JFA_BIAS_RELPOS32) if bias_grad else JFA_BIAS_NONE
    return int(lib().jfa_bwd_ex_workspace_size(plan.handle, DTYPES[dtype], kind))


def jfa_bwd_ex(plan: Plan, Q, K, V, O, dO, lse, bias, scale=None, dQ=None, dK=None, dV=None, dbias=None,
               workspace=None, stream=None, dense_bias=None):
    """jfa_bwd plus the gradient of the bias: of the bucket table [H, 32], or with
    dense_bias of the dense per-pair bias [H, P] (fp32).  Returns (dQ, dK, dV, dbias)."""
    dt = _dtype_code(Q)
    scale = 1.0 / float(plan.D) ** 0.5 if scale is None else float(scale)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    if dbias is None:
        shape = (plan.H, 32) if dense_bias is None else tuple(dense_bias.shape)
        dbias = torch.empty(shape, dtype=torch.float32, device=Q.device)
    need = jfa_bwd_ex_workspace_size(plan, Q.dtype, dense=dense_bias is not None)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=Q.device)
    bk, bp = _bias_args(bias, dense_bias)
    _check("jfa_bwd_ex", lib().jfa_bwd_ex(plan.handle, dt, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _dtype_code(O),
                                          _ptr(dO), _ptr(lse), bk, bp, scale, _ptr(dQ), _ptr(dK), _ptr(dV),
                                          _ptr(dbias), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                          _stream(stream)))
    return dQ, dK, dV, dbias


def jfa_bwd_static_scratch(plan: Plan, Q, K, V, O, dO, lse, bias=None, scale=None, dQ=None, dK=None, dV=None,
                           stream=None):
    """jfa_bwd with the library's static scratch array in place of a workspace, for
    callers that cannot allocate device memory: pass dQ, dK and dV preallocated and
    this binding allocates nothing either.  Returns (dQ, dK, dV)."""
    dt = _dtype_code(Q)
    scale = 1.0 / float(plan.D) ** 0.5 if scale is None else float(scale)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    bk, bp = _bias_args(bias)
    _check("jfa_bwd_static_scratch", lib().jfa_bwd_static_scratch(
        plan.handle, dt, _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _dtype_code(O), _ptr(dO), _ptr(lse), bk, bp, scale,
        _ptr(dQ), _ptr(dK), _ptr(dV), _stream(stream)))
    return dQ, dK, dV


def jfa_plan_device_status(plan: Plan, stream=None) -> int:
    return int(lib().jfa_plan_device_status(plan.handle, _stream(stream)))


KERNEL_KINDS = ["fwd", "bwd_pre", "bwd_main", "bwd_post", "bwd_dq"]


def jfa_plan_set_work_item(plan: Plan, pass_: int, index: int, item):
    """Test hook: overwrite work item `index` of pass 0 (forward), 1 (dK/dV), 2 (dQ), 3 (the
    short-query backward) or 4 (the short-query forward) with the four ints of `item` (see
    include/jfa.h)."""
    buf = np.ascontiguousarray(np.asarray(item, dtype=np.int32).reshape(4))
    _check("jfa_plan_set_work_item", lib().jfa_plan_set_work_item(plan.handle, int(pass_), int(index),
                                                                    buf.ctypes.data_as(ctypes.c_void_p)))


def jfa_plan_set_deterministic(plan: Plan, enable: bool = True):
    """enable: always the two-pass bf16 backward, the same bit for bit on every run; off
    (the default): the planner's choice, the fused backward on short sequences (whose dQ
    can differ in its last bit between runs), the two-pass one on long ones."""
    _check("jfa_plan_set_deterministic", lib().jfa_plan_set_deterministic(plan.handle, int(bool(enable))))


def jfa_plan_set_timing(plan: Plan, enable: bool = True):
    _check("jfa_plan_set_timing", lib().jfa_plan_set_timing(plan.handle, int(bool(enable))))


def jfa_plan_kernel_times(plan: Plan) -> dict:
    """{kind: (total_ms, launches)} since the previous query (synchronises)."""
    ms = (ctypes.c_double * len(KERNEL_KINDS))()
    n = (ctypes.c_int64 * len(KERNEL_KINDS))()
    _check("jfa_plan_kernel_times", lib().jfa_plan_kernel_times(plan.handle, ms, n))
    return {k: (float(ms[i]), int(n[i])) for i, k in enumerate(KERNEL_KINDS)}


def jfa_partition_sequences(q_offsets, kv_offsets, H: int, causal: bool, n_parts: int, window=None):
    """Host LPT split of a batch's sequences over n_parts GPUs.  Returns (part_of_seq int32 [B],
    part_cost int64 [n_parts])."""
    qo, ko = _i32(q_offsets), _i32(kv_offsets)
    B = qo.size - 1
    part = np.zeros(max(B, 1), dtype=np.int32)
    cost = np.zeros(int(n_parts), dtype=np.int64)
    _check("jfa_partition_sequences", lib().jfa_partition_sequences(
        qo.ctypes.data_as(ctypes.c_void_p), ko.ctypes.data_as(ctypes.c_void_p), int(B), int(H), int(bool(causal)),
        _win(window), int(n_parts), part.ctypes.data_as(ctypes.c_void_p), cost.ctypes.data_as(ctypes.c_void_p)))
    return part[:B], cost


def jfa_partition_users(q_offsets, kv_offsets, kv_index, H: int, causal: bool, n_parts: int, window=None):
    """Host LPT split of a shared key/value batch's users (with all their query sets) over
    n_parts GPUs.  Returns (part_of_user int32 [U], part_cost int64 [n_parts])."""
    qo, ko, ki = _i32(q_offsets), _i32(kv_offsets), _i32(kv_index)
    B, U = qo.size - 1, ko.size - 1
    part = np.zeros(max(U, 1), dtype=np.int32)
    cost = np.zeros(int(n_parts), dtype=np.int64)
    vp = ctypes.c_void_p
    _check("jfa_partition_users", lib().jfa_partition_users(
        qo.ctypes.data_as(vp), int(B), ko.ctypes.data_as(vp), int(U), ki.ctypes.data_as(vp), int(H),
        int(bool(causal)), _win(window), int(n_parts), part.ctypes.data_as(vp), cost.ctypes.data_as(vp)))
    return part[:U], cost


def shard(batch, rank: int, world: int):
    """The part of `batch` that rank `rank` of `world` processes (a workloads.Batch,
    repacked), by the LPT splits above: sequences, or for a shared key/value batch users
    with all their query sets.  The parts are independent, so their results are exactly
    the full batch's results for those sequences (users)."""
    from . import workloads
    if getattr(batch, "kv_map", None) is not None:
        part, _ = jfa_partition_users(batch.q_off, batch.kv_off, batch.kv_map, batch.H, batch.causal, world,
                                      window=getattr(batch, "window", None))
        return workloads.subset_users(batch, np.nonzero(part == rank)[0])
    part, _ = jfa_partition_sequences(batch.q_off, batch.kv_off, batch.H, batch.causal, world,
                                      window=getattr(batch, "window", None))
    seqs = np.nonzero(part == rank)[0]
    return workloads.subset(batch, seqs)


def jfa_worklist_size(q_offsets, kv_offsets, H: int, causal: bool, pass_: int, window=None) -> int:
    qo, ko = _i32(q_offsets), _i32(kv_offsets)
    n = ctypes.c_int64()
    _check("jfa_worklist_size", lib().jfa_worklist_size(qo.ctypes.data_as(ctypes.c_void_p),
                                                         ko.ctypes.data_as(ctypes.c_void_p), qo.size - 1, int(H),
                                                         int(bool(causal)), _win(window), int(pass_),
                                                         ctypes.byref(n)))
    return int(n.value)


def jfa_worklist_build(q_offsets, kv_offsets, H: int, causal: bool, pass_: int, n_ctas: int, window=None):
    """Host planner.  Returns (items int32 [n,4] (seq, head, tile, inner), cta_offsets [n_ctas+1],
    cta_cost [n_ctas])."""
    qo, ko = _i32(q_offsets), _i32(kv_offsets)
    n = jfa_worklist_size(qo, ko, H, causal, pass_, window)
    items = np.zeros((max(n, 1), 4), dtype=np.int32)
    offs = np.zeros(n_ctas + 1, dtype=np.int32)
    cost = np.zeros(n_ctas, dtype=np.int64)
    _check("jfa_worklist_build", lib().jfa_worklist_build(
        qo.ctypes.data_as(ctypes.c_void_p), ko.ctypes.data_as(ctypes.c_void_p), qo.size - 1, int(H),
        int(bool(causal)), _win(window), int(pass_), int(n_ctas), items.ctypes.data_as(ctypes.c_void_p),
        offs.ctypes.data_as(ctypes.c_void_p), cost.ctypes.data_as(ctypes.c_void_p)))
    return items[:n], offs, cost


# --------------------------------------------------------------------------- paged cache


class Cache:
    """Owns a jfa_cache handle and keeps the cache's arrays alive.  dtype: of the rows that are
    appended and attended with."""

    def __init__(self, handle, K, V, scales=None):
        self.handle, self.K, self.V, self.scales = handle, K, V, scales
        self.n_pages, self.page_size, self.Hkv, self.D = K.shape
        self.dtype, self.device = K.dtype, K.device
        if scales is not None:  # 4 bits: two codes in a byte
            self.D, self.dtype = 2 * self.D, torch.bfloat16
        # what the compiled calls check against
        self.info = _cache_calls().describe(handle.value or 0, K, scales is not None)

    def __del__(self):
        try:
            if self.handle is not None and _lib is not None:
                _lib.jfa_cache_destroy(self.handle)
        finally:
            self.handle = None


def _bad(fn: str, what: str):
    raise JFAError(f"{fn} ({what})", JFA_ERR_INVALID_ARG)


def jfa_cache_create(K: torch.Tensor, V: torch.Tensor, stream=None) -> Cache:
    """A handle on caches K, V [n_pages, page_size, Hkv, D] (bf16 or fp32, on the current CUDA
    device; any strides that are multiples of 16 bytes with a dense last dimension, so
    head-major pages are given as a permuted view)."""
    fn = "jfa_cache_create"
    if K.dim() != 4 or K.shape != V.shape or K.dtype != V.dtype or K.device != V.device or not K.is_cuda:
        _bad(fn, "K and V must be CUDA tensors of one shape [n_pages, page_size, Hkv, D] and type")
    if K.device.index != torch.cuda.current_device():
        _bad(fn, f"K and V lie on {K.device}, which is not the current device")
    if K.stride(3) != 1 or V.stride(3) != 1:
        _bad(fn, "the head dimension must be dense")
    n, ps, Hkv, D = K.shape
    # (a dimension of one element leaves its stride free)
    ks, vs = ((ctypes.c_int64 * 3)(*[t.stride(i) if t.shape[i] > 1 else D for i in range(3)]) for t in (K, V))
    h = ctypes.c_void_p()
    _check(fn, lib().jfa_cache_create(_dtype_code(K), Hkv, D, ps, n, K.data_ptr(), V.data_ptr(), ks, vs,
                                      _stream(stream), ctypes.byref(h)))
    return Cache(h, K, V)


def jfa_cache_create_quantized(K: torch.Tensor, V: torch.Tensor, K_scales: torch.Tensor, V_scales: torch.Tensor,
                               k_factor: float = 1.0, v_factor: float = 1.0, stream=None) -> Cache:
    """A handle on a cache held in 4 bits: codes K, V uint8 [n_pages, page_size, Hkv, D / 2] (any
    strides that are multiples of 16 bytes with a dense last dimension; head-major pages, given
    as a permuted view, are read fastest) and scales uint8 or float8_e4m3fn
    [n_pages, Hkv, page_size, D / 16] (the last two dimensions dense), on the current CUDA
    device.  It is used like jfa_cache_create's, with bf16 rows."""
    fn = "jfa_cache_create_quantized"
    if (K.dim() != 4 or K.shape != V.shape or K.dtype != torch.uint8 or V.dtype != torch.uint8 or not K.is_cuda
            or K.device != V.device):
        _bad(fn, "K and V must be uint8 CUDA tensors of one shape [n_pages, page_size, Hkv, D / 2]")
    if K.device.index != torch.cuda.current_device():
        _bad(fn, f"K and V lie on {K.device}, which is not the current device")
    n, ps, Hkv, half = K.shape
    for s in (K_scales, V_scales):
        if (s.shape != (n, Hkv, ps, half // 8) or half % 8 or s.dtype not in (torch.uint8, torch.float8_e4m3fn)
                or s.device != K.device):
            _bad(fn, "scales must be e4m3 tensors [n_pages, Hkv, page_size, D / 16] on the codes' device")
        if s.stride(3) != 1 or (ps > 1 and s.stride(2) != half // 8):
            _bad(fn, "a head's scales of one page must lie in one piece")
    if K.stride(3) != 1 or V.stride(3) != 1:
        _bad(fn, "the head dimension must be dense")
    # (a dimension of one element leaves its stride free)
    ks, vs = ((ctypes.c_int64 * 3)(*[t.stride(i) if t.shape[i] > 1 else -(-half // 16) * 16 for i in range(3)])
              for t in (K, V))
    piece = -(-ps * (half // 8) // 16) * 16
    kss, vss = ((ctypes.c_int64 * 2)(*[t.stride(i) if t.shape[i] > 1 else piece for i in range(2)])
                for t in (K_scales, V_scales))
    h = ctypes.c_void_p()
    _check(fn, lib().jfa_cache_create_quantized(Hkv, 2 * half, ps, n, K.data_ptr(), V.data_ptr(), ks, vs,
                                                K_scales.data_ptr(), V_scales.data_ptr(), kss, vss, float(k_factor),
                                                float(v_factor), _stream(stream), ctypes.byref(h)))
    return Cache(h, K, V, (K_scales, V_scales))


def jfa_cache_destroy(cache: Cache):
    if cache.handle is not None:
        _check("jfa_cache_destroy", lib().jfa_cache_destroy(cache.handle))
        cache.handle = cache.info = None


def jfa_cache_device_status(cache: Cache, stream=None) -> int:
    return int(lib().jfa_cache_device_status(cache.handle, _stream(stream)))


def jfa_cache_append(cache: Cache, K, V, q_offsets, kv_lens, page_table, Q=None, Q_out=None, rot=None,
                     rot_kind="half", stream=None):
    """Appends the new tokens' K, V [T, Hkv, D] to their slots.  rot: the rotation's table
    [rot_len, rot_dim] (cosines, then sines, fp32), applied to the keys and to Q [T, H, D]
    (into Q_out, which may be Q; allocated if None).  Returns Q_out (None without Q)."""
    if Q is not None and Q_out is None:
        with torch.cuda.stream(stream):
            Q_out = torch.empty(Q.shape, dtype=Q.dtype, device=Q.device)
    try:
        status = _calls.append(cache.info, K, V, q_offsets, kv_lens, page_table, Q, Q_out, rot,
                               ROT_KINDS.get(rot_kind, -1) if isinstance(rot_kind, str) else rot_kind,
                               None if stream is None else stream.cuda_stream)
    except (ValueError, TypeError, OverflowError) as e:
        raise JFAError(f"jfa_cache_append ({e})", JFA_ERR_INVALID_ARG) from None
    if status != JFA_OK:
        raise JFAError("jfa_cache_append", status)
    return Q_out


def jfa_cache_workspace_size(cache: Cache, H: int) -> int:
    return int(lib().jfa_cache_workspace_size(cache.handle, int(H)))


def jfa_cache_workspace(cache: Cache, H: int) -> torch.Tensor:
    """A workspace for jfa_cache_fwd, with the part that must start zero cleared on the
    current stream.  Calls that may overlap need one each."""
    n = jfa_cache_workspace_size(cache, H)
    if n == 0:
        _bad("jfa_cache_workspace", "H must be a multiple of the cache's heads")
    ws = torch.empty(n, dtype=torch.uint8, device=cache.device)
    ws[:JFA_CACHE_ZERO_BYTES].zero_()
    return ws


def jfa_cache_fwd(cache: Cache, Q, q_offsets, kv_lens, page_table, bias=None, scale=None, causal=True, window=None,
                  max_q_len=None, O=None, lse=None, out_dtype=None, workspace=None, stream=None):
    """Attention of the new tokens Q [T, H, D] over the cache.  Returns (O, lse).  bias: the
    bucket table [H, 32]; max_q_len: an upper bound of the batch's query lengths (it chooses
    the kernel); workspace: jfa_cache_workspace's, kept by the caller (one is made if None)."""
    if O is None or lse is None or workspace is None:
        with torch.cuda.stream(stream):  # what is made here belongs to the stream that writes it
            if O is None:
                O = torch.empty(Q.shape, dtype=out_dtype or Q.dtype, device=Q.device)
            if lse is None:
                lse = torch.empty(Q.shape[:2], dtype=torch.float32, device=Q.device)
            if workspace is None:
                workspace = jfa_cache_workspace(cache, Q.shape[1] if Q.dim() == 3 else 0)
    try:
        status = _calls.fwd(cache.info, Q, q_offsets, kv_lens, page_table, bias,
                            cache.D ** -0.5 if scale is None else scale, causal, window, max_q_len, O, lse, workspace,
                            None if stream is None else stream.cuda_stream)
    except (ValueError, TypeError, OverflowError) as e:
        raise JFAError(f"jfa_cache_fwd ({e})", JFA_ERR_INVALID_ARG) from None
    if status != JFA_OK:
        raise JFAError("jfa_cache_fwd", status)
    return O, lse


def _compiled(fn, call, *args):
    """A compiled call whose failed checks become this binding's error."""
    try:
        status = call(*args)
    except (ValueError, TypeError, OverflowError) as e:
        raise JFAError(f"{fn} ({e})", JFA_ERR_INVALID_ARG) from None
    if status != JFA_OK:
        raise JFAError(fn, status)


def _raw(stream):
    return None if stream is None else stream.cuda_stream


def jfa_cache_read(cache: Cache, T: int, q_offsets, kv_lens, page_table, K=None, V=None, stream=None):
    """The rows of the T new tokens as the cache holds them, K and V [T, Hkv, D] (allocated if
    None), which are returned."""
    if K is None or V is None:
        with torch.cuda.stream(stream):
            K = torch.empty(T, cache.Hkv, cache.D, dtype=cache.dtype, device=cache.device) if K is None else K
            V = torch.empty(T, cache.Hkv, cache.D, dtype=cache.dtype, device=cache.device) if V is None else V
    _compiled("jfa_cache_read", _calls.read, cache.info, T, q_offsets, kv_lens, page_table, K, V, _raw(stream))
    return K, V


def jfa_cache_summarize(cache: Cache, bounds, T: int, q_offsets, kv_lens, page_table, stream=None):
    """Brings bounds (bf16 [n_pages, Hkv, 2, D]: least and largest keys of each page) up to date
    for the pages of the T new tokens.  Returns bounds."""
    _compiled("jfa_cache_summarize", _calls.summarize, cache.info, cache.n_pages, bounds, T, q_offsets, kv_lens,
              page_table, _raw(stream))
    return bounds


def jfa_cache_select_workspace_size(cache: Cache, T: int, max_pages: int) -> int:
    return int(lib().jfa_cache_select_workspace_size(cache.handle, int(T), int(max_pages)))


def jfa_cache_select_workspace(cache: Cache, T: int, max_pages: int) -> torch.Tensor:
    """A workspace for jfa_cache_select on up to T new tokens.  Calls that may overlap need one
    each."""
    n = jfa_cache_select_workspace_size(cache, T, max_pages)
    if n == 0:
        _bad("jfa_cache_select_workspace", "T and max_pages must not be negative, nor more than jfa_cache_select takes")
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def jfa_cache_select(cache: Cache, bounds, Q, q_offsets, kv_lens, page_table, n_blocks: int, n_first: int = 1,
                     n_last: int = 1, max_q_len=None, blocks=None, workspace=None, stream=None):
    """The blocks (pages) that each new token attends to, by the score of their bounds: blocks
    [T, Hkv, n_blocks] int32, ascending, then -1 (allocated if None), which is returned."""
    if blocks is None or workspace is None:
        with torch.cuda.stream(stream):
            if blocks is None:
                blocks = torch.empty(Q.shape[0], cache.Hkv, max(int(n_blocks), 0), dtype=torch.int32, device=Q.device)
            if workspace is None:
                workspace = jfa_cache_select_workspace(cache, Q.shape[0], page_table.shape[-1])
    _compiled("jfa_cache_select", _calls.select, cache.info, cache.n_pages, bounds, Q, q_offsets, kv_lens, page_table,
              n_blocks, n_first, n_last, max_q_len, blocks, workspace, _raw(stream))
    return blocks


def jfa_cache_fwd_blocks(cache: Cache, Q, q_offsets, kv_lens, page_table, blocks, bias=None, scale=None, O=None,
                         lse=None, out_dtype=None, workspace=None, stream=None):
    """Causal attention of the new tokens Q [T, H, D] over the blocks [T, Hkv, n] listed for
    them.  Returns (O, lse).  The other arguments are jfa_cache_fwd's."""
    if O is None or lse is None or workspace is None:
        with torch.cuda.stream(stream):
            if O is None:
                O = torch.empty(Q.shape, dtype=out_dtype or Q.dtype, device=Q.device)
            if lse is None:
                lse = torch.empty(Q.shape[:2], dtype=torch.float32, device=Q.device)
            if workspace is None:
                workspace = jfa_cache_workspace(cache, Q.shape[1] if Q.dim() == 3 else 0)
    _compiled("jfa_cache_fwd_blocks", _calls.fwd_blocks, cache.info, Q, q_offsets, kv_lens, page_table, blocks, bias,
              cache.D ** -0.5 if scale is None else scale, O, lse, workspace, _raw(stream))
    return O, lse


# --------------------------------------------------------------------------- convenience


def plan_for(batch, stream=None, deterministic=False) -> Plan:
    """The plan of a workloads.Batch: shared key/value when it has a query-set-to-user map.
    deterministic: the two-pass backward (see jfa_plan_set_deterministic)."""
    if getattr(batch, "kv_map", None) is not None:
        plan = jfa_plan_create_shared_kv(batch.q_off, batch.kv_off, batch.kv_map, batch.H, batch.D, batch.mode,
                                         batch.causal, stream, window=getattr(batch, "window", None))
    else:
        plan = jfa_plan_create(batch.q_off, batch.kv_off, batch.H, batch.D, batch.mode, batch.causal, stream,
                               window=getattr(batch, "window", None))
    if deterministic:
        jfa_plan_set_deterministic(plan, True)
    return plan


class JaggedAttention(torch.autograd.Function):
    """The forward and backward passes as one torch.autograd function (argument marshalling
    only: both passes run in the library's kernels, on the current stream).

    Q [T_q, H, D], K, V [T_kv, H, D] (bf16 or fp32, contiguous); bias: the bucket table
    [H, 32], or with dense set the dense per-pair bias [H, P] (fp32), or None.  Returns O in
    Q's dtype.  The bias gradient is computed only when the bias requires one."""

    @staticmethod
    def forward(ctx, Q, K, V, bias, plan, scale, dense):
        O, lse = jfa_fwd(plan, Q, K, V, None if dense else bias, scale, dense_bias=bias if dense else None)
        ctx.plan, ctx.scale, ctx.dense = plan, scale, dense
        ctx.save_for_backward(Q, K, V, O, lse, bias)
        return O

    @staticmethod
    def backward(ctx, dO):
        Q, K, V, O, lse, bias = ctx.saved_tensors
        dO = dO.to(Q.dtype).contiguous()
        table, dense = (None, bias) if ctx.dense else (bias, None)
        if bias is not None and ctx.needs_input_grad[3]:
            dQ, dK, dV, dbias = jfa_bwd_ex(ctx.plan, Q, K, V, O, dO, lse, table, ctx.scale, dense_bias=dense)
        else:
            (dQ, dK, dV), dbias = jfa_bwd(ctx.plan, Q, K, V, O, dO, lse, table, ctx.scale, dense_bias=dense), None
        return dQ, dK, dV, dbias, None, None, None


def jagged_attention(Q, K, V, q_offsets=None, kv_offsets=None, bias=None, mode="softmax", causal=False,
                     window=None, scale=None, plan=None, dense_bias=False, kv_index=None, deterministic=False):
    """Differentiable jagged attention.  Builds the plan from the offsets (kv_index: shared
    key/value, query set b attending to user kv_index[b]) unless one is given; a plan can be
    reused while the batch's shape is the same.  deterministic: a new plan runs the two-pass
    backward (see jfa_plan_set_deterministic).  See JaggedAttention for the tensors."""
    if plan is None:
        H, D = int(Q.shape[1]), int(Q.shape[2])
        if kv_index is not None:
            plan = jfa_plan_create_shared_kv(q_offsets, kv_offsets, kv_index, H, D, mode, causal, window=window)
        else:
            plan = jfa_plan_create(q_offsets, kv_offsets, H, D, mode, causal, window=window)
        if deterministic:
            jfa_plan_set_deterministic(plan, True)
    return JaggedAttention.apply(Q, K, V, bias, plan, scale, bool(dense_bias))


def attention(batch, with_backward=True, stream=None, out_dtype=None, bias_grad=False, deterministic=False):
    """Run forward (and backward) for a workloads.Batch on the GPU: returns dict of tensors
    (with bias_grad, also "dbias", the gradient of the batch's bias table).  deterministic:
    the two-pass backward (see jfa_plan_set_deterministic)."""
    plan = plan_for(batch, stream, deterministic)
    dense = getattr(batch, "dense", None)
    O, lse = jfa_fwd(plan, batch.Q, batch.K, batch.V, batch.bias, batch.scale, stream=stream, out_dtype=out_dtype,
                     dense_bias=dense)
    out = {"O": O, "lse": lse, "plan": plan}
    if with_backward and bias_grad:
        dQ, dK, dV, dbias = jfa_bwd_ex(plan, batch.Q, batch.K, batch.V, O, batch.dO, lse, batch.bias, batch.scale,
                                       stream=stream, dense_bias=dense)
        out.update(dQ=dQ, dK=dK, dV=dV, dbias=dbias)
    elif with_backward:
        dQ, dK, dV = jfa_bwd(plan, batch.Q, batch.K, batch.V, O, batch.dO, lse, batch.bias, batch.scale,
                             stream=stream, dense_bias=dense)
        out.update(dQ=dQ, dK=dK, dV=dV)
    return out
