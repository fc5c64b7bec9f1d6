"""ctypes binding of libla2.so (C ABI in ``include/la2.h``).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels. The raw functions keep the C names and argument order
and return the C status code. ``forward`` / ``backward`` below take torch
tensors, allocate outputs and the workspace with torch (PyTorch is only the
allocator and the stream provider here) and raise ``La2Error`` on a non-zero
status. Importing this module fails loudly when the library is missing.
"""

from __future__ import annotations

import contextlib
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libla2.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libla2.so not found at {LIB_PATH}; build it with "
        "`python -m linear_attention_la2_b200.build` (nvcc, sm_100a)")

_lib = ctypes.CDLL(LIB_PATH)

LA2_OK = 0
LA2_ERR_INVALID_ARG = 1
LA2_ERR_UNSUPPORTED = 2
LA2_ERR_WORKSPACE = 3
LA2_ERR_CUDA = 4
LA2_ERR_TIMEOUT = 5
LA2_F32 = 0
LA2_BF16 = 1

_i64 = ctypes.c_int64
_int = ctypes.c_int
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t
_f64 = ctypes.c_double
_pi64 = ctypes.POINTER(ctypes.c_int64)

_SIGS = {
    "la2_workspace_size": (_sz, [_i64, _i64, _i64, _i64, _i64, _int, _int, _int, _int]),
    "la2_forward": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _int, _int, _int,
                           _vp, _sz, _vp]),
    "la2_backward": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _int,
                            _int, _int, _vp, _sz, _vp]),
    "la2_workspace_size_gqa": (_sz, [_i64, _i64, _i64, _i64, _i64, _i64, _int, _int, _int, _int]),
    "la2_forward_gqa": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _int, _int,
                               _int, _vp, _sz, _vp]),
    "la2_backward_gqa": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64,
                                _i64, _int, _int, _int, _vp, _sz, _vp]),
    "la2_workspace_size_sp": (_sz, [_i64, _i64, _i64, _i64, _i64, _int, _int, _int]),
    "la2_forward_sp": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _int,
                              _int, _vp, _sz, _vp]),
    "la2_backward_sp": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _i64, _i64, _i64,
                               _i64, _i64, _i64, _int, _int, _vp, _sz, _vp]),
    "la2_workspace_size_decay": (_sz, [_i64, _i64, _i64, _i64, _i64, _int, _int, _int]),
    "la2_forward_decay": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _int, _int,
                                 _vp, _sz, _vp]),
    "la2_backward_decay": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                  _i64, _int, _int, _vp, _sz, _vp]),
    "la2_check": (_int, [_vp]),
    "la2_status_string": (ctypes.c_char_p, [_int]),
    "la2_set_chunk_len": (_int, [_i64]),
    "la2_plan_ranges": (_i64, [_i64, _i64, _i64, _i64, _i64, _int, _int, _int, _int,
                               ctypes.POINTER(_i64), _i64]),
    "la2_set_spin_limit": (_int, [_i64]),
    "la2_profile_enable": (_int, [_int]),
    "la2_profile_num_kernels": (_int, []),
    "la2_profile_kernel_name": (ctypes.c_char_p, [_int]),
    "la2_profile_collect": (_int, [_int, ctypes.POINTER(_i64), ctypes.POINTER(ctypes.c_double)]),
    "la2_version": (_int, []),
    "la2_forward_noalloc": (_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _int, _int,
                                   _int, _vp]),
    "la2_kv_state_workspace_size": (_sz, [_i64, _i64, _i64, _i64, _i64, _int]),
    "la2_kv_state": (_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _int, _vp, _sz, _vp]),
    "la2_decode_step": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _vp]),
    "la2_workspace_size_gated": (_sz, [_i64, _i64, _i64, _i64, _i64, _int, _int]),
    "la2_forward_gated": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _int, _vp, _sz,
                                 _vp]),
    "la2_backward_gated": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                  _i64, _int, _vp, _sz, _vp]),
    "la2_kv_state_gated_workspace_size": (_sz, [_i64, _i64, _i64, _i64, _i64, _int]),
    "la2_kv_state_gated": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _int, _vp,
                                  _sz, _vp]),
    "la2_decode_step_gated": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64,
                                     _int, _vp]),
    "la2_qk_norm_rope": (_int, [_vp, _vp, _pi64, _pi64, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                _i64, _i64, _i64, _pi64, _f64, _f64, _f64, _f64, _int, _vp]),
    "la2_qk_norm_rope_backward_workspace_size": (_sz, [_i64, _i64, _i64, _i64, _i64]),
    "la2_qk_norm_rope_backward": (_int, [_vp, _vp, _vp, _vp, _pi64, _pi64, _vp, _vp, _vp, _vp, _vp, _vp,
                                         _vp, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _pi64, _f64, _f64,
                                         _f64, _f64, _int, _vp, _sz, _vp]),
    "la2_state_copy": (_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _vp]),
    "la2_state_compact": (_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp]),
}

EXPORTED = tuple(_SIGS)

for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

# Raw C entry points, same names and argument order as include/la2.h.
la2_workspace_size = _lib.la2_workspace_size
la2_forward = _lib.la2_forward
la2_backward = _lib.la2_backward
la2_check = _lib.la2_check
la2_workspace_size_gqa = _lib.la2_workspace_size_gqa
la2_forward_gqa = _lib.la2_forward_gqa
la2_backward_gqa = _lib.la2_backward_gqa
la2_workspace_size_sp = _lib.la2_workspace_size_sp
la2_forward_sp = _lib.la2_forward_sp
la2_backward_sp = _lib.la2_backward_sp
la2_workspace_size_decay = _lib.la2_workspace_size_decay
la2_forward_decay = _lib.la2_forward_decay
la2_backward_decay = _lib.la2_backward_decay
la2_set_chunk_len = _lib.la2_set_chunk_len
la2_plan_ranges = _lib.la2_plan_ranges
la2_set_spin_limit = _lib.la2_set_spin_limit
la2_profile_enable = _lib.la2_profile_enable
la2_profile_num_kernels = _lib.la2_profile_num_kernels
la2_version = _lib.la2_version
la2_forward_noalloc = _lib.la2_forward_noalloc
la2_kv_state_workspace_size = _lib.la2_kv_state_workspace_size
la2_kv_state = _lib.la2_kv_state
la2_decode_step = _lib.la2_decode_step
la2_workspace_size_gated = _lib.la2_workspace_size_gated
la2_forward_gated = _lib.la2_forward_gated
la2_backward_gated = _lib.la2_backward_gated
la2_kv_state_gated_workspace_size = _lib.la2_kv_state_gated_workspace_size
la2_kv_state_gated = _lib.la2_kv_state_gated
la2_decode_step_gated = _lib.la2_decode_step_gated
la2_qk_norm_rope = _lib.la2_qk_norm_rope
la2_qk_norm_rope_backward_workspace_size = _lib.la2_qk_norm_rope_backward_workspace_size
la2_qk_norm_rope_backward = _lib.la2_qk_norm_rope_backward
la2_state_copy = _lib.la2_state_copy
la2_state_compact = _lib.la2_state_compact
NOALLOC_SCRATCH_BYTES = 32 << 20


def plan_ranges(B, H, N, d, dv, causal, block, dtype_code, is_backward=False):
    """Range starts (in blocks of the flattened B*H*ceil(N/block) list) the
    library will use for these arguments."""
    R = la2_plan_ranges(B, H, N, d, dv, int(causal), block, dtype_code, int(is_backward), None, 0)
    if R < 0:
        raise La2Error(LA2_ERR_INVALID_ARG)
    buf = (_i64 * (R + 1))()
    la2_plan_ranges(B, H, N, d, dv, int(causal), block, dtype_code, int(is_backward), buf, R + 1)
    return list(buf)


def la2_status_string(code: int) -> str:
    return _lib.la2_status_string(code).decode()


def la2_profile_kernel_name(kernel: int) -> str:
    s = _lib.la2_profile_kernel_name(kernel)
    return s.decode() if s else ""


def la2_profile_collect(kernel: int):
    n = _i64(0)
    ms = ctypes.c_double(0.0)
    st = _lib.la2_profile_collect(kernel, ctypes.byref(n), ctypes.byref(ms))
    _raise(st)
    return int(n.value), float(ms.value)


class La2Error(RuntimeError):
    def __init__(self, code: int):
        super().__init__(la2_status_string(code))
        self.code = code


def _raise(code: int):
    if code != LA2_OK:
        raise La2Error(code)


# ------------------------------------------------------------ torch helpers


def _dtype_code(t):
    import torch

    if t.dtype == torch.bfloat16:
        return LA2_BF16
    if t.dtype == torch.float32:
        return LA2_F32
    raise La2Error(LA2_ERR_UNSUPPORTED)


def _stream_handle(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return _vp(stream.cuda_stream)


def _ptr(t):
    return _vp(t.data_ptr()) if t is not None and t.numel() > 0 else _vp(0)


def workspace_bytes(B, H, N, d, dv, causal, block, dtype_code, is_backward) -> int:
    n = la2_workspace_size(B, H, N, d, dv, int(causal), block, dtype_code, int(is_backward))
    if n == ctypes.c_size_t(-1).value:
        raise La2Error(LA2_ERR_INVALID_ARG)
    return int(n)


def _workspace(nbytes, device, stream):
    """Scratch for one call, allocated on the stream the kernels run on, so the
    caching allocator cannot hand it to other work while they still use it."""
    import torch

    if nbytes == 0:
        return None
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _check_inputs(*ts):
    for t in ts:
        if not t.is_cuda:
            raise La2Error(LA2_ERR_INVALID_ARG)
        if not t.is_contiguous():
            raise La2Error(LA2_ERR_INVALID_ARG)


def _check_like(ref, shape, dtype, *ts):
    """Every tensor in ``ts`` must have ``shape``, ``dtype`` and ref's device:
    the library sizes every tensor map and loop from q's shape, so a shorter
    k, v, dO or output would be read or written past its end."""
    for t in ts:
        if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != ref.device:
            raise La2Error(LA2_ERR_INVALID_ARG)


def _check_workspace(ws, need, device):
    import torch

    if ws is None:
        if need:
            raise La2Error(LA2_ERR_WORKSPACE)
        return
    if not ws.is_cuda or ws.device != device or not ws.is_contiguous() or ws.dtype != torch.uint8:
        raise La2Error(LA2_ERR_INVALID_ARG)


def _kv_heads(q, k, v):
    """K/V head count of a call: k, v [B,Hkv,N,.] with Hkv dividing q's H."""
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise La2Error(LA2_ERR_INVALID_ARG)
    H, Hkv = q.shape[1], k.shape[1]
    if (H > 0 and (Hkv < 1 or H % Hkv)) or (H == 0 and Hkv != 0):
        raise La2Error(LA2_ERR_INVALID_ARG)
    return Hkv


def workspace_bytes_gqa(B, H, Hkv, N, d, dv, causal, block, dtype_code, is_backward) -> int:
    n = la2_workspace_size_gqa(B, H, Hkv, N, d, dv, int(causal), block, dtype_code, int(is_backward))
    if n == ctypes.c_size_t(-1).value:
        raise La2Error(LA2_ERR_INVALID_ARG)
    return int(n)


def forward(q, k, v, causal: bool = True, block: int = 64, out=None, workspace=None, stream=None):
    """O = ((Q K^T) ⊙ M) V for [B,H,N,d] CUDA tensors; returns O. k and v may
    hold fewer heads (grouped K/V heads: query head h reads K/V head
    h // (H // Hkv))."""
    import torch

    _check_inputs(q, k, v)
    Hkv = _kv_heads(q, k, v)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    _check_like(q, (B, Hkv, N, d), q.dtype, k)
    _check_like(q, (B, Hkv, N, dv), q.dtype, v)
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=q.dtype, device=q.device)
    _check_inputs(out)
    _check_like(q, (B, H, N, dv), q.dtype, out)
    need = workspace_bytes_gqa(B, H, Hkv, N, d, dv, causal, block, dt, False)
    ws = workspace if workspace is not None else _workspace(need, q.device, stream)
    _check_workspace(ws, need, q.device)
    _raise(la2_forward_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, Hkv, N, d, dv, int(causal),
                           block, dt, _ptr(ws), ws.numel() if ws is not None else 0,
                           _stream_handle(stream)))
    return out


def backward(q, k, v, do, causal: bool = True, block: int = 64, outs=None, workspace=None,
             stream=None):
    """Gradients (dQ, dK, dV) of <dO, O> for the same op; returns a tuple. With
    grouped K/V heads dK and dV are the sums over each group's query heads."""
    import torch

    _check_inputs(q, k, v, do)
    Hkv = _kv_heads(q, k, v)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    _check_like(q, (B, Hkv, N, d), q.dtype, k)
    _check_like(q, (B, Hkv, N, dv), q.dtype, v)
    _check_like(q, (B, H, N, dv), q.dtype, do)
    if outs is None:
        outs = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    dq, dk, dvv = outs
    _check_inputs(dq, dk, dvv)
    _check_like(q, q.shape, q.dtype, dq)
    _check_like(q, (B, Hkv, N, d), q.dtype, dk)
    _check_like(q, (B, Hkv, N, dv), q.dtype, dvv)
    need = workspace_bytes_gqa(B, H, Hkv, N, d, dv, causal, block, dt, True)
    ws = workspace if workspace is not None else _workspace(need, q.device, stream)
    _check_workspace(ws, need, q.device)
    _raise(la2_backward_gqa(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dvv), B,
                            H, Hkv, N, d, dv, int(causal), block, dt, _ptr(ws),
                            ws.numel() if ws is not None else 0, _stream_handle(stream)))
    return dq, dk, dvv


def workspace_bytes_decay(B, H, N, d, dv, block, dtype_code, is_backward) -> int:
    n = la2_workspace_size_decay(B, H, N, d, dv, block, dtype_code, int(is_backward))
    if n == ctypes.c_size_t(-1).value:
        raise La2Error(LA2_ERR_INVALID_ARG)
    return int(n)


def _decay_rates(lam, q, stream):
    """Per-head rates as a float32 CUDA tensor of H values on q's device (a
    copy, when one is needed, is made on the stream the kernels run on)."""
    import torch

    lam = torch.as_tensor(lam, dtype=torch.float32).reshape(-1)
    if lam.numel() != q.shape[1]:
        raise La2Error(LA2_ERR_INVALID_ARG)
    if stream is None:
        return lam.to(q.device).contiguous()
    with torch.cuda.stream(stream):
        return lam.to(q.device).contiguous()


def forward_decay(q, k, v, lam, block: int = 64, out=None, workspace=None, stream=None):
    """Decayed causal form: o_t = sum_{s<=t} lam_h^(t-s) (q_t . k_s) v_s for
    [B,H,N,d] CUDA tensors and H per-head rates ``lam``; returns O."""
    import torch

    _check_inputs(q, k, v)
    if q.dim() != 4:
        raise La2Error(LA2_ERR_INVALID_ARG)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    _check_like(q, q.shape, q.dtype, k)
    _check_like(q, (B, H, N, dv), q.dtype, v)
    rates = _decay_rates(lam, q, stream)
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=q.dtype, device=q.device)
    _check_inputs(out)
    _check_like(q, (B, H, N, dv), q.dtype, out)
    need = workspace_bytes_decay(B, H, N, d, dv, block, dt, False)
    ws = workspace if workspace is not None else _workspace(need, q.device, stream)
    _check_workspace(ws, need, q.device)
    _raise(la2_forward_decay(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(rates), B, H, N, d, dv,
                             block, dt, _ptr(ws), ws.numel() if ws is not None else 0,
                             _stream_handle(stream)))
    return out


def backward_decay(q, k, v, do, lam, block: int = 64, outs=None, workspace=None, stream=None):
    """Gradients (dQ, dK, dV) of <dO, O> for the decayed causal form."""
    import torch

    _check_inputs(q, k, v, do)
    if q.dim() != 4:
        raise La2Error(LA2_ERR_INVALID_ARG)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    _check_like(q, q.shape, q.dtype, k)
    _check_like(q, (B, H, N, dv), q.dtype, v, do)
    rates = _decay_rates(lam, q, stream)
    if outs is None:
        outs = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    dq, dk, dvv = outs
    _check_inputs(dq, dk, dvv)
    _check_like(q, q.shape, q.dtype, dq, dk)
    _check_like(q, (B, H, N, dv), q.dtype, dvv)
    need = workspace_bytes_decay(B, H, N, d, dv, block, dt, True)
    ws = workspace if workspace is not None else _workspace(need, q.device, stream)
    _check_workspace(ws, need, q.device)
    _raise(la2_backward_decay(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dvv),
                              _ptr(rates), B, H, N, d, dv, block, dt, _ptr(ws),
                              ws.numel() if ws is not None else 0, _stream_handle(stream)))
    return dq, dk, dvv


def kv_state(k, v, state=None, workspace=None, stream=None):
    """state += sum_t k_t^T v_t per sequence; k [B,H,N,d], v [B,H,N,dv] CUDA
    tensors, state [B,H,d,dv] float32 (zeros if omitted). Returns the state."""
    import torch

    _check_inputs(k, v)
    if k.dim() != 4 or v.dim() != 4:
        raise La2Error(LA2_ERR_INVALID_ARG)
    B, H, N, d = k.shape
    dv = v.shape[-1]
    dt = _dtype_code(k)
    _check_like(k, (B, H, N, dv), k.dtype, v)
    if state is None:
        state = torch.zeros((B, H, d, dv), dtype=torch.float32, device=k.device)
    _check_inputs(state)
    _check_like(k, (B, H, d, dv), torch.float32, state)
    need = la2_kv_state_workspace_size(B, H, N, d, dv, dt)
    if need == ctypes.c_size_t(-1).value:
        raise La2Error(LA2_ERR_INVALID_ARG)
    ws = workspace if workspace is not None else _workspace(need, k.device, stream)
    _check_workspace(ws, need, k.device)
    _raise(la2_kv_state(_ptr(k), _ptr(v), _ptr(state), B, H, N, d, dv, dt, _ptr(ws),
                        ws.numel() if ws is not None else 0, _stream_handle(stream)))
    return state


def decode_step(q, k, v, state, out=None, stream=None):
    """One RNN-mode token per sequence: state += k^T v, o = q state. q, k [B,H,d],
    v [B,H,dv] CUDA tensors, state [B,H,d,dv] float32 (updated in place). Returns o."""
    import torch

    _check_inputs(q, k, v, state)
    if q.dim() != 3 or v.dim() != 3:
        raise La2Error(LA2_ERR_INVALID_ARG)
    B, H, d = q.shape
    dv = v.shape[-1]
    _dtype_code(q)
    _check_like(q, q.shape, q.dtype, k)
    _check_like(q, (B, H, dv), q.dtype, v)
    _check_like(q, (B, H, d, dv), torch.float32, state)
    if out is None:
        out = torch.empty((B, H, dv), dtype=q.dtype, device=q.device)
    _check_inputs(out)
    _check_like(q, (B, H, dv), q.dtype, out)
    _raise(la2_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(state), B, H, d, dv,
                           _dtype_code(q), _stream_handle(stream)))
    return out


def check(stream=None):
    _raise(la2_check(_stream_handle(stream)))


def _states_arg(states, q):
    """(pointer, count) of a [n,B,H,d,dv] float32 stack of states (None: none)."""
    import torch

    if states is None or states.shape[0] == 0:
        return _vp(0), 0
    B, H, _, d = q.shape
    _check_inputs(states)
    if states.dim() != 5 or tuple(states.shape[1:4]) != (B, H, d) or states.dtype != torch.float32 \
            or states.device != q.device:
        raise La2Error(LA2_ERR_INVALID_ARG)
    return _ptr(states), int(states.shape[0])


def forward_sp(q, k, v, prefix_states=None, block: int = 64, out=None, workspace=None, stream=None):
    """Causal output of one part of longer sequences: ``prefix_states``
    [n,B,H,d,dv] float32 sum to the KV state of everything before the part."""
    import torch

    _check_inputs(q, k, v)
    if q.dim() != 4 or v.dim() != 4:
        raise La2Error(LA2_ERR_INVALID_ARG)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    _check_like(q, q.shape, q.dtype, k)
    _check_like(q, (B, H, N, dv), q.dtype, v)
    if out is None:
        out = torch.empty((B, H, N, dv), dtype=q.dtype, device=q.device)
    _check_inputs(out)
    _check_like(q, (B, H, N, dv), q.dtype, out)
    pp, npre = _states_arg(prefix_states, q)
    need = la2_workspace_size_sp(B, H, N, d, dv, block, dt, 0)
    if need == ctypes.c_size_t(-1).value:
        raise La2Error(LA2_ERR_INVALID_ARG)
    ws = workspace if workspace is not None else _workspace(need, q.device, stream)
    _check_workspace(ws, need, q.device)
    _raise(la2_forward_sp(_ptr(q), _ptr(k), _ptr(v), _ptr(out), pp, npre, B, H, N, d, dv, block, dt,
                          _ptr(ws), ws.numel() if ws is not None else 0, _stream_handle(stream)))
    return out


def backward_sp(q, k, v, do, prefix_states=None, suffix_states=None, block: int = 64, outs=None,
                workspace=None, stream=None):
    """Gradients of one part of longer sequences: ``prefix_states`` sum to the
    KV state before the part, ``suffix_states`` to sum q^T dO after it."""
    import torch

    _check_inputs(q, k, v, do)
    if q.dim() != 4 or v.dim() != 4:
        raise La2Error(LA2_ERR_INVALID_ARG)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    _check_like(q, q.shape, q.dtype, k)
    _check_like(q, (B, H, N, dv), q.dtype, v, do)
    if outs is None:
        outs = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    dq, dk, dvv = outs
    _check_inputs(dq, dk, dvv)
    _check_like(q, q.shape, q.dtype, dq, dk)
    _check_like(q, (B, H, N, dv), q.dtype, dvv)
    pp, npre = _states_arg(prefix_states, q)
    sp, nsuf = _states_arg(suffix_states, q)
    need = la2_workspace_size_sp(B, H, N, d, dv, block, dt, 1)
    if need == ctypes.c_size_t(-1).value:
        raise La2Error(LA2_ERR_INVALID_ARG)
    ws = workspace if workspace is not None else _workspace(need, q.device, stream)
    _check_workspace(ws, need, q.device)
    _raise(la2_backward_sp(_ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(dq), _ptr(dk), _ptr(dvv), pp,
                           npre, sp, nsuf, B, H, N, d, dv, block, dt, _ptr(ws),
                           ws.numel() if ws is not None else 0, _stream_handle(stream)))
    return dq, dk, dvv


# ---------------------------------------------------------------- gated form


def _sized(n) -> int:
    if n == ctypes.c_size_t(-1).value:
        raise La2Error(LA2_ERR_INVALID_ARG)
    return int(n)


def workspace_bytes_gated(B, H, N, d, dv, dtype_code, is_backward) -> int:
    return _sized(la2_workspace_size_gated(B, H, N, d, dv, dtype_code, int(is_backward)))


_HERE = contextlib.nullcontext()


def _call_on(ref, stream):
    """Context of one call: ref's device and the call's stream are current, so what
    is allocated inside belongs to the stream that the kernels run on."""
    import torch

    if stream is not None:
        if stream.device != ref.device:
            raise La2Error(LA2_ERR_INVALID_ARG)
        return torch.cuda.stream(stream)
    if ref.device.index == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(ref.device)


def forward_gated(q, k, v, gate, out=None, workspace=None, stream=None):
    """Gated form: KV_t = exp(gate_t) KV_(t-1) + k_t^T v_t, o_t = q_t KV_t for
    [B,H,N,d] CUDA tensors and log gates [B,H,N] of the same type (-inf restarts
    the state); returns O."""
    import torch

    _check_inputs(q, k, v, gate)
    if q.dim() != 4 or v.dim() != 4:
        raise La2Error(LA2_ERR_INVALID_ARG)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    _check_like(q, q.shape, q.dtype, k)
    _check_like(q, (B, H, N, dv), q.dtype, v)
    _check_like(q, (B, H, N), q.dtype, gate)
    with _call_on(q, stream):
        if out is None:
            out = torch.empty((B, H, N, dv), dtype=q.dtype, device=q.device)
        _check_inputs(out)
        _check_like(q, (B, H, N, dv), q.dtype, out)
        need = workspace_bytes_gated(B, H, N, d, dv, dt, False)
        ws = workspace if workspace is not None else _workspace(need, q.device, None)
        _check_workspace(ws, need, q.device)
        _raise(la2_forward_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(out), B, H, N, d, dv, dt,
                                 _ptr(ws), ws.numel() if ws is not None else 0, _stream_handle(stream)))
    return out


def backward_gated(q, k, v, gate, do, outs=None, workspace=None, stream=None):
    """Gradients (dQ, dK, dV, dGate) of <dO, O> for the gated form; dGate is the
    gradient by the log gates."""
    import torch

    _check_inputs(q, k, v, gate, do)
    if q.dim() != 4 or v.dim() != 4:
        raise La2Error(LA2_ERR_INVALID_ARG)
    B, H, N, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    _check_like(q, q.shape, q.dtype, k)
    _check_like(q, (B, H, N, dv), q.dtype, v, do)
    _check_like(q, (B, H, N), q.dtype, gate)
    with _call_on(q, stream):
        if outs is None:
            outs = tuple(torch.empty_like(t) for t in (q, k, v, gate))
        dq, dk, dvv, dgate = outs
        _check_inputs(dq, dk, dvv, dgate)
        _check_like(q, q.shape, q.dtype, dq, dk)
        _check_like(q, (B, H, N, dv), q.dtype, dvv)
        _check_like(q, (B, H, N), q.dtype, dgate)
        need = workspace_bytes_gated(B, H, N, d, dv, dt, True)
        ws = workspace if workspace is not None else _workspace(need, q.device, None)
        _check_workspace(ws, need, q.device)
        _raise(la2_backward_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(do), _ptr(dq), _ptr(dk),
                                  _ptr(dvv), _ptr(dgate), B, H, N, d, dv, dt, _ptr(ws),
                                  ws.numel() if ws is not None else 0, _stream_handle(stream)))
    return dq, dk, dvv, dgate


def _index_list(ref, t, n=None):
    """A contiguous int32 index list on ref's device (length ``n`` if given)."""
    import torch

    _check_inputs(t)
    if t.dim() != 1 or t.dtype != torch.int32 or t.device != ref.device or (n is not None and t.numel() != n):
        raise La2Error(LA2_ERR_INVALID_ARG)
    return t


def kv_state_gated(k, v, gate, state=None, slots=None, workspace=None, stream=None):
    """The gated state after a prefill of k [B,H,N,d], v [B,H,N,dv] with log gates
    [B,H,N], continuing ``state`` [S,H,d,dv] float32 in place (zeros [B,H,d,dv] if
    omitted). Row b updates slot ``slots[b]`` (int32 CUDA tensor, -1: skipped), or
    slot b. Returns the state."""
    import torch

    _check_inputs(k, v, gate)
    if k.dim() != 4 or v.dim() != 4:
        raise La2Error(LA2_ERR_INVALID_ARG)
    B, H, N, d = k.shape
    dv = v.shape[-1]
    dt = _dtype_code(k)
    _check_like(k, (B, H, N, dv), k.dtype, v)
    _check_like(k, (B, H, N), k.dtype, gate)
    if state is None and slots is not None:
        raise La2Error(LA2_ERR_INVALID_ARG)
    with _call_on(k, stream):
        if state is None:
            state = torch.zeros((B, H, d, dv), dtype=torch.float32, device=k.device)
        S = _pool_slots(k, state, (H, d, dv), B, slots)
        need = _sized(la2_kv_state_gated_workspace_size(B, H, N, d, dv, dt))
        ws = workspace if workspace is not None else _workspace(need, k.device, None)
        _check_workspace(ws, need, k.device)
        _raise(la2_kv_state_gated(_ptr(k), _ptr(v), _ptr(gate), _ptr(state), _ptr(slots), S, B, H, N, d, dv,
                                  dt, _ptr(ws), ws.numel() if ws is not None else 0,
                                  _stream_handle(stream)))
    return state


def _pool_slots(ref, state, tail, B, slots):
    """Slot count of a pool [S,H,d,dv] that B batch rows work on."""
    import torch

    _check_inputs(state)
    if state.dim() != 4 or tuple(state.shape[1:]) != tuple(tail) or state.dtype != torch.float32 \
            or state.device != ref.device:
        raise La2Error(LA2_ERR_INVALID_ARG)
    if slots is not None:
        _index_list(ref, slots, B)
    elif state.shape[0] != B:
        raise La2Error(LA2_ERR_INVALID_ARG)
    return state.shape[0]


def decode_step_gated(q, k, v, gate, state, slots=None, out=None, stream=None):
    """One gated token per row: S <- exp(gate) S + k^T v, o = q S. q, k [B,H,d],
    v [B,H,dv], log gates [B,H]; ``state`` [S,H,d,dv] float32 is updated in place at
    ``slots`` (int32 CUDA tensor [B], -1: the row is skipped and its output left as
    it was), or at slot b for row b. Returns o (zeros behind skipped rows when
    ``out`` is omitted)."""
    import torch

    _check_inputs(q, k, v, gate)
    if q.dim() != 3 or v.dim() != 3:
        raise La2Error(LA2_ERR_INVALID_ARG)
    B, H, d = q.shape
    dv = v.shape[-1]
    dt = _dtype_code(q)
    _check_like(q, q.shape, q.dtype, k)
    _check_like(q, (B, H, dv), q.dtype, v)
    _check_like(q, (B, H), q.dtype, gate)
    S = _pool_slots(q, state, (H, d, dv), B, slots)
    with _call_on(q, stream):
        if out is None:
            make = torch.empty if slots is None else torch.zeros
            out = make((B, H, dv), dtype=q.dtype, device=q.device)
        _check_inputs(out)
        _check_like(q, (B, H, dv), q.dtype, out)
        _raise(la2_decode_step_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(gate), _ptr(out), _ptr(state),
                                     _ptr(slots), S, B, H, d, dv, dt, _stream_handle(stream)))
    return out


# --------------------------------------------------------------- state slots


def state_copy(state, src, dst, stream=None):
    """Slot dst[i] of the pool ``state`` [S,H,d,dv] float32 <- slot src[i], or zeros
    where src[i] is -1; dst[i] = -1 does nothing (int32 CUDA lists). Returns the pool."""
    import torch

    _check_inputs(state)
    if state.dim() != 4 or state.dtype != torch.float32:
        raise La2Error(LA2_ERR_INVALID_ARG)
    n = _index_list(state, src).numel()
    _index_list(state, dst, n)
    S, H, d, dv = state.shape
    with _call_on(state, stream):
        _raise(la2_state_copy(_ptr(state), _ptr(src), _ptr(dst), n, S, H, d, dv, _stream_handle(stream)))
    return state


def state_compact(state, live, moved=None, stream=None):
    """Moves the live slots (int32 CUDA list ``live`` [S], non-zero) of the pool
    ``state`` [S,H,d,dv] float32 to its front. Returns the new slot of every old one
    (int32 [S], -1: was not live)."""
    import torch

    _check_inputs(state)
    if state.dim() != 4 or state.dtype != torch.float32:
        raise La2Error(LA2_ERR_INVALID_ARG)
    S, H, d, dv = state.shape
    _index_list(state, live, S)
    with _call_on(state, stream):
        if moved is None:
            moved = torch.empty_like(live)
        _index_list(state, moved, S)
        _raise(la2_state_compact(_ptr(state), _ptr(live), _ptr(moved), S, H, d, dv, _stream_handle(stream)))
    return moved


# ------------------------------------------- queries and keys: norm, rotation


def _strided(x):
    """(data pointer, element strides of batch, token, head) of a [B,N,heads,d]
    CUDA tensor with a dense last dimension."""
    if not x.is_cuda or x.dim() != 4 or (x.shape[-1] > 1 and x.stride(-1) != 1):
        raise La2Error(LA2_ERR_INVALID_ARG)
    return _ptr(x), (_i64 * 3)(*x.stride()[:3])


def _rope_args(q, k, wq, wk, positions, rot, sections):
    import torch

    qp, qs = _strided(q)
    kp, ks = _strided(k)
    B, N, H, d = q.shape
    Hkv = k.shape[2]
    _check_like(q, (B, N, Hkv, d), q.dtype, k)
    dt = _dtype_code(q)
    for w in (wq, wk):
        if w is not None:
            _check_inputs(w)
            _check_like(q, (d,), q.dtype, w)
    rot = d if rot is None else int(rot)
    axes = 1
    if positions is not None:
        _check_inputs(positions)
        axes = positions.shape[0] if positions.dim() == 3 else 1
        if positions.dtype != torch.int32 or positions.device != q.device \
                or tuple(positions.shape[-2:]) != (B, N) or positions.dim() not in (2, 3):
            raise La2Error(LA2_ERR_INVALID_ARG)
    elif sections is not None:
        axes = len(sections)
    if sections is not None and len(sections) != axes:
        raise La2Error(LA2_ERR_INVALID_ARG)
    sec = None if sections is None else (_i64 * axes)(*[int(x) for x in sections])
    return qp, kp, qs, ks, B, N, H, Hkv, d, rot, axes, sec, dt


def qk_norm_rope(q, k, wq=None, wk=None, positions=None, base: float = 10000.0, rot=None, sections=None,
                 eps: float = 1e-6, q_scale: float = 1.0, k_scale: float = 1.0, outs=None, stream=None):
    """RMS norm (weights ``wq``, ``wk`` [d], None: ones) and position rotation of
    every head's queries and keys: q [B,N,H,d], k [B,N,Hkv,d] (any strides, dense last
    dimension) to dense [B,H,N,d], [B,Hkv,N,d], scaled by q_scale, k_scale.
    positions: int32 CUDA tensor [B,N] or [axes,B,N] (None: 0..N-1); ``sections`` are
    the pairs of each axis, adding up to rot/2; the first ``rot`` values turn (None:
    all). Returns (q_out, k_out)."""
    import torch

    qp, kp, qs, ks, B, N, H, Hkv, d, rot, axes, sec, dt = _rope_args(q, k, wq, wk, positions, rot, sections)
    with _call_on(q, stream):
        if outs is None:
            outs = (torch.empty((B, H, N, d), dtype=q.dtype, device=q.device),
                    torch.empty((B, Hkv, N, d), dtype=q.dtype, device=q.device))
        qo, ko = outs
        _check_inputs(qo, ko)
        _check_like(q, (B, H, N, d), q.dtype, qo)
        _check_like(q, (B, Hkv, N, d), q.dtype, ko)
        _raise(la2_qk_norm_rope(qp, kp, qs, ks, _ptr(wq), _ptr(wk), _ptr(positions), _ptr(qo), _ptr(ko), B, N,
                                H, Hkv, d, rot, axes, sec, base, eps, q_scale, k_scale, dt,
                                _stream_handle(stream)))
    return qo, ko


def qk_norm_rope_backward(dq_out, dk_out, q, k, wq=None, wk=None, positions=None, base: float = 10000.0,
                          rot=None, sections=None, eps: float = 1e-6, q_scale: float = 1.0,
                          k_scale: float = 1.0, outs=None, workspace=None, stream=None):
    """Gradients (dq [B,N,H,d], dk [B,N,Hkv,d], dwq, dwk) of ``qk_norm_rope`` from
    dq_out [B,H,N,d], dk_out [B,Hkv,N,d] and the forward's arguments (dwq, dwk are
    None where the weight is)."""
    import torch

    qp, kp, qs, ks, B, N, H, Hkv, d, rot, axes, sec, dt = _rope_args(q, k, wq, wk, positions, rot, sections)
    _check_inputs(dq_out, dk_out)
    _check_like(q, (B, H, N, d), q.dtype, dq_out)
    _check_like(q, (B, Hkv, N, d), q.dtype, dk_out)
    with _call_on(q, stream):
        if outs is None:
            outs = (torch.empty((B, N, H, d), dtype=q.dtype, device=q.device),
                    torch.empty((B, N, Hkv, d), dtype=q.dtype, device=q.device),
                    None if wq is None else torch.empty_like(wq), None if wk is None else torch.empty_like(wk))
        dq, dk, dwq, dwk = outs
        _check_inputs(dq, dk, *(w for w in (dwq, dwk) if w is not None))
        _check_like(q, (B, N, H, d), q.dtype, dq)
        _check_like(q, (B, N, Hkv, d), q.dtype, dk)
        _check_like(q, (d,), q.dtype, *(w for w in (dwq, dwk) if w is not None))
        need = _sized(la2_qk_norm_rope_backward_workspace_size(B, N, H, Hkv, d))
        ws = workspace if workspace is not None else _workspace(need, q.device, None)
        _check_workspace(ws, need, q.device)
        _raise(la2_qk_norm_rope_backward(_ptr(dq_out), _ptr(dk_out), qp, kp, qs, ks, _ptr(wq), _ptr(wk),
                                         _ptr(positions), _ptr(dq), _ptr(dk), _ptr(dwq), _ptr(dwk), B, N, H,
                                         Hkv, d, rot, axes, sec, base, eps, q_scale, k_scale, dt, _ptr(ws),
                                         ws.numel() if ws is not None else 0, _stream_handle(stream)))
    return dq, dk, dwq, dwk
