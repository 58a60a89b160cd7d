"""Binding of liblvx.so (argument marshalling only), by ctypes.

Each ``lvx_*`` function here has the C entry point's name and meaning (see
``include/lvx.h``).  Sizes are read from tensor shapes, pointers from
``data_ptr()``, the stream from ``torch.cuda.current_stream()`` unless one is
given.  Every step of the computation runs in the library's kernels.  Four allocating calls
(rope_axes, head_norm_rope, head_norm_rope_backward, attention_prefix) go through the
extension ``_calls.so``, which takes their arguments in less time.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("LVX_LIBRARY", os.path.join(_HERE, "liblvx.so"))

LVX_FP32 = 0
LVX_BF16 = 1
STATUS = {0: "LVX_OK", 1: "LVX_ERR_INVALID_ARG", 2: "LVX_ERR_UNSUPPORTED",
          3: "LVX_ERR_WORKSPACE", 4: "LVX_ERR_CUDA", 5: "LVX_ERR_DEVICE_TIMEOUT"}


class LvxError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}")
        self.status = status


_lib = None

LVX_PAIR_HALF = 0
LVX_PAIR_ADJACENT = 1

_c_int, _c_float, _c_size, _vp = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p
_c_i64 = ctypes.c_int64

_SIGS = {
    "lvx_status_string": ([_c_int], ctypes.c_char_p),
    "lvx_version": ([], _c_int),
    "lvx_attn_fwd_workspace": ([_c_int] * 8 + [_c_int], _c_size),
    "lvx_attn_fwd": ([_vp] * 5 + [_c_int] * 8 + [_c_int, _c_float, _vp, _c_size, _vp], _c_int),
    "lvx_merge_partials": ([_vp] * 4 + [_c_int] * 5 + [_c_int, _vp], _c_int),
    "lvx_attn_fwd_partials": ([_vp] * 5 + [_c_int] * 8 + [_c_int, _c_float, _vp], _c_int),
    "lvx_attn_fwd_noalloc": ([_vp] * 5 + [_c_int] * 8 + [_c_int, _c_float, _vp], _c_int),
    "lvx_attn_bwd_workspace": ([_c_int] * 7 + [_c_int], _c_size),
    "lvx_attn_bwd": ([_vp] * 9 + [_c_int] * 7 + [_c_int, _c_float, _vp, _c_size, _vp], _c_int),
    "lvx_attn_bwd_accumulate": ([_vp] * 9 + [_c_int] * 7 + [_c_int, _c_float, _vp, _c_size, _vp],
                                _c_int),
    "lvx_kv_recompute": ([_vp] * 5 + [_c_int] * 5 + [_c_int, _vp], _c_int),
    "lvx_kv_recompute_bwd": ([_vp] * 8 + [_c_int] * 5 + [_c_int, _vp], _c_int),
    "lvx_attn_fwd_recompute_workspace": ([_c_int] * 8 + [_c_int], _c_size),
    "lvx_attn_fwd_recompute": ([_vp] * 6 + [_c_int] * 8 + [_c_int, _c_float, _vp, _c_size, _vp],
                               _c_int),
    "lvx_attn_bwd_recompute_workspace": ([_c_int] * 8 + [_c_int], _c_size),
    "lvx_attn_bwd_recompute": ([_vp] * 11 + [_c_int] * 8 + [_c_int, _c_float, _vp, _c_size, _vp],
                               _c_int),
    "lvx_rope_axes": ([_vp] * 7 + [_c_int] * 8 + [_c_i64] * 4 + [_c_int, _vp], _c_int),
    "lvx_head_norm_rope": ([_vp] * 9 + [_c_int] * 7 + [_c_float] + [_c_i64] * 4 + [_c_int, _vp],
                           _c_int),
    "lvx_head_norm_rope_bwd_workspace": ([_c_int], _c_size),
    "lvx_head_norm_rope_bwd": ([_vp] * 13 + [_c_int] * 7 + [_c_float] + [_c_i64] * 6 +
                               [_c_int, _vp, _c_size, _vp], _c_int),
    "lvx_attn_prefix_workspace": ([_c_int] * 7 + [_c_int], _c_size),
    "lvx_attn_prefix": ([_vp] * 8 + [_c_int] * 7 + [_c_int, _c_float, _vp, _c_size, _vp], _c_int),
    "lvx_last_device_error": ([_vp], _c_int),
    "lvx_selftest_wait_timeout": ([_vp], _c_int),
    "lvx_selftest_prefix_plan": ([_c_int] * 7 + [_c_int, _vp], _c_int),
}


def lib() -> ctypes.CDLL:
    """Loads liblvx.so once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m blockwise_long_context_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(status: int, where: str) -> None:
    if status != 0:
        raise LvxError(status, where)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return LVX_FP32
    if t.dtype == torch.bfloat16:
        return LVX_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def lvx_status_string(status: int) -> str:
    return lib().lvx_status_string(status).decode()


def lvx_attn_fwd_workspace(B, H, H_kv, S_Q, S_KV, d, n_blocks, causal, dtype: int) -> int:
    return lib().lvx_attn_fwd_workspace(B, H, H_kv, S_Q, S_KV, d, n_blocks, int(causal), dtype)


def lvx_attn_bwd_workspace(B, H, H_kv, S_Q, S_KV, d, causal, dtype: int) -> int:
    return lib().lvx_attn_bwd_workspace(B, H, H_kv, S_Q, S_KV, d, int(causal), dtype)


def lvx_attn_fwd(q, k, v, out, lse, n_blocks: int, causal: bool = False, scale: float = 0.0,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """q [B,S_Q,H,d], k/v [B,S_KV,H_kv,d], out like q, lse [B,H,S_Q] fp32."""
    B, S_Q, H, d = q.shape
    S_KV, H_kv = k.shape[1], k.shape[2]
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().lvx_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, H_kv, S_Q,
                              S_KV, d, n_blocks, int(causal), _dt(q), float(scale),
                              _ptr(workspace), ws, _stream(stream)), "lvx_attn_fwd")


def lvx_attn_fwd_noalloc(q, k, v, out, lse, n_blocks: int, causal: bool = False,
                         scale: float = 0.0, stream=None) -> None:
    """lvx_attn_fwd for callers that cannot allocate: the block partials live in
    the library's fixed 64 MiB device array instead of a caller workspace."""
    B, S_Q, H, d = q.shape
    S_KV, H_kv = k.shape[1], k.shape[2]
    _check(lib().lvx_attn_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, H_kv,
                                      S_Q, S_KV, d, n_blocks, int(causal), _dt(q), float(scale),
                                      _stream(stream)), "lvx_attn_fwd_noalloc")


def lvx_attn_fwd_partials(q, k, v, o_parts, l_parts, scale: float = 0.0, stream=None,
                          causal: bool = False) -> None:
    """q [B,S_Q,H,d], k/v [B,S_KV,H_kv,d] (a shard of the keys/values) ->
    o_parts [n,B,H,S_Q,d] fp32, l_parts [n,B,H,S_Q] fp32; n is o_parts.shape[0].
    causal: key j visible to row r iff j <= r (S_Q == S_KV)."""
    B, S_Q, H, d = q.shape
    S_KV, H_kv = k.shape[1], k.shape[2]
    n = o_parts.shape[0]
    _check(lib().lvx_attn_fwd_partials(_ptr(q), _ptr(k), _ptr(v), _ptr(o_parts), _ptr(l_parts), B, H,
                                       H_kv, S_Q, S_KV, d, n, int(bool(causal)), _dt(q), float(scale),
                                       _stream(stream)), "lvx_attn_fwd_partials")


def lvx_merge_partials(o_parts, l_parts, out, lse, stream=None) -> None:
    """o_parts [n,B,H,S_Q,d] fp32, l_parts [n,B,H,S_Q] fp32 -> out [B,S_Q,H,d], lse [B,H,S_Q]."""
    n, B, H, S_Q, d = o_parts.shape
    _check(lib().lvx_merge_partials(_ptr(o_parts), _ptr(l_parts), _ptr(out), _ptr(lse), n, B, H,
                                    S_Q, d, _dt(out), _stream(stream)), "lvx_merge_partials")


def lvx_attn_bwd(q, k, v, out, lse, dout, dq, dk, dv, causal: bool = False, scale: float = 0.0,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    B, S_Q, H, d = q.shape
    S_KV, H_kv = k.shape[1], k.shape[2]
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().lvx_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout),
                              _ptr(dq), _ptr(dk), _ptr(dv), B, H, H_kv, S_Q, S_KV, d,
                              int(causal), _dt(q), float(scale), _ptr(workspace), ws,
                              _stream(stream)), "lvx_attn_bwd")


def lvx_attn_bwd_accumulate(q, k, v, out, lse, dout, dq, dk, dv, causal: bool = False,
                            scale: float = 0.0, workspace: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """As lvx_attn_bwd, with dq, dk, dv float32 arrays the gradients are added to."""
    B, S_Q, H, d = q.shape
    S_KV, H_kv = k.shape[1], k.shape[2]
    for t in (dq, dk, dv):
        if t.dtype != torch.float32:
            raise TypeError("lvx_attn_bwd_accumulate adds into float32 gradients")
    if workspace is None:
        workspace = bwd_workspace(q, k, causal, stream)
    ws = workspace.numel() * workspace.element_size()
    _check(lib().lvx_attn_bwd_accumulate(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                         _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), B, H, H_kv, S_Q,
                                         S_KV, d, int(causal), _dt(q), float(scale),
                                         _ptr(workspace), ws, _stream(stream)),
           "lvx_attn_bwd_accumulate")


def lvx_kv_recompute(y, w_k, w_v, k, v, H_kv: int, d: int, stream=None) -> None:
    """y [B,S_KV,d_embed], w [d_embed, H_kv*d] -> k, v [B,S_KV,H_kv,d]."""
    B, S_KV, d_embed = y.shape
    _check(lib().lvx_kv_recompute(_ptr(y), _ptr(w_k), _ptr(w_v), _ptr(k), _ptr(v), B, S_KV,
                                  d_embed, H_kv, d, _dt(y), _stream(stream)), "lvx_kv_recompute")


def lvx_kv_recompute_bwd(y, w_k, w_v, dk, dv, dy, dw_k, dw_v, stream=None) -> None:
    """y [B,S_KV,d_embed], w [d_embed,H_kv*d], dk/dv [B,S_KV,H_kv,d] ->
    dy like y, dw_k/dw_v like w (dW = y^T dK, dy = dK W_k^T + dV W_v^T)."""
    B, S_KV, d_embed = y.shape
    H_kv, d = dk.shape[2], dk.shape[3]
    _check(lib().lvx_kv_recompute_bwd(_ptr(y), _ptr(w_k), _ptr(w_v), _ptr(dk), _ptr(dv), _ptr(dy),
                                      _ptr(dw_k), _ptr(dw_v), B, S_KV, d_embed, H_kv, d, _dt(y),
                                      _stream(stream)), "lvx_kv_recompute_bwd")


def lvx_attn_fwd_recompute_workspace(B, H, H_kv, S_Q, S_KV, d, d_embed, n_blocks, dtype: int) -> int:
    return lib().lvx_attn_fwd_recompute_workspace(B, H, H_kv, S_Q, S_KV, d, d_embed, n_blocks, dtype)


def lvx_attn_bwd_recompute_workspace(B, H, H_kv, S_Q, S_KV, d, d_embed, n_blocks, dtype: int) -> int:
    return lib().lvx_attn_bwd_recompute_workspace(B, H, H_kv, S_Q, S_KV, d, d_embed, n_blocks, dtype)


def lvx_attn_fwd_recompute(q, y, w_k, w_v, out, lse, H_kv: int, n_blocks: int, scale: float = 0.0,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """q [B,S_Q,H,d], y [B,S_KV,d_embed], w [d_embed,H_kv*d] -> out like q,
    lse [B,H,S_Q] fp32, with K, V regenerated from y one key block at a time."""
    B, S_Q, H, d = q.shape
    S_KV, d_embed = y.shape[1], y.shape[2]
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().lvx_attn_fwd_recompute(_ptr(q), _ptr(y), _ptr(w_k), _ptr(w_v), _ptr(out), _ptr(lse),
                                        B, H, H_kv, S_Q, S_KV, d, d_embed, n_blocks, _dt(q),
                                        float(scale), _ptr(workspace), ws, _stream(stream)),
           "lvx_attn_fwd_recompute")


def lvx_attn_bwd_recompute(q, y, w_k, w_v, out, lse, dout, dq, dy, dw_k, dw_v, H_kv: int,
                           n_blocks: int, scale: float = 0.0,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of attention(q, y W_k, y W_v): dq like q, dy like y (bf16), dw_k,
    dw_v [d_embed, H_kv*d] float32, with K, V regenerated one key block at a time."""
    B, S_Q, H, d = q.shape
    S_KV, d_embed = y.shape[1], y.shape[2]
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().lvx_attn_bwd_recompute(_ptr(q), _ptr(y), _ptr(w_k), _ptr(w_v), _ptr(out), _ptr(lse),
                                        _ptr(dout), _ptr(dq), _ptr(dy), _ptr(dw_k), _ptr(dw_v), B, H,
                                        H_kv, S_Q, S_KV, d, d_embed, n_blocks, _dt(q), float(scale),
                                        _ptr(workspace), ws, _stream(stream)),
           "lvx_attn_bwd_recompute")


def _device(t: torch.Tensor) -> int:
    """Index of t's GPU.  (The calls below are made once a layer and token: their checks are written for
    the fewest tensor attributes, each of which costs 0.1 us; a device object costs more.)"""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be contiguous CUDA tensors")
    return dev


def _launch(name: str, dev: int, stream, *args) -> None:
    """Calls the entry point `name` with its arguments and a stream of GPU `dev`, which becomes the
    current device for the call."""
    if stream is None:   # current_stream(dev).cuda_stream without the Stream object (2 us)
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    fn = getattr(_lib or lib(), name)
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status != 0:
        raise LvxError(status, name)


def _on(stream, dev):
    """Makes `stream` (a Stream or a raw handle; None: the current one as it is) the current stream."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    return torch.cuda.stream(stream)


def _scratch(nbytes: int, dev, stream) -> torch.Tensor:
    """A workspace for launches on `stream` (None: the current one), from the memory of that stream: what is
    given the same memory once the workspace is dropped comes after the launches."""
    with _on(stream, dev):
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def _few(*sizes) -> None:
    """Sizes that the C entry points take as int."""
    if max(sizes) > 0x7fffffff:
        raise ValueError("sizes of 2^31 or more")


def _dense(t, shape, dtype, dev: int, name: str) -> Optional[int]:
    """Pointer of a contiguous tensor of that shape, dtype and GPU."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: not a contiguous tensor on cuda:{dev}")
    return t.data_ptr()


def _strided(t, shape, dtype, dev: int, name: str) -> int:
    """Elements between the tokens of t, a tensor [B, S, heads, d] of that shape, dtype and GPU: heads
    dense, tokens at one stride."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, not {dtype}")
    if t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name}: {tuple(t.shape)} on {t.device}, not {tuple(shape)} on cuda:{dev}")
    B, S, heads, d = shape
    sb, ss, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (heads > 1 and sh != d) or (B > 1 and S > 1 and sb != S * ss):
        raise ValueError(f"{name}: heads must be dense and tokens evenly spaced")
    return ss if S > 1 else sb if B > 1 else heads * d


def _ref(q, k):
    """(B, S, d, dtype, GPU) of queries and keys, one of which may be None."""
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("queries and keys are both None")
    _dt(ref)
    shape = ref.shape
    if len(shape) != 4:
        raise ValueError("queries and keys must be [B, S, heads, d]")
    return shape[0], shape[1], shape[3], ref.dtype, _device(ref)


def _side(ref, names, x, *others):
    """(heads, [pointer, token stride] of each of x and the others, which have its shape); of a side that
    is not there, zeros."""
    if x is None:
        return 0, [None, 0] * (1 + len(others))
    B, S, d, dtype, dev = ref
    shape = x.shape
    if len(shape) != 4 or shape[0] != B or shape[1] != S or shape[3] != d:
        raise ValueError(f"{names[0]}: shape {tuple(shape)}, not [{B}, {S}, heads, {d}]")
    heads = shape[2]
    at = []
    for t in (x, *others):
        if t is None:
            raise ValueError(f"{names[len(at) // 2]} is None")
        at.append(t.data_ptr())
        if t.is_contiguous() and t.dtype is dtype and t.get_device() == dev and t.shape == shape:
            at.append(heads * d)
        else:
            at.append(_strided(t, shape, dtype, dev, names[len(at) // 2]))
    return heads, at


def _turns(ref, pos, inv_freq, axis_of):
    """(pointers of pos, inv_freq, axis_of; n_axes, n_freq), or none of them."""
    if pos is None:
        return None, None, None, 0, 0
    if inv_freq is None or axis_of is None:
        raise TypeError("pos and axis_of must be int32, inv_freq float32")
    B, S, _, _, dev = ref
    shape, n = pos.shape, inv_freq.shape
    if len(shape) != 3 or len(n) != 1:
        raise ValueError("pos must be [n_axes, B, S], inv_freq and axis_of [n_freq]")
    return (_dense(pos, (shape[0], B, S), torch.int32, dev, "pos"),
            _dense(inv_freq, n, torch.float32, dev, "inv_freq"),
            _dense(axis_of, n, torch.int32, dev, "axis_of"), shape[0], n[0])


def _weight(w, ref, name: str):
    return None if w is None else _dense(w, (ref[2],), ref[3], ref[4], name)


def lvx_rope_axes(q, k, pos, inv_freq, axis_of, q_out, k_out, adjacent: bool = False,
                  inverse: bool = False, stream=None) -> None:
    """Rotary positions with several axes: q [B,S,H,d], k [B,S,H_kv,d] (either may be None, with its
    output), pos [n_axes,B,S] int32, inv_freq [n_freq] fp32, axis_of [n_freq] int32.  Tensors may be
    slices of one projection; q_out, k_out may be q, k.  inverse: the gradient of the rotation."""
    ref = B, S, d, dtype, dev = _ref(q, k)
    _few(B * S)
    pp, pi, pa, n_axes, n_freq = _turns(ref, pos, inv_freq, axis_of)
    H, (q_, qs, qo_, qos) = _side(ref, ("q", "q_out"), q, q_out)
    H_kv, (k_, ks, ko_, kos) = _side(ref, ("k", "k_out"), k, k_out)
    _launch("lvx_rope_axes", dev, stream, q_, k_, qo_, ko_, pp, pi, pa, B * S, H, H_kv, d, n_axes,
            n_freq, 1 if adjacent else 0, 1 if inverse else 0, qs, ks, qos, kos,
            LVX_BF16 if dtype is torch.bfloat16 else LVX_FP32)


def lvx_head_norm_rope(q, k, w_q, w_k, q_out, k_out, pos=None, inv_freq=None, axis_of=None,
                       eps: float = 1e-6, adjacent: bool = False, stream=None) -> None:
    """The RMS norm of every head of q and k (weights [d] or None), then the rotation of
    lvx_rope_axes (left out when pos is None), in one pass."""
    ref = B, S, d, dtype, dev = _ref(q, k)
    _few(B * S)
    pp, pi, pa, n_axes, n_freq = _turns(ref, pos, inv_freq, axis_of)
    H, (q_, qs, qo_, qos) = _side(ref, ("q", "q_out"), q, q_out)
    H_kv, (k_, ks, ko_, kos) = _side(ref, ("k", "k_out"), k, k_out)
    _launch("lvx_head_norm_rope", dev, stream, q_, k_, _weight(w_q, ref, "w_q"),
            _weight(w_k, ref, "w_k"), qo_, ko_, pp, pi, pa, B * S, H, H_kv, d, n_axes, n_freq,
            1 if adjacent else 0, eps, qs, ks, qos, kos,
            LVX_BF16 if dtype is torch.bfloat16 else LVX_FP32)


def lvx_head_norm_rope_bwd_workspace(d: int) -> int:
    return lib().lvx_head_norm_rope_bwd_workspace(d)


def lvx_head_norm_rope_bwd(q, k, w_q, w_k, dq_out, dk_out, dq, dk, dw_q, dw_k, pos=None,
                           inv_freq=None, axis_of=None, eps: float = 1e-6, adjacent: bool = False,
                           workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gradients of lvx_head_norm_rope from its inputs and dq_out, dk_out: dq, dk like q, k (they may
    be dq_out, dk_out), dw_q, dw_k [d] float32 (or None)."""
    ref = B, S, d, dtype, dev = _ref(q, k)
    _few(B * S)
    pp, pi, pa, n_axes, n_freq = _turns(ref, pos, inv_freq, axis_of)
    H, (q_, qs, gq_, gqs, dq_, dqs) = _side(ref, ("q", "dq_out", "dq"), q, dq_out, dq)
    H_kv, (k_, ks, gk_, gks, dk_, dks) = _side(ref, ("k", "dk_out", "dk"), k, dk_out, dk)
    wq_ = None if dw_q is None else _dense(dw_q, (d,), torch.float32, dev, "dw_q")
    wk_ = None if dw_k is None else _dense(dw_k, (d,), torch.float32, dev, "dw_k")
    if workspace is None:
        workspace = _scratch(lvx_head_norm_rope_bwd_workspace(d), dev, stream)
    elif workspace.get_device() != dev:
        raise ValueError(f"workspace is on {workspace.device}, not on cuda:{dev}")
    _launch("lvx_head_norm_rope_bwd", dev, stream, q_, k_, _weight(w_q, ref, "w_q"),
            _weight(w_k, ref, "w_k"), gq_, gk_, dq_, dk_, wq_, wk_, pp, pi, pa, B * S, H, H_kv, d,
            n_axes, n_freq, 1 if adjacent else 0, eps, qs, ks, gqs, gks, dqs, dks,
            LVX_BF16 if dtype is torch.bfloat16 else LVX_FP32, _ptr(workspace),
            workspace.numel() * workspace.element_size())


def lvx_attn_prefix_workspace(B, H, H_kv, S_Q, S_P, S_cap, d, dtype: int) -> int:
    return lib().lvx_attn_prefix_workspace(B, H, H_kv, S_Q, S_P, S_cap, d, dtype)


def lvx_attn_prefix(q, k_prefix, v_prefix, k_suffix, v_suffix, suffix_len, out, lse,
                    scale: float = 0.0, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """q [B,S_Q,H,d], a shared prefix k/v [S_P,H_kv,d], suffix caches k/v [B,S_cap,H_kv,d] of which
    suffix_len [B] int32 keys are valid (either pair may be None) -> out like q, lse [B,H,S_Q] fp32.
    A workspace that the call takes itself belongs to `stream`."""
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [B, S_Q, H, d]")
    B, S_Q, H, d = shape
    dtype, dev, dt = q.dtype, q.get_device(), _dt(q)
    some = k_prefix if k_prefix is not None else k_suffix
    if some is None:
        raise ValueError("neither a prefix nor a suffix")
    if some.dim() < 3:
        raise ValueError("k_prefix must be [S_P, H_kv, d], k_suffix [B, S_cap, H_kv, d]")
    H_kv, S_P, S_cap = some.shape[-2], 0, 0
    kp_ = vp_ = ks_ = vs_ = n_ = None
    if k_prefix is not None:
        S_P = k_prefix.shape[0]
        kp_ = _dense(k_prefix, (S_P, H_kv, d), dtype, dev, "k_prefix")
        if S_P > 0 and v_prefix is None:
            raise ValueError("v_prefix is None")
    if v_prefix is not None:
        vp_ = _dense(v_prefix, (S_P, H_kv, d), dtype, dev, "v_prefix")
    if k_suffix is not None:
        S_cap = k_suffix.shape[1]
        ks_ = _dense(k_suffix, (B, S_cap, H_kv, d), dtype, dev, "k_suffix")
        if S_cap > 0 and v_suffix is None:
            raise ValueError("v_suffix is None")
        if S_cap > 0 and suffix_len is None:
            raise TypeError(f"suffix_len must be [{B}] int32")
    if v_suffix is not None:
        vs_ = _dense(v_suffix, (B, S_cap, H_kv, d), dtype, dev, "v_suffix")
    if S_cap > 0:
        n_ = _dense(suffix_len, (B,), torch.int32, dev, "suffix_len")
    _few(B, S_Q, H, S_P, S_cap)
    q_, out_ = _dense(q, shape, dtype, _device(q), "q"), _dense(out, shape, dtype, dev, "out")
    lse_ = _dense(lse, (B, H, S_Q), torch.float32, dev, "lse")
    if workspace is None:
        workspace = prefix_workspace(q, H_kv, S_P, S_cap, stream)
    elif workspace.get_device() != dev:
        raise ValueError(f"workspace is on {workspace.device}, not on cuda:{dev}")
    _launch("lvx_attn_prefix", dev, stream, q_, kp_, vp_, ks_, vs_, n_, out_, lse_, B, H, H_kv, S_Q,
            S_P, S_cap, d, dt, scale, _ptr(workspace), workspace.numel() * workspace.element_size())


def lvx_last_device_error(stream=None) -> None:
    _check(lib().lvx_last_device_error(_stream(stream)), "lvx_last_device_error")


def lvx_selftest_wait_timeout(stream=None) -> None:
    _check(lib().lvx_selftest_wait_timeout(_stream(stream)), "lvx_selftest_wait_timeout")


def lvx_selftest_prefix_plan(B, H, H_kv, S_Q, S_P, S_cap, d, dtype: int) -> dict:
    """How lvx_attn_prefix takes a problem of these sizes: the kernels ("rows", "tc" or "fp32") of the
    prefix's and the suffixes' parts, the parts and their keys, and whether it takes requests whole."""
    plan = (_c_int * 7)()
    _check(lib().lvx_selftest_prefix_plan(B, H, H_kv, S_Q, S_P, S_cap, d, dtype, plan), "lvx_selftest_prefix_plan")
    kernels = ("rows", "tc", "fp32")
    return {"prefix": kernels[plan[0]], "suffix": kernels[plan[1]], "n_pre": plan[2], "pre_len": plan[3],
            "n_suf": plan[4], "suf_len": plan[5], "whole": bool(plan[6])}


# ------------------------------------------------------------------ conveniences

def fwd_workspace(q, k, n_blocks: int, causal: bool = False) -> Optional[torch.Tensor]:
    B, S_Q, H, d = q.shape
    S_KV, H_kv = k.shape[1], k.shape[2]
    nbytes = lvx_attn_fwd_workspace(B, H, H_kv, S_Q, S_KV, d, n_blocks, causal, _dt(q))
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=q.device)


def bwd_workspace(q, k, causal: bool = False, stream=None) -> torch.Tensor:
    B, S_Q, H, d = q.shape
    S_KV, H_kv = k.shape[1], k.shape[2]
    nbytes = lvx_attn_bwd_workspace(B, H, H_kv, S_Q, S_KV, d, causal, _dt(q))
    return _scratch(nbytes, q.device, stream)


def fwd_partials_view(workspace: torch.Tensor, n, B, H, S_Q, d):
    """(O_parts [n,B,H,S_Q,d], L_parts [n,B,H,S_Q]) views of a forward workspace."""
    o_bytes = (n * B * H * S_Q * d * 4 + 255) // 256 * 256
    O = workspace[: n * B * H * S_Q * d * 4].view(torch.float32).view(n, B, H, S_Q, d)
    L = workspace[o_bytes: o_bytes + n * B * H * S_Q * 4].view(torch.float32).view(n, B, H, S_Q)
    return O, L


def attention_forward(q, k, v, n_blocks: int, causal: bool = False, scale: float = 0.0):
    """Allocates outputs and workspace, runs lvx_attn_fwd, returns (out, lse)."""
    B, S_Q, H, d = q.shape
    out = torch.empty_like(q)
    lse = torch.empty(B, H, S_Q, dtype=torch.float32, device=q.device)
    ws = fwd_workspace(q, k, n_blocks, causal)
    lvx_attn_fwd(q, k, v, out, lse, n_blocks, causal, scale, ws)
    return out, lse


def kv_recompute_backward(y, w_k, w_v, dk, dv):
    """Allocates dy, dw_k, dw_v and runs lvx_kv_recompute_bwd; returns them."""
    dy = torch.empty_like(y); dw_k = torch.empty_like(w_k); dw_v = torch.empty_like(w_v)
    lvx_kv_recompute_bwd(y, w_k, w_v, dk, dv, dy, dw_k, dw_v)
    return dy, dw_k, dw_v


def recompute_workspaces(q, y, H_kv: int, n_blocks: int):
    """(forward, backward) workspaces of the recomputing entry points."""
    B, S_Q, H, d = q.shape
    S_KV, d_embed = y.shape[1], y.shape[2]
    f = lvx_attn_fwd_recompute_workspace(B, H, H_kv, S_Q, S_KV, d, d_embed, n_blocks, _dt(q))
    b = lvx_attn_bwd_recompute_workspace(B, H, H_kv, S_Q, S_KV, d, d_embed, n_blocks, _dt(q))
    if f == 0 or b == 0:
        raise LvxError(2, "recompute_workspaces: unsupported shape or dtype")
    return (torch.empty(f, dtype=torch.uint8, device=q.device),
            torch.empty(b, dtype=torch.uint8, device=q.device))


def attention_backward(q, k, v, out, lse, dout, causal: bool = False, scale: float = 0.0):
    dq = torch.empty_like(q); dk = torch.empty_like(k); dv = torch.empty_like(v)
    ws = bwd_workspace(q, k, causal)
    lvx_attn_bwd(q, k, v, out, lse, dout, dq, dk, dv, causal, scale, ws)
    return dq, dk, dv


_calls = None


def _load_calls():
    """The extension that makes the allocating calls below for arguments in order (csrc/host/lvx_calls.cpp);
    it returns NotImplemented for the others, which the Python functions check and refuse."""
    global _calls
    path = os.path.join(_HERE, "_calls.so")
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m blockwise_long_context_b200.build`")
    from . import _calls as m
    m.use(*(ctypes.cast(getattr(lib(), n), ctypes.c_void_p).value for n in (
        "lvx_rope_axes", "lvx_head_norm_rope", "lvx_head_norm_rope_bwd", "lvx_head_norm_rope_bwd_workspace",
        "lvx_attn_prefix", "lvx_attn_prefix_workspace")))
    _calls = m
    return m


def _like(t):
    return None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)


def rope_axes(q, k, pos, inv_freq, axis_of, adjacent: bool = False, inverse: bool = False):
    """Allocates the outputs, runs lvx_rope_axes, returns (q_out, k_out)."""
    made = (_calls or _load_calls()).rope_axes(q, k, pos, inv_freq, axis_of, adjacent, inverse)
    if made is not NotImplemented:
        return made
    q_out, k_out = _like(q), _like(k)
    lvx_rope_axes(q, k, pos, inv_freq, axis_of, q_out, k_out, adjacent, inverse)
    return q_out, k_out


def head_norm_rope(q, k, w_q, w_k, pos=None, inv_freq=None, axis_of=None, eps: float = 1e-6,
                   adjacent: bool = False):
    """Allocates the outputs, runs lvx_head_norm_rope, returns (q_out, k_out)."""
    made = (_calls or _load_calls()).head_norm_rope(q, k, w_q, w_k, pos, inv_freq, axis_of, eps, adjacent)
    if made is not NotImplemented:
        return made
    q_out, k_out = _like(q), _like(k)
    lvx_head_norm_rope(q, k, w_q, w_k, q_out, k_out, pos, inv_freq, axis_of, eps, adjacent)
    return q_out, k_out


def head_norm_rope_backward(q, k, w_q, w_k, dq_out, dk_out, pos=None, inv_freq=None, axis_of=None,
                            eps: float = 1e-6, adjacent: bool = False):
    """Allocates dq, dk and the float32 weight gradients, runs lvx_head_norm_rope_bwd, returns
    (dq, dk, dw_q, dw_k); a side that is None has None gradients, and so has a weight that is None."""
    made = (_calls or _load_calls()).head_norm_rope_backward(q, k, w_q, w_k, dq_out, dk_out, pos, inv_freq,
                                                             axis_of, eps, adjacent)
    if made is not NotImplemented:
        return made
    dq, dk = _like(q), _like(k)
    dw_q, dw_k = (None if t is None or w is None else
                  torch.empty(t.shape[-1], dtype=torch.float32, device=t.device)
                  for t, w in ((q, w_q), (k, w_k)))
    lvx_head_norm_rope_bwd(q, k, w_q, w_k, dq_out, dk_out, dq, dk, dw_q, dw_k, pos, inv_freq, axis_of,
                           eps, adjacent)
    return dq, dk, dw_q, dw_k


def prefix_workspace(q, H_kv: int, S_P: int, S_cap: int, stream=None) -> torch.Tensor:
    """The workspace of lvx_attn_prefix for queries like q, for calls on `stream` (None: the current one)."""
    if not q.is_cuda:
        raise ValueError("tensors must be contiguous CUDA tensors")
    B, S_Q, H, d = q.shape
    nbytes = lvx_attn_prefix_workspace(B, H, H_kv, S_Q, S_P, S_cap, d, _dt(q))
    if nbytes == 0:
        raise LvxError(2, "prefix_workspace: invalid or unsupported shape")
    return _scratch(nbytes, q.get_device(), stream)


def attention_prefix(q, k_prefix, v_prefix, k_suffix=None, v_suffix=None, suffix_len=None,
                     scale: float = 0.0):
    """Allocates outputs and workspace, runs lvx_attn_prefix, returns (out, lse)."""
    made = (_calls or _load_calls()).attention_prefix(q, k_prefix, v_prefix, k_suffix, v_suffix, suffix_len, scale)
    if made is not NotImplemented:
        return made
    B, S_Q, H, d = q.shape
    out = torch.empty_like(q)
    lse = torch.empty(B, H, S_Q, dtype=torch.float32, device=q.device)
    lvx_attn_prefix(q, k_prefix, v_prefix, k_suffix, v_suffix, suffix_len, out, lse, scale)
    return out, lse
