"""Thin ctypes binding of libhstu_attn.so (C ABI in include/hstu_attn.h).

Argument marshalling only: tensors become raw device pointers plus the current CUDA
stream; every step of the computation runs in the library's kernels.  There is no CPU
path: without the built library, or with tensors not on a CUDA device, calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import NamedTuple, Optional

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhstu_attn.so")

HSTU_F32, HSTU_BF16 = 0, 1
STATUS_NAMES = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace too small",
                4: "CUDA error", 5: "invalid device data"}
DEV_BAD_OFFSETS, DEV_BAD_COUNTS, DEV_SEQ_TOO_LONG, DEV_WAIT_TIMEOUT = 0x1, 0x2, 0x4, 0x8
DEV_BAD_EXPERT = 0x10

EXPORTED = ["hstu_attn_fwd_workspace_size", "hstu_attn_fwd", "hstu_attn_bwd_workspace_size",
            "hstu_attn_bwd", "hstu_attn_read_device_status", "hstu_attn_debug_mask",
            "hstu_attn_debug_kernel_mask", "hstu_attn_set_wait_test",
            "hstu_stochastic_length", "hstu_gather_rows", "hstu_jagged_concat",
            "hstu_layer_norm_rows", "hstu_uvqk_proj", "hstu_out_proj",
            "hstu_rms_norm_rows", "hstu_rms_norm_rows_e4m3",
            "hstu_rms_norm_rows_bwd_workspace_size", "hstu_rms_norm_rows_bwd",
            "hstu_expert_sort_workspace_size", "hstu_expert_sort", "hstu_expert_dispatch",
            "hstu_expert_combine", "hstu_expert_combine_bwd", "hstu_expert_proj",
            "hstu_expert_proj_e4m3", "hstu_expert_proj_bwd",
            "hstu_expert_proj_bwd_workspace_size",
            "hstu_attn_time_thresholds", "hstu_attn_set_stage_events", "hstu_status_string",
            "hstu_attn_version"]
STAGES = {"fwd_attn": 0, "fwd_norm": 1, "bwd_norm": 2, "bwd_attn": 3}


class HstuError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s failed: %s (status %d)" % (what, STATUS_NAMES.get(status, "?"), status))
        self.status = status


class Params(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("d_qk", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("max_seqlen", ctypes.c_int32), ("max_attn_len", ctypes.c_int32),
                ("total_tokens", ctypes.c_int64), ("alpha", ctypes.c_float),
                ("ln_eps", ctypes.c_float), ("rel_bias_len", ctypes.c_int32),
                ("time_bias_len", ctypes.c_int32), ("time_bucket_div", ctypes.c_double),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]

# mask variants (Params.flags)
FLAG_CTX_SEES_HISTORY, FLAG_REL_ABS, FLAG_CANDIDATES_ONLY = 0x1, 0x2, 0x4


_lib = None
_VP = ctypes.c_void_p


def lib():
    """Load libhstu_attn.so (build it with `python -m jagged_hstu_attention_02_b200.build`)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libhstu_attn.so is not built (%s); run "
                               "`python -m jagged_hstu_attention_02_b200.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(Params)
        sz = ctypes.POINTER(ctypes.c_size_t)
        L.hstu_attn_fwd_workspace_size.argtypes = [P, sz]
        L.hstu_attn_bwd_workspace_size.argtypes = [P, sz]
        L.hstu_attn_fwd.argtypes = [P] + [_VP] * 15 + [ctypes.c_size_t, _VP]
        L.hstu_attn_bwd.argtypes = [P] + [_VP] * 21 + [ctypes.c_size_t, _VP]
        L.hstu_attn_read_device_status.argtypes = [_VP, _VP, ctypes.POINTER(ctypes.c_int32)]
        L.hstu_attn_debug_mask.argtypes = [P, _VP, _VP, _VP, ctypes.c_int32, ctypes.c_int32, _VP,
                                           _VP]
        L.hstu_attn_debug_kernel_mask.argtypes = [P, _VP, _VP, _VP] + [ctypes.c_int32] * 5 + [
            _VP, _VP]
        L.hstu_attn_time_thresholds.argtypes = [ctypes.c_double, ctypes.c_int32,
                                                ctypes.POINTER(ctypes.c_uint64)]
        L.hstu_attn_set_stage_events.argtypes = [ctypes.c_int32, _VP, _VP]
        L.hstu_attn_set_wait_test.argtypes = [ctypes.c_int64, ctypes.c_int32]
        L.hstu_stochastic_length.argtypes = [_VP, _VP, _VP, ctypes.c_int32, ctypes.c_int64, _VP,
                                             ctypes.c_int32, _VP, _VP, _VP, _VP]
        L.hstu_layer_norm_rows.argtypes = [_VP, _VP, ctypes.c_int64, ctypes.c_int32,
                                           ctypes.c_float, _VP]
        L.hstu_uvqk_proj.argtypes = [_VP, _VP, _VP, ctypes.c_int64] + [ctypes.c_int32] * 5 + \
            [_VP] * 6
        L.hstu_out_proj.argtypes = [_VP, _VP, _VP, _VP, ctypes.c_int64, ctypes.c_int32,
                                    ctypes.c_int32, _VP, _VP, _VP]
        L.hstu_gather_rows.argtypes = [_VP, ctypes.c_int64, _VP, _VP, ctypes.c_int64, _VP, _VP]
        L.hstu_jagged_concat.argtypes = [ctypes.c_int32, ctypes.POINTER(_VP),
                                         ctypes.POINTER(_VP), ctypes.c_int32, ctypes.c_int64,
                                         _VP, _VP, _VP]
        i32, i64, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        L.hstu_rms_norm_rows.argtypes = [_VP] * 3 + [i64, i32, f32, i32] + [_VP] * 4
        L.hstu_rms_norm_rows_e4m3.argtypes = [_VP] * 3 + [i64, i32, f32, i32, i32] + [_VP] * 5
        L.hstu_rms_norm_rows_bwd_workspace_size.argtypes = [i64, i32, sz]
        L.hstu_rms_norm_rows_bwd.argtypes = [_VP] * 5 + [i64, i32, i32] + [_VP] * 3 + [
            ctypes.c_size_t, _VP]
        L.hstu_expert_sort_workspace_size.argtypes = [i64, i32, i32, sz]
        L.hstu_expert_sort.argtypes = [_VP, i32, i64, i32, i32] + [_VP] * 5 + [ctypes.c_size_t,
                                                                              _VP]
        L.hstu_expert_dispatch.argtypes = [_VP, i64, _VP, i32, _VP, i64, i32, i64] + [_VP] * 3
        L.hstu_expert_combine.argtypes = [_VP] * 4 + [i64, i32, i64, i32, i32] + [_VP] * 2
        L.hstu_expert_combine_bwd.argtypes = [_VP] * 4 + [i64, i32, i64, i32, i32] + [_VP] * 3
        L.hstu_expert_proj.argtypes = [_VP] * 3 + [i64, i32, i32, i32, i32] + [_VP] * 4
        L.hstu_expert_proj_e4m3.argtypes = [_VP] * 5 + [i64, i32, i32, i32, i32] + [_VP] * 3
        L.hstu_expert_proj_bwd.argtypes = [_VP] * 5 + [i64, i32, i32, i32] + [_VP] * 4 + [
            ctypes.c_size_t, _VP]
        L.hstu_expert_proj_bwd_workspace_size.argtypes = [i64, i32, i32, i32, sz]
        L.hstu_status_string.restype = ctypes.c_char_p
        L.hstu_status_string.argtypes = [ctypes.c_int]
        L.hstu_attn_version.restype = ctypes.c_int32
        for name in EXPORTED:
            f = getattr(L, name)
            if name not in ("hstu_status_string", "hstu_attn_version"):
                f.restype = ctypes.c_int
        _lib = L
    return _lib


def _check(status: int, what: str):
    if status != 0:
        raise HstuError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return HSTU_F32
    if t.dtype == torch.bfloat16:
        return HSTU_BF16
    raise ValueError("unsupported dtype %s" % t.dtype)


def make_params(q, v, seq_offsets, *, alpha, max_seqlen, max_attn_len=0, rel_bias=None,
                time_bias=None, time_bucket_div=0.301, ln_eps=1e-5, mask_flags=0) -> Params:
    T, H, dqk = q.shape
    return Params(batch=seq_offsets.numel() - 1, num_heads=H, d_qk=dqk, d_v=v.shape[2],
                  max_seqlen=int(max_seqlen), max_attn_len=int(max_attn_len), total_tokens=T,
                  alpha=float(alpha), ln_eps=float(ln_eps),
                  rel_bias_len=0 if rel_bias is None else rel_bias.numel(),
                  time_bias_len=0 if time_bias is None else time_bias.numel(),
                  time_bucket_div=float(time_bucket_div), dtype=dtype_code(q),
                  flags=int(mask_flags))


def fwd_workspace_size(params: Params) -> int:
    n = ctypes.c_size_t()
    _check(lib().hstu_attn_fwd_workspace_size(ctypes.byref(params), ctypes.byref(n)),
           "hstu_attn_fwd_workspace_size")
    return n.value


def bwd_workspace_size(params: Params) -> int:
    n = ctypes.c_size_t()
    _check(lib().hstu_attn_bwd_workspace_size(ctypes.byref(params), ctypes.byref(n)),
           "hstu_attn_bwd_workspace_size")
    return n.value


@dataclass
class Saved:
    y: torch.Tensor
    mean: torch.Tensor
    rstd: torch.Tensor


def fwd(q, k, v, u, seq_offsets, num_contextuals=None, num_targets=None, timestamps=None,
        rel_bias=None, time_bias=None, *, alpha, max_seqlen, max_attn_len=0,
        time_bucket_div=0.301, ln_eps=1e-5, mask_flags=0, training=False, out=None,
        workspace=None, saved: Optional[Saved] = None, stream=None):
    """out [T, H*d_v] (and Saved(y, mean, rstd) when training)."""
    p = make_params(q, v, seq_offsets, alpha=alpha, max_seqlen=max_seqlen,
                    max_attn_len=max_attn_len, rel_bias=rel_bias, time_bias=time_bias,
                    time_bucket_div=time_bucket_div, ln_eps=ln_eps, mask_flags=mask_flags)
    T, H, dv = v.shape
    dev = q.device
    if out is None:
        out = torch.empty((T, H * dv), dtype=q.dtype, device=dev)
    if training and saved is None:
        saved = Saved(torch.empty((T, H * dv), dtype=torch.float32, device=dev),
                      torch.empty(T, dtype=torch.float32, device=dev),
                      torch.empty(T, dtype=torch.float32, device=dev))
    if workspace is None:
        workspace = torch.empty(fwd_workspace_size(p), dtype=torch.uint8, device=dev)
    st = lib().hstu_attn_fwd(
        ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(u), _ptr(seq_offsets),
        _ptr(num_contextuals), _ptr(num_targets), _ptr(timestamps), _ptr(rel_bias),
        _ptr(time_bias), _ptr(out), _ptr(saved.y if training else None),
        _ptr(saved.mean if training else None), _ptr(saved.rstd if training else None),
        _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "hstu_attn_fwd")
    fwd.last_workspace = workspace
    return (out, saved) if training else out


def bwd(dout, q, k, v, u, seq_offsets, num_contextuals=None, num_targets=None, timestamps=None,
        rel_bias=None, time_bias=None, *, saved: Saved, alpha, max_seqlen, max_attn_len=0,
        time_bucket_div=0.301, ln_eps=1e-5, mask_flags=0, grads=None, workspace=None,
        stream=None):
    """(dq, dk, dv, du, d_rel_bias or None, d_time_bias or None)."""
    p = make_params(q, v, seq_offsets, alpha=alpha, max_seqlen=max_seqlen,
                    max_attn_len=max_attn_len, rel_bias=rel_bias, time_bias=time_bias,
                    time_bucket_div=time_bucket_div, ln_eps=ln_eps, mask_flags=mask_flags)
    dev = q.device
    if grads is None:
        grads = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v),
                 torch.empty_like(u),
                 None if rel_bias is None else torch.empty_like(rel_bias),
                 None if time_bias is None else torch.empty_like(time_bias))
    dq, dk, dv, du, drel, dtb = grads
    if workspace is None:
        workspace = torch.empty(bwd_workspace_size(p), dtype=torch.uint8, device=dev)
    st = lib().hstu_attn_bwd(
        ctypes.byref(p), _ptr(dout), _ptr(q), _ptr(k), _ptr(v), _ptr(u), _ptr(seq_offsets),
        _ptr(num_contextuals), _ptr(num_targets), _ptr(timestamps), _ptr(rel_bias),
        _ptr(time_bias), _ptr(saved.y), _ptr(saved.mean), _ptr(saved.rstd), _ptr(dq), _ptr(dk),
        _ptr(dv), _ptr(du), _ptr(drel), _ptr(dtb), _ptr(workspace), workspace.numel(),
        _stream(stream))
    _check(st, "hstu_attn_bwd")
    bwd.last_workspace = workspace
    return grads


def read_device_status(workspace: torch.Tensor, stream=None) -> int:
    code = ctypes.c_int32(0)
    st = lib().hstu_attn_read_device_status(_ptr(workspace), _stream(stream), ctypes.byref(code))
    if st not in (0, 5):
        _check(st, "hstu_attn_read_device_status")
    return code.value


def debug_mask(params: Params, seq_offsets, num_contextuals, num_targets, seq: int, seq_len: int,
               stream=None) -> torch.Tensor:
    """[seq_len, seq_len] bool mask of sequence `seq` as the device predicate evaluates it."""
    words = (seq_len * seq_len + 31) // 32
    bits = torch.zeros(max(words, 1), dtype=torch.int32, device=seq_offsets.device)
    _check(lib().hstu_attn_debug_mask(ctypes.byref(params), _ptr(seq_offsets),
                                      _ptr(num_contextuals), _ptr(num_targets), seq, seq_len,
                                      _ptr(bits), _stream(stream)), "hstu_attn_debug_mask")
    b = bits.cpu().numpy().view("uint32")
    import numpy as np
    flat = ((b[:, None] >> np.arange(32, dtype=np.uint32)[None, :]) & 1).astype(bool).reshape(-1)
    return torch.from_numpy(flat[:seq_len * seq_len].reshape(seq_len, seq_len).copy())


def debug_kernel_mask(params: Params, seq_offsets, num_contextuals, num_targets, seq: int,
                      kernel: str, row_begin: int, row_count: int, key_count: int,
                      stream=None):
    """[row_count, key_count] bool mask of sequence `seq` as the tensor-core forward
    (kernel "fwd") or backward ("bwd") decides it, rows from row_begin."""
    import numpy as np
    words = row_count * key_count // 32
    bits = torch.zeros(max(words, 1), dtype=torch.int32, device=seq_offsets.device)
    _check(lib().hstu_attn_debug_kernel_mask(
        ctypes.byref(params), _ptr(seq_offsets), _ptr(num_contextuals), _ptr(num_targets), seq,
        {"fwd": 0, "bwd": 1}[kernel], row_begin, row_count, key_count, _ptr(bits),
        _stream(stream)), "hstu_attn_debug_kernel_mask")
    b = bits.cpu().numpy().view("uint32")[:words]
    flat = ((b[:, None] >> np.arange(32, dtype=np.uint32)[None, :]) & 1).astype(bool).reshape(-1)
    return torch.from_numpy(flat.reshape(row_count, key_count).copy())


def time_thresholds(div: float, nb: int):
    """Host-side threshold table the device compares |dt| against (uint64, nb-1 entries)."""
    arr = (ctypes.c_uint64 * max(nb - 1, 1))()
    _check(lib().hstu_attn_time_thresholds(float(div), int(nb), arr), "hstu_attn_time_thresholds")
    return [int(arr[i]) for i in range(nb - 1)]


def set_stage_events(stage: str, start=None, stop=None):
    """Record torch.cuda.Event `start`/`stop` around the kernels of `stage` in every later
    fwd/bwd call (None clears).  The events must stay alive while set."""
    sp = None if start is None else ctypes.c_void_p(start.cuda_event)
    ep = None if stop is None else ctypes.c_void_p(stop.cuda_event)
    _check(lib().hstu_attn_set_stage_events(STAGES[stage], sp, ep), "hstu_attn_set_stage_events")


def set_wait_test(limit_cycles: int = 0, stall: bool = False):
    """Test hook: shorten the kernels' pipeline waits and make one of them run out."""
    _check(lib().hstu_attn_set_wait_test(int(limit_cycles), 1 if stall else 0),
           "hstu_attn_set_wait_test")


# ------------------------------------------------------------------ jagged operations

MAX_CONCAT_PARTS = 16

def stochastic_length(seq_offsets, num_contextuals, num_targets, keys, budget: int,
                      status=None, stream=None):
    """(kept rows [T] int64 (first new_offsets[-1] valid), new offsets [B+1] int64)."""
    T = int(keys.numel())
    B = seq_offsets.numel() - 1
    rows = torch.empty(max(T, 1), dtype=torch.int64, device=seq_offsets.device)
    offs = torch.empty(B + 1, dtype=torch.int64, device=seq_offsets.device)
    _check(lib().hstu_stochastic_length(_ptr(seq_offsets), _ptr(num_contextuals),
                                        _ptr(num_targets), B, T, _ptr(keys), int(budget),
                                        _ptr(rows), _ptr(offs), _ptr(status), _stream(stream)),
           "hstu_stochastic_length")
    return rows, offs


def gather_rows(src, rows, n_rows, max_rows: int, out=None, stream=None):
    """out[r] = src[rows[r]] for r < n_rows (a device scalar tensor), up to max_rows rows."""
    if out is None:
        out = torch.empty((max_rows,) + tuple(src.shape[1:]), dtype=src.dtype, device=src.device)
    row_bytes = src[0].numel() * src.element_size() if src.numel() else 1
    _check(lib().hstu_gather_rows(_ptr(src), row_bytes, _ptr(rows), _ptr(n_rows), int(max_rows),
                                  _ptr(out), _stream(stream)), "hstu_gather_rows")
    return out


def jagged_concat(parts, out=None, stream=None):
    """parts: list of (values [T_q, ...], offsets [B+1]); (values, offsets) of the per-sequence
    concatenation."""
    vals0, offs0 = parts[0]
    B = offs0.numel() - 1
    total = sum(int(v.shape[0]) for v, _ in parts)
    if out is None:
        out = torch.empty((total,) + tuple(vals0.shape[1:]), dtype=vals0.dtype,
                          device=vals0.device)
    out_offs = torch.empty(B + 1, dtype=torch.int64, device=offs0.device)
    n = len(parts)
    V = (_VP * n)(*[_ptr(v) for v, _ in parts])
    O = (_VP * n)(*[_ptr(o) for _, o in parts])
    row_bytes = vals0[0].numel() * vals0.element_size() if vals0.numel() else \
        int(np.prod(vals0.shape[1:])) * vals0.element_size()
    _check(lib().hstu_jagged_concat(n, V, O, B, row_bytes, _ptr(out), _ptr(out_offs),
                                    _stream(stream)), "hstu_jagged_concat")
    return out, out_offs


# ------------------------------------------------------------------ the layer around the path

def layer_norm_rows(x, eps=1e-5, out=None, stream=None):
    """LayerNorm (no affine) of every row of the bf16 matrix x."""
    if out is None:
        out = torch.empty_like(x)
    _check(lib().hstu_layer_norm_rows(_ptr(x), _ptr(out), x.shape[0], x.shape[1], float(eps),
                                      _stream(stream)), "hstu_layer_norm_rows")
    return out


def uvqk_proj(x, w, bias, num_heads, d_qk, d_v, silu=False, status=None, stream=None):
    """(u [T, H*d_v], v [T,H,d_v], q [T,H,d_qk], k [T,H,d_qk]) of the fused projection."""
    T = x.shape[0]
    dev, dt = x.device, x.dtype
    u = torch.empty((T, num_heads * d_v), dtype=dt, device=dev)
    v = torch.empty((T, num_heads, d_v), dtype=dt, device=dev)
    q = torch.empty((T, num_heads, d_qk), dtype=dt, device=dev)
    k = torch.empty((T, num_heads, d_qk), dtype=dt, device=dev)
    _check(lib().hstu_uvqk_proj(_ptr(x), _ptr(w), _ptr(bias), T, x.shape[1], num_heads, d_qk,
                                d_v, 1 if silu else 0, _ptr(u), _ptr(v), _ptr(q), _ptr(k),
                                _ptr(status), _stream(stream)), "hstu_uvqk_proj")
    return u, v, q, k


def out_proj(z, w_o, bias=None, x=None, status=None, stream=None):
    """z [T, d_in] w_o [d_in, d_model] (+ bias) (+ x): the output projection and residual."""
    T, d_model = z.shape[0], w_o.shape[1]
    out = torch.empty((T, d_model), dtype=z.dtype, device=z.device)
    _check(lib().hstu_out_proj(_ptr(z), _ptr(w_o), _ptr(bias), _ptr(x), T, z.shape[1], d_model,
                               _ptr(out), _ptr(status), _stream(stream)), "hstu_out_proj")
    return out


def layer_fwd(x, seq_offsets, num_contextuals, num_targets, timestamps, rel_bias, time_bias,
              w_uvqk, b_uvqk, w_o, b_o, *, num_heads, d_qk, d_v, alpha, max_seqlen,
              max_attn_len=0, time_bucket_div=0.301, ln_eps=1e-5, mask_flags=0,
              uvqk_silu=False, stream=None):
    """One HSTU layer on jagged tokens x [T, d_model] (bf16): input LayerNorm, fused U/V/Q/K
    projection, attention with LayerNorm and U gating, output projection with bias and the
    residual.  Returns dict(xn, u, v, q, k, attn, o)."""
    xn = layer_norm_rows(x, ln_eps, stream=stream)
    u, v, q, k = uvqk_proj(xn, w_uvqk, b_uvqk, num_heads, d_qk, d_v, silu=uvqk_silu,
                           stream=stream)
    attn = fwd(q, k, v, u, seq_offsets, num_contextuals, num_targets, timestamps, rel_bias,
               time_bias, alpha=alpha, max_seqlen=max_seqlen, max_attn_len=max_attn_len,
               time_bucket_div=time_bucket_div, ln_eps=ln_eps, mask_flags=mask_flags,
               stream=stream)
    o = out_proj(attn, w_o, b_o, x, stream=stream)
    return dict(xn=xn, u=u, v=v, q=q, k=k, attn=attn, o=o)


# ------------------------------------------------------------------ mixture of experts

F8 = torch.float8_e4m3fn
# These calls run for a few microseconds on small batches, so what the host does around them is
# kept short: one check per tensor, which yields its address, and the stream's handle as an integer.
_CODES = {torch.float32: HSTU_F32, torch.bfloat16: HSTU_BF16}
# handle of a device's current stream, and the current device, without the objects and checks
# around them where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _elsewhere(dev, stream):
    """Whether a call on tensors of device `dev` has to change the device or the stream first."""
    return dev >= 0 and (stream is not None or dev != _device())


def _place(dev, stream):
    """Context for `stream` (of device `dev`), or for that device's current stream."""
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device_index != dev:
        raise ValueError("stream and tensors must be on the same device")
    return torch.cuda.stream(stream)


def _on_cuda(dev):
    if dev < 0:
        raise ValueError("tensors must live on a CUDA device")


def _expect(t, name, dtype, shape, dev):
    """Address of an optional tensor, checked for its type, shape, device and layout."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise ValueError("%s must be %s, not %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must be %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    if t.get_device() != dev:
        raise ValueError("%s must be on the other tensors' device" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _expect_32(*sizes):
    """Sizes that the C ABI takes as 32 bits (ctypes would cut larger ones)."""
    if max(sizes) >= 2 ** 31:
        raise ValueError("a size of 2^31 or more: %s" % (sizes,))


def _expect_rows(t, name):
    """(rows, width, dtype code) of a matrix of rows."""
    if t.dim() != 2:
        raise ValueError("%s must be [rows, width]" % name)
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError("unsupported dtype %s" % t.dtype)
    rows, width = t.shape
    if width >= 2 ** 31:
        _expect_32(width)
    return rows, width, code


def _expect_status(status, dev):
    if status is None:
        return None
    if status.numel() < 1:
        raise ValueError("status must hold an int32")
    return _expect(status, "status", torch.int32, status.shape, dev)


@functools.lru_cache(maxsize=1024)
def _workspace_size(name, *sizes):
    """Bytes that the named workspace-size entry point asks for."""
    n = ctypes.c_size_t()
    _check(getattr(lib(), name)(*sizes, ctypes.byref(n)), name)
    return n.value


def _workspace(like, given, size, dev):
    """(address, bytes, tensor) of the workspace: the given one, or a new one of `size` bytes."""
    if given is None:
        if size == 0:
            return None, 0, None
        given = like.new_empty((size,), dtype=torch.uint8)
    return _expect(given, "workspace", given.dtype, given.shape, dev), \
        given.numel() * given.element_size(), given


class RmsNorm(NamedTuple):
    """Results of rms_norm_rows: y (e4m3 with scales, or the rows' type), the stored sum (x
    itself without a residual) and, when training, rstd."""
    y: torch.Tensor
    scales: Optional[torch.Tensor]
    sum: torch.Tensor
    rstd: Optional[torch.Tensor]


def rms_norm_rows(x, weight=None, residual=None, *, eps=1e-5, e4m3=False, group=0,
                  training=False, out: Optional[RmsNorm] = None, stream=None) -> RmsNorm:
    """RMS norm of the rows of h = x (+ residual), times weight (fp32).  e4m3: y in 8 bits with
    one fp32 scale per row (group 0) or per `group` (32, 64, 128) columns, y ~ q * scale.
    training keeps rstd for rms_norm_rows_bwd.  out: a result to write into again; its sum only
    with a residual (the sum of a call without one is that call's x)."""
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return rms_norm_rows(x, weight, residual, eps=eps, e4m3=e4m3, group=group,
                                 training=training, out=out)
    rows, width, code = _expect_rows(x, "x")
    if group not in (0, 32, 64, 128):
        raise ValueError("group must be 0, 32, 64 or 128")
    if group and not e4m3:
        raise ValueError("group is for the e4m3 output")
    shape, dtype = x.shape, x.dtype
    px = _expect(x, "x", dtype, shape, dev)
    pw = _expect(weight, "weight", torch.float32, (width,), dev)
    pr = _expect(residual, "residual", dtype, shape, dev)
    groups = -(-width // group) if group else 1
    _on_cuda(dev)
    if out is None:
        out = RmsNorm(torch.empty_like(x, dtype=F8) if e4m3 else torch.empty_like(x),
                      x.new_empty((rows, groups), dtype=torch.float32) if e4m3 else None,
                      x if residual is None else torch.empty_like(x),
                      x.new_empty((rows,), dtype=torch.float32) if training else None)
        py, psum = out.y.data_ptr(), out.sum.data_ptr()
        psc = out.scales.data_ptr() if e4m3 else None
        pst = out.rstd.data_ptr() if training else None
    else:
        py = _expect(out.y, "out.y", F8 if e4m3 else dtype, shape, dev)
        psc = _expect(out.scales, "out.scales", torch.float32, (rows, groups), dev)
        psum = _expect(out.sum, "out.sum", dtype, shape, dev)
        pst = _expect(out.rstd, "out.rstd", torch.float32, (rows,), dev)
        if (e4m3 and psc is None) or (training and pst is None):
            raise ValueError("out lacks scales or rstd")
        out = RmsNorm(out.y, out.scales if e4m3 else None, x if residual is None else out.sum,
                      out.rstd)
    if residual is None:
        psum = None
    if e4m3:
        st = lib().hstu_rms_norm_rows_e4m3(px, pr, pw, rows, width, eps, code, group, py, psc, psum,
                                           pst, _raw_stream(dev))
    else:
        st = lib().hstu_rms_norm_rows(px, pr, pw, rows, width, eps, code, py, psum, pst,
                                      _raw_stream(dev))
    _check(st, "hstu_rms_norm_rows")
    return out


def rms_norm_rows_bwd(dy, sum, rstd, weight=None, *, dsum=None, grads=None, workspace=None,
                      stream=None):
    """(dx, dweight or None) of rms_norm_rows at its stored sum; dx is the gradient of x and of
    the residual, dsum the gradient that reaches the sum by other ways."""
    dev = dy.get_device()
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return rms_norm_rows_bwd(dy, sum, rstd, weight, dsum=dsum, grads=grads,
                                     workspace=workspace)
    rows, width, code = _expect_rows(dy, "dy")
    shape, dtype = dy.shape, dy.dtype
    pdy = _expect(dy, "dy", dtype, shape, dev)
    ph = _expect(sum, "sum", dtype, shape, dev)
    pst = _expect(rstd, "rstd", torch.float32, (rows,), dev)
    pw = _expect(weight, "weight", torch.float32, (width,), dev)
    pds = _expect(dsum, "dsum", dtype, shape, dev)
    _on_cuda(dev)
    if grads is None:
        grads = (torch.empty_like(dy), None if weight is None else torch.empty_like(weight))
    dx, dw = grads
    pdx = _expect(dx, "dx", dtype, shape, dev)
    pdw = _expect(dw, "dweight", torch.float32, (width,), dev)
    need = 0 if dw is None else _workspace_size("hstu_rms_norm_rows_bwd_workspace_size", rows, width)
    pws, nws, workspace = _workspace(dy, workspace, need, dev)
    _check(lib().hstu_rms_norm_rows_bwd(pdy, ph, pst, pw, pds, rows, width, code, pdx, pdw, pws, nws,
                                        _raw_stream(dev)), "hstu_rms_norm_rows_bwd")
    return grads


class Routing(NamedTuple):
    """Where expert_sort puts the pairs: slots [tokens, choices] (the pair's sorted row, -1 for
    none), offsets [experts + 1] of the sorted rows, rows [tokens * choices] (each sorted row's
    token, as gather_rows takes them; offsets[-1] of them)."""
    slots: torch.Tensor
    offsets: torch.Tensor
    rows: Optional[torch.Tensor]


def expert_sort(expert_ids, num_experts: int, *, status=None, out: Optional[Routing] = None,
                workspace=None, stream=None) -> Routing:
    """Sorts the pairs of expert_ids [tokens, choices] (int32 or int64; negative: no expert) by
    expert, in the order of the pairs within an expert."""
    dev = expert_ids.get_device()
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return expert_sort(expert_ids, num_experts, status=status, out=out,
                               workspace=workspace)
    if expert_ids.dim() != 2:
        raise ValueError("expert_ids must be [tokens, choices]")
    dtype = expert_ids.dtype
    if dtype not in (torch.int32, torch.int64):
        raise ValueError("expert_ids must be int32 or int64")
    T, k = shape = expert_ids.shape
    _expect_32(k, num_experts)
    pid = _expect(expert_ids, "expert_ids", dtype, shape, dev)
    pst = _expect_status(status, dev)
    _on_cuda(dev)
    need = _workspace_size("hstu_expert_sort_workspace_size", T, k, num_experts)
    if out is None:
        out = Routing(expert_ids.new_empty(shape, dtype=torch.int32),
                      expert_ids.new_empty((num_experts + 1,), dtype=torch.int64),
                      expert_ids.new_empty((T * k,), dtype=torch.int64))
    ps = _expect(out.slots, "out.slots", torch.int32, shape, dev)
    po = _expect(out.offsets, "out.offsets", torch.int64, (num_experts + 1,), dev)
    pr = _expect(out.rows, "out.rows", torch.int64, (T * k,), dev)
    pws, nws, workspace = _workspace(expert_ids, workspace, need, dev)
    _check(lib().hstu_expert_sort(pid, 1 if dtype == torch.int64 else 0, T, k, num_experts, ps, po,
                                  pr, pst, pws, nws, _raw_stream(dev)), "hstu_expert_sort")
    return out


def _expect_slots(slots, dev):
    """(tokens, choices, address)."""
    if slots.dim() != 2:
        raise ValueError("slots must be [tokens, choices]")
    T, k = shape = slots.shape
    if k >= 2 ** 31:
        _expect_32(k)
    return T, k, _expect(slots, "slots", torch.int32, shape, dev)


def expert_dispatch(x, slots, *, scales=None, out=None, scales_out=None, stream=None):
    """xs [tokens * choices, ...]: row t of x at every slots[t, j]; with scales (one row of fp32
    per token, e.g. of e4m3 rows) (xs, their scales).  Rows that no slot names are left as they
    were in out."""
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return expert_dispatch(x, slots, scales=scales, out=out, scales_out=scales_out)
    T, k, ps = _expect_slots(slots, dev)
    shape, dtype = x.shape, x.dtype
    if len(shape) < 2 or shape[0] != T:
        raise ValueError("x must be [tokens, ...] with the slots' tokens")
    px = _expect(x, "x", dtype, shape, dev)
    if scales_out is not None and scales is None:
        raise ValueError("scales_out without scales")
    psc = pso = None
    n_scales = 0
    if scales is not None:
        if scales.dim() != 2:
            raise ValueError("scales must be [tokens, n]")
        n_scales = scales.shape[1]
        _expect_32(n_scales)
        psc = _expect(scales, "scales", torch.float32, (T, n_scales), dev)
    _on_cuda(dev)
    if out is None:
        out = x.new_empty((T * k,) + tuple(shape[1:]))
    elif out.shape[1:] != shape[1:]:
        raise ValueError("out must have rows like x")
    po = _expect(out, "out", dtype, out.shape, dev)
    most = out.shape[0]
    if scales is not None:
        if scales_out is None:
            scales_out = scales.new_empty((most, n_scales))
        pso = _expect(scales_out, "scales_out", torch.float32, (most, n_scales), dev)
    row = shape[1:].numel()
    if row == 0 and n_scales:                       # the scales are all there is to move
        px, row, po, psc, pso = psc, 4 * n_scales, pso, None, None
    else:
        row *= x.element_size()
    if row:
        _check(lib().hstu_expert_dispatch(px, row, psc, n_scales, ps, T, k, most,
                                          po, pso, _raw_stream(dev)), "hstu_expert_dispatch")
    return out if scales is None else (out, scales_out)


def expert_combine(y, slots, weights=None, *, residual=None, out=None, stream=None):
    """out [tokens, width] = residual + sum over j of weights[:, j] * y[slots[:, j]]."""
    dev = y.get_device()
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return expert_combine(y, slots, weights, residual=residual, out=out)
    T, k, ps = _expect_slots(slots, dev)
    rows, width, code = _expect_rows(y, "y")
    shape, dtype = (T, width), y.dtype
    py = _expect(y, "y", dtype, y.shape, dev)
    pw = _expect(weights, "weights", torch.float32, (T, k), dev)
    pr = _expect(residual, "residual", dtype, shape, dev)
    _on_cuda(dev)
    if out is None:
        out = y.new_empty(shape)
    po = _expect(out, "out", dtype, shape, dev)
    _check(lib().hstu_expert_combine(py, ps, pw, pr, T, k, rows, width, code, po, _raw_stream(dev)),
           "hstu_expert_combine")
    return out


def expert_combine_bwd(dout, y, slots, weights=None, *, grads=None, stream=None):
    """(dy, dweights or None) of expert_combine; rows of dy that no slot names are left as they
    were.  The residual's gradient is dout itself."""
    dev = y.get_device()
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return expert_combine_bwd(dout, y, slots, weights, grads=grads)
    T, k, ps = _expect_slots(slots, dev)
    rows, width, code = _expect_rows(y, "y")
    dtype = y.dtype
    py = _expect(y, "y", dtype, y.shape, dev)
    pdo = _expect(dout, "dout", dtype, (T, width), dev)
    pw = _expect(weights, "weights", torch.float32, (T, k), dev)
    _on_cuda(dev)
    if grads is None:
        grads = (torch.empty_like(y), None if weights is None else torch.empty_like(weights))
    dy, dw = grads
    pdy = _expect(dy, "dy", dtype, y.shape, dev)
    pdw = _expect(dw, "dweights", torch.float32, (T, k), dev)
    _check(lib().hstu_expert_combine_bwd(pdo, py, ps, pw, T, k, rows, width, code, pdy, pdw,
                                         _raw_stream(dev)), "hstu_expert_combine_bwd")
    return grads


def expert_dispatch_bwd(dxs, slots, *, out=None, stream=None):
    """dx [tokens, width] of expert_dispatch: each token's sum over its sorted rows."""
    return expert_combine(dxs, slots, out=out, stream=stream)


def _expect_proj(x, w):
    if x.dim() != 2 or w.dim() != 3:
        raise ValueError("x must be [rows, d_in] and w [experts, ., .]")
    _expect_32(x.shape[1], *w.shape)


def expert_proj(x, w, offsets, *, silu=False, pre=None, out=None, status=None, stream=None):
    """out [rows, d_out]: each expert's rows offsets[e] .. offsets[e+1] of x [rows, d_in] (bf16)
    times w[e] of [experts, d_in, d_out], SiLU after it when silu (the product itself then to
    pre, when given).  Rows of no expert are left as they were in out."""
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return expert_proj(x, w, offsets, silu=silu, pre=pre, out=out, status=status)
    _expect_proj(x, w)
    S, K = x.shape
    E, N = w.shape[0], w.shape[2]
    if pre is not None and not silu:
        raise ValueError("pre is for the product ahead of the SiLU")
    px = _expect(x, "x", torch.bfloat16, (S, K), dev)
    pw = _expect(w, "w", torch.bfloat16, (E, K, N), dev)
    pof = _expect(offsets, "offsets", torch.int64, (E + 1,), dev)
    pp = _expect(pre, "pre", torch.bfloat16, (S, N), dev)
    pst = _expect_status(status, dev)
    _on_cuda(dev)
    if out is None:
        out = x.new_empty((S, N))
    po = _expect(out, "out", torch.bfloat16, (S, N), dev)
    _check(lib().hstu_expert_proj(px, pw, pof, S, E, K, N, 1 if silu else 0, po, pp, pst,
                                  _raw_stream(dev)), "hstu_expert_proj")
    return out


def expert_proj_e4m3(x, x_scales, w, w_scales, offsets, *, silu=False, out=None, status=None,
                     stream=None):
    """expert_proj of e4m3 rows x [rows, d_in] with scales (one fp32 per row) and e4m3 weights w
    [experts, d_out, d_in] with scales [experts, d_out]; out is bf16."""
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return expert_proj_e4m3(x, x_scales, w, w_scales, offsets, silu=silu, out=out,
                                    status=status)
    _expect_proj(x, w)
    S, K = x.shape
    E, N = w.shape[0], w.shape[1]
    px = _expect(x, "x", F8, (S, K), dev)
    pw = _expect(w, "w", F8, (E, N, K), dev)
    pxs = _expect(x_scales, "x_scales", torch.float32, (S, 1) if x_scales.dim() == 2 else (S,), dev)
    pws = _expect(w_scales, "w_scales", torch.float32, (E, N), dev)
    pof = _expect(offsets, "offsets", torch.int64, (E + 1,), dev)
    pst = _expect_status(status, dev)
    _on_cuda(dev)
    if out is None:
        out = x.new_empty((S, N), dtype=torch.bfloat16)
    po = _expect(out, "out", torch.bfloat16, (S, N), dev)
    _check(lib().hstu_expert_proj_e4m3(px, pxs, pw, pws, pof, S, E, K, N, 1 if silu else 0, po, pst,
                                       _raw_stream(dev)), "hstu_expert_proj_e4m3")
    return out


def expert_proj_bwd(dout, x, w, offsets, *, silu_pre=None, grads=None, status=None,
                    workspace=None, stream=None):
    """(dx, dw) of expert_proj's product.  With silu_pre (x = SiLU(silu_pre)), dx is the gradient
    of silu_pre.  grads: (dx, dw) to write into, None in the place of one not wanted; rows of dx
    of no expert are left as they were."""
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return expert_proj_bwd(dout, x, w, offsets, silu_pre=silu_pre, grads=grads,
                                   status=status, workspace=workspace)
    _expect_proj(x, w)
    S, K = x.shape
    E, N = w.shape[0], w.shape[2]
    px = _expect(x, "x", torch.bfloat16, (S, K), dev)
    pw = _expect(w, "w", torch.bfloat16, (E, K, N), dev)
    pdo = _expect(dout, "dout", torch.bfloat16, (S, N), dev)
    pp = _expect(silu_pre, "silu_pre", torch.bfloat16, (S, K), dev)
    pof = _expect(offsets, "offsets", torch.int64, (E + 1,), dev)
    pst = _expect_status(status, dev)
    _on_cuda(dev)
    if grads is None:
        grads = (torch.empty_like(x), torch.empty_like(w))
    dx, dw = grads
    pdx = _expect(dx, "dx", torch.bfloat16, (S, K), dev)
    pdw = _expect(dw, "dw", torch.bfloat16, (E, K, N), dev)
    need = 0 if dw is None else _workspace_size("hstu_expert_proj_bwd_workspace_size", S, E, K, N)
    pws, nws, workspace = _workspace(x, workspace, need, dev)
    _check(lib().hstu_expert_proj_bwd(pdo, px, pw, pof, pp, S, E, K, N, pdx, pdw, pst, pws, nws,
                                      _raw_stream(dev)), "hstu_expert_proj_bwd")
    return grads


def expert_layer_fwd(x, residual, norm_weight, expert_ids, gates, w_in, w_out, *, ln_eps=1e-5,
                     training=False, status=None, stream=None):
    """A mixture-of-experts layer on tokens x [T, d_model] (bf16) behind a residual stream:
    h = x + residual, each token's experts' SiLU(norm(h) w_in[e]) w_out[e], weighted by gates
    [T, choices] and added to h.  w_in [E, d_model, d_ff], or (e4m3 [E, d_ff, d_model], scales
    [E, d_ff]) for the 8-bit product (inference); w_out [E, d_ff, d_model].  Returns dict(o, sum,
    rstd, routing, xs, pre, z, y); expert_layer_bwd takes it after training=True."""
    dev = x.get_device()
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return expert_layer_fwd(x, residual, norm_weight, expert_ids, gates, w_in, w_out,
                                    ln_eps=ln_eps, training=training, status=status)
    eight = isinstance(w_in, (tuple, list))
    if eight and training:
        raise ValueError("the 8-bit product has no backward")
    E = w_out.shape[0]
    n = rms_norm_rows(x, norm_weight, residual, eps=ln_eps, e4m3=eight, training=training)
    r = expert_sort(expert_ids, E, status=status)
    pre = None
    if eight:
        xs, sc = expert_dispatch(n.y, r.slots, scales=n.scales)
        z = expert_proj_e4m3(xs, sc, w_in[0], w_in[1], r.offsets, silu=True, status=status)
    else:
        xs = expert_dispatch(n.y, r.slots)
        if training:
            pre = x.new_empty((xs.shape[0], w_in.shape[2]))
        z = expert_proj(xs, w_in, r.offsets, silu=True, pre=pre, status=status)
    y = expert_proj(z, w_out, r.offsets, status=status)
    o = expert_combine(y, r.slots, gates, residual=n.sum)
    return dict(o=o, sum=n.sum, rstd=n.rstd, routing=r, xs=xs, pre=pre, z=z, y=y)


def expert_layer_bwd(do, saved, norm_weight, gates, w_in, w_out, *, status=None, stream=None):
    """Gradients of expert_layer_fwd(..., training=True), whose result is `saved`: dict(dx (of x
    and of residual alike), dnorm_weight, dgates, dw_in, dw_out)."""
    dev = do.get_device()
    if _elsewhere(dev, stream):
        with _place(dev, stream):
            return expert_layer_bwd(do, saved, norm_weight, gates, w_in, w_out, status=status)
    r = saved["routing"]
    dy, dgates = expert_combine_bwd(do, saved["y"], r.slots, gates)
    dpre, dw_out = expert_proj_bwd(dy, saved["z"], w_out, r.offsets, silu_pre=saved["pre"],
                                   status=status)
    dxs, dw_in = expert_proj_bwd(dpre, saved["xs"], w_in, r.offsets, status=status)
    dn = expert_dispatch_bwd(dxs, r.slots)
    dx, dnw = rms_norm_rows_bwd(dn, saved["sum"], saved["rstd"], norm_weight, dsum=do)
    return dict(dx=dx, dnorm_weight=dnw, dgates=dgates, dw_in=dw_in, dw_out=dw_out)


def version() -> int:
    return int(lib().hstu_attn_version())


# ------------------------------------------------------------------ batch helpers

def batch_to_device(b, device="cuda"):
    """Device tensors of a synth.Batch (values already exact in the batch dtype)."""
    dt = torch.float32 if b.dtype == "f32" else torch.bfloat16

    def T(a, dtype=None):
        if a is None:
            return None
        t = torch.from_numpy(a)
        if dtype is not None:
            t = t.to(dtype)
        return t.to(device).contiguous()

    return dict(q=T(b.q, dt), k=T(b.k, dt), v=T(b.v, dt), u=T(b.u, dt),
                seq_offsets=T(b.seq_offsets), num_contextuals=T(b.num_contextuals),
                num_targets=T(b.num_targets), timestamps=T(b.timestamps),
                rel_bias=T(b.rel_bias), time_bias=T(b.time_bias),
                dout=T(b.dout, dt) if b.dout is not None else None)


def batch_kwargs(b):
    return dict(alpha=b.alpha, max_seqlen=b.max_seqlen, max_attn_len=b.max_attn_len,
                time_bucket_div=b.time_bucket_div, ln_eps=b.ln_eps,
                mask_flags=int(getattr(b, "mask_flags", 0)))


def run_fwd(b, dev_tensors=None, training=False, **kw):
    t = batch_to_device(b) if dev_tensors is None else dev_tensors
    args = batch_kwargs(b)
    args.update(kw)
    return fwd(t["q"], t["k"], t["v"], t["u"], t["seq_offsets"], t["num_contextuals"],
               t["num_targets"], t["timestamps"], t["rel_bias"], t["time_bias"],
               training=training, **args)


def run_bwd(b, saved, dout=None, dev_tensors=None, **kw):
    t = batch_to_device(b) if dev_tensors is None else dev_tensors
    if dout is None:
        dout = t["dout"]
    args = batch_kwargs(b)
    args.update(kw)
    return bwd(dout, t["q"], t["k"], t["v"], t["u"], t["seq_offsets"], t["num_contextuals"],
               t["num_targets"], t["timestamps"], t["rel_bias"], t["time_bias"], saved=saved,
               **args)
