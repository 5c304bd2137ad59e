"""Python binding of include/kda_layers.h: the operators around the KDA layers
of a hybrid stack (projections with their epilogue, linear attention with one
decay per head, the paged key-value cache and attention over it).

As in ``kda``, every step runs in the CUDA library; this module checks shapes,
dtypes, devices and strides, passes pointers and the stream, and turns a non-OK
status into ``KDAError``.  Inputs [T, H, d] may be slices of a wider row-major
tensor (a fused projection): a row (the last two axes) is dense, the rows any
stride apart.  Outputs and workspaces that a call allocates come from the memory
of the stream it runs on (`stream`, or torch's current one); outputs may be used
on the current stream as well, once it waits for `stream`, and any tensor of the
call may be dropped before the call has run.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .kda import KDA_BF16, KDA_F32, KDA_OK, KDAError, _empty, _record, lib

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "sigmoid": 4}
_CODE = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}
_P, _I, _L, _F, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_SIGNATURES = {
    "kda_linear": (_I, [_P, _L, _P, _P, _P, _P, _L, _L, _L, _I, _I, _P, _P]),
    "kda_decay_prefill_workspace_size": (_Z, [_L, _I, _I, _I, _I, _I]),
    "kda_decay_prefill": (_I, [_P, _L, _P, _L, _P, _L, _P, _P, _I, _L, _I, _I, _I, _I, _F, _P, _P, _P, _P, _Z, _P, _P]),
    "kda_decay_decode": (_I, [_P, _L, _P, _L, _P, _L, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _F, _P, _P]),
    "kda_paged_append": (_I, [_P, _L, _P, _L, _P, _P, _I, _I, _P, _I, _P, _P, _I, _L, _I, _I, _I, _P, _P]),
    "kda_paged_decode_workspace_size": (_Z, [_I, _L, _I, _I, _I, _I]),
    "kda_paged_decode": (_I, [_P, _L, _P, _P, _I, _I, _P, _I, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P, _Z, _P, _P]),
    "kda_paged_append_q8": (_I, [_P, _L, _P, _L, _P, _P, _P, _P, _I, _I, _I, _P, _I, _P, _P, _I, _L, _I, _I, _I, _P, _P]),
    "kda_paged_decode_q8_workspace_size": (_Z, [_I, _L, _I, _I, _I, _I]),
    "kda_paged_decode_q8": (_I, [_P, _L, _P, _P, _P, _P, _I, _I, _I, _P, _I, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P, _Z, _P, _P]),
    "kda_pages_resize_workspace_size": (_Z, [_I, _I, _I]),
    "kda_pages_resize": (_I, [_P, _I, _I, _P, _P, _I, _P, _I, _P, _Z, _P, _P]),
    "kda_pages_fork_workspace_size": (_Z, [_I, _I, _I]),
    "kda_pages_fork": (_I, [_P, _P, _I, _P, _I, _I, _P, _P, _I, _P, _P, _P, _I, _I, _P, _Z, _P, _P]),
    "kda_pages_compact_workspace_size": (_Z, [_I]),
    "kda_pages_compact": (_I, [_P, _P, _I, _P, _I, _I, _P, _I, _P, _P, _P, _Z, _P, _P]),
}
_fns: dict = {}
# torch's current stream of a device as an integer, without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = getattr(lib(), name)
        f.restype, f.argtypes = _SIGNATURES[name]
        _fns[name] = f
    return f


def _dense(t, name, shape, dtype, device):
    """`t` is a contiguous tensor of this shape, dtype and device; its pointer (None for None)."""
    if t is None:
        return None
    if type(t) is torch.Tensor and t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, shape, width, dtype, device):
    """`t` is a tensor of this shape whose rows (all axes but the first, `width` elements) are dense; its row stride."""
    if type(t) is torch.Tensor and t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return width
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return width
    inner = 1
    for n, st in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and st != inner:
            raise ValueError(f"{name}: the rows of [T, ...] must be dense")
        inner *= n
    if t.shape[0] > 1 and t.stride(0) < width:
        raise ValueError(f"{name}: rows overlap (row stride {t.stride(0)}, {width} elements)")
    return max(t.stride(0), width)


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _dims(t, name, n):
    if not isinstance(t, torch.Tensor) or t.dim() != n:
        raise ValueError(f"{name} must be a tensor of {n} axes")
    return t.shape


def _code(dtype, name):
    c = _CODE.get(dtype)
    if c is None:
        raise TypeError(f"{name}: unsupported dtype {dtype}")
    return c


@functools.lru_cache(maxsize=4096)
def _size(name, device, *args):
    """Workspace bytes on `device`, whose number of SMs they depend on."""
    with torch.cuda.device(device):
        return _fn(name)(*args)


def _call(name, device, stream, outputs, *args):
    """Runs `name` on `device` and `stream` (torch's current one by default); `outputs`
    were allocated for the call, and the current stream may use them too."""
    index = device.index
    if stream is None:
        raw = _raw_stream(index)
    else:
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the inputs on {device}")
        raw = stream.cuda_stream
        if raw != _raw_stream(index):
            for t in outputs:
                t.record_stream(torch.cuda.current_stream(device))
    if index == _current_device():
        st = _fn(name)(*args, raw)
    else:
        with torch.cuda.device(device):
            st = _fn(name)(*args, raw)
    if st != KDA_OK:
        raise KDAError(st, name)


def _status(status, device):
    if status is None:
        return None
    if not isinstance(status, torch.Tensor) or status.device != device or status.numel() * status.element_size() < 4:
        raise ValueError("status must be a tensor of at least 4 bytes on the inputs' device")
    return status.data_ptr()


def linear(x, w, bias=None, residual=None, act="none", out=None, out_dtype=None, status=None, stream=None):
    """act(x w^T + bias) + residual for x [M, K] bf16 (rows any stride apart), w
    [N, K] bf16, bias [N] f32, residual [M, N] of the output's dtype (bf16, or
    out_dtype=torch.float32).  act: one of ACTIVATIONS."""
    dev = _cuda(x, "x")
    M, K = _dims(x, "x", 2)
    ldx = _rows(x, "x", (M, K), K, torch.bfloat16, dev)
    N = _dims(w, "w", 2)[0]
    wp = _dense(w, "w", (N, K), torch.bfloat16, dev)
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(ACTIVATIONS)}, got {act!r}")
    new = []
    if out is None:
        out = _empty(stream, (M, N), torch.bfloat16 if out_dtype is None else out_dtype, dev)
        new.append(out)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"out is {out.dtype}, out_dtype {out_dtype}")
    code = _code(out.dtype, "out")
    _call("kda_linear", dev, stream, new, x.data_ptr(), ldx, wp, _dense(bias, "bias", (N,), torch.float32, dev),
          _dense(residual, "residual", (M, N), out.dtype, dev), _dense(out, "out", (M, N), out.dtype, dev), M, N, K,
          ACTIVATIONS[act], code, _status(status, dev))
    if stream is not None:
        _record(stream, x, w, bias, residual, out, status)
    return out


def decay_prefill_workspace_size(total_tokens, num_seqs, H, dk, dv, dtype=torch.bfloat16) -> int:
    return int(_fn("kda_decay_prefill_workspace_size")(total_tokens, num_seqs, H, dk, dv, _code(dtype, "dtype")))


def decay_prefill(q, k, v, log_decay, cu_seqlens, initial_state=None, final_state=None, out=None, scale=1.0,
                  workspace=None, want_final_state=True, status=None, stream=None):
    """Linear attention with one decay per head over packed sequences.

    q, k [T, H, dk], v [T, H, dv] (bf16 or f32, all the same; rows any stride
    apart); log_decay [H] f32; cu_seqlens [N + 1] int32; initial_state
    [N, H, dk, dv] f32 or None.  Returns (out [T, H, dv], final_state or None)."""
    dev = _cuda(q, "q")
    dt = q.dtype
    code = _code(dt, "q")
    T, H, dk = _dims(q, "q", 3)
    dv = _dims(v, "v", 3)[2]
    ldq = _rows(q, "q", (T, H, dk), H * dk, dt, dev)
    ldk = _rows(k, "k", (T, H, dk), H * dk, dt, dev)
    ldv = _rows(v, "v", (T, H, dv), H * dv, dt, dev)
    lp = _dense(log_decay, "log_decay", (H,), torch.float32, dev)
    N = _dims(cu_seqlens, "cu_seqlens", 1)[0] - 1
    cp = _dense(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    new = []
    if final_state is None and want_final_state:
        final_state = _empty(stream, (N, H, dk, dv), torch.float32, dev)
        new.append(final_state)
    if out is None:
        out = _empty(stream, (T, H, dv), dt, dev)
        new.append(out)
    if workspace is None:
        size = _size("kda_decay_prefill_workspace_size", dev, T, N, H, dk, dv, code)
        if size:
            workspace = _empty(stream, size, torch.uint8, dev)
    size = 0 if workspace is None else _dims(workspace, "workspace", 1)[0]
    wp = _dense(workspace, "workspace", (size,), torch.uint8, dev)
    _call("kda_decay_prefill", dev, stream, new, q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, lp, cp, N, T,
          H, dk, dv, code, scale, _dense(initial_state, "initial_state", (N, H, dk, dv), torch.float32, dev),
          _dense(final_state, "final_state", (N, H, dk, dv), torch.float32, dev),
          _dense(out, "out", (T, H, dv), dt, dev), wp, size,
          _status(status, dev))
    if stream is not None:
        _record(stream, q, k, v, log_decay, cu_seqlens, initial_state, final_state, out, workspace, status)
    return out, final_state


def decay_decode(q, k, v, log_decay, state_pool, slot_ids=None, out=None, scale=1.0, status=None, stream=None):
    """One token per sequence of the same mixer; the states in the pool [P, H,
    dk, dv] f32 are updated in place.  q, k [N, H, dk], v [N, H, dv]; slot_ids
    [N] int32 (negative: padding row) or None for slot i = i.  Returns out [N, H, dv]."""
    dev = _cuda(q, "q")
    dt = q.dtype
    code = _code(dt, "q")
    N, H, dk = _dims(q, "q", 3)
    dv = _dims(v, "v", 3)[2]
    ldq = _rows(q, "q", (N, H, dk), H * dk, dt, dev)
    ldk = _rows(k, "k", (N, H, dk), H * dk, dt, dev)
    ldv = _rows(v, "v", (N, H, dv), H * dv, dt, dev)
    P = _dims(state_pool, "state_pool", 4)[0]
    new = []
    if out is None:
        out = _empty(stream, (N, H, dv), dt, dev)
        new.append(out)
    _call("kda_decay_decode", dev, stream, new, q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv,
          _dense(log_decay, "log_decay", (H,), torch.float32, dev),
          _dense(state_pool, "state_pool", (P, H, dk, dv), torch.float32, dev), P,
          _dense(slot_ids, "slot_ids", (N,), torch.int32, dev), _dense(out, "out", (N, H, dv), dt, dev), N, H, dk,
          dv, code, scale, _status(status, dev))
    if stream is not None:
        _record(stream, q, k, v, log_decay, state_pool, slot_ids, out, status)
    return out


def paged_append(k, v, k_cache, v_cache, page_table, start_pos, cu_seqlens=None, status=None, stream=None):
    """Writes new tokens' k and v [T, Hkv, d] into the pages [P, Hkv, page_size, d]
    of a cache: token t of sequence i goes to position start_pos[i] + t -
    cu_seqlens[i] (cu_seqlens None: one token per sequence)."""
    dev = _cuda(k, "k")
    dt = k.dtype
    code = _code(dt, "k")
    T, H, d = _dims(k, "k", 3)
    ldk = _rows(k, "k", (T, H, d), H * d, dt, dev)
    ldv = _rows(v, "v", (T, H, d), H * d, dt, dev)
    P, _, ps, _ = _dims(k_cache, "k_cache", 4)
    kp = _dense(k_cache, "k_cache", (P, H, ps, d), dt, dev)
    vp = _dense(v_cache, "v_cache", (P, H, ps, d), dt, dev)
    N, cols = _dims(page_table, "page_table", 2)
    tp = _dense(page_table, "page_table", (N, cols), torch.int32, dev)
    _call("kda_paged_append", dev, stream, (), k.data_ptr(), ldk, v.data_ptr(), ldv, kp, vp, P, ps, tp, cols,
          _dense(start_pos, "start_pos", (N,), torch.int32, dev),
          _dense(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev), N, T, H, d, code, _status(status, dev))
    if stream is not None:
        _record(stream, k, v, k_cache, v_cache, page_table, start_pos, cu_seqlens, status)


def paged_decode_workspace_size(num_seqs, max_tokens, Hq, Hkv, d, dtype=torch.bfloat16) -> int:
    """Workspace bytes of paged_decode for tables of max_tokens = max_pages * page_size tokens."""
    return int(_fn("kda_paged_decode_workspace_size")(num_seqs, max_tokens, Hq, Hkv, d, _code(dtype, "dtype")))


def paged_decode(q, k_cache, v_cache, page_table, seq_lens, scale=None, out=None, lse=None, return_lse=False,
                 workspace=None, status=None, stream=None):
    """Attention of one token per sequence over the first seq_lens[i] tokens of
    its paged cache.  q [N, Hq, d]; caches [P, Hkv, page_size, d]; page_table
    [N, max_pages] int32; seq_lens [N] int32; scale defaults to d^-1/2.  Returns
    out [N, Hq, d], or (out, lse [N, Hq] f32) with return_lse."""
    dev = _cuda(q, "q")
    dt = q.dtype
    code = _code(dt, "q")
    N, Hq, d = _dims(q, "q", 3)
    ldq = _rows(q, "q", (N, Hq, d), Hq * d, dt, dev)
    P, Hkv, ps, _ = _dims(k_cache, "k_cache", 4)
    kp = _dense(k_cache, "k_cache", (P, Hkv, ps, d), dt, dev)
    vp = _dense(v_cache, "v_cache", (P, Hkv, ps, d), dt, dev)
    cols = _dims(page_table, "page_table", 2)[1]
    tp = _dense(page_table, "page_table", (N, cols), torch.int32, dev)
    new = []
    if out is None:
        out = _empty(stream, (N, Hq, d), dt, dev)
        new.append(out)
    if lse is None and return_lse:
        lse = _empty(stream, (N, Hq), torch.float32, dev)
        new.append(lse)
    if workspace is None:
        size = _size("kda_paged_decode_workspace_size", dev, N, cols * ps, Hq, Hkv, d, code)
        workspace = _empty(stream, size, torch.uint8, dev)
    size = _dims(workspace, "workspace", 1)[0]
    _call("kda_paged_decode", dev, stream, new, q.data_ptr(), ldq, kp, vp, P, ps, tp, cols,
          _dense(seq_lens, "seq_lens", (N,), torch.int32, dev), N, Hq, Hkv, d, code,
          d ** -0.5 if scale is None else scale, _dense(out, "out", (N, Hq, d), dt, dev),
          _dense(lse, "lse", (N, Hq), torch.float32, dev), _dense(workspace, "workspace", (size,), torch.uint8, dev),
          size, _status(status, dev))
    if stream is not None:
        _record(stream, q, k_cache, v_cache, page_table, seq_lens, out, lse, workspace, status)
    return (out, lse) if return_lse else out


def _cache_q8(k_cache, v_cache, k_scale, v_scale, H, d, dev):
    """The shapes and pointers of a cache in 8 bits: pages, page size, block, and four pointers."""
    shape, blocks = _dims(k_cache, "k_cache", 4), _dims(k_scale, "k_scale", 3)
    P, _, ps, _ = shape
    n, index, f8, f32 = blocks[2], dev.index, torch.float8_e4m3fn, torch.float32
    if (type(k_cache) is type(v_cache) is type(k_scale) is type(v_scale) is torch.Tensor and shape == (P, H, ps, d)
            and blocks == (P, H, n) and v_cache.shape == shape and v_scale.shape == blocks
            and k_cache.dtype is v_cache.dtype is f8 and k_scale.dtype is v_scale.dtype is f32
            and k_cache.get_device() == v_cache.get_device() == k_scale.get_device() == v_scale.get_device() == index
            and k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous() and v_scale.is_contiguous()
            and n and ps % n == 0):
        return P, ps, ps // n, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr()
    # which of it is wrong (a subclass of Tensor is not)
    kp, vp = (_dense(t, name, (P, H, ps, d), f8, dev) for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")))
    if n == 0 or ps % n:
        raise ValueError(f"k_scale has {n} blocks for pages of {ps} tokens")
    ksp, vsp = (_dense(t, name, (P, H, n), f32, dev) for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")))
    return P, ps, ps // n, kp, vp, ksp, vsp


def paged_append_q8(k, v, k_cache, v_cache, k_scale, v_scale, page_table, start_pos, cu_seqlens=None, status=None,
                    stream=None):
    """paged_append into a cache in 8 bits: k_cache, v_cache [P, Hkv, page_size, d] e4m3, k_scale, v_scale [P, Hkv,
    page_size / block] f32 with a power of two for each block of 16, 32, 64 or 128 tokens (a value is its code times
    its block's scale).  A partly filled block's scale grows where new tokens need it, and its codes follow."""
    dev = _cuda(k, "k")
    dt = k.dtype
    code = _code(dt, "k")
    T, H, d = _dims(k, "k", 3)
    ldk = _rows(k, "k", (T, H, d), H * d, dt, dev)
    ldv = _rows(v, "v", (T, H, d), H * d, dt, dev)
    P, ps, block, kp, vp, ksp, vsp = _cache_q8(k_cache, v_cache, k_scale, v_scale, H, d, dev)
    N, cols = _dims(page_table, "page_table", 2)
    tp = _dense(page_table, "page_table", (N, cols), torch.int32, dev)
    _call("kda_paged_append_q8", dev, stream, (), k.data_ptr(), ldk, v.data_ptr(), ldv, kp, vp, ksp, vsp, P, ps, block, tp,
          cols, _dense(start_pos, "start_pos", (N,), torch.int32, dev),
          _dense(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev), N, T, H, d, code, _status(status, dev))
    if stream is not None:
        _record(stream, k, v, k_cache, v_cache, k_scale, v_scale, page_table, start_pos, cu_seqlens, status)


def paged_decode_q8_workspace_size(num_seqs, max_tokens, Hq, Hkv, d, dtype=torch.bfloat16) -> int:
    """Workspace bytes of paged_decode_q8 for tables of max_tokens = max_pages * page_size tokens."""
    return int(_fn("kda_paged_decode_q8_workspace_size")(num_seqs, max_tokens, Hq, Hkv, d, _code(dtype, "dtype")))


def paged_decode_q8(q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, scale=None, out=None, lse=None,
                    return_lse=False, workspace=None, status=None, stream=None):
    """paged_decode over a cache in 8 bits (as for paged_append_q8).  q [N, Hq, d] bf16 or f32, as out."""
    dev = _cuda(q, "q")
    dt = q.dtype
    code = _code(dt, "q")
    N, Hq, d = _dims(q, "q", 3)
    ldq = _rows(q, "q", (N, Hq, d), Hq * d, dt, dev)
    Hkv = _dims(k_cache, "k_cache", 4)[1]
    P, ps, block, kp, vp, ksp, vsp = _cache_q8(k_cache, v_cache, k_scale, v_scale, Hkv, d, dev)
    cols = _dims(page_table, "page_table", 2)[1]
    tp = _dense(page_table, "page_table", (N, cols), torch.int32, dev)
    new, lsep, wp = [], None, None
    if out is None:
        out = _empty(stream, (N, Hq, d), dt, dev)
        outp = out.data_ptr()
        new.append(out)
    else:
        outp = _dense(out, "out", (N, Hq, d), dt, dev)
    if lse is not None:
        lsep = _dense(lse, "lse", (N, Hq), torch.float32, dev)
    elif return_lse:
        lse = _empty(stream, (N, Hq), torch.float32, dev)
        lsep = lse.data_ptr()
        new.append(lse)
    if workspace is not None:
        size = _dims(workspace, "workspace", 1)[0]
        wp = _dense(workspace, "workspace", (size,), torch.uint8, dev)
    else:
        size = _size("kda_paged_decode_q8_workspace_size", dev, N, cols * ps, Hq, Hkv, d, code)
        if size:
            workspace = _empty(stream, size, torch.uint8, dev)
            wp = workspace.data_ptr()
    _call("kda_paged_decode_q8", dev, stream, new, q.data_ptr(), ldq, kp, vp, ksp, vsp, P, ps, block, tp, cols,
          _dense(seq_lens, "seq_lens", (N,), torch.int32, dev), N, Hq, Hkv, d, code,
          d ** -0.5 if scale is None else scale, outp, lsep, wp, size, _status(status, dev))
    if stream is not None:
        _record(stream, q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, out, lse, workspace, status)
    return (out, lse) if return_lse else out
