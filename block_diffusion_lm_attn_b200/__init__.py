"""Python binding of libbdattn.so, the B200 block-diffusion attention library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/bd_attn.h``.  There is no
CPU or PyTorch fallback; if the library is missing or cannot be loaded,
every call raises.

Two layers:
  * ``bd_attn_fwd`` / ``bd_attn_decode`` / ``bd_attn_decode_workspace_bytes``
    / ``bd_attn_get_device_status`` / ``bd_attn_status_string`` take the C
    arguments one to one (device pointers as ints, stream as an int handle)
    and return the status code.
  * ``fwd`` / ``decode`` take torch CUDA tensors, check shapes, allocate the
    outputs if not given, call the C entry point on the current stream and
    raise ``BdAttnError`` on a non-OK status.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbdattn.so")

BD_OK = 0
BD_ERR_INVALID_ARG = 1
BD_ERR_UNSUPPORTED = 2
BD_ERR_CUDA = 3
BD_ERR_DEVICE_TIMEOUT = 4

EXPORTED = ("bd_attn_fwd", "bd_attn_decode", "bd_attn_decode_workspace_bytes",
            "bd_attn_get_device_status", "bd_attn_status_string",
            "bd_spec_accept", "bd_cache_append", "bd_cache_crop",
            "bd_sprint_prune", "bd_sprint_workspace_bytes", "bd_attn_bwd",
            "bd_attn_bwd_workspace_bytes", "bd_rope_table", "bd_rope",
            "bd_cache_append_q8", "bd_cache_read_q8", "bd_attn_decode_q8",
            "bd_spec_verify")

# scalings of rope_table
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}


class BdAttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s failed: %s (status %d)" %
                         (what, bd_attn_status_string(status), status))
        self.status = status


_lib = None


def load(path: str = LIB_PATH):
    """Load libbdattn.so (built by ``build.build()``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(
            "libbdattn.so not built at %s: run "
            "`python -m block_diffusion_lm_attn_b200.build`" % path)
    lib = ctypes.CDLL(path)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.bd_attn_fwd.restype = i
    lib.bd_attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, f, vp]
    lib.bd_attn_decode.restype = i
    lib.bd_attn_decode.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i,
                                   vp, i, vp, ctypes.c_size_t]
    lib.bd_attn_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.bd_attn_decode_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.bd_attn_get_device_status.restype = i
    lib.bd_attn_get_device_status.argtypes = [vp]
    lib.bd_attn_status_string.restype = ctypes.c_char_p
    lib.bd_attn_status_string.argtypes = [i]
    lib.bd_attn_bwd.restype = i
    lib.bd_attn_bwd.argtypes = [vp] * 9 + [i, i, i, i, i, i, f, vp, vp,
                                           ctypes.c_size_t]
    lib.bd_attn_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.bd_attn_bwd_workspace_bytes.argtypes = [i, i, i]
    lib.bd_spec_accept.restype = i
    lib.bd_spec_accept.argtypes = [vp, vp, vp, i, i, vp]
    lib.bd_cache_append.restype = i
    lib.bd_cache_append.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
    lib.bd_cache_crop.restype = i
    lib.bd_cache_crop.argtypes = [vp, i, i, vp]
    lib.bd_sprint_prune.restype = i
    lib.bd_sprint_prune.argtypes = [vp, vp, vp, vp, vp, f, f, f, vp, vp, vp,
                                    vp, vp, i, i, i, i, vp, vp,
                                    ctypes.c_size_t]
    lib.bd_sprint_workspace_bytes.restype = ctypes.c_size_t
    lib.bd_sprint_workspace_bytes.argtypes = [i, i]
    dbl, sz = ctypes.c_double, ctypes.c_size_t
    lib.bd_rope_table.restype = i
    lib.bd_rope_table.argtypes = [vp, vp, i, dbl, i, dbl, i, dbl, dbl]
    lib.bd_rope.restype = i
    lib.bd_rope.argtypes = [vp] * 7 + [i] * 8 + [f, i, vp]
    lib.bd_cache_append_q8.restype = i
    lib.bd_cache_append_q8.argtypes = [vp] * 8 + [i] * 7 + [vp]
    lib.bd_cache_read_q8.restype = i
    lib.bd_cache_read_q8.argtypes = [vp] * 7 + [i] * 5 + [vp]
    lib.bd_attn_decode_q8.restype = i
    lib.bd_attn_decode_q8.argtypes = [vp] * 8 + [i] * 6 + [vp, i, i, vp, sz]
    lib.bd_spec_verify.restype = i
    lib.bd_spec_verify.argtypes = [vp] * 8 + [i] * 3 + [vp]
    _lib = lib
    return lib


# ---------------------------------------------------------------------------
# one-to-one C entry points


def bd_attn_fwd(q, k, v, out, lse, B, Hq, Hkv, L, b, d, scale, stream):
    return load().bd_attn_fwd(q, k, v, out, lse, B, Hq, Hkv, L, b, d, scale,
                              stream)


def bd_attn_decode(q_blk, k_cache, v_cache, cache_len, out, lse, B, Hq, Hkv,
                   b, d, intra_block_mode, stream, S_cap, workspace,
                   workspace_bytes):
    return load().bd_attn_decode(q_blk, k_cache, v_cache, cache_len, out, lse,
                                 B, Hq, Hkv, b, d, intra_block_mode, stream,
                                 S_cap, workspace, workspace_bytes)


def bd_attn_decode_workspace_bytes(B, Hq, Hkv, b, d, S_cap):
    return int(load().bd_attn_decode_workspace_bytes(B, Hq, Hkv, b, d, S_cap))


def bd_attn_get_device_status(stream):
    return load().bd_attn_get_device_status(stream)


def bd_attn_status_string(status):
    return load().bd_attn_status_string(status).decode()


def bd_attn_bwd(q, k, v, out, lse, dout, dq, dk, dv, B, Hq, Hkv, L, b, d,
                scale, stream, workspace, workspace_bytes):
    return load().bd_attn_bwd(q, k, v, out, lse, dout, dq, dk, dv, B, Hq, Hkv,
                              L, b, d, scale, stream, workspace,
                              workspace_bytes)


def bd_attn_bwd_workspace_bytes(B, Hq, L):
    return int(load().bd_attn_bwd_workspace_bytes(B, Hq, L))


def bd_spec_accept(draft, target, n_accept, B, b, stream):
    return load().bd_spec_accept(draft, target, n_accept, B, b, stream)


def bd_cache_append(k_cache, v_cache, cache_len, k_new, v_new, n_new, B, Hkv,
                    b, d, S_cap, stream):
    return load().bd_cache_append(k_cache, v_cache, cache_len, k_new, v_new,
                                  n_new, B, Hkv, b, d, S_cap, stream)


def bd_cache_crop(cache_len, B, max_len, stream):
    return load().bd_cache_crop(cache_len, B, max_len, stream)


def bd_sprint_prune(k_cache, v_cache, cache_len, conf, modality, alpha,
                    keep_text, keep_image, k_out, v_out, kept, new_len, score,
                    B, Hkv, d, S_cap, stream, workspace, workspace_bytes):
    return load().bd_sprint_prune(k_cache, v_cache, cache_len, conf, modality,
                                  alpha, keep_text, keep_image, k_out, v_out,
                                  kept, new_len, score, B, Hkv, d, S_cap,
                                  stream, workspace, workspace_bytes)


def bd_sprint_workspace_bytes(B, S_cap):
    return int(load().bd_sprint_workspace_bytes(B, S_cap))


def bd_rope_table(inv_freq, mscale, rot_dim, base, scaling, factor,
                  trained_len, beta_fast, beta_slow):
    return load().bd_rope_table(inv_freq, mscale, rot_dim, base, scaling,
                                factor, trained_len, beta_fast, beta_slow)


def bd_rope(q, k, q_out, k_out, inv_freq, start, positions, B, Hq, Hkv, N, d,
            rot_dim, period, interleaved, mscale, adjoint, stream):
    return load().bd_rope(q, k, q_out, k_out, inv_freq, start, positions, B,
                          Hq, Hkv, N, d, rot_dim, period, interleaved, mscale,
                          adjoint, stream)


def bd_cache_append_q8(k_cache, v_cache, k_scale, v_scale, cache_len, k_new,
                       v_new, n_new, B, Hkv, b, d, S_cap, group, advance,
                       stream):
    return load().bd_cache_append_q8(k_cache, v_cache, k_scale, v_scale,
                                     cache_len, k_new, v_new, n_new, B, Hkv,
                                     b, d, S_cap, group, advance, stream)


def bd_cache_read_q8(k_cache, v_cache, k_scale, v_scale, cache_len, k_out,
                     v_out, B, Hkv, d, S_cap, group, stream):
    return load().bd_cache_read_q8(k_cache, v_cache, k_scale, v_scale,
                                   cache_len, k_out, v_out, B, Hkv, d, S_cap,
                                   group, stream)


def bd_attn_decode_q8(q_blk, k_cache, v_cache, k_scale, v_scale, cache_len,
                      out, lse, B, Hq, Hkv, b, d, intra_block_mode, stream,
                      S_cap, group, workspace, workspace_bytes):
    return load().bd_attn_decode_q8(q_blk, k_cache, v_cache, k_scale, v_scale,
                                    cache_len, out, lse, B, Hq, Hkv, b, d,
                                    intra_block_mode, stream, S_cap, group,
                                    workspace, workspace_bytes)


def bd_spec_verify(draft, draft_prob, target_prob, u_accept, u_sample,
                   n_draft, n_accept, next_token, B, b, V, stream):
    return load().bd_spec_verify(draft, draft_prob, target_prob, u_accept,
                                 u_sample, n_draft, n_accept, next_token, B,
                                 b, V, stream)


def bd_attn_debug_inject_fault(kind):
    """Test hook (include/bd_attn_debug.h): arm (1) or disarm (0) a one-shot
    fault that makes a bounded wait of the next head-dim-128 launch run out."""
    fn = load().bd_attn_debug_inject_fault
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_int]
    return fn(kind)


def bd_attn_debug_fwd_kernel(Hq, Hkv, d):
    """Test hook (include/bd_attn_debug.h): which forward kernel runs for
    these sizes (2 paired tcgen05, 1 one-tile tcgen05, 0 mma.sync, -1 none)."""
    fn = load().bd_attn_debug_fwd_kernel
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_int] * 3
    return fn(Hq, Hkv, d)


def bd_attn_debug_reset_sched():
    """Test hook (include/bd_attn_debug.h): synchronise the device and zero
    every work-counter pair of the persistent kernels."""
    fn = load().bd_attn_debug_reset_sched
    fn.restype = ctypes.c_int
    fn.argtypes = []
    return fn()


def bd_attn_debug_set_grid(ctas):
    """Test hook (include/bd_attn_debug.h): cap the grid of the persistent
    head-dim-128 kernels at `ctas` CTAs (0 restores one CTA per SM)."""
    fn = load().bd_attn_debug_set_grid
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_int]
    return fn(ctas)


def bd_attn_debug_set_chunk(groups):
    """Test hook (include/bd_attn_debug.h): fix the chunk size of the work
    lists at `groups` heads / head pairs / kv-head groups (0 restores the
    defaults)."""
    fn = load().bd_attn_debug_set_chunk
    fn.restype = ctypes.c_int
    fn.argtypes = [ctypes.c_int]
    return fn(groups)


# ---------------------------------------------------------------------------
# torch-tensor conveniences


def _stream_handle(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _new(make, stream, *args, **kw):
    """make(*args, **kw), an output that is made here, on the stream that the
    call launches to: its memory then is that stream's, not what work queued on
    the current one may still be using."""
    if stream is None:
        return make(*args, **kw)
    import torch
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def fwd(q, k, v, L: int, b: int, scale: float | None = None, out=None,
        lse=None, stream=None):
    """Training/prefill block-diffusion attention on CUDA tensors.

    q [B,Hq,2L,d], k, v [B,Hkv,2L,d] bf16 contiguous.  Returns (out, lse)."""
    import torch
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    if N != 2 * L or tuple(k.shape) != (B, Hkv, N, d) or v.shape != k.shape:
        raise ValueError("shape mismatch")
    for t in (q, k, v):
        if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
            raise ValueError("q, k, v must be contiguous bf16 CUDA tensors")
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = _new(torch.empty_like, stream, q)
    if lse is None:
        lse = _new(torch.empty, stream, (B, Hq, N), device=q.device, dtype=torch.float32)
    st = bd_attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                     lse.data_ptr(), B, Hq, Hkv, L, b, d, float(scale),
                     _stream_handle(stream))
    if st != BD_OK:
        raise BdAttnError(st, "bd_attn_fwd")
    return out, lse


def bwd(q, k, v, out, lse, dout, L: int, b: int, scale: float | None = None,
        dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward of ``fwd``: gradients of q, k, v given dout (the gradient of
    out), out and lse from the forward.  Returns (dq, dk, dv)."""
    import torch
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    if N != 2 * L or tuple(k.shape) != (B, Hkv, N, d) or v.shape != k.shape:
        raise ValueError("shape mismatch")
    if out.shape != q.shape or dout.shape != q.shape or tuple(lse.shape) != (B, Hq, N):
        raise ValueError("shape mismatch")
    for t_, w in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _check(t_, torch.bfloat16, w)
    _check(lse, torch.float32, "lse")
    if scale is None:
        scale = d ** -0.5
    dq = _new(torch.empty_like, stream, q) if dq is None else dq
    dk = _new(torch.empty_like, stream, k) if dk is None else dk
    dv = _new(torch.empty_like, stream, v) if dv is None else dv
    nb = bd_attn_bwd_workspace_bytes(B, Hq, L)
    if workspace is None:
        workspace = _new(torch.empty, stream, nb, dtype=torch.uint8, device=q.device)
    st = bd_attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                     lse.data_ptr(), dout.data_ptr(), dq.data_ptr(),
                     dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, L, b, d,
                     float(scale), _stream_handle(stream), workspace.data_ptr(),
                     workspace.numel() * workspace.element_size())
    if st != BD_OK:
        raise BdAttnError(st, "bd_attn_bwd")
    return dq, dk, dv


def decode(q_blk, k_cache, v_cache, cache_len, mode: int, out=None, lse=None,
           workspace=None, stream=None):
    """Block-decode attention on CUDA tensors.

    q_blk [B,Hq,b,d]; k_cache, v_cache [B,Hkv,S_cap,d] bf16; cache_len int32
    [B] on the device; mode 0 bidirectional, 1 causal, 2 cross-attention to
    the prefix only.  ``workspace`` is an
    optional uint8 CUDA tensor of at least ``workspace_bytes(...)`` bytes
    (None: the library's own per-device buffer).  Returns (out, lse)."""
    import torch
    B, Hq, b, d = q_blk.shape
    Hkv, S_cap = k_cache.shape[1], k_cache.shape[2]
    if tuple(k_cache.shape) != (B, Hkv, S_cap, d) or v_cache.shape != k_cache.shape:
        raise ValueError("shape mismatch")
    if not (cache_len.is_cuda and cache_len.dtype == torch.int32
            and cache_len.numel() == B):
        raise ValueError("cache_len must be an int32 CUDA tensor of B entries")
    for t in (q_blk, k_cache, v_cache):
        if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
            raise ValueError("q_blk and caches must be contiguous bf16 CUDA")
    if out is None:
        out = _new(torch.empty_like, stream, q_blk)
    if lse is None:
        lse = _new(torch.empty, stream, (B, Hq, b), device=q_blk.device, dtype=torch.float32)
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = bd_attn_decode(q_blk.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                        cache_len.data_ptr(), out.data_ptr(), lse.data_ptr(),
                        B, Hq, Hkv, b, d, int(mode), _stream_handle(stream),
                        S_cap, ws_ptr, ws_bytes)
    if st != BD_OK:
        raise BdAttnError(st, "bd_attn_decode")
    return out, lse


def _check(t, dtype, what):
    import torch
    if not (t.is_cuda and t.dtype == dtype and t.is_contiguous()):
        raise ValueError("%s must be a contiguous %s CUDA tensor" % (what, dtype))


def spec_accept(draft, target, n_accept=None, stream=None):
    """Longest matching prefix of draft and target ([B, b] int32 CUDA).
    Returns n_accept [B] int32 on the device."""
    import torch
    _check(draft, torch.int32, "draft")
    _check(target, torch.int32, "target")
    B, b = draft.shape
    if tuple(target.shape) != (B, b):
        raise ValueError("shape mismatch")
    if n_accept is None:
        n_accept = _new(torch.empty, stream, B, dtype=torch.int32, device=draft.device)
    st = bd_spec_accept(draft.data_ptr(), target.data_ptr(),
                        n_accept.data_ptr(), B, b, _stream_handle(stream))
    if st != BD_OK:
        raise BdAttnError(st, "bd_spec_accept")
    return n_accept


def cache_append(k_cache, v_cache, cache_len, n_new, k_new=None, v_new=None,
                 stream=None):
    """Append rows 0..n_new[i]-1 of k_new/v_new [B,Hkv,b,d] (or of the rows
    already at the cache tail, if None) and advance cache_len, in place."""
    import torch
    B, Hkv, S_cap, d = k_cache.shape
    for t, w in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _check(t, torch.bfloat16, w)
    _check(cache_len, torch.int32, "cache_len")
    _check(n_new, torch.int32, "n_new")
    if k_new is None:
        b = S_cap
        kp = vp = None
    else:
        b = k_new.shape[2]
        kp, vp = k_new.data_ptr(), v_new.data_ptr()
    st = bd_cache_append(k_cache.data_ptr(), v_cache.data_ptr(),
                         cache_len.data_ptr(), kp, vp, n_new.data_ptr(), B,
                         Hkv, b, d, S_cap, _stream_handle(stream))
    if st != BD_OK:
        raise BdAttnError(st, "bd_cache_append")


def cache_crop(cache_len, max_len: int, stream=None):
    import torch
    _check(cache_len, torch.int32, "cache_len")
    st = bd_cache_crop(cache_len.data_ptr(), cache_len.numel(), int(max_len),
                       _stream_handle(stream))
    if st != BD_OK:
        raise BdAttnError(st, "bd_cache_crop")


def sprint_prune(k_cache, v_cache, cache_len, conf, modality, alpha=0.5,
                 keep_text=1.0, keep_image=0.8, k_out=None, v_out=None,
                 want_score=False, workspace=None, stream=None):
    """Sparse prefix retention on CUDA tensors.  Returns (k_out, v_out,
    kept [B,S_cap] int32, new_len [B] int32, score [B,S_cap] fp64 or None)."""
    import torch
    B, Hkv, S_cap, d = k_cache.shape
    for t, w in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _check(t, torch.bfloat16, w)
    _check(cache_len, torch.int32, "cache_len")
    _check(conf, torch.float32, "conf")
    _check(modality, torch.uint8, "modality")
    dev = k_cache.device
    if k_out is None:
        k_out = _new(torch.empty_like, stream, k_cache)
    if v_out is None:
        v_out = _new(torch.empty_like, stream, v_cache)
    kept = _new(torch.empty, stream, (B, S_cap), dtype=torch.int32, device=dev)
    new_len = _new(torch.empty, stream, B, dtype=torch.int32, device=dev)
    score = (_new(torch.zeros, stream, (B, S_cap), dtype=torch.float64, device=dev)
             if want_score else None)
    nb = bd_sprint_workspace_bytes(B, S_cap)
    if workspace is None:
        workspace = _new(torch.empty, stream, nb, dtype=torch.uint8, device=dev)
    st = bd_sprint_prune(k_cache.data_ptr(), v_cache.data_ptr(),
                         cache_len.data_ptr(), conf.data_ptr(),
                         modality.data_ptr(), float(alpha), float(keep_text),
                         float(keep_image), k_out.data_ptr(), v_out.data_ptr(),
                         kept.data_ptr(), new_len.data_ptr(),
                         score.data_ptr() if score is not None else None,
                         B, Hkv, d, S_cap, _stream_handle(stream),
                         workspace.data_ptr(),
                         workspace.numel() * workspace.element_size())
    if st != BD_OK:
        raise BdAttnError(st, "bd_sprint_prune")
    return k_out, v_out, kept, new_len, score


# ---------------------------------------------------------------------------
# the serving step over a KV cache in 8 bits


def _check_on(t, dtype, shape, dev, what):
    """t is a contiguous tensor of this type and shape on CUDA device `dev`
    (its index).  Written for the good case: a serving step makes five such
    calls a layer, each with up to eight tensors."""
    if (t.dtype is dtype and t.get_device() == dev and t.shape == shape
            and dev >= 0 and t.is_contiguous()):
        return
    if t.dtype is not dtype or t.get_device() != dev or dev < 0 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor on %s" %
                         (what, dtype, "cuda" if dev < 0 else "cuda:%d" % dev))
    raise ValueError("%s must have the shape %s" % (what, tuple(shape)))


def _launch(fn, dev, stream, args, tail=()):
    """fn(*args, stream, *tail) with device `dev` current (a launch goes to the
    current device); stream None: that device's current stream."""
    import torch
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _launch(fn, dev, stream, args, tail)
    handle = (torch._C._cuda_getCurrentRawStream(dev) if stream is None
              else stream.cuda_stream)
    return fn(*args, handle, *tail)


def rope_table(rot_dim: int, base: float = 10000.0, scaling: str = "plain",
               factor: float = 1.0, trained_len: int = 0,
               beta_fast: float = 32.0, beta_slow: float = 1.0,
               device="cuda"):
    """Frequencies of rotary positions: (inv_freq [rot_dim / 2] fp64 on
    ``device``, mscale).  ``scaling``: "plain", "linear" (positions divided by
    ``factor``), "ntk" (a larger base) or "yarn" (slow pairs divided by
    ``factor``, pairs that turn more than ``beta_fast`` times over
    ``trained_len`` kept, in between a ramp linear in the turns, and an
    attention factor ``mscale``).  ``rope`` takes any other ``inv_freq`` too."""
    import torch
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s" % sorted(ROPE_SCALINGS))
    inv_freq = torch.empty(max(1, int(rot_dim) // 2), dtype=torch.float64)
    mscale = ctypes.c_float()
    st = bd_rope_table(inv_freq.data_ptr(), ctypes.addressof(mscale),
                       int(rot_dim), float(base), ROPE_SCALINGS[scaling],
                       float(factor), int(trained_len), float(beta_fast),
                       float(beta_slow))
    if st != BD_OK:
        raise BdAttnError(st, "bd_rope_table")
    return inv_freq.to(device), mscale.value


def rope(q, k, inv_freq, start=None, positions=None, period: int | None = None,
         interleaved: bool = False, mscale: float = 1.0,
         adjoint: bool = False, q_out=None, k_out=None, stream=None):
    """Rotary positions of q [B,Hq,N,d] and k [B,Hkv,N,d] (or None), bf16 CUDA.

    Row r of sequence i stands at ``positions[i, r]`` (int32 [B,N]) or at
    ``start[i] + r % period`` (start int32 [B], None: 0; period None: N).  The
    first 2 * len(inv_freq) dims turn, ``inv_freq`` and ``mscale`` as from
    ``rope_table``.  ``adjoint`` maps gradients of the outputs to those of the
    inputs.  q_out may be q and k_out may be k.  Returns (q_out, k_out)."""
    import torch
    B, Hq, N, d = q.shape
    dev = q.get_device()
    bf = torch.bfloat16
    _check_on(q, bf, q.shape, dev, "q")
    Hkv = 0
    if k is not None:
        Hkv = k.shape[1]
        _check_on(k, bf, (B, Hkv, N, d), dev, "k")
        if k_out is None:
            k_out = _new(torch.empty_like, stream, k)
        else:
            _check_on(k_out, bf, k.shape, dev, "k_out")
    elif k_out is not None:
        raise ValueError("k_out without k")
    if q_out is None:
        q_out = _new(torch.empty_like, stream, q)
    else:
        _check_on(q_out, bf, q.shape, dev, "q_out")
    _check_on(inv_freq, torch.float64, (inv_freq.numel(),), dev, "inv_freq")
    if start is not None:
        _check_on(start, torch.int32, (B,), dev, "start")
    if positions is not None:
        _check_on(positions, torch.int32, (B, N), dev, "positions")
    st = _launch(load().bd_rope, dev, stream, (
        q.data_ptr(), None if k is None else k.data_ptr(),
        q_out.data_ptr(), None if k is None else k_out.data_ptr(),
        inv_freq.data_ptr(), None if start is None else start.data_ptr(),
        None if positions is None else positions.data_ptr(), B, Hq, Hkv, N,
        d, 2 * inv_freq.numel(), N if period is None else period,
        int(interleaved), mscale, int(adjoint)))
    if st != BD_OK:
        raise BdAttnError(st, "bd_rope")
    return q_out, k_out


def _check_q8(k_cache, v_cache, k_scale, v_scale, cache_len, group):
    import torch
    B, Hkv, S_cap, d = shape = k_cache.shape
    dev = k_cache.get_device()
    if group not in (16, 32, 64, 128):
        raise ValueError("group must be 16, 32, 64 or 128")
    e4m3, f32 = torch.float8_e4m3fn, torch.float32
    _check_on(k_cache, e4m3, shape, dev, "k_cache")
    _check_on(v_cache, e4m3, shape, dev, "v_cache")
    groups = (B, Hkv, -(-S_cap // group))
    _check_on(k_scale, f32, groups, dev, "k_scale")
    _check_on(v_scale, f32, groups, dev, "v_scale")
    _check_on(cache_len, torch.int32, (B,), dev, "cache_len")
    return dev


def cache_append_q8(k_cache, v_cache, k_scale, v_scale, cache_len, k_new,
                    v_new, group: int, n_new=None, advance: bool = True,
                    stream=None):
    """Quantise rows 0..n_new[i]-1 (None: all) of k_new/v_new [B,Hkv,b,d] bf16
    into the cache in 8 bits (e4m3 codes [B,Hkv,S_cap,d] and fp32 scales
    [B,Hkv,ceil(S_cap/group)]) behind its cache_len[i] rows, in place, and
    advance cache_len.  ``advance=False``: the rows are a draft, to be attended
    to and overwritten.  k_new = v_new = None with n_new: the rows are there
    already, only the lengths advance."""
    import torch
    dev = _check_q8(k_cache, v_cache, k_scale, v_scale, cache_len, group)
    B, Hkv, S_cap, d = k_cache.shape
    kp = vp = None
    if k_new is None and v_new is None:
        if n_new is None:
            raise ValueError("nothing to append: neither rows nor n_new")
        b = S_cap
    else:
        if k_new is None or v_new is None:
            raise ValueError("k_new and v_new must be given together")
        b = k_new.shape[2]
        _check_on(k_new, torch.bfloat16, (B, Hkv, b, d), dev, "k_new")
        _check_on(v_new, torch.bfloat16, (B, Hkv, b, d), dev, "v_new")
        kp, vp = k_new.data_ptr(), v_new.data_ptr()
    if n_new is not None:
        _check_on(n_new, torch.int32, (B,), dev, "n_new")
    st = _launch(load().bd_cache_append_q8, dev, stream, (
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), cache_len.data_ptr(), kp, vp,
        None if n_new is None else n_new.data_ptr(), B, Hkv, b, d, S_cap,
        group, int(advance)))
    if st != BD_OK:
        raise BdAttnError(st, "bd_cache_append_q8")


def cache_read_q8(k_cache, v_cache, k_scale, v_scale, cache_len, group: int,
                  k_out=None, v_out=None, stream=None):
    """Rows 0..cache_len[i]-1 of the cache in 8 bits as bf16.  Returns (k_out,
    v_out) [B,Hkv,S_cap,d]; later rows are left as they are (0 in outputs that
    are made here)."""
    import torch
    dev = _check_q8(k_cache, v_cache, k_scale, v_scale, cache_len, group)
    B, Hkv, S_cap, d = shape = k_cache.shape
    outs = []
    for t, w in ((k_out, "k_out"), (v_out, "v_out")):
        if t is None:
            t = _new(torch.zeros, stream, shape, dtype=torch.bfloat16, device=k_cache.device)
        else:
            _check_on(t, torch.bfloat16, shape, dev, w)
        outs.append(t)
    k_out, v_out = outs
    st = _launch(load().bd_cache_read_q8, dev, stream, (
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), cache_len.data_ptr(), k_out.data_ptr(),
        v_out.data_ptr(), B, Hkv, d, S_cap, group))
    if st != BD_OK:
        raise BdAttnError(st, "bd_cache_read_q8")
    return k_out, v_out


def decode_q8(q_blk, k_cache, v_cache, k_scale, v_scale, cache_len, mode: int,
              group: int, out=None, lse=None, workspace=None, stream=None):
    """``decode`` over the cache in 8 bits of ``cache_append_q8``: same masks,
    modes, outputs and workspace.  Returns (out, lse)."""
    import torch
    dev = _check_q8(k_cache, v_cache, k_scale, v_scale, cache_len, group)
    B, Hq, b, d = q_blk.shape
    Hkv, S_cap = k_cache.shape[1], k_cache.shape[2]
    if k_cache.shape[0] != B or k_cache.shape[3] != d:
        raise ValueError("shape mismatch")
    _check_on(q_blk, torch.bfloat16, q_blk.shape, dev, "q_blk")
    if out is None:
        out = _new(torch.empty_like, stream, q_blk)
    else:
        _check_on(out, torch.bfloat16, q_blk.shape, dev, "out")
    if lse is None:
        lse = _new(torch.empty, stream, (B, Hq, b), device=q_blk.device, dtype=torch.float32)
    else:
        _check_on(lse, torch.float32, (B, Hq, b), dev, "lse")
    ws_ptr, ws_bytes = None, 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous on cuda:%d" % dev)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = _launch(load().bd_attn_decode_q8, dev, stream, (
        q_blk.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), cache_len.data_ptr(),
        out.data_ptr(), lse.data_ptr(), B, Hq, Hkv, b, d, mode),
        (S_cap, group, ws_ptr, ws_bytes))
    if st != BD_OK:
        raise BdAttnError(st, "bd_attn_decode_q8")
    return out, lse


def spec_verify(draft, draft_prob, target_prob, u_accept, u_sample,
                n_draft=None, n_accept=None, next_token=None, stream=None):
    """Accept a prefix of draft [B,b] int32 by speculative sampling and draw
    the token behind it: draft_prob [B,b,V] fp32 (None: the draft was not
    sampled), target_prob [B,b+1,V] fp32, random numbers u_accept [B,b] and
    u_sample [B] fp32 in [0,1), n_draft [B] int32 (None: b).  n_accept or
    next_token may be n_draft.  Returns (n_accept [B], next_token [B]) int32 on
    the device."""
    import torch
    B, b = draft.shape
    V = target_prob.shape[-1]
    dev = draft.get_device()
    i32, f32 = torch.int32, torch.float32
    _check_on(draft, i32, (B, b), dev, "draft")
    _check_on(target_prob, f32, (B, b + 1, V), dev, "target_prob")
    _check_on(u_accept, f32, (B, b), dev, "u_accept")
    _check_on(u_sample, f32, (B,), dev, "u_sample")
    if draft_prob is not None:
        _check_on(draft_prob, f32, (B, b, V), dev, "draft_prob")
    if n_draft is not None:
        _check_on(n_draft, i32, (B,), dev, "n_draft")
    if n_accept is None:
        n_accept = _new(torch.empty, stream, B, dtype=i32, device=draft.device)
    else:
        _check_on(n_accept, i32, (B,), dev, "n_accept")
    if next_token is None:
        next_token = _new(torch.empty, stream, B, dtype=i32, device=draft.device)
    else:
        _check_on(next_token, i32, (B,), dev, "next_token")
    st = _launch(load().bd_spec_verify, dev, stream, (
        draft.data_ptr(), None if draft_prob is None else draft_prob.data_ptr(),
        target_prob.data_ptr(), u_accept.data_ptr(), u_sample.data_ptr(),
        None if n_draft is None else n_draft.data_ptr(),
        n_accept.data_ptr(), next_token.data_ptr(), B, b, V))
    if st != BD_OK:
        raise BdAttnError(st, "bd_spec_verify")
    return n_accept, next_token


def workspace_bytes(B, Hq, Hkv, b, d, S_cap) -> int:
    return bd_attn_decode_workspace_bytes(B, Hq, Hkv, b, d, S_cap)


def device_status(stream=None) -> int:
    return bd_attn_get_device_status(_stream_handle(stream))


def bd_attn_decode_noalloc(q_blk, k_cache, v_cache, cache_len, out, lse, B,
                           Hq, Hkv, b, d, intra_block_mode, stream, S_cap):
    """One-to-one binding of the C entry point that decodes without
    allocating: its split-KV scratch is a fixed array inside the library
    (see include/bd_attn.h), for callers that cannot allocate device memory
    at decode time."""
    fn = load().bd_attn_decode_noalloc
    vp, i = ctypes.c_void_p, ctypes.c_int
    fn.restype = i
    fn.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp, i]
    return fn(q_blk, k_cache, v_cache, cache_len, out, lse, B, Hq, Hkv, b, d,
              intra_block_mode, stream, S_cap)
