"""Allocating wrappers over the C ABI: build the output tensors with torch,
call ``gbn_norm_fwd`` / ``gbn_norm_bwd`` (and the softmax, rotary position and
paged cache entry points) and raise on a non-OK status.

The work itself runs in the library's CUDA kernels; these functions only
allocate device memory and marshal arguments.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import gbnorm as G
from ._build import torch_tag

_NORM = {"layernorm": G.GBN_LAYERNORM, "rmsnorm": G.GBN_RMSNORM}
_SCALING = {"none": G.GBN_SCALING_NONE, "delayed": G.GBN_SCALING_DELAYED_TENSOR,
            "mxfp8": G.GBN_SCALING_MXFP8_1D}
_LAYOUT = {"rowwise": G.GBN_LAYOUT_ROWWISE, "colwise": G.GBN_LAYOUT_COLWISE,
           "rowwise_colwise": G.GBN_LAYOUT_ROWWISE_COLWISE}


def _check(st, where):
    if st != G.GBN_OK:
        raise G.GbnError(st, where)


def _roundup(a, b):
    return (a + b - 1) // b * b


def mx_scale_shapes(rows, hidden, swizzled=False):
    """Shapes of the MXFP8 (rowwise, colwise) E8M0 scale buffers.  Swizzled:
    padded to the 128 x 4 tiles of the GEMM order (colwise as the transposed
    operand: hidden outer, rows/32 inner)."""
    if not swizzled:
        return (rows, hidden // 32), (rows // 32, hidden)
    return ((_roundup(rows, 128), _roundup(hidden // 32, 4)),
            (_roundup(hidden, 128), _roundup(rows // 32, 4)))


def fwd_outputs(rows, hidden, in_dtype, norm="layernorm", scaling="none", layout="rowwise",
                device="cuda", training=True, swizzled_scales=False):
    """Allocates every output buffer the forward writes for this configuration."""
    dev = torch.device(device)
    o = {"out": None, "colwise_out": None, "mu": None, "rsigma": None, "scale_inv": None,
         "colwise_scale_inv": None, "updated_amax": None}
    rowwise = scaling == "none" or layout != "colwise"
    colwise = scaling != "none" and layout != "rowwise"
    if rowwise:
        o["out"] = torch.empty(rows, hidden, dtype=in_dtype if scaling == "none" else torch.uint8,
                               device=dev)
    if training:
        o["rsigma"] = torch.empty(rows, dtype=torch.float32, device=dev)
        if norm == "layernorm":
            o["mu"] = torch.empty(rows, dtype=torch.float32, device=dev)
    if scaling == "delayed":
        o["updated_amax"] = torch.empty(1, dtype=torch.float32, device=dev)
        if rowwise:
            o["scale_inv"] = torch.empty(1, dtype=torch.float32, device=dev)
        if colwise:
            o["colwise_out"] = torch.empty(hidden, rows, dtype=torch.uint8, device=dev)
            o["colwise_scale_inv"] = torch.empty(1, dtype=torch.float32, device=dev)
    elif scaling == "mxfp8":
        rs, cs = mx_scale_shapes(rows, hidden, swizzled_scales)
        if rowwise:
            o["scale_inv"] = torch.empty(rs, dtype=torch.uint8, device=dev)
        if colwise:
            o["colwise_out"] = torch.empty(rows, hidden, dtype=torch.uint8, device=dev)
            o["colwise_scale_inv"] = torch.empty(cs, dtype=torch.uint8, device=dev)
    return o


def norm_fwd(x, gamma, beta=None, *, norm="layernorm", eps=1e-5, zero_centered_gamma=False,
             scaling="none", layout="rowwise", scale=None, amax=None, sm_margin=0,
             training=True, outputs=None, stream=None, swizzled_scales=False, workspace=None):
    """Runs the fused forward; returns the dict of output tensors.
    ``swizzled_scales`` (MXFP8): scales in the padded, tiled GEMM order.
    ``workspace``: a uint8 device tensor of at least the queried size; allocated
    here when the call needs one (columnwise layouts of long rows without the
    mu / rsigma outputs)."""
    rows, hidden = x.shape
    o = outputs if outputs is not None else fwd_outputs(rows, hidden, x.dtype, norm, scaling,
                                                        layout, x.device, training,
                                                        swizzled_scales)
    in_dt = G.TORCH_DTYPE[x.dtype]
    out_dt = in_dt if scaling == "none" else G.GBN_E4M3
    lay = _LAYOUT[layout] | (G.GBN_LAYOUT_SWIZZLED_SCALES if swizzled_scales else 0)
    if workspace is None and (o["rsigma"] is None or (norm == "layernorm" and o["mu"] is None)):
        st, n = G.gbn_norm_fwd_workspace_size(rows, hidden, in_dt, G.TORCH_DTYPE[gamma.dtype],
                                              out_dt, _NORM[norm], _SCALING[scaling], lay,
                                              zero_centered_gamma, sm_margin, training)
        _check(st, "gbn_norm_fwd_workspace_size")
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    st = G.gbn_norm_fwd(x, gamma, beta, scale, amax, o["out"], o["colwise_out"], o["mu"],
                        o["rsigma"], o["scale_inv"], o["colwise_scale_inv"], o["updated_amax"],
                        workspace, workspace.numel() if workspace is not None else 0, rows,
                        hidden, in_dt, G.TORCH_DTYPE[gamma.dtype], out_dt, _NORM[norm],
                        _SCALING[scaling], lay, zero_centered_gamma, eps, sm_margin, stream)
    _check(st, "gbn_norm_fwd")
    return o


def bwd_workspace(rows, hidden, in_dtype, w_dtype, norm="layernorm", zero_centered_gamma=False,
                  sm_margin=0, device="cuda"):
    st, n = G.gbn_norm_bwd_workspace_size(rows, hidden, G.TORCH_DTYPE[in_dtype],
                                          G.TORCH_DTYPE[w_dtype], _NORM[norm],
                                          zero_centered_gamma, sm_margin)
    _check(st, "gbn_norm_bwd_workspace_size")
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def norm_bwd(dz, x, mu, rsigma, gamma, dresidual=None, *, norm="layernorm",
             zero_centered_gamma=False, sm_margin=0, workspace=None, dx=None, dgamma=None,
             dbeta=None, stream=None):
    """Runs the fused backward; returns (dx, dgamma, dbeta or None)."""
    rows, hidden = x.shape
    if workspace is None:
        workspace = bwd_workspace(rows, hidden, x.dtype, gamma.dtype, norm, zero_centered_gamma,
                                  sm_margin, x.device)
    dx = torch.empty_like(x) if dx is None else dx
    dgamma = torch.empty_like(gamma) if dgamma is None else dgamma
    if norm == "layernorm" and dbeta is None:
        dbeta = torch.empty_like(gamma)
    st = G.gbn_norm_bwd(dz, x, mu if norm == "layernorm" else None, rsigma, gamma, dresidual, dx,
                        dgamma, dbeta if norm == "layernorm" else None, workspace,
                        workspace.numel(), rows, hidden, G.TORCH_DTYPE[x.dtype],
                        G.TORCH_DTYPE[gamma.dtype], _NORM[norm], zero_centered_gamma, sm_margin,
                        stream)
    _check(st, "gbn_norm_bwd")
    return dx, dgamma, dbeta if norm == "layernorm" else None


_SOFTMAX_MASK = {"none": G.GBN_SOFTMAX_NO_MASK, "padding": G.GBN_SOFTMAX_PADDING,
                 "causal": G.GBN_SOFTMAX_CAUSAL_UPPER,
                 "causal_aligned": G.GBN_SOFTMAX_CAUSAL_ALIGNED}


def softmax_fwd(x, scale=1.0, mask_kind="none", mask=None, out=None, stream=None):
    """Scaled (masked) softmax over the last axis of x [batches, heads, sq, sk];
    mask [mask_batches, 1, sq, sk] uint8 (nonzero = masked) for "padding"."""
    b, h, sq, sk = x.shape
    y = torch.empty_like(x) if out is None else out
    mb = 0 if mask is None else mask.shape[0]
    st = G.gbn_softmax_fwd(x, mask, y, b, h, sq, sk, mb, G.TORCH_DTYPE[x.dtype],
                           _SOFTMAX_MASK[mask_kind], scale, stream)
    _check(st, "gbn_softmax_fwd")
    return y


def softmax_bwd(dy, y, scale=1.0, out=None, stream=None):
    """dx = scale * y * (dy - sum(dy * y)) over the last axis."""
    sk = y.shape[-1]
    dx = torch.empty_like(dy) if out is None else out
    st = G.gbn_softmax_bwd(dy, y, dx, y.numel() // sk, sk, G.TORCH_DTYPE[y.dtype], scale, stream)
    _check(st, "gbn_softmax_bwd")
    return dx


# ---- rotary positions and the paged key/value cache

def _shortcut():
    """The shortcut of the usual calls (csrc/fastcall.cpp), or None: they work without it, and one
    compiled against another torch would read its objects wrongly."""
    try:
        from . import _fastcall as fast
    except ImportError:
        return None
    if getattr(fast, "built_for", None) != torch_tag():
        return None
    fast.setup(*(ctypes.cast(getattr(G.library(), n), ctypes.c_void_p).value
                 for n in ("gbn_rope_fwd", "gbn_rope_bwd", "gbn_paged_append",
                           "gbn_paged_attention", "gbn_paged_attention_workspace_size")))
    return fast


_fast = _shortcut()


def _taken(r, where):
    """What the shortcut returned: the results, or the status of a refused call."""
    if type(r) is int:
        raise G.GbnError(r, where)
    return r


_ROPE_LAYOUT = {"half": G.GBN_ROPE_HALF, "interleaved": G.GBN_ROPE_INTERLEAVED}
_NO_STRIDES = (0, 0, 0)
_INT_DTYPES = (torch.int32, torch.int64)


def _launch(where, fn, args, device_index, stream):
    """Calls a C entry point that takes a packed argument struct, with the
    tensors' device current (the launch and the current stream go by it)."""
    if device_index == torch.cuda.current_device():
        st = fn(args, G.current_stream(device_index) if stream is None else G._stream(stream))
    else:
        with torch.cuda.device(device_index):
            st = fn(args, G._stream(stream))
    if st:
        raise G.GbnError(st, where)


def _on_stream(stream, device, fn, *args, **kw):
    """fn(...) with ``stream`` current, so that what it allocates belongs to the
    stream that uses it (a workspace allocated on another stream could be handed
    out again there while this one still works in it)."""
    if not isinstance(stream, torch.cuda.Stream):  # a raw handle, or an object that holds one
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        stream = torch.cuda.ExternalStream(handle, device=device)
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _on_gpu(t):
    if t.device.type != "cuda":
        raise ValueError(f"expected CUDA tensors, got one on {t.device}")


def _same(name, t, dtype, device, dims=None):
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected {dims}")


def _inner(name, t):
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")


def rope_frequencies(rotary_dim, base=10000.0, *, scaling="none", factor=1.0,
                     original_length=None, fast_turns=32.0, slow_turns=1.0, device="cuda"):
    """Radians per position of each pair: base^(-2i / rotary_dim), fp64
    [rotary_dim / 2], scaled for contexts ``factor`` times longer:

    * "linear": every frequency divided by ``factor``;
    * "ntk": the base enlarged so that the slowest pair slows down by
      ``factor`` and the fastest not at all;
    * "yarn": by how often a pair turns within ``original_length`` positions:
      kept from ``fast_turns`` on, divided by ``factor`` up to ``slow_turns``, a
      linear ramp over the pair's index between (``rope_mscale`` goes with it).
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even and positive, got {rotary_dim}")
    if not base > 0 or not factor >= 1.0:
        raise ValueError("base must be positive and factor at least 1")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    if scaling == "ntk" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = torch.pow(torch.tensor(float(base), dtype=torch.float64), -2.0 * i / rotary_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if original_length is None:
            raise ValueError('"yarn" needs original_length')
        if not base > 1.0 or not fast_turns > slow_turns > 0:
            raise ValueError("base must exceed 1 and fast_turns slow_turns")

        def index_of(turns):  # the (fractional) pair that turns this often
            return (rotary_dim * math.log(original_length / (turns * 2 * math.pi))
                    / (2 * math.log(base)))

        lo = max(0.0, math.floor(index_of(fast_turns)))
        # Beyond the last pair where even that one turns oftener than slow_turns.
        hi = min(rotary_dim - 1.0, math.ceil(index_of(slow_turns)))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        f = f * (1 - ramp) + f / factor * ramp
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device)


def rope_mscale(factor):
    """The amplitude that goes with "yarn" frequencies: 0.1 ln(factor) + 1."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0


def _output_like(t):
    """An output like t, the elements of a head side by side.  (Where t's elements share memory,
    empty_like orders the dimensions by their strides, and the last may not be the innermost.)"""
    o = torch.empty_like(t)
    return o if o.stride(-1) == 1 else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _rope_tensor(name, t, o, x):
    """Checks q or k against x (whichever of them is given first), and its output."""
    if t.dim() != 4:
        raise ValueError(f"{name}: expected [batch, seq, heads, head_dim], got {tuple(t.shape)}")
    _same(name, t, x.dtype, x.device)
    if t.shape[:2] != x.shape[:2] or t.shape[3] != x.shape[3]:
        raise ValueError(f"{name}: shape {tuple(t.shape)} does not go with {tuple(x.shape)}")
    _inner(name, t)
    if o is not None:
        _same(name + "_out", o, x.dtype, x.device)
        if o.shape != t.shape:
            raise ValueError(f"{name}_out: shape {tuple(o.shape)}, expected {tuple(t.shape)}")
        _inner(name + "_out", o)


def _check_rope(q, k, inv_freq, positions, q_out, k_out):
    if q is None and k is None:
        raise ValueError("q and k are both None")
    x = q if q is not None else k
    for name, t, o in (("q", q, q_out), ("k", k, k_out)):
        if t is not None:
            _rope_tensor(name, t, o, x)
    if x.dtype not in G.TORCH_DTYPE:
        raise ValueError(f"unsupported dtype {x.dtype}")
    _same("inv_freq", inv_freq, torch.float64, x.device, 1)
    if not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be contiguous")
    if positions is not None:
        b, s = x.shape[:2]
        if positions.dtype not in _INT_DTYPES or positions.device != x.device:
            raise ValueError("positions: int32 or int64 on the tensors' device")
        if positions.shape not in ((s,), (1, s), (b, s)):
            raise ValueError(f"positions: shape {tuple(positions.shape)}, expected "
                             f"({s},), (1, {s}) or ({b}, {s})")
        if s > 1 and positions.stride(-1) != 1:
            raise ValueError("positions must be contiguous along the sequence")
    _on_gpu(x)


def _rope(call, where, q, k, inv_freq, positions, layout, mscale, q_out, k_out, stream):
    if stream is not None and (q_out is None and q is not None or k_out is None and k is not None):
        _check_rope(q, k, inv_freq, positions, q_out, k_out)
        return _on_stream(stream, inv_freq.device, _rope, call, where, q, k, inv_freq, positions,
                          layout, mscale, q_out, k_out, None)
    # The usual call in one expression; anything else goes through the checks one by one.
    if not (q is not None and k is not None and q_out is None and k_out is None
            and positions is not None and q.dim() == 4 == k.dim() and q.stride(3) == 1 == k.stride(3)
            and positions.is_contiguous() and q.shape[:2] == k.shape[:2] == positions.shape
            and q.shape[3] == k.shape[3] and q.dtype is k.dtype and q.dtype in G.TORCH_DTYPE
            and positions.dtype in _INT_DTYPES and inv_freq.dtype is torch.float64
            and inv_freq.dim() == 1 and inv_freq.is_contiguous() and q.is_cuda
            and q.get_device() == k.get_device() == positions.get_device()
            == inv_freq.get_device()):
        _check_rope(q, k, inv_freq, positions, q_out, k_out)
    x = k if q is None else q
    b, s, _, d = x.shape
    hq = hk = qa = ka = qoa = koa = 0
    qs = ks = qo = ko = _NO_STRIDES
    if q is not None:
        q_out = _output_like(q) if q_out is None else q_out
        hq, qs, qo, qa, qoa = q.shape[2], q.stride(), q_out.stride(), q.data_ptr(), q_out.data_ptr()
    if k is not None:
        k_out = _output_like(k) if k_out is None else k_out
        hk, ks, ko, ka, koa = k.shape[2], k.stride(), k_out.stride(), k.data_ptr(), k_out.data_ptr()
    pos_stride, pos_bytes, pa = 0, 8, 0
    if positions is not None:
        pos_bytes, pa = positions.itemsize, positions.data_ptr()
        if positions.dim() == 2 and positions.shape[0] > 1:
            pos_stride = positions.stride(0)
    _launch(where, call,
            G.rope_args(qa, ka, pa, inv_freq.data_ptr(), qoa, koa, b, s, hq, hk, d,
                        2 * inv_freq.shape[0], qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], qo[0],
                        qo[1], qo[2], ko[0], ko[1], ko[2], pos_stride, pos_bytes,
                        G.TORCH_DTYPE[x.dtype], _ROPE_LAYOUT[layout], mscale),
            x.get_device(), stream)
    return q_out, k_out


def rope_fwd(q, k, inv_freq, positions=None, *, layout="half", mscale=1.0, q_out=None, k_out=None,
             stream=None):
    """Rotates q and k [batch, seq, heads, head_dim] (either may be None) to
    their positions ([seq], [1, seq] or [batch, seq] int32 / int64; None: 0, 1,
    ...) and returns (q_out, k_out), new tensors unless given (q and k
    themselves may be).  ``inv_freq``: ``rope_frequencies(rotary_dim)``; of the
    head's elements the first rotary_dim = 2 * len(inv_freq) turn.  ``layout``:
    pairs (i, i + rotary_dim / 2) ("half") or (2i, 2i + 1) ("interleaved")."""
    if _fast is not None and q_out is None and k_out is None and stream is None:
        r = _fast.rope(0, q, k, inv_freq, positions, _ROPE_LAYOUT[layout], mscale)
        if r is not None:
            return _taken(r, "gbn_rope_fwd")
    return _rope(G.library().gbn_rope_fwd, "gbn_rope_fwd", q, k, inv_freq, positions, layout, mscale, q_out,
                 k_out, stream)


def rope_bwd(dq, dk, inv_freq, positions=None, *, layout="half", mscale=1.0, dq_out=None,
             dk_out=None, stream=None):
    """Gradients of ``rope_fwd``'s inputs from those of its outputs."""
    if _fast is not None and dq_out is None and dk_out is None and stream is None:
        r = _fast.rope(1, dq, dk, inv_freq, positions, _ROPE_LAYOUT[layout], mscale)
        if r is not None:
            return _taken(r, "gbn_rope_bwd")
    return _rope(G.library().gbn_rope_bwd, "gbn_rope_bwd", dq, dk, inv_freq, positions, layout, mscale,
                 dq_out, dk_out, stream)


_E4M3_DTYPES = (torch.uint8, torch.float8_e4m3fn)


def _cache_dtype(k_cache, v_cache, dtype):
    c = k_cache.dtype
    if c in _E4M3_DTYPES and v_cache.dtype in _E4M3_DTYPES:
        return G.GBN_E4M3
    if v_cache.dtype != c:
        raise ValueError(f"v_cache: dtype {v_cache.dtype}, expected {c}")
    if c != dtype:
        raise ValueError(f"cache dtype {c}: expected {dtype}, or E4M3 codes (uint8, float8_e4m3fn)")
    return G.TORCH_DTYPE[c]


def _check_paged(x, k_cache, v_cache, cu_seqlens, kv_lens, block_table):
    """What both paged calls need of their tensors, one by one."""
    dev = x.device
    if x.dim() != 3:
        raise ValueError(f"expected [tokens, heads, head_dim], got {tuple(x.shape)}")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"unsupported dtype {x.dtype}: bfloat16 or float16")
    _cache_dtype(k_cache, v_cache, x.dtype)
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("caches: [pages, page_size, kv_heads, head_dim], the same for both; got "
                         f"{tuple(k_cache.shape)} and {tuple(v_cache.shape)}")
    if k_cache.shape[3] != x.shape[2]:
        raise ValueError(f"caches: head_dim {k_cache.shape[3]}, expected {x.shape[2]}")
    if k_cache.device != dev or v_cache.device != dev:
        raise ValueError(f"caches: not on {dev}")
    _inner("k_cache", k_cache)
    _inner("v_cache", v_cache)
    _same("cu_seqlens", cu_seqlens, torch.int32, dev, 1)
    _same("kv_lens", kv_lens, torch.int32, dev, 1)
    _same("block_table", block_table, torch.int32, dev, 2)
    n = kv_lens.shape[0]
    if cu_seqlens.shape[0] != n + 1 or block_table.shape[0] != n:
        raise ValueError(f"{n} kv_lens need {n + 1} cu_seqlens and {n} block_table rows, got "
                         f"{cu_seqlens.shape[0]} and {block_table.shape[0]}")
    if not (cu_seqlens.is_contiguous() and kv_lens.is_contiguous()):
        raise ValueError("cu_seqlens and kv_lens must be contiguous")
    _inner("block_table", block_table)


def _paged_args(x, k_cache, v_cache, cu_seqlens, kv_lens, block_table):
    """Checks what both paged calls share; (cache dtype, kv heads, head_dim)."""
    dt, i32 = x.dtype, torch.int32
    # The usual call in one expression; anything else goes through the checks one by one.
    if not (x.dim() == 3 and (dt is torch.bfloat16 or dt is torch.float16)
            and k_cache.dtype is v_cache.dtype and k_cache.dim() == 4
            and k_cache.shape == v_cache.shape and k_cache.shape[3] == x.shape[2]
            and k_cache.stride(3) == 1 == v_cache.stride(3)
            and cu_seqlens.dtype is i32 and kv_lens.dtype is i32 and block_table.dtype is i32
            and cu_seqlens.is_contiguous() and kv_lens.is_contiguous()
            and block_table.is_contiguous() and cu_seqlens.dim() == 1 == kv_lens.dim()
            and block_table.dim() == 2 and cu_seqlens.shape[0] - 1 == kv_lens.shape[0]
            == block_table.shape[0]
            and x.get_device() == k_cache.get_device() == v_cache.get_device()
            == cu_seqlens.get_device() == kv_lens.get_device() == block_table.get_device()):
        _check_paged(x, k_cache, v_cache, cu_seqlens, kv_lens, block_table)
    cdt = G.TORCH_DTYPE[dt] if k_cache.dtype is dt else _cache_dtype(k_cache, v_cache, dt)
    return cdt, k_cache.shape[2], k_cache.shape[3]


def _scalar(name, t, dev):
    _same(name, t, torch.float32, dev)
    if t.numel() != 1:
        raise ValueError(f"{name}: one element, got {t.numel()}")


def paged_append(k, v, k_cache, v_cache, cu_seqlens, kv_lens, block_table, *, q=None,
                 inv_freq=None, layout="half", mscale=1.0, k_scale=None, v_scale=None, q_out=None,
                 stream=None):
    """Writes the new tokens' k and v [tokens, kv_heads, head_dim] into the
    paged caches [pages, page_size, kv_heads, head_dim] (bf16 / f16 like k, or
    E4M3 codes as uint8 / float8_e4m3fn, then with k_scale and v_scale, fp32
    [1]).  Sequence b's tokens are rows cu_seqlens[b] .. cu_seqlens[b+1] - 1
    and become its last keys: kv_lens[b] counts them.  With ``inv_freq`` the
    keys are rotated to their positions on the way, and ``q`` [tokens, heads,
    head_dim], if given, into ``q_out`` (returned; a new tensor unless given,
    and then with unwritten padding rows)."""
    if _fast is not None and q_out is None and stream is None:
        r = _fast.append(k, v, k_cache, v_cache, cu_seqlens, kv_lens, block_table, q, inv_freq,
                         _ROPE_LAYOUT[layout], mscale, k_scale, v_scale)
        if r is not None:
            return _taken(r, "gbn_paged_append")
    cdt, hk, d = _paged_args(k, k_cache, v_cache, cu_seqlens, kv_lens, block_table)
    dev = k.device
    if stream is not None and q is not None and q_out is None and k.is_cuda:
        return _on_stream(stream, dev, paged_append, k, v, k_cache, v_cache, cu_seqlens, kv_lens,
                          block_table, q=q, inv_freq=inv_freq, layout=layout, mscale=mscale,
                          k_scale=k_scale, v_scale=v_scale)
    dt = k.dtype
    if v.dtype is not dt or v.dim() != 3 or v.get_device() != k.get_device():
        _same("v", v, dt, dev, 3)
    if v.shape != k.shape or k.shape[1] != hk:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)}: expected "
                         f"[tokens, {hk}, {d}]")
    _inner("k", k)
    _inner("v", v)
    hq, qs, qo = 0, (0, 0), (0, 0)
    if q is not None:
        if q.dtype is not dt or q.dim() != 3 or q.get_device() != k.get_device():
            _same("q", q, dt, dev, 3)
        if q.shape[0] != k.shape[0] or q.shape[2] != d:
            raise ValueError(f"q: shape {tuple(q.shape)} does not go with k {tuple(k.shape)}")
        _inner("q", q)
        if q_out is None:
            q_out = _output_like(q)
        else:
            _same("q_out", q_out, k.dtype, dev, 3)
            if q_out.shape != q.shape:
                raise ValueError(f"q_out: shape {tuple(q_out.shape)}, expected {tuple(q.shape)}")
            _inner("q_out", q_out)
        hq, qs, qo = q.shape[1], q.stride(), q_out.stride()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rot = 0
    if inv_freq is not None:
        _same("inv_freq", inv_freq, torch.float64, dev, 1)
        if not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be contiguous")
        rot = 2 * inv_freq.shape[0]
    if cdt == G.GBN_E4M3:
        if k_scale is None or v_scale is None:
            raise ValueError("E4M3 caches need k_scale and v_scale")
        _scalar("k_scale", k_scale, dev)
        _scalar("v_scale", v_scale, dev)
    _on_gpu(k)
    ks, vs, kc, vc = k.stride(), v.stride(), k_cache.stride(), v_cache.stride()
    _launch("gbn_paged_append", G.library().gbn_paged_append,
            G.append_args(0 if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
                          0 if q is None else q_out.data_ptr(), k_cache.data_ptr(),
                          v_cache.data_ptr(), 0 if inv_freq is None else inv_freq.data_ptr(),
                          0 if k_scale is None else k_scale.data_ptr(),
                          0 if v_scale is None else v_scale.data_ptr(), cu_seqlens.data_ptr(),
                          kv_lens.data_ptr(), block_table.data_ptr(), k.shape[0],
                          kv_lens.shape[0], hq, hk, d, rot, k_cache.shape[0], k_cache.shape[1],
                          block_table.shape[1], block_table.stride(0), qs[0], qs[1], ks[0], ks[1],
                          vs[0], vs[1], qo[0], qo[1], kc[0], kc[1], kc[2], vc[0], vc[1], vc[2],
                          G.TORCH_DTYPE[k.dtype], cdt, _ROPE_LAYOUT[layout], mscale),
            k.get_device(), stream)
    return q_out


@functools.lru_cache(maxsize=4096)
def _attention_bytes(device_index, *sizes):
    """Workspace bytes of an attention call, by its sizes (and the device's)."""
    with torch.cuda.device(device_index):
        st, n = G.gbn_paged_attention_workspace_size(*sizes)
    _check(st, "gbn_paged_attention_workspace_size")
    return n


def paged_attention_workspace(q, k_cache, block_table, *, max_q, max_kv=None, causal=True,
                              window=0):
    """A workspace for ``paged_attention`` calls of these sizes (None: they need none)."""
    cdt = _cache_dtype(k_cache, k_cache, q.dtype)
    mkv = min(block_table.shape[1] * k_cache.shape[1], 1 << 30) if max_kv is None else max_kv
    _on_gpu(q)
    n = _attention_bytes(q.get_device(), q.shape[0], block_table.shape[0], q.shape[1],
                         k_cache.shape[2], q.shape[2], k_cache.shape[1], block_table.shape[1],
                         max_q, mkv, window, bool(causal), G.TORCH_DTYPE[q.dtype], cdt)
    return torch.empty(n, dtype=torch.uint8, device=q.device) if n else None


def paged_attention(q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, *, max_q, max_kv=None,
                    scale=None, causal=True, window=0, k_scale_inv=None, v_scale_inv=None,
                    return_lse=False, out=None, lse=None, workspace=None, stream=None):
    """Attention of the new tokens q [tokens, heads, head_dim] over the paged
    caches (arguments as in ``paged_append``, which has run before).  max_q and
    max_kv bound the new tokens per sequence and kv_lens (max_kv: by default
    the table's room).  ``scale``: 1 / sqrt(head_dim) by default.  ``causal``:
    bottom-right aligned; ``window`` > 0: only the last ``window`` positions up
    to the token's own.  Returns out, or (out, lse) with ``return_lse``; both
    are new tensors unless given (padding rows are not written).
    ``workspace``: ``paged_attention_workspace``; allocated here when needed."""
    if (_fast is not None and out is None and lse is None and workspace is None
            and stream is None):
        r = _fast.attention(q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, max_q, max_kv,
                            scale, causal, window, k_scale_inv, v_scale_inv, return_lse)
        if r is not None:
            return _taken(r, "gbn_paged_attention")
    cdt, hk, d = _paged_args(q, k_cache, v_cache, cu_seqlens, kv_lens, block_table)
    dev, t, hq = q.device, q.shape[0], q.shape[1]
    _inner("q", q)
    if stream is not None and q.is_cuda:
        return _on_stream(stream, dev, paged_attention, q, k_cache, v_cache, cu_seqlens, kv_lens,
                          block_table, max_q=max_q, max_kv=max_kv, scale=scale, causal=causal,
                          window=window, k_scale_inv=k_scale_inv, v_scale_inv=v_scale_inv,
                          return_lse=return_lse, out=out, lse=lse, workspace=workspace)
    if out is None:
        out = _output_like(q)
    else:
        _same("out", out, q.dtype, dev, 3)
        if out.shape != q.shape:
            raise ValueError(f"out: shape {tuple(out.shape)}, expected {tuple(q.shape)}")
        _inner("out", out)
        if out.data_ptr() == q.data_ptr() and q.numel():
            raise ValueError("out must not be q")
    if return_lse and lse is None:
        lse = torch.empty(t, hq, dtype=torch.float32, device=dev)
    elif lse is not None:
        _same("lse", lse, torch.float32, dev)
        if lse.shape != (t, hq) or not lse.is_contiguous():
            raise ValueError(f"lse: contiguous [{t}, {hq}] expected")
    if cdt == G.GBN_E4M3:
        if k_scale_inv is None or v_scale_inv is None:
            raise ValueError("E4M3 caches need k_scale_inv and v_scale_inv")
        _scalar("k_scale_inv", k_scale_inv, dev)
        _scalar("v_scale_inv", v_scale_inv, dev)
    page, pages = k_cache.shape[1], block_table.shape[1]
    mkv = min(pages * page, 1 << 30) if max_kv is None else max_kv
    dt = G.TORCH_DTYPE[q.dtype]
    n = kv_lens.shape[0]
    _on_gpu(q)
    size = 0
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace: contiguous, on {dev}")
        size = workspace.numel() * workspace.element_size()
    else:
        size = _attention_bytes(q.get_device(), t, n, hq, hk, d, page, pages, max_q, mkv, window,
                                bool(causal), dt, cdt)
        if size:
            workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    qs, os, kc, vc = q.stride(), out.stride(), k_cache.stride(), v_cache.stride()
    _launch("gbn_paged_attention", G.library().gbn_paged_attention,
            G.attention_args(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                             cu_seqlens.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(),
                             0 if k_scale_inv is None else k_scale_inv.data_ptr(),
                             0 if v_scale_inv is None else v_scale_inv.data_ptr(),
                             out.data_ptr(), 0 if lse is None else lse.data_ptr(),
                             0 if workspace is None else workspace.data_ptr(), size, t, n, hq, hk,
                             d, k_cache.shape[0], page, pages, block_table.stride(0), max_q, mkv,
                             qs[0], qs[1], os[0], os[1], kc[0], kc[1], kc[2], vc[0], vc[1], vc[2],
                             window, dt, cdt, 1 if causal else 0,
                             d ** -0.5 if scale is None else scale),
            q.get_device(), stream)
    return (out, lse) if return_lse else out
