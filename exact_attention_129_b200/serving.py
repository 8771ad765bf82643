"""Rotary positions and the paged key/value cache: the binding of attn_rotary,
attn_paged_append and attn_paged_fwd (``include/attn.h``).

A cache is a pool of pages, ``[num_pages, page_size, nheads_kv, head_dim]`` in
bf16 or e4m3 with any order of the outer dimensions in memory (a pool laid out
``[num_pages, nheads_kv, page_size, head_dim]`` is passed as
``pool.transpose(1, 2)``), and an int32 block table ``[batch, pages_per_seq]``.
An e4m3 cache has fp32 scales ``[num_pages, nheads_kv]`` for keys and values.
One decoding step of a layer is

    seqlens_k += 1
    q = attn_paged_append(k, v, k_cache, v_cache, block_table, cu, seqlens_k, 1,
                          k_scale=ks, v_scale=vs, q=q, inv_freq=inv_freq)
    out, _ = attn_paged_fwd(q, k_cache, v_cache, block_table, cu, seqlens_k, 1,
                            max_seqlen_k, k_scale=ks, v_scale=vs)
"""
from __future__ import annotations

import ctypes
import math
import struct
import sys

import torch

__all__ = ["rope_frequencies", "attn_rotary", "rotary", "attn_paged_append", "attn_paged_fwd",
           "paged_workspace_size"]

_ea = sys.modules[__package__]  # the package's checks and loader, looked up at each call

CACHE_TYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}
_CACHE = struct.Struct("5P7q6i")  # attn_paged_cache_t


def declare(lib):
    """Argument types of this module's part of the C ABI."""
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    rows = [vp, i64, i64]
    lib.attn_rotary.argtypes = rows * 4 + [vp, i32, i32, f32, i32, vp, vp, vp, i32, i32, i32, i32,
                                           i32, i32, vp]
    lib.attn_rotary.restype = ctypes.c_int
    lib.attn_paged_append.argtypes = [ctypes.c_char_p] + rows * 4 + [
        vp, vp, i32, i32, i32, i32, vp, i32, i32, f32, vp]
    lib.attn_paged_append.restype = ctypes.c_int
    lib.attn_paged_fwd.argtypes = [ctypes.c_char_p, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32,
                                   i32, i32, f32, i32, i32, vp, vp, vp, ctypes.c_size_t, vp]
    lib.attn_paged_fwd.restype = ctypes.c_int
    lib.attn_paged_workspace_size.argtypes = [ctypes.c_char_p, i32, i32, i32, i32, i32, i32, i32,
                                              i32, i32]
    lib.attn_paged_workspace_size.restype = ctypes.c_size_t


def rope_frequencies(rot_dim, base=10000.0, *, scaling=None, factor=1.0, original_max=None,
                     beta_fast=32.0, beta_slow=1.0, device=None):
    """Angles per position of ``rot_dim / 2`` pairs (fp64 tensor) and the factor
    on the rotated values.

    ``scaling`` stretches them for contexts ``factor`` times the trained one:
    None; "linear" (every angle divided by the factor); "ntk" (the base raised,
    so that the fastest pair keeps its angle and the slowest is divided by the
    factor); "yarn" (pairs that turn more than ``beta_fast`` times over
    ``original_max`` positions keep their angle, those under ``beta_slow`` turns
    are divided, a linear ramp between; the factor on the values is
    0.1 ln(factor) + 1)."""
    rot_dim = int(rot_dim)
    if rot_dim < 16 or rot_dim % 16:
        raise ValueError(f"rot_dim must be a positive multiple of 16, got {rot_dim}")
    if not base > 1 or not factor >= 1:
        raise ValueError("base must be above 1 and factor at least 1")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    freq, mscale = float(base) ** (-2 * i / rot_dim), 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "ntk":
        freq = (float(base) * factor ** (rot_dim / (rot_dim - 2))) ** (-2 * i / rot_dim)
    elif scaling == "yarn":
        if original_max is None or not original_max > 0 or not beta_fast > beta_slow:
            raise ValueError("yarn needs original_max > 0 and beta_fast > beta_slow")
        turns = original_max * freq / (2 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
        mscale = 0.1 * math.log(factor) + 1
    elif scaling is not None:
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq.to(device) if device is not None else freq, mscale


def _call(dev, name, *args):
    """A C ABI function with `dev` current, on its current stream."""
    fn = getattr(_ea.library(), name)
    if dev.type == "cuda" and dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            rc = fn(*args, _ea._stream(dev))
    else:
        rc = fn(*args, _ea._stream(dev))
    if rc != 0:
        raise _ea.AttnError(name, rc)


def _rows(name, t, dev, shape=None):
    """A bf16 [tokens, heads, head_dim] tensor or view that the kernels can read
    or write in 16-byte pieces: (pointer, token stride, head stride)."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim], got shape {tuple(t.shape)}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    st, sh, sd = t.stride()
    if sd != 1 or st % 8 or sh % 8 or t.data_ptr() % 16:
        raise ValueError(f"{name} must have a contiguous head_dim, strides that are multiples of 8 "
                         f"and a 16-byte aligned start, got strides {tuple(t.stride())}")
    return t.data_ptr(), st, sh


def _out_rows(name, out, src, dev):
    """(pointer, strides) of an output for the rows `src`: another tensor, or the
    very same memory."""
    p = _rows(name, out, dev, src.shape)
    st, sh, _ = out.stride()
    t, h, d = out.shape
    # distinct elements for distinct (token, head): no two threads may write one
    small, big = sorted(((abs(st), t), (abs(sh), h)))
    if (small[1] > 1 and small[0] < d) or (big[1] > 1 and big[0] < small[0] * (small[1] - 1) + d):
        raise ValueError(f"{name} overlaps itself, strides {tuple(out.stride())}")
    return p


def _ints(name, t, dev, shape):
    if t.dtype != torch.int32 or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    return t.data_ptr()


def _cu(name, t):
    if t.dim() != 1 or t.numel() < 2:
        raise ValueError(f"{name} must be a 1-D int32 tensor of batch + 1 offsets")
    return t.numel() - 1


def _freqs(inv_freq, dev, head_dim):
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous 1-D float64 tensor")
    if inv_freq.device != dev:
        raise ValueError(f"inv_freq is on {inv_freq.device}, expected {dev}")
    n = inv_freq.numel()
    if n % 8 or 2 * n > head_dim:
        raise ValueError(f"2 * len(inv_freq) must be a multiple of 16 up to head_dim {head_dim}, "
                         f"got {2 * n}")
    return inv_freq.data_ptr(), n


def attn_rotary(q, k, inv_freq, *, cu_seqlens=None, offsets=None, positions=None,
                interleaved=False, mscale=1.0, inverse=False, q_out=None, k_out=None):
    """Rotates the first ``2 * len(inv_freq)`` elements of each row of q [T,Hq,D]
    and k [T,Hkv,D] (or None) by its position; returns (q_out, k_out).

    Pairs are (x[i], x[i + R/2]), or (x[2i], x[2i+1]) with ``interleaved``.  Row t
    has the position ``positions[t]``; or t - cu_seqlens[b] (+ offsets[b]) in its
    segment b; or t.  ``inverse`` turns the other way (the gradient).  q and k may
    be strided views; an output may be its input.  Rows behind the last segment
    are left as they were in outputs passed in, and zero in outputs made here."""
    dev = q.device
    qp = _rows("q", q, dev)
    t, hq, d = q.shape
    kp, hkv = (None, 0, 0), 0
    if k is not None:
        kp, hkv = _rows("k", k, dev), k.shape[1]
        if k.shape[0] != t or k.shape[2] != d:
            raise ValueError(f"k {tuple(k.shape)} does not match q {tuple(q.shape)}")
    elif k_out is not None:
        raise ValueError("k_out without k")
    fp, nf = _freqs(inv_freq, dev, d)
    if positions is not None and cu_seqlens is not None:
        raise ValueError("positions and cu_seqlens exclude each other")
    if offsets is not None and cu_seqlens is None:
        raise ValueError("offsets need cu_seqlens")
    batch, pp, cp, op = 0, None, None, None
    if positions is not None:
        pp = _ints("positions", positions, dev, (t,))
    if cu_seqlens is not None:
        batch = _cu("cu_seqlens", cu_seqlens)
        cp = _ints("cu_seqlens", cu_seqlens, dev, (batch + 1,))
        if offsets is not None:
            op = _ints("offsets", offsets, dev, (batch,))
    if cu_seqlens is not None and (q_out is None) != (k is not None and k_out is None) and \
            k is not None:
        raise ValueError("with cu_seqlens, pass both outputs or neither")
    zero = q_out is None
    qop = _out_rows("q_out", q_out, q, dev) if q_out is not None else None
    kop = _out_rows("k_out", k_out, k, dev) if k_out is not None else None
    _ea._check_cuda(q)
    if qop is None:
        q_out = torch.empty((t, hq, d), dtype=q.dtype, device=dev)
        qop = (q_out.data_ptr(), hq * d, d)
    if k is not None and kop is None:
        k_out = torch.empty((t, hkv, d), dtype=k.dtype, device=dev)
        kop = (k_out.data_ptr(), hkv * d, d)
    if k is None:
        kop = (None, 0, 0)
    if t:
        _call(dev, "attn_rotary", *qp, *kp, *qop, *kop, fp, nf, bool(interleaved), float(mscale),
              bool(inverse), pp, cp, op, batch, zero, t, hq, hkv, d)
    return q_out, k_out


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, inv_freq, cu_seqlens, offsets, positions, interleaved, mscale):
        ctx.save_for_backward(inv_freq, cu_seqlens, offsets, positions)
        ctx.args = (interleaved, mscale)
        return attn_rotary(q, k, inv_freq, cu_seqlens=cu_seqlens, offsets=offsets,
                           positions=positions, interleaved=interleaved, mscale=mscale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk):
        inv_freq, cu_seqlens, offsets, positions = ctx.saved_tensors
        interleaved, mscale = ctx.args
        grads = [g if need else None for g, need in zip((dq, dk), ctx.needs_input_grad)]
        live = [_plain(g) for g in grads if g is not None]
        if live:
            back = attn_rotary(live[0], live[1] if len(live) > 1 else None, inv_freq,
                               cu_seqlens=cu_seqlens, offsets=offsets, positions=positions,
                               interleaved=interleaved, mscale=mscale, inverse=True)
            back = iter(back)
            grads = [None if g is None else next(back) for g in grads]
        return (*grads, None, None, None, None, None, None)


def _plain(t):
    """A gradient as the kernels can read it."""
    st, sh, sd = t.stride()
    return t if sd == 1 and st % 8 == 0 and sh % 8 == 0 and t.data_ptr() % 16 == 0 else \
        t.clone(memory_format=torch.contiguous_format)


def rotary(q, k, inv_freq, *, cu_seqlens=None, offsets=None, positions=None, interleaved=False,
           mscale=1.0):
    """Differentiable attn_rotary: the gradient is the inverse rotation."""
    return _Rotary.apply(q, k, inv_freq, cu_seqlens, offsets, positions, bool(interleaved),
                         float(mscale))


def _cache(k_cache, v_cache, k_scale, v_scale, block_table, dev):
    """attn_paged_cache_t of the tensors, and (nheads_kv, head_dim)."""
    kind = CACHE_TYPES.get(k_cache.dtype)
    if kind is None:
        raise ValueError(f"k_cache must be bfloat16 or float8_e4m3fn, got {k_cache.dtype}")
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, nheads_kv, head_dim] "
                         f"of one type, got {tuple(shape)} and {tuple(v_cache.shape)}")
    pages, page, hkv, d = shape
    if page not in (16, 32, 64, 128):
        raise ValueError(f"page_size must be 16, 32, 64 or 128, got {page}")
    step = 16 if kind else 8
    strides = []
    for n, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if t.device != dev:
            raise ValueError(f"{n} is on {t.device}, expected {dev}")
        s = t.stride()
        if s[3] != 1 or s[0] % step or s[1] % step or s[2] % step or t.data_ptr() % 16:
            raise ValueError(f"{n} must have a contiguous head_dim, strides that are multiples of "
                             f"16 bytes and a 16-byte aligned start, got strides {s}")
        strides += s[:3]
    scales = [None, None]
    if kind:
        for i, (n, t) in enumerate((("k_scale", k_scale), ("v_scale", v_scale))):
            if t is None or t.dtype != torch.float32 or tuple(t.shape) != (pages, hkv) or \
                    not t.is_contiguous() or t.device != dev:
                raise ValueError(f"{n} must be a contiguous float32 tensor of shape {(pages, hkv)} "
                                 f"on {dev} for an e4m3 cache")
            scales[i] = t.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError("scales belong to an e4m3 cache")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be int32 [batch, pages_per_seq] with contiguous rows")
    if block_table.device != dev:
        raise ValueError(f"block_table is on {block_table.device}, expected {dev}")
    return _CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), scales[0] or 0, scales[1] or 0,
                       block_table.data_ptr(), *strides, block_table.stride(0), kind, pages, page,
                       block_table.shape[1], hkv, d), hkv, d


def attn_paged_append(k, v, k_cache, v_cache, block_table, cu_seqlens, seqlens_k, max_seqlen, *,
                      k_scale=None, v_scale=None, q=None, q_out=None, inv_freq=None,
                      interleaved=False, mscale=1.0):
    """Writes the new rows k, v [T,Hkv,D] of each sequence into its pages, k
    rotated by its position (``inv_freq`` None: as it is), and returns q [T,Hq,D]
    rotated the same way (None without q).

    ``cu_seqlens`` packs the new rows, at most ``max_seqlen`` for a sequence;
    ``seqlens_k`` [batch] counts each sequence's tokens, the new ones included.
    An e4m3 cache is written under one power-of-two scale per page and head,
    which grows as larger values arrive (see attn_paged_append in attn.h); the
    scales are updated in place.  ``q_out`` may be q; rows behind the last
    sequence are left as they were."""
    dev = k.device
    kp = _rows("k", k, dev)
    vp = _rows("v", v, dev, k.shape)
    cache, hkv, d = _cache(k_cache, v_cache, k_scale, v_scale, block_table, dev)
    t = k.shape[0]
    if k.shape[1] != hkv or k.shape[2] != d:
        raise ValueError(f"k {tuple(k.shape)} does not match the cache's {hkv} heads of {d}")
    batch = _cu("cu_seqlens", cu_seqlens)
    cp = _ints("cu_seqlens", cu_seqlens, dev, (batch + 1,))
    sp = _ints("seqlens_k", seqlens_k, dev, (batch,))
    if block_table.shape[0] != batch:
        raise ValueError(f"block_table has {block_table.shape[0]} rows for {batch} sequences")
    qp, qop, hq = (None, 0, 0), (None, 0, 0), 0
    if q is not None:
        qp, hq = _rows("q", q, dev), q.shape[1]
        if q.shape[0] != t or q.shape[2] != d:
            raise ValueError(f"q {tuple(q.shape)} does not match k {tuple(k.shape)}")
        if q_out is not None:
            qop = _out_rows("q_out", q_out, q, dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    fp, nf = (None, 0) if inv_freq is None else _freqs(inv_freq, dev, d)
    _ea._check_cuda(k)
    if q is not None and q_out is None:
        q_out = torch.empty((t, hq, d), dtype=q.dtype, device=dev)
        qop = (q_out.data_ptr(), hq * d, d)
    if t:
        _call(dev, "attn_paged_append", cache, *kp, *vp, *qp, *qop, cp, sp, batch, t,
              int(max_seqlen), hq, fp, nf, bool(interleaved), float(mscale))
    return q_out


def paged_workspace_size(k_cache, v_cache, block_table, batch, total_q, max_seqlen_q, max_seqlen_k,
                         nheads_q, *, k_scale=None, v_scale=None, causal=False, window=None,
                         num_splits=0) -> int:
    """Bytes of workspace attn_paged_fwd needs for these arguments."""
    cache = _cache(k_cache, v_cache, k_scale, v_scale, block_table, k_cache.device)[0]
    wl, wr = _ea._window(window)
    return int(_ea.library().attn_paged_workspace_size(
        cache, batch, total_q, int(max_seqlen_q), int(max_seqlen_k), nheads_q, bool(causal), wl,
        wr, int(num_splits)))


def attn_paged_fwd(q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k, max_seqlen_q,
                   max_seqlen_k, *, k_scale=None, v_scale=None, scale=None, causal=False,
                   window=None, softcap=0.0, return_lse=True, out=None, lse=None, num_splits=0,
                   workspace=None):
    """Attention of the packed query rows q [T,Hq,D] over a paged cache; returns
    (out, lse or None).

    ``seqlens_k`` [batch] counts each sequence's keys; with ``causal`` or
    ``window`` its query rows are the last ones.  ``scale``, ``window`` and
    ``softcap`` are as in attn_fwd.  ``num_splits`` 0 lets the library cut the keys
    into parts; ``workspace`` (at least paged_workspace_size bytes) is allocated
    if None."""
    dev = q.device
    if q.dim() != 3:
        raise ValueError(f"q must be [tokens, heads, head_dim], got shape {tuple(q.shape)}")
    _ea._check_layout("q", q, torch.bfloat16)
    t, hq, d = q.shape
    cache, hkv, dc = _cache(k_cache, v_cache, k_scale, v_scale, block_table, dev)
    if dc != d:
        raise ValueError(f"q and the cache differ in head_dim: {d} and {dc}")
    if hq % hkv:
        raise ValueError(f"nheads_q {hq} is not a multiple of nheads_kv {hkv}")
    batch = _cu("cu_seqlens_q", cu_seqlens_q)
    cp = _ints("cu_seqlens_q", cu_seqlens_q, dev, (batch + 1,))
    sp = _ints("seqlens_k", seqlens_k, dev, (batch,))
    if block_table.shape[0] != batch:
        raise ValueError(f"block_table has {block_table.shape[0]} rows for {batch} sequences")
    _ea._check_like("out", out, q.shape, torch.bfloat16, dev)
    _ea._check_like("lse", lse, (hq, t), torch.float32, dev)
    if workspace is not None and (not workspace.is_contiguous() or workspace.device != dev):
        raise ValueError("workspace must be a contiguous tensor on q's device")
    _ea._check_cuda(q)
    if scale is None:
        scale = d ** -0.5
    if out is None:
        out = torch.empty_like(q)
    if not return_lse:
        lse = None
    elif lse is None:
        lse = torch.empty((hq, t), device=dev, dtype=torch.float32)
    if t == 0:
        return out, lse
    wl, wr = _ea._window(window)
    max_q, max_k, splits = int(max_seqlen_q), int(max_seqlen_k), int(num_splits)
    causal = bool(causal)
    if workspace is None:
        need = _ea.library().attn_paged_workspace_size(cache, batch, t, max_q, max_k, hq, causal,
                                                       wl, wr, splits)
        if need:
            workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    _call(dev, "attn_paged_fwd", cache, q.data_ptr(), cp, sp, batch, t, max_q, max_k, hq,
          float(scale), causal, wl, wr, float(softcap or 0.0), splits, bool(return_lse),
          out.data_ptr(), None if lse is None else lse.data_ptr(),
          None if workspace is None else workspace.data_ptr(),
          0 if workspace is None else workspace.numel() * workspace.element_size())
    return out, lse
