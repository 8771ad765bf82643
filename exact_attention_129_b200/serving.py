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
import importlib.util
import math
import os
import sys

import torch

__all__ = ["rope_frequencies", "attn_rotary", "rotary", "attn_paged_append", "attn_paged_fwd",
           "paged_workspace_size"]

_ea = sys.modules[__package__]  # the package's loader, looked up when it is needed

ABI = ("attn_rotary", "attn_paged_append", "attn_paged_fwd", "attn_paged_workspace_size")
_binding = None


def binding_path() -> str:
    """The compiled binding for the running Python and torch.  It is built against their
    C++ headers, so another version of either has another file and never loads this one."""
    tag = f"{sys.implementation.cache_tag}-torch{torch.__version__}"
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), f"_serving.{tag}.so")


def _load():
    """The compiled binding, bound to the loaded libattn.so."""
    global _binding
    path = binding_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m "
                          "exact_attention_129_b200.build`")
    lib = _ea.library()
    spec = importlib.util.spec_from_file_location(f"{__package__}._serving", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.init(_ea.AttnError,
                *(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in ABI), True)
    _binding = module
    return module


def rope_frequencies(rot_dim, base=10000.0, *, scaling=None, factor=1.0, original_max=None,
                     beta_fast=32.0, beta_slow=1.0, device=None):
    """Angles per position of ``rot_dim / 2`` pairs (fp64 tensor) and the factor
    on the rotated values.

    ``scaling`` stretches them for contexts ``factor`` times the trained one:
    None; "linear" (every angle divided by the factor); "ntk" (the base raised,
    so that the fastest pair keeps its angle and the slowest is divided by the
    factor); "yarn" (pairs that turn more than ``beta_fast`` times over
    ``original_max`` positions keep their angle, those under ``beta_slow`` turns
    are divided, a ramp between that is linear in the number of turns, as the YaRN
    paper defines it; the factor on the values is 0.1 ln(factor) + 1).  Some released
    checkpoints ramp linearly in the pair's index between two rounded bounds instead,
    which gives other angles in the middle: compute ``inv_freq`` as such a checkpoint
    does and pass that."""
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


def attn_rotary(q, k, inv_freq, *, cu_seqlens=None, offsets=None, positions=None,
                interleaved=False, mscale=1.0, inverse=False, q_out=None, k_out=None):
    """Rotates the first ``2 * len(inv_freq)`` elements of each row of q [T,Hq,D]
    and k [T,Hkv,D] (or None) by its position; returns (q_out, k_out).

    Pairs are (x[i], x[i + R/2]), or (x[2i], x[2i+1]) with ``interleaved``.  Row t
    has the position ``positions[t]``; or t - cu_seqlens[b] (+ offsets[b]) in its
    segment b; or t.  ``inverse`` turns the other way (the gradient).  q and k may
    be strided views; an output may be its input.  Rows behind the last segment
    are left as they were in outputs passed in, and zero in outputs made here."""
    return (_binding or _load()).rotary(q, k, inv_freq, cu_seqlens, offsets, positions,
                                        interleaved, mscale, inverse, q_out, k_out)


def rotary(q, k, inv_freq, *, cu_seqlens=None, offsets=None, positions=None, interleaved=False,
           mscale=1.0):
    """Differentiable attn_rotary: the gradient, of q and k, is the inverse rotation.

    A backward can be captured into a CUDA graph only when no eager graph of the same
    leaves is alive: torch refuses the capture otherwise, which can end the process, so
    drop the outputs of eager calls first."""
    return (_binding or _load()).rotary_grad(q, k, inv_freq, cu_seqlens, offsets, positions,
                                             interleaved, mscale)


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
    sequence are left as they were (undefined in an output made here)."""
    return (_binding or _load()).append(k, v, k_cache, v_cache, block_table, cu_seqlens, seqlens_k,
                                        max_seqlen, k_scale, v_scale, q, q_out, inv_freq,
                                        interleaved, mscale)


def paged_workspace_size(k_cache, v_cache, block_table, batch, total_q, max_seqlen_q, max_seqlen_k,
                         nheads_q, *, k_scale=None, v_scale=None, causal=False, window=None,
                         num_splits=0) -> int:
    """Bytes of workspace attn_paged_fwd needs for these arguments."""
    return (_binding or _load()).workspace_size(
        k_cache, v_cache, block_table, k_scale, v_scale, batch, total_q, max_seqlen_q,
        max_seqlen_k, nheads_q, causal, *_ea._window(window), num_splits)


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
    if None.  With ``num_splits`` 0 and many rows it may hold bf16 copies of all keys
    and values (up to 4 GiB): any other number avoids them."""
    return (_binding or _load()).fwd(q, k_cache, v_cache, block_table, cu_seqlens_q, seqlens_k,
                                     max_seqlen_q, max_seqlen_k, k_scale, v_scale, scale, causal,
                                     window, softcap, return_lse, out, lse, num_splits, workspace)
