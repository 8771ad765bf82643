"""Plain 64-bit definitions of rotary positions, the paged append and attention
over a paged cache, and the error bounds their GPU tests use (CPU only)."""
from __future__ import annotations

import math

import torch

E4M3 = torch.float8_e4m3fn
U_BF16 = 2.0 ** -8   # half a step, relative to the value
U_F16 = 2.0 ** -11
U_E4M3 = 2.0 ** -4
# fp32 cosines and sines of an angle rounded to fp32 in half turns, times mscale,
# and the two products of a pair: each part is within a few 2^-24 of its factor
ROT_ERR = 2.0 ** -20


def rotate(x, pos, inv_freq, mscale=1.0, interleaved=False, inverse=False):
    """x [T, H, D] float64 rotated by positions [T]."""
    x = x.double()
    half = inv_freq.numel()
    ang = pos.double()[:, None] * inv_freq.double()[None, :]
    c = (mscale * ang.cos())[:, None]
    s = (mscale * ang.sin())[:, None] * (-1 if inverse else 1)
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * c - b * s, b * c + a * s
    return y


def rotate_slack(x, inv_freq, mscale=1.0, interleaved=False):
    """Bound on the fp32 part of the error: ROT_ERR * m * (|a| + |b|) per pair, 0 elsewhere."""
    x = x.double().abs()
    half = inv_freq.numel()
    y = torch.zeros_like(x)
    if interleaved:
        p = x[..., 0:2 * half:2] + x[..., 1:2 * half:2]
        y[..., 0:2 * half:2] = y[..., 1:2 * half:2] = p
    else:
        p = x[..., :half] + x[..., half:2 * half]
        y[..., :half] = y[..., half:2 * half] = p
    return ROT_ERR * abs(mscale) * y


def positions(cu, offsets=None):
    """Positions of the packed rows of segments cu (a list)."""
    offsets = offsets or [0] * (len(cu) - 1)
    return torch.cat([torch.arange(o, o + b - a) for a, b, o in zip(cu, cu[1:], offsets)]
                     + [torch.zeros(0, dtype=torch.long)])


def need_exponent(y):
    """Least e >= -64 with max |y| <= 448 * 2^e over the finite y."""
    y = y.double().abs()
    y = y[torch.isfinite(y)]
    top = float(y.max()) if y.numel() else 0.0
    if top == 0.0:
        return -64
    m, e = math.frexp(top)  # 448 = 0.875 * 2^9
    return max(-64, e - 9 + (1 if m > 0.875 else 0))


def to_e4m3(x):
    """float64 -> e4m3, ties to even; not finite -> NaN.  The argument fits fp32 exactly."""
    return x.float().to(E4M3)


def append(x, cache, scale, table, cu, lens):
    """The bf16 rows x [T, H, D] into cache [pages, page, H, D] (in place), scale
    [pages, H] for e4m3."""
    page = cache.shape[1]
    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b]
        start = lens[b] - n
        lo = max(start, 0)
        j = lo // page
        while j * page < lens[b] and n > 0:
            a, z = max(lo, j * page), min(lens[b], (j + 1) * page)
            if j >= table.shape[1]:
                break
            at = int(table[b, j])
            if 0 <= at < cache.shape[0]:
                rows = x[cu[b] + a - start:cu[b] + z - start]
                if scale is None:
                    cache[at, a - j * page:z - j * page] = rows
                else:
                    for h in range(x.shape[1]):
                        need = 2.0 ** need_exponent(rows[:, h])
                        old = float(scale[at, h])
                        new = need if a == j * page else max(old, need)
                        if a > j * page and new > old:
                            kept = cache[at, :a - j * page, h].double() * (old / new)
                            cache[at, :a - j * page, h] = to_e4m3(kept)
                        scale[at, h] = new
                        cache[at, a - j * page:z - j * page, h] = to_e4m3(
                            rows[:, h].double() / new)
            j += 1


def keys_of(cache, scale, table_row, n):
    """The first n tokens of a sequence, float64 [n, H, D]."""
    page = cache.shape[1]
    at = table_row[:-(-n // page)].long()
    x = cache[at].double()
    if scale is not None:
        x = x * scale[at].double()[:, None, :, None]
    return x.flatten(0, 1)[:n]


def attend(q, k_cache, v_cache, k_scale, v_scale, table, cu, lens, scale, causal=False,
           window=None, softcap=0.0):
    """(O [T, Hq, D], LSE [Hq, T], sum_j p_j |v_j|), float64; rows of no sequence are NaN."""
    t, hq, d = q.shape
    hkv = k_cache.shape[2]
    left, right = (-1, -1) if window is None else window
    out = torch.full((t, hq, d), math.nan, dtype=torch.float64)
    pabs = out.clone()
    lse = torch.full((hq, t), math.nan, dtype=torch.float64)
    for b in range(len(cu) - 1):
        nq, nk = cu[b + 1] - cu[b], lens[b]
        rows = slice(cu[b], cu[b + 1])
        if nq == 0:
            continue
        k = keys_of(k_cache, k_scale, table[b], nk).repeat_interleave(hq // hkv, 1)
        v = keys_of(v_cache, v_scale, table[b], nk).repeat_interleave(hq // hkv, 1)
        s = torch.einsum("ihd,jhd->hij", q[rows].double(), k) * scale
        if softcap > 0:
            s = softcap * torch.tanh(s / softcap)
        i = torch.arange(nq)[:, None] + nk - nq
        j = torch.arange(nk)[None, :]
        see = torch.ones(nq, nk, dtype=torch.bool)
        if causal:
            see &= j <= i
        if right >= 0:
            see &= j <= i + right
        if left >= 0:
            see &= j >= i - left
        s = s.masked_fill(~see, -math.inf)
        lse[:, rows] = torch.logsumexp(s, -1) if nk else torch.full((hq, nq), -math.inf)
        m = lse[:, rows][..., None]
        p = torch.where(see & (m > -math.inf), torch.exp(s - torch.where(m > -math.inf, m, 0.0)),
                        0.0)
        # a key that a row does not see contributes nothing, whatever its value is
        vz = torch.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0)
        out[rows] = torch.einsum("hij,jhd->ihd", p, vz)
        pabs[rows] = torch.einsum("hij,jhd->ihd", p, vz.abs())
        bad = (~torch.isfinite(v)).double()
        hit = torch.einsum("hij,jhd->ihd", see.double().expand(hq, nq, nk), bad) > 0
        out[rows] = torch.where(hit, math.nan, out[rows])
    return out, lse, pabs


def o_bound(ref, pabs, e4m3):
    """|O - ref|: O rounded to bf16 (half a step of |ref|), P rounded to bf16, or
    to f16 for e4m3 (half a step of each weight, sum_j p_j |v_j| in all), and
    2^-11 of that sum for the fp32 scores, exponentials and sums."""
    p = (U_F16 if e4m3 else U_BF16) + 2.0 ** -11
    return U_BF16 * (1 + 2.0 ** -6) * ref.abs() + p * (1 + 2.0 ** -6) * pabs + 1e-30


class Cache:
    """A pool with pages dealt out at random to sequences of the given lengths."""

    def __init__(self, lens, room, hkv, d, page, e4m3, head_major=True, seed=0, spread=1.0,
                 junk=None, spare=3):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(a, r) // page) for a, r in zip(lens, room)]
        self.pages = sum(need) + spare
        width = max(need + [1])
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), width), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.page, self.lens, self.e4m3 = page, list(lens), e4m3
        for name in ("k", "v"):
            x = torch.randn(self.pages, page, hkv, d, generator=g, dtype=torch.float64)
            x *= torch.exp(spread * torch.randn(self.pages, 1, hkv, 1, generator=g,
                                                dtype=torch.float64))
            scale = None
            if e4m3:
                scale = torch.empty(self.pages, hkv)
                for i in range(self.pages):
                    for h in range(hkv):
                        scale[i, h] = 2.0 ** need_exponent(x[i, :, h])
                x = to_e4m3((x / scale[:, None, :, None].double()).float().double())
            else:
                x = x.to(torch.bfloat16)
            if junk is not None:  # slots that hold no token of a sequence
                owner = torch.zeros(self.pages, page, dtype=torch.bool)
                for b, n in enumerate(lens):
                    for t in range(n):
                        owner[self.table[b, t // page], t % page] = True
                x = torch.where(owner[:, :, None, None], x.float(), junk).to(x.dtype)
            if head_major:
                x = x.transpose(1, 2).contiguous().transpose(1, 2)
            setattr(self, name, x)
            setattr(self, name + "_scale", scale)

    def to(self, dev):
        """(k, v, table, scales as keyword arguments) on a device, strides kept."""
        def move(x):
            y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=dev)
            return y.copy_(x)
        kw = {"k_scale": self.k_scale.to(dev), "v_scale": self.v_scale.to(dev)} if self.e4m3 else {}
        return move(self.k), move(self.v), self.table.to(dev), kw
