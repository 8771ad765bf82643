"""Cases for the serving operators: rotary positions, appending to a paged
key/value cache, and attention over that cache.

``run`` computes a case either in plain torch operations (``own`` false) or
through the package's entry points (``own`` true); ``exact`` gives the same
outputs from the definitions in 64 bits.

A cache is a pool of pages, indexed [page, token of the page, key/value head,
head_dim]; ``block_table[b, j]`` is the page of sequence b's tokens
[j * page_size, (j + 1) * page_size).  An e4m3 cache has one fp32 scale for each
(page, key/value head), for the keys and for the values.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -64  # smallest block scale: 2^-64


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # training: the packed batch of the framework's varlen workload, forward and gradient
        _rotary("rotary, packed batch, train", 16384, 128, 4096, 32, 8, 128, 128, False, "none",
                True),
        # one 128K sequence, GQA-8 at head_dim 256, a quarter of the head rotated, long-context frequencies
        _rotary("rotary, 128K, part of the head", 131072, 131072, 131072, 8, 1, 256, 64, True,
                "yarn", False),
        # the tokens of one decoding step of four sequences: latency
        _rotary("rotary, 4 single tokens", 4, 1, 1, 32, 8, 128, 128, False, "linear", False),
        # a decoding step of 64 sequences into an 8-bit cache, q rotated too
        _append("append, 64 single tokens", 64, 1, 1, 1, 512, 32, 8, 128, 128, False, "e4m3", 64,
                True, True),
        # a packed batch of prompts into an 8-bit cache
        _append("append, prompts", 9, 128, 4096, 0, 0, 32, 8, 128, 128, False, "e4m3", 64, True,
                True),
        # drafted tokens of a small batch, small pages, bf16
        _append("append, drafts", 7, 1, 5, 1, 700, 16, 16, 64, 32, True, "bf16", 16, False, False),
        # one sequence of about a thousand tokens: latency
        _attend("attend, one short sequence", 1, 1, 1, 1000, 1000, 32, 8, 128, "e4m3", 64, True,
                -1, 0.0),
        # decoding over long contexts
        _attend("attend, 16 x 64K", 16, 1, 1, 65536, 65536, 32, 8, 128, "e4m3", 64, True, -1, 0.0),
        # a ragged decoding batch over a bf16 cache of small pages, tokens before heads
        _attend("attend, ragged batch", 128, 1, 1, 1, 8192, 32, 8, 128, "bf16", 16, False, -1, 0.0),
        # drafted tokens verified at once, GQA-8, head_dim 256, capped scores
        _attend("attend, drafts", 32, 1, 5, 100, 16384, 8, 1, 256, "e4m3", 128, True, -1, 50.0),
        # a sliding window, MHA, head_dim 64
        _attend("attend, window", 16, 1, 1, 9000, 16384, 16, 16, 64, "e4m3", 32, True, 4095, 0.0),
        # the next chunk of two long prompts
        _attend("attend, prompt chunks", 2, 1024, 1024, 16000, 16384, 32, 8, 128, "e4m3", 64, True,
                -1, 0.0),
    ]


def _rotary(name, tokens, lo, hi, hq, hkv, d, rot, interleaved, scaling, train):
    return {"name": name, "op": "rotary", "tokens": tokens, "lo": lo, "hi": hi, "hq": hq,
            "hkv": hkv, "d": d, "rot": rot, "interleaved": interleaved, "scaling": scaling,
            "train": train, "mix": 1}


def _append(name, batch, n_lo, n_hi, old_lo, old_hi, hq, hkv, d, rot, interleaved, kind, page,
            with_q, head_major):
    return {"name": name, "op": "append", "batch": batch, "n_lo": n_lo, "n_hi": n_hi,
            "old_lo": old_lo, "old_hi": old_hi, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "interleaved": interleaved, "kind": kind, "page": page, "with_q": with_q,
            "head_major": head_major, "mix": 1}


def _attend(name, batch, n_lo, n_hi, k_lo, k_hi, hq, hkv, d, kind, page, head_major, left, cap):
    return {"name": name, "op": "attend", "batch": batch, "n_lo": n_lo, "n_hi": n_hi,
            "k_lo": k_lo, "k_hi": k_hi, "hq": hq, "hkv": hkv, "d": d, "kind": kind, "page": page,
            "head_major": head_major, "left": left, "cap": cap, "mix": 1}


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


HEADS = [(32, 8, 128), (8, 1, 256), (16, 16, 64), (8, 2, 64), (4, 4, 128), (6, 2, 128), (8, 8, 256),
         (5, 1, 64)]


def draw(rng):
    op = rng.choice(["rotary", "append", "attend"])
    hq, hkv, d = rng.choice(HEADS)
    mix = rng.randrange(1 << 30)
    if op == "rotary":
        tokens = _spread(rng, 1, min(131072, (1 << 27) // (hq * d)))
        lo = _spread(rng, 1, tokens)
        c = _rotary("", tokens, lo, _spread(rng, lo, tokens), hq, hkv, d,
                    16 * rng.randint(1, d // 16), rng.random() < 0.5,
                    rng.choice(["none", "linear", "ntk", "yarn"]), rng.random() < 0.5)
    elif op == "append":
        batch = _spread(rng, 1, 256)
        n_hi = _spread(rng, 1, max(1, min(4096, 20000 // batch)))
        old_hi = _spread(rng, 1, max(1, min(4096, 40000 // batch)))
        c = _append("", batch, rng.randint(0, n_hi), n_hi, rng.randint(0, old_hi), old_hi, hq, hkv,
                    d, 16 * rng.randint(1, d // 16), rng.random() < 0.5,
                    rng.choice(["e4m3", "bf16"]), rng.choice([16, 32, 64, 128]),
                    rng.random() < 0.6, rng.random() < 0.5)
    else:
        batch = _spread(rng, 1, 128)
        k_hi = _spread(rng, 1, max(16, min(131072, (1 << 29) // (batch * hkv * d))))
        few = rng.random() < 0.7
        n_hi = _spread(rng, 1, 8 if few else max(8, min(1024, (1 << 29) // (batch * hq * k_hi))))
        n_hi = max(1, min(n_hi, (1 << 29) // (batch * hq * k_hi)))
        c = _attend("", batch, rng.randint(1, n_hi), n_hi, rng.randint(0, k_hi), k_hi, hq, hkv, d,
                    rng.choice(["e4m3", "bf16"]), rng.choice([16, 32, 64, 128]),
                    rng.random() < 0.5, rng.choice([-1, -1, _spread(rng, 1, k_hi)]),
                    rng.choice([0.0, 0.0, 30.0]))
    del c["name"]
    c["mix"] = mix
    return c


def _lengths(case):
    """Lengths of a case's sequences, from the case alone: (new tokens or query
    rows, tokens before them or keys)."""
    r = random.Random(case["mix"])
    if case["op"] == "rotary":
        left, n = case["tokens"], []
        while left > 0:
            n.append(min(left, r.randint(case["lo"], case["hi"])))
            left -= n[-1]
        # where each sequence begins: its tokens may follow others seen before
        return n, [0 if case["train"] else r.randint(0, 100000) for _ in n]
    n = [r.randint(case["n_lo"], case["n_hi"]) for _ in range(case["batch"])]
    n[0] = max(n[0], 1)
    if case["op"] == "append":
        return n, [r.randint(case["old_lo"], case["old_hi"]) for _ in range(case["batch"])]
    return n, [r.randint(case["k_lo"], case["k_hi"]) for _ in range(case["batch"])]


def _cu(n):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return cu


def _visible(rows, keys, left):
    """(row, key) pairs that a causal mask and a left window bound allow."""
    total = 0
    for nq, nk in zip(rows, keys):
        for i in range(nq):
            hi = min(nk - 1, i + nk - nq)
            lo = 0 if left < 0 else max(0, i + nk - nq - left)
            total += max(0, hi - lo + 1)
    return total


def work(case):
    n, before = _lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    t = sum(n)
    if case["op"] == "rotary":
        row = (hq + hkv) * d * 2
        passes = 2 if case["train"] else 1
        return {"bytes": passes * t * 2 * row + 8.0 * case["rot"] / 2,
                "flops": passes * t * (hq + hkv) * case["rot"] * 3.0}
    size = 1 if case["kind"] == "e4m3" else 2
    if case["op"] == "append":
        bytes_ = 2.0 * t * hkv * d * (2 + size) + (4.0 * t * hq * d if case["with_q"] else 0.0)
        return {"bytes": bytes_,
                "flops": 3.0 * t * case["rot"] * (hkv + (hq if case["with_q"] else 0))}
    # keys that some row of the sequence sees
    seen = 0
    for nq, nk in zip(n, before):
        lo = 0 if case["left"] < 0 else max(0, nk - nq - case["left"])
        seen += max(0, nk - lo)
    return {"bytes": 2.0 * seen * hkv * d * size + 4.0 * t * hq * d + 4.0 * t * hq,
            "flops": 4.0 * _visible(n, before, case["left"]) * hq * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _frequencies(rot, scaling):
    """Angle per position of each pair (64 bits), and the factor on cos and sin."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    base, factor, trained = 10000.0, 8.0, 8192.0
    plain = base ** (-2.0 * i / rot)
    if scaling == "none":
        return plain, 1.0
    if scaling == "linear":
        return plain / factor, 1.0
    if scaling == "ntk":
        return (base * factor ** (rot / max(rot - 2.0, 1.0))) ** (-2.0 * i / rot), 1.0
    # yarn: frequencies that turn often over the trained length stay, slow ones are stretched
    turns = trained * plain / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
    return plain * keep + plain / factor * (1 - keep), 0.1 * math.log(factor) + 1.0


def _pow2(e):
    """2^e for whole e, without rounding, in 64 bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _ints(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _pool(pages, page, hkv, d, kind, head_major, gen, dev):
    """A pool of written pages and its scales (None for bf16)."""
    shape = (pages, hkv, page, d) if head_major else (pages, page, hkv, d)
    x = torch.randn(shape, generator=gen, device=dev)
    view = x.transpose(1, 2) if head_major else x
    view *= torch.exp(0.4 * torch.randn((pages, 1, hkv, 1), generator=gen, device=dev))
    if kind == "bf16":
        x = x.to(torch.bfloat16)
        return (x.transpose(1, 2) if head_major else x), None
    top = torch.linalg.vector_norm(view, ord=math.inf, dim=(1, 3)) / E4M3_MAX
    m, e = torch.frexp(top)
    scale = _pow2(e - (m == 0.5).int()).float()
    view /= scale[:, None, :, None]
    x = x.to(torch.float8_e4m3fn)
    return (x.transpose(1, 2) if head_major else x), scale


def _table(lengths, page, gen, dev):
    """A block table with every sequence's pages scattered over the pool; rows
    are padded with page 0."""
    need = [-(-n // page) for n in lengths]
    total, width = max(1, sum(need)), max(1, max(need))
    at = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    counts = torch.tensor(need, device=dev)
    start = counts.cumsum(0) - counts
    j = torch.arange(width, device=dev)
    inside = j[None, :] < counts[:, None]
    idx = (start[:, None] + j[None, :]).clamp(max=total - 1)
    return torch.where(inside, at[idx], torch.zeros((), dtype=torch.int32, device=dev)), total


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(int(seed))
    n, before = _lengths(case)
    hq, hkv, d, t = case["hq"], case["hkv"], case["d"], sum(n)
    s = {"case": case, "cu": _ints(_cu(n), dev)}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev).to(torch.bfloat16)

    if case["op"] == "rotary":
        freq, s["mscale"] = _frequencies(case["rot"], case["scaling"])
        s["inv_freq"] = freq.to(dev)
        s["offsets"] = _ints(before, dev)
        if case["train"]:
            s["q"] = normal(t, hq, d).requires_grad_(True)
            s["k"] = normal(t, hkv, d).requires_grad_(True)
            s["dq"], s["dk"] = normal(t, hq, d), normal(t, hkv, d)
        else:  # views of one fused projection
            qkv = normal(t, hq + 2 * hkv, d)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hkv]
        return s
    s["max_n"] = max(n)
    if case["op"] == "append":
        freq, s["mscale"] = _frequencies(case["rot"], "none")
        s["inv_freq"] = freq.to(dev)
        lengths = [a + b for a, b in zip(n, before)]
        qkv = normal(t, hq + 2 * hkv, d)
        qkv *= torch.exp(0.4 * torch.randn((t, hq + 2 * hkv, 1), generator=gen,
                                           device=dev)).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        lengths = before
        s["q"] = normal(t, hq, d)
        s["max_k"] = max(lengths)
    s["seqlens"] = _ints(lengths, dev)
    s["table"], pages = _table(lengths, case["page"], gen, dev)
    for x in ("k", "v"):
        s[x + "_cache"], s[x + "_scale"] = _pool(pages, case["page"], hkv, d, case["kind"],
                                                 case["head_major"], gen, dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return {"rotary": _run_rotary, "append": _run_append, "attend": _run_attend}[
        s["case"]["op"]](s)


def _run_rotary(s):
    c = s["case"]
    if own:
        import exact_attention_129_b200 as ea
        args = dict(cu_seqlens=s["cu"], offsets=s["offsets"], interleaved=c["interleaved"],
                    mscale=s["mscale"])
        if not c["train"]:
            return ea.attn_rotary(s["q"], s["k"], s["inv_freq"], **args)
        q, k = ea.rotary(s["q"], s["k"], s["inv_freq"], **args)
        return (q, k) + torch.autograd.grad((q, k), (s["q"], s["k"]), (s["dq"], s["dk"]))
    pos = _positions(s["cu"], s["offsets"], s["q"].shape[0])
    cos, sin = _cos_sin(pos, s["inv_freq"], s["mscale"])
    with torch.no_grad():
        out = tuple(_turn(x, cos, sin, c["interleaved"]) for x in (s["q"], s["k"]))
        if c["train"]:
            out += tuple(_turn(x, cos, -sin, c["interleaved"]) for x in (s["dq"], s["dk"]))
    return out


def _positions(cu, offsets, tokens):
    t = torch.arange(tokens, device=cu.device)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    return t - cu[b] + offsets[b]


def _cos_sin(pos, inv_freq, mscale):
    a = pos.double()[:, None] * inv_freq[None, :]
    return (mscale * torch.cos(a)).float()[:, None], (mscale * torch.sin(a)).float()[:, None]


def _turn(x, cos, sin, interleaved):
    """Rotates the pairs of x's first 2 * cos.shape[-1] elements; rounds once."""
    rot = 2 * cos.shape[-1]
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    y = torch.empty_like(x)
    ya, yb = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = ya, yb
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ya, yb
    y[..., rot:] = x[..., rot:]
    return y.to(torch.bfloat16)


def _run_append(s):
    c = s["case"]
    if own:
        import exact_attention_129_b200 as ea
        q = ea.attn_paged_append(
            s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["seqlens"],
            s["max_n"], k_scale=s["k_scale"], v_scale=s["v_scale"],
            q=s["q"] if c["with_q"] else None, inv_freq=s["inv_freq"],
            interleaved=c["interleaved"], mscale=s["mscale"])
    else:
        page = c["page"]
        n = (s["cu"][1:] - s["cu"][:-1]).long()
        start = s["seqlens"].long() - n
        t = torch.arange(s["k"].shape[0], device=s["cu"].device)
        b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
        pos = t - s["cu"][b] + start[b]
        cos, sin = _cos_sin(pos, s["inv_freq"], s["mscale"])
        at, slot = s["table"][b, pos // page].long(), pos % page
        q = _turn(s["q"], cos, sin, c["interleaved"]) if c["with_q"] else None
        _put(_turn(s["k"], cos, sin, c["interleaved"]), s["k_cache"], s["k_scale"], at, slot)
        _put(s["v"], s["v_cache"], s["v_scale"], at, slot)
    out = {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if q is not None:
        out["q"] = q
    if s["k_scale"] is not None:  # an e4m3 value stands for itself times its block's scale
        out["k_scale"], out["v_scale"] = s["k_scale"], s["v_scale"]
    return out


def _put(x, cache, scale, at, slot):
    """Writes the tokens x [T, heads, d] to (page at, slot) of a cache."""
    if scale is None:
        cache[at, slot] = x
        return
    x = x.float()
    pages = cache.shape[0]
    top = torch.zeros_like(scale).index_reduce_(0, at, x.abs().amax(-1), "amax")
    m, e = torch.frexp(top / E4M3_MAX)  # top = m 2^e * 448, 0.5 <= m < 1
    need = _pow2((e - (m == 0.5).int()).clamp(min=MIN_EXP)).float()
    need = torch.where(top > 0, need, torch.full_like(need, 2.0 ** MIN_EXP))
    first = torch.full((pages,), cache.shape[1], device=at.device).index_reduce_(0, at, slot,
                                                                                "amin")
    touched = first < cache.shape[1]
    new = torch.where((first == 0)[:, None], need, torch.maximum(scale, need))
    new = torch.where(touched[:, None], new, scale)
    # earlier tokens of a page whose scale grew
    grown = torch.unique(at)
    old = cache[grown].float() * (scale[grown] / new[grown])[:, None, :, None]
    keep = torch.arange(cache.shape[1], device=at.device)[None, :] < first[grown][:, None]
    cache[grown] = torch.where(keep[:, :, None, None], old, cache[grown].float()).to(cache.dtype)
    cache[at, slot] = (x / new[at][:, :, None]).to(cache.dtype)
    scale.copy_(new)


def _run_attend(s):
    c = s["case"]
    scale = c["d"] ** -0.5
    if own:
        import exact_attention_129_b200 as ea
        return ea.attn_paged_fwd(
            s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["seqlens"], s["max_n"],
            s["max_k"], k_scale=s["k_scale"], v_scale=s["v_scale"], scale=scale, causal=True,
            window=(c["left"], -1), softcap=c["cap"])
    q, cu, lens = s["q"], s["cu"], s["seqlens"].long()
    rows, hq, d = q.shape
    hkv, batch, width = s["k_cache"].shape[2], lens.numel(), s["table"].shape[1]
    keys = width * c["page"]

    def gather(cache, scales):
        x = cache[s["table"].long()].float()  # [batch, width, page, heads, d]
        if scales is not None:
            x *= scales[s["table"].long()][:, :, None, :, None]
        return x.reshape(batch, keys, hkv, d).transpose(1, 2)

    n = (cu[1:] - cu[:-1]).long()
    i = torch.arange(s["max_n"], device=q.device)
    at = (cu[:-1, None] + i[None, :]).clamp(max=rows - 1)  # [batch, max_n]
    x = (q[at].float() * scale).view(batch, s["max_n"], hkv, hq // hkv, d)
    x = x.permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)  # group, then row
    p = x @ gather(s["k_cache"], s["k_scale"]).transpose(2, 3)
    if c["cap"] > 0:
        p = p.div_(c["cap"]).tanh_().mul_(c["cap"])
    j = torch.arange(keys, device=q.device)[None, None, :]
    edge = (i[None, :] + (lens - n)[:, None])[:, :, None]  # last key of each row
    see = (j <= edge) & (j < lens[:, None, None])
    if c["left"] >= 0:
        see = see & (j >= edge - c["left"])
    p = p.view(batch, hkv, hq // hkv, s["max_n"], keys)
    p.masked_fill_(~see[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = p.view(batch, hkv, -1, keys) @ gather(s["v_cache"], s["v_scale"])
    o = o.view(batch, hkv, hq // hkv, s["max_n"], d) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log())[..., 0]
    # back to packed rows
    t = torch.arange(rows, device=q.device)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    r = t - cu[b]
    o = o.permute(0, 3, 1, 2, 4)[b, r].reshape(rows, hq, d)
    lse = lse.permute(0, 3, 1, 2)[b, r].reshape(rows, hq)
    return o.to(torch.bfloat16), lse.t().contiguous()


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"rotary": _exact_rotary, "append": _exact_append, "attend": _exact_attend}[
            case["op"]](s)


def _exact_turn(x, pos, inv_freq, mscale, interleaved, sign=1.0):
    """Pairs as complex numbers, times mscale * e^(i sign pos inv_freq)."""
    x = x.double().clone()
    half = inv_freq.numel()
    z = torch.polar(torch.full((), mscale, dtype=torch.float64, device=x.device),
                    sign * torch.outer(pos.double(), inv_freq))[:, None]
    if interleaved:
        pairs = x[..., :2 * half].unflatten(-1, (half, 2))
    else:
        pairs = x[..., :2 * half].unflatten(-1, (2, half)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    x[..., :2 * half] = (y if interleaved else y.transpose(-1, -2)).flatten(-2)
    return x


def _each(s):
    """(sequence, its slice of the packed rows) for the sequences that have rows."""
    cu = s["cu"].tolist()
    return [(b, slice(cu[b], cu[b + 1])) for b in range(len(cu) - 1) if cu[b + 1] > cu[b]]


def _exact_rotary(s):
    c = s["case"]
    off = s["offsets"].tolist()
    pos = torch.cat([torch.arange(off[b], off[b] + r.stop - r.start, device=s["q"].device)
                     for b, r in _each(s)])
    args = (pos, s["inv_freq"], s["mscale"], c["interleaved"])
    out = (_exact_turn(s["q"], *args), _exact_turn(s["k"], *args))
    if c["train"]:
        out += (_exact_turn(s["dq"], *args, -1.0), _exact_turn(s["dk"], *args, -1.0))
    return out


def _nearest(x, bits, least):
    """x rounded to `bits` significant bits, ties to even, steps no finer than `least`."""
    step = _pow2(torch.frexp(x)[1] - bits).clamp(min=least)
    return torch.round(x / step) * step


def _exact_append(s):
    c, page = s["case"], s["case"]["page"]
    lens, table = s["seqlens"].tolist(), s["table"].tolist()
    out = {"k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    if c["kind"] == "e4m3":
        out["k_scale"], out["v_scale"] = s["k_scale"].double(), s["v_scale"].double()
    q = []
    for b, r in _each(s):
        pos = torch.arange(lens[b] - (r.stop - r.start), lens[b], device=s["cu"].device)
        args = (pos, s["inv_freq"], s["mscale"], c["interleaved"])
        if c["with_q"]:
            q.append(_exact_turn(s["q"][r], *args))
        # what a cache holds is a bf16 value, and in 8 bits that value rounded again
        new = {"k": _nearest(_exact_turn(s["k"][r], *args), 8, 2.0 ** -133),
               "v": s["v"][r].double()}
        lo, hi = int(pos[0]), int(pos[-1]) + 1
        for j in range(lo // page, -(-hi // page)):
            a, z = max(lo, j * page), min(hi, (j + 1) * page)
            at, slots = table[b][j], slice(a - j * page, z - j * page)
            for x in ("k", "v"):
                y, pool = new[x][a - lo:z - lo], out[x + "_cache"]
                if c["kind"] == "bf16":
                    pool[at, slots] = y
                    continue
                scales = out[x + "_scale"]
                top = y.abs().amax((0, 2)).clamp(min=E4M3_MAX * 2.0 ** MIN_EXP)
                m, e = torch.frexp(top)  # 448 = 0.875 * 2^9
                need = _pow2(e - 9 + (m > 0.875).int())
                if a > j * page:
                    old = scales[at].clone()
                    need = torch.maximum(old, need)
                    kept = pool[at, :a - j * page] * (old / need)[:, None]
                    pool[at, :a - j * page] = _nearest(kept, 4, 2.0 ** -9)
                scales[at] = need
                pool[at, slots] = _nearest(y / need[:, None], 4, 2.0 ** -9)
    if q:
        out["q"] = torch.cat(q)
    return out


def _exact_attend(s):
    c = s["case"]
    q, scale, page = s["q"], c["d"] ** -0.5, c["page"]
    group = c["hq"] // c["hkv"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full((c["hq"], q.shape[0]), -math.inf, dtype=torch.float64, device=q.device)
    lens = s["seqlens"].tolist()
    for b, r in _each(s):
        nq, nk = r.stop - r.start, lens[b]
        if nk == 0:
            continue
        pages = s["table"][b, :-(-nk // page)].long()
        i = torch.arange(nq, device=q.device)[:, None] + nk - nq
        j = torch.arange(nk, device=q.device)[None, :]
        hide = (j > i) | ((j < i - c["left"]) if c["left"] >= 0 else (j < 0))
        blind = hide.all(1)
        for h in range(c["hkv"]):
            def rows(x):
                y = s[x + "_cache"][pages, :, h].double()
                if c["kind"] == "e4m3":
                    y = y * s[x + "_scale"][pages, h].double()[:, None, None]
                return y.flatten(0, 1)[:nk]
            heads = slice(h * group, (h + 1) * group)
            a = torch.einsum("ihd,jd->hij", q[r, heads].double(), rows("k")) * scale
            if c["cap"] > 0:
                a = c["cap"] * torch.tanh(a / c["cap"])
            a = a.masked_fill(hide, -math.inf)
            m = torch.logsumexp(a, -1)
            lse[heads, r] = m
            p = torch.exp(a - m[..., None]).masked_fill(blind[:, None], 0.0)
            out[r, heads] = torch.einsum("hij,jd->ihd", p, rows("v"))
    return out, lse
