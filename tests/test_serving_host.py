"""Host side of the rotary and paged-cache entry points, on CPU: refusals of the
C ABI and of the binding, the sizes the binding marshals, the frequency scalings,
and the plain definitions the GPU tests compare with."""
import ctypes
import math
import struct

import pytest
import torch

import exact_attention_129_b200 as ea
from exact_attention_129_b200 import serving
from exact_attention_129_b200 import build as eab
from tests import serving_ref as sr

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    eab.build()
    return ea.library()


# ---------------------------------------------------------------------------
# C ABI refusals: host checks, before any device call
# ---------------------------------------------------------------------------
def _rotary(lib, **kw):
    a = dict(q=16, qst=1024, qsh=128, k=16, kst=256, ksh=128, qo=16, ko=16, f=8, nf=64, m=1.0,
             pos=0, cu=16, off=0, batch=1, total=4, hq=8, hkv=2, d=128)
    a.update(kw)
    vp = ctypes.c_void_p
    return lib.attn_rotary(vp(a["q"]), a["qst"], a["qsh"], vp(a["k"]), a["kst"], a["ksh"],
                           vp(a["qo"]), a["qst"], a["qsh"], vp(a["ko"]), a["kst"], a["ksh"],
                           vp(a["f"]), a["nf"], 0, a["m"], 0, vp(a["pos"]), vp(a["cu"]),
                           vp(a["off"]), a["batch"], 0, a["total"], a["hq"], a["hkv"], a["d"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(q=0), 1), (dict(q=8), 1), (dict(ko=0), 1), (dict(k=0), 1), (dict(qst=1028), 1),
    (dict(ksh=4), 1), (dict(f=0), 1), (dict(f=4), 1), (dict(nf=12), 1), (dict(nf=72), 1),
    (dict(nf=-8), 1), (dict(m=math.inf), 1), (dict(m=math.nan), 1), (dict(cu=0, off=16), 1),
    (dict(pos=16), 1), (dict(cu=18), 1), (dict(batch=0), 1), (dict(total=-1), 1), (dict(hq=0), 1),
    (dict(hkv=0), 1), (dict(d=96), 2), (dict(d=32), 2),
])
def test_rotary_refuses(lib, bad, code):
    assert _rotary(lib, **bad) == code


def _cache(**kw):
    a = dict(k=16, v=16, ks=16, vs=16, table=16, kp=8192, kt=128, kh=8192 * 2, vp=8192, vt=128,
             vh=8192 * 2, ts=4, type=1, pages=8, page=64, per=4, hkv=2, d=128)
    a.update(kw)
    return struct.pack("5P7q6i", *a.values())


BAD_CACHE = [
    (dict(k=0), 1), (dict(v=8), 1), (dict(table=0), 1), (dict(table=2), 1), (dict(ks=0), 1),
    (dict(vs=2), 1), (dict(kt=72), 1), (dict(vh=8), 1), (dict(type=2), 1), (dict(pages=-1), 1),
    (dict(per=-1), 1), (dict(hkv=0), 1), (dict(d=80), 2), (dict(page=8), 2), (dict(page=48), 2),
    (dict(page=256), 2),
]


def _append(lib, cache=None, **kw):
    a = dict(k=16, st=256, sh=128, v=16, q=16, qst=1024, qo=16, cu=16, lens=16, batch=2, total=6,
             max=3, hq=8, f=8, nf=64, m=1.0)
    a.update(kw)
    vp = ctypes.c_void_p
    return lib.attn_paged_append(cache or _cache(), vp(a["k"]), a["st"], a["sh"], vp(a["v"]),
                                 a["st"], a["sh"], vp(a["q"]), a["qst"], 128, vp(a["qo"]), a["qst"],
                                 128, vp(a["cu"]), vp(a["lens"]), a["batch"], a["total"], a["max"],
                                 a["hq"], vp(a["f"]), a["nf"], 0, a["m"], None)


@pytest.mark.parametrize("bad,code", [
    (dict(k=0), 1), (dict(v=8), 1), (dict(qo=0), 1), (dict(st=4), 1), (dict(qst=12), 1),
    (dict(cu=0), 1), (dict(lens=0), 1), (dict(lens=6), 1), (dict(batch=0), 1), (dict(total=-2), 1),
    (dict(max=-1), 1), (dict(hq=0), 1), (dict(f=0), 1), (dict(nf=4), 1), (dict(m=math.nan), 1),
])
def test_append_refuses(lib, bad, code):
    assert _append(lib, **bad) == code


@pytest.mark.parametrize("bad,code", BAD_CACHE)
def test_cache_refusals(lib, bad, code):
    assert _append(lib, _cache(**bad)) == code
    assert _paged(lib, _cache(**bad)) == code
    assert lib.attn_paged_workspace_size(_cache(**bad), 2, 6, 3, 100, 8, 1, -1, -1, 4) == 0


def _paged(lib, cache=None, **kw):
    a = dict(q=16, cu=16, lens=16, batch=2, total=6, mq=3, mk=100, hq=8, scale=0.1, wl=-1, cap=0.0,
             splits=0, rl=1, out=16, lse=16, ws=256, bytes=1 << 30)
    a.update(kw)
    vp = ctypes.c_void_p
    return lib.attn_paged_fwd(cache or _cache(), vp(a["q"]), vp(a["cu"]), vp(a["lens"]), a["batch"],
                              a["total"], a["mq"], a["mk"], a["hq"], a["scale"], 1, a["wl"], -1,
                              a["cap"], a["splits"], a["rl"], vp(a["out"]), vp(a["lse"]),
                              vp(a["ws"]), a["bytes"], None)


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(q=8), dict(cu=0), dict(lens=2), dict(batch=0), dict(total=-1), dict(mq=-1),
    dict(mk=-1), dict(mk=1 << 30), dict(hq=7), dict(hq=0), dict(scale=0.0),
    dict(scale=math.nan), dict(cap=-1.0), dict(cap=math.inf), dict(splits=-1), dict(splits=129),
    dict(out=0), dict(out=8), dict(lse=0), dict(lse=2),
])
def test_paged_fwd_refuses(lib, bad):
    assert _paged(lib, **bad) == 1


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
class CacheStruct(ctypes.Structure):  # attn_paged_cache_t
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "block_table")] +
                [(n, ctypes.c_int64) for n in ("k_s_page", "k_s_token", "k_s_head", "v_s_page",
                                               "v_s_token", "v_s_head", "table_stride")] +
                [(n, ctypes.c_int32) for n in ("type", "num_pages", "page_size", "pages_per_seq",
                                               "nheads_kv", "head_dim")])


class Recorder:
    """Functions of the C ABI's types that write their arguments down, as callbacks."""

    def __init__(self, lib):
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        cache, rows, size = ctypes.POINTER(CacheStruct), [vp, i64, i64], ctypes.c_size_t
        types = {
            "attn_rotary": [i32] + rows * 4 + [vp, i32, i32, f32, i32, vp, vp, vp] + [i32] * 6 + [vp],
            "attn_paged_append": [i32, cache] + rows * 4 + [vp, vp, i32, i32, i32, i32, vp, i32, i32,
                                                            f32, vp],
            "attn_paged_fwd": [i32, cache, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, i32, i32,
                               f32, i32, i32, vp, vp, vp, size, vp],
            "attn_paged_workspace_size": [size, cache] + [i32] * 9,
        }
        self.calls, self.code = [], 0
        self.functions = [ctypes.CFUNCTYPE(*types[n])(self._recorder(n)) for n in serving.ABI]
        self.addresses = [ctypes.cast(f, ctypes.c_void_p).value for f in self.functions]

    def _recorder(self, name):
        def f(*args):
            args = tuple([getattr(a.contents, n) for n, _ in CacheStruct._fields_]
                         if isinstance(a, ctypes.POINTER(CacheStruct)) else a for a in args)
            self.calls.append((name, args))
            return 4096 if name.endswith("workspace_size") else self.code
        return f


@pytest.fixture
def rec(lib):
    r = Recorder(lib)
    binding = serving._binding or serving._load()
    binding.init(ea.AttnError, *r.addresses, False)
    yield r
    serving._load()


def _problem(t=5, hq=4, hkv=2, d=64, page=16, e4m3=True, lens=(9, 20)):
    c = sr.Cache(lens, lens, hkv, d, page, e4m3)
    cu = torch.tensor([0, 2, t], dtype=torch.int32)
    return dict(q=torch.zeros(t, hq, d, dtype=BF), k=torch.zeros(t, hkv, d, dtype=BF),
                v=torch.zeros(t, hkv, d, dtype=BF), kc=c.k, vc=c.v, table=c.table, cu=cu,
                lens=torch.tensor(lens, dtype=torch.int32),
                f=ea.rope_frequencies(d)[0], kw={"k_scale": c.k_scale, "v_scale": c.v_scale}
                if e4m3 else {})


def test_binding_marshals_append_and_attention(rec):
    p = _problem()
    q = ea.attn_paged_append(p["k"], p["v"], p["kc"], p["vc"], p["table"], p["cu"], p["lens"], 3,
                             q=p["q"], inv_freq=p["f"], mscale=1.5, interleaved=True, **p["kw"])
    name, a = rec.calls[-1]
    assert name == "attn_paged_append" and q.shape == p["q"].shape and q is not p["q"]
    cache = tuple(a[0])
    assert cache[0] == p["kc"].data_ptr() and cache[2] == p["kw"]["k_scale"].data_ptr()
    assert cache[5:8] == (16 * 2 * 64, 64, 16 * 64)  # a head-major pool: page, token, head
    assert cache[11] == p["table"].shape[1]
    assert cache[12:] == (1, p["kc"].shape[0], 16, p["table"].shape[1], 2, 64)
    assert a[2:4] == (128, 64) and a[8:10] == (256, 64)
    assert a[15:19] == (2, 5, 3, 4) and a[20:23] == (32, True, 1.5)
    out, lse = ea.attn_paged_fwd(p["q"], p["kc"], p["vc"], p["table"], p["cu"], p["lens"], 3, 20,
                                 causal=True, window=(7, None), softcap=3.0, **p["kw"])
    names = [c[0] for c in rec.calls]
    assert names[-2:] == ["attn_paged_workspace_size", "attn_paged_fwd"]
    a = rec.calls[-1][1]
    assert a[4:9] == (2, 5, 3, 20, 4) and math.isclose(a[9], 64 ** -0.5)
    assert a[10:16] == (True, 7, -1, 3.0, 0, True) and a[19] == 4096
    assert out.shape == p["q"].shape and lse.shape == (4, 5)
    assert ea.attn_paged_fwd(p["q"], p["kc"], p["vc"], p["table"], p["cu"], p["lens"], 3, 20,
                             return_lse=False, **p["kw"])[1] is None


def test_binding_marshals_rotary(rec):
    p = _problem(d=128)
    qkv = torch.zeros(5, 8, 128, dtype=BF)
    q, k = ea.attn_rotary(qkv[:, :4], qkv[:, 4:6], p["f"], cu_seqlens=p["cu"])
    a = rec.calls[-1][1]
    assert a[1:3] == (1024, 128) and a[4:6] == (1024, 128) and a[7:9] == (512, 128)
    assert a[13] == 64 and a[19] is None and a[20:26] == (2, True, 5, 4, 2, 128)
    assert q.is_contiguous() and k.shape == (5, 2, 128)
    # in place, through the views
    ea.attn_rotary(qkv[:, :4], None, p["f"], q_out=qkv[:, :4])
    a = rec.calls[-1][1]
    assert a[6] == a[0] and a[7:9] == (1024, 128) and a[3] is None and a[24] == 0
    # autograd: one call forward, one backward with inverse set
    x = torch.randn(5, 4, 128).to(BF).requires_grad_(True)
    y = torch.randn(5, 2, 128).to(BF).requires_grad_(True)
    n = len(rec.calls)
    a, b = ea.rotary(x, y, p["f"])
    torch.autograd.grad((a, b), (x, y), (torch.zeros_like(a), torch.zeros_like(b)))
    assert [c[1][16] for c in rec.calls[n:]] == [False, True]


@pytest.mark.parametrize("case", [
    "q_dtype", "q_rank", "q_stride", "q_start", "k_rows", "freq_dtype", "freq_len", "freq_odd",
    "pos_dtype", "pos_len", "both", "offsets", "cu_len", "out_shape", "out_overlap", "k_out"])
def test_rotary_binding_refuses(case):
    q, k = torch.zeros(6, 4, 64, dtype=BF), torch.zeros(6, 2, 64, dtype=BF)
    f, kw = ea.rope_frequencies(64)[0], {}
    cu = torch.tensor([0, 6], dtype=torch.int32)
    if case == "q_dtype":
        q = q.float()
    elif case == "q_rank":
        q = q.reshape(6, 256)
    elif case == "q_stride":
        q = torch.zeros(6, 4, 68, dtype=BF)[..., :64]
    elif case == "q_start":
        q = torch.zeros(6 * 256 + 8, dtype=BF)[1:1537].view(6, 4, 64)
    elif case == "k_rows":
        k = k[:5]
    elif case == "freq_dtype":
        f = f.float()
    elif case == "freq_len":
        f = ea.rope_frequencies(128)[0]
    elif case == "freq_odd":
        f = f[:4].contiguous()
    elif case == "pos_dtype":
        kw["positions"] = torch.zeros(6, dtype=torch.int64)
    elif case == "pos_len":
        kw["positions"] = torch.zeros(5, dtype=torch.int32)
    elif case == "both":
        kw.update(positions=torch.zeros(6, dtype=torch.int32), cu_seqlens=cu)
    elif case == "offsets":
        kw["offsets"] = torch.zeros(1, dtype=torch.int32)
    elif case == "cu_len":
        kw["cu_seqlens"] = cu[:1]
    elif case == "out_shape":
        kw["q_out"] = torch.zeros(6, 4, 128, dtype=BF)
    elif case == "out_overlap":
        kw["q_out"] = torch.zeros(6, 1, 64, dtype=BF).expand(6, 4, 64)
    elif case == "k_out":
        kw["k_out"], k = torch.zeros_like(k), None
    with pytest.raises(ValueError) as e:
        ea.attn_rotary(q, k, f, **kw)
    assert "CUDA tensors only" not in str(e.value)


@pytest.mark.parametrize("case", [
    "cache_type", "cache_shapes", "page", "cache_stride", "no_scale", "scale_shape", "scale_bf16",
    "table_dtype", "table_rows", "heads", "head_dim", "lens_len", "lens_dtype", "cu", "v_shape"])
def test_paged_binding_refuses(case):
    p = _problem()
    if case == "cache_type":
        p["kc"] = p["kc"].float()
    elif case == "cache_shapes":
        p["vc"] = p["vc"][:-1]
    elif case == "page":
        p["kc"], p["vc"] = p["kc"][:, :8], p["vc"][:, :8]
    elif case == "cache_stride":
        s = p["kc"].shape
        p["kc"] = torch.zeros(s[0], s[1], s[2], s[3] + 8).to(sr.E4M3)[..., :s[3]]
    elif case == "no_scale":
        p["kw"].pop("v_scale")
    elif case == "scale_shape":
        p["kw"]["k_scale"] = p["kw"]["k_scale"][:-1]
    elif case == "scale_bf16":
        p["kc"], p["vc"] = p["kc"].to(BF), p["vc"].to(BF)
    elif case == "table_dtype":
        p["table"] = p["table"].long()
    elif case == "table_rows":
        p["table"] = p["table"][:1]
    elif case == "heads":
        p["q"] = torch.zeros(5, 3, 64, dtype=BF)
        p["k"] = torch.zeros(5, 1, 64, dtype=BF)
        p["v"] = p["k"]
    elif case == "head_dim":
        p["q"], p["k"] = torch.zeros(5, 4, 128, dtype=BF), torch.zeros(5, 2, 128, dtype=BF)
        p["v"] = p["k"]
    elif case == "lens_len":
        p["lens"] = p["lens"][:1]
    elif case == "lens_dtype":
        p["lens"] = p["lens"].long()
    elif case == "cu":
        p["cu"] = p["cu"][:1]
    elif case == "v_shape":
        p["v"] = p["v"][:4]
    with pytest.raises(ValueError) as e:
        ea.attn_paged_append(p["k"], p["v"], p["kc"], p["vc"], p["table"], p["cu"], p["lens"], 3,
                             **p["kw"])
    assert "CUDA tensors only" not in str(e.value)
    if case != "v_shape":
        with pytest.raises(ValueError) as e:
            ea.attn_paged_fwd(p["q"], p["kc"], p["vc"], p["table"], p["cu"], p["lens"], 3, 20,
                              **p["kw"])
        assert "CUDA tensors only" not in str(e.value)


def test_an_empty_pool_is_refused(lib):
    assert _append(lib, _cache(pages=0)) == 1
    assert _paged(lib, _cache(pages=0)) == 1


def test_errors_of_a_backward_reach_the_caller(rec):
    x = torch.zeros(5, 4, 128, dtype=BF).requires_grad_(True)
    y, _ = ea.rotary(x, None, ea.rope_frequencies(128)[0])
    rec.code = 3
    with pytest.raises(RuntimeError, match="attn_rotary"):
        y.backward(torch.zeros_like(y))
    rec.code = 0
    y, _ = ea.rotary(x, None, ea.rope_frequencies(128)[0])
    y.backward(torch.zeros_like(y))
    rec.code = 3
    with pytest.raises(ea.AttnError):
        ea.rotary(x, None, ea.rope_frequencies(128)[0])


def test_a_frequency_that_wants_a_gradient_is_refused(rec):
    f = ea.rope_frequencies(128)[0].requires_grad_(True)
    with pytest.raises(ValueError, match="inv_freq"):
        ea.rotary(torch.zeros(5, 4, 128, dtype=BF), None, f)


@pytest.mark.parametrize("case", ["heads", "tokens", "pages"])
def test_append_refuses_a_pool_that_overlaps_itself(rec, case):
    p = _problem()
    n, page, h, d = p["kc"].shape
    dims = {"heads": (n, page, 1, d), "tokens": (n, 1, h, d), "pages": (1, page, h, d)}[case]
    one = torch.zeros(dims).to(sr.E4M3).expand(n, page, h, d)
    for kc, vc in ((one, p["vc"]), (p["kc"], one)):
        with pytest.raises(ValueError, match="overlap"):
            ea.attn_paged_append(p["k"], p["v"], kc, vc, p["table"], p["cu"], p["lens"], 3,
                                 **p["kw"])
    ea.attn_paged_fwd(p["q"], one, one, p["table"], p["cu"], p["lens"], 3, 20, **p["kw"])


def test_cpu_tensors_are_refused():
    p = _problem()
    with pytest.raises(ValueError, match="CUDA tensors only"):
        ea.attn_rotary(p["q"], p["k"], p["f"])
    with pytest.raises(ValueError, match="CUDA tensors only"):
        ea.attn_paged_append(p["k"], p["v"], p["kc"], p["vc"], p["table"], p["cu"], p["lens"], 3,
                             **p["kw"])
    with pytest.raises(ValueError, match="CUDA tensors only"):
        ea.attn_paged_fwd(p["q"], p["kc"], p["vc"], p["table"], p["cu"], p["lens"], 3, 20,
                          **p["kw"])


# ---------------------------------------------------------------------------
# frequencies
# ---------------------------------------------------------------------------
def test_rope_frequencies():
    f, m = ea.rope_frequencies(64, 500.0)
    assert m == 1.0 and f.dtype == torch.float64 and f.shape == (32,)
    for i in (0, 1, 31):
        assert math.isclose(f[i], 500.0 ** (-2 * i / 64), rel_tol=1e-14)
    lin, _ = ea.rope_frequencies(64, 500.0, scaling="linear", factor=4)
    assert torch.allclose(lin * 4, f, rtol=1e-14, atol=0)
    ntk, _ = ea.rope_frequencies(64, 500.0, scaling="ntk", factor=4)
    assert ntk[0] == 1.0 and math.isclose(ntk[31] * 4, f[31], rel_tol=1e-12)
    y, m = ea.rope_frequencies(64, 500.0, scaling="yarn", factor=4, original_max=2048)
    turns = 2048 * f / (2 * math.pi)
    assert math.isclose(m, 0.1 * math.log(4) + 1)
    assert torch.equal(y[turns >= 32], f[turns >= 32]) and (turns >= 32).any()
    slow = turns <= 1
    assert slow.any() and torch.allclose(y[slow] * 4, f[slow], rtol=1e-14, atol=0)
    mid = ~slow & (turns < 32)
    assert mid.any() and bool(((y[mid] < f[mid]) & (y[mid] > f[mid] / 4)).all())


@pytest.mark.parametrize("kw", [dict(rot_dim=24), dict(rot_dim=0), dict(base=1.0),
                                dict(factor=0.5), dict(scaling="other"),
                                dict(scaling="yarn", factor=2)])
def test_rope_frequencies_refuses(kw):
    kw = {"rot_dim": 64, **kw}
    with pytest.raises(ValueError):
        ea.rope_frequencies(kw.pop("rot_dim"), **kw)


# ---------------------------------------------------------------------------
# the plain definitions themselves
# ---------------------------------------------------------------------------
def test_reference_rotation_is_orthogonal_and_its_inverse_the_gradient():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(3, 2, 64, generator=g, dtype=torch.float64)
    f = ea.rope_frequencies(48)[0]
    pos = torch.tensor([0, 5, 100000])
    for inter in (False, True):
        y = sr.rotate(x, pos, f, 1.3, inter)
        assert torch.equal(y[..., 48:], x[..., 48:])
        assert torch.allclose(y[..., :48].norm(dim=-1), 1.3 * x[..., :48].norm(dim=-1))
        w = torch.randn(x.shape, generator=g, dtype=torch.float64)
        z = x.clone().requires_grad_(True)
        grad = torch.autograd.grad((sr.rotate(z, pos, f, 1.3, inter) * w).sum(), z)[0]
        assert torch.allclose(grad, sr.rotate(w, pos, f, 1.3, inter, inverse=True))
        eps = 1e-6  # and by differences
        for at in ((0, 1, 3), (2, 0, 40), (1, 1, 60)):
            d = torch.zeros_like(x)
            d[at] = eps
            num = ((sr.rotate(x + d, pos, f, 1.3, inter) - sr.rotate(x - d, pos, f, 1.3, inter))
                   * w).sum() / (2 * eps)
            assert abs(float(num - grad[at])) < 1e-8


def test_reference_scale_is_the_least_power_of_two():
    for top in (448.0, 449.0, 1.0, 1.75, 1.7578125, 2.0 ** -80, 3e38, 0.0):
        e = sr.need_exponent(torch.tensor([top, -top / 2, math.inf, math.nan]))
        assert top <= 448 * 2.0 ** e and (e == -64 or top > 448 * 2.0 ** (e - 1))
