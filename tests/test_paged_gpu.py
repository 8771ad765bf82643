"""Appending to a paged cache and attention over it, on the GPU, against the
64-bit definitions."""
import math

import pytest
import torch

import exact_attention_129_b200 as ea
from tests import serving_ref as sr
from tests.gpu_helpers import LSE_TOL, guarded_empty, guards_intact
from tests.serving_ref import Cache

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rows(t, h, d, seed, spread=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, h, d, generator=g) * torch.exp(spread * torch.randn(t, h, 1, generator=g))
    return x.to(BF)


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def cu_of(n):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return cu


def bits(x):
    return x.view(torch.uint8 if x.dtype == sr.E4M3 else torch.int16)


def same_codes(a, b):
    """Equal bit for bit, any NaN alike."""
    x, y = bits(a.contiguous()), bits(b.contiguous())
    nan = a.float().isnan().reshape(x.shape) & b.float().isnan().reshape(y.shape)
    return bool(((x == y) | nan).all())


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
APPENDS = [  # new tokens, tokens before them
    ([1], [0]), ([1, 1, 1], [0, 15, 16]), ([3, 0, 8, 1], [14, 5, 120, 0]),
    ([9, 40], [0, 7]), ([200, 1, 0, 129], [30, 300, 2, 127]),
]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
def test_append(d, page, e4m3):
    hkv = 3
    for n, before in APPENDS:
        for head_major in (True, False):
            lens, cu = [a + b for a, b in zip(n, before)], cu_of(n)
            c = Cache(before, lens, hkv, d, page, e4m3, head_major, seed=len(n), spread=1.5)
            k, v = rows(cu[-1], hkv, d, 1), rows(cu[-1], hkv, d, 2)
            kc, vc, table, kw = c.to("cuda")
            ea.attn_paged_append(k.cuda(), v.cuda(), kc, vc, table, i32(cu), i32(lens), max(n),
                                 **kw)
            for x, pool, got, name in ((k, c.k, kc, "k"), (v, c.v, vc, "v")):
                scale = getattr(c, name + "_scale")
                sr.append(x, pool, scale, c.table, cu, lens)
                assert same_codes(got.cpu(), pool), (n, before, head_major, name)
                if e4m3:
                    assert torch.equal(kw[name + "_scale"].cpu(), scale)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,rot,inter", [(64, 32, False), (128, 128, False), (128, 80, True),
                                         (256, 256, True), (256, 64, False)])
def test_append_rotates_as_rotary_does(e4m3, d, rot, inter):
    hq, hkv, page = 6, 2, 32
    f, m = ea.rope_frequencies(rot, scaling="yarn", factor=8, original_max=4096)
    for n, before in (([3, 1, 0, 8], [40, 0, 9, 100000]), ([90, 5, 33], [0, 61, 100])):
        lens, cu = [a + b for a, b in zip(n, before)], cu_of(n)
        q, k, v = (rows(cu[-1], h, d, s).cuda() for s, h in enumerate((hq, hkv, hkv)))
        c = Cache([0] * len(n), [min(x, 200) for x in lens], hkv, d, page, e4m3, seed=7)
        # far positions share few pages: the table names them at the end of its row
        width = -(-max(lens) // page)
        table = torch.full((len(n), width), -1, dtype=torch.int32)
        for b, (x, y) in enumerate(zip(before, lens)):
            for j in range(x // page, -(-y // page)):
                table[b, j] = c.table[b, j - x // page]
        kc, vc, _, kw = c.to("cuda")
        kc2, vc2, _, kw2 = c.to("cuda")
        args = (table.cuda(), i32(cu), i32(lens), max(n))
        qo = ea.attn_paged_append(k, v, kc, vc, *args, q=q, inv_freq=f.cuda(), interleaved=inter,
                                  mscale=m, **kw)
        qr, kr = ea.attn_rotary(q, k, f.cuda(), cu_seqlens=i32(cu), offsets=i32(before),
                                interleaved=inter, mscale=m)
        assert torch.equal(qo, qr)
        ea.attn_paged_append(kr, v, kc2, vc2, *args, **kw2)
        assert same_codes(kc, kc2) and same_codes(vc, vc2)
        for name in kw:
            assert torch.equal(kw[name], kw2[name])


def test_append_holds_what_is_not_finite_as_nan():
    d, page = 64, 16
    k = rows(4, 2, d, 3)
    k[0, 0, 5], k[1, 1, 7], k[2, 0, 9], k[3, 1] = math.inf, math.nan, -math.inf, 0.0
    for n in ([4], [2, 2]):  # both kernels: 4 tokens of one page, then padded to many
        cu, before = cu_of(n), [6] * len(n)
        lens = [a + b for a, b in zip(n, before)]
        c = Cache(before, lens, 2, d, page, True, seed=3, spread=3.0)
        for max_n in (max(n), 40):
            kc, vc, table, kw = c.to("cuda")
            ea.attn_paged_append(k.cuda(), k.cuda(), kc, vc, table, i32(cu), i32(lens), max_n, **kw)
            ref, scale = c.k.clone(), c.k_scale.clone()
            sr.append(k, ref, scale, c.table, cu, lens)
            assert same_codes(kc.cpu(), ref) and torch.equal(kw["k_scale"].cpu(), scale)
            assert bool(torch.isfinite(kw["k_scale"]).all())


@pytest.mark.parametrize("max_n", [8, 64])
def test_append_leaves_the_rest_alone(max_n):
    # pages of nobody, slots behind the tokens, rows behind the last sequence, table
    # entries outside the pool and positions outside the table
    d, page, hkv = 64, 16, 2
    c = Cache([20, 3], [40, 16], hkv, d, page, True, seed=5)
    c.table[0, 1] = 10 ** 6     # tokens 16 .. 31 of sequence 0 go nowhere
    n, lens = [7, 5], [27, 20]  # sequence 1: tokens 15 .. 19, its row has 1 usable page + -7s
    cu = [0, 7, 12]
    k, q = rows(15, hkv, d, 6).cuda(), rows(15, 4, d, 7).cuda()
    kc, vc, table, kw = c.to("cuda")
    out = torch.full_like(q, 3.0)
    f = ea.rope_frequencies(d)[0].cuda()
    ea.attn_paged_append(k, k, kc, vc, table, i32(cu), i32(lens), max_n, q=q, q_out=out, inv_freq=f,
                         **kw)
    kr = ea.attn_rotary(k[:12], None, f, cu_seqlens=i32(cu), offsets=i32([20, 15]))[0]
    for x, pool, got, name in ((kr.cpu(), c.k, kc, "k"), (k.cpu(), c.v, vc, "v")):
        scale = getattr(c, name + "_scale")
        sr.append(x, pool, scale, c.table, cu, lens)
        assert same_codes(got.cpu(), pool) and torch.equal(kw[name + "_scale"].cpu(), scale)
    assert bool((out[12:] == 3).all())
    assert torch.equal(out[:12], ea.attn_rotary(q[:12], None, f, cu_seqlens=i32(cu),
                                                offsets=i32([20, 15]))[0])


def test_append_views_and_queries_in_place():
    d, page = 128, 64
    n, before = [5, 1], [61, 0]
    cu, lens = cu_of(n), [66, 1]
    qkv = rows(6, 8, d, 8)
    f = ea.rope_frequencies(d)[0].cuda()
    c = Cache(before, lens, 2, d, page, True)
    for max_n in (5, 100):
        a, b = c.to("cuda"), c.to("cuda")
        dev = qkv.cuda()
        q, k, v = dev[:, :4], dev[:, 4:6], dev[:, 6:]
        want = ea.attn_paged_append(k.contiguous(), v.contiguous(), a[0], a[1], a[2], i32(cu),
                                    i32(lens), max_n, q=q.contiguous(), inv_freq=f, **a[3])
        got = ea.attn_paged_append(k, v, b[0], b[1], b[2], i32(cu), i32(lens), max_n, q=q, q_out=q,
                                   inv_freq=f, **b[3])
        assert torch.equal(got, want) and got.data_ptr() == dev.data_ptr()
        assert torch.equal(dev[:, 4:].cpu(), qkv[:, 4:])
        assert same_codes(a[0], b[0]) and same_codes(a[1], b[1])


@pytest.mark.parametrize("e4m3", [False, True])
def test_append_with_more_new_tokens_than_the_length(e4m3):
    # positions -7 .. 12 and -3 .. 0: the tokens before position 0 go nowhere, the
    # queries are rotated by their positions in both kernels
    d, page, hkv, n, lens = 64, 16, 2, [20, 4], [13, 1]
    cu = cu_of(n)
    f = ea.rope_frequencies(d)[0].cuda()
    k, q = rows(24, hkv, d, 71).cuda(), rows(24, 4, d, 72).cuda()
    off = i32([x - y for x, y in zip(lens, n)])
    want = ea.attn_rotary(q, None, f, cu_seqlens=i32(cu), offsets=off)[0]
    kr = ea.attn_rotary(k, None, f, cu_seqlens=i32(cu), offsets=off)[0].cpu()
    c = Cache([0, 0], lens, hkv, d, page, e4m3, seed=7)
    sr.append(kr, c.k, c.k_scale, c.table, cu, lens)
    for j in (0, 1):  # the sequences together (20 new tokens), and the second alone (4)
        c2 = Cache([0, 0], lens, hkv, d, page, e4m3, seed=7)
        kc, vc, table, kw = c2.to("cuda")
        a = cu[j]
        got = ea.attn_paged_append(k[a:], k[a:], kc, vc, table[j:], i32([x - a for x in cu[j:]]),
                                   i32(lens[j:]), max(n[j:]), q=q[a:], inv_freq=f, **kw)
        assert torch.equal(got, want[a:])
        for b in range(j, 2):
            at = int(c.table[b, 0])
            assert same_codes(kc[at].cpu(), c.k[at])


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attend(c, q, n, *, hq, splits=0, max_k=None, **mask):
    """Runs the kernel between guard bands and compares with the definition."""
    cu = cu_of(n)
    kc, vc, table, kw = c.to("cuda")
    obuf, out, og = guarded_empty(q.shape, BF, kc.device)
    lbuf, lse, lg = guarded_empty((hq, q.shape[0]), torch.float32, kc.device)
    scale = q.shape[2] ** -0.5
    ea.attn_paged_fwd(q.cuda(), kc, vc, table, i32(cu), i32(c.lens), max(n),
                      max(c.lens) if max_k is None else max_k, num_splits=splits, out=out, lse=lse,
                      scale=scale, **mask, **kw)
    rc, msg = ea.last_device_error()
    assert rc == 0, msg
    assert guards_intact(obuf, og) and guards_intact(lbuf, lg)
    ref, ref_lse, pabs = sr.attend(q, c.k, c.v, c.k_scale, c.v_scale, c.table, cu, c.lens, scale,
                                   **mask)
    # from 128 rows of a group on, an unsplit call runs attn_fwd on packed bf16 copies: the codes
    # times their power-of-two scales are exact in bf16, and P is rounded to bf16 (half a step,
    # 2^-8 of each weight) where the paged kernel rounds it to f16
    f16 = c.e4m3 and (splits != 0 or max(n) * (hq // c.k.shape[2]) < 128)
    compare(out[:cu[-1]], lse[:, :cu[-1]], ref[:cu[-1]], ref_lse[:, :cu[-1]], pabs[:cu[-1]], f16)
    return out, lse


def compare(out, lse, ref, ref_lse, pabs, e4m3):
    out, lse = out.cpu().double(), lse.cpu().double()
    assert torch.equal(out.isnan(), ref.isnan())
    err = (out - ref).abs().nan_to_num(0.0)
    bound = sr.o_bound(ref, pabs, e4m3).nan_to_num(1.0)
    assert bool((err <= bound).all()), float((err / bound).max())
    none = ref_lse == -math.inf
    assert torch.equal(lse == -math.inf, none)
    fine = torch.isfinite(ref_lse)
    assert float((lse - ref_lse)[fine].abs().max() if fine.any() else 0.0) <= LSE_TOL


GROUPS = [(4, 4), (8, 2), (8, 1), (5, 1), (6, 2)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [16, 128])
def test_single_tokens(d, e4m3, page):
    lens = [1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 128, 200, 600]
    for i, (hq, hkv) in enumerate(GROUPS):
        # NaN where no token is: it must not reach the result
        c = Cache(lens, lens, hkv, d, page, e4m3, head_major=i % 2 == 0, seed=i, junk=math.nan)
        q = rows(len(lens), hq, d, 10 + i, 0.2)
        attend(c, q, [1] * len(lens), hq=hq, causal=i % 2 == 1)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("splits", [1, 2, 7, 128])
def test_splits_give_the_same(d, e4m3, splits):
    lens = [900, 3, 0, 257]
    c = Cache(lens, lens, 2, d, 32, e4m3, seed=1, junk=math.nan)
    q = rows(4, 8, d, 20, 0.2)
    attend(c, q, [1] * 4, hq=8, splits=splits)
    # a bound far above the lengths cuts them into empty parts
    attend(c, q, [1] * 4, hq=8, splits=splits, max_k=50000)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("most", [2, 5, 13, 30])
def test_several_rows(d, e4m3, most):
    # rows of a group fill 8, 16, 32 and 64 columns, and more than one tile
    n = [most, 0, 1, max(1, most - 1), 2]
    lens = [300, 70, 0, most, 129]
    for hq, hkv in ((4, 4), (8, 2), (5, 1)):
        c = Cache(lens, lens, hkv, d, 64, e4m3, seed=most, junk=math.nan)
        q = rows(sum(n) + 3, hq, d, 30 + most, 0.2)
        attend(c, q, n, hq=hq, causal=True)
        attend(c, q, n, hq=hq, causal=False, splits=3)


@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_that_see_no_key(e4m3):
    # more rows than keys: the first ones see none under a causal mask
    n, lens = [6, 3, 1], [2, 0, 0]
    c = Cache(lens, [16] * 3, 2, 64, 16, e4m3, seed=2, junk=math.nan)
    q = rows(10, 4, 64, 40)
    for splits in (0, 2):
        out, lse = attend(c, q, n, hq=4, causal=True, splits=splits)
        assert not out[:4].any() and bool((lse[:, :4] == -math.inf).all())
        assert not out[6:].any() and bool((lse[:, 6:] == -math.inf).all())


@pytest.mark.parametrize("d,e4m3", [(64, True), (128, False), (128, True), (256, True)])
@pytest.mark.parametrize("window", [(0, 0), (1, -1), (15, 0), (64, 3), (100, -1), (-1, 2),
                                    (500, 500)])
def test_windows(d, e4m3, window):
    n, lens = [1, 4, 12, 1], [333, 260, 12, 90]
    c = Cache(lens, lens, 2, d, 32, e4m3, seed=4, junk=math.nan)
    q = rows(sum(n), 6, d, 50, 0.2)
    for causal in (False, True):
        for splits in (0, 3):
            attend(c, q, n, hq=6, causal=causal, window=window, splits=splits)


@pytest.mark.parametrize("d,e4m3", [(64, False), (128, True), (256, True)])
@pytest.mark.parametrize("cap", [1.5, 30.0])
def test_softcap(d, e4m3, cap):
    n, lens = [1, 5, 2], [200, 90, 2]
    c = Cache(lens, lens, 1, d, 64, e4m3, seed=5)
    q = rows(sum(n), 8, d, 60, 0.2)
    attend(c, q, n, hq=8, causal=True, softcap=cap)
    attend(c, q, n, hq=8, causal=True, softcap=cap, window=(50, -1), splits=2)


def test_scales_far_apart():
    # value scales 2^-40 .. 2^40 over the pages, and keys that favour any of them
    d, page = 128, 16
    lens = [400, 130]
    c = Cache(lens, lens, 2, d, page, True, seed=6)
    g = torch.Generator().manual_seed(6)
    c.v_scale = 2.0 ** torch.randint(-40, 41, c.v_scale.shape, generator=g).float()
    q = rows(2, 8, d, 70, 0.2)
    attend(c, q, [1, 1], hq=8)
    # queries of any size: the row is brought into f16's range by its own largest element
    for f in (2.0 ** -60, 2.0 ** 12):
        small = (rows(2, 8, d, 71, 0.2).double() * f).to(BF)
        c2 = Cache(lens, lens, 2, d, page, True, seed=7)
        c2.k_scale = c2.k_scale / f
        attend(c2, small, [1, 1], hq=8)


def test_one_heavy_key_among_many_light_ones():
    # the light keys' weights are near 2^-20 of the heavy one's: together they count
    d, n = 64, 20000
    c = Cache([n], [n], 1, d, 128, True, seed=8, spread=0.0)
    c.k[:] = 0.0
    c.k[int(c.table[0, 5]), 17, 0] = torch.full((d,), 8.0).to(sr.E4M3)
    c.k_scale[:] = 1.0
    q = torch.full((1, 1, d), 13.9 / 64.0).to(BF)
    attend(c, q, [1], hq=1)


@pytest.mark.parametrize("e4m3", [False, True])
def test_not_finite_keys_and_values(e4m3):
    # NaN in a visible key or value reaches exactly the rows that see it
    d, page = 64, 16
    lens, n = [100, 50], [1, 1]
    for where in ("k", "v"):
        c = Cache(lens, lens, 2, d, page, e4m3, seed=9)
        getattr(c, where)[int(c.table[1, 2]), 3, 1, 5] = math.nan
        q = rows(2, 4, d, 80, 0.2)
        kc, vc, table, kw = c.to("cuda")
        out, lse = ea.attn_paged_fwd(q.cuda(), kc, vc, table, i32([0, 1, 2]), i32(lens), 1, 100,
                                     **kw)
        bad = out.isnan().cpu()
        want = torch.zeros_like(bad)
        if where == "k":
            want[1, 2:] = True
        else:
            want[1, 2:, 5] = True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (12, 2), (20, 2)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_not_finite_values_behind_the_mask(d, e4m3, hq, hkv, bad):
    """A value that is not finite reaches the rows that see its key and no other
    row of the call, whichever kernel the number of rows selects."""
    if e4m3 and bad == math.inf:
        return  # e4m3 has no infinity
    page, n, lens = 32, [4, 3, 1], [90, 40, 17]
    c = Cache(lens, lens, hkv, d, page, e4m3, seed=21, junk=math.nan)

    def put(seq, pos, head, col):
        c.v[int(c.table[seq, pos // page]), pos % page, head, col] = bad

    put(0, 88, 1, 3)    # seen by the third and fourth of four rows
    put(0, 89, 0, d - 1)  # by the last only
    put(1, 10, 0, 7)    # under the window: by the first two of three rows
    q = rows(sum(n), hq, d, 120, 0.2)
    for splits in (0, 2):
        cu = cu_of(n)
        kc, vc, table, kw = c.to("cuda")
        args = dict(causal=True, window=(28, -1))
        out, lse = ea.attn_paged_fwd(q.cuda(), kc, vc, table, i32(cu), i32(lens), 4, 90,
                                     num_splits=splits, **args, **kw)
        ref, ref_lse, pabs = sr.attend(q, c.k, c.v, c.k_scale, c.v_scale, c.table, cu, lens,
                                       d ** -0.5, **args)
        got = out.cpu().double()
        assert torch.equal(~torch.isfinite(got), ref.isnan())
        compare(torch.where(ref.isnan(), ref, got), lse, ref, ref_lse, pabs, e4m3)


def test_cut_off_lengths_and_bad_pages():
    # lengths past the block table are cut there; pages outside the pool read as zeros
    d, page = 128, 32
    c = Cache([64, 50], [64, 64], 2, d, page, True, seed=10)
    q = rows(2, 4, d, 90, 0.2)
    kc, vc, table, kw = c.to("cuda")
    args = (q.cuda(), kc, vc)
    want = ea.attn_paged_fwd(*args, table, i32([0, 1, 2]), i32([64, 50]), 1, 64, **kw)
    got = ea.attn_paged_fwd(*args, table, i32([0, 1, 2]), i32([1000, 50]), 1, 64, **kw)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    bad = table.clone()
    bad[0, 1] = 10 ** 7
    got = ea.attn_paged_fwd(*args, bad, i32([0, 1, 2]), i32([64, 50]), 1, 64, **kw)
    assert torch.equal(want[0][1], got[0][1]) and bool(torch.isfinite(got[0]).all())


def test_a_pool_past_32_bits():
    # element offsets above 2^31 (a 2.4 GB pool), the last pages used
    d, page, hkv = 128, 128, 8
    pages = (1 << 31) // (page * hkv * d) + 2000
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough memory")
    dev = torch.device("cuda")
    c = Cache([300], [300], hkv, d, page, True, seed=11, spare=0)
    kc = torch.zeros(pages, hkv, page, d, dtype=sr.E4M3, device=dev).transpose(1, 2)
    vc = torch.zeros_like(kc)
    ks, vs = (torch.ones(pages, hkv, device=dev) for _ in range(2))
    for i in range(c.pages):
        at = pages - 1 - i
        kc[at], vc[at], ks[at], vs[at] = (x[i].to(dev) for x in (c.k, c.v, c.k_scale, c.v_scale))
    table = (pages - 1 - c.table).to(dev)
    q = rows(1, 32, d, 100, 0.2)
    k = rows(1, hkv, d, 101)
    ea.attn_paged_append(k.cuda(), k.cuda(), kc, vc, table, i32([0, 1]), i32([300]), 1, k_scale=ks,
                         v_scale=vs)
    out, lse = ea.attn_paged_fwd(q.cuda(), kc, vc, table, i32([0, 1]), i32([300]), 1, 300,
                                 k_scale=ks, v_scale=vs)
    sr.append(k, c.k, c.k_scale, c.table, [0, 1], [300])
    sr.append(k, c.v, c.v_scale, c.table, [0, 1], [300])
    ref = sr.attend(q, c.k, c.v, c.k_scale, c.v_scale, c.table, [0, 1], [300], d ** -0.5)
    compare(out, lse, *ref, True)


def test_workspace_of_the_callers():
    d, lens = 128, [700, 20]
    c = Cache(lens, lens, 2, d, 64, True, seed=12)
    q = rows(2, 8, d, 110, 0.2).cuda()
    kc, vc, table, kw = c.to("cuda")
    args = (q, kc, vc, table, i32([0, 1, 2]), i32(lens), 1, 700)
    want = ea.attn_paged_fwd(*args, num_splits=5, **kw)
    need = ea.paged_workspace_size(kc, vc, table, 2, 2, 1, 700, 8, num_splits=5, **kw)
    assert need > 0
    assert ea.paged_workspace_size(kc, vc, table, 2, 2, 1, 700, 8, num_splits=1, **kw) == 0
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN wherever it is read
    got = ea.attn_paged_fwd(*args, num_splits=5, workspace=ws, **kw)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    with pytest.raises(ea.AttnError):
        ea.attn_paged_fwd(*args, num_splits=5, workspace=ws[:need - 256], **kw)


def test_decoding_steps_equal_attention_over_the_whole():
    """Prompts appended, then tokens one by one and a few at a time, in a captured
    graph too: the attention over the bf16 cache equals attn_fwd on the rotated rows
    within the rounding of P and O, and the e4m3 cache its own definition."""
    hq, hkv, d, page = 8, 2, 128, 32
    prompt, steps = [50, 7, 129], [1, 1, 3, 1]
    total = [p + sum(steps) for p in prompt]
    f = ea.rope_frequencies(d)[0].cuda()
    q, k, v = (rows(sum(total), h, d, 200 + h, 0.2) for h in (hq, hkv, hkv + 1))
    v = v[:, :hkv].contiguous()
    cu_all = cu_of(total)
    qr, kr = ea.attn_rotary(q.cuda(), k.cuda(), f, cu_seqlens=i32(cu_all))
    full, full_lse = ea.attn_fwd(qr, kr, v.cuda(), i32(cu_all), i32(cu_all), max(total), max(total),
                                 causal=True)
    for e4m3 in (False, True):
        c = Cache([0] * 3, total, hkv, d, page, e4m3, seed=13)
        kc, vc, table, kw = c.to("cuda")
        lens = torch.zeros(3, dtype=torch.int32, device="cuda")
        at = [0, 0, 0]
        for step in [prompt] + [[s] * 3 for s in steps]:
            cu = cu_of(step)
            pick = torch.cat([torch.arange(cu_all[b] + at[b], cu_all[b] + at[b] + step[b])
                              for b in range(3)])
            at = [a + s for a, s in zip(at, step)]
            lens += i32(step)
            qo = ea.attn_paged_append(k[pick].cuda(), v[pick].cuda(), kc, vc, table, i32(cu), lens,
                                      max(step), q=q[pick].cuda(), inv_freq=f, **kw)
            assert torch.equal(qo, qr[pick.cuda()])
            out, lse = ea.attn_paged_fwd(qo, kc, vc, table, i32(cu), lens, max(step), max(total),
                                         causal=True, **kw)
            scales = [x.cpu() for x in kw.values()] or [None, None]
            ref = sr.attend(qo.cpu(), kc.cpu(), vc.cpu(), *scales, c.table, cu, at, d ** -0.5,
                            causal=True)
            # the prompts' rows take the packed copies, with P in bf16 (see attend())
            compare(out, lse, *ref, e4m3 and max(step) * (hq // hkv) < 128)
            if not e4m3:
                # both are within the bound of the same reference
                gap = (out - full[pick.cuda()]).abs().cpu().double()
                assert bool((gap <= 2 * sr.o_bound(ref[0], ref[2], False)).all())
                assert float((lse - full_lse[:, pick.cuda()]).abs().max()) <= 2 * LSE_TOL


def test_a_captured_step_replays():
    hq, hkv, d, page = 8, 2, 64, 16
    lens0 = [30, 15, 200]
    c = Cache(lens0, [x + 4 for x in lens0], hkv, d, page, True, seed=14)
    f = ea.rope_frequencies(d)[0].cuda()
    cu = i32([0, 1, 2, 3])
    q, k, v = (rows(3, h, d, 300 + i).cuda() for i, h in enumerate((hq, hkv, hkv)))
    a, b = c.to("cuda"), c.to("cuda")
    lens_a, lens_b = i32(lens0), i32(lens0)

    def step(pool, lens):
        lens += 1
        qo = ea.attn_paged_append(k, v, pool[0], pool[1], pool[2], cu, lens, 1, q=q, inv_freq=f,
                                  **pool[3])
        return ea.attn_paged_fwd(qo, pool[0], pool[1], pool[2], cu, lens, 1, 204, causal=True,
                                 num_splits=2, **pool[3])

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(a, lens_a)
    for i in range(4):
        for x, h, s in ((q, hq, 0), (k, hkv, 1), (v, hkv, 2)):
            x.copy_(rows(3, h, d, 400 + 10 * i + s))
        graph.replay()
        want = step(b, lens_b)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert same_codes(a[0], b[0]) and torch.equal(a[3]["v_scale"], b[3]["v_scale"])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("mask", [dict(causal=True), dict(), dict(causal=True, window=(70, -1)),
                                  dict(window=(5, 200), softcap=20.0)])
def test_prompt_chunks(d, e4m3, mask):
    # enough rows for the packed copies: ragged chunks, sequences without rows or keys
    n, lens = [150, 0, 33, 1, 70], [400, 300, 33, 257, 0]
    for hq, hkv, page in ((4, 2, 32), (5, 1, 128)):
        c = Cache(lens, lens, hkv, d, page, e4m3, seed=15, junk=math.nan)
        q = rows(sum(n) + 2, hq, d, 500, 0.2)
        attend(c, q, n, hq=hq, **mask)


def test_prompt_chunks_and_single_rows_agree():
    # one call with many rows, and the same rows a few at a time
    d, hq, hkv = 128, 8, 2
    n, lens = [100, 40], [300, 1000]
    c = Cache(lens, lens, hkv, d, 64, True, seed=16, junk=math.nan)
    q = rows(140, hq, d, 510, 0.2)
    whole = attend(c, q, n, hq=hq, causal=True)
    kc, vc, table, kw = c.to("cuda")
    for i in range(0, 100, 20):
        part = ea.attn_paged_fwd(q[i:i + 20].cuda(), kc, vc, table[:1], i32([0, 20]),
                                 i32([220 + i]), 20, 1000, causal=True, **{
                                     k: v for k, v in kw.items()})
        assert float((part[1] - whole[1][:, i:i + 20]).abs().max()) <= 2 * LSE_TOL


# ---------------------------------------------------------------------------
# 9 rows of a group and more over the pages themselves
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("most", [9, 16, 17, 33, 64, 65, 127, 128, 129, 300])
def test_rows_of_a_group(d, e4m3, most):
    # each number of rows a CTA can hold, one below and above it, and several row tiles
    page = {64: 16, 128: 64, 256: 128}[d]
    n, lens = [most, 0, 2, 1], [most + 200, 50, 131, 640]
    c = Cache(lens, lens, 1, d, page, e4m3, seed=most, junk=math.nan, head_major=most % 2 == 0)
    q = rows(sum(n) + 2, 1, d, 600 + most, 0.3)
    attend(c, q, n, hq=1, causal=True, splits=1)
    attend(c, q, n, hq=1, window=(130, 40), softcap=15.0, splits=4)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("e4m3", [False, True])
def test_rows_of_a_group_and_every_page(page, e4m3):
    # parts begin at any page, lengths end inside a tile, a page and a 16-key block
    n, lens = [5, 4, 5, 3, 1], [1000, 383, 129, 5, 64]
    for d, head_major in ((64, False), (128, True), (256, False)):
        c = Cache(lens, lens, 2, d, page, e4m3, seed=page, junk=math.nan, head_major=head_major)
        q = rows(sum(n), 10, d, 620, 0.3)
        for splits, window in ((1, None), (3, None), (7, (300, 10))):
            attend(c, q, n, hq=10, causal=window is None, window=window, splits=splits)


def test_queries_of_uneven_size():
    # one element far above the others of its row: the small ones decide the scores too
    d, n, lens = 128, [20], [500]
    c = Cache(lens, lens, 1, d, 64, True, seed=31)
    c.k[:, :, :, 5] = 0.0
    q = rows(20, 1, d, 630, 0.0)
    q[:, :, 5] = 256.0
    cu = [0, 20]
    kc, vc, table, kw = c.to("cuda")
    out, lse = ea.attn_paged_fwd(q.cuda(), kc, vc, table, i32(cu), i32(lens), 20, 500,
                                 num_splits=1, **kw)
    ref, ref_lse, pabs = sr.attend(q, c.k, c.v, c.k_scale, c.v_scale, c.table, cu, lens, d ** -0.5)
    # an element of q is off by at most 2^-17 of 256, so a score by at most
    # e = 2^-9 d^-1/2 max_j sum |k_j|, a weight by the factor exp(2 e) and O by that
    # much of sum p |v|, beyond the bound of the other roundings
    keys = sr.keys_of(c.k, c.k_scale, c.table[0], 500)
    e = 2.0 ** -9 * d ** -0.5 * float(keys.abs().sum(-1).max())
    err = (out.cpu().double() - ref).abs()
    assert bool((err <= sr.o_bound(ref, pabs, True) + math.expm1(2 * e) * pabs).all())
    assert float((lse.cpu().double() - ref_lse).abs().max()) <= LSE_TOL + e


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [1, 6, 30])
def test_heads_that_share_memory(e4m3, n):
    # a pool of one head seen as four (stride 0) gives what four copies give
    d, page, lens = 128, 32, [200]
    c = Cache(lens, lens, 1, d, page, e4m3, seed=41)
    kc, vc, table, kw = c.to("cuda")
    many = {k: v.expand(-1, 4).contiguous() for k, v in kw.items()}
    q = rows(n, 16, d, 640, 0.3).cuda()
    args = (table, i32([0, n]), i32(lens), n, 200)
    want = ea.attn_paged_fwd(q, kc.expand(-1, -1, 4, -1).contiguous(),
                             vc.expand(-1, -1, 4, -1).contiguous(), *args, num_splits=2, **many)
    got = ea.attn_paged_fwd(q, kc.expand(-1, -1, 4, -1), vc.expand(-1, -1, 4, -1), *args,
                            num_splits=2, **many)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("d,n", [(128, 1), (128, 4), (128, 12), (256, 5), (64, 100)])
def test_two_streams_and_a_graph(d, n):
    # calls at once on two streams, each with its own workspace, and a captured call
    # replayed after its inputs changed
    lens = [700, 900]
    cu = i32([0, n, 2 * n])
    sides, pools, qs, want = [torch.cuda.Stream() for _ in range(2)], [], [], []
    for i in range(2):
        c = Cache(lens, lens, 2, d, 64, True, seed=50 + i)
        pools.append(c.to("cuda"))
        qs.append(rows(2 * n, 8, d, 650 + i, 0.3).cuda())

    def call(i):
        kc, vc, table, kw = pools[i]
        return ea.attn_paged_fwd(qs[i], kc, vc, table, cu, i32lens, n, 900, causal=True, **kw)

    i32lens = i32(lens)
    want = [call(i) for i in range(2)]
    for side in sides:
        side.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for i, side in enumerate(sides):
            with torch.cuda.stream(side):
                got[i].append(call(i))
    for side in sides:
        torch.cuda.current_stream().wait_stream(side)
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g[0], want[i][0]) and torch.equal(g[1], want[i][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = call(0)
    qs[0].copy_(rows(2 * n, 8, d, 660, 0.3))
    i32lens -= 37
    graph.replay()
    again = call(0)
    assert torch.equal(g[0], again[0]) and torch.equal(g[1], again[1])


@pytest.mark.parametrize("n", [1, 5, 20, 200])
def test_rows_of_no_sequence_stay(n):
    # a batch padded behind its last sequence: those rows are neither read nor written
    d, lens = 128, [600, 300]
    c = Cache(lens, lens, 2, d, 64, True, seed=61)
    kc, vc, table, kw = c.to("cuda")
    q = rows(2 * n + 7, 8, d, 670, 0.3)
    q[2 * n:] = math.nan
    for splits in (0, 1, 3):
        out = torch.full_like(q, 3.0).cuda()
        lse = torch.full((8, 2 * n + 7), 3.0, device="cuda")
        ea.attn_paged_fwd(q.cuda(), kc, vc, table, i32([0, n, 2 * n]), i32(lens), n, 600, out=out,
                          lse=lse, num_splits=splits, **kw)
        assert bool((out[2 * n:] == 3).all()) and bool((lse[:, 2 * n:] == 3).all())
        assert bool(torch.isfinite(out).all())


def test_rows_of_a_group_in_a_pool_past_32_bits():
    d, page, hkv, n = 128, 64, 8, 12
    pages = (1 << 31) // (page * hkv * d) + 2000
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("not enough memory")
    dev = torch.device("cuda")
    c = Cache([300], [300], hkv, d, page, True, seed=71, spare=0)
    kc = torch.zeros(pages, hkv, page, d, dtype=sr.E4M3, device=dev).transpose(1, 2)
    vc = torch.zeros_like(kc)
    ks, vs = (torch.ones(pages, hkv, device=dev) for _ in range(2))
    for i in range(c.pages):
        at = pages - 1 - i
        kc[at], vc[at], ks[at], vs[at] = (x[i].to(dev) for x in (c.k, c.v, c.k_scale, c.v_scale))
    q = rows(n, 32, d, 680, 0.2)
    out, lse = ea.attn_paged_fwd(q.cuda(), kc, vc, (pages - 1 - c.table).to(dev), i32([0, n]),
                                 i32([300]), n, 300, causal=True, k_scale=ks, v_scale=vs)
    ref = sr.attend(q, c.k, c.v, c.k_scale, c.v_scale, c.table, [0, n], [300], d ** -0.5,
                    causal=True)
    compare(out, lse, *ref, True)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 128)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [1, 4, 10, 40, 100])
def test_pages_outside_the_pool(d, page, e4m3, n):
    # table entries that name no page of the pool read as pages of zeros, in every kernel
    lens = [400, 300]
    c = Cache(lens, lens, 2, d, page, e4m3, seed=81)
    used = {int(x) for b, m in enumerate(lens) for x in c.table[b, :-(-m // page)]}
    empty = next(i for i in range(c.pages) if i not in used)
    c.k[empty], c.v[empty] = 0, 0
    if e4m3:
        c.k_scale[empty] = c.v_scale[empty] = 1.0
    q = rows(2 * n, 4, d, 690 + n, 0.3)
    kc, vc, table, kw = c.to("cuda")
    for (b, j), name in zip(((0, 1), (0, 0), (1, 2)), (10 ** 7, -1, c.pages)):
        table[b, j] = name
        c.table[b, j] = empty
    for splits in (0, 1, 3):
        out, lse = ea.attn_paged_fwd(q.cuda(), kc, vc, table, i32([0, n, 2 * n]), i32(lens), n,
                                     400, causal=True, num_splits=splits, **kw)
        ref = sr.attend(q, c.k, c.v, c.k_scale, c.v_scale, c.table, [0, n, 2 * n], lens,
                        d ** -0.5, causal=True)
        # P in f16 except where an unsplit call of many rows packs its keys (see attend())
        compare(out, lse, *ref, e4m3 and (splits != 0 or 2 * n < 128))
