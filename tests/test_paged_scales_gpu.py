"""Scales of an e4m3 cache that another quantiser wrote: any positive number, where the
append itself makes powers of two.  On the GPU, against the 64-bit definitions."""
import math

import pytest
import torch

import exact_attention_129_b200 as ea
from tests import serving_ref as sr
from tests.serving_ref import Cache
from tests.test_paged_gpu import BF, compare, cu_of, i32, rows, same_codes

pytestmark = pytest.mark.gpu


def foreign(c, seed):
    """The cache's scales times numbers in [1, 2)."""
    g = torch.Generator().manual_seed(seed)
    for name in ("k_scale", "v_scale"):
        s = getattr(c, name)
        setattr(c, name, (s * (1 + torch.rand(s.shape, generator=g))).float())
    return c


@pytest.mark.parametrize("max_n", [8, 64])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_append_rounds_ties_to_even(d, max_n):
    # y / s half way between two codes, for scales whose rounded reciprocal is above 1 / s
    # (1.75 is the smallest), and a zero with a sign
    page, n, before = 32, [3, 4], [5, 9]
    cu, lens = cu_of(n), [a + b for a, b in zip(n, before)]
    for s in (1.75, 0.875, 1.5, 1.0, 1.1, 448.0 / 7):
        c = Cache(before, lens, 2, d, page, True, seed=91)
        c.k_scale[:], c.v_scale[:] = s, s * 4
        x = torch.zeros(sum(n), 2, d, dtype=torch.float64)
        ties = torch.tensor([(m / 16) * 2.0 ** e for m in range(17, 32, 2) for e in range(-5, 6)])
        for i in range(d):
            x[:, :, i] = ties[i % len(ties)] * s * (-1) ** (i // len(ties))
        x[0, 0, 0], x[1, 1, 1] = -0.0, 0.0
        x = x.to(BF)
        kc, vc, table, kw = c.to("cuda")
        ea.attn_paged_append(x.cuda(), (4 * x.float()).to(BF).cuda(), kc, vc, table, i32(cu),
                             i32(lens), max_n, **kw)
        sr.append(x, c.k, c.k_scale, c.table, cu, lens)
        sr.append((4 * x.float()).to(BF), c.v, c.v_scale, c.table, cu, lens)
        assert same_codes(kc.cpu(), c.k) and same_codes(vc.cpu(), c.v), s
        assert torch.equal(kw["k_scale"].cpu(), c.k_scale)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [[1, 1, 1], [5, 2, 1], [14, 3, 1], [40, 9, 1], [100, 30, 1]])
def test_attention_over_the_pages(monkeypatch, d, n):
    monkeypatch.setenv("ATTN_PAGED_PACK", "0")
    lens = [400, 130, 65]
    c = foreign(Cache(lens, lens, 2, d, 32, True, seed=92, junk=math.nan), 92)
    q = rows(sum(n), 4, d, 700, 0.2)
    kc, vc, table, kw = c.to("cuda")
    ref = sr.attend(q, c.k, c.v, c.k_scale, c.v_scale, c.table, cu_of(n), lens, d ** -0.5,
                    causal=True)
    for splits in (0, 1, 3):
        out, lse = ea.attn_paged_fwd(q.cuda(), kc, vc, table, i32(cu_of(n)), i32(lens), max(n),
                                     400, causal=True, num_splits=splits, **kw)
        compare(out, lse, *ref, True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("splits", [0, 3])
def test_attention_through_packed_copies(monkeypatch, d, splits):
    # code times scale is rounded to bf16 there: compared with the definition over the
    # values so rounded, which is what the copies hold
    monkeypatch.setenv("ATTN_PAGED_PACK", "1")
    n, lens = [140, 30, 1], [400, 130, 65]
    c = foreign(Cache(lens, lens, 2, d, 32, True, seed=93, junk=math.nan), 93)
    q = rows(sum(n), 4, d, 710, 0.2)
    kc, vc, table, kw = c.to("cuda")
    held = []
    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        held.append((x.float() * s[:, None, :, None]).to(BF))
    ref = sr.attend(q, *held, None, None, c.table, cu_of(n), lens, d ** -0.5, causal=True)
    out, lse = ea.attn_paged_fwd(q.cuda(), kc, vc, table, i32(cu_of(n)), i32(lens), max(n), 400,
                                 causal=True, num_splits=splits, **kw)
    compare(out, lse, *ref, False)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [3, 20])
def test_append_at_the_last_positions(e4m3, n):
    # positions up to 2^31 - 2 lie past any block table: nothing is written, and the
    # queries are rotated by them all the same, in both kernels
    d, page, top = 64, 16, 2 ** 31 - 1
    c = Cache([16], [16], 2, d, page, e4m3, seed=94)
    k, q = rows(n, 2, d, 95).cuda(), rows(n, 4, d, 96).cuda()
    kc, vc, table, kw = c.to("cuda")
    f = ea.rope_frequencies(d)[0].cuda()
    out = ea.attn_paged_append(k, k, kc, vc, table, i32([0, n]), i32([top]), n, q=q, inv_freq=f,
                               **kw)
    pos = torch.arange(top - n, top, dtype=torch.int64)
    want = ea.attn_rotary(q, None, f, positions=pos.int().cuda())[0]
    assert torch.equal(out, want)
    # in place: each row is rotated once
    ea.attn_paged_append(k, k, kc, vc, table, i32([0, n]), i32([top]), n, q=q, q_out=q, inv_freq=f,
                         **kw)
    assert torch.equal(q, want)
    assert same_codes(kc.cpu(), c.k) and same_codes(vc.cpu(), c.v)
