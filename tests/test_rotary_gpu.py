"""Rotary positions on the GPU against the 64-bit definition."""
import pytest
import torch

import exact_attention_129_b200 as ea
from tests import serving_ref as sr
from tests.gpu_helpers import guarded_empty, guards_intact

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rows(t, h, d, seed, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, h, d, generator=g) * torch.exp(spread * torch.randn(t, h, 1, generator=g))
    return x.to(BF)


def check(got, x, pos, f, mscale=1.0, inter=False, inverse=False):
    """Half a bf16 step of the exact value, plus the fp32 part."""
    ref = sr.rotate(x, pos, f, mscale, inter, inverse)
    slack = sr.rotate_slack(x, f, mscale, inter)
    err = (got.cpu().double() - ref).abs()
    bound = sr.U_BF16 * (ref.abs() + slack) + slack
    assert bool((err <= bound).all()), float((err - bound).max())
    r = 2 * f.numel()
    assert torch.equal(got.cpu()[..., r:], x[..., r:])  # what is not rotated is copied


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 48), (256, 256),
                                   (256, 96), (256, 16)])
@pytest.mark.parametrize("inter", [False, True])
def test_segments_and_offsets(d, rot, inter):
    cu, off = [0, 1, 1, 70, 203], [3, 9, 0, 130000]
    t = cu[-1]
    q, k = rows(t, 5, d, 1), rows(t, 2, d, 2)
    f, m = ea.rope_frequencies(rot, scaling="yarn", factor=16, original_max=8192)
    args = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                offsets=torch.tensor(off, dtype=torch.int32).cuda(), interleaved=inter, mscale=m)
    pos = sr.positions(cu, off)
    qo, ko = ea.attn_rotary(q.cuda(), k.cuda(), f.cuda(), **args)
    check(qo, q, pos, f, m, inter)
    check(ko, k, pos, f, m, inter)
    qi, ki = ea.attn_rotary(q.cuda(), k.cuda(), f.cuda(), inverse=True, **args)
    check(qi, q, pos, f, m, inter, True)
    check(ki, k, pos, f, m, inter, True)


@pytest.mark.parametrize("t", [0, 1, 2, 33])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (32, 8), (7, 3)])
def test_rows_positions_and_no_k(t, hq, hkv):
    q, k = rows(t, hq, 128, 3), rows(t, hkv, 128, 4)
    f = ea.rope_frequencies(128)[0]
    qo, ko = ea.attn_rotary(q.cuda(), k.cuda(), f.cuda())
    check(qo, q, torch.arange(t), f)
    check(ko, k, torch.arange(t), f)
    g = torch.Generator().manual_seed(5)
    pos = torch.randint(0, 2 ** 24, (t,), generator=g, dtype=torch.int32)
    qo, ko = ea.attn_rotary(q.cuda(), None, f.cuda(), positions=pos.cuda())
    assert ko is None
    check(qo, q, pos, f)


def test_many_tokens_and_heads_in_groups():
    # more blocks than one round of the grid, heads split into uneven groups
    t, d = 5000, 64
    q, k = rows(t, 13, d, 6), rows(t, 13, d, 7)
    f = ea.rope_frequencies(d)[0]
    qo, ko = ea.attn_rotary(q.cuda(), k.cuda(), f.cuda())
    check(qo, q, torch.arange(t), f)
    check(ko, k, torch.arange(t), f)


@pytest.mark.parametrize("inter", [False, True])
def test_views_in_place_and_guards(inter):
    t, d = 77, 128
    f = ea.rope_frequencies(96)[0]
    qkv = rows(t, 8, d, 8)
    want = ea.attn_rotary(qkv[:, :4].contiguous().cuda(), qkv[:, 4:6].contiguous().cuda(), f.cuda(),
                          interleaved=inter)
    dev = qkv.cuda()
    q, k = dev[:, :4], dev[:, 4:6]
    ea.attn_rotary(q, k, f.cuda(), interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(dev[:, 6:].cpu(), qkv[:, 6:])
    # heads before tokens in memory, outputs between guard bands
    ht = qkv[:, :4].transpose(0, 1).contiguous().cuda().transpose(0, 1)
    buf, out, n = guarded_empty((4, t, d), BF, dev.device)
    ea.attn_rotary(ht, None, f.cuda(), interleaved=inter, q_out=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), want[0]) and guards_intact(buf, n)


def test_rows_behind_the_last_segment():
    t, d = 20, 64
    q, k = rows(t, 2, d, 9), rows(t, 1, d, 10)
    f = ea.rope_frequencies(d)[0].cuda()
    cu = torch.tensor([2, 5, 13], dtype=torch.int32).cuda()
    qo, ko = ea.attn_rotary(q.cuda(), k.cuda(), f, cu_seqlens=cu)
    for x in (qo, ko):
        assert not x[:2].any() and not x[13:].any()
    keep = [torch.full_like(x, 7.0).cuda() for x in (q, k)]
    ea.attn_rotary(q.cuda(), k.cuda(), f, cu_seqlens=cu, q_out=keep[0], k_out=keep[1])
    for x, y in zip(keep, (qo, ko)):
        assert bool((x[:2] == 7).all()) and bool((x[13:] == 7).all())
        assert torch.equal(x[2:13], y[2:13])


def test_not_finite_values_stay_in_their_pair():
    q = rows(3, 2, 64, 11)
    q[1, 0, 3], q[2, 1, 40] = float("nan"), float("inf")
    f = ea.rope_frequencies(64)[0]
    out = ea.attn_rotary(q.cuda(), None, f.cuda())[0].cpu()
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[1, 0, 3] = want[1, 0, 35] = want[2, 1, 40] = want[2, 1, 8] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (128, 64, True), (256, 256, False)])
def test_gradient(d, rot, inter):
    cu, t = [0, 40, 41, 130], 150  # 20 rows of padding behind the last segment
    f, m = ea.rope_frequencies(rot, scaling="yarn", factor=4, original_max=4096)
    q, k = rows(t, 4, d, 12), rows(t, 2, d, 13)
    wq, wk = rows(t, 4, d, 14), rows(t, 2, d, 15)
    cud = torch.tensor(cu, dtype=torch.int32).cuda()
    qd, kd = q.cuda().requires_grad_(True), k.cuda().requires_grad_(True)
    qo, ko = ea.rotary(qd, kd, f.cuda(), cu_seqlens=cud, interleaved=inter, mscale=m)
    dq, dk = torch.autograd.grad((qo, ko), (qd, kd), (wq.cuda(), wk.cuda()))
    n, pos = cu[-1], sr.positions(cu)
    for got, w in ((dq, wq), (dk, wk)):
        check(got[:n], w[:n], pos, f, m, inter, True)
        assert not got[n:].any()
    # against differences of the kernel's own forward: <R(x + e) - R(x - e), w> = <2e, dx>,
    # with e a power of two and x = 0, so that the forward's bf16 rounding is all there is
    g = torch.Generator().manual_seed(16)
    for _ in range(4):
        e = torch.zeros(t, 4, d)
        at = (int(torch.randint(0, n, (1,), generator=g)), 1,
              int(torch.randint(0, d, (1,), generator=g)))
        e[at] = 0.5
        plus = ea.attn_rotary(e.to(BF).cuda(), None, f.cuda(), cu_seqlens=cud, interleaved=inter,
                              mscale=m)[0].cpu().double()
        num = float((2 * plus * wq.double()).sum())
        # two elements, each off by half a step; the gradient by half a step too
        slack = 1.01 * sr.U_BF16 * (float((2 * plus * wq.double()).abs().sum()) +
                                    abs(float(dq[at]))) + 1e-5
        assert abs(num - float(dq[at])) <= slack


def test_gradient_of_one_input_and_of_views():
    t, d = 9, 128
    f = ea.rope_frequencies(d)[0].cuda()
    q, k, w = rows(t, 4, d, 17).cuda(), rows(t, 2, d, 18).cuda(), rows(t, 2, d, 19).cuda()
    full = ea.attn_rotary(w, None, f, inverse=True)[0]
    kd = k.clone().requires_grad_(True)
    ko = ea.rotary(q, kd, f)[1]
    assert torch.equal(torch.autograd.grad(ko, kd, w)[0], full)
    # a gradient without a contiguous last dimension, as sum() and a transpose give
    ko = ea.rotary(q, kd, f)[1]
    wt = w.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(torch.autograd.grad(ko, kd, wt)[0], full)
    ko = ea.rotary(q, kd, f)[1]
    ones = ea.attn_rotary(torch.ones_like(w), None, f, inverse=True)[0]
    assert torch.equal(torch.autograd.grad(ko.sum(), kd)[0], ones)
    qd = q.clone().requires_grad_(True)
    qo, none = ea.rotary(qd, None, f)
    assert none is None
    assert torch.equal(torch.autograd.grad(qo, qd, q)[0],
                       ea.attn_rotary(q, None, f, inverse=True)[0])


def test_in_a_graph_and_on_another_stream():
    t, d = 300, 128
    f = ea.rope_frequencies(d)[0].cuda()
    q, k = rows(t, 4, d, 20).cuda(), rows(t, 2, d, 21).cuda()
    want = ea.attn_rotary(q, k, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ea.attn_rotary(q, k, f)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ea.attn_rotary(q, k, f)
    q.copy_(rows(t, 4, d, 22))
    graph.replay()
    assert torch.equal(got[0], ea.attn_rotary(q, k, f)[0]) and torch.equal(got[1], want[1])


def test_gradient_in_a_graph():
    # forward and backward captured, after an eager pass over the same leaves; the eager
    # graph is gone by then, because torch would run its accumulation nodes, which the
    # leaves keep as long as a graph lives, on the eager stream and refuse the capture
    t, d = 130, 128
    f = ea.rope_frequencies(d)[0].cuda()
    q, k = (rows(t, h, d, 30 + h).cuda().requires_grad_(True) for h in (4, 2))
    g = [rows(t, h, d, 40 + h).cuda() for h in (4, 2)]
    want = torch.autograd.grad(ea.rotary(q, k, f), (q, k), g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(ea.rotary(q, k, f), (q, k), g)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    for x in g:
        x.neg_()
    graph.replay()
    assert all(torch.equal(-a, b) for a, b in zip(want, got))
    again = torch.autograd.grad(ea.rotary(q, k, f), (q, k), g)
    assert all(torch.equal(a, b) for a, b in zip(again, got))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("both", [False, True])
def test_gradient_of_the_gradient(inter, both):
    # y = R x, so dx(w) = R^T w, which is linear in w: the gradient of <dx(w), u> by w is R u,
    # the gradient of <dx(w(x)), u> by x goes on through w(x), and a third one turns back again
    t, d = 21, 128
    f, m = ea.rope_frequencies(d, scaling="yarn", factor=4, original_max=4096)
    f, cu = f.cuda(), torch.tensor([0, 9, 21], dtype=torch.int32).cuda()
    how = dict(cu_seqlens=cu, interleaved=inter, mscale=m)
    heads = (4, 2) if both else (4,)
    x, w, u, z = ([rows(t, h, d, s + h).cuda() for h in heads] for s in (50, 60, 70, 80))
    for part in (x, w, u):
        for i in part:
            i.requires_grad_(True)

    def turn(p, inverse):
        out = ea.attn_rotary(p[0].detach(), p[1].detach() if both else None, f, inverse=inverse,
                             **how)
        return out if both else out[:1]

    y = ea.rotary(x[0], x[1] if both else None, f, **how)[:len(heads)]
    dx = torch.autograd.grad(y, x, w, create_graph=True)
    assert all(i.requires_grad for i in dx)
    for got, want in zip(dx, turn(w, True)):
        assert torch.equal(got, want)
    ddw = torch.autograd.grad(dx, w, u, create_graph=True)
    for got, want in zip(ddw, turn(u, False)):
        assert torch.equal(got, want)
    for got, want in zip(torch.autograd.grad(ddw, u, z), turn(z, True)):
        assert torch.equal(got, want)
    # through w(x) = x: d/dx <R^T x, u> = R u
    y = ea.rotary(x[0], x[1] if both else None, f, **how)[:len(heads)]
    dx = torch.autograd.grad(y, x, x, create_graph=True)
    for got, want in zip(torch.autograd.grad(dx, x, [i.detach() for i in u]), turn(u, False)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("offset", [0, 10 ** 6, -500])
def test_pairs_that_nearly_cancel(inter, offset):
    # a cos - b sin is far below a and b: what is left shows the error of cosine and sine,
    # which are to be the 64-bit ones rounded to fp32 once.  With u = 2^-24, half a step:
    # |a c| u for the product with a rounded c; 2 |b s| u for b s, rounded itself; u of the
    # result; and 2^-30 (|a| + |b|) for the sine and cosine before their rounding
    t, d = 200000, 64
    f = ea.rope_frequencies(d, 500000.0)[0]
    x = rows(t, 1, d, 23)
    out = ea.attn_rotary(x.cuda(), None, f.cuda(), cu_seqlens=torch.tensor([0, t]).int().cuda(),
                         offsets=torch.tensor([offset]).int().cuda(), interleaved=inter)[0].cpu()
    ang = (torch.arange(t, dtype=torch.float64) + offset)[:, None] * f[None, :]
    c, s = ang.cos(), ang.sin()

    def halves(y):
        y = y[:, 0].double()
        return (y[:, 0::2], y[:, 1::2]) if inter else (y[:, :d // 2], y[:, d // 2:])

    a, b = halves(x)
    ga, gb = halves(out)
    seen = 0
    for got, p, q in ((ga, a * c, -b * s), (gb, b * c, a * s)):
        want = p + q
        u = 2.0 ** -24
        bound = u * (p.abs() + 2 * q.abs() + want.abs()) + 2.0 ** -30 * (a.abs() + b.abs())
        close = want.abs() < 2.0 ** -12
        seen += int(close.sum())
        err = (got - want).abs()
        assert bool((err <= bound + sr.U_BF16 * (want.abs() + bound))[close].all()), float(
            (err / bound)[close].max())
    assert seen > 1000
