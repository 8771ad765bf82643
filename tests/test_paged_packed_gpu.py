"""Attention over a paged cache through packed bf16 copies of its keys and values, on
the GPU, against the 64-bit definitions.

The library takes that way for calls with many rows, by an estimate.  Most tests here
ask for it (ATTN_PAGED_PACK=1), and every one checks by the workspace that the call
takes it.  The workspace holds NaN before the call, so nothing that the copies leave out
can be read unnoticed."""
import math

import pytest
import torch

import exact_attention_129_b200 as ea
from tests import serving_ref as sr
from tests.gpu_helpers import guarded_empty, guards_intact
from tests.serving_ref import Cache
from tests.test_paged_gpu import BF, compare, cu_of, i32, rows

pytestmark = pytest.mark.gpu


@pytest.fixture
def pack(monkeypatch):
    monkeypatch.setenv("ATTN_PAGED_PACK", "1")


def align256(n):
    return -(-n // 256) * 256


def copies(batch, max_k, hkv, d):
    """Bytes of the packed keys and values: every sequence at its longest, and 128 rows of pad."""
    return 2 * align256(batch * (max_k + 128) * hkv * d * 2)


def way(need, c, q, batch, max_k, hq):
    """("pages", parts) or ("packed", parts) for a workspace of `need` bytes: the parts of O
    and their LSE alone, or beside the copies and the segments' offsets."""
    t, d = q.shape[0], q.shape[2]
    for parts in range(1, 129):
        if need == (align256(parts * t * hq * d * 4) + parts * t * hq * 4 if parts > 1 else 0):
            return "pages", parts
    room = need - copies(batch, max_k, c.k.shape[2], d)
    assert room > 0
    return "packed", max(1, room // (t * hq * d * 4))


def run(c, q, n, *, hq, splits=0, max_k=None, packed=True, cu=None, **mask):
    """(out, lse) between guard bands, the workspace full of NaN; asserts which way is taken."""
    cu = cu_of(n) if cu is None else cu
    kc, vc, table, kw = c.to("cuda")
    max_k = max(c.lens) if max_k is None else max_k
    where = {k: v for k, v in mask.items() if k != "softcap"}
    need = ea.paged_workspace_size(kc, vc, table, len(n), q.shape[0], max(n), max_k, hq,
                                   num_splits=splits, **where, **kw)
    name, parts = way(need, c, q, len(n), max_k, hq)
    assert name == ("packed" if packed else "pages")
    assert splits == 0 or parts == splits or (not packed and parts <= splits)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    obuf, out, og = guarded_empty(q.shape, BF, kc.device)
    lbuf, lse, lg = guarded_empty((hq, q.shape[0]), torch.float32, kc.device)
    ea.attn_paged_fwd(q.cuda(), kc, vc, table, i32(cu), i32(c.lens), max(n), max_k,
                      num_splits=splits, out=out, lse=lse, workspace=ws, **mask, **kw)
    rc, msg = ea.last_device_error()
    assert rc == 0, msg
    assert guards_intact(obuf, og) and guards_intact(lbuf, lg)
    return out, lse


def check(c, q, n, *, hq, f16=False, **how):
    """run() and compare: P rounded to bf16 by attn_fwd; f16 where the paged kernels run on e4m3."""
    out, lse = run(c, q, n, hq=hq, **how)
    mask = {k: v for k, v in how.items() if k in ("causal", "window", "softcap")}
    cu = cu_of(n)
    ref, ref_lse, pabs = sr.attend(q, c.k, c.v, c.k_scale, c.v_scale, c.table, cu, c.lens,
                                   q.shape[2] ** -0.5, **mask)
    t = cu[-1]
    compare(out[:t], lse[:, :t], ref[:t], ref_lse[:, :t], pabs[:t], f16)
    return out, lse


MASKS = [dict(causal=True), dict(), dict(causal=True, window=(70, -1)),
         dict(window=(5, 200), softcap=20.0), dict(causal=True, softcap=30.0),
         dict(window=(0, 0))]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("mask", MASKS)
def test_values(pack, d, e4m3, mask):
    # ragged chunks, sequences without rows or keys, more rows than keys, lengths that end
    # inside a page; NaN in every slot of a page that holds no token
    n, lens = [150, 0, 33, 1, 70, 260, 9], [400, 300, 33, 257, 0, 700, 5]
    for hq, hkv, page, major in ((4, 2, 32, True), (5, 1, 128, False), (2, 2, 16, True)):
        c = Cache(lens, lens, hkv, d, page, e4m3, major, seed=15, junk=math.nan)
        q = rows(sum(n), hq, d, 500, 0.2)
        for splits in (0, 1, 3):
            check(c, q, n, hq=hq, splits=splits, **mask)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("splits", [0, 2])
def test_sequences_without_keys(pack, e4m3, splits):
    # every row sees nothing: max_seqlen_k 0, and an empty block table
    c = Cache([0, 0], [0, 0], 2, 128, 64, e4m3, seed=16)
    q = rows(130, 4, 128, 505, 0.2)
    for max_k in (0, 300):
        out, lse = check(c, q, [100, 30], hq=4, splits=splits, max_k=max_k, causal=True)
        assert not out.any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("d,e4m3,n,lens,hq,hkv,parts", [
    (128, True, [500, 100], [3000, 2100], 8, 2, 4), (64, True, [500, 100], [3000, 2100], 8, 2, 4),
    (64, False, [500, 100, 500, 500], [2000, 600, 500, 1500], 16, 4, 1)])
def test_the_rule_takes_the_copies_for_many_rows(d, e4m3, n, lens, hq, hkv, parts):
    c = Cache(lens, lens, hkv, d, 64, e4m3, seed=17, junk=math.nan)
    q = rows(sum(n), hq, d, 510, 0.2)
    kc, vc, table, kw = c.to("cuda")
    need = ea.paged_workspace_size(kc, vc, table, len(n), sum(n), max(n), max(lens), hq,
                                   causal=True, **kw)
    assert way(need, c, q, len(n), max(lens), hq) == ("packed", parts)
    check(c, q, n, hq=hq, causal=True)
    # a window leaves too little work for them
    check(c, q, n, hq=hq, packed=False, f16=e4m3, causal=True, window=(300, -1))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
def test_the_same_rows_over_the_pages_themselves(monkeypatch, d, e4m3):
    # the same call both ways: the paged kernels are held to their own rounding of P
    n, lens = [150, 60, 1], [400, 61, 257]
    c = Cache(lens, lens, 2, d, 64, e4m3, seed=18, junk=math.nan)
    q = rows(sum(n), 4, d, 520, 0.2)
    for mask in MASKS[:4]:
        for switch in ("0", "1"):
            monkeypatch.setenv("ATTN_PAGED_PACK", switch)
            check(c, q, n, hq=4, packed=switch == "1", f16=e4m3 and switch == "0", **mask)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (256, 128)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_outside_the_pool(pack, d, page, e4m3):
    n, lens = [140, 40], [400, 300]
    c = Cache(lens, lens, 2, d, page, e4m3, seed=81)
    used = {int(x) for b, m in enumerate(lens) for x in c.table[b, :-(-m // page)]}
    empty = next(i for i in range(c.pages) if i not in used)
    c.k[empty], c.v[empty] = 0, 0
    if e4m3:
        c.k_scale[empty] = c.v_scale[empty] = 1.0
    q = rows(sum(n), 4, d, 530, 0.3)
    bad = {(0, 1): 10 ** 7, (0, 0): -1, (1, 2): c.pages}
    for at in bad:
        c.table[at] = empty
    ref, ref_lse, pabs = sr.attend(q, c.k, c.v, c.k_scale, c.v_scale, c.table, cu_of(n), lens,
                                   d ** -0.5, causal=True)
    for at, page_id in bad.items():
        c.table[at] = page_id
    for splits in (0, 2):
        out, lse = run(c, q, n, hq=4, splits=splits, causal=True)
        compare(out, lse, ref, ref_lse, pabs, False)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("most,way_to", [(1, "0"), (5, "0"), (16, "0"), (60, "0"), (140, "0"),
                                         (140, "1")])
@pytest.mark.parametrize("cap", [1e4, 1e6, 1e30])
def test_large_softcaps(monkeypatch, d, e4m3, most, way_to, cap):
    # far above the scores the cap changes them by less than rounding, and must not
    # cost their low bits
    monkeypatch.setenv("ATTN_PAGED_PACK", way_to)
    n, lens = [most, 1], [most + 200, 70]
    c = Cache(lens, lens, 2, d, 64, e4m3, seed=19, junk=math.nan)
    q = rows(sum(n), 4, d, 525, 0.2)
    for mask in (dict(causal=True), dict(window=(90, 10))):
        check(c, q, n, hq=4, packed=way_to == "1", softcap=cap, f16=e4m3 and way_to == "0",
              splits=2, **mask)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,way_to", [(1, "0"), (5, "0"), (12, "0"), (40, "0"), (130, "0"),
                                      (130, "1")])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_the_same_bits_whatever_ran_before(monkeypatch, d, e4m3, n, way_to, cap):
    # a call's last tile is partly loaded: what an earlier call left in shared memory, large
    # keys here, must not decide how its scores are computed
    monkeypatch.setenv("ATTN_PAGED_PACK", way_to)
    seqs, size = 148, 228  # every SM, and 100 keys of a second tile
    c = Cache([size] * 4, [256] * 4, 1, d, 16, e4m3, seed=20)
    kc, vc, table, kw = c.to("cuda")
    table = table.repeat(seqs // 4, 1)
    big = torch.full_like(kc.float(), 448.0)
    big[:, ::2] = -448.0
    big = big.to(kc.dtype)
    q = rows(seqs * n, 1, d, 560, 0.0).cuda()
    cu = i32([n * i for i in range(seqs + 1)])

    def call(keys, length):
        return ea.attn_paged_fwd(q, keys, vc, table, cu, i32([length] * seqs), n, 256, causal=True,
                                 window=(200, 0), softcap=cap, num_splits=1, **kw)

    got = []
    for before in (torch.zeros_like(kc.float()).to(kc.dtype), big, kc):
        call(before, 256)
        got.append(call(kc, size))
    assert bool(torch.isfinite(got[0][0]).all())
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])


# (rows, parts) and the way: 65 to 128 rows and more over the pages, and the copies
ODD = [(65, 1, "0"), (128, 3, "0"), (140, 1, "0"), (65, 0, "1"), (140, 0, "1"), (140, 3, "1")]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("most,splits,way_to", ODD)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_not_finite_values_behind_the_mask(monkeypatch, d, e4m3, most, splits, way_to, bad):
    """A value that is not finite reaches the rows that see its key and no other row."""
    if e4m3 and bad == math.inf:
        return  # e4m3 has no infinity
    monkeypatch.setenv("ATTN_PAGED_PACK", way_to)
    page, n, lens = 32, [most, 70, 1, 40], [most + 200, 90, 17, 300]
    c = Cache(lens, lens, 2, d, page, e4m3, seed=21, junk=math.nan)

    def put(seq, pos, head, col):
        c.v[int(c.table[seq, pos // page]), pos % page, head, col] = bad

    put(0, lens[0] - 2, 1, 3)     # seen by the last two rows
    put(0, lens[0] - 1, 0, d - 1)  # by the last only
    put(0, 240, 1, 9)             # by the rows from 40 on, under no window
    put(1, 10, 0, 7)              # under the window: by the first rows only
    q = rows(sum(n), 2, d, 120, 0.2)
    for args in (dict(causal=True), dict(causal=True, window=(28, -1))):
        out, lse = run(c, q, n, hq=2, splits=splits, packed=way_to == "1", **args)
        ref, ref_lse, pabs = sr.attend(q, c.k, c.v, c.k_scale, c.v_scale, c.table, cu_of(n), lens,
                                       d ** -0.5, **args)
        got = out.cpu().double()
        assert torch.equal(~torch.isfinite(got), ref.isnan())
        compare(torch.where(ref.isnan(), ref, got), lse, ref, ref_lse, pabs, False)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("most,splits,way_to", [(1, 1, "0"), (1, 3, "0"), (5, 2, "0"),
                                                (20, 1, "0")] + ODD)
def test_not_finite_keys_and_queries(monkeypatch, d, e4m3, most, splits, way_to):
    """A key that is not finite makes O and the LSE of the rows that see it NaN, a query
    its own; with the keys in parts too, where only one of them has it."""
    monkeypatch.setenv("ATTN_PAGED_PACK", way_to)
    page, n, lens = 32, [most, most, 1], [most + 200, most + 90, 400]
    c = Cache(lens, lens, 2, d, page, e4m3, seed=22, junk=math.nan)
    q = rows(sum(n), 4, d, 121, 0.2)
    ref, ref_lse, pabs = sr.attend(q, c.k, c.v, c.k_scale, c.v_scale, c.table, cu_of(n), lens,
                                   d ** -0.5, causal=True)
    # a key of the last position, seen by the last row; and one seen by every row
    for seq, pos, seen in ((0, lens[0] - 1, slice(most - 1, most)), (1, 3, slice(most, 2 * most))):
        c.k[int(c.table[seq, pos // page]), pos % page, seq, 5] = math.nan
        heads = slice(2 * seq, 2 * seq + 2)  # those of key/value head seq
        ref[seen, heads] = pabs[seen, heads] = math.nan
        ref_lse[heads, seen] = math.nan
    q[2 * most, 1, 7] = math.nan  # the single row of the third sequence, one head
    ref[2 * most, 1] = pabs[2 * most, 1] = math.nan
    ref_lse[1, 2 * most] = math.nan
    out, lse = run(c, q, n, hq=4, splits=splits, packed=way_to == "1", causal=True)
    assert torch.equal(lse.cpu().isnan(), ref_lse.isnan())
    compare(out, lse, ref, ref_lse, pabs, False)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("splits", [0, 1, 2, 7])
def test_rows_of_no_sequence_stay(pack, d, splits):
    # a batch padded behind its last sequence: those rows are neither read nor written, in
    # one part or several
    n, lens = [140, 3], [600, 300]
    c = Cache(lens, lens, 2, d, 64, True, seed=61)
    q = rows(sum(n) + 9, 8, d, 670, 0.3)
    q[sum(n):] = math.nan
    out, lse = check(c, q, n, hq=8, splits=splits, causal=True)
    # the sentinels of guarded_empty
    assert bool((out[sum(n):].view(torch.int16) == 0x7FC1).all())
    assert bool((lse[:, sum(n):].view(torch.int32) == 0x7FC00001).all())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_two_streams_and_a_graph(pack, d):
    # calls at once on two streams, each with its own workspace; a captured call replayed
    # after its inputs changed; each call gives the same bits every time
    n, lens = [150, 30], [700, 900]
    cu, i32lens = i32(cu_of(n)), i32(lens)
    sides, pools, qs = [torch.cuda.Stream() for _ in range(2)], [], []
    for i in range(2):
        c = Cache(lens, lens, 2, d, 64, True, seed=50 + i)
        pools.append(c.to("cuda"))
        qs.append(rows(sum(n), 8, d, 650 + i, 0.3).cuda())

    def call(i, splits=0):
        kc, vc, table, kw = pools[i]
        assert ea.paged_workspace_size(kc, vc, table, 2, sum(n), max(n), 900, 8, causal=True,
                                       num_splits=splits, **kw) >= copies(2, 900, 2, d)
        return ea.attn_paged_fwd(qs[i], kc, vc, table, cu, i32lens, max(n), 900, causal=True,
                                 num_splits=splits, **kw)

    for splits in (0, 3):
        want = [call(i, splits) for i in range(2)]
        for side in sides:
            side.wait_stream(torch.cuda.current_stream())
        got = [[], []]
        for _ in range(5):
            for i, side in enumerate(sides):
                with torch.cuda.stream(side):
                    got[i].append(call(i, splits))
        for side in sides:
            torch.cuda.current_stream().wait_stream(side)
        for i in range(2):
            for g in got[i]:
                assert torch.equal(g[0], want[i][0]) and torch.equal(g[1], want[i][1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g = call(0, splits)
        qs[0].copy_(rows(sum(n), 8, d, 660 + splits, 0.3))
        i32lens -= 37
        graph.replay()
        again = call(0, splits)
        assert torch.equal(g[0], again[0]) and torch.equal(g[1], again[1])
