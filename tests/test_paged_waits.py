"""CPU checks of what the paged tcgen05 kernel does when a bounded wait runs out.

The kernel's warps leave their tile loops one by one then, so nothing inside a
loop may wait for other warps without a bound: no named barrier and no barrier of
the block.  Shown on the source; no test makes a wait run out in this kernel."""
import os
import re

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "exact_attention_129_b200", "csrc")
BARRIER = re.compile(r"named_bar_sync|__syncthreads|bar\.sync|cluster_sync")


def kernel():
    src = open(os.path.join(CSRC, "paged_tc.cuh")).read()
    src = re.sub(r"//[^\n]*", "", src)
    return src[src.index("attn_paged_tc_kernel("):]


def roles():
    """The branches of the kernel by warps: softmax, values, loads, MMAs."""
    src = kernel()
    at = [re.search(x, src).start() for x in (
        r"if \(warp < 4\) \{", r"\} else if \(warp < 8\) \{", r"\} else if \(warp == 9\) \{",
        r"\} else \{\s*named_bar_sync\(1, 160\)")]
    end = src.index("\n  }\n", at[3])
    return [src[a:z] for a, z in zip(at, at[1:] + [end])]


def braces(src, at):
    """src from its first brace behind `at` to the matching one."""
    at = src.index("{", at)
    depth = 0
    for i in range(at, len(src)):
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        if depth == 0:
            return src[at:i + 1]
    raise AssertionError("unbalanced")


@pytest.mark.parametrize("role", range(4))
def test_no_barrier_inside_a_tile_loop(role):
    src = roles()[role]
    loops = [braces(src, m.start()) for m in re.finditer(r"for \([^;]*;[^;]*t < tiles;", src)]
    assert loops
    for loop in loops:
        assert "wait" in loop and not BARRIER.search(loop)
        # nor in what the loop calls by name
        for name in set(re.findall(r"\b([a-z_]+)\(", loop)):
            m = re.search(r"auto %s = \[" % name, src)
            if m:
                assert not BARRIER.search(braces(src, m.end())), name


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("esz", [1, 2])
def test_the_words_a_warp_clears_are_those_it_notes(d, esz):
    bk, words = (64 if d == 256 else 128), d // 32
    cpr = d * esz // 16
    step, keys = 128 // cpr, 32 // cpr
    n = bk // step
    cleared = {}
    for warp in range(4):
        for lane in range(32):
            for i in range(lane, 2 * n * keys * words, 32):
                word, k, sign = i % words, i // words % (n * keys), i // (words * n * keys)
                key = k // keys * step + warp * keys + k % keys
                assert (sign, key, word) not in cleared
                cleared[sign, key, word] = warp
    assert len(cleared) == 2 * bk * words
    for lt in range(128):  # the keys and columns a thread looks at
        for i in range(n):
            key = lt // cpr + i * step
            for col in range(lt % cpr * (16 // esz), (lt % cpr + 1) * (16 // esz)):
                assert cleared[0, key, col // 32] == cleared[1, key, col // 32] == lt // 32


def test_copies_and_mmas_end_before_their_memory_goes():
    # another warp's wait can run out after the loading warp or the MMA warp has gone
    # through its tiles: only behind the block's last barrier is it known whether one did
    src = kernel()
    last = src.rindex("__syncthreads()")
    for role in roles()[2:]:
        assert "drain" not in role and "*abort" not in role
    tail = src[last:]
    gave_up = braces(tail, tail.index("if (*abort)"))
    assert "mbar_wait_drain(&landed[u % STAGES], (u / STAGES) & 1" in gave_up
    assert "max(0, issued - STAGES)" in gave_up and "globaltimer_ns() - t0 < " in gave_up
    assert tail.index("if (*abort)") < tail.index("tmem_dealloc")


@pytest.mark.parametrize("stages", [3, 4])
@pytest.mark.parametrize("issued", [0, 1, 2, 3, 4, 5, 11])
def test_the_drain_waits_for_the_last_phase_of_every_stage(stages, issued):
    # mbarrier phases count from 0 per stage; waiting for the parity of a phase that is
    # done, or whose successor has begun and is not done, returns
    last = {}
    for t in range(issued):
        last[t % stages] = t // stages
    waits = {u % stages: (u // stages) & 1 for u in range(max(0, issued - stages), issued)}
    assert waits == {s: phase & 1 for s, phase in last.items()}
