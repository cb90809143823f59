"""How the 4-bit chunk kernel (attn4_tc_kernel) hands key tiles over, checked on
the host.

Four warps make key tiles from codes.  A key row out of fp16's range is divided
by a power of two; that factor, and a mark of the warp that wrote any, go into a
slot of shared memory, and the warpgroups that turn scores into weights multiply
by it.  A key tile's stage is free when the tensor core has done its Q K^T, which
says nothing of the warpgroups: they read marks and factors only after that.  So
the slots are a ring of their own, and it has to be deep enough that no slot is
written again while a warpgroup may still read it.

This runs the hand-over as a discrete-event model with random interleavings (see
test_tc_pipeline_protocol.py): every wait is by parity as in the kernel, products
and commits complete in issue order.  Rings whose absence only gives the agents
more freedom (units, queries, raw codes, values) are left out.  The depths are
the kernel's own, printed by a host program that includes its source.
"""
import os
import random
import shutil
import subprocess

import pytest

from group_quantized_moe_gb300 import build_lib
from test_tc_pipeline_protocol import Barrier, Violation, check

PROGRAM = r"""
#include <cstdio>
#include <type_traits>
#include "attn_tc_body.cuh"
using namespace qmm;
// slots of marks and factors; where the kernel names none, one a key stage
template <typename C, typename = void> struct Slots { static constexpr int n = C::stages / 2; };
template <typename C> struct Slots<C, std::void_t<decltype(C::key_slots)>> { static constexpr int n = C::key_slots; };
int main() {
  printf("%d %d\n%d %d\n", Tc<1, false, true>::stages, Slots<Tc<1, false, true>>::n, Tc<2, false, true>::stages,
         Slots<Tc<2, false, true>>::n);
}
"""


def run(units, stages, slots, seed):
    """units: (two query tiles, key tiles, how many of them query tile A reaches)."""
    rng = random.Random(seed)
    freed, clean = [Barrier(1) for _ in range(stages)], [Barrier(4) for _ in range(stages)]
    s_full, o_full = [Barrier(1), Barrier(1)], [Barrier(1), Barrier(1)]
    p_full = [[Barrier(4), Barrier(4)] for _ in range(2)]
    tile_of = [[None] * 4 for _ in range(stages)]             # what each warp's rows of a stage hold
    factors = [[[None, None] for _ in range(4)] for _ in range(slots)]  # slot, warp, half
    marks = [[None] * 4 for _ in range(slots)]
    pipe = []

    def wait(bar, parity):
        while not bar.test(parity):
            yield bar, parity

    def maker(k):
        t = 0
        for _, tiles, _ in units:
            for _ in range(tiles):
                s, slot = 2 * t % stages, t % slots
                yield from wait(freed[s], (2 * t // stages & 1) ^ 1)
                for half in range(2):
                    yield
                    factors[slot][k][half] = t
                tile_of[s][k] = t
                yield
                marks[slot][k] = t
                clean[s].arrive()
                t += 1

    def issuer():
        n0, np = 0, [0, 0]
        for pair, tiles, reach in units:
            step = 1 if pair else 2
            cur, last = [0, 0 if pair else 1], [min(tiles, reach) if pair else tiles, tiles]
            held, w = [False, False], 0
            while held[0] or held[1] or cur[0] < last[0] or cur[1] < last[1]:
                more, frees = cur[w] < last[w], not pair or w
                if held[w]:
                    for half in range(2):
                        yield from wait(p_full[w][half], np[w] & 1)
                    np[w] += 1
                    if pair and not more:
                        pipe.append(("commit", o_full[w]))
                if more:
                    t = n0 + cur[w]
                    s = 2 * t % stages
                    yield from wait(clean[s], 2 * t // stages & 1)
                    pipe.append(("scores", s, t))
                    pipe.append(("commit", s_full[w]))
                    if frees:
                        pipe.append(("commit", freed[s]))
                    yield
                held[w] = more
                cur[w] += step
                w ^= 1
            if not pair:
                pipe.append(("commit", o_full[0]))
                if tiles > 1:
                    pipe.append(("commit", o_full[1]))
            n0 += tiles

    def warpgroup(w):  # one of its four warps
        n0, nt, no = 0, 0, 0
        for pair, tiles, reach in units:
            first, last = (0 if pair else w), (min(tiles, reach) if pair and w == 0 else tiles)
            mine = range(first, last, 1 if pair else 2)
            for i in mine:
                t = n0 + i
                slot = t % slots
                yield from wait(s_full[w], nt & 1)
                nt += 1
                check(marks[slot] == [t] * 4, f"tile {t}: marks of {marks[slot]}")
                for c in range(4):
                    yield
                    check(all(f[c >> 1] == t for f in factors[slot]), f"tile {t}: factors of {factors[slot]}")
                for half in range(2):
                    yield
                    p_full[w][half].arrive()
            if len(mine):
                yield from wait(o_full[w], no & 1)
                no += 1
            n0 += tiles

    agents = [maker(k) for k in range(4)] + [issuer()] + [warpgroup(w) for w in (0, 1) for _ in range(4)]
    speed = {id(a): rng.expovariate(1.0) + 1e-3 for a in agents}
    p_pipe = rng.uniform(0.05, 0.6)
    live = {id(a): [a, None] for a in agents}
    while live or pipe:
        if pipe and rng.random() < p_pipe:
            op = pipe.pop(0)
            if op[0] == "commit":
                op[1].arrive()
            else:
                check(tile_of[op[1]] == [op[2]] * 4, f"scores of tile {op[2]} from {tile_of[op[1]]}")
            continue
        ready = [v for v in live.values() if v[1] is None or v[1][0].test(v[1][1])]
        if not ready:
            check(pipe, "deadlock: every agent waits and nothing is in flight")
            continue
        v = rng.choices(ready, weights=[speed[id(x[0])] for x in ready])[0]
        try:
            v[1] = next(v[0])
        except StopIteration:
            del live[id(v[0])]


def some_units(seed):
    rng = random.Random(seed)
    units = []
    for _ in range(6):
        tiles, pair = rng.randint(1, 9), rng.random() < 0.5
        units.append((pair, tiles, rng.randint(0, tiles)))
    return units


@pytest.fixture(scope="module")
def depths(tmp_path_factory):
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not found")
    d = tmp_path_factory.mktemp("kv4")
    src, exe = d / "depths.cu", d / "depths"
    src.write_text(PROGRAM)
    subprocess.run([build_lib._nvcc(), *build_lib.ARCH, *build_lib.FLAGS, "-I", build_lib.CSRC, str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    return [tuple(map(int, line.split())) for line in subprocess.check_output([str(exe)], text=True).splitlines()]


def test_marks_and_factors_outlive_their_readers(depths):
    """No slot is written before the warpgroups have read it, no stage before its product."""
    assert [s for s, _ in depths] == [8, 4]
    for stages, slots in depths:
        for seed in range(400):
            run(some_units(seed), stages, slots, seed)


@pytest.mark.parametrize("stages", [8, 4])
def test_a_slot_a_stage_is_caught(stages):
    """As many slots as key stages: the commit that frees a stage lets a slot be
    written under its readers."""
    with pytest.raises(Violation):
        for seed in range(400):
            run(some_units(seed), stages, stages // 2, seed)
