"""The cross attention's ring of value tiles, every schedule of a small model of
it (no GPU).

The producer fills a stage, the warp that writes zeros over value rows that
must not count ("fixer") passes it, the MMA warp reads it. A wait names the
parity of a phase only, so a warp that falls a whole turn of the ring behind
takes a later phase for its own. The model has the arrivals that the kernel's
source gives the barrier on which the producer waits for an empty stage.
"""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "audio_diffusion_transformer_h3_b200", "csrc")


class Barrier:
    """(phases completed, arrivals still missing) as a tuple in the state."""

    @staticmethod
    def passes(bar, parity):
        return bar[0] & 1 != parity   # the phase with that parity is not the current one

    @staticmethod
    def arrive(bar, count):
        phases, missing = bar
        return (phases + 1, count) if missing == 1 else (phases, missing - 1)


def find_fault(tiles, fixed, stages, empty_count, fixer_releases):
    """The first schedule's end that is wrong, or None: a warp at a tile that its
    stage does not hold, or no warp that can go on."""
    def parity(j):
        return j // stages & 1

    def replace(t, i, x):
        return t[:i] + (x,) + t[i + 1:]

    # (producer, fixer, MMA: tile; full, empty, fix barriers; tile in each stage)
    start = (0, 0, 0, ((0, 1),) * stages, ((0, empty_count),) * stages, ((0, 1),) * stages,
             (-1,) * stages)
    seen, todo = {start}, [start]
    while todo:
        p, f, m, full, empty, fix, held = todo.pop()
        steps = []
        if p < tiles:
            s = p % stages
            if Barrier.passes(empty[s], parity(p) ^ 1):
                steps.append((p + 1, f, m, replace(full, s, Barrier.arrive(full[s], 1)), empty, fix,
                              replace(held, s, p)))
        if f < tiles:
            s = f % stages
            if Barrier.passes(full[s], parity(f)):
                if held[s] != f:
                    return f"the fixer of tile {f} finds tile {held[s]}"
                steps.append((p, f + 1, m, full,
                              replace(empty, s, Barrier.arrive(empty[s], empty_count))
                              if fixer_releases else empty,
                              replace(fix, s, Barrier.arrive(fix[s], 1)) if f in fixed else fix, held))
        if m < tiles:
            s = m % stages
            turn = sum(1 for j in fixed if j < m and j % stages == s) & 1
            if Barrier.passes(full[s], parity(m)) and (m not in fixed or Barrier.passes(fix[s], turn)):
                if held[s] != m or (m in fixed and f <= m):
                    return f"the MMA of tile {m} finds tile {held[s]}, fixer at {f}"
                e = empty[s]
                for _ in range(2):   # one commit for each query tile
                    e = Barrier.arrive(e, empty_count)
                steps.append((p, f, m + 1, full, replace(empty, s, e), fix, held))
        if not steps and not (p == f == m == tiles):
            return f"stuck: producer at {p}, fixer at {f}, MMA at {m}"
        for x in steps:
            if x not in seen:
                seen.add(x)
                todo.append(x)
    return None


def _kernel():
    """(arrivals of the empty barrier, whether the fixer is one of them)"""
    with open(os.path.join(CSRC, "cross_attn.cuh")) as f:
        text = f.read()
    count = int(re.search(r"mbar_init\(&bars\[CB_VEMPTY \+ s\], (\d+)\)", text).group(1))
    fixer = text[text.index("== value rows that must not count"):text.index("== MMA issuer")]
    return count, "CB_VEMPTY" in fixer


@pytest.mark.parametrize("stages", [2, 4])
@pytest.mark.parametrize("tiles,fixed", [(9, {8}), (12, {3, 11}), (7, {2}), (10, set(range(10))),
                                         (10, set()), (11, {0, 1, 9, 10})])
def test_no_schedule_loses_a_phase(stages, tiles, fixed):
    count, releases = _kernel()
    assert count == 2 + releases
    assert find_fault(tiles, fixed, stages, count, releases) is None


def test_the_model_sees_a_fixer_that_holds_nothing_back():
    assert find_fault(9, {8}, 2, 2, False) is not None
