"""The tile rings of the paged forward as a random-schedule model on the CPU: a producer, copies that
land in any order, and consumers whose waits see one parity bit. A ring whose stages are passed
between consumer groups can take an old phase for the one it waits for; the layouts the kernels
compile keep every stage with one group, or let every consumer see every phase."""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _passed(done, phase):
    """try_wait with a parity bit: the last completed phase has the same parity."""
    return done > 0 and (done - 1) % 2 == phase % 2


def _run(stages, groups, tiles, seed):
    """'ok', or how it fails. Group g takes tiles g, g + groups, ..."""
    r = random.Random(seed)
    full, empty, held, flying = [0] * stages, [0] * stages, [None] * stages, {}
    made, at = 0, list(range(groups))
    while any(t < tiles for t in at):
        moves = [("land", s) for s in flying]
        if made < tiles and (made < stages or _passed(empty[made % stages], made // stages - 1)):
            moves.append(("make", made % stages))
        moves += [("take", g) for g in range(groups) if at[g] < tiles and _passed(full[at[g] % stages], at[g] // stages)]
        if not moves:
            return "deadlock"
        what, x = r.choice(moves)
        if what == "make":
            if x in flying:
                return "overwrite"
            flying[x] = made
            made += 1
        elif what == "land":
            held[x] = flying.pop(x)
            full[x] += 1
        else:
            s = at[x] % stages
            if held[s] != at[x] or s in flying:
                return "stale"
            empty[s] += 1
            at[x] += groups
    return "ok"


def _rows_layouts():
    """(stages, groups) of every instantiation of the few-rows kernel, from its sources' constants."""
    src = open(os.path.join(ROOT, "block_sparse_attention_37_b200", "csrc", "paged_rows.cu")).read()
    budget, cap = map(int, re.search(r"FIT = \((\d+) \* 1024\) / STAGE;.*?FIT > (\d+)", src, re.S).groups())
    out = set()
    for d in (64, 128):
        for e4m3 in (False, True):
            stage = 2 * 64 * d * (1 if e4m3 else 2) + (1024 if e4m3 else 0)
            for groups in {2 if e4m3 or d == 64 else 1, 1}:
                out.add((min(budget * 1024 // stage, cap) // groups * groups, groups))
    return sorted(out)


@pytest.mark.parametrize("stages,groups", _rows_layouts())
def test_the_compiled_rings_never_read_a_stale_tile(stages, groups):
    assert stages >= 2 and stages % groups == 0
    assert {_run(stages, groups, 40, s) for s in range(300)} == {"ok"}


def test_the_model_sees_a_ring_passed_between_groups():
    assert "stale" in {_run(3, 2, 40, s) for s in range(300)}
