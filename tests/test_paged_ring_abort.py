"""The few-rows kernel's tile ring when waits run out, as a random-schedule model on the CPU: a producer,
copies that land in any order and as late as they like, and groups of warps that walk the run's
pieces and meet at each piece's end. Any wait may give up from some point on. However it ends, no
copy may be in flight when the last warp is through, and none may be issued over another.

What the kernel does is read from its source: whether the producer always drains its last stages or
only sees to it once the CTA has aborted, and whether a warp whose wait gave up takes further tiles."""
import os
import random
import re

import pytest

from test_abort_drains import drains_behind_the_flag
from test_paged_ring import _rows_layouts

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_37_b200", "csrc")


def source_forms():
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "paged_rows.cu")).read())
    return {"always_drain": not drains_behind_the_flag(code),
            "dead_warps_stay_dead": bool(re.search(r"bool ok = true;\s*SplitItem split", code))
            and bool(re.search(r"for \(int it = [^;]+; ok && it < q\.m;", code))}


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.done = count, 0, 0

    def arrive(self):
        self.pending += 1
        if self.pending == self.count:
            self.pending, self.done = 0, self.done + 1

    def test(self, phase):
        return (self.done & 1) != (phase & 1)


def run(stages, groups, seed, withhold=-1, forms=None):
    """'ok', or how it fails; two warps a group."""
    f = source_forms() if forms is None else forms
    r = random.Random(seed)
    pieces = [r.choice([1, 2, 3, 7, 12]) for _ in range(r.choice([1, 2, 4]))]
    full, empty = [Bar(1) for _ in range(stages)], [Bar(2) for _ in range(stages)]
    flying, flag, now, at = {}, [False], [0], r.randrange(300)
    meet = {"n": 0, "gen": 0}
    warps = 2 * groups

    def wait(b, phase):
        while not b.test(phase):
            if flag[0] or (now[0] > at and r.random() < 0.02):
                return False
            yield
        yield
        return True

    def producer():
        k, ok = 0, True
        for m in pieces:
            for _ in range(m):
                if k >= stages:
                    ok = yield from wait(empty[k % stages], k // stages - 1)
                if not ok:
                    flag[0] = True
                    break
                if k != withhold:
                    if k % stages in flying:
                        raise AssertionError("loaded over a copy in flight")
                    flying[k % stages] = full[k % stages]
                k += 1
                yield
            if not ok:
                break
        if f["always_drain"] or flag[0]:
            for t in range(max(0, k - stages), k):
                if t != withhold:
                    while not full[t % stages].test(t // stages):
                        yield

    def warp(g):
        k, ok = 0, True
        for m in pieces:
            if not f["dead_warps_stay_dead"]:
                ok = True
            it = (g + groups - k % groups) % groups
            while ok and it < m:
                ok = yield from wait(full[(k + it) % stages], (k + it) // stages)
                if not ok:
                    flag[0] = True
                    break
                empty[(k + it) % stages].arrive()
                it += groups
            k += m
            gen = meet["gen"]
            meet["n"] += 1
            if meet["n"] == warps:
                meet["n"], meet["gen"] = 0, gen + 1
            while meet["gen"] == gen:
                yield

    live = {"p": producer(), **{f"w{i}": warp(i // 2) for i in range(warps)}}
    slow = r.choice([1.0, 0.02])
    for _ in range(30000):
        now[0] += 1
        if not live:
            return "copies in flight at the end" if flying else "ok"
        c = r.choice(list(live) + (["land"] if flying and r.random() < slow else []))
        if c == "land":
            flying.pop(r.choice(sorted(flying))).arrive()
            continue
        try:
            next(live[c])
        except StopIteration:
            del live[c]
        except AssertionError as e:
            return str(e)
    return "never ends"


@pytest.mark.parametrize("withheld", [False, True])
@pytest.mark.parametrize("stages,groups", _rows_layouts())
def test_a_cta_that_gives_up_leaves_nothing_in_flight(stages, groups, withheld):
    for seed in range(300):
        assert (seed, run(stages, groups, seed, seed % 9 if withheld else -1)) == (seed, "ok")


@pytest.mark.parametrize("form", ["always_drain", "dead_warps_stay_dead"])
def test_the_model_sees_the_forms_that_were_once_there(form):
    forms = {"always_drain": True, "dead_warps_stay_dead": True, form: False}
    assert any(run(s, g, seed, seed % 9 if seed % 2 else -1, forms) != "ok" for s, g in _rows_layouts() for seed in range(400))
