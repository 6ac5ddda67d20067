"""A model of the paged tile kernel's synchronisation, run on the CPU under random schedules.

The agents follow paged_tiles_kernel's code: the producers of Q, K and V (bf16: with the tiles whose
rows it clears; e4m3: code pieces and their converters), the MMA issuer with its long-run loop, and
the softmax warps, two (a row's column halves) in a pair. mbarriers are modelled by their completed
phases and the one-bit parity test; copies land in any order, MMAs and commits complete in issue
order. In half of the runs waits give up at random, as when a wait limit runs out. Checked:

* no deadlock, in an aborting CTA either;
* every read finds its own tile, piece or exchanged value: Q, K, V, V codes and scales, K scales,
  sigma, S, P, O, the word that a row's two warps exchange;
* nothing is loaded over a copy in flight or an operand that an issued MMA still reads, no barrier is
  armed twice in a phase;
* when the CTA ends no copy and no MMA is in flight.

Planted mistakes, each of which the model must see: a shorter scale ring, no flush of the PV that
holds up a V stage, the row tiles always in one order, drains only of a CTA that has already
aborted, stages released by a failed wait, and no barrier between the two uses of the exchange word.
Stage counts and the forms of the last three are read from the kernel's source."""
import os
import random
import re

import pytest

from test_abort_drains import drains_behind_the_flag

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_37_b200", "csrc")
SRC = open(os.path.join(CSRC, "paged_tiles.cu")).read()


def _ternary(e, env):
    """A C conditional expression over D, E4M3, SPLIT and other constants."""
    e = e.strip()
    depth, q = 0, None
    for i, ch in enumerate(e):
        if ch == "(":
            depth += 1
        elif ch == ")":
            depth -= 1
        elif ch == "?" and depth == 0:
            q = i
            break
    if q is None:
        if e.startswith("(") and e.endswith(")") and "?" in e:
            return _ternary(e[1:-1], env)
        return eval(e.replace("&&", " and ").replace("!", " not "), {}, env)
    n = 0
    for i in range(q + 1, len(e)):
        n += {"?": 1, ":": -1}.get(e[i], 0) if _level(e, i) == 0 else 0
        if n < 0:
            return _ternary(e[q + 1:i] if eval(e[:q].replace("&&", " and ").replace("!", " not "), {}, env) else e[i + 1:], env)
    raise ValueError(e)


def _level(e, at):
    return e[:at].count("(") - e[:at].count(")")


def config(d, e4m3, split):
    env = {"D": d, "E4M3": e4m3, "SPLIT": split}
    for name in ("SK", "SV", "RAW", "R"):
        env[name] = int(_ternary(re.search(rf"int {name} = ([^;]+);", SRC).group(1), env))
    return env


def source_forms():
    """How the kernel is written, for the mistakes that were once in it."""
    code = re.sub(r"//[^\n]*", "", SRC)
    return {"always_drain": not drains_behind_the_flag(code),
            "commit_if_ok": bool(re.search(r"if \(ok\) tc_commit_warp\(&k_empty\[st\]\)", code))
            and bool(re.search(r"if \(!ok\) break;\s*tc_commit_warp\(&k_empty\[ks\]\)", code)),
            "word_barrier": bool(re.search(r"top = max\(top, __float_as_uint\(\*mx_other\)\);\s*named_bar\(pair_bar, 64\);", code))}


class Fault(AssertionError):
    pass


def need(ok, what):
    if not ok:
        raise Fault(what)


class Bar:
    moves = 0  # arrivals anywhere: an agent may arrive and then find that it has to wait

    def __init__(self, count):
        self.count, self.arrived, self.done = count, 0, 0

    def arrive(self):
        Bar.moves += 1
        self.arrived += 1
        if self.arrived == self.count:
            self.arrived, self.done = 0, self.done + 1

    def test(self, phase):
        return (self.done & 1) != (phase & 1)


class Named:
    def __init__(self, count):
        self.count, self.n, self.gen = count, 0, 0

    def sync(self):
        g = self.gen
        Bar.moves += 1
        self.n += 1
        if self.n == self.count:
            self.n, self.gen = 0, self.gen + 1
        while self.gen == g:
            yield False
        yield True


WARPS = 4   # softmax warps of a row tile in the model: two pairs
CONV = 2    # converter warps


class Piece:
    """m tiles; ranges of the two row tiles (SPLIT: alternate tiles); which pairs have written rows."""

    def __init__(self, r, split):
        self.split, self.m = split, r.choice([1, 1, 2, 3, 5, 8, 13, 20])
        # (a row tile that keeps keys has a written row)
        self.rows = [r.choice([[True, True], [True, False], [True, True], [False, True]]) for _ in range(2)]
        self.clear = [r.random() < 0.15 for _ in range(self.m)]
        if split:
            self.rows[1] = self.rows[0]
            self.a, self.e = [0, 0], [self.m if r.random() < 0.95 else 0] * 2
        else:
            kind = r.random()
            self.a, self.e = [0, 0], [self.m, self.m]
            if kind < 0.4:      # causal: the upper tile ends earlier
                self.e[0] = r.randint(0, self.m)
            elif kind < 0.6:    # window: and begins earlier
                self.e[0], self.a[1] = r.randint(0, self.m), r.randint(0, self.m)
            elif kind < 0.75:   # one row tile
                w = r.randint(0, 1)
                self.e[w] = 0
            elif kind < 0.85:   # anything
                for w in range(2):
                    self.a[w], self.e[w] = sorted((r.randint(0, self.m), r.randint(0, self.m)))

    def mask(self, i):
        if self.split:
            return 1 << (i & 1) if i < self.e[0] else 0
        return sum(1 << w for w in range(2) if self.a[w] <= i < self.e[w])

    def last(self, i, w):
        return i + 2 >= self.e[0] if self.split else i + 1 == self.e[w]

    def any(self, w):
        return self.e[0] > w if self.split else self.e[w] > self.a[w]


def run(d, e4m3, split, seed, aborts=False, withhold=-1, plant=(), steps=200000):
    r = random.Random(seed)
    cfg = config(d, e4m3, split)
    SK, SV, RAW, R = cfg["SK"], cfg["SV"], cfg["RAW"], cfg["R"]
    form = source_forms()
    for name in plant:
        if name == "short ring":
            R = 2
        elif name in form:
            form[name] = False
    pieces = [Piece(r, split) for _ in range(r.choice([1, 2, 3, 5]))]
    slots = 1 if split else 2
    bars, named = {}, {}

    def bar(name, i=0):
        count = {"q_ready": WARPS, "p_full": WARPS, "o_free": WARPS, "v_full": CONV if e4m3 else 1,
                 "raw_empty": CONV}.get(name, 1)
        return bars.setdefault((name, i), Bar(count))

    def nb(name, count):
        return named.setdefault(name, Named(count))

    held = {}       # (kind, slot) -> what lies there
    flying = {}     # (kind, slot) -> landing
    pipe = []       # issued MMAs and commits, in order
    st = {"flag": False, "void": False, "drains": set()}

    def data(ok, what):
        need(st["void"] or ok, what)

    give_up = {"at": r.randrange(400) if aborts else None, "n": 0}

    def wait(b, phase):
        while True:
            if b.test(phase):
                yield True
                return True
            if st["flag"] or (aborts and give_up["n"] > give_up["at"] and r.random() < 0.02):
                st["void"] = True  # from here on results may be anything, and accesses must still be sound
                return False
            yield False

    def drain(b, phase, who):
        while not b.test(phase):
            st["drains"].add(who)
            yield False
        st["drains"].discard(who)

    def reads(kind, i):
        return any(op[0] == "mma" and (kind, i) in op[2] for op in pipe)

    def tma(kind, i, what, b):
        need((kind, i) not in flying, f"{kind} {i}: loaded over a copy in flight")
        need(not reads(kind, i), f"{kind} {i}: loaded over an operand in use")
        held[kind, i] = None

        def land():
            held[kind, i] = what
            b.arrive()
        flying[kind, i] = land

    def fail():
        st["flag"] = True

    # ------------------------------------------------------------------ producers
    def q_producer():
        pc, ok = 0, True
        for pc_, _ in enumerate(pieces):
            if pc > 0:
                ok = yield from wait(bar("q_empty"), pc - 1)
                for w in range(slots):
                    ok = ok and (yield from wait(bar("q_full", w), pc - 1))
                if not ok:
                    fail()
                    break
            for w in range(slots):
                tma("q", w, ("q", pc), bar("q_full", w))
            pc += 1
            yield True
        if pc > 0 and (form["always_drain"] or st["flag"]):
            for w in range(slots):
                yield from drain(bar("q_full", w), pc - 1, "q")

    def kv_producer(kind):
        S = SK if kind == "k" else SV
        k = landed = 0
        ok = True
        for p in pieces:
            for i in range(p.m):
                if p.mask(i) == 0:
                    continue
                s = k % S
                if k >= S:
                    ok = yield from wait(bar(kind + "_empty", s), k // S - 1)
                if not ok:
                    fail()
                    break
                if kind == "k" and k == withhold:
                    k += 1
                    continue
                clear = kind == "v" and p.clear[i]
                tma(kind, s, k, bar("v_land") if clear else bar(kind + "_full", s))
                if e4m3:
                    tma("sc", k % R, k, bar("sc_full", k % R))
                yield True
                if clear:
                    ok = yield from wait(bar("v_land"), landed)
                    landed += 1
                    if not ok:
                        fail()
                        yield from drain(bar("v_land"), landed - 1, kind)
                        break
                    data(held["v", s] == k, "cleared another tile")
                    bar("v_full", s).arrive()
                k += 1
            if not ok:
                break
        if form["always_drain"] or st["flag"]:
            for t in range(max(0, k - S), k):
                if kind == "v" or t != withhold:
                    yield from drain(bar(kind + "_full", t % S), t // S, kind)
            for t in range(max(0, k - R), k) if e4m3 else ():
                if t != withhold:
                    yield from drain(bar("sc_full", t % R), t // R, kind)

    def code_producer():
        c = k = 0
        ok = True
        for p in pieces:
            for i in range(p.m):
                if p.mask(i) == 0:
                    continue
                for x in range(2):
                    if c >= RAW:
                        ok = yield from wait(bar("raw_empty", c % RAW), c // RAW - 1)
                    if not ok:
                        fail()
                        break
                    tma("raw", c % RAW, c, bar("raw_full", c % RAW))
                    if x == 0:
                        held["land", k % RAW] = k
                    yield True
                    c += 1
                if not ok:
                    break
                k += 1
            if not ok:
                break
        if form["always_drain"] or st["flag"]:
            for t in range(max(0, c - RAW), c):
                yield from drain(bar("raw_full", t % RAW), t // RAW, "raw")

    def converter(cw):
        c = k = 0
        ok = True
        for p in pieces:
            for i in range(p.m):
                if p.mask(i) == 0:
                    continue
                for half in range(2):
                    ok = yield from wait(bar("raw_full", c % RAW), c // RAW)
                    if ok and half == 0:
                        data(held["land", k % RAW] == k, "V scales of another tile")
                        if r.random() < 0.3:  # (the same for every warp in the kernel; waiting more often is no harm)
                            ok = yield from wait(bar("raw_full", (c + 1) % RAW), (c + 1) // RAW)
                            data(not ok or held["raw", (c + 1) % RAW] == c + 1, "codes of another piece")
                        if cw == 0:
                            held["sig", k % R] = k
                            bar("sig_full", k % R).arrive()
                        if k >= SV:
                            ok = ok and (yield from wait(bar("v_empty", k % SV), k // SV - 1))
                    if not ok:
                        fail()
                        break
                    data(held["raw", c % RAW] == c and held["land", k % RAW] == k, "codes or scales of another piece")
                    need(not reads("v", k % SV), "V converted over an operand in use")
                    held["v", k % SV] = k
                    yield True
                    data(held["raw", c % RAW] == c, "codes replaced under the converter")
                    bar("raw_empty", c % RAW).arrive()
                    if half == 1:
                        bar("v_full", k % SV).arrive()
                    c += 1
                if not ok:
                    break
                k += 1
            if not ok:
                break

    # ------------------------------------------------------------------ issuer
    tile = [{"pt": -1, "np": 0, "nf": 0, "fresh": False, "last": False} for _ in range(2)]
    s_of, p_of = [None, None], [None, None]      # whose S lies in tensor memory, whose P is ready
    o_busy = [False, False]                      # O holds results that were not read yet

    def commit(b):
        pipe.append(("commit", b))

    def pv(w, u, fresh):
        data(held.get(("v", u % SV)) == u and ("v", u % SV) not in flying, "PV on another V tile")
        data(p_of[w] == u, "PV before its P")
        data(not (fresh and o_busy[w]), "PV over an O that was not read")
        p_of[w] = None
        o_busy[w] = True
        pipe.append(("mma", ("pv", w, u), {("v", u % SV), ("p", w), ("o", w)}))

    def qk(w, k, pc):
        data(held.get(("k", k % SK)) == k and ("k", k % SK) not in flying, "QK on another K tile")
        q = held.get(("q", 0 if split else w))
        data(q == (("Q8" if e4m3 else "q"), pc), "QK on another Q")
        data(s_of[w] is None and p_of[w] is None, "QK over S or P in use")
        s_of[w] = ("flying", k)
        pipe.append(("mma", ("qk", w, k), {("k", k % SK), ("q", 0 if split else w), ("s", w)}))

    def issuer():
        v_seen = k = 0
        rem = [[] for _ in range(SV)]
        ok, issued = True, False
        for pc, p in enumerate(pieces):
            if not ok:
                break
            for w in range(slots):
                ok = ok and (yield from wait(bar("q_ready" if e4m3 else "q_full", w), pc))
            for t in tile:
                t["fresh"] = True
            i = 0
            while i <= p.m and ok:
                flush = i == p.m
                nw = 0 if flush else p.mask(i)
                if nw == 0 and not flush:
                    i += 1
                    continue
                s = k % SK
                if (not e4m3 and not split and nw == 3 and all(t["pt"] == k - 1 and not t["fresh"] for t in tile)):
                    n = min(p.e) - i
                    for x in range(n):
                        if not ok:
                            break
                        kk = k + x
                        ok = (yield from wait(bar("k_full", kk % SK), kk // SK)) and (
                            yield from wait(bar("v_full", (kk - 1) % SV), (kk - 1) // SV))
                        for w in range(2):
                            ok = ok and (yield from wait(bar("p_full", w), tile[w]["np"]))
                            if not ok:
                                break
                            pv(w, kk - 1, False)
                            if w:
                                commit(bar("v_empty", (kk - 1) % SV))
                            qk(w, kk, pc)
                            commit(bar("s_full", w))
                            yield True
                        if not ok and form["commit_if_ok"]:
                            break
                        commit(bar("k_empty", kk % SK))
                        for t in tile:
                            t["np"] += 1
                    k += n
                    v_seen = k - 1
                    rem = [[] for _ in range(SV)]
                    rem[(k - 1) % SV] = [k - 1, k - 1]
                    for w, t in enumerate(tile):
                        t["pt"], t["last"] = k - 1, i + n == p.e[w]
                    i += n
                    continue
                if not flush:
                    ok = yield from wait(bar("k_full", s), k // SK)
                else:
                    commit(bar("q_empty"))
                w0 = 1 if nw == 1 and "one order" not in plant else 0
                for w in (w0, 1 - w0):
                    t = tile[w]
                    held_up = t["pt"] <= k - SV and "no flush" not in plant
                    if ok and t["pt"] >= 0 and (flush or (nw >> w) & 1 or held_up):
                        u = t["pt"]
                        while v_seen <= u and ok:
                            ok = yield from wait(bar("v_full", v_seen % SV), v_seen // SV)
                            v_seen += 1
                        fresh = t["fresh"]
                        if fresh:
                            if t["nf"] > 0:
                                ok = ok and (yield from wait(bar("o_free", w), t["nf"] - 1))
                            t["nf"] += 1
                        ok = ok and (yield from wait(bar("p_full", w), t["np"]))
                        t["np"] += 1
                        if ok:
                            pv(w, u, fresh)
                            if t["last"]:
                                commit(bar("o_ready", w))
                            data(u in rem[u % SV] and len(set(rem[u % SV])) == 1, "a V stage's users mixed up")
                            rem[u % SV] = rem[u % SV][1:]
                            if not rem[u % SV]:
                                commit(bar("v_empty", u % SV))
                            yield True
                        t["fresh"], t["pt"] = False, -1
                    if ok and (nw >> w) & 1:
                        qk(w, k, pc)
                        commit(bar("s_full", w))
                        issued = True
                        rem[k % SV].append(k)
                        t["pt"], t["last"] = k, p.last(i, w)
                        yield True
                if not flush:
                    if ok or not form["commit_if_ok"]:
                        commit(bar("k_empty", s))
                    k += 1
                i += 1
        if not ok:
            fail()
        while issued and pipe:
            yield False

    # ------------------------------------------------------------------ softmax
    words = {}

    def softmax(w, pr, hf):
        j = pj = k = 0
        ok = True
        pair = f"pair {w} {pr}"

        def other(want):
            got = words[w, pr, 1 - hf]
            data(got == want, f"exchange word {got}, not {want}")
        for pc, p in enumerate(pieces):
            if e4m3:
                if not split or w == 0:
                    q = ("q", 0 if split else w)
                    ok = ok and (yield from wait(bar("q_full", w), pc))
                    data(not ok or held[q] == ("q", pc), "Q of another piece")
                    words[w, pr, hf] = ("q", pc)
                    yield from nb(f"rows {w}", WARPS).sync()
                    other(("q", pc))
                    if form["word_barrier"]:
                        yield from nb(pair, 2).sync()
                    if not ok:
                        fail()
                    bar("q_ready", w).arrive()
                    if bar("q_ready", w).arrived == 0 and ok:
                        held[q] = ("Q8", pc)
                    yield True
                else:
                    ok = ok and (yield from wait(bar("q_ready", 0), pc))
            jp = 0
            for i in range(p.m):
                nw = p.mask(i)
                if nw == 0:
                    continue
                kk = k
                k += 1
                if not (nw >> w) & 1:
                    continue
                ok = ok and (yield from wait(bar("s_full", w), j))
                if p.rows[w][pr]:
                    if e4m3:
                        ok = ok and (yield from wait(bar("sc_full", kk % R), kk // R))
                    for half in range(2):
                        if ok:
                            data(s_of[w] == ("there", kk), "another tile's S")
                            data(not e4m3 or held["sc", kk % R] == kk, "another tile's K scales")
                            data(not reads("p", w), "P written under a PV")
                        if half == 0:
                            words[w, pr, hf] = ("t", kk)
                            yield from nb(pair, 2).sync()
                            other(("t", kk))
                        yield True
                    if e4m3:
                        ok = ok and (yield from wait(bar("sig_full", kk % R), kk // R))
                        data(not ok or held["sig", kk % R] == kk, "another tile's sigma")
                    if ok and jp > 0:
                        data(not reads("o", w), "O rescaled under a PV")
                if ok:
                    b = bar("p_full", w)
                    b.arrive()
                    if b.arrived == 0:
                        s_of[w], p_of[w] = None, kk
                j += 1
                jp += 1
            if jp > 0 and ok:
                ok = yield from wait(bar("o_ready", w), pj)
                pj += 1
            if not ok:
                fail()
            words[w, pr, hf] = ("l", pc)
            yield from nb(pair, 2).sync()
            other(("l", pc))
            yield from nb(pair, 2).sync()
            for _ in range(2):
                data(not (ok and jp > 0) or not reads("o", w), "O read under a PV")
                yield True
                if split:
                    for _ in range(2):
                        yield from nb("rows", 2 * WARPS).sync()
            if p.any(w):
                b = bar("o_free", w)
                b.arrive()
                if b.arrived == 0:
                    o_busy[w] = False

    live = {"q": q_producer(), "k": kv_producer("k"), "issuer": issuer()}
    if e4m3:
        live["raw"] = code_producer()
        for cw in range(CONV):
            live[f"conv{cw}"] = converter(cw)
    else:
        live["v"] = kv_producer("v")
    for w in range(2):
        for pr in range(2):
            for hf in range(2):
                live[f"soft{w}{pr}{hf}"] = softmax(w, pr, hf)
    # in some runs copies land slowly
    slow, idle = r.choice([1.0, 1.0, 0.05]), {}
    for _ in range(steps):
        give_up["n"] += 1
        if not live:
            need(not flying, f"copies in flight at the end: {sorted(flying)}")
            need(not any(op[0] == "mma" for op in pipe), "MMAs in flight at the end")
            return "ok"
        choices = list(live) + (["land"] if flying and r.random() < slow else []) + (["pipe"] if pipe else [])
        c = r.choice(choices)
        if c == "land":
            flying.pop(r.choice(sorted(flying)))()
            idle = {}
        elif c == "pipe":
            op = pipe.pop(0)
            if op[0] == "commit":
                op[1].arrive()
            elif op[1][0] == "qk":
                s_of[op[1][1]] = ("there", op[1][2])
            idle = {}
        else:
            try:
                before = Bar.moves
                if next(live[c]) or Bar.moves != before:
                    idle = {}
                else:
                    idle[c] = idle.get(c, 0) + 1
            except StopIteration:
                del live[c]
                idle = {}
            if not flying and not pipe and live and all(idle.get(x, 0) >= (400 if aborts else 4) for x in live):
                return "a drain that never ends" if st["drains"] else "deadlock"
    return "too long"


CONFIGS = [(d, e4m3, split) for d in (64, 128) for e4m3 in (False, True) for split in (False, True)]


def _outcome(*a, **kw):
    try:
        return run(*a, **kw)
    except Fault as f:
        return str(f)


@pytest.mark.parametrize("d,e4m3,split", CONFIGS)
def test_every_schedule_ends_and_reads_its_own(d, e4m3, split):
    for seed in range(60):
        assert (seed, _outcome(d, e4m3, split, seed)) == (seed, "ok")


@pytest.mark.parametrize("d,e4m3,split", CONFIGS)
def test_a_cta_that_gives_up_ends_without_anything_in_flight(d, e4m3, split):
    for seed in range(100):
        assert (seed, _outcome(d, e4m3, split, seed, aborts=True)) == (seed, "ok")


@pytest.mark.parametrize("d,e4m3,split", CONFIGS)
def test_a_withheld_tile_ends_without_anything_in_flight(d, e4m3, split):
    for seed in range(60):
        assert (seed, _outcome(d, e4m3, split, seed, aborts=True, withhold=seed % 7)) == (seed, "ok")


PLANTS = [  # mistake, configuration, with waits that give up, what shows it
    ("short ring", (128, True, False), False, ""), ("no flush", (128, False, False), False, ""),
    ("one order", (128, False, False), False, ""), ("always_drain", (64, True, True), True, "in flight at the end"),
    ("commit_if_ok", (128, False, False), True, "in flight"), ("word_barrier", (128, True, False), False, "exchange word")]


@pytest.mark.parametrize("plant,cfg,aborts,shows", PLANTS, ids=[p[0] for p in PLANTS])
def test_the_model_sees_planted_mistakes(plant, cfg, aborts, shows):
    seen = set()
    for seed in range(600):
        seen.add(_outcome(*cfg, seed, aborts=aborts, withhold=seed % 7 if aborts else -1, plant=(plant,)))
        if any(s != "ok" and shows in s for s in seen):
            return
    raise AssertionError(seen)
