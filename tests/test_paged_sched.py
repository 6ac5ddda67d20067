"""The cut of the paged forward's work, compiled for the host from the kernels' own sources: the key
spans of every row tile against the rows they stand for, and the runs against a plain walk."""
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_sparse_attention_37_b200", "csrc")

SRC = r'''
#include <cstdio>
#include <cstring>
#include "paged_sched.cuh"
using namespace bsa;
int main() {
  char op[8];
  while (scanf("%7s", op) == 1) {
    if (op[0] == 's') {  // spans: rows keys N G causal window n kv -> lines of lo hi clo chi t0 nt
      int rows, keys, N, G, causal, window, n, kv;
      if (scanf("%d %d %d %d %d %d %d %d", &rows, &keys, &N, &G, &causal, &window, &n, &kv) != 8) return 1;
      PagedParams p;
      std::memset(&p, 0, sizeof(p));
      p.N = N; p.G = G; p.causal = causal; p.window = window; p.f_n = make_fastdiv(N);
      const int rts = (G * N + rows - 1) / rows;
      for (int rt = 0; rt < rts; ++rt) {
        ItemSpan s = rows == 16 ? item_span<16, 64>(p, n, kv, rt)
                   : rows == 128 ? item_span<128, 128>(p, n, kv, rt) : item_span<256, 128>(p, n, kv, rt);
        printf("%d %d %d %d %d %d\n", s.lo, s.hi, s.clo, s.chi, s.t0, s.nt);
      }
    } else {  // runs: total grid min -> ctas, then start of each run and the run of each tile
      long long total; int grid, mn;
      if (scanf("%lld %d %d", &total, &grid, &mn) != 3) return 1;
      const int c = run_ctas(total, grid, mn);
      printf("%d\n", c);
      for (int i = 0; i <= c; ++i) printf("%lld ", run_start(total, i, c));
      for (long long x = 0; x < total; ++x) printf("%d ", run_of(total, x, c));
      printf("\n");
    }
  }
  return 0;
}
'''


@pytest.fixture(scope="module")
def tool(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged_sched")
    src, exe = d / "t.cu", d / "t"
    src.write_text(SRC)
    from block_sparse_attention_37_b200 import build
    subprocess.run([build.nvcc_path(), "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a", "-I", CSRC, "-o", str(exe), str(src)],
                   check=True, capture_output=True, text=True)
    return str(exe)


def _ask(tool, text):
    return subprocess.run([tool], input=text, capture_output=True, text=True, check=True).stdout.strip().split("\n")


def _want(rows, keys, N, G, causal, window, n, kv):
    out = []
    for rt in range(-(-G * N // rows)):
        toks = [r % N for r in range(rt * rows, min((rt + 1) * rows, G * N)) if r % N < n]
        kept = []
        for t in toks:
            pos = kv - n + t
            lo, hi = 0, kv
            if causal:
                hi = min(max(pos + 1, 0), kv)
                if window:
                    lo = min(max(pos - window + 1, 0), kv)
            kept.append((lo, hi))
        out.append(kept)
    return out


@pytest.mark.parametrize("rows,keys", [(16, 64), (128, 128), (256, 128)])
def test_spans_cover_their_rows_and_little_else(tool, rows, keys):
    rng = np.random.default_rng(rows)
    asks, wants = [], []
    for _ in range(250):
        G = int(rng.choice([1, 2, 3, 4, 5, 8]))
        N = int(rng.choice([1, 2, 3, 7, 16, 33, 100, 127, 128, 129, 300]))
        n = int(rng.integers(0, N + 1))
        kv = int(rng.choice([0, 1, n, n + 1, 64, 65, 128, 500, 1000]))
        causal = int(rng.integers(0, 2))
        window = int(rng.choice([0, 1, 5, 64, 200, 2**31 - 1])) if causal else 0
        asks.append(f"s {rows} {keys} {N} {G} {causal} {window} {n} {kv}")
        wants.append((asks[-1], _want(rows, keys, N, G, causal, window, n, kv), N, n))
    lines = iter(_ask(tool, "\n".join(asks)))
    for what, tiles, N, n in wants:
        for kept in tiles:
            lo, hi, clo, chi, t0, nt = map(int, next(lines).split())
            if not kept:
                assert nt == 0, what
                continue
            assert nt >= 1, what
            some = [(a, b) for a, b in kept if a < b]
            if not some:
                assert lo == hi == 0 and nt == 1, what
                continue
            # [lo, hi) holds every kept key; [clo, chi) lies inside every row's
            assert lo <= min(a for a, _ in some) and hi >= max(b for _, b in some), what
            assert clo >= max(a for a, _ in kept) and chi <= min(b for _, b in kept) or clo >= chi, what
            assert t0 == lo // keys and (t0 + nt) * keys >= hi > (t0 + nt - 1) * keys, what
            # tight unless the tile's rows run over from one head to the next
            if n == N and len(kept) <= N:
                assert hi <= max(b for _, b in some) + N, what


def test_runs_partition_the_line(tool):
    asks = [(t, g, m) for t in (0, 1, 2, 7, 100, 1000, 4097) for g in (1, 2, 148, 296) for m in (1, 2, 8)]
    lines = _ask(tool, "\n".join(f"r {t} {g} {m}" for t, g, m in asks))
    lines = [x for x in lines if x.strip()]
    for i, (t, g, m) in enumerate(asks):
        c = int(lines[2 * i])
        v = list(map(int, lines[2 * i + 1].split()))
        starts, of = v[:c + 1], v[c + 1:]
        assert 1 <= c <= g and c <= max(1, -(-t // m)) and starts[0] == 0 and starts[-1] == t and len(of) == t
        assert all(b - a in (t // c, t // c + 1) for a, b in zip(starts, starts[1:]))
        for x, r in enumerate(of):
            assert starts[r] <= x < starts[r + 1]
