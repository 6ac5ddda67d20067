// How the paged forward's work is cut: shared by its kernels, and compiled
// for the host by the index tests.
//
// An item is one tile of ROWS packed query rows of one (sequence, key/value
// head). The G query heads that share the head and the chunk's N tokens are
// one run of G * N rows in memory (row = g * N + token), so a tile is
// consecutive rows whatever G and N are, and grouped heads read K and V once.
// An item's cost is the number of KT-key tiles that its rows keep. The items'
// tiles form one line, cut into equal runs, one a CTA: lengths of any
// mixture, few long sequences or many short ones, load every CTA alike, and
// the host needs no lengths. A run that starts or ends inside an item leaves
// a partial result (running maximum, sum, unnormalised output) in the
// workspace; each CTA leaves at most two, one for the item it starts in and
// one for the item it ends in. The item's first CTA names it to the combine
// kernel, which joins the partials in the order of the CTAs: the result does
// not depend on timing.
// Where the table's width bounds every item to a few tiles, the line counts
// items instead (whole_items): nothing is split and no join is launched.
#pragma once

#include "paged.cuh"

namespace bsa {

// The kept keys of one tile of rows: [lo, hi) holds every key that any of its
// rows keeps, [clo, chi) the keys that all of them keep (possibly empty), t0
// and nt the key tiles over [lo, hi). nt = 0: no row of the tile is written;
// rows that are written but keep no key have one tile with lo = hi.
struct ItemSpan {
  int lo, hi, clo, chi, t0, nt;
};

__host__ __device__ __forceinline__ int clamp0(long long x, int top) {
  return x < 0 ? 0 : x > top ? top : (int)x;
}

template <int ROWS, int KT>
__host__ __device__ __forceinline__ ItemSpan item_span(const PagedParams& p, int n, int kv, int rt) {
  ItemSpan s{0, 0, 0, 0, 0, 0};
  if (n <= 0) return s;
  const int r0 = rt * ROWS;
  const long long end = (long long)r0 + ROWS;
  const int r1 = (int)(end < (long long)p.G * p.N ? end : (long long)p.G * p.N) - 1;
  const int a0 = fdiv(r0, p.f_n), a1 = fdiv(r1, p.f_n);
  const int n0 = r0 - a0 * p.N, n1 = r1 - a1 * p.N;
  // first and last written token of the tile (its rows may run over heads)
  int first = n0, last = n1 < n - 1 ? n1 : n - 1;
  if (a0 != a1) {
    first = 0;
    if (a1 > a0 + 1 || n - 1 >= n0) last = n - 1;
  }
  if (first > last) return s;
  const long long off = (long long)kv - n;  // position of the chunk's token 0
  s.hi = s.chi = kv;
  if (p.causal) {
    s.hi = clamp0(off + last + 1, kv);
    s.chi = clamp0(off + first + 1, kv);
    if (p.window > 0) {
      s.lo = clamp0(off + first - p.window + 1, kv);
      s.clo = clamp0(off + last - p.window + 1, kv);
    }
  }
  if (s.hi <= s.lo) {
    s.lo = s.hi = 0;
    s.nt = 1;
    return s;
  }
  s.t0 = s.lo / KT;
  s.nt = (s.hi - 1) / KT - s.t0 + 1;
  return s;
}

// One run: `left` tiles from tile `t` of the item (idx, hk), idx = sequence *
// row tiles + row tile, heads inside idx; `pos` is the run's start on the
// line of `total` tiles cut for `ctas` CTAs.
struct Run {
  long long total, pos;
  int ctas, idx, hk, t;
  long long left;
};

__host__ __device__ __forceinline__ long long run_start(long long total, int c, int ctas) { return total * c / ctas; }

// The CTA whose run holds tile x of the line.
__host__ __device__ __forceinline__ int run_of(long long total, long long x, int ctas) {
  return (int)(((x + 1) * ctas - 1) / total);
}

// CTAs that get a run: fewer when they would have less than `min_tiles` each.
__host__ __device__ __forceinline__ int run_ctas(long long total, int grid, int min_tiles) {
  const long long c = (total + min_tiles - 1) / min_tiles;
  return c < 1 ? 1 : c > grid ? grid : (int)c;
}

// What a CTA tells the combine kernel: the item that starts in its run and
// ends in a later one (parts = 0: there is none), and how many CTAs hold it.
struct SplitItem {
  int idx, hk, parts, pad;
};

// Partial results: slot 2c for the item CTA c starts inside of, 2c + 1 for
// the one that starts in c's run and goes on; each ROWS rows.
struct PagedWork {
  SplitItem* split;  // [ctas]
  float2* ml;        // [2 ctas][ROWS]: running maximum (log2 units), sum
  float* o;          // [2 ctas][ROWS][d], unnormalised
};

#ifdef __CUDACC__
// The CTA's run (every thread of a block of NT threads calls it, `sh` is
// scratch of 2 + NT / 32 long longs plus a Run behind a barrier). Each thread
// sums a chunk of the items, a scan places the chunks on the line, and the
// thread whose chunk holds the run's start looks it up.
// An item's length on the line.
__device__ __forceinline__ int line_tiles(const PagedParams& p, const ItemSpan& s) {
  return p.whole_items ? (s.nt > 0) : s.nt;
}

template <int ROWS, int KT, int NT, bool READ_ONLY = false>
__device__ Run find_run(const PagedParams& p, int row_tiles, int min_tiles, Run* run_sh, long long* sh) {
  constexpr int W = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int items = p.B * row_tiles;
  const int chunk = (items + NT - 1) / NT;
  const long long i0 = (long long)tid * chunk;
  const int first = (int)(i0 < items ? i0 : items), last = (int)(i0 + chunk < items ? i0 + chunk : items);
  long long sum = 0;
  for (int i = first, b = -1; i < last; ++i) {
    SeqLen s;
    if (i / row_tiles != b) b = i / row_tiles;
    s = seq_lens<READ_ONLY>(p, b);
    sum += line_tiles(p, item_span<ROWS, KT>(p, s.n, s.kv, i - b * row_tiles));
  }
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  long long before = inc - sum, all = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += sh[w];
    all += sh[w];
  }
  const long long total = all * p.Hkv;
  const int ctas = run_ctas(total, gridDim.x, p.whole_items ? 1 : min_tiles);
  const int c = blockIdx.x;
  const long long s0 = c < ctas ? run_start(total, c, ctas) : total;
  const long long s1 = c < ctas ? run_start(total, c + 1, ctas) : total;
  if (tid == 0 && s0 >= s1) *run_sh = Run{total, s0, ctas, 0, 0, 0, 0};
  long long at = before * p.Hkv;
  if (s0 < s1 && s0 >= at && s0 < at + sum * p.Hkv) {
    for (int i = first; i < last; ++i) {
      const int b = i / row_tiles;
      const SeqLen s = seq_lens<READ_ONLY>(p, b);
      const int nt = line_tiles(p, item_span<ROWS, KT>(p, s.n, s.kv, i - b * row_tiles));
      const long long w = (long long)nt * p.Hkv;
      if (s0 < at + w) {
        const long long d = s0 - at;
        *run_sh = Run{total, s0, ctas, i, (int)(d / nt), (int)(d % nt), s1 - s0};
        break;
      }
      at += w;
    }
  }
  __syncthreads();
  return *run_sh;
}

// The piece of the item under `r` that belongs to the run.
struct Piece {
  int b, rt, hk, n, kv;
  ItemSpan s;
  int t, m;  // tiles t .. t + m - 1 of the item's nt
  __device__ bool whole() const { return t == 0 && m == s.nt; }
};

// Next piece of the run; r.left > 0 on entry.
template <int ROWS, int KT, bool READ_ONLY = false>
__device__ __forceinline__ Piece next_piece(const PagedParams& p, int row_tiles, Run& r) {
  Piece q;
  for (;;) {
    q.b = r.idx / row_tiles;
    q.rt = r.idx - q.b * row_tiles;
    const SeqLen s = seq_clamped<READ_ONLY>(p, q.b);
    q.n = s.n;
    q.kv = s.kv;
    q.s = item_span<ROWS, KT>(p, s.n, s.kv, q.rt);
    if (q.s.nt > 0) break;
    ++r.idx;  // the run has tiles left, so an item with tiles follows
  }
  q.hk = r.hk;
  q.t = r.t;
  const long long rest = q.s.nt - q.t;
  q.m = p.whole_items || rest < r.left ? (int)rest : (int)r.left;
  const int step = p.whole_items ? 1 : q.m;
  r.left -= step;
  r.pos += step;
  r.t = 0;
  if (++r.hk == p.Hkv) {
    r.hk = 0;
    ++r.idx;
  }
  return q;
}

// Which rows of the whole chunk a query row keeps: [lo, hi).
__device__ __forceinline__ void row_keys(const PagedParams& p, int n, int kv, int token, int& lo, int& hi) {
  lo = 0;
  hi = kv;
  if (p.causal) {
    const long long pos = (long long)kv - n + token;
    hi = clamp0(pos + 1, kv);
    if (p.window > 0) lo = clamp0(pos - p.window + 1, kv);
  }
}
#endif

}  // namespace bsa
