// The paged forward for at most 16 packed query rows a key/value head (single
// tokens, and a few), and the kernel that joins split results.
//
// The work is reading the kept K and V once: 2 d values a token and head
// against 4 d flops a row, a few flops a byte, so HBM bounds it and the
// kernel's task is to keep copies in flight. Persistent CTAs (two an SM) each
// walk one run of the line of 64-key tiles (paged_sched.cuh); a producer warp
// keeps a ring of tiles full with TMA, a lane a copy (page tables are read by
// the lanes that need them), and groups of four warps take tiles in turn:
// warp w of a group has keys 16w .. 16w + 15 of its tiles for all rows, with a
// softmax state of its own, so the warps meet only where an item ends. The
// products are m16n8k16 warp MMAs with the keys (S^T = K Q^T) and then the
// channels (O^T = V^T P^T) as the long side, so eight rows fill them: a
// tcgen05 tile would be filled to a sixteenth, and at the rate HBM delivers
// keys (23 bytes a clock and SM) the warp MMAs are busy a fifth of the time.
// The lines are cut to equal runs, so one long sequence fills the GPU like
// many short ones.
//
// e4m3: codes become fp16 in registers (exact). K's scale multiplies the
// logit; V's, over sigma, the weight: sigma is a power of two, the largest V
// scale the warp has met of a token that is not all zeros, so the weights stay
// in fp16's range, and O carries 1 / sigma as it carries the running maximum.
// Weights are held times 2^12: what fp16 flushes of (weight times V scale) is
// below 2^-36 of the largest V scale, and 11 bits of weight round less than
// bf16's eight.
#include "paged_sched.cuh"
#include "tiles.cuh"

#include <cuda_fp16.h>

namespace bsa {

constexpr int kRowsTile = 16;     // query rows of an item
constexpr int kRowsKeys = 64;     // keys of a tile
// A run is at least this many tiles (one token, 16 heads, 437 to 20,000 keys:
// 1 gives within 2% of it, 4 is up to 7% slower).
constexpr int kRowsMinTiles = 2;
constexpr float kRowsTau = 3.f;   // the state moves when a row's maximum grows by more than 2^3
constexpr float kRowsGain = 4096.f;  // e4m3: weights (at most 2^3) are held times this in fp16

// R8: query rows in eights. NG: groups of four consumer warps.
template <int D, bool E4M3, int R8, int NG>
struct RowsCfg {
  static constexpr int WARPS = 4 * NG;
  static constexpr int THREADS = 32 * WARPS + 32;
  static constexpr int TOKEN = D * (E4M3 ? 1 : 2);         // bytes of a token's K
  static constexpr int KBYTES = kRowsKeys * TOKEN;
  static constexpr int SCALES = E4M3 ? kRowsKeys * 4 : 0;  // bytes of K's scales
  static constexpr int STAGE = 2 * KBYTES + (E4M3 ? 1024 : 0);  // K, V, scales (1024-aligned stages)
  // as many stages as two CTAs an SM have room for, at most 8. A multiple of
  // the groups: every stage then belongs to one group, which sees each of its
  // phases. With a stage passed from group to group, one could wait for a
  // phase while the other's tile is still in flight and take the phase before
  // (same parity) for it.
  static constexpr int FIT = (104 * 1024) / STAGE;
  static constexpr int STAGES = (FIT > 8 ? 8 : FIT) / NG * NG;
  static constexpr int TPR = 2;                            // 16-channel tiles of O joined a round
  static constexpr int XCH_OFF = STAGES * STAGE;
  static constexpr int ML_OFF = XCH_OFF + WARPS * TPR * R8 * 512;
  static constexpr int BAR_OFF = ML_OFF + 2 * WARPS * 8 * R8 * 4;
  static constexpr int MISC_OFF = BAR_OFF + 2 * STAGES * 8;
  static constexpr int SMEM = MISC_OFF + 16 + sizeof(Run) + 16 * 8;
  static constexpr int ALLOC = SMEM + 1024;
  static_assert(ALLOC <= 113 * 1024, "two CTAs an SM");
  static_assert(STAGES >= 2 && STAGES % NG == 0, "a stage belongs to one group");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void lds128(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 8 x 8 16-bit matrix over the warp, transposed
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool HALF>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if constexpr (HALF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two e4m3 codes as an fp16 pair, from the low and the high half of w.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  uint32_t y;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(y) : "r"(w));
  return y;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  uint32_t y;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(y) : "r"(w));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int N>
__device__ __forceinline__ void rows_bar() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

template <int D, bool E4M3, int R8, int NG>
__global__ void __launch_bounds__(RowsCfg<D, E4M3, R8, NG>::THREADS, 2)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const PagedParams p, const PagedWork wk) {
  using C = RowsCfg<D, E4M3, R8, NG>;
  constexpr int S = C::STAGES, W = C::WARPS;
  constexpr int NR = 2 * R8;  // rows a thread holds: 2t, 2t + 1 of each eight
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + S;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF);
  Run* run_sh = reinterpret_cast<Run*>(smem + C::MISC_OFF + 16);
  long long* scan_sh = reinterpret_cast<long long*>(smem + C::MISC_OFF + 16 + sizeof(Run));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;

  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the kernel before may have written what is read here
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // (the barriers are published by find_run's own block barriers)
  Run run = find_run<kRowsTile, kRowsKeys, C::THREADS>(p, 1, kRowsMinTiles, run_sh, scan_sh);

  if (warp == W) {
    // ------------------------------------------------------------- producer
    const int per = min(1 << p.page_log2, kRowsKeys);  // tokens a copy covers: a page, or a tile of a long page
    const int sub = kRowsKeys / per;
    const int kind = lane & 3, piece = lane >> 2;
    const uint32_t copy_bytes = (uint32_t)per * C::TOKEN * 2 + (E4M3 ? (uint32_t)per * 8 : 0u);
    int k = 0;
    bool ok = true;
    while (run.left > 0 && ok) {
      const Piece q = next_piece<kRowsTile, kRowsKeys>(p, 1, run);
      int j0 = (q.s.t0 + q.t) * kRowsKeys + piece * per;  // first token of this lane's copies
      auto keeps = [&](int j) { return piece < sub && j < q.s.hi && j + per > q.s.lo; };
      int next = keeps(j0) ? table_entry(p, q.b, j0) : 0;
      for (int i = 0; i < q.m; ++i, ++k, j0 += kRowsKeys) {
        const int st = k % S;
        const bool mine = keeps(j0);
        const int entry = next;  // the next tile's is on its way while this one waits for its stage
        next = i + 1 < q.m && keeps(j0 + kRowsKeys) ? table_entry(p, q.b, j0 + kRowsKeys) : 0;
        if (k >= S) ok = warp_all(mbar_wait(&empty[st], (uint32_t)(k / S - 1) & 1u, abort_flag, p.wait_limit_ns));
        if (!ok) {
          cta_fail(abort_flag, BSA_DEVERR_TIMEOUT);
          break;
        }
        if (k == p.withhold_tile) continue;  // failure-detection test: never loaded
        const uint32_t copies = __popc(__ballot_sync(0xffffffffu, mine && kind == 0));
        if (lane == 0) mbar_arrive_expect_tx(&full[st], copies * copy_bytes);
        __syncwarp();
        if (mine) {
          const int pg = checked_page(p, entry);
          uint8_t* dk = smem + st * C::STAGE;
          const int slot = j0 & ((1 << p.page_log2) - 1);
          const int z = pg * p.Hkv + q.hk;
          if constexpr (E4M3) {
            uint8_t* d = dk + (kind & 1) * C::KBYTES + piece * per * C::TOKEN;
            if (kind < 2)
              tma_load_3d(d, kind ? &tmV : &tmK, &full[st], 0, slot * D / 128, z);
            else
              bulk_load_1d(dk + 2 * C::KBYTES + (kind & 1) * C::SCALES + piece * per * 4,
                           ((kind & 1) ? p.v_scale : p.k_scale) + cache_row(p, pg, q.hk, j0), per * 4, &full[st]);
          } else {
            const int ch = kind >> 1;  // 64-channel half of a d = 128 row
            if (ch * 64 < D)
              tma_load_3d(dk + (kind & 1) * C::KBYTES + ch * kRowsKeys * 128 + piece * per * 128,
                          (kind & 1) ? &tmV : &tmK, &full[st], ch * 64, slot, z);
          }
        }
        __syncwarp();
      }
    }
    // copies in flight land before the CTA ends, whether or not it aborts:
    // consumers may give up on them after this warp is through
    if (lane == 0)
      for (int t = max(0, k - S); t < k; ++t)
        if (t != p.withhold_tile) mbar_drain(&full[t % S], (uint32_t)(t / S) & 1u);
    return;
  }

  // --------------------------------------------------------------- consumers
  const int g = lane >> 2, t4 = lane & 3, w4 = warp & 3, grp = warp >> 2;
  const uint32_t sbase = smem_u32(smem);
  // where this lane's first reads of a tile's K and V lie (128-byte swizzle:
  // 16-byte unit u of 128-byte row r sits at u ^ (r & 7)); the tile starts on
  // 1024 bytes, so the further units of a row are an XOR away
  uint32_t k_off, v_off;
  if constexpr (E4M3) {
    const uint32_t kl = (16 * w4 + g) * C::TOKEN + 16 * t4, vl = (16 * w4 + (lane & 15)) * C::TOKEN + (lane >> 4) * 16;
    k_off = kl ^ ((kl >> 3) & 0x70u);
    v_off = vl ^ ((vl >> 3) & 0x70u);
  } else {
    const uint32_t kk = 16 * w4 + (lane & 15), vk = 16 * w4 + (lane >> 4) * 8 + (lane & 7);
    k_off = kk * 128 + (((lane >> 4) ^ (kk & 7)) << 4);
    v_off = vk * 128 + ((((lane >> 3) & 1) ^ (vk & 7)) << 4);
  }
  float* sm_m = reinterpret_cast<float*>(smem + C::ML_OFF);
  float* sm_l = sm_m + W * 8 * R8;
  const int rows = p.G * p.N;
  int k = 0;  // tiles of the run before this piece
  bool ok = true;
  SplitItem split{0, 0, 0, 0};
  while (run.left > 0) {
    const long long at = run.pos;
    const Piece q = next_piece<kRowsTile, kRowsKeys>(p, 1, run);
    if (q.t == 0 && q.m < q.s.nt)
      split = SplitItem{q.b, q.hk, run_of(run.total, at + q.s.nt - 1, run.ctas) - cta + 1, 0};
    const size_t row_base = (size_t)(q.b * p.Hkv + q.hk) * rows;
    // this thread's rows of S^T and O^T: 2t, 2t + 1 of each eight
    int lo[NR], hi[NR];
    bool written[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int r = 8 * (i >> 1) + 2 * t4 + (i & 1);
      const int tok = r < rows ? r - fdiv(r, p.f_n) * p.N : 0;
      written[i] = r < rows && tok < q.n;
      row_keys(p, q.n, q.kv, tok, lo[i], hi[i]);
    }
    // Q as B fragments, row g of each eight. bf16: k-step s covers channels
    // 16 s .. 16 s + 15 in order. e4m3: fp16 after a power-of-two scale of
    // the row (exact down to 2^-17 of its largest value, an error of at most
    // 2^-25 of it below), in the order in which a lane's 16-byte reads of K
    // deliver the channels (see below).
    uint32_t qf[R8][D / 16][2];
    float zs[NR];  // row factor of the logits
#pragma unroll
    for (int e = 0; e < R8; ++e) {
      const int r = 8 * e + g;
      const int tok = r < rows ? r - fdiv(r, p.f_n) * p.N : 0;
      const bool have = r < rows && tok < q.n;
      const __nv_bfloat16* src = p.Q + (row_base + r) * D;
      if constexpr (E4M3) {
        uint2 x[D / 16];
        uint32_t top = 0u;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          x[s] = make_uint2(0u, 0u);
          if (have) x[s] = *reinterpret_cast<const uint2*>(src + 64 * (s >> 2) + 16 * t4 + 4 * (s & 3));
          const uint32_t u = __vmaxu2(x[s].x & 0x7fff7fffu, x[s].y & 0x7fff7fffu);
          top = max(top, max(u & 0xffffu, u >> 16));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e with e the exponent of the largest value, inside the normal range
        const int ex = min(max((int)(top >> 7), 1), 253);
        const float down = __int_as_float((254 - ex) << 23), up = __int_as_float(ex << 23);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          qf[e][s][0] = pack_f16x2(__uint_as_float(x[s].x << 16) * down, __uint_as_float(x[s].x & 0xffff0000u) * down);
          qf[e][s][1] = pack_f16x2(__uint_as_float(x[s].y << 16) * down, __uint_as_float(x[s].y & 0xffff0000u) * down);
        }
        // rows 2t and 2t + 1 are held by the lanes 8t and 8t + 4
        zs[2 * e] = __shfl_sync(0xffffffffu, up, 8 * t4) * p.scale_log2;
        zs[2 * e + 1] = __shfl_sync(0xffffffffu, up, 8 * t4 + 4) * p.scale_log2;
      } else {
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          qf[e][s][0] = have ? *reinterpret_cast<const uint32_t*>(src + 16 * s + 2 * t4) : 0u;
          qf[e][s][1] = have ? *reinterpret_cast<const uint32_t*>(src + 16 * s + 8 + 2 * t4) : 0u;
        }
        zs[2 * e] = zs[2 * e + 1] = p.scale_log2;
      }
    }
    float o[R8][D / 16][4];
#pragma unroll
    for (int e = 0; e < R8; ++e)
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[e][i][0] = o[e][i][1] = o[e][i][2] = o[e][i][3] = 0.f;
    float m[NR], mu[NR], l[NR];  // running maximum (log2 units), the same or 0 before there is one, sum
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      m[i] = kNegInf;
      mu[i] = l[i] = 0.f;
    }
    // e4m3: a power of two, at least every finite V scale of a token with values so far, and gain / sigma
    float sigma = 0x1p-112f, rs = kRowsGain / 0x1p-112f;

    // the group's tiles: every NG-th of the run
    for (int it = (grp + NG - k % NG) % NG; ok && it < q.m; it += NG) {
      const int st = (k + it) % S;
      const int key0 = (q.s.t0 + q.t + it) * kRowsKeys;
      const bool edge = key0 < q.s.clo || key0 + kRowsKeys > q.s.chi;
      ok = warp_all(mbar_wait(&full[st], (uint32_t)((k + it) / S) & 1u, abort_flag, p.wait_limit_ns));
      if (!ok) {
        // every warp sees the flag in its next wait; all go on to the same
        // block barriers, so none is left behind in one (the output is void).
        // This warp takes no further tile: an arrival out of turn would let
        // the producer load over a copy in flight
        cta_fail(abort_flag, BSA_DEVERR_TIMEOUT);
        break;
      }
      const uint32_t kb = sbase + st * C::STAGE, vb = kb + C::KBYTES;
      // S^T[16 keys][rows]
      float s2[R8][4];
#pragma unroll
      for (int e = 0; e < R8; ++e) s2[e][0] = s2[e][1] = s2[e][2] = s2[e][3] = 0.f;
      const float* scl = reinterpret_cast<const float*>(smem + st * C::STAGE + 2 * C::KBYTES) + 16 * w4 + g;
      if constexpr (E4M3) {
        // lane (key g, t) reads bytes 16 t .. 16 t + 15 of each 64-byte half:
        // word s of it holds the four channels of k-step s
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          uint32_t x[4], y[4];
          lds128(x, (kb + k_off) ^ (64 * h));
          lds128(y, D == 64 ? (kb + k_off + 512) ^ 64 : (kb + k_off + 1024) ^ (64 * h));
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const uint32_t a0 = codes_lo(x[s]), a1 = codes_lo(y[s]), a2 = codes_hi(x[s]), a3 = codes_hi(y[s]);
#pragma unroll
            for (int e = 0; e < R8; ++e) mma16<true>(s2[e], a0, a1, a2, a3, qf[e][4 * h + s][0], qf[e][4 * h + s][1]);
          }
        }
        const float k0 = scl[0], k1 = scl[8];
#pragma unroll
        for (int e = 0; e < R8; ++e) {
          s2[e][0] *= k0;
          s2[e][1] *= k0;
          s2[e][2] *= k1;
          s2[e][3] *= k1;
        }
      } else {
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          uint32_t x[4];
          ldsm4(x, (kb + (s >> 2) * kRowsKeys * 128 + k_off) ^ (32 * (s & 3)));
#pragma unroll
          for (int e = 0; e < R8; ++e) mma16<false>(s2[e], x[0], x[1], x[2], x[3], qf[e][s][0], qf[e][s][1]);
        }
      }
      const int j0 = key0 + 16 * w4 + g;  // this thread's keys: j0 and j0 + 8
      if (edge) {
#pragma unroll
        for (int e = 0; e < R8; ++e)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int j = j0 + 8 * (c >> 1), i = 2 * e + (c & 1);
            if (j < lo[i] || j >= hi[i]) s2[e][c] = kNegInf;
          }
      }
      // online softmax; the state moves only when a row's maximum grows by
      // more than 2^kRowsTau (or a V scale passes sigma), which a vote finds
      // without the maximum itself
      bool over = false;
#pragma unroll
      for (int i = 0; i < NR; ++i)
        over |= fmaxf(s2[i >> 1][i & 1], s2[i >> 1][2 + (i & 1)]) * zs[i] > m[i] + kRowsTau;
      float v0 = 0.f, v1 = 0.f;
      if constexpr (E4M3) {
        v0 = scl[C::SCALES / 4];
        v1 = scl[C::SCALES / 4 + 8];
        if (edge) {  // scales of keys no row keeps may be anything
          v0 = j0 >= q.s.lo && j0 < q.s.hi ? v0 : 0.f;
          v1 = j0 + 8 >= q.s.lo && j0 + 8 < q.s.hi ? v1 : 0.f;
        }
        over |= fmaxf(v0, v1) > sigma;
      }
      if (__any_sync(0xffffffffu, over)) {
        float alpha[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          float x = fmaxf(s2[i >> 1][i & 1], s2[i >> 1][2 + (i & 1)]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x *= zs[i];
          alpha[i] = 1.f;
          if (x > m[i] + kRowsTau) {
            alpha[i] = fast_exp2(m[i] - x);
            m[i] = x;
          }
          l[i] *= alpha[i];
        }
        if constexpr (E4M3) {
          // A token of zeros adds nothing whatever its scale (1, as it is
          // written): it must not move sigma, above which V's weights would
          // sink into fp16's subnormals, and its own weight must stay finite.
          // Four lanes read a key's codes; only scales above sigma need it.
          if (__any_sync(0xffffffffu, fmaxf(v0, v1) > sigma)) {
            const uint32_t lin = (16 * w4 + g) * D + t4 * (D / 4);
            const uint32_t at = vb + (lin ^ ((lin >> 3) & 0x70u));
            uint32_t z0 = 0u, z1 = 0u;
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
              uint32_t x[4], y[4];
              lds128(x, at ^ (16 * h));
              lds128(y, D == 64 ? (at + 512) ^ 64 : (at + 1024) ^ (16 * h));
              z0 |= x[0] | x[1] | x[2] | x[3];
              z1 |= y[0] | y[1] | y[2] | y[3];
            }
            z0 |= __shfl_xor_sync(0xffffffffu, z0, 1);
            z1 |= __shfl_xor_sync(0xffffffffu, z1, 1);
            z0 |= __shfl_xor_sync(0xffffffffu, z0, 2);
            z1 |= __shfl_xor_sync(0xffffffffu, z1, 2);
            if (v0 > sigma && (z0 & 0x7f7f7f7fu) == 0u) v0 = 0.f;
            if (v1 > sigma && (z1 & 0x7f7f7f7fu) == 0u) v1 = 0.f;
          }
          // the largest finite scale of the warp's keys, as bits
          const uint32_t b0 = __float_as_uint(v0), b1 = __float_as_uint(v1);
          const uint32_t top =
              __reduce_max_sync(0xffffffffu, max(b0 < 0x7f800000u ? b0 : 0u, b1 < 0x7f800000u ? b1 : 0u));
          if (top > __float_as_uint(sigma)) {
            const float up = __uint_as_float(min((top + 0x7fffffu) & 0x7f800000u, 0x7f000000u));
            const float beta = sigma / up;
            sigma = up;
            rs = kRowsGain / sigma;
#pragma unroll
            for (int i = 0; i < NR; ++i) alpha[i] *= beta;
          }
        }
#pragma unroll
        for (int e = 0; e < R8; ++e)
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[e][i][0] *= alpha[2 * e];
            o[e][i][1] *= alpha[2 * e + 1];
            o[e][i][2] *= alpha[2 * e];
            o[e][i][3] *= alpha[2 * e + 1];
          }
#pragma unroll
        for (int i = 0; i < NR; ++i) mu[i] = m[i] == kNegInf ? 0.f : m[i];
      }
      uint32_t pf[R8][2];
#pragma unroll
      for (int e = 0; e < R8; ++e) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int i = 2 * e + (c & 1);
          s2[e][c] = fast_exp2(fmaf(s2[e][c], zs[i], -mu[i]));
          l[i] += s2[e][c];
        }
        if constexpr (E4M3) {
          const float f0 = v0 * rs, f1 = v1 * rs;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float x = s2[e][c] * (c < 2 ? f0 : f1);
            // a masked key adds nothing, whatever its scale
            s2[e][c] = edge && s2[e][c] == 0.f ? 0.f : x;
          }
          pf[e][0] = movm(pack_f16x2(s2[e][0], s2[e][1]));
          pf[e][1] = movm(pack_f16x2(s2[e][2], s2[e][3]));
        } else {
          pf[e][0] = movm(pack_bf16x2(s2[e][0], s2[e][1]));
          pf[e][1] = movm(pack_bf16x2(s2[e][2], s2[e][3]));
        }
      }
      uint32_t vm[2] = {0xffffffffu, 0xffffffffu};  // V of keys no row keeps reads as zero
      if (edge) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int j = key0 + 16 * w4 + 8 * h + 2 * t4;
          if (j < q.s.lo || j >= q.s.hi) vm[h] &= 0xffff0000u;
          if (j + 1 < q.s.lo || j + 1 >= q.s.hi) vm[h] &= 0x0000ffffu;
        }
      }
      // O^T += V^T P^T: matrices of eight keys x 16 bytes, transposed on the way in
      if constexpr (E4M3) {
        // 16-bit columns are channel pairs: channel 2g of a 16-byte unit is
        // row g of the tile, channel 2g + 1 row g + 8
#pragma unroll
        for (int h = 0; h < D / 32; ++h) {
          uint32_t x[4];
          ldsm4t(x, (vb + v_off) ^ (32 * h));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t y = __byte_perm(x[2 * u], 0u, 0x3120), z = __byte_perm(x[2 * u + 1], 0u, 0x3120);
            uint32_t a0 = codes_lo(y), a1 = codes_hi(y), a2 = codes_lo(z), a3 = codes_hi(z);
            if (edge) {
              a0 &= vm[0];
              a1 &= vm[0];
              a2 &= vm[1];
              a3 &= vm[1];
            }
#pragma unroll
            for (int e = 0; e < R8; ++e) mma16<true>(o[e][2 * h + u], a0, a1, a2, a3, pf[e][0], pf[e][1]);
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < D / 16; ++h) {
          uint32_t x[4];
          ldsm4t(x, (vb + (h >> 2) * kRowsKeys * 128 + v_off) ^ (32 * (h & 3)));
          if (edge) {
            x[0] &= vm[0];
            x[1] &= vm[0];
            x[2] &= vm[1];
            x[3] &= vm[1];
          }
#pragma unroll
          for (int e = 0; e < R8; ++e) mma16<false>(o[e][h], x[0], x[1], x[2], x[3], pf[e][0], pf[e][1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    k += q.m;

    // ------------------------------------------------ join the warps
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 4);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 8);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 16);
      if (g == 0) {
        const int at8 = warp * 8 * R8 + 8 * (i >> 1) + 2 * t4 + (i & 1);
        sm_m[at8] = m[i];
        sm_l[at8] = l[i];
      }
    }
    rows_bar<32 * W>();
    float M[NR], L[NR], sc[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int at8 = 8 * (i >> 1) + 2 * t4 + (i & 1);
      M[i] = kNegInf;
      L[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) M[i] = fmaxf(M[i], sm_m[w * 8 * R8 + at8]);
      const float mu = M[i] == kNegInf ? 0.f : M[i];
#pragma unroll
      for (int w = 0; w < W; ++w) L[i] += sm_l[w * 8 * R8 + at8] * fast_exp2(sm_m[w * 8 * R8 + at8] - mu);
      sc[i] = fast_exp2(m[i] - mu);
      if constexpr (E4M3) sc[i] *= sigma * (1.f / kRowsGain);
    }
    // TPR of O's tiles a round; warp w of the round's tiles sums and stores tile w
    const bool whole = q.whole();
    const size_t slot = 2 * (size_t)cta + (q.t == 0 ? 1 : 0);
    float4* slots = reinterpret_cast<float4*>(smem + C::XCH_OFF);
#pragma unroll
    for (int rd = 0; rd < D / 16 / C::TPR; ++rd) {
#pragma unroll
      for (int u = 0; u < C::TPR; ++u)
#pragma unroll
        for (int e = 0; e < R8; ++e) {
          const float(&x)[4] = o[e][rd * C::TPR + u];
          slots[((warp * C::TPR + u) * R8 + e) * 32 + lane] =
              make_float4(x[0] * sc[2 * e], x[1] * sc[2 * e + 1], x[2] * sc[2 * e], x[3] * sc[2 * e + 1]);
        }
      rows_bar<32 * W>();
      // (tile u, eight e) of the round by one warp
      if (warp < C::TPR * R8) {
        const int u = warp / R8, e = warp % R8;
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float4 x = slots[((w * C::TPR + u) * R8 + e) * 32 + lane];
          acc[0] += x.x;
          acc[1] += x.y;
          acc[2] += x.z;
          acc[3] += x.w;
        }
        const int t16 = rd * C::TPR + u;
        const int d0 = 16 * t16 + (E4M3 ? 2 * g : g), d1 = d0 + (E4M3 ? 1 : 8);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = 8 * e + 2 * t4 + c;
          // this row's sums are held under index 2 e + c
          float Lr = L[c], Mr = M[c];
          bool wr = written[c];
          if (R8 == 2 && e == 1) {
            Lr = L[NR - 2 + c];
            Mr = M[NR - 2 + c];
            wr = written[NR - 2 + c];
          }
          if (!wr) continue;
          if (whole) {
            const float inv = Lr > 0.f ? 1.f / Lr : Lr == 0.f ? 0.f : Lr;
            __nv_bfloat16* dst = p.O + (row_base + r) * D;
            if constexpr (E4M3) {
              *reinterpret_cast<uint32_t*>(dst + d0) = pack_bf16x2(acc[c] * inv, acc[2 + c] * inv);
            } else {
              dst[d0] = __float2bfloat16(acc[c] * inv);
              dst[d1] = __float2bfloat16(acc[2 + c] * inv);
            }
          } else {
            float* dst = wk.o + (slot * kRowsTile + r) * D;
            dst[d0] = acc[c];
            dst[d1] = acc[2 + c];
            if (rd == 0 && u == 0 && g == 0) wk.ml[slot * kRowsTile + r] = make_float2(Mr, Lr);
          }
        }
      }
      rows_bar<32 * W>();
    }
  }
  if (tid == 0) wk.split[cta] = split;
}

// Joins the partial results of split items, in the order of the CTAs that
// left them: grid (CTAs of the forward, y); block (c, y) takes rows y, y +
// gridDim.y, ... of the item that starts in CTA c's run and ends in another's.
// The warps share an item's parts, lanes its channels.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedParams p, const PagedWork wk, int row_tiles) {
  constexpr int V = D / 32;
  __shared__ float acc_sh[8][D];
  __shared__ float l_sh[8];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const SplitItem it = wk.split[blockIdx.x];
  if (it.parts <= 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = it.idx / row_tiles, rt = it.idx - b * row_tiles;
  const int rows = min(ROWS, p.G * p.N - rt * ROWS);
  const SeqLen s = seq_clamped(p, b);
  // part i: slot 2c + 1 of the first CTA, slot 2 (c + i) of the others
  auto slot = [&](int i) -> size_t { return i == 0 ? 2 * (size_t)blockIdx.x + 1 : 2 * ((size_t)blockIdx.x + i); };
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    const int R = rt * ROWS + r;
    if (R - fdiv(R, p.f_n) * p.N >= s.n) continue;  // padding (uniform over the block)
    float M = kNegInf;
    for (int i = lane; i < it.parts; i += 32) M = fmaxf(M, wk.ml[slot(i) * ROWS + r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float mu = M == kNegInf ? 0.f : M;
    float acc[V], l = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
#pragma unroll 4
    for (int i = warp; i < it.parts; i += 8) {
      const size_t at = slot(i) * ROWS + r;
      const float2 ml = wk.ml[at];
      const float w = fast_exp2(ml.x - mu);
      l += ml.y * w;
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] += wk.o[at * D + c * 32 + lane] * w;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < V; ++c) acc_sh[warp][c * 32 + lane] = acc[c];
    if (lane == 0) l_sh[warp] = l;
    __syncthreads();
    if (threadIdx.x < D) {
      float x = 0.f, L = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        x += acc_sh[w][threadIdx.x];
        L += l_sh[w];
      }
      const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;
      p.O[((size_t)(b * p.Hkv + it.hk) * p.G * p.N + R) * D + threadIdx.x] = __float2bfloat16(x * inv);
    }
  }
}

template <int D, bool E4M3, int R8, int NG>
static cudaError_t launch_rows_d(const CUtensorMap& k, const CUtensorMap& v, const PagedParams& p, const PagedWork& w,
                                 int grid, cudaStream_t stream) {
  using C = RowsCfg<D, E4M3, R8, NG>;
  auto fn = paged_rows_kernel<D, E4M3, R8, NG>;
  static DeviceOnce once;
  cudaError_t e = once.run(
      [&]() -> cudaError_t { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::ALLOC); });
  if (e != cudaSuccess) return e;
  if ((e = launch_after(fn, dim3(grid), C::THREADS, C::ALLOC, stream, k, v, p, w)) != cudaSuccess) return e;
  if (p.whole_items) return cudaSuccess;
  const int rows = p.G * p.N;
  return launch_after(paged_join_kernel<D, kRowsTile>, dim3(grid, min(rows, 8)), 256, 0, stream, p, w, 1);
}

template <int D, bool E4M3>
static cudaError_t launch_rows_any(const CUtensorMap& k, const CUtensorMap& v, const PagedParams& p,
                                   const PagedWork& w, int grid, cudaStream_t stream) {
  // Up to eight rows leave the registers for a second group of warps, which
  // the conversion of e4m3 codes needs; bf16 at d = 128 has three stages' room
  // and one group keeps up with HBM.
  constexpr int NG = E4M3 || D == 64 ? 2 : 1;
  if (p.G * p.N <= 8) return launch_rows_d<D, E4M3, 1, NG>(k, v, p, w, grid, stream);
  return launch_rows_d<D, E4M3, 2, 1>(k, v, p, w, grid, stream);
}

cudaError_t launch_paged_rows(const CUtensorMap& k, const CUtensorMap& v, const PagedParams& p, const PagedWork& w,
                              int grid, cudaStream_t stream) {
  if (p.d == 64)
    return p.e4m3 ? launch_rows_any<64, true>(k, v, p, w, grid, stream)
                  : launch_rows_any<64, false>(k, v, p, w, grid, stream);
  return p.e4m3 ? launch_rows_any<128, true>(k, v, p, w, grid, stream)
                : launch_rows_any<128, false>(k, v, p, w, grid, stream);
}

}  // namespace bsa
