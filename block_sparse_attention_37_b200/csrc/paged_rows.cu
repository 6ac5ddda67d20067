// The paged forward for at most 16 packed query rows a key/value head (single
// tokens, and a few), and the kernel that joins split results.
//
// The work is reading the kept K and V once: 2 d values a token and head
// against 4 d flops a row, a few flops a byte, so HBM bounds it and the
// kernel's task is to keep copies in flight. Persistent CTAs (two an SM) each
// walk one run of the line of 64-key tiles (paged_sched.cuh); a producer warp
// keeps a ring of tiles full with TMA, a lane a copy (page tables are read by
// the lanes that need them), and four warps consume: warp w takes keys 16w ..
// 16w + 15 of every tile for all rows, with a softmax state of its own, so
// the warps meet only where an item ends. The products are m16n8k16 warp
// MMAs: with 16 rows a tcgen05 tile would be filled to an eighth, and at the
// rate HBM delivers keys (23 bytes a clock and SM) the warp MMAs are busy a
// fifth of the time. The lines are cut to equal runs, so one long sequence
// fills the GPU like many short ones.
//
// e4m3: codes become bf16 in registers (exact). K's scale multiplies the
// logit, V's the weight before its rounding to bf16, so neither adds an error.
#include "paged_sched.cuh"
#include "tiles.cuh"

namespace bsa {

constexpr int kRowsTile = 16;    // query rows of an item
constexpr int kRowsKeys = 64;    // keys of a tile
constexpr int kRowsThreads = 160;
constexpr int kRowsMinTiles = 2;  // a run is at least this many tiles

template <int D, bool E4M3>
struct RowsCfg {
  static constexpr int TOKEN = D * (E4M3 ? 1 : 2);         // bytes of a token's K
  static constexpr int KBYTES = kRowsKeys * TOKEN;
  static constexpr int SCALES = E4M3 ? kRowsKeys * 4 : 0;  // bytes of K's scales
  static constexpr int STAGE = 2 * KBYTES + (E4M3 ? 1024 : 0);  // K, V, scales (1024-aligned stages)
  // as many stages as two CTAs an SM have room for, at most 8
  static constexpr int FIT = (100 * 1024) / STAGE;
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int XCH_OFF = STAGES * STAGE;           // exchange of the warps' outputs: a quarter each
  static constexpr int ML_OFF = XCH_OFF + kRowsTile * D * 4;
  static constexpr int BAR_OFF = ML_OFF + 2 * 4 * kRowsTile * 4;
  static constexpr int MISC_OFF = BAR_OFF + 2 * STAGES * 8;
  static constexpr int SMEM = MISC_OFF + 16 + sizeof(Run) + 8 * 8;
  static constexpr int ALLOC = SMEM + 1024;
};
static_assert(RowsCfg<128, false>::ALLOC <= 113 * 1024 && RowsCfg<64, false>::ALLOC <= 113 * 1024 &&
                  RowsCfg<128, true>::ALLOC <= 113 * 1024 && RowsCfg<64, true>::ALLOC <= 113 * 1024,
              "two CTAs an SM");

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
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bits(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }
// Bytes 0 and 2, and bytes 1 and 3, of four codes as bf16 pairs.
__device__ __forceinline__ uint32_t codes_even(uint32_t w) { return bits(e4m3_pair(w << 8, w << 4)); }
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) { return bits(e4m3_pair(w, w >> 4)); }

__device__ __forceinline__ void rows_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int D, bool E4M3>
__global__ void __launch_bounds__(kRowsThreads, 2)
    paged_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                      const PagedParams p, const PagedWork wk) {
  using C = RowsCfg<D, E4M3>;
  constexpr int S = C::STAGES;
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
  Run run = find_run<kRowsTile, kRowsKeys, kRowsThreads>(p, 1, kRowsMinTiles, run_sh, scan_sh);

  if (warp == 4) {
    // ------------------------------------------------------------- producer
    const int per = min(1 << p.page_log2, kRowsKeys);  // tokens a copy covers: a page, or a tile of a long page
    const int sub = kRowsKeys / per;
    const int kind = lane & 3, piece = lane >> 2;
    const uint32_t copy_bytes = (uint32_t)per * C::TOKEN * 2 + (E4M3 ? (uint32_t)per * 8 : 0u);
    int k = 0;
    bool ok = true;
    while (run.left > 0 && ok) {
      const Piece q = next_piece<kRowsTile, kRowsKeys>(p, 1, run);
      for (int i = 0; i < q.m; ++i, ++k) {
        const int st = k % S;
        const int key0 = (q.s.t0 + q.t + i) * kRowsKeys;
        const int j0 = key0 + piece * per;
        const bool mine = piece < sub && j0 < q.s.hi && j0 + per > q.s.lo;
        int pg = 0;
        if (mine) pg = max(page_of(p, q.b, j0), 0);
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
    // copies in flight land before the CTA ends (an aborting CTA's consumers may not wait for them)
    if (*abort_flag && lane == 0)
      for (int t = max(0, k - S); t < k; ++t)
        if (t != p.withhold_tile) mbar_drain(&full[t % S], (uint32_t)(t / S) & 1u);
    return;
  }

  // --------------------------------------------------------------- consumers
  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t sbase = smem_u32(smem);
  float* xch = reinterpret_cast<float*>(smem + C::XCH_OFF);
  float* sm_m = reinterpret_cast<float*>(smem + C::ML_OFF);
  float* sm_l = sm_m + 4 * kRowsTile;
  const int rows = p.G * p.N;
  int k = 0;
  SplitItem split{0, 0, 0, 0};
  while (run.left > 0) {
    const long long at = run.pos;
    const Piece q = next_piece<kRowsTile, kRowsKeys>(p, 1, run);
    if (q.t == 0 && q.m < q.s.nt)
      split = SplitItem{q.b, q.hk, run_of(run.total, at + q.s.nt - 1, run.ctas) - cta + 1, 0};
    // the rows of this thread: g and g + 8
    const size_t row_base = (size_t)(q.b * p.Hkv + q.hk) * rows;
    int lo[2], hi[2];
    bool written[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      const int tok = r < rows ? r - fdiv(r, p.f_n) * p.N : 0;
      written[i] = r < rows && tok < q.n;
      row_keys(p, q.n, q.kv, tok, lo[i], hi[i]);
    }
    // Q as A fragments. bf16: k-step s covers channels 16 s .. 16 s + 15 in
    // order. e4m3: the order of the channels inside the steps is the one in
    // which a lane's 16-byte reads of K deliver them (see below); a dot
    // product does not mind.
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __nv_bfloat16* src = p.Q + (row_base + g + 8 * i) * D;
        if constexpr (E4M3) {
          uint2 x = make_uint2(0u, 0u);
          if (written[i]) x = __ldg(reinterpret_cast<const uint2*>(src + 64 * (s >> 2) + 16 * t4 + 4 * (s & 3)));
          qf[s][i] = __byte_perm(x.x, x.y, 0x5410);
          qf[s][2 + i] = __byte_perm(x.x, x.y, 0x7632);
        } else {
          qf[s][i] = written[i] ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * s + 2 * t4)) : 0u;
          qf[s][2 + i] = written[i] ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * s + 8 + 2 * t4)) : 0u;
        }
      }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};

    for (int it = 0; it < q.m; ++it, ++k) {
      const int st = k % S;
      const int key0 = (q.s.t0 + q.t + it) * kRowsKeys;
      const bool edge = key0 < q.s.clo || key0 + kRowsKeys > q.s.chi;
      if (!warp_all(mbar_wait(&full[st], (uint32_t)(k / S) & 1u, abort_flag, p.wait_limit_ns))) {
        // every warp sees the flag in its next wait; all go on to the same
        // block barriers, so none is left behind in one (the output is void)
        cta_fail(abort_flag, BSA_DEVERR_TIMEOUT);
        k += q.m - it;
        break;
      }
      const uint32_t kb = sbase + st * C::STAGE, vb = kb + C::KBYTES;
      // S[16 rows][16 keys]: two n-tiles of eight keys
      float s2[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        s2[nt][0] = s2[nt][1] = s2[nt][2] = s2[nt][3] = 0.f;
        if constexpr (E4M3) {
          // lane (key g, t) reads bytes 16 t .. 16 t + 15 of each 64-byte half:
          // word s of it is k-step s's four values, even bytes then odd bytes
          const int key = 16 * warp + 8 * nt + g;
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            const uint32_t lin = key * C::TOKEN + 64 * h + 16 * t4;
            uint32_t x[4];
            lds128(x, kb + (lin ^ ((lin >> 3) & 0x70u)));
#pragma unroll
            for (int s = 0; s < 4; ++s) mma16(s2[nt], qf[4 * h + s], codes_even(x[s]), codes_odd(x[s]));
          }
          const float2 sk =
              *reinterpret_cast<const float2*>(smem + st * C::STAGE + 2 * C::KBYTES + (16 * warp + 8 * nt + 2 * t4) * 4);
          s2[nt][0] *= sk.x;
          s2[nt][1] *= sk.y;
          s2[nt][2] *= sk.x;
          s2[nt][3] *= sk.y;
        } else {
          const int key = 16 * warp + 8 * nt + (lane & 7);
#pragma unroll
          for (int h = 0; h < D / 32; ++h) {
            const int u = 4 * h + (lane >> 3);  // 16-byte unit of the row
            uint32_t x[4];
            ldsm4(x, kb + (u >> 3) * kRowsKeys * 128 + key * 128 + (((u ^ key) & 7) << 4));
            mma16(s2[nt], qf[2 * h], x[0], x[1]);
            mma16(s2[nt], qf[2 * h + 1], x[2], x[3]);
          }
        }
      }
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int j = key0 + 16 * warp + 8 * nt + 2 * t4 + (c & 1);
            if (j < lo[c >> 1] || j >= hi[c >> 1]) s2[nt][c] = kNegInf;
          }
      }
      // online softmax; the state moves only when a row's maximum grows by
      // more than 2^8 (weights then reach 2^8, within bf16's range)
      bool moved = false;
      float mu[2];
      float alpha[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = fmaxf(fmaxf(s2[0][2 * i], s2[0][2 * i + 1]), fmaxf(s2[1][2 * i], s2[1][2 * i + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        x *= p.scale_log2;
        alpha[i] = 1.f;
        if (x > m[i] + 8.f) {
          alpha[i] = fast_exp2(m[i] - x);
          m[i] = x;
          moved = true;
        }
        mu[i] = m[i] == kNegInf ? 0.f : m[i];
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= alpha[0];
          o[i][1] *= alpha[0];
          o[i][2] *= alpha[1];
          o[i][3] *= alpha[1];
        }
        l[0] *= alpha[0];
        l[1] *= alpha[1];
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          s2[nt][c] = fast_exp2(fmaf(s2[nt][c], p.scale_log2, -mu[c >> 1]));
          l[c >> 1] += s2[nt][c];
        }
      uint32_t vm[2] = {0xffffffffu, 0xffffffffu};  // V of keys no row keeps reads as zero
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int j = key0 + 16 * warp + 8 * nt + 2 * t4;
          if (j < q.s.lo || j >= q.s.hi) vm[nt] &= 0xffff0000u;
          if (j + 1 < q.s.lo || j + 1 >= q.s.hi) vm[nt] &= 0x0000ffffu;
        }
      }
      if constexpr (E4M3) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          float2 sv = *reinterpret_cast<const float2*>(smem + st * C::STAGE + 2 * C::KBYTES + C::SCALES +
                                                       (16 * warp + 8 * nt + 2 * t4) * 4);
          if (edge) {
            if (!(vm[nt] & 0xffffu)) sv.x = 0.f;
            if (!(vm[nt] >> 16)) sv.y = 0.f;
          }
          s2[nt][0] *= sv.x;
          s2[nt][1] *= sv.y;
          s2[nt][2] *= sv.x;
          s2[nt][3] *= sv.y;
        }
      }
      const uint32_t pf[4] = {pack_bf16x2(s2[0][0], s2[0][1]), pack_bf16x2(s2[0][2], s2[0][3]),
                              pack_bf16x2(s2[1][0], s2[1][1]), pack_bf16x2(s2[1][2], s2[1][3])};
      // O += P V: matrices of eight keys x 16 bytes, transposed on the way in
      const int vkey = 16 * warp + (lane & 15);
#pragma unroll
      for (int h = 0; h < C::TOKEN / 32; ++h) {
        const int u = 2 * h + (lane >> 4);
        uint32_t x[4];
        if constexpr (E4M3) {
          // 16-bit columns are channel pairs: even channels make one n-tile, odd ones the next
          const uint32_t lin = vkey * C::TOKEN + u * 16;
          ldsm4t(x, vb + (lin ^ ((lin >> 3) & 0x70u)));
          mma16(o[4 * h], pf, codes_even(x[0]), codes_even(x[1]));
          mma16(o[4 * h + 1], pf, codes_odd(x[0]), codes_odd(x[1]));
          mma16(o[4 * h + 2], pf, codes_even(x[2]), codes_even(x[3]));
          mma16(o[4 * h + 3], pf, codes_odd(x[2]), codes_odd(x[3]));
        } else {
          ldsm4t(x, vb + (u >> 3) * kRowsKeys * 128 + vkey * 128 + (((u ^ vkey) & 7) << 4));
          if (edge) {
            x[0] &= vm[0];
            x[1] &= vm[1];
            x[2] &= vm[0];
            x[3] &= vm[1];
          }
          mma16(o[2 * h], pf, x[0], x[1]);
          mma16(o[2 * h + 1], pf, x[2], x[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }

    // ------------------------------------------------ join the four warps
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (t4 == 0) {
        sm_m[warp * kRowsTile + g + 8 * i] = m[i];
        sm_l[warp * kRowsTile + g + 8 * i] = l[i];
      }
    }
    rows_bar();
    float M[2], L[2], sc[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      M[i] = kNegInf;
      L[i] = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) M[i] = fmaxf(M[i], sm_m[w * kRowsTile + g + 8 * i]);
      const float mu = M[i] == kNegInf ? 0.f : M[i];
#pragma unroll
      for (int w = 0; w < 4; ++w)
        L[i] += sm_l[w * kRowsTile + g + 8 * i] * fast_exp2(sm_m[w * kRowsTile + g + 8 * i] - mu);
      sc[i] = fast_exp2(m[i] - mu);
    }
    // each warp ends with a quarter of the channels, summed over the warps
    constexpr int QT = D / 32;  // n-tiles a quarter
    float own[QT][4];
    float4* slots = reinterpret_cast<float4*>(xch);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
#pragma unroll
      for (int i = 0; i < QT; ++i)
        slots[(warp * QT + i) * 32 + lane] = make_float4(o[w * QT + i][0] * sc[0], o[w * QT + i][1] * sc[0],
                                                         o[w * QT + i][2] * sc[1], o[w * QT + i][3] * sc[1]);
      rows_bar();
      if (w == warp)
#pragma unroll
        for (int i = 0; i < QT; ++i) {
          const float4 x0 = slots[i * 32 + lane], x1 = slots[(QT + i) * 32 + lane];
          const float4 x2 = slots[(2 * QT + i) * 32 + lane], x3 = slots[(3 * QT + i) * 32 + lane];
          own[i][0] = (x0.x + x1.x) + (x2.x + x3.x);
          own[i][1] = (x0.y + x1.y) + (x2.y + x3.y);
          own[i][2] = (x0.z + x1.z) + (x2.z + x3.z);
          own[i][3] = (x0.w + x1.w) + (x2.w + x3.w);
        }
      rows_bar();
    }
    const bool whole = q.whole();
    const size_t slot = 2 * (size_t)cta + (q.t == 0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!written[i]) continue;
      const int r = g + 8 * i;
      const float inv = !whole ? 1.f : L[i] > 0.f ? 1.f / L[i] : L[i] == 0.f ? 0.f : L[i];
      float* po = wk.o + (slot * kRowsTile + r) * D;
      __nv_bfloat16* oo = p.O + (row_base + r) * D;
      if constexpr (E4M3) {
#pragma unroll
        for (int h = 0; h < QT / 2; ++h) {
          const int d = 16 * (warp * QT / 2 + h) + 4 * t4;
          const float4 x = make_float4(own[2 * h][2 * i] * inv, own[2 * h + 1][2 * i] * inv,
                                       own[2 * h][2 * i + 1] * inv, own[2 * h + 1][2 * i + 1] * inv);
          if (whole)
            *reinterpret_cast<uint2*>(oo + d) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
          else
            *reinterpret_cast<float4*>(po + d) = x;
        }
      } else {
#pragma unroll
        for (int h = 0; h < QT; ++h) {
          const int d = 8 * (warp * QT + h) + 2 * t4;
          const float a = own[h][2 * i] * inv, b = own[h][2 * i + 1] * inv;
          if (whole)
            *reinterpret_cast<uint32_t*>(oo + d) = pack_bf16x2(a, b);
          else
            *reinterpret_cast<float2*>(po + d) = make_float2(a, b);
        }
      }
      if (!whole && warp == 0 && t4 == 0) wk.ml[slot * kRowsTile + r] = make_float2(M[i], L[i]);
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const SplitItem it = wk.split[blockIdx.x];
  if (it.parts <= 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = it.idx / row_tiles, rt = it.idx - b * row_tiles;
  const int rows = min(ROWS, p.G * p.N - rt * ROWS);
  const SeqLen s = clamp_lens(p, p.n_new ? __ldg(p.n_new + b) : p.N, __ldg(p.kv_len + b));
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

template <class K, class... A>
static cudaError_t launch_after(K kernel, dim3 grid, unsigned block, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, bool E4M3>
static cudaError_t launch_rows_d(const CUtensorMap& k, const CUtensorMap& v, const PagedParams& p, const PagedWork& w,
                                 int grid, cudaStream_t stream) {
  using C = RowsCfg<D, E4M3>;
  auto fn = paged_rows_kernel<D, E4M3>;
  static DeviceOnce once;
  cudaError_t e = once.run(
      [&]() -> cudaError_t { return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::ALLOC); });
  if (e != cudaSuccess) return e;
  fn<<<grid, kRowsThreads, C::ALLOC, stream>>>(k, v, p, w);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int rows = p.G * p.N;
  return launch_after(paged_join_kernel<D, kRowsTile>, dim3(grid, min(rows, 8)), 256, stream, p, w, 1);
}

cudaError_t launch_paged_rows(const CUtensorMap& k, const CUtensorMap& v, const PagedParams& p, const PagedWork& w,
                              int grid, cudaStream_t stream) {
  if (p.d == 64)
    return p.e4m3 ? launch_rows_d<64, true>(k, v, p, w, grid, stream)
                  : launch_rows_d<64, false>(k, v, p, w, grid, stream);
  return p.e4m3 ? launch_rows_d<128, true>(k, v, p, w, grid, stream)
                : launch_rows_d<128, false>(k, v, p, w, grid, stream);
}

}  // namespace bsa
