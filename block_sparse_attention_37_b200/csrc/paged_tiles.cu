// The paged forward for more than 16 packed query rows a key/value head:
// chunks of a prompt, blocks of tokens denoised together.
//
// Persistent CTAs, one an SM, each walk one run of the line of 128-key tiles
// (paged_sched.cuh). An item is 256 query rows: two 128-row tiles that share
// every K and V tile (a causal chunk's upper tile skips the keys only the
// lower one keeps). With at most 128 rows (SPLIT) both hold the same rows and
// take alternate key tiles; their results are joined in the CTA, so the
// tensor core still has two independent softmaxes to work between. Either way
// it runs one row tile's PV and next QK^T under the other's softmax. A row
// tile's softmax is two warpgroups, each half of the columns: a tile's chain
// QK^T - softmax - PV is what a row tile waits for, and eight warps shorten
// it (one warpgroup each: causal chunk 972 us, two: 943).
// Roles:
//   warp 0      TMA producer of K (a lane a copy: a page's part of a tile)
//   warp 1      TMEM allocator and tcgen05.mma issuer
//   warp 2      TMA producer of V; clears the rows of V no key owns
//   warp 3      TMA producer of Q, ahead of the item's first product
//   warps 4-19  the softmax warpgroups: row tile 0, columns 0-63 and 64-127,
//               then row tile 1
//   warps 20-23 (e4m3) converters: warp 2 then loads V as codes, and these
//               four turn them into the fp16 tiles that PV reads
// Tensor memory: S at 128w with P written over it, O at 256 + Dw.
//
// e4m3: QK^T runs on K's codes as they are (kind::f8f6f4, twice the 16-bit
// rate): each row of Q, scaled by a power of two, is the sum of two e4m3
// values, its rounding and the rest, which hold bf16's eight bits exactly down
// to 2^-9 of the row's largest value (2^-17 of it bounds the error below), so
// two products give the logits and take the time of one in bf16. K's scale
// multiplies the logits. PV runs in fp16: V is code times (scale / sigma), the
// quotient rounded to 11 bits and the product once more (sigma a power of two,
// the largest V scale of the piece so far of a token that is not all zeros), the
// weights fp16 times 2^12 (what is flushed is below 2^-36 of the largest); O is
// rescaled when sigma grows. A scale below 2^-21 of sigma has fewer bits: the
// quotient is then subnormal in fp16. Weights in e4m3 would lose those below
// 2^-18, which a long context's sum needs.
#include <type_traits>

#include "mma_steps.cuh"
#include "paged_sched.cuh"
#include "tiles.cuh"

namespace bsa {

constexpr int kTileKeys = 128;
// A run is at least this many tiles (one sequence of 437 to 20,000 keys, 32
// and 300 rows: 2 gives 10% less to 5% more, 8 up to 60% more).
constexpr int kTilesMin = 4;

template <int D, bool E4M3, bool SPLIT>
struct TilesCfg {
  static constexpr int THREADS = E4M3 ? 768 : 640;
  static constexpr int CHUNK = 128 * 128;          // 128 rows of 128 bytes
  static constexpr int QSLOTS = SPLIT ? 1 : 2;
  static constexpr int QTILE = 128 * D * 2;        // bf16, or e4m3 twice
  static constexpr int KTILE = 128 * D * (E4M3 ? 1 : 2);
  static constexpr int VTILE = 128 * D * 2;
  // Stages as shared memory allows. V's are held through a softmax, so where
  // HBM is the bound (SPLIT) it gets the room of the second Q slot.
  static constexpr int SK = D == 64 ? 4 : !E4M3 ? 2 : SPLIT ? 4 : 3;
  static constexpr int SV = D == 64 ? (SPLIT ? 6 : 4) : SPLIT && !E4M3 ? 3 : 2;
  static constexpr int RAW = !E4M3 ? 0 : D == 64 ? 8 : 4;  // V code pieces of 64 keys
  static constexpr int RAW_BYTES = 64 * D;
  // Scale and sigma ring: an entry is written again only when the K tile SK + SV
  // later is loaded, after the product of the tile SV later, before which the
  // issuer flushes the PVs (and so outlives the softmaxes) of this one
  static constexpr int R = E4M3 ? SK + SV : 0;
  static constexpr int K_OFF = QSLOTS * QTILE;
  static constexpr int V_OFF = K_OFF + SK * KTILE;
  static constexpr int RAW_OFF = V_OFF + SV * VTILE;
  static constexpr int XCH_OFF = RAW_OFF + RAW * RAW_BYTES;     // SPLIT: 2 x 16 channels of 128 rows, fp32
  static constexpr int LAND_OFF = XCH_OFF + (SPLIT ? 128 * 32 * 4 : 0);  // [RAW][128] V scales as loaded
  static constexpr int KSC_OFF = LAND_OFF + RAW * 512;          // [R][128] K scales
  static constexpr int SIG_OFF = KSC_OFF + R * 512;             // [R] sigma of a tile
  static constexpr int ML_OFF = SIG_OFF + (E4M3 ? 64 : 0);      // [128] row tile 1's (m, l, factor) (SPLIT)
  static constexpr int ZS_OFF = ML_OFF + (SPLIT ? 128 * 16 : 0);  // [128] row factors (SPLIT, e4m3)
  static constexpr int MX_OFF = ZS_OFF + (SPLIT && E4M3 ? 512 : 0);  // [2][2][128] exchange of a row's two halves
  static constexpr int BAR_OFF = MX_OFF + 4 * 128 * 4;
  static constexpr int NBAR = 4 + 1 + 2 * SK + 2 * SV + 1 + 8 + 1 + 2 * RAW + 2 * R;
  static constexpr int MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr int SMEM = MISC_OFF + 16 + sizeof(Run) + 24 * 8;
  static constexpr int ALLOC = SMEM + 1024;
  static_assert(ALLOC <= 227 * 1024, "smem budget");
  static_assert(SV <= 8 && R <= 16, "two bits a V stage; sigma's room");
};

// Instruction descriptor for kind::f16 with fp16 A and B and fp32 D.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Shared-memory matrix descriptor of K-major rows of 64 bytes, 64-byte swizzle
// (16-byte unit u of row r sits at u ^ ((r >> 1) & 3)).
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)1 << 16;          // leading offset (unused by swizzled K-major)
  d |= (uint64_t)(512 >> 4) << 32; // eight rows
  d |= (uint64_t)1 << 46;          // descriptor version for sm_100
  d |= (uint64_t)4 << 61;          // SWIZZLE_64B
  return d;
}

// S (+)= A K^T over D / 32 k-steps of 32 e4m3 values (K-major rows of D bytes).
template <int KK>
__device__ __forceinline__ void qk8_part(uint32_t s_tmem, uint64_t qd, uint64_t kd, uint32_t idesc, uint32_t acc) {
  umma8_ss_at_warp<KK * 2, KK * 2>(s_tmem, qd, kd, idesc, KK > 0 ? 1u : acc);
}
template <int... KK>
__device__ __forceinline__ void qk8_sum(uint32_t s_tmem, uint64_t qd, uint64_t kd, uint32_t idesc, uint32_t acc,
                                        std::integer_sequence<int, KK...>) {
  (qk8_part<KK>(s_tmem, qd, kd, idesc, acc), ...);
}

// O (+)= P V over 8 k-steps of 16 keys, the weights of keys 0-63 in columns
// 0-31 of S's place and those of keys 64-127 in columns 64-95.
template <int KK>
__device__ __forceinline__ void pv_half_step(uint32_t o_tmem, uint32_t p_tmem, uint64_t vd, uint32_t idesc,
                                             uint32_t first) {
  umma_ts_at_warp<(KK >> 2) * 64 + (KK & 3) * 8, KK * 2048 / 16>(o_tmem, p_tmem, vd, idesc,
                                                                  (KK > 0 || !first) ? 1u : 0u);
}
template <int... KK>
__device__ __forceinline__ void pv_halves(uint32_t o_tmem, uint32_t p_tmem, uint64_t vd, uint32_t idesc,
                                          uint32_t first, std::integer_sequence<int, KK...>) {
  (pv_half_step<KK>(o_tmem, p_tmem, vd, idesc, first), ...);
}

// Which row tiles need key tile kt (absolute) of a piece, and whether one needs
// any. Every role asks the same questions.
template <bool SPLIT>
struct TileNeed {
  int a0, e0, a1, e1;  // tile ranges of the row tiles
  int first;           // the piece's first tile (SPLIT)
  __device__ __forceinline__ TileNeed(const PagedParams& p, const Piece& q) {
    first = q.s.t0 + q.t;
    const int end = first + q.m;
    if constexpr (SPLIT) {
      const bool any = q.s.lo < q.s.hi;
      a0 = a1 = first;
      e0 = e1 = any ? end : first;
    } else {
      const ItemSpan x = item_span<128, kTileKeys>(p, q.n, q.kv, 2 * q.rt);
      ItemSpan y{0, 0, 0, 0, 0, 0};
      if ((long long)q.rt * 256 + 128 < (long long)p.G * p.N) y = item_span<128, kTileKeys>(p, q.n, q.kv, 2 * q.rt + 1);
      a0 = max(first, x.t0);
      e0 = x.lo < x.hi ? min(end, x.t0 + x.nt) : a0;
      a1 = max(first, y.t0);
      e1 = y.lo < y.hi ? min(end, y.t0 + y.nt) : a1;
    }
  }
  __device__ __forceinline__ int mask(int kt) const {
    if constexpr (SPLIT) return kt < e0 ? 1 << ((kt - first) & 1) : 0;
    return (kt >= a0 && kt < e0 ? 1 : 0) | (kt >= a1 && kt < e1 ? 2 : 0);
  }
  // is kt, needed by w, the last that w needs?
  __device__ __forceinline__ bool last(int kt, int w) const {
    if constexpr (SPLIT) return kt + 2 >= e0;
    return kt + 1 == (w ? e1 : e0);
  }
  __device__ __forceinline__ bool any(int w) const {
    if constexpr (SPLIT) return e0 - first > w;
    return w ? e1 > a1 : e0 > a0;
  }
};

// 32 lanes x 32-bit, 8 consecutive columns per thread.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// The rest of a bounded wait whose first try did not find the phase complete;
// kept out of line for e4m3, whose roles' loops outgrow the instruction cache.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t limit_ns) {
  return warp_all(mbar_wait(bar, parity, abort_flag, limit_ns));
}

__device__ __forceinline__ void mul2(float& x0, float& x1, float c0, float c1) {
  uint64_t v, c;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x0), "f"(x1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(c0), "f"(c1));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(v), "l"(c));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x0), "=f"(x1) : "l"(v));
}

template <int D, bool E4M3, bool SPLIT>
__global__ void __launch_bounds__(TilesCfg<D, E4M3, SPLIT>::THREADS, 1)
    paged_tiles_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const PagedParams p, const PagedWork wk,
                       int row_tiles) {
  using C = TilesCfg<D, E4M3, SPLIT>;
  constexpr int SK = C::SK, SV = C::SV, ROWS = SPLIT ? 128 : 256;
  constexpr float kTau = E4M3 ? 3.f : 8.f;    // the state moves when a row's maximum grows by more than 2^kTau
  constexpr float kGain = E4M3 ? 12.f : 0.f;  // log2 of what the weights are held times
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::K_OFF;
  uint8_t* sV = smem + C::V_OFF;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);  // [2]
  uint64_t* q_ready = q_full + 2;    // [2] e4m3: Q converted
  uint64_t* q_empty = q_ready + 2;   // every QK^T of the piece complete
  uint64_t* k_full = q_empty + 1;    // [SK]
  uint64_t* k_empty = k_full + SK;
  uint64_t* v_full = k_empty + SK;   // [SV]
  uint64_t* v_empty = v_full + SV;
  uint64_t* v_land = v_empty + SV;   // V of a tile with rows to clear
  uint64_t* s_full = v_land + 1;     // [2]
  uint64_t* p_full = s_full + 2;     // [2]
  uint64_t* o_ready = p_full + 2;    // [2]
  uint64_t* o_free = o_ready + 2;    // [2] O read by the softmax
  uint64_t* mma_done = o_free + 2;
  uint64_t* raw_full = mma_done + 1; // [RAW]
  uint64_t* raw_empty = raw_full + C::RAW;
  uint64_t* sc_full = raw_empty + C::RAW;  // [R] e4m3: K scales of a tile
  uint64_t* sig_full = sc_full + C::R;     // [R] e4m3: sigma of a tile
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  Run* run_sh = reinterpret_cast<Run*>(smem + C::MISC_OFF + 16);
  long long* scan_sh = reinterpret_cast<long long*>(smem + C::MISC_OFF + 16 + sizeof(Run));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  asm volatile("griddepcontrol.launch_dependents;");
  if (tid == 0) {
    for (int w = 0; w < 2; ++w) {
      mbar_init(&q_full[w], 1);
      mbar_init(&q_ready[w], 8);  // (an arrival a warp)
      mbar_init(&s_full[w], 1);
      mbar_init(&p_full[w], 8);
      mbar_init(&o_ready[w], 1);
      mbar_init(&o_free[w], 8);
    }
    mbar_init(q_empty, 1);
    mbar_init(v_land, 1);
    mbar_init(mma_done, 1);
    for (int s = 0; s < SK; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < SV; ++s) {
      mbar_init(&v_full[s], E4M3 ? 4 : 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < C::RAW; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], 4);
    }
    for (int s = 0; s < C::R; ++s) {
      mbar_init(&sc_full[s], 1);
      mbar_init(&sig_full[s], 1);
    }
    misc[1] = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(misc, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  Run run = find_run<ROWS, kTileKeys, C::THREADS, kReadOnly>(p, row_tiles, kTilesMin, run_sh, scan_sh);  // block barriers
  tc_fence_after();
  const uint32_t tmem = misc[0];

  auto teardown = [&]() {
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    const uint32_t a = smem_u32(bar);
    if (warp_all(mbar_try_wait(a, parity & 1u))) return true;
    if constexpr (E4M3) return wait_slow(bar, parity & 1u, abort_flag, p.wait_limit_ns);
    return warp_all(mbar_wait(bar, parity & 1u, abort_flag, p.wait_limit_ns));
  };
  const int page_mask = (1 << p.page_log2) - 1;

  if (warp < 4) {
    if (warp == 3) {
      // ------------------------------------------------------------- Q producer
      int pc = 0;
      bool ok = true;
      for (; run.left > 0 && ok; ++pc) {
        const Piece q = next_piece<ROWS, kTileKeys, kReadOnly>(p, row_tiles, run);
        if (pc > 0) {  // the slots are free, and their last tiles have landed
          ok = wait(q_empty, pc - 1);
          for (int w = 0; w < (SPLIT ? 1 : 2); ++w) ok = ok && wait(&q_full[w], pc - 1);
          if (!ok) {
            cta_fail(abort_flag, BSA_DEVERR_TIMEOUT);
            break;
          }
        }
        if (lane == 0)
          for (int w = 0; w < (SPLIT ? 1 : 2); ++w) {
            mbar_arrive_expect_tx(&q_full[w], C::QTILE);
            for (int c = 0; c < D / 64; ++c)
              for (int h2 = 0; h2 < 2; ++h2)  // rows past the head's G N read as zeros
                tma_load_3d(sQ + w * C::QTILE + c * C::CHUNK + h2 * (C::CHUNK / 2), &tmQ, &q_full[w], c * 64,
                            q.rt * ROWS + 128 * w + 64 * h2, q.b * p.Hkv + q.hk);
          }
        __syncwarp();
      }
      // here and in the producers below: copies in flight land before the CTA
      // ends, whether or not it aborts (the softmax may yet give up on them)
      if (pc > 0 && lane == 0)
        for (int w = 0; w < (SPLIT ? 1 : 2); ++w) mbar_drain(&q_full[w], (uint32_t)(pc - 1) & 1u);
    } else if (warp == 2 && E4M3) {
      if constexpr (E4M3) {
        // ------------------------------------------------------- V code producer
        // pieces of 64 keys; the tile's scales land with the first
        const int per = min(page_mask + 1, 64), sub = 64 / per;
        const int part = lane & 3, role = lane >> 2;  // role 0: codes, 1 and 2: scales of the low and high half
        int c = 0, k = 0;
        bool ok = true;
        while (run.left > 0 && ok) {
          const Piece q = next_piece<ROWS, kTileKeys, kReadOnly>(p, row_tiles, run);
          const TileNeed<SPLIT> need(p, q);
          // lane l < 2 sub holds the table entry of tokens l per .. of a tile;
          // the next tile's is on its way while this one's pieces wait
          auto keeps = [&](int j) { return j < q.s.hi && j + per > q.s.lo; };
          auto entry_of = [&](int kt) {
            const int j = kt * kTileKeys + lane * per;
            return lane < 2 * sub && keeps(j) ? table_entry<kReadOnly>(p, q.b, j) : 0;
          };
          int next = entry_of(q.s.t0 + q.t);
          for (int i = 0; i < q.m && ok; ++i) {
            const int kt = q.s.t0 + q.t + i;
            const int entry = next;
            if (i + 1 < q.m) next = entry_of(kt + 1);
            if (need.mask(kt) == 0) continue;
            const int page = lane < 2 * sub && keeps(kt * kTileKeys + lane * per) ? checked_page(p, entry) : 0;
            for (int x = 0; x < 2; ++x, ++c) {
              const int half = role == 0 ? x : (role - 1) & 1;
              const int j0 = kt * kTileKeys + 64 * half + part * per;
              const bool mine = part < sub && keeps(j0) && (role == 0 || (x == 0 && role <= 2));
              const int pg = __shfl_sync(0xffffffffu, page, half * sub + part);
              const int st = c % C::RAW;
              if (c >= C::RAW) ok = wait(&raw_empty[st], c / C::RAW - 1);
              if (!ok) {
                cta_fail(abort_flag, BSA_DEVERR_TIMEOUT);
                break;
              }
              const uint32_t codes = __popc(__ballot_sync(0xffffffffu, mine && role == 0));
              const uint32_t scales = __popc(__ballot_sync(0xffffffffu, mine && role != 0));
              if (lane == 0) mbar_arrive_expect_tx(&raw_full[st], codes * per * D + scales * per * 4);
              __syncwarp();
              if (mine) {
                if (role == 0)
                  tma_load_3d(smem + C::RAW_OFF + st * C::RAW_BYTES + part * per * D, &tmV, &raw_full[st], 0,
                              (j0 & page_mask) * D / 128, pg * p.Hkv + q.hk);
                else
                  bulk_load_1d(smem + C::LAND_OFF + (k % C::RAW) * 512 + (64 * half + part * per) * 4,
                               p.v_scale + cache_row(p, pg, q.hk, j0), per * 4, &raw_full[st]);
              }
              __syncwarp();
            }
            ++k;
          }
        }
        if (lane == 0)
          for (int t = max(0, c - C::RAW); t < c; ++t) mbar_drain(&raw_full[t % C::RAW], (uint32_t)(t / C::RAW) & 1u);
      }
    } else if (warp == 0 || warp == 2) {
      // --------------------------------------------------------- K and V producers
      auto produce = [&](auto ring) {
        constexpr bool IS_K = decltype(ring)::value;
        constexpr int S = IS_K ? SK : SV;
        constexpr int ROW = E4M3 ? D : 128;  // bytes of a token's row in one copy
        uint64_t* const full = IS_K ? k_full : v_full;
        uint64_t* const empty = IS_K ? k_empty : v_empty;
        const int per = min(page_mask + 1, kTileKeys), sub = kTileKeys / per;
        // a lane a copy: role = 64-channel half, or (e4m3) the K scales
        const int part = lane & 7, role = lane >> 3;
        const bool copies_tile = role < (E4M3 ? 1 : D / 64);
        int k = 0, landed = 0;
        bool ok = true;
        while (run.left > 0 && ok) {
          const Piece q = next_piece<ROWS, kTileKeys, kReadOnly>(p, row_tiles, run);
          const TileNeed<SPLIT> need(p, q);
          int j0 = (q.s.t0 + q.t) * kTileKeys + part * per;  // first token of this lane's copies
          auto keeps = [&](int j) { return part < sub && role < 2 && j < q.s.hi && j + per > q.s.lo; };
          int next = keeps(j0) ? table_entry<kReadOnly>(p, q.b, j0) : 0;
          for (int i = 0; i < q.m; ++i, j0 += kTileKeys) {
            const int kt = q.s.t0 + q.t + i;
            const bool mine = keeps(j0);
            const int entry = next;  // the next tile's is on its way while this one waits for its stage
            next = i + 1 < q.m && keeps(j0 + kTileKeys) ? table_entry<kReadOnly>(p, q.b, j0 + kTileKeys) : 0;
            if (need.mask(kt) == 0) continue;
            const int st = k % S, key0 = kt * kTileKeys;
            if (k >= S) ok = wait(&empty[st], k / S - 1);
            if (!ok) {
              cta_fail(abort_flag, BSA_DEVERR_TIMEOUT);
              break;
            }
            if (IS_K && k == p.withhold_tile) {  // failure-detection test
              ++k;
              continue;
            }
            // V rows of no kept key: their weights are zero, but whatever
            // the slots hold (NaN, even) must not meet them
            const bool clear = !IS_K && (key0 < q.s.lo || key0 + kTileKeys > q.s.hi);
            uint64_t* bar = clear ? v_land : &full[st];
            const uint32_t copies = __popc(__ballot_sync(0xffffffffu, mine && copies_tile));
            if (lane == 0) {
              mbar_arrive_expect_tx(bar, copies * per * ROW);
              if constexpr (E4M3) mbar_arrive_expect_tx(&sc_full[k % C::R], copies * per * 4);
            }
            __syncwarp();
            uint8_t* tile = IS_K ? sK + st * C::KTILE : sV + st * C::VTILE;
            if (mine) {
              const int pg = checked_page(p, entry);
              if (copies_tile) {
                tma_load_3d(tile + role * C::CHUNK + part * per * ROW, IS_K ? &tmK : &tmV, bar, role * 64,
                            j0 & page_mask, pg * p.Hkv + q.hk);
              } else if constexpr (E4M3) {
                bulk_load_1d(smem + C::KSC_OFF + (k % C::R) * 512 + part * per * 4,
                             p.k_scale + cache_row(p, pg, q.hk, j0), per * 4, &sc_full[k % C::R]);
              }
            }
            __syncwarp();
            if (clear) {
              ok = wait(v_land, landed++);
              if (!ok) {
                cta_fail(abort_flag, BSA_DEVERR_TIMEOUT);
                if (lane == 0) mbar_drain(v_land, (uint32_t)(landed - 1) & 1u);
                break;
              }
              const int a = max(q.s.lo - key0, 0), e = min(q.s.hi - key0, kTileKeys);  // rows [a, e) stay
              constexpr int U = D / 8;  // 16-byte units of a row
              for (int x = lane; x < (kTileKeys - (e - a)) * U; x += 32) {
                const int u = x % U, r0 = x / U;
                const int r = r0 < a ? r0 : r0 - a + e;
                *reinterpret_cast<uint4*>(tile + (u >> 3) * C::CHUNK + r * 128 + (u & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&full[st]);
            }
            ++k;
          }
        }
        // a stage whose tile was cleared by this warp has landed already
        if (lane == 0) {
          for (int t = max(0, k - S); t < k; ++t)
            if (!IS_K || t != p.withhold_tile) mbar_drain(&full[t % S], (uint32_t)(t / S) & 1u);
          if constexpr (E4M3)
            for (int t = max(0, k - C::R); t < k; ++t)
              if (t != p.withhold_tile) mbar_drain(&sc_full[t % C::R], (uint32_t)(t / C::R) & 1u);
        }
      };
      if (warp == 0)
        produce(std::true_type{});
      else
        produce(std::false_type{});
    } else if (warp == 1) {
      // ------------------------------------------------------------- MMA issuer
      constexpr uint32_t idesc_qk = E4M3 ? idesc_e4m3_f32(128, 128) : idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t idesc_pv = E4M3 ? idesc_f16_f32(128, D, true) : idesc_bf16_f32(128, D, false, true);
      const uint32_t sQa = smem_u32(sQ), sKa = smem_u32(sK), sVa = smem_u32(sV);
      struct RowTile {
        int pt;      // tile whose PV is outstanding (-1: none)
        int np, nf;  // PVs issued, pieces begun
        bool fresh;  // the next PV is the piece's first
        bool last;   // the outstanding PV is the piece's last
      };
      RowTile cur{-1, 0, 0, false, false}, oth = cur;
      int v_seen = 0, k = 0, pc = 0;
      uint32_t rem = 0u;  // row tiles still to use a stage's V, two bits a stage
      bool ok = true, issued = false;
      // e4m3: one code site for PV and one for QK^T, the row tiles taking turns
      // in `cur`; with a copy a call this loop outgrew the instruction cache
      // (ragged chunks 342 -> 275 us). bf16 has room for a copy a row tile.
      for (; run.left > 0 && ok; ++pc) {
        const Piece q = next_piece<ROWS, kTileKeys, kReadOnly>(p, row_tiles, run);
        const TileNeed<SPLIT> need(p, q);
        for (int w = 0; w < (SPLIT ? 1 : 2) && ok; ++w) ok = wait(E4M3 ? &q_ready[w] : &q_full[w], pc);
        cur.fresh = oth.fresh = true;
#pragma unroll 1
        for (int i = 0; i <= q.m && ok; ++i) {
          const int kt = q.s.t0 + q.t + i;
          const bool flush = i == q.m;  // the piece's last PVs
          const int nw = flush ? 0 : need.mask(kt);
          if (nw == 0 && !flush) continue;
          const int st = k % SK;
          if constexpr (!E4M3 && !SPLIT) {
            // The long run of tiles both row tiles need, each with its PV of
            // the tile before outstanding: the same steps without the
            // bookkeeping, which otherwise takes the issuer longer between two
            // products than the tensor pipe has work queued
            if (nw == 3 && cur.pt == k - 1 && oth.pt == k - 1 && !cur.fresh && !oth.fresh) {
              const int n = min(need.e0, need.e1) - kt;  // such tiles from here on, at least this one
              int ks = st, kp = (k / SK) & 1, vs = (k - 1) % SV, vp = ((k - 1) / SV) & 1;
#pragma unroll 1
              for (int x = 0; x < n && ok; ++x) {
                const uint64_t vd = smem_desc_sw128(sVa + vs * C::VTILE, C::CHUNK, 1024);
                const uint64_t kd = smem_desc_sw128(sKa + ks * C::KTILE, 16, 1024);
                ok = wait(&k_full[ks], kp) && wait(&v_full[vs], vp);
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                  ok = ok && wait(&p_full[w], w ? oth.np : cur.np);
                  if (!ok) break;
                  tc_fence_after();
                  pv_halves(tmem + 256 + w * D, tmem + 128 * w, vd, idesc_pv, 0u, std::make_integer_sequence<int, 8>{});
                  if (w) tc_commit_warp(&v_empty[vs]);
                  qk_all(tmem + 128 * w, smem_desc_sw128(sQa + w * C::QTILE, 16, 1024), kd, idesc_qk,
                         std::make_integer_sequence<int, D / 16>{});
                  tc_commit_warp(&s_full[w]);
                }
                if (!ok) break;
                tc_commit_warp(&k_empty[ks]);
                ++cur.np;
                ++oth.np;
                if (++ks == SK) {
                  ks = 0;
                  kp ^= 1;
                }
                if (++vs == SV) {
                  vs = 0;
                  vp ^= 1;
                }
              }
              k += n;
              v_seen = k - 1;
              rem = 2u << (2 * ((k - 1) % SV));
              cur.pt = oth.pt = k - 1;
              cur.last = kt + n == need.e0;
              oth.last = kt + n == need.e1;
              i += n - 1;
              continue;
            }
          }
          if (!flush)
            ok = wait(&k_full[st], k / SK);
          else
            tc_commit_warp(q_empty);
          // a row tile that does not need tile k goes first: its outstanding
          // PV may be the last user of the V stage tile k is about to count on
          const int w0 = nw == 1 ? 1 : 0;
          if (w0) {
            const RowTile t = cur;
            cur = oth;
            oth = t;
          }
#pragma unroll(E4M3 ? 1 : 2)
          for (int s = 0; s < 2; ++s) {
            const int w = w0 ^ s;
            // PV of the tile before: P lies over S, and the tensor pipe keeps
            // issue order. One that holds up the V stage of tile k goes out
            // although its row tile does not need tile k.
            if (ok && cur.pt >= 0 && (flush || ((nw >> w) & 1) || cur.pt <= k - SV)) {
              const int u = cur.pt, sv = u % SV;
              // V tiles are observed in tile order, so the parity test never
              // meets another phase of a shared stage
              for (; v_seen <= u && ok; ++v_seen) ok = wait(&v_full[v_seen % SV], v_seen / SV);
              if (cur.fresh) {  // O of the piece before has been read
                if (cur.nf > 0) ok = ok && wait(&o_free[w], cur.nf - 1);
                ++cur.nf;
              }
              ok = ok && wait(&p_full[w], cur.np);
              ++cur.np;
              if (ok) {
                tc_fence_after();
                pv_halves(tmem + 256 + w * D, tmem + 128 * w, smem_desc_sw128(sVa + sv * C::VTILE, C::CHUNK, 1024),
                          idesc_pv, cur.fresh ? 1u : 0u, std::make_integer_sequence<int, 8>{});
                if (cur.last) tc_commit_warp(&o_ready[w]);
                rem -= 1u << (2 * sv);
                if (((rem >> (2 * sv)) & 3u) == 0u) tc_commit_warp(&v_empty[sv]);
              }
              cur.fresh = false;
              cur.pt = -1;
            }
            if (ok && ((nw >> w) & 1)) {
              tc_fence_after();
              const uint32_t qa = sQa + (SPLIT ? 0 : w) * C::QTILE, ka = sKa + st * C::KTILE;
              if constexpr (!E4M3) {
                qk_all(tmem + 128 * w, smem_desc_sw128(qa, 16, 1024), smem_desc_sw128(ka, 16, 1024), idesc_qk,
                       std::make_integer_sequence<int, D / 16>{});
              } else {
#pragma unroll 1
                for (int h = 0; h < 2; ++h)  // the row's rounding, then the rest
                  qk8_sum(tmem + 128 * w,
                          D == 128 ? smem_desc_sw128(qa + h * 128 * D, 16, 1024) : smem_desc_sw64(qa + h * 128 * D),
                          D == 128 ? smem_desc_sw128(ka, 16, 1024) : smem_desc_sw64(ka), idesc_qk, (uint32_t)h,
                          std::make_integer_sequence<int, D / 32>{});
              }
              tc_commit_warp(&s_full[w]);
              issued = true;
              rem += 1u << (2 * (k % SV));
              cur.pt = k;
              cur.last = need.last(kt, w);
            }
            const RowTile t = cur;
            cur = oth;
            oth = t;
          }
          if (w0) {
            const RowTile t = cur;
            cur = oth;
            oth = t;
          }
          if (!flush) {
            // (a stage whose tile was waited for in vain is not free: its copies may be in flight)
            if (ok) tc_commit_warp(&k_empty[st]);
            ++k;
          }
        }
      }
      if (!ok) cta_fail(abort_flag, BSA_DEVERR_TIMEOUT);
      // tensor memory is freed only once every issued MMA has completed
      if (issued) {
        tc_commit_warp(mma_done);
        mbar_drain(mma_done, 0u);
      }
    }
    teardown();
  } else if (warp < 20) {
    // --------------------------------------------------------------- softmax
    const int w = (warp - 4) >> 3, hf = ((warp - 4) >> 2) & 1, q4 = warp & 3;
    const int r = q4 * 32 + lane;
    const int pair_bar = 4 + 4 * w + q4;  // this warp and the one with the rows' other columns
    const int kc = 64 * hf, oc = D / 2 * hf;  // first of this thread's columns of S, of O
    float* mx_mine = reinterpret_cast<float*>(smem + C::MX_OFF) + (2 * w + hf) * 128 + r;
    const float* mx_other = reinterpret_cast<float*>(smem + C::MX_OFF) + (2 * w + 1 - hf) * 128 + r;
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t stm = tmem + lane_off + 128 * w, otm = tmem + lane_off + 256 + w * D;
    const int slot_row = (SPLIT ? 0 : 128 * w) + r;  // row of the item
    float4* ml_sh = reinterpret_cast<float4*>(smem + C::ML_OFF);
    float* zs_sh = reinterpret_cast<float*>(smem + C::ZS_OFF);
    int j = 0, pj = 0, k = 0, pc = 0;  // tiles and pieces of this row tile, tiles and pieces of the CTA
    bool ok = true;
    SplitItem split{0, 0, 0, 0};
    for (; run.left > 0; ++pc) {
      const long long at = run.pos;
      const Piece q = next_piece<ROWS, kTileKeys, kReadOnly>(p, row_tiles, run);
      if (q.t == 0 && q.m < q.s.nt)
        split = SplitItem{q.b * row_tiles + q.rt, q.hk, run_of(run.total, at + q.s.nt - 1, run.ctas) - (int)blockIdx.x + 1, 0};
      const TileNeed<SPLIT> need(p, q);
      const int R = q.rt * ROWS + slot_row;  // packed row of the head
      const int tok = R < p.G * p.N ? R - fdiv(R, p.f_n) * p.N : 0;
      const bool written = R < p.G * p.N && tok < q.n;
      const bool warp_rows = __any_sync(0xffffffffu, written);
      int lo, hi;
      row_keys(p, q.n, q.kv, tok, lo, hi);
      if (!written) lo = hi = 0;
      // keys that every written row of the warp keeps
      const int clo = __reduce_max_sync(0xffffffffu, written ? lo : 0);
      const int chi = __reduce_min_sync(0xffffffffu, written ? hi : 0x7fffffff);
      float zs = p.scale_log2;
      if constexpr (E4M3) {
        if (!SPLIT || w == 0) {
          // this thread's half row of Q in place as two e4m3 parts, after a
          // power-of-two scale that leaves the row's largest value in [2^7, 2^8)
          ok = ok && wait(&q_full[w], pc);
          uint8_t* base = sQ + (SPLIT ? 0 : w) * C::QTILE;
          constexpr int U = D / 16;  // 16-byte units of the half row
          uint4 x[U];
          uint32_t top = 0u;
#pragma unroll
          for (int e = 0; e < U; ++e) {
            const int u = U * hf + e;
            x[e] = *reinterpret_cast<const uint4*>(base + (u >> 3) * C::CHUNK + r * 128 + (((u ^ r) & 7) << 4));
            const uint32_t y = __vmaxu2(__vmaxu2(x[e].x & 0x7fff7fffu, x[e].y & 0x7fff7fffu),
                                        __vmaxu2(x[e].z & 0x7fff7fffu, x[e].w & 0x7fff7fffu));
            top = max(top, max(y & 0xffffu, y >> 16));
          }
          *mx_mine = __uint_as_float(top);
          named_bar(1 + w, 256);  // every row is read: at d = 64 the two forms lie elsewhere
          top = max(top, __float_as_uint(*mx_other));
          named_bar(pair_bar, 64);  // read: a piece without tiles goes on to its sums in the same word
          // 2^(7 - e), e the exponent of the largest value, kept in the normal range
          const int ex = min(max((int)(top >> 7), 8), 253);
          const float down = __int_as_float((261 - ex) << 23);
          zs *= top < 0x7f80u ? __int_as_float((ex - 7) << 23) : __int_as_float(0x7fc00000);  // a row with inf or NaN
#pragma unroll
          for (int e = 0; e < U / 2; ++e) {  // 16 values: a unit of each form
            const int u = U / 2 * hf + e;
            uint32_t hw[4], lw[4];
            const uint32_t v[8] = {x[2 * e].x, x[2 * e].y, x[2 * e].z, x[2 * e].w,
                                   x[2 * e + 1].x, x[2 * e + 1].y, x[2 * e + 1].z, x[2 * e + 1].w};
#pragma unroll
            for (int n = 0; n < 8; ++n) {
              const float a = __uint_as_float(v[n] << 16) * down, b = __uint_as_float(v[n] & 0xffff0000u) * down;
              const uint32_t hi = e4m3x2(a, b);
              const uint32_t h2 = codes_lo(hi);
              const float2 hf2 = __half22float2(*reinterpret_cast<const __half2*>(&h2));
              const uint32_t lo8 = e4m3x2(a - hf2.x, b - hf2.y);
              if (n & 1) {
                hw[n >> 1] |= hi << 16;
                lw[n >> 1] |= lo8 << 16;
              } else {
                hw[n >> 1] = hi;
                lw[n >> 1] = lo8;
              }
            }
            const int off = D == 128 ? r * 128 + (((u ^ r) & 7) << 4) : r * 64 + (((u ^ (r >> 1)) & 3) << 4);
            *reinterpret_cast<uint4*>(base + off) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
            *reinterpret_cast<uint4*>(base + 128 * D + off) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
          }
          if constexpr (SPLIT)
            if (hf == 0) zs_sh[r] = zs;
          if (!ok) cta_fail(abort_flag, BSA_DEVERR_TIMEOUT);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_ready[w]);
        } else {
          // row tile 0's warpgroups convert; they cannot pass this piece's join
          // before this one
          ok = ok && wait(&q_ready[0], pc);
          zs = zs_sh[r];
        }
      }
      float m = kNegInf, l = 0.f, sig = 1.f;
      int jp = 0;  // tiles of this row tile in the piece
      // An aborting CTA walks its tiles without waiting or computing: a row's
      // two warps meet in a barrier every tile, so neither may leave early.
      for (int i = 0; i < q.m; ++i) {
        const int kt = q.s.t0 + q.t + i;
        const int nw = need.mask(kt);
        if (nw == 0) continue;
        const int kk = k++;
        if (!((nw >> w) & 1)) continue;
        ok = ok && wait(&s_full[w], j);
        tc_fence_after();
        if (warp_rows) {
          const int key0 = kt * kTileKeys;
          const float4* ks = reinterpret_cast<const float4*>(smem + C::KSC_OFF + (E4M3 ? kk % C::R : 0) * 512);
          if constexpr (E4M3) ok = ok && wait(&sc_full[kk % C::R], kk / C::R);
          const bool edge = key0 < clo || key0 + kTileKeys > chi;
          const int first = lo - key0, n = hi - lo;  // the row keeps columns [first, first + n)
          // CH scores of the row, masked. They are read twice, for the maximum
          // and for the weights, in loops that stay rolled: unrolled over a
          // whole row in registers this code outgrew the instruction cache
          // beside the other roles' (a third slower for e4m3). The converters'
          // threads leave e4m3 fewer registers (16 scores at a time: 264 us
          // for the ragged chunks, 32: 274).
          constexpr int CH = E4M3 ? 16 : 32;
          auto scores = [&](int c, float (&x)[CH]) {
            if constexpr (CH == 32)
              tmem_ld32(stm + kc + CH * c, x);
            else
              tmem_ld16(stm + kc + CH * c, x);
            tc_wait_ld();
            if constexpr (E4M3) {
#pragma unroll
              for (int e = 0; e < CH / 4; ++e) {
                const float4 s4 = ks[kc / 4 + CH / 4 * c + e];
                mul2(x[4 * e], x[4 * e + 1], s4.x, s4.y);
                mul2(x[4 * e + 2], x[4 * e + 3], s4.z, s4.w);
              }
            }
            if (edge) {
#pragma unroll
              for (int e = 0; e < CH; ++e) x[e] = (uint32_t)(kc + CH * c + e - first) < (uint32_t)n ? x[e] : kNegInf;
            }
          };
          float top = kNegInf;
#pragma unroll 1
          for (int c = 0; c < (ok ? 64 / CH : 0); ++c) {
            float x[CH];
            scores(c, x);
            float t0 = max3f(x[0], x[1], x[2]), t1 = max3f(x[3], x[4], x[5]);
#pragma unroll
            for (int e = 6; e < CH - 2; e += 4) {
              t0 = max3f(t0, x[e], x[e + 1]);
              t1 = max3f(t1, x[e + 2], x[e + 3]);
            }
            top = max3f(max3f(t0, x[CH - 2], x[CH - 1]), t1, top);
          }
          // the row's maximum over both halves
          *mx_mine = top;
          named_bar(pair_bar, 64);
          top = fmaxf(top, *mx_other) * zs;
          float alpha = 1.f;
          if (top > m + kTau) {
            alpha = fast_exp2(m - top);
            m = top;
          }
          const float off = kGain - (m == kNegInf ? 0.f : m);
          // P over this half's own columns of S, behind the scores read: S(j)
          // landing implies PV(j-1) is complete
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll 1
          for (int c = 0; c < (ok ? 64 / CH : 0); ++c) {
            float x[CH];
            scores(c, x);
            uint32_t pk[CH / 2];
#pragma unroll
            for (int e = 0; e < CH / 2; ++e) {
              float a = x[2 * e], b = x[2 * e + 1];
              fma2(a, b, zs, off);
              a = fast_exp2(a);
              b = fast_exp2(b);
              add2(sum0, sum1, a, b);
              pk[e] = E4M3 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
            }
            if constexpr (CH == 32)
              tmem_st16(stm + kc + 16 * c, pk);
            else
              tmem_st8(stm + kc + 8 * c, pk);
          }
          l = l * alpha + (sum0 + sum1);
          if constexpr (E4M3) {
            ok = ok && wait(&sig_full[kk % C::R], kk / C::R);
            const float now = *reinterpret_cast<const float*>(smem + C::SIG_OFF + (kk % C::R) * 4);
            if (jp > 0) alpha *= sig / now;  // both powers of two
            sig = now;
          }
          if (ok && jp > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[16];
              tmem_ld16(otm + oc + c * 16, o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= alpha;
              tmem_st16(otm + oc + c * 16, reinterpret_cast<uint32_t*>(o));
            }
          }
          tc_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&p_full[w]);
        ++j;
        ++jp;
      }
      if (jp > 0) {
        ok = ok && wait(&o_ready[w], pj++);
        tc_fence_after();
      }
      if (!ok) cta_fail(abort_flag, BSA_DEVERR_TIMEOUT);
      const bool have = ok && jp > 0;

      // ------------------------------------------------------------ epilogue
      const bool whole = q.whole();
      const size_t slot = 2 * (size_t)blockIdx.x + (q.t == 0 ? 1 : 0);
      const size_t obase = ((size_t)(q.b * p.Hkv + q.hk) * p.G * p.N + R) * D;
      // the row's sum over both halves
      *mx_mine = l;
      named_bar(pair_bar, 64);
      l += *mx_other;
      named_bar(pair_bar, 64);
      // 16 channels of a row, scaled and stored: the output, or a partial result
      auto store = [&](int c, float (&o)[16], float f) {
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] *= f;
        if (!written) return;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(p.O + obase + oc + c * 16);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            dst[e] = make_uint4(pack_bf16x2(o[8 * e], o[8 * e + 1]), pack_bf16x2(o[8 * e + 2], o[8 * e + 3]),
                                pack_bf16x2(o[8 * e + 4], o[8 * e + 5]), pack_bf16x2(o[8 * e + 6], o[8 * e + 7]));
        } else {
          // [slot][four channels][row]: a warp's rows side by side
          float4* dst = reinterpret_cast<float4*>(wk.o) + (slot * (D / 4) + oc / 4 + c * 4) * ROWS + slot_row;
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e * ROWS] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      };
      auto load = [&](int c, float (&o)[16]) {
        if (have) {
          tmem_ld16(otm + oc + c * 16, o);
          tc_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0.f;
        }
      };
      const float unit = E4M3 ? sig * (1.f / 128.f) : 1.f;  // what O is held over
      auto inverse = [&](float x) { return !whole ? 1.f : x > 0.f ? 1.f / x : x == 0.f ? 0.f : x; };
      if constexpr (SPLIT) {
        // row tile 1 hands its results over, 16 channels a warpgroup at a time
        float4* xch = reinterpret_cast<float4*>(smem + C::XCH_OFF) + hf * 4 * 128;
        float f0 = 0.f, f1 = 0.f;
        if (w == 1 && hf == 0) ml_sh[r] = make_float4(m, l, unit, 0.f);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[16];
          load(c, o);
          if (w == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              xch[e * 128 + r] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
          named_bar(3, 512);
          if (w == 0) {
            if (c == 0) {
              const float4 x = ml_sh[r];
              const float M = fmaxf(m, x.x), mu = M == kNegInf ? 0.f : M;
              const float e0 = fast_exp2(m - mu), e1 = fast_exp2(x.x - mu);
              m = M;
              l = l * e0 + x.y * e1;
              f0 = e0 * unit * inverse(l);
              f1 = e1 * x.z * inverse(l);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 x = xch[e * 128 + r];
              o[4 * e] = o[4 * e] * f0 + x.x * f1;
              o[4 * e + 1] = o[4 * e + 1] * f0 + x.y * f1;
              o[4 * e + 2] = o[4 * e + 2] * f0 + x.z * f1;
              o[4 * e + 3] = o[4 * e + 3] * f0 + x.w * f1;
            }
            store(c, o, 1.f);
          }
          named_bar(3, 512);
        }
      } else {
        const float f = unit * inverse(l);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[16];
          load(c, o);
          store(c, o, f);
        }
      }
      if (!whole && written && hf == 0 && (!SPLIT || w == 0)) wk.ml[slot * ROWS + slot_row] = make_float2(m, l);
      if (need.any(w)) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[w]);
      }
    }
    if (warp == 4 && lane == 0) wk.split[blockIdx.x] = split;
    teardown();
  } else {
    if constexpr (E4M3) {
      // ------------------------------------------------------------- converters
      const int cw = warp - 20;
      int c = 0, k = 0;
      bool ok = true;
      while (run.left > 0 && ok) {
        const Piece q = next_piece<ROWS, kTileKeys, kReadOnly>(p, row_tiles, run);
        const TileNeed<SPLIT> need(p, q);
        float sig = 0x1p-112f;
        for (int i = 0; i < q.m && ok; ++i) {
          const int kt = q.s.t0 + q.t + i;
          if (need.mask(kt) == 0) continue;
          const int st = k % SV, key0 = kt * kTileKeys;
          const bool edge = key0 < q.s.lo || key0 + kTileKeys > q.s.hi;
          const float* land = reinterpret_cast<const float*>(smem + C::LAND_OFF + (k % C::RAW) * 512);
          for (int half = 0; half < 2; ++half, ++c) {
            ok = wait(&raw_full[c % C::RAW], c / C::RAW);
            if (ok && half == 0) {
              // sigma from the tile's V scales; every warp finds the same
              const int j4 = key0 + 4 * lane;
              const float4 f = reinterpret_cast<const float4*>(land)[lane];
              const float fs[4] = {f.x, f.y, f.z, f.w};
              uint32_t b[4];  // as bits; 0 for what does not count
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                b[e] = __float_as_uint(fs[e]);
                if (b[e] >= 0x7f800000u || (edge && (j4 + e < q.s.lo || j4 + e >= q.s.hi))) b[e] = 0u;
              }
              uint32_t top = __reduce_max_sync(0xffffffffu, max(max(b[0], b[1]), max(b[2], b[3])));
              if (top > __float_as_uint(sig)) {
                // A token of zeros adds nothing whatever its scale (1, as it
                // is written): it must not move sigma, or V's small values
                // would sink into fp16's subnormals. Of the tokens with the
                // largest scale one must have a value, or the next largest
                // scale is looked at; the second half's codes land first.
                ok = wait(&raw_full[(c + 1) % C::RAW], (c + 1) / C::RAW);
                while (ok && top > __float_as_uint(sig)) {
                  const uint8_t* codes = smem + C::RAW_OFF + ((c + (lane >> 4)) % C::RAW) * C::RAW_BYTES;
                  bool some = false;
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    if (b[e] != top) continue;
                    uint32_t any = 0u;
#pragma unroll 1
                    for (int u = 0; u < D / 16; ++u) {
                      const uint32_t lin = (4 * (lane & 15) + e) * D + u * 16;
                      const uint4 y = *reinterpret_cast<const uint4*>(codes + (lin ^ ((lin >> 3) & 0x70u)));
                      any |= y.x | y.y | y.z | y.w;
                    }
                    if (any & 0x7f7f7f7fu)
                      some = true;
                    else
                      b[e] = 0u;
                  }
                  if (__any_sync(0xffffffffu, some)) break;
                  top = __reduce_max_sync(0xffffffffu, max(max(b[0], b[1]), max(b[2], b[3])));
                }
                if (top > __float_as_uint(sig)) sig = __uint_as_float(min((top + 0x7fffffu) & 0x7f800000u, 0x7f000000u));
              }
              if (cw == 0 && lane == 0) {
                *reinterpret_cast<float*>(smem + C::SIG_OFF + (k % C::R) * 4) = sig;
                mbar_arrive(&sig_full[k % C::R]);
              }
              if (k >= SV) ok = ok && wait(&v_empty[st], k / SV - 1);
            }
            if (!ok) {
              cta_fail(abort_flag, BSA_DEVERR_TIMEOUT);
              break;
            }
            const uint8_t* raw = smem + C::RAW_OFF + (c % C::RAW) * C::RAW_BYTES;
            uint8_t* tile = sV + st * C::VTILE;
            constexpr int UNITS = D / 16;                  // 16-code units of a token
            constexpr int STEP = 128 / UNITS;              // tokens a step of the warpgroup covers
            const int u = lane % UNITS;
            const float up = 128.f / sig;
#pragma unroll
            for (int e = 0; e < 64 / STEP; ++e) {
              const int key = e * STEP + cw * (32 / UNITS) + lane / UNITS;  // of the piece
              const uint32_t lin = key * D + u * 16;
              const uint4 y = *reinterpret_cast<const uint4*>(raw + (lin ^ ((lin >> 3) & 0x70u)));
              uint32_t h[8] = {codes_lo(y.x), codes_hi(y.x), codes_lo(y.y), codes_hi(y.y),
                               codes_lo(y.z), codes_hi(y.z), codes_lo(y.w), codes_hi(y.w)};
              const int row = 64 * half + key;
              const float f = land[row];  // (above sigma: a token of zeros; NaN stays)
              const float s = (f > sig && f <= 3.402823466e38f ? sig : f) * up;
              const uint32_t s2 = pack_f16x2(s, s);
              // rows of no kept key are cleared: their codes and scales may be anything
              const bool out = edge && (key0 + row < q.s.lo || key0 + row >= q.s.hi);
#pragma unroll
              for (int n = 0; n < 8; ++n) {
                const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&h[n]), *reinterpret_cast<const __half2*>(&s2));
                h[n] = out ? 0u : *reinterpret_cast<const uint32_t*>(&z);
              }
              uint8_t* dst = tile + (u >> 2) * C::CHUNK + row * 128;
              const int a = 2 * (u & 3);
              *reinterpret_cast<uint4*>(dst + (((a ^ row) & 7) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(dst + ((((a + 1) ^ row) & 7) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&raw_empty[c % C::RAW]);
              if (half == 1) mbar_arrive(&v_full[st]);
            }
          }
          ++k;
        }
      }
      teardown();
    }
  }
}

// Joins the partial results of split items (see paged_join_kernel): grid
// (CTAs of the forward, 8), a thread a row and some groups of four channels,
// rows side by side as they were stored.
template <int D, int ROWS>
__global__ void __launch_bounds__(256) paged_join_tiles_kernel(const PagedParams p, const PagedWork wk, int row_tiles) {
  constexpr int CPT = ROWS * (D / 4) / 2048;  // channel groups a thread
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const SplitItem it = wk.split[blockIdx.x];
  if (it.parts <= 1) return;
  const int b = it.idx / row_tiles, rt = it.idx - b * row_tiles;
  const SeqLen s = seq_clamped(p, b);
  const int x = blockIdx.y * 256 + threadIdx.x;
  const int r = x % ROWS, c0 = x / ROWS;  // channel groups c0, c0 + 2048 / ROWS, ...
  const int R = rt * ROWS + r;
  if (R >= p.G * p.N || R - fdiv(R, p.f_n) * p.N >= s.n) return;
  auto slot = [&](int i) -> size_t { return i == 0 ? 2 * (size_t)blockIdx.x + 1 : 2 * ((size_t)blockIdx.x + i); };
  // the maximum first: the sums over the parts are then independent loads
  float m = kNegInf, l = 0.f;
#pragma unroll 4
  for (int i = 0; i < it.parts; ++i) m = fmaxf(m, wk.ml[slot(i) * ROWS + r].x);
  const float mu = m == kNegInf ? 0.f : m;
  float4 acc[CPT];
#pragma unroll
  for (int c = 0; c < CPT; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < it.parts; ++i) {
    const float2 ml = wk.ml[slot(i) * ROWS + r];
    const float4* o = reinterpret_cast<const float4*>(wk.o) + (slot(i) * (D / 4) + c0) * ROWS + r;
    const float e = fast_exp2(ml.x - mu);
    l += ml.y * e;
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const float4 v = o[c * 2048];
      acc[c].x += v.x * e;
      acc[c].y += v.y * e;
      acc[c].z += v.z * e;
      acc[c].w += v.w * e;
    }
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  __nv_bfloat16* dst = p.O + ((size_t)(b * p.Hkv + it.hk) * p.G * p.N + R) * D + 4 * c0;
#pragma unroll
  for (int c = 0; c < CPT; ++c)
    *reinterpret_cast<uint2*>(dst + c * (4 * 2048 / ROWS)) =
        make_uint2(pack_bf16x2(acc[c].x * inv, acc[c].y * inv), pack_bf16x2(acc[c].z * inv, acc[c].w * inv));
}

// The same for few items, whose parts are many: grid (CTAs of the forward,
// ROWS / 32 * D / 16), a block 32 rows and four groups of four channels, its
// eight warps sharing the parts (one item in 40 parts: 23 us the other way).
template <int D, int ROWS>
__global__ void __launch_bounds__(256) paged_join_parts_kernel(const PagedParams p, const PagedWork wk, int row_tiles) {
  __shared__ float4 acc_sh[8][4][32];
  __shared__ float2 ml_sh[8][32];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const SplitItem it = wk.split[blockIdx.x];
  if (it.parts <= 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = it.idx / row_tiles, rt = it.idx - b * row_tiles;
  const SeqLen s = seq_clamped(p, b);
  const int r = (blockIdx.y % (ROWS / 32)) * 32 + lane, c0 = blockIdx.y / (ROWS / 32) * 4;
  const int R = rt * ROWS + r;
  const bool written = R < p.G * p.N && R - fdiv(R, p.f_n) * p.N < s.n;
  if (!__any_sync(0xffffffffu, written)) return;  // the same rows in every warp of the block
  auto slot = [&](int i) -> size_t { return i == 0 ? 2 * (size_t)blockIdx.x + 1 : 2 * ((size_t)blockIdx.x + i); };
  // each warp's own parts against their own maximum, then the warps' sums
  float m = kNegInf, l = 0.f;
  if (written)
#pragma unroll 8
    for (int i = warp; i < it.parts; i += 8) m = fmaxf(m, wk.ml[slot(i) * ROWS + r].x);
  const float mu = m == kNegInf ? 0.f : m;
  float4 acc[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (written)
#pragma unroll 4
    for (int i = warp; i < it.parts; i += 8) {
      const float2 ml = wk.ml[slot(i) * ROWS + r];
      const float4* o = reinterpret_cast<const float4*>(wk.o) + (slot(i) * (D / 4) + c0) * ROWS + r;
      const float e = fast_exp2(ml.x - mu);
      l += ml.y * e;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 v = o[c * ROWS];
        acc[c].x += v.x * e;
        acc[c].y += v.y * e;
        acc[c].z += v.z * e;
        acc[c].w += v.w * e;
      }
    }
#pragma unroll
  for (int c = 0; c < 4; ++c) acc_sh[warp][c][lane] = acc[c];
  ml_sh[warp][lane] = make_float2(m, l);
  __syncthreads();
  if (warp >= 4 || !written) return;  // warp c finishes channel group c
  float M = kNegInf;
#pragma unroll
  for (int w = 0; w < 8; ++w) M = fmaxf(M, ml_sh[w][lane].x);
  const float Mu = M == kNegInf ? 0.f : M;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float e = fast_exp2(ml_sh[w][lane].x - Mu);
    const float4 v = acc_sh[w][warp][lane];
    x.x += v.x * e;
    x.y += v.y * e;
    x.z += v.z * e;
    x.w += v.w * e;
    l += ml_sh[w][lane].y * e;
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  *reinterpret_cast<uint2*>(p.O + ((size_t)(b * p.Hkv + it.hk) * p.G * p.N + R) * D + 4 * (c0 + warp)) =
      make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
}

template <int D, bool E4M3, bool SPLIT>
static cudaError_t launch_tiles_d(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                  const PagedParams& p, const PagedWork& w, int row_tiles, int grid,
                                  cudaStream_t stream) {
  using C = TilesCfg<D, E4M3, SPLIT>;
  auto fn = paged_tiles_kernel<D, E4M3, SPLIT>;
  static DeviceOnce once;
  cudaError_t e = once.run([&]() -> cudaError_t {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::ALLOC);
  });
  if (e != cudaSuccess) return e;
  // (a dependent launch gains nothing here: a CTA takes an SM of its own)
  fn<<<grid, C::THREADS, C::ALLOC, stream>>>(q, k, v, p, w, row_tiles);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (p.whole_items) return cudaSuccess;
  constexpr int ROWS = SPLIT ? 128 : 256;
  if ((long long)p.B * p.Hkv * row_tiles * 8 <= grid)  // eight parts an item, or more
    return launch_after(paged_join_parts_kernel<D, ROWS>, dim3(grid, ROWS / 32 * (D / 16)), 256, 0, stream, p, w, row_tiles);
  return launch_after(paged_join_tiles_kernel<D, ROWS>, dim3(grid, 8), 256, 0, stream, p, w, row_tiles);
}

template <int D, bool E4M3>
static cudaError_t launch_tiles_any(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                    const PagedParams& p, const PagedWork& w, int rows, int row_tiles, int grid,
                                    cudaStream_t stream) {
  return rows == 128 ? launch_tiles_d<D, E4M3, true>(q, k, v, p, w, row_tiles, grid, stream)
                     : launch_tiles_d<D, E4M3, false>(q, k, v, p, w, row_tiles, grid, stream);
}

cudaError_t launch_paged_tiles(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedParams& p,
                               const PagedWork& w, int rows, int row_tiles, int grid, cudaStream_t stream) {
  if (p.d == 64)
    return p.e4m3 ? launch_tiles_any<64, true>(q, k, v, p, w, rows, row_tiles, grid, stream)
                  : launch_tiles_any<64, false>(q, k, v, p, w, rows, row_tiles, grid, stream);
  return p.e4m3 ? launch_tiles_any<128, true>(q, k, v, p, w, rows, row_tiles, grid, stream)
                : launch_tiles_any<128, false>(q, k, v, p, w, rows, row_tiles, grid, stream);
}

}  // namespace bsa
