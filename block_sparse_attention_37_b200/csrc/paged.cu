// Writing the paged key/value cache and reading it back: one pass over the
// chunk, bound by the bytes it reads and writes.
//
// A row is one token of one key/value head, d values, held by d / 8 lanes
// (bf16) or d / 16 (e4m3: the copies are short, and finding a row's page and
// converting it would otherwise take more issue slots than the bytes take
// time), K's and V's row of a token side by side in the same lanes, so the page
// lookup is paid once for both. The rows
// of the [B, Hkv, N, d] tensor are numbered flat: a block of consecutive rows
// is contiguous in the tensor and, page by page, in the cache, and a decode
// step's single tokens fill blocks as well as a long prompt does.
#include "paged.cuh"

namespace bsa {

__device__ __forceinline__ float pg_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float pg_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Largest |x| of eight bf16 as an integer of the magnitude's bits: bf16 bits
// order like the values, and NaN comes out above infinity, so a row with a
// value that is not finite shows in the maximum.
__device__ __forceinline__ uint32_t amax_bits8(const uint4& v) {
  uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// The scale and code factor of a row from its largest magnitude (bf16 bits).
__device__ __forceinline__ void row_scale(uint32_t amax_bits, float& s, float& r) {
  const float amax = __uint_as_float(amax_bits << 16);
  if (amax_bits >= 0x7f80u) {  // infinity or NaN in the row
    s = __int_as_float(0x7fc00000);
    r = 0.f;
  } else if (amax < 0x1p-100f) {  // 448 / amax would leave the fp32 range
    s = r = 1.f;
  } else {
    s = __fdiv_rn(amax, 448.f);
    r = __fdiv_rn(448.f, amax);
  }
}

__device__ __forceinline__ uint2 row_codes8(const uint4& v, float r) {
  uint2 o;
  o.x = e4m3x2(pg_lo(v.x) * r, pg_hi(v.x) * r) | (e4m3x2(pg_lo(v.y) * r, pg_hi(v.y) * r) << 16);
  o.y = e4m3x2(pg_lo(v.z) * r, pg_hi(v.z) * r) | (e4m3x2(pg_lo(v.w) * r, pg_hi(v.w) * r) << 16);
  return o;
}

// Two e4m3 codes in the low byte of each half of `w` (sign, exponent and
// mantissa moved to where bf16 has them: 2^-120 of the value) times 2^120:
// exact, subnormal codes included.
__device__ __forceinline__ __nv_bfloat162 e4m3_pair(uint32_t sign, uint32_t mag) {
  const uint32_t w = (sign & 0x80008000u) | (mag & 0x07f007f0u);
  const uint32_t k = 0x7b807b80u;  // bf16 2^120, twice
  return __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&k));
}

// Four codes (bytes 0..3 of w) times s, as bf16 in order.
__device__ __forceinline__ uint2 dequant4(uint32_t w, float s) {
  const float2 e = __bfloat1622float2(e4m3_pair(w << 8, w << 4));  // bytes 0 and 2
  const float2 o = __bfloat1622float2(e4m3_pair(w, w >> 4));       // bytes 1 and 3
  return make_uint2(pack_bf16x2(e.x * s, o.x * s), pack_bf16x2(e.y * s, o.y * s));
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(256) paged_append_kernel(const PagedParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // before any read or write
  constexpr int W = E4M3 ? 2 : 1;  // 16-byte units of bf16 a lane
  constexpr int LANES = D / (8 * W), ROWS = 256 / LANES;
  const int grp = threadIdx.x / LANES, l = threadIdx.x % LANES;
  const long long rows = (long long)p.B * p.Hkv * p.N;
  const long long r = (long long)blockIdx.x * ROWS + grp;
  uint4 k[W], v[W];
#pragma unroll
  for (int w = 0; w < W; ++w) k[w] = v[w] = make_uint4(0u, 0u, 0u, 0u);
  long long dst = -1;
  if (r < rows) {
    const int bh = fdiv((int)r, p.f_n), n = (int)r - bh * p.N;
    const int b = fdiv(bh, p.f_hkv), hk = bh - b * p.Hkv;
    const SeqLen s = seq_lens(p, b);
    if (n < s.n) {
#pragma unroll
      for (int w = 0; w < W; ++w) {
        k[w] = reinterpret_cast<const uint4*>(p.new_k)[(r * LANES + l) * W + w];
        v[w] = reinterpret_cast<const uint4*>(p.new_v)[(r * LANES + l) * W + w];
      }
      // the position by the length as given: one that runs past the table
      // must not move the chunk over tokens that are there
      const long long j = (long long)p.kv_len[b] - s.n + n;
      if (j < 0 || j >= (long long)p.max_pages << p.page_log2) {
        record_error(BSA_DEVERR_BAD_INDEX);
      } else {
        const int pg = page_of(p, b, (int)j);
        if (pg >= 0) dst = cache_row(p, pg, hk, (int)j);
      }
    }
  }
  if constexpr (E4M3) {
    uint32_t mk = max(amax_bits8(k[0]), amax_bits8(k[W - 1])), mv = max(amax_bits8(v[0]), amax_bits8(v[W - 1]));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      mk = max(mk, __shfl_xor_sync(0xffffffffu, mk, o));
      mv = max(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    if (dst < 0) return;
    float sk, rk, sv, rv;
    row_scale(mk, sk, rk);
    row_scale(mv, sv, rv);
    const uint2 k0 = row_codes8(k[0], rk), k1 = row_codes8(k[W - 1], rk);
    const uint2 v0 = row_codes8(v[0], rv), v1 = row_codes8(v[W - 1], rv);
    // a row that is not finite holds zero codes under its NaN scale
    reinterpret_cast<uint4*>(p.k)[dst * LANES + l] = rk == 0.f ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(k0.x, k0.y, k1.x, k1.y);
    reinterpret_cast<uint4*>(p.v)[dst * LANES + l] = rv == 0.f ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(v0.x, v0.y, v1.x, v1.y);
    if (l == 0) {
      p.k_scale[dst] = sk;
      p.v_scale[dst] = sv;
    }
  } else {
    if (dst < 0) return;
    reinterpret_cast<uint4*>(p.k)[dst * LANES + l] = k[0];
    reinterpret_cast<uint4*>(p.v)[dst * LANES + l] = v[0];
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(256) paged_read_kernel(const PagedParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // before any read or write
  constexpr int W = E4M3 ? 2 : 1;
  constexpr int LANES = D / (8 * W), ROWS = 256 / LANES;
  const int grp = threadIdx.x / LANES, l = threadIdx.x % LANES;
  const long long rows = (long long)p.B * p.Hkv * p.N;
  const long long r = (long long)blockIdx.x * ROWS + grp;
  if (r >= rows) return;
  const int bh = fdiv((int)r, p.f_n), n = (int)r - bh * p.N;
  const int b = fdiv(bh, p.f_hkv), hk = bh - b * p.Hkv;
  const int first = p.begin ? p.begin[b] : 0;
  const SeqLen s = clamp_lens(p, 0, p.kv_len[b]);
  if (s.bad || first < 0) record_error(BSA_DEVERR_BAD_INDEX);
  const long long j = (long long)max(first, 0) + n;
  long long src = -1;
  if (j < s.kv) {
    const int pg = page_of(p, b, (int)j);
    if (pg >= 0) src = cache_row(p, pg, hk, (int)j);
  }
  uint4 k[W], v[W];
#pragma unroll
  for (int w = 0; w < W; ++w) k[w] = v[w] = make_uint4(0u, 0u, 0u, 0u);
  if (src >= 0) {
    if constexpr (E4M3) {
      // eight codes of each half row: a lane's stores lie side by side with its
      // neighbours' (16 codes in a row: 86 us for 407 MB, against 65)
      const float sk = p.k_scale[src], sv = p.v_scale[src];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const uint2 ck = reinterpret_cast<const uint2*>(p.k)[(src * W + w) * LANES + l];
        const uint2 cv = reinterpret_cast<const uint2*>(p.v)[(src * W + w) * LANES + l];
        const uint2 k0 = dequant4(ck.x, sk), k1 = dequant4(ck.y, sk);
        const uint2 v0 = dequant4(cv.x, sv), v1 = dequant4(cv.y, sv);
        k[w] = make_uint4(k0.x, k0.y, k1.x, k1.y);
        v[w] = make_uint4(v0.x, v0.y, v1.x, v1.y);
      }
    } else {
      k[0] = reinterpret_cast<const uint4*>(p.k)[src * LANES + l];
      v[0] = reinterpret_cast<const uint4*>(p.v)[src * LANES + l];
    }
  }
#pragma unroll
  for (int w = 0; w < W; ++w) {
    reinterpret_cast<uint4*>(p.new_k)[(r * W + w) * LANES + l] = k[w];
    reinterpret_cast<uint4*>(p.new_v)[(r * W + w) * LANES + l] = v[w];
  }
}

template <int D, bool E4M3>
static cudaError_t launch_copy(bool append, const PagedParams& p, cudaStream_t stream) {
  const long long per = 256 / (D / (E4M3 ? 16 : 8));
  const long long rows = (long long)p.B * p.Hkv * p.N;
  const unsigned grid = (unsigned)((rows + per - 1) / per);
  return append ? launch_after(paged_append_kernel<D, E4M3>, dim3(grid), 256, 0, stream, p)
                : launch_after(paged_read_kernel<D, E4M3>, dim3(grid), 256, 0, stream, p);
}

static cudaError_t launch_copy_any(bool append, const PagedParams& p, cudaStream_t stream) {
  if (p.d == 64) return p.e4m3 ? launch_copy<64, true>(append, p, stream) : launch_copy<64, false>(append, p, stream);
  return p.e4m3 ? launch_copy<128, true>(append, p, stream) : launch_copy<128, false>(append, p, stream);
}

cudaError_t launch_paged_append(const PagedParams& p, cudaStream_t stream) { return launch_copy_any(true, p, stream); }
cudaError_t launch_paged_read(const PagedParams& p, cudaStream_t stream) { return launch_copy_any(false, p, stream); }

}  // namespace bsa
