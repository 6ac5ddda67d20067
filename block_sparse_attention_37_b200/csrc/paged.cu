// Writing the paged key/value cache and reading it back: one pass over the
// chunk, bound by the bytes it reads and writes.
//
// A row is one token of one key/value head, d values. d / 8 lanes hold a row,
// eight values (16 bytes of bf16) a lane, K's and V's row of a token side by
// side in the same lanes, so the page lookup is paid once for both. The rows
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

// U: rows a lane group keeps in flight (see launch_copy_any).
template <int D, bool E4M3, int U>
__global__ void __launch_bounds__(256) paged_append_kernel(const PagedParams p) {
  constexpr int LANES = D / 8;
  constexpr int GROUPS = 256 / LANES;
  const int grp = threadIdx.x / LANES, l = threadIdx.x % LANES;
  const long long rows = (long long)p.B * p.Hkv * p.N;
  const long long r0 = (long long)blockIdx.x * (GROUPS * U) + grp;
  uint4 k[U], v[U];
  long long dst[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long r = r0 + u * GROUPS;
    dst[u] = -1;
    k[u] = v[u] = make_uint4(0u, 0u, 0u, 0u);
    if (r >= rows) continue;
    const int bh = fdiv((int)r, p.f_n), n = (int)r - bh * p.N;
    const int b = fdiv(bh, p.f_hkv), hk = bh - b * p.Hkv;
    const SeqLen s = seq_lens(p, b);
    if (n >= s.n) continue;
    k[u] = __ldg(reinterpret_cast<const uint4*>(p.new_k) + r * LANES + l);
    v[u] = __ldg(reinterpret_cast<const uint4*>(p.new_v) + r * LANES + l);
    const int j = s.kv - s.n + n;
    if (j < 0) {
      record_error(BSA_DEVERR_BAD_INDEX);
      continue;
    }
    const int pg = page_of(p, b, j);
    if (pg >= 0) dst[u] = cache_row(p, pg, hk, j);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if constexpr (E4M3) {
      uint32_t mk = amax_bits8(k[u]), mv = amax_bits8(v[u]);
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) {
        mk = max(mk, __shfl_xor_sync(0xffffffffu, mk, o));
        mv = max(mv, __shfl_xor_sync(0xffffffffu, mv, o));
      }
      if (dst[u] < 0) continue;
      float sk, rk, sv, rv;
      row_scale(mk, sk, rk);
      row_scale(mv, sv, rv);
      // a row that is not finite holds zero codes under its NaN scale
      const uint2 ck = rk == 0.f ? make_uint2(0u, 0u) : row_codes8(k[u], rk);
      const uint2 cv = rv == 0.f ? make_uint2(0u, 0u) : row_codes8(v[u], rv);
      reinterpret_cast<uint2*>(p.k)[dst[u] * LANES + l] = ck;
      reinterpret_cast<uint2*>(p.v)[dst[u] * LANES + l] = cv;
      if (l == 0) {
        p.k_scale[dst[u]] = sk;
        p.v_scale[dst[u]] = sv;
      }
    } else {
      if (dst[u] < 0) continue;
      reinterpret_cast<uint4*>(p.k)[dst[u] * LANES + l] = k[u];
      reinterpret_cast<uint4*>(p.v)[dst[u] * LANES + l] = v[u];
    }
  }
}

template <int D, bool E4M3, int U>
__global__ void __launch_bounds__(256) paged_read_kernel(const PagedParams p) {
  constexpr int LANES = D / 8;
  constexpr int GROUPS = 256 / LANES;
  const int grp = threadIdx.x / LANES, l = threadIdx.x % LANES;
  const long long rows = (long long)p.B * p.Hkv * p.N;
  const long long r0 = (long long)blockIdx.x * (GROUPS * U) + grp;
  long long src[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long r = r0 + u * GROUPS;
    src[u] = -1;
    if (r >= rows) continue;
    const int bh = fdiv((int)r, p.f_n), n = (int)r - bh * p.N;
    const int b = fdiv(bh, p.f_hkv), hk = bh - b * p.Hkv;
    int kv = __ldg(p.kv_len + b);
    int first = p.begin ? __ldg(p.begin + b) : 0;
    const SeqLen s = clamp_lens(p, 0, kv);
    if (s.bad || first < 0) record_error(BSA_DEVERR_BAD_INDEX);
    const long long j = (long long)max(first, 0) + n;
    if (j >= s.kv) continue;
    const int pg = page_of(p, b, (int)j);
    if (pg >= 0) src[u] = cache_row(p, pg, hk, (int)j);
  }
  uint4 k[U], v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    k[u] = v[u] = make_uint4(0u, 0u, 0u, 0u);
    if (src[u] < 0) continue;
    if constexpr (E4M3) {
      const uint2 ck = __ldg(reinterpret_cast<const uint2*>(p.k) + src[u] * LANES + l);
      const uint2 cv = __ldg(reinterpret_cast<const uint2*>(p.v) + src[u] * LANES + l);
      const float sk = __ldg(p.k_scale + src[u]), sv = __ldg(p.v_scale + src[u]);
      const uint2 k0 = dequant4(ck.x, sk), k1 = dequant4(ck.y, sk);
      const uint2 v0 = dequant4(cv.x, sv), v1 = dequant4(cv.y, sv);
      k[u] = make_uint4(k0.x, k0.y, k1.x, k1.y);
      v[u] = make_uint4(v0.x, v0.y, v1.x, v1.y);
    } else {
      k[u] = __ldg(reinterpret_cast<const uint4*>(p.k) + src[u] * LANES + l);
      v[u] = __ldg(reinterpret_cast<const uint4*>(p.v) + src[u] * LANES + l);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long r = r0 + u * GROUPS;
    if (r >= rows) continue;
    reinterpret_cast<uint4*>(p.new_k)[r * LANES + l] = k[u];
    reinterpret_cast<uint4*>(p.new_v)[r * LANES + l] = v[u];
  }
}

template <int D, bool E4M3, int U>
static cudaError_t launch_copy(bool append, const PagedParams& p, cudaStream_t stream) {
  const long long per = 256 / (D / 8) * U;
  const long long rows = (long long)p.B * p.Hkv * p.N;
  const unsigned grid = (unsigned)((rows + per - 1) / per);
  if (append)
    paged_append_kernel<D, E4M3, U><<<grid, 256, 0, stream>>>(p);
  else
    paged_read_kernel<D, E4M3, U><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

// bf16 rows are long enough to fill the memory pipe one a lane group (append of
// 211 MB: 33.6 us with one, 34.2 with two, against 32.6 at the copy bandwidth).
// e4m3 rows have fewer bytes and more between load and store: two, once there
// are rows for every SM (209 MB: 52.4 us with two, 53.9 with one, 57.1 with
// four); one keeps a decode step's 512 rows spread wider (2.2 us against 3.0).
template <int D>
static cudaError_t launch_copy_d(bool append, const PagedParams& p, cudaStream_t stream) {
  if (!p.e4m3) return launch_copy<D, false, 1>(append, p, stream);
  if ((long long)p.B * p.Hkv * p.N < 65536) return launch_copy<D, true, 1>(append, p, stream);
  return launch_copy<D, true, 2>(append, p, stream);
}

static cudaError_t launch_copy_any(bool append, const PagedParams& p, cudaStream_t stream) {
  return p.d == 64 ? launch_copy_d<64>(append, p, stream) : launch_copy_d<128>(append, p, stream);
}

cudaError_t launch_paged_append(const PagedParams& p, cudaStream_t stream) { return launch_copy_any(true, p, stream); }
cudaError_t launch_paged_read(const PagedParams& p, cudaStream_t stream) { return launch_copy_any(false, p, stream); }

}  // namespace bsa
