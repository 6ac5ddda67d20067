// Attention of a chunk's queries over the paged cache: one warp a query row,
// the row's kept keys one after another with an online softmax.
#include "paged.cuh"

namespace bsa {

template <int D, bool E4M3>
__device__ __forceinline__ void paged_vec(const uint8_t* base, const float* scale, long long row, int lane, float* x) {
  constexpr int PER = D / 32;
  if constexpr (E4M3) {
    const float s = __ldg(scale + row);
    const uint8_t* c = base + row * D + lane * PER;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t w = c[i];
      x[i] = __bfloat162float(__low2bfloat16(e4m3_pair(w << 8, w << 4))) * s;
    }
  } else {
    const __nv_bfloat16* c = reinterpret_cast<const __nv_bfloat16*>(base) + row * D + lane * PER;
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = __bfloat162float(c[i]);
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(256) paged_forward_kernel(const PagedParams p) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31;
  const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= (long long)p.B * p.H * p.N) return;
  const int bh = fdiv((int)r, p.f_n), n = (int)r - bh * p.N;
  const int b = bh / p.H, h = bh - b * p.H, hk = h / p.G;
  const SeqLen s = seq_lens(p, b);
  if (n >= s.n) return;
  const int pos = s.kv - s.n + n;
  int hi = s.kv, lo = 0;
  if (p.causal) {
    hi = min(hi, pos + 1);
    if (p.window > 0) lo = max(0, pos - p.window + 1);
  }
  float q[PER], o[PER], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    q[i] = __bfloat162float(p.Q[r * D + lane * PER + i]) * p.scale_log2;
    o[i] = 0.f;
  }
  for (int j = lo; j < hi; ++j) {
    const int pg = max(page_of(p, b, j), 0);
    const long long row = cache_row(p, pg, hk, j);
    float x[PER], z = 0.f;
    paged_vec<D, E4M3>(p.k, p.k_scale, row, lane, x);
#pragma unroll
    for (int i = 0; i < PER; ++i) z = fmaf(q[i], x[i], z);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) z += __shfl_xor_sync(0xffffffffu, z, w);
    const float mn = fmaxf(m, z);
    const float a = exp2f(m - mn), e = exp2f(z - mn);
    m = mn;
    l = l * a + e;
    paged_vec<D, E4M3>(p.v, p.v_scale, row, lane, x);
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = fmaf(e, x[i], o[i] * a);
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
  for (int i = 0; i < PER; ++i) p.O[r * D + lane * PER + i] = __float2bfloat16(o[i] * inv);
}

cudaError_t launch_paged_forward(const PagedParams& p, cudaStream_t stream) {
  const long long rows = (long long)p.B * p.H * p.N;
  const unsigned grid = (unsigned)((rows + 7) / 8);
  if (p.d == 64)
    p.e4m3 ? paged_forward_kernel<64, true><<<grid, 256, 0, stream>>>(p)
           : paged_forward_kernel<64, false><<<grid, 256, 0, stream>>>(p);
  else
    p.e4m3 ? paged_forward_kernel<128, true><<<grid, 256, 0, stream>>>(p)
           : paged_forward_kernel<128, false><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace bsa
