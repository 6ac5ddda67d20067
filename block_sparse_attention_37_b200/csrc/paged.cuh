// The paged key/value cache as the kernels see it, and their launchers.
#pragma once

#include "common.cuh"

namespace bsa {

struct PagedParams {
  int B, H, Hkv, N, d;
  int n_pages, max_pages, page_log2;
  int e4m3;
  uint8_t* k;  // [n_pages, Hkv, page, d], bf16 or e4m3 codes
  uint8_t* v;
  float* k_scale;  // [n_pages, Hkv, page], e4m3 only
  float* v_scale;
  const int32_t* table;   // [B, max_pages]
  const int32_t* kv_len;  // [B]
  const int32_t* n_new;   // [B] or null: N each (append, forward)
  const int32_t* begin;   // [B] or null: 0 each (read)
  __nv_bfloat16* new_k;   // [B, Hkv, N, d]: source of an append, destination of a read
  __nv_bfloat16* new_v;
  FastDiv f_n, f_hkv;
  // forward
  const __nv_bfloat16* Q;  // [B, H, N, d]
  __nv_bfloat16* O;
  int G;                   // query heads a key/value head
  int causal, window;
  int whole_items;         // runs hold whole items: nothing is split
  float scale_log2;        // scale * log2(e)
  uint64_t wait_limit_ns;  // failure detection: as in AttnParams
  int withhold_tile;
};

// A sequence's chunk and cache lengths, clamped to what the arguments hold.
struct SeqLen {
  int n, kv;
  bool bad;
};

__host__ __device__ __forceinline__ SeqLen clamp_lens(const PagedParams& p, int n, int kv) {
  SeqLen s{n, kv, false};
  const long long cap = (long long)p.max_pages << p.page_log2;
  if (kv < 0 || kv > cap) {
    s.bad = true;
    s.kv = kv < 0 ? 0 : (int)cap;
  }
  if (n < 0 || n > p.N) {
    s.bad = true;
    s.n = n < 0 ? 0 : p.N;
  }
  return s;
}

// Lengths and table entries. What the kernel before writes is not read-only
// for the lifetime of a kernel launched as its dependent (launch_after), and
// griddepcontrol.wait orders no load of the read-only path: such kernels read
// by ordinary loads. READ_ONLY is for kernels launched the plain way.
constexpr bool kReadOnly = true;
template <bool READ_ONLY>
__device__ __forceinline__ int load_i32(const int32_t* a) {
  return READ_ONLY ? __ldg(a) : *a;
}

template <bool READ_ONLY = false>
__device__ __forceinline__ SeqLen seq_clamped(const PagedParams& p, int b) {
  return clamp_lens(p, p.n_new ? load_i32<READ_ONLY>(p.n_new + b) : p.N, load_i32<READ_ONLY>(p.kv_len + b));
}

template <bool READ_ONLY = false>
__device__ __forceinline__ SeqLen seq_lens(const PagedParams& p, int b) {
  const SeqLen s = seq_clamped<READ_ONLY>(p, b);
  if (s.bad) record_error(BSA_DEVERR_BAD_INDEX);
  return s;
}

// The page of position j of sequence b (j inside the table's row); -1, with
// the fault recorded, for an index outside the cache.
__device__ __forceinline__ int page_of(const PagedParams& p, int b, int j) {
  const int pg = p.table[(size_t)b * p.max_pages + (j >> p.page_log2)];
  if (pg < 0 || pg >= p.n_pages) {
    record_error(BSA_DEVERR_BAD_INDEX);
    return -1;
  }
  return pg;
}

// The same in two steps, for producers that look a tile ahead: the entry is
// read early and checked when the copy goes out; an index outside the cache
// is recorded and page 0 read in its place.
template <bool READ_ONLY = false>
__device__ __forceinline__ int table_entry(const PagedParams& p, int b, int j) {
  return load_i32<READ_ONLY>(p.table + (size_t)b * p.max_pages + (j >> p.page_log2));
}
__device__ __forceinline__ int checked_page(const PagedParams& p, int entry) {
  if (entry >= 0 && entry < p.n_pages) return entry;
  record_error(BSA_DEVERR_BAD_INDEX);
  return 0;
}

// Row (token and head) index of slot j % page of page pg: rows hold d values.
__host__ __device__ __forceinline__ long long cache_row(const PagedParams& p, int pg, int hk, int j) {
  return (((long long)pg * p.Hkv + hk) << p.page_log2) + (j & ((1 << p.page_log2) - 1));
}

#ifdef __CUDACC__
// A launch that may be scheduled while the kernel before it finishes; every
// kernel launched so waits (griddepcontrol.wait) before it reads memory, and
// reads by ordinary loads (see load_i32).
template <class K, class... A>
static cudaError_t launch_after(K kernel, dim3 grid, unsigned block, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

cudaError_t launch_paged_append(const PagedParams& p, cudaStream_t stream);
cudaError_t launch_paged_read(const PagedParams& p, cudaStream_t stream);
struct PagedWork;
// The forward for G * N <= 16: k and v map the pages in boxes of one 64-key
// tile's part of a page; grid = persistent CTAs.
cudaError_t launch_paged_rows(const CUtensorMap& k, const CUtensorMap& v, const PagedParams& p, const PagedWork& w,
                              int grid, cudaStream_t stream);
// The forward for more rows: items of `rows` (128 or 256) packed rows, q maps
// [B * Hkv, G * N, d].
cudaError_t launch_paged_tiles(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PagedParams& p,
                               const PagedWork& w, int rows, int row_tiles, int grid, cudaStream_t stream);

}  // namespace bsa
