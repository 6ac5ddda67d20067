// C ABI of the paged cache (include/bsa.h): argument checks and launches. No
// allocation, no host synchronisation, no CPU fallback.
#include <cmath>
#include <cstring>

#include "paged_sched.cuh"

namespace bsa {
namespace {

// The checks every call on a cache shares; fills the parameters they agree on.
int paged_params(const bsa_dims* dims, const bsa_paged_cache* c, PagedParams* out) {
  int st = check_dims(dims);
  if (st != BSA_OK) return st;
  if (!c) return BSA_ERR_INVALID_ARG;
  if (c->kind != BSA_CACHE_BF16 && c->kind != BSA_CACHE_E4M3) return BSA_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->Hkv < 1 || c->max_pages < 1 || c->page < 1 || c->d != dims->d) return BSA_ERR_INVALID_ARG;
  if (!c->k || !c->v || !c->table || !c->kv_len || !aligned16(c->k) || !aligned16(c->v)) return BSA_ERR_INVALID_ARG;
  const bool e4m3 = c->kind == BSA_CACHE_E4M3;
  if (e4m3 && (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale)))
    return BSA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return BSA_ERR_UNSUPPORTED;
  if (c->page < 16 || c->page > 1024 || (c->page & (c->page - 1))) return BSA_ERR_UNSUPPORTED;
  if ((long long)c->max_pages * c->page > (1ll << 30)) return BSA_ERR_UNSUPPORTED;
  if ((long long)dims->B * c->Hkv * dims->N > 0x7fffffffll) return BSA_ERR_UNSUPPORTED;
  if ((long long)c->n_pages * c->Hkv > 0x7fffffffll) return BSA_ERR_UNSUPPORTED;
  PagedParams& p = *out;
  std::memset(&p, 0, sizeof(p));
  p.B = dims->B;
  p.H = dims->H;
  p.Hkv = c->Hkv;
  p.N = dims->N;
  p.d = dims->d;
  p.n_pages = c->n_pages;
  p.max_pages = c->max_pages;
  while ((1 << p.page_log2) < c->page) ++p.page_log2;
  p.e4m3 = e4m3;
  p.k = static_cast<uint8_t*>(c->k);
  p.v = static_cast<uint8_t*>(c->v);
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.table = c->table;
  p.kv_len = c->kv_len;
  p.f_n = make_fastdiv(p.N);
  p.f_hkv = make_fastdiv(p.Hkv);
  return BSA_OK;
}

// The further checks of the forward (everything but Q, O and the workspace).
int paged_forward_params(const bsa_dims* dims, const bsa_paged_cache* c, PagedParams* p) {
  const int st = paged_params(dims, c, p);
  if (st != BSA_OK) return st;
  if (dims->H % c->Hkv != 0) return BSA_ERR_INVALID_ARG;
  if ((long long)dims->B * dims->H * dims->N > 0x7fffffffll) return BSA_ERR_UNSUPPORTED;
  p->G = dims->H / c->Hkv;
  return BSA_OK;
}

// The cache's K or V for TMA, in boxes of a page's part of a `keys`-token
// tile: rows of 128 bytes, 128-byte swizzle (a bf16 token is one or two
// 64-channel halves; e4m3 codes at d = 64 lie two tokens a row). `rows64`:
// e4m3 at d = 64 as rows of 64 bytes, 64-byte swizzle (an MMA operand).
int make_page_map(CUtensorMap* m, const PagedParams& p, const void* base, int keys, bool rows64 = false) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return BSA_ERR_CUDA;
  const int page = 1 << p.page_log2;
  const int box_tokens = page < keys ? page : keys;
  const bool half = p.e4m3 && p.d == 64 && !rows64;  // two tokens a 128-byte row
  const cuuint64_t inner = !p.e4m3 ? p.d : rows64 ? 64 : 128, rows = half ? page / 2 : page;
  const cuuint64_t row_bytes = p.e4m3 ? inner : inner * 2;
  cuuint64_t dims[3] = {inner, rows, (cuuint64_t)p.n_pages * p.Hkv};
  cuuint64_t strides[2] = {row_bytes, rows * row_bytes};
  cuuint32_t box[3] = {p.e4m3 ? (cuuint32_t)inner : 64u, (cuuint32_t)(half ? box_tokens / 2 : box_tokens), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, p.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  rows64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BSA_OK : BSA_ERR_CUDA;
}

// How a forward is cut: rows of an item, keys of a tile, persistent CTAs.
struct PagedCut {
  int rows, keys, row_tiles, grid;
};

PagedCut paged_cut(const PagedParams& p) {
  // Up to 16 rows a key/value head the warp MMAs keep up with HBM; more rows
  // need the tensor core's tiles, 128 rows or 256 an item. Both sides of each
  // switch, 32 sequences of 150 to 8,100 tokens, 8 key/value heads, d = 128:
  // 16 rows 107 us with warp MMAs, 128 in tiles (e4m3 96 and 191); 20 to 128
  // rows 128 to 152 us as an item of 128, 142 to 162 as half an item of 256
  // (e4m3 191 to 212, 234 to 257).
  const long long rows = (long long)p.G * p.N;
  PagedCut c;
  c.rows = rows <= 16 ? 16 : rows <= 128 ? 128 : 256;
  c.keys = c.rows == 16 ? 64 : 128;
  c.row_tiles = ceil_div(rows, c.rows);
  c.grid = (c.rows == 16 ? 2 : 1) * num_sms();
  // Few items of many rows: as many CTAs as give each item the same number, so
  // that items of one length are cut into whole runs and no CTA fills its
  // pipeline for two (32 items of 32 tiles: 27.6 us with 128 CTAs, 31.6 with
  // 148). From two CTAs an item on the idle SMs cost as much; the few-rows
  // kernel is bound by HBM and keeps every CTA.
  const long long items = (long long)p.B * p.Hkv * c.row_tiles;
  if (c.rows != 16 && 4 * items <= c.grid) c.grid = (int)(c.grid / items * items);
  return c;
}

// The items' tiles fit the arithmetic of the line (paged_sched.cuh).
bool paged_line_fits(const PagedParams& p, const PagedCut& c) {
  const double tiles = (double)(((long long)p.max_pages << p.page_log2) / c.keys + 2);
  return (double)p.B * p.Hkv * c.row_tiles * tiles * c.grid < 4e18 && (long long)p.B * c.row_tiles <= 0x7fffffffll;
}

struct PagedLayout {
  size_t split, ml, o, total;
};

PagedLayout paged_layout(const PagedParams& p, const PagedCut& c) {
  PagedLayout L;
  L.split = 0;
  L.ml = align256((size_t)c.grid * sizeof(SplitItem));
  L.o = L.ml + align256((size_t)2 * c.grid * c.rows * sizeof(float2));
  L.total = L.o + (size_t)2 * c.grid * c.rows * p.d * sizeof(float);
  return L;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" {

int bsa_paged_append(const bsa_dims* dims, const void* K, const void* V, const int32_t* n_new,
                     const bsa_paged_cache* cache, void* stream) {
  PagedParams p;
  const int st = paged_params(dims, cache, &p);
  if (st != BSA_OK) return st;
  if (!K || !V || !aligned16(K) || !aligned16(V)) return BSA_ERR_INVALID_ARG;
  p.new_k = static_cast<__nv_bfloat16*>(const_cast<void*>(K));
  p.new_v = static_cast<__nv_bfloat16*>(const_cast<void*>(V));
  p.n_new = n_new;
  return cuda_status(launch_paged_append(p, static_cast<cudaStream_t>(stream)));
}

int bsa_paged_read(const bsa_dims* dims, const bsa_paged_cache* cache, const int32_t* begin, void* K, void* V,
                   void* stream) {
  PagedParams p;
  const int st = paged_params(dims, cache, &p);
  if (st != BSA_OK) return st;
  if (!K || !V || !aligned16(K) || !aligned16(V)) return BSA_ERR_INVALID_ARG;
  p.new_k = static_cast<__nv_bfloat16*>(K);
  p.new_v = static_cast<__nv_bfloat16*>(V);
  p.begin = begin;
  return cuda_status(launch_paged_read(p, static_cast<cudaStream_t>(stream)));
}

size_t bsa_paged_workspace_size(const bsa_dims* dims, const bsa_paged_cache* cache) {
  PagedParams p;
  if (paged_forward_params(dims, cache, &p) != BSA_OK) return 0;
  const PagedCut c = paged_cut(p);
  return paged_line_fits(p, c) ? paged_layout(p, c).total : 0;
}

int bsa_paged_forward(const bsa_dims* dims, const void* Q, const int32_t* n_new, const bsa_paged_cache* cache,
                      int32_t causal, int32_t window, float scale, void* workspace, size_t workspace_bytes,
                      void* O, void* stream) {
  PagedParams p;
  int st = paged_forward_params(dims, cache, &p);
  if (st != BSA_OK) return st;
  const PagedCut c = paged_cut(p);
  if (!paged_line_fits(p, c)) return BSA_ERR_UNSUPPORTED;
  if (!Q || !O || !aligned16(Q) || !aligned16(O)) return BSA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return BSA_ERR_INVALID_ARG;
  if (window < 0 || (window > 0 && !causal)) return BSA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale <= 0.f) return BSA_ERR_INVALID_ARG;
  const PagedLayout L = paged_layout(p, c);
  if (!workspace || workspace_bytes < L.total || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return BSA_ERR_WORKSPACE;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.O = static_cast<__nv_bfloat16*>(O);
  p.n_new = n_new;
  p.causal = causal;
  p.window = window;
  p.scale_log2 = scale * 1.4426950408889634f;
  // Items of at most eight tiles are not worth a split and its join (a token
  // over 437 keys, 16 heads, on the GPU: 8.8 us in one launch, 9.8 us in two).
  // The host knows the table's width, not the lengths: a table for a longer
  // context takes the two launches.
  p.whole_items = ((long long)p.max_pages << p.page_log2) <= 8ll * c.keys;
  p.wait_limit_ns = g_wait_limit_ns.load();
  p.withhold_tile = g_withheld_tile.load();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const PagedWork w{reinterpret_cast<SplitItem*>(ws + L.split), reinterpret_cast<float2*>(ws + L.ml),
                    reinterpret_cast<float*>(ws + L.o)};
  CUtensorMap mk, mv, mq;
  // e4m3 V is converted on its way, 64 keys at a time; K is an operand as it lies
  const bool tiles = c.rows != 16;
  if ((st = make_page_map(&mk, p, p.k, c.keys, tiles && p.e4m3 && p.d == 64)) != BSA_OK) return st;
  if ((st = make_page_map(&mv, p, p.v, p.e4m3 ? 64 : c.keys)) != BSA_OK) return st;
  if (!tiles) return cuda_status(launch_paged_rows(mk, mv, p, w, c.grid, s));
  if ((st = make_map(&mq, Q, (long long)p.B * p.Hkv, p.G * p.N, p.d)) != BSA_OK) return st;
  return cuda_status(launch_paged_tiles(mq, mk, mv, p, w, c.rows, c.row_tiles, c.grid, s));
}

}  // extern "C"
