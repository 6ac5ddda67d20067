// C ABI of the paged cache (include/bsa.h): argument checks and launches. No
// allocation, no host synchronisation, no CPU fallback.
#include <cmath>
#include <cstring>

#include "paged.cuh"

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
  return paged_forward_params(dims, cache, &p) == BSA_OK ? 256 : 0;
}

int bsa_paged_forward(const bsa_dims* dims, const void* Q, const int32_t* n_new, const bsa_paged_cache* cache,
                      int32_t causal, int32_t window, float scale, void* workspace, size_t workspace_bytes,
                      void* O, void* stream) {
  PagedParams p;
  const int st = paged_forward_params(dims, cache, &p);
  if (st != BSA_OK) return st;
  if (!Q || !O || !aligned16(Q) || !aligned16(O)) return BSA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return BSA_ERR_INVALID_ARG;
  if (window < 0 || (window > 0 && !causal)) return BSA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale <= 0.f) return BSA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < bsa_paged_workspace_size(dims, cache) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return BSA_ERR_WORKSPACE;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.O = static_cast<__nv_bfloat16*>(O);
  p.n_new = n_new;
  p.causal = causal;
  p.window = window;
  p.scale_log2 = scale * 1.4426950408889634f;
  return cuda_status(launch_paged_forward(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
