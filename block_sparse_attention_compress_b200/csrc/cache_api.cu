// C entries of the paged cache: argument checks and launches.  See include/nsa.h for the contract.
#include <cmath>
#include <cstdint>

#include "../../include/nsa.h"
#include "kernels.h"

static_assert(nsa::kErrCache == NSA_CODE_CACHE, "one code for a skipped token");

namespace {

constexpr int64_t kMaxCapacity = int64_t(1) << 30;   // tokens per sequence: positions and tile ends stay in 32 bits
constexpr int kMaxGroup = 16, kMaxNew = 16;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The cache's description, and with `pools` its pointers.
nsa_status check_cache(const nsa_cache* c, bool pools) {
  if (!c) return NSA_ERR_INVALID_ARG;
  if (c->format != NSA_CACHE_BF16 && c->format != NSA_CACHE_INT4) return NSA_ERR_INVALID_ARG;
  if (c->batch < 1 || c->h_kv < 1 || c->d_k < 1 || c->d_v < 1 || c->page_size < 1 || c->n_pages < 1 ||
      c->max_pages < 1)
    return NSA_ERR_INVALID_ARG;
  if (!((c->d_k == 64 && c->d_v == 64) || (c->d_k == 128 && c->d_v == 128) || (c->d_k == 192 && c->d_v == 128)))
    return NSA_ERR_UNSUPPORTED;
  if (c->batch > 65535 || c->h_kv > 65535) return NSA_ERR_UNSUPPORTED;
  if (c->page_size % 16 && (c->max_pages > 1 || c->format == NSA_CACHE_INT4)) return NSA_ERR_UNSUPPORTED;
  if ((int64_t)c->max_pages * c->page_size > kMaxCapacity) return NSA_ERR_UNSUPPORTED;
  if (!pools) return NSA_OK;
  if (!c->k || !c->v || !c->page_table || !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4) ||
      !aligned(c->status, 4))
    return NSA_ERR_INVALID_ARG;
  if (c->format == NSA_CACHE_INT4 &&
      (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)))
    return NSA_ERR_INVALID_ARG;
  return NSA_OK;
}

nsa::CacheArgs cache_args(const nsa_cache* c) {
  nsa::CacheArgs a{};
  a.k = c->k; a.v = c->v; a.k_scale = c->k_scale; a.v_scale = c->v_scale;
  a.page_table = c->page_table; a.status = c->status;
  a.batch = c->batch; a.h_kv = c->h_kv; a.dk = c->d_k; a.dv = c->d_v;
  a.page_size = c->page_size; a.n_pages = c->n_pages; a.max_pages = c->max_pages;
  a.int4 = c->format == NSA_CACHE_INT4;
  return a;
}

// The rows an append or a read names; rows out.
nsa_status check_rows(const nsa_cache* c, const int32_t* seqlens, const int32_t* cu, int32_t n_new, int32_t total,
                      nsa::RowsArgs* r) {
  if (!seqlens || !aligned(seqlens, 4) || !aligned(cu, 4)) return NSA_ERR_INVALID_ARG;
  if (cu ? total < 1 : n_new < 1) return NSA_ERR_INVALID_ARG;
  const int64_t rows = cu ? total : (int64_t)c->batch * n_new;
  if (rows > INT32_MAX) return NSA_ERR_UNSUPPORTED;
  r->seqlens = seqlens; r->cu = cu; r->n_new = cu ? 0 : n_new; r->rows = (int)rows;
  return NSA_OK;
}

nsa_status check_attention(const nsa_cache* c, const nsa_cache_attention_args* a, bool pools) {
  nsa_status st = check_cache(c, pools);
  if (st != NSA_OK) return st;
  if (!a || a->n_new < 1 || a->h_q < 1 || a->h_q % c->h_kv || a->max_seqlen < 1 || a->window < 0)
    return NSA_ERR_INVALID_ARG;
  if (a->max_seqlen > (int64_t)c->max_pages * c->page_size) return NSA_ERR_INVALID_ARG;
  if (!(a->softmax_scale >= 0.f) || std::isinf(a->softmax_scale) || !(a->softcap >= 0.f) || std::isinf(a->softcap))
    return NSA_ERR_INVALID_ARG;
  if (a->n_new > kMaxNew || a->h_q / c->h_kv > kMaxGroup) return NSA_ERR_UNSUPPORTED;
  return NSA_OK;
}

nsa::CacheAttnArgs attention_args(const nsa_cache* c, const nsa_cache_attention_args* a) {
  nsa::CacheAttnArgs r{};
  r.seqlens = a->seqlens; r.slopes = a->slopes; r.lse = a->lse; r.workspace = a->workspace;
  r.scale = a->softmax_scale > 0.f ? a->softmax_scale : 1.f / std::sqrt((float)c->d_k);
  // a cap above 2^100 leaves every score that a softmax can tell apart as it is
  r.softcap = a->softcap < 0x1p100f ? a->softcap : 0.f;
  r.inv_softcap = r.softcap > 0.f ? std::fmin(1.f / r.softcap, 3e38f) : 0.f;
  r.n_new = a->n_new; r.h_q = a->h_q; r.G = a->h_q / c->h_kv; r.max_seqlen = a->max_seqlen;
  r.window = a->window < a->max_seqlen ? a->window : 0;   // reaches every token: none
  return r;
}

nsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? NSA_OK : NSA_ERR_CUDA; }

}  // namespace

extern "C" {

nsa_status nsa_cache_append(const nsa_cache* cache, const nsa_cache_append_args* a, void* stream) {
  nsa_status st = check_cache(cache, true);
  if (st != NSA_OK) return st;
  if (!a || !a->k || !a->v || !aligned(a->k, 16) || !aligned(a->v, 16)) return NSA_ERR_INVALID_ARG;
  nsa::RowsArgs r{};
  st = check_rows(cache, a->seqlens, a->cu_seqlens, a->n_new, a->total_tokens, &r);
  if (st != NSA_OK) return st;
  if (a->k_stride < (int64_t)cache->h_kv * cache->d_k || a->v_stride < (int64_t)cache->h_kv * cache->d_v ||
      a->k_stride % 8 || a->v_stride % 8)
    return NSA_ERR_INVALID_ARG;
  if (a->cos_sin && (!aligned(a->cos_sin, 16) || a->n_positions < 1 || a->rot_dim < 16 || a->rot_dim % 16 ||
                     a->rot_dim > cache->d_k || (a->interleaved != 0 && a->interleaved != 1)))
    return NSA_ERR_INVALID_ARG;
  if ((a->q != nullptr) != (a->q_out != nullptr)) return NSA_ERR_INVALID_ARG;
  if (a->q && (!aligned(a->q, 16) || !aligned(a->q_out, 16) || a->h_q < 1 || a->h_q > 65535 ||
               a->q_stride < (int64_t)a->h_q * cache->d_k || a->q_stride % 8))
    return NSA_ERR_INVALID_ARG;
  nsa::AppendArgs p{};
  p.k = a->k; p.v = a->v; p.q = a->q; p.q_out = a->q_out; p.cos_sin = a->cos_sin;
  p.k_stride = a->k_stride; p.v_stride = a->v_stride; p.q_stride = a->q_stride;
  p.n_positions = a->n_positions; p.rot = a->rot_dim; p.interleaved = a->interleaved; p.h_q = a->h_q;
  return from_cuda(nsa::launch_cache_append(cache_args(cache), r, p, static_cast<cudaStream_t>(stream)));
}

nsa_status nsa_cache_read(const nsa_cache* cache, const int32_t* seqlens, const int32_t* cu_seqlens, int32_t n_new,
                          int32_t total_tokens, void* k_out, void* v_out, void* stream) {
  nsa_status st = check_cache(cache, true);
  if (st != NSA_OK) return st;
  if (!k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16)) return NSA_ERR_INVALID_ARG;
  nsa::RowsArgs r{};
  st = check_rows(cache, seqlens, cu_seqlens, n_new, total_tokens, &r);
  if (st != NSA_OK) return st;
  return from_cuda(nsa::launch_cache_read(cache_args(cache), r, k_out, v_out, static_cast<cudaStream_t>(stream)));
}

size_t nsa_cache_attention_workspace(const nsa_cache* cache, const nsa_cache_attention_args* args) {
  if (check_attention(cache, args, false) != NSA_OK) return 0;
  return nsa::cache_attn_workspace(cache_args(cache), attention_args(cache, args));
}

nsa_status nsa_cache_attention(const nsa_cache* cache, const void* q, const nsa_cache_attention_args* a, void* out,
                               void* stream) {
  nsa_status st = check_attention(cache, a, true);
  if (st != NSA_OK) return st;
  if (!q || !out || !a->seqlens || !aligned(q, 16) || !aligned(out, 16) || !aligned(a->seqlens, 4) ||
      !aligned(a->slopes, 4) || !aligned(a->lse, 4))
    return NSA_ERR_INVALID_ARG;
  const nsa::CacheArgs c = cache_args(cache);
  nsa::CacheAttnArgs r = attention_args(cache, a);
  r.q = q;
  r.out = out;
  const size_t need = nsa::cache_attn_workspace(c, r);
  if (need && (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < need)) return NSA_ERR_WORKSPACE;
  if (!nsa::cache_attn_fits(c, r)) return NSA_ERR_UNSUPPORTED;
  return from_cuda(nsa::launch_cache_attn(c, r, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
