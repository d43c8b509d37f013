// kv_api.cu -- the C ABI of the plain paged cache (include/deltakv.h):
// workspace layout, validation, dispatch.
#include <algorithm>
#include <cstdint>

#include "internal.h"

using namespace dkv;

namespace dkv {

KvWorkspace kv_workspace(const Plan& p, int max_len) {
  const auto& c = p.cfg;
  const int64_t BH = (int64_t)c.batch * c.kv_heads;
  KvWorkspace w{};
  size_t off = kErrBytes;
  w.part = off;
  off = align256(off + (size_t)kKvMaxGrid * 2 * kv_part_floats(p.G, c.d_h) * 4);
  w.norm = off;
  off = align256(off + (size_t)(BH * p.G) * 8);
  w.attend_end = off;
  w.dots = off;
  w.weights_end = align256(off + (size_t)(BH * max_len * p.G) * 4);
  off = kErrBytes;
  w.count = off;
  off = align256(off + (size_t)BH * 4);
  w.hole = off;  // at most half of a pair's rows move
  off = align256(off + (size_t)(BH * (max_len / 2)) * 4);
  w.move = off;
  off = align256(off + (size_t)(BH * (max_len / 2)) * 4);
  w.evict_end = off;
  return w;
}

}  // namespace dkv

namespace {

bool aligned(const void* ptr, uintptr_t n) { return ((uintptr_t)ptr & (n - 1)) == 0; }

// Rows of d elements at b * sb + h * sh share none: one stride steps over all rows of the other.  (A stride of a
// dimension of one counts for nothing.)
bool rows_apart(int64_t B, int64_t H, int64_t sb, int64_t sh, int64_t d) {
  if (B == 1 || H == 1) return (B == 1 || sb >= d) && (H == 1 || sh >= d);
  return (sh >= d && (sb - d) / sh >= H - 1) || (sb >= d && (sh - d) / sb >= B - 1);
}

deltakv_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DELTAKV_OK : DELTAKV_ERR_CUDA; }

// log2 of a page's rows, or -1 where the size is not built
int page_log_of(int32_t tokens_per_page) {
  for (int l = 4; l <= 8; ++l)
    if (tokens_per_page == 1 << l) return l;
  return -1;
}

deltakv_status check_pool(int32_t n_pages, int32_t tokens_per_page) {
  if (n_pages < 1) return DELTAKV_ERR_INVALID_ARG;
  if (page_log_of(tokens_per_page) < 0) return DELTAKV_ERR_UNSUPPORTED;
  if ((int64_t)n_pages * tokens_per_page > INT32_MAX) return DELTAKV_ERR_UNSUPPORTED;
  return DELTAKV_OK;
}

// Check what every kv call shares and build the kernels' view.
deltakv_status make_view(const Plan& p, const deltakv_kv_cache* c, void* workspace, KvView& v) {
  if (!c || !c->pool || !c->page_table || !c->lens || !workspace) return DELTAKV_ERR_INVALID_ARG;
  deltakv_status st = check_pool(c->n_pages, c->tokens_per_page);
  if (st != DELTAKV_OK) return st;
  if (c->max_len < 1 || c->max_len > p.cfg.max_T) return DELTAKV_ERR_INVALID_ARG;
  // the kernels count 16-row units of all pairs, and 1024-row blocks of a grid, in 32 bits; a warp's look ahead
  // reaches up to two batches of eight by 32 units past the last
  constexpr int64_t kMostUnits = INT32_MAX - 1024;
  if ((int64_t)p.cfg.batch * p.cfg.kv_heads > (INT32_MAX >> 4) ||
      (int64_t)p.cfg.batch * p.cfg.kv_heads * ceil_div64(c->max_len, 16) > kMostUnits)
    return DELTAKV_ERR_UNSUPPORTED;
  if (c->max_pages < ceil_div64(c->max_len, c->tokens_per_page)) return DELTAKV_ERR_INVALID_ARG;
  if (!aligned(c->pool, 16) || !aligned(workspace, 16) || !aligned(c->page_table, 4) || !aligned(c->lens, 4))
    return DELTAKV_ERR_ALIGNMENT;
  v.k = (char*)c->pool;
  v.v = v.k + (size_t)c->n_pages * c->tokens_per_page * p.cfg.d_h * p.esize;
  v.ptab = c->page_table;
  v.lens = c->lens;
  v.n_pages = c->n_pages;
  v.page_log = page_log_of(c->tokens_per_page);
  v.max_pages = c->max_pages;
  v.max_len = c->max_len;
  v.err = (uint32_t*)workspace;
  return DELTAKV_OK;
}

}  // namespace

extern "C" {

deltakv_status deltakv_kv_pool_layout(deltakv_plan_t plan, int32_t n_pages, int32_t tokens_per_page,
                                      int32_t max_len, deltakv_kv_layout* out) {
  if (!plan || !out) return DELTAKV_ERR_INVALID_ARG;
  const Plan& p = plan->p;
  deltakv_status st = check_pool(n_pages, tokens_per_page);
  if (st != DELTAKV_OK) return st;
  if (max_len < 1 || max_len > p.cfg.max_T) return DELTAKV_ERR_INVALID_ARG;
  const size_t plane = (size_t)n_pages * tokens_per_page * p.cfg.d_h * p.esize;
  const KvWorkspace w = kv_workspace(p, max_len);
  out->k_offset = 0;
  out->v_offset = plane;
  out->pool_bytes = 2 * plane;
  out->workspace_bytes = std::max(w.attend_end, w.evict_end);
  out->weights_workspace_bytes = std::max(out->workspace_bytes, w.weights_end);
  return DELTAKV_OK;
}

deltakv_status deltakv_kv_append(deltakv_plan_t plan, const deltakv_kv_cache* cache, int32_t n_new,
                                 const void* K, const void* V, const int64_t kv_strides[3],
                                 const int32_t* n_tokens, const int32_t* first_pos, float* weights,
                                 int32_t* pos, int32_t cap, const float* token_weights,
                                 void* workspace, size_t workspace_bytes, deltakv_stream_t stream) {
  NvtxRange nvtx("deltakv_kv_append");
  if (!plan || n_new < 0) return DELTAKV_ERR_INVALID_ARG;
  if (n_new == 0) return DELTAKV_OK;
  const Plan& p = plan->p;
  KvView v{};
  deltakv_status st = make_view(p, cache, workspace, v);
  if (st != DELTAKV_OK) return st;
  if (!K || !V || !kv_strides || (pos && !first_pos)) return DELTAKV_ERR_INVALID_ARG;
  if ((weights || pos) && cap < cache->max_len) return DELTAKV_ERR_INVALID_ARG;
  if ((int64_t)p.cfg.batch * p.cfg.kv_heads * ceil_div64(n_new, 64) > INT32_MAX) return DELTAKV_ERR_UNSUPPORTED;
  if (workspace_bytes < kErrBytes) return DELTAKV_ERR_WORKSPACE;
  for (int i = 0; i < 3; ++i)
    if (kv_strides[i] < 0 || (kv_strides[i] * p.esize) % 16 != 0) return DELTAKV_ERR_ALIGNMENT;
  if (kv_strides[2] < p.cfg.d_h) return DELTAKV_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(n_tokens, 4) || !aligned(first_pos, 4) ||
      !aligned(weights, 16) || !aligned(pos, 16) || !aligned(token_weights, 4))
    return DELTAKV_ERR_ALIGNMENT;
  const KVView kv{K, V, kv_strides[0], kv_strides[1], kv_strides[2]};
  return from_cuda(launch_kv_append(p, v, n_new, kv, n_tokens, first_pos, weights, pos, cap, token_weights,
                                    (cudaStream_t)stream));
}

deltakv_status deltakv_kv_decode_attention(deltakv_plan_t plan, const deltakv_kv_cache* cache, const void* q,
                                           const int64_t q_strides[2], float* out, const int64_t out_strides[2],
                                           float* lse, float* weights, int32_t cap, float decay, void* workspace,
                                           size_t workspace_bytes, deltakv_stream_t stream) {
  NvtxRange nvtx("deltakv_kv_decode_attention");
  if (!plan) return DELTAKV_ERR_INVALID_ARG;
  const Plan& p = plan->p;
  KvView v{};
  deltakv_status st = make_view(p, cache, workspace, v);
  if (st != DELTAKV_OK) return st;
  if (!q || !q_strides || !out || !out_strides) return DELTAKV_ERR_INVALID_ARG;
  // the comparisons are false for a NaN
  if (weights && (cap < cache->max_len || !(decay >= 0.f && decay <= 3.402823466e38f))) return DELTAKV_ERR_INVALID_ARG;
  const KvWorkspace w = kv_workspace(p, cache->max_len);
  if (workspace_bytes < (weights ? w.weights_end : w.attend_end)) return DELTAKV_ERR_WORKSPACE;
  if (q_strides[0] < 0 || q_strides[1] < 0 || out_strides[0] < 0 || out_strides[1] < 0)
    return DELTAKV_ERR_INVALID_ARG;
  if ((q_strides[0] * p.esize) % 16 || (q_strides[1] * p.esize) % 16 || (out_strides[0] * 4) % 16 ||
      (out_strides[1] * 4) % 16)
    return DELTAKV_ERR_ALIGNMENT;
  if (!rows_apart(p.cfg.batch, p.cfg.q_heads, out_strides[0], out_strides[1], p.cfg.d_h))
    return DELTAKV_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(weights, 16)) return DELTAKV_ERR_ALIGNMENT;
  return from_cuda(launch_kv_attend(p, v, q, q_strides[0], q_strides[1], out, out_strides[0], out_strides[1], lse,
                                    weights, cap, decay, workspace, (cudaStream_t)stream));
}

deltakv_status deltakv_kv_evict(deltakv_plan_t plan, const deltakv_kv_cache* cache, const int32_t* budget,
                                int32_t n_first, int32_t n_recent, const float* weights, const int32_t* pos,
                                float* weights_out, int32_t* pos_out, int32_t cap, int32_t* lens_out,
                                void* workspace, size_t workspace_bytes, deltakv_stream_t stream) {
  NvtxRange nvtx("deltakv_kv_evict");
  if (!plan) return DELTAKV_ERR_INVALID_ARG;
  const Plan& p = plan->p;
  KvView v{};
  deltakv_status st = make_view(p, cache, workspace, v);
  if (st != DELTAKV_OK) return st;
  if (!budget || !weights || !pos || !weights_out || !pos_out || !lens_out) return DELTAKV_ERR_INVALID_ARG;
  if (n_first < 0 || n_recent < 0 || (int64_t)n_first + n_recent > p.cfg.max_T || cap < cache->max_len)
    return DELTAKV_ERR_INVALID_ARG;
  if (workspace_bytes < kv_workspace(p, cache->max_len).evict_end) return DELTAKV_ERR_WORKSPACE;
  if (!aligned(budget, 4) || !aligned(lens_out, 4) || !aligned(weights, 16) || !aligned(pos, 16) ||
      !aligned(weights_out, 16) || !aligned(pos_out, 16))
    return DELTAKV_ERR_ALIGNMENT;
  return from_cuda(launch_kv_evict(p, v, budget, n_first, n_recent, weights, pos, weights_out, pos_out, cap, lens_out,
                                   workspace, (cudaStream_t)stream));
}

}  // extern "C"
