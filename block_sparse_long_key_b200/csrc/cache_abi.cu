// C ABI of the paged 8-bit cache: argument checks, workspace carving and
// launches.  See include/moba.h for the contract.
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "moba.h"
#include "cache.cuh"

using moba::cache::bf16;
using moba::cache::Plan;
using moba::cache::RowPlan;
using moba::cache::View;

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool sizes_ok(const moba_cache* c) {
  if (!c) return false;
  if (c->rows < 1 || c->n_pages < 1 || c->max_blocks < 1 || c->h_kv < 1) return false;
  if (c->head_dim != 64 && c->head_dim != 128) return false;
  if (c->block_size != 16 && c->block_size != 32 && c->block_size != 64 && c->block_size != 128) return false;
  if (c->kind != MOBA_CACHE_E4M3 && c->kind != MOBA_CACHE_INT8) return false;
  if (c->conv_width < 0 || c->conv_width > moba::cache::kMaxWidth) return false;
  if (c->set_back < 0 || c->set_back > moba::cache::kHistRing + 1 - (c->conv_width > 1 ? c->conv_width : 1)) return false;
  if ((long long)c->n_pages * c->block_size >= (1LL << 31)) return false;
  if ((long long)c->max_blocks * c->block_size >= (1LL << 31)) return false;
  if (c->rows > (1 << 24) || c->h_kv > 65535) return false;
  return true;
}

bool step_ok(const moba_cache* c, int total_new, int h_q, int topk) {
  if (total_new < 0 || h_q < 1 || h_q > 65535 || h_q % c->h_kv != 0 || topk < 1 || topk > 64) return false;
  const long long widest = c->head_dim > topk ? c->head_dim : topk;
  return (long long)total_new * h_q * widest < (1LL << 31);
}

int check_ptrs(std::initializer_list<const void*> ps) {
  for (const void* p : ps) {
    if (!p) return MOBA_EINVAL;
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return MOBA_EALIGN;
  }
  return MOBA_OK;
}

int check_ws(const void* ws, size_t have, size_t need) {
  if (!ws) return MOBA_EINVAL;
  if (reinterpret_cast<uintptr_t>(ws) % kAlign != 0) return MOBA_EALIGN;
  return have < need ? MOBA_EWORKSPACE : MOBA_OK;
}

int check_plan(const moba_cache_plan* p) {
  if (!p || p->total_new < 0) return MOBA_EINVAL;
  int rc = check_ptrs({p->cu_new});
  if (rc != MOBA_OK || p->total_new == 0) return rc;
  return check_ptrs({p->token_row, p->token_pos, p->slot_map});
}

// A step without tokens: nothing to do but for the status word, where there is one.
int no_tokens(void* ws, size_t bytes, void* stream) {
  if (!ws) return MOBA_OK;
  const int rc = check_ws(ws, bytes, kAlign);
  if (rc != MOBA_OK) return rc;
  return cudaMemsetAsync(ws, 0, 2 * sizeof(int32_t), static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOBA_OK : MOBA_ELAUNCH;
}

View view_of(const moba_cache* c) {
  View v;
  v.rows = c->rows, v.n_pages = c->n_pages, v.max_blocks = c->max_blocks, v.h_kv = c->h_kv;
  v.d = c->head_dim, v.B = c->block_size, v.kind = c->kind, v.conv_width = c->conv_width;
  v.k = static_cast<uint8_t*>(c->k), v.v = static_cast<uint8_t*>(c->v);
  v.k_scale = c->k_scale, v.v_scale = c->v_scale;
  v.cent = static_cast<bf16*>(c->cent);
  v.tail_k = static_cast<bf16*>(c->tail_k), v.tail_v = static_cast<bf16*>(c->tail_v);
  v.hist = static_cast<bf16*>(c->hist);
  v.table = c->block_table, v.state = c->row_state, v.free_pages = c->free_pages;
  v.ring = reinterpret_cast<long long*>(c->ring);
  return v;
}

Plan plan_of(const moba_cache_plan* p) { return Plan{p->total_new, p->cu_new, p->token_row, p->token_pos, p->slot_map}; }

// Everything that holds keys and values.
int check_store(const moba_cache* c) {
  int rc = check_ptrs({c->k, c->v, c->k_scale, c->v_scale, c->cent, c->tail_k, c->tail_v, c->block_table, c->row_state});
  if (rc == MOBA_OK && c->conv_width > 1) rc = check_ptrs({c->hist});
  return rc;
}

size_t workspace_need(const moba_cache* c, int total_new, int h_q) {
  const View v = view_of(c);
  size_t most = (size_t)c->rows * sizeof(RowPlan);
  const size_t a = moba::cache::route_scratch(v, total_new, h_q), b = moba::cache::attn_scratch(v, total_new, h_q);
  if (a > most) most = a;
  if (b > most) most = b;
  return kAlign + align_up(most);
}

#define MOBA_TRY(expr)                              \
  do {                                              \
    if ((expr) != cudaSuccess) return MOBA_ELAUNCH; \
  } while (0)

}  // namespace

extern "C" {

size_t moba_cache_workspace_size(const moba_cache* cache, int total_new, int h_q) {
  if (!sizes_ok(cache) || !step_ok(cache, total_new, h_q, 1)) return 0;
  return workspace_need(cache, total_new, h_q);
}

int moba_cache_reset(const moba_cache* cache, void* stream) {
  if (!sizes_ok(cache)) return MOBA_EINVAL;
  int rc = check_store(cache);
  if (rc == MOBA_OK) rc = check_ptrs({cache->free_pages, cache->ring});
  if (rc != MOBA_OK) return rc;
  MOBA_TRY(moba::cache::launch_reset(view_of(cache), static_cast<cudaStream_t>(stream)));
  return MOBA_OK;
}

int moba_cache_tables(const moba_cache* cache, const int32_t* new_len, int32_t* row_state_out, int64_t* ring_out,
                      const moba_cache_plan* plan, void* workspace, size_t workspace_bytes, void* stream) {
  if (!sizes_ok(cache)) return MOBA_EINVAL;
  int rc = check_ptrs({cache->block_table, cache->row_state, cache->free_pages, cache->ring, new_len});
  if (rc == MOBA_OK) rc = check_plan(plan);
  if (rc != MOBA_OK) return rc;
  if ((long long)plan->total_new * cache->h_kv * cache->head_dim >= (1LL << 31)) return MOBA_EINVAL;
  if (!row_state_out) row_state_out = cache->row_state;
  if (!ring_out) ring_out = cache->ring;
  if ((rc = check_ptrs({row_state_out, ring_out})) != MOBA_OK) return rc;
  const size_t need = kAlign + align_up((size_t)cache->rows * sizeof(RowPlan));
  if ((rc = check_ws(workspace, workspace_bytes, need)) != MOBA_OK) return rc;
  char* ws = static_cast<char*>(workspace);
  MOBA_TRY(moba::cache::launch_tables(view_of(cache), new_len, row_state_out, reinterpret_cast<long long*>(ring_out),
                                      plan_of(plan), reinterpret_cast<RowPlan*>(ws + kAlign),
                                      reinterpret_cast<int32_t*>(ws), static_cast<cudaStream_t>(stream)));
  return MOBA_OK;
}

int moba_cache_append(const moba_cache* cache, const moba_cache_plan* plan, const void* k, const void* v,
                      const float* conv_w, void* workspace, size_t workspace_bytes, void* stream) {
  if (!sizes_ok(cache)) return MOBA_EINVAL;
  int rc = check_plan(plan);
  if (rc == MOBA_OK) rc = check_store(cache);
  if (rc != MOBA_OK) return rc;
  if ((long long)plan->total_new * cache->h_kv * cache->head_dim >= (1LL << 31)) return MOBA_EINVAL;
  if (plan->total_new == 0) return no_tokens(workspace, workspace_bytes, stream);
  if ((rc = check_ptrs({k, v})) != MOBA_OK) return rc;
  if (cache->conv_width > 0 && (rc = check_ptrs({conv_w})) != MOBA_OK) return rc;
  if ((rc = check_ws(workspace, workspace_bytes, kAlign)) != MOBA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t* status = static_cast<int32_t*>(workspace);
  MOBA_TRY(cudaMemsetAsync(status, 0, 2 * sizeof(int32_t), st));
  MOBA_TRY(moba::cache::launch_append(view_of(cache), plan_of(plan), static_cast<const bf16*>(k),
                                      static_cast<const bf16*>(v), conv_w,
                                      cache->conv_width > 1 ? cache->conv_width - 1 + cache->set_back : 0, status, st));
  return MOBA_OK;
}

int moba_cache_route(const moba_cache* cache, const moba_cache_plan* plan, const void* q, int h_q, int topk,
                     int32_t* sel_idx, void* workspace, size_t workspace_bytes, void* stream) {
  if (!sizes_ok(cache)) return MOBA_EINVAL;
  int rc = check_plan(plan);
  if (rc == MOBA_OK) rc = check_ptrs({cache->cent, cache->block_table, cache->row_state});
  if (rc != MOBA_OK) return rc;
  if (!step_ok(cache, plan->total_new, h_q, topk)) return MOBA_EINVAL;
  if (plan->total_new == 0) return no_tokens(workspace, workspace_bytes, stream);
  if ((rc = check_ptrs({q, sel_idx})) != MOBA_OK) return rc;
  if ((rc = check_ws(workspace, workspace_bytes, workspace_need(cache, plan->total_new, h_q))) != MOBA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  MOBA_TRY(moba::cache::launch_route(view_of(cache), plan_of(plan), static_cast<const bf16*>(q), h_q, topk, sel_idx,
                                     ws + kAlign, reinterpret_cast<int32_t*>(ws), st));
  return MOBA_OK;
}

int moba_cache_attention(const moba_cache* cache, const moba_cache_plan* plan, const void* q, int h_q,
                         const int32_t* sel_idx, int topk, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (!sizes_ok(cache)) return MOBA_EINVAL;
  int rc = check_plan(plan);
  if (rc == MOBA_OK) rc = check_store(cache);
  if (rc != MOBA_OK) return rc;
  if (!step_ok(cache, plan->total_new, h_q, sel_idx ? topk : 1)) return MOBA_EINVAL;
  if (plan->total_new == 0) return no_tokens(workspace, workspace_bytes, stream);
  if ((rc = check_ptrs({q, out, lse})) != MOBA_OK) return rc;
  if (sel_idx && (rc = check_ptrs({sel_idx})) != MOBA_OK) return rc;
  if ((rc = check_ws(workspace, workspace_bytes, workspace_need(cache, plan->total_new, h_q))) != MOBA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  MOBA_TRY(cudaMemsetAsync(ws, 0, 2 * sizeof(int32_t), st));
  MOBA_TRY(moba::cache::launch_attention(view_of(cache), plan_of(plan), static_cast<const bf16*>(q), h_q, sel_idx, topk,
                                         static_cast<bf16*>(out), lse, ws + kAlign, reinterpret_cast<int32_t*>(ws),
                                         st));
  return MOBA_OK;
}

}  // extern "C"
