// Attention of new queries over the paged 8-bit cache:
//   s_i = q . (k8_i ks) / sqrt(d),  out = sum_i softmax(s)_i v8_i vs,  lse = log sum_i exp(s_i)
// over the tokens at positions <= the query's of the listed blocks (or all).
#include <cuda_fp8.h>
#include <math_constants.h>

#include "cache.cuh"

namespace moba {
namespace cache {
namespace {

template <int KIND>
__device__ __forceinline__ float decode8(uint8_t x) {
  if constexpr (KIND == 0) return __half2float(__half(__nv_cvt_fp8_to_halfraw(x, __NV_E4M3)));
  else return (float)(int8_t)x;
}

// One warp per (token, query head), one key at a time.
template <int KIND, int D>
__global__ void __launch_bounds__(128)
attn_simple_kernel(View c, Plan p, const bf16* __restrict__ q, int h_q, const int32_t* __restrict__ sel, int topk,
                   bf16* __restrict__ out, float* __restrict__ lse, int32_t* status) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= (long long)p.T * h_q) return;
  const int t = (int)(item / h_q), h = (int)(item % h_q);
  const int row = __ldg(p.row + t);
  if (row < 0 || row >= c.rows) return;
  int pos = __ldg(p.pos + t);
  const int len = c.state[2 * row], held = c.state[2 * row + 1];
  if (pos >= 0 && (pos >= len || pos / c.B >= held)) {
    if (lane == 0) set_status(status, kStatusBadTable);
    pos = -1;
  }
  const int own = pos < 0 ? -1 : pos / c.B;
  const int head = h / (h_q / c.h_kv);
  float qr[E], o[E], m = -CUDART_INF_F, l = 0.f;
  for (int i = 0; i < E; ++i) {
    qr[i] = __bfloat162float(q[(size_t)item * D + lane * E + i]) * rsqrtf((float)D);
    o[i] = 0.f;
  }
  const int32_t* list = sel ? sel + (size_t)item * topk : nullptr;
  const int count = pos < 0 ? 0 : (list ? topk : own + 1);
  int prev = -1;
  for (int e = 0; e < count; ++e) {
    const int j = list ? __ldg(list + e) : e;
    if (j == -1) continue;
    if (j <= prev || j > own) {
      if (lane == 0) set_status(status, kStatusBadSelIdx);
      continue;
    }
    prev = j;
    const bool full = (j + 1) * c.B <= len;
    const int pg = block_page(c, row, j);
    if (pg < 0) {
      if (lane == 0) set_status(status, kStatusBadTable);
      continue;
    }
    const size_t at = (size_t)pg * c.h_kv + head;
    const size_t tl = (((size_t)row * 2 + (j & 1)) * c.h_kv + head) * c.B * D;
    const int n = min(c.B, pos - j * c.B + 1);
    for (int i = 0; i < n; ++i) {
      float s = 0.f, vv[E];
      for (int x = 0; x < E; ++x) {
        const size_t el = (size_t)i * D + lane * E + x;
        const float kk = full ? decode8<KIND>(c.k[at * c.B * D + el]) * c.k_scale[at] : __bfloat162float(c.tail_k[tl + el]);
        vv[x] = full ? decode8<KIND>(c.v[at * c.B * D + el]) * c.v_scale[at] : __bfloat162float(c.tail_v[tl + el]);
        s += qr[x] * kk;
      }
      for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(~0u, s, off);
      const float mn = fmaxf(m, s);
      const float a = mn == -CUDART_INF_F ? 1.f : __expf(m - mn), w = mn == -CUDART_INF_F ? 0.f : __expf(s - mn);
      l = l * a + w;
      for (int x = 0; x < E; ++x) o[x] = o[x] * a + w * vv[x];
      m = mn;
    }
  }
  for (int x = 0; x < E; ++x) out[(size_t)item * D + lane * E + x] = __float2bfloat16_rn(l > 0.f ? o[x] / l : (l == 0.f ? 0.f : l));
  if (lane == 0) lse[item] = m + logf(l);
}

}  // namespace

size_t attn_scratch(const View&, int, int) { return 0; }

cudaError_t launch_attention(const View& c, const Plan& p, const bf16* q, int h_q, const int32_t* sel, int topk,
                             bf16* out, float* lse, void* scratch, int32_t* status, cudaStream_t st) {
  const long long items = (long long)p.T * h_q;
  const unsigned grid = (unsigned)((items + 3) / 4);
#define LAUNCH(KIND, D) attn_simple_kernel<KIND, D><<<grid, 128, 0, st>>>(c, p, q, h_q, sel, topk, out, lse, status)
  if (c.kind == 0) {
    if (c.d == 64) LAUNCH(0, 64); else LAUNCH(0, 128);
  } else {
    if (c.d == 64) LAUNCH(1, 64); else LAUNCH(1, 128);
  }
#undef LAUNCH
  return cudaGetLastError();
}

}  // namespace cache
}  // namespace moba
