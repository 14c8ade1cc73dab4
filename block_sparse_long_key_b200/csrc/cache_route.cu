// Routing of new queries over the cached centroids: the topk - 1 earlier
// blocks with the largest q . (hi + lo), ties to the lower block, and the
// query's own block.
#include <math_constants.h>

#include "cache.cuh"

namespace moba {
namespace cache {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ double exact_score(const bf16* q, const bf16* hi, const bf16* lo, int d) {
  double s = 0.0;
  for (int i = 0; i < d; ++i)
    s += (double)__bfloat162float(q[i]) * ((double)__bfloat162float(hi[i]) + (double)__bfloat162float(lo[i]));
  return isnan(s) ? -CUDART_INF : s;
}

// One CTA per (token, query head): every score in 64 bits, then topk - 1
// rounds of an argmax.
__global__ void __launch_bounds__(kThreads)
route_simple_kernel(View c, Plan p, const bf16* __restrict__ q, int h_q, int topk, int32_t* sel, double* score,
                    int32_t* status) {
  __shared__ double best_s[kThreads];
  __shared__ int best_j[kThreads];
  __shared__ int picked[64];
  const int t = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int row = __ldg(p.row + t);
  if (row < 0 || row >= c.rows) return;
  const int pos = __ldg(p.pos + t);
  int32_t* out = sel + ((size_t)t * h_q + h) * topk;
  if (pos < 0 || pos >= c.state[2 * row] || pos / c.B >= c.state[2 * row + 1]) {
    if (pos >= 0 && tid == 0) set_status(status, kStatusBadTable);
    for (int i = tid; i < topk; i += kThreads) out[i] = -1;
    return;
  }
  const int own = pos / c.B;
  const int head = h / (h_q / c.h_kv);
  const bf16* qr = q + ((size_t)t * h_q + h) * c.d;
  double* sc = score + ((size_t)t * h_q + h) * c.max_blocks;
  for (int j = tid; j < own; j += kThreads) {
    const int pg = block_page(c, row, j);
    if (pg < 0) {
      set_status(status, kStatusBadTable);
      sc[j] = -CUDART_INF;
      continue;
    }
    const bf16* hi = c.cent + ((size_t)pg * c.h_kv + head) * c.d;
    sc[j] = exact_score(qr, hi, hi + (size_t)c.n_pages * c.h_kv * c.d, c.d);
  }
  __syncthreads();
  const int want = min(topk - 1, own);
  double last_s = CUDART_INF;
  int last_j = -1;
  for (int i = 0; i < want; ++i) {
    double bs = -CUDART_INF;
    int bj = 1 << 30;
    for (int j = tid; j < own; j += kThreads) {
      const double s = sc[j];
      const bool after = s < last_s || (s == last_s && j > last_j);
      if (after && (s > bs || (s == bs && j < bj))) bs = s, bj = j;
    }
    best_s[tid] = bs, best_j[tid] = bj;
    __syncthreads();
    for (int off = kThreads / 2; off; off >>= 1) {
      if (tid < off && (best_s[tid + off] > best_s[tid] ||
                        (best_s[tid + off] == best_s[tid] && best_j[tid + off] < best_j[tid]))) {
        best_s[tid] = best_s[tid + off];
        best_j[tid] = best_j[tid + off];
      }
      __syncthreads();
    }
    last_s = best_s[0], last_j = best_j[0];
    if (tid == 0) picked[i] = last_j;
    __syncthreads();
  }
  if (tid < topk) {
    int v = -1;
    if (tid < want) {  // ascending: the pick with `tid` smaller ones
      for (int i = 0; i < want; ++i) {
        int below = 0;
        for (int k = 0; k < want; ++k) below += picked[k] < picked[i];
        if (below == tid) v = picked[i];
      }
    } else if (tid == want) {
      v = own;
    }
    out[tid] = v;
  }
}

}  // namespace

size_t route_scratch(const View& c, int T, int h_q) { return (size_t)T * h_q * c.max_blocks * sizeof(double); }

cudaError_t launch_route(const View& c, const Plan& p, const bf16* q, int h_q, int topk, int32_t* sel, void* scratch,
                         int32_t* status, cudaStream_t st) {
  route_simple_kernel<<<dim3(p.T, h_q), kThreads, 0, st>>>(c, p, q, h_q, topk, sel, static_cast<double*>(scratch),
                                                           status);
  return cudaGetLastError();
}

}  // namespace cache
}  // namespace moba
