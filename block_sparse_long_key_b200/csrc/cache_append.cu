// Writes new keys and values into the paged 8-bit cache.
//
//   k'_t = bf16(k_t + SiLU(sum_{l < W} w_l (.) k_{t-l}))       (key conv, optional)
//   block complete: s = max(amax / M, 2^-126), x8 = rn(x / s); c = mean k', hi = bf16(c), lo = bf16(c - hi)
//   else: bf16 tail
//
// The unit of work is a run: the new tokens of one row inside one block.  One
// CTA per (run, KV head).  A block that becomes complete is gathered in
// shared memory (its earlier tokens from the tail, the new ones converted),
// its largest magnitude found, and written once in 8 bits.
//
// A row's first run is the only one that may need what the step replaces: the
// tail bank of its block (its earlier tokens) and the raw-key history.  Its
// CTA therefore also does the replacing: it takes the second run along where
// that reads history too (the first run has fewer than W - 1 tokens), then
// writes the tail tokens of the later block that shares its bank, and the
// history, behind a barrier.
#include <cuda_fp8.h>

#include "cache.cuh"

namespace moba {
namespace cache {
namespace {

constexpr int kThreads = 128;

// 8-bit code of x / s (IEEE division, nearest, ties to even).
template <int KIND>
__device__ __forceinline__ uint8_t encode8(float x, float s) {
  const float y = __fdiv_rn(x, s);
  if constexpr (KIND == 0) return (uint8_t)__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  else return (uint8_t)(int8_t)max(-127, min(127, __float2int_rn(y)));
}

struct RowInfo {
  int row, t_begin, t_end;  // the row's new tokens
  int pos0;                 // position of t_begin
  int len;                  // tokens after the step
};

// Channel ch of k' for the row's new token `rel` (fp32 before its rounding to
// bf16).  64-bit sums: k' then does not depend on their order, and neither do
// the 8-bit codes and centroids that follow from it.
__device__ __forceinline__ float conv_key(const View& c, const RowInfo& R, const bf16* k, const float* w, int rel,
                                          int head, int ch) {
  const size_t stride = (size_t)c.h_kv * c.d;
  const float x0 = __bfloat162float(k[(size_t)(R.t_begin + rel) * stride + head * c.d + ch]);
  if (c.conv_width == 0) return x0;
  double z = 0.0;
  for (int l = 0; l < c.conv_width; ++l) {
    const int rl = rel - l;
    float x = 0.f;
    if (rl >= 0) x = __bfloat162float(k[(size_t)(R.t_begin + rl) * stride + head * c.d + ch]);
    else if (R.pos0 + rl >= 0)
      x = __bfloat162float(
          c.hist[(((size_t)R.row * kHistRing + ((R.pos0 + rl) & (kHistRing - 1))) * c.h_kv + head) * c.d + ch]);
    z += (double)w[((size_t)head * c.d + ch) * c.conv_width + l] * (double)x;
  }
  return (float)((double)x0 + z / (1.0 + exp(-z)));
}

__device__ __forceinline__ bf16 finite16(float x, bool* bad) {
  bf16 y = __float2bfloat16_rn(x);
  if (!(fabsf(__bfloat162float(y)) <= 3.4e38f)) {  // NaN or infinite
    *bad = true;
    y = __float2bfloat16_rn(0.f);
  }
  return y;
}

__device__ __forceinline__ bf16* tail_at(bf16* tail, const View& c, int row, int j, int head, int off) {
  return tail + ((((size_t)row * 2 + (j & 1)) * c.h_kv + head) * c.B + off) * c.d;
}

template <int KIND>
__device__ void encode_block(const View& c, const bf16* tile, uint8_t* dst, float* scale, int pg, int head,
                             float* red) {
  const int n = c.B * c.d, tid = threadIdx.x;
  float m = 0.f;
  for (int i = tid; i < n; i += kThreads) m = fmaxf(m, fabsf(__bfloat162float(tile[i])));
  for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, off));
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
  m = red[0];
  for (int i = 1; i < kThreads / 32; ++i) m = fmaxf(m, red[i]);
  const float s = fmaxf(m * (KIND == 0 ? 1.f / 448.f : 1.f / 127.f), 1.17549435e-38f);
  const size_t at = (size_t)pg * c.h_kv + head;
  for (int i = tid; i < n; i += kThreads) dst[at * n + i] = encode8<KIND>(__bfloat162float(tile[i]), s);
  if (tid == 0) scale[at] = s;
  __syncthreads();
}

template <int KIND>
__global__ void __launch_bounds__(kThreads)
append_kernel(View c, Plan p, const bf16* __restrict__ k, const bf16* __restrict__ v, const float* __restrict__ w,
              int per_token, int32_t* status) {
  extern __shared__ __align__(16) unsigned char smem[];
  bf16* tile = reinterpret_cast<bf16*>(smem);  // [B][d]
  __shared__ float red[kThreads / 32];
  const int tid = threadIdx.x, head = blockIdx.y, B = c.B, d = c.d;
  const int u = blockIdx.x;
  const int total = min(__ldg(p.cu + c.rows), p.T);
  // ---- which run
  RowInfo R;
  int first_rel;  // first token of this run, relative to the row's first
  if (per_token) {
    if (u >= total) return;
    R.row = __ldg(p.row + u);
    if ((unsigned)R.row >= (unsigned)c.rows) return;
    R.t_begin = __ldg(p.cu + R.row);
    first_rel = u - R.t_begin;
    if (first_rel < 0) return;
    R.pos0 = __ldg(p.pos + R.t_begin);
    if (first_rel > 0 && (R.pos0 + first_rel) % B != 0) return;
  } else {
    int lo = 0, hi = c.rows;  // largest row with cu / B + 2 row <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu + mid) / B + 2 * mid <= u) lo = mid; else hi = mid;
    }
    R.row = lo;
    R.t_begin = __ldg(p.cu + lo);
    const int i = u - (R.t_begin / B + 2 * lo);  // block number within the row's touched blocks
    if (R.t_begin >= total) return;
    R.pos0 = __ldg(p.pos + R.t_begin);
    if (R.pos0 < 0) return;
    first_rel = i == 0 ? 0 : (R.pos0 / B + i) * B - R.pos0;
  }
  R.t_end = min(__ldg(p.cu + R.row + 1), total);
  const int n = R.t_end - R.t_begin;
  if (R.t_begin < 0) return;
  if (n <= 0 || first_rel >= n || R.pos0 < 0) return;
  R.len = R.pos0 + n;
  if (c.state[2 * R.row] != R.len || (long long)R.len > (long long)c.max_blocks * B) {
    if (tid == 0) set_status(status, kStatusBadTable);
    return;
  }
  const int W = c.conv_width, Wm1 = W > 0 ? W - 1 : 0;
  const int j_first = R.pos0 / B, j_last = (R.len - 1) / B;
  const int n_first = min(n, (j_first + 1) * B - R.pos0);  // tokens of the row's first run
  int j0 = (R.pos0 + first_rel) / B, j1 = j0;
  const bool is_first = j0 == j_first;
  const bool second_along = n_first < Wm1 && n > n_first;  // the second run reads history too
  if (second_along) {
    if (j0 == j_first + 1) return;
    if (is_first) j1 = j_first + 1;
  }
  const bool has_old = R.pos0 % B != 0;
  bool bad = false;
  const size_t stride = (size_t)c.h_kv * d;
  for (int j = j0; j <= j1; ++j) {
    const int lo = max(R.pos0, j * B) - j * B, hi = min(R.len, (j + 1) * B) - j * B;  // new tokens inside the block
    const int rel0 = j * B - R.pos0;
    const bool full = (j + 1) * B <= R.len;
    // A later block in the first block's bank: written by the first run's CTA, below.
    const bool keep = j >= j_last - 1 && !(has_old && j > j_first && ((j ^ j_first) & 1) == 0);
    int pg = -1;
    if (full) {
      const int slot = __ldg(p.slot + R.t_begin + rel0 + lo);
      if (slot >= 0 && slot / B < c.n_pages) pg = slot / B;
      else if (tid == 0) set_status(status, kStatusBadTable);
    }
    for (int kv = 0; kv < 2; ++kv) {
      bf16* tail = kv ? c.tail_v : c.tail_k;
      for (int i = tid; i < hi * d; i += kThreads) {
        const int off = i / d, ch = i % d;
        bf16 x;
        if (off < lo) {
          if (!full) continue;
          x = tail_at(tail, c, R.row, j, head, off)[ch];
        } else {
          const int rel = rel0 + off;
          const float y = kv ? __bfloat162float(v[(size_t)(R.t_begin + rel) * stride + head * d + ch])
                             : conv_key(c, R, k, w, rel, head, ch);
          x = finite16(y, &bad);
          if (keep) tail_at(tail, c, R.row, j, head, off)[ch] = x;
        }
        if (full) tile[i] = x;
      }
      if (!full) continue;
      __syncthreads();
      if (pg >= 0) {
        encode_block<KIND>(c, tile, kv ? c.v : c.k, kv ? c.v_scale : c.k_scale, pg, head, red);
        if (!kv && tid < d) {
          double s = 0.0;  // exact for bf16 keys within 2^40 of one another
          for (int i = 0; i < B; ++i) s += (double)__bfloat162float(tile[i * d + tid]);
          const float m = (float)(s / B);
          const bf16 h = __float2bfloat16_rn(m);
          const size_t at = ((size_t)pg * c.h_kv + head) * d + tid;
          c.cent[at] = h;
          c.cent[(size_t)c.n_pages * c.h_kv * d + at] = __float2bfloat16_rn(m - __bfloat162float(h));
        }
      }
      __syncthreads();
    }
  }
  if (is_first) {
    __syncthreads();
    if (has_old) {
      int jc = j_last;  // the later one of the last two blocks in the first block's bank
      if ((jc ^ j_first) & 1) --jc;
      if (jc > j_first) {
        const int hi = min(R.len, (jc + 1) * B) - jc * B;
        for (int kv = 0; kv < 2; ++kv)
          for (int i = tid; i < hi * d; i += kThreads) {
            const int off = i / d, ch = i % d, rel = jc * B + off - R.pos0;
            const float y = kv ? __bfloat162float(v[(size_t)(R.t_begin + rel) * stride + head * d + ch])
                               : conv_key(c, R, k, w, rel, head, ch);
            tail_at(kv ? c.tail_v : c.tail_k, c, R.row, jc, head, off)[ch] = finite16(y, &bad);
          }
      }
    }
    __syncthreads();
    const int m = min(n, Wm1);
    for (int i = tid; i < m * d; i += kThreads) {
      const int rel = n - m + i / d, ch = i % d;
      c.hist[(((size_t)R.row * kHistRing + ((R.pos0 + rel) & (kHistRing - 1))) * c.h_kv + head) * d + ch] =
          k[(size_t)(R.t_begin + rel) * stride + head * d + ch];
    }
  }
  if (bad) set_status(status, kStatusNonFinite);
}

}  // namespace

cudaError_t launch_append(const View& c, const Plan& p, const bf16* k, const bf16* v, const float* conv_w,
                          int32_t* status, cudaStream_t st) {
  const long long runs = (long long)p.T / c.B + 2ll * c.rows;
  const int per_token = p.T <= runs;
  const dim3 grid((unsigned)(per_token ? p.T : runs), c.h_kv);
  const size_t smem = (size_t)c.B * c.d * sizeof(bf16);
  if (c.kind == 0) append_kernel<0><<<grid, kThreads, smem, st>>>(c, p, k, v, conv_w, per_token, status);
  else append_kernel<1><<<grid, kThreads, smem, st>>>(c, p, k, v, conv_w, per_token, status);
  return cudaGetLastError();
}

}  // namespace cache
}  // namespace moba
