// Writes new keys and values into the paged 8-bit cache.
//
//   k'_t = bf16(k_t + SiLU(sum_{l < W} w_l (.) k_{t-l}))       (key conv, optional)
//   block complete: s = max(amax r, 2^-126), x8 = rn(x / s); c = mean k', hi = bf16(c), lo = bf16(c - hi)
//   else: bf16 tail
//
// The unit of work is a run: the new tokens of one row inside one block.  One
// CTA of 128 threads per (run, KV head); a thread holds 8 channels of
// consecutive tokens of the block in registers (NCH = B d / 1024 pieces of 16
// bytes), so a complete block is read once (its earlier tokens from the tail),
// its largest magnitude agreed on, and its codes written once.  Bound by HBM
// for prompts, by latency for single tokens.
//
// A row's first run is the only one that may need what the step replaces: the
// tail bank of its block (its earlier tokens) and the raw-key history.  Its
// CTA therefore also does the replacing: it takes the second run along where
// that reads history too (the first run has fewer than W - 1 tokens), then
// writes the tail tokens of the later block that shares its bank, and the
// history, behind a barrier.
//
// Rounding that depends on nothing but the inputs.  k' is the rounding (to
// fp32, then bf16) of the value summed in 64 bits: it is formed in 32 bits
// first, with a bound E on its error, and again in 64 bits only where a bf16
// rounding boundary lies within E (about one element in a thousand).  A
// block's sum is kept in 64 bits, where sums of bf16 values are exact unless
// their exponents span more than 2^38.
#include <cuda_fp8.h>

#include "cache.cuh"

namespace moba {
namespace cache {
namespace {

constexpr int kThreads = 128;

struct RowInfo {
  int row, t_begin;  // the row's first new token
  int pos0;          // and its position
  int n;             // new tokens
  int len;           // tokens after the step
};

__device__ __forceinline__ bool finite_pair(uint32_t w) {
  return (w & 0x7f80u) != 0x7f80u && (w & 0x7f800000u) != 0x7f800000u;
}

// Zero in place of NaN and infinities.
__device__ __forceinline__ uint4 finite8(uint4 x, bool* bad) {
  uint32_t* w = &x.x;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!finite_pair(w[i])) {
      *bad = true;
      if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
      if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0xffffu;
    }
  return x;
}

// 8 raw-key channels of the token `rel` of the row's new ones; negative: from the history; zero before the row.
template <int D>
__device__ __forceinline__ uint4 raw_key(const View& c, const RowInfo& R, const bf16* k, int head, int ch, int rel) {
  if (rel >= 0) return __ldg(reinterpret_cast<const uint4*>(k + ((size_t)(R.t_begin + rel) * c.h_kv + head) * D + ch));
  const int pos = R.pos0 + rel;
  if (pos < 0) return make_uint4(0, 0, 0, 0);
  return *reinterpret_cast<const uint4*>(c.hist +
                                         (((size_t)R.row * kHistRing + (pos & (kHistRing - 1))) * c.h_kv + head) * D + ch);
}

__device__ __noinline__ float conv_in_64(const float* x, const float* w, int W) {
  double z = 0.0;
  for (int l = 0; l < W; ++l) z += (double)w[l] * (double)x[l];
  return (float)((double)x[0] + z / (1.0 + exp(-z)));
}

// k' of 8 channels of token rel.
template <int D>
__device__ __forceinline__ uint4 conv8(const View& c, const RowInfo& R, const bf16* k, const float* w, int head, int ch,
                                       int rel) {
  const int W = c.conv_width;
  float x0[8], z[8], size[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = size[e] = 0.f;
  for (int l = 0; l < W; ++l) {
    float x[8];
    bf16x8_to_f32(raw_key<D>(c, R, k, head, ch, rel - l), x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float wl = __ldg(w + ((size_t)head * D + ch + e) * W + l);
      if (l == 0) x0[e] = x[e];
      z[e] = fmaf(wl, x[e], z[e]);
      size[e] += fabsf(wl * x[e]);
    }
  }
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y[e] = x0[e] + __fdividef(z[e], 1.f + __expf(-z[e]));
    // sum: W 2^-24 size; SiLU: slope at most 1.1, its own error 2^-21 |z| (1 + |z| / 2^2 for the exponent's argument)
    const float E = 9.5367432e-7f * (fabsf(x0[e]) + size[e] * (1.2f + 0.25f * fminf(fabsf(z[e]), 88.f)));
    const uint16_t a = __bfloat16_as_ushort(__float2bfloat16_rn(y[e] - E));
    const uint16_t b = __bfloat16_as_ushort(__float2bfloat16_rn(y[e] + E));
    if (a != b || !(fabsf(z[e]) < 80.f)) {
      float xs[kMaxWidth], ws[kMaxWidth];
      for (int l = 0; l < W; ++l) {
        float x[8];
        bf16x8_to_f32(raw_key<D>(c, R, k, head, ch, rel - l), x);
        xs[l] = x[e];
        ws[l] = __ldg(w + ((size_t)head * D + ch + e) * W + l);
      }
      y[e] = conv_in_64(xs, ws, W);
    }
  }
  return f32_to_bf16x8(y);
}

template <int D>
__device__ __forceinline__ uint4* tail_at(bf16* tail, const View& c, int row, int j, int head, int off, int ch) {
  return reinterpret_cast<uint4*>(tail + ((((size_t)row * 2 + (j & 1)) * c.h_kv + head) * c.B + off) * D + ch);
}

// Codes of 8 values x / s.  The quotient is x r with r = rn(1 / s), corrected
// once by its remainder (Markstein's correction step): within 2^-40 of half a
// unit of its last place, so its rounding to 8 bits is the exact quotient's.
// Scales where the remainder could leave the normal range are divided.
template <int KIND>
__device__ __forceinline__ uint2 encode8(uint4 u, float s, float r, bool divide) {
  float x[8];
  bf16x8_to_f32(u, x);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float y = x[e] * r;
    x[e] = divide ? __fdiv_rn(x[e], s) : fmaf(fmaf(-y, s, x[e]), r, y);
  }
  uint2 o;
  if constexpr (KIND == 0) {
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      p[e] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * e], x[2 * e + 1]), __NV_SATFINITE, __NV_E4M3);
    o.x = p[0] | p[1] << 16, o.y = p[2] | p[3] << 16;
  } else {
    // adding 1.5 x 2^23 rounds to a whole number, ties to even; its low byte is the code (|x| <= 127 (1 + 2^-22))
    uint32_t b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) b[e] = __float_as_uint(x[e] + 12582912.f);
    o.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    o.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  }
  return o;
}

struct Shared {
  float red[kThreads / 32];
  double sum[kThreads * 8];  // block sums of the token groups
};

// Codes, scale (and centroid) of a complete block held in registers.
template <int KIND, int D, int NCH, bool KEY>
__device__ __forceinline__ void write_block(const View& c, uint4* x, int pg, int head, Shared& sh) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES, B = NCH * GROUPS;
  const int tid = threadIdx.x, ck = tid % LANES, grp = tid / LANES;
  __nv_bfloat162 m2 = __float2bfloat162_rn(0.f);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) m2 = __hmax2(m2, __habs2(h[e]));
  }
  float m = fmaxf(__low2float(m2), __high2float(m2));
#pragma unroll
  for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, off));
  if ((tid & 31) == 0) sh.red[tid >> 5] = m;
  if constexpr (KEY) {
    double s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.0;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      float f[8];
      bf16x8_to_f32(x[i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] += (double)f[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sh.sum[(grp * 8 + e) * LANES + ck] = s[e];
  }
  __syncthreads();
  m = fmaxf(fmaxf(sh.red[0], sh.red[1]), fmaxf(sh.red[2], sh.red[3]));
  const float s = fmaxf(m * (KIND == 0 ? 1.f / 448.f : 1.f / 127.f), 1.17549435e-38f);
  const float r = __frcp_rn(s);
  const bool divide = s < 8.6736174e-19f;  // 2^-60
  const size_t at = (size_t)pg * c.h_kv + head;
  uint8_t* dst = (KEY ? c.k : c.v) + at * (B * D) + ck * 8;
#pragma unroll
  for (int i = 0; i < NCH; ++i)
    *reinterpret_cast<uint2*>(dst + (grp * NCH + i) * D) = encode8<KIND>(x[i], s, r, divide);
  if (tid == 0) (KEY ? c.k_scale : c.v_scale)[at] = s;
  if constexpr (KEY) {
    if (tid < D) {
      double t = 0.0;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) t += sh.sum[(g * 8 + (tid & 7)) * LANES + tid / 8];
      const float mean = (float)(t * (1.0 / B));
      const bf16 hi = __float2bfloat16_rn(mean);
      c.cent[at * D + tid] = hi;
      c.cent[((size_t)c.n_pages * c.h_kv + at) * D + tid] = __float2bfloat16_rn(mean - __bfloat162float(hi));
    }
  }
  __syncthreads();
}

template <int KIND, int D, int NCH, bool CONV>
__global__ void __launch_bounds__(kThreads)
append_kernel(View c, Plan p, const bf16* __restrict__ k, const bf16* __restrict__ v, const float* __restrict__ w,
              int per_token, int32_t* status) {
  constexpr int LANES = D / 8, GROUPS = kThreads / LANES, B = NCH * GROUPS;
  __shared__ Shared sh;
  const int tid = threadIdx.x, head = blockIdx.y, u = blockIdx.x;
  const int ch = tid % LANES * 8, off0 = tid / LANES * NCH;  // this thread's channels and first token of a block
  const int total = min(__ldg(p.cu + c.rows), p.T);
  // ---- which run
  RowInfo R;
  int first_rel;  // its first token, relative to the row's first
  if (per_token) {
    if (u >= total) return;
    R.row = __ldg(p.row + u);
    const int pos = __ldg(p.pos + u);
    if ((unsigned)R.row >= (unsigned)c.rows) return;
    R.t_begin = __ldg(p.cu + R.row);
    first_rel = u - R.t_begin;
    if (R.t_begin < 0 || first_rel < 0 || pos < first_rel) return;
    R.pos0 = pos - first_rel;
    if (first_rel > 0 && pos % B != 0) return;
  } else {
    int lo = 0, hi = c.rows;  // largest row with cu / B + 2 row <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu + mid) / B + 2 * mid <= u) lo = mid; else hi = mid;
    }
    R.row = lo;
    R.t_begin = __ldg(p.cu + lo);
    if (R.t_begin < 0 || R.t_begin >= total) return;
    R.pos0 = __ldg(p.pos + R.t_begin);
    if (R.pos0 < 0) return;
    const int i = u - (R.t_begin / B + 2 * lo);  // number of the block among the row's touched ones
    first_rel = i == 0 ? 0 : (R.pos0 / B + i) * B - R.pos0;
  }
  R.n = min(__ldg(p.cu + R.row + 1), total) - R.t_begin;
  if (R.n <= 0 || first_rel >= R.n) return;
  const int len = c.state[2 * R.row];
  if ((long long)R.pos0 + R.n != len || len > (long long)c.max_blocks * B) {
    if (tid == 0) set_status(status, kStatusBadTable);
    return;
  }
  R.len = len;
  const int Wm1 = CONV ? c.conv_width - 1 : 0;
  const int j_first = R.pos0 / B, j_last = (R.len - 1) / B;
  const int n_first = min(R.n, (j_first + 1) * B - R.pos0);  // tokens of the row's first run
  const int j0 = (R.pos0 + first_rel) / B;
  int j1 = j0;
  const bool is_first = j0 == j_first;
  if (n_first < Wm1 && R.n > n_first) {  // the second run reads history too
    if (j0 == j_first + 1) return;
    if (is_first) j1 = j_first + 1;
  }
  const bool has_old = R.pos0 % B != 0;
  bool bad = false;
  auto new_key = [&](int rel) {
    uint4 x;
    if constexpr (CONV) x = conv8<D>(c, R, k, w, head, ch, rel);
    else x = raw_key<D>(c, R, k, head, ch, rel);
    return finite8(x, &bad);
  };
  auto new_val = [&](int rel) {
    return finite8(__ldg(reinterpret_cast<const uint4*>(v + ((size_t)(R.t_begin + rel) * c.h_kv + head) * D + ch)), &bad);
  };
  for (int j = j0; j <= j1; ++j) {
    const int lo = max(R.pos0 - j * B, 0), hi = min(R.len - j * B, B);  // new tokens inside the block
    const int rel0 = j * B - R.pos0;
    // A later block in the first block's bank is written by the first run's CTA, below.
    const bool keep = j >= j_last - 1 && !(has_old && j > j_first && ((j ^ j_first) & 1) == 0);
    int pg = -1;
    if (hi == B) {
      const int slot = __ldg(p.slot + R.t_begin + rel0 + lo);
      if (slot >= 0 && slot / B < c.n_pages) pg = slot / B;
      else if (tid == 0) set_status(status, kStatusBadTable);
    }
    uint4 x[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int off = off0 + i;
      x[i] = make_uint4(0, 0, 0, 0);
      if (off < lo) {
        if (pg >= 0) x[i] = *tail_at<D>(c.tail_k, c, R.row, j, head, off, ch);
      } else if (off < hi) {
        x[i] = new_key(rel0 + off);
      }
    }
    if (keep) {
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (off0 + i >= lo && off0 + i < hi) *tail_at<D>(c.tail_k, c, R.row, j, head, off0 + i, ch) = x[i];
    }
    if (pg >= 0) write_block<KIND, D, NCH, true>(c, x, pg, head, sh);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int off = off0 + i;
      x[i] = make_uint4(0, 0, 0, 0);
      if (off < lo) {
        if (pg >= 0) x[i] = *tail_at<D>(c.tail_v, c, R.row, j, head, off, ch);
      } else if (off < hi) {
        x[i] = new_val(rel0 + off);
      }
    }
    if (keep) {
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (off0 + i >= lo && off0 + i < hi) *tail_at<D>(c.tail_v, c, R.row, j, head, off0 + i, ch) = x[i];
    }
    if (pg >= 0) write_block<KIND, D, NCH, false>(c, x, pg, head, sh);
  }
  if (is_first) {
    if (has_old) {
      int jc = j_last;  // the later one of the last two blocks in the first block's bank
      if ((jc ^ j_first) & 1) --jc;
      if (jc > j_first) {
        __syncthreads();  // the earlier tokens have been read
        const int hi = min(R.len - jc * B, B), rel0 = jc * B - R.pos0;
        for (int off = off0; off < min(off0 + NCH, hi); ++off) {
          *tail_at<D>(c.tail_k, c, R.row, jc, head, off, ch) = new_key(rel0 + off);
          *tail_at<D>(c.tail_v, c, R.row, jc, head, off, ch) = new_val(rel0 + off);
        }
      }
    }
    if constexpr (CONV) {
      __syncthreads();  // the history has been read
      const int m = min(R.n, Wm1), i = tid / LANES;
      if (i < m) {
        const int rel = R.n - m + i;
        *reinterpret_cast<uint4*>(
            c.hist + (((size_t)R.row * kHistRing + ((R.pos0 + rel) & (kHistRing - 1))) * c.h_kv + head) * D + ch) =
            raw_key<D>(c, R, k, head, ch, rel);
      }
    }
  }
  if (bad) set_status(status, kStatusNonFinite);
}

template <int KIND, int D, int NCH>
cudaError_t launch_one(const View& c, const Plan& p, const bf16* k, const bf16* v, const float* w, int32_t* status,
                       cudaStream_t st) {
  // Runs of a row start at index cu / B + 2 row at the earliest; with few tokens a row every token stands for its run.
  const long long runs = (long long)p.T / c.B + 2ll * c.rows;
  const int per_token = p.T <= runs;
  const dim3 grid((unsigned)(per_token ? p.T : runs), c.h_kv);
  if (c.conv_width > 0) append_kernel<KIND, D, NCH, true><<<grid, kThreads, 0, st>>>(c, p, k, v, w, per_token, status);
  else append_kernel<KIND, D, NCH, false><<<grid, kThreads, 0, st>>>(c, p, k, v, w, per_token, status);
  return cudaGetLastError();
}

template <int KIND, int D>
cudaError_t launch_block(const View& c, const Plan& p, const bf16* k, const bf16* v, const float* w, int32_t* status,
                         cudaStream_t st) {
  switch (c.B * D / 1024) {
    case 1: if constexpr (D == 64) return launch_one<KIND, D, 1>(c, p, k, v, w, status, st);
    case 2: return launch_one<KIND, D, 2>(c, p, k, v, w, status, st);
    case 4: return launch_one<KIND, D, 4>(c, p, k, v, w, status, st);
    case 8: return launch_one<KIND, D, 8>(c, p, k, v, w, status, st);
    default: if constexpr (D == 128) return launch_one<KIND, D, 16>(c, p, k, v, w, status, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_append(const View& c, const Plan& p, const bf16* k, const bf16* v, const float* conv_w,
                          int32_t* status, cudaStream_t st) {
  if (c.d == 64)
    return c.kind == 0 ? launch_block<0, 64>(c, p, k, v, conv_w, status, st)
                       : launch_block<1, 64>(c, p, k, v, conv_w, status, st);
  return c.kind == 0 ? launch_block<0, 128>(c, p, k, v, conv_w, status, st)
                     : launch_block<1, 128>(c, p, k, v, conv_w, status, st);
}

}  // namespace cache
}  // namespace moba
