// Writes new keys and values into the paged 8-bit cache.
//
//   k'_t = bf16(k_t + SiLU(sum_{l < W} w_l (.) k_{t-l}))       (key conv, optional)
//   block complete: s = max(amax r, 2^-126), x8 = rn(x / s); c = mean k', hi = bf16(c), lo = bf16(c - hi)
//   else: bf16 tail
//
// The unit of work is a run: the new tokens of one row inside one block.  A
// CTA takes a run for some KV heads in turn, the next head's tokens on their
// way (cp.async) while one is rounded.  A thread holds 8 channels of NCH
// consecutive tokens of the block in registers, so a complete block is read
// once (its earlier tokens from the tail), its largest magnitudes agreed on,
// and its codes written once.  Bound by HBM for prompts (four of 8K to 64K
// tokens, 8 heads of 128: 764 MB in 141 us, 5.4 TB/s, 83 % of a copy's rate),
// by instruction issue with the conv (64K tokens, 16 heads of 64, width 4: 275
// us, without conv 87), by a chain of look-ups for single tokens (64 rows with
// conv 10.7 us).
//
// A row's first run is the only one that may need what the step replaces: the
// tail bank of its block (its earlier tokens) and the raw-key history.  Its
// CTA therefore also does the replacing: it takes the second run along where
// that reads history too (the first run has fewer than W - 1 tokens), then
// writes the tail tokens of the later block that shares its bank, and the
// history, behind a barrier.  The history takes more of a step than the next
// one's taps reach (W - 1): as many more as a length may be set back by, for
// where part of the step is taken back its tokens are what comes before.
//
// Rounding that depends on nothing but the inputs.  k' is the rounding (to
// fp32, then bf16) of the value summed in 64 bits: it is formed in 32 bits
// first, with a bound E on its error, and again in 64 bits only where a bf16
// rounding boundary lies within E (about one element in a thousand).  A
// block's sum is that of its threads' sums (of at most 8 tokens, in 32 bits,
// an eighth of each so that none overflows) in 64 bits, in a fixed order.
#include <cuda_fp8.h>

#include "cache.cuh"

namespace moba {
namespace cache {
namespace {

__device__ __forceinline__ void cp_async16(void* smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem_u32(smem)), "l"(gmem));
}

constexpr int kFewTokens = 4;  // see append_kernel
constexpr int kDoubts = 512;   // roundings in doubt held per tile

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

// One channel of k' in 64 bits: taps x0 .. x7 (zero from the width on), weights w[0, W).
__device__ __noinline__ float conv_in_64(float x0, float x1, float x2, float x3, float x4, float x5, float x6, float x7,
                                         const float* w, int W) {
  const float x[kMaxWidth] = {x0, x1, x2, x3, x4, x5, x6, x7};
  double z = 0.0;
#pragma unroll
  for (int l = 0; l < kMaxWidth; ++l)
    if (l < W) z += (double)__ldg(w + l) * (double)x[l];
  return (float)((double)x0 + z / (1.0 + exp(-z)));
}

// Element e of 8 bf16.
__device__ __forceinline__ float element(const uint4& u, int e) {
  const uint32_t w = e < 2 ? u.x : (e < 4 ? u.y : (e < 6 ? u.z : u.w));
  return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
}

// k' of 8 channels of a token; tap(l): their raw keys l tokens before.  w: the head's weights [d, W]; ws: the same as
// [W, d] in shared memory, channels in the order of wplace, or null (a lane's 8 x W weights are then read one by one,
// which a CTA that converts many tokens would feel).  `doubt(e)` takes note of a channel whose rounding 32 bits do not
// settle and returns true, or returns false: then it is settled here.
template <int D, typename G, typename F>
__device__ __forceinline__ uint4 conv8(int W, const float* w, const float* ws, int ch, G tap, F doubt) {
  uint4 raw[kMaxWidth];
#pragma unroll
  for (int l = 0; l < kMaxWidth; ++l) raw[l] = l < W ? tap(l) : make_uint4(0, 0, 0, 0);
  float x0[8], z[8], size[8];
  bf16x8_to_f32(raw[0], x0);
#pragma unroll
  for (int e = 0; e < 8; ++e) z[e] = size[e] = 0.f;
  const float* wc = w + (size_t)ch * W;
#pragma unroll
  for (int l = 0; l < kMaxWidth; ++l)
    if (l < W) {
      float x[8], wl[8];
      bf16x8_to_f32(raw[l], x);
      if (ws) {
        *reinterpret_cast<float4*>(wl) = *reinterpret_cast<const float4*>(ws + l * D + ch / 2);
        *reinterpret_cast<float4*>(wl + 4) = *reinterpret_cast<const float4*>(ws + l * D + D / 2 + ch / 2);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) wl[e] = __ldg(wc + e * W + l);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        z[e] = fmaf(wl[e], x[e], z[e]);
        size[e] = fmaf(fabsf(wl[e]), fabsf(x[e]), size[e]);
      }
    }
  // In units of 2^-24: the sum is off by W size, SiLU (slope at most 1.1) carries that and adds 12 of its own value
  // (exponential, quotient) and 2 |z| of its value for the exponent's argument (|z SiLU(z)| <= size where that counts),
  // the last sum and the rounding to 32 bits 2 of the result.  1.1 W + 16 with room, and 2^-140 for what the steps lose
  // below the normal range (2^-150 each):
  const float e1 = 5.9604645e-8f * (1.2f * (float)W + 18.f);
  float y[8];
  uint32_t open = 0;  // channels whose rounding is not settled
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y[e] = x0[e] + __fdividef(z[e], 1.f + __expf(-z[e]));
    const float E = fmaf(size[e], e1, fmaf(fabsf(x0[e]), 1.1920929e-7f, 7.1746481e-43f));
    const uint32_t both = pack_bf16(y[e] - E, y[e] + E);
    open |= (uint32_t)(__byte_perm(both, 0, 0x1032) != both || !(fabsf(z[e]) < 80.f)) << e;
  }
  uint4 r = f32_to_bf16x8(y);
  while (open) {
    const int e = __ffs(open) - 1;
    open &= open - 1;
    if (doubt(e)) continue;
    const float v = conv_in_64(element(raw[0], e), element(raw[1], e), element(raw[2], e), element(raw[3], e),
                               element(raw[4], e), element(raw[5], e), element(raw[6], e), element(raw[7], e), wc + e * W, W);
    const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    uint32_t* word = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e >> 1 == i) word[i] = e & 1 ? (word[i] & 0xffffu) | h << 16 : (word[i] & 0xffff0000u) | h;
  }
  return r;
}

template <int D>
__device__ __forceinline__ uint4* tail_at(bf16* tail, const View& c, int row, int j, int head, int off, int ch) {
  return reinterpret_cast<uint4*>(tail + ((((size_t)row * 2 + (j & 1)) * c.h_kv + head) * c.B + off) * D + ch);
}

// Codes of 8 values x / s, r = rn(1 / s).  The quotient is x r, corrected
// once by its remainder (Markstein's correction step): within 2^-40 of half a
// unit of its last place, so its rounding to 8 bits is the exact quotient's.
// Scales where the remainder could leave the normal range are divided.
template <int KIND, bool DIVIDE>
__device__ __forceinline__ uint2 encode8(uint4 u, float s, float r) {
  float x[8];
  bf16x8_to_f32(u, x);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (DIVIDE) {
      x[e] = __fdiv_rn(x[e], s);
    } else {
      const float y = x[e] * r;
      x[e] = fmaf(fmaf(-y, s, x[e]), r, y);
    }
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

// Threads and pieces of 16 bytes per thread for a tile of B tokens x D channels.
template <int D, int BLK>
struct Shape {
  static constexpr int THREADS = BLK * D >= 8192 ? 256 : 128;
  static constexpr int NCH = BLK * D / 8 / THREADS;
  static constexpr int LANES = D / 8;               // threads across a token
  static constexpr int GROUPS = THREADS / LANES;    // token groups of NCH consecutive tokens
  static constexpr int STAGE = 2 * NCH * THREADS;   // 16-byte slots of one head's K and V
  static constexpr int RAW = (BLK + kMaxWidth - 1) * LANES;  // slots of a head's raw keys, with the taps before the block
  static constexpr int bytes(bool conv) { return 2 * STAGE * 16 + THREADS * 8 * 4 + (conv ? 2 * RAW * 16 : 0); }
  static_assert(NCH * GROUPS == BLK && NCH <= 8, "tile");
};

// Where the sum of channel 8 ck + e of a token group is kept: 8 rows of D / 8 values, rotated so that both the threads
// that hold 8 channels each and those that take one channel each meet every bank once.
template <int D>
__device__ __forceinline__ int sum_place(int ck, int e) {
  return e * (D / 8) + ((ck + (D == 128 ? 2 * e : e)) & (D / 8 - 1));
}

template <int NCH>
__device__ __forceinline__ float amax8(const uint4* x) {
  __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) m = __hmax2_nan(m, __habs2(h[e]));
  }
  const float a = __low2float(m), b = __high2float(m);
  return a > b || a != a ? a : b;  // NaN stays
}

// Largest magnitude; NaN and infinities, if any, become zero first.
template <int NCH>
__device__ __forceinline__ float finite_amax(uint4* x, bool* bad) {
  float m = amax8<NCH>(x);
  if (!(m <= 3.4e38f)) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) x[i] = finite8(x[i], bad);
    m = amax8<NCH>(x);
  }
  return m;
}

template <int KIND>
__device__ __noinline__ uint2 encode8_divide(uint4 u, float s) {
  return encode8<KIND, true>(u, s, 0.f);
}

template <int KIND, int D, int BLK>
__device__ __forceinline__ void write_codes(uint8_t* dst, const uint4* x, float s) {
  using S = Shape<D, BLK>;
  const float r = __frcp_rn(s);
  dst += (threadIdx.x / S::LANES * S::NCH) * D + threadIdx.x % S::LANES * 8;
  if (s < 8.6736174e-19f) {  // 2^-60
#pragma unroll 1
    for (int i = 0; i < S::NCH; ++i) {
      uint4 u = x[0];
#pragma unroll
      for (int k = 1; k < S::NCH; ++k)
        if (k == i) u = x[k];
      *reinterpret_cast<uint2*>(dst + i * D) = encode8_divide<KIND>(u, s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < S::NCH; ++i) *reinterpret_cast<uint2*>(dst + i * D) = encode8<KIND, false>(x[i], s, r);
  }
}

template <int KIND>
__device__ __forceinline__ float scale_of(float m) {
  return fmaxf(m * (KIND == 0 ? 1.f / 448.f : 1.f / 127.f), 1.17549435e-38f);
}

template <int KIND, int D, int BLK, bool CONV>
__global__ void __launch_bounds__(Shape<D, BLK>::THREADS, (CONV || Shape<D, BLK>::NCH > 4 ? 512 : 768) / Shape<D, BLK>::THREADS)
append_kernel(View c, Plan p, const bf16* __restrict__ k, const bf16* __restrict__ v, const float* __restrict__ w,
              int raw_kept, int per_token, int heads_per_cta, int32_t* status) {
  using S = Shape<D, BLK>;
  constexpr int THREADS = S::THREADS, NCH = S::NCH, LANES = S::LANES, GROUPS = S::GROUPS, B = BLK;
  extern __shared__ __align__(16) unsigned char smem[];
  uint4* ring = reinterpret_cast<uint4*>(smem);                            // [2][K, V][NCH][THREADS]
  float* gsum = reinterpret_cast<float*>(smem + 2 * S::STAGE * 16);        // [GROUPS][D], swizzled
  uint4* raws = reinterpret_cast<uint4*>(smem + 2 * S::STAGE * 16 + THREADS * 8 * 4);  // [2][BLK + 7][LANES], conv only
  __shared__ float red[2][THREADS / 32];
  __shared__ int n_doubt, doubts[CONV ? kDoubts : 1];
  __shared__ __align__(16) float wsm[CONV ? 2 * kMaxWidth * D : 4];  // two heads' conv weights [W, d]
  const int tid = threadIdx.x, u = blockIdx.x;
  const int head0 = blockIdx.y * heads_per_cta, head1 = min(c.h_kv, head0 + heads_per_cta);
  const int ch = tid % LANES * 8, off0 = tid / LANES * NCH;  // this thread's channels and first token of a block
  // ---- which run.  Loads that do not need one another's answers are made together.
  RowInfo R;
  int first_rel;  // its first token, relative to the row's first
  int end, len, total;
  if (per_token) {
    const int row = __ldg(p.row + u), pos = __ldg(p.pos + u);
    total = __ldg(p.cu + c.rows);
    if ((unsigned)row >= (unsigned)c.rows) return;
    R.row = row;
    R.t_begin = __ldg(p.cu + row);
    end = __ldg(p.cu + row + 1);
    len = c.state[2 * row];
    first_rel = u - R.t_begin;
    if (R.t_begin < 0 || first_rel < 0 || pos < first_rel || u >= total) return;
    R.pos0 = pos - first_rel;
    if (first_rel > 0 && pos % B != 0) return;
  } else {
    total = __ldg(p.cu + c.rows);
    int lo = 0, hi = c.rows;  // largest row with cu / B + 2 row <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu + mid) / B + 2 * mid <= u) lo = mid; else hi = mid;
    }
    R.row = lo;
    R.t_begin = __ldg(p.cu + lo);
    end = __ldg(p.cu + lo + 1);
    len = c.state[2 * lo];
    if (R.t_begin < 0 || R.t_begin >= min(total, p.T)) return;
    R.pos0 = __ldg(p.pos + R.t_begin);
    if (R.pos0 < 0) return;
    const int i = u - (R.t_begin / B + 2 * lo);  // number of the block among the row's touched ones
    if (i < 0) return;
    first_rel = i == 0 ? 0 : (R.pos0 / B + i) * B - R.pos0;
  }
  R.n = min(end, min(total, p.T)) - R.t_begin;
  if (R.n <= 0 || first_rel >= R.n) return;
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

  // k' straight from memory
  auto key_now = [&](int head, int rel) {
    if constexpr (CONV)
      return conv8<D>(c.conv_width, w + (size_t)head * D * c.conv_width, nullptr, ch,
                      [&](int l) { return raw_key<D>(c, R, k, head, ch, rel - l); }, [](int) { return false; });
    else return raw_key<D>(c, R, k, head, ch, rel);
  };
  if (R.n <= kFewTokens && R.n == n_first && R.len % B != 0) {
    // A few tokens of an unfinished block (a generated token, mostly): one CTA for all heads, a thread group per
    // (token, head).  With a CTA per head, one group in 16 would work.
    if (blockIdx.y > 0) return;
    for (int i = tid / LANES; i < R.n * c.h_kv; i += GROUPS) {
      const int rel = i / c.h_kv, head = i % c.h_kv;
      const size_t at = ((size_t)(R.t_begin + rel) * c.h_kv + head) * D + ch;
      const uint4 y = __ldg(reinterpret_cast<const uint4*>(v + at));
      const uint4 x = key_now(head, rel);
      *tail_at<D>(c.tail_k, c, R.row, j0, head, R.pos0 % B + rel, ch) = finite8(x, &bad);
      *tail_at<D>(c.tail_v, c, R.row, j0, head, R.pos0 % B + rel, ch) = finite8(y, &bad);
    }
    if constexpr (CONV) {
      __syncthreads();  // the history has been read
      const int m = min(R.n, raw_kept);
      for (int i = tid / LANES; i < m * c.h_kv; i += GROUPS) {
        const int rel = R.n - m + i / c.h_kv, head = i % c.h_kv;
        *reinterpret_cast<uint4*>(
            c.hist + (((size_t)R.row * kHistRing + ((R.pos0 + rel) & (kHistRing - 1))) * c.h_kv + head) * D + ch) =
            raw_key<D>(c, R, k, head, ch, rel);
      }
    }
    if (bad) set_status(status, kStatusNonFinite);
    return;
  }

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
    // Copies of a head's tokens on their way: a thread reads only the slots that it fills itself.
    auto fetch = [&](int head) {
      if (head < head1) {
        uint4* dst = ring + ((head - head0) & 1) * S::STAGE + tid;
        if (lo == 0 && hi == B) {  // a whole block of new tokens
          const size_t at = ((size_t)(R.t_begin + rel0 + off0) * c.h_kv + head) * D + ch;
          const size_t row = (size_t)c.h_kv * D;
#pragma unroll
          for (int i = 0; i < NCH; ++i) {
            if (!CONV) cp_async16(dst + i * THREADS, k + at + i * row);
            cp_async16(dst + (NCH + i) * THREADS, v + at + i * row);
          }
        } else {
#pragma unroll
          for (int i = 0; i < NCH; ++i) {
            const int off = off0 + i;
            const bool fresh = off >= lo && off < hi, old = off < lo && pg >= 0;
            const size_t at = ((size_t)(R.t_begin + (fresh ? rel0 + off : 0)) * c.h_kv + head) * D + ch;
            const void* ks = old ? (const void*)tail_at<D>(c.tail_k, c, R.row, j, head, off, ch) : (const void*)(k + at);
            const void* vs = old ? (const void*)tail_at<D>(c.tail_v, c, R.row, j, head, off, ch) : (const void*)(v + at);
            if (!CONV || !fresh) cp_async16_zfill(dst + i * THREADS, ks, old || fresh);
            cp_async16_zfill(dst + (NCH + i) * THREADS, vs, old || fresh);
          }
        }
        if constexpr (CONV) {  // raw keys of the new tokens and of the W - 1 before them
          uint4* rd = raws + ((head - head0) & 1) * S::RAW;
          for (int i = tid; i < S::RAW; i += THREADS) {
            const int off = i / LANES - (kMaxWidth - 1), rel = rel0 + off, cc = i % LANES * 8;
            if (off < lo - Wm1 || off >= hi) continue;
            const bf16* at = k;
            if (rel >= 0) at = k + ((size_t)(R.t_begin + rel) * c.h_kv + head) * D + cc;
            else if (R.pos0 + rel >= 0)
              at = c.hist + (((size_t)R.row * kHistRing + ((R.pos0 + rel) & (kHistRing - 1))) * c.h_kv + head) * D + cc;
            cp_async16_zfill(rd + i, at, R.pos0 + rel >= 0);
          }
        }
      }
      cp_async_commit();
    };
    fetch(head0);
    // the next head's conv weights wait in registers; [d, W] goes to [W, d]
    constexpr int NWR = CONV ? kMaxWidth * D / THREADS : 1;
    float wnext[NWR];
    int wplace[NWR];
#pragma unroll
    for (int i = 0; i < NWR; ++i) {
      const int at = tid + i * THREADS, W = CONV ? c.conv_width : 1;
      const int cc = at / W;  // of 8 channels the first 4 and the last 4 apart, so that neighbours read side by side
      wplace[i] = at < D * W ? at % W * D + (cc >> 2 & 1) * (D / 2) + (cc >> 3) * 4 + (cc & 3) : -1;
    }
    auto ask_weights = [&](int head) {
      if constexpr (CONV) {
#pragma unroll
        for (int i = 0; i < NWR; ++i)
          if (wplace[i] >= 0 && head < head1)
            wnext[i] = __ldg(w + (size_t)head * D * c.conv_width + tid + i * THREADS);
      }
    };
    ask_weights(head0);
    for (int head = head0; head < head1; ++head) {
      fetch(head + 1);
      uint4 x[NCH], y[NCH];
      uint4* src = ring + ((head - head0) & 1) * S::STAGE + tid;
      if constexpr (CONV) {  // the converted tokens go where copies of the others go
        const uint4* rs = raws + ((head - head0) & 1) * S::RAW + (kMaxWidth - 1) * LANES;
        float* ws = wsm + (head & 1) * kMaxWidth * D;
        const float* wh = w + (size_t)head * D * c.conv_width;
        const int W = c.conv_width;
#pragma unroll
        for (int i = 0; i < NWR; ++i)
          if (wplace[i] >= 0) ws[wplace[i]] = wnext[i];
        ask_weights(head + 1);
        if (tid == 0) n_doubt = 0;
        cp_async_wait<1>();
        __syncthreads();
        // Roundings in doubt are noted and settled together, a thread each.
        const int i1 = min(hi - off0, NCH);
#pragma unroll 1
        for (int i = max(lo - off0, 0); i < i1; ++i)
          src[i * THREADS] = conv8<D>(W, wh, ws, ch, [&](int l) { return rs[(off0 + i - l) * LANES + ch / 8]; },
                                      [&](int e) {
                                        const int at = atomicAdd(&n_doubt, 1);
                                        if (at >= kDoubts) return false;
                                        doubts[at] = (off0 + i) * D + ch + e;
                                        return true;
                                      });
        __syncthreads();
        if (n_doubt > 0) {
          for (int at = tid; at < min(n_doubt, kDoubts); at += THREADS) {
            const int off = doubts[at] / D, cc = doubts[at] % D;
            float xs[kMaxWidth];
#pragma unroll
            for (int l = 0; l < kMaxWidth; ++l)
              xs[l] = l < W ? __bfloat162float(reinterpret_cast<const bf16*>(rs + (off - l) * LANES)[cc]) : 0.f;
            const float z = conv_in_64(xs[0], xs[1], xs[2], xs[3], xs[4], xs[5], xs[6], xs[7], wh + (size_t)cc * W, W);
            // into the slot of the thread that holds it
            uint4* slot = ring + ((head - head0) & 1) * S::STAGE + off % NCH * THREADS + off / NCH * LANES + cc / 8;
            reinterpret_cast<bf16*>(slot)[cc & 7] = __float2bfloat16_rn(z);
          }
          __syncthreads();
        }
      }
      cp_async_wait<1>();
#pragma unroll
      for (int i = 0; i < NCH; ++i) x[i] = src[i * THREADS], y[i] = src[(NCH + i) * THREADS];
      float mk = finite_amax<NCH>(x, &bad), mv = finite_amax<NCH>(y, &bad);
      if (keep) {
#pragma unroll
        for (int i = 0; i < NCH; ++i)
          if (off0 + i >= lo && off0 + i < hi) {
            *tail_at<D>(c.tail_k, c, R.row, j, head, off0 + i, ch) = x[i];
            *tail_at<D>(c.tail_v, c, R.row, j, head, off0 + i, ch) = y[i];
          }
      }
      if (pg < 0) continue;
#pragma unroll
      for (int off = 16; off; off >>= 1) {
        mk = fmaxf(mk, __shfl_xor_sync(~0u, mk, off));
        mv = fmaxf(mv, __shfl_xor_sync(~0u, mv, off));
      }
      if ((tid & 31) == 0) red[0][tid >> 5] = mk, red[1][tid >> 5] = mv;
      // An eighth of the sum of this thread's tokens (8 at most: it stays finite where the sum would not; an eighth of a
      // bf16 is exact in 32 bits): exact unless their exponents span more than 2^13.
      float s[8];
      bf16x8_to_f32(x[0], s);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] *= 0.125f;
#pragma unroll
      for (int i = 1; i < NCH; ++i) {
        float f[8];
        bf16x8_to_f32(x[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = fmaf(f[e], 0.125f, s[e]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) gsum[off0 / NCH * D + sum_place<D>(tid % LANES, e)] = s[e];
      __syncthreads();
      mk = red[0][0], mv = red[1][0];
#pragma unroll
      for (int i = 1; i < THREADS / 32; ++i) mk = fmaxf(mk, red[0][i]), mv = fmaxf(mv, red[1][i]);
      const float sk = scale_of<KIND>(mk), sv = scale_of<KIND>(mv);
      const size_t at = (size_t)pg * c.h_kv + head;
      write_codes<KIND, D, BLK>(c.k + at * (B * D), x, sk);
      write_codes<KIND, D, BLK>(c.v + at * (B * D), y, sv);
      if (tid == 0) c.k_scale[at] = sk, c.v_scale[at] = sv;
      if (tid < D) {
        double t = 0.0;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) t += (double)gsum[g * D + sum_place<D>(tid >> 3, tid & 7)];
        const float mean = (float)(t * (8.0 / B));
        const bf16 hi16 = __float2bfloat16_rn(mean);
        c.cent[at * D + tid] = hi16;
        c.cent[((size_t)c.n_pages * c.h_kv + at) * D + tid] = __float2bfloat16_rn(mean - __bfloat162float(hi16));
      }
      __syncthreads();
    }
    cp_async_wait<0>();
  }
  if (is_first) {
    int jc = j_last;  // the later one of the last two blocks in the first block's bank
    if ((jc ^ j_first) & 1) --jc;
    const bool replace = has_old && jc > j_first;
    if (replace || CONV) __syncthreads();  // the earlier tokens and the history have been read
    for (int head = head0; head < head1; ++head) {
      if (replace) {
        const int hi = min(R.len - jc * B, B), rel0 = jc * B - R.pos0;
        for (int off = off0; off < min(off0 + NCH, hi); ++off) {
          const uint4 x = key_now(head, rel0 + off);
          const size_t at = ((size_t)(R.t_begin + rel0 + off) * c.h_kv + head) * D + ch;
          *tail_at<D>(c.tail_k, c, R.row, jc, head, off, ch) = finite8(x, &bad);
          *tail_at<D>(c.tail_v, c, R.row, jc, head, off, ch) = finite8(__ldg(reinterpret_cast<const uint4*>(v + at)), &bad);
        }
      }
      if constexpr (CONV) {
        const int m = min(R.n, raw_kept);
        for (int i = tid / LANES; i < m; i += GROUPS) {
          const int rel = R.n - m + i;
          *reinterpret_cast<uint4*>(
              c.hist + (((size_t)R.row * kHistRing + ((R.pos0 + rel) & (kHistRing - 1))) * c.h_kv + head) * D + ch) =
              raw_key<D>(c, R, k, head, ch, rel);
        }
      }
    }
  }
  if (bad) set_status(status, kStatusNonFinite);
}

template <int KIND, int D, int BLK>
cudaError_t launch_one(const View& c, const Plan& p, const bf16* k, const bf16* v, const float* w, int raw_kept, int32_t* status,
                       cudaStream_t st) {
  using S = Shape<D, BLK>;
  // Runs of a row start at index cu / B + 2 row at the earliest; with few tokens a row every token stands for its run.
  const long long runs = (long long)p.T / c.B + 2ll * c.rows;
  const int per_token = p.T <= runs;
  const long long n = per_token ? p.T : runs;
  // Heads one after the other in a CTA share its look-ups and overlap copies with rounding, as long as the GPU is
  // filled (16 CTAs per SM), evenly.
  long long per = n * c.h_kv / (16 * 148);
  per = per < 1 ? 1 : (per > c.h_kv ? c.h_kv : per);
  const long long parts = (c.h_kv + per - 1) / per;
  per = (c.h_kv + parts - 1) / parts;
  const dim3 grid((unsigned)n, (unsigned)((c.h_kv + per - 1) / per));
  cudaError_t e;
  if (c.conv_width > 0) {
    if ((e = cudaFuncSetAttribute(append_kernel<KIND, D, BLK, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  S::bytes(true))) != cudaSuccess)
      return e;
    append_kernel<KIND, D, BLK, true><<<grid, S::THREADS, S::bytes(true), st>>>(c, p, k, v, w, raw_kept, per_token, (int)per, status);
  } else {
    if ((e = cudaFuncSetAttribute(append_kernel<KIND, D, BLK, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  S::bytes(false))) != cudaSuccess)
      return e;
    append_kernel<KIND, D, BLK, false><<<grid, S::THREADS, S::bytes(false), st>>>(c, p, k, v, w, raw_kept, per_token, (int)per, status);
  }
  return cudaGetLastError();
}

template <int KIND, int D>
cudaError_t launch_block(const View& c, const Plan& p, const bf16* k, const bf16* v, const float* w, int raw_kept, int32_t* status,
                         cudaStream_t st) {
  switch (c.B) {
    case 16: return launch_one<KIND, D, 16>(c, p, k, v, w, raw_kept, status, st);
    case 32: return launch_one<KIND, D, 32>(c, p, k, v, w, raw_kept, status, st);
    case 64: return launch_one<KIND, D, 64>(c, p, k, v, w, raw_kept, status, st);
    default: return launch_one<KIND, D, 128>(c, p, k, v, w, raw_kept, status, st);
  }
}

}  // namespace

cudaError_t launch_append(const View& c, const Plan& p, const bf16* k, const bf16* v, const float* conv_w,
                          int raw_kept, int32_t* status, cudaStream_t st) {
  if (c.d == 64)
    return c.kind == 0 ? launch_block<0, 64>(c, p, k, v, conv_w, raw_kept, status, st)
                       : launch_block<1, 64>(c, p, k, v, conv_w, raw_kept, status, st);
  return c.kind == 0 ? launch_block<0, 128>(c, p, k, v, conv_w, raw_kept, status, st)
                     : launch_block<1, 128>(c, p, k, v, conv_w, raw_kept, status, st);
}

}  // namespace cache
}  // namespace moba
