// Attention of new queries over the paged 8-bit cache:
//   s_i = q . (k8_i ks) / sqrt(d),  out = sum_i softmax(s)_i v8_i vs,  lse = log sum_i exp(s_i)
// over the tokens at positions <= the query's of the listed blocks (or all).
//
// Arithmetic.  An 8-bit code (e4m3 or int8) is exactly an fp16 value, so a page
// is multiplied as fp16 with fp32 sums and the block's scales stay outside:
// ks scales the score, vs is carried in the exponent.  With
//   x_i = s_i log2 e + log2 vs,   M = running max of x_i,   w_i = 2^(x_i - M + 15)
// the output is sum w_i v8_i / (2^15 l), l = sum w_i 2^-15 / vs = sum 2^(s_i log2 e - M),
// and log2 of the softmax sum is M + log2 l.  So no block's product has to be
// scaled on its own, whatever the spread of the scales (vs is taken as at
// least 2^-100, so that 1 / vs and l stay finite; the rest of a smaller scale
// is multiplied into w_i).  Queries are fp16 after a power of two per row that
// brings the row's largest magnitude to [2^8, 2^9): exact down to 2^-22 of
// it.  Weights are rounded to fp16 (2^-11, the offset 2^15 keeps weights down
// to 2^-29 of the largest out of the subnormals); their sum is kept in fp32
// from the unrounded ones.
//
// A partial block is bf16 (the tail) and is multiplied as bf16, its weights
// as hi + lo.
//
// Fragments (mma.m16n8k16; lane = 4 g + t).  Keys come 16 tokens (a unit) at a
// time.  Scores: A = queries, B = keys; column n of n-tile i is the unit's
// token 4 (n / 2) + 2 i + n % 2, and the k index runs over channels such that a
// lane's share of a key row is 16 contiguous bytes.  Then a lane's weights are
// those of tokens 4 t .. 4 t + 3, already in the layout of the A operand of
// the product with V, and its share of V is 4 token rows of D / 8 contiguous
// channels, transposed 4 x 4 bytes in registers; column n of output n-tile i
// is channel (D / 8) n + i.
#include <cuda_fp16.h>
#include <math_constants.h>

#include "cache.cuh"

namespace moba {
namespace cache {
namespace {

constexpr int kUnit = 16;        // tokens per unit
constexpr int kPair = 2;         // units per softmax step
constexpr float kOffset = 15.f;  // exponent of the largest weight
constexpr int kListCap = 256;    // list entries held in shared memory at a time

// ---------------------------------------------------------------- fragments
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8-bit codes to two fp16 pairs, exactly.
template <int KIND>
__device__ __forceinline__ void widen(uint32_t x, uint32_t& lo, uint32_t& hi) {
  if constexpr (KIND == 0) {
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
  } else {
    // 0x64bb is 1024 + bb; with bb = x + 128 subtract 1152.
    x ^= 0x80808080u;
    const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const __half2 ra = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 rb = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    lo = *reinterpret_cast<const uint32_t*>(&ra);
    hi = *reinterpret_cast<const uint32_t*>(&rb);
  }
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 4 x 4 byte transpose: x[i] = row i, y[c] = column c.
__device__ __forceinline__ void transpose4(const uint32_t* x, uint32_t* y) {
  const uint32_t a = __byte_perm(x[0], x[1], 0x5140), b = __byte_perm(x[2], x[3], 0x5140);
  const uint32_t c = __byte_perm(x[0], x[1], 0x7362), d = __byte_perm(x[2], x[3], 0x7362);
  y[0] = __byte_perm(a, b, 0x5410), y[1] = __byte_perm(a, b, 0x7632);
  y[2] = __byte_perm(c, d, 0x5410), y[3] = __byte_perm(c, d, 0x7632);
}

// Shared-memory places of the 16-byte chunk ck of row r of a unit's K and V
// (16 rows of D bytes).  Swizzled so that the fragment reads below touch every
// bank once per phase.
template <int D>
__device__ __forceinline__ uint32_t k_place(int r, int ck) {
  if constexpr (D == 128) return r * 128 + ((ck ^ ((r & 1) << 2)) << 4);
  else return r * 64 + (ck << 4);
}
template <int D>
__device__ __forceinline__ uint32_t v_place(int r, int ck) {
  const int x = 2 * ((r >> 2) & 3);
  if constexpr (D == 128) return r * 128 + ((ck ^ x) << 4);
  else return (r >> 1) * 128 + ((((r & 1) * 4 + ck) ^ x) << 4);
}

// Starts the copy of one unit (K, then V) into shared memory; zeros where
// there is none.
template <int D>
__device__ __forceinline__ void fetch_unit(unsigned char* dst, const uint8_t* kp, const uint8_t* vp, bool valid, int lane) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int c = lane + 32 * i, r = c / (D / 16), ck = c % (D / 16);
    cp_async16_zfill(dst + k_place<D>(r, ck), kp + c * 16, valid);
    cp_async16_zfill(dst + 16 * D + v_place<D>(r, ck), vp + c * 16, valid);
  }
}

// Scores of one unit: s[i][*] of n-tile i.  qf: D / 16 fragments of the queries.
template <int D, int KIND>
__device__ __forceinline__ void unit_scores(const unsigned char* kt, const uint32_t (*qf)[4], float (*s)[4], int g, int t) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = (g >> 1) * 4 + 2 * i + (g & 1);
#pragma unroll
    for (int x = 0; x < 4; ++x) s[i][x] = 0.f;
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh) {
      const uint4 w = *reinterpret_cast<const uint4*>(kt + k_place<D>(r, 4 * hh + t));
      const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t b0, b1;
        widen<KIND>(ws[x], b0, b1);
        mma_f16(s[i], qf[hh * 4 + x], b0, b1);
      }
    }
  }
}

// o += weights (A fragment pf) times the unit's V.
template <int D, int KIND>
__device__ __forceinline__ void unit_values(const unsigned char* vt, const uint32_t* pf, float (*o)[4], int g, int t) {
  constexpr int NW = D / 32;  // words of 4 channels per lane and token
  uint32_t x[4][NW];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * t + i;
    if constexpr (D == 128) {
      const uint4 w = *reinterpret_cast<const uint4*>(vt + v_place<D>(r, g));
      x[i][0] = w.x, x[i][1] = w.y, x[i][2] = w.z, x[i][3] = w.w;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(vt + v_place<D>(r, g >> 1) + (g & 1) * 8);
      x[i][0] = w.x, x[i][1] = w.y;
    }
  }
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const uint32_t in[4] = {x[0][w], x[1][w], x[2][w], x[3][w]};
    uint32_t y[4];
    transpose4(in, y);
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
      uint32_t b0, b1;
      widen<KIND>(y[ch], b0, b1);
      mma_f16(o[4 * w + ch], pf, b0, b1);
    }
  }
}

// Running softmax state of a warp's 16 rows (this lane: rows g and g + 8).
template <int D>
struct State {
  float m[2], l[2];
  float o[D / 8][4];
  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -CUDART_INF_F;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[i][x] = 0.f;
  }
  // Raises the reference to cover `mx` (this lane's maxima over its columns).
  __device__ __forceinline__ void raise(float mx0, float mx1) {
    float mx[2] = {mx0, mx1};
    bool up = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(~0u, mx[r], 2));
      up |= mx[r] > m[r];
    }
    if (__any_sync(~0u, up)) {
      float a[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float n = fmaxf(m[r], mx[r]);
        a[r] = n > m[r] ? fast_exp2(m[r] - n) : 1.f;  // m = -inf: 0
        m[r] = n;
        l[r] *= a[r];
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= a[0], o[i][1] *= a[0];
        o[i][2] *= a[1], o[i][3] *= a[1];
      }
    }
  }
  // Subtrahend of the exponent: w = 2^(x - base).
  __device__ __forceinline__ float base(int r) const { return (m[r] == -CUDART_INF_F ? 0.f : m[r]) - kOffset; }
};

// One block as the unit loop sees it.
struct __align__(16) Entry {
  int page;  // -1: skip
  int j;
  float ks;
  float lv;    // log2 of the V scale, taken as at least 2^-100
  float rest;  // V scale over that (1 but for smaller scales)
  float inv;   // 2^-15 over that
  float pad[2];
};

__device__ __forceinline__ Entry make_entry(const View& c, int page, int j, int head) {
  const size_t at = (size_t)page * c.h_kv + head;
  const float s = __ldg(c.v_scale + at), vs = fmaxf(s, 7.8886090522101181e-31f);
  return Entry{page, j, __ldg(c.k_scale + at), log2f(vs), s / vs, (1.f / 32768.f) / vs, {0.f, 0.f}};
}

struct Tile {
  int row;        // request
  int head;       // KV head
  int t0;         // first token of the request's part of the step
  int r0;         // first flattened row (token * G + group member) of the tile
  int nrows;      // flattened rows of the request
  int max_pos;    // largest position among the tile's rows
};

template <int D>
struct Layout {
  static constexpr int kStage = kPair * 2 * kUnit * D;  // bytes of a pair of units, K and V
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kQ = 16 * (D + 8) * 2;           // bf16 queries, rows padded by 16 bytes
  static constexpr int kList = kListCap * (int)sizeof(Entry);
  static constexpr int bytes(int nw) { return kList + kQ + nw * kStages * kStage; }
  static constexpr int kORow = D + 4;                   // floats per merged row: D, then m, l
  static_assert(16 * kORow * 4 <= kStages * kStage, "merge buffer fits the ring");
};

// One partial-block unit (16 tokens from `first` on, `n` of them real) from the tail.
template <int D>
__device__ __forceinline__ void tail_unit(const bf16* tk, const bf16* tv, int first, int n, int pos_first,
                                          const bf16* qs, const float* fac, const int* pos, State<D>& st, int g, int t) {
  float s[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = first + (g >> 1) * 4 + 2 * i + (g & 1);
#pragma unroll
    for (int x = 0; x < 4; ++x) s[i][x] = 0.f;
#pragma unroll
    for (int hh = 0; hh < D / 64; ++hh) {
      uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (r < n) {
        const uint4* src = reinterpret_cast<const uint4*>(tk + (size_t)r * D + 64 * hh + 16 * t);
        w[0] = src[0], w[1] = src[1];
      }
      const uint32_t ws[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bf16* q0 = qs + g * (D + 8) + 64 * hh + 16 * t + 4 * x;
        const bf16* q1 = q0 + 8 * (D + 8);
        const uint2 a = *reinterpret_cast<const uint2*>(q0), b = *reinterpret_cast<const uint2*>(q1);
        const uint32_t qa[4] = {a.x, b.x, a.y, b.y};
        mma_bf16(s[i], qa, ws[2 * x], ws[2 * x + 1]);
      }
    }
  }
  float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int p = pos_first + first + 4 * t + 2 * i + (x & 1), r = x >> 1;
      s[i][x] = p <= pos[r] && first + 4 * t + 2 * i + (x & 1) < n ? s[i][x] * fac[r] : -CUDART_INF_F;
      mx[r] = fmaxf(mx[r], s[i][x]);
    }
  st.raise(mx[0], mx[1]);
  const float base[2] = {st.base(0), st.base(1)};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      s[i][x] = fast_exp2(s[i][x] - base[x >> 1]);
      st.l[x >> 1] += s[i][x] * (1.f / 32768.f);
    }
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float a = s[i][2 * r], b = s[i][2 * r + 1];
      const uint32_t h = pack_bf16(a, b);
      hi[2 * i + r] = h;
      lo[2 * i + r] = pack_bf16(a - __uint_as_float(h << 16), b - __uint_as_float(h & 0xffff0000u));
    }
#pragma unroll
  for (int half = 0; half < D / 64; ++half) {  // 8 channels per lane at a time
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = first + 4 * t + i;
      w[i] = make_uint4(0, 0, 0, 0);
      if (r < n) w[i] = *reinterpret_cast<const uint4*>(tv + (size_t)r * D + (D / 8) * g + 8 * half);
    }
    const uint32_t* ww[4] = {&w[0].x, &w[1].x, &w[2].x, &w[3].x};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t b0 = __byte_perm(ww[0][i], ww[1][i], e ? 0x7632 : 0x5410);
        const uint32_t b1 = __byte_perm(ww[2][i], ww[3][i], e ? 0x7632 : 0x5410);
        mma_bf16(st.o[8 * half + 2 * i + e], hi, b0, b1);
        mma_bf16(st.o[8 * half + 2 * i + e], lo, b0, b1);
      }
  }
}

// A CTA takes up to 16 query rows that read the same blocks: the query heads
// of a KV head's group over some tokens of one request (all blocks), or one
// (token, query head) with its own list (selected).  Its warps take pairs of
// units in turn, each with its own ring of copies in flight, and are merged at
// the end; with several splits the split's result goes to `part`.
template <int D, int KIND, int NW, bool SEL>
__global__ void __launch_bounds__(NW * 32)
attn_kernel(View c, Plan p, const bf16* __restrict__ q, int h_q, const int32_t* __restrict__ sel, int topk,
            int per_token, int split_blocks, int nsplit, bf16* __restrict__ out, float* __restrict__ lse,
            float* __restrict__ part, int32_t* status) {
  using Ly = Layout<D>;
  extern __shared__ __align__(128) unsigned char smem[];
  Entry* list = reinterpret_cast<Entry*>(smem);
  bf16* qs = reinterpret_cast<bf16*>(smem + Ly::kList);
  unsigned char* ring = smem + Ly::kList + Ly::kQ + (threadIdx.x >> 5) * Ly::kStages * Ly::kStage;
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int G = h_q / c.h_kv;

  // ---- the tile
  Tile T;
  int split = 0;
  if constexpr (SEL) {
    const int tok = blockIdx.x, h = blockIdx.y;
    T.row = __ldg(p.row + tok);
    if ((unsigned)T.row >= (unsigned)c.rows) return;
    T.head = h / G;
    T.t0 = tok;
    T.r0 = h % G;
    T.nrows = h % G + 1;
  } else {
    T.head = blockIdx.y;
    split = blockIdx.z;
    const int u = blockIdx.x;
    if (per_token) {
      const int tiles = (G + 15) / 16;
      T.t0 = u / tiles;
      T.row = __ldg(p.row + T.t0);
      if ((unsigned)T.row >= (unsigned)c.rows) return;
      T.r0 = (u % tiles) * 16;
      T.nrows = G;
    } else {
      int lo = 0, hi = c.rows;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((long long)__ldg(p.cu + mid) * G / 16 + mid <= u) lo = mid; else hi = mid;
      }
      T.row = lo;
      T.t0 = __ldg(p.cu + lo);
      T.r0 = (int)(u - ((long long)T.t0 * G / 16 + lo)) * 16;
      T.nrows = (min(__ldg(p.cu + lo + 1), p.T) - T.t0) * G;
      if (T.r0 >= T.nrows) return;
    }
  }
  const int len = c.state[2 * T.row], held = c.state[2 * T.row + 1];
  const int rows = min(16, T.nrows - T.r0);  // real rows of the tile
  // Position of a tile row; -1 for rows that see nothing.
  auto pos_of = [&](int r) {
    if (r >= rows) return -1;
    const int x = __ldg(p.pos + T.t0 + (T.r0 + r) / G);
    return x < len && x / c.B < held ? x : -1;
  };
  int pos[2] = {pos_of(g), pos_of(g + 8)};
  int mp = max(pos[0], pos[1]);
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) mp = max(mp, __shfl_xor_sync(~0u, mp, off));
  T.max_pos = mp;
  if (tid < rows && split == 0 && pos_of(tid) != __ldg(p.pos + T.t0 + (T.r0 + tid) / G)) set_status(status, kStatusBadTable);

  // ---- queries: bf16 in shared memory, fp16 fragments after scaling by a power of two
  auto item_of = [&](int r) {  // (token, query head) of a tile row
    return (size_t)(T.t0 + (T.r0 + r) / G) * h_q + T.head * G + (T.r0 + r) % G;
  };
  for (int i = tid; i < 16 * (D / 8); i += NW * 32) {
    const int r = i / (D / 8), ck = i % (D / 8);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < rows) x = *reinterpret_cast<const uint4*>(q + item_of(r) * D + ck * 8);
    *reinterpret_cast<uint4*>(qs + r * (D + 8) + ck * 8) = x;
  }
  const int own = mp < 0 ? -1 : mp / c.B;
  const bool tail = own >= 0 && (long long)(own + 1) * c.B > len;  // the last block is partial
  int b0 = 0, b1 = own + 1;                                        // blocks of this CTA
  bool my_tail = tail;
  if constexpr (!SEL) {
    b0 = min(b1, split * split_blocks);
    const int e = min(b1, b0 + split_blocks);
    my_tail = tail && e == b1 && b0 < b1;
    b1 = e;
    if (split > 0 && b0 >= b1) return;
  }
  __syncthreads();
  uint32_t qf[D / 16][4];
  float fac[2];
  {
    float am[2] = {0.f, 0.f};
    uint2 raw[2][D / 16];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        raw[r][k] = *reinterpret_cast<const uint2*>(qs + (g + 8 * r) * (D + 8) + 64 * (k / 4) + 16 * t + 4 * (k % 4));
        const uint32_t w[2] = {raw[r][k].x, raw[r][k].y};
#pragma unroll
        for (int e = 0; e < 2; ++e)
          am[r] = fmaxf(am[r], fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      am[r] = fmaxf(am[r], __shfl_xor_sync(~0u, am[r], 1));
      am[r] = fmaxf(am[r], __shfl_xor_sync(~0u, am[r], 2));
      // exponent of the largest magnitude, kept where the factors are normal
      const int e = max(-100, min(127, (int)((__float_as_uint(am[r]) >> 23) & 255) - 127));
      const float up = __uint_as_float((uint32_t)(8 - e + 127) << 23);
      fac[r] = __uint_as_float((uint32_t)(e - 8 + 127) << 23) * (kLog2e * rsqrtf((float)D));
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t w[2] = {raw[r][k].x, raw[r][k].y};
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2)
          qf[k][2 * e2 + r] = pack_f16(__uint_as_float(w[e2] << 16) * up, __uint_as_float(w[e2] & 0xffff0000u) * up);
      }
    }
  }
  int min_pos = min(g < rows ? pos[0] : 0x7fffffff, g + 8 < rows ? pos[1] : 0x7fffffff);
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) min_pos = min(min_pos, __shfl_xor_sync(~0u, min_pos, off));

  State<D> st;
  st.clear();
  const int upb = c.B / kUnit;
  const size_t page_bytes = (size_t)c.B * D;
  bool tail_done = !my_tail;

  // ---- chunks of the list
  const int n_list = SEL ? topk : (my_tail ? b1 - 1 : b1) - b0;
  int done = 0;
  do {
    const int n = SEL ? n_list : min(kListCap, n_list - done);
    if constexpr (SEL) {
      if (warp == 0) {
        int count = 0, prev = -1;
        bool want_tail = false;
        for (int base = 0; base < n; base += 32) {
          const int e = base + lane;
          const int j = e < n ? __ldg(sel + ((size_t)T.t0 * h_q + T.head * G + T.r0) * topk + e) : -1;
          const bool in = j >= 0 && j <= own;
          int top = in ? j : -1;  // running maximum before this lane
          for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(~0u, top, off);
            if (lane >= off) top = max(top, o);
          }
          int before = __shfl_up_sync(~0u, top, 1);
          before = max(prev, lane ? before : -1);
          prev = max(prev, __shfl_sync(~0u, top, 31));
          bool ok = in && j > before;
          if (j != -1 && own >= 0 && !ok) set_status(status, kStatusBadSelIdx);
          if (ok && tail && j == own) {
            want_tail = true;
            ok = false;
          }
          const int pg = ok ? block_page(c, T.row, j) : -1;
          if (ok && pg < 0) {
            set_status(status, kStatusBadTable);
            ok = false;
          }
          const uint32_t m = __ballot_sync(~0u, ok);
          if (ok) list[count + __popc(m & ((1u << lane) - 1))] = make_entry(c, pg, j, T.head);
          count += __popc(m);
        }
        want_tail = __any_sync(~0u, want_tail);
        if (lane == 0) s_count = count | (want_tail ? 1 << 16 : 0);
      }
    } else {
      for (int e = tid; e < n; e += NW * 32) {
        const int j = b0 + done + e;
        const int pg = block_page(c, T.row, j);
        if (pg < 0) set_status(status, kStatusBadTable);
        list[e] = pg >= 0 ? make_entry(c, pg, j, T.head) : Entry{-1, j, 0.f, 0.f, 0.f, 0.f, {0.f, 0.f}};
      }
    }
    __syncthreads();
    int count = n;
    if constexpr (SEL) {
      count = s_count & 0xffff;
      tail_done = !(s_count >> 16);
    }
    // Units of the listed blocks; the last one may end before its block does.
    int units = count * upb;
    if (count > 0 && list[count - 1].j == own) units -= upb - (mp - own * c.B) / kUnit - 1;
    const int pairs = (units + kPair - 1) / kPair;
    const int mine = warp < pairs ? (pairs - warp + NW - 1) / NW : 0;
    auto fetch = [&](int i) {
      if (i < mine) {
        unsigned char* dst = ring + (i % Ly::kStages) * Ly::kStage;
#pragma unroll
        for (int x = 0; x < kPair; ++x) {
          const int u = (warp + i * NW) * kPair + x;
          const Entry e = list[u < units ? u / upb : 0];
          const bool ok = u < units && e.page >= 0;
          const size_t at = ok ? ((size_t)e.page * c.h_kv + T.head) * page_bytes + (size_t)(u % upb) * (kUnit * D) : 0;
          fetch_unit<D>(dst + x * 2 * kUnit * D, c.k + at, c.v + at, ok, lane);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < Ly::kStages - 1; ++i) fetch(i);
    // the partial block's units go round the warps while the first copies are in flight
    if (!tail_done) {
      const int n_tail = mp - own * c.B + 1;
      const size_t at = (((size_t)T.row * 2 + (own & 1)) * c.h_kv + T.head) * page_bytes;
      const float f[2] = {kLog2e * rsqrtf((float)D), kLog2e * rsqrtf((float)D)};
      for (int u = (NW - 1 - warp); u * kUnit < n_tail; u += NW)
        tail_unit<D>(c.tail_k + at, c.tail_v + at, u * kUnit, n_tail, own * c.B, qs, f, pos, st, g, t);
      tail_done = true;
    }
    for (int i = 0; i < mine; ++i) {
      fetch(i + Ly::kStages - 1);
      cp_async_wait<Ly::kStages - 1>();
      __syncwarp();
      const unsigned char* src = ring + (i % Ly::kStages) * Ly::kStage;
      float s[2 * kPair][4];
      float mx[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
      for (int x = 0; x < kPair; ++x) {
        const int u = (warp + i * NW) * kPair + x;
        unit_scores<D, KIND>(src + x * 2 * kUnit * D, qf, s + 2 * x, g, t);
        const Entry e = list[u < units ? u / upb : 0];
        const int p0 = u < units && e.page >= 0 ? e.j * c.B + (u % upb) * kUnit : 0x7fffffff - kUnit;
        const float f[2] = {fac[0] * e.ks, fac[1] * e.ks};
        const bool cut = p0 + kUnit - 1 > min_pos;
#pragma unroll
        for (int n8 = 0; n8 < 2; ++n8)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float& z = s[2 * x + n8][y];
            z = fmaf(z, f[y >> 1], e.lv);
            if (cut && p0 + 4 * t + 2 * n8 + (y & 1) > pos[y >> 1]) z = -CUDART_INF_F;
            mx[y >> 1] = fmaxf(mx[y >> 1], z);
          }
      }
      st.raise(mx[0], mx[1]);
      const float base[2] = {st.base(0), st.base(1)};
#pragma unroll
      for (int x = 0; x < kPair; ++x) {
        const int u = (warp + i * NW) * kPair + x;
        const float rest = list[u < units ? u / upb : 0].rest, inv = list[u < units ? u / upb : 0].inv;
        uint32_t pf[4];
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int n8 = 0; n8 < 2; ++n8) {
          float* z = s[2 * x + n8];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            z[y] = fast_exp2(z[y] - base[y >> 1]);
            sum[y >> 1] += z[y];
          }
          pf[2 * n8] = pack_f16(z[0] * rest, z[1] * rest);
          pf[2 * n8 + 1] = pack_f16(z[2] * rest, z[3] * rest);
        }
        st.l[0] += sum[0] * inv, st.l[1] += sum[1] * inv;
        unit_values<D, KIND>(src + x * 2 * kUnit * D + kUnit * D, pf, st.o, g, t);
      }
      __syncwarp();
    }
    cp_async_wait<0>();
    __syncthreads();
    done += n;
  } while (!SEL && done < n_list);

  // ---- merge the warps
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    st.l[r] += __shfl_xor_sync(~0u, st.l[r], 1);
    st.l[r] += __shfl_xor_sync(~0u, st.l[r], 2);
  }
  float* buf = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float* b = buf + (g + 8 * r) * Ly::kORow;
    if (g + 8 * r < rows) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        b[(D / 8) * (2 * t) + i] = st.o[i][2 * r];
        b[(D / 8) * (2 * t + 1) + i] = st.o[i][2 * r + 1];
      }
      if (t == 0) b[D] = st.m[r], b[D + 1] = st.l[r];
    }
  }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(smem + Ly::kList + Ly::kQ);
  constexpr int kStep = Ly::kStages * Ly::kStage / 4;
  for (int i = tid; i < rows * (D / 4); i += NW * 32) {
    const int r = i / (D / 4), ch = (i % (D / 4)) * 4;
    float M = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, all[w * kStep + r * Ly::kORow + D]);
    float l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float* b = all + w * kStep + r * Ly::kORow;
      const float a = b[D] == -CUDART_INF_F ? (b[D + 1] == b[D + 1] ? 0.f : 1.f) : fast_exp2(b[D] - M);
      l += a * b[D + 1];
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] += a * b[ch + x];
    }
    const size_t item = item_of(r);
    if (nsplit == 1) {
      const float inv = l == 0.f ? 0.f : 1.f / (32768.f * l);
      uint2 y;
      y.x = pack_bf16(o[0] * inv, o[1] * inv), y.y = pack_bf16(o[2] * inv, o[3] * inv);
      *reinterpret_cast<uint2*>(out + item * D + ch) = y;
      if (ch == 0) lse[item] = l == 0.f ? -CUDART_INF_F : (M + log2f(l)) * 0.69314718055994531f;
    } else {
      float* b = part + (item * nsplit + split) * Ly::kORow;
      *reinterpret_cast<float4*>(b + ch) = make_float4(o[0], o[1], o[2], o[3]);
      if (ch == 0) b[D] = M, b[D + 1] = l;
    }
  }
}

// Joins the splits of one (token, query head) per warp.
template <int D>
__global__ void __launch_bounds__(128)
merge_kernel(View c, Plan p, int h_q, int split_blocks, int nsplit, const float* __restrict__ part,
             bf16* __restrict__ out, float* __restrict__ lse) {
  constexpr int kORow = Layout<D>::kORow, E = D / 32;
  const int lane = threadIdx.x & 31;
  const size_t item = (size_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= (size_t)p.T * h_q) return;
  const int tok = (int)(item / h_q), row = __ldg(p.row + tok);
  if ((unsigned)row >= (unsigned)c.rows) return;
  const int pos = __ldg(p.pos + tok);
  // splits that wrote: as many as the tile's furthest row needs; a row's own are the first of those
  const int n = pos < 0 || pos >= c.state[2 * row] || pos / c.B >= c.state[2 * row + 1] ? 0 : pos / c.B / split_blocks + 1;
  const float* b = part + item * nsplit * kORow;
  float M = -CUDART_INF_F, l = 0.f, o[E];
#pragma unroll
  for (int x = 0; x < E; ++x) o[x] = 0.f;
  for (int s = 0; s < n; ++s) M = fmaxf(M, b[s * kORow + D]);
  for (int s = 0; s < n; ++s) {
    const float m = b[s * kORow + D], ls = b[s * kORow + D + 1];
    const float a = m == -CUDART_INF_F ? (ls == ls ? 0.f : 1.f) : fast_exp2(m - M);
    l += a * ls;
#pragma unroll
    for (int x = 0; x < E; ++x) o[x] += a * b[s * kORow + lane * E + x];
  }
  const float inv = l == 0.f ? 0.f : 1.f / (32768.f * l);
#pragma unroll
  for (int x = 0; x < E; x += 2)
    *reinterpret_cast<uint32_t*>(out + item * D + lane * E + x) = pack_bf16(o[x] * inv, o[x + 1] * inv);
  if (lane == 0) lse[item] = l == 0.f ? -CUDART_INF_F : (M + log2f(l)) * 0.69314718055994531f;
}

// How a step over all blocks is cut up.
struct Cut {
  bool many;       // tiles of 128 rows (cache_attn_rows.cu) instead of 16
  bool per_token;  // tiles of 16: each token on its own, or a request's tokens together, whichever bound is less
  long long tiles;
  int split_blocks, nsplit;
};

// Long rows are cut into splits of whole blocks, so that even few tiles fill
// the GPU: about four CTAs per SM counted over rows of full length, and at
// least 512 tokens each (a split costs a partial result of D + 4 floats per
// query row, written and read back).
Cut cut_of(const View& c, int T, int h_q) {
  const int G = h_q / c.h_kv;
  const long long a = (long long)T * ((G + 15) / 16), b = (long long)T * G / 16 + c.rows;
  const long long big = (long long)T * G / 128 + (T < c.rows ? T : c.rows);
  Cut x;
  x.per_token = a <= b;
  x.tiles = x.per_token ? a : b;
  x.many = x.tiles >= 2 * big;
  if (x.many) x.tiles = (long long)T * G / 128 + c.rows;
  const long long ctas = (x.many ? big : x.tiles) * c.h_kv;
  const long long want = ((x.many ? 6 : 4) * 148 + ctas - 1) / ctas;
  const long long step = x.many && c.B < 128 ? 128 / c.B : 1;  // splits of whole key tiles
  const long long least = (512 + c.B - 1) / c.B;
  long long blocks = (c.max_blocks + want - 1) / want;
  if (blocks < least) blocks = least;
  blocks = (blocks + step - 1) / step * step;
  x.split_blocks = (int)blocks;
  x.nsplit = (int)((c.max_blocks + blocks - 1) / blocks);
  return x;
}

template <int D, int KIND>
cudaError_t launch_all(const View& c, const Plan& p, const bf16* q, int h_q, const int32_t* sel, int topk, bf16* out,
                       float* lse, float* part, int32_t* status, cudaStream_t st) {
  using Ly = Layout<D>;
  cudaError_t e;
  if (sel) {
    const dim3 grid(p.T, h_q);
    // few rows: more warps each, so that their blocks are read at once
    if ((long long)p.T * h_q > 2 * 148) {
      constexpr int NW = 4;
      if ((e = cudaFuncSetAttribute(attn_kernel<D, KIND, NW, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Ly::bytes(NW))) != cudaSuccess)
        return e;
      attn_kernel<D, KIND, NW, true><<<grid, NW * 32, Ly::bytes(NW), st>>>(c, p, q, h_q, sel, topk, 0, 0, 1, out, lse,
                                                                          nullptr, status);
    } else {
      constexpr int NW = 8;
      if ((e = cudaFuncSetAttribute(attn_kernel<D, KIND, NW, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Ly::bytes(NW))) != cudaSuccess)
        return e;
      attn_kernel<D, KIND, NW, true><<<grid, NW * 32, Ly::bytes(NW), st>>>(c, p, q, h_q, sel, topk, 0, 0, 1, out, lse,
                                                                          nullptr, status);
    }
    return cudaGetLastError();
  }
  const Cut x = cut_of(c, p.T, h_q);
  if (x.many) {
    e = launch_attention_rows(c, p, q, h_q, (int)x.tiles, x.split_blocks, x.nsplit, out, lse, part, status, st);
    if (e != cudaSuccess || x.nsplit == 1) return e;
  } else {
    constexpr int NW = 4;
    if ((e = cudaFuncSetAttribute(attn_kernel<D, KIND, NW, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  Ly::bytes(NW))) != cudaSuccess)
      return e;
    attn_kernel<D, KIND, NW, false><<<dim3((unsigned)x.tiles, c.h_kv, x.nsplit), NW * 32, Ly::bytes(NW), st>>>(
        c, p, q, h_q, nullptr, 0, x.per_token, x.split_blocks, x.nsplit, out, lse, part, status);
    if ((e = cudaGetLastError()) != cudaSuccess || x.nsplit == 1) return e;
  }
  const long long items = (long long)p.T * h_q;
  merge_kernel<D><<<(unsigned)((items + 3) / 4), 128, 0, st>>>(c, p, h_q, x.split_blocks, x.nsplit, part, out, lse);
  return cudaGetLastError();
}

}  // namespace

size_t attn_scratch(const View& c, int T, int h_q) {
  if (T == 0) return 0;
  const Cut x = cut_of(c, T, h_q);
  return x.nsplit == 1 ? 0 : (size_t)T * h_q * x.nsplit * (c.d + 4) * sizeof(float);
}

cudaError_t launch_attention(const View& c, const Plan& p, const bf16* q, int h_q, const int32_t* sel, int topk,
                             bf16* out, float* lse, void* scratch, int32_t* status, cudaStream_t st) {
  float* part = static_cast<float*>(scratch);
  if (c.d == 64)
    return c.kind == 0 ? launch_all<64, 0>(c, p, q, h_q, sel, topk, out, lse, part, status, st)
                       : launch_all<64, 1>(c, p, q, h_q, sel, topk, out, lse, part, status, st);
  return c.kind == 0 ? launch_all<128, 0>(c, p, q, h_q, sel, topk, out, lse, part, status, st)
                     : launch_all<128, 1>(c, p, q, h_q, sel, topk, out, lse, part, status, st);
}

}  // namespace cache
}  // namespace moba
