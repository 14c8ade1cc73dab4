// Attention of new queries over the paged 8-bit cache:
//   s_i = q . (k8_i ks) / sqrt(d),  out = sum_i softmax(s)_i v8_i vs,  lse = log sum_i exp(s_i)
// over the tokens at positions <= the query's of the listed blocks (or all).
//
// Arithmetic.  An 8-bit code (e4m3 or int8) is exactly an fp16 value, so a page
// is multiplied as fp16 with fp32 sums and the block's scales stay outside:
// ks scales the score, vs is carried in the exponent.  With
//   x_i = s_i log2 e + log2 vs,   M >= max x_i - 8,   w_i = 2^(x_i - M + 7) <= 2^15
// the output is sum w_i v8_i / (2^7 l), l = sum w_i 2^-7 / vs = sum 2^(s_i log2 e - M),
// and log2 of the softmax sum is M + log2 l.  The reference M follows the
// running maximum only when that has grown by more than 8, so in most steps
// nothing is reduced across lanes or rescaled.  So no block's product has to be
// scaled on its own (vs is taken as at least 2^-100, so that 1 / vs and l stay
// finite; the rest of a smaller scale is multiplied into w_i).  Beside blocks of
// ordinary size the w_i of a scale below 2^-40 (of zeros, mostly) may be 0 in 32
// bits; what they add to l is formed without vs.  Of larger scales those that one
// row sees may lie 2^100 apart.  Queries are fp16 after a power of two per row that
// brings the row's largest magnitude to [2^8, 2^9): exact down to 2^-22 of
// it.  Weights are rounded to fp16 (2^-11; those below 2^-21 of the one at the
// reference are subnormal, with steps of 2^-31 of it); their sum is kept in fp32
// from the unrounded ones.  Where all of a row's scales are below 2^-100 (values
// below 2^-91) the steps stay those of a scale of 2^-100: an output is then off
// by up to 2^-132 times the largest code for each key.
//
// A partial block is bf16 (the tail) and is multiplied as bf16, its weights
// 2^(s_i log2 e - M + 7) as hi + lo; in M it counts with its largest |v| / 448.
//
// Fragments (mma.m16n8k16; lane = 4 g + t).  Keys come 16 tokens (a unit) at a
// time and are the M side of both products, so that up to 8 query rows (the
// heads of a group) fill the N side: scores^T = K q^T, out^T = V^T w^T.  Row r
// of the scores is the unit's token 4 (r / 2) + r % 2 (r < 8; + 2 for r + 8),
// and the k index runs over channels such that a lane's share of a key row is
// 16 contiguous bytes.  Transposed in place (movmatrix), a lane's weights are
// those of tokens 4 t .. 4 t + 3; its share of V is those 4 token rows of D / 8
// contiguous channels, transposed 4 x 4 bytes in registers, and row r of
// output tile i is channel (D / 8) (r % 8) + 2 i + r / 8.
//
// Each warp has its own ring of pages on their way (cp.async) and its own
// softmax, joined at the end of the CTA; no warp waits for another.  Bound by
// HBM: 24 single tokens of 32 heads over 4K to 64K keys of 8 heads of 128
// (1.17 GB) 212 us, of which the kernel about 205 at 5.7 TB/s; 64 rows of 16 heads of 64 over their 32 selected blocks of 32 (134
// MB) 33 us, 4.3 TB/s, the rest the look-ups before the first page.  One token
// over 64K keys of 8 heads 39 us, of 32 selected blocks 10.
#include <math_constants.h>

#include "cache.cuh"

namespace moba {
namespace cache {
namespace {

constexpr int kUnit = 16;        // tokens per unit
constexpr int kPair = 2;         // units per softmax step
constexpr int kListCap = 128;    // list entries held in shared memory at a time

// 2^x down to the end of 32 bits (fast_exp2 gives 0 from 2^-126 on).
__device__ __forceinline__ float exp2_small(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------- fragments
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Scores of one unit for 8 NT query rows: s[n][0, 1] of token 4 (g / 2) + g % 2 and rows 8 n + 2 t, + 1; s[n][2, 3] of
// the token 2 behind.  qf[n][k]: the queries' fragments.
template <int D, int KIND, int NT>
__device__ __forceinline__ void unit_scores(const unsigned char* kt, const uint32_t (*qf)[D / 16][2], float (*s)[4], int g, int t) {
  const int r = (g >> 1) * 4 + (g & 1);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
#pragma unroll
  for (int hh = 0; hh < D / 64; ++hh) {
    const uint4 u = *reinterpret_cast<const uint4*>(kt + k_place<D>(r, 4 * hh + t));
    const uint4 v = *reinterpret_cast<const uint4*>(kt + k_place<D>(r + 2, 4 * hh + t));
    const uint32_t us[4] = {u.x, u.y, u.z, u.w}, vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      uint32_t a[4];
      widen<KIND>(us[x], a[0], a[2]);
      widen<KIND>(vs[x], a[1], a[3]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(s[n], a, qf[n][hh * 4 + x][0], qf[n][hh * 4 + x][1]);
    }
  }
}

// o += the unit's V times weights (B fragments pf).
template <int D, int KIND, int NT>
__device__ __forceinline__ void unit_values(const unsigned char* vt, const uint32_t (*pf)[2], float (*o)[D / 16][4], int g, int t) {
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
    for (int c2 = 0; c2 < 2; ++c2) {
      uint32_t a[4];
      widen<KIND>(y[2 * c2], a[0], a[2]);
      widen<KIND>(y[2 * c2 + 1], a[1], a[3]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(o[n][2 * w + c2], a, pf[n][0], pf[n][1]);
    }
  }
}

// Running softmax state of a warp's 8 NT rows (this lane: rows 8 n + 2 t + b).
template <int D, int NT>
struct State {
  float m[NT][2], l[NT][2];
  float o[NT][D / 16][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -CUDART_INF_F;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[n][i][x] = 0.f;
    }
  }
  // Raises the references to mx (this lane's maxima over its tokens) where one has been outgrown by more than the slack.
  __device__ __forceinline__ void raise(float (*mx)[2]) {
    bool up = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) up |= mx[n][0] > m[n][0] + kSlack || mx[n][1] > m[n][1] + kSlack;  // m = -inf: any
    if (__any_sync(~0u, up)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float a[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float x = mx[n][b];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, off));
          x = fmaxf(m[n][b], x);
          const float h = x > m[n][b] ? fast_exp2(0.5f * (m[n][b] - x)) : 1.f;  // m = -inf: 0
          a[b] = h * h;
          m[n][b] = x;
          l[n][b] = l[n][b] * h * h;  // in halves: l may be as large as a is small
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[n][i][0] *= a[0], o[n][i][1] *= a[1];
          o[n][i][2] *= a[0], o[n][i][3] *= a[1];
        }
      }
    }
  }
  // Subtrahend of the exponent: w = 2^(x - base).
  __device__ __forceinline__ float base(int n, int b) const {
    return (m[n][b] == -CUDART_INF_F ? 0.f : m[n][b]) - kOffset;
  }
};

// One block as the unit loop sees it.
struct __align__(16) Entry {
  long long at;  // byte offset of its K and V tiles; -1: skip
  int pos;       // position of its first token
  float ks;
  float lv;      // log2 of the V scale, taken as at least 2^-100
  float rest;    // V scale over that (1 but for smaller scales)
  float inv;     // 2^-7 over lv's; 0 for a scale below 2^-40, whose weights are added to l without it
  float pad;
};

__device__ __forceinline__ Entry make_entry(const View& c, int page, int j, int head) {
  const size_t at = (size_t)page * c.h_kv + head;
  const float s = __ldg(c.v_scale + at), vs = fmaxf(s, 7.8886090522101181e-31f);
  return Entry{(long long)at * c.B * c.d, j * c.B, __ldg(c.k_scale + at), log2f(vs), s / vs,
               s < kSmallScale ? 0.f : (1.f / 128.f) / vs, 0.f};
}

// How the tiles of attn_kernel are found, and what each does of its row.
enum : int { kPerToken, kSearch, kSlots };
struct Few {
  int mode;
  int limit;      // query rows per KV head from which a request is left to cache_attn_rows.cu
  int slot_rows;  // kSlots: rows per request
  int split_blocks, nsplit;
};

struct Tile {
  int row;        // request
  int head;       // KV head
  int t0;         // first token of the request's part of the step
  int r0;         // first flattened row (token * G + group member) of the tile
  int nrows;      // flattened rows of the request
};

template <int D>
struct Layout {
  static constexpr int kStage = kPair * 2 * kUnit * D;  // bytes of a pair of units, K and V
  static constexpr int kStages = D == 128 ? 2 : 3;
  static constexpr int kList = kListCap * (int)sizeof(Entry);
  static constexpr int q_bytes(int nt) { return 8 * nt * (D + 8) * 2; }  // bf16 queries, rows padded by 16 bytes
  static constexpr int bytes(int nw, int nt) { return kList + q_bytes(nt) + nw * kStages * kStage; }
  static constexpr int kORow = D + 4;                   // floats per merged row: D, then m, l
  static_assert(16 * kORow * 4 <= kStages * kStage, "merge buffer fits the ring");
};

// One unit of the partial block (16 tokens from `first` on; n tokens of the block are real) from the tail, as bf16.
template <int D, int NT>
__device__ __forceinline__ void tail_unit(const bf16* tk, const bf16* tv, int first, int n_tok, int pos_first,
                                          const bf16* qs, const int (*pos)[2], State<D, NT>& st, int g, int t) {
  float s[NT][4];
  const int r = first + (g >> 1) * 4 + (g & 1);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 4; ++x) s[n][x] = 0.f;
#pragma unroll
  for (int hh = 0; hh < D / 64; ++hh) {
    uint4 u[2][2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      u[e][0] = u[e][1] = make_uint4(0, 0, 0, 0);
      if (r + 2 * e < n_tok) {
        const uint4* src = reinterpret_cast<const uint4*>(tk + (size_t)(r + 2 * e) * D + 64 * hh + 16 * t);
        u[e][0] = src[0], u[e][1] = src[1];
      }
    }
    const uint32_t us[8] = {u[0][0].x, u[0][0].y, u[0][0].z, u[0][0].w, u[0][1].x, u[0][1].y, u[0][1].z, u[0][1].w};
    const uint32_t vs[8] = {u[1][0].x, u[1][0].y, u[1][0].z, u[1][0].w, u[1][1].x, u[1][1].y, u[1][1].z, u[1][1].w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t a[4] = {us[2 * x], vs[2 * x], us[2 * x + 1], vs[2 * x + 1]};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint2 b = *reinterpret_cast<const uint2*>(qs + (8 * n + g) * (D + 8) + 64 * hh + 16 * t + 4 * x);
        mma_bf16(s[n], a, b.x, b.y);
      }
    }
  }
  // The reference takes the unit's V at its largest magnitude, as it takes a page at its scale.
  uint4 w[D / 64][4];
  float am = 0.f;
#pragma unroll
  for (int half = 0; half < D / 64; ++half)  // 8 channels per lane at a time
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[half][i] = make_uint4(0, 0, 0, 0);
      if (first + 4 * t + i < n_tok)
        w[half][i] = *reinterpret_cast<const uint4*>(tv + (size_t)(first + 4 * t + i) * D + (D / 8) * g + 8 * half);
      float f[8];
      bf16x8_to_f32(w[half][i], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) am = fmaxf(am, fabsf(f[e]));
    }
#pragma unroll
  for (int off = 16; off; off >>= 1) am = fmaxf(am, __shfl_xor_sync(~0u, am, off));
  const float lv = log2f(fmaxf(am * (1.f / 448.f), 7.8886090522101181e-31f));
  const float fac = kLog2e * rsqrtf((float)D);
  float mx[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    mx[n][0] = mx[n][1] = -CUDART_INF_F;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int tok = r + (x & 2), b = x & 1;
      s[n][x] = tok < n_tok && pos_first + tok <= pos[n][b] ? s[n][x] * fac : -CUDART_INF_F;
      mx[n][b] = fmaxf(mx[n][b], s[n][x] + lv);
    }
  }
  st.raise(mx);
  // weights 2^(s - M + 7): at most 2^(15 - lv), within bf16; from 2^-112 down where lv is largest, so not cut at 2^-126
  uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float base[2] = {st.base(n, 0), st.base(n, 1)};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      s[n][x] = exp2_small(s[n][x] - base[x & 1]);
      st.l[n][x & 1] += s[n][x] * (1.f / 128.f);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float a = s[n][2 * e], b = s[n][2 * e + 1];
      const uint32_t h = pack_bf16(a, b);
      hi[n][e] = transpose8x8(h);
      lo[n][e] = transpose8x8(pack_bf16(a - __uint_as_float(h << 16), b - __uint_as_float(h & 0xffff0000u)));
    }
  }
#pragma unroll
  for (int half = 0; half < D / 64; ++half) {
    const uint32_t* ww[4] = {&w[half][0].x, &w[half][1].x, &w[half][2].x, &w[half][3].x};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a[4] = {__byte_perm(ww[0][i], ww[1][i], 0x5410), __byte_perm(ww[0][i], ww[1][i], 0x7632),
                             __byte_perm(ww[2][i], ww[3][i], 0x5410), __byte_perm(ww[2][i], ww[3][i], 0x7632)};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_bf16(st.o[n][4 * half + i], a, hi[n][0], hi[n][1]);
        mma_bf16(st.o[n][4 * half + i], a, lo[n][0], lo[n][1]);
      }
    }
  }
}

// A CTA takes up to 8 NT query rows that read the same blocks: the query heads
// of a KV head's group over some tokens of one request (all blocks), or one
// (token, query head) with its own list (selected).  Its warps take pairs of
// units in turn, each with its own ring of copies in flight, and are merged at
// the end; with several splits the split's result goes to `part`.
template <int D, int KIND, int NW, int NT, bool SEL>
__global__ void __launch_bounds__(NW * 32, NW <= 4 ? (D == 128 ? 12 : 16) / NW : 1)
attn_kernel(View c, Plan p, const bf16* __restrict__ q, int h_q, const int32_t* __restrict__ sel, int topk,
            Few few, bf16* __restrict__ out, float* __restrict__ lse, float* __restrict__ part, int32_t* status) {
  using Ly = Layout<D>;
  constexpr int TR = 8 * NT;  // rows of a tile
  extern __shared__ __align__(128) unsigned char smem[];
  Entry* list = reinterpret_cast<Entry*>(smem);
  bf16* qs = reinterpret_cast<bf16*>(smem + Ly::kList);
  unsigned char* ring = smem + Ly::kList + Ly::q_bytes(NT) + (threadIdx.x >> 5) * Ly::kStages * Ly::kStage;
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int G = h_q / c.h_kv;
  const int lb = 31 - __clz(c.B), lu = lb - 4;  // log2 of the tokens and units of a block

  if constexpr (!SEL) asm volatile("griddepcontrol.launch_dependents;");  // cache_attn_rows.cu: nothing there waits for this
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
    if (few.mode == kPerToken) {
      const int tiles = (G + TR - 1) / TR;
      T.t0 = u / tiles;
      T.row = __ldg(p.row + T.t0);
      if ((unsigned)T.row >= (unsigned)c.rows) return;
      T.r0 = (u % tiles) * TR;
      T.nrows = G;
    } else {
      if (few.mode == kSlots) {
        const int slots = few.slot_rows / TR;
        T.row = u / slots;
        T.t0 = __ldg(p.cu + T.row);
        T.r0 = (u % slots) * TR;
      } else {
        auto place = [&](int r) { return (long long)__ldg(p.cu + r) * G / TR + r; };
        T.row = last_row(c.rows, u, place);
        T.t0 = __ldg(p.cu + T.row);
        T.r0 = (int)(u - place(T.row)) * TR;
      }
      T.nrows = (int)min(request_rows(p, T.row, G), (long long)few.limit);
      if (T.t0 < 0 || T.r0 < 0 || T.r0 >= T.nrows || T.nrows == few.limit) return;
    }
  }
  const int len = c.state[2 * T.row], held = min(c.state[2 * T.row + 1], c.max_blocks);
  const int rows = min(TR, T.nrows - T.r0);  // real rows of the tile
  // Position of a tile row; -1 for rows that see nothing.
  auto pos_of = [&](int r) {
    if (r >= rows) return -1;
    const int x = __ldg(p.pos + T.t0 + (T.r0 + r) / G);
    return x < len && x >> lb < held ? x : -1;
  };
  int pos[NT][2], mp = -1, min_pos = 0x7fffffff;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int r = 8 * n + 2 * t + b;
      pos[n][b] = pos_of(r);
      mp = max(mp, pos[n][b]);
      if (r < rows) min_pos = min(min_pos, pos[n][b]);
    }
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    mp = max(mp, __shfl_xor_sync(~0u, mp, off));
    min_pos = min(min_pos, __shfl_xor_sync(~0u, min_pos, off));
  }
  // (behind the look-ups above, which this one then overlaps)
  if (!SEL && few.mode == kPerToken && few.limit != 0x7fffffff && request_rows(p, T.row, G) >= few.limit) return;
  if (tid < rows && split == 0 && pos_of(tid) != __ldg(p.pos + T.t0 + (T.r0 + tid) / G)) set_status(status, kStatusBadTable);

  // ---- queries: bf16 in shared memory, fp16 fragments after scaling by a power of two
  auto item_of = [&](int r) {  // (token, query head) of a tile row
    return (size_t)(T.t0 + (T.r0 + r) / G) * h_q + T.head * G + (T.r0 + r) % G;
  };
  auto part_of = [&](int r) {  // where its splits' results go
    return few.mode == kSlots ? ((size_t)T.row * few.slot_rows + T.r0 + r) * c.h_kv + T.head : item_of(r);
  };
  for (int i = tid; i < TR * (D / 8); i += NW * 32) {
    const int r = i / (D / 8), ck = i % (D / 8);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < rows) x = *reinterpret_cast<const uint4*>(q + item_of(r) * D + ck * 8);
    *reinterpret_cast<uint4*>(qs + r * (D + 8) + ck * 8) = x;
  }
  const int own = mp < 0 ? -1 : mp >> lb;
  const bool tail = own >= 0 && (long long)(own + 1) * c.B > len;  // the last block is partial
  int b0 = 0, b1 = own + 1;                                        // blocks of this CTA
  bool my_tail = tail;
  if constexpr (!SEL) {
    b0 = min(b1, split * few.split_blocks);
    const int e = min(b1, b0 + few.split_blocks);
    my_tail = tail && e == b1 && b0 < b1;
    b1 = e;
    if (split > 0 && b0 >= b1) return;
  }
  __syncthreads();
  uint32_t qf[NT][D / 16][2];
  float fac[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float am = 0.f;
    uint2 raw[D / 16];
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      raw[k] = *reinterpret_cast<const uint2*>(qs + (8 * n + g) * (D + 8) + 64 * (k / 4) + 16 * t + 4 * (k % 4));
      const uint32_t w[2] = {raw[k].x, raw[k].y};
#pragma unroll
      for (int e = 0; e < 2; ++e)
        am = fmaxf(am, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u))));
    }
    am = fmaxf(am, __shfl_xor_sync(~0u, am, 1));
    am = fmaxf(am, __shfl_xor_sync(~0u, am, 2));
    // exponent of the largest magnitude, kept where the factors are normal
    const int e = max(-100, min(127, (int)((__float_as_uint(am) >> 23) & 255) - 127));
    const float up = __uint_as_float((uint32_t)(8 - e + 127) << 23);
    const float down = __uint_as_float((uint32_t)(e - 8 + 127) << 23) * (kLog2e * rsqrtf((float)D));
    fac[n][0] = __shfl_sync(~0u, down, 8 * t);      // of row 8 n + 2 t
    fac[n][1] = __shfl_sync(~0u, down, 8 * t + 4);  // and the next
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t w[2] = {raw[k].x, raw[k].y};
#pragma unroll
      for (int e2 = 0; e2 < 2; ++e2)
        qf[n][k][e2] = pack_f16(__uint_as_float(w[e2] << 16) * up, __uint_as_float(w[e2] & 0xffff0000u) * up);
    }
  }

  State<D, NT> st;
  st.clear();
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
        list[e] = pg >= 0 ? make_entry(c, pg, j, T.head) : Entry{-1, j * c.B, 0.f, 0.f, 0.f, 0.f, 0.f};
      }
    }
    __syncthreads();
    int count = n;
    if constexpr (SEL) {
      count = s_count & 0xffff;
      tail_done = !(s_count >> 16);
    }
    // Units of the listed blocks; the last one may end before its block does.
    int units = count << lu;
    if (count > 0 && list[count - 1].pos == own * c.B) units -= (1 << lu) - (mp - own * c.B) / kUnit - 1;
    const int pairs = (units + kPair - 1) / kPair;
    const int mine = warp < pairs ? (pairs - warp + NW - 1) / NW : 0;
    auto fetch = [&](int i) {
      if (i < mine) {
        unsigned char* dst = ring + (i % Ly::kStages) * Ly::kStage;
#pragma unroll
        for (int x = 0; x < kPair; ++x) {
          const int u = (warp + i * NW) * kPair + x;
          const long long off = list[u < units ? u >> lu : 0].at;
          const bool ok = u < units && off >= 0;
          const size_t at = ok ? off + (u & ((1 << lu) - 1)) * (kUnit * D) : 0;
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
      for (int u = (NW - 1 - warp); u * kUnit < n_tail; u += NW)
        tail_unit<D, NT>(c.tail_k + at, c.tail_v + at, u * kUnit, n_tail, own * c.B, qs, pos, st, g, t);
      tail_done = true;
    }
    for (int i = 0; i < mine; ++i) {
      fetch(i + Ly::kStages - 1);
      cp_async_wait<Ly::kStages - 1>();
      __syncwarp();
      const unsigned char* src = ring + (i % Ly::kStages) * Ly::kStage;
      float s[kPair][NT][4], mx[NT][2];
      bool small = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = -CUDART_INF_F;
#pragma unroll
      for (int x = 0; x < kPair; ++x) {
        const int u = (warp + i * NW) * kPair + x;
        unit_scores<D, KIND, NT>(src + x * 2 * kUnit * D, qf, s[x], g, t);
        const Entry e = list[u < units ? u >> lu : 0];
        small |= e.inv == 0.f;
        const int p0 = u < units && e.at >= 0 ? e.pos + (u & ((1 << lu) - 1)) * kUnit : 0x7fffffff - kUnit;
        const int tok = p0 + 4 * (g >> 1) + (g & 1);
        const bool cut = p0 + kUnit - 1 > min_pos;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float f[2] = {fac[n][0] * e.ks, fac[n][1] * e.ks};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float& z = s[x][n][y];
            z = fmaf(z, f[y & 1], e.lv);
          }
        }
        if (cut) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if (tok + (y & 2) > pos[n][y & 1]) s[x][n][y] = -CUDART_INF_F;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mx[n][0] = fmaxf(mx[n][0], fmaxf(s[x][n][0], s[x][n][2]));
          mx[n][1] = fmaxf(mx[n][1], fmaxf(s[x][n][1], s[x][n][3]));
        }
      }
      st.raise(mx);
      if (small) {  // what the weights of small V scales add to l, without the scale
#pragma unroll
        for (int x = 0; x < kPair; ++x) {
          const int u = (warp + i * NW) * kPair + x;
          const float lv = list[u < units ? u >> lu : 0].lv;
          if (list[u < units ? u >> lu : 0].inv != 0.f) continue;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              st.l[n][y & 1] += fast_exp2(s[x][n][y] - lv - (st.base(n, y & 1) + kOffset));
        }
      }
#pragma unroll
      for (int x = 0; x < kPair; ++x) {
        const int u = (warp + i * NW) * kPair + x;
        const float rest = list[u < units ? u >> lu : 0].rest, inv = list[u < units ? u >> lu : 0].inv;
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float* z = s[x][n];
          const float base[2] = {st.base(n, 0), st.base(n, 1)};
#pragma unroll
          for (int y = 0; y < 4; ++y) z[y] = fast_exp2(z[y] - base[y & 1]);
          st.l[n][0] = fmaf(z[0] + z[2], inv, st.l[n][0]);
          st.l[n][1] = fmaf(z[1] + z[3], inv, st.l[n][1]);
          pf[n][0] = transpose8x8(pack_f16(z[0] * rest, z[1] * rest));
          pf[n][1] = transpose8x8(pack_f16(z[2] * rest, z[3] * rest));
        }
        unit_values<D, KIND, NT>(src + x * 2 * kUnit * D + kUnit * D, pf, st.o, g, t);
      }
      __syncwarp();
    }
    cp_async_wait<0>();
    __syncthreads();
    done += n;
  } while (!SEL && done < n_list);

  // ---- merge the warps
  float* buf = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float l = st.l[n][b];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(~0u, l, off);
      const int r = 8 * n + 2 * t + b;
      if (r < rows) {
        float* d = buf + r * Ly::kORow;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float2*>(d + (D / 8) * g + 2 * i) = make_float2(st.o[n][i][b], st.o[n][i][2 + b]);
        if (g == 0) d[D] = st.m[n][b], d[D + 1] = l;
      }
    }
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(smem + Ly::kList + Ly::q_bytes(NT));
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
      const float h = b[D] == -CUDART_INF_F ? (b[D + 1] == b[D + 1] ? 0.f : 1.f) : fast_exp2(0.5f * (b[D] - M)), a = h * h;
      l += h * b[D + 1] * h;
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] += a * b[ch + x];
    }
    const size_t item = item_of(r);
    if (few.nsplit == 1) {
      const float inv = l == 0.f ? 0.f : 1.f / (128.f * l);
      uint2 y;
      y.x = pack_bf16(o[0] * inv, o[1] * inv), y.y = pack_bf16(o[2] * inv, o[3] * inv);
      *reinterpret_cast<uint2*>(out + item * D + ch) = y;
      if (ch == 0) lse[item] = l == 0.f ? -CUDART_INF_F : (M + log2f(l)) * 0.69314718055994531f;
    } else {
      float* b = part + (part_of(r) * few.nsplit + split) * Ly::kORow;
      *reinterpret_cast<float4*>(b + ch) = make_float4(o[0], o[1], o[2], o[3]);
      if (ch == 0) b[D] = M, b[D + 1] = l;
    }
  }
}

// Joins the splits of a (token, query head): WARPS warps take its splits in turn, four at a time in flight.
template <int D, int WARPS>
__global__ void __launch_bounds__(128)
merge_kernel(View c, Plan p, int h_q, Many many, Few few, const float* __restrict__ part_many,
             const float* __restrict__ part_few, bf16* __restrict__ out, float* __restrict__ lse) {
  constexpr int kORow = Layout<D>::kORow, E = D / 32;
  __shared__ float so[WARPS > 1 ? 4 : 1][D], sm[4], sl[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned item = blockIdx.x * (4 / WARPS) + warp / WARPS;  // T h_q d is below 2^31
  if (item >= (unsigned)p.T * h_q) return;
  const int tok = item / (unsigned)h_q, row = __ldg(p.row + tok), pos = __ldg(p.pos + tok);
  if ((unsigned)row >= (unsigned)c.rows) return;
  const int lb = 31 - __clz(c.B), len = c.state[2 * row], held = min(c.state[2 * row + 1], c.max_blocks);
  int split_blocks = few.split_blocks, nsplit = few.nsplit;
  bool known = true;
  size_t place = item;
  const float* part = part_few;
  if (many.limit) {
    const int G = h_q / c.h_kv, h = item - (unsigned)tok * h_q;
    if (request_rows(p, row, G) >= many.limit) {
      split_blocks = many.split_blocks, nsplit = many.nsplit, part = part_many;
    } else if (few.mode == kSlots) {
      const long long r = ((long long)tok - __ldg(p.cu + row)) * G + h % G;
      known = r >= 0 && r < few.slot_rows;
      place = ((size_t)row * few.slot_rows + (known ? r : 0)) * c.h_kv + h / G;
    }
  }
  if (nsplit == 1) return;
  const float* b = part + place * nsplit * kORow;
  // splits that wrote: as many as the tile's furthest row needs; a row's own are the first of those
  const bool sees = known && pos >= 0 && pos < len && pos >> lb < held;
  const int n = sees ? (pos >> lb) / split_blocks + 1 : 0;
  float M = -CUDART_INF_F, l = 0.f, o[E];
#pragma unroll
  for (int x = 0; x < E; ++x) o[x] = 0.f;
  for (int s0 = warp % WARPS * 4; s0 < n; s0 += 4 * WARPS) {
    float m[4], ls[4], v[4][E], top = M;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* d = b + min(s0 + i, n - 1) * kORow;
      m[i] = s0 + i < n ? d[D] : -CUDART_INF_F;
      ls[i] = s0 + i < n ? d[D + 1] : 0.f;
      if constexpr (E == 4) {
        const float4 y = *reinterpret_cast<const float4*>(d + 4 * lane);
        v[i][0] = y.x, v[i][1] = y.y, v[i][2] = y.z, v[i][3] = y.w;
      } else {
        const float2 y = *reinterpret_cast<const float2*>(d + 2 * lane);
        v[i][0] = y.x, v[i][1] = y.y;
      }
      top = fmaxf(top, m[i]);
    }
    const float h0 = M == -CUDART_INF_F ? 0.f : fast_exp2(0.5f * (M - top)), a0 = h0 * h0;
    l = l * h0 * h0;
#pragma unroll
    for (int x = 0; x < E; ++x) o[x] *= a0;
    M = top;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float h = m[i] == -CUDART_INF_F ? (ls[i] == ls[i] ? 0.f : 1.f) : fast_exp2(0.5f * (m[i] - top)), a = h * h;
      l += h * ls[i] * h;
#pragma unroll
      for (int x = 0; x < E; ++x) o[x] += s0 + i < n ? a * v[i][x] : 0.f;
    }
  }
  if constexpr (WARPS == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / (128.f * l);
#pragma unroll
    for (int x = 0; x < E; ++x) o[x] = l == 0.f ? 0.f : o[x] * inv;
    bf16* y = out + (size_t)item * D + E * lane;
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
    else
      *reinterpret_cast<uint32_t*>(y) = pack_bf16(o[0], o[1]);
    if (lane == 0) lse[item] = l == 0.f ? -CUDART_INF_F : (M + log2f(l)) * 0.69314718055994531f;
  } else {
#pragma unroll
    for (int x = 0; x < E; ++x) so[warp][E * lane + x] = o[x];
    if (lane == 0) sm[warp] = M, sl[warp] = l;
    __syncthreads();
    const int ch = threadIdx.x;
    if (ch >= D) return;
    M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    l = 0.f;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float h = sm[w] == -CUDART_INF_F ? (sl[w] == sl[w] ? 0.f : 1.f) : fast_exp2(0.5f * (sm[w] - M));
      l += h * sl[w] * h;
      y += h * h * so[w][ch];
    }
    out[item * D + ch] = __float2bfloat16_rn(l == 0.f ? 0.f : y / (128.f * l));
    if (ch == 0) lse[item] = l == 0.f ? -CUDART_INF_F : (M + log2f(l)) * 0.69314718055994531f;
  }
}

// How a step over all blocks is cut up.
struct Cut {
  bool with_many;  // a request may reach the limit
  bool wide;       // tiles of 16 rows instead of 8
  long long tiles, many_tiles;
  Few few;
  Many many;
  size_t part_many, part_few;  // floats of splits' results
};

// Requests with few query rows per KV head go in tiles of 8 or 16 (attn_kernel), those with many in tiles of 128
// (cache_attn_rows.cu).  Only the device knows which a request is, so both kernels are launched where a request could
// reach the limit, and each leaves the other's rows alone.  Measured in tiles of 16 and of 128: d = 128, 48 rows of each
// of 16 requests over 17K keys 255 and 300 us, 64 rows 326 and 300; d = 64, 80 rows of each of 4 requests 199 and 214
// us, 96 rows 235 and 203.
//
// Long rows are cut into splits of whole blocks, so that even few or uneven rows fill the GPU: about 24 CTAs per SM
// counted over rows of full length (tiles of 128 rows: 8), and at least 1024 tokens each (512): a split costs a partial
// result of D + 4 floats per query row, written and read back.  With 8, 16, 24 and 32 per SM: 24 single tokens over 4K
// to 64K keys 247, 219, 214 and 215 us, 16 over 30K each 171, 177, 184 and 189, 512 tokens beside 63 single ones 603,
// 606, 559 and 563.  Tiles of 128 with 4, 6 and 8 per SM: 16 requests of 16
// tokens, 4 heads each, over 4K to 30K keys 276, 283 and 241 us; 13 uneven requests of 4 to 700 tokens 455, 446 and
// 380; 3 chunks of 312 to 513 tokens 403, 413 and 410.
Cut cut_of(const View& c, int T, int h_q) {
  const int G = h_q / c.h_kv;
  const long long all = (long long)T * G;
  const int limit = c.d == 128 ? 64 : 96;
  Cut x = {};
  x.with_many = all >= limit;
  // tiles, by what a tile's place says: a token, a place among all tokens, or a place among its request's
  const long long by[3] = {(long long)T * ((G + 15) / 16), all / 16 + c.rows,
                           x.with_many ? (long long)c.rows * (limit / 16) : 0x7fffffffffffll};
  x.few.mode = by[0] <= by[1] && by[0] <= by[2] ? kPerToken : (by[1] <= by[2] ? kSearch : kSlots);
  x.few.limit = x.with_many ? limit : 0x7fffffff;
  x.few.slot_rows = limit;
  x.wide = x.few.mode != kPerToken || G > 8;
  x.tiles = by[x.few.mode];
  const int active = T < c.rows ? T : c.rows;
  {
    const long long ctas = (x.few.mode == kSlots ? active : x.tiles) * c.h_kv;
    const long long want = (24 * 148 + ctas - 1) / ctas;
    const long long least = 1024 / c.B;
    long long blocks = (c.max_blocks + want - 1) / want;
    if (blocks < least) blocks = least;
    // a little more than one wave of CTAs (3 per SM at d = 128, 4 at 64) is worse than one of longer ones (2 rows of
    // 30000 keys, 8 KV heads: 42.5 us as 16 CTAs per SM would have it, 35 in one wave)
    const long long slots = (c.d == 128 ? 3 : 4) * 148, total = ctas * ((c.max_blocks + blocks - 1) / blocks);
    if (total > slots && total < 2 * slots && ctas <= slots)
      blocks = (c.max_blocks + slots / ctas - 1) / (slots / ctas);
    if (x.few.mode == kSlots) {  // most of these CTAs may find nothing to do: four waves of them are enough
      long long n = 4 * slots / (x.tiles * c.h_kv);
      if (n < 1) n = 1;
      if (blocks < (c.max_blocks + n - 1) / n) blocks = (c.max_blocks + n - 1) / n;
    }
    x.few.split_blocks = (int)blocks;
    x.few.nsplit = (int)((c.max_blocks + blocks - 1) / blocks);
  }
  if (x.with_many) {
    // n >= 64 query rows from `first` on cover at least n / 64 >= ceil(n / 128) multiples of 64: places enough, and few
    // where few tokens meet many rows
    const long long most = all / limit;  // requests that can reach the limit
    const long long ctas = (all / 128 + (most < active ? most : active)) * c.h_kv;
    long long want = (8 * 148 + ctas - 1) / ctas;
    const long long step = c.B < 128 ? 128 / c.B : 1;  // splits of whole key tiles
    x.many.per_row = all / 128 + c.rows <= all / 64;
    x.many_tiles = x.many.per_row ? all / 128 + c.rows : all / 64;
    // no more tokens than rows are mostly single ones, with nothing to do here: one wave of CTAs
    if (T <= c.rows && want > 2 * 148 / (x.many_tiles * c.h_kv)) want = 2 * 148 / (x.many_tiles * c.h_kv);
    if (want < 1) want = 1;
    long long blocks = (c.max_blocks + want - 1) / want;
    if (blocks < 512 / c.B) blocks = 512 / c.B;
    blocks = (blocks + step - 1) / step * step;
    x.many.limit = limit;
    x.many.split_blocks = (int)blocks;
    x.many.nsplit = (int)((c.max_blocks + blocks - 1) / blocks);
  }
  const size_t row = (size_t)c.d + 4;
  if (x.many.nsplit > 1) x.part_many = (size_t)T * h_q * x.many.nsplit * row;
  if (x.few.nsplit > 1)
    x.part_few = (x.few.mode == kSlots ? (size_t)c.rows * limit * c.h_kv : (size_t)T * h_q) * x.few.nsplit * row;
  return x;
}

template <int D, int KIND, int NW, int NT, bool SEL>
cudaError_t launch_one(const View& c, const Plan& p, const bf16* q, int h_q, const int32_t* sel, int topk, dim3 grid,
                       const Few& few, bf16* out, float* lse, float* part, int32_t* status, cudaStream_t st) {
  constexpr int smem = Layout<D>::bytes(NW, NT);
  const cudaError_t e = cudaFuncSetAttribute(attn_kernel<D, KIND, NW, NT, SEL>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attn_kernel<D, KIND, NW, NT, SEL><<<grid, NW * 32, smem, st>>>(c, p, q, h_q, sel, topk, few, out, lse, part, status);
  return cudaGetLastError();
}

template <int D, int KIND>
cudaError_t launch_all(const View& c, const Plan& p, const bf16* q, int h_q, const int32_t* sel, int topk, bf16* out,
                       float* lse, float* part, int32_t* status, cudaStream_t st) {
  if (sel) {
    const dim3 grid(p.T, h_q);
    const Few one{kPerToken, 0x7fffffff, 0, 0, 1};
    // Two warps a row leave the least to the last wave (1024 rows of 32 blocks of 32: 35 us with four, 31.7 with two,
    // 33.6 with one); few rows take more, so that their blocks are read at once.
    if ((long long)p.T * h_q > 2 * 148)
      return launch_one<D, KIND, 2, 1, true>(c, p, q, h_q, sel, topk, grid, one, out, lse, part, status, st);
    return launch_one<D, KIND, 8, 1, true>(c, p, q, h_q, sel, topk, grid, one, out, lse, part, status, st);
  }
  const Cut x = cut_of(c, p.T, h_q);
  float* part_few = part + x.part_many;
  const dim3 grid((unsigned)x.tiles, c.h_kv, x.few.nsplit);
  cudaError_t e =
      x.wide ? launch_one<D, KIND, 4, 2, false>(c, p, q, h_q, nullptr, 0, grid, x.few, out, lse, part_few, status, st)
             : launch_one<D, KIND, 4, 1, false>(c, p, q, h_q, nullptr, 0, grid, x.few, out, lse, part_few, status, st);
  if (e != cudaSuccess) return e;
  if (x.with_many) e = launch_attention_rows(c, p, q, h_q, (int)x.many_tiles, x.many, out, lse, part, status, st);
  if (e != cudaSuccess) return e;
  if (x.part_many + x.part_few == 0) return cudaSuccess;
  const long long items = (long long)p.T * h_q;
  // (38K rows of 2 splits: a warp each 438 us in all, a CTA each 472; 768 rows of up to 13: 214 and 210; 32 rows of 64:
  // 48 and 40)
  const int most = x.few.nsplit > x.many.nsplit ? x.few.nsplit : x.many.nsplit;
  if (most <= 8 || items > 2 * 16 * 148)
    merge_kernel<D, 1><<<(unsigned)((items + 3) / 4), 128, 0, st>>>(c, p, h_q, x.many, x.few, part, part_few, out, lse);
  else
    merge_kernel<D, 4><<<(unsigned)items, 128, 0, st>>>(c, p, h_q, x.many, x.few, part, part_few, out, lse);
  return cudaGetLastError();
}

}  // namespace

size_t attn_scratch(const View& c, int T, int h_q) {
  if (T == 0) return 0;
  const Cut x = cut_of(c, T, h_q);
  return (x.part_many + x.part_few) * sizeof(float);
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
