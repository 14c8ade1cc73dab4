// Routing of new queries over the cached centroids: the topk - 1 earlier
// blocks with the largest s_j = q . (hi_j + lo_j), ties to the lower block,
// and the query's own block.
//
// Screen and rescore.  Reading hi alone halves the bytes, and
//   |s_j - q . hi_j| <= |q| |lo_j| <= |q| |hi_j| 2^-8 (1 + 2^-8)
// because lo is what rounding to hi left (half a unit of hi's 8-bit
// significand); the rounding of the 32-bit sums is far below.  With e the
// largest such bound over a row's blocks, any value b that at least K = topk - 1
// screen scores reach gives: every block of the true top K has a screen score
// >= b - 2 e.  Kernel one writes the screen scores (mma.m16n8k16, bf16, tiles
// of 16 query rows of one request and KV head against 8 blocks); in kernel two
// a warp takes a query row: b is the K-th largest of the maxima of 128 disjoint
// subsets (about 1.1 K blocks pass), passing blocks whose screen score is more
// than 2 e above the K-th largest are in, and the few others are scored in 64
// bits and ranked by (score, block).  Products of bf16 are exact in 64 bits
// and their sums are off by 2^-46 at most, so the result is that of exact
// arithmetic unless two scores agree to 14 digits.
//
// Measured: 64 rows of up to 64K tokens (2048 blocks), 16 heads of 64: 38.6 us, 145 MB of centroids with lo and 73
// without; kernel one 27 us of it at 2.6 TB/s (uneven rows, short loops behind dependent look-ups), kernel two 17 (a
// chain of about 40 warp-wide steps per query row), overlapped at the seam.  One row 19 us, nearly all of it that
// chain.  530 tokens of 32 heads: 30 and 60 us, bound by issue.
#include <math_constants.h>

#include <climits>

#include "cache.cuh"

namespace moba {
namespace cache {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kSelWarps = 4;
constexpr int kCand = 256;       // candidates held per warp (at most 32 x 32)
constexpr float kNone = -3.4e38f; // below every finite screen score that can win
// Squares below the normal range of 32 bits lose up to 2^-150 each, 2^-143 in a sum: added to the sums, so that the bound
// holds for magnitudes whose squares vanish (below 2^-70 all blocks are then candidates, and scored in 64 bits).
constexpr float kLostSquares = 7.1746481e-43f;  // 2^-140
constexpr size_t kScratch = (size_t)256 << 20;  // screen scores held at a time

struct Slab {
  int t0, t1;        // tokens of this launch
  int per_token;     // tiles: each token on its own (1) or a request's tokens together (0)
  int chunk;         // blocks per CTA of kernel one
  int nchunk;
  int stride;        // floats per screen-score row
  int tiles;         // bound on the tiles of the launch
};

// Row r's part of the slab.
__device__ __forceinline__ int clip(int x, const Slab& s) { return min(max(x, s.t0), s.t1); }

// First tile of request r (tiles of a request's rows; relative to the slab).
__device__ __forceinline__ int tile_base(const Plan& p, const Slab& s, int r, int G) {
  return (int)((long long)(clip(__ldg(p.cu + r), s) - s.t0) * G / 16) + r;
}

// Number of earlier blocks of a token at `pos`, or -1 (sees nothing), -2 (plan entry out of range).
__device__ __forceinline__ int own_block(const View& c, int row, int pos) {
  if (pos < 0) return -1;
  const int j = pos >> (31 - __clz(c.B));
  return pos < c.state[2 * row] && j < min(c.state[2 * row + 1], c.max_blocks) ? j : -2;
}

// SHARE: the CTA's warps take the blocks of one tile in turn; else each has a tile of its own, and neighbours (mostly of
// one request) find one another's centroids in L1.
template <int D, bool SHARE>
__global__ void __launch_bounds__(kScoreThreads)
score_kernel(View c, Plan p, Slab sl, const bf16* __restrict__ q, int h_q, float* __restrict__ score,
             float* __restrict__ hmax, int32_t* status) {
  constexpr int NT = 4, WARPS = kScoreThreads / 32;  // n-tiles (of 8 blocks) per warp and step
  __shared__ __align__(16) bf16 qbuf[(SHARE ? 1 : WARPS) * 16 * (D + 8)];
  __shared__ float smax[WARPS];
  cudaTriggerProgrammaticLaunchCompletion();  // select_kernel may start; it waits for this grid's end where it has to
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  if (sl.t0 == 0 && tid == 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) status[0] = status[1] = 0;
  const int G = h_q / c.h_kv, head = blockIdx.y, u = SHARE ? blockIdx.x : blockIdx.x * WARPS + warp;
  bf16* qs = qbuf + (SHARE ? 0 : warp * 16 * (D + 8));
  int row, tok0, r0, nrows;
  if (sl.per_token) {
    const int tiles = (G + 15) / 16;
    tok0 = sl.t0 + u / tiles;
    if (tok0 >= sl.t1) return;
    row = __ldg(p.row + tok0);
    if ((unsigned)row >= (unsigned)c.rows) return;
    r0 = (u % tiles) * 16;
    nrows = G;
  } else {
    int lo = 0, hi = c.rows;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile_base(p, sl, mid, G) <= u) lo = mid; else hi = mid;
    }
    row = lo;
    tok0 = clip(__ldg(p.cu + row), sl);
    r0 = (u - tile_base(p, sl, row, G)) * 16;
    nrows = (clip(__ldg(p.cu + row + 1), sl) - tok0) * G;
    if (r0 < 0 || r0 >= nrows) return;
  }
  const int rows = min(16, nrows - r0);
  int nb = 0;
  if (lane < rows) nb = max(0, own_block(c, row, __ldg(p.pos + tok0 + (r0 + lane) / G)));
  for (int off = 1; off < 16; off <<= 1) nb = max(nb, __shfl_xor_sync(~0u, nb, off));
  nb = __shfl_sync(~0u, nb, 0);
  const int j0 = blockIdx.z * sl.chunk, j1 = min(nb, j0 + sl.chunk);
  const size_t at_max = ((size_t)u * c.h_kv + head) * sl.nchunk + blockIdx.z;
  if (j0 >= j1) return;
  auto item_of = [&](int r) { return (size_t)(tok0 + (r0 + r) / G) * h_q + head * G + (r0 + r) % G; };
  for (int i = SHARE ? tid : lane; i < 16 * (D / 8); i += SHARE ? kScoreThreads : 32) {
    const int r = i / (D / 8), ck = i % (D / 8);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < rows) x = *reinterpret_cast<const uint4*>(q + item_of(r) * D + ck * 8);
    *reinterpret_cast<uint4*>(qs + r * (D + 8) + ck * 8) = x;
  }
  if constexpr (SHARE) __syncthreads(); else __syncwarp();
  // Lane's share of a row: channels 64 hh + 16 t .. + 15; k-step x of a half takes 4 of them.
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const bf16* a = qs + g * (D + 8) + 64 * (k / 4) + 16 * t + 4 * (k % 4);
    const uint2 x = *reinterpret_cast<const uint2*>(a), y = *reinterpret_cast<const uint2*>(a + 8 * (D + 8));
    qf[k][0] = x.x, qf[k][1] = y.x, qf[k][2] = x.y, qf[k][3] = y.y;
  }
  float most = 0.f;
  float* dst[2];  // screen scores of this lane's rows
#pragma unroll
  for (int r = 0; r < 2; ++r)
    dst[r] = g + 8 * r < rows ? score + (item_of(g + 8 * r) - (size_t)sl.t0 * h_q) * sl.stride + 2 * t : nullptr;
  constexpr int STEP = (SHARE ? WARPS : 1) * NT * 8;
  const int first = j0 + (SHARE ? warp * NT * 8 : 0);
  auto page_at = [&](int j) { return j < j1 ? __ldg(c.table + (size_t)row * c.max_blocks + j) : 0; };
  int next = page_at(first + lane);
  for (int j = first; j < j1; j += STEP) {
    const int mine = (unsigned)next < (unsigned)c.n_pages ? next : -1;
    if (j + lane < j1 && mine < 0) most = CUDART_NAN_F;  // no such page: the row is looked at block by block
    next = page_at(j + STEP + lane);
    uint4 w[NT][D / 64][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int pg = __shfl_sync(~0u, mine, n * 8 + g);
      const uint4* src = reinterpret_cast<const uint4*>(c.cent + ((size_t)max(pg, 0) * c.h_kv + head) * D + 16 * t);
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
        for (int x = 0; x < 2; ++x)
          w[n][hh][x] = pg >= 0 && j + n * 8 + g < j1 ? __ldg(src + hh * 8 + x) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float s[4] = {0.f, 0.f, 0.f, 0.f}, sq = 0.f;
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh) {
        const uint32_t ws[8] = {w[n][hh][0].x, w[n][hh][0].y, w[n][hh][0].z, w[n][hh][0].w,
                                w[n][hh][1].x, w[n][hh][1].y, w[n][hh][1].z, w[n][hh][1].w};
#pragma unroll
        for (int x = 0; x < 4; ++x) mma_bf16(s, qf[hh * 4 + x], ws[2 * x], ws[2 * x + 1]);
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const float a = __uint_as_float(ws[x] << 16), b = __uint_as_float(ws[x] & 0xffff0000u);
          sq = fmaf(a, a, fmaf(b, b, sq));
        }
      }
      sq += __shfl_xor_sync(~0u, sq, 1);
      sq += __shfl_xor_sync(~0u, sq, 2);
      most = sq > most || sq != sq ? sq : most;  // NaN stays (nothing compares with it)
      const int jj = j + n * 8 + 2 * t;
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (dst[r]) {
          if (jj + 1 < j1) *reinterpret_cast<float2*>(dst[r] + j + n * 8) = make_float2(s[2 * r], s[2 * r + 1]);
          else if (jj < j1) dst[r][j + n * 8] = s[2 * r];
        }
    }
  }
  for (int off = 1; off < 32; off <<= 1) {
    const float o = __shfl_xor_sync(~0u, most, off);
    most = o > most || o != o ? o : most;
  }
  if constexpr (SHARE) {
    if (lane == 0) smax[warp] = most;
    __syncthreads();
    if (tid == 0) {
      for (int i = 1; i < WARPS; ++i) most = smax[i] > most || smax[i] != smax[i] ? smax[i] : most;
      hmax[at_max] = most;
    }
  } else if (lane == 0) {
    hmax[at_max] = most;
  }
}

// Order-preserving key of a float that is not NaN, and back.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }

// Order-preserving whole number of a score (comparing doubles takes several times as long); NaN counts as -infinity,
// -0 as 0.
__device__ __forceinline__ long long order_of(double s) {
  const long long b = __double_as_longlong(s + 0.0);
  return isnan(s) ? LLONG_MIN : b ^ ((b >> 63) & LLONG_MAX);
}

// One warp's candidates.
struct List {
  long long exact[kCand];  // order_of an exact score
  float screen[kCand];
  int j[kCand];
  int todo[kCand];         // list positions of the candidates being scored,
  int page[kCand];         // their pages, then the upper words of their exact scores
};

// 64-bit scores of the candidates i < n for which `want(i)`, 16 at a time (2 lanes each); their list positions stay in
// todo, the upper words of their scores in page; returns their number.
template <int D, typename F>
__device__ __forceinline__ int rescore(const View& c, int row, int head, const bf16* q, List& ls, int n,
                                       int32_t* status, F want) {
  constexpr int V = D / 16;  // 16-byte pieces per lane
  const int lane = threadIdx.x & 31, sub = lane & 1;
  int m = 0;
  for (int x = 0; x < n; x += 32) {
    const bool w = x + lane < n && want(x + lane);
    const int pg = w ? block_page(c, row, ls.j[x + lane]) : -1;
    if (w && pg < 0) set_status(status, kStatusBadTable);
    const uint32_t b = __ballot_sync(~0u, w);
    const int at = m + __popc(b & ((1u << lane) - 1));
    if (w) ls.todo[at] = x + lane, ls.page[at] = pg;
    m += __popc(b);
  }
  __syncwarp();
  for (int base = 0; base < m; base += 16) {
    const int k = base + (lane >> 1);
    const int pg = k < m ? ls.page[k] : -1;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    if (pg >= 0) {
      const uint4* hi = reinterpret_cast<const uint4*>(c.cent + ((size_t)pg * c.h_kv + head) * D) + sub;
      const uint4* lo = hi + (size_t)c.n_pages * c.h_kv * (D / 8);
      uint4 u[V], v[V];
#pragma unroll
      for (int x = 0; x < V; ++x) u[x] = __ldg(hi + 2 * x), v[x] = __ldg(lo + 2 * x);
#pragma unroll
      for (int x = 0; x < V; ++x) {
        float a[8], b[8], f[8];
        bf16x8_to_f32(u[x], a);
        bf16x8_to_f32(v[x], b);
        bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(q) + sub + 2 * x), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e & 3] += (double)f[e] * ((double)a[e] + (double)b[e]);
      }
    }
    double r = (s[0] + s[1]) + (s[2] + s[3]);
    r += __shfl_xor_sync(~0u, r, 1);
    if (k < m && sub == 0) {
      const long long o = pg < 0 ? LLONG_MIN : order_of(r);
      ls.exact[ls.todo[k]] = o;
      ls.page[k] = (int)(o >> 32);
    }
  }
  __syncwarp();
  return m;
}

// Whether candidate (s, j) is among the best K of the list positions todo[0, m) (all positions when todo is null).
__device__ __forceinline__ bool among(const List& ls, const int* todo, int m, int K, long long s, int j) {
  int above = 0;
#pragma unroll 4
  for (int k = 0; k < m; ++k) {
    const int i = todo ? todo[k] : k;
    const long long o = ls.exact[i];
    above += o > s || (o == s && ls.j[i] < j);
  }
  return above < K;
}

// Rows with more candidates than the list holds, or screen scores that do not count (bar = -infinity): blocks in
// order, all that reach the bar scored in 64 bits, the best K staying whenever the list is full.  Returns how many are
// in the list; all have their exact scores.
template <int D>
__device__ __noinline__ int many_candidates(const View& c, int row, int head, const bf16* q, List& ls, const float* sc,
                                            int own, float bar, int K, int32_t* status) {
  const int lane = threadIdx.x & 31;
  int n = 0, scored = 0;
  for (int base = 0; base < own; base += 32) {
    const int j = base + lane;
    const bool in = j < own && (bar == -CUDART_INF_F || sc[j] >= bar);
    const uint32_t m = __ballot_sync(~0u, in);
    if (in) ls.j[n + __popc(m & ((1u << lane) - 1))] = j;
    n += __popc(m);
    __syncwarp();
    if (n > kCand - 32) {
      rescore<D>(c, row, head, q, ls, n, status, [&](int i) { return i >= scored; });
      uint32_t keep = 0;  // ranks need the whole list: first all of them, then the moves
      for (int x = 0; x * 32 < n; ++x) {
        const int i = x * 32 + lane;
        if (i < n && among(ls, nullptr, n, K, ls.exact[i], ls.j[i])) keep |= 1u << x;
      }
      __syncwarp();
      int kept = 0;
      for (int x = 0; x * 32 < n; ++x) {
        const bool k = keep >> x & 1;
        const long long s = k ? ls.exact[x * 32 + lane] : 0;
        const int jj = k ? ls.j[x * 32 + lane] : 0;
        const uint32_t b = __ballot_sync(~0u, k);
        const int at = kept + __popc(b & ((1u << lane) - 1));  // at most x * 32 + lane
        __syncwarp();
        if (k) ls.exact[at] = s, ls.j[at] = jj;
        kept += __popc(b);
      }
      __syncwarp();
      n = scored = kept;
    }
  }
  rescore<D>(c, row, head, q, ls, n, status, [&](int i) { return i >= scored; });
  return n;
}

// The K-th largest of the warp's keys (N per lane; at least K of them real), to 16 bits (a bf16) from below: two bits a
// step, the three counts in one sum.
template <int N>
__device__ __forceinline__ uint32_t kth_key(const uint32_t* key, int K) {
  uint32_t b = 0;
#pragma unroll 1
  for (int bit = 30; bit >= 16; bit -= 2) {
    uint32_t cnt = 0;
#pragma unroll
    for (int x = 0; x < N; ++x)
#pragma unroll
      for (int s = 1; s < 4; ++s) cnt += (uint32_t)(key[x] >= (b | (uint32_t)s << bit)) << (10 * (s - 1));
    cnt = __reduce_add_sync(~0u, cnt);  // at most 32 N = 256 each
    const int s = ((int)(cnt & 1023) >= K) + ((int)(cnt >> 10 & 1023) >= K) + ((int)(cnt >> 20) >= K);
    b |= (uint32_t)s << bit;
  }
  return b;
}

// One warp per (token, query head).  HELD: pieces of 4 screen scores per lane and batch (a batch: 128 HELD blocks).
template <int D, int HELD>
__global__ void __launch_bounds__(kSelWarps * 32)
select_kernel(View c, Plan p, Slab sl, const bf16* __restrict__ q, int h_q, int topk, const float* __restrict__ score,
              const float* __restrict__ hmax, int32_t* __restrict__ sel, int32_t* status) {
  __shared__ List lists[kSelWarps];
  const int lane = threadIdx.x & 31;
  List& ls = lists[threadIdx.x >> 5];
  const int local = blockIdx.x * kSelWarps + (threadIdx.x >> 5);  // item of the slab
  if (local >= (sl.t1 - sl.t0) * h_q) return;
  const int tok = sl.t0 + local / h_q, h = local % h_q;
  const size_t item = (size_t)tok * h_q + h;
  const bf16* qr = q + item * D;
  uint32_t qw[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) qw[i] = __ldg(reinterpret_cast<const uint32_t*>(qr) + lane + 32 * i);
  const int row = __ldg(p.row + tok), pos = __ldg(p.pos + tok);
  if ((unsigned)row >= (unsigned)c.rows) {
    cudaGridDependencySynchronize();  // a step of padding only waits, too: what comes after finds score_kernel done
    return;
  }
  int32_t* out = sel + item * topk;
  const int own = own_block(c, row, pos);
  cudaGridDependencySynchronize();  // the screen scores are there
  const int K = topk - 1;
  if (own <= K) {  // every earlier block; none (-1) for a token that sees nothing
    if (own == -2 && lane == 0) set_status(status, kStatusBadTable);
    for (int i = lane; i < topk; i += 32) out[i] = i <= own ? i : -1;
    return;
  }
  if (K == 0) {
    if (lane == 0) out[0] = own;
    return;
  }
  const int G = h_q / c.h_kv, head = h / G;
  const float* sc = score + (size_t)local * sl.stride;
  // ---- screen scores: piece r of a lane is blocks base + 128 r + 4 lane .. + 3, what lies behind `own` is kNone
  auto piece = [&](int j) {
    float4 v = make_float4(kNone, kNone, kNone, kNone);
    if (j < own) v = *reinterpret_cast<const float4*>(sc + j);
    if (j + 1 >= own) v.y = kNone;
    if (j + 2 >= own) v.z = kNone;
    if (j + 3 >= own) v.w = kNone;
    return v;
  };
  // the largest of this lane's subsets, and (rows of one batch) of its pieces
  float mx[4] = {kNone, kNone, kNone, kNone}, pm[HELD];
  for (int base = 0; base < own; base += HELD * 128) {
    float4 v[HELD];
#pragma unroll
    for (int r = 0; r < HELD; ++r) {
      const int j = base + 128 * r + 4 * lane;
      if (base + 128 * r + 128 <= own) v[r] = *reinterpret_cast<const float4*>(sc + j);
      else v[r] = piece(j);
    }
#pragma unroll
    for (int r = 0; r < HELD; ++r) {
      mx[0] = fmaxf(mx[0], v[r].x), mx[1] = fmaxf(mx[1], v[r].y);
      mx[2] = fmaxf(mx[2], v[r].z), mx[3] = fmaxf(mx[3], v[r].w);
      pm[r] = fmaxf(fmaxf(v[r].x, v[r].y), fmaxf(v[r].z, v[r].w));
    }
  }
  // ---- twice the error bound: 2 |q| max |hi| (2^-8 + 2^-10), and room for products below the normal range
  float sq = 0.f, hm = 0.f;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const float a = __uint_as_float(qw[i] << 16), b = __uint_as_float(qw[i] & 0xffff0000u);
    sq = fmaf(a, a, fmaf(b, b, sq));
  }
  const int tile = sl.per_token ? (tok - sl.t0) * ((G + 15) / 16) + (h % G) / 16
                                : tile_base(p, sl, row, G) + ((tok - clip(__ldg(p.cu + row), sl)) * G + h % G) / 16;
  for (int i = lane; i * sl.chunk < own; i += 32) {
    const float x = hmax[((size_t)min(max(tile, 0), sl.tiles - 1) * c.h_kv + head) * sl.nchunk + i];
    hm = x > hm || x != x ? x : hm;  // NaN stays
  }
  for (int off = 16; off; off >>= 1) {
    sq += __shfl_xor_sync(~0u, sq, off);
    const float x = __shfl_xor_sync(~0u, hm, off);
    hm = x > hm || x != x ? x : hm;
  }
  // |q . hi| and all its partial sums are at most this: up to 2^126 no screen score can be other than finite
  const float size = sqrtf(sq + kLostSquares) * sqrtf(hm + kLostSquares);
  const bool odd = !(size <= 8.5070592e37f);
  const float e2 = 2.f * (size * 4.8828125e-3f + 1e-30f);
  // K-th largest of the subsets' maxima (K < own, so as many subsets hold a block), from below; 64 subsets do for small K
  float bar = -CUDART_INF_F;
  if (!odd) {
    uint32_t key[4];
    if (K <= 20) {
      key[0] = key_of(fmaxf(mx[0], mx[1])), key[1] = key_of(fmaxf(mx[2], mx[3]));
      bar = own > 64 ? of_key(kth_key<2>(key, K)) - e2 : bar;
    }
    if (K > 20 || own <= 64) {
#pragma unroll
      for (int x = 0; x < 4; ++x) key[x] = key_of(mx[x]);
      bar = of_key(kth_key<4>(key, K)) - e2;
    }
  }
  // ---- candidates, in no order: pieces with one as bits, then those pieces once more
  int n = 0;
  if (!odd) {
    for (int base = 0; base < own; base += HELD * 128) {
      uint32_t hit = 0;
      if (own <= HELD * 128) {
#pragma unroll
        for (int r = 0; r < HELD; ++r) hit |= (uint32_t)(pm[r] >= bar) << r;
      } else {
#pragma unroll
        for (int r = 0; r < HELD; ++r) {
          const float4 v = piece(base + 128 * r + 4 * lane);
          hit |= (uint32_t)(fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) >= bar) << r;
        }
      }
      while (__any_sync(~0u, hit)) {
        const int j = base + 128 * (__ffs(hit) - 1) + 4 * lane;
        float4 v = make_float4(kNone, kNone, kNone, kNone);
        if (hit) v = piece(j);
        hit &= hit - 1;
        const float s[4] = {v.x, v.y, v.z, v.w};
        int at = n;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t m = __ballot_sync(~0u, s[x] >= bar);
          at += __popc(m & ((1u << lane) - 1));
          n += __popc(m);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (s[x] >= bar) {
            if (at < kCand) ls.screen[at] = s[x], ls.j[at] = j + x;
            ++at;
          }
      }
    }
    __syncwarp();
  }
  // picks: this lane's list positions lane + 32 x, as bits
  uint32_t picks = 0;
  if (odd || n > kCand) {
    n = many_candidates<D>(c, row, head, qr, ls, sc, own, odd ? -CUDART_INF_F : bar, K, status);
    for (int x = 0; x * 32 < n; ++x) {
      const int i = x * 32 + lane;
      if (i < n && among(ls, nullptr, n, K, ls.exact[i], ls.j[i])) picks |= 1u << x;
    }
  } else {
    // Candidates more than 2 e above the K-th largest screen score are in; only the others have to be told apart.
    uint32_t key[kCand / 32];
#pragma unroll
    for (int x = 0; x < kCand / 32; ++x) key[x] = x * 32 + lane < n ? key_of(ls.screen[x * 32 + lane]) : 0;
    const uint32_t kth = n <= 64 ? kth_key<2>(key, K) : (n <= 128 ? kth_key<4>(key, K) : kth_key<kCand / 32>(key, K));
    const float sure = of_key(kth | 0xffffu) + e2;
    int n_sure = 0;
    uint32_t is_sure = 0;
#pragma unroll
    for (int x = 0; x < kCand / 32; ++x)
      if (x * 32 < n) {
        const bool s = x * 32 + lane < n && of_key(key[x]) > sure;
        is_sure |= (uint32_t)s << x;
        n_sure += __popc(__ballot_sync(~0u, s));
      }
    const int m = rescore<D>(c, row, head, qr, ls, n, status, [&](int i) { return !(is_sure >> (i >> 5) & 1); });
    picks = is_sure;
    // the ones in doubt, two per lane, against all of them: by the upper words of their scores, where those decide
    for (int first = 0; first < m; first += 64) {
      int above[2] = {0, 0}, same[2] = {0, 0}, k2[2], w[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        k2[x] = first + 32 * x + lane;
        w[x] = ls.page[min(k2[x], m - 1)];
      }
#pragma unroll 8
      for (int k = 0; k < m; ++k) {
        const int o = ls.page[k];
#pragma unroll
        for (int x = 0; x < 2; ++x) above[x] += o > w[x], same[x] += o == w[x];
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (k2[x] < m) {
          const int i = ls.todo[k2[x]];
          const bool in = same[x] == 1 ? above[x] < K - n_sure : among(ls, ls.todo, m, K - n_sure, ls.exact[i], ls.j[i]);
          ls.screen[i] = in ? 1.f : 0.f;  // screen scores are done with
        }
    }
    __syncwarp();
    for (int x = 0; x * 32 < n; ++x) {
      const int i = x * 32 + lane;
      if (i < n && !(is_sure >> x & 1) && ls.screen[i] != 0.f) picks |= 1u << x;
    }
  }
  // ---- in ascending order
  __syncwarp();
  int k = 0;
  for (int x = 0; x * 32 < n; ++x) {
    const bool s = picks >> x & 1;
    const uint32_t b = __ballot_sync(~0u, s);
    if (s) ls.todo[k + __popc(b & ((1u << lane) - 1))] = ls.j[x * 32 + lane];
    k += __popc(b);
  }
  __syncwarp();
  for (int i = lane; i < topk; i += 32) {
    if (i < k) {
      const int j = ls.todo[i];
      int below = 0;
#pragma unroll 8
      for (int y = 0; y < k; ++y) below += ls.todo[y] < j;
      out[below] = j;
    } else {
      out[i] = i == k ? own : -1;
    }
  }
}

// Tiles of 16 rows, per KV head.
long long tiles_of(const View& c, int T, int h_q, int* per_token) {
  const int G = h_q / c.h_kv;
  const long long a = (long long)T * ((G + 15) / 16), b = (long long)T * G / 16 + c.rows;
  *per_token = a <= b;
  return a <= b ? a : b;
}

int stride_of(const View& c) { return (c.max_blocks + 3) / 4 * 4; }

int slab_tokens(const View& c, int T, int h_q) {
  const long long per = (long long)h_q * stride_of(c) * sizeof(float);
  const long long n = (long long)kScratch / per;
  return (int)(n < 1 ? 1 : (n < T ? n : T));
}

// Blocks per CTA of kernel one: the more, the less a tile's look-ups cost, as long as 8 CTAs per SM remain (4 where each
// warp of a CTA has a tile of its own).  A whole call for 64 rows of ragged length up to 2048 blocks takes 49.4, 40.9,
// 37.6 and 38.6 us with at most 128, 256, 512 and 1024; a single row's kernel one 6.5 us with 128 and 8.7 with 256.
int chunk_of(const View& c, int slab, int h_q) {
  int per_token;
  long long tiles = tiles_of(c, slab, h_q, &per_token) * c.h_kv;
  if (!per_token) tiles /= kScoreThreads / 32;
  int chunk = 128;
  const long long least = (per_token ? 8 : 4) * 148;
  while (chunk < 1024 && tiles * ((c.max_blocks + 2 * chunk - 1) / (2 * chunk)) >= least) chunk *= 2;
  while ((c.max_blocks + chunk - 1) / chunk > 65535) chunk *= 2;
  return chunk;
}

template <int D>
cudaError_t launch_slab(const View& c, const Plan& p, const Slab& sl, long long tiles, const bf16* q, int h_q, int topk,
                        float* score, float* hmax, int32_t* sel, int32_t* status, cudaStream_t st) {
  constexpr int WARPS = kScoreThreads / 32;
  if (sl.per_token) {
    const dim3 grid((unsigned)tiles, c.h_kv, sl.nchunk);
    score_kernel<D, true><<<grid, kScoreThreads, 0, st>>>(c, p, sl, q, h_q, score, hmax, status);
  } else {
    const dim3 grid((unsigned)((tiles + WARPS - 1) / WARPS), c.h_kv, sl.nchunk);
    score_kernel<D, false><<<grid, kScoreThreads, 0, st>>>(c, p, sl, q, h_q, score, hmax, status);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((long long)(sl.t1 - sl.t0) * h_q + kSelWarps - 1) / kSelWarps));
  cfg.blockDim = dim3(kSelWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  // The longest rows' scores should be one batch: a second look at them is then not a second read.  Half the registers
  // do where no row is longer than 1024 blocks (530 x 32 rows of up to 1017 blocks: 89 us in all, against 107).
  if (c.max_blocks <= 1024)
    return cudaLaunchKernelEx(&cfg, select_kernel<D, 8>, c, p, sl, q, h_q, topk, (const float*)score, (const float*)hmax, sel,
                              status);
  return cudaLaunchKernelEx(&cfg, select_kernel<D, 16>, c, p, sl, q, h_q, topk, (const float*)score, (const float*)hmax, sel,
                            status);
}

}  // namespace

size_t route_scratch(const View& c, int T, int h_q) {
  if (T == 0) return 0;
  const int n = slab_tokens(c, T, h_q), chunk = chunk_of(c, n, h_q);
  int per_token;
  const long long tiles = tiles_of(c, n, h_q, &per_token) + kScoreThreads / 32;
  return ((size_t)n * h_q * stride_of(c) + (size_t)tiles * c.h_kv * ((c.max_blocks + chunk - 1) / chunk)) * sizeof(float);
}

cudaError_t launch_route(const View& c, const Plan& p, const bf16* q, int h_q, int topk, int32_t* sel, void* scratch,
                         int32_t* status, cudaStream_t st) {
  const int step = slab_tokens(c, p.T, h_q);
  float* score = static_cast<float*>(scratch);
  float* hmax = score + (size_t)step * h_q * stride_of(c);
  for (int t0 = 0; t0 < p.T; t0 += step) {
    Slab sl;
    sl.t0 = t0, sl.t1 = t0 + step < p.T ? t0 + step : p.T;
    const long long tiles = tiles_of(c, sl.t1 - t0, h_q, &sl.per_token);
    sl.chunk = chunk_of(c, step, h_q);
    sl.nchunk = (c.max_blocks + sl.chunk - 1) / sl.chunk;
    sl.stride = stride_of(c);
    sl.tiles = (int)tiles;
    const cudaError_t e = c.d == 64 ? launch_slab<64>(c, p, sl, tiles, q, h_q, topk, score, hmax, sel, status, st)
                                    : launch_slab<128>(c, p, sl, tiles, q, h_q, topk, score, hmax, sel, status, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace cache
}  // namespace moba
