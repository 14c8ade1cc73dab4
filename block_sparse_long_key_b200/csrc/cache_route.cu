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
// of 16 query rows of one request and KV head against 8 blocks); kernel two
// takes as b the K-th largest of the 128 maxima its threads find in disjoint
// subsets (about 1.1 K blocks pass), scores the passing blocks in 64 bits, and
// ranks them by (score, block).  Products of bf16 are exact in 64 bits and
// their sums are off by 2^-46 at most, so the result is that of exact
// arithmetic unless two scores agree to 14 digits.
#include <math_constants.h>

#include "cache.cuh"

namespace moba {
namespace cache {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kSelThreads = 128;
constexpr int kCand = 512;       // candidates ranked at a time
constexpr size_t kScratch = (size_t)256 << 20;  // screen scores held at a time

struct Slab {
  int t0, t1;        // tokens of this launch
  int per_token;     // tiles: each token on its own (1) or a request's tokens together (0)
  int chunk;         // blocks per CTA of kernel one
  int nchunk;
  int stride;        // floats per screen-score row
};

// Row r's part of the slab.
__device__ __forceinline__ int clip(int x, const Slab& s) { return min(max(x, s.t0), s.t1); }

// First tile of request r (tiles of a request's rows; relative to the slab).
__device__ __forceinline__ int tile_base(const Plan& p, const Slab& s, int r, int G) {
  return (int)((long long)(clip(__ldg(p.cu + r), s) - s.t0) * G / 16) + r;
}

// Number of earlier blocks of a token, or -1 (sees nothing), -2 (plan entry out of range).
__device__ __forceinline__ int own_block(const View& c, const Plan& p, int row, int tok) {
  const int pos = __ldg(p.pos + tok);
  if (pos < 0) return -1;
  return pos < c.state[2 * row] && pos / c.B < c.state[2 * row + 1] ? pos / c.B : -2;
}

template <int D>
__global__ void __launch_bounds__(kScoreThreads)
score_kernel(View c, Plan p, Slab sl, const bf16* __restrict__ q, int h_q, float* __restrict__ score,
             float* __restrict__ hmax, int32_t* status) {
  constexpr int NT = 4;  // n-tiles (of 8 blocks) per warp and step
  __shared__ __align__(16) bf16 qs[16 * (D + 8)];
  __shared__ float smax[kScoreThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int G = h_q / c.h_kv, head = blockIdx.y, u = blockIdx.x;
  int row, tok0, r0, nrows;
  if (sl.per_token) {
    const int tiles = (G + 15) / 16;
    tok0 = sl.t0 + u / tiles;
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
    if (r0 >= nrows) return;
  }
  const int rows = min(16, nrows - r0);
  int nb = 0;
  if (lane < rows) nb = max(0, own_block(c, p, row, tok0 + (r0 + lane) / G));
  for (int off = 1; off < 16; off <<= 1) nb = max(nb, __shfl_xor_sync(~0u, nb, off));
  nb = __shfl_sync(~0u, nb, 0);
  const int j0 = blockIdx.z * sl.chunk, j1 = min(nb, j0 + sl.chunk);
  const size_t at_max = ((size_t)u * c.h_kv + head) * sl.nchunk + blockIdx.z;
  if (j0 >= j1) return;
  auto item_of = [&](int r) { return (size_t)(tok0 + (r0 + r) / G) * h_q + head * G + (r0 + r) % G; };
  for (int i = tid; i < 16 * (D / 8); i += kScoreThreads) {
    const int r = i / (D / 8), ck = i % (D / 8);
    uint4 x = make_uint4(0, 0, 0, 0);
    if (r < rows) x = *reinterpret_cast<const uint4*>(q + item_of(r) * D + ck * 8);
    *reinterpret_cast<uint4*>(qs + r * (D + 8) + ck * 8) = x;
  }
  __syncthreads();
  // Lane's share of a row: channels 64 hh + 16 t .. + 15; k-step x of a half takes 4 of them.
  uint32_t qf[D / 16][4];
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const bf16* a = qs + g * (D + 8) + 64 * (k / 4) + 16 * t + 4 * (k % 4);
    const uint2 x = *reinterpret_cast<const uint2*>(a), y = *reinterpret_cast<const uint2*>(a + 8 * (D + 8));
    qf[k][0] = x.x, qf[k][1] = y.x, qf[k][2] = x.y, qf[k][3] = y.y;
  }
  float most = 0.f;
  for (int j = j0 + warp * NT * 8; j < j1; j += kScoreThreads / 32 * NT * 8) {
    int mine = -1;
    if (j + lane < j1) {
      mine = block_page(c, row, j + lane);
      if (mine < 0) set_status(status, kStatusBadTable);
    }
    uint4 w[NT][D / 64][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int pg = __shfl_sync(~0u, mine, n * 8 + g);
      const uint4* src = reinterpret_cast<const uint4*>(c.cent + ((size_t)max(pg, 0) * c.h_kv + head) * D + 16 * t);
#pragma unroll
      for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
        for (int x = 0; x < 2; ++x) w[n][hh][x] = pg >= 0 ? __ldg(src + hh * 8 + x) : make_uint4(0, 0, 0, 0);
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
      most = sq > most || sq != sq ? sq : most;
      const int jj = j + n * 8 + 2 * t;
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (g + 8 * r < rows) {
          float* dst = score + item_of(g + 8 * r) * sl.stride - (size_t)sl.t0 * h_q * sl.stride + jj;
          if (jj + 1 < j1) *reinterpret_cast<float2*>(dst) = make_float2(s[2 * r], s[2 * r + 1]);
          else if (jj < j1) *dst = s[2 * r];
        }
    }
  }
  for (int off = 4; off < 32; off <<= 1) {
    const float o = __shfl_xor_sync(~0u, most, off);
    most = o > most || o != o ? o : most;
  }
  if (lane == 0) smax[warp] = most;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < kScoreThreads / 32; ++i) most = smax[i] > most || smax[i] != smax[i] ? smax[i] : most;
    hmax[at_max] = most;
  }
}

// 64-bit scores of candidates [from, n): 8 lanes each.
template <int D>
__device__ void rescore(const View& c, int row, int head, const bf16* q, const int* cj, double* cs, int from, int n) {
  const int sub = threadIdx.x & 7;
  for (int base = from; base < n; base += kSelThreads / 8) {
    const int i = base + (threadIdx.x >> 3);
    double s = 0.0;
    if (i < n) {
      const int pg = block_page(c, row, cj[i]);
      if (pg >= 0) {
        const bf16* hi = c.cent + ((size_t)pg * c.h_kv + head) * D + sub * (D / 8);
        const bf16* lo = hi + (size_t)c.n_pages * c.h_kv * D;
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          float a[8], b[8], y[8];
          bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(hi) + x), a);
          bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(lo) + x), b);
          bf16x8_to_f32(*reinterpret_cast<const uint4*>(q + sub * (D / 8) + 8 * x), y);
#pragma unroll
          for (int k = 0; k < 8; ++k) s += (double)y[k] * ((double)a[k] + (double)b[k]);
        }
      } else {
        s = -CUDART_INF;
      }
    }
    for (int off = 1; off < 8; off <<= 1) s += __shfl_xor_sync(~0u, s, off);
    if (i < n && sub == 0) cs[i] = isnan(s) ? -CUDART_INF : s;
  }
}

template <int D>
__global__ void __launch_bounds__(kSelThreads)
select_kernel(View c, Plan p, Slab sl, const bf16* __restrict__ q, int h_q, int topk, const float* __restrict__ score,
              const float* __restrict__ hmax, int32_t* __restrict__ sel, int32_t* status) {
  __shared__ __align__(16) bf16 qs[D];
  __shared__ float top[kSelThreads];
  __shared__ double cs[kCand];
  __shared__ int cj[kCand];
  __shared__ int n_cand;
  __shared__ float s_b, s_norm;
  const int tid = threadIdx.x, lane = tid & 31, h = blockIdx.y;
  const int tok = sl.t0 + blockIdx.x;
  const int row = __ldg(p.row + tok);
  if ((unsigned)row >= (unsigned)c.rows) return;
  const size_t item = (size_t)tok * h_q + h;
  int32_t* out = sel + item * topk;
  const int own = own_block(c, p, row, tok);
  if (own < 0) {
    if (own == -2 && tid == 0) set_status(status, kStatusBadTable);
    if (tid < topk) out[tid] = -1;
    return;
  }
  const int K = topk - 1;
  if (own <= K) {  // every earlier block
    if (tid < topk) out[tid] = tid <= own ? tid : -1;
    return;
  }
  if (K == 0) {
    if (tid == 0) out[0] = own;
    return;
  }
  const int G = h_q / c.h_kv, head = h / G;
  const float* sc = score + ((size_t)blockIdx.x * h_q + h) * sl.stride;
  // ---- error bound e, and b
  if (tid < 32) {
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const bf16 x = q[item * D + lane * (D / 32) + i];
      qs[lane * (D / 32) + i] = x;
      const float f = __bfloat162float(x);
      sq = fmaf(f, f, sq);
    }
    for (int off = 16; off; off >>= 1) sq += __shfl_xor_sync(~0u, sq, off);
    int tile;
    if (sl.per_token) {
      tile = (tok - sl.t0) * ((G + 15) / 16) + (h % G) / 16;
    } else {
      tile = tile_base(p, sl, row, G) + ((tok - clip(__ldg(p.cu + row), sl)) * G + h % G) / 16;
    }
    float m = 0.f;
    bool bad = false;
    for (int i = lane; i * sl.chunk < own; i += 32) {
      const float x = hmax[((size_t)tile * c.h_kv + head) * sl.nchunk + i];
      bad |= !(x <= 3.0e38f);
      m = fmaxf(m, x);
    }
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, off));
    bad = __any_sync(~0u, bad) || !(sq <= 3.0e38f);
    // |q| max |hi| (2^-8 + 2^-10), and room for products below the normal range
    if (lane == 0) s_norm = bad ? CUDART_INF_F : sqrtf(sq) * sqrtf(m) * 4.8828125e-3f + 1e-30f;
  }
  float mx = -CUDART_INF_F;
  bool odd = false;  // a screen score that is not finite
  for (int j = tid; j < own; j += kSelThreads) {
    const float s = sc[j];
    odd |= !(fabsf(s) <= 3.0e38f);
    mx = fmaxf(mx, s);
  }
  top[tid] = mx;
  if (tid == 0) s_b = -CUDART_INF_F, n_cand = 0;
  odd = __syncthreads_or(odd);
  if (tid < own) {  // K < own subsets hold a block; the K-th largest maximum has K - 1 above or beside it
    int above = 0, same = 0;
#pragma unroll 8
    for (int i = 0; i < kSelThreads; ++i) {
      above += top[i] > mx;
      same += top[i] == mx;
    }
    if (above < K && above + same >= K) s_b = mx;
  }
  __syncthreads();
  const float e2 = 2.f * s_norm;
  const float bar = odd || !(e2 <= 3.0e38f) ? -CUDART_INF_F : s_b - e2;
  // ---- candidates; when the list is full the best K of it stay
  auto keep_best = [&](int from) {  // cj[0, n) with exact scores below `from`
    __syncthreads();
    const int n = n_cand;
    rescore<D>(c, row, head, qs, cj, cs, from, n);
    __syncthreads();
    double ks[kCand / kSelThreads];
    int kj[kCand / kSelThreads], kr[kCand / kSelThreads];
#pragma unroll
    for (int x = 0; x < kCand / kSelThreads; ++x) {
      const int i = tid + x * kSelThreads;
      kr[x] = K;
      if (i < n) {
        const double s = cs[i];
        const int j = cj[i];
        int above = 0;
        for (int k = 0; k < n; ++k) {
          const double o = cs[k];
          above += o > s || (o == s && cj[k] < j);
        }
        ks[x] = s, kj[x] = j, kr[x] = above;
      }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kCand / kSelThreads; ++x)
      if (kr[x] < K) cs[kr[x]] = ks[x], cj[kr[x]] = kj[x];
    if (tid == 0) n_cand = min(n, K);
    __syncthreads();
  };
  int scored = 0;
  for (int base = 0; base < own; base += kSelThreads) {
    const int j = base + tid;
    const bool in = j < own && (sc[j] >= bar || odd);
    const uint32_t m = __ballot_sync(~0u, in);
    if (m) {
      int at = 0;
      if (lane == 0) at = atomicAdd(&n_cand, __popc(m));
      at = __shfl_sync(~0u, at, 0) + __popc(m & ((1u << lane) - 1));
      if (in) cj[at] = j;
    }
    // room for one more round?  (uniform: decided from the shared count)
    if (bar == -CUDART_INF_F || (base / kSelThreads) % 3 == 2) {
      __syncthreads();
      const int n = n_cand;
      __syncthreads();
      if (n > kCand - 3 * kSelThreads) {
        keep_best(scored);
        scored = n_cand;
      }
    }
  }
  keep_best(scored);
  const int n = n_cand;
  if (tid < n) {
    const int j = cj[tid];
    int below = 0;
    for (int i = 0; i < n; ++i) below += cj[i] < j;
    out[below] = j;
  }
  for (int i = n + tid; i < topk; i += kSelThreads) out[i] = i == n ? own : -1;
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

int chunk_of(const View&) { return 256; }

}  // namespace

size_t route_scratch(const View& c, int T, int h_q) {
  if (T == 0) return 0;
  const int n = slab_tokens(c, T, h_q);
  int per_token;
  const long long tiles = tiles_of(c, n, h_q, &per_token);
  const int nchunk = (c.max_blocks + chunk_of(c) - 1) / chunk_of(c);
  return ((size_t)n * h_q * stride_of(c) + (size_t)tiles * c.h_kv * nchunk) * sizeof(float);
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
    sl.chunk = chunk_of(c);
    sl.nchunk = (c.max_blocks + sl.chunk - 1) / sl.chunk;
    sl.stride = stride_of(c);
    const dim3 g1((unsigned)tiles, c.h_kv, sl.nchunk), g2(sl.t1 - t0, h_q);
    if (c.d == 64) {
      score_kernel<64><<<g1, kScoreThreads, 0, st>>>(c, p, sl, q, h_q, score, hmax, status);
      select_kernel<64><<<g2, kSelThreads, 0, st>>>(c, p, sl, q, h_q, topk, score, hmax, sel, status);
    } else {
      score_kernel<128><<<g1, kScoreThreads, 0, st>>>(c, p, sl, q, h_q, score, hmax, status);
      select_kernel<128><<<g2, kSelThreads, 0, st>>>(c, p, sl, q, h_q, topk, score, hmax, sel, status);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace cache
}  // namespace moba
