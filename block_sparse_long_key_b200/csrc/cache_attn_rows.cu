// Attention over the whole cache for many new queries of a request (chunks of
// a prompt): the arithmetic of cache_attn.cu on tcgen05.
//
// A CTA takes 128 query rows ((token, group member) of one request and KV
// head; row = TMEM lane = softmax thread) and walks key tiles of 64 positions.
//   producers (4 warps)  8-bit pages -> fp16 K and V tiles in shared memory
//                        (128-byte swizzle, two of each); the partial block's
//                        bf16 goes the same way under powers of two that bring
//                        the largest key to 2^14 (all bits of elements down to
//                        2^-31 of it, smaller ones in steps of 2^-38) and the
//                        largest value to 2^7, as large as codes are, so that
//                        what weights lose counts as much beside both (values
//                        keep all bits down to 2^-24 of it, then steps of 2^-31)
//   products (1 thread)  S = Q K^T (M = 128, N = 64, K = d) into one of two
//                        TMEM tiles, O += P V (N = d, K = 64)
//   softmax (4 warps)    S from TMEM, weights back into its columns as fp16
// The scores of tile i + 1 are formed while the softmax is at tile i, so the
// softmax warps wait for nobody in the steady state.  S and O take 256 TMEM
// columns and the tiles 96 KB (d = 128): two CTAs share an SM.  The reference
// of a row moves only when its maximum grows by more than 2^8, so O (in TMEM)
// is seldom rescaled: weights are 2^(x - m + 7) <= 2^15.
//
// Measured on 3 chunks of 312 to 513 tokens, 32 heads of 128 over 8 KV heads (251 GFLOP): 406 us with the join, 0.62
// PFLOP/s, the tensor pipe busy 32 % of the time.  What bounds it is the softmax warps' chain per tile (load from TMEM,
// maximum, exponentials, store) and the widening of the codes, which share the issue slots (53 % taken).  Two score
// tiles and a warp for the products took it from 475 to 461 us, one pair of scales per tile to 438, exponentials under
// the reference as it is to 396 (with fewer splits).  Eight softmax warps took 454 us where four took 437.
#include <cuda_fp8.h>
#include <math_constants.h>

#include "cache.cuh"
#include "tc.cuh"

namespace moba {
namespace cache {
namespace {

constexpr int kRows = 128;      // query rows per CTA
constexpr int kKeys = 64;       // key positions per tile
constexpr int kUnits = 4;       // units of 16 positions per tile, one per producer warp
constexpr int kTailK = 14;      // exponents that the largest key and value of a partial block are brought to: a key's
constexpr int kTailV = 7;       // smallest bits count, a value is to be as large as an 8-bit code beside the same scale
constexpr int kThreads = 288;   // 4 softmax warps, 4 producer warps, 1 warp for the products

template <int D>
struct Layout {
  static constexpr int KB = D / 64;
  static constexpr uint32_t Q_REGION = 128 * 128;              // 128 rows of 64 fp16
  static constexpr uint32_t REGION = kKeys * 128;              // 64 keys of 64 fp16
  static constexpr uint32_t TILE = KB * REGION;
  static constexpr uint32_t Q_OFF = 0, K_OFF = KB * Q_REGION, V_OFF = K_OFF + 2 * TILE;
  static constexpr uint32_t UNIT_OFF = V_OFF + 2 * TILE;       // float4 [2][kUnits]: ks, log2 vs, rest, 2^-7 / vs (0: small)
  static constexpr uint32_t RED_OFF = UNIT_OFF + 2 * kUnits * 16;
  static constexpr uint32_t MB_OFF = RED_OFF + 64;             // K full, V full, S full, P full, O done: two each
  static constexpr uint32_t HOLD_OFF = MB_OFF + 80;
  static constexpr uint32_t FAIL_OFF = HOLD_OFF + 4;
  static constexpr uint32_t BYTES = FAIL_OFF + 16 + 1024;
  static constexpr uint32_t TM_S = 0, TM_O = 2 * kKeys, TMEM_COLS = 256;
};

// Instruction descriptor: fp16 operands, fp32 sums.
constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 16 codes to 32 bytes of fp16.
template <int KIND>
__device__ __forceinline__ void widen16(uint4 w, uint4& a, uint4& b) {
  widen<KIND>(w.x, a.x, a.y);
  widen<KIND>(w.y, a.z, a.w);
  widen<KIND>(w.z, b.x, b.y);
  widen<KIND>(w.w, b.z, b.w);
}

// Bounded wait for phase `parity`: the clock is looked at once in 1024 tries.
__device__ __forceinline__ bool wait(uint32_t addr, uint32_t parity, uint64_t limit_ns = 2000000000ull) {
  uint64_t t0 = 0;
  for (uint32_t n = 1;; ++n) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done) : "r"(addr), "r"(parity) : "memory");
    if (done) return true;
    if ((n & 1023u) == 0) {
      const uint64_t now = tc::globaltimer();
      if (t0 == 0) t0 = now;
      else if (now - t0 > limit_ns) return false;
    }
  }
}

// 32 lanes x 16 consecutive columns: thread t of the warp writes its lane's.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Two fp32 at a time.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// Exponent of a magnitude, within what keeps 2^(14 - e) and 2^(e - 14) normal.
__device__ __forceinline__ int exponent(float m) { return max(-100, min(127, (int)((__float_as_uint(m) >> 23) & 255) - 127)); }

// 8 bf16 times a power of two, as fp16.
__device__ __forceinline__ uint4 scale8(uint4 x, float up) {
  float f[8];
  bf16x8_to_f32(x, f);
  return make_uint4(pack_f16(f[0] * up, f[1] * up), pack_f16(f[2] * up, f[3] * up), pack_f16(f[4] * up, f[5] * up),
                    pack_f16(f[6] * up, f[7] * up));
}

__device__ __forceinline__ float amax8(uint4 x, float m) {
  float f[8];
  bf16x8_to_f32(x, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
  return m;
}

// What the weights of a tile's small V scales add to l, without the scale: from the scores once more (UK keys under one
// pair of scales).  Out of line: it is seldom called, and in place it cost every tile (blocks of 32: 459 to 478 us).
template <int UK>
__device__ __noinline__ float small_scales(uint32_t tm_s, const float4* prm, float fac, int nvis, float m) {
  float sum = 0.f;
#pragma unroll 1
  for (int x0 = 0; x0 < kKeys; x0 += 16) {
    const float4 pr = prm[x0 / UK];
    if (pr.w != 0.f) continue;
    const float f1 = fmaxf(fac * pr.x, 7.5231639e-37f);
    uint32_t w[16];
    tc::tmem_ld16(tm_s + x0, w);
    tc::tmem_ld_wait();
#pragma unroll
    for (int x = 0; x < 16; ++x)
      if (x0 + x < nvis) sum += fast_exp2(fmaf(__uint_as_float(w[x]), f1, m == -CUDART_INF_F ? 0.f : -m));
  }
  return sum;
}

// This kernel shares nothing with the one before it (attn_kernel on the requests with few rows) and starts as soon as
// that one's last CTAs have; what comes after must find both done, so the first CTA ends behind it.
__device__ __forceinline__ void end_of_cta() {
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ONE: blocks of at least a key tile, so that a tile has one pair of scales.
template <int D, int KIND, bool ONE>
__global__ void __launch_bounds__(kThreads, 2)
attn_rows_kernel(View c, Plan p, const bf16* __restrict__ q, int h_q, Many many,
                 bf16* __restrict__ out, float* __restrict__ lse, float* __restrict__ part, int32_t* status) {
  using Ly = Layout<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  const uint32_t sbase = smem_u32(sm);
  // barriers of tile i: the one of its parity, whose phase is i / 2
  const uint32_t mb_k = sbase + Ly::MB_OFF, mb_v = mb_k + 16, mb_s = mb_k + 32, mb_p = mb_k + 48, mb_o = mb_k + 64;
  auto got = [&](uint32_t mb, int i) { return wait(mb + 8 * (i & 1), (i >> 1) & 1); };
  volatile int* fail = reinterpret_cast<volatile int*>(sm + Ly::FAIL_OFF);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lb = 31 - __clz(c.B);
  const int G = h_q / c.h_kv, head = blockIdx.y, split = blockIdx.z, u0 = blockIdx.x;

  // ---- the tile's rows
  auto place = [&](int r) {
    const long long first = (long long)__ldg(p.cu + r) * G;
    return many.per_row ? first / kRows + r : first / 64;
  };
  const int row = last_row(c.rows, u0, place), t0 = __ldg(p.cu + row);
  const int r0 = (int)(u0 - place(row)) * kRows;
  const long long nrows = request_rows(p, row, G);
  if (t0 < 0 || r0 < 0 || r0 >= nrows || nrows < many.limit) return end_of_cta();
  const int rows = (int)min((long long)kRows, nrows - r0);
  const int len = c.state[2 * row], held = min(c.state[2 * row + 1], c.max_blocks);
  auto pos_of = [&](int r) {
    const int x = __ldg(p.pos + t0 + (r0 + r) / G);
    return x < len && x >> lb < held ? x : -1;
  };
  int mp = -1;  // largest position of the tile
  for (int r = lane; r < rows; r += 32) mp = max(mp, pos_of(r));
  mp = __reduce_max_sync(~0u, mp);
  const int own = mp < 0 ? -1 : mp >> lb;
  const int b0 = min(own + 1, split * many.split_blocks), b1 = min(own + 1, b0 + many.split_blocks);
  if (split > 0 && b0 >= b1) return end_of_cta();
  const int kt0 = b0 * c.B / kKeys;                                  // split_blocks * B is a multiple of kKeys
  const int kend = min(b1 * c.B, mp + 1);                            // first position behind this CTA's keys
  const int nt = mp < 0 ? 0 : (kend - kt0 * kKeys + kKeys - 1) / kKeys;
  const int tail0 = (long long)(own + 1) * c.B > len ? own * c.B : 0x7fffffff;  // first position read from the tail

  if (tid == 0) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      tc::mbar_init(mb_k + 8 * x, 4);
      tc::mbar_init(mb_v + 8 * x, 4);
      tc::mbar_init(mb_s + 8 * x, 1);
      tc::mbar_init(mb_p + 8 * x, 4);
      tc::mbar_init(mb_o + 8 * x, 1);
    }
    tc::mbar_init_fence();
    *fail = 0;
  }
  if (warp == 4) tc::tmem_alloc(sbase + Ly::HOLD_OFF, Ly::TMEM_COLS);

  // ---- queries: fp16 after a power of two per row that brings the largest magnitude to [2^8, 2^9)
  float fac = 0.f;
  int pos = -1;
  size_t item = 0;
  if (warp < 4) {
    float m = 0.f;
    if (tid < rows) {
      pos = pos_of(tid);
      if (split == 0 && pos != __ldg(p.pos + t0 + (r0 + tid) / G)) set_status(status, kStatusBadTable);
      item = (size_t)(t0 + (r0 + tid) / G) * h_q + head * G + (r0 + tid) % G;
    }
    auto piece = [&](int i) {
      return tid < rows ? __ldg(reinterpret_cast<const uint4*>(q + item * D) + i) : make_uint4(0, 0, 0, 0);
    };
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) m = amax8(piece(i), m);
    const int e = exponent(m);
    const float up = pow2f(8 - e);
    fac = pow2f(e - 8) * (kLog2e * rsqrtf((float)D));
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i)
      *reinterpret_cast<uint4*>(sm + Ly::Q_OFF + (i / 8) * Ly::Q_REGION + tc::sw128_offset(tid, i % 8)) = scale8(piece(i), up);
    tc::fence_proxy_async();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + Ly::HOLD_OFF);
  const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
  float m = -CUDART_INF_F, l = 0.f;

  if (warp >= 4 && warp < 8) {
    // =============================================================== producers
    const int pw = warp - 4;
    int tail_e[2] = {0, 0};
    if (nt > 0 && kend > tail0) {  // exponents of the tail's largest key and value
      float am[2] = {0.f, 0.f};
      const int n = (mp + 1 - tail0) * (D / 8);
      const size_t at = (((size_t)row * 2 + (own & 1)) * c.h_kv + head) * c.B * D;
      for (int i = tid - 128; i < n; i += 128) {
        am[0] = amax8(*(reinterpret_cast<const uint4*>(c.tail_k + at) + i), am[0]);
        am[1] = amax8(*(reinterpret_cast<const uint4*>(c.tail_v + at) + i), am[1]);
      }
      float* red = reinterpret_cast<float*>(sm + Ly::RED_OFF);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
#pragma unroll
        for (int off = 16; off; off >>= 1) am[z] = fmaxf(am[z], __shfl_xor_sync(~0u, am[z], off));
        if (lane == 0) red[z * 4 + pw] = am[z];
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
      for (int z = 0; z < 2; ++z)
        tail_e[z] = exponent(fmaxf(fmaxf(red[4 * z], red[4 * z + 1]), fmaxf(red[4 * z + 2], red[4 * z + 3])));
    }
    // This warp's unit of a tile is pw.  Piece z: 16 codes a lane, of row 8 (z / KB) + lane / 4 and the channels
    // 64 (z % KB) + 16 (lane % 4) on; 8 lanes then store two rows' 64 bytes, every bank once.
    constexpr int NP = D / 32;
    const int rr = lane >> 2, cq = lane & 3;
    const uint32_t code_at = rr * D + cq * 16;
    const uint32_t put_a = rr * 128 + ((2 * cq ^ rr) << 4), put_b = rr * 128 + (((2 * cq + 1) ^ rr) << 4);
    auto unit_pos = [&](int i) { return (kt0 + i) * kKeys + pw * 16; };
    // A unit's table entry (only loaded here: nothing waits for it), and what it says: page; -1: zeros; -2: tail.
    auto unit_entry = [&](int i) {
      const int ps = unit_pos(i);
      return i < nt && ps < kend && ps < tail0 ? __ldg(c.table + (size_t)row * c.max_blocks + (ps >> lb)) : 0;
    };
    auto unit_page = [&](int entry, int i) {
      const int ps = unit_pos(i);
      if (i >= nt || ps >= kend) return -1;
      if (ps >= tail0) return -2;
      if ((unsigned)entry < (unsigned)c.n_pages) return entry;
      set_status(status, kStatusBadTable);
      return -1;
    };
    auto put = [&](uint32_t base, int z, uint4 a, uint4 b) {
      unsigned char* dst = sm + base + (z % Ly::KB) * Ly::REGION + (2 * pw + z / Ly::KB) * 1024;
      *reinterpret_cast<uint4*>(dst + put_a) = a;
      *reinterpret_cast<uint4*>(dst + put_b) = b;
    };
    auto put_tail = [&](uint32_t base, const bf16* tail, int i, float up) {
      const size_t at = (((size_t)row * 2 + (own & 1)) * c.h_kv + head) * c.B * D;
      const int first = unit_pos(i) - tail0, n = mp + 1 - tail0;
#pragma unroll 1
      for (int z = 0; z < NP; ++z) {
        const int r = first + 8 * (z / Ly::KB) + rr;
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (r < n) {
          const uint4* src = reinterpret_cast<const uint4*>(tail + at + (size_t)r * D + 64 * (z % Ly::KB) + 16 * cq);
          a = scale8(src[0], up), b = scale8(src[1], up);
        }
        put(base, z, a, b);
      }
    };
    // Registers hold one tile's pieces; a tile's are asked for as soon as the ones before have been stored.
    uint4 kr[NP], vr[NP];
    float sc[2] = {0.f, 1.f};  // the unit's scales
    auto ask = [&](uint4* r, const uint8_t* base, int pg, int i) {
      const size_t at = pg >= 0 ? ((size_t)pg * c.h_kv + head) * c.B * D + (size_t)(unit_pos(i) & (c.B - 1)) * D + code_at : 0;
#pragma unroll
      for (int z = 0; z < NP; ++z) {
        r[z] = make_uint4(0, 0, 0, 0);
        if (pg >= 0) r[z] = __ldg(reinterpret_cast<const uint4*>(base + at + (z / Ly::KB) * 8 * D + (z % Ly::KB) * 64));
      }
    };
    auto ask_scales = [&](int pg) {
      if (pg >= 0) {
        const size_t at = (size_t)pg * c.h_kv + head;
        sc[0] = __ldg(c.k_scale + at), sc[1] = __ldg(c.v_scale + at);
      }
    };
    int pg = unit_page(unit_entry(0), 0), next = unit_entry(1);
    ask(kr, c.k, pg, 0);
    ask(vr, c.v, pg, 0);
    ask_scales(pg);
    for (int i = 0; i < nt; ++i) {
      const uint32_t k_tile = Ly::K_OFF + (i & 1) * Ly::TILE, v_tile = Ly::V_OFF + (i & 1) * Ly::TILE;
      // K tile free: the scores of tile i - 2 are done
      if (!__all_sync(~0u, i < 2 || got(mb_s, i - 2))) { *fail = 1; break; }
      if (pg == -2) {
        put_tail(k_tile, c.tail_k, i, pow2f(kTailK - tail_e[0]));
      } else {
#pragma unroll
        for (int z = 0; z < NP; ++z) {
          uint4 a, b;
          widen16<KIND>(kr[z], a, b);
          put(k_tile, z, a, b);
        }
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(mb_k + 8 * (i & 1));
      const float ks = pg >= 0 ? sc[0] : (pg == -2 ? pow2f(tail_e[0] - kTailK) : 0.f);
      const float vs = pg >= 0 ? sc[1] : (pg == -2 ? pow2f(tail_e[1] - kTailV) : 1.f);
      const int now = pg;
      pg = unit_page(next, i + 1);
      next = unit_entry(i + 2);
      ask(kr, c.k, pg, i + 1);
      ask_scales(pg);
      // V tile (and the unit's scales) free: the product of tile i - 2 is done, so its weights are, too
      if (!__all_sync(~0u, i < 2 || got(mb_o, i - 2))) { *fail = 1; break; }
      if (lane == 0) {
        const float vc = fmaxf(vs, 7.8886090522101181e-31f);  // 2^-100
        float4* unit = reinterpret_cast<float4*>(sm + Ly::UNIT_OFF + ((i & 1) * kUnits + pw) * 16);
        *unit = make_float4(ks, now == -1 ? -CUDART_INF_F : log2f(vc), 1.f, (1.f / 128.f) / vc);  // nothing: weights 0
        if (vs < kSmallScale) unit->z = vs / vc * 0.99999994f, unit->w = 0.f;  // below 1, and the same to 16 bits
      }
      if (now == -2) {
        put_tail(v_tile, c.tail_v, i, pow2f(kTailV - tail_e[1]));
      } else {
#pragma unroll
        for (int z = 0; z < NP; ++z) {
          uint4 a, b;
          widen16<KIND>(vr[z], a, b);
          put(v_tile, z, a, b);
        }
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(mb_v + 8 * (i & 1));
      ask(vr, c.v, pg, i + 1);
    }
  } else if (warp == 8) {
    // =============================================================== products
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_f16(kRows, kKeys, 0), id_o = idesc_f16(kRows, D, 1);
      auto scores = [&](int i) {
        tc::fence_after_sync();
        const uint32_t k_tile = sbase + Ly::K_OFF + (i & 1) * Ly::TILE;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_bf16_ss(tmem + Ly::TM_S + (i & 1) * kKeys,
                          tc::smem_desc(sbase + Ly::Q_OFF + (kk >> 2) * Ly::Q_REGION + (kk & 3) * 32, 16, 1024, tc::kLayoutSW128),
                          tc::smem_desc(k_tile + (kk >> 2) * Ly::REGION + (kk & 3) * 32, 16, 1024, tc::kLayoutSW128), id_s,
                          kk > 0);
        tc::mma_commit(mb_s + 8 * (i & 1));
      };
      bool ok = nt == 0 || got(mb_k, 0);
      if (nt > 0 && ok) scores(0);
      for (int i = 0; ok && i < nt; ++i) {
        if (i + 1 < nt) {  // the next scores go where the weights of tile i - 1 were: its product must be done
          ok = got(mb_k, i + 1) && (i == 0 || got(mb_o, i - 1)) ;
          if (!ok) break;
          scores(i + 1);
        }
        ok = got(mb_v, i) && got(mb_p, i);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t v_tile = sbase + Ly::V_OFF + (i & 1) * Ly::TILE;
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          tc::mma_bf16_ts(tmem + Ly::TM_O, tmem + Ly::TM_S + (i & 1) * kKeys + kk * 8,
                          tc::smem_desc(v_tile + kk * 2048, Ly::REGION, 1024, tc::kLayoutSW128), id_o, i > 0 || kk > 0);
        tc::mma_commit(mb_o + 8 * (i & 1));
      }
      if (!ok) *fail = 1;
    }
    __syncwarp();
  } else {
    // =============================================================== softmax
    for (int i = 0; i < nt; ++i) {
      if (!__all_sync(~0u, got(mb_s, i))) { *fail = 1; break; }
      tc::fence_after_sync();
      const uint32_t tm_s = tmem + lane_base + Ly::TM_S + (i & 1) * kKeys;
      const float4* prm = reinterpret_cast<const float4*>(sm + Ly::UNIT_OFF + (i & 1) * kUnits * 16);
      const int nvis = min(kKeys, min(pos + 1, kend) - (kt0 + i) * kKeys);  // visible keys of this row, from the first
      uint32_t s[2][32];  // scores; from its start on, pairs of weights take their place
      auto load = [&]() {
        tc::tmem_ld32(tm_s, s[0]);
        tc::tmem_ld32(tm_s + 32, s[1]);
        tc::tmem_ld_wait();
        if (!__all_sync(~0u, nvis == kKeys)) {
#pragma unroll
          for (int x = 0; x < kKeys; ++x)
            if (x >= nvis) s[x / 32][x % 32] = 0xff800000u;
        }
      };
      load();
      // the units' scales come with the V tile
      if (!__all_sync(~0u, got(mb_v, i))) { *fail = 1; break; }
      constexpr int NU = ONE ? 1 : kUnits, UK = kKeys / NU;  // groups of keys under one pair of scales
      bool odd, ok = true;  // odd: a V scale below 2^-40
      // Weights under the reference as it is, and the tile's maximum beside them (the exponentials leave room for it).
      // Where a row's maximum has outgrown its reference, which is seldom, the reference is moved and the tile done again.
      while (true) {
        const float off = kOffset - (m == -CUDART_INF_F ? 0.f : m);
        float mx = -CUDART_INF_F, add = 0.f;
        odd = false;
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const float4 pr = prm[u];
          // at least 2^-120, so that -infinity stays itself; smaller factors meet scores that they make zero anyway
          const float f1 = fmaxf(fac * pr.x, 7.5231639e-37f);
          const uint64_t f = pair(f1, f1), b = pair(pr.y + off, pr.y + off);
          uint64_t sum[2] = {0, 0};  // two zeros each
          float top[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
          for (int x = 0; x < UK; x += 2) {
            const int k = u * UK + x;
            const float s0 = __uint_as_float(s[k / 32][k % 32]), s1 = __uint_as_float(s[k / 32][k % 32 + 1]);
            float e0, e1;
            unpair(fma2(pair(s0, s1), f, b), e0, e1);
            top[0] = fmaxf(top[0], s0), top[1] = fmaxf(top[1], s1);
            e0 = fast_exp2(e0), e1 = fast_exp2(e1);
            sum[x / 2 & 1] = add2(sum[x / 2 & 1], pair(e0, e1));
            s[0][k / 2] = pack_f16(e0, e1);
          }
          mx = fmaxf(mx, fmaf(fmaxf(top[0], top[1]), f1, pr.y));
          float s0, s1;
          unpair(add2(sum[0], sum[1]), s0, s1);
          add = fmaf(s0 + s1, pr.w, add);
          odd |= pr.z != 1.f;
        }
        const bool up = mx > m + kSlack;  // m = -infinity: any
        if (!__any_sync(~0u, up)) {
          l += add;
          break;
        }
        const float half = up ? fast_exp2(0.5f * (m - mx)) : 1.f, a = half * half;
        if (up) m = mx;
        l = l * half * half;  // l may be as large as a is small
        if (i > 0) {
          ok = __all_sync(~0u, got(mb_o, i - 1));
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll 1
          for (int h = 0; h < D / 16; ++h) {
            uint32_t o[16];
            tc::tmem_ld16(tmem + lane_base + Ly::TM_O + h * 16, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * a);
            tmem_st16(tmem + lane_base + Ly::TM_O + h * 16, o);
          }
        }
        load();
      }
      if (!ok) { *fail = 1; break; }
      if (__any_sync(~0u, odd)) [[unlikely]] {
        l += small_scales<UK>(tm_s, prm, fac, nvis, m);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const float z = prm[u].z;  // as little as 2^-26: not a factor for 16 bits
#pragma unroll
          for (int x = 0; x < UK / 2; ++x) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&s[0][u * UK / 2 + x]));
            s[0][u * UK / 2 + x] = pack_f16(y.x * z, y.y * z);
          }
        }
      }
      tc::tmem_st32(tm_s, s[0]);
      tc::tmem_st_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(mb_p + 8 * (i & 1));
    }
    // ---- result
    bool fine = nt == 0 || got(mb_o, nt - 1);
    fine = __all_sync(~0u, fine) && !*fail;
    if (!fine) *fail = 1;
    tc::fence_after_sync();
    if (fine) {
      const float inv = l == 0.f ? 0.f : 1.f / (128.f * l);
#pragma unroll 1
      for (int h = 0; h < D / 16; ++h) {
        uint32_t o[16];
        if (nt > 0) {
          tc::tmem_ld16(tmem + lane_base + Ly::TM_O + h * 16, o);
          tc::tmem_ld_wait();
        } else {
#pragma unroll
          for (int x = 0; x < 16; ++x) o[x] = 0;
        }
        if (tid < rows) {
          if (many.nsplit == 1) {
#pragma unroll
            for (int x = 0; x < 16; x += 8) {
              uint4 y;
              uint32_t* yy = &y.x;
#pragma unroll
              for (int z = 0; z < 4; ++z)
                yy[z] = pack_bf16(l == 0.f ? 0.f : __uint_as_float(o[x + 2 * z]) * inv,
                                  l == 0.f ? 0.f : __uint_as_float(o[x + 2 * z + 1]) * inv);
              *reinterpret_cast<uint4*>(out + item * D + h * 16 + x) = y;
            }
          } else {
            float* b = part + (item * many.nsplit + split) * (D + 4);
#pragma unroll
            for (int x = 0; x < 16; x += 4) *reinterpret_cast<uint4*>(b + h * 16 + x) = make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
          }
        }
      }
      if (tid < rows) {
        if (many.nsplit == 1) {
          lse[item] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * 0.69314718055994531f;
        } else {
          float* b = part + (item * many.nsplit + split) * (D + 4);
          b[D] = m, b[D + 1] = l;
        }
      }
    }
    tc::fence_before_sync();
  }
  __syncthreads();
  if (*fail) {
    // A completion never arrived: record it and give what is in flight a bounded chance to drain.
    if (tid == 0) set_status(status, kStatusTimeout);
    for (int x = 0; x < 4; ++x) {
      wait(mb_s + 8 * (x & 1), x >> 1, 50000000ull);
      wait(mb_o + 8 * (x & 1), x >> 1, 50000000ull);
    }
    __syncthreads();
  }
  if (warp == 4) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, Ly::TMEM_COLS);
  }
  end_of_cta();
}

template <int D, int KIND, bool ONE>
cudaError_t launch_one(const View& c, const Plan& p, const bf16* q, int h_q, int tiles, const Many& many,
                       bf16* out, float* lse, float* part, int32_t* status, cudaStream_t st) {
  constexpr int smem = Layout<D>::BYTES;
  const cudaError_t e =
      cudaFuncSetAttribute(attn_rows_kernel<D, KIND, ONE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles, c.h_kv, many.nsplit);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_rows_kernel<D, KIND, ONE>, c, p, q, h_q, many, out, lse, part, status);
}

template <int D, int KIND>
cudaError_t launch(const View& c, const Plan& p, const bf16* q, int h_q, int tiles, const Many& many,
                   bf16* out, float* lse, float* part, int32_t* status, cudaStream_t st) {
  return c.B >= kKeys
             ? launch_one<D, KIND, true>(c, p, q, h_q, tiles, many, out, lse, part, status, st)
             : launch_one<D, KIND, false>(c, p, q, h_q, tiles, many, out, lse, part, status, st);
}

}  // namespace

cudaError_t launch_attention_rows(const View& c, const Plan& p, const bf16* q, int h_q, int tiles, const Many& many,
                                  bf16* out, float* lse, float* part, int32_t* status, cudaStream_t st) {
  if (c.d == 64)
    return c.kind == 0 ? launch<64, 0>(c, p, q, h_q, tiles, many, out, lse, part, status, st)
                       : launch<64, 1>(c, p, q, h_q, tiles, many, out, lse, part, status, st);
  return c.kind == 0 ? launch<128, 0>(c, p, q, h_q, tiles, many, out, lse, part, status, st)
                     : launch<128, 1>(c, p, q, h_q, tiles, many, out, lse, part, status, st);
}

}  // namespace cache
}  // namespace moba
