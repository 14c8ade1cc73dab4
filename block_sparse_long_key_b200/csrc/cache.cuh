// Internal view of the paged 8-bit cache (include/moba.h) and the launchers
// of its kernels.  As in launch.h, every launcher enqueues on `st` and
// returns the launch status; none allocates or synchronises.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moba {
namespace cache {

typedef __nv_bfloat16 bf16;

enum : int32_t {
  kStatusNoPages = 1 << 4,    // a row was refused
  kStatusBadTable = 1 << 5,   // row state, page number or plan entry out of range; skipped
  kStatusNonFinite = 1 << 6   // a NaN or infinity was stored as 0
};

constexpr int kHistRing = 16;  // raw keys kept per row for the key conv
constexpr int kMaxWidth = 8;

// Device pointers and sizes of a cache; kernels take it by value.
struct View {
  int rows, n_pages, max_blocks, h_kv, d, B, kind, conv_width;
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  bf16* cent;
  bf16* tail_k;
  bf16* tail_v;
  bf16* hist;
  int32_t* table;
  int32_t* state;
  int32_t* free_pages;
  long long* ring;
};

struct Plan {
  int T;
  int32_t* cu;
  int32_t* row;
  int32_t* pos;
  int32_t* slot;
};

// What kernel one of moba_cache_tables leaves for kernel two, per row.
struct RowPlan {
  int32_t length;  // tokens before the step
  int32_t held;    // pages before the step
  int32_t from;    // ring index of the first page taken (releasing rows: of the first page given back)
  int32_t flags;   // kRowServed, kRowRelease
};
constexpr int kRowServed = 1, kRowRelease = 2;

cudaError_t launch_reset(const View& c, cudaStream_t st);
cudaError_t launch_tables(const View& c, const int32_t* new_len, int32_t* state_out, long long* ring_out,
                          const Plan& p, RowPlan* rp, int32_t* status, cudaStream_t st);
// raw_kept: of a step's raw keys, how many go to the history (conv_width - 1 + set_back; no conv: 0).
cudaError_t launch_append(const View& c, const Plan& p, const bf16* k, const bf16* v, const float* conv_w,
                          int raw_kept, int32_t* status, cudaStream_t st);
// Workspace of the router and of attention beyond the status word, in bytes.
size_t route_scratch(const View& c, int T, int h_q);
cudaError_t launch_route(const View& c, const Plan& p, const bf16* q, int h_q, int topk, int32_t* sel, void* scratch,
                         int32_t* status, cudaStream_t st);
size_t attn_scratch(const View& c, int T, int h_q);
cudaError_t launch_attention(const View& c, const Plan& p, const bf16* q, int h_q, const int32_t* sel, int topk,
                             bf16* out, float* lse, void* scratch, int32_t* status, cudaStream_t st);
// Attention over all blocks for the requests of a step that have at least `limit` query rows per KV head
// (cache_attn_rows.cu); split_blocks * B is a multiple of 128.
struct Many {
  int limit;    // at least 64
  int per_row;  // a row's tiles of 128 begin at place cu * G / 128 + row (1), or at cu * G / 64 (0)
  int split_blocks, nsplit;
};
cudaError_t launch_attention_rows(const View& c, const Plan& p, const bf16* q, int h_q, int tiles, const Many& many,
                                  bf16* out, float* lse, float* part, int32_t* status, cudaStream_t st);

// Query rows per KV head of a request in this step (below 1 if the plan makes no sense).
__device__ __forceinline__ long long request_rows(const Plan& p, int row, int G) {
  return ((long long)min(__ldg(p.cu + row + 1), p.T) - __ldg(p.cu + row)) * G;
}

// The last of rows 0 .. rows - 1 that begins at or before place u (row 0 if none does), by a whole warp: two look-ups one
// after the other for 1024 rows, where halving takes ten of them.
template <class F>
__device__ __forceinline__ int last_row(int rows, long long u, F&& place) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = rows;
  while (n > 1) {
    const int step = (n + 31) / 32, i = lane * step;
    const unsigned before = __ballot_sync(~0u, i < n && (i == 0 || place(lo + i) <= u));
    const int k = (31 - __clz(before)) * step;
    lo += k, n = min(step, n - k);
  }
  return lo;
}

// ---- what both attention kernels share (the arithmetic: cache_attn.cu)
constexpr float kOffset = 7.f;                 // exponent of a weight at the reference
constexpr float kSlack = 8.f;                  // growth of a row's maximum that leaves its reference alone
constexpr float kSmallScale = 9.0949470e-13f;  // 2^-40: V scales below add to the sum of weights by themselves

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

// Where block j of a row is read from: its page (complete blocks), its tail
// bank, or nowhere (an entry out of range).
__device__ __forceinline__ int block_page(const View& c, int row, int j) {
  if (j < 0 || j >= c.max_blocks) return -1;
  const int pg = __ldg(c.table + (size_t)row * c.max_blocks + j);
  return (unsigned)pg < (unsigned)c.n_pages ? pg : -1;
}

}  // namespace cache
}  // namespace moba
