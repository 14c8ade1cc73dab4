// Block tables and slot maps of the paged cache, built on the device from the
// rows' lengths, so that no step waits for the host.
//
// Row r with L tokens in `held` pages, getting n more, needs
//   need_r = max(0, ceil((L + n) / B) - held)
// pages.  They come from a FIFO ring of free pages in row order, so row r's
// are ring entries [head + S_r - need_r, head + S_r) with S the inclusive sum
// of need: a scan.  Row r is served iff S_r <= free pages.  Pages of finished
// rows go behind the ring's end and can be taken from the next step on, so
// what is taken and what is given back never meet.
//
// Kernel one scans the rows in one CTA and writes the state after the step
// (it is the only one to read the state before, so both may be one buffer);
// kernel two lists the tokens, four per thread.  A page is first used by
// the token at its start (pages are taken only for blocks without tokens), so
// that token's thread writes the block table entry.
//
// Nothing here reads more than a few KB per thousand tokens: the time is that of a chain of dependent look-ups and
// barriers.  64 rows of one token 6.4 us; 1024 rows of 869K tokens (the token lists are 10 MB) 13 us, of which kernel
// two about 5.
#include "cache.cuh"

namespace moba {
namespace cache {
namespace {

constexpr int kScanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kCuShared = 4096;  // rows whose first tokens fit shared memory

struct Sums {
  long long tokens, need, gone;
};

__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return Sums{a.tokens + b.tokens, a.need + b.need, a.gone + b.gone};
}

__device__ __forceinline__ Sums shfl_up(const Sums& s, int off) {
  return Sums{__shfl_up_sync(~0u, s.tokens, off), __shfl_up_sync(~0u, s.need, off), __shfl_up_sync(~0u, s.gone, off)};
}

// Inclusive scan over the CTA.
__device__ Sums block_scan(Sums s, Sums* warp_sums) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  for (int off = 1; off < 32; off <<= 1) {
    const Sums o = shfl_up(s, off);
    if (lane >= off) s = s + o;
  }
  if (lane == 31) warp_sums[w] = s;
  __syncthreads();
  if (w == 0) {
    Sums t = lane < nw ? warp_sums[lane] : Sums{0, 0, 0};
    for (int off = 1; off < 32; off <<= 1) {
      const Sums o = shfl_up(t, off);
      if (lane >= off) t = t + o;
    }
    if (lane < nw) warp_sums[lane] = t;
  }
  __syncthreads();
  return w ? s + warp_sums[w - 1] : s;
}

// Lists the tokens 4 i .. 4 i + 3 (of `total`; the arrays end at T) and enters the pages whose first token is among
// them in the block table.
__device__ __forceinline__ void fill_tokens(const View& c, const Plan& p, const RowPlan* rp, const int* cu, int i, int total,
                                            int32_t* status) {
  const int lb = 31 - __clz(c.B), first = 4 * i;
  int out[3][4];
  int lo = 0, hi = c.rows;  // largest row whose tokens begin at or before `first`
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= first) lo = mid; else hi = mid;
  }
  int row = lo - 1, begin = 0, end = first, block = -1, page = -1;  // the row of the last token, its tokens, its last page
  RowPlan q{0, 0, 0, 0};
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int t = first + x;
    out[0][x] = out[1][x] = out[2][x] = -1;
    if (t >= total) continue;
    while (t >= end && row + 1 < c.rows) {
      ++row;
      begin = cu[row];
      end = row + 1 < c.rows ? cu[row + 1] : total;
      if (t < end) q = rp[row], block = -1;
    }
    out[0][x] = row;
    if (!(q.flags & kRowServed)) continue;
    const int pos = q.length + t - begin, j = pos >> lb, off = pos & (c.B - 1);
    if (j != block || off == 0) {
      int32_t* entry = c.table + (size_t)row * c.max_blocks + j;
      if (j < q.held) {
        page = *entry;
      } else {
        // from < n_pages and j - held < n_pages: one turn of the ring at most
        long long at = (long long)q.from + (j - q.held);
        if (at >= c.n_pages) at -= c.n_pages;
        page = c.free_pages[at];
        if (off == 0) *entry = page;
      }
      block = j;
      if ((unsigned)page >= (unsigned)c.n_pages) {
        set_status(status, kStatusBadTable);
        page = -1;
      }
    }
    out[1][x] = pos;
    if (page >= 0) out[2][x] = page * c.B + off;
  }
  int32_t* dst[3] = {p.row, p.pos, p.slot};
#pragma unroll
  for (int y = 0; y < 3; ++y) {
    if (first + 4 <= p.T) {
      *reinterpret_cast<int4*>(dst[y] + first) = make_int4(out[y][0], out[y][1], out[y][2], out[y][3]);
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (first + x < p.T) dst[y][first + x] = out[y][x];
    }
  }
}

// Gives the finished rows' pages back: warp `warp` of `nwarps` looks at 32 rows at once (one look-up after another cost
// 36 us for 1024 rows) and writes out a row's pages together.
__device__ __forceinline__ void release_rows(const View& c, const RowPlan* rp, int warp, int nwarps) {
  const int lane = threadIdx.x & 31;
  for (int r0 = warp; r0 < c.rows; r0 += 32 * nwarps) {
    const int mine = r0 + lane * nwarps;
    RowPlan q{0, 0, 0, 0};
    if (mine < c.rows) q = rp[mine];
    for (unsigned left = __ballot_sync(~0u, q.flags & kRowRelease); left; left &= left - 1) {
      const int src = __ffs(left) - 1;
      const int held = __shfl_sync(~0u, q.held, src), from = __shfl_sync(~0u, q.from, src);
      const int32_t* pages = c.table + (size_t)(r0 + src * nwarps) * c.max_blocks;
#pragma unroll 4
      for (int i = lane; i < held; i += 32) {
        long long at = (long long)from + i;
        if (at >= c.n_pages) at -= c.n_pages;
        if (at < c.n_pages) c.free_pages[at] = pages[i];
      }
    }
  }
}

__global__ void __launch_bounds__(kScanThreads)
scan_kernel(View c, const int32_t* new_len, int32_t* state_out, long long* ring_out, Plan p, RowPlan* rp, int alone,
            int32_t* status) {
  __shared__ Sums warp_sums[32];
  __shared__ Sums carry;
  __shared__ unsigned long long taken;
  const int tid = threadIdx.x;
  long long head = c.ring[0], tail = c.ring[1];
  const bool ring_ok = head >= 0 && tail >= head && tail - head <= c.n_pages;
  if (!ring_ok) head = tail = 0;
  const long long avail = tail - head;
  if (tid == 0) {
    status[0] = ring_ok ? 0 : kStatusBadTable;
    status[1] = 0;
    carry = Sums{0, 0, 0};
    taken = 0;
    p.cu[0] = 0;
  }
  __syncthreads();
  for (int base = 0; base < c.rows; base += kScanThreads) {
    const int r = base + tid;
    int L = 0, held = 0, n = 0;
    bool ok = true;
    long long total = 0;
    Sums s{0, 0, 0};
    if (r < c.rows) {
      L = c.state[2 * r], held = c.state[2 * r + 1], n = new_len[r];
      if (L < 0 || held < 0 || held > c.max_blocks || L > (long long)held * c.B) {
        set_status(status, kStatusBadTable);
        ok = false;
        L = held = 0;
      }
      total = ((long long)L + max(n, 0) + c.B - 1) / c.B;
      if (total > c.max_blocks) {
        set_status(status, kStatusNoPages);
        ok = false;
      }
      s.tokens = max(n, 0);
      if (ok && n >= 0) s.need = max(total - held, 0ll);
      if (n < 0) s.gone = held;
    }
    const Sums mine = s;
    int got = 0;  // pages this row takes
    s = block_scan(s, warp_sums) + carry;
    if (r < c.rows) {
      if (mine.need > 0 && s.need > avail) {
        set_status(status, kStatusNoPages);
        ok = false;
      }
      if (s.tokens > p.T) {
        if (n > 0) ok = false;
        set_status(status, kStatusBadSeqlens);
      }
      RowPlan q;
      q.length = L, q.held = held;
      q.flags = n < 0 ? kRowRelease : (ok ? kRowServed : 0);
      const long long from = n < 0 ? tail + s.gone - mine.gone : head + s.need - mine.need;
      q.from = (int)(from % c.n_pages);
      rp[r] = q;
      p.cu[r + 1] = (int)(s.tokens < p.T ? s.tokens : p.T);
      if (n < 0) {
        state_out[2 * r] = 0, state_out[2 * r + 1] = 0;
      } else if (ok) {
        state_out[2 * r] = L + n, state_out[2 * r + 1] = held + (int)mine.need;
        got = (int)mine.need;
      } else {
        state_out[2 * r] = c.state[2 * r], state_out[2 * r + 1] = c.state[2 * r + 1];
      }
    }
    got = __reduce_add_sync(~0u, got);
    if ((tid & 31) == 0 && got) atomicAdd(&taken, (unsigned long long)got);
    __syncthreads();
    if (tid == kScanThreads - 1) carry = s;
    __syncthreads();
  }
  if (tid == 0) {
    if (carry.gone > c.n_pages - avail) atomicOr(status, kStatusBadTable);
    ring_out[0] = head + (long long)taken;
    ring_out[1] = tail + carry.gone;
  }
  if (!alone) return;
  // small steps end here, without a second launch (the loop's last barrier has published rp and cu)
  const int total = (int)min(carry.tokens, (long long)p.T);
  for (int i = tid; i < (p.T + 3) / 4; i += kScanThreads) fill_tokens(c, p, rp, p.cu, i, total, status);
  release_rows(c, rp, tid >> 5, kScanThreads / 32);
}

__global__ void __launch_bounds__(kFillThreads) fill_kernel(View c, Plan p, const RowPlan* rp, int32_t* status) {
  __shared__ int cu[kCuShared];
  const bool here = c.rows <= kCuShared;
  if (here) {
    for (int i = threadIdx.x; i < c.rows; i += kFillThreads) cu[i] = __ldg(p.cu + i);
    __syncthreads();
  }
  const int nth = gridDim.x * kFillThreads;
  const int total = __ldg(p.cu + c.rows);
  const int n4 = p.T / 4 + (p.T % 4 != 0);
  for (int i = blockIdx.x * kFillThreads + threadIdx.x; i < n4; i += nth)
    fill_tokens(c, p, rp, here ? cu : p.cu, i, total, status);
  // counted from the last CTA, whose own tokens are the fewest
  release_rows(c, rp, (int)(gridDim.x - 1 - blockIdx.x) * (kFillThreads / 32) + (threadIdx.x >> 5),
               (int)gridDim.x * (kFillThreads / 32));
}

__global__ void __launch_bounds__(kFillThreads) reset_kernel(View c) {
  const size_t nth = (size_t)gridDim.x * kFillThreads;
  const size_t i0 = (size_t)blockIdx.x * kFillThreads + threadIdx.x;
  for (size_t i = i0; i < (size_t)c.n_pages; i += nth) c.free_pages[i] = (int)i;
  for (size_t i = i0; i < (size_t)c.rows * c.max_blocks; i += nth) c.table[i] = -1;
  for (size_t i = i0; i < (size_t)c.rows * 2; i += nth) c.state[i] = 0;
  const size_t tail = (size_t)c.rows * 2 * c.h_kv * c.B * c.d / 8;
  const uint4 z = make_uint4(0, 0, 0, 0);
  for (size_t i = i0; i < tail; i += nth) {
    reinterpret_cast<uint4*>(c.tail_k)[i] = z;
    reinterpret_cast<uint4*>(c.tail_v)[i] = z;
  }
  if (c.conv_width > 1)
    for (size_t i = i0; i < (size_t)c.rows * kHistRing * c.h_kv * c.d / 8; i += nth)
      reinterpret_cast<uint4*>(c.hist)[i] = z;
  if (i0 == 0) {
    c.ring[0] = 0;
    c.ring[1] = c.n_pages;
  }
}

}  // namespace

cudaError_t launch_reset(const View& c, cudaStream_t st) {
  reset_kernel<<<592, kFillThreads, 0, st>>>(c);
  return cudaGetLastError();
}

cudaError_t launch_tables(const View& c, const int32_t* new_len, int32_t* state_out, long long* ring_out,
                          const Plan& p, RowPlan* rp, int32_t* status, cudaStream_t st) {
  // One CTA lists up to four tokens per thread in less time than a second launch takes (512 rows: 4096 tokens 8.3 us in
  // one launch and 8.9 in two, 6144 tokens 10.4 and 9.0; 2000 rows of two tokens 16.4 and 14.4).
  const int alone = p.T <= 4 * kScanThreads && c.rows <= kScanThreads;
  scan_kernel<<<1, kScanThreads, 0, st>>>(c, new_len, state_out, ring_out, p, rp, alone, status);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || alone) return e;
  const int work = p.T / 4 + 1 > c.rows ? p.T / 4 + 1 : c.rows;
  const int grid = (work + kFillThreads - 1) / kFillThreads;
  fill_kernel<<<grid < 1184 ? grid : 1184, kFillThreads, 0, st>>>(c, p, rp, status);
  return cudaGetLastError();
}

}  // namespace cache
}  // namespace moba
