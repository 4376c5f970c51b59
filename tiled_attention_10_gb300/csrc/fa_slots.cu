/*
 * fa_slots.cu -- fa_paged_slots: the arrays of a paged step from its request
 * lengths (formulas in include/fa_api.h).
 *
 * Every output follows from two running sums over the requests (new tokens,
 * new pages).  A block takes both sums itself, in shared memory, and then
 * finds the request of each of its rows and of each of its new pages by
 * bisection; so one launch does all, with no pass that others wait for.  New
 * entries are taken from the free list by the blocks that need them, never
 * from the table another block is writing.  Latency is what counts: a few loads
 * one after another, 5.4 us for 128 requests of a token, 6.4 for 32 of 2000 (the
 * sums of 16384 requests cost a block 128 KB of L2 reads).
 */
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/fa_api.h"
#include "fa_launch.cuh"

namespace {

constexpr int kThreads = 512;

struct SlotParams {
  const int32_t* past_k;
  const int32_t* new_q;
  const int32_t* free_pages;
  int64_t n_free;
  int32_t* block_table;
  int32_t* cu_q;
  int32_t* seqused_k;
  int32_t* positions;
  int64_t* slot_map;
  int32_t* pages_taken;
  int64_t cap;        // max_pages * page_size
  int64_t total_q;
  int32_t n_seqs, max_pages;
  int64_t page_size;
};

struct Request {
  int64_t past, fresh, held;  // tokens held before, added, held after
};

__device__ __forceinline__ Request request(const SlotParams& p, int s) {
  const int64_t past = min(max(static_cast<int64_t>(p.past_k[s]), int64_t(0)), p.cap);
  const int64_t fresh = max(static_cast<int64_t>(p.new_q[s]), int64_t(0));
  return Request{past, fresh, min(past + fresh, p.cap)};
}

__device__ __forceinline__ int64_t pages_of(const SlotParams& p, int64_t tokens) {
  // 32-bit division where it is enough: tokens < 2^31 for all but huge tables
  const int64_t t = tokens + p.page_size - 1;
  if (t <= 0xffffffffll && p.page_size <= 0xffffffffll)
    return static_cast<uint32_t>(t) / static_cast<uint32_t>(p.page_size);
  return t / p.page_size;
}

// The last s in [0, n) with start[s] <= x (start[0] = 0, non-decreasing): the
// request that row or page x belongs to when x < start[n].
__device__ __forceinline__ int find(const int32_t* start, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) fa_slots_kernel(const SlotParams p) {
  extern __shared__ int32_t sums[];
  int32_t* const cu = sums;                    // [n + 1] rows before each request, clipped
  int32_t* const pg = sums + p.n_seqs + 1;     // [n + 1] pages before each request
  __shared__ int64_t warp_rows[kThreads / 32], warp_pages[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = p.n_seqs;
  fa::wait_for_stream();
  fa::let_next_start();

  // Running sums: each thread a contiguous run of requests, then the runs.
  const int per = (n + kThreads - 1) / kThreads;
  const int s0 = min(n, tid * per), s1 = min(n, s0 + per);
  int64_t rows = 0, pages = 0;
  for (int s = s0; s < s1; ++s) {
    const Request r = request(p, s);
    rows += r.fresh;
    pages += pages_of(p, r.held) - pages_of(p, r.past);
  }
  int64_t rows_in = rows, pages_in = pages;    // inclusive over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, rows_in, o);
    const int64_t b = __shfl_up_sync(0xffffffffu, pages_in, o);
    if (lane >= o) { rows_in += a; pages_in += b; }
  }
  if (lane == 31) { warp_rows[warp] = rows_in; warp_pages[warp] = pages_in; }
  __syncthreads();
  int64_t row0 = rows_in - rows, page0 = pages_in - pages;
  for (int w = 0; w < warp; ++w) { row0 += warp_rows[w]; page0 += warp_pages[w]; }
  for (int s = s0; s < s1; ++s) {
    const Request r = request(p, s);
    cu[s] = static_cast<int32_t>(min(row0, p.total_q));
    pg[s] = static_cast<int32_t>(page0);       // < n_seqs * max_pages < 2^31
    row0 += r.fresh;
    page0 += pages_of(p, r.held) - pages_of(p, r.past);
  }
  if (s0 < n && s1 == n) {                     // the thread of the last request
    cu[n] = static_cast<int32_t>(min(row0, p.total_q));
    pg[n] = static_cast<int32_t>(page0);
  }
  __syncthreads();

  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + tid;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t s = first; s < n; s += step) {
    p.cu_q[s] = cu[s];
    p.seqused_k[s] = static_cast<int32_t>(request(p, static_cast<int>(s)).held);
  }
  if (first == 0) {
    p.cu_q[n] = cu[n];
    p.pages_taken[0] = pg[n];
  }
  for (int64_t i = first; i < pg[n]; i += step) {
    const int s = find(pg, n, static_cast<int32_t>(i));
    const int64_t col = pages_of(p, request(p, s).past) + i - pg[s];
    p.block_table[static_cast<int64_t>(s) * p.max_pages + col] = i < p.n_free ? p.free_pages[i] : -1;
  }
  for (int64_t t = first; t < p.total_q; t += step) {
    int64_t slot = -1, pos = 0;
    if (t < cu[n]) {
      const int s = find(cu, n, static_cast<int32_t>(t));
      const Request r = request(p, s);
      pos = r.past + t - cu[s];
      if (pos < p.cap) {
        const int64_t have = pages_of(p, r.past);
        const int64_t col = pages_of(p, pos + 1) - 1;   // pos / page_size
        int32_t page;
        if (col < have) {
          page = p.block_table[static_cast<int64_t>(s) * p.max_pages + col];
        } else {
          const int64_t i = pg[s] + col - have;
          page = i < p.n_free ? p.free_pages[i] : -1;
        }
        if (page >= 0) slot = static_cast<int64_t>(page) * p.page_size + (pos - col * p.page_size);
      }
    }
    p.positions[t] = static_cast<int32_t>(min(pos, int64_t(INT32_MAX)));
    p.slot_map[t] = slot;
  }
}

struct Range {
  const void* p;
  int64_t bytes;
};
bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.bytes > 0 && b.bytes > 0 && x < y + static_cast<uintptr_t>(b.bytes) &&
         y < x + static_cast<uintptr_t>(a.bytes);
}
bool off(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

}  // namespace

extern "C" fa_status_t fa_paged_slots(const int32_t* past_k, const int32_t* new_q,
                                      const int32_t* free_pages, int64_t n_free,
                                      int32_t* block_table, int64_t n_seqs,
                                      int64_t max_pages_per_seq, int64_t page_size, int64_t total_q,
                                      int32_t* cu_seqlens_q, int32_t* seqused_k,
                                      int32_t* positions, int64_t* slot_map, int32_t* pages_taken,
                                      cudaStream_t stream) {
  if (!past_k || !new_q || !block_table || !cu_seqlens_q || !seqused_k || !pages_taken)
    return FA_ERR_INVALID_ARG;
  if (n_seqs < 1 || max_pages_per_seq < 1 || page_size < 1 || total_q < 0 || n_free < 0)
    return FA_ERR_INVALID_ARG;
  if (n_free > 0 && !free_pages) return FA_ERR_INVALID_ARG;
  if (total_q > 0 && (!positions || !slot_map)) return FA_ERR_INVALID_ARG;
  if (off(past_k, 4) || off(new_q, 4) || off(free_pages, 4) || off(block_table, 4) ||
      off(cu_seqlens_q, 4) || off(seqused_k, 4) || off(positions, 4) || off(slot_map, 8) ||
      off(pages_taken, 4))
    return FA_ERR_MISALIGNED;
  if (n_seqs > FA_SLOTS_MAX_SEQS || max_pages_per_seq > INT32_MAX / n_seqs ||
      total_q > INT32_MAX - 1024 || n_free > INT32_MAX ||
      page_size > INT32_MAX / max_pages_per_seq)
    return FA_ERR_UNSUPPORTED;
  const Range in[3] = {{past_k, n_seqs * 4}, {new_q, n_seqs * 4}, {free_pages, n_free * 4}};
  const Range out[6] = {{block_table, n_seqs * max_pages_per_seq * 4}, {cu_seqlens_q, n_seqs * 4 + 4},
                        {seqused_k, n_seqs * 4}, {positions, total_q * 4}, {slot_map, total_q * 8},
                        {pages_taken, 4}};
  for (int i = 0; i < 6; ++i) {
    for (const Range& r : in)
      if (overlap(out[i], r)) return FA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return FA_ERR_INVALID_ARG;
  }

  SlotParams p = {};
  p.past_k = past_k; p.new_q = new_q; p.free_pages = free_pages; p.n_free = n_free;
  p.block_table = block_table; p.cu_q = cu_seqlens_q; p.seqused_k = seqused_k;
  p.positions = positions; p.slot_map = slot_map; p.pages_taken = pages_taken;
  p.cap = max_pages_per_seq * page_size;
  p.total_q = total_q;
  p.n_seqs = static_cast<int32_t>(n_seqs);
  p.max_pages = static_cast<int32_t>(max_pages_per_seq);
  p.page_size = page_size;
  const size_t smem = static_cast<size_t>(n_seqs + 1) * 8;
  if (smem > fa::kFreeSmem &&
      cudaFuncSetAttribute(fa_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>((FA_SLOTS_MAX_SEQS + 1) * 8)) != cudaSuccess)
    return FA_ERR_CUDA;
  // A block for 512 rows, at most one on each of 152 SMs: more would repeat
  // the sums without spreading the rows any further.
  const int64_t want = (std::max(total_q, n_seqs) + kThreads - 1) / kThreads;
  const fa::Launch c(dim3(static_cast<unsigned>(std::min<int64_t>(want, 152))), kThreads, smem, stream);
  return cudaLaunchKernelEx(&c.cfg, fa_slots_kernel, p) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
