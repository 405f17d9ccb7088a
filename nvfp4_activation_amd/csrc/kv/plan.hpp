// Block table entries, slots and offsets of one step from the requests'
// lengths (include/nvfp4rq.h, nvfp4_kv_plan).
//
// What a request adds, tokens and pages, is summed over the requests before
// it.  Every workgroup forms both running sums for itself: a lane adds up a
// run of ceil(requests / kPlanThreads) requests, and a scan over the
// workgroup gives each run's start in LDS.  It then takes its share of the
// requests, of the new pages and of the tokens, finds each one's run in LDS and
// its place or its request by walking the run.  A page id is read from the free list, not
// from the entry that another workgroup writes, so nothing is handed from one
// workgroup to another and one launch does.
//
// Bound by latency: 64 requests take 4.4 us and 4096 requests with 65111 tokens
// in all, 467 of them chunks of up to 257, 11.8 us (16 us with the offsets on
// one workgroup): 3.5 us of that to add up, 2 us to scan, the rest to walk.
// With 1024 threads a workgroup they take 5.9 and 10.4 us, with the loads of
// eight requests at once 4.9 and 17.4 us.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "host.hpp"

namespace nvfp4rq {
namespace {

constexpr int kPlanThreads = 512;

struct PlanArgs {
  const int32_t *cached, *added;
  int32_t* table;
  const int32_t *free_pages, *head_in;
  int64_t *slots, max_tokens;
  int32_t *cu_q, *kv_lens, *head_out, *missing;
  int64_t table_width, free_count;
  int32_t requests, shift;
};

struct PlanRequest {
  int64_t cached, added;
  int64_t have, fresh, narrow;  // entries held, entries to write, pages past the width
};

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int shift) {
  return (tokens + (int64_t{1} << shift) - 1) >> shift;
}

__device__ __forceinline__ PlanRequest plan_request(const PlanArgs& a, int64_t r) {
  PlanRequest q;
  const int32_t c = a.cached[r], n = a.added[r];
  q.cached = c > 0 ? c : 0;
  q.added = n > 0 ? n : 0;
  const int64_t held = pages_of(q.cached, a.shift), wants = pages_of(q.cached + q.added, a.shift);
  q.have = held < a.table_width ? held : a.table_width;
  const int64_t want = wants < a.table_width ? wants : a.table_width;
  q.fresh = want - q.have;
  q.narrow = wants - (want > held ? want : held);
  if (q.narrow < 0) q.narrow = 0;
  return q;
}

// Inclusive sum over the workgroup of one value per thread; every thread calls
// it.
__device__ __forceinline__ int64_t scan_add(int64_t v, int64_t* wave_sums) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  if (lane == 63) wave_sums[w] = v;
  __syncthreads();
  for (int i = 0; i < w; ++i) v += wave_sums[i];
  __syncthreads();
  return v;
}

// The last i with start[i] <= x, start[0] = 0 <= x.
__device__ __forceinline__ int run_of(const int64_t* start, int64_t x) {
  int lo = 0;
#pragma unroll
  for (int step = kPlanThreads / 2; step > 0; step >>= 1)
    if (start[lo + step] <= x) lo += step;
  return lo;
}

__global__ __launch_bounds__(kPlanThreads) void kv_plan_kernel(PlanArgs a) {
  __shared__ int64_t token_start[kPlanThreads], page_start[kPlanThreads];
  __shared__ int64_t wave_sums[kPlanThreads / 64];
  __shared__ int64_t totals[2];
  const int tid = threadIdx.x;
  const int64_t n = a.requests, run = (n + kPlanThreads - 1) / kPlanThreads;
  const int64_t r0 = tid * run, r1 = r0 + run < n ? r0 + run : n;
  int64_t tokens = 0, fresh = 0, narrow = 0;
  for (int64_t r = r0; r < r1; ++r) {
    const PlanRequest q = plan_request(a, r);
    tokens += q.added;
    fresh += q.fresh;
    narrow += q.narrow;
  }
  const int64_t token_end = scan_add(tokens, wave_sums);
  const int64_t page_end = scan_add(fresh, wave_sums);
  token_start[tid] = token_end - tokens;
  page_start[tid] = page_end - fresh;
  if (tid == kPlanThreads - 1) {
    totals[0] = token_end;
    totals[1] = page_end;
  }
  __syncthreads();
  const int64_t all_tokens = totals[0], all_pages = totals[1];
  const int64_t head = *a.head_in > 0 ? *a.head_in : 0;
  auto page_id = [&](int64_t p) -> int32_t {  // the p-th page that this step takes
    return head + p < a.free_count ? a.free_pages[head + p] : -1;
  };

  if (blockIdx.x == 0) {
    const int64_t all_narrow = scan_add(narrow, wave_sums);
    if (tid == kPlanThreads - 1) {
      a.cu_q[n] = static_cast<int32_t>(all_tokens);
      const int64_t left = head < a.free_count ? a.free_count - head : 0;
      const int64_t got = all_pages < left ? all_pages : left;
      *a.head_out = static_cast<int32_t>(head + got);
      a.missing[0] = static_cast<int32_t>(all_pages - got + all_narrow);
      a.missing[1] = static_cast<int32_t>(all_tokens > a.max_tokens ? all_tokens - a.max_tokens : 0);
    }
  }

  const int64_t first = static_cast<int64_t>(blockIdx.x) * kPlanThreads + tid;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kPlanThreads;
  for (int64_t r = first; r < n; r += stride) {
    const int64_t i = r / run;
    int64_t at = token_start[i];
    for (int64_t o = i * run; o < r; ++o) at += a.added[o] > 0 ? a.added[o] : 0;
    const PlanRequest q = plan_request(a, r);
    a.cu_q[r] = static_cast<int32_t>(at);
    a.kv_lens[r] = static_cast<int32_t>(q.cached + q.added);
  }
  for (int64_t p = first; p < all_pages; p += stride) {
    const int i = run_of(page_start, p);
    int64_t at = page_start[i], r = i * run;
    PlanRequest q = plan_request(a, r);
    while (p >= at + q.fresh) {  // p < all_pages: ends within the run
      at += q.fresh;
      q = plan_request(a, ++r);
    }
    a.table[r * a.table_width + q.have + (p - at)] = page_id(p);
  }
  for (int64_t t = first; t < a.max_tokens; t += stride) {
    int64_t slot = -1;
    if (t < all_tokens) {
      const int i = run_of(token_start, t);
      int64_t at = token_start[i], page = page_start[i], r = i * run;
      PlanRequest q = plan_request(a, r);
      while (t >= at + q.added) {
        at += q.added;
        page += q.fresh;
        q = plan_request(a, ++r);
      }
      const int64_t pos = q.cached + (t - at), col = pos >> a.shift;
      if (col < a.table_width) {
        const int64_t id = col < q.have ? a.table[r * a.table_width + col] : page_id(page + (col - q.have));
        if (id >= 0) slot = (id << a.shift) + (pos & ((int64_t{1} << a.shift) - 1));
      }
    }
    a.slots[t] = slot;
  }
}

}  // namespace
}  // namespace nvfp4rq
