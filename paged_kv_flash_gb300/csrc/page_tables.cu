// page_tables.cu -- block tables, slot maps and lengths of a step, built on
// the GPU from the requests' lengths (TileInfer.jl "Performance" page, "Fused
// kernels, FlashAttention and PagedAttention": the block table that maps
// positions to pages), with the free pages in a ring.
//
// Two launches.  The plan kernel, one CTA, sums tokens and pages over the
// requests (first the totals, so that a step that does not fit is refused
// before anything is written, then the prefix sums) and writes the new
// lengths and the ring's new state; being one CTA, it may write them over its
// inputs.  The fill kernel, the whole GPU, works from those outputs alone (the
// old lengths and the old ends of the ring follow from the new ones and the
// sums), one thread per new token, per page taken and per page freed, each of
// which finds its request by binary search in a prefix sum.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace {

using namespace pkv;

__device__ uint32_t g_err_tables;

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;

__device__ __forceinline__ int pages_of(int len) { return (len + kPageSize - 1) / kPageSize; }

// Last b with cu[b] <= t (cu written by an earlier kernel of the step).
__device__ __forceinline__ int find_owner(const int32_t* cu, int batch, int t) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

struct Counts {
  int tokens, taken, freed;
};

__device__ __forceinline__ Counts counts_of(int len, int fresh) {
  Counts c{0, 0, 0};
  if (fresh < 0) {
    c.freed = pages_of(len);
  } else {
    c.tokens = fresh;
    c.taken = pages_of(len + fresh) - pages_of(len);
  }
  return c;
}

__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const __grid_constant__ pkv_host::TablesLaunch a) {
  pdl_trigger();                                   // the fill kernel may be placed now
  constexpr uint32_t FULL = 0xffffffffu;
  __shared__ long long total[3];
  __shared__ int bad;
  __shared__ int wsum[3][32], carry[3];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    bad = 0;
    total[0] = total[1] = total[2] = 0;
  }
  if (tid < 3) carry[tid] = 0;
  __syncthreads();

  // totals and checks
  const int most = a.max_pages * kPageSize;
  long long sum[3] = {0, 0, 0};
  bool wrong = false;
  for (long long b = tid; b < a.batch; b += kPlanThreads) {
    const int len = a.seq_lens[b], fresh = a.new_lens[b];
    if (len < 0 || len > most || (long long)len + fresh > most) {
      wrong = true;
      continue;
    }
    const Counts c = counts_of(len, fresh);
    sum[0] += c.tokens;
    sum[1] += c.taken;
    sum[2] += c.freed;
  }
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    for (int x = 16; x >= 1; x >>= 1) sum[j] += __shfl_xor_sync(FULL, sum[j], x);
    if (lane == 0 && sum[j]) atomicAdd(reinterpret_cast<unsigned long long*>(&total[j]),
                                       (unsigned long long)sum[j]);
  }
  if (wrong) bad = 1;
  const int head = a.ring_state[0], count = a.ring_state[1];
  __syncthreads();
  const int cap = a.ring_capacity;
  const bool refuse =
      bad || head < 0 || head >= cap || count < 0 || count > cap || total[1] > count ||
      (long long)count - total[1] + total[2] > cap || total[0] > 2147483647ll ||
      (a.slots && total[0] > a.slot_capacity);
  if (refuse) {
    for (long long b = tid; b <= a.batch; b += kPlanThreads) {
      a.cu_new[b] = a.taken[b] = a.freed[b] = 0;
      if (b < a.batch) a.seq_lens_out[b] = a.seq_lens[b];
    }
    if (tid == 0) {
      a.ring_state_out[0] = head;
      a.ring_state_out[1] = count;
      atomicOr(&g_err_tables, kErrBadIndex);
    }
    return;
  }

  // prefix sums, 1,024 requests at a time
  for (long long base = 0; base < a.batch; base += kPlanThreads) {
    const long long b = base + tid;
    const bool on = b < a.batch;
    const int len = on ? a.seq_lens[b] : 0, fresh = on ? a.new_lens[b] : 0;
    const Counts c = counts_of(len, fresh);
    int v[3] = {c.tokens, c.taken, c.freed};
#pragma unroll
    for (int j = 0; j < 3; ++j) {
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int up = __shfl_up_sync(FULL, v[j], x);
        if (lane >= x) v[j] += up;
      }
      if (lane == 31) wsum[j][warp] = v[j];
    }
    __syncthreads();
    if (warp < 3) {
      int w = wsum[warp][lane];
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int up = __shfl_up_sync(FULL, w, x);
        if (lane >= x) w += up;
      }
      wsum[warp][lane] = w;
    }
    __syncthreads();
    if (on) {
      int32_t* out[3] = {a.cu_new, a.taken, a.freed};
#pragma unroll
      for (int j = 0; j < 3; ++j)
        out[j][b + 1] = carry[j] + v[j] + (warp ? wsum[j][warp - 1] : 0);
      a.seq_lens_out[b] = fresh < 0 ? 0 : len + fresh;
    }
    __syncthreads();
    if (tid < 3) carry[tid] += wsum[tid][31];
    __syncthreads();
  }
  if (tid == 0) {
    a.cu_new[0] = a.taken[0] = a.freed[0] = 0;
    a.ring_state_out[0] = (int)(((long long)head + total[1]) % cap);
    a.ring_state_out[1] = (int)(count - total[1] + total[2]);
  }
}

__global__ void __launch_bounds__(kFillThreads)
    fill_kernel(const __grid_constant__ pkv_host::TablesLaunch a) {
  pdl_wait();                                      // the plan's outputs
  const int B = a.batch, cap = a.ring_capacity;
  const int tokens = a.slots ? a.cu_new[B] : 0, taken = a.taken[B], freed = a.freed[B];
  const int head_new = a.ring_state_out[0], count_new = a.ring_state_out[1];
  const int head = (int)((((long long)head_new - taken) % cap + cap) % cap);   // before the step
  const int tail = (int)((((long long)head_new + count_new - freed) % cap + cap) % cap);
  const long long work = (long long)tokens + taken + freed;
  for (long long i = (long long)blockIdx.x * kFillThreads + threadIdx.x; i < work;
       i += (long long)gridDim.x * kFillThreads) {
    if (i < tokens) {
      const int t = (int)i, b = find_owner(a.cu_new, B, t);
      const int first = a.cu_new[b];
      const int len = a.seq_lens_out[b] - (a.cu_new[b + 1] - first);    // before the step
      const int p = len + (t - first), lp = p / kPageSize, held = pages_of(len);
      const int page = lp < held
                           ? a.table[(size_t)b * a.max_pages + lp]
                           : a.ring[((long long)head + a.taken[b] + (lp - held)) % cap];
      const bool ok = page >= 0 && page < a.num_pages;
      if (!ok) atomicOr(&g_err_tables, kErrBadIndex);
      a.slots[t] = ok ? page * kPageSize + p % kPageSize : -1;
    } else if (i < (long long)tokens + taken) {
      const int j = (int)(i - tokens), b = find_owner(a.taken, B, j);
      const int len = a.seq_lens_out[b] - (a.cu_new[b + 1] - a.cu_new[b]);
      const int page = a.ring[((long long)head + j) % cap];
      if (page < 0 || page >= a.num_pages) atomicOr(&g_err_tables, kErrBadIndex);
      a.table[(size_t)b * a.max_pages + pages_of(len) + (j - a.taken[b])] = page;
    } else {
      const int j = (int)(i - tokens - taken), b = find_owner(a.freed, B, j);
      const int page = a.table[(size_t)b * a.max_pages + (j - a.freed[b])];
      if (page < 0 || page >= a.num_pages) atomicOr(&g_err_tables, kErrBadIndex);
      a.ring[((long long)tail + j) % cap] = page;
    }
  }
}

}  // namespace

namespace pkv_host {

cudaError_t launch_tables(const TablesLaunch& a, cudaStream_t s) {
  plan_kernel<<<1, kPlanThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // one thread per token and page as far as the host knows them (the slot
  // map's size and four pages per request), at most eight CTAs per SM
  const long long guess = (long long)a.slot_capacity + 4ll * a.batch;
  const int grid = (int)std::max<long long>(
      1, std::min<long long>((guess + kFillThreads - 1) / kFillThreads, 8ll * sm_count()));
  return launch_dependent(fill_kernel, dim3(grid), dim3(kFillThreads), s, a);
}

uint32_t take_tables_error(cudaStream_t s) { return take_error_word(&g_err_tables, s); }

}  // namespace pkv_host
