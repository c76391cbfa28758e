// The bookkeeping of one serving step from request lengths alone: which rows
// of the token batch belong to which request, which blocks each request takes
// from the free list, and the slot and position of every row.
//
//   rows[b]  = sum of added[0 .. b)            first[b] = taken + sum of need[0 .. b)
//   need[b]  = ceil(total / block) - ceil(cached / block),  total = cached + added
//   table[b][had + i] = free[first[b] + i],    slot(p) = table[b][p / block] * block + p % block
//
// A few kilobytes in and out: the launch is all there is to it, so everything
// is one kernel.  Every CTA repeats the two prefix sums over the requests (at
// most 16 lengths per thread), keeps them in shared memory, and then finds the
// request of each of its token rows and new blocks by bisection; a row in a
// block that this step hands out reads its id from the free list, not from the
// table entry that another CTA writes.  Measured: 4.3 us each call in a graph
// for 192 requests of one token.
#include <cstdint>

#include "common.cuh"
#include "serving.cuh"
#include "sm100.cuh"

namespace hbl {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct Lengths {
  int cached, total;    // cached tokens, tokens after the step
  int64_t had, need;    // blocks before, blocks this step adds
  int added;
};

__device__ __forceinline__ Lengths lengths_of(const KvPlanArgs& a, int b) {
  Lengths n;
  n.cached = max(a.cached[b], 0);
  n.added = min(max(a.added[b], 0), INT32_MAX - n.cached);
  n.total = n.cached + n.added;
  const int64_t had = ((int64_t)n.cached + a.block - 1) / a.block, want = ((int64_t)n.total + a.block - 1) / a.block;
  n.had = had < a.width ? had : a.width;
  n.need = (want < a.width ? want : a.width) - n.had;
  return n;
}

// the last b in [0, B) with start[b] <= i (start rising, start[0] = 0)
__device__ __forceinline__ int request_of(const int64_t* start, int B, int64_t i) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) kv_plan_kernel(const KvPlanArgs a) {
  extern __shared__ int64_t sums[];  // rows [B + 1], then blocks [B + 1]
  int64_t* rows = sums;
  int64_t* blocks = sums + a.B + 1;
  __shared__ int64_t warp_rows[kWarps], warp_blocks[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int64_t r = 0, n = 0;
  for (int b = b0; b < b1; ++b) {
    const Lengths l = lengths_of(a, b);
    r += l.added;
    n += l.need;
  }
  int64_t ri = r, ni = n;  // inclusive over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ru = __shfl_up_sync(0xffffffffu, ri, o), nu = __shfl_up_sync(0xffffffffu, ni, o);
    if (lane >= o) {
      ri += ru;
      ni += nu;
    }
  }
  if (lane == 31) {
    warp_rows[warp] = ri;
    warp_blocks[warp] = ni;
  }
  __syncthreads();
  int64_t rbase = ri - r, nbase = ni - n;
  for (int w = 0; w < warp; ++w) {
    rbase += warp_rows[w];
    nbase += warp_blocks[w];
  }
  for (int b = b0; b < b1; ++b) {
    const Lengths l = lengths_of(a, b);
    rows[b] = rbase;
    blocks[b] = nbase;
    rbase += l.added;
    nbase += l.need;
    if (blockIdx.x == 0) {
      a.total[b] = l.total;
      a.row_start[b] = (int)(rows[b] < a.T ? rows[b] : a.T);
    }
  }
  if (b1 == a.B && (b0 < a.B || tid == 0)) {
    rows[a.B] = rbase;
    blocks[a.B] = nbase;
  }
  __syncthreads();
  const int64_t nrows = rows[a.B] < a.T ? rows[a.B] : a.T, nblocks = blocks[a.B];
  const int64_t taken = max(a.taken[0], 0);
  if (blockIdx.x == 0 && tid == 0) {
    a.row_start[a.B] = (int)nrows;
    const int64_t after = taken + nblocks;
    a.taken_out[0] = (int)(after < INT32_MAX ? after : INT32_MAX);
  }
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < nblocks; i += stride) {
    const int b = request_of(blocks, a.B, i);
    const Lengths l = lengths_of(a, b);
    const int64_t at = taken + i;
    a.table[(int64_t)b * a.width + l.had + (i - blocks[b])] = at < a.num_free ? a.free_blocks[at] : -1;
  }
  for (int64_t t = (int64_t)blockIdx.x * kThreads + tid; t < a.T; t += stride) {
    int slot = -1, pos = -1;
    if (t < nrows) {
      const int b = request_of(rows, a.B, t);
      const Lengths l = lengths_of(a, b);
      pos = l.cached + (int)(t - rows[b]);
      const int64_t col = pos / a.block;
      if (col < l.had + l.need) {
        int id;
        if (col < l.had) {
          id = a.table[(int64_t)b * a.width + col];
        } else {
          const int64_t at = taken + blocks[b] + (col - l.had);
          id = at < a.num_free ? a.free_blocks[at] : -1;
        }
        const int64_t s = (int64_t)id * a.block + pos % a.block;
        if (id >= 0 && s <= INT32_MAX) slot = (int)s;
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream) {
  const int64_t need = (a.T + kThreads - 1) / kThreads, cap = (int64_t)sm100_host::sm_count() * 2;
  const size_t smem = (size_t)(a.B + 1) * 2 * sizeof(int64_t);  // 64 KB + 16 at 4096 requests
  static std::atomic<bool> done[sm100_host::kMaxDevices];
  cudaError_t e = sm100_host::ensure_smem(kv_plan_kernel, (kMaxRequests + 1) * 2 * (int)sizeof(int64_t), done);
  if (e != cudaSuccess) return e;
  kv_plan_kernel<<<(unsigned)(need < cap ? need : cap), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace hbl
