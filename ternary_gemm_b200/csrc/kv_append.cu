// Writing K and V rows into the paged 8-bit cache: one absmax gamma per (block
// of tokens, head), codes under the QKV-state quantizer's rule,
//
//   gamma' = max(gamma of the block's earlier tokens, max|x| of the new rows)
//   r = L / (2 (gamma' + eps)),  q = clip(rint(fl(fl(x r) + L/2)), 0, L),  L = 2^b - 1
//
// and earlier codes of the block requantized from (float)(2 q - L) *
// fl(gamma / L) where gamma grew.  The rows of one block stand together in the
// batch, so the first of them (the leader: its predecessor's slot is not the
// one before, or its own starts a block) finds the run by reading slots alone.
//
// A CTA takes a group of rows, one head, and K or V, and works on the runs
// that begin in its group: long runs with all its threads, short ones (a
// decode step's single rows) a warp each, the rows held in registers between
// the maximum and the codes.  Bytes are all there is to it: 2 (4) in and 1 out
// per value; for few rows, the launch and four dependent reads.  Measured: six
// prompts of up to 2731 rows (32 heads of 128, 350 MB in and out) 70 us, 5.0
// TB/s, 76% of a plain copy's rate (eleven instructions a value keep the issue
// slots 61% busy beside it); 64 single rows 4 us each call in a graph.
#include <cstdint>

#include "common.cuh"
#include "rowkit.cuh"
#include "serving.cuh"
#include "sm100.cuh"

namespace hbl {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxGroup = 64;   // rows of a CTA
constexpr int kMaxBlock = 128;
constexpr int kMaxSpan = 8;     // heads of a CTA
// vectors of eight values that a thread holds: 64 rows of 128 (float: 32 rows)
template <bool BF16>
constexpr int kHold = BF16 ? 8 : 4;

__device__ __forceinline__ uint32_t code_of(float x, float r, float half, int L) {
  const int c = __float2int_rn(__fadd_rn(__fmul_rn(x, r), half));
  return (uint32_t)min(max(c, 0), L);
}

// A code in the low byte.  With |x| <= gamma the sum lies in [0, L] (a
// rounding of r moves it by less than a half), so adding 1.5 * 2^23 rounds it
// to the nearest integer, ties to even, into the low mantissa bits, and no clip
// is left to do; a mask keeps what NaN gives within the codes.  Scalar
// operations: the packed f32x2 multiply and add come out fused, one rounding
// short of the rule.
__device__ __forceinline__ uint32_t code_bits(float x, float r, float half) {
  return __float_as_uint(__fadd_rn(__fadd_rn(__fmul_rn(x, r), half), q::kMagic));
}

__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a & 0x7FFF7FFFu), "r"(b & 0x7FFF7FFFu));
  return d;
}

// eight values of a row, as they lie in memory
template <bool BF16>
struct Vec8 {
  uint4 raw[BF16 ? 1 : 2] = {};
  __device__ __forceinline__ void load(const char* x) {
    const uint4* p = reinterpret_cast<const uint4*>(x);
    raw[0] = __ldg(p);
    if constexpr (!BF16) raw[1] = __ldg(p + 1);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (BF16) {
      rowkit::bf16x8_to_f32(raw[0], v);
    } else {
      const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
    }
  }
  __device__ __forceinline__ float top() const {
    if constexpr (BF16) {
      // the larger magnitude of each pair, in pairs (a NaN gives way to a number)
      const uint32_t m = max_abs2(max_abs2(raw[0].x, raw[0].y), max_abs2(raw[0].z, raw[0].w));
      return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    } else {
      float v[8], m = 0.0f;
      values(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
      return m;
    }
  }
  __device__ __forceinline__ uint2 codes(float r, float half, uint32_t mask) const {
    float v[8];
    values(v);
    uint32_t q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = code_bits(v[e], r, half);
    return make_uint2(q::gather_low_bytes(q[0], q[1], q[2], q[3]) & mask, q::gather_low_bytes(q[4], q[5], q[6], q[7]) & mask);
  }
};

struct Run {
  int row;     // first row (relative to the group)
  int n;       // rows
  int slot;
};

// One run with `threads` threads (a warp or the CTA); reduce: their common
// maximum, ready before any of them goes on to write.
template <bool BF16, int kThreadsOf, typename Reduce>
__device__ __forceinline__ void write_run(const KvAppendArgs& a, const void* x, int64_t stride, int64_t row, int n,
                                          int slot, int h, uint8_t* all_codes, float* all_scales, int thread,
                                          Reduce&& reduce) {
  const int shift = 31 - __clz(a.D / 8);                     // vectors per row and head
  const int block_shift = 31 - __clz(a.block);
  const int place = slot & (a.block - 1);
  const int64_t tile = (int64_t)(slot >> block_shift) * a.H + h;
  uint8_t* codes = all_codes + (tile << block_shift) * a.D;
  float* scale = all_scales + tile;
  const int count = n << shift;
  // a thread keeps its column and goes down the rows (there are at most 32 vectors in one)
  constexpr int kSize = BF16 ? 2 : 4;
  const char* from = reinterpret_cast<const char*>(x) +
                     ((row + (thread >> shift)) * stride + (int64_t)h * a.D + ((thread & ((1 << shift) - 1)) << 3)) * kSize;
  const int64_t down = (kThreadsOf >> shift) * stride * kSize;
  const float old = place ? *scale : 0.0f;
  Vec8<BF16> held[kHold<BF16>];
  float m = 0.0f;
  const bool full = count == kHold<BF16> * kThreadsOf;  // a block's worth: no bounds to look at
  if (full) {
#pragma unroll
    for (int j = 0; j < kHold<BF16>; ++j) held[j].load(from + j * down);
  } else {
#pragma unroll
    for (int j = 0; j < kHold<BF16>; ++j) {
      held[j] = Vec8<BF16>();
      if (thread + j * kThreadsOf < count) held[j].load(from + j * down);
    }
  }
#pragma unroll
  for (int j = 0; j < kHold<BF16>; ++j) m = fmaxf(m, held[j].top());
  // the largest blocks of the widest heads are read twice
  for (int j = kHold<BF16>; thread + j * kThreadsOf < count; ++j) {
    Vec8<BF16> v;
    v.load(from + j * down);
    m = fmaxf(m, v.top());
  }
  m = reduce(m);
  const int L = (1 << a.bits) - 1;
  const uint32_t mask = (uint32_t)L * 0x01010101u;
  const float gamma = fmaxf(old, m);
  const float r = __fdiv_rn((float)L, __fmul_rn(2.0f, __fadd_rn(gamma, 1e-5f))), half = 0.5f * (float)L;
  if (place && gamma > old) {
    const float u = __fdiv_rn(old, (float)L);
    uint32_t* words = reinterpret_cast<uint32_t*>(codes);
    for (int i = thread; i < place * a.D / 4; i += kThreadsOf) {
      const uint32_t w = words[i];
      uint32_t out = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int q = (int)((w >> (8 * e)) & 0xFFu);
        out |= code_of(__fmul_rn((float)(2 * q - L), u), r, half, L) << (8 * e);
      }
      words[i] = out;
    }
  }
  uint2* to = reinterpret_cast<uint2*>(codes + place * a.D) + thread;
  if (full) {
#pragma unroll
    for (int j = 0; j < kHold<BF16>; ++j) to[j * kThreadsOf] = held[j].codes(r, half, mask);
  } else {
#pragma unroll
    for (int j = 0; j < kHold<BF16>; ++j)
      if (thread + j * kThreadsOf < count) to[j * kThreadsOf] = held[j].codes(r, half, mask);
  }
  for (int j = kHold<BF16>; thread + j * kThreadsOf < count; ++j) {
    Vec8<BF16> v;
    v.load(from + j * down);
    to[j * kThreadsOf] = v.codes(r, half, mask);
  }
  if (thread == 0 && !(place && gamma == old)) *scale = gamma;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, BF16 ? 6 : 5) kv_append_kernel(const KvAppendArgs a, const int group, const int span) {
  __shared__ Run runs[2][kMaxGroup];  // long ones, short ones
  __shared__ int count[2];
  __shared__ float tops[2][kWarps];
  __shared__ uint32_t heads[((kMaxGroup + kMaxBlock) / kThreads + 1) * kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * group;
  const int h0 = blockIdx.y * span, h1 = min(h0 + span, a.H);
  const bool is_v = blockIdx.z != 0;
  const int64_t nslots = a.num_blocks * a.block;
  if (tid < 2) count[tid] = 0;
  // which rows of the group and of a block's length behind it begin a run (rows without a slot, and the batch's end,
  // do; place group + block counts as a beginning)
  int s = -1;
  bool head = true;
#pragma unroll
  for (int i = 0; i < (kMaxGroup + kMaxBlock) / kThreads + 1; ++i) {
    const int at = tid + i * kThreads;
    const int64_t t = row0 + at;
    int s_at = -1;
    bool head_at = true;
    if (at < group + a.block && t < a.T) {
      s_at = a.slots[t];
      head_at = s_at < 0 || (s_at & (a.block - 1)) == 0 || t == 0 || a.slots[t - 1] != s_at - 1;
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, head_at);
    if (lane == 0) heads[i * kWarps + warp] = bits;
    if (i == 0) s = s_at, head = head_at;
  }
  __syncthreads();
  if (tid < group && head && s >= 0 && s < nslots) {
    // the run ends before the next head (there is one at group + block at the latest)
    int word = (tid + 1) >> 5;
    uint32_t left = heads[word] >> ((tid + 1) & 31) << ((tid + 1) & 31);
    while (left == 0) left = heads[++word];
    const int n = word * 32 + __ffs(left) - 1 - tid;
    const int kind = n * a.D > 32 * 8 * 2 ? 0 : 1;
    runs[kind][atomicAdd(&count[kind], 1)] = {tid, n, s};
  }
  __syncthreads();
  const void* x = is_v ? a.v : a.k;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  uint8_t* codes = is_v ? a.v_codes : a.k_codes;
  float* scales = is_v ? a.v_scales : a.k_scales;
  for (int h = h0; h < h1; ++h) {
    for (int i = warp; i < count[1]; i += kWarps) {
      const Run r = runs[1][i];
      write_run<BF16, 32>(a, x, stride, row0 + r.row, r.n, r.slot, h, codes, scales, lane, [&](float m) {
        return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
      });
    }
  }
  int parity = 0;
  for (int i = 0; i < count[0]; ++i) {
    const Run r = runs[0][i];
    for (int h = h0; h < h1; ++h) {
      write_run<BF16, kThreads>(a, x, stride, row0 + r.row, r.n, r.slot, h, codes, scales, tid, [&](float m) {
        m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
        if (lane == 0) tops[parity][warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, tops[parity][w]);
        parity ^= 1;
        return m;
      });
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  // Rows per CTA, then heads: as many as leave about thirty CTAs per SM, so
  // that a decode batch has one row and head a CTA, and a prompt shares the
  // search for its runs among several heads.
  const int64_t ctas = a.T * a.H * 2, want = (int64_t)sm100_host::sm_count() * 32;
  int group = 1, span = 1;
  while (group < kMaxGroup && ctas / (group * 2) >= want) group *= 2;
  while (span < kMaxSpan && ctas / ((int64_t)group * span * 2) >= want) span *= 2;
  const dim3 grid((unsigned)((a.T + group - 1) / group), (unsigned)((a.H + span - 1) / span), 2);
  if (a.bf16)
    kv_append_kernel<true><<<grid, kThreads, 0, stream>>>(a, group, span);
  else
    kv_append_kernel<false><<<grid, kThreads, 0, stream>>>(a, group, span);
  return cudaGetLastError();
}

}  // namespace hbl
