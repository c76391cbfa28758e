// Writing K and V rows into the paged 8-bit cache: one absmax gamma per (block
// of tokens, head), codes under the QKV-state quantizer's rule,
//
//   gamma' = max(gamma of the block's earlier tokens, max|x| of the new rows)
//   r = L / (2 (gamma' + eps)),  q = clip(rint(fl(fl(x r) + L/2)), 0, L),  L = 2^b - 1
//
// and earlier codes of the block requantized from (float)(2 q - L) *
// fl(gamma / L) where gamma grew.  The rows of one block stand together in the
// batch at consecutive slots, so the first of them (the leader: its
// predecessor's slot is not the one before, or its own starts a block) finds the
// run by reading slots alone.
//
// A CTA takes a group of rows, some heads, and K or V, and works on the runs
// that begin in its group: long runs with all its threads, short ones (a
// decode step's single rows) a warp each, the rows held in registers between
// the maximum and the codes.  The rows of the next head are on their way into
// shared memory while one is worked on (directly into registers, with more
// CTAs an SM to hide it, six prompts took 70 us instead of 64).  Bytes are all
// there is to it: 2 (4) in and 1 out per value; for few rows, the launch and
// four dependent reads.  Measured: six prompts of up to 2731 rows (32 heads of
// 128, 350 MB in and out) 64 us, 5.5 TB/s, 84% of a plain copy's rate (float
// rows 153 us, 58%; 8 heads of 256 in blocks of 128, whose rows past a thread's
// registers are read twice, 50%); 64 single rows 4 us each call in a graph; 2048
// single rows into blocks of 64 that all grow, codes read and written again,
// 162 us, 3.3 TB/s.
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

// Two codes in the low bytes.  With |x| <= gamma the sum lies in [0, L] (a
// rounding of r moves it by less than a half), so adding 1.5 * 2^23 rounds it
// to the nearest integer, ties to even, into the low mantissa bits, and no clip
// is left to do; a mask keeps what NaN gives within the codes.  The products
// are scalar: a packed f32x2 multiply comes out fused with the packed addition
// behind it, one rounding short of the rule.
__device__ __forceinline__ void code_bits2(float x0, float x1, float r, float half, uint32_t& c0, uint32_t& c1) {
  asm("{\n\t.reg .b64 P, H, M;\n\t"
      "mov.b64 P, {%2, %3};\n\tmov.b64 H, {%4, %4};\n\tmov.b64 M, {%5, %5};\n\t"
      "add.rn.f32x2 P, P, H;\n\tadd.rn.f32x2 P, P, M;\n\tmov.b64 {%0, %1}, P;\n\t}"
      : "=r"(c0), "=r"(c1)
      : "f"(__fmul_rn(x0, r)), "f"(__fmul_rn(x1, r)), "f"(half), "f"(q::kMagic));
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
  // the largest magnitudes so far (a NaN gives way to a number): in pairs for bf16, their signs of no meaning
  __device__ __forceinline__ void join(uint32_t& most) const {
    if constexpr (BF16) {
      const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(most) : "r"(w[e]));
    } else {
      float v[8], m = __uint_as_float(most);
      values(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
      most = __float_as_uint(m);
    }
  }
  static __device__ __forceinline__ float top(uint32_t most) {
    if constexpr (BF16)
      return fmaxf(__uint_as_float(most << 16 & 0x7FFFFFFFu), __uint_as_float(most & 0x7FFF0000u));
    else
      return __uint_as_float(most);
  }
  __device__ __forceinline__ uint2 codes(float r, float half, uint32_t mask) const {
    float v[8];
    values(v);
    uint32_t q[8];
#pragma unroll
    for (int e = 0; e < 8; e += 2) code_bits2(v[e], v[e + 1], r, half, q[e], q[e + 1]);
    return make_uint2(q::gather_low_bytes(q[0], q[1], q[2], q[3]) & mask, q::gather_low_bytes(q[4], q[5], q[6], q[7]) & mask);
  }
};

struct Run {
  int row;     // first row (relative to the group)
  int n;       // rows
  int slot;
};

// Where a thread's vectors of a run lie: it keeps its column and goes down the
// rows (there are at most 32 vectors in one).
template <bool BF16, int kThreadsOf>
struct Column {
  const char* from;
  int64_t down;
  int count;  // vectors of the run
  __device__ __forceinline__ Column(const KvAppendArgs& a, const void* x, int64_t stride, int64_t row, int n, int h, int thread) {
    constexpr int kSize = BF16 ? 2 : 4;
    const int shift = 31 - __clz(a.D / 8);  // vectors per row and head
    from = reinterpret_cast<const char*>(x) +
           ((row + (thread >> shift)) * stride + (int64_t)h * a.D + ((thread & ((1 << shift) - 1)) << 3)) * kSize;
    down = (kThreadsOf >> shift) * stride * kSize;
    count = n << shift;
  }
  // a block's worth: no bounds to look at
  __device__ __forceinline__ bool full() const { return count == kHold<BF16> * kThreadsOf; }
};

// One run with kThreadsOf threads (a warp or the CTA).  take: the first vectors
// of the thread; reduce: the threads' common maximum, ready before any of them
// goes on to write.
template <bool BF16, int kThreadsOf, typename Take, typename Reduce>
__device__ __forceinline__ void write_run(const KvAppendArgs& a, const Column<BF16, kThreadsOf>& at, int slot, int h,
                                          uint8_t* all_codes, float* all_scales, int thread, Take&& take, Reduce&& reduce) {
  const int block_shift = 31 - __clz(a.block);
  const int place = slot & (a.block - 1);
  const int64_t tile = (int64_t)(slot >> block_shift) * a.H + h;
  uint8_t* codes = all_codes + (tile << block_shift) * a.D;
  float* scale = all_scales + tile;
  const float old = place ? *scale : 0.0f;
  Vec8<BF16> held[kHold<BF16>];
  uint32_t most = 0;
  const bool full = at.full();
  const int count = at.count;
  take(held);
#pragma unroll
  for (int j = 0; j < kHold<BF16>; ++j) held[j].join(most);
  // the largest blocks of the widest heads are read twice
  for (int j = kHold<BF16>; thread + j * kThreadsOf < count; ++j) {
    Vec8<BF16> v;
    v.load(at.from + j * at.down);
    v.join(most);
  }
  const float m = reduce(Vec8<BF16>::top(most));
  const int L = (1 << a.bits) - 1;
  const uint32_t mask = (uint32_t)L * 0x01010101u;
  const float gamma = fmaxf(old, m);
  const float r = __fdiv_rn((float)L, __fmul_rn(2.0f, __fadd_rn(gamma, 1e-5f))), half = 0.5f * (float)L;
  if (place && gamma > old) {
    const float u = __fdiv_rn(old, (float)L);
    uint4* earlier = reinterpret_cast<uint4*>(codes);
#pragma unroll 2
    for (int i = thread; i < place * a.D / 16; i += kThreadsOf) {
      const uint4 v = earlier[i];
      const uint32_t words[4] = {v.x, v.y, v.z, v.w};
      uint32_t out[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        out[w] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int q = (int)((words[w] >> (8 * e)) & 0xFFu);
          out[w] |= code_of(__fmul_rn((float)(2 * q - L), u), r, half, L) << (8 * e);
        }
      }
      earlier[i] = make_uint4(out[0], out[1], out[2], out[3]);
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
    v.load(at.from + j * at.down);
    to[j * kThreadsOf] = v.codes(r, half, mask);
  }
  if (thread == 0 && !(place && gamma == old)) *scale = gamma;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 5) kv_append_kernel(const KvAppendArgs a, const int group, const int span) {
  constexpr int kPieces = BF16 ? 1 : 2;                             // 16-byte pieces of a vector
  constexpr int kStage = kHold<BF16> * kPieces * 16 * kThreads;     // bytes
  __shared__ __align__(16) uint8_t ring[2 * kStage];
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
      const Column<BF16, 32> at(a, x, stride, row0 + r.row, r.n, h, lane);
      auto take = [&](Vec8<BF16> (&held)[kHold<BF16>]) {
#pragma unroll
        for (int j = 0; j < kHold<BF16>; ++j) {
          held[j] = Vec8<BF16>();
          if (lane + j * 32 < at.count) held[j].load(at.from + j * at.down);
        }
      };
      write_run<BF16, 32>(a, at, r.slot, h, codes, scales, lane, take, [&](float m) {
        return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
      });
    }
  }
  // Long runs: the next run's (or head's) vectors are on their way while one is worked on.  A thread copies what it
  // will read itself, so its own wait is all the ordering there is.
  int parity = 0, run = 0, h = h0;
  const int runs_here = count[0];
  const uint32_t mine = sm100::smem_u32(ring) + tid * 16;
  auto fetch = [&](int i, int head_of, int stage) {
    if (i < runs_here) {
      const Run r = runs[0][i];
      const Column<BF16, kThreads> at(a, x, stride, row0 + r.row, r.n, head_of, tid);
      const uint32_t to = mine + stage * kStage;
      const bool full = at.full();
#pragma unroll
      for (int j = 0; j < kHold<BF16>; ++j) {
        if (full || tid + j * kThreads < at.count) {
#pragma unroll
          for (int y = 0; y < kPieces; ++y) cp_async16(to + (j * kPieces + y) * (16 * kThreads), at.from + j * at.down + 16 * y);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(0, h0, 0);
  while (run < runs_here) {
    const int next_h = h + 1 < h1 ? h + 1 : h0, next_run = h + 1 < h1 ? run : run + 1;
    fetch(next_run, next_h, parity ^ 1);
    const Run r = runs[0][run];
    const Column<BF16, kThreads> at(a, x, stride, row0 + r.row, r.n, h, tid);
    auto take = [&](Vec8<BF16> (&held)[kHold<BF16>]) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      const bool full = at.full();
#pragma unroll
      for (int j = 0; j < kHold<BF16>; ++j) {
        held[j] = Vec8<BF16>();
        if (full || tid + j * kThreads < at.count) {
#pragma unroll
          for (int y = 0; y < kPieces; ++y) held[j].raw[y] = lds128(mine + parity * kStage + (j * kPieces + y) * (16 * kThreads));
        }
      }
    };
    write_run<BF16, kThreads>(a, at, r.slot, h, codes, scales, tid, take, [&](float m) {
      m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
      if (lane == 0) tops[parity][warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, tops[parity][w]);
      parity ^= 1;
      return m;
    });
    run = next_run;
    h = next_h;
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  // Rows per CTA, then heads: as many as leave about thirty CTAs per SM, so
  // that a decode batch has one row and head a CTA, and a prompt shares the
  // search for its runs among several heads.  (About twelve: 69 us instead of
  // 64 for the six prompts, the last ones running alone.)
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
