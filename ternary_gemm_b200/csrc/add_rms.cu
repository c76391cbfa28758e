// The join between two sublayers: residual addition, RMSNorm with a gain, and
// the per-token quantizer of the next BitLinear, and its straight-through
// gradient.
//
//   h = round(x + residual),  rstd = 1 / sqrt(mean h^2 + eps),  t = fl(fl(h rstd) gain)
//   codes, scale = the H-BitLinear quantizer of t (quant.cuh)
//   g_x = g_h + rstd (g_t gain - n mean(g_t gain n)),  g_gain = sum_rows g_t n,  n = h rstd
//
// Both are bound by the rows' bytes (forward 7 per bf16 element, backward 8),
// so a row is read once: T threads hold it in registers, E vectors of eight
// values each (16-byte accesses, neighbouring threads on neighbouring
// vectors), through the row's reductions until it is written.  T = K / 32 up
// to the next power of two keeps 32 values a thread; rows past 16384 take 64.
// Short rows share a CTA.  The mean of h^2 (and of |t| for INT4) is a double
// sum rounded once, so that the codes follow from h bit for bit whatever the
// order of the sum; conversions and double adds hide behind the loads.
//
// The gain's gradient is summed over the rows in registers by a grid that
// stays (a CTA's rows one after the other), then over the CTAs by a second
// kernel, in double and in fixed order (in float: 0.1 to 0.3 us less, and errors
// of 1.06e-7 of the norm instead of 0.77e-7 at 1001 float rows).
//
// Measured at 8192 bf16 rows of 4096: forward 42 us, 5.6 TB/s, 85% of a plain
// copy's rate; gradient 49 us, 5.5 TB/s, 83% (about 45 of them the rows, the
// rest the sum over CTAs and its launch).  Other rows reach less: bf16 of 2560
// 75% and 72%, 5552 72% and 70%, 11008 68% and 70%, just above a power of two
// (1040, 2064) 60%, for threads and shared memory go by the next power; float
// rows 52 to 67%.  One row of 2560: 3.3 us on the device.
#include <cstdint>

#include "common.cuh"
#include "quant.cuh"
#include "rowkit.cuh"
#include "serving.cuh"
#include "sm100.cuh"

namespace hbl {
namespace {

using rowkit::AddD;
using rowkit::MaxF;
using rowkit::RowReduce;

template <int T_, int E_>
struct Rows {
  static constexpr int T = T_, E = E_;
  static constexpr int kThreads = T < 128 ? 128 : T;
  static constexpr int R = kThreads / T;           // rows per CTA
  static constexpr int kWarpsPerRow = T > 32 ? T / 32 : 1;
};

// eight values at element i: plain loads (h may be written over x or residual)
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (BF16) {
    rowkit::bf16x8_to_f32(*reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i), v);
  } else {
    const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
    const float4 a = f[0], b = f[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ uint4 bf16x8(const float (&v)[8]) {
  return make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) = bf16x8(v);
  } else {
    float4* f = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
    f[0] = make_float4(v[0], v[1], v[2], v[3]);
    f[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// The rows that a CTA takes next are on their way while it works on one: a
// thread copies into shared memory the vectors that it will read itself, so
// that its own wait is all the ordering there is, and the copies hold no
// registers.

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// a vector (eight values) of this thread: its place in the ring
template <typename S, bool BF16>
__device__ __forceinline__ uint32_t slot_of(uint32_t row, int tensor, int j) {
  return row + ((tensor * S::E + j) * (BF16 ? 1 : 2)) * (16 * S::kThreads) + threadIdx.x * 16;
}
template <typename S, bool BF16>
__device__ __forceinline__ void copy8(uint32_t slot, const void* p, int64_t i) {
  const char* from = reinterpret_cast<const char*>(p) + i * (BF16 ? 2 : 4);
  cp_async16(slot, from);
  if constexpr (!BF16) cp_async16(slot + 16 * S::kThreads, from + 16);
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
template <typename S, bool BF16>
__device__ __forceinline__ void take8(uint32_t slot, float (&v)[8]) {
  const uint4 a = lds128(slot);
  if constexpr (BF16) {
    rowkit::bf16x8_to_f32(a, v);
  } else {
    const uint4 b = lds128(slot + 16 * S::kThreads);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
  }
}

// the gain of this thread's vectors, held where 32 values a thread leave room
template <typename S>
__device__ __forceinline__ void load_gain(const float* gain, int j, int vectors, float (&w)[8]) {
  const int i = j * S::T + threadIdx.x % S::T;
  if (gain && i < vectors) {
    rowkit::load8<false>(gain, i * 8, w);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.0f;
  }
}

// CTAs per SM and rows in shared memory per CTA for rows of `bytes` over all
// the tensors that are copied: as many CTAs as their registers allow (at most
// 128 a thread) while two rows each fit, a third where it fits too; rows that
// do not fit twice are read straight into registers (no stages).
struct Flow {
  int blocks, stages;
};
constexpr int most_blocks(int threads) { return 512 / threads; }
constexpr Flow flow_for(int threads, int bytes) {
  const int room = 224 * 1024;
  for (int blocks = most_blocks(threads); blocks >= 1; blocks /= 2)
    for (int stages = 3; stages >= 2; --stages)
      if (blocks * stages * bytes <= room) return {blocks, stages};
  return {most_blocks(threads), 0};
}

// kStages 0: a CTA per S::R rows, read straight into registers; else a grid
// that stays, its rows copied kStages - 1 ahead
template <typename S, bool BF16, int BITS, int kStages, int kBlocks>
__global__ void __launch_bounds__(S::kThreads, kBlocks)
add_rms_quant_kernel(const void* x, const void* residual, int64_t M, int K, const float* __restrict__ gain, void* h,
                     int8_t* codes, float* scales) {
  constexpr int T = S::T, E = S::E, WPR = S::kWarpsPerRow;
  constexpr uint32_t kRow = 2 * E * S::kThreads * (BF16 ? 16 : 32);
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  __shared__ double red_d[2][2][S::R * WPR];
  __shared__ float red_f[2][S::R * WPR];
  const int rl = threadIdx.x / T, t = threadIdx.x % T;
  const int vectors = K / 8;
  const int64_t step = (int64_t)gridDim.x * S::R;
  const uint32_t ring = sm100::smem_u32(ring_bytes);

  float w[kStages > 0 ? E : 1][8];
  if constexpr (kStages > 0) {
#pragma unroll
    for (int j = 0; j < E; ++j) load_gain<S>(gain, j, vectors, w[j]);
  }
  auto fetch = [&](int64_t row, uint32_t at) {
    if (row < M) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int i = j * T + t;
        if (i < vectors) {
          copy8<S, BF16>(slot_of<S, BF16>(at, 0, j), x, row * K + i * 8);
          if (residual) copy8<S, BF16>(slot_of<S, BF16>(at, 1, j), residual, row * K + i * 8);
        }
      }
    }
    cp_commit();
  };
  int64_t row = (int64_t)blockIdx.x * S::R + rl;
  uint32_t here = ring, next = ring;
  if constexpr (kStages > 0) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      fetch(row + i * step, next);
      next += kRow;
    }
  }
  int parity = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * S::R; row0 < M; row0 += step, row += step, parity ^= 1) {
    const bool active = row < M;
    const int64_t base = (active ? row : 0) * K;
    if constexpr (kStages > 0) {
      fetch(row + (kStages - 1) * step, next);
      next = next == ring + (kStages - 1) * kRow ? ring : next + kRow;
      cp_wait<kStages - 1>();
    }
    float v[E][8];
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int i = j * T + t;
      if (active && i < vectors) {
        if constexpr (kStages > 0)
          take8<S, BF16>(slot_of<S, BF16>(here, 0, j), v[j]);
        else
          load8<BF16>(x, base + i * 8, v[j]);
        if (residual) {
          float r[8];
          if constexpr (kStages > 0)
            take8<S, BF16>(slot_of<S, BF16>(here, 1, j), r);
          else
            load8<BF16>(residual, base + i * 8, r);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] = __fadd_rn(v[j][e], r[e]);
          if constexpr (BF16) rowkit::bf16x8_to_f32(bf16x8(v[j]), v[j]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = 0.0f;
      }
    }
    if constexpr (kStages > 0) here = here == ring + (kStages - 1) * kRow ? ring : here + kRow;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int i = j * T + t;
      if (h && active && i < vectors) store8<BF16>(h, base + i * 8, v[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fma((double)v[j][e], (double)v[j][e], ss);
    }
    ss = RowReduce<T, WPR>::run(ss, AddD(), red_d[parity][0], rl, t);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn((float)(ss / (double)K), 1e-5f)));
    float top = 0.0f;
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if constexpr (kStages == 0) load_gain<S>(gain, j, vectors, w[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[j][e] = __fmul_rn(__fmul_rn(v[j][e], rstd), w[kStages > 0 ? j : 0][e]);  // times 1 is exact
        if constexpr (BITS == 8)
          top = fmaxf(top, fabsf(v[j][e]));
        else
          sum += q::abs_f64(v[j][e]);
      }
    }
    q::RowParams p;
    if constexpr (BITS == 8)
      p = q::params_int8(RowReduce<T, WPR>::run(top, MaxF(), red_f[parity], rl, t));
    else
      p = q::params_int4(RowReduce<T, WPR>::run(sum, AddD(), red_d[parity][1], rl, t), K);
    if (!active) continue;
    if (t == 0) scales[row] = p.scale();
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int i = j * T + t;
      uint32_t m[8];
#pragma unroll
      for (int e = 0; e < 8; e += 2) rowkit::magic2(v[j][e], v[j][e + 1], p.r, m[e], m[e + 1]);
      if constexpr (BITS == 4) {
#pragma unroll
        for (int e = 0; e < 8; ++e) m[e] = q::clip_magic_int4(m[e]);
      }
      if (i < vectors)
        *reinterpret_cast<uint2*>(codes + base + i * 8) =
            make_uint2(q::gather_low_bytes(m[0], m[1], m[2], m[3]), q::gather_low_bytes(m[4], m[5], m[6], m[7]));
    }
  }
}

// ---------------------------------------------------------------- gradient

// B blocks of an SM as one, which leaves one row of partial sums instead of B
// (592 of them took 8 us to add up at 4096 columns).
template <typename S, int B>
struct Wide {
  static constexpr int T = S::T, E = S::E;
  static constexpr int kThreads = B * S::kThreads;
  static constexpr int R = B * S::R;
  static constexpr int kWarpsPerRow = S::kWarpsPerRow;
};

// A grid that stays: a thread's columns of the gain's sums stay in registers
// over its rows.  kStages as above (three tensors a row).  Row r goes to CTA
// r mod grid, so that few rows still take many SMs.
template <typename S, bool BF16, bool GT16, int kStages>
__global__ void __launch_bounds__(S::kThreads, most_blocks(S::kThreads))
add_rms_grad_kernel(const void* __restrict__ h, int64_t M, int K, const float* __restrict__ gain,
                    const void* __restrict__ g_t, const void* g_h, void* g_x, float* __restrict__ sums) {
  constexpr int T = S::T, E = S::E, WPR = S::kWarpsPerRow;
  constexpr bool kRinged = kStages > 0, kGain = kRinged && E <= 4;
  constexpr uint32_t kH = E * S::kThreads * (BF16 ? 16 : 32), kT = E * S::kThreads * (GT16 ? 16 : 32);
  constexpr uint32_t kRow = 2 * kH + kT;  // h, g_h, g_t
  extern __shared__ __align__(16) uint8_t ring_bytes[];
  __shared__ float2 red[2][S::R * WPR];
  const int rl = threadIdx.x / T, t = threadIdx.x % T;
  const int vectors = K / 8;
  const float inv_k = __fdiv_rn(1.0f, (float)K);
  // Row sums are taken of h 2^-8: h^2 over at most 2^15 columns stays in float wherever its mean does, which is where
  // the forward's rstd is not 0.  Powers of two: the same bits.
  constexpr float kDown = 0x1p-8f;
  const float mean_h2 = inv_k * 0x1p16f, mean_gh = inv_k * 0x1p8f;
  const int64_t grid = gridDim.x, step = grid * S::R;
  const uint32_t ring = sm100::smem_u32(ring_bytes);
  float acc[E][8], w[kGain ? E : 1][8];
#pragma unroll
  for (int j = 0; j < E; ++j) {
    if constexpr (kGain) load_gain<S>(gain, j, vectors, w[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[j][e] = 0.0f;
  }
  auto fetch = [&](int64_t row, uint32_t at) {
    if (row < M) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int i = j * T + t;
        if (i < vectors) {
          copy8<S, BF16>(slot_of<S, BF16>(at, 0, j), h, row * K + i * 8);
          copy8<S, GT16>(slot_of<S, GT16>(at + 2 * kH, 0, j), g_t, row * K + i * 8);
          if (g_h) copy8<S, BF16>(slot_of<S, BF16>(at, 1, j), g_h, row * K + i * 8);
        }
      }
    }
    cp_commit();
  };
  int64_t row = blockIdx.x + rl * grid;
  uint32_t here = ring, next = ring;
  if constexpr (kRinged) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      fetch(row + i * step, next);
      next += kRow;
    }
  }
  int parity = 0;
  for (int64_t row0 = blockIdx.x; row0 < M; row0 += step, row += step, parity ^= 1) {
    const bool active = row < M;
    const int64_t base = (active ? row : 0) * K;
    if constexpr (kRinged) {
      fetch(row + (kStages - 1) * step, next);
      next = next == ring + (kStages - 1) * kRow ? ring : next + kRow;
      cp_wait<kStages - 1>();
    }
    auto read = [&](int j, float (&hv)[8], float (&gv)[8]) {
      const int i = j * T + t;
      if (active && i < vectors) {
        if constexpr (kRinged) {
          take8<S, BF16>(slot_of<S, BF16>(here, 0, j), hv);
          take8<S, GT16>(slot_of<S, GT16>(here + 2 * kH, 0, j), gv);
        } else {
          load8<BF16>(h, base + i * 8, hv);
          load8<GT16>(g_t, base + i * 8, gv);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) hv[e] = gv[e] = 0.0f;
      }
    };
    // both passes over the row read it from the ring (without one: from L2 the second time)
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      float hv[8], gv[8], s = 0.0f, d = 0.0f;
      read(j, hv, gv);
      if constexpr (!kGain) load_gain<S>(gain, j, vectors, w[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = hv[e] * kDown;
        s = fmaf(v, v, s);
        d = fmaf(gv[e] * w[kGain ? j : 0][e], v, d);
      }
      ss += s;
      dot += d;
    }
#pragma unroll
    for (int o = (T < 32 ? T : 32) / 2; o >= 1; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    if constexpr (T > 32) {
      if ((t & 31) == 0) red[parity][rl * WPR + (t >> 5)] = make_float2(ss, dot);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + rl), "n"(T) : "memory");  // the row's threads
      ss = dot = 0.0f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) {
        const float2 r = red[parity][rl * WPR + i];
        ss += r.x;
        dot += r.y;
      }
    }
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(ss, mean_h2, 1e-5f)));
    const float c = dot * rstd * mean_gh;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int i = j * T + t;
      const bool there = active && i < vectors;
      float hv[8], gv[8], out[8];
      read(j, hv, gv);
      if constexpr (!kGain) load_gain<S>(gain, j, vectors, w[0]);
      if (g_h && there) {
        if constexpr (kRinged)
          take8<S, BF16>(slot_of<S, BF16>(here, 1, j), out);
        else
          load8<BF16>(g_h, base + i * 8, out);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = hv[e] * rstd;
        acc[j][e] = fmaf(gv[e], n, acc[j][e]);
        out[e] = fmaf(rstd, fmaf(-n, c, gv[e] * w[kGain ? j : 0][e]), out[e]);
      }
      if (there) store8<BF16>(g_x, base + i * 8, out);
    }
    if constexpr (kRinged) here = here == ring + (kStages - 1) * kRow ? ring : here + kRow;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the sum over CTAs waits for the grid's end
  if (!sums) return;
  sums += (int64_t)blockIdx.x * K;
  if constexpr (S::R == 1) {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int i = j * T + t;
      if (i < vectors) store8<false>(sums, i * 8, acc[j]);
    }
  } else {
    // the CTA's rows, in order, through the ring's memory
    static_assert(kRinged && 2 * kRow >= S::R * T * E * 32, "the sums fit the ring");
    float4* part = reinterpret_cast<float4*>(ring_bytes);  // [row][half of a vector][vector]
    cp_wait<0>();
    __syncthreads();
#pragma unroll
    for (int j = 0; j < E; ++j) {
      float4* to = part + rl * 2 * T * E + j * T + t;
      to[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
      to[T * E] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < vectors; i += S::kThreads) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float4 s = part[half * T * E + i];
#pragma unroll
        for (int r = 1; r < S::R; ++r) {
          const float4 v = part[(2 * r + half) * T * E + i];
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        reinterpret_cast<float4*>(sums)[2 * i + half] = s;
      }
    }
  }
}

// g_gain[k] = sum of the partial sums [count][K], in double: 32 columns per CTA,
// 32 warps on every 32nd row (the partial sums are in L2: round trips are what
// counts)
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32)
gain_sum_kernel(const float* sums, int count, int K, float* g_gain) {
  __shared__ double part[kSumWarps][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  double s = 0.0;
  if (k < K) {
#pragma unroll 8
    for (int i = warp; i < count; i += kSumWarps) s += (double)sums[(int64_t)i * K + k];
  }
  part[warp][lane] = s;
  __syncthreads();
  s = part[lane][warp];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int to = blockIdx.x * 32 + warp;
  if (lane == 0 && to < K) g_gain[to] = (float)s;
}

// f(Rows<T, E>()) for the rows of K values
template <typename F>
cudaError_t by_length(int64_t K, F&& f) {
  if (K <= 1024) return f(Rows<32, 4>());
  if (K <= 2048) return f(Rows<64, 4>());
  if (K <= 4096) return f(Rows<128, 4>());
  if (K <= 8192) return f(Rows<256, 4>());
  if (K <= 16384) return f(Rows<512, 4>());
  return f(Rows<512, 8>());
}

template <typename Kernel, typename... Args>
cudaError_t start(Kernel kernel, std::atomic<bool> (&done)[sm100_host::kMaxDevices], int64_t grid, int threads, int smem,
                  cudaStream_t stream, Args... args) {
  if (smem) {
    cudaError_t e = sm100_host::ensure_smem(kernel, smem, done);
    if (e != cudaSuccess) return e;
  }
  kernel<<<(unsigned)grid, threads, smem, stream>>>(args...);
  return cudaGetLastError();
}

// CTAs of the gradient, and rows of partial sums of the gain's
int64_t grad_grid(int64_t M, int blocks) {
  const int64_t cap = (int64_t)sm100_host::sm_count() * blocks;
  return M < cap ? M : cap;
}

template <typename S>
int64_t staying_grid(int64_t M, int blocks) {
  const int64_t need = (M + S::R - 1) / S::R, cap = (int64_t)sm100_host::sm_count() * blocks;
  return need < cap ? need : cap;
}

template <typename S, bool BF16, int BITS>
cudaError_t launch_quant(const void* x, const void* residual, int64_t M, int64_t K, const float* gain, void* h,
                         int8_t* codes, float* scales, cudaStream_t stream) {
  constexpr int row_bytes = 2 * S::E * S::kThreads * (BF16 ? 16 : 32);
  constexpr Flow flow = flow_for(S::kThreads, row_bytes);
  static std::atomic<bool> done[sm100_host::kMaxDevices];
  const int64_t need = (M + S::R - 1) / S::R, grid = staying_grid<S>(M, flow.blocks);
  // less than two rounds of the staying grid: nothing to copy ahead
  if (flow.stages == 0 || need < 2 * grid)
    return start(add_rms_quant_kernel<S, BF16, BITS, 0, most_blocks(S::kThreads)>, done, need, S::kThreads, 0, stream, x,
                 residual, M, (int)K, gain, h, codes, scales);
  return start(add_rms_quant_kernel<S, BF16, BITS, flow.stages, flow.blocks>, done, grid, S::kThreads,
               flow.stages * row_bytes, stream, x, residual, M, (int)K, gain, h, codes, scales);
}

// B blocks of an SM as one (1: as they are)
template <typename S, int B, bool BF16, bool GT16>
cudaError_t launch_grad_of(const void* h, int64_t M, int64_t K, const float* gain, const void* g_t, const void* g_h,
                           void* g_x, float* g_gain, float* sums, cudaStream_t stream) {
  constexpr int row_bytes = S::E * S::kThreads * (2 * (BF16 ? 16 : 32) + (GT16 ? 16 : 32));
  constexpr Flow flow = flow_for(S::kThreads, row_bytes);
  using W = Wide<S, B>;
  static std::atomic<bool> done[sm100_host::kMaxDevices];
  const int64_t grid = grad_grid(M, flow.blocks / B);
  cudaError_t e = start(add_rms_grad_kernel<W, BF16, GT16, flow.stages>, done, grid, W::kThreads,
                        flow.stages * B * row_bytes, stream, h, M, (int)K, gain, g_t, g_h, g_x, g_gain ? sums : nullptr);
  if (e != cudaSuccess || !g_gain) return e;
  return sm100_host::launch_pdl(gain_sum_kernel, (unsigned)((K + 31) / 32), kSumWarps * 32, 0, stream, 1, (const float*)sums,
                                (int)grid, (int)K, g_gain);
}

// Wide blocks where an SM has at least three rounds of their rows: 8192 bf16
// rows of 4096 take 47.7 us so and 51.8 as separate blocks, 1001 float rows of
// 2560 (3.4 rounds) 15.4 and 16.4; but 809 bf16 rows of 5552 (2.7 rounds) 13.5
// and 11.9, and 64 of 4096 6.8 and 4.9.
constexpr int kWideRounds = 3;
template <typename S, bool BF16, bool GT16>
cudaError_t launch_grad(const void* h, int64_t M, int64_t K, const float* gain, const void* g_t, const void* g_h,
                        void* g_x, float* g_gain, float* sums, cudaStream_t stream) {
  constexpr int B = flow_for(S::kThreads, S::E * S::kThreads * (2 * (BF16 ? 16 : 32) + (GT16 ? 16 : 32))).blocks;
  if constexpr (B > 1) {
    if (M >= (int64_t)kWideRounds * sm100_host::sm_count() * Wide<S, B>::R)
      return launch_grad_of<S, B, BF16, GT16>(h, M, K, gain, g_t, g_h, g_x, g_gain, sums, stream);
  }
  return launch_grad_of<S, 1, BF16, GT16>(h, M, K, gain, g_t, g_h, g_x, g_gain, sums, stream);
}

}  // namespace

cudaError_t launch_add_rms_quant(const void* x, const void* residual, bool bf16, int64_t M, int64_t K,
                                 const float* gain, int bits, void* h, int8_t* codes, float* scales,
                                 cudaStream_t stream) {
  return by_length(K, [&](auto rows) {
    using S = decltype(rows);
    auto go = bf16 ? (bits == 8 ? launch_quant<S, true, 8> : launch_quant<S, true, 4>)
                   : (bits == 8 ? launch_quant<S, false, 8> : launch_quant<S, false, 4>);
    return go(x, residual, M, K, gain, h, codes, scales, stream);
  });
}

size_t add_rms_backward_workspace(int64_t M, int64_t K) {
  size_t bytes = 0;
  by_length(K, [&](auto rows) {
    bytes = (size_t)grad_grid(M, most_blocks(decltype(rows)::kThreads)) * (size_t)K * 4;
    return cudaSuccess;
  });
  return bytes;
}

cudaError_t launch_add_rms_quant_backward(const void* h, bool bf16, int64_t M, int64_t K, const float* gain,
                                          const void* g_t, bool gt_bf16, const void* g_h, void* g_x, float* g_gain,
                                          void* workspace, cudaStream_t stream) {
  return by_length(K, [&](auto rows) {
    using S = decltype(rows);
    auto go = bf16 ? (gt_bf16 ? launch_grad<S, true, true> : launch_grad<S, true, false>)
                   : (gt_bf16 ? launch_grad<S, false, true> : launch_grad<S, false, false>);
    return go(h, M, K, gain, g_t, g_h, g_x, g_gain, reinterpret_cast<float*>(workspace), stream);
  });
}

}  // namespace hbl
