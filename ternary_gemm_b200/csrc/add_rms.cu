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
// kernel in fixed order.
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

template <typename S, bool BF16, int BITS>
__global__ void __launch_bounds__(S::kThreads)
add_rms_quant_kernel(const void* x, const void* residual, int64_t M, int K, const float* __restrict__ gain, void* h,
                     int8_t* codes, float* scales) {
  constexpr int T = S::T, E = S::E, WPR = S::kWarpsPerRow;
  __shared__ double red_d[2][S::R * WPR];
  __shared__ float red_f[S::R * WPR];
  const int rl = threadIdx.x / T, t = threadIdx.x % T;
  const int64_t row = (int64_t)blockIdx.x * S::R + rl;
  const bool active = row < M;
  const int64_t base = (active ? row : 0) * K;
  const int vectors = K / 8;

  float v[E][8];
  double ss = 0.0;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int i = j * T + t;
    if (active && i < vectors) {
      load8<BF16>(x, base + i * 8, v[j]);
      if (residual) {
        float r[8];
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
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int i = j * T + t;
    if (h && active && i < vectors) store8<BF16>(h, base + i * 8, v[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fma((double)v[j][e], (double)v[j][e], ss);
  }
  ss = RowReduce<T, WPR>::run(ss, AddD(), red_d[0], rl, t);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn((float)(ss / (double)K), 1e-5f)));
  float top = 0.0f;
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int i = j * T + t;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] = __fmul_rn(v[j][e], rstd);
    if (gain && i < vectors) {
      float w[8];
      rowkit::load8<false>(gain, i * 8, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = __fmul_rn(v[j][e], w[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (BITS == 8)
        top = fmaxf(top, fabsf(v[j][e]));
      else
        sum += q::abs_f64(v[j][e]);
    }
  }
  q::RowParams p;
  if constexpr (BITS == 8)
    p = q::params_int8(RowReduce<T, WPR>::run(top, MaxF(), red_f, rl, t));
  else
    p = q::params_int4(RowReduce<T, WPR>::run(sum, AddD(), red_d[1], rl, t), K);
  if (!active) return;
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

// ---------------------------------------------------------------- gradient

// CTAs per SM of the gradient: its registers hold h, g_t and the gain's sums
template <typename S>
constexpr int grad_blocks() {
  return S::E > 4 ? 1 : (S::kThreads <= 128 ? 3 : (S::kThreads <= 256 ? 2 : 1));
}

template <typename S, bool BF16, bool GT16>
__global__ void __launch_bounds__(S::kThreads, grad_blocks<S>())
add_rms_grad_kernel(const void* __restrict__ h, int64_t M, int K, const float* __restrict__ gain,
                    const void* __restrict__ g_t, const void* g_h, void* g_x, float* __restrict__ sums) {
  constexpr int T = S::T, E = S::E, WPR = S::kWarpsPerRow;
  constexpr bool kHold = E <= 4;  // longer rows are read again (from L2) for their outputs
  __shared__ float2 red[2][S::R * WPR];
  const int rl = threadIdx.x / T, t = threadIdx.x % T;
  const int vectors = K / 8;
  const float inv_k = __fdiv_rn(1.0f, (float)K);
  float acc[E][8];
#pragma unroll
  for (int j = 0; j < E; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[j][e] = 0.0f;

  int parity = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * S::R; row0 < M; row0 += (int64_t)gridDim.x * S::R, parity ^= 1) {
    const bool active = row0 + rl < M;
    const int64_t base = (active ? row0 + rl : 0) * K;
    float a[kHold ? E : 1][8], g[kHold ? E : 1][8];
    float ss = 0.0f, dot = 0.0f;
    auto read = [&](int j, float (&hv)[8], float (&gv)[8]) {
      const int i = j * T + t;
      if (active && i < vectors) {
        load8<BF16>(h, base + i * 8, hv);
        load8<GT16>(g_t, base + i * 8, gv);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) hv[e] = gv[e] = 0.0f;
      }
    };
    auto gains = [&](int j, float (&w)[8]) {
      const int i = j * T + t;
      if (gain && i < vectors) {
        rowkit::load8<false>(gain, i * 8, w);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
      }
    };
    if constexpr (kHold) {
#pragma unroll
      for (int j = 0; j < E; ++j) read(j, a[j], g[j]);
    }
#pragma unroll
    for (int j = 0; j < E; ++j) {
      float w[8];
      gains(j, w);
      if constexpr (!kHold) read(j, a[0], g[0]);
      float s = 0.0f, d = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float hv = a[kHold ? j : 0][e];
        s = fmaf(hv, hv, s);
        d = fmaf(g[kHold ? j : 0][e] * w[e], hv, d);
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
      __syncthreads();
      ss = dot = 0.0f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) {
        const float2 r = red[parity][rl * WPR + w];
        ss += r.x;
        dot += r.y;
      }
    }
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(fmaf(ss, inv_k, 1e-5f)));
    const float c = dot * rstd * inv_k;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int i = j * T + t;
      float w[8], out[8];
      gains(j, w);
      if constexpr (!kHold) read(j, a[0], g[0]);
      const bool there = active && i < vectors;
      if (g_h && there) {
        load8<BF16>(g_h, base + i * 8, out);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = a[kHold ? j : 0][e] * rstd, gv = g[kHold ? j : 0][e];
        acc[j][e] = fmaf(gv, n, acc[j][e]);
        out[e] = fmaf(rstd, fmaf(-n, c, gv * w[e]), out[e]);
      }
      if (there) store8<BF16>(g_x, base + i * 8, out);
    }
  }
  if (!sums) return;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    const int i = j * T + t;
    if (i < vectors) store8<false>(sums, ((int64_t)blockIdx.x * S::R + rl) * K + i * 8, acc[j]);
  }
}

// g_gain[k] = sum of the partial sums [count][K]: 32 columns per CTA, eight
// warps on every eighth row
__global__ void __launch_bounds__(256) gain_sum_kernel(const float* __restrict__ sums, int count, int K, float* g_gain) {
  __shared__ float part[8][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.0f;
  if (k < K) {
#pragma unroll 8
    for (int i = warp; i < count; i += 8) s += sums[(int64_t)i * K + k];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && k < K) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += part[w][lane];
    g_gain[k] = s;
  }
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

template <typename S>
int64_t grad_grid(int64_t M) {
  const int64_t need = (M + S::R - 1) / S::R, cap = (int64_t)sm100_host::sm_count() * grad_blocks<S>();
  return need < cap ? need : cap;
}

}  // namespace

cudaError_t launch_add_rms_quant(const void* x, const void* residual, bool bf16, int64_t M, int64_t K,
                                 const float* gain, int bits, void* h, int8_t* codes, float* scales,
                                 cudaStream_t stream) {
  return by_length(K, [&](auto rows) {
    using S = decltype(rows);
    const unsigned grid = (unsigned)((M + S::R - 1) / S::R);
    auto kernel = bf16 ? (bits == 8 ? add_rms_quant_kernel<S, true, 8> : add_rms_quant_kernel<S, true, 4>)
                       : (bits == 8 ? add_rms_quant_kernel<S, false, 8> : add_rms_quant_kernel<S, false, 4>);
    kernel<<<grid, S::kThreads, 0, stream>>>(x, residual, M, (int)K, gain, h, codes, scales);
    return cudaGetLastError();
  });
}

size_t add_rms_backward_workspace(int64_t M, int64_t K) {
  size_t bytes = 0;
  by_length(K, [&](auto rows) {
    using S = decltype(rows);
    bytes = (size_t)grad_grid<S>(M) * S::R * (size_t)K * 4;
    return cudaSuccess;
  });
  return bytes;
}

cudaError_t launch_add_rms_quant_backward(const void* h, bool bf16, int64_t M, int64_t K, const float* gain,
                                          const void* g_t, bool gt_bf16, const void* g_h, void* g_x, float* g_gain,
                                          void* workspace, cudaStream_t stream) {
  return by_length(K, [&](auto rows) {
    using S = decltype(rows);
    const int64_t grid = grad_grid<S>(M);
    float* sums = g_gain ? reinterpret_cast<float*>(workspace) : nullptr;
    auto kernel = bf16 ? (gt_bf16 ? add_rms_grad_kernel<S, true, true> : add_rms_grad_kernel<S, true, false>)
                       : (gt_bf16 ? add_rms_grad_kernel<S, false, true> : add_rms_grad_kernel<S, false, false>);
    kernel<<<(unsigned)grid, S::kThreads, 0, stream>>>(h, M, (int)K, gain, g_t, g_h, g_x, sums);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !g_gain) return e;
    return sm100_host::launch_pdl(gain_sum_kernel, (unsigned)((K + 31) / 32), 256, 0, stream, 1, (const float*)sums,
                                  (int)(grid * S::R), (int)K, g_gain);
  });
}

}  // namespace hbl
