// The join between two sublayers: residual addition, RMSNorm with a gain, and
// the per-token quantizer of the next BitLinear, and its straight-through
// gradient.
//
//   h = round(x + residual),  rstd = 1 / sqrt(mean h^2 + eps),  t = fl(fl(h rstd) gain)
//   codes, scale = the H-BitLinear quantizer of t (quant.cuh)
//   g_x = g_h + rstd (g_t gain - n mean(g_t gain n)),  g_gain = sum_rows g_t n,  n = h rstd
//
// The mean of h^2 is a double sum rounded once, so that the codes follow from
// h bit for bit whatever the order of the sum.
#include <cstdint>

#include "common.cuh"
#include "quant.cuh"
#include "serving.cuh"
#include "sm100.cuh"

namespace hbl {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float ld(const void* p, bool bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16)
              : reinterpret_cast<const float*>(p)[i];
}

__device__ __forceinline__ float round_bf16(float v) {
  uint32_t u;
  asm("{\n\t.reg .b16 h;\n\tcvt.rn.bf16.f32 h, %1;\n\tmov.b32 %0, {0, h};\n\t}" : "=r"(u) : "f"(v));
  return __uint_as_float(u);
}

__device__ __forceinline__ void st(void* p, bool bf16, int64_t i, float v) {
  if (bf16)
    reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(__float_as_uint(round_bf16(v)) >> 16);
  else
    reinterpret_cast<float*>(p)[i] = v;
}

template <typename V, typename Op>
__device__ V block_all(V v, Op op, V* red) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < kThreads / 32; ++w) v = op(v, red[w]);
  return v;
}

struct Add {
  template <typename V>
  __device__ V operator()(V a, V b) const { return a + b; }
};
struct Max {
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

__global__ void __launch_bounds__(kThreads)
add_rms_quant_kernel(const void* x, const void* residual, bool bf16, int K, const float* gain, int bits, void* h,
                     int8_t* codes, float* scales) {
  extern __shared__ float row[];
  __shared__ double red_d[kThreads / 32];
  __shared__ float red_f[kThreads / 32];
  const int64_t base = (int64_t)blockIdx.x * K;
  double ss = 0.0;
  for (int i = threadIdx.x; i < K; i += kThreads) {
    float v = ld(x, bf16, base + i);
    if (residual) v = __fadd_rn(v, ld(residual, bf16, base + i));
    if (bf16) v = round_bf16(v);
    if (h) st(h, bf16, base + i, v);
    row[i] = v;
    ss += (double)v * (double)v;
  }
  ss = block_all(ss, Add(), red_d);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn((float)(ss / (double)K), 1e-5f)));
  float m = 0.0f;
  double sum = 0.0;
  for (int i = threadIdx.x; i < K; i += kThreads) {
    float t = __fmul_rn(row[i], rstd);
    if (gain) t = __fmul_rn(t, gain[i]);
    row[i] = t;
    m = fmaxf(m, fabsf(t));
    sum += fabs((double)t);
  }
  q::RowParams p;
  if (bits == 8)
    p = q::params_int8(block_all(m, Max(), red_f));
  else
    p = q::params_int4(block_all(sum, Add(), red_d), K);
  for (int i = threadIdx.x; i < K; i += kThreads) {
    const int c = q::rint_code(row[i], p.r);
    codes[base + i] = (int8_t)(bits == 8 ? max(-128, min(127, c)) : q::clip_int4(c));
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = p.scale();
}

__global__ void __launch_bounds__(kThreads)
add_rms_backward_kernel(const void* h, bool bf16, int K, const float* gain, const void* g_t, bool gt_bf16,
                        const void* g_h, void* g_x, float* rstds) {
  __shared__ float red_f[kThreads / 32];
  const int64_t base = (int64_t)blockIdx.x * K;
  float ss = 0.0f, dot = 0.0f;
  for (int i = threadIdx.x; i < K; i += kThreads) {
    const float v = ld(h, bf16, base + i), g = ld(g_t, gt_bf16, base + i) * (gain ? gain[i] : 1.0f);
    ss += v * v;
    dot += g * v;
  }
  ss = block_all(ss, Add(), red_f);
  dot = block_all(dot, Add(), red_f);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(ss / (float)K + 1e-5f));
  const float c = dot * rstd / (float)K;
  for (int i = threadIdx.x; i < K; i += kThreads) {
    const float v = ld(h, bf16, base + i), g = ld(g_t, gt_bf16, base + i) * (gain ? gain[i] : 1.0f);
    st(g_x, bf16, base + i, (g_h ? ld(g_h, bf16, base + i) : 0.0f) + rstd * (g - v * rstd * c));
  }
  if (threadIdx.x == 0) rstds[blockIdx.x] = rstd;
}

__global__ void __launch_bounds__(kThreads)
gain_grad_kernel(const void* h, bool bf16, int64_t M, int K, const void* g_t, bool gt_bf16, const float* rstds,
                 float* g_gain) {
  const int k = blockIdx.x * kThreads + threadIdx.x;
  if (k >= K) return;
  double s = 0.0;
  for (int64_t m = 0; m < M; ++m) s += (double)(ld(g_t, gt_bf16, m * K + k) * (ld(h, bf16, m * K + k) * rstds[m]));
  g_gain[k] = (float)s;
}

}  // namespace

cudaError_t launch_add_rms_quant(const void* x, const void* residual, bool bf16, int64_t M, int64_t K,
                                 const float* gain, int bits, void* h, int8_t* codes, float* scales,
                                 cudaStream_t stream) {
  static std::atomic<bool> done[sm100_host::kMaxDevices];
  cudaError_t e = sm100_host::ensure_smem(add_rms_quant_kernel, 32768 * 4, done);
  if (e != cudaSuccess) return e;
  add_rms_quant_kernel<<<(unsigned)M, kThreads, (size_t)K * 4, stream>>>(x, residual, bf16, (int)K, gain, bits, h,
                                                                         codes, scales);
  return cudaGetLastError();
}

size_t add_rms_backward_workspace(int64_t M, int64_t K) { return (size_t)M * 4; }

cudaError_t launch_add_rms_quant_backward(const void* h, bool bf16, int64_t M, int64_t K, const float* gain,
                                          const void* g_t, bool gt_bf16, const void* g_h, void* g_x, float* g_gain,
                                          void* workspace, cudaStream_t stream) {
  float* rstds = reinterpret_cast<float*>(workspace);
  add_rms_backward_kernel<<<(unsigned)M, kThreads, 0, stream>>>(h, bf16, (int)K, gain, g_t, gt_bf16, g_h, g_x, rstds);
  if (g_gain)
    gain_grad_kernel<<<(unsigned)((K + kThreads - 1) / kThreads), kThreads, 0, stream>>>(h, bf16, M, (int)K, g_t,
                                                                                         gt_bf16, rstds, g_gain);
  return cudaGetLastError();
}

}  // namespace hbl
