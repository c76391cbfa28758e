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
#include <cstdint>

#include "common.cuh"
#include "serving.cuh"
#include "sm100.cuh"

namespace hbl {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxBlock = 128;

__device__ __forceinline__ float value_at(const void* x, bool bf16, int64_t i) {
  return bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(x)[i] << 16)
              : reinterpret_cast<const float*>(x)[i];
}

__device__ __forceinline__ uint8_t code_of(float x, float r, float half, int L) {
  const int c = __float2int_rn(__fadd_rn(__fmul_rn(x, r), half));
  return (uint8_t)min(max(c, 0), L);
}

__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a) {
  __shared__ uint32_t top;
  __shared__ int run;
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, tid = threadIdx.x;
  const bool is_v = blockIdx.z != 0;
  const int64_t nslots = a.num_blocks * a.block;
  const int s0 = a.slots[t];
  if (s0 < 0 || s0 >= nslots) return;
  const int place = s0 % a.block;
  if (place != 0 && t > 0 && a.slots[t - 1] == s0 - 1) return;  // the run's first row does it
  if (tid == 0) {
    int n = 1;
    while (place + n < a.block && t + n < a.T && a.slots[t + n] == s0 + n) ++n;
    run = n;
    top = 0;
  }
  __syncthreads();
  const int n = run;
  const void* x = is_v ? a.v : a.k;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const int64_t tile = (int64_t)(s0 / a.block) * a.H + h;
  uint8_t* codes = (is_v ? a.v_codes : a.k_codes) + tile * a.block * a.D;
  float* scale = (is_v ? a.v_scales : a.k_scales) + tile;
  float m = 0.0f;
  for (int i = tid; i < n * a.D; i += kThreads)
    m = fmaxf(m, fabsf(value_at(x, a.bf16, (t + i / a.D) * stride + (int64_t)h * a.D + i % a.D)));
  atomicMax(&top, __float_as_uint(m));
  __syncthreads();
  const int L = (1 << a.bits) - 1;
  const float old = place ? *scale : 0.0f;
  const float gamma = fmaxf(old, __uint_as_float(top));
  const float r = __fdiv_rn((float)L, __fmul_rn(2.0f, __fadd_rn(gamma, 1e-5f))), half = 0.5f * (float)L;
  if (gamma > old && place) {
    const float u = __fdiv_rn(old, (float)L);
    for (int i = tid; i < place * a.D; i += kThreads)
      codes[i] = code_of(__fmul_rn((float)(2 * (int)codes[i] - L), u), r, half, L);
  }
  for (int i = tid; i < n * a.D; i += kThreads)
    codes[place * a.D + i] = code_of(value_at(x, a.bf16, (t + i / a.D) * stride + (int64_t)h * a.D + i % a.D), r, half, L);
  __syncthreads();
  if (tid == 0) *scale = gamma;
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream) {
  kv_append_kernel<<<dim3((unsigned)a.T, (unsigned)a.H, 2), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace hbl
