// Causal attention over the paged 8-bit cache.  A code q of block c and head h
// stands for (2 q - L) u, u = fl(gamma[c][h] / L), L = 2^bits - 1; with the
// running maximum m and sum l of a softmax,
//
//   s_j = scale u_k(j) sum_d q_d (2 k_jd - L),   o = sum_j exp(s_j - m) u_v(j) (2 v_jd - L) / l
//
// One warp per (row, query head), its lanes over the head dimension.
#include <cstdint>

#include "common.cuh"
#include "serving.cuh"
#include "sm100.cuh"

namespace hbl {
namespace {

constexpr int kThreads = 128;

__global__ void __launch_bounds__(kThreads) kv_attention_kernel(const KvAttentionArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = w / a.Hq;
  const int head = (int)(w % a.Hq), kvh = head / (a.Hq / a.Hkv);
  if (t >= a.T || t < a.row_start[0] || t >= a.row_start[a.B]) return;
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.row_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int b = lo;
  const int64_t limit = a.width * a.block;
  const int64_t pos = (int64_t)a.total[b] - a.row_start[b + 1] + t;
  const int64_t keys = pos + 1 < limit ? pos + 1 : limit;
  const int V = a.D / 32;
  const float L = (float)((1 << a.bits) - 1);
  const float scale = a.scale ? *a.scale : rsqrtf((float)a.D);
  float q[8], o[8], m = -INFINITY, l = 0.0f;
  for (int i = 0; i < V; ++i) {
    const int64_t at = t * a.q_stride + (int64_t)head * a.D + lane * V + i;
    q[i] = a.q_bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.q)[at] << 16)
                    : reinterpret_cast<const float*>(a.q)[at];
    o[i] = 0.0f;
  }
  for (int64_t j = 0; j < keys; ++j) {
    const int id = a.table[(int64_t)b * a.width + j / a.block];
    if (id < 0 || id >= a.num_blocks) continue;
    const int64_t tile = (int64_t)id * a.Hkv + kvh, at = (tile * a.block + j % a.block) * a.D + lane * V;
    float s = 0.0f;
    for (int i = 0; i < V; ++i) s += q[i] * (2.0f * (float)a.k_codes[at + i] - L);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= scale * __fdiv_rn(a.k_scales[tile], L);
    const float u = __fdiv_rn(a.v_scales[tile], L);
    const float m1 = fmaxf(m, s), f = __expf(m - m1), p = __expf(s - m1);
    l = l * f + p;
    for (int i = 0; i < V; ++i) o[i] = o[i] * f + p * u * (2.0f * (float)a.v_codes[at + i] - L);
    m = m1;
  }
  for (int i = 0; i < V; ++i) {
    const float v = l > 0.0f ? o[i] / l : (l == 0.0f ? 0.0f : l);
    const int64_t at = (t * a.Hq + head) * a.D + lane * V + i;
    if (a.o_bf16) {
      uint16_t b16;
      asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b16) : "f"(v));
      reinterpret_cast<uint16_t*>(a.o)[at] = b16;
    } else {
      reinterpret_cast<float*>(a.o)[at] = v;
    }
  }
}

}  // namespace

size_t kv_attention_workspace(int64_t T, int Hq, int Hkv, int D, int B) { return 256; }

cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t stream) {
  const int64_t warps = a.T * a.Hq;
  kv_attention_kernel<<<(unsigned)((warps + 3) / 4), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace hbl
