// Internal declarations of the serving and norm operators: the paged 8-bit
// cache (plan, append, attention) and the residual + RMSNorm + quantizer row
// kernels.  Nothing here is part of the public ABI (include/hbl.h is).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace hbl {

constexpr int kMaxRequests = 4096;  // the plan and the attention scan them in shared memory

// A weight of the attention is exp(score) u, u = gamma / L of its block of
// values, and the softmax sum holds weights over u.  A block with u below the
// first of these (2 to the second) counts as all zeros.  Its weights enter no
// product: where the running maximum (or reference) is taken they stand as if u
// were that, below every block with values, and in the sum they are held without
// u.  A term of the sum is then at most 2^(15 + 100); the sum is kept times
// 2^-20, so that fewer than 2^31 tokens stay below 2^126 in float, and the
// largest float values (u = 2^120) leave terms of 2^(15 - 120 - 20).  (Codes of
// so small a gamma hold nothing: with the rule's 1e-5 beside it x r vanishes next
// to L / 2 from gamma = 2^-42 down, and all codes are one.)
constexpr float kLeastValueScale = 0x1p-100f, kLeastValueLog = -100.0f;
constexpr float kSumScale = 0x1p-20f;

// 2^d for d <= 0 in two factors, the second 1 down to 2^-100.  A sum that zeros
// have made large takes both, and keeps what 2^d alone would lose below float's
// smallest number when values of large u follow them; of outputs the first
// leaves nothing that counts.
struct Shrink {
  float near, far;
};

struct KvPlanArgs {
  const int32_t *cached, *added;
  int B, block;
  const int32_t* free_blocks;
  int64_t num_free;
  const int32_t* taken;
  int32_t* table;
  int64_t width, T;
  int32_t *total, *row_start, *slots, *positions, *taken_out;
};
cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream);

struct KvAppendArgs {
  const void *k, *v;
  bool bf16;
  int64_t T;
  int H, D;
  int64_t k_stride, v_stride;  // elements
  const int32_t* slots;
  int bits;
  int64_t num_blocks;
  int block;
  uint8_t* k_codes;
  float* k_scales;
  uint8_t* v_codes;
  float* v_scales;
};
cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t stream);

struct KvAttentionArgs {
  const void* q;
  bool q_bf16;
  int64_t T, q_stride;  // q_stride in elements
  int Hq, Hkv, D;
  const int32_t *row_start, *total;
  int B;
  const int32_t* table;
  int64_t width, num_blocks;
  int block, bits;
  const uint8_t* k_codes;
  const float* k_scales;
  const uint8_t* v_codes;
  const float* v_scales;
  const float* scale;  // device scalar, or null for 1 / sqrt(D)
  void* o;
  bool o_bf16;
  void* workspace;
};
size_t kv_attention_workspace(int64_t T, int Hq, int Hkv, int D, int B);
cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t stream);
// The same with 256-row tiles on tcgen05 (kv_attention_prompt.cu), for bf16
// queries of head dimension 64 or 128 where enough full row tiles' worth of
// CTAs are at work at once.
bool kv_attention_prompt_supports(const KvAttentionArgs& a);
size_t kv_attention_prompt_workspace(int D);
cudaError_t launch_kv_attention_prompt(const KvAttentionArgs& a, cudaStream_t stream);

cudaError_t launch_add_rms_quant(const void* x, const void* residual, bool bf16, int64_t M, int64_t K,
                                 const float* gain, int bits, void* h, int8_t* codes, float* scales,
                                 cudaStream_t stream);
size_t add_rms_backward_workspace(int64_t M, int64_t K);
cudaError_t launch_add_rms_quant_backward(const void* h, bool bf16, int64_t M, int64_t K, const float* gain,
                                          const void* g_t, bool gt_bf16, const void* g_h, void* g_x, float* g_gain,
                                          void* workspace, cudaStream_t stream);

}  // namespace hbl
