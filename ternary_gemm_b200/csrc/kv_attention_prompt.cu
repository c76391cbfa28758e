// Causal attention over the paged 8-bit cache for many rows per request
// (prompts and chunks of them): bf16 queries, head dimension 64 or 128.
//
// The arithmetic is that of kv_attention.cu: centred codes k' = k - z and
// v' = v - z enter the products exactly as fp16,
//
//   s_j = scale u_k(j) (2 sum_d q_d k'_jd + sum_d q_d)
//   w_j = exp(s_j) u_v(j),   o = sum_j w_j (2 v'_j + 1) / sum_j w_j / u_v(j)
//
// and the weights are held under a reference that is a row's maximum when it
// first sees a token (its largest weight there is 2^7) and moves only when the
// weights of half a tile add up to more than 2^15: no weight can pass fp16's
// range, no maximum is taken of a tile, and the accumulator in tensor memory is
// seldom rescaled.  fp16 keeps 11 bits of all weights down to 2^-21 of the
// reference's at the least; the 1 beside 2 v' and the sum below take them
// unrounded.  (A reference that followed after four powers of
// two, which some warp of a CTA met in every other tile: 571 us at three
// requests of up to 2048 rows over 8192 tokens; after eight, with a maximum of
// every tile: 406; without: 379, and 367 with the start and end of a CTA
// shortened.)
//
// Rows are many, so this is a matter of the tensor cores: a CTA takes 256 rows
// of one cached head (two tiles of 128, query heads of the group times the
// request's rows) over tiles of 128 tokens.
//   warps 0-3, 4-7  softmax of the first and the second row tile, a row per
//                   thread: scores from tensor memory, weights back into it
//   warps 8-11      codes from the pages (16-byte loads, a tile ahead in
//                   registers) to fp16 in the 128-byte-swizzled layout, K and V
//                   alike, two stages each
//   warp 12         issues tcgen05.mma kind::f16: S = Q K^T from shared memory,
//                   O += W V with W from tensor memory (it lies where S was),
//                   the two row tiles in turn, so that one tile's softmax runs
//                   under the other's products
// Measured there: 369 us, 860 TFLOP/s of the causal products, 52% of the
// rate of a long library product (heads of 64: 319 us, 500 TFLOP/s, 30%); 4000 clocks for 256 rows over 128 tokens, of
// which the products take 2050 and a row tile's softmax 2700 (the exponentials
// of both 2050, at their unit's rate).  What bounds it is the chain of a row
// tile: its next scores go where its weights lie, so they are begun only when
// the products with those have been issued.
// Where there are too few items for the SMs, several CTAs share the tokens of
// one and a second kernel joins their parts: one request of 1024 rows over
// 16384 tokens 95 us instead of 347.
// Every mbarrier wait is bounded; a CTA that gives up sets the device error
// word, waits for its products and frees its tensor memory.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "serving.cuh"
#include "sm100.cuh"

namespace hbl {
namespace {

using namespace sm100;

constexpr int kRowsM = 128;               // rows of one tile
constexpr int kRows = 2 * kRowsM;         // rows of a CTA
constexpr int kKeys = 128;                // tokens of a tile
constexpr int kThreads = 13 * 32;
constexpr int kMeta = 4;                  // slots of page scales
constexpr int kMostSplits = 32;           // CTAs that share an item's tokens at most
constexpr int kLeastTiles = 4;            // and the tiles that each of them has at least
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kS = 0, kO = 256;      // tensor memory columns: S0 and S1 (W in their place), O0 and O1
constexpr float kTop = 7.0f;              // log2 of the weight at the reference maximum
constexpr float kMost = 32768.0f;         // what the weights of half a tile may add up to before the reference follows
constexpr float kLog2e = 1.4426950408889634f;

// kind::f16, D f32, A and B fp16, M = 128: scores (both K-major, N = 128 tokens), outputs (B MN-major, N = D)
constexpr uint32_t kIdescS = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
template <int D>
constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);

template <int D>
struct Shape {
  static constexpr int kHalves = D / 64;             // blocks of 64 values: 128 rows of 128 bytes
  static constexpr int kBlock = 128 * 128;
  static constexpr int kTile = kHalves * kBlock;     // a Q, K or V tile in fp16
  static constexpr size_t kSmem = 1024 + 6 * (size_t)kTile + kMeta * 8 * 16 + 256;
  static constexpr int kVectors = D / 16;            // 16-byte code vectors per converting thread and tile
};

// Descriptors differ in their low words alone (the address, in 16-byte units).
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t a_high, uint32_t b, uint32_t b_high, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 A, B;\n\t"
      "mov.b64 A, {%1, %2};\n\tmov.b64 B, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], A, B, %5, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(a_high), "r"(b), "r"(b_high), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_high, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 B;\n\t"
      "mov.b64 B, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], B, %4, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(b_high), "r"(idesc), "r"(accumulate));
}

// true in one lane of the warp, the same one every time
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// A bounded wait of the whole warp, with one answer for all its lanes (the
// limit may run out for some while others see the phase end).
__device__ __forceinline__ bool await(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err) {
  const bool there = wait_bounded_warp(bar, parity, abort_flag, err);
  return __all_sync(0xffffffffu, there) != 0;
}

// sixteen columns of this thread's lane; the registers hold them after landed()
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void landed(uint32_t (&r)[32], uint32_t (&q)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                      "+r"(r[i + 6]), "+r"(r[i + 7]));
    asm volatile("" : "+r"(q[i]), "+r"(q[i + 1]), "+r"(q[i + 2]), "+r"(q[i + 3]), "+r"(q[i + 4]), "+r"(q[i + 5]),
                      "+r"(q[i + 6]), "+r"(q[i + 7]));
  }
}
__device__ __forceinline__ void landed(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// (a0, a1) * m + c
__device__ __forceinline__ void fma2(float& a0, float& a1, float m, float c) {
  asm("{\n\t.reg .b64 A, M, C;\n\t"
      "mov.b64 A, {%0, %1};\n\tmov.b64 M, {%2, %2};\n\tmov.b64 C, {%3, %3};\n\t"
      "fma.rn.f32x2 A, A, M, C;\n\tmov.b64 {%0, %1}, A;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "f"(m), "f"(c));
}
__device__ __forceinline__ void add2(float& s0, float& s1, float a0, float a1) {
  asm("{\n\t.reg .b64 A, S;\n\t"
      "mov.b64 A, {%2, %3};\n\tmov.b64 S, {%0, %1};\n\t"
      "add.rn.f32x2 S, S, A;\n\tmov.b64 {%0, %1}, S;\n\t}"
      : "+f"(s0), "+f"(s1)
      : "f"(a0), "f"(a1));
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// place of 16 bytes (eight fp16 values) of row t in a block of 64 values
__device__ __forceinline__ uint32_t swizzled(int t, int piece) { return (uint32_t)(t * 128 + ((piece ^ (t & 7)) << 4)); }

__device__ __forceinline__ Shrink shrink(float d) { return {ex2(fmaxf(d, -100.0f)), ex2(fminf(d + 100.0f, 0.0f))}; }

// What a row's scores of sixteen tokens of one page are to be multiplied by and
// added to, the inverse of the values' scale as it is in the weights, and what
// the weights count for the reference: 1, or less for a page whose values are
// all zero, the weights of which stand as they go into the sum (0: no page).
struct Page {
  float f2, c, inv, part;
  __device__ __forceinline__ bool some() const { return part == 1.0f; }
};
__device__ __forceinline__ Page page_at(uint32_t pages, int grp, float q_scale, float q_sum) {
  const uint4 p = lds128(pages + grp * 16);
  const float f = q_scale * __uint_as_float(p.x);
  return {2.0f * f, fmaf(q_sum, f, __uint_as_float(p.y)), __uint_as_float(p.z), __uint_as_float(p.w)};
}

// The CTA's item: which request, its rows, and where they stand.
struct Item {
  int b, row0, n;        // request, its first row of the batch, its rows
  int first;             // first of the CTA's rows, in (row, head of the group) order
  int keys, pos0;        // tokens that the table can hold; position of the request's first row
};

// Rows r, r + step, ... in (row of the batch, head of the group) order, with
// the divisions by the group's size taken once.
struct Walk {
  int tok, head, g, tok_step, head_step;
  __device__ __forceinline__ Walk(int r, int step, int group)
      : tok(r / group), head(r % group), g(group), tok_step(step / group), head_step(step % group) {}
  __device__ __forceinline__ void next() {
    tok += tok_step;
    head += head_step;
    if (head >= g) head -= g, ++tok;
  }
};

// What the CTAs leave in the workspace where several share an item: for each
// row (reference, sum of the weights over it) and its outputs unscaled, and for
// each item what the joining kernel has to know (parts 0: nothing to join).
struct Joined {
  int first, rows, row0, h, parts;
};
struct Parts {
  float* o;         // [CTAs][256][D]
  float2* ml;       // [CTAs][256]
  Joined* item;     // [items]
};
__host__ __device__ inline Parts parts_of(void* workspace, int64_t ctas, int D) {
  Parts p;
  p.o = reinterpret_cast<float*>(workspace);
  p.ml = reinterpret_cast<float2*>(p.o + (size_t)ctas * kRows * D);
  p.item = reinterpret_cast<Joined*>(p.ml + (size_t)ctas * kRows);
  return p;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
kv_attention_prompt_kernel(const KvAttentionArgs a, const int splits, int* err) {
  using S = Shape<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t q_at = smem_u32(base), k_at = q_at + 2 * S::kTile, v_at = k_at + 2 * S::kTile;
  const uint32_t meta_at = v_at + 2 * S::kTile;
  float4* meta = reinterpret_cast<float4*>(base + 6 * S::kTile);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + 6 * S::kTile + kMeta * 8 * 16);
  uint64_t *kfull = bars, *kempty = bars + 2, *vfull = bars + 4, *vempty = bars + 6, *sfull = bars + 8,
           *pready = bars + 10, *odone = bars + 14, *mready = bars + 16, *qready = bars + 20, *drain = bars + 21,
           *ofinal = bars + 22;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 24);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ Item item;
  __shared__ int64_t warp_sums[kThreads / 32];

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int g = a.Hq / a.Hkv;
  const int split = blockIdx.x % splits, h = blockIdx.x / splits % a.Hkv;
  const int64_t rank = blockIdx.x / splits / a.Hkv;
  const Parts parts = parts_of(a.workspace, gridDim.x, D);

  // ---- which 256 rows: the request whose row tiles hold this CTA's rank
  {
    const int per = (a.B + kThreads - 1) / kThreads, b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
    auto rows_of = [&](int b, int& row0) {
      row0 = min(max(a.row_start[b], 0), (int)a.T);
      return min(max(a.row_start[b + 1], row0), (int)a.T) - row0;
    };
    if (tid == 0) item.b = -1;
    int64_t s = 0;
    int row0;
    for (int b = b0; b < b1; ++b) s += ((int64_t)rows_of(b, row0) * g + kRows - 1) / kRows;
    int64_t inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int64_t at = inc - s;
    for (int w = 0; w < warp; ++w) at += warp_sums[w];
    if (rank >= at && rank < at + s) {
      for (int b = b0; b < b1; ++b) {
        const int n = rows_of(b, row0);
        const int tiles = (int)(((int64_t)n * g + kRows - 1) / kRows);
        if (rank < at + tiles) {
          const int total = max(a.total[b], 0);
          const int64_t limit = a.width * a.block;
          // the last rows see most tokens: they go first
          item = {b, row0, n, (int)(tiles - 1 - (rank - at)) * kRows, limit < total ? (int)limit : total, total - n};
          break;
        }
        at += tiles;
      }
    }
    __syncthreads();
  }
  const Item it = item;
  // tokens that the last row of a tile sees, in tiles
  const int rows = it.n * g;
  auto tiles_of = [&](int mt) {
    const int last = min(it.first + (mt + 1) * kRowsM, rows) - 1;
    if (last < it.first + mt * kRowsM) return 0;
    const int sees = min(it.pos0 + last / g + 1, it.keys);
    return sees > 0 ? (sees - 1) / kKeys + 1 : 0;
  };
  const int seen0 = it.b < 0 ? 0 : tiles_of(0), seen1 = it.b < 0 ? 0 : tiles_of(1), seen = max(seen0, seen1);
  // this CTA's share of them
  const int used = min(splits, max(seen / kLeastTiles, 1));
  if (splits > 1 && split == 0 && tid == 0)
    parts.item[blockIdx.x / splits] = {it.first, min(rows - it.first, kRows), it.row0, h, it.b < 0 || used == 1 ? 0 : used};
  if (it.b < 0 || split >= used) return;
  const int i0 = (int)((int64_t)seen * split / used), i1 = (int)((int64_t)seen * (split + 1) / used);
  const int n0 = max(min(seen0, i1) - i0, 0), n1 = max(min(seen1, i1) - i0, 0), n = max(n0, n1);
  const int tok0 = i0 * kKeys;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], 4);
      mbar_init(&kempty[i], 1);
      mbar_init(&vfull[i], 4);
      mbar_init(&vempty[i], 1);
      mbar_init(&sfull[i], 1);
      mbar_init(&pready[2 * i], 4);
      mbar_init(&pready[2 * i + 1], 4);
      mbar_init(&odone[i], 1);
      mbar_init(&ofinal[i], 1);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(&mready[i], 4);
    mbar_init(qready, 8);
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 12) tmem_alloc(tmem_slot, kTmemCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp < 8) {
    // ------------------------------------------------ softmax: one row per thread
    const int mt = warp >> 2, mine = mt ? n1 : n0;
    const int row = it.first + mt * kRowsM + (warp & 3) * 32 + lane;
    const bool live = row < rows;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + kS + mt * 128 + lanes, o_tm = tmem + kO + mt * D + lanes;
    const float scale = a.scale ? *a.scale : rsqrtf((float)D);
    // The warp's rows: copied by neighbouring lanes into their places, then turned to fp16 there, a row's largest value
    // in [2^10, 2^11), by the row's thread.  In short loops: the code runs once a CTA, and fetching it costs most.
    float q_scale, q_sum = 0.0f;
    {
      constexpr int kLanes = D / 8, kStep = 32 / kLanes;  // lanes per row, rows per copy
      const uint32_t tile = q_at + mt * S::kTile;
      const int piece = lane % kLanes, t0 = (warp & 3) * 32 + lane / kLanes, r0 = it.first + mt * kRowsM + t0;
      const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)it.row0 * a.q_stride + (int64_t)h * g * D + piece * 8;
      Walk at(r0, kStep, g);
#pragma unroll 2
      for (int x = 0; x < kLanes; ++x) {
        const bool there = r0 + x * kStep < rows;
        const uint16_t* from = there ? q + (int64_t)at.tok * a.q_stride + at.head * D : q;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         tile + (piece / 8) * S::kBlock + swizzled(t0 + x * kStep, piece % 8)),
                     "l"(from), "r"(there ? 16 : 0)
                     : "memory");
        at.next();
      }
      asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
      __syncwarp();
      const int t = (warp & 3) * 32 + lane;
      uint32_t top = 0;
#pragma unroll 4
      for (int i = 0; i < kLanes; ++i) {
        const uint4 v = lds128(tile + (i / 8) * S::kBlock + swizzled(t, i % 8));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          asm("max.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(w[e] & 0x7FFF7FFFu));  // a NaN gives way to a number
      }
      const float amax = fmaxf(__uint_as_float(top << 16), __uint_as_float(top & 0xFFFF0000u));
      const int e2 = max((int)(__float_as_uint(amax) >> 23) - 127, -100);
      const float up = __uint_as_float((uint32_t)(127 + 10 - e2) << 23), down = __uint_as_float((uint32_t)(127 - 10 + e2) << 23);
      const float sign = scale < 0.0f ? -up : up;
      q_scale = fabsf(scale) * kLog2e * down;
#pragma unroll 2
      for (int i = 0; i < kLanes; ++i) {
        const uint32_t place = tile + (i / 8) * S::kBlock + swizzled(t, i % 8);
        const uint4 v = lds128(place);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[e] = pack2(__uint_as_float(w[e] << 16) * sign, __uint_as_float(w[e] & 0xFFFF0000u) * sign);
          const __half2 hv = *reinterpret_cast<const __half2*>(&o[e]);
          q_sum += __low2float(hv) + __high2float(hv);
        }
        sts128(place, o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qready);
    }

    float ref = -INFINITY, l = 0.0f, ws = 0.0f;
    // tokens that the row sees; rows that are none see all (their scores are 0)
    const int sees = live ? min(it.pos0 + row / g + 1, it.keys) - tok0 : INT32_MAX;
    bool ok = true;
    for (int i = 0; i < mine; ++i) {
      if (!await(&mready[i % kMeta], (uint32_t)(i / kMeta) & 1u, abort_flag, err) ||
          !await(&sfull[mt], (uint32_t)i & 1u, abort_flag, err)) {
        ok = false;
        break;
      }
      fence_after();
      const int lim = sees - i * kKeys;
      const bool masked = __any_sync(0xffffffffu, lim < kKeys);
      const uint32_t pages = meta_at + (i % kMeta) * 128;
      // the tile in two halves, so that the products of the first begin while the second is worked on
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const uint32_t from = s_tm + 64 * half;
        const int first = 64 * half;
        uint32_t w[4][8];
        float sum, all, most;
        // one reading of the half's scores: weights under the reference (-inf: 0 in its place) and their sums
        auto weigh = [&](auto with_mask) {
          const float off = kTop - (ref == -INFINITY ? 0.0f : ref);
          // all of the half at once: what lies between two waits for tensor memory is scheduled as one piece
          uint32_t s[2][32];
          tmem_ld32_nowait(from, s[0]);
          tmem_ld32_nowait(from + 32, s[1]);
          landed(s[0], s[1]);
          sum = all = most = 0.0f;
#pragma unroll
          for (int grp = 0; grp < 4; ++grp) {
            const Page p = page_at(pages, 4 * half + grp, q_scale, q_sum);
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(s[grp >> 1][16 * (grp & 1) + e]);
#pragma unroll
            for (int e = 0; e < 16; e += 2) fma2(v[e], v[e + 1], p.f2, p.c + off);
            if constexpr (decltype(with_mask)::value) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (first + 16 * grp + e >= lim) v[e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = ex2(v[e]);
            float s0 = v[0], s1 = v[1];
#pragma unroll
            for (int e = 2; e < 16; e += 2) add2(s0, s1, v[e], v[e + 1]);
#pragma unroll
            for (int e = 0; e < 8; ++e) w[grp][e] = pack2(v[2 * e], v[2 * e + 1]);
            s0 += s1;
            most = fmaf(s0, p.part, most);
            sum = fmaf(s0, p.inv, sum);
            // a page whose values are all zero takes part in the sum alone
            all += p.some() ? s0 : 0.0f;
            if (!p.some()) {
#pragma unroll
              for (int e = 0; e < 8; ++e) w[grp][e] = 0u;
            }
          }
        };
        // the row's maximum over the half (in log2 units, values' scale included)
        auto maximum = [&] {
          float top = -INFINITY;
#pragma unroll 1
          for (int grp = 0; grp < 4; ++grp) {
            const Page p = page_at(pages, 4 * half + grp, q_scale, q_sum);
            const float c = p.some() ? p.c : p.c + kLeastValueLog;
            uint32_t s[16];
            tmem_ld16(from + 16 * grp, s);
            landed(s);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (first + 16 * grp + e < lim) top = fmaxf(top, fmaf(__uint_as_float(s[e]), p.f2, c));
          }
          return top;
        };
        auto run = [&] {
          if (masked)
            weigh(std::true_type());
          else
            weigh(std::false_type());
        };
        run();
        // No weight is above the sum of the half's: while that is at most 2^15 the reference holds, and no maximum is
        // taken.  Above it (an infinity with it), and until a row has seen a token, the reference moves.
        const bool follow = most > kMost || ref == -INFINITY;
        if (__any_sync(0xffffffffu, follow)) {
          const float top = maximum();
          const float next = follow ? fmaxf(ref, top) : ref;
          const Shrink to_next = shrink(ref == -INFINITY ? -INFINITY : ref - next);
          const float grow = to_next.near;
          if (i + half > 0) {
            // the products up to the half before this one (the one before that is known to have ended)
            if (!await(&odone[mt], (uint32_t)(half ^ 1), abort_flag, err)) {
              ok = false;
              break;
            }
            fence_after();
            const float by = follow && next != ref ? grow : 1.0f;
#pragma unroll 1
            for (int x = 0; x < D; x += 16) {
              uint32_t r[16];
              tmem_ld16(o_tm + x, r);
              landed(r);
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * by);
              tmem_st16(o_tm + x, r);
            }
          }
          if (follow && next != ref) {
            l = l * to_next.far * grow;
            ws *= grow;
            ref = next;
          }
          run();
        }
        l = fmaf(sum, kSumScale, l);
        ws += all;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t r[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) r[e] = w[2 * x + e / 8][e % 8];
          tmem_st16(s_tm + 32 * half + 16 * x, r);
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pready[2 * mt + half]);
      }
      if (!ok) break;
    }
    // ---- o = (2 O + sum of the weights) / l
    // Below, a warp of 128-value rows writes over the Q rows of its neighbours: they have all been written (and turned)
    // once qready completes, and read once the tile's products have ended.  A row tile that sees no token has no
    // products to wait for, so it waits for the Q rows alone.
    if (ok) ok = mine > 0 ? await(&ofinal[mt], 0, abort_flag, err) : await(qready, 0, abort_flag, err);
    fence_after();
    if (ok && used > 1) {
      // a part: unscaled, under this CTA's reference
      const int t = mt * kRowsM + (warp & 3) * 32 + lane;
      float4* to = reinterpret_cast<float4*>(parts.o + ((int64_t)blockIdx.x * kRows + t) * D);
#pragma unroll 1
      for (int x = 0; x < D; x += 16) {
        uint32_t r[16];
        if (mine > 0) {
          tmem_ld16(o_tm + x, r);
          landed(r);
        }
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = mine > 0 ? fmaf(2.0f, __uint_as_float(r[e]), ws) : 0.0f;
        if (live) {
#pragma unroll
          for (int e = 0; e < 4; ++e) to[x / 4 + e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
        __syncwarp();
      }
      if (live) parts.ml[(int64_t)blockIdx.x * kRows + t] = make_float2(ref, l);
    } else if (ok) {
      const float inv = l == 0.0f ? 0.0f : __fdiv_rn(kSumScale, l);
      // through the warp's part of the Q tile, free by now, so that lanes write whole rows
      const uint32_t stage = q_at + mt * S::kTile + (warp & 3) * (32 * D * 2);
      constexpr int kLanes = D / 8;
      auto place = [&](int r, int piece) { return stage + r * (D * 2) + ((piece ^ (r & 7)) << 4); };
#pragma unroll 1
      for (int x = 0; x < D; x += 16) {
        uint32_t r[16];
        float v[16];
        if (mine > 0) {
          tmem_ld16(o_tm + x, r);
          landed(r);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = mine > 0 ? fmaf(2.0f, __uint_as_float(r[e]), ws) * inv : 0.0f;
        if (a.o_bf16) {
          uint32_t p[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[e]) : "f"(v[2 * e + 1]), "f"(v[2 * e]));
          sts128(place(lane, x / 8), p[0], p[1], p[2], p[3]);
          sts128(place(lane, x / 8 + 1), p[4], p[5], p[6], p[7]);
        } else if (live) {
          const int64_t at = ((int64_t)(it.row0 + row / g) * a.Hq + (int64_t)h * g + row % g) * D;
          float4* to = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.o) + at + x);
#pragma unroll
          for (int e = 0; e < 4; ++e) to[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
        __syncwarp();
      }
      if (a.o_bf16) {
        constexpr int kStep = 32 / kLanes;
        const int r0 = it.first + mt * kRowsM + (warp & 3) * 32 + lane / kLanes;
        Walk to(r0, kStep, g);
#pragma unroll 2
        for (int x = 0; x < kLanes; ++x) {
          const uint4 v = lds128(place(x * kStep + lane / kLanes, lane % kLanes));
          if (r0 + x * kStep < rows)
            *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.o) +
                                      ((int64_t)(it.row0 + to.tok) * a.Hq + (int64_t)h * g + to.head) * D + lane % kLanes * 8) = v;
          to.next();
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------ codes to fp16, 32 tokens of a tile per warp
    const int cw = warp - 8;
    constexpr int kPerHalf = S::kHalves;   // neighbouring vectors alternate between the halves of a token's row
    const int32_t* pages = a.table + (int64_t)it.b * a.width;
    const int block_shift = 31 - __clz(a.block);
    const int L = (1 << a.bits) - 1;
    const uint32_t minus = 0xE400E400u | ((uint32_t)(1 << (a.bits - 1)) * 0x10001u);  // -(1024 + z), twice
    auto page_of = [&](int i, int grp) {
      const int tok = tok0 + i * kKeys + cw * 32 + grp * 16;
      const int v = i < n && tok < it.keys ? pages[tok >> block_shift] : -1;
      return v >= 0 && v < a.num_blocks ? v : -1;
    };
    const int my_tok = lane >> 2, my_piece = lane & 3;
    auto load = [&](const uint8_t* codes, int i, const int (&id)[2], uint4 (&v)[S::kVectors]) {
#pragma unroll
      for (int j = 0; j < S::kVectors; ++j) {
        const int half = j % kPerHalf, tok = (j / kPerHalf) * 8 + my_tok;   // tok < 32
        const int page = id[(j / kPerHalf) >> 1];
        const int64_t from =
            (((int64_t)page * a.Hkv + h) * a.block + ((tok0 + i * kKeys + cw * 32 + tok) & (a.block - 1))) * D + half * 64 + my_piece * 16;
        v[j] = page >= 0 ? *reinterpret_cast<const uint4*>(codes + from) : make_uint4(0, 0, 0, 0);
      }
    };
    auto convert = [&](uint32_t tile, const int (&id)[2], const uint4 (&v)[S::kVectors]) {
#pragma unroll
      for (int j = 0; j < S::kVectors; ++j) {
        const int half = j % kPerHalf, tok = cw * 32 + (j / kPerHalf) * 8 + my_tok;
        const bool there = id[(j / kPerHalf) >> 1] >= 0;
        const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          asm("add.rn.f16x2 %0, %1, %2;" : "=r"(o[2 * e]) : "r"(__byte_perm(w[e], 0x64646464u, 0x4140u)), "r"(minus));
          asm("add.rn.f16x2 %0, %1, %2;" : "=r"(o[2 * e + 1]) : "r"(__byte_perm(w[e], 0x64646464u, 0x4342u)), "r"(minus));
        }
        if (!there) {  // the warp's tokens of one page: a branch for all lanes
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = 0u;
        }
        const uint32_t at = tile + half * S::kBlock;
        sts128(at + swizzled(tok, 2 * my_piece), o[0], o[1], o[2], o[3]);
        sts128(at + swizzled(tok, 2 * my_piece + 1), o[4], o[5], o[6], o[7]);
      }
    };
    int id[2], next[2];
    uint4 kv[S::kVectors], vv[S::kVectors];
    float ks = 0.0f, vs = 0.0f;  // scales of the page of the group that this lane (0 or 1) writes down
#pragma unroll
    for (int e = 0; e < 2; ++e) id[e] = page_of(0, e), next[e] = page_of(1, e);
    load(a.k_codes, 0, id, kv);
    load(a.v_codes, 0, id, vv);
    auto scales = [&](const int (&of)[2]) {
      const int page = lane == 0 ? of[0] : of[1];
      if (lane < 2 && page >= 0) {
        ks = a.k_scales[(int64_t)page * a.Hkv + h];
        vs = a.v_scales[(int64_t)page * a.Hkv + h];
      }
    };
    scales(id);
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      const uint32_t reuse = ((uint32_t)(i >> 1) & 1u) ^ 1u;
      if (!await(&kempty[st], reuse, abort_flag, err)) break;
      if (lane < 2) {
        const bool there = (lane == 0 ? id[0] : id[1]) >= 0;
        const float vu = __fdiv_rn(vs, (float)L);
        const bool some = vu >= kLeastValueScale;
        const float lu = some ? __log2f(vu) : 0.0f;
        meta[(i % kMeta) * 8 + cw * 2 + lane] =
            there ? make_float4(__fdiv_rn(ks, (float)L), lu, ex2(-lu), some ? 1.0f : kLeastValueScale)
                  : make_float4(0.0f, -INFINITY, 0.0f, 0.0f);
      }
      convert(k_at + st * S::kTile, id, kv);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&mready[i % kMeta]);
        mbar_arrive(&kfull[st]);
      }
      if (i + 1 < n) {
        load(a.k_codes, i + 1, next, kv);
        scales(next);
      }
      if (!await(&vempty[st], reuse, abort_flag, err)) break;
      convert(v_at + st * S::kTile, id, vv);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&vfull[st]);
      if (i + 1 < n) load(a.v_codes, i + 1, next, vv);
#pragma unroll
      for (int e = 0; e < 2; ++e) id[e] = next[e], next[e] = page_of(i + 2, e);
    }
  } else {
    // ------------------------------------------------ products
    // The whole warp goes through the loop, so that addresses and descriptors stay in uniform registers and an issue
    // is few instructions between the softmax warps' (one lane's branch cost 40% more time per product).
    const uint64_t q0 = sdesc_k_sw128(q_at), k0 = sdesc_k_sw128(k_at), v0 = sdesc_mn_sw128(v_at, S::kBlock);
    const uint32_t q_lo = (uint32_t)q0, k_lo = (uint32_t)k0, v_lo = (uint32_t)v0;
    const uint32_t k_hi = (uint32_t)(k0 >> 32), v_hi = (uint32_t)(v0 >> 32);  // Q's is K's
    auto scores = [&](auto mt, uint32_t k) {
      if (elect_one()) {
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint32_t in = (x / 4) * (S::kBlock / 16) + 2 * (x % 4);
          mma_ss(tmem + kS + mt * 128, q_lo + mt * (S::kTile / 16) + in, k_hi, k + in, k_hi, kIdescS, x > 0 ? 1u : 0u);
        }
        umma_commit(&sfull[mt]);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) umma_commit(bar);
      __syncwarp();
    };
    bool ok = n == 0 || (await(qready, 0, abort_flag, err) && await(&kfull[0], 0, abort_flag, err));
    if (ok && n > 0) {
      fence_after();
      if (n0 > 0) scores(std::integral_constant<int, 0>(), k_lo);
      if (n1 > 0) scores(std::integral_constant<int, 1>(), k_lo);
      commit(&kempty[0]);
    }
    for (int i = 0; i < n && ok; ++i) {
      const int st = i & 1, nst = st ^ 1;
      const uint32_t v = v_lo + st * (S::kTile / 16), k = k_lo + nst * (S::kTile / 16);
      ok = await(&vfull[st], (uint32_t)(i >> 1) & 1u, abort_flag, err) &&
           (i + 1 >= n || await(&kfull[nst], (uint32_t)((i + 1) >> 1) & 1u, abort_flag, err));
      if (!ok) break;
      auto row_tile = [&](auto mt) {
        const int mine = mt ? n1 : n0;
        if (i < mine) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!await(&pready[2 * mt + half], (uint32_t)i & 1u, abort_flag, err)) return false;
            fence_after();
            if (elect_one()) {
#pragma unroll
              for (int y = 0; y < kKeys / 32; ++y)
                mma_ts(tmem + kO + mt * D, tmem + kS + mt * 128 + 32u * half + 8u * y, v + 512u * half + 128u * y, v_hi,
                       kIdescO<D>, half + y > 0 ? 1u : (uint32_t)(i > 0));
              umma_commit(&odone[mt]);
              if (half == 1 && i + 1 == mine) umma_commit(&ofinal[mt]);
            }
            __syncwarp();
          }
          if (i + 1 < mine) scores(mt, k);
        }
        return true;
      };
      ok = row_tile(std::integral_constant<int, 0>()) && row_tile(std::integral_constant<int, 1>());
      if (!ok) break;
      commit(&vempty[st]);
      if (i + 1 < n) commit(&kempty[nst]);
    }
    // all products issued are complete before tensor memory is freed
    if (elect_one()) {
      umma_commit(drain);
      drain_wait(drain, 0, err);
    }
    __syncwarp();
  }

  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 12) tmem_dealloc(tmem, kTmemCols);
}

// Joins the parts of a row, in order: a CTA takes 32 rows of an item, a warp
// one row after the other.
template <int D>
__global__ void __launch_bounds__(256) kv_attention_prompt_join_kernel(const KvAttentionArgs a, const int splits) {
  constexpr int V = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t items = gridDim.x / (kRows / 32), at = blockIdx.x / (kRows / 32);
  const Parts parts = parts_of(a.workspace, items * splits, D);
  const Joined it = parts.item[at];
  if (it.parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = a.Hq / a.Hkv;
  const int first = (blockIdx.x % (kRows / 32)) * 32;
  for (int t = first + warp; t < min(first + 32, it.rows); t += 8) {
    auto slot = [&](int p) { return (at * splits + p) * kRows + t; };
    const float2 ml = lane < it.parts ? parts.ml[slot(lane)] : make_float2(-INFINITY, 0.0f);
    float top = ml.x;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const Shrink by = shrink(ml.x - (top == -INFINITY ? 0.0f : top));
    const float f = by.near;
    float sum = f * (by.far * ml.y);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll 4
    for (int p = 0; p < it.parts; ++p) {
      const float by = __shfl_sync(0xffffffffu, f, p);
      const float* from = parts.o + slot(p) * D + lane * V;
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const float2 v = *reinterpret_cast<const float2*>(from + i);
        acc[i] = fmaf(by, v.x, acc[i]);
        acc[i + 1] = fmaf(by, v.y, acc[i + 1]);
      }
    }
    const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(kSumScale, sum);
    const int row = it.first + t;
    const int64_t to = ((int64_t)(it.row0 + row / g) * a.Hq + (int64_t)it.h * g + row % g) * D + lane * V;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float x = acc[i] * inv, y = acc[i + 1] * inv;
      if (a.o_bf16) {
        uint32_t p;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p) : "f"(y), "f"(x));
        *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.o) + to + i) = p;
      } else {
        *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.o) + to + i) = make_float2(x, y);
      }
    }
  }
}

// How a batch is laid out: a CTA for each row tile that it can have, whatever
// its rows' split over the requests, and as many CTAs per item as fill the SMs
// where there are few items and the table is long.
struct Layout {
  int64_t items;
  int splits;
};
Layout layout_of(const KvAttentionArgs& a) {
  Layout l;
  l.items = ((a.T * (a.Hq / a.Hkv) + kRows - 1) / kRows + a.B - 1) * a.Hkv;
  const int64_t room = sm100_host::sm_count() / l.items, tiles = a.width * a.block / kKeys / kLeastTiles;
  l.splits = (int)std::max<int64_t>(1, std::min({room, tiles, (int64_t)kMostSplits}));
  return l;
}

template <int D>
cudaError_t launch(const KvAttentionArgs& a, cudaStream_t stream) {
  int* err = device_error_word();
  if (!err) return cudaErrorInvalidValue;
  static std::atomic<bool> done[sm100_host::kMaxDevices];
  cudaError_t e = sm100_host::ensure_smem(kv_attention_prompt_kernel<D>, (int)Shape<D>::kSmem, done);
  if (e != cudaSuccess) return e;
  const Layout l = layout_of(a);
  kv_attention_prompt_kernel<D><<<(unsigned)(l.items * l.splits), kThreads, Shape<D>::kSmem, stream>>>(a, l.splits, err);
  e = cudaGetLastError();
  if (e != cudaSuccess || l.splits == 1) return e;
  return sm100_host::launch_pdl(kv_attention_prompt_join_kernel<D>, (unsigned)(l.items * (kRows / 32)), 256, 0, stream, 1,
                                a, l.splits);
}

}  // namespace

// The tensor cores' tiles pay where enough of them are at work and full.  With
// P the CTAs at once times the share of their 256 rows that is used (on
// average over the requests), the measured times cross at P near 18, or 45
// where CTAs share their items' tokens (a share costs its CTA about 12 us of
// start and end and the join).  At 32 heads over 8 and 64 requests of 4096
// tokens: about 25 rows a head and request, P = 15, 181 us here against 152 in
// kv_attention.cu; 50 rows, P = 28, 192 against 277.  One request of 16384,
// shared: 64 rows, P = 36, 48 us against 41; 128 rows, P = 72, 48 against 62;
// 1024 rows, 95 against 347.  The average is all the host knows: one prompt of
// 2048 rows over 4096 tokens beside 63 single rows comes here whole, 417 us,
// where two calls take 111 and 123.
constexpr int64_t kWorkAlone = 18, kWorkShared = 45;
bool kv_attention_prompt_supports(const KvAttentionArgs& a) {
  if (!a.q_bf16 || (a.D != 64 && a.D != 128)) return false;
  const int64_t rows = a.T * (a.Hq / a.Hkv);
  const Layout l = layout_of(a);
  if (l.items * l.splits > INT32_MAX / (kRows / 32)) return false;
  const int64_t tiles = std::max((rows / a.B + kRows - 1) / kRows, (int64_t)1) * a.B;  // of equal requests
  const int64_t ctas = std::min(tiles * a.Hkv * l.splits, (int64_t)sm100_host::sm_count());
  return rows * ctas >= (l.splits == 1 ? kWorkAlone : kWorkShared) * tiles * kRows;
}

size_t kv_attention_prompt_workspace(int D) {
  const size_t ctas = (size_t)sm100_host::sm_count();  // items are split over CTAs only as far as there are SMs
  return ctas * (kRows * (D * 4 + 8) + sizeof(Joined));
}

cudaError_t launch_kv_attention_prompt(const KvAttentionArgs& a, cudaStream_t stream) {
  return a.D == 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace hbl
