// Causal attention over the paged 8-bit cache, for few rows per request
// (decode and draft steps) and every head dimension and type.
//
// A code q of block c and head h stands for (2 q - L) u, u = fl(gamma / L),
// L = 2^bits - 1.  With z = 2^(bits - 1), 2 q - L = 2 (q - z) + 1, so on
// centred integer codes k' = k - z, v' = v - z (exact in fp16)
//
//   s_j = scale u_k(j) (2 sum_d q_d k'_jd + sum_d q_d)
//   w_j = exp(s_j) u_v(j),   o = sum_j w_j (2 v'_j + 1) / sum_j w_j / u_v(j)
//
// The value blocks' scale is part of the weight, so the running maximum is
// that of s_j + ln u_v(j): the weights that enter the second product lie in
// [0, 2^15] with the largest near the top, where fp16 keeps 11 bits of
// everything down to 2^-29 of it.  Their rounding falls on 2 v'_j; the 1 beside
// it and the sum below take them as they were.  What blocks of zeros do to the
// sum is said at kLeastValueScale.  Queries are scaled by a power of two per
// row into fp16 (bf16 values exactly; float ones as two fp16 parts, 22 bits,
// and the weights too).
//
// One step takes thirty-two tokens (each sixteen of them lie in one block)
// against eight or sixteen rows (query heads of one cached head, times the request's rows).
// Both products have the codes as their 16-row operand and the rows as the
// 8-column one, S^T = K Q^T and O^T = V^T W^T, so that the few rows of a decode
// step cost no empty half of a product.  Such a step is bound by the codes'
// bytes: one warp is a pipeline of its own (cp.async into its stages, mma.sync
// m16n8k16, no block barrier), and all warps of the grid share the cache's
// tiles evenly: the tiles of all (request, row tile, head) items stand in one
// line, each warp takes the same length of it.  A warp that covers an item
// whole writes o; parts go to the workspace as (max, sum, o) and a second
// kernel joins them in order.
//
// Measured (codes' bytes over the call's time): 64 requests of up to 8192
// tokens, 32 heads over 8 of 128: 109 us, 5.3 TB/s, 80% of a plain copy's rate;
// two of up to 131072: 78 us, 5.4 TB/s, 83%.  (Heads of 64: 70%, of 256: 69%, of
// 32: 50%; float queries at 128: 76%; four rows a request: 54%, float 41%.)  The
// main kernel alone moves its bytes at 5.7 TB/s; what is left is the join (4 us), the first loads of
// every warp, and shares that end unevenly.  One request of 777 tokens takes 12 us
// on the device: two launches and a chain of six dependent reads (lengths,
// table, scales, codes, part, parts of others).
#include <cstdint>
#include <utility>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "serving.cuh"
#include "sm100.cuh"

namespace hbl {
namespace {

using sm100::smem_u32;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kJoinThreads = 256;
constexpr int kTok = 16;        // tokens that surely lie in one block
constexpr int kStep = 2 * kTok; // tokens of a tile: two products' depth
constexpr float kTop = 15.0f;   // log2 of the largest weight in the second product
constexpr float kLog2e = 1.4426950408889634f;
// a warp takes at least this many tiles of the line
constexpr int kMinTiles = 2;

// Blocks per SM and stages per warp: copies in flight (over 100 KB on an SM)
// and warps enough to hide the products' latency, at the registers that the
// accumulators (4 NT D / 16 per thread) and the queries leave.  At D = 128 two
// blocks with two tiles ahead took 77 us where three with one ahead took 80
// (two requests of 131072 tokens), and 23 against 25 (one of 32768).  Past some
// 2100 requests their prefix sums leave room for one of the two.
__host__ __device__ constexpr int blocks_per_sm(int D, int NT, bool f32) {
  const int weight = D * NT * (f32 ? 3 : 2);   // registers go with accumulators and query parts
  return D == 256 ? 1 : (D == 128 ? 2 : (weight <= 128 ? 4 : 3));
}
__host__ __device__ constexpr int stages_of(int D) { return D == 256 ? 2 : (D >= 64 ? 3 : 6); }

// Rows, tiles per row tile, and row tiles of a request.
struct Request {
  int row0;         // first row of the batch
  int n;            // rows
  int keys;         // tokens that the table can hold of it
  int pos0;         // position of its first row (negative where it has fewer tokens than rows)
  int tiles;        // 32-token tiles of one item
  int64_t items;    // row tiles x cached heads
};

__device__ __forceinline__ Request request_of(const KvAttentionArgs& a, int b, int rows_per_tile) {
  Request r;
  const int T = (int)a.T;
  r.row0 = min(max(a.row_start[b], 0), T);
  r.n = min(max(a.row_start[b + 1], r.row0), T) - r.row0;
  const int total = max(a.total[b], 0);
  const int64_t limit = a.width * a.block;
  r.pos0 = total - r.n;
  r.keys = limit < total ? (int)limit : total;
  r.tiles = max((int)(((int64_t)r.keys + kStep - 1) / kStep), 1);  // a request without tokens still writes its zeros
  r.items = ((int64_t)r.n * (a.Hq / a.Hkv) + rows_per_tile - 1) / rows_per_tile * a.Hkv;
  return r;
}

// How the line of tiles is shared out: a warp takes `per` places of it.  Where
// the items are few beside the warps, each begins a share of its own (`pitch`
// places of the line, a multiple of per, for its tiles): a warp that went on
// from one item to the next would take twice as long as the others.
struct Line {
  int64_t units, per;
  bool padded;
  __device__ __forceinline__ int64_t pitch(const Request& r) const {
    return padded ? (r.tiles + per - 1) / per * per : r.tiles;
  }
};

// Sum over the CTA of s, and what lies before this thread's.
__device__ __forceinline__ int64_t scan(int64_t s, int64_t* warp_sums, int64_t& before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  before = inc - s;
  int64_t all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sums[w];
    all += warp_sums[w];
  }
  return all;
}

// Prefix sums of the requests' places in shared memory, by the whole CTA.
__device__ __forceinline__ Line lay_line(const KvAttentionArgs& a, int rows_per_tile, int64_t workers, int64_t* start,
                                         int64_t (*warp_sums)[kWarps]) {
  const int tid = threadIdx.x;
  const int each = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * each, a.B), b1 = min(b0 + each, a.B);
  int64_t tiles = 0, items = 0, before, unused;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b, rows_per_tile);
    start[b] = tiles;
    tiles += r.tiles * r.items;
    items += r.items;
  }
  Line line;
  line.units = scan(tiles, warp_sums[0], before);
  items = scan(items, warp_sums[1], unused);
  line.padded = items <= workers / 4;
  const int64_t shares = line.padded ? workers - items : workers;  // of `per` places: an item's last one may not be full
  line.per = max((line.units + shares - 1) / shares, (int64_t)kMinTiles);
  if (line.padded) {
    tiles = 0;
    for (int b = b0; b < b1; ++b) {
      const Request r = request_of(a, b, rows_per_tile);
      start[b] = tiles;
      tiles += line.pitch(r) * r.items;
    }
    line.units = scan(tiles, warp_sums[2], before);
  }
  for (int b = b0; b < b1; ++b) start[b] += before;
  if (tid == 0) start[a.B] = line.units;
  __syncthreads();
  return line;
}

// the request of a place in the line (start rising; equal starts: the last,
// which is the one that has tiles)
__device__ __forceinline__ int find_request(const int64_t* start, int B, int64_t u) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// two of a word's bytes (selector: byte, 0x64, byte, 0x64) as fp16 1024 + q,
// then minus 1024 + z: the centred codes, exactly
__device__ __forceinline__ uint32_t codes2(uint32_t w, uint32_t sel, uint32_t minus) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(__byte_perm(w, 0x64646464u, sel)), "r"(minus));
  return d;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ float half_lo(uint32_t v) { return __half2float(__ushort_as_half((unsigned short)(v & 0xFFFFu))); }
__device__ __forceinline__ float half_hi(uint32_t v) { return __half2float(__ushort_as_half((unsigned short)(v >> 16))); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ Shrink shrink(float d) { return {ex2(fmaxf(d, -100.0f)), ex2(fminf(d + 100.0f, 0.0f))}; }

// 8 x 8 matrix of fp16 pairs across the warp, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

template <int kOff>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0+%2], [%1+%2], 16;" ::"r"(dst), "l"(src), "n"(kOff) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int kOff>
__device__ __forceinline__ void ldmatrix4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4+%5];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr), "n"(kOff)
               : "memory");
}

template <int kOff>
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4+%5];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr), "n"(kOff)
               : "memory");
  return v;
}
template <int kOff>
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2+%3];" : "=r"(v.x), "=r"(v.y) : "r"(addr), "n"(kOff) : "memory");
  return v;
}

// f(0), f(1), ... f(N - 1) with the argument a constant
template <int... I, typename F>
__device__ __forceinline__ void unrolled(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void unrolled(F&& f) {
  unrolled(std::make_integer_sequence<int, N>(), static_cast<F&&>(f));
}

// over the eight lanes that hold one row's tokens
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

template <bool BF16, int N>
__device__ __forceinline__ void store_row(void* o, int64_t at, const float (&v)[N]) {
  if constexpr (N == 1) {
    if (BF16)
      reinterpret_cast<__nv_bfloat16*>(o)[at] = __float2bfloat16_rn(v[0]);
    else
      reinterpret_cast<float*>(o)[at] = v[0];
  } else {
    uint32_t w[N];
#pragma unroll
    for (int i = 0; i < N / (BF16 ? 2 : 1); ++i) {
      if (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[(2 * i + 1) % N]), "f"(v[2 * i % N]));
      else
        w[i] = __float_as_uint(v[i]);
    }
    char* to = reinterpret_cast<char*>(o) + at * (BF16 ? 2 : 4);
    if constexpr (N * (BF16 ? 2 : 4) == 4)
      *reinterpret_cast<uint32_t*>(to) = w[0];
    else if constexpr (N * (BF16 ? 2 : 4) == 8)
      *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2 % N], w[3 % N]);
  }
}

// Where a 16-byte piece of a token's row lies in a staged tile: K is read 16
// bytes a lane, a quad per token, so rows of 128 bytes and more put odd
// tokens' halves the other way round; V is read by ldmatrix, eight tokens at
// one column, so its pieces are spread over all eight 16-byte bank groups.
template <int D>
__device__ __forceinline__ int k_place(int tok, int piece) {
  return tok * D + 16 * (D >= 128 ? piece ^ ((tok & 1) << 2) : piece);
}
template <int D>
__device__ __forceinline__ int v_place(int tok, int piece) {
  constexpr int kPer = D >= 128 ? 1 : 128 / D;       // rows per 128 bytes
  constexpr int kMask = D >= 128 ? 7 : D / 16 - 1;
  return tok * D + 16 * (piece ^ ((tok / kPer) & kMask));
}

// Eight query rows as the B operand of the first product.  Lane c of a quad
// holds values 64 j + 16 c .. + 15 of row lane / 4 (D = 32: 8 c .. + 7), four
// per 16-deep step, the same order in which it reads the codes of a token.
template <int D, int NT, bool F32>
struct Query {
  static constexpr int kSteps = D / 16;
  uint32_t hi[NT][kSteps][2];
  uint32_t lo[F32 ? NT : 1][F32 ? kSteps : 1][2];
  // of rows 2 c and 2 c + 1 of each eight: the sum of a row's values as they
  // enter the product, and what a product of them is to be multiplied by (in
  // log2 units, without u_k)
  float sum[NT][2], scale[NT][2];
};

template <int D, int NT, bool F32>
__device__ __forceinline__ void load_query(const KvAttentionArgs& a, const Request& r, int row0, int h, int lane,
                                           float scale, Query<D, NT, F32>& q) {
  constexpr int kPer = D >= 64 ? 16 : 8;       // values per lane and part
  constexpr int kParts = D >= 64 ? D / 64 : 1;
  const int g = a.Hq / a.Hkv;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = row0 + nt * 8 + (lane >> 2);
    const bool live = row < r.n * g;
    const int64_t at = live ? (int64_t)(r.row0 + row / g) * a.q_stride + ((int64_t)h * g + row % g) * D : 0;
    float v[kParts][kPer];
#pragma unroll
    for (int j = 0; j < kParts; ++j)
#pragma unroll
      for (int i = 0; i < kPer; i += 8) {
        float* d = &v[j][i];
        if (!live) {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] = 0.0f;
        } else if (F32) {
          const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) + at + 64 * j +
                                                            (lane & 3) * kPer + i);
          const float4 x = p[0], y = p[1];
          d[0] = x.x, d[1] = x.y, d[2] = x.z, d[3] = x.w, d[4] = y.x, d[5] = y.y, d[6] = y.z, d[7] = y.w;
        } else {
          const uint4 x = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) + at + 64 * j +
                                                          (lane & 3) * kPer + i);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            d[2 * e] = __uint_as_float(w[e] << 16);
            d[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
          }
        }
      }
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < kParts; ++j)
#pragma unroll
      for (int i = 0; i < kPer; ++i) top = fmaxf(top, fabsf(v[j][i]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the row's largest value into [2^10, 2^11): a power of two, its inverse
    // kept for the scores (zero and tiny rows are scaled as 2^-100 would be)
    const int e = max((int)(__float_as_uint(top) >> 23) - 127, -100);
    const float up = __uint_as_float((uint32_t)(127 + 10 - e) << 23), down = __uint_as_float((uint32_t)(127 - 10 + e) << 23);
    const float sign = scale < 0.0f ? -up : up;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kParts; ++j)
#pragma unroll
      for (int s = 0; s < kPer / 4; ++s)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float x = v[j][4 * s + 2 * k] * sign, y = v[j][4 * s + 2 * k + 1] * sign;
          const uint32_t hi = pack2(x, y);
          q.hi[nt][j * (kPer / 4) + s][k] = hi;
          sum += half_lo(hi) + half_hi(hi);
          if constexpr (F32) {
            const uint32_t lo = pack2(x - half_lo(hi), y - half_hi(hi));
            q.lo[nt][j * (kPer / 4) + s][k] = lo;
            sum += half_lo(lo) + half_hi(lo);
          }
        }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    const float f = fabsf(scale) * kLog2e * down;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      q.sum[nt][x] = __shfl_sync(0xffffffffu, sum, 4 * (2 * (lane & 3) + x));
      q.scale[nt][x] = __shfl_sync(0xffffffffu, f, 4 * (2 * (lane & 3) + x));
    }
  }
}

// What a warp leaves in the workspace: (max, sum, o) of a part of an item (in
// slot 2 w the part that it begins in the middle of an item, in slot 2 w + 1
// the one that it leaves unfinished), and a record of the item that it began
// and did not end.  A CTA whose whole share lies in one item joins its warps'
// parts itself and leaves one, in its first warp's name.
struct Record {
  int64_t mid_cta, last_cta;  // the parts: `head` warps from this one on, `mid` CTAs from mid_cta on, `tail` warps
  int head, mid, tail;        // from the first of last_cta on; none at all: no open item
  int row, rows, h;           // first of the item's rows (in the request), their number, cached head
  int row0;                   // the request's first row of the batch
};
struct Parts {
  float* o;        // [slots][rows][D]
  float2* ml;      // [slots][rows]
  Record* record;  // [workers]
};

__host__ __device__ inline Parts parts_of(void* workspace, int64_t workers, int D, int rows) {
  Parts p;
  p.o = reinterpret_cast<float*>(workspace);
  p.ml = reinterpret_cast<float2*>(p.o + (size_t)workers * 2 * rows * D);
  p.record = reinterpret_cast<Record*>(p.ml + (size_t)workers * 2 * rows);
  return p;
}

template <int D, int NT, bool F32>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(D, NT, F32)) kv_attention_kernel(const KvAttentionArgs a) {
  constexpr int kStages = stages_of(D);
  constexpr int kHalf = kTok * D;           // bytes of sixteen tokens of K or V
  constexpr int kStage = 4 * kHalf;         // K and V of a tile: K, V of the first sixteen tokens, K, V of the others
  constexpr int kSegs = D / 16;
  constexpr int kRows = 8 * NT;
  constexpr int kCopies = kHalf >= 512 ? kHalf / 512 : 1;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t warp_sums[3][kWarps];
  __shared__ float2 cta_ml[kWarps][kRows];
  int64_t* start = reinterpret_cast<int64_t*>(smem + kWarps * kStages * kStage);

  // programmatic dependent of the stream's previous kernel: nothing is read before it has ended, and the joining
  // kernel may start from here on (it waits for this one before it reads the parts)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int64_t workers = (int64_t)gridDim.x * kWarps;
  const Line line = lay_line(a, kRows, workers, start, warp_sums);
  const int64_t units = line.units, per = line.per;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3, gid = lane >> 2;
  const int64_t worker = (int64_t)blockIdx.x * kWarps + warp;
  int64_t u = worker * per;
  const int64_t u_end = min(u + per, units);
  const Parts parts = parts_of(a.workspace, workers, D, kRows);
  const uint32_t ring = smem_u32(smem + warp * kStages * kStage);
  const int block_shift = 31 - __clz(a.block);
  const int L = (1 << a.bits) - 1;
  const uint32_t minus = 0xE400E400u | ((uint32_t)(1 << (a.bits - 1)) * 0x10001u);  // -(1024 + z), twice
  const float scale = a.scale ? *a.scale : rsqrtf((float)D);
  const int g = a.Hq / a.Hkv;
  // the CTA's share, and whether one item holds it
  const int64_t c0 = (int64_t)blockIdx.x * kWarps * per, c1 = min(c0 + kWarps * per, units);
  bool alone = false;
  if (c0 < c1) {
    const int b = find_request(start, a.B, c0);
    const int64_t pitch = line.pitch(request_of(a, b, kRows));
    alone = c1 <= start[b] + ((c0 - start[b]) / pitch + 1) * pitch;
  }
  if ((u >= u_end || (alone && warp != 0)) && lane == 0) {
    Record& rec = parts.record[worker];
    rec.head = rec.mid = rec.tail = 0;
  }

  // where this lane's copies land and its reads begin within a stage
  const uint32_t k_to = k_place<D>(lane / (D / 16), lane % (D / 16));
  const uint32_t v_to = v_place<D>(lane / (D / 16), lane % (D / 16));
  const uint32_t k_from = D >= 64 ? k_place<D>(gid, c) : gid * D + 8 * c;
  const uint32_t v_from = kHalf + v_place<D>(lane & 15, lane >> 4);

  while (u < u_end) {
    const int b = find_request(start, a.B, u);
    const Request r = request_of(a, b, kRows);
    const int64_t in_request = u - start[b], pitch = line.pitch(r);
    const int64_t item = in_request / pitch;
    const int t0 = (int)(in_request - item * pitch);              // first tile of the item here
    const int t1 = (int)min((int64_t)r.tiles, t0 + (u_end - u));  // end of the tiles here
    const int row_tile = (int)(item / a.Hkv), row0 = row_tile * kRows;
    const int h = (int)(item - (int64_t)row_tile * a.Hkv);
    const int64_t i0 = u - t0;
    u = line.padded ? u_end : u + (t1 - t0);

    // tokens that the tile's first and last row see, and tiles to work on (none: n <= 0)
    const int all_see = min(r.pos0 + row0 / g + 1, r.keys);
    const int any_sees = min(r.pos0 + (min(row0 + kRows, r.n * g) - 1) / g + 1, r.keys);
    const int n = min(t1, any_sees > 0 ? (any_sees - 1) / kStep + 1 : 0) - t0;
    const int first = t0 * 2, seen = any_sees > 0 ? (any_sees - 1) / kTok + 1 - first : 0;  // the same in sixteens

    float o[NT][kSegs][4];
    float m[NT][2], l[NT][2], w_sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int s = 0; s < kSegs; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][s][i] = 0.0f;
#pragma unroll
      for (int x = 0; x < 2; ++x) m[nt][x] = -INFINITY, l[nt][x] = 0.0f, w_sum[nt][x] = 0.0f;
    }

    // blocks and scales of 32 sixteens of tokens at a time, one per lane, a group ahead
    const int32_t* pages = a.table + (int64_t)b * a.width;
    // (id; scale of the keys; log2 of the values' scale; 0, 1 for values that are all zero, 2 for an absent block)
    int id_now, id_next, kind_now, kind_next;
    float ku_now, lu_now, ku_next, lu_next;
    auto page_of = [&](int i) {
      const int v = i + lane < seen ? pages[((first + i + lane) * kTok) >> block_shift] : -1;
      return v >= 0 && v < a.num_blocks ? v : -1;
    };
    auto scales_of = [&](int id, float& ku, float& lu, int& kind) {
      ku = lu = 0.0f;
      kind = 2;
      if (id >= 0) {
        const int64_t tile = (int64_t)id * a.Hkv + h;
        const float k = a.k_scales[tile], v = a.v_scales[tile];
        ku = __fdiv_rn(k, (float)L);
        const float vu = __fdiv_rn(v, (float)L);
        kind = vu >= kLeastValueScale ? 0 : 1;
        lu = kind == 0 ? __log2f(vu) : kLeastValueLog;
      }
    };
    id_now = page_of(0);
    id_next = page_of(32);

    uint32_t into = 0;      // the stage that the next copies fill
    auto issue = [&](int i, int id_of_group) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int id = __shfl_sync(0xffffffffu, id_of_group, (2 * i + half) & 31);
        if (i < n && id >= 0) {
          const int64_t from =
              (((int64_t)id * a.Hkv + h) * a.block + (((first + 2 * i + half) * kTok) & (a.block - 1))) * D + lane * 16;
          const uint8_t *k_src = a.k_codes + from, *v_src = a.v_codes + from;
          const uint32_t to = ring + into + half * 2 * kHalf;
          if (kHalf >= 512 || lane < kHalf / 16)
            unrolled<kCopies>([&](auto x) {
              cp_async16<x * 512>(to + k_to, k_src);
              // 32 pieces on, the token's part of the place changes by a constant
              cp_async16<x * 512>(to + kHalf + (v_to ^ (v_place<D>(x * 32 / (D / 16), 0) & 112)), v_src);
            });
        }
      }
      cp_commit();
      into = into == (kStages - 1) * kStage ? 0 : into + kStage;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, id_now);
    scales_of(id_now, ku_now, lu_now, kind_now);
    scales_of(id_next, ku_next, lu_next, kind_next);
    Query<D, NT, F32> q;
    load_query<D, NT, F32>(a, r, row0, h, lane, scale, q);

    uint32_t stage = ring;
    for (int i = 0; i < n; ++i) {
      if (i != 0 && (i & 15) == 0) {
        id_now = id_next;
        ku_now = ku_next;
        lu_now = lu_next;
        kind_now = kind_next;
        id_next = page_of(2 * i + 32);
        scales_of(id_next, ku_next, lu_next, kind_next);
      }
      cp_wait<kStages - 2>();
      __syncwarp();  // tile i has landed for all lanes, and all have read the stage that the next copies overwrite
      issue(i + kStages - 1, (i & 15) + kStages - 1 < 16 ? id_now : id_next);

      float s[2][NT][4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[half][nt][x] = 0.0f;
      }
      unrolled<2>([&](auto half) {
        constexpr int kAt = half * 2 * kHalf;
        auto steps = [&](int step, uint32_t w0, uint32_t w1) {
          const uint32_t k[4] = {codes2(w0, 0x4140u, minus), codes2(w1, 0x4140u, minus), codes2(w0, 0x4342u, minus),
                                 codes2(w1, 0x4342u, minus)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (F32) {
              // from 0 and added with a rounding: the tensor cores' own sums drop what lies below the last bit
              float t[4] = {};
              mma(t, k, q.hi[nt][step]);
              mma(t, k, q.lo[nt][step]);
#pragma unroll
              for (int e = 0; e < 4; ++e) s[half][nt][e] += t[e];
            } else {
              mma(s[half][nt], k, q.hi[nt][step]);
            }
          }
        };
        if constexpr (D >= 64) {
          unrolled<D / 64>([&](auto j) {
            // D >= 128: the halves of odd tokens stand the other way round
            const uint32_t at = D >= 128 ? stage + (k_from ^ (64 * (j & 1))) : stage + k_from;
            const uint4 x0 = lds128<kAt + (j >> 1) * 128>(at), x1 = lds128<kAt + (j >> 1) * 128 + 8 * D>(at);
            steps(4 * j, x0.x, x1.x);
            steps(4 * j + 1, x0.y, x1.y);
            steps(4 * j + 2, x0.z, x1.z);
            steps(4 * j + 3, x0.w, x1.w);
          });
        } else {
          const uint2 x0 = lds64<kAt>(stage + k_from), x1 = lds64<kAt + 8 * D>(stage + k_from);
          steps(0, x0.x, x1.x);
          steps(1, x0.y, x1.y);
        }
      });

      int kind[2];
      float ku[2], lu[2], inv_vu[2], lift[2];  // lift: what takes u out of the weights of zeros for the sum
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int from = (2 * i + half) & 31;
        kind[half] = __shfl_sync(0xffffffffu, kind_now, from);
        ku[half] = __shfl_sync(0xffffffffu, ku_now, from);
        lu[half] = __shfl_sync(0xffffffffu, lu_now, from);
        lift[half] = kind[half] == 1 ? -kLeastValueLog : 0.0f;
        inv_vu[half] = kind[half] == 1 ? 1.0f : ex2(-lu[half]);
      }
      const int tok0 = (first + 2 * i) * kTok;
      const bool masked = kind[0] == 2 || kind[1] == 2 || tok0 + kStep > all_see;
      float grow[NT][2];
      bool grows = false;
      uint32_t w_hi[2][NT][2], w_lo[2][F32 ? NT : 1][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // s[.][.][0], [1]: token lane / 4, rows 2 c and 2 c + 1; [2], [3]: token lane / 4 + 8.  p: its log2 weight
        float p[2][2][2];
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float f = q.scale[nt][x] * ku[half], f0 = fmaf(q.sum[nt][x], f, lu[half]), f2 = 2.0f * f;
            p[half][0][x] = fmaf(s[half][nt][x], f2, f0);
            p[half][1][x] = fmaf(s[half][nt][2 + x], f2, f0);
          }
        if (masked) {
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int sees = min(r.pos0 + (row0 + nt * 8 + 2 * c + x) / g + 1, r.keys) - tok0 - half * kTok;
              if (kind[half] == 2 || gid >= sees) p[half][0][x] = -INFINITY;
              if (kind[half] == 2 || gid + 8 >= sees) p[half][1][x] = -INFINITY;
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float top = fmaxf(
              m[nt][x], row_max(fmaxf(fmaxf(p[0][0][x], p[0][1][x]), fmaxf(p[1][0][x], p[1][1][x]))));
          // a row that has seen nothing keeps -inf, with 0 in its place in the differences
          const float base = top == -INFINITY ? 0.0f : top, off = kTop - base;
          const float rise = m[nt][x] - base;  // shrink(), its second factor where there is one
          grow[nt][x] = ex2(fmaxf(rise, -100.0f));
          if (rise < -100.0f) l[nt][x] *= ex2(rise + 100.0f);
          grows |= grow[nt][x] != 1.0f;
          m[nt][x] = top;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            p[half][0][x] = ex2(p[half][0][x] + (off + lift[half]));
            p[half][1][x] = ex2(p[half][1][x] + (off + lift[half]));
          }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // a block whose values are all zero takes part in the sum alone
          const bool zero = kind[half] == 1;
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t hi = zero ? 0u : pack2(p[half][y][0], p[half][y][1]);
            w_hi[half][nt][y] = transpose8(hi);
            if constexpr (F32)
              w_lo[half][nt][y] = transpose8(zero ? 0u : pack2(p[half][y][0] - half_lo(hi), p[half][y][1] - half_hi(hi)));
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float s0 = p[0][0][x] + p[0][1][x], s1 = p[1][0][x] + p[1][1][x];
          w_sum[nt][x] = fmaf(w_sum[nt][x], grow[nt][x], (kind[0] == 1 ? 0.0f : s0) + (kind[1] == 1 ? 0.0f : s1));
          l[nt][x] = fmaf(l[nt][x], grow[nt][x], kSumScale * fmaf(s0, inv_vu[0], s1 * inv_vu[1]));
        }
      }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < kSegs; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[nt][x][y] *= grow[nt][y & 1];
      }
      unrolled<kSegs / 2>([&](auto pair) {
        // four 8 x 16-byte matrices: tokens 0-7 and 8-15 at two neighbouring 16-byte columns; a register holds two
        // tokens at two columns, the even column of a pair in rows 0-7 of the product and the odd one in rows 8-15
        constexpr int x = 2 * pair;
        const uint32_t at = stage + (v_from ^ (16 * (x & 6)));
        // The tensor cores' sums drop what lies below the accumulator's last bit, always toward zero: over the hundreds
        // of products of a long item that would show in float outputs (1.5e-6 of them at 2448 tokens).  A tile's
        // products of float queries begin at 0, and an ordinary addition takes them to the row's.
        [[maybe_unused]] float of_tile[2][F32 ? NT : 1][4] = {};
        unrolled<2>([&](auto half) {
          uint32_t w[4];
          ldmatrix4t<half * 2 * kHalf + (x >> 3) * 128>(at, w);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t v[4] = {codes2(w[2 * y], 0x4240u, minus), codes2(w[2 * y], 0x4341u, minus),
                                   codes2(w[2 * y + 1], 0x4240u, minus), codes2(w[2 * y + 1], 0x4341u, minus)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (F32) {
                mma(of_tile[y][nt], v, w_hi[half][nt]);
                mma(of_tile[y][nt], v, w_lo[half][nt]);
              } else {
                mma(o[nt][x + y], v, w_hi[half][nt]);
              }
            }
          }
        });
        if constexpr (F32) {
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nt][x + y][e] += of_tile[y][nt][e];
        }
      });
      stage = stage == ring + (kStages - 1) * kStage ? ring : stage + kStage;
    }
    cp_wait<0>();
    __syncwarp();  // the ring is free for the next item

    const bool whole = t0 == 0 && t1 == r.tiles && !alone;
    const int64_t slot = worker * 2 + (t0 == 0 ? 1 : 0);
    // parts go to the workspace, or to this warp's own stages for the CTA to join
    float* part = alone ? reinterpret_cast<float*>(smem + warp * kStages * kStage) : parts.o + slot * kRows * D;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float sum = row_sum(l[nt][x]), ws = row_sum(w_sum[nt][x]);
        const int in_tile = nt * 8 + 2 * c + x, row = row0 + in_tile;
        if (row >= r.n * g) continue;
        const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(kSumScale, sum);
        const int64_t at = ((int64_t)(r.row0 + row / g) * a.Hq + (int64_t)h * g + row % g) * D;
#pragma unroll
        for (int s = 0; s < kSegs; ++s) {
          float v[2] = {fmaf(2.0f, o[nt][s][x], ws), fmaf(2.0f, o[nt][s][2 + x], ws)};
          if (whole) {
            v[0] *= inv, v[1] *= inv;
            if (a.o_bf16)
              store_row<true>(a.o, at + 16 * s + 2 * gid, v);
            else
              store_row<false>(a.o, at + 16 * s + 2 * gid, v);
          } else {
            store_row<false>(part, in_tile * D + 16 * s + 2 * gid, v);
          }
        }
        if (!whole && gid == 0) {
          if (alone)
            cta_ml[warp][in_tile] = make_float2(m[nt][x], sum);
          else
            parts.ml[slot * kRows + in_tile] = make_float2(m[nt][x], sum);
        }
      }
    if (alone) {
      // every warp of the CTA that has a share comes here once
      const int shares = (int)((c1 - c0 + per - 1) / per);
      asm volatile("bar.sync 1, %0;" ::"r"(shares * 32) : "memory");
      const bool all = i0 >= c0 && i0 + r.tiles <= c1;
      const int64_t to = ((int64_t)blockIdx.x * kWarps * 2 + (i0 >= c0 ? 1 : 0)) * kRows;
      for (int y = warp; y < kRows && row0 + y < r.n * g; y += shares) {
        float top = -INFINITY, sum = 0.0f;
        for (int w = 0; w < shares; ++w) top = fmaxf(top, cta_ml[w][y].x);
        const float base = top == -INFINITY ? 0.0f : top;
        float v[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) v[i] = 0.0f;
        for (int w = 0; w < shares; ++w) {
          const Shrink by = shrink(cta_ml[w][y].x - base);
          const float f = by.near;
          sum = fmaf(f, by.far * cta_ml[w][y].y, sum);
          const float* from = reinterpret_cast<const float*>(smem + w * kStages * kStage) + y * D;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) v[i] = fmaf(f, from[i * 32 + lane], v[i]);
        }
        const int row = row0 + y;
        const int64_t at = ((int64_t)(r.row0 + row / g) * a.Hq + (int64_t)h * g + row % g) * D;
        const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(kSumScale, sum);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          if (!all)
            parts.o[(to + y) * D + i * 32 + lane] = v[i];
          else if (a.o_bf16)
            reinterpret_cast<__nv_bfloat16*>(a.o)[at + i * 32 + lane] = __float2bfloat16_rn(v[i] * inv);
          else
            reinterpret_cast<float*>(a.o)[at + i * 32 + lane] = v[i] * inv;
        }
        if (!all && lane == 0) parts.ml[to + y] = make_float2(top, sum);
      }
    }
    if (u >= u_end && lane == 0 && (!alone || warp == 0)) {
      Record rec;
      rec.head = rec.mid = rec.tail = 0;
      if (alone ? i0 >= c0 && i0 + r.tiles > c1 : t0 == 0 && t1 < r.tiles) {
        // an item begun here and left open; CTAs that lie in it whole left one part each
        const int64_t i1 = i0 + r.tiles, w1 = (i1 - 1) / per, share = kWarps * per;
        const int64_t first_cta = blockIdx.x;
        rec.last_cta = w1 / kWarps;
        const bool last_in = rec.last_cta * share >= i0 && min((rec.last_cta + 1) * share, units) <= i0 + pitch;
        rec.head = alone ? 0 : (int)(min(w1, first_cta * kWarps + kWarps - 1) - worker + 1);
        rec.mid_cta = alone ? first_cta : first_cta + 1;
        rec.mid = (int)max((last_in ? rec.last_cta : rec.last_cta - 1) - rec.mid_cta + 1, (int64_t)0);
        rec.tail = last_in || rec.last_cta == first_cta ? 0 : (int)(w1 - rec.last_cta * kWarps + 1);
        rec.row = row0;
        rec.rows = min(kRows, r.n * g - row0);
        rec.h = h;
        rec.row0 = r.row0;
      }
      parts.record[worker] = rec;
    }
  }
}

// Joins the parts of the items that more than one warp worked on: CTA i those
// that the warps of CTA i began and left open, a warp per row.
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) kv_attention_join_kernel(const KvAttentionArgs a) {
  constexpr int kRows = 8 * NT;
  constexpr int V = D >= 128 ? 4 : D / 32;       // neighbouring values per lane
  constexpr int kCols = D / (32 * V);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the parts are the previous kernel's; every CTA waits, so that the end of this grid is the end of that one too
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Parts parts = parts_of(a.workspace, (int64_t)gridDim.x * kWarps, D, kRows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = a.Hq / a.Hkv;
  int dealt = 0;  // rows dealt out to the warps so far
  int counts = 0;  // of the record that a lane looks at: all at once, most are empty
  if (lane < kWarps) {
    const Record& rec = parts.record[(int64_t)blockIdx.x * kWarps + lane];
    counts = rec.head + rec.mid + rec.tail;
  }
  for (int own = 0; own < kWarps; ++own) {
    const int64_t w0 = (int64_t)blockIdx.x * kWarps + own;
    const int count = __shfl_sync(0xffffffffu, counts, own);
    if (count == 0) continue;
    const Record rec = parts.record[w0];
    for (int y = (warp - dealt) & (kJoinThreads / 32 - 1); y < rec.rows; y += kJoinThreads / 32) {
      auto slot = [&](int p) {
        const int64_t w = p < rec.head ? w0 + p
                                       : (p < rec.head + rec.mid ? (rec.mid_cta + p - rec.head) * kWarps
                                                                 : rec.last_cta * kWarps + p - rec.head - rec.mid);
        return (w * 2 + (p == 0 ? 1 : 0)) * kRows + y;
      };
      float acc[kCols][V], top = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kCols; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[j][i] = 0.0f;
      // eight parts at a time, their loads together, under a running maximum
      constexpr int kAhead = 8;
      for (int p0 = 0; p0 < count; p0 += kAhead) {
        float2 ml[kAhead];
        float part[kAhead][kCols][V];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          ml[e] = make_float2(-INFINITY, 0.0f);
          if (p0 + e < count) {
            const int64_t at = slot(p0 + e);
            ml[e] = parts.ml[at];
#pragma unroll
            for (int j = 0; j < kCols; ++j) {
              const float* from = parts.o + at * D + j * 32 * V + lane * V;
              if constexpr (V == 4) {
                const float4 v = *reinterpret_cast<const float4*>(from);
                part[e][j][0] = v.x, part[e][j][1] = v.y, part[e][j][2] = v.z, part[e][j][3] = v.w;
              } else {
#pragma unroll
                for (int i = 0; i < V; ++i) part[e][j][i] = from[i];
              }
            }
          }
        }
        float now = top;
#pragma unroll
        for (int e = 0; e < kAhead; ++e) now = fmaxf(now, ml[e].x);
        const float base = now == -INFINITY ? 0.0f : now;
        const Shrink to_now = shrink(top - base);
        const float f0 = to_now.near;
        top = now;
        sum = sum * to_now.far * f0;
#pragma unroll
        for (int j = 0; j < kCols; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) acc[j][i] *= f0;
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          if (p0 + e < count) {
            const Shrink by = shrink(ml[e].x - base);
            const float f = by.near;
            sum = fmaf(f, by.far * ml[e].y, sum);
#pragma unroll
            for (int j = 0; j < kCols; ++j)
#pragma unroll
              for (int i = 0; i < V; ++i) acc[j][i] = fmaf(f, part[e][j][i], acc[j][i]);
          }
        }
      }
      const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(kSumScale, sum);
      const int row = rec.row + y;
      const int64_t at = ((int64_t)(rec.row0 + row / g) * a.Hq + (int64_t)rec.h * g + row % g) * D + lane * V;
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[j][i] *= inv;
        if (a.o_bf16)
          store_row<true>(a.o, at + j * 32 * V, acc[j]);
        else
          store_row<false>(a.o, at + j * 32 * V, acc[j]);
      }
    }
    dealt += rec.rows;
  }
}

template <int D, int NT, bool F32>
cudaError_t launch(const KvAttentionArgs& a, cudaStream_t stream) {
  const unsigned grid = (unsigned)(sm100_host::sm_count() * blocks_per_sm(D, NT, F32));
  constexpr int ring = kWarps * stages_of(D) * 2 * kStep * D;
  static std::atomic<bool> done[sm100_host::kMaxDevices];
  cudaError_t e = sm100_host::ensure_smem(kv_attention_kernel<D, NT, F32>, ring + (kMaxRequests + 1) * 8, done);
  if (e != cudaSuccess) return e;
  e = sm100_host::launch_pdl(kv_attention_kernel<D, NT, F32>, grid, kThreads, ring + (size_t)(a.B + 1) * 8, stream, 1, a);
  if (e != cudaSuccess) return e;
  return sm100_host::launch_pdl(kv_attention_join_kernel<D, NT>, grid, kJoinThreads, 0, stream, 1, a);
}

template <int D>
cudaError_t launch_d(const KvAttentionArgs& a, cudaStream_t stream) {
  // Rows of one request and cached head, on average: up to eight share one
  // pass over the codes in half the products that sixteen need.
  // At D = 256 sixteen bf16 rows spill a little (300 bytes) and are kept for
  // prompts, the only path that those have: two chunks of 512 rows over 4096
  // tokens, 16 heads over 4, take 374 us so and 413 with eight; 32 x 4 draft
  // rows, 32 heads over 8, 135 and 133, 64 single rows, 32 heads over 2, 111
  // and 108.
  const bool few = a.T * (a.Hq / a.Hkv) <= (int64_t)8 * a.B;
  if (a.q_bf16) return few ? launch<D, 1, false>(a, stream) : launch<D, 2, false>(a, stream);
  if constexpr (D == 256) return launch<D, 1, true>(a, stream);  // sixteen float rows would not fit the registers
  else return few ? launch<D, 1, true>(a, stream) : launch<D, 2, true>(a, stream);
}

}  // namespace

size_t kv_attention_workspace(int64_t T, int Hq, int Hkv, int D, int B) {
  (void)T, (void)Hq, (void)Hkv, (void)B;
  size_t most = D == 64 || D == 128 ? kv_attention_prompt_workspace(D) : 0;
  for (int NT = 1; NT <= 2; ++NT) {
    const size_t workers = (size_t)sm100_host::sm_count() * blocks_per_sm(D, NT, false) * kWarps;
    const size_t bytes = workers * (2 * 8 * NT * (D * 4 + 8) + sizeof(Record));
    most = bytes > most ? bytes : most;
  }
  return (most + 255) & ~(size_t)255;
}

cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t stream) {
  if (kv_attention_prompt_supports(a)) return launch_kv_attention_prompt(a, stream);
  switch (a.D) {
    case 32: return launch_d<32>(a, stream);
    case 64: return launch_d<64>(a, stream);
    case 128: return launch_d<128>(a, stream);
    case 256: return launch_d<256>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace hbl
