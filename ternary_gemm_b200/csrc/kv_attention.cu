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
// everything down to 2^-29 of it.  Queries are scaled by a power of two per
// row into fp16 (bf16 values exactly; float ones as two fp16 parts, 22 bits,
// and the weights too).
//
// One step takes sixteen tokens, which always lie in one block, against eight
// or sixteen rows (query heads of one cached head, times the request's rows).
// Both products have the codes as their 16-row operand and the rows as the
// 8-column one, S^T = K Q^T and O^T = V^T W^T, so that the few rows of a decode
// step cost no empty half of a product.  Such a step is bound by the codes'
// bytes: one warp is a pipeline of its own (cp.async into its stages, mma.sync
// m16n8k16, no block barrier), and all warps of the grid share the cache's
// tiles evenly: the tiles of all (request, row tile, head) items stand in one
// line, each warp takes the same length of it.  A warp that covers an item
// whole writes o; parts go to the workspace as (max, sum, o) and a second
// kernel joins them in order.
#include <cstdint>

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
constexpr int kTok = 16;        // tokens of a tile
constexpr float kTop = 15.0f;   // log2 of the largest weight in the second product
constexpr float kLog2e = 1.4426950408889634f;
// a warp takes at least this many tiles of the line
constexpr int kMinTiles = 4;

// Blocks per SM and stages per warp: copies in flight (over 100 KB on an SM)
// and warps enough to hide the products' latency, at the registers that the
// accumulators (4 NT D / 16 per thread) and the queries leave.
__host__ __device__ constexpr int blocks_per_sm(int D, int NT, bool f32) {
  const int weight = D * NT * (f32 ? 3 : 2);   // registers go with accumulators and query parts
  return weight <= 256 ? 4 : (weight <= 384 ? 3 : (weight <= 768 ? 2 : 1));
}
__host__ __device__ constexpr int stages_of(int D) { return D >= 128 ? 3 : 6; }

// Rows, tiles per row tile, and row tiles of a request.
struct Request {
  int row0;         // first row of the batch
  int n;            // rows
  int keys;         // tokens that the table can hold of it
  int pos0;         // position of its first row (negative where it has fewer tokens than rows)
  int tiles;        // 16-token tiles of one item
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
  r.tiles = max((int)(((int64_t)r.keys + kTok - 1) / kTok), 1);  // a request without tokens still writes its zeros
  r.items = ((int64_t)r.n * (a.Hq / a.Hkv) + rows_per_tile - 1) / rows_per_tile * a.Hkv;
  return r;
}

// Prefix sums of the requests' tiles in shared memory, by the whole CTA.
__device__ __forceinline__ int64_t lay_line(const KvAttentionArgs& a, int rows_per_tile, int64_t* start,
                                            int64_t* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int64_t s = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b, rows_per_tile);
    start[b] = s;
    s += r.tiles * r.items;
  }
  int64_t inc = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int64_t base = inc - s, all = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += warp_sums[w];
    all += warp_sums[w];
  }
  for (int b = b0; b < b1; ++b) start[b] += base;
  if (tid == 0) start[a.B] = all;
  __syncthreads();
  return all;
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

// 8 x 8 matrix of fp16 pairs across the warp, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
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
  if (BF16) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    if constexpr (N == 4)
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(o) + at) = make_uint2(w[0], w[N / 2 - 1]);
    else
      *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(o) + at) = w[0];
  } else if constexpr (N == 4) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(o) + at) = make_float4(v[0], v[1], v[N - 2], v[N - 1]);
  } else {
    *reinterpret_cast<float2*>(reinterpret_cast<float*>(o) + at) = make_float2(v[0], v[1]);
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
// and did not end.
struct Record {
  int64_t i0, i1, per;  // the item's tiles in the line, and a warp's share
  int b, row0, h, open; // open: there is such an item
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
  constexpr int kHalf = kTok * D;           // bytes of one of K and V in a stage
  constexpr int kStage = 2 * kHalf;
  constexpr int kSegs = D / 16;
  constexpr int kRows = 8 * NT;
  constexpr int kCopies = kHalf >= 512 ? kHalf / 512 : 1;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t warp_sums[kWarps];
  int64_t* start = reinterpret_cast<int64_t*>(smem + kWarps * kStages * kStage);

  // programmatic dependent of the stream's previous kernel: nothing is read before it has ended, and the joining
  // kernel may start from here on (it waits for this one before it reads the parts)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int64_t workers = (int64_t)gridDim.x * kWarps;
  const int64_t units = lay_line(a, kRows, start, warp_sums);
  const int64_t per = max((units + workers - 1) / workers, (int64_t)kMinTiles);
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
  if (u >= u_end && lane == 0) parts.record[worker].open = 0;

  // where this lane's copies land and its reads begin within a stage
  const uint32_t k_to = k_place<D>(lane / (D / 16), lane % (D / 16));
  const uint32_t v_to = v_place<D>(lane / (D / 16), lane % (D / 16));
  const uint32_t k_from = D >= 64 ? k_place<D>(gid, c) : gid * D + 8 * c;
  const uint32_t v_from = kHalf + v_place<D>(lane & 15, lane >> 4);

  while (u < u_end) {
    const int b = find_request(start, a.B, u);
    const Request r = request_of(a, b, kRows);
    const int64_t in_request = u - start[b];
    const int64_t item = in_request / r.tiles;
    const int t0 = (int)(in_request - item * r.tiles);            // first tile of the item here
    const int t1 = (int)min((int64_t)r.tiles, t0 + (u_end - u));  // end of the tiles here
    const int row_tile = (int)(item / a.Hkv), row0 = row_tile * kRows;
    const int h = (int)(item - (int64_t)row_tile * a.Hkv);
    const int64_t i0 = u - t0;
    u += t1 - t0;

    Query<D, NT, F32> q;
    load_query<D, NT, F32>(a, r, row0, h, lane, scale, q);
    // tokens that the tile's first and last row see, and tiles to work on (none: n <= 0)
    const int all_see = min(r.pos0 + row0 / g + 1, r.keys);
    const int any_sees = min(r.pos0 + (min(row0 + kRows, r.n * g) - 1) / g + 1, r.keys);
    const int n = min(t1, any_sees > 0 ? (any_sees - 1) / kTok + 1 : 0) - t0;

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

    // blocks and scales of 32 tiles at a time, one per lane, a group ahead
    const int32_t* pages = a.table + (int64_t)b * a.width;
    int id_now, id_next;
    float ku_now, vu_now, ku_next, vu_next;
    auto look_up = [&](int first, int& id, float& ku, float& vu) {
      id = -1;
      ku = 0.0f;
      vu = 1.0f;
      if (first + lane < n) {
        const int v = pages[((t0 + first + lane) * kTok) >> block_shift];
        if (v >= 0 && v < a.num_blocks) {
          id = v;
          const int64_t tile = (int64_t)v * a.Hkv + h;
          ku = __fdiv_rn(a.k_scales[tile], (float)L);
          vu = __fdiv_rn(a.v_scales[tile], (float)L);
        }
      }
    };
    look_up(0, id_now, ku_now, vu_now);
    look_up(32, id_next, ku_next, vu_next);

    uint32_t into = 0;      // the stage that the next copies fill
    auto issue = [&](int i, int id_of_group) {
      const int id = __shfl_sync(0xffffffffu, id_of_group, i & 31);
      if (i < n && id >= 0) {
        const int64_t from = (((int64_t)id * a.Hkv + h) * a.block + (((t0 + i) * kTok) & (a.block - 1))) * D + lane * 16;
        const uint8_t *k_src = a.k_codes + from, *v_src = a.v_codes + from;
        const uint32_t to = ring + into;
        if (kHalf >= 512 || lane < kHalf / 16) {
#pragma unroll
          for (int x = 0; x < kCopies; ++x) {
            cp_async16(to + k_to + x * 512, k_src + x * 512);
            // 32 pieces on, the token's part of the place changes by a constant
            cp_async16(to + kHalf + (v_to ^ (v_place<D>(x * 32 / (D / 16), 0) & 112)) + x * 512, v_src + x * 512);
          }
        }
      }
      cp_commit();
      into = into == (kStages - 1) * kStage ? 0 : into + kStage;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, id_now);

    uint32_t stage = ring;
    for (int i = 0; i < n; ++i) {
      if (i != 0 && (i & 31) == 0) {
        id_now = id_next;
        ku_now = ku_next;
        vu_now = vu_next;
        look_up(i + 32, id_next, ku_next, vu_next);
      }
      cp_wait<kStages - 2>();
      __syncwarp();  // tile i has landed for all lanes, and all have read the stage that the next copies overwrite
      issue(i + kStages - 1, (i & 31) + kStages - 1 < 32 ? id_now : id_next);

      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[nt][x] = 0.0f;
      if constexpr (D >= 64) {
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          // D >= 128: the halves of odd tokens stand the other way round
          const uint32_t at = D >= 128 ? stage + ((k_from ^ (64 * (j & 1))) + 128 * (j >> 1)) : stage + k_from;
          const uint4 x0 = lds128(at), x1 = lds128(at + 8 * D);
          const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t k[4] = {codes2(w0[x], 0x4140u, minus), codes2(w1[x], 0x4140u, minus),
                                   codes2(w0[x], 0x4342u, minus), codes2(w1[x], 0x4342u, minus)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma(s[nt], k, q.hi[nt][4 * j + x]);
              if constexpr (F32) mma(s[nt], k, q.lo[nt][4 * j + x]);
            }
          }
        }
      } else {
        const uint2 x0 = lds64(stage + k_from), x1 = lds64(stage + k_from + 8 * D);
        const uint32_t w0[2] = {x0.x, x0.y}, w1[2] = {x1.x, x1.y};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t k[4] = {codes2(w0[x], 0x4140u, minus), codes2(w1[x], 0x4140u, minus),
                                 codes2(w0[x], 0x4342u, minus), codes2(w1[x], 0x4342u, minus)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma(s[nt], k, q.hi[nt][x]);
            if constexpr (F32) mma(s[nt], k, q.lo[nt][x]);
          }
        }
      }

      const bool here = __shfl_sync(0xffffffffu, id_now, i & 31) >= 0;
      const float ku = __shfl_sync(0xffffffffu, ku_now, i & 31), vu = __shfl_sync(0xffffffffu, vu_now, i & 31);
      // a block whose values are all zero (below 1e-30) takes part in the sum alone
      const bool zero = !(vu >= 1e-30f);
      const float lu = __log2f(zero ? 1e-30f : vu), inv_vu = ex2(-lu);
      const int tok0 = (t0 + i) * kTok;
      const bool masked = !here || tok0 + kTok > all_see;
      float grow[NT][2];
      bool grows = false;
      uint32_t w_hi[NT][2], w_lo[F32 ? NT : 1][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // s[0], s[1]: token lane / 4, rows 2 c and 2 c + 1; s[2], s[3]: token lane / 4 + 8
        float p[2][2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float f1 = q.scale[nt][x] * ku, f0 = q.sum[nt][x] * f1, f = 2.0f * f1;
          p[0][x] = fmaf(s[nt][x], f, f0);
          p[1][x] = fmaf(s[nt][2 + x], f, f0);
        }
        if (masked) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int sees = min(r.pos0 + (row0 + nt * 8 + 2 * c + x) / g + 1, r.keys) - tok0;
            if (!here || gid >= sees) p[0][x] = -INFINITY;
            if (!here || gid + 8 >= sees) p[1][x] = -INFINITY;
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float top = fmaxf(m[nt][x], row_max(fmaxf(p[0][x], p[1][x])) + lu);
          // a row that has seen nothing keeps -inf, with 0 in its place in the differences
          const float base = top == -INFINITY ? 0.0f : top, off = lu + kTop - base;
          grow[nt][x] = ex2(m[nt][x] - base);
          grows |= grow[nt][x] != 1.0f;
          m[nt][x] = top;
          p[0][x] = ex2(p[0][x] + off);
          p[1][x] = ex2(p[1][x] + off);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t hi = zero ? 0u : pack2(p[y][0], p[y][1]);
          w_hi[nt][y] = transpose8(hi);
          if constexpr (F32) w_lo[nt][y] = transpose8(zero ? 0u : pack2(p[y][0] - half_lo(hi), p[y][1] - half_hi(hi)));
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float sum = p[0][x] + p[1][x];
          w_sum[nt][x] = fmaf(w_sum[nt][x], grow[nt][x], zero ? 0.0f : sum);
          l[nt][x] = fmaf(l[nt][x], grow[nt][x], sum * inv_vu);
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
#pragma unroll
      for (int x = 0; x < kSegs; x += 2) {
        // four 8 x 16-byte matrices: tokens 0-7 and 8-15 at two neighbouring 16-byte columns; a register holds two
        // tokens at two columns, the even column of a pair in rows 0-7 of the product and the odd one in rows 8-15
        uint32_t w[4];
        ldmatrix4t(stage + (D >= 128 ? (v_from ^ (16 * (x & 6))) + 128 * (x >> 3) : v_from ^ (16 * x)), w);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t v[4] = {codes2(w[2 * y], 0x4240u, minus), codes2(w[2 * y], 0x4341u, minus),
                                 codes2(w[2 * y + 1], 0x4240u, minus), codes2(w[2 * y + 1], 0x4341u, minus)};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma(o[nt][x + y], v, w_hi[nt]);
            if constexpr (F32) mma(o[nt][x + y], v, w_lo[nt]);
          }
        }
      }
      stage = stage == ring + (kStages - 1) * kStage ? ring : stage + kStage;
    }
    cp_wait<0>();
    __syncwarp();  // the ring is free for the next item

    const bool whole = t0 == 0 && t1 == r.tiles;
    const int64_t slot = worker * 2 + (t0 == 0 ? 1 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float sum = row_sum(l[nt][x]), ws = row_sum(w_sum[nt][x]);
        const int in_tile = nt * 8 + 2 * c + x, row = row0 + in_tile;
        if (row >= r.n * g) continue;
        const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
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
            store_row<false>(parts.o, (slot * kRows + in_tile) * D + 16 * s + 2 * gid, v);
          }
        }
        if (!whole && gid == 0) parts.ml[slot * kRows + in_tile] = make_float2(m[nt][x], sum);
      }
    if (u >= u_end && lane == 0) {
      Record rec;
      rec.i0 = i0;
      rec.i1 = i0 + r.tiles;
      rec.per = per;
      rec.b = b;
      rec.row0 = row0;
      rec.h = h;
      rec.open = t0 == 0 && t1 < r.tiles;
      parts.record[worker] = rec;
    }
  }
}

// Joins the parts of an item that more than one warp worked on: CTA w the item
// that warp w began and left open.  A warp takes a row and every n-th part.
template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads) kv_attention_join_kernel(const KvAttentionArgs a) {
  constexpr int kRows = 8 * NT;
  constexpr int kJoinWarps = kJoinThreads / 32;
  constexpr int V = D / 32;
  __shared__ float part_o[kJoinWarps][D];
  __shared__ float2 part_ml[kJoinWarps];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the parts are the previous kernel's; every CTA waits, so that the end of this grid is the end of that one too
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t workers = gridDim.x, w0 = blockIdx.x;
  const Parts parts = parts_of(a.workspace, workers, D, kRows);
  const Record rec = parts.record[w0];
  if (!rec.open) return;
  const Request r = request_of(a, rec.b, kRows);
  const int count = (int)((rec.i1 - 1) / rec.per - w0 + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = a.Hq / a.Hkv;
  const int rows = min(kRows, r.n * g - rec.row0);
  const int sharing = rows >= kJoinWarps ? 1 : kJoinWarps / rows;   // warps per row
  for (int y0 = 0; y0 < rows; y0 += kJoinWarps / sharing) {
    const int y = y0 + warp / sharing, first = warp % sharing;
    const bool on = y < rows && warp < kJoinWarps / sharing * sharing;
    float acc[V], top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    if (on) {
      auto slot = [&](int p) { return (p == 0 ? w0 * 2 + 1 : (w0 + p) * 2) * kRows + y; };
      for (int p = first + sharing * lane; p < count; p += sharing * 32) top = fmaxf(top, parts.ml[slot(p)].x);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll 8
      for (int p = first; p < count; p += sharing) {
        const int64_t at = slot(p);
        const float2 ml = parts.ml[at];
        const float f = ex2(ml.x - base);
        sum = fmaf(f, ml.y, sum);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(f, parts.o[at * D + i * 32 + lane], acc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) part_o[warp][i * 32 + lane] = acc[i];
    if (lane == 0) part_ml[warp] = make_float2(top, sum);
    __syncthreads();
    if (on && first == 0) {
      for (int w = warp; w < warp + sharing; ++w) top = fmaxf(top, part_ml[w].x);
      const float base = top == -INFINITY ? 0.0f : top;
      sum = 0.0f;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      float v2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int w = warp; w < warp + sharing; ++w) {
        const float f = ex2(part_ml[w].x - base);
        sum = fmaf(f, part_ml[w].y, sum);
        if (4 * lane < D) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = fmaf(f, part_o[w][4 * lane + i], v[i]);
        }
        if constexpr (D == 256) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v2[i] = fmaf(f, part_o[w][128 + 4 * lane + i], v2[i]);
        }
      }
      const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
      const int row = rec.row0 + y;
      const int64_t at = ((int64_t)(r.row0 + row / g) * a.Hq + (int64_t)rec.h * g + row % g) * D + 4 * lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= inv, v2[i] *= inv;
      if (4 * lane < D) {
        if (a.o_bf16)
          store_row<true>(a.o, at, v);
        else
          store_row<false>(a.o, at, v);
      }
      if constexpr (D == 256) {
        if (a.o_bf16)
          store_row<true>(a.o, at + 128, v2);
        else
          store_row<false>(a.o, at + 128, v2);
      }
    }
    __syncthreads();
  }
}

template <int D, int NT, bool F32>
cudaError_t launch(const KvAttentionArgs& a, cudaStream_t stream) {
  const unsigned grid = (unsigned)(sm100_host::sm_count() * blocks_per_sm(D, NT, F32));
  constexpr int ring = kWarps * stages_of(D) * 2 * kTok * D;
  static std::atomic<bool> done[sm100_host::kMaxDevices];
  cudaError_t e = sm100_host::ensure_smem(kv_attention_kernel<D, NT, F32>, ring + (kMaxRequests + 1) * 8, done);
  if (e != cudaSuccess) return e;
  e = sm100_host::launch_pdl(kv_attention_kernel<D, NT, F32>, grid, kThreads, ring + (size_t)(a.B + 1) * 8, stream, 1, a);
  if (e != cudaSuccess) return e;
  return sm100_host::launch_pdl(kv_attention_join_kernel<D, NT>, grid * kWarps, kJoinThreads, 0, stream, 1, a);
}

template <int D>
cudaError_t launch_d(const KvAttentionArgs& a, cudaStream_t stream) {
  // Rows of one request and cached head, on average: up to eight share one
  // pass over the codes in half the products that sixteen need.
  const bool few = a.T * (a.Hq / a.Hkv) <= (int64_t)8 * a.B;
  if (a.q_bf16) return few ? launch<D, 1, false>(a, stream) : launch<D, 2, false>(a, stream);
  if constexpr (D == 256) return launch<D, 1, true>(a, stream);  // sixteen float rows would not fit the registers
  else return few ? launch<D, 1, true>(a, stream) : launch<D, 2, true>(a, stream);
}

}  // namespace

size_t kv_attention_workspace(int64_t T, int Hq, int Hkv, int D, int B) {
  (void)T, (void)Hq, (void)Hkv, (void)B;
  size_t most = 0;
  for (int NT = 1; NT <= 2; ++NT) {
    const size_t workers = (size_t)sm100_host::sm_count() * blocks_per_sm(D, NT, false) * kWarps;
    const size_t bytes = workers * (2 * 8 * NT * (D * 4 + 8) + sizeof(Record));
    most = bytes > most ? bytes : most;
  }
  return (most + 255) & ~(size_t)255;
}

cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t stream) {
  switch (a.D) {
    case 32: return launch_d<32>(a, stream);
    case 64: return launch_d<64>(a, stream);
    case 128: return launch_d<128>(a, stream);
    case 256: return launch_d<256>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace hbl
