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
// One 16 x 16 tile step: sixteen rows (query heads of one cached head, times
// the request's rows) against sixteen tokens, which always lie in one block.
// Rows of a decode step are few, so the step is bound by the codes' bytes: one
// warp is a pipeline of its own (cp.async into its stages, mma.sync m16n8k16,
// no block barrier), and all warps of the grid share the cache's tiles evenly:
// the tiles of all (request, row tile, head) items stand in one line, each
// warp takes the same length of it.  A warp that covers an item whole writes
// o; parts go to the workspace as (max, sum, o) and a second kernel joins them
// in order.
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
constexpr int kRows = 16;       // rows of a tile
constexpr int kTok = 16;        // tokens of a tile
constexpr float kTop = 15.0f;   // log2 of the largest weight in the second product
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kJoinRows = 4;    // CTAs of the joining kernel per split item

// Blocks per SM and stages per warp: enough copies in flight on an SM (over
// 100 KB) at the registers that the accumulators leave.
__host__ __device__ constexpr int blocks_per_sm(int D, bool f32) { return D == 256 ? 1 : (D == 128 ? (f32 ? 2 : 3) : 4); }
__host__ __device__ constexpr int stages_of(int D) { return D == 256 ? 4 : (D == 128 ? 4 : 6); }

struct Plan {             // how the line of tiles is shared out
  int64_t units, per;     // tiles in all, tiles per warp
};

// Rows, tiles per row tile, and row tiles of a request.
struct Request {
  int64_t row0;     // first row of the batch
  int n;            // rows
  int64_t keys;     // tokens that the table can hold of it
  int64_t pos0;     // position of its first row (negative where it has fewer tokens than rows)
  int64_t tiles;    // 16-token tiles of one item
  int64_t items;    // row tiles x cached heads
};

__device__ __forceinline__ Request request_of(const KvAttentionArgs& a, int b) {
  Request r;
  const int64_t lo = min(max((int64_t)a.row_start[b], (int64_t)0), a.T);
  const int64_t hi = min(max((int64_t)a.row_start[b + 1], lo), a.T);
  r.row0 = lo;
  r.n = (int)(hi - lo);
  const int64_t total = a.total[b], limit = a.width * a.block;
  r.pos0 = total - r.n;
  r.keys = min(max(total, (int64_t)0), limit);
  r.tiles = max((r.keys + kTok - 1) / kTok, (int64_t)1);  // a request without tokens still writes its zeros
  r.items = ((int64_t)r.n * (a.Hq / a.Hkv) + kRows - 1) / kRows * a.Hkv;
  return r;
}

// Prefix sums of the requests' tiles in shared memory, by the whole CTA.
__device__ __forceinline__ Plan plan_line(const KvAttentionArgs& a, int64_t* start, int64_t* warp_sums, int64_t workers,
                                          int min_tiles) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int64_t s = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b);
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
  Plan p;
  p.units = all;
  p.per = max((all + workers - 1) / workers, (int64_t)min_tiles);
  return p;
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

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// two of a word's bytes (selector: byte, 0x64, byte, 0x64) as fp16 1024 + q,
// then minus 1024 + z: the centred codes, exactly
__device__ __forceinline__ uint32_t codes2(uint32_t w, uint32_t sel, uint32_t minus) {
  return hadd2(__byte_perm(w, 0x64646464u, sel), minus);
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

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

__device__ __forceinline__ void store4(void* o, bool bf16, int64_t at, float4 v) {
  if (bf16) {
    uint32_t x, y;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(v.y), "f"(v.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(v.w), "f"(v.z));
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(o) + at) = make_uint2(x, y);
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(o) + at) = v;
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

// Sixteen consecutive (D = 32: eight) values of a query row per lane and
// 64-value part, as fragments of the first product: lane c of a quad holds
// values 64 j + 16 c .. + 15 (D = 32: 8 c .. + 7), four per 16-deep step, the
// same order in which it reads the codes of a token.
template <int D, bool F32>
struct Query {
  static constexpr int kSteps = D / 16;
  uint32_t hi[kSteps][4];
  uint32_t lo[F32 ? kSteps : 1][4];
  float sum[2];     // sum of the row's values as they enter the product
  float scale[2];   // what a product of them is to be multiplied by (log2 units, without u_k)
};

template <int D, bool F32>
__device__ __forceinline__ void load_query(const KvAttentionArgs& a, const Request& r, int64_t row_tile, int h, int lane,
                                           float scale, Query<D, F32>& q) {
  constexpr int kPer = D >= 64 ? 16 : 8;       // values per lane and part
  constexpr int kParts = D >= 64 ? D / 64 : 1;
  const int g = a.Hq / a.Hkv;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int64_t row = row_tile * kRows + (lane >> 2) + 8 * half;
    const bool live = row < (int64_t)r.n * g;
    const int64_t at = live ? (r.row0 + row / g) * a.q_stride + ((int64_t)h * g + row % g) * D : 0;
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
    top = quad_max(top);
    // the row's largest value into [2^10, 2^11): a power of two, its inverse
    // kept for the scores (zero and tiny rows are scaled as 2^-100 would be)
    const int e = max((int)(__float_as_uint(top) >> 23) - 127, -100);
    const float up = __uint_as_float((uint32_t)(127 + 10 - e) << 23), down = __uint_as_float((uint32_t)(127 - 10 + e) << 23);
    const float sign = scale < 0.0f ? -up : up;
    q.scale[half] = fabsf(scale) * kLog2e * down;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kParts; ++j)
#pragma unroll
      for (int s = 0; s < kPer / 4; ++s)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float x = v[j][4 * s + 2 * k] * sign, y = v[j][4 * s + 2 * k + 1] * sign;
          const uint32_t hi = pack2(x, y);
          q.hi[j * (kPer / 4) + s][half + 2 * k] = hi;
          sum += half_lo(hi) + half_hi(hi);
          if constexpr (F32) {
            const uint32_t lo = pack2(x - half_lo(hi), y - half_hi(hi));
            q.lo[j * (kPer / 4) + s][half + 2 * k] = lo;
            sum += half_lo(lo) + half_hi(lo);
          }
        }
    q.sum[half] = quad_sum(sum);
  }
}

// (max, sum, o) of a part of an item: slot 2 w is the part that warp w begins
// in the middle of an item, slot 2 w + 1 the one that it leaves unfinished.
struct Parts {
  float* o;    // [slots][16][D]
  float2* ml;  // [slots][16]
};

__host__ __device__ inline Parts parts_of(void* workspace, int64_t workers, int D) {
  Parts p;
  p.o = reinterpret_cast<float*>(workspace);
  p.ml = reinterpret_cast<float2*>(p.o + (size_t)workers * 2 * kRows * D);
  return p;
}

template <int D, bool F32>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(D, F32))
kv_attention_kernel(const KvAttentionArgs a, const int min_tiles) {
  constexpr int kStages = stages_of(D);
  constexpr int kHalf = kTok * D;           // bytes of one of K and V in a stage
  constexpr int kStage = 2 * kHalf;
  constexpr int kSegs = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t warp_sums[kWarps];
  int64_t* start = reinterpret_cast<int64_t*>(smem + kWarps * kStages * kStage);

  // programmatic dependent of the stream's previous kernel: nothing is read before it has ended, and the joining
  // kernel may start from here on (it waits for this one before it reads the parts)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int64_t workers = (int64_t)gridDim.x * kWarps;
  const Plan plan = plan_line(a, start, warp_sums, workers, min_tiles);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3;
  const int64_t worker = (int64_t)blockIdx.x * kWarps + warp;
  int64_t u = worker * plan.per;
  const int64_t u_end = min(u + plan.per, plan.units);
  const Parts parts = parts_of(a.workspace, workers, D);
  uint8_t* ring = smem + warp * kStages * kStage;
  const uint32_t ring_addr = smem_u32(ring);
  const int block_shift = 31 - __clz(a.block);
  const int L = (1 << a.bits) - 1;
  const uint32_t minus = 0xE400E400u | ((uint32_t)(1 << (a.bits - 1)) * 0x10001u);  // -(1024 + z), twice
  const float scale = a.scale ? *a.scale : rsqrtf((float)D);
  const int g = a.Hq / a.Hkv;

  while (u < u_end) {
    const int b = find_request(start, a.B, u);
    const Request r = request_of(a, b);
    const int64_t in_request = u - start[b];
    const int64_t item = in_request / r.tiles;
    const int64_t t0 = in_request - item * r.tiles;               // first tile of the item here
    const int64_t t1 = min(r.tiles, t0 + (u_end - u));            // end of the tiles here
    const int64_t row_tile = item / a.Hkv;
    const int h = (int)(item - row_tile * a.Hkv);
    u += t1 - t0;

    Query<D, F32> q;
    load_query<D, F32>(a, r, row_tile, h, lane, scale, q);
    // tokens that this lane's two rows, and the tile's first and last row, see
    int64_t sees[2];
#pragma unroll
    for (int half = 0; half < 2; ++half)
      sees[half] = min(r.pos0 + (row_tile * kRows + (lane >> 2) + 8 * half) / g + 1, r.keys);
    const int64_t all_see = min(r.pos0 + row_tile * kRows / g + 1, r.keys);
    const int64_t last_row = min(row_tile * kRows + kRows, (int64_t)r.n * g) - 1;
    const int64_t any_sees = min(r.pos0 + last_row / g + 1, r.keys);
    const int64_t seen_tiles = any_sees > 0 ? (any_sees + kTok - 1) / kTok : 0;
    const int n = (int)(min(t1, seen_tiles) - t0);                // tiles to work on (none: n <= 0)

    float o[kSegs][2][4];
#pragma unroll
    for (int s = 0; s < kSegs; ++s)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[s][p][i] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, w_sum[2] = {0.0f, 0.0f};

    // blocks and scales of 32 tiles at a time, one per lane, a group ahead
    int id_now = -1, id_next = -1;
    float ku_now = 0.0f, vu_now = 1.0f, ku_next = 0.0f, vu_next = 1.0f;
    auto look_up = [&](int first, int& id, float& ku, float& vu) {
      const int i = first + lane;
      id = -1;
      ku = 0.0f;
      vu = 1.0f;
      if (i < n) {
        const int v = a.table[(int64_t)b * a.width + (((t0 + i) * kTok) >> block_shift)];
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

    auto issue = [&](int i, int group) {
      if (i < n) {
        const int id = __shfl_sync(0xffffffffu, (i >> 5) == group ? id_now : id_next, i & 31);
        if (id >= 0) {
          const int64_t tok = (t0 + i) * kTok;
          const int64_t from = (((int64_t)id * a.Hkv + h) * a.block + (tok & (a.block - 1))) * D;
          const uint32_t to = ring_addr + (uint32_t)(i % kStages) * kStage;
#pragma unroll
          for (int x = 0; x < kHalf / 512 + (kHalf % 512 != 0); ++x) {
            const int piece = x * 32 + lane, t = piece / (D / 16), p = piece % (D / 16);
            if (kHalf % 512 == 0 || piece < kHalf / 16) {
              cp_async16(to + k_place<D>(t, p), a.k_codes + from + piece * 16);
              cp_async16(to + kHalf + v_place<D>(t, p), a.v_codes + from + piece * 16);
            }
          }
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, 0);

    for (int i = 0; i < n; ++i) {
      if (i != 0 && (i & 31) == 0) {
        id_now = id_next;
        ku_now = ku_next;
        vu_now = vu_next;
        look_up(i + 32, id_next, ku_next, vu_next);
      }
      cp_wait<kStages - 2>();
      __syncwarp();  // tile i has landed for all lanes, and all have read the stage that the next copies overwrite
      issue(i + kStages - 1, i >> 5);

      const uint8_t* k_tile = ring + (i % kStages) * kStage;
      const uint32_t v_tile = ring_addr + (uint32_t)(i % kStages) * kStage + kHalf;
      float s[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
        for (int x = 0; x < 4; ++x) s[nt][x] = 0.0f;
        const int tok = nt * 8 + (lane >> 2);
        if constexpr (D >= 64) {
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            const uint4 w = *reinterpret_cast<const uint4*>(k_tile + k_place<D>(tok, 4 * j + c));
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t b0 = codes2(ww[x], 0x4140u, minus), b1 = codes2(ww[x], 0x4342u, minus);
              mma(s[nt], q.hi[4 * j + x], b0, b1);
              if constexpr (F32) mma(s[nt], q.lo[4 * j + x], b0, b1);
            }
          }
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(k_tile + tok * D + 8 * c);
          const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t b0 = codes2(ww[x], 0x4140u, minus), b1 = codes2(ww[x], 0x4342u, minus);
            mma(s[nt], q.hi[x], b0, b1);
            if constexpr (F32) mma(s[nt], q.lo[x], b0, b1);
          }
        }
      }

      const bool here = __shfl_sync(0xffffffffu, id_now, i & 31) >= 0;
      const float ku = __shfl_sync(0xffffffffu, ku_now, i & 31), vu = __shfl_sync(0xffffffffu, vu_now, i & 31);
      // a block whose values are all zero (below 1e-30) takes part in the sum alone
      const bool zero = !(vu >= 1e-30f);
      const float lu = __log2f(zero ? 1e-30f : vu), inv_vu = ex2(-lu);
      const int64_t tok0 = (t0 + i) * kTok;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float f = 2.0f * q.scale[half] * ku, f0 = q.sum[half] * q.scale[half] * ku;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) s[nt][2 * half + x] = fmaf(s[nt][2 * half + x], f, f0);
      }
      if (!here || tok0 + kTok > all_see) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (!here || tok0 + nt * 8 + 2 * c + x >= sees[half]) s[nt][2 * half + x] = -INFINITY;
      }
      float grow[2], off[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float top = fmaxf(fmaxf(s[0][2 * half], s[0][2 * half + 1]), fmaxf(s[1][2 * half], s[1][2 * half + 1]));
        top = fmaxf(m[half], quad_max(top) + lu);
        // a row that has seen nothing keeps -inf, with 0 in its place in the differences
        const float base = top == -INFINITY ? 0.0f : top;
        grow[half] = ex2(m[half] - base);
        off[half] = lu + kTop - base;
        m[half] = top;
      }
      if (__any_sync(0xffffffffu, grow[0] != 1.0f || grow[1] != 1.0f)) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          l[half] *= grow[half];
          w_sum[half] *= grow[half];
#pragma unroll
          for (int x = 0; x < kSegs; ++x)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              o[x][p][2 * half] *= grow[half];
              o[x][p][2 * half + 1] *= grow[half];
            }
        }
      }
      uint32_t w_hi[4], w_lo[4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float tile_sum = 0.0f;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float x = ex2(s[nt][2 * half] + off[half]), y = ex2(s[nt][2 * half + 1] + off[half]);
          tile_sum += x + y;
          const uint32_t hi = zero ? 0u : pack2(x, y);
          w_hi[half + 2 * nt] = hi;
          if constexpr (F32) w_lo[half + 2 * nt] = zero ? 0u : pack2(x - half_lo(hi), y - half_hi(hi));
        }
        if (!zero) w_sum[half] += tile_sum;
        l[half] = fmaf(tile_sum, inv_vu, l[half]);
      }
#pragma unroll
      for (int x = 0; x < kSegs; x += 2) {
        // four 8 x 16-byte matrices: tokens 0-7 and 8-15 at two neighbouring 16-byte columns
        const int tok = lane & 15, piece = x + (lane >> 4);
        uint32_t w[4];
        ldmatrix4t(v_tile + v_place<D>(tok, piece), w);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          // a register holds two tokens at two columns: even columns and odd ones are products of their own
          const uint32_t e0 = codes2(w[2 * y], 0x4240u, minus), e1 = codes2(w[2 * y + 1], 0x4240u, minus);
          const uint32_t d0 = codes2(w[2 * y], 0x4341u, minus), d1 = codes2(w[2 * y + 1], 0x4341u, minus);
          mma(o[x + y][0], w_hi, e0, e1);
          mma(o[x + y][1], w_hi, d0, d1);
          if constexpr (F32) {
            mma(o[x + y][0], w_lo, e0, e1);
            mma(o[x + y][1], w_lo, d0, d1);
          }
        }
      }
    }
    cp_wait<0>();
    __syncwarp();  // the ring is free for the next item

    const bool whole = t0 == 0 && t1 == r.tiles;
    const int64_t slot = worker * 2 + (t0 == 0 ? 1 : 0);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float sum = quad_sum(l[half]), ws = quad_sum(w_sum[half]);
      const int64_t row = row_tile * kRows + (lane >> 2) + 8 * half;
      if (row >= (int64_t)r.n * g) continue;
      const int in_tile = (lane >> 2) + 8 * half;
      const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
      const int64_t at = ((r.row0 + row / g) * a.Hq + (int64_t)h * g + row % g) * D;
#pragma unroll
      for (int x = 0; x < kSegs; ++x) {
        float4 v;
        v.x = fmaf(2.0f, o[x][0][2 * half], ws);
        v.y = fmaf(2.0f, o[x][1][2 * half], ws);
        v.z = fmaf(2.0f, o[x][0][2 * half + 1], ws);
        v.w = fmaf(2.0f, o[x][1][2 * half + 1], ws);
        if (whole) {
          v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
          store4(a.o, a.o_bf16, at + 16 * x + 4 * c, v);
        } else {
          *reinterpret_cast<float4*>(parts.o + (slot * kRows + in_tile) * D + 16 * x + 4 * c) = v;
        }
      }
      if (!whole && c == 0) parts.ml[slot * kRows + in_tile] = make_float2(m[half], sum);
    }
  }
}

// Joins the parts of each item that more than one warp worked on: the CTAs of
// place w look at the border between warps w - 1 and w, and where it is the
// first border inside an item, they join that item (rows y, y + 4, ...).
template <int D>
__global__ void __launch_bounds__(kThreads)
kv_attention_join_kernel(const KvAttentionArgs a, const int64_t workers, const int min_tiles) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t warp_sums[kWarps];
  __shared__ float red[kWarps][D + 1];
  __shared__ float tops[kWarps];
  int64_t* start = reinterpret_cast<int64_t*>(smem);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Plan plan = plan_line(a, start, warp_sums, workers, min_tiles);
  const int64_t w0 = (int64_t)blockIdx.x, border = (w0 + 1) * plan.per;
  bool mine = border < plan.units;
  Request r;
  int64_t item = 0, i0 = 0, i1 = 0;
  if (mine) {
    const int b = find_request(start, a.B, border);
    r = request_of(a, b);
    item = (border - start[b]) / r.tiles;
    i0 = start[b] + item * r.tiles;
    i1 = i0 + r.tiles;
    mine = i0 < border && i0 >= w0 * plan.per;  // the item begins in warp w0's share
  }
  // the parts are the previous kernel's; every CTA waits, so that the end of this grid is the end of that one too
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!mine) return;
  const int64_t w1 = (i1 - 1) / plan.per;
  const int count = (int)(w1 - w0 + 1);
  const Parts parts = parts_of(a.workspace, workers, D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = a.Hq / a.Hkv;
  const int64_t row_tile = item / a.Hkv;
  const int h = (int)(item - row_tile * a.Hkv);
  constexpr int V = D / 32;
  for (int y = blockIdx.y; y < kRows; y += kJoinRows) {
    const int64_t row = row_tile * kRows + y;
    if (row >= (int64_t)r.n * g) break;
    auto slot = [&](int p) { return (p == 0 ? w0 * 2 + 1 : (w0 + p) * 2) * kRows + y; };
    float top = -INFINITY;
    for (int p = threadIdx.x; p < count; p += kThreads) top = fmaxf(top, parts.ml[slot(p)].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    __syncthreads();
    if (lane == 0) tops[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, tops[w]);
    if (top == -INFINITY) top = 0.0f;
    float acc[V], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll 4
    for (int p = warp; p < count; p += kWarps) {
      const int64_t at = slot(p);
      const float2 ml = parts.ml[at];
      const float f = ex2(ml.x - top);
      sum = fmaf(f, ml.y, sum);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(f, parts.o[at * D + i * 32 + lane], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) red[warp][i * 32 + lane] = acc[i];
    if (lane == 0) red[warp][D] = sum;
    __syncthreads();
    const int64_t at = ((r.row0 + row / g) * a.Hq + (int64_t)h * g + row % g) * D;
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += red[w][D];
    const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
    for (int d = 4 * threadIdx.x; d < D; d += 4 * kThreads) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        v.x += red[w][d];
        v.y += red[w][d + 1];
        v.z += red[w][d + 2];
        v.w += red[w][d + 3];
      }
      v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
      store4(a.o, a.o_bf16, at + d, v);
    }
  }
}

constexpr int kMinTiles = 4;

template <int D, bool F32>
cudaError_t launch(const KvAttentionArgs& a, cudaStream_t stream) {
  const unsigned grid = (unsigned)(sm100_host::sm_count() * blocks_per_sm(D, F32));
  const size_t scan = (size_t)(a.B + 1) * 8;
  constexpr int ring = kWarps * stages_of(D) * 2 * kTok * D;
  static std::atomic<bool> done[sm100_host::kMaxDevices];
  cudaError_t e = sm100_host::ensure_smem(kv_attention_kernel<D, F32>, ring + (kMaxRequests + 1) * 8, done);
  if (e != cudaSuccess) return e;
  e = sm100_host::launch_pdl(kv_attention_kernel<D, F32>, grid, kThreads, ring + scan, stream, 1, a, kMinTiles);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid * kWarps, kJoinRows, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = scan;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv_attention_join_kernel<D>, a, (int64_t)grid * kWarps, kMinTiles);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const KvAttentionArgs& a, cudaStream_t stream) {
  return a.q_bf16 ? launch<D, false>(a, stream) : launch<D, true>(a, stream);
}

}  // namespace

size_t kv_attention_workspace(int64_t T, int Hq, int Hkv, int D, int B) {
  (void)T, (void)Hq, (void)Hkv, (void)B;
  const size_t workers = (size_t)sm100_host::sm_count() * blocks_per_sm(D, false) * kWarps;
  return (workers * 2 * kRows * (D * 4 + 8) + 255) & ~(size_t)255;
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
