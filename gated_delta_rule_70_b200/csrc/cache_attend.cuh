// What the two kernels of the attention over the paged 8-bit cache share: how the work is laid out over the
// blocks, the widening of codes, and the join of an item's parts.
//
// A work item is one (sequence, tile of query rows, key / value head); a query row is a (new token, query
// head of the group) pair, so grouped heads share every cached byte that is read.  The items' tiles of cached
// tokens form one line, which the grid's blocks share out equally: a long sequence spreads over many blocks, a
// block takes several short ones.  An item that lies in several blocks leaves partial results (running
// maximum, sum, unnormalised output) in the workspace, and a second kernel joins them in the order of the
// blocks, so results do not depend on timing.
//
// Scales: with ks, vs the page's scales, weights are kept as w_j = exp2(s_j + log2 vs_j - m), m a running
// reference for s_j + log2 vs_j some powers of two below their maximum, so that w fills fp16's range from the top,
// and the sum takes w_j / vs_j.  A query row is brought to [2^14, 2^15) by a power of two first, so its fp16 copy
// is exact for bf16 inputs.
#pragma once

#include <cuda_fp16.h>

#include "kda_common.cuh"
#include "kda_internal.h"
#include "tma_host.h"
#include "umma.cuh"

namespace kda {
namespace attend {

using namespace umma;

constexpr int kBlocks = 148;                          // one per SM (shared memory allows one)
constexpr int kLensInSmem = 2048;

struct StageInfo {          // per 16 tokens of the stage
  float kf[4];              // key scale
  float lv[4];              // log2 of the value scale
  float iv[4];              // 1 / value scale
  uint8_t valid[4];         // 1: loaded, and 2: the value scale is NaN (kNanScale)
  uint32_t turn;            // of the tile that the stage was given last (~0: none)
  uint32_t pad[2];
};

// A NaN value scale is no factor that weights and sums could carry: its values count as NaN codes, at a scale of
// 2^-60, so that the rows that see one of them are NaN and nothing else is.
constexpr uint32_t kNanScale = 2;

struct AttendParams {
  int N, T, Hq, Hk, G;      // G: query heads per key / value head
  int P, log_page, max_pages, num_pages;
  int RT;                   // row tiles per (sequence, key / value head)
  int whole;                // items are not split: block b takes items b, b + grid, ...
  int box, boxes;           // tokens per TMA box, boxes per stage
  int64_t q_stride;
  float scale;
  const void *q;
  const float *k_scale, *v_scale;
  const int32_t *table, *lens;
  void *o;
  float *lse;
  int *status;
  int4 *desc;               // workspace: per block the split item that begins in it
  float *parts;             // workspace: per block two partial results
  uint32_t polls;           // of an ordinary wait
  int expire;               // failure test: one of the readers of each item gives up before its first tile
  CUtensorMap map_k, map_v;
};

__device__ __forceinline__ int clamp_len(int len, int cap) { return len < 0 ? 0 : (len > cap ? cap : len); }

// Tokens that the last row of row tile rt sees, and its tiles (one at least, so that every item is somebody's).
__device__ __forceinline__ int visible(int len, int T, int G, int rows, int rt) {
  const int last = min(T - 1, ((rt + 1) * rows - 1) / G);
  return len - T + last + 1;
}
__device__ __forceinline__ int tiles_of(int seen, int tile) { return seen <= tile ? 1 : (seen + tile - 1) / tile; }

// The items of this block, one after another: (sequence, row tile, head) and a range of its tiles.  On the
// line an item is LEAD places longer than its tiles: what its own start and end cost, in tiles.
template <int R, int TILE, int LEAD> struct Walker {
  const AttendParams *pp;
  const int32_t *lens;       // shared memory copy, or pp->lens
  int64_t left;              // places still to take (split) / the item (whole)
  uint32_t stop;             // the line's place behind the current item
  int n, rt, h, len, tiles;
  int t0, t1;                // tile range of the current item in this block
  bool starts, ends;         // the range holds the item's first / last tile

  __device__ Walker(const AttendParams &p_, const int32_t *lens_) : pp(&p_), lens(lens_) {}
  __device__ void enter() {
    len = clamp_len(lens[n], pp->max_pages * pp->P);
    tiles = tiles_of(visible(len, pp->T, pp->G, R, rt), TILE);
  }
  // split: `first` is the block's first place on the line, `sums` the exclusive sums of chunks of `per`
  // (sequence, row tile) pairs
  __device__ bool begin_split(uint32_t first, int count, const uint32_t *sums, int per) {
    left = count;
    if (count <= 0) return false;
    int lo = 0, hi = 255;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sums[mid] <= first) lo = mid; else hi = mid - 1;
    }
    uint32_t at = first - sums[lo];
    const int m = lo * per;
    n = m / pp->RT; rt = m - n * pp->RT;
    enter();
    while (at >= (uint32_t)(tiles + LEAD) * pp->Hk) {
      at -= (uint32_t)(tiles + LEAD) * pp->Hk;
      if (++rt == pp->RT) { rt = 0; ++n; }
      enter();
    }
    h = (int)(at / (uint32_t)(tiles + LEAD));
    at -= (uint32_t)(h * (tiles + LEAD));
    stop = first - at;
    return take((int)at);
  }
  // From the item's place `at` on; false where the block's share ends before the item's first tile.
  __device__ bool take(int at) {
    const int to = left < tiles + LEAD - at ? at + (int)left : tiles + LEAD;
    left -= to - at;
    stop += tiles + LEAD;
    t0 = max(at - LEAD, 0); t1 = to - LEAD;
    starts = t0 == 0; ends = t1 == tiles;
    return t1 > 0;
  }
  __device__ bool begin_whole(int64_t item) {
    if (item >= (int64_t)pp->N * pp->RT * pp->Hk) return false;
    const int64_t m = item / pp->Hk;
    h = (int)(item - m * pp->Hk);
    n = (int)(m / pp->RT); rt = (int)(m - (int64_t)n * pp->RT);
    enter();
    left = item; t0 = 0; t1 = tiles; starts = ends = true;
    return true;
  }
  __device__ bool next() {
    if (pp->whole) return begin_whole(left + gridDim.x);
    if (left <= 0) return false;
    if (++h == pp->Hk) {
      h = 0;
      if (++rt == pp->RT) { rt = 0; ++n; }
      enter();
    }
    return take(0);
  }
};

// Every block lays out the line by itself: the places before each chunk of (sequence, row tile) pairs go to
// sums[0 .. 255] (sums: 266 words), the block's own range of the line is [first, first + sums[264]).  At
// least `least` places a block.
struct Line { uint32_t first, share; int per; };
template <int R, int TILE, int LEAD>
__device__ __forceinline__ Line lay_out(const AttendParams &p, const int32_t *lens, uint32_t *sums, uint32_t least) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, cap = p.max_pages * p.P;
  Line line;
  line.per = (p.N * p.RT + 255) / 256;
  uint32_t sum = 0;
  if (threadIdx.x < 256) {
    const int m0 = threadIdx.x * line.per, m1 = min(m0 + line.per, p.N * p.RT);
    int n = m0 / p.RT, rt = m0 - n * p.RT;
    for (int m = m0; m < m1; ++m) {
      sum += tiles_of(visible(clamp_len(lens[n], cap), p.T, p.G, R, rt), TILE) + LEAD;
      if (++rt == p.RT) { rt = 0; ++n; }
    }
    sum *= p.Hk;
    uint32_t run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(~0u, run, o);
      if (lane >= o) run += up;
    }
    sums[threadIdx.x] = run - sum;                    // within the warp
    if (lane == 31) sums[256 + warp] = run;
  }
  __syncthreads();
  uint32_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const uint32_t x = sums[256 + w];
    if (w < warp) before += x;
    total += x;
  }
  if (threadIdx.x < 256) sums[threadIdx.x] += before;
  line.share = (total + gridDim.x - 1) / gridDim.x;
  line.share = line.share < least ? least : line.share;
  line.first = line.share * blockIdx.x;
  if (threadIdx.x == 0) sums[264] = line.first < total ? min(line.share, total - line.first) : 0;
  __syncthreads();
  return line;
}

// Two e4m3 codes (the low / high half of w) to fp16, exactly.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
// fp16 pairs; what is beyond fp16's range (a weight whose reference, with scores from 2^24 on, was rounded by more than
// fp16 has room for above 2^15) becomes the largest.
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
// The output row of query row r of a (sequence, key / value head); rows are counted in 32 bits.
__device__ __forceinline__ int out_row(const AttendParams &p, int n, int h, int r) {
  const int t = r / p.G;
  return (n * p.T + t) * p.Hq + h * p.G + (r - t * p.G);
}
// A finished row's factor on its output, and its lse.
__device__ __forceinline__ float row_factor(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }   // no weight: o = 0
__device__ __forceinline__ void store_lse(const AttendParams &p, int row, float m, float sum) {
  if (p.lse != nullptr) p.lse[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
}
// Four channels of a finished row.
template <typename IO, int D>
__device__ __forceinline__ void store_row(const AttendParams &p, int row, int q, float4 x, float f) {
  IO *dst = static_cast<IO *>(p.o) + (int64_t)row * D + 4 * q;
  if constexpr (sizeof(IO) == 2) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x * f, x.y * f), b = __floats2bfloat162_rn(x.z * f, x.w * f);
    *reinterpret_cast<uint2 *>(dst) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                                 *reinterpret_cast<const uint32_t *>(&b));
  } else {
    *reinterpret_cast<float4 *>(dst) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
  }
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
// The whole warp waits for a phase; false if the wait ran out.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase, uint32_t polls) {
  return __all_sync(~0u, mbar_wait_bounded(bar, phase & 1, polls));
}
// exp2 of a difference from a maximum that may be -inf (no weight yet).
__device__ __forceinline__ float fade(float m, float top) { return m == -INFINITY ? 0.f : ex2(m - top); }

// Joins the parts of the item that begins in block blockIdx.x and ends in a later one: four warps take
// every fourth part of a row, a lane D / 32 channels.  A latency of dependent loads (desc, maxima, sums, outputs),
// 4 to 6 us behind the last block; set up while the attention runs, which saves a launch's 3 us.
template <typename IO, int D, int R>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ AttendParams p) {
  constexpr int kPart = R * D + 2 * R, V = D / 32;
  __shared__ float factor[kBlocks], red[4];
  __shared__ __align__(16) float acc[4][D];
  cudaGridDependencySynchronize();
  const int4 d = p.desc[blockIdx.x];
  if (d.x < 0) return;
  const int parts = d.w - (int)blockIdx.x + 1, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  auto part = [&](int i) { return p.parts + ((int64_t)(blockIdx.x + i) * 2 + (i == 0)) * kPart; };
  for (int row = blockIdx.y; row < R && d.y * R + row < p.T * p.G; row += gridDim.y) {
    float M = -INFINITY, sum = 0.f;
    for (int i = threadIdx.x; i < parts; i += 128) M = fmaxf(M, factor[i] = part(i)[R * D + row]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
    if (lane == 0) red[warp] = M;
    __syncthreads();
    M = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    __syncthreads();
    for (int i = threadIdx.x; i < parts; i += 128) {
      const float f = fade(factor[i], M);
      factor[i] = f;
      sum = fmaf(f, part(i)[R * D + R + row], sum);   // (0 of a part without weight, NaN of one whose scores all are)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = (red[0] + red[1]) + (red[2] + red[3]);
    float x[V] = {};
#pragma unroll 8
    for (int i = warp; i < parts; i += 4) {
      const float f = factor[i];
      const float *y = part(i) + row * D + lane * V;
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = fmaf(f, y[e], x[e]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) acc[warp][lane * V + e] = x[e];
    __syncthreads();
    if (threadIdx.x < D / 4) {
      float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float4 y = *reinterpret_cast<const float4 *>(&acc[w][4 * threadIdx.x]);
        r.x += y.x; r.y += y.y; r.z += y.z; r.w += y.w;
      }
      const int to = out_row(p, d.x, d.z, d.y * R + row);
      store_row<IO, D>(p, to, threadIdx.x, r, row_factor(sum));
      if (threadIdx.x == 0) store_lse(p, to, M, sum);
    }
    __syncthreads();
  }
}

// The join, set up while the attention still runs (it waits for the whole grid before it reads anything).  Up to
// 32 rows of an item side by side: with 16 the items of 128 rows took 2 to 4 us more, with 64 no less.
template <typename IO, int D, int R>
cudaError_t launch_join(const AttendParams &p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kBlocks, R < 32 ? R : 32);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_join_kernel<IO, D, R>, p);
}

// The tensor maps of the two caches: boxes of p.box tokens.
inline bool encode_maps(AttendParams &p, const kda_cache &c, CUtensorMapSwizzle swizzle) {
  const uint64_t rows = (uint64_t)c.num_pages * c.num_kv_heads * c.page_tokens;
  const int D = c.head_dim;
  return encode_rows(&p.map_k, c.k_cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, D, D, p.box, D, swizzle) &&
         encode_rows(&p.map_v, c.v_cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, D, D, p.box, D, swizzle);
}

// The kernel for many query rows (kda_cache_attend_wide.cu): bf16 calls with more than wide_from(D) rows per key /
// value head (item_rows has both sides' times).
constexpr int wide_from(int D) { return D == 64 ? 32 : 16; }
constexpr int kWideTile = 128, kWideItem = 128;                  // tokens of a tile; rows of an item
constexpr int kWideStage = 64;                                   // tokens of a stage
// What an item's own start and end cost it, in tiles (64 sequences of up to 12345 tokens, 4 new ones, 8 query
// heads each: 131 us without it, 121 with 2, 115 with 4, 119 with 6).
constexpr int kWideLead = 4;
cudaError_t launch_wide(AttendParams p, const kda_cache &c, int64_t items, cudaStream_t stream);

}  // namespace attend
}  // namespace kda
