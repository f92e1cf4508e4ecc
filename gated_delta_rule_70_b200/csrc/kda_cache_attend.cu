// Attention over the paged 8-bit cache.
//
// A work item is one (sequence, tile of query rows, key / value head); a query row is a (new token, query
// head of the group) pair, so grouped heads share every cached byte that is read.  The items' tiles (32
// cached tokens of 128 channels, or 64 of 64) form one line, which the grid's blocks share out equally: a long sequence spreads over
// many blocks, a block takes several short ones.  An item that lies in several blocks leaves partial
// results (running maximum, sum, unnormalised output) in the workspace, and a second kernel joins them
// in the order of the blocks, so results do not depend on timing.
//
// A block: two or three producer warps bring tiles by TMA into a ring of 8 KB stages (one box per page, rows
// swizzled in shared memory), one or two bring the next item's queries as fp16 fragments, and twelve
// consumer warps each own 16 query rows (an m-tile) and every KL-th tile, with a running maximum, sum
// and output of their own, so no warp waits for another until the item ends.
//
// One warp and tile: S = Q K^T and O += P V by mma.sync m16n8k16 with fp16 operands and fp32
// accumulation.  e4m3 codes are exact in fp16.  The contraction's order is free, so the channels of a
// key row go to the lanes as the 16-byte pieces they load; the order of the 8 tokens of an n-tile is
// free too and is sigma(n) = n (even), n ^ 4 (odd: 1 -> 5, 3 -> 7, 5 -> 1, 7 -> 3), which makes the key
// loads (two tokens x four pieces per phase) and the value loads (four tokens x two pieces) free of
// bank conflicts under the hardware's swizzle; the accumulators of S are then the A operand of P V as they lie.
//
// Scales: with ks, vs the page's scales, weights are kept as w_j = exp2(s_j + log2 vs_j - m), m the
// running maximum of s_j + log2 vs_j, so w is at most 1 and holds in fp16 whatever the scales are, and the
// sum takes w_j / vs_j.  A query row is brought to [2^14, 2^15) by a power of two first, so its fp16
// copy is exact for bf16 inputs (fp32 inputs and their weights go as two fp16 parts each).
#include <cuda_fp16.h>

#include "kda_common.cuh"
#include "kda_internal.h"
#include "tma_host.h"
#include "umma.cuh"

namespace kda {
namespace {

using namespace umma;

constexpr int kBlocks = 148;                   // one per SM (shared memory allows one)
constexpr int kConsumers = 12;                 // warps
constexpr int kThreads = (kConsumers + 4) * 32;
// Registers: 16 warps leave 128 a thread; the producer's warpgroup gives up 48 of them for the three
// consumer warpgroups (3 x 144 + 80 = 4 x 128), whose output fragments would spill otherwise.
constexpr int kProducerRegs = 80, kConsumerRegs = 144;
constexpr int kLensInSmem = 2048;
template <int D> constexpr int kTile = 4096 / D;      // cached tokens per stage: 4 KB of keys, 4 KB of values

struct StageInfo {          // per 16 tokens of the stage
  float kf[4];              // key scale
  float lv[4];              // log2 of the value scale
  float iv[4];              // 1 / value scale
  uint8_t valid[4];         // loaded
  uint32_t turn;            // of the tile that the stage was given last
  uint32_t pad[2];
};

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
  uint32_t polls;
  CUtensorMap map_k, map_v;
};

template <typename IO, int D, int MT> struct Layout {
  static constexpr int kRows = 16 * MT, kLanes = kConsumers / MT;   // query rows per item, tiles at a time
  static constexpr int kHalf = (kLanes + 1) / 2;                    // of them, those that write the merge buffer last
  static constexpr int kStages = MT == 1 ? 18 : MT == 2 ? 16 : 10;
  static constexpr int kLoaders = MT < 2 ? MT : 2, kProducers = 4 - kLoaders;   // warps for queries and for tiles
  static constexpr uint32_t kOwn = kStages / kProducers;            // stages of a producer
  static constexpr uint32_t kQParts = sizeof(IO) / 2;               // fp16 parts of a query
  static constexpr uint32_t kQSlot = MT * kQParts * (D / 16) * 32 * 16;     // fragments of one item
  static constexpr uint32_t kMerge = kStages * 8192;                // [kHalf][kRows][D] fp32
  static constexpr uint32_t kQ = kMerge + kHalf * kRows * D * 4;    // two slots
  static constexpr uint32_t kQFactor = kQ + 2 * kQSlot;             // two slots of [kRows]
  static constexpr uint32_t kStats = kQFactor + 2 * kRows * 4;      // [kConsumers][16] x (m, l)
  static constexpr uint32_t kInfo = kStats + kConsumers * 16 * 8;
  static constexpr uint32_t kBars = kInfo + kStages * (uint32_t)sizeof(StageInfo);
  static constexpr uint32_t kSums = kBars + (2 * kStages + 4) * 8;  // 256 int64 prefix sums + total
  static constexpr uint32_t kLens = kSums + 258 * 8;
  static constexpr uint32_t kBytes = kLens + kLensInSmem * 4;
  static constexpr int kPart = kRows * D + 2 * kRows;               // floats of a partial result
  static_assert(kStages % kProducers == 0, "each stage has one producer");
  static_assert(kBytes <= 232448, "shared memory of one block");
};

__device__ __forceinline__ int clamp_len(int len, int cap) { return len < 0 ? 0 : (len > cap ? cap : len); }

// Tokens that the last row of row tile rt sees, and its tiles (one at least, so that every item is somebody's).
__device__ __forceinline__ int visible(int len, int T, int G, int rows, int rt) {
  const int last = min(T - 1, ((rt + 1) * rows - 1) / G);
  return len - T + last + 1;
}
__device__ __forceinline__ int tiles_of(int seen, int tile) { return seen <= tile ? 1 : (seen + tile - 1) / tile; }

// The items of this block, one after another: (sequence, row tile, head) and a range of its tiles.
template <int R, int TILE> struct Walker {
  const AttendParams *pp;
  const int32_t *lens;       // shared memory copy, or pp->lens
  int64_t left;              // tiles still to take (split) / items (whole)
  int n, rt, h, len, tiles;
  int t0, t1;                // tile range of the current item in this block
  bool starts, ends;         // the range holds the item's first / last tile

  __device__ Walker(const AttendParams &p_, const int32_t *lens_) : pp(&p_), lens(lens_) {}
  __device__ void enter() {
    len = clamp_len(lens[n], pp->max_pages * pp->P);
    tiles = tiles_of(visible(len, pp->T, pp->G, R, rt), TILE);
  }
  // split: `tile` is the block's first tile on the line, `sums` the exclusive sums of chunks of `per`
  // (sequence, row tile) pairs
  __device__ bool begin_split(int64_t tile, int64_t count, const int64_t *sums, int per) {
    left = count;
    if (left <= 0) return false;
    int lo = 0, hi = 255;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sums[mid] <= tile) lo = mid; else hi = mid - 1;
    }
    int64_t at = tile - sums[lo];
    int m = lo * per;
    n = m / pp->RT; rt = m - n * pp->RT;
    enter();
    while (at >= (int64_t)tiles * pp->Hk) {
      at -= (int64_t)tiles * pp->Hk;
      if (++rt == pp->RT) { rt = 0; ++n; }
      enter();
    }
    h = (int)(at / tiles);
    t0 = (int)(at - (int64_t)h * tiles);
    take();
    return true;
  }
  __device__ void take() {
    t1 = left < tiles - t0 ? t0 + (int)left : tiles;
    starts = t0 == 0; ends = t1 == tiles;
    left -= t1 - t0;
  }
  __device__ bool begin_whole(int64_t item) {
    if (item >= (int64_t)pp->N * pp->RT * pp->Hk) return false;
    h = (int)(item % pp->Hk);
    const int64_t m = item / pp->Hk;
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
    t0 = 0;
    take();
    return true;
  }
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// The fp16 parts that pack_f16 rounded off.
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  return pack_f16(a - f.x, b - f.y);
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// One lane's piece of a value row: the channels [g D/8, (g + 1) D/8).
template <int D> struct Piece { uint32_t w[D / 32]; };
template <int D> __device__ __forceinline__ Piece<D> load_value(uint32_t vb, int token, int g) {
  Piece<D> r;
  if constexpr (D == 128) {
    const uint4 v = lds128(vb + token * 128 + ((g ^ (token & 7)) << 4));
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  } else {
    const uint2 v = lds64(vb + token * 64 + ((((g >> 1) ^ ((token >> 1) & 3)) << 4) | ((g & 1) << 3)));
    r.w[0] = v.x; r.w[1] = v.y;
  }
  return r;
}

// Where the 16-byte chunk q of a row of the merge buffer lies: the lanes of a store phase (two rows, four
// lanes' pieces) and the readers of a row both meet eight different bank groups.
template <int D> __device__ __forceinline__ int merge_chunk(int row, int q) {
  const int key = D == 128 ? ((row & 1) << 2 | q >> 3) : ((row & 1) << 1 | q >> 3);
  return q ^ key;
}

// Four channels of a finished row: the output over the sum; channel 0's holder adds lse.
template <typename IO, int D>
__device__ __forceinline__ void store_row(const AttendParams &p, int n, int h, int r, int q, float4 x, float m,
                                          float sum) {
  const int t = r / p.G;
  const int64_t row = ((int64_t)n * p.T + t) * p.Hq + h * p.G + (r - t * p.G);
  const float f = sum == 0.f ? 0.f : 1.f / sum;       // no weight at all: o = 0
  IO *dst = static_cast<IO *>(p.o) + row * D + 4 * q;
  if constexpr (sizeof(IO) == 2) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x * f, x.y * f), b = __floats2bfloat162_rn(x.z * f, x.w * f);
    *reinterpret_cast<uint2 *>(dst) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                                 *reinterpret_cast<const uint32_t *>(&b));
  } else {
    *reinterpret_cast<float4 *>(dst) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
  }
  if (q == 0 && p.lse != nullptr) p.lse[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
}

// Until the stage has been given its tile of that turn (bounded; sixteen reads take about one poll's time).
__device__ __forceinline__ bool wait_turn(const volatile uint32_t *turn, uint32_t want, uint32_t polls) {
  for (uint32_t i = 0; i < 16 * polls; ++i)
    if (*turn == want) return true;
  return false;
}

template <typename IO, int D, int MT>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ AttendParams p) {
  using L = Layout<IO, D, MT>;
  constexpr bool kSplitIO = sizeof(IO) == 4;          // fp32 calls: two fp16 parts of q and of the weights
  constexpr int R = L::kRows, KL = L::kLanes, NT = D / 8, NS = L::kStages;   // NT: n-tiles of the output
  constexpr int TILE = kTile<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
  StageInfo *info = reinterpret_cast<StageInfo *>(smem + L::kInfo);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBars), *empty = full + NS;
  uint64_t *qfull = empty + NS, *qempty = qfull + 2;
  int64_t *sums = reinterpret_cast<int64_t *>(smem + L::kSums);
  int32_t *slens = reinterpret_cast<int32_t *>(smem + L::kLens);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      // unloaded groups of 16 tokens keep valid = 0 beyond the tile's own
      *reinterpret_cast<uint32_t *>(info[i].valid) = 0;
      info[i].turn = ~0u;
      mbar_init(full + i, p.boxes);
      mbar_init(empty + i, MT);
    }
    for (int i = 0; i < 2; ++i) { mbar_init(qfull + i, L::kLoaders); mbar_init(qempty + i, kConsumers); }
    mbar_fence_init();
    tma_prefetch_desc(&p.map_k);
    tma_prefetch_desc(&p.map_v);
  }
  const int cap = p.max_pages * p.P;
  const bool small = p.N <= kLensInSmem;
  for (int n = threadIdx.x; n < p.N && (small || blockIdx.x == 0); n += kThreads) {
    const int len = p.lens[n];
    if (small) slens[n] = len;
    if (blockIdx.x == 0 && p.status != nullptr && (len < 0 || len > cap)) atomicOr(p.status, ERR_BAD_LENGTH);
  }
  __syncthreads();
  const int32_t *lens = small ? slens : p.lens;
  const int64_t pairs = (int64_t)p.N * p.RT;
  const int per = (int)((pairs + 255) / 256);
  int64_t first = 0, share = 0;
  if (!p.whole) {
    // every block lays out the line by itself: tiles before each chunk of `per` pairs
    int64_t sum = 0;
    if (threadIdx.x < 256) {
      const int64_t m0 = (int64_t)threadIdx.x * per, m1 = min(m0 + per, pairs);
      int n = (int)(m0 / p.RT), rt = (int)(m0 - (int64_t)n * p.RT);
      for (int64_t m = m0; m < m1; ++m) {
        sum += tiles_of(visible(clamp_len(lens[n], cap), p.T, p.G, R, rt), TILE);
        if (++rt == p.RT) { rt = 0; ++n; }
      }
      sum *= p.Hk;
      int64_t run = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(~0u, run, o);
        if (lane >= o) run += up;
      }
      sums[threadIdx.x] = run - sum;                  // within the warp
      if (lane == 31) reinterpret_cast<int64_t *>(smem + L::kStats)[warp] = run;
    }
    __syncthreads();
    const int64_t *warp_sums = reinterpret_cast<const int64_t *>(smem + L::kStats);
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += warp_sums[w];
      total += warp_sums[w];
    }
    if (threadIdx.x < 256) sums[threadIdx.x] += before;
    __syncthreads();
    share = (total + gridDim.x - 1) / gridDim.x;
    share = share < KL ? KL : share;                  // a tile for each lane of warps at least
    first = share * blockIdx.x;
    if (threadIdx.x == 0) sums[256] = total - first;
    __syncthreads();
  }
  Walker<R, TILE> it(p, lens);
  bool more = p.whole ? it.begin_whole(blockIdx.x) : it.begin_split(first, min(share, sums[256]), sums, per);

  if (warp >= kConsumers) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kProducerRegs));
    bool dead = p.polls == 0 && more;
    if (warp >= kConsumers + L::kProducers) {
      // ---------------------------------------------------------------- queries
      // Each row by a power of two in [2^14, 2^15), as fp16 A fragments; the channels of k-step s are
      // 16 c + 4 s .. + 3 (s < 4) and 64 + 16 c + 4 (s - 4) .. + 3.
      const int loader = warp - kConsumers - L::kProducers, rows = p.T * p.G;
      for (uint32_t i = 0; more && !dead; more = it.next(), ++i) {
        const uint32_t slot = i & 1;
        if (i >= 2 && !__all_sync(~0u, mbar_wait_bounded(qempty + slot, (i / 2 - 1) & 1, p.polls))) { dead = true; break; }
        for (int mt = loader; mt < MT; mt += L::kLoaders) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int row = mt * 16 + g + 8 * half, r = min(it.rt * R + row, rows - 1), t = r / p.G;
            const IO *src = static_cast<const IO *>(p.q) + ((int64_t)it.n * p.T + t) * p.q_stride +
                            (int64_t)(it.h * p.G + r - t * p.G) * D + 16 * c;
            float x[D / 4];
            float big = 0.f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              float y[8];
              load8(src + (k / 2) * 64 + (k % 2) * 8, y);
#pragma unroll
              for (int e = 0; e < 8; ++e) { x[8 * k + e] = y[e]; big = fmaxf(big, fabsf(y[e])); }
            }
            big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
            big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
            int e = 14 - ((int)(__float_as_uint(big) >> 23) - 127);
            e = e < -120 ? -120 : (e > 120 ? 120 : e);
            const float up = __uint_as_float((uint32_t)(127 + e) << 23);
            const float down = __uint_as_float((uint32_t)(127 - e) << 23);
            if (c == 0) reinterpret_cast<float *>(smem + L::kQFactor)[slot * R + row] = p.scale * kLog2e * down;
            uint32_t *dst = reinterpret_cast<uint32_t *>(smem + L::kQ + slot * L::kQSlot) +
                            (mt * L::kQParts * (D / 16) * 32 + lane) * 4 + half;
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float a = x[4 * s + 2 * k] * up, b = x[4 * s + 2 * k + 1] * up;
                const uint32_t hi = pack_f16(a, b);
                dst[s * 128 + 2 * k] = hi;
                if constexpr (kSplitIO) dst[(D / 16 + s) * 128 + 2 * k] = pack_rest(a, b, hi);
              }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(qfull + slot);
      }
      if (dead && lane == 0 && p.status != nullptr) atomicOr(p.status, ERR_TIMEOUT_ATTEND);
      return;
    }
    // ------------------------------------------------------------------ producers
    // A lane has one box of a tile to itself, from the table entry to the copy, so the several hundred cycles
    // of one warp's way through that are shared by several tiles.  A stage has one producer for good, which
    // has seen all its earlier turns: a parity could not tell another's turns apart.
    bool bad = false;
    uint32_t issued = 0;
    const int per_batch = 32 / p.boxes;               // tiles whose pages the lanes look up at once
    const int groups = (TILE / 16) / p.boxes;         // 16-token groups per box
    const int b = lane % p.boxes, ahead = lane / p.boxes;
    // A batch: tiles [t, t + count) of one item; in each lane the first cache row of its box (-1: nothing to
    // load) and its scales.  The next batch is looked up before the present one is issued, across items too.
    struct Batch { int count, row; float ks, vs; };
    int at = it.t0;
    auto look_up = [&](Batch &x) {
      x.count = 0;
      x.row = -1;
      x.ks = x.vs = 1.f;
      if (!more) return;
      x.count = min(per_batch, it.t1 - at);
      const int token = (at + ahead) * TILE + b * p.box;
      if (ahead < x.count && token < visible(it.len, p.T, p.G, R, it.rt)) {
        const int page = p.table[(int64_t)it.n * p.max_pages + (token >> p.log_page)];
        if (page >= 0 && page < p.num_pages) {
          const int tile = page * p.Hk + it.h;
          x.ks = p.k_scale[tile];
          x.vs = p.v_scale[tile];
          x.row = (tile << p.log_page) + (token & (p.P - 1));
        } else {
          bad = true;
        }
      }
      at += x.count;
      if (at >= it.t1) { more = it.next(); at = it.t0; }
    };
    Batch x, y;
    look_up(x);
    while (x.count > 0 && !dead) {
      look_up(y);
      const float vs = fminf(fmaxf(x.vs, 0x1p-60f), 0x1p60f), lv = log2f(vs), iv = 1.f / vs;
      const uint32_t tile = issued + ahead, turn = tile / NS, s = tile - turn * NS;
      const uint32_t bytes = x.row >= 0 ? 2 * p.box * D : 0;
      unsigned char *dst = smem + s * 8192 + b * p.box * D;
      const bool own = ahead < x.count && s / L::kOwn == warp - kConsumers;
      const uint32_t last = (issued + x.count - 1) / NS;
      for (uint32_t now = issued / NS; now <= last; ++now) {
        const bool mine = own && turn == now;
        if (!__all_sync(~0u, !mine || turn == 0 || mbar_wait_bounded(empty + s, (turn - 1) & 1, p.polls))) {
          dead = true;
          issued = max(issued, now * NS);             // what this batch has sent before
          break;
        }
        if (mine) {
          for (int i = b * groups; i < (b + 1) * groups; ++i) {
            info[s].kf[i] = x.ks;
            info[s].lv[i] = lv;
            info[s].iv[i] = iv;
            info[s].valid[i] = x.row >= 0;
          }
          *const_cast<volatile uint32_t *>(&info[s].turn) = turn;
          mbar_arrive_expect_tx(full + s, bytes);
          if (x.row >= 0) {
            tma_load_2d(dst, &p.map_k, 0, x.row, full + s);
            tma_load_2d(dst + 4096, &p.map_v, 0, x.row, full + s);
          }
        }
        __syncwarp();
      }
      if (!dead) issued += x.count;
      x = y;
    }
    if (bad && p.status != nullptr) atomicOr(p.status, ERR_BAD_PAGE);
    if (dead && lane == 0 && p.status != nullptr) atomicOr(p.status, ERR_TIMEOUT_ATTEND);
    // no copy is left in flight when the block ends, whether or not a consumer waited for it
    for (uint32_t i = issued > NS ? issued - NS : 0; i < issued; ++i)
      if (i % NS / L::kOwn == warp - kConsumers) mbar_wait_bounded(full + i % NS, (i / NS) & 1, kWaitPolls);
    return;
  }

  // -------------------------------------------------------------------- consumers
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kConsumerRegs));
  const int mt = warp % MT, kl = warp / MT;
  const int rows = p.T * p.G;
  const int sg = g ^ ((g & 1) << 2);                  // sigma(g): the token of the lane's key column
  const int ca = 2 * c, cb = (2 * c + 1) ^ 4;         // sigma(2c), sigma(2c + 1): the tokens of its score columns
  const uint32_t ring = smem_u32(smem);
  float *merge = reinterpret_cast<float *>(smem + L::kMerge);
  float2 *stats = reinterpret_cast<float2 *>(smem + L::kStats);
  constexpr uint32_t kAllValid = TILE == 64 ? 0x01010101u : 0x0101u;
  bool dead = false;
  int4 split = make_int4(-1, 0, 0, 0);
  uint32_t done = 0;                                  // tiles of the items before

  for (uint32_t item = 0; more; more = it.next(), ++item) {
    const int row0 = it.rt * R + mt * 16;
    // tokens that a row sees: all below its limit.  Rows behind the last one repeat it.
    auto limit = [&](int r) { return it.len - p.T + min(r, rows - 1) / p.G + 1; };
    const int lim0 = limit(row0 + g), lim1 = limit(row0 + g + 8);
    const int low = limit(row0), high = limit(row0 + 15);

    const uint32_t slot = item & 1;
    if (!dead) dead = !__all_sync(~0u, mbar_wait_bounded(qfull + slot, (item / 2) & 1, p.polls));
    const uint32_t qf = ring + L::kQ + slot * L::kQSlot + (mt * L::kQParts * (D / 16) * 32 + lane) * 16;
    const float *factor = reinterpret_cast<const float *>(smem + L::kQFactor) + slot * R + mt * 16;
    const float rf0 = dead ? 0.f : factor[g], rf1 = dead ? 0.f : factor[g + 8];

    float o[NT][4] = {}, m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    for (int u = it.t0 + kl; u < it.t1; u += KL) {
      const uint32_t at = done + (u - it.t0), s = at % NS;
      // A parity tells a phase only from its neighbour, and the stage's previous tile was another warp's: it
      // may still be on its way although later ones have come.  So the tile's turn is waited for first, which
      // the producer writes when the stage is free for it: the barrier is in that phase or just past it then.
      if (!dead) dead = !__all_sync(~0u, wait_turn(&info[s].turn, at / NS, p.polls));
      if (!dead) dead = !__all_sync(~0u, mbar_wait_bounded(full + s, (at / NS) & 1, p.polls));
      if (dead) continue;
      const int base = u * TILE;
      if (base < high) {
        const uint32_t kb = ring + s * 8192, vb = kb + 4096;
        const uint32_t valid = *reinterpret_cast<const uint32_t *>(info[s].valid);
        const bool masked = base + TILE > low || valid != kAllValid;
        float sc[TILE / 8][4] = {};
#pragma unroll
        for (int part = 0; part < D / 64; ++part) {   // the pieces c and c + 4 of the key rows
          uint4 w[TILE / 8];
#pragma unroll
          for (int nt = 0; nt < TILE / 8; ++nt) {
            const int token = 8 * nt + sg;
            w[nt] = D == 128 ? lds128(kb + token * 128 + (((c + 4 * part) ^ sg) << 4))
                             : lds128(kb + token * 64 + ((c ^ ((token >> 1) & 3)) << 4));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 qh = lds128(qf + (4 * part + k) * 512);
            const uint32_t a[4] = {qh.x, qh.y, qh.z, qh.w};
            uint4 ql;
            if constexpr (kSplitIO) ql = lds128(qf + (D / 16 + 4 * part + k) * 512);
#pragma unroll
            for (int nt = 0; nt < TILE / 8; ++nt) {
              const uint32_t v = k == 0 ? w[nt].x : k == 1 ? w[nt].y : k == 2 ? w[nt].z : w[nt].w;
              const uint32_t b0 = codes_lo(v), b1 = codes_hi(v);
              mma_f16(sc[nt], a, b0, b1);
              if constexpr (kSplitIO) {
                const uint32_t al[4] = {ql.x, ql.y, ql.z, ql.w};
                mma_f16(sc[nt], al, b0, b1);
              }
            }
          }
        }
        float x0 = m0, x1 = m1;
#pragma unroll
        for (int nt = 0; nt < TILE / 8; ++nt) {
          const float kf = info[s].kf[nt / 2], lv = info[s].lv[nt / 2];
          const float f0 = rf0 * kf, f1 = rf1 * kf;
          sc[nt][0] = fmaf(sc[nt][0], f0, lv);
          sc[nt][1] = fmaf(sc[nt][1], f0, lv);
          sc[nt][2] = fmaf(sc[nt][2], f1, lv);
          sc[nt][3] = fmaf(sc[nt][3], f1, lv);
          if (masked) {
            const bool in = valid >> (8 * (nt / 2)) & 1;
            const int ta = base + 8 * nt + ca, tb = base + 8 * nt + cb;
            if (!in || ta >= lim0) sc[nt][0] = -INFINITY;
            if (!in || tb >= lim0) sc[nt][1] = -INFINITY;
            if (!in || ta >= lim1) sc[nt][2] = -INFINITY;
            if (!in || tb >= lim1) sc[nt][3] = -INFINITY;
          }
          x0 = fmaxf(x0, fmaxf(sc[nt][0], sc[nt][1]));
          x1 = fmaxf(x1, fmaxf(sc[nt][2], sc[nt][3]));
        }
#pragma unroll
        for (int i = 1; i < 4; i <<= 1) {
          x0 = fmaxf(x0, __shfl_xor_sync(~0u, x0, i));
          x1 = fmaxf(x1, __shfl_xor_sync(~0u, x1, i));
        }
        const float z0 = x0 == -INFINITY ? 0.f : x0, z1 = x1 == -INFINITY ? 0.f : x1;
        if (__any_sync(~0u, x0 != m0 || x1 != m1)) {
          const float a0 = ex2(m0 - z0), a1 = ex2(m1 - z1);
          l0 *= a0;
          l1 *= a1;
#pragma unroll
          for (int i = 0; i < NT; ++i) { o[i][0] *= a0; o[i][1] *= a0; o[i][2] *= a1; o[i][3] *= a1; }
        }
        m0 = x0;
        m1 = x1;
        bool nan = false;
#pragma unroll
        for (int j = 0; j < TILE / 16; ++j) {
          const float iv = info[s].iv[j];
          uint32_t pf[4], pl[4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float (&w)[4] = sc[2 * j + k];
            w[0] = ex2(w[0] - z0); w[1] = ex2(w[1] - z0);
            w[2] = ex2(w[2] - z1); w[3] = ex2(w[3] - z1);
            l0 = fmaf(w[0] + w[1], iv, l0);
            l1 = fmaf(w[2] + w[3], iv, l1);
            pf[2 * k] = pack_f16(w[0], w[1]);
            pf[2 * k + 1] = pack_f16(w[2], w[3]);
            if constexpr (kSplitIO) {
              pl[2 * k] = pack_rest(w[0], w[1], pf[2 * k]);
              pl[2 * k + 1] = pack_rest(w[2], w[3], pf[2 * k + 1]);
            }
          }
          const int tok[4] = {16 * j + ca, 16 * j + cb, 16 * j + ca + 8, 16 * j + cb + 8};
          Piece<D> v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = load_value<D>(vb, tok[k], g);
            if (masked) {
              // a code that no row sees becomes 0: its weight is 0, but 0 * NaN would not be.  A NaN that
              // some rows see and others do not is put in its rows by hand below.
              const bool in = valid >> (8 * j) & 1, none = !in || base + tok[k] >= high, some = base + tok[k] >= low;
#pragma unroll
              for (int i = 0; i < D / 32; ++i) {
                if (none) v[k].w[i] = 0;
                if (some) {
                  const uint32_t is = __vcmpeq4(v[k].w[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                  nan |= is != 0;
                  v[k].w[i] &= ~is;
                }
              }
            }
          }
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const uint32_t e0 = __byte_perm(v[0].w[i], v[1].w[i], 0x5140), e1 = __byte_perm(v[0].w[i], v[1].w[i], 0x7362);
            const uint32_t e2 = __byte_perm(v[2].w[i], v[3].w[i], 0x5140), e3 = __byte_perm(v[2].w[i], v[3].w[i], 0x7362);
            const uint32_t b[4][2] = {{codes_lo(e0), codes_lo(e2)}, {codes_hi(e0), codes_hi(e2)},
                                      {codes_lo(e1), codes_lo(e3)}, {codes_hi(e1), codes_hi(e3)}};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              mma_f16(o[4 * i + k], pf, b[k][0], b[k][1]);
              if constexpr (kSplitIO) mma_f16(o[4 * i + k], pl, b[k][0], b[k][1]);
            }
          }
        }
        if (masked && __any_sync(~0u, nan)) {
          const int to = min(base + TILE, high);
          for (int token = max(base, low); token < to; ++token) {
            if (!(valid >> (8 * ((token - base) / 16)) & 1)) continue;
#pragma unroll
            for (int k = 0; k < 2; ++k) {             // the lane's output columns: pieces 2 c and 2 c + 1
              const Piece<D> v = load_value<D>(vb, token - base, 2 * c + k);
#pragma unroll
              for (int i = 0; i < NT; ++i)
                if ((v.w[i / 4] >> (8 * (i % 4)) & 0x7f) == 0x7f) {
                  if (token < lim0) o[i][k] = __int_as_float(0x7fffffff);
                  if (token < lim1) o[i][2 + k] = __int_as_float(0x7fffffff);
                }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + s);
    }
    if (lane == 0 && !dead) mbar_arrive(qempty + slot);

    // ---- the KL warps of an m-tile meet: the upper half leaves its outputs, the lower half adds its own,
    // and all of them sum up what the lower half has left
#pragma unroll
    for (int i = 1; i < 4; i <<= 1) {
      l0 += __shfl_xor_sync(~0u, l0, i);
      l1 += __shfl_xor_sync(~0u, l1, i);
    }
    if (c == 0) {
      stats[warp * 16 + g] = make_float2(m0, l0);
      stats[warp * 16 + g + 8] = make_float2(m1, l1);
    }
    named_sync(1, kConsumers * 32);
    float M0 = m0, M1 = m1;
#pragma unroll
    for (int k = 0; k < KL; ++k) {
      M0 = fmaxf(M0, stats[k * R + mt * 16 + g].x);
      M1 = fmaxf(M1, stats[k * R + mt * 16 + g + 8].x);
    }
    const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - M0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M1);
    auto leave = [&](int lane_slot, bool add) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float *dst = merge + (lane_slot * R + mt * 16 + g + 8 * half) * D;
        const float f = half ? f1 : f0;
#pragma unroll
        for (int k = 0; k < 2; ++k)                   // pieces 2 c and 2 c + 1 of the row
#pragma unroll
          for (int i = 0; i < NT / 4; ++i) {
            float4 *to = reinterpret_cast<float4 *>(dst + 4 * merge_chunk<D>(g, (2 * c + k) * (NT / 4) + i));
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            if (add) y = *to;
            *to = make_float4(fmaf(o[4 * i][2 * half + k], f, y.x), fmaf(o[4 * i + 1][2 * half + k], f, y.y),
                              fmaf(o[4 * i + 2][2 * half + k], f, y.z), fmaf(o[4 * i + 3][2 * half + k], f, y.w));
          }
      }
    };
    if (kl >= L::kHalf) leave(kl - L::kHalf, false);
    named_sync(1, kConsumers * 32);
    if (kl < L::kHalf) leave(kl, kl + L::kHalf < KL);
    named_sync(1, kConsumers * 32);
    float *part = it.starts && it.ends ? nullptr
                                       : p.parts + ((int64_t)blockIdx.x * 2 + (it.starts ? 1 : 0)) * L::kPart;
    for (int i = threadIdx.x; i < R * (D / 4); i += kConsumers * 32) {
      const int row = i / (D / 4), q = i % (D / 4);
      float M = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < KL; ++k) M = fmaxf(M, stats[k * R + row].x);
#pragma unroll
      for (int k = 0; k < KL; ++k) {
        const float2 ml = stats[k * R + row];
        sum += ml.x == -INFINITY ? 0.f : ml.y * ex2(ml.x - M);
      }
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < L::kHalf; ++k) {
        const float4 y = *reinterpret_cast<const float4 *>(merge + (k * R + row) * D + 4 * merge_chunk<D>(row, q));
        x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
      }
      if (part != nullptr) {
        *reinterpret_cast<float4 *>(part + row * D + 4 * q) = x;
        if (q == 0) { part[R * D + row] = M; part[R * D + R + row] = sum; }
      } else if (it.rt * R + row < rows) {
        store_row<IO, D>(p, it.n, it.h, it.rt * R + row, q, x, M, sum);
      }
    }
    if (it.starts && !it.ends)
      split = make_int4(it.n, it.rt, it.h, (int)((first + done + it.tiles - 1) / share));
    done += it.t1 - it.t0;
    named_sync(1, kConsumers * 32);                   // the buffers are free again
  }
  if (dead && lane == 0 && p.status != nullptr) atomicOr(p.status, ERR_TIMEOUT_ATTEND);
  if (!p.whole && threadIdx.x == 0) p.desc[blockIdx.x] = split;
}

// Joins the parts of the item that begins in block blockIdx.x and ends in a later one: four warps take
// every fourth part of a row, a lane D / 32 channels.
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
      const float m = factor[i], f = m == -INFINITY ? 0.f : ex2(m - M);
      factor[i] = f;
      sum += m == -INFINITY ? 0.f : f * part(i)[R * D + R + row];
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
      store_row<IO, D>(p, d.x, d.z, d.y * R + row, threadIdx.x, r, M, sum);
    }
    __syncthreads();
  }
}

int row_tiles(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

template <typename IO, int D, int MT>
cudaError_t launch(AttendParams p, const kda_cache &c, int64_t items, cudaStream_t stream) {
  using L = Layout<IO, D, MT>;
  const CUtensorMapSwizzle swizzle = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  const uint64_t rows = (uint64_t)c.num_pages * c.num_kv_heads * c.page_tokens;
  if (!encode_rows(&p.map_k, c.k_cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, D, D, p.box, D, swizzle) ||
      !encode_rows(&p.map_v, c.v_cache, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, rows, D, D, p.box, D, swizzle))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<IO, D, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       L::kBytes);
  if (e != cudaSuccess) return e;
  const unsigned grid = p.whole && items < kBlocks ? (unsigned)items : kBlocks;
  attend_kernel<IO, D, MT><<<grid, kThreads, L::kBytes, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.whole) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kBlocks, 16);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_join_kernel<IO, D, 16 * MT>, p);
}

template <typename IO, int D>
cudaError_t launch_rows(const AttendParams &p, const kda_cache &c, int64_t items, int mt, cudaStream_t stream) {
  if (mt == 1) return launch<IO, D, 1>(p, c, items, stream);
  if (mt == 2) return launch<IO, D, 2>(p, c, items, stream);
  return launch<IO, D, 4>(p, c, items, stream);
}

}  // namespace

size_t cache_attend_workspace(const kda_cache &c, const kda_cache_attend_args &a) {
  const int64_t rows = 16 * row_tiles(a.num_new * (a.num_heads / c.num_kv_heads));
  const int64_t bytes = kBlocks * 16 + kBlocks * 2 * (rows * c.head_dim + 2 * rows) * 4;
  return (size_t)((bytes + 255) / 256 * 256);
}

cudaError_t launch_cache_attend(const kda_cache &c, const kda_cache_attend_args &a, void *workspace,
                                cudaStream_t stream) {
  AttendParams p{};
  p.N = c.num_seqs; p.T = a.num_new; p.Hq = a.num_heads; p.Hk = c.num_kv_heads; p.G = p.Hq / p.Hk;
  p.P = c.page_tokens; p.log_page = p.P == 16 ? 4 : p.P == 32 ? 5 : p.P == 64 ? 6 : 7; p.max_pages = c.max_pages; p.num_pages = c.num_pages;
  const int mt = row_tiles(p.T * p.G), R = 16 * mt;
  p.RT = (p.T * p.G + R - 1) / R;
  const int tile = c.head_dim == 128 ? kTile<128> : kTile<64>;
  p.box = p.P < tile ? p.P : tile;
  p.boxes = tile / p.box;
  p.q_stride = a.q_stride; p.scale = a.scale; p.q = a.q;
  p.k_scale = c.k_scale; p.v_scale = c.v_scale; p.table = c.block_table; p.lens = c.seq_lens;
  p.o = a.o; p.lse = a.lse; p.status = a.status;
  p.polls = wait_polls_for(a.flags);
  p.desc = static_cast<int4 *>(workspace);
  p.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + kBlocks * 16);
  const int64_t items = (int64_t)p.N * p.RT * p.Hk;
  // No item has more tiles than its block takes at a time: splitting would only add the join.
  p.whole = ((int64_t)p.max_pages * p.P + tile - 1) / tile <= kConsumers / mt;
  const bool bf16 = a.io_dtype == KDA_BF16;
  if (c.head_dim == 128)
    return bf16 ? launch_rows<__nv_bfloat16, 128>(p, c, items, mt, stream)
                : launch_rows<float, 128>(p, c, items, mt, stream);
  return bf16 ? launch_rows<__nv_bfloat16, 64>(p, c, items, mt, stream)
              : launch_rows<float, 64>(p, c, items, mt, stream);
}

}  // namespace kda
