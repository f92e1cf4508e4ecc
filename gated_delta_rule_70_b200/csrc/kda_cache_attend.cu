// Attention over the paged 8-bit cache.
//
// A work item is one (sequence, tile of query rows, key / value head); a query row is a (new token, query
// head of the group) pair, so grouped heads share every cached byte that is read.  The items' tiles (32
// cached tokens of 128 channels, or 64 of 64) form one line, which the grid's blocks share out equally: a
// long sequence spreads over many blocks, a block takes several short ones.  An item that lies in several
// blocks leaves partial results (running maximum, sum, unnormalised output) in the workspace, and a second
// kernel joins them in the order of the blocks, so results do not depend on timing.
//
// A block has warps of four kinds, which meet at mbarriers alone:
//   producers  bring tiles by TMA into a ring of 8 KB stages (one box per page, rows swizzled);
//   the loader brings the next item's queries as fp16 fragments;
//   consumers  own 8 NR query rows and every KL-th tile of the item, with a running maximum, sum and output
//              of their own, so none waits for another: at the item's end each leaves its output in shared
//              memory and goes on to the next item;
//   the merger sums up what they left and stores it.
//
// One consumer and tile: S^T = K Q^T and O^T += V^T P^T by mma.sync m16n8k16 with fp16 operands and fp32
// accumulation: cached tokens (then channels) are the 16 rows and query rows the 8 columns, so few query
// rows waste little and a widened key or value serves all NR columns' tiles.  e4m3 codes are exact in fp16.
// The contraction's order is free, so the channels of a key row go to the lanes as the 16-byte pieces they
// load; the order of 8 tokens is free too and is sigma(n) = n (even), n ^ 4 (odd: 1 -> 5, 3 -> 7, 5 -> 1,
// 7 -> 3), which makes the key loads (two tokens x four pieces per phase) and the value loads (four tokens x
// two pieces) free of bank conflicts under the hardware's swizzle.  P^T goes from the accumulators of S^T to
// the B operand through movmatrix.
//
// Scales: with ks, vs the page's scales, weights are kept as w_j = exp2(s_j + log2 vs_j - m + 15), m the
// running maximum of s_j + log2 vs_j, so w is at most 2^15, and the sum takes w_j / vs_j.  A query row is brought
// to [2^14, 2^15) by a power of two first, so its fp16 copy is exact for bf16 inputs (fp32 inputs and their
// weights go as two fp16 parts each).
// A weight's rounding to fp16 (2^-11) is below that of a bf16 output, down to 2^-29 of the row's largest w, from
// where on fp16's subnormals lose up to 2^-40 of it each.  (With 1 as the largest w that begins at 2^-14: the many
// small weights of a long sequence, beside one token with nearly all of the weight, came out up to 100 % wrong.)
// The second part of an fp32 call's weight is what the first rounded off times 2^11, against the values times 2^-11
// (exact: codes are multiples of 2^-9 with four digits): 2^-22 down to 2^-29 of the largest, 2^-51 of it below.
// A tensor-core sum is truncated, so a long one drifts towards zero: by half of 2^-24 for each 16 tokens.  In fp32
// calls the products of 16 tokens are therefore added to the output by ordinary additions (60000 tokens of one sign,
// 64 rows: 8.3e-5 off without them, 2.7e-7 with).  Both together cost 4 to 8 % with one column tile (64 sequences
// of up to 4000 tokens, 2 heads x 128, 8 rows: 37.5 -> 39.8 us) and 9 to 23 % with two (16 rows 55.9 -> 61.2, 32
// rows 81.9 -> 100.8).  bf16 calls do without: 262144 tokens in one block come out as far from the exact mean as that
// mean rounded to bf16.
//
// Bound by HBM for long sequences: 262144 tokens x 4 heads x 128 take 57 us, 4.7 TB/s of codes; 3 us pass before
// the line is laid out and 5 more until the first tiles are there, then codes come at 6.1 TB/s, and the join ends
// 4 us after the last block.  256 sequences of up to 16384 tokens (2 heads x 128, mean 1500) take 50 us, 4.0 TB/s:
// each start of a sequence costs a block as much as eight tiles, in which its consumers have fewer tiles than
// they are or wait for the merge buffer.  Short calls are latency: one tile's way through the chain is 12 us.
// On the way: a block for each query row 82 ms for the long sequence; tiles in the ring with eight consumers 95,
// twelve and two producers 78, query rows as the products' 8 columns instead of their 16 rows 73 (cold caches).
// Units dealt out by a counter instead of equal shares even the blocks' unequal bandwidth out, but their join
// and their starts cost more (83 to 110 us), and results would depend on timing.
#include "cache_attend.cuh"

namespace kda {
namespace {

using namespace attend;

constexpr int kStageBytes = 8192;                     // 4 KB of keys, 4 KB of values
constexpr int kProducers = 2;                         // warps; a stage belongs to one of them
template <int D> constexpr int kTile = 4096 / D;      // cached tokens per stage
// What an item's own start and end cost, in tiles.  256 sequences of up to 16384 tokens, one to ten items to a
// block: with none counted the blocks ended 1.7 us later for each of their items (42 to 69 us), with 12 they end
// 0.85 us earlier; 6 to 12 are equal in time, 16 costs 2 us.
constexpr int kLead = 8;

// NR: query column tiles (of 8) per consumer; MT: row groups of an item.
template <typename IO, int D, int NR, int MT> struct Layout {
  static constexpr int kConsumers = 12, kWarps = kConsumers + 4;
  // Registers: with two column tiles the warpgroup of producers, loader and merger gives up some of its share
  // (65536 / threads) for the consumers' output fragments (16 NR x D / 64 a thread).  fp32, 16 rows of 128 channels
  // (64 sequences of up to 4000 tokens): 69.9 us with 80 / 144, 61.2 with 56 / 152; bf16, 16 rows of 64: 33.3 and
  // 34.4, and 35.5 with equal shares.  With one column tile 80 / 144 only spilled in the others (bf16: 112 bytes; the
  // batch of 256 sequences 49.8 -> 49.3 us without).
  static constexpr int kOtherRegs = NR == 1 ? 128 : sizeof(IO) == 4 ? 56 : 80;
  static constexpr int kConsumerRegs = NR == 1 ? 128 : sizeof(IO) == 4 ? 152 : 144;
  static_assert(kOtherRegs + kConsumers / 4 * kConsumerRegs == kWarps / 4 * 128, "register pool");
  static constexpr int kRows = 8 * NR * MT, kLanes = kConsumers / MT;       // query rows, tiles at a time
  // Outputs of the item in shared memory at a time: with more than one column tile the upper half of the
  // lanes leaves its own first and the lower half adds to it.
  static constexpr int kSlots = NR == 1 ? kLanes : (kLanes + 1) / 2;
  static constexpr int kStages = MT == 1 ? 18 : MT == 2 ? 16 : 10;
  static constexpr uint32_t kOwn = kStages / kProducers;            // stages of a producer
  static constexpr uint32_t kQParts = sizeof(IO) / 2;               // fp16 parts of a query
  static constexpr uint32_t kQSlot = kRows / 8 * kQParts * (D / 32) * 512;  // fragments of one item
  static constexpr uint32_t kMerge = kStages * kStageBytes;         // [kSlots][kRows][D] fp32
  static constexpr uint32_t kQ = kMerge + kSlots * kRows * D * 4;   // two slots
  static constexpr uint32_t kQFactor = kQ + 2 * kQSlot;             // two slots of [kRows] (factor, limit)
  static constexpr uint32_t kStats = kQFactor + 2 * kRows * 8;      // [kLanes][kRows] x (m, l)
  static constexpr uint32_t kInfo = kStats + kLanes * kRows * 8;
  static constexpr uint32_t kBars = kInfo + kStages * (uint32_t)sizeof(StageInfo);
  static constexpr uint32_t kSums = kBars + (2 * kStages + 7) * 8;  // 256 prefix sums, 8 of warps, the rest
  static constexpr uint32_t kLens = kSums + 266 * 4;
  static constexpr uint32_t kBytes = kLens + kLensInSmem * 4;
  static constexpr int kPart = kRows * D + 2 * kRows;               // floats of a partial result
  static_assert(kLanes >= 3, "the merger keeps three values of a row");
  static_assert(kStages % kProducers == 0, "each stage has one producer");
  static_assert(kInfo % 16 == 0 && kBars % 8 == 0 && kBytes <= 232448, "shared memory of one block");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of fp16 pairs (row lane / 4, columns 2 (lane % 4), + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
constexpr float kUp = 15.f;                           // the largest weight, as a power of two
constexpr float kRestUp = 2048.f;                     // factor on the second part of a weight
// The parts that pack_f16 rounded off, times `up`.
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi, float up) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
  return pack_f16((a - f.x) * up, (b - f.y) * up);
}
// Values for the second part of a weight.
__device__ __forceinline__ uint32_t rest_down(uint32_t v) {
  const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&v), __float2half2_rn(1.f / kRestUp));
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
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

// Where the 16-byte chunk q of a row of the merge buffer lies: the lanes of a store phase (rows 2 c, pieces
// g and g + 1) meet eight different bank groups.
template <int D> __device__ __forceinline__ int merge_chunk(int row, int q) {
  const int c = (row >> 1) & 3;
  return q ^ (D == 128 ? c : (c & 1) | (c >> 1) << 2);
}

// Until the stage has been given its tile of that turn (bounded: a poll of a barrier suspends for 4 us, sixteen
// reads take a twentieth of that).
__device__ __forceinline__ bool wait_turn(const volatile uint32_t *turn, uint32_t want, uint32_t polls) {
  for (uint32_t i = 0; i < 16 * polls; ++i)
    if (*turn == want) return true;
  return false;
}
template <typename IO, int D, int NR, int MT>
__global__ void __launch_bounds__(Layout<IO, D, NR, MT>::kWarps * 32, 1)
attend_kernel(const __grid_constant__ AttendParams p) {
  using L = Layout<IO, D, NR, MT>;
  constexpr bool kSplitIO = sizeof(IO) == 4;          // fp32 calls: two fp16 parts of q and of the weights
  constexpr int R = L::kRows, KL = L::kLanes, SL = L::kSlots, NS = L::kStages, TILE = kTile<D>;
  constexpr int kThreads = L::kWarps * 32, MI = TILE / 16, OI = D / 16;   // token tiles, output channel tiles
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c = lane % 4;
  StageInfo *info = reinterpret_cast<StageInfo *>(smem + L::kInfo);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBars), *empty = full + NS;
  uint64_t *qfull = empty + NS, *qempty = qfull + 2;  // queries: two slots
  uint64_t *left_up = qempty + 2, *left_all = left_up + 1, *merged = left_all + 1;   // the merge buffer
  uint32_t *sums = reinterpret_cast<uint32_t *>(smem + L::kSums);
  int32_t *slens = reinterpret_cast<int32_t *>(smem + L::kLens);
  float2 *stats = reinterpret_cast<float2 *>(smem + L::kStats);
  float *merge = reinterpret_cast<float *>(smem + L::kMerge);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      // unloaded groups of 16 tokens keep valid = 0 beyond the tile's own
      *reinterpret_cast<uint32_t *>(info[i].valid) = 0;
      info[i].turn = ~0u;
      mbar_init(full + i, p.boxes);
      mbar_init(empty + i, MT);
    }
    for (int i = 0; i < 2; ++i) { mbar_init(qfull + i, 1); mbar_init(qempty + i, L::kConsumers); }
    mbar_init(left_up, (KL - SL) * MT + (KL == SL));  // never waited for without an upper half
    mbar_init(left_all, SL * MT);
    mbar_init(merged, 1);
    mbar_fence_init();
  }
  if (threadIdx.x == 32) {
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
  Line line{0, 0, 0};
  if (!p.whole) line = lay_out<R, TILE, kLead>(p, lens, sums, KL);   // a tile for each lane of consumers at least
  // the join may be set up now: it waits for the whole grid before it reads anything
  cudaTriggerProgrammaticLaunchCompletion();
  Walker<R, TILE, kLead> it(p, lens);
  bool more = p.whole ? it.begin_whole(blockIdx.x) : it.begin_split(line.first, (int)sums[264], sums, line.per);
  bool dead = false;

  if (warp >= L::kConsumers) {
    if constexpr (NR > 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(L::kOtherRegs));
    const int other = warp - L::kConsumers, rows = p.T * p.G;
    if (other == kProducers) {
      // ---------------------------------------------------------------- the loader
      // Each query row by a power of two in [2^14, 2^15), as fp16 B fragments; the channels of k-step s are
      // 16 c + 4 s .. + 3 (s < 4) and 64 + 16 c + 4 (s - 4) .. + 3.  With it the row's factor on the scores
      // and its limit: the row sees the tokens below.  Rows behind the last one repeat it.
      for (uint32_t i = 0; more && !dead; more = it.next(), ++i) {
        const uint32_t slot = i & 1;
        if (i >= 2 && !warp_wait(qempty + slot, i / 2 - 1, p.polls)) { dead = true; break; }
        for (int nt = 0; nt < R / 8; ++nt) {
          const int row = nt * 8 + g, r = min(it.rt * R + row, rows - 1), t = r / p.G;
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
          if (c == 0)
            reinterpret_cast<float2 *>(smem + L::kQFactor)[slot * R + row] =
                make_float2(p.scale * kLog2e * down, __int_as_float(it.len - p.T + t + 1));
          uint4 *dst = reinterpret_cast<uint4 *>(smem + L::kQ + slot * L::kQSlot) + nt * L::kQParts * (D / 32) * 32 + lane;
#pragma unroll
          for (int s = 0; s < D / 32; ++s) {          // two k-steps
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float a = x[8 * s + 2 * k] * up, b = x[8 * s + 2 * k + 1] * up;
              hi[k] = pack_f16(a, b);
              lo[k] = kSplitIO ? pack_rest(a, b, hi[k], 1.f) : 0;
            }
            dst[s * 32] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if constexpr (kSplitIO) dst[(D / 32 + s) * 32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(qfull + slot);
      }
      if (dead && lane == 0 && p.status != nullptr) atomicOr(p.status, ERR_TIMEOUT_ATTEND);
      return;
    }
    if (other == kProducers + 1) {
      // ---------------------------------------------------------------- the merger
      int4 split = make_int4(-1, 0, 0, 0);
      for (uint32_t i = 0; more && !dead; more = it.next(), ++i) {
        const int used = min(it.t1 - it.t0, SL);      // the lanes that had a tile
        if (!warp_wait(left_all, i, p.polls)) { dead = true; break; }
        float *part = it.starts && it.ends ? nullptr
                                           : p.parts + ((int64_t)blockIdx.x * 2 + (it.starts ? 1 : 0)) * L::kPart;
        // Each lane's share of the row's weight, over its m; then, in places that are free by then, the row's
        // factor on its output and its place, so that the loop below waits for neither: with them in it an item of
        // 64 rows took 23 us here.
        const int real = min(R, rows - it.rt * R);
        for (int row = lane; row < R; row += 32) {
          float2 ml[SL];
          float M = -INFINITY, sum = 0.f;
#pragma unroll
          for (int k = 0; k < SL; ++k) {
            ml[k] = k < used ? stats[k * R + row] : make_float2(-INFINITY, 0.f);
            M = fmaxf(M, ml[k].x);
          }
#pragma unroll
          for (int k = 0; k < SL; ++k) {
            const float f = fade(ml[k].x, M);
            sum = fmaf(f, ml[k].y, sum);
            stats[k * R + row].x = f;
          }
          if (row >= real) continue;
          const int to = out_row(p, it.n, it.h, it.rt * R + row);
          stats[R + row].y = row_factor(sum);
          stats[2 * R + row].y = __int_as_float(to);
          if (part != nullptr) {
            part[R * D + row] = M;
            part[R * D + R + row] = sum;
          } else {
            store_lse(p, to, M, sum);
          }
        }
        __syncwarp();
#pragma unroll (R >= 32 ? 4 : 1)
        for (int at = lane; at < real * (D / 4); at += 32) {
          const int row = at / (D / 4), q = at % (D / 4);
          const float *src = merge + row * D + 4 * merge_chunk<D>(row, q);
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < SL; ++k)
            if (k < used) {
              const float f = stats[k * R + row].x;
              const float4 y = *reinterpret_cast<const float4 *>(src + k * R * D);
              x.x = fmaf(f, y.x, x.x); x.y = fmaf(f, y.y, x.y); x.z = fmaf(f, y.z, x.z); x.w = fmaf(f, y.w, x.w);
            }
          if (part != nullptr) {
            *reinterpret_cast<float4 *>(part + row * D + 4 * q) = x;
          } else {
            store_row<IO, D>(p, __float_as_int(stats[2 * R + row].y), q, x, stats[R + row].y);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(merged);
        if (it.starts && !it.ends) split = make_int4(it.n, it.rt, it.h, (int)((it.stop - 1) / line.share));
      }
      if (dead && lane == 0 && p.status != nullptr) atomicOr(p.status, ERR_TIMEOUT_ATTEND);
      if (!p.whole && lane == 0) p.desc[blockIdx.x] = split;
      return;
    }
    // ------------------------------------------------------------------ producers
    // A lane has one box of a tile to itself, from the table entry to the copy, so the several hundred cycles
    // of one warp's way through that are shared by several tiles.  A stage has one producer for good, which
    // has seen all its earlier turns: a parity could not tell another's turns apart.
    bool bad = false;
    uint32_t issued = 0, sent = 0, last_stage = 0, last_phase = 0;
    const int per_batch = 32 / p.boxes;               // tiles whose pages the lanes look up at once
    const int groups = MI / p.boxes;                  // 16-token groups per box
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
      const uint32_t tile = issued + ahead, turn = tile / NS, s = tile - turn * NS;
      const uint32_t bytes = x.row >= 0 ? 2 * p.box * D : 0;
      unsigned char *dst = smem + s * kStageBytes + b * p.box * D;
      const bool own = ahead < x.count && s / L::kOwn == other;
      const uint32_t last = (issued + x.count - 1) / NS;
      for (uint32_t now = issued / NS; now <= last; ++now) {
        // each box goes out as soon as its stage is free; a stage's next turn only after this one
        bool pending = own && turn == now;
        for (uint32_t poll = 0; __any_sync(~0u, pending); ++poll) {
          if (poll >= p.polls) { dead = true; break; }
          const bool ready = pending && (turn == 0 || mbar_try_wait(empty + s, (turn - 1) & 1));
          if (ready) {
            pending = false;
            last_stage = s;
            last_phase = turn & 1;
            // the copies first: they do not wait for the scales to come (the barrier's phase stays open until
            // the arrival below, whatever has been copied by then)
            if (x.row >= 0) {
              tma_load_2d(dst, &p.map_k, 0, x.row, full + s);
              tma_load_2d(dst + kStageBytes / 2, &p.map_v, 0, x.row, full + s);
            }
            const float vs = fminf(fmaxf(x.vs, 0x1p-60f), 0x1p60f), lv = log2f(vs), iv = 1.f / vs;
            for (int i = b * groups; i < (b + 1) * groups; ++i) {
              info[s].kf[i] = x.ks;
              info[s].lv[i] = lv;
              info[s].iv[i] = iv;
              info[s].valid[i] = x.row < 0 ? 0 : x.vs != x.vs ? 1 | kNanScale : 1;
            }
            *const_cast<volatile uint32_t *>(&info[s].turn) = turn;
            mbar_arrive_expect_tx(full + s, bytes);
          }
          __syncwarp();
        }
        if (dead) {
          sent = __ballot_sync(~0u, own && turn == now && !pending);
          issued = max(issued, now * NS);             // what this batch has sent in earlier turns
          break;
        }
      }
      if (!dead) issued += x.count;
      x = y;
    }
    if (bad && p.status != nullptr) atomicOr(p.status, ERR_BAD_PAGE);
    if (dead && lane == 0 && p.status != nullptr) atomicOr(p.status, ERR_TIMEOUT_ATTEND);
    // No copy is left in flight when the block ends, whether or not a consumer waited for it: each stage by its last
    // turn.  After a wait that ran out in the middle of a turn that is this turn for the boxes that had been sent; the
    // turn before is not waited for on their stages, its parity would not come again.  (The many-row kernel goes by the
    // turns in `info`, without this record; here that cost 1.0 of 50 us, by another allocation of registers.)
    const bool late = sent >> lane & 1;
    for (uint32_t i = issued > NS ? issued - NS : 0; i < issued; ++i)
      if (i % NS / L::kOwn == other && !__any_sync(~0u, late && last_stage == i % NS))
        mbar_wait_bounded(full + i % NS, (i / NS) & 1, kWaitPolls);
    if (late) mbar_wait_bounded(full + last_stage, last_phase, kWaitPolls);
    return;
  }

  // -------------------------------------------------------------------- consumers
  if constexpr (NR > 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(L::kConsumerRegs));
  const int mt = warp % MT, kl = warp / MT;
  const int sg = g ^ ((g & 1) << 2);                  // sigma(g): the token of the lane's score rows
  const int ca = 2 * c, cb = (2 * c + 1) ^ 4;         // sigma(2c), sigma(2c + 1): the tokens of its value pairs
  const uint32_t ring = smem_u32(smem);
  constexpr uint32_t kAllValid = MI == 4 ? 0x01010101u : 0x0101u;
  uint32_t done = 0;                                  // tiles of the items before
  if (p.expire && kl == 0) dead = more;               // its stages are never given back: the others' waits run out

  for (uint32_t item = 0; more && !dead; more = it.next(), ++item) {
    const uint32_t slot = item & 1;
    if (!warp_wait(qfull + slot, item / 2, p.polls)) { dead = true; break; }
    const uint32_t qf = ring + L::kQ + slot * L::kQSlot + (mt * NR * L::kQParts * (D / 32) * 32 + lane) * 16;
    // (factor, limit) of the lane's query rows 8 n + 2 c + e
    const float2 *factor = reinterpret_cast<const float2 *>(smem + L::kQFactor) + slot * R + mt * 8 * NR;
    auto limit = [&](int row) { return __float_as_int(factor[row].y); };
    const int low = limit(0), high = limit(8 * NR - 1);
    float rf[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) { rf[n][0] = factor[8 * n + 2 * c].x; rf[n][1] = factor[8 * n + 2 * c + 1].x; }

    // o: channel tile i, rows' tile n: channels 16 g + 2 i (0, 1) and + 1 (2, 3) of rows 2 c (0, 2) and + 1 (1, 3)
    float o[OI][NR][4] = {}, m[NR][2], l[NR][2] = {};
#pragma unroll
    for (int n = 0; n < NR; ++n) m[n][0] = m[n][1] = -INFINITY;
    for (int u = it.t0 + kl; u < it.t1; u += KL) {
      const uint32_t at = done + (u - it.t0), s = at % NS;
      // A parity tells a phase only from its neighbour, and the stage's previous tile was another warp's: it
      // may still be on its way although later ones have come.  So the tile's turn is waited for first, which
      // the producer writes when the stage is free for it: the barrier is in that phase or just past it then.
      dead = !__all_sync(~0u, wait_turn(&info[s].turn, at / NS, p.polls)) || !warp_wait(full + s, at / NS, p.polls);
      if (dead) break;
      const int base = u * TILE;
      if (base < high) {
        const uint32_t kb = ring + s * kStageBytes, vb = kb + kStageBytes / 2;
        const uint32_t valid = *reinterpret_cast<const uint32_t *>(info[s].valid);
        const bool masked = base + TILE > low || valid != kAllValid;
        float sc[MI][NR][4] = {};
#pragma unroll
        for (int part = 0; part < D / 64; ++part) {   // the pieces c and c + 4 of the key rows
          uint4 w[MI][2];
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int token = 16 * i + 8 * k + sg;
              w[i][k] = D == 128 ? lds128(kb + token * 128 + (((c + 4 * part) ^ sg) << 4))
                                 : lds128(kb + token * 64 + ((c ^ ((token >> 1) & 3)) << 4));
            }
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            uint4 qh[NR], ql[NR];
#pragma unroll
            for (int n = 0; n < NR; ++n) {
              qh[n] = lds128(qf + (n * L::kQParts * (D / 32) + 2 * part + k2) * 512);
              if constexpr (kSplitIO) ql[n] = lds128(qf + (n * L::kQParts * (D / 32) + D / 32 + 2 * part + k2) * 512);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int i = 0; i < MI; ++i) {
                const uint32_t w0 = word_of(w[i][0], 2 * k2 + k), w1 = word_of(w[i][1], 2 * k2 + k);
                const uint32_t a[4] = {codes_lo(w0), codes_lo(w1), codes_hi(w0), codes_hi(w1)};
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                  mma_f16(sc[i][n], a, word_of(qh[n], 2 * k), word_of(qh[n], 2 * k + 1));
                  if constexpr (kSplitIO) mma_f16(sc[i][n], a, word_of(ql[n], 2 * k), word_of(ql[n], 2 * k + 1));
                }
              }
          }
        }
        float top[NR][2], z[NR][2];                   // the maximum; the reference of the weights (0 while there is none)
        bool grew = false;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          float x0 = m[n][0], x1 = m[n][1];
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            float (&v)[4] = sc[i][n];
            const float kf = info[s].kf[i], lv = info[s].lv[i], f0 = rf[n][0] * kf, f1 = rf[n][1] * kf;
            v[0] = fmaf(v[0], f0, lv); v[1] = fmaf(v[1], f1, lv);
            v[2] = fmaf(v[2], f0, lv); v[3] = fmaf(v[3], f1, lv);
            if (masked) {
              const bool in = valid >> (8 * i) & 1;
              const int ta = base + 16 * i + sg, tb = ta + 8;
              const int l0 = limit(8 * n + 2 * c), l1 = limit(8 * n + 2 * c + 1);
              if (!in || ta >= l0) v[0] = -INFINITY;
              if (!in || ta >= l1) v[1] = -INFINITY;
              if (!in || tb >= l0) v[2] = -INFINITY;
              if (!in || tb >= l1) v[3] = -INFINITY;
            }
            x0 = fmaxf(x0, fmaxf(v[0], v[2]));
            x1 = fmaxf(x1, fmaxf(v[1], v[3]));
          }
#pragma unroll
          for (int i = 4; i < 32; i <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(~0u, x0, i));
            x1 = fmaxf(x1, __shfl_xor_sync(~0u, x1, i));
          }
          top[n][0] = x0;
          top[n][1] = x1;
          z[n][0] = x0 == -INFINITY ? 0.f : x0 - kUp;
          z[n][1] = x1 == -INFINITY ? 0.f : x1 - kUp;
          grew |= x0 != m[n][0] || x1 != m[n][1];
        }
        if (__any_sync(~0u, grew)) {
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const float a0 = ex2(m[n][0] - kUp - z[n][0]), a1 = ex2(m[n][1] - kUp - z[n][1]);
            l[n][0] *= a0;
            l[n][1] *= a1;
#pragma unroll
            for (int i = 0; i < OI; ++i) {
              o[i][n][0] *= a0; o[i][n][1] *= a1; o[i][n][2] *= a0; o[i][n][3] *= a1;
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NR; ++n) { m[n][0] = top[n][0]; m[n][1] = top[n][1]; }
        bool nan = false;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const float iv = info[s].iv[i];
          uint32_t pb[NR][2], pl[NR][2];
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            float (&v)[4] = sc[i][n];
            v[0] = ex2(v[0] - z[n][0]); v[1] = ex2(v[1] - z[n][1]);
            v[2] = ex2(v[2] - z[n][0]); v[3] = ex2(v[3] - z[n][1]);
            l[n][0] = fmaf(v[0] + v[2], iv, l[n][0]);
            l[n][1] = fmaf(v[1] + v[3], iv, l[n][1]);
            const uint32_t h0 = pack_f16(v[0], v[1]), h1 = pack_f16(v[2], v[3]);
            pb[n][0] = transpose8(h0);
            pb[n][1] = transpose8(h1);
            if constexpr (kSplitIO) {
              pl[n][0] = transpose8(pack_rest(v[0], v[1], h0, kRestUp));
              pl[n][1] = transpose8(pack_rest(v[2], v[3], h1, kRestUp));
            }
          }
          const int tok[4] = {16 * i + ca, 16 * i + cb, 16 * i + ca + 8, 16 * i + cb + 8};
          Piece<D> v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = load_value<D>(vb, tok[k], g);
            if (masked) {
              // a code that no row sees becomes 0: its weight is 0, but 0 * NaN would not be.  A NaN that
              // some rows see and others do not is put in its rows by hand below.
              const bool in = valid >> (8 * i) & 1, none = !in || base + tok[k] >= high, some = base + tok[k] >= low;
#pragma unroll
              for (int j = 0; j < D / 32; ++j) {
                if (valid >> (8 * i) & kNanScale) v[k].w[j] = 0x7f7f7f7f;
                if (none) v[k].w[j] = 0;
                if (some) {
                  const uint32_t is = __vcmpeq4(v[k].w[j] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                  nan |= is != 0;
                  v[k].w[j] &= ~is;
                }
              }
            }
          }
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint32_t e0 = __byte_perm(v[0].w[j], v[1].w[j], 0x5140), e1 = __byte_perm(v[0].w[j], v[1].w[j], 0x7362);
            const uint32_t e2 = __byte_perm(v[2].w[j], v[3].w[j], 0x5140), e3 = __byte_perm(v[2].w[j], v[3].w[j], 0x7362);
            const uint32_t a0[4] = {codes_lo(e0), codes_hi(e0), codes_lo(e2), codes_hi(e2)};
            const uint32_t a1[4] = {codes_lo(e1), codes_hi(e1), codes_lo(e3), codes_hi(e3)};
            if constexpr (!kSplitIO) {
#pragma unroll
              for (int n = 0; n < NR; ++n) {
                mma_f16(o[2 * j][n], a0, pb[n][0], pb[n][1]);
                mma_f16(o[2 * j + 1][n], a1, pb[n][0], pb[n][1]);
              }
            } else {
              const uint32_t b0[4] = {rest_down(a0[0]), rest_down(a0[1]), rest_down(a0[2]), rest_down(a0[3])};
              const uint32_t b1[4] = {rest_down(a1[0]), rest_down(a1[1]), rest_down(a1[2]), rest_down(a1[3])};
#pragma unroll
              for (int n = 0; n < NR; ++n) {
                float t0[4] = {}, t1[4] = {};
                mma_f16(t0, b0, pl[n][0], pl[n][1]);
                mma_f16(t1, b1, pl[n][0], pl[n][1]);
                mma_f16(t0, a0, pb[n][0], pb[n][1]);
                mma_f16(t1, a1, pb[n][0], pb[n][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) { o[2 * j][n][e] += t0[e]; o[2 * j + 1][n][e] += t1[e]; }
              }
            }
          }
        }
        if (masked && __any_sync(~0u, nan)) {
          const int to = min(base + TILE, high);
          for (int token = max(base, low); token < to; ++token) {
            const uint32_t is = valid >> (8 * ((token - base) / 16));
            if (!(is & 1)) continue;
            const Piece<D> v = load_value<D>(vb, token - base, g);   // the lane's output channels
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              if ((is & kNanScale) || (v.w[i / 4] >> (8 * (i % 4)) & 0x7f) == 0x7f) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    if (token < limit(8 * n + 2 * c + e)) o[i / 2][n][2 * (i % 2) + e] = __int_as_float(0x7fffffff);
              }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + s);
    }
    if (dead) break;
    if (lane == 0) mbar_arrive(qempty + slot);

    // ---- the outputs, to the merger
    const int count = it.t1 - it.t0;
    if (item > 0 && !warp_wait(merged, item - 1, p.polls)) { dead = true; break; }
    const bool upper = kl >= SL, add = !upper && kl + SL < KL && kl + SL < count;   // an output to add one's own to
    if (KL > SL && !upper && !warp_wait(left_up, item, p.polls)) { dead = true; break; }
    if (kl < count) {                                 // (without a tile there is no output)
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[n][e];
#pragma unroll
          for (int i = 4; i < 32; i <<= 1) sum += __shfl_xor_sync(~0u, sum, i);
          const int row = mt * 8 * NR + 8 * n + 2 * c + e;
          const float own = m[n][e] - kUp;            // what the output and the sum are relative to
          float M = own, f = 1.f, fy = 0.f;
          if (add) {
            const float2 ml = stats[(kl + SL) * R + row];
            M = fmaxf(M, ml.x);
            f = fade(own, M);
            fy = fade(ml.x, M);
            sum = f * sum + fy * ml.y;
          }
          if (g == 0) stats[kl * R + row] = make_float2(M, sum);
          float *dst = merge + ((upper ? kl - SL : kl) * R + row) * D;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {          // channels 16 g + 4 i .. + 3 (D = 128)
            float4 *to = reinterpret_cast<float4 *>(dst + 4 * merge_chunk<D>(row, g * (D / 32) + i));
            float4 x = make_float4(o[2 * i][n][e], o[2 * i][n][2 + e], o[2 * i + 1][n][e], o[2 * i + 1][n][2 + e]);
            if (add) {
              const float4 y = *to;
              x = make_float4(f * x.x + fy * y.x, f * x.y + fy * y.y, f * x.z + fy * y.z, f * x.w + fy * y.w);
            }
            *to = x;
          }
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(upper ? left_up : left_all);
    done += count;
  }
  if (dead && lane == 0 && p.status != nullptr) atomicOr(p.status, ERR_TIMEOUT_ATTEND);
}

// Tiles that a block takes of an item at a time.
constexpr int lanes_of(int rows) { return rows == kWideItem ? 1 : rows <= 16 ? 12 : rows == 32 ? 6 : 3; }

// Items with no more tiles than a block takes at a time are not split: that would only add the join.  (Nor
// is a line of tiles that 32 bits cannot count.)
bool whole_items(const kda_cache &c, int rows, int64_t items) {
  const bool wide = rows == kWideItem;
  const int tile = wide ? kWideTile : 4096 / c.head_dim, lead = wide ? kWideLead : kLead;
  const int64_t tiles = ((int64_t)c.max_pages * c.page_tokens + tile - 1) / tile;
  return tiles <= lanes_of(rows) || items > INT32_MAX / (tiles + lead);
}

template <typename IO, int D, int NR, int MT>
cudaError_t launch(AttendParams p, const kda_cache &c, int64_t items, cudaStream_t stream) {
  using L = Layout<IO, D, NR, MT>;
  if (!encode_maps(p, c, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attend_kernel<IO, D, NR, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       L::kBytes);
  if (e != cudaSuccess) return e;
  static_assert(L::kLanes == lanes_of(L::kRows), "what decides about whole items");
  const unsigned grid = p.whole && items < kBlocks ? (unsigned)items : kBlocks;
  attend_kernel<IO, D, NR, MT><<<grid, L::kWarps * 32, L::kBytes, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.whole) return e;
  return launch_join<IO, D, L::kRows>(p, stream);
}

template <typename IO, int D>
cudaError_t launch_rows(const AttendParams &p, const kda_cache &c, int64_t items, int R, cudaStream_t stream) {
  if (R == 8) return launch<IO, D, 1, 1>(p, c, items, stream);
  if constexpr (sizeof(IO) == 4 || wide_from(D) == 32) {
    if (R == 32) return launch<IO, D, 2, 2>(p, c, items, stream);
  }
  if constexpr (sizeof(IO) == 4) {
    if (R == 64) return launch<IO, D, 2, 4>(p, c, items, stream);
  }
  return launch<IO, D, 2, 1>(p, c, items, stream);
}

// Query rows of an item: the fewest column tiles of 8 that hold them, up to 64; bf16 calls with more than wide_from
// rows (per sequence and key / value head) take the tensor cores' kernel and its 128.  That kernel widens every tile
// once for all rows, this one once for every 16 of them.  64 sequences of up to 12345 tokens, 4 heads, that kernel
// against this one (us, cold):
//                  24 rows     32 rows     40 rows     64 rows
//   64 channels    93 /  75    95 /  77    97 / 108   101 / 114
//   128 channels  112 /  99   114 / 103   116 / 159   122 / 167
// With 128 channels the limit is 16 all the same: it was set when this kernel took 132 and 142 there, and the sizes
// of workspaces go by it.
int item_rows(int64_t rows, bool bf16, int D) {
  if (bf16 && rows > wide_from(D)) return kWideItem;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

}  // namespace

size_t cache_attend_workspace(const kda_cache &c, const kda_cache_attend_args &a) {
  const int64_t all = (int64_t)a.num_new * (a.num_heads / c.num_kv_heads);
  const int64_t rows = item_rows(all, a.io_dtype == KDA_BF16, c.head_dim);
  if (whole_items(c, (int)rows, c.num_seqs * ((all + rows - 1) / rows) * c.num_kv_heads)) return 0;
  const int64_t bytes = kBlocks * 16 + kBlocks * 2 * (rows * c.head_dim + 2 * rows) * 4;
  return (size_t)((bytes + 255) / 256 * 256);
}

cudaError_t launch_cache_attend(const kda_cache &c, const kda_cache_attend_args &a, void *workspace,
                                cudaStream_t stream) {
  AttendParams p{};
  p.N = c.num_seqs; p.T = a.num_new; p.Hq = a.num_heads; p.Hk = c.num_kv_heads; p.G = p.Hq / p.Hk;
  p.P = c.page_tokens; p.log_page = p.P == 16 ? 4 : p.P == 32 ? 5 : p.P == 64 ? 6 : 7;
  p.max_pages = c.max_pages; p.num_pages = c.num_pages;
  const bool bf16 = a.io_dtype == KDA_BF16;
  const int R = item_rows(p.T * p.G, bf16, c.head_dim);
  p.RT = (p.T * p.G + R - 1) / R;
  const int tile = R == kWideItem ? kWideStage : c.head_dim == 128 ? kTile<128> : kTile<64>;
  p.box = p.P < tile ? p.P : tile;
  p.boxes = tile / p.box;
  p.q_stride = a.q_stride; p.scale = a.scale; p.q = a.q;
  p.k_scale = c.k_scale; p.v_scale = c.v_scale; p.table = c.block_table; p.lens = c.seq_lens;
  p.o = a.o; p.lse = a.lse; p.status = a.status;
  p.expire = (a.flags & KDA_FLAG_TEST_EXPIRE_WAITS) != 0;
  p.polls = p.expire ? 1u << 12 : kWaitPolls;
  p.desc = static_cast<int4 *>(workspace);
  p.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + kBlocks * 16);
  const int64_t items = (int64_t)p.N * p.RT * p.Hk;
  p.whole = whole_items(c, R, items);
  if (R == kWideItem) return launch_wide(p, c, items, stream);
  if (c.head_dim == 128)
    return bf16 ? launch_rows<__nv_bfloat16, 128>(p, c, items, R, stream)
                : launch_rows<float, 128>(p, c, items, R, stream);
  return bf16 ? launch_rows<__nv_bfloat16, 64>(p, c, items, R, stream)
              : launch_rows<float, 64>(p, c, items, R, stream);
}

}  // namespace kda
