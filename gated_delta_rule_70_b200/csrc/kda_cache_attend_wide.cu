// Attention over the paged 8-bit cache for many query rows per key / value head (speculative tokens of wide
// groups, chunks of a prompt), on the tcgen05 tensor cores: S = Q K^T and O += P V with the item's 128 query rows
// as the rows of both products, so a thread owns a row and no softmax step crosses lanes.
//
// A block of sixteen warps:
//   warp 0       brings 64 cached tokens at a time by TMA into a ring (e4m3, one box per page);
//   warps 4-7    widen them to fp16 (exact) in the layouts the products read, two buffers of 128 tokens each
//                for keys and for values;
//   warp 1       issues the products of a tile of 128 tokens;
//   warps 8-11 and 12-15, two softmax groups: both own every row, the first the tile's first 64 tokens, the
//                second the others.  They agree on the tile's maximum through shared memory, keep a sum each,
//                and bring the queries and store the outputs half a row each.
// Tensor memory (D = 128): two S of 128 columns, whose first 64 then take P (fp16 pairs), O of 128, Q of 64
// (fp16 pairs; as a shared-memory operand the 128 x 128 Q would be read again for every tile).
//
// The reference of the weights is not the exact running maximum: it follows the maximum only when that has
// grown by more than 2^3.5, so the output in tensor memory is rescaled a few times per item instead of with every
// tile.  It lies 2^12 below the maximum it was taken from: weights reach 2^15.5 at most (fp16 holds 2^16 less
// 2^5) and keep their 2^-11 down to 2^-26 of the row's largest; below, fp16's subnormals lose up to 2^-37 of it
// each.  (With 2^8, 1 us less in the case below, and a largest weight of 1 that began at 2^-14: the many small weights of a long sequence, beside
// one token with nearly all of the weight, came out up to 100 % wrong.)
//
// Measured: 512 new tokens of 32 query heads on 4 x 128, 4 sequences of up to 8192 tokens: 320 us, 601 TFLOP/s of
// the products' work that the mask leaves; the tensor pipe is active for 30 % of the time.  A tile takes 2800
// cycles, and two chains are that long: the issuing thread (eight products 650 to 800 cycles, twice, a wait 250 to
// 350, a commit 200) and a softmax warp (scores there 290, loaded 270, their maximum 260, agreed with the other
// group 390, 64 exponentials 1285 with 1024 for the two warps that share a special-function unit, weights stored
// and handed over 330).  Both groups are in the same phase of a tile because they agree on its maximum.
// Slower forms of it, or no faster:
//   tiles of 64 tokens, each group its own (445 us): the issuing thread's waits and commits, about 1200 cycles a
//     tile whatever its size, and products of 64 columns, which run at 60 % of the rate of 128;
//   tiles of 128 tokens, each group its own, the reference handed on from tile to tile (450 us): a group's next
//     scores then wait for its last weights' products, 2300 cycles, and 128 scores a row do not fit in registers;
//   eight widening warps, or codes loaded a part ahead (no change); keys and values issued by two warps (349 us).
#include "cache_attend.cuh"

namespace kda {
namespace attend {
namespace {

constexpr int kTile = kWideTile, kHalf = kTile / 2, kRows = kWideItem, kThreads = 512;
constexpr int kLead = kWideLead;
constexpr int kBuffers = 2, kStages = 4;              // of a tile; of half a tile
// Registers: 512 threads share 65536; the softmax groups hold half a row's 64 scores each.
constexpr int kIssueRegs = 72, kWidenRegs = 88, kSoftmaxRegs = 176;
static_assert(kIssueRegs + kWidenRegs + 2 * kSoftmaxRegs == 4 * 128, "register pool");
constexpr float kUp = 12.f;                           // the largest weight when its reference is taken, as a power of two
constexpr float kSlack = 3.5f;                        // powers of two that a later one may exceed that by
static_assert(kUp + kSlack < 16.f, "weights in fp16");

template <int D> struct Wide {
  static constexpr uint32_t kOperand = kTile * D * 2;               // a widened tile of keys or values
  static constexpr uint32_t kStageBytes = 2 * kHalf * D;            // codes of half a tile's keys and values
  static constexpr uint32_t kRing = 2 * kBuffers * kOperand;        // (keys' buffers, values' buffers, ring)
  static constexpr uint32_t kInfo = kRing + kStages * kStageBytes;  // StageInfo of stages, then of half tiles
  static constexpr uint32_t kNan = kInfo + (kStages + 8) * (uint32_t)sizeof(StageInfo);   // (half tiles of four tiles)
  static constexpr uint32_t kNanBytes = kTile * D / 8;              // per buffer: a bit for each value
  static constexpr uint32_t kMax = kNan + kBuffers * kNanBytes;     // [2 buffers][2 groups][kRows] maxima
  static constexpr uint32_t kSum = kMax + 4 * kRows * 4;            // [2 groups][kRows] sums, then maxima of q
  static constexpr uint32_t kSeen = kSum + 4 * kRows * 4;           // [2 groups][kRows][D / 32] NaN bits
  static constexpr uint32_t kBars = kSeen + 2 * kRows * (D / 8);
  static constexpr uint32_t kSums = kBars + (2 * kStages + 7 * kBuffers + 20) * 8;
  static constexpr uint32_t kLens = kSums + 266 * 4;
  static constexpr uint32_t kBytes = kLens + kLensInSmem * 4;
  static_assert(kNan % 16 == 0 && kBars % 8 == 0 && kBytes <= 232448, "shared memory of one block");
  // tensor memory columns
  static constexpr uint32_t kS = 0, kO = 2 * kTile, kQ = kO + D;
  static_assert(kQ + D / 2 <= 512, "tensor memory");
  static constexpr int kPart = kRows * D + 2 * kRows;
};

// Instruction descriptor for kind::f16 with fp16 A and B and fp32 accumulation (as make_idesc_bf16).
constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// A widened tile: 128 token rows of 64 channels (128 bytes, swizzled) for each 64 channels.
// Keys: K-major; values: MN-major (channels).  A k-step's descriptor is the tile's with the start address
// (in units of 16 bytes) moved on: 16 channels, or 16 tokens.
__device__ __forceinline__ uint64_t key_desc(uint32_t base) { return make_desc(base, 16, 1024, LAYOUT_SW128); }
__device__ __forceinline__ uint64_t value_desc(uint32_t base) {
  return make_desc(base, kTile * 128, 1024, LAYOUT_SW128);
}
constexpr uint32_t key_step(int s) { return ((s >> 2) * kTile * 128 + (s & 3) * 32) >> 4; }
constexpr uint32_t value_step(int s) { return s * 2048 >> 4; }

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// The largest of three; a NaN does not enter.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The pieces of 16 codes of half a tile, number `at` of them: which row and which piece of the row.  D = 128:
// eight neighbours are the lower (or upper) four pieces of rows r and r ^ 5, which meet eight bank groups in
// the codes (rows of 128 bytes under the 128-byte swizzle) and in each store of the widened tile.
template <int D> __device__ __forceinline__ int2 piece_of(int at) {
  if constexpr (D == 64) return make_int2(at >> 2, at & 3);
  const int pair = at >> 3, row = ((pair >> 1) & 3) * 2 + (pair >> 3) * 8;
  return make_int2(row ^ (at & 4 ? 5 : 0), (at & 3) | (pair & 1) << 2);
}
// Widens a piece into the tile at `dst`: 32 bytes of fp16 as two 16-byte units.
__device__ __forceinline__ void widen_piece(uint32_t dst, int row, int c, uint4 w) {
  const int unit = (c & 3) * 2;
  const uint32_t to = dst + (c >> 2) * (kTile * 128) + row * 128;
  sts128(to + ((unit ^ (row & 7)) << 4), make_uint4(codes_lo(w.x), codes_hi(w.x), codes_lo(w.y), codes_hi(w.y)));
  sts128(to + (((unit + 1) ^ (row & 7)) << 4), make_uint4(codes_lo(w.z), codes_hi(w.z), codes_lo(w.w), codes_hi(w.w)));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attend_wide_kernel(const __grid_constant__ AttendParams p) {
  using L = Wide<D>;
  using IO = __nv_bfloat16;
  constexpr int DW = D / 32;                          // words of a row's channel bits
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  StageInfo *info = reinterpret_cast<StageInfo *>(smem + L::kInfo), *wide_info = info + kStages;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBars), *empty = full + kStages;
  // of the tile's buffers, by tile % 2: widened keys and values there / used up, scores, weights, outputs
  uint64_t *k_full = empty + kStages, *k_free = k_full + kBuffers, *v_full = k_free + kBuffers;
  uint64_t *v_free = v_full + kBuffers, *s_full = v_free + kBuffers, *p_full = s_full + kBuffers;
  uint64_t *o_done = p_full + kBuffers;
  uint64_t *agreed = o_done + kBuffers;               // maxima: [buffer][quarter of the rows]
  uint64_t *q_max = agreed + 8, *q_full = q_max + 4, *ended = q_full + 1;   // [quarter], one, [quarter]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ended + 4);
  uint32_t *sums = reinterpret_cast<uint32_t *>(smem + L::kSums);
  int32_t *slens = reinterpret_cast<int32_t *>(smem + L::kLens);
  float *maxima = reinterpret_cast<float *>(smem + L::kMax), *ends = reinterpret_cast<float *>(smem + L::kSum);
  uint32_t *seen_nan = reinterpret_cast<uint32_t *>(smem + L::kSeen);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      *reinterpret_cast<uint32_t *>(info[i].valid) = 0;
      info[i].turn = ~0u;
      mbar_init(full + i, p.boxes);
      mbar_init(empty + i, 4);
    }
    for (int i = 0; i < kBuffers; ++i) {
      mbar_init(k_full + i, 4);
      mbar_init(k_free + i, 1);
      mbar_init(v_full + i, 4);
      mbar_init(v_free + i, 1);
      mbar_init(s_full + i, 2);
      mbar_init(p_full + i, 8);
      mbar_init(o_done + i, 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(agreed + i, 2);
    for (int i = 0; i < 4; ++i) { mbar_init(q_max + i, 2); mbar_init(ended + i, 2); }
    mbar_init(q_full, 8);
    mbar_fence_init();
  }
  if (threadIdx.x == 64) {
    tma_prefetch_desc(&p.map_k);
    tma_prefetch_desc(&p.map_v);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  const int cap = p.max_pages * p.P;
  const bool small = p.N <= kLensInSmem;
  for (int n = threadIdx.x; n < p.N && (small || blockIdx.x == 0); n += kThreads) {
    const int len = p.lens[n];
    if (small) slens[n] = len;
    if (blockIdx.x == 0 && p.status != nullptr && (len < 0 || len > cap)) atomicOr(p.status, ERR_BAD_LENGTH);
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int32_t *lens = small ? slens : p.lens;
  Line line{0, 0, 0};
  if (!p.whole) line = lay_out<kRows, kTile, kLead>(p, lens, sums, 1);
  // the join may be set up now: it waits for the whole grid before it reads anything
  cudaTriggerProgrammaticLaunchCompletion();
  Walker<kRows, kTile, kLead> it(p, lens);
  bool more = p.whole ? it.begin_whole(blockIdx.x) : it.begin_split(line.first, (int)sums[264], sums, line.per);
  bool dead = false;
  const int rows = p.T * p.G;
  const uint32_t smem0 = smem_u32(smem);
  // tokens that a row of the item sees: all below
  auto limit = [&](int row) { return it.len - p.T + min(it.rt * kRows + row, rows - 1) / p.G + 1; };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kIssueRegs));
    if (warp == 0) {
      // -------------------------------------------------------------- the producer
      // A lane has one box of a tile to itself; a batch is what the lanes look up at once, and the next batch
      // is looked up before the present one is issued, across items too.
      bool bad = false;
      uint32_t issued = 0;
      const int per_batch = 32 / p.boxes, groups = 4 / p.boxes;   // half tiles; 16-token groups of a box
      const int b = lane % p.boxes, ahead = lane / p.boxes;
      struct Batch { int count, row; float ks, vs; };
      int at = 2 * it.t0;                             // half tiles
      auto look_up = [&](Batch &x) {
        x.count = 0;
        x.row = -1;
        x.ks = x.vs = 1.f;
        if (!more) return;
        x.count = min(per_batch, 2 * it.t1 - at);
        const int token = (at + ahead) * kHalf + b * p.box;
        if (ahead < x.count && token < visible(it.len, p.T, p.G, kRows, it.rt)) {
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
        if (at >= 2 * it.t1) { more = it.next(); at = 2 * it.t0; }
      };
      Batch x, y;
      look_up(x);
      while (x.count > 0 && !dead) {
        look_up(y);
        const uint32_t tile = issued + ahead, turn = tile / kStages, s = tile - turn * kStages;
        const uint32_t bytes = x.row >= 0 ? 2 * p.box * D : 0;
        unsigned char *dst = smem + L::kRing + s * L::kStageBytes + b * p.box * D;
        const uint32_t last = (issued + x.count - 1) / kStages;
        for (uint32_t now = issued / kStages; now <= last; ++now) {
          // each box goes out as soon as its stage is free; a stage's next turn only after this one
          bool pending = ahead < x.count && turn == now;
          for (uint32_t poll = 0; __any_sync(~0u, pending); ++poll) {
            if (poll >= p.polls) { dead = true; break; }
            if (pending && (turn == 0 || mbar_try_wait(empty + s, (turn - 1) & 1))) {
              pending = false;
              if (x.row >= 0) {
                tma_load_2d(dst, &p.map_k, 0, x.row, full + s);
                tma_load_2d(dst + L::kStageBytes / 2, &p.map_v, 0, x.row, full + s);
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
          if (dead) break;
        }
        issued += x.count;
        x = y;
      }
      if (bad && p.status != nullptr) atomicOr(p.status, ERR_BAD_PAGE);
      // no copy is left in flight when the block ends: each stage by the turn it was given last, which after a wait
      // that ran out is not the same for all
      __syncwarp();
      for (int s = 0; s < kStages; ++s) {
        const uint32_t turn = *const_cast<volatile uint32_t *>(&info[s].turn);
        if (turn != ~0u) mbar_wait_bounded(full + s, turn & 1, kWaitPolls);
      }
    } else if (warp == 1 && lane == 0) {
      // -------------------------------------------------------------- the products
      // S of tile i goes out before O of tile i - 1: the softmax groups find their next scores there when they
      // are done with the last, and the weights are multiplied while they work on those.  S i takes the place
      // of P i - 2, so O i - 2 has to be done.
      const uint32_t id_s = idesc_f16(128, kTile, 0), id_o = idesc_f16(128, D, 1);
      uint32_t done = 0;                              // tiles of the items before
      uint64_t *last = nullptr;                       // the latest commit and its phase
      uint32_t last_phase = 0;
      auto wait = [&](uint64_t *bar, uint32_t phase) {
        dead = dead || !mbar_wait_bounded(bar, phase & 1, p.polls);
        return !dead;
      };
      for (uint32_t item = 0; more && wait(q_full, item); more = it.next(), ++item) {
        const int count = it.t1 - it.t0;
        for (int i = 0; i <= count; ++i) {
          if (i < count) {
            const uint32_t tile = done + i, buf = tile & 1, turn = tile >> 1;
            if (!wait(k_full + buf, turn) || (turn > 0 && !wait(o_done + buf, turn - 1))) break;
            fence_after_sync();
            // (s_full takes an arrival of this thread beside the products': it hands on what the widening warps
            // wrote, the scales; k_full itself may be two phases on by the time a softmax warp looks)
            mbar_arrive(s_full + buf);
            const uint64_t keys = key_desc(smem0 + buf * L::kOperand);
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              mma_ts(tmem + L::kS + buf * kTile, tmem + L::kQ + s * 8, keys + key_step(s), id_s, s > 0);
            mma_commit(s_full + buf);
            mma_commit(k_free + buf);
            last = k_free + buf;
            last_phase = turn;
          }
          if (i > 0) {
            const uint32_t tile = done + i - 1, buf = tile & 1, turn = tile >> 1;
            if (!wait(v_full + buf, turn) || !wait(p_full + buf, turn)) break;
            fence_after_sync();
            const uint64_t values = value_desc(smem0 + (kBuffers + buf) * L::kOperand);
#pragma unroll
            for (int s = 0; s < kTile / 16; ++s)
              mma_ts(tmem + L::kO, tmem + L::kS + buf * kTile + s * 8, values + value_step(s), id_o, i > 1 || s > 0);
            mma_commit(o_done + buf);
            mma_commit(v_free + buf);
            last = v_free + buf;
            last_phase = turn;
          }
        }
        if (dead) break;
        done += count;
      }
      // nothing of this block's may still run on the tensor cores when tensor memory is freed
      if (last != nullptr) (void)mbar_wait_bounded(last, last_phase & 1, kWaitPolls);
    }
    __syncwarp();
  } else if (warp < 8) {
    // ------------------------------------------------------------------ widening
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kWidenRegs));
    const int tid = threadIdx.x - 128;
    constexpr int kPieces = kHalf * D / 16 / 128, kRow = D / 16;   // 16-code pieces a thread has of a half; of a row
    uint32_t tile = 0;
    for (; more && !dead; more = it.next()) {
      const int low = limit(0), high = limit(kRows - 1);
      for (int u = it.t0; u < it.t1; ++u, ++tile) {
        const uint32_t buf = tile & 1, turn = tile >> 1;
#pragma unroll
        for (int v = 0; v < 2; ++v) {                 // keys, then values
          if (turn > 0 && !warp_wait((v ? v_free : k_free) + buf, turn - 1, p.polls)) { dead = true; break; }
          const uint32_t dst = smem0 + (v * kBuffers + buf) * L::kOperand;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t stage = 2 * tile + half, s = stage % kStages;
            if (v == 0 && !warp_wait(full + s, stage / kStages, p.polls)) { dead = true; break; }
            const uint32_t src = smem0 + L::kRing + s * L::kStageBytes + v * (L::kStageBytes / 2);
            const int base = u * kTile + half * kHalf;
            const uint32_t valid = *reinterpret_cast<const uint32_t *>(info[s].valid);
            uint4 w[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
              const int2 at = piece_of<D>(tid + i * 128);
              w[i] = lds128(src + at.x * D + ((D == 128 ? at.y ^ (at.x & 7) : at.y) << 4));
            }
            uint32_t found = 0;
            if (v == 0) {
              // (four tiles' worth: the scales of tile - 2 may still be read when its keys are used up)
              StageInfo &to = wide_info[2 * (tile & 3) + half];
              if (tid < 4) {
                to.kf[tid] = info[s].kf[tid];
                to.lv[tid] = info[s].lv[tid];
                to.iv[tid] = info[s].iv[tid];
                if (tid == 0) *reinterpret_cast<uint32_t *>(to.valid) = valid;
              }
            } else if (base + kHalf > low || valid != 0x01010101u) {
              // a value that no row sees becomes 0: its weight is 0, but 0 * NaN would not be.  A NaN that some
              // rows see and others do not becomes 0 too, and a bit by which the rows that see it find it.
              uint16_t *nan = reinterpret_cast<uint16_t *>(smem + L::kNan + buf * L::kNanBytes) + half * kHalf * kRow;
#pragma unroll
              for (int i = 0; i < kPieces; ++i) {
                const int2 at = piece_of<D>(tid + i * 128);
                const int row = at.x;
                uint32_t e[4] = {w[i].x, w[i].y, w[i].z, w[i].w}, bits = 0;
                const bool none = !(valid >> (8 * (row / 16)) & 1) || base + row >= high, some = base + row >= low;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (valid >> (8 * (row / 16)) & kNanScale) e[k] = 0x7f7f7f7f;
                  if (none) e[k] = 0;
                  if (some) {
                    const uint32_t is = __vcmpeq4(e[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                    e[k] &= ~is;
                    bits |= ((is & 0x01010101u) * 0x01020408u >> 24 & 15u) << (4 * k);
                  }
                }
                nan[row * kRow + at.y] = (uint16_t)bits;
                found |= bits;
                w[i] = make_uint4(e[0], e[1], e[2], e[3]);
              }
            }
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
              const int2 at = piece_of<D>(tid + i * 128);
              widen_piece(dst, half * kHalf + at.x, at.y, w[i]);
            }
            if (v == 1) {
              // each widening warp's byte: it found a NaN, so the bits are worth reading
              found = __any_sync(~0u, found != 0);
              __syncwarp();
              if (lane == 0) {
                reinterpret_cast<uint8_t *>(wide_info[2 * (tile & 3) + half].pad)[warp - 4] = (uint8_t)found;
                mbar_arrive(empty + s);
              }
            }
          }
          if (dead) break;
          fence_proxy_async_smem();                   // the products read it through the async proxy
          __syncwarp();
          if (lane == 0) mbar_arrive((v ? v_full : k_full) + buf);
        }
        if (dead) break;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftmaxRegs));
    const int x = warp >= 12, row = threadIdx.x & 127, quarter = warp & 3;
    const uint32_t tm = tmem + ((uint32_t)quarter * 32u << 16);      // the warp's lanes of tensor memory
    int4 split = make_int4(-1, 0, 0, 0);
    uint32_t done = 0;
    // a value of each row's other half, through shared memory and a barrier of the two warps that share the rows
    auto exchange = [&](float *place, uint64_t *bar, uint32_t phase, float mine, float &other) {
      place[x * kRows + row] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
      if (!warp_wait(bar, phase, p.polls)) return false;
      other = place[(1 - x) * kRows + row];
      return true;
    };
    for (uint32_t item = 0; more && !dead; more = it.next(), ++item) {
      const int lim = limit(row), low = limit(0), r = min(it.rt * kRows + row, rows - 1), t = r / p.G;
      float rf;
      {
        // half the row of q, by a power of two in [2^14, 2^15), to tensor memory; rows behind the last repeat it
        const IO *src = static_cast<const IO *>(p.q) + ((int64_t)it.n * p.T + t) * p.q_stride +
                        (int64_t)(it.h * p.G + r - t * p.G) * D + x * (D / 2);
        Held8<IO> q[D / 16];
        float big = 0.f, other = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) q[i].load(src + 8 * i);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) big = fmaxf(big, q[i].amax());
        if (!exchange(ends + 2 * kRows, q_max + quarter, item, big, other)) { dead = true; break; }
        big = fmaxf(big, other);
        int e = 14 - ((int)(__float_as_uint(big) >> 23) - 127);
        e = e < -120 ? -120 : (e > 120 ? 120 : e);
        const float up = __uint_as_float((uint32_t)(127 + e) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
        rf = p.scale * kLog2e * down;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float y[8];
            q[4 * i + k].get(y);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * k + j] = pack_f16(y[2 * j] * up, y[2 * j + 1] * up);
          }
          tmem_st16(tm + L::kQ + x * (D / 4) + 16 * i, w);
        }
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      if (p.expire && x == 0) { dead = true; break; } // the scores' products are under way, the others' waits run out
      const int count = it.t1 - it.t0;
      float m = -INFINITY, l = 0.f;
      uint32_t nans[DW] = {};
      for (int i = 0; i < count; ++i) {
        const uint32_t tile = done + i, buf = tile & 1, turn = tile >> 1;
        if (!warp_wait(s_full + buf, turn, p.polls)) { dead = true; break; }
        fence_after_sync();
        uint32_t sr[2][32];
        tmem_ld32(tm + L::kS + buf * kTile + x * kHalf, sr[0]);
        tmem_ld32(tm + L::kS + buf * kTile + x * kHalf + 32, sr[1]);
        const StageInfo &sc = wide_info[2 * (tile & 3) + x];
        const int base = (it.t0 + i) * kTile + x * kHalf;
        const uint32_t valid = *reinterpret_cast<const uint32_t *>(sc.valid);
        const bool masked = base + kHalf > low || valid != 0x01010101u;
        float kf[4], lv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) { kf[k] = rf * sc.kf[k]; lv[k] = sc.lv[k]; }
        float tops[4];                                // of each 16 tokens, which share a factor
        tmem_wait_ld();
        if (!masked && fminf(fminf(kf[0], kf[1]), fminf(kf[2], kf[3])) >= 0.f) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint32_t (&v)[32] = sr[g / 2];
            const int c = g % 2 * 16;
            float t = max3(__uint_as_float(v[c]), __uint_as_float(v[c + 1]), __uint_as_float(v[c + 2]));
#pragma unroll
            for (int j = 3; j < 15; j += 2) t = max3(t, __uint_as_float(v[c + j]), __uint_as_float(v[c + j + 1]));
            tops[g] = fmaf(fmaxf(t, __uint_as_float(v[c + 15])), kf[g], lv[g]);
          }
        } else {
          // the hidden scores become -inf; what is kept here needs no factor any more
#pragma unroll
          for (int k = 0; k < 4; ++k) tops[k] = -INFINITY;
#pragma unroll
          for (int j = 0; j < kHalf; ++j) {
            float s = fmaf(__uint_as_float(sr[j / 32][j % 32]), kf[j / 16], lv[j / 16]);
            if (base + j >= lim || !(valid >> (8 * (j / 16)) & 1)) s = -INFINITY;
            sr[j / 32][j % 32] = __float_as_uint(s);
            tops[j / 16] = fmaxf(tops[j / 16], s);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) { kf[k] = 1.f; lv[k] = 0.f; }
        }
        float top = fmaxf(m, fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]))), other;
        // (also: both halves' scores of these rows are in registers, P may take their place)
        fence_before_sync();
        if (!exchange(maxima + buf * 2 * kRows, agreed + 4 * buf + quarter, turn, top, other)) { dead = true; break; }
        fence_after_sync();
        top = fmaxf(top, other);
        const bool grew = m != -INFINITY && top - m > kUp + kSlack;
        if (m == -INFINITY) m = top - kUp;            // no weight yet: the output is 0, the reference free
        if (__any_sync(~0u, grew)) {
          const float old = m;
          m = fmaxf(m, top - kUp);
          const float f = m == old ? 1.f : ex2(old - m);
          l *= f;
          // the products are done with this item's output so far (the tile before has the other buffer)
          if (!warp_wait(o_done + (buf ^ 1), (tile - 1) >> 1, p.polls)) { dead = true; break; }
          fence_after_sync();
          uint32_t w[32];
#pragma unroll 1
          for (int c = x * (D / 2); c < (x + 1) * (D / 2); c += 32) {
            tmem_ld32(tm + L::kO + c, w);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * f);
            tmem_st32(tm + L::kO + c, w);
          }
        }
        const float z = m == -INFINITY ? 0.f : m;
        uint32_t pr[32];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float2 factor = make_float2(kf[g], kf[g]), shift = make_float2(lv[g], lv[g]);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = 16 * g + 2 * j;
            float2 w = fma2(make_float2(__uint_as_float(sr[c / 32][c % 32]), __uint_as_float(sr[c / 32][c % 32 + 1])),
                            factor, shift);
            // (apart from the product, so that the difference from the maximum, which was rounded like this score, is
            // exact: with -z as a part of the product's shift, 3 us less in the case above, scores beyond 2^22 gave
            // weights beyond fp16)
            w = add2(w, make_float2(-z, -z));
            w.x = ex2(w.x);
            w.y = ex2(w.y);
            sum = add2(sum, w);
            pr[8 * g + j] = pack_f16(w.x, w.y);
          }
          l = fmaf(sum.x + sum.y, sc.iv[g], l);
        }
        tmem_st32(tm + L::kS + buf * kTile + x * (kHalf / 2), pr);
        if (masked) {                                 // NaN values that this row sees and others do not
          if (!warp_wait(v_full + buf, turn, p.polls)) { dead = true; break; }
          const uint32_t *bits = reinterpret_cast<const uint32_t *>(smem + L::kNan + buf * L::kNanBytes) + x * kHalf * DW;
          const int to = sc.pad[0] == 0 ? 0 : min(base + kHalf, lim);
          for (int token = max(base, low); token < to; ++token)
#pragma unroll
            for (int k = 0; k < DW; ++k) nans[k] |= bits[(token - base) * DW + k];
        }
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + buf);
      }
      if (dead) break;
      // ---- the item's end: each group stores half of every row
      const uint32_t end = done + count - 1;
      if (!warp_wait(o_done + (end & 1), end >> 1, p.polls)) { dead = true; break; }
      fence_after_sync();
#pragma unroll
      for (int k = 0; k < DW; ++k) seen_nan[(x * kRows + row) * DW + k] = nans[k];
      float other;
      if (!exchange(ends, ended + quarter, item, l, other)) { dead = true; break; }
      const float sum = x == 0 ? l + other : other + l;   // (the same order in both)
      const bool whole = it.starts && it.ends, real = it.rt * kRows + row < rows;
      float *part = p.parts + ((int64_t)blockIdx.x * 2 + (it.starts ? 1 : 0)) * L::kPart;
      const int64_t orow = ((int64_t)it.n * p.T + t) * p.Hq + it.h * p.G + (r - t * p.G);
      const float f = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;     // no weight at all: o = 0
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const int c = x * (D / 2) + 32 * j;
        uint32_t a[32];
        tmem_ld32(tm + L::kO + c, a);
        tmem_wait_ld();
        const uint32_t bad = seen_nan[row * DW + c / 32] | seen_nan[(kRows + row) * DW + c / 32];
        float y[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          y[k] = __uint_as_float(a[k]) * f;
          if (bad >> k & 1) y[k] = __int_as_float(0x7fffffff);
        }
        if (real && whole) {
          IO *dst = static_cast<IO *>(p.o) + orow * D + c;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float z[8] = {y[8 * k], y[8 * k + 1], y[8 * k + 2], y[8 * k + 3],
                                y[8 * k + 4], y[8 * k + 5], y[8 * k + 6], y[8 * k + 7]};
            store8(dst + 8 * k, z);
          }
        } else if (real) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<float4 *>(part + row * D + c + 4 * k) =
                make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
        }
      }
      if (x == 0 && real && whole) {
        if (p.lse != nullptr) p.lse[orow] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
      } else if (x == 0 && real) {
        part[kRows * D + row] = m;
        part[kRows * D + kRows + row] = sum;
      }
      fence_before_sync();                            // (the loads above, before the next item's products)
      if (it.starts && !it.ends)
        split = make_int4(it.n, it.rt, it.h, (int)((it.stop - 1) / line.share));
      done += count;
    }
    if (!p.whole && threadIdx.x == 256) p.desc[blockIdx.x] = split;
  }
  if (dead && lane == 0 && p.status != nullptr) atomicOr(p.status, ERR_TIMEOUT_ATTEND);
  __syncwarp();
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(AttendParams p, const kda_cache &c, int64_t items, cudaStream_t stream) {
  using L = Wide<D>;
  if (!encode_maps(p, c, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attend_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  const unsigned grid = p.whole && items < kBlocks ? (unsigned)items : kBlocks;
  attend_wide_kernel<D><<<grid, kThreads, L::kBytes, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.whole) return e;
  return launch_join<__nv_bfloat16, D, kRows>(p, stream);
}

}  // namespace

cudaError_t launch_wide(AttendParams p, const kda_cache &c, int64_t items, cudaStream_t stream) {
  return c.head_dim == 128 ? launch<128>(p, c, items, stream) : launch<64>(p, c, items, stream);
}

}  // namespace attend
}  // namespace kda
