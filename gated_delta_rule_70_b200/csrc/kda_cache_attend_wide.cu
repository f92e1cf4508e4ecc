// Attention over the paged 8-bit cache for many query rows per key / value head (speculative tokens of wide
// groups, chunks of a prompt), on the tcgen05 tensor cores: S = Q K^T and O += P V with the item's 128 query rows
// as the rows of both products, so a thread owns a row and no softmax step crosses lanes.
//
// A block of sixteen warps:
//   warp 0       brings tiles of 64 cached tokens by TMA into a ring (e4m3, one box per page);
//   warps 4-7    widen them to fp16 (exact) in the layouts the products read, four buffers;
//   warp 1       issues the products;
//   warps 8-11 and 12-15, two softmax groups that take the tiles in turn, each with a running reference, sum
//                and output of its own; the first also brings the queries and, at the item's end, adds the
//                second's output to its own and stores.
// Tensor memory (D = 128, all 512 columns): two S of 64, two P of 32 (fp16 pairs), two O of 128, Q of 64 (fp16
// pairs; as a shared-memory operand the 128 x 128 Q would be read again for every tile, and with the widened
// tiles shared memory is what bounds the loop).
//
// The reference of the weights is not the exact running maximum: it follows the maximum only when that has
// grown by more than 2^8, so weights reach 2^8 at most (fp16 holds 2^15) and the output in tensor memory is
// rescaled a few times per item instead of with every tile.
#include "cache_attend.cuh"

namespace kda {
namespace attend {
namespace {

constexpr int kTile = kWideTile, kRows = kWideItem, kThreads = 512;
constexpr int kBuffers = 4, kStages = 4;
// Registers: 512 threads share 65536; the softmax groups hold a row's 64 scores each.
constexpr int kIssueRegs = 72, kWidenRegs = 88, kSoftmaxRegs = 176;
static_assert(kIssueRegs + kWidenRegs + 2 * kSoftmaxRegs == 4 * 128, "register pool");
constexpr float kSlack = 8.f;                         // powers of two that a weight may exceed 1 by

template <int D> struct Wide {
  static constexpr uint32_t kOperand = kTile * D * 2;               // a widened tile of keys or values
  static constexpr uint32_t kStageBytes = 2 * kTile * D;            // codes of keys and values
  static constexpr uint32_t kRing = kBuffers * 2 * kOperand;
  static constexpr uint32_t kInfo = kRing + kStages * kStageBytes;  // StageInfo of stages, then of buffers
  static constexpr uint32_t kNan = kInfo + (kStages + kBuffers) * (uint32_t)sizeof(StageInfo);
  static constexpr uint32_t kNanBytes = kTile * D / 8;              // per buffer: a bit for each value
  static constexpr uint32_t kFactor = kNan + kBuffers * kNanBytes;  // [kRows]
  static constexpr uint32_t kSecond = kFactor + kRows * 4;          // the second group's (m, l) and NaN bits, by row
  static constexpr uint32_t kSecondBytes = 8 + D / 8;
  static constexpr uint32_t kBars = kSecond + kRows * kSecondBytes;
  static constexpr uint32_t kSums = kBars + (2 * kStages + 2 * kBuffers + 12) * 8;
  static constexpr uint32_t kLens = kSums + 266 * 4;
  static constexpr uint32_t kBytes = kLens + kLensInSmem * 4;
  static_assert(kNan % 16 == 0 && kBars % 8 == 0 && kBytes <= 232448, "shared memory of one block");
  // tensor memory columns
  static constexpr uint32_t kS = 0, kP = 2 * kTile, kO = kP + kTile, kQ = kO + 2 * D;
  static_assert(kQ + D / 2 <= 512, "tensor memory");
  static constexpr int kPart = kRows * D + 2 * kRows;
};

// Instruction descriptor for kind::f16 with fp16 A and B and fp32 accumulation (as make_idesc_bf16).
constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// A widened tile: 64 token rows of 64 channels (128 bytes, swizzled) for each 64 channels.
// Keys: K-major; values: MN-major (channels).  A k-step's descriptor is the tile's with the start address
// (in units of 16 bytes) moved on: 16 channels, or 16 tokens.
__device__ __forceinline__ uint64_t key_desc(uint32_t base) { return make_desc(base, 16, 1024, LAYOUT_SW128); }
__device__ __forceinline__ uint64_t value_desc(uint32_t base) {
  return make_desc(base, kTile * 128, 1024, LAYOUT_SW128);
}
constexpr uint32_t key_step(int s) { return ((s >> 2) * kTile * 128 + (s & 3) * 32) >> 4; }
constexpr uint32_t value_step(int s) { return s * 2048 >> 4; }

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attend_wide_kernel(const __grid_constant__ AttendParams p) {
  using L = Wide<D>;
  using IO = __nv_bfloat16;
  constexpr int DW = D / 32;                          // words of a row's channel bits
  extern __shared__ __align__(1024) unsigned char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  StageInfo *info = reinterpret_cast<StageInfo *>(smem + L::kInfo), *wide_info = info + kStages;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::kBars), *empty = full + kStages;
  uint64_t *kv_full = empty + kStages, *kv_free = kv_full + kBuffers;
  uint64_t *s_full = kv_free + kBuffers, *s_free = s_full + 2, *p_full = s_free + 2, *pv_done = p_full + 2;
  uint64_t *q_full = pv_done + 2, *second_full = q_full + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(second_full + 1);
  uint32_t *sums = reinterpret_cast<uint32_t *>(smem + L::kSums);
  int32_t *slens = reinterpret_cast<int32_t *>(smem + L::kLens);
  float *factors = reinterpret_cast<float *>(smem + L::kFactor);
  float2 *second = reinterpret_cast<float2 *>(smem + L::kSecond);                    // [kRows]
  uint32_t *second_nan = reinterpret_cast<uint32_t *>(smem + L::kSecond + kRows * 8);  // [kRows][DW]

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      *reinterpret_cast<uint32_t *>(info[i].valid) = 0;
      mbar_init(full + i, p.boxes);
      mbar_init(empty + i, 4);
    }
    for (int i = 0; i < kBuffers; ++i) { mbar_init(kv_full + i, 4); mbar_init(kv_free + i, 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(s_free + i, 4);
      mbar_init(p_full + i, 4);
      mbar_init(pv_done + i, 1);
    }
    mbar_init(q_full, 4);
    mbar_init(second_full, 4);
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
  if (!p.whole) line = lay_out<kRows, kTile>(p, lens, sums, 2);   // a tile for each softmax group at least
  // the join may be set up now: it waits for the whole grid before it reads anything
  cudaTriggerProgrammaticLaunchCompletion();
  Walker<kRows, kTile> it(p, lens);
  bool more = p.whole ? it.begin_whole(blockIdx.x) : it.begin_split(line.first, (int)sums[264], sums, line.per);
  bool dead = p.polls == 0 && more;
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
      uint32_t issued = 0, sent = 0, last_stage = 0, last_phase = 0;
      const int per_batch = 32 / p.boxes, groups = 4 / p.boxes;
      const int b = lane % p.boxes, ahead = lane / p.boxes;
      struct Batch { int count, row; float ks, vs; };
      int at = it.t0;
      auto look_up = [&](Batch &x) {
        x.count = 0;
        x.row = -1;
        x.ks = x.vs = 1.f;
        if (!more) return;
        x.count = min(per_batch, it.t1 - at);
        const int token = (at + ahead) * kTile + b * p.box;
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
        if (at >= it.t1) { more = it.next(); at = it.t0; }
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
          const bool own = ahead < x.count && turn == now;
          bool pending = own;
          for (uint32_t poll = 0; __any_sync(~0u, pending); ++poll) {
            if (poll >= p.polls) { dead = true; break; }
            if (pending && (turn == 0 || mbar_try_wait(empty + s, (turn - 1) & 1))) {
              pending = false;
              last_stage = s;
              last_phase = turn & 1;
              if (x.row >= 0) {
                tma_load_2d(dst, &p.map_k, 0, x.row, full + s);
                tma_load_2d(dst + L::kStageBytes / 2, &p.map_v, 0, x.row, full + s);
              }
              const float vs = fminf(fmaxf(x.vs, 0x1p-60f), 0x1p60f), lv = log2f(vs), iv = 1.f / vs;
              for (int i = b * groups; i < (b + 1) * groups; ++i) {
                info[s].kf[i] = x.ks;
                info[s].lv[i] = lv;
                info[s].iv[i] = iv;
                info[s].valid[i] = x.row >= 0;
              }
              mbar_arrive_expect_tx(full + s, bytes);
            }
            __syncwarp();
          }
          if (dead) {
            sent = __ballot_sync(~0u, own && !pending);
            issued = max(issued, now * kStages);      // what this batch has sent in earlier turns
            break;
          }
        }
        if (!dead) issued += x.count;
        x = y;
      }
      if (bad && p.status != nullptr) atomicOr(p.status, ERR_BAD_PAGE);
      // no copy is left in flight when the block ends, whether or not somebody waited for it
      for (uint32_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
        mbar_wait_bounded(full + i % kStages, (i / kStages) & 1, kWaitPolls);
      if (sent >> lane & 1) mbar_wait_bounded(full + last_stage, last_phase, kWaitPolls);
    } else if (warp == 1 && lane == 0) {
      // -------------------------------------------------------------- the products
      // S of tile i goes out before O of tile i - 2: a softmax group finds its next scores there when it is
      // done with the last, and its weights are multiplied while it works on those (with O of tile i - 1
      // there, a group waited as long for scores as it worked on them: 484 us for attend_chunk_512).
      const uint32_t id_s = idesc_f16(128, kTile, 0), id_o = idesc_f16(128, D, 1);
      uint32_t done = 0, turns[2] = {0, 0};           // tiles of the items before; of each softmax group
      uint64_t *last = nullptr;                       // the latest commit and its phase
      uint32_t last_phase = 0;
      auto wait = [&](uint64_t *bar, uint32_t phase) {
        dead = dead || !mbar_wait_bounded(bar, phase & 1, p.polls);
        return !dead;
      };
      for (uint32_t item = 0; more && wait(q_full, item); more = it.next(), ++item) {
        const int count = it.t1 - it.t0;
        for (int i = 0; i < count + 2; ++i) {
          const int x = i & 1;                        // (of tile i - 2 too)
          if (i < count) {
            const uint32_t tile = done + i, buf = tile % kBuffers, turn = turns[x] + (i > 1);
            if (!wait(kv_full + buf, tile / kBuffers) || (turn > 0 && !wait(s_free + x, turn - 1))) break;
            fence_after_sync();
            const uint64_t keys = key_desc(smem0 + buf * 2 * L::kOperand);
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              mma_ts(tmem + L::kS + x * kTile, tmem + L::kQ + s * 8, keys + key_step(s), id_s, s > 0);
            mma_commit(s_full + x);
            last = s_full + x;
            last_phase = turn;
          }
          if (i > 1 && i - 2 < count) {
            const uint32_t tile = done + i - 2, buf = tile % kBuffers;
            if (!wait(p_full + x, turns[x])) break;
            fence_after_sync();
            const uint64_t values = value_desc(smem0 + buf * 2 * L::kOperand + L::kOperand);
#pragma unroll
            for (int s = 0; s < kTile / 16; ++s)
              mma_ts(tmem + L::kO + x * D, tmem + L::kP + x * (kTile / 2) + s * 8, values + value_step(s), id_o,
                     i > 3 || s > 0);
            mma_commit(pv_done + x);
            mma_commit(kv_free + buf);
            last = kv_free + buf;
            last_phase = tile / kBuffers;
            ++turns[x];
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
    uint32_t tile = 0;
    for (; more && !dead; more = it.next()) {
      const int low = limit(0), high = limit(kRows - 1);
      for (int u = it.t0; u < it.t1; ++u, ++tile) {
        const uint32_t s = tile % kStages, buf = tile % kBuffers;
        if (!warp_wait(full + s, tile / kStages, p.polls) ||
            (tile >= kBuffers && !warp_wait(kv_free + buf, tile / kBuffers - 1, p.polls))) {
          dead = true;
          break;
        }
        const int base = u * kTile;
        const uint32_t valid = *reinterpret_cast<const uint32_t *>(info[s].valid);
        const bool masked = base + kTile > low || valid != 0x01010101u;
        const uint32_t src = smem0 + L::kRing + s * L::kStageBytes;
        const uint32_t dst = smem0 + buf * 2 * L::kOperand;
        uint16_t *nan = reinterpret_cast<uint16_t *>(smem + L::kNan + buf * L::kNanBytes);
        if (tid < 4) {
          wide_info[buf].kf[tid] = info[s].kf[tid];
          wide_info[buf].lv[tid] = info[s].lv[tid];
          wide_info[buf].iv[tid] = info[s].iv[tid];
          if (tid == 0) *reinterpret_cast<uint32_t *>(wide_info[buf].valid) = valid;
        }
#pragma unroll
        for (int v = 0; v < 2; ++v)                   // keys, values
#pragma unroll
          for (int i = 0; i < kTile * D / 16 / 128; ++i) {
            const int at = tid + i * 128, row = at / (D / 16), c = at % (D / 16);   // 16 channels of a token
            uint4 w = lds128(src + v * (L::kStageBytes / 2) + row * D + c * 16);
            if (v == 1 && masked) {
              // a value that no row sees becomes 0: its weight is 0, but 0 * NaN would not be.  A NaN that some
              // rows see and others do not becomes 0 too, and a bit by which the rows that see it find it.
              const bool none = !(valid >> (8 * (row / 16)) & 1) || base + row >= high;
              if (none) w = make_uint4(0, 0, 0, 0);
              uint32_t bits = 0;
              if (base + row >= low) {
                uint32_t *e = &w.x;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const uint32_t is = __vcmpeq4(e[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                  e[k] &= ~is;
                  bits |= ((is & 0x01010101u) * 0x01020408u >> 24 & 15u) << (4 * k);
                }
              }
              nan[at] = (uint16_t)bits;
            }
            // 32 bytes of fp16 as two 16-byte units; the upper four pieces of a row store theirs in the other
            // order, so that eight lanes meet eight bank groups
            const uint4 lo = make_uint4(codes_lo(w.x), codes_hi(w.x), codes_lo(w.y), codes_hi(w.y));
            const uint4 hi = make_uint4(codes_lo(w.z), codes_hi(w.z), codes_lo(w.w), codes_hi(w.w));
            const int turn = (c >> 2) & 1, unit = (c & 3) * 2;
            const uint32_t to = dst + v * L::kOperand + (c >> 2) * (kTile * 128) + row * 128;
            sts128(to + (((unit + turn) ^ (row & 7)) << 4), turn ? hi : lo);
            sts128(to + (((unit + 1 - turn) ^ (row & 7)) << 4), turn ? lo : hi);
          }
        fence_proxy_async_smem();                     // the products read it through the async proxy
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(kv_full + buf);
          mbar_arrive(empty + s);
        }
      }
      if (dead) break;
    }
  } else {
    // ------------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftmaxRegs));
    const int x = warp >= 12, row = threadIdx.x & 127;
    const uint32_t tm = tmem + ((uint32_t)(warp & 3) * 32u << 16);   // the warp's lanes of tensor memory
    int4 split = make_int4(-1, 0, 0, 0);
    uint32_t done = 0, turn = 0;
    for (uint32_t item = 0; more && !dead; more = it.next(), ++item) {
      const int lim = limit(row), low = limit(0), high = limit(kRows - 1), r = min(it.rt * kRows + row, rows - 1);
      if (x == 0) {
        // the row of q, by a power of two in [2^14, 2^15), to tensor memory; rows behind the last repeat it
        const int t = r / p.G;
        const IO *src = static_cast<const IO *>(p.q) + ((int64_t)it.n * p.T + t) * p.q_stride +
                        (int64_t)(it.h * p.G + r - t * p.G) * D;
        Held8<IO> q[D / 8];
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) q[i].load(src + 8 * i);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) big = fmaxf(big, q[i].amax());
        int e = 14 - ((int)(__float_as_uint(big) >> 23) - 127);
        e = e < -120 ? -120 : (e > 120 ? 120 : e);
        const float up = __uint_as_float((uint32_t)(127 + e) << 23), down = __uint_as_float((uint32_t)(127 - e) << 23);
        factors[row] = p.scale * kLog2e * down;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float y[8];
            q[4 * i + k].get(y);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * k + j] = pack_f16(y[2 * j] * up, y[2 * j + 1] * up);
          }
          tmem_st16(tm + L::kQ + 16 * i, w);
        }
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      // (the second group: also so that it leaves no new (m, l) before the first has read the last)
      if (!warp_wait(q_full, item, p.polls)) { dead = true; break; }
      const float rf = factors[row];
      const int count = it.t1 - it.t0;
      float m = -INFINITY, l = 0.f;
      uint32_t nans[DW] = {};
      for (int i = x; i < count; i += 2, ++turn) {
        const uint32_t tile = done + i, buf = tile % kBuffers;
        // (the scales' wait: s_full says that the tile is widened; waiting for that itself makes it visible)
        if (!warp_wait(s_full + x, turn, p.polls) || !warp_wait(kv_full + buf, tile / kBuffers, p.polls)) {
          dead = true;
          break;
        }
        fence_after_sync();
        uint32_t sr[2][32];
        tmem_ld32(tm + L::kS + x * kTile, sr[0]);
        tmem_ld32(tm + L::kS + x * kTile + 32, sr[1]);
        tmem_wait_ld();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free + x);
        const int base = (it.t0 + i) * kTile;
        const uint32_t valid = *reinterpret_cast<const uint32_t *>(wide_info[buf].valid);
        const bool masked = base + kTile > low || valid != 0x01010101u;
        float kf[4], lv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) { kf[k] = rf * wide_info[buf].kf[k]; lv[k] = wide_info[buf].lv[k]; }
        float tops[4] = {m, m, m, m};                 // (four chains)
        if (!masked) {
#pragma unroll
          for (int j = 0; j < kTile; ++j)
            tops[j % 4] = fmaxf(tops[j % 4], fmaf(__uint_as_float(sr[j / 32][j % 32]), kf[j / 16], lv[j / 16]));
        } else {
          // the hidden scores become -inf; what is kept here needs no factor any more
#pragma unroll
          for (int j = 0; j < kTile; ++j) {
            float s = fmaf(__uint_as_float(sr[j / 32][j % 32]), kf[j / 16], lv[j / 16]);
            if (base + j >= lim || !(valid >> (8 * (j / 16)) & 1)) s = -INFINITY;
            sr[j / 32][j % 32] = __float_as_uint(s);
            tops[j % 4] = fmaxf(tops[j % 4], s);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) { kf[k] = 1.f; lv[k] = 0.f; }
        }
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        const bool grew = m != -INFINITY && top > m + kSlack;
        const bool fresh = m == -INFINITY;            // no weight yet: the output is 0, the reference free
        if (fresh) m = top;
        const float old = m;
        const bool rescale = __any_sync(~0u, grew);
        if (rescale) m = fmaxf(m, top);
        const float z = m == -INFINITY ? 0.f : m;
        // O and P of this group's last tile: the products are done with them
        if (turn > 0 && !warp_wait(pv_done + x, turn - 1, p.polls)) { dead = true; break; }
        if (rescale) {
          fence_after_sync();
          const float f = m == old ? 1.f : ex2(old - m);
          l *= f;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t w[32];
            tmem_ld32(tm + L::kO + x * D + c, w);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * f);
            tmem_st32(tm + L::kO + x * D + c, w);
          }
        }
        uint32_t pr[32];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float shift = lv[g] - z;
          float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = 16 * g + 2 * j;
            const float a = ex2(fmaf(__uint_as_float(sr[c / 32][c % 32]), kf[g], shift));
            const float b = ex2(fmaf(__uint_as_float(sr[c / 32][c % 32 + 1]), kf[g], shift));
            sum0 += a;
            sum1 += b;
            pr[8 * g + j] = pack_f16(a, b);
          }
          l = fmaf(sum0 + sum1, wide_info[buf].iv[g], l);
        }
        tmem_st32(tm + L::kP + x * (kTile / 2), pr);
        if (masked) {                                 // NaN values that this row sees and others do not
          const uint32_t *bits = reinterpret_cast<const uint32_t *>(smem + L::kNan + buf * L::kNanBytes);
          const int to = min(base + kTile, lim);
          for (int token = max(base, low); token < to; ++token)
#pragma unroll
            for (int k = 0; k < DW; ++k) nans[k] |= bits[(token - base) * DW + k];
        }
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + x);
      }
      if (dead) break;
      const bool used = count > x;                    // this group had a tile
      if (used && !warp_wait(pv_done + x, turn - 1, p.polls)) { dead = true; break; }
      fence_after_sync();
      if (x == 1) {
        second[row] = make_float2(m, l);
#pragma unroll
        for (int k = 0; k < DW; ++k) second_nan[row * DW + k] = nans[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(second_full);
      } else {
        if (!warp_wait(second_full, item, p.polls)) { dead = true; break; }
        fence_after_sync();
        const float2 ml = second[row];
        const float M = fmaxf(m, ml.x), fa = fade(m, M), fb = fade(ml.x, M), sum = fa * l + fb * ml.y;
        const bool whole = it.starts && it.ends, real = it.rt * kRows + row < rows;
        float *part = p.parts + ((int64_t)blockIdx.x * 2 + (it.starts ? 1 : 0)) * L::kPart;
        const int t = r / p.G;
        const int64_t orow = ((int64_t)it.n * p.T + t) * p.Hq + it.h * p.G + (r - t * p.G);
        const float f = !whole ? 1.f : sum == 0.f ? 0.f : 1.f / sum;     // no weight at all: o = 0
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t a[32], b[32];
          tmem_ld32(tm + L::kO + c, a);
          if (count > 1) tmem_ld32(tm + L::kO + D + c, b);
          tmem_wait_ld();
          const uint32_t bad = nans[c / 32] | second_nan[row * DW + c / 32];
          float y[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            y[k] = __uint_as_float(a[k]) * fa;
            if (count > 1) y[k] = fmaf(__uint_as_float(b[k]), fb, y[k]);
            if (bad >> k & 1) y[k] = __int_as_float(0x7fffffff);
            y[k] *= f;
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
        if (real && whole) {
          if (p.lse != nullptr) p.lse[orow] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
        } else if (real) {
          part[kRows * D + row] = M;
          part[kRows * D + kRows + row] = sum;
        }
        fence_before_sync();                          // (the loads above, before the next item's products)
        if (it.starts && !it.ends)
          split = make_int4(it.n, it.rt, it.h, (int)((line.first + done + it.tiles - 1) / line.share));
      }
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
  if (!encode_maps(p, c, CU_TENSOR_MAP_SWIZZLE_NONE)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attend_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  // as in the kernel for few rows: short items whole, and a line that 32 bits cannot count
  const int64_t tiles = ((int64_t)p.max_pages * p.P + kTile - 1) / kTile;
  p.whole = tiles <= 2 || items > INT32_MAX / tiles;
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
