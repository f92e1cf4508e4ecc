// Rotary positions on the q and k heads of a batch of tokens.
//
//   (a, b) -> amplitude (a cos t - b sin t, b cos t + a sin t),   t = position * frequency[pair]
//
// The angle only matters modulo one turn, so it is formed there: the frequency in turns per token
// becomes a 64-bit fraction of a turn, and position * fraction wraps modulo 2^64 = one turn by itself.
// The top 32 bits, taken as a signed fraction of a turn, go to sincospi: a far position loses no more digits than
// the frequency's own rounding times its distance, at one integer multiplication in the place of an fp64 range
// reduction.  (sincospi takes the fraction as fp32, 2^-25 of a half-turn: fp32 outputs are 1.3 times as far off as
// with angles taken in fp64, 5.4e-8 against 4.2e-8.)
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256;

struct RopeParams {
  int64_t tokens;
  int heads[2], D, rot;
  const void *in[2];
  void *out[2];
  int64_t in_stride[2], out_stride[2];
  const int32_t *positions;
  const double *frequencies;
  float amplitude;
  int inverse;
  int copy;        // the channels behind rot are copied (0: in place, they stay)
  int tile;        // tokens per block
  int head_lanes, token_lanes;   // heads and tokens that a block's threads take side by side
};

__device__ __forceinline__ uint64_t turn_fraction(double radians_per_token) {
  double t = radians_per_token * 0.15915494309189535;  // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);   // 2^64; t <= 1 - 2^-53 stays below
}

// amplitude (cos, sin) of position * fraction turns
__device__ __forceinline__ float2 cos_sin(uint64_t fraction, int32_t position, float amplitude, int inverse) {
  const uint64_t phase = fraction * (uint64_t)(int64_t)position + 0x80000000ull;
  float s, c;
  sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
  return make_float2(amplitude * c, inverse ? -amplitude * s : amplitude * s);
}

__device__ __forceinline__ void rotate(float &a, float &b, float2 cs) {
  const float x = a * cs.x - b * cs.y;
  b = b * cs.x + a * cs.y;
  a = x;
}

// Half layout whose pair count is a multiple of 8: a unit is 8 pairs (two 16-byte rows of bf16), or 8
// copied channels.  Interleaved layout: a unit is 8 channels, of which those below rot are rotated.
// Otherwise (kScalar) a unit is one pair or one copied channel.
enum { kHalf8 = 0, kInterleaved = 1, kScalar = 2 };

// A block has p.tile tokens: their cosines and sines go to shared memory once, for all heads; then a
// thread keeps one unit u of the head, takes a token's cosines and sines of it into registers and goes over
// the token's heads, kBatch at a time, all loads before the first store (in flight: 128 bytes a thread in the
// half layout; four rows of fp32 were slower than two, 78 us against 69, for the registers they take).
//
// Bound by HBM: 32768 tokens x 40 heads x 128 in bf16 take 119 us, 5.7 TB/s of the tensors read and written;
// 76091 tokens x 9 heads x 64 in fp32 68 us, 5.2 TB/s.  Rows of (token, head) dealt out to the threads one by
// one, with a row's cosines read again for each, took 130 us at 73 % of the issue slots (now 49 %).
template <typename T, int FORM>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;
  __shared__ uint64_t fraction[128];
  extern __shared__ float2 cs[];           // [tile][pairs], a unit's pairs apart from one another
  const int half = p.rot / 2;
  const int64_t t0 = (int64_t)blockIdx.x * p.tile;
  const int nt = (int)(p.tokens - t0 < p.tile ? p.tokens - t0 : p.tile);
  constexpr int kPairs = FORM == kHalf8 ? 8 : FORM == kInterleaved ? 4 : 1;   // of a unit
  const int turned = (half + kPairs - 1) / kPairs, pitch = turned * kPairs;
  for (int i = threadIdx.x; i < half; i += kThreads) fraction[i] = turn_fraction(p.frequencies[i]);
  __syncthreads();
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, pair = i - t * half;
    cs[t * pitch + pair % kPairs * turned + pair / kPairs] =
        cos_sin(fraction[pair], p.positions[t0 + t], p.amplitude, p.inverse);
  }
  __syncthreads();

  const int rest = !p.copy ? 0 : FORM == kHalf8 ? (p.D - p.rot) / 8 : FORM == kInterleaved
                   ? p.D / 8 - turned : p.D - p.rot;
  const int units = turned + rest, u = threadIdx.x % units, lane = threadIdx.x / units;
  const int hl = lane % p.head_lanes, tl = lane / p.head_lanes;
  if (tl >= p.token_lanes) return;
  const bool turn = u < turned;
  const bool whole = 4 * u + 3 < half;     // interleaved: all four pairs are rotated
  // the unit's first channel; in the half layout a pair's second one lies `half` on
  const int ch = FORM == kHalf8 ? (turn ? 8 * u : p.rot + 8 * (u - turned))
                 : FORM == kInterleaved ? 8 * u : (turn ? u : p.rot + u - turned);
  const int step = p.head_lanes * p.D;
  for (int t = tl; t < nt; t += p.token_lanes) {
    float2 c[kPairs];
    if (turn) {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) c[j] = cs[t * pitch + j * turned + u];
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const T *x = static_cast<const T *>(p.in[which]) + (t0 + t) * p.in_stride[which] + hl * p.D + ch;
      T *y = static_cast<T *>(p.out[which]) + (t0 + t) * p.out_stride[which] + hl * p.D + ch;
      for (int h = hl; h < p.heads[which]; h += kBatch * p.head_lanes) {
        Held8<T> ra[kBatch], rb[kBatch];
        T sa[kBatch], sb[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (h + k * p.head_lanes < p.heads[which]) {
            if constexpr (FORM == kScalar) {
              sa[k] = x[k * step];
              if (turn) sb[k] = x[k * step + half];
            } else {
              ra[k].load(x + k * step);
              if (FORM == kHalf8 && turn) rb[k].load(x + k * step + half);
            }
          }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          if (h + k * p.head_lanes < p.heads[which]) {
            float a[8], b[8];
            if constexpr (FORM == kHalf8) {
              ra[k].get(a);
              if (turn) {
                rb[k].get(b);
#pragma unroll
                for (int j = 0; j < 8; ++j) rotate(a[j], b[j], c[j]);
                store8(y + k * step + half, b);
              }
              store8(y + k * step, a);
            } else if constexpr (FORM == kInterleaved) {
              ra[k].get(a);
              if (turn) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (whole || 4 * u + j < half) rotate(a[2 * j], a[2 * j + 1], c[j]);
              }
              store8(y + k * step, a);
            } else {
              a[0] = to_f32(sa[k]);
              if (turn) {
                b[0] = to_f32(sb[k]);
                rotate(a[0], b[0], c[0]);
                y[k * step + half] = from_f32<T>(b[0]);
              }
              y[k * step] = from_f32<T>(a[0]);
            }
          }
        x += kBatch * step;
        y += kBatch * step;
      }
    }
  }
}

template <typename T>
cudaError_t launch(const RopeParams &p, int form, cudaStream_t stream) {
  const unsigned grid = (unsigned)((p.tokens + p.tile - 1) / p.tile);
  const size_t smem = (size_t)p.tile * (p.rot / 2 + 7) * sizeof(float2);
  if (form == kHalf8) rope_kernel<T, kHalf8><<<grid, kThreads, smem, stream>>>(p);
  else if (form == kInterleaved) rope_kernel<T, kInterleaved><<<grid, kThreads, smem, stream>>>(p);
  else rope_kernel<T, kScalar><<<grid, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const kda_rope_args &a, cudaStream_t stream) {
  RopeParams p;
  p.tokens = a.num_tokens;
  p.heads[0] = a.q_heads; p.heads[1] = a.k_heads;
  p.D = a.head_dim; p.rot = a.rot_dim;
  p.in[0] = a.q; p.in[1] = a.k; p.out[0] = a.q_out; p.out[1] = a.k_out;
  p.in_stride[0] = a.q_stride; p.in_stride[1] = a.k_stride;
  p.out_stride[0] = a.q_out_stride; p.out_stride[1] = a.k_out_stride;
  p.positions = a.positions; p.frequencies = a.frequencies;
  p.amplitude = a.amplitude; p.inverse = a.inverse != 0;
  p.copy = a.q != a.q_out || (a.k_heads > 0 && a.k != a.k_out);
  const int half = a.rot_dim / 2;
  const int form = a.layout == KDA_ROPE_INTERLEAVED ? kInterleaved : half % 8 == 0 ? kHalf8 : kScalar;
  const int rest = p.copy ? a.head_dim - a.rot_dim : 0;
  const int units = form == kHalf8 ? half / 8 + rest / 8
                    : form == kInterleaved ? (p.copy ? a.head_dim / 8 : (half + 3) / 4) : half + rest;
  const int lanes = kThreads / units;
  // Few tokens: as many heads side by side as there are lanes, a token or two a block, for latency.  Many:
  // a power of two of heads that divides both counts, so no lane idles at a token's end, but at most 16
  // tokens side by side; and up to four rounds of them a block to share its set-up (32 KB of cosines and
  // sines at most), as long as there are four blocks for each place on the GPU.
  const int most = a.q_heads > a.k_heads ? a.q_heads : a.k_heads;
  p.head_lanes = most < lanes ? most : lanes;
  int turns = 1;
  if (a.num_tokens >= 4096) {
    const int both = a.q_heads | a.k_heads;
    int even = both & -both;
    while (lanes / even > 16 && even < most) even *= 2;
    while (even > lanes) even /= 2;
    p.head_lanes = even;
    const int64_t spread = a.num_tokens / (lanes / even * 1776), room = 4096 / (lanes / even * (half + 7));
    turns = (int)(spread < room ? spread : room);
    turns = turns < 1 ? 1 : turns > 4 ? 4 : turns;
  }
  p.token_lanes = lanes / p.head_lanes;
  p.tile = p.token_lanes * turns;
  return a.io_dtype == KDA_BF16 ? launch<__nv_bfloat16>(p, form, stream) : launch<float>(p, form, stream);
}

}  // namespace kda
