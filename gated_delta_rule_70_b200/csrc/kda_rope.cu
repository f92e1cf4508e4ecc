// Rotary positions on the q and k heads of a batch of tokens.
//
//   (a, b) -> amplitude (a cos t - b sin t, b cos t + a sin t),   t = position * frequency[pair]
//
// The angle only matters modulo one turn, so it is formed there: the frequency in turns per token
// becomes a 64-bit fraction of a turn, and position * fraction wraps modulo 2^64 = one turn by itself.
// The top 32 bits, taken as a signed fraction of a turn, go to sincospi: no far position loses digits, at
// one integer multiplication in the place of an fp64 range reduction.
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
// thread keeps one unit u of the head and takes every RL-th (token, head) row, kBatch of them at a time, all
// loads before the first store.  Bound by HBM; with one row at a time the loads in flight were too few
// (32768 tokens x 40 heads x 128 bf16: 152 us).
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
  const int rest = !p.copy ? 0 : FORM == kHalf8 ? (p.D - p.rot) / 8 : FORM == kInterleaved
                   ? p.D / 8 - turned : p.D - p.rot;
  const int units = turned + rest;
  const int RL = kThreads / units, u = threadIdx.x % units, H = p.heads[0] + p.heads[1];
  const int rows = threadIdx.x < RL * units ? nt * H : 0;
  const bool turn = u < turned;
  // the unit's first channel; in the half layout a pair's second one lies `half` on
  const int ch = FORM == kHalf8 ? (turn ? 8 * u : p.rot + 8 * (u - turned))
                 : FORM == kInterleaved ? 8 * u : (turn ? u : p.rot + u - turned);
  Held8<T> ra[kBatch], rb[kBatch];
  T sa[kBatch], sb[kBatch];
  T *to[kBatch];
  int token[kBatch];
  auto load = [&](int row0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int row = row0 + k * RL;
      if (row >= rows) break;
      const int t = row / H, hh = row - t * H;
      const int which = hh >= p.heads[0], h = hh - (which ? p.heads[0] : 0);
      token[k] = t;
      to[k] = static_cast<T *>(p.out[which]) + (t0 + t) * p.out_stride[which] + h * p.D + ch;
      const T *x = static_cast<const T *>(p.in[which]) + (t0 + t) * p.in_stride[which] + h * p.D + ch;
      if constexpr (FORM == kScalar) {
        sa[k] = x[0];
        if (turn) sb[k] = x[half];
      } else {
        ra[k].load(x);
        if (FORM == kHalf8 && turn) rb[k].load(x + half);
      }
    }
  };
  int row0 = threadIdx.x / units;
  load(row0);                              // the first rows come while the angles are made

  for (int i = threadIdx.x; i < half; i += kThreads) fraction[i] = turn_fraction(p.frequencies[i]);
  __syncthreads();
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, pair = i - t * half;
    cs[t * pitch + pair % kPairs * turned + pair / kPairs] =
        cos_sin(fraction[pair], p.positions[t0 + t], p.amplitude, p.inverse);
  }
  __syncthreads();

  while (row0 < rows) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (row0 + k * RL >= rows) break;
      T *y = to[k];
      const float2 *c = cs + token[k] * pitch + u;
      float a[8], b[8];
      if constexpr (FORM == kHalf8) {
        ra[k].get(a);
        if (turn) {
          rb[k].get(b);
#pragma unroll
          for (int j = 0; j < 8; ++j) rotate(a[j], b[j], c[j * turned]);
          store8(y + half, b);
        }
        store8(y, a);
      } else if constexpr (FORM == kInterleaved) {
        ra[k].get(a);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * u + j < half) rotate(a[2 * j], a[2 * j + 1], c[j * turned]);
        store8(y, a);
      } else {
        a[0] = to_f32(sa[k]);
        if (turn) {
          b[0] = to_f32(sb[k]);
          rotate(a[0], b[0], c[0]);
          y[half] = from_f32<T>(b[0]);
        }
        y[0] = from_f32<T>(a[0]);
      }
    }
    row0 += RL * kBatch;
    load(row0);
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
  // few tokens: one a block, for as many blocks as there are; many: eight share a block's set-up
  p.tile = a.num_tokens >= 8 * 592 ? 8 : a.num_tokens >= 4 * 592 ? 4 : a.num_tokens >= 2 * 592 ? 2 : 1;
  const int form = a.layout == KDA_ROPE_INTERLEAVED ? kInterleaved
                   : (a.rot_dim / 2) % 8 == 0       ? kHalf8
                                                    : kScalar;
  return a.io_dtype == KDA_BF16 ? launch<__nv_bfloat16>(p, form, stream) : launch<float>(p, form, stream);
}

}  // namespace kda
