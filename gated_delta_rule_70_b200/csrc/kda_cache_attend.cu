// Attention over the paged 8-bit cache, one block per query row: each warp takes every fourth cached
// token with its own running maximum and sum, and the four meet at the end.
#include <cuda_fp8.h>

#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kWarps = 4;

struct AttendParams {
  kda_cache c;
  const void *q;
  int64_t q_stride;
  int T, Hq;
  float scale;
  void *o;
  float *lse;
  int *status;
};

template <int V> __device__ __forceinline__ void load_codes(const uint8_t *p, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3)));
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) attend_row_kernel(AttendParams p) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t row = blockIdx.x;
  const int64_t tok = row / p.Hq;
  const int hq = (int)(row - tok * p.Hq), n = (int)(tok / p.T), t = (int)(tok - (int64_t)n * p.T);
  const int hk = hq / (p.Hq / p.c.num_kv_heads), P = p.c.page_tokens;
  int64_t len = p.c.seq_lens[n];
  const int64_t cap = (int64_t)p.c.max_pages * P;
  if ((len < 0 || len > cap) && p.status != nullptr && threadIdx.x == 0) atomicOr(p.status, ERR_BAD_LENGTH);
  len = len < 0 ? 0 : (len > cap ? cap : len);
  const int64_t seen = len - p.T + t + 1;
  float q[V], acc[V] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
    q[i] = to_f32(static_cast<const T *>(p.q)[tok * p.q_stride + hq * D + lane * V + i]);
  for (int64_t j = warp; j < seen; j += kWarps) {
    const int32_t pg = p.c.block_table[(int64_t)n * p.c.max_pages + j / P];
    if (pg < 0 || pg >= p.c.num_pages) {
      if (p.status != nullptr && lane == 0) atomicOr(p.status, ERR_BAD_PAGE);
      continue;
    }
    const int64_t tile = (int64_t)pg * p.c.num_kv_heads + hk;
    const int64_t at = (tile * P + j % P) * D + lane * V;
    float x[V], s = 0.f;
    load_codes(static_cast<const uint8_t *>(p.c.k_cache) + at, x);
#pragma unroll
    for (int i = 0; i < V; ++i) s += q[i] * x[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    s *= p.scale * p.c.k_scale[tile];
    const float mn = fmaxf(m, s), a = expf(m - mn), w = expf(s - mn);
    m = mn;
    l = l * a + w;
    load_codes(static_cast<const uint8_t *>(p.c.v_cache) + at, x);
    const float vs = fminf(fmaxf(p.c.v_scale[tile], 0x1p-60f), 0x1p60f);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = acc[i] * a + w * vs * x[i];
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
  for (int i = 0; i < V; ++i) so[warp][lane * V + i] = acc[i];
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm[w]);
  l = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float f = sl[w] == 0.f ? 0.f : expf(sm[w] - m);
    l += f * sl[w];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += f * so[w][lane * V + i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    static_cast<T *>(p.o)[row * D + lane * V + i] = from_f32<T>(l == 0.f ? 0.f : acc[i] / l);
  if (p.lse != nullptr && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t cache_attend_workspace(const kda_cache &, const kda_cache_attend_args &) { return 256; }

cudaError_t launch_cache_attend(const kda_cache &c, const kda_cache_attend_args &a, void *, cudaStream_t stream) {
  AttendParams p{c, a.q, a.q_stride, a.num_new, a.num_heads, a.scale, a.o, a.lse, a.status};
  const unsigned grid = (unsigned)((int64_t)c.num_seqs * a.num_new * a.num_heads);
  const bool bf16 = a.io_dtype == KDA_BF16;
  if (c.head_dim == 128) {
    if (bf16) attend_row_kernel<__nv_bfloat16, 128><<<grid, kWarps * 32, 0, stream>>>(p);
    else attend_row_kernel<float, 128><<<grid, kWarps * 32, 0, stream>>>(p);
  } else {
    if (bf16) attend_row_kernel<__nv_bfloat16, 64><<<grid, kWarps * 32, 0, stream>>>(p);
    else attend_row_kernel<float, 64><<<grid, kWarps * 32, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace kda
