// The append to the paged 8-bit cache: quantises new keys and values, one block per page, head and
// tensor that gets new tokens.
#include <cuda_fp8.h>

#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kMinExp = -60, kMaxExp = 60;   // exponents of the scales written

struct AppendParams {
  kda_cache c;
  const void *x[2];
  int64_t stride[2];
  int new_tokens;        // dense: per sequence; varlen: packed total
  const int32_t *cu;
  int pages_per_seq;     // dense: page slots per sequence
  int *status;
};

// The smallest power of two s with amax <= 448 s (448 = 0.875 * 2^9), its exponent held to [-60, 60].
__device__ __forceinline__ float power_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  // amax = m 2^e, m in [0.5, 1): e = biased - 126, and 0.875 is 0x600000 in the mantissa bits
  int e = (int)(u >> 23) - 126 - 9 + ((u & 0x7fffffu) > 0x600000u);
  e = e < kMinExp ? kMinExp : (e > kMaxExp ? kMaxExp : e);   // zero and subnormals land on the lower bound
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ uint2 quantise8(const float (&x)[8]) {
  uint2 r;
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
  r.x = h[0] | ((uint32_t)h[1] << 16);
  r.y = h[2] | ((uint32_t)h[3] << 16);
  return r;
}

__device__ __forceinline__ void dequantise8(uint2 r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint8_t b = (uint8_t)((i < 4 ? r.x : r.y) >> (8 * (i & 3)));
    x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
  }
}

// x / s.  The scales that this kernel writes are powers of two, whose reciprocal is exact; a scale that
// somebody else wrote is divided by.
__device__ __forceinline__ void divide8(float (&x)[8], float s) {
  if ((__float_as_uint(s) & 0x7fffffu) == 0 && s > 0x1p-100f && s < 0x1p100f) {
    const float r = 1.f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= r;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] / s;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendParams p) {
  const int P = p.c.page_tokens, N = p.c.num_seqs;
  const int64_t slot = blockIdx.x;
  const int h = blockIdx.y, which = blockIdx.z;
  const bool first = blockIdx.x == 0 && h == 0 && which == 0;
  // varlen: sequence n owns the page slots from floor(cu[n] / P) + 2 n on, enough for its pages
  // wherever they begin (c tokens touch at most floor(c / P) + 2 pages)
  int n;
  int64_t j, row0, count;
  if (p.cu == nullptr) {
    n = (int)(slot / p.pages_per_seq);
    j = slot - (int64_t)n * p.pages_per_seq;
    row0 = (int64_t)n * p.new_tokens;
    count = p.new_tokens;
  } else {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      int64_t c = p.cu[mid];
      if (c / P + 2 * (int64_t)mid <= slot) lo = mid; else hi = mid - 1;
    }
    n = lo;
    int64_t end;
    seq_bounds(p.cu, n, 0, p.new_tokens, row0, end);
    count = end - row0;
    j = slot - (row0 / P + 2 * (int64_t)n);
    if (first && p.status != nullptr && threadIdx.x == 0) {
      bool bad = p.cu[0] != 0 || p.cu[N] != p.new_tokens;
      for (int i = 0; i < N; ++i) bad |= p.cu[i + 1] < p.cu[i];
      if (bad) atomicOr(p.status, ERR_BAD_CU_SEQLENS);
    }
  }
  if (n >= N || j < 0 || count <= 0) return;
  const int64_t len = p.c.seq_lens[n], cap = (int64_t)p.c.max_pages * P;
  if (j == 0 && h == 0 && which == 0 && threadIdx.x == 0 && p.status != nullptr && (len < 0 || len > cap))
    atomicOr(p.status, ERR_BAD_LENGTH);
  const int64_t start = len - count;                       // position of the first new token
  const int64_t begin0 = start > 0 ? start : 0, end0 = len < cap ? len : cap;
  const int64_t page = begin0 / P + j;
  const int64_t begin = page * P > begin0 ? page * P : begin0;
  const int64_t end = (page + 1) * P < end0 ? (page + 1) * P : end0;
  if (begin >= end) return;
  const int32_t pg = p.c.block_table[(int64_t)n * p.c.max_pages + page];
  if (pg < 0 || pg >= p.c.num_pages) {
    if (threadIdx.x == 0 && p.status != nullptr) atomicOr(p.status, ERR_BAD_PAGE);
    return;
  }
  const int kept = (int)(begin - page * P);                // earlier tokens of the page
  const int64_t tile = (int64_t)pg * p.c.num_kv_heads + h;
  float *scale = (which ? p.c.v_scale : p.c.k_scale) + tile;
  uint8_t *codes = static_cast<uint8_t *>(which ? p.c.v_cache : p.c.k_cache) + tile * P * D;
  const T *x = static_cast<const T *>(p.x[which]) + (row0 + (begin - start)) * p.stride[which] + h * D;
  const int64_t stride = p.stride[which];

  constexpr int V = D / 8;                                 // 8-channel vectors per token
  const int vectors = (int)(end - begin) * V;
  float amax = 0.f;
  for (int i = threadIdx.x; i < vectors; i += kThreads) {
    float y[8];
    load8(x + (int64_t)(i / V) * stride + (i % V) * 8, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(y[e]));   // a NaN does not enter
  }
  __shared__ float part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) amax = fmaxf(amax, part[i]);
  float s = power_scale(amax);
  if (kept > 0) {
    const float old = *scale;
    s = fmaxf(old, s);
    if (s != old) {
      const float ratio = old / s;
      for (int i = threadIdx.x; i < kept * V; i += kThreads) {
        float y[8];
        uint2 *at = reinterpret_cast<uint2 *>(codes) + i;
        dequantise8(*at, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= ratio;
        *at = quantise8(y);
      }
    }
  }
  __syncthreads();                                         // everybody has read the old scale
  if (threadIdx.x == 0) *scale = s;
  for (int i = threadIdx.x; i < vectors; i += kThreads) {
    float y[8];
    load8(x + (int64_t)(i / V) * stride + (i % V) * 8, y);
    divide8(y, s);
    reinterpret_cast<uint2 *>(codes)[kept * V + i] = quantise8(y);
  }
}

}  // namespace

cudaError_t launch_cache_append(const kda_cache &c, const kda_cache_append_args &a, cudaStream_t stream) {
  AppendParams p;
  p.c = c;
  p.x[0] = a.k; p.x[1] = a.v;
  p.stride[0] = a.k_stride; p.stride[1] = a.v_stride;
  p.new_tokens = a.num_new; p.cu = a.cu_seqlens; p.status = a.status;
  const int P = c.page_tokens;
  p.pages_per_seq = (int)(((int64_t)a.num_new + P - 2) / P + 1);
  const int64_t slots = a.cu_seqlens != nullptr ? a.num_new / P + 2 * (int64_t)c.num_seqs
                                                : (int64_t)c.num_seqs * p.pages_per_seq;
  const dim3 grid((unsigned)slots, c.num_kv_heads, 2);
  const bool bf16 = a.io_dtype == KDA_BF16;
  if (c.head_dim == 128) {
    if (bf16) append_kernel<__nv_bfloat16, 128><<<grid, kThreads, 0, stream>>>(p);
    else append_kernel<float, 128><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (bf16) append_kernel<__nv_bfloat16, 64><<<grid, kThreads, 0, stream>>>(p);
    else append_kernel<float, 64><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace kda
