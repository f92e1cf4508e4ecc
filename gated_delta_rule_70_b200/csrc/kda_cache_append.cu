// The append to the paged 8-bit cache: quantises new keys and values.  A unit is one page, head and tensor
// (keys or values) that gets new tokens; one to eight warps take it, so that the new values stay in
// registers between the search for their largest and their division by the scale: one pass over the input.
// Bound by HBM for prompts (32768 tokens of 8 heads x 128 in bf16, pages of 64: 42 us, 4.8 TB/s of the new
// values and the codes), with the dependent loads of a unit (length, table, scale) behind its other units' data;
// by those loads alone for single tokens.
#include <cuda_fp8.h>

#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMinExp = -60, kMaxExp = 60;   // exponents of the scales written

struct AppendParams {
  kda_cache c;
  const void *x[2];
  int64_t stride[2];
  int new_tokens;        // dense: per sequence; varlen: packed total
  const int32_t *cu;
  int slots;             // page slots of the call
  int log_page;
  int pages_per_seq;     // dense: page slots per sequence
  int warps;             // per unit: 1, 2, 4 or 8
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
  asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}" : "=r"(r.x) : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
  asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}" : "=r"(r.y) : "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

__device__ __forceinline__ void dequantise8(uint2 r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint8_t b = (uint8_t)((i < 4 ? r.x : r.y) >> (8 * (i & 3)));
    x[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
  }
}

// VPT: 8-channel vectors of new values that a thread holds at most.
template <typename T, int D, int VPT>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int V = D / 8;                                 // vectors per token
  const int P = p.c.page_tokens, N = p.c.num_seqs, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const uint32_t units = 2 * p.c.num_kv_heads, per_block = kWarps / p.warps;
  const uint32_t id = blockIdx.x * per_block + warp / p.warps;           // of the unit
  const int slot = (int)(id / units);
  const int unit = (int)(id - slot * units), h = unit >> 1, which = unit & 1;
  const int at = threadIdx.x % (32 * p.warps), step = 32 * p.warps;      // the thread in the unit
  // varlen: sequence n owns the page slots from floor(cu[n] / P) + 2 n on, enough for its pages
  // wherever they begin (c tokens touch at most floor(c / P) + 2 pages)
  int n = 0;
  int64_t j = 0, row0 = 0, count = 0;
  if (slot < p.slots && p.cu == nullptr) {
    n = (int)((uint32_t)slot / (uint32_t)p.pages_per_seq);
    j = slot - n * p.pages_per_seq;
    row0 = (int64_t)n * p.new_tokens;
    count = p.new_tokens;
  } else if (slot < p.slots) {
    for (int left = N; left > 1;) {                        // 32 places of the sequences left at a time
      const int stride = (left + 31) / 32, i = n + lane * stride;
      const bool below = lane * stride < left && ((int64_t)p.cu[i] >> p.log_page) + 2 * (int64_t)i <= slot;
      const uint32_t m = __ballot_sync(~0u, below);
      const int k = m == 0 ? 0 : 31 - __clz(m);
      n += k * stride;
      left = min(stride, left - k * stride);
    }
    int64_t end;
    seq_bounds(p.cu, n, 0, p.new_tokens, row0, end);
    count = end - row0;
    j = slot - ((row0 >> p.log_page) + 2 * (int64_t)n);
  }
  if (p.cu != nullptr && blockIdx.x == 0 && warp == 0 && p.status != nullptr) {
    bool bad = lane == 0 && (p.cu[0] != 0 || p.cu[N] != p.new_tokens);
    for (int i = lane; i < N; i += 32) bad |= p.cu[i + 1] < p.cu[i];
    if (bad) atomicOr(p.status, ERR_BAD_CU_SEQLENS);
  }
  // the unit's page and its new tokens [begin, end) (positions in the sequence), if it has any
  int64_t begin = 0, start = 0;
  int kept = 0, fresh = 0;
  const int32_t *table = nullptr;
  if (j >= 0 && count > 0) {
    const int64_t len = p.c.seq_lens[n], cap = (int64_t)p.c.max_pages * P;
    if (j == 0 && unit == 0 && lane == 0 && p.status != nullptr && (len < 0 || len > cap))
      atomicOr(p.status, ERR_BAD_LENGTH);
    start = len - count;                                   // position of the first new token
    const int64_t begin0 = start > 0 ? start : 0, end0 = len < cap ? len : cap;
    const int64_t page = (begin0 >> p.log_page) + j;
    begin = page * P > begin0 ? page * P : begin0;
    const int64_t end = (page + 1) * P < end0 ? (page + 1) * P : end0;
    if (begin < end) {
      kept = (int)(begin - page * P);                      // earlier tokens of the page
      fresh = (int)(end - begin);
      table = p.c.block_table + (int64_t)n * p.c.max_pages + page;
    }
  }
  const int64_t stride = p.stride[which];
  const T *x = static_cast<const T *>(p.x[which]) + (row0 + (begin - start)) * stride + h * D;
  const int vectors = fresh * V;
  Held8<T> raw[VPT];
  // a thread's vectors lie a whole number of tokens apart (step is a multiple of V)
  const T *from = x + (int64_t)(at / V) * stride + (at % V) * 8;
  const int64_t apart = (int64_t)(step / V) * stride;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {                          // the values come while the table is looked up
    const int i = at + k * step;
    if (i < vectors) raw[k].load(from + k * apart);
  }
  const int pg = fresh > 0 ? *table : 0;
  const bool good = pg >= 0 && pg < p.c.num_pages;
  if (!good && lane == 0 && p.status != nullptr) atomicOr(p.status, ERR_BAD_PAGE);
  const int64_t tile = good ? (int64_t)pg * p.c.num_kv_heads + h : 0;
  float *scale = (which ? p.c.v_scale : p.c.k_scale) + tile;
  uint2 *codes = reinterpret_cast<uint2 *>(static_cast<uint8_t *>(which ? p.c.v_cache : p.c.k_cache) + tile * P * D);
  const float old = good && kept > 0 ? *scale : 0.f;
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < VPT; ++k)
    if (at + k * step < vectors) amax = fmaxf(amax, raw[k].amax());
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  if (p.warps > 1) {                                       // (also: everybody has read the old scale)
    __shared__ float part[kWarps];
    if (lane == 0) part[warp] = amax;
    __syncthreads();
    for (int i = 0; i < p.warps; ++i) amax = fmaxf(amax, part[warp / p.warps * p.warps + i]);
  }
  if (fresh == 0 || !good) return;
  float s = power_scale(amax);
  if (kept > 0) {
    s = fmaxf(old, s);
    if (s != old) {
      const float ratio = old / s;
      for (int i = at; i < kept * V; i += step) {
        float z[8];
        dequantise8(codes[i], z);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] *= ratio;
        codes[i] = quantise8(z);
      }
    }
  }
  __syncwarp();
  if (at == 0) *scale = s;
  codes += kept * V + at;
  // x / s: the scales that this kernel writes are powers of two, whose reciprocal is exact; a scale that
  // somebody else wrote is divided by
  if ((__float_as_uint(s) & 0x7fffffu) == 0 && s > 0x1p-100f && s < 0x1p100f) {
    const float r = 1.f / s;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      if (at + k * step < vectors) {
        float y[8];
        raw[k].get(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= r;
        codes[k * step] = quantise8(y);
      }
  } else {
#pragma unroll 1
    for (int i = at; i < vectors; i += step) {            // rare, and read once more
      Held8<T> again;
      float y[8];
      again.load(from);
      again.get(y);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] / s;
      *codes = quantise8(y);
      from += apart;
      codes += step;
    }
  }
}

// Pages that num_new tokens touch at most, wherever they begin; the page slots of a call.
int pages_per_sequence(const kda_cache &c, const kda_cache_append_args &a) {
  return (int)(((int64_t)a.num_new + c.page_tokens - 2) / c.page_tokens + 1);
}
int64_t page_slots(const kda_cache &c, const kda_cache_append_args &a) {
  return a.cu_seqlens != nullptr ? a.num_new / c.page_tokens + 2 * (int64_t)c.num_seqs
                                 : (int64_t)c.num_seqs * pages_per_sequence(c, a);
}

template <typename T, int D>
cudaError_t launch(AppendParams p, cudaStream_t stream) {
  // New values of a page at most, in vectors.  A thread holds one of them, four, or eight: four where one warp
  // is enough for the page, or with fp32 (32768 tokens of 4 x 128 in pages of 64: 35 us against 47 with eight,
  // whose 106 registers leave too few blocks on an SM to hide the way from the table to the scale); eight with
  // bf16 (8 x 128: 47 us against 53 with four), and where eight warps with four are too few.
  const int most = (p.c.page_tokens < p.new_tokens ? p.c.page_tokens : p.new_tokens) * (D / 8);
  const int hold = most <= 32 ? 1 : most <= 128 || (sizeof(T) == 4 && most <= 1024) ? 4 : 8;
  for (p.warps = 1; p.warps < kWarps && p.warps * 32 * hold < most; p.warps *= 2) {}
  const int per_block = kWarps / p.warps;
  const int64_t all = (int64_t)p.slots * 2 * p.c.num_kv_heads, grid = (all + per_block - 1) / per_block;
  if (hold == 1) append_kernel<T, D, 1><<<(unsigned)grid, kThreads, 0, stream>>>(p);
  else if (hold == 4) append_kernel<T, D, 4><<<(unsigned)grid, kThreads, 0, stream>>>(p);
  else append_kernel<T, D, 8><<<(unsigned)grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

int64_t cache_append_units(const kda_cache &c, const kda_cache_append_args &a) {
  return page_slots(c, a) * 2 * c.num_kv_heads;
}

cudaError_t launch_cache_append(const kda_cache &c, const kda_cache_append_args &a, cudaStream_t stream) {
  AppendParams p;
  p.c = c;
  p.x[0] = a.k; p.x[1] = a.v;
  p.stride[0] = a.k_stride; p.stride[1] = a.v_stride;
  p.new_tokens = a.num_new; p.cu = a.cu_seqlens; p.status = a.status;
  const int P = c.page_tokens;
  p.pages_per_seq = pages_per_sequence(c, a);
  p.slots = (int)page_slots(c, a);
  p.log_page = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
  const bool bf16 = a.io_dtype == KDA_BF16;
  if (c.head_dim == 128) return bf16 ? launch<__nv_bfloat16, 128>(p, stream) : launch<float, 128>(p, stream);
  return bf16 ? launch<__nv_bfloat16, 64>(p, stream) : launch<float, 64>(p, stream);
}

}  // namespace kda
