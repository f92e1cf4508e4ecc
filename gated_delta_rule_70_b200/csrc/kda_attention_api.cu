// C ABI of the softmax-attention layer's operators (declared in include/kda.h): the checks of
// rotary positions, the append to the paged 8-bit cache and the attention over it.
#include <cmath>
#include <cstdint>

#include "kda_common.cuh"
#include "kda_internal.h"

namespace {

using namespace kda;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

#define KDA_CHECK(cond) do { if (!(cond)) return KDA_ERR_INVALID_ARGUMENT; } while (0)

kda_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

bool known_dtype(int t) { return t == KDA_BF16 || t == KDA_FP32; }

// Tokens of `row` elements each, `stride` elements apart.
bool good_stride(int64_t stride, int64_t row) { return stride >= row && stride % 8 == 0; }

constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 4096;   // places of a block table's row

// The sizes of a cache, before any pointer is looked at.
kda_status check_cache_sizes(const kda_cache *c) {
  KDA_CHECK(c != nullptr);
  KDA_CHECK(c->num_seqs >= 0 && c->num_kv_heads >= 1 && c->num_pages >= 1 && c->max_pages >= 1);
  if (c->head_dim != 64 && c->head_dim != 128) return KDA_ERR_UNSUPPORTED;
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
    return KDA_ERR_UNSUPPORTED;
  if (c->num_kv_heads > 64) return KDA_ERR_UNSUPPORTED;
  // token positions are counted in 32 bits, and up to 2048 tokens beyond a sequence's end are (not read)
  if ((int64_t)c->num_pages * c->num_kv_heads > INT32_MAX / c->page_tokens ||
      (int64_t)c->max_pages * c->page_tokens > kMaxTokens)
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda_status check_cache_pointers(const kda_cache *c) {
  for (const void *p : {(const void *)c->k_cache, (const void *)c->v_cache})
    KDA_CHECK(p != nullptr && aligned16(p));
  for (const void *p : {(const void *)c->k_scale, (const void *)c->v_scale,
                        (const void *)c->block_table, (const void *)c->seq_lens})
    KDA_CHECK(p != nullptr && aligned4(p));
  return KDA_OK;
}

kda_status check_attend_sizes(const kda_cache *c, const kda_cache_attend_args *a) {
  kda_status st = check_cache_sizes(c);
  if (st != KDA_OK) return st;
  KDA_CHECK(a != nullptr);
  KDA_CHECK(known_dtype(a->io_dtype) && a->num_new >= 1 && a->num_heads >= 1);
  KDA_CHECK(a->num_heads % c->num_kv_heads == 0 && std::isfinite(a->scale));
  KDA_CHECK((a->flags & ~KDA_FLAG_TEST_EXPIRE_WAITS) == 0);
  if (a->num_heads > 256) return KDA_ERR_UNSUPPORTED;
  // query rows and row tiles are counted in 32 bits
  if ((int64_t)c->num_seqs * a->num_new > INT32_MAX / a->num_heads) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_rope_frequencies(const kda_rope_config *c, double *frequencies, float *amplitude) {
  KDA_CHECK(c != nullptr && frequencies != nullptr && amplitude != nullptr);
  KDA_CHECK(c->rot_dim >= 2 && c->rot_dim <= 256 && c->rot_dim % 2 == 0);
  KDA_CHECK(std::isfinite(c->base) && c->base > 1.0);
  const int rot = c->rot_dim;
  double base = c->base, mul = 1.0, low = 0.0, high = 0.0;
  *amplitude = 1.f;
  switch (c->scaling) {
    case KDA_ROPE_UNSCALED: break;
    case KDA_ROPE_LINEAR:
    case KDA_ROPE_NTK:
    case KDA_ROPE_YARN: KDA_CHECK(std::isfinite(c->factor) && c->factor >= 1.0); break;
    default: return KDA_ERR_INVALID_ARGUMENT;
  }
  if (c->scaling == KDA_ROPE_LINEAR) mul = 1.0 / c->factor;
  if (c->scaling == KDA_ROPE_NTK) {
    KDA_CHECK(rot >= 4);
    base *= std::pow(c->factor, (double)rot / (rot - 2));
  }
  if (c->scaling == KDA_ROPE_YARN) {
    KDA_CHECK(std::isfinite(c->original_context) && c->original_context > 0.0);
    KDA_CHECK(std::isfinite(c->beta_fast) && c->beta_fast > c->beta_slow && c->beta_slow > 0.0);
    // the (fractional) pair that turns `b` times within the original context
    auto pair_of = [&](double b) {
      return rot * std::log(c->original_context / (b * 2.0 * M_PI)) / (2.0 * std::log(base));
    };
    low = std::fmax(std::floor(pair_of(c->beta_fast)), 0.0);
    high = std::fmin(std::ceil(pair_of(c->beta_slow)), (double)(rot - 1));
    *amplitude = (float)(0.1 * std::log(c->factor) + 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot) * mul;
    if (c->scaling == KDA_ROPE_YARN) {
      const double r = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
      f = f * (1.0 - r) + f / c->factor * r;
    }
    frequencies[i] = f;
  }
  return KDA_OK;
}

kda_status kda_rope(const kda_rope_args *a, void *stream) {
  KDA_CHECK(a != nullptr);
  KDA_CHECK(known_dtype(a->io_dtype) && a->num_tokens >= 0 && std::isfinite(a->amplitude));
  KDA_CHECK(a->layout == KDA_ROPE_HALF || a->layout == KDA_ROPE_INTERLEAVED);
  KDA_CHECK(a->q_heads >= 1 && a->k_heads >= 0 && a->head_dim >= 1);
  KDA_CHECK(a->rot_dim >= 2 && a->rot_dim % 2 == 0 && a->rot_dim <= a->head_dim);
  if (a->head_dim % 8 != 0 || a->head_dim > 256 || a->q_heads > 256 || a->k_heads > 256)
    return KDA_ERR_UNSUPPORTED;
  kda_status st = check_tokens(a->num_tokens);
  if (st != KDA_OK) return st;
  KDA_CHECK(good_stride(a->q_stride, (int64_t)a->q_heads * a->head_dim) &&
            good_stride(a->q_out_stride, (int64_t)a->q_heads * a->head_dim));
  KDA_CHECK(a->q != a->q_out || a->q_stride == a->q_out_stride);
  if (a->k_heads > 0) {
    KDA_CHECK(good_stride(a->k_stride, (int64_t)a->k_heads * a->head_dim) &&
              good_stride(a->k_out_stride, (int64_t)a->k_heads * a->head_dim));
    KDA_CHECK(a->k != a->k_out || a->k_stride == a->k_out_stride);
  }
  if (a->num_tokens == 0) return KDA_OK;
  KDA_CHECK(a->q != nullptr && aligned16(a->q) && a->q_out != nullptr && aligned16(a->q_out));
  if (a->k_heads > 0)
    KDA_CHECK(a->k != nullptr && aligned16(a->k) && a->k_out != nullptr && aligned16(a->k_out));
  KDA_CHECK(a->positions != nullptr && aligned4(a->positions));
  KDA_CHECK(a->frequencies != nullptr && (reinterpret_cast<uintptr_t>(a->frequencies) & 7u) == 0);
  return cuda_status(launch_rope(*a, static_cast<cudaStream_t>(stream)));
}

kda_status kda_cache_append(const kda_cache *c, const kda_cache_append_args *a, void *stream_) {
  kda_status st = check_cache_sizes(c);
  if (st != KDA_OK) return st;
  KDA_CHECK(a != nullptr);
  KDA_CHECK(known_dtype(a->io_dtype) && a->num_new >= 0);
  KDA_CHECK(good_stride(a->k_stride, (int64_t)c->num_kv_heads * c->head_dim) &&
            good_stride(a->v_stride, (int64_t)c->num_kv_heads * c->head_dim));
  KDA_CHECK(a->status == nullptr || aligned4(a->status));
  st = check_tokens(a->cu_seqlens != nullptr ? (int64_t)a->num_new : (int64_t)c->num_seqs * a->num_new);
  if (st != KDA_OK) return st;
  if (cache_append_units(*c, *a) > INT32_MAX) return KDA_ERR_UNSUPPORTED;   // counted in 32 bits
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const bool work = c->num_seqs > 0 && a->num_new > 0;
  if (work) {
    st = check_cache_pointers(c);
    if (st != KDA_OK) return st;
    KDA_CHECK(a->k != nullptr && aligned16(a->k) && a->v != nullptr && aligned16(a->v));
    KDA_CHECK(a->cu_seqlens == nullptr || aligned4(a->cu_seqlens));
  }
  if (a->status != nullptr && cudaMemsetAsync(a->status, 0, sizeof(int32_t), stream) != cudaSuccess)
    return KDA_ERR_CUDA;
  return work ? cuda_status(launch_cache_append(*c, *a, stream)) : KDA_OK;
}

size_t kda_cache_attend_workspace_size(const kda_cache *c, const kda_cache_attend_args *a) {
  return check_attend_sizes(c, a) == KDA_OK ? cache_attend_workspace(*c, *a) : 0;
}

kda_status kda_cache_attend(const kda_cache *c, const kda_cache_attend_args *a, void *workspace,
                            size_t workspace_bytes, void *stream_) {
  kda_status st = check_attend_sizes(c, a);
  if (st != KDA_OK) return st;
  KDA_CHECK(good_stride(a->q_stride, (int64_t)a->num_heads * c->head_dim));
  KDA_CHECK(a->status == nullptr || aligned4(a->status));
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (c->num_seqs > 0) {
    st = check_cache_pointers(c);
    if (st != KDA_OK) return st;
    KDA_CHECK(a->q != nullptr && aligned16(a->q) && a->o != nullptr && aligned16(a->o));
    KDA_CHECK(a->lse == nullptr || aligned4(a->lse));
    const size_t need = cache_attend_workspace(*c, *a);
    if (need > 0 && (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
                     workspace_bytes < need))
      return KDA_ERR_WORKSPACE;
  }
  if (a->status != nullptr && cudaMemsetAsync(a->status, 0, sizeof(int32_t), stream) != cudaSuccess)
    return KDA_ERR_CUDA;
  return c->num_seqs > 0 ? cuda_status(launch_cache_attend(*c, *a, workspace, stream)) : KDA_OK;
}

}  // extern "C"
