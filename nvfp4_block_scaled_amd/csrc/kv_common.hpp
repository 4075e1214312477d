// What the key/value cache's kernels share: the page layout of nvfp4.h as
// offsets, 16-bit loads and stores, and the host-side argument checks.
#pragma once

#include "common.hpp"

namespace nvfp4 {

// A 16-byte vector that may lie at any 4-byte (loads of code rows) or 8-byte
// boundary: head dimensions that are no multiple of 32 have rows of 8 (2 j + 1)
// bytes.
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));
typedef u32x2_t u32x2_a4 __attribute__((aligned(4)));

// The cache as the kernels see it. Byte offsets inside one head's part of a
// page fit 32 bits (256 tokens x 256 elements x 9/8); page offsets are 64-bit.
struct KvView {
  uint8_t *pages;
  int64_t page_stride;
  int32_t num_pages;
  int32_t log_p;       // log2 of the page size
  int32_t heads;
  int32_t D;
  const float *k_g, *v_g;

  __host__ __device__ __forceinline__ uint32_t P() const { return 1u << log_p; }
  __host__ __device__ __forceinline__ uint32_t k_scales() const { return ((uint32_t)D << log_p) / 2; }
  __host__ __device__ __forceinline__ uint32_t v_codes() const { return ((uint32_t)D << log_p) / 16 * 9; }
  __host__ __device__ __forceinline__ uint32_t v_scales() const { return ((uint32_t)D << log_p) / 16 * 17; }
  __host__ __device__ __forceinline__ uint32_t head_bytes() const { return ((uint32_t)D << log_p) / 8 * 9; }
};

// The most workgroups of 256 threads in a launch along one dimension: the runtime
// counts threads in 32 bits and drops the rest without an error.
constexpr int64_t kMostWorkgroups = 0xFFFFFF;

// CUs of the current device; 256 where there is none (config.hip).
int device_cus_or_default();

inline bool kv_geometry_ok(int32_t page_size, int32_t kv_heads, int32_t head_dim) {
  return (page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128 || page_size == 256) &&
         kv_heads >= 1 && kv_heads <= 65535 && head_dim >= 16 && head_dim <= 256 && head_dim % 16 == 0;
}

inline int64_t kv_page_bytes_of(int32_t page_size, int32_t kv_heads, int32_t head_dim) {
  return (int64_t)kv_heads * page_size * (head_dim / 16) * 18;
}

// Checks a cache descriptor and turns it into the kernels' view of it.
inline nvfp4_status kv_view(const nvfp4_kv_cache *c, KvView *v) {
  if (!c) return NVFP4_ERR_NULL;
  if (!kv_geometry_ok(c->page_size, c->kv_heads, c->head_dim)) return NVFP4_ERR_SHAPE;
  if (c->num_pages < 1 || c->num_pages > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  if (c->page_stride < kv_page_bytes_of(c->page_size, c->kv_heads, c->head_dim)) return NVFP4_ERR_SHAPE;
  if (c->page_stride > INT64_MAX / c->num_pages) return NVFP4_ERR_SHAPE;
  if (!c->pages) return NVFP4_ERR_NULL;
  if (!aligned(c->pages, 16) || c->page_stride % 16 != 0) return NVFP4_ERR_ALIGN;
  if ((c->k_g && !aligned(c->k_g, 4)) || (c->v_g && !aligned(c->v_g, 4))) return NVFP4_ERR_ALIGN;
  v->pages = c->pages;
  v->page_stride = c->page_stride;
  v->num_pages = (int32_t)c->num_pages;
  v->log_p = __builtin_ctz((unsigned)c->page_size);
  v->heads = c->kv_heads;
  v->D = c->head_dim;
  v->k_g = c->k_g;
  v->v_g = c->v_g;
  return NVFP4_OK;
}

// Alignment of a [tokens][heads][D] tensor (elements of 2 or 4 bytes).
inline bool kv_rows_aligned(const nvfp4_rows &r) {
  return aligned(r.base, 16) && r.token_stride % 8 == 0 && r.head_stride % 8 == 0;
}

// Eight consecutive 16-bit elements (16-byte aligned) as FP32 values (exact).
template <bool F16>
__device__ __forceinline__ void unpack8(const u32x4_t w, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t u = w[i];
    if (F16) {
      half2_t h;
      __builtin_memcpy(&h, &u, 4);
      x[2 * i] = (float)h[0];
      x[2 * i + 1] = (float)h[1];
    } else {
      x[2 * i] = __uint_as_float(u << 16);
      x[2 * i + 1] = __uint_as_float(u & 0xFFFF0000u);
    }
  }
}

// One FP32 value rounded to nearest even in 16 bits.
template <bool F16>
__device__ __forceinline__ uint16_t pack1(float x) {
  if (F16) {
    const _Float16 h = (_Float16)x;
    uint16_t b;
    __builtin_memcpy(&b, &h, 2);
    return b;
  }
  return f32_to_bf16_rne(x);
}

template <bool F16>
__device__ __forceinline__ u32x4_t pack8(const float (&x)[8]) {
  u32x4_t w;
#pragma unroll
  for (int i = 0; i < 4; i++)
    w[i] = (uint32_t)pack1<F16>(x[2 * i]) | ((uint32_t)pack1<F16>(x[2 * i + 1]) << 16);
  return w;
}

}  // namespace nvfp4
