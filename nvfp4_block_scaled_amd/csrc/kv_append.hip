// Append to and read from the NVFP4 key/value cache.
//
// Append: a query or key head of D elements turns in pairs (a, b) by the angle
// of its position,  a' = a cos - b sin,  b' = b cos + a sin,  and a key or value
// block of 16 is held as  s = E4M3(amax / 6 * g),  code = E2M1(x * (g / s)).
// Every step is one IEEE FP32 operation (no contraction), so the cache's bytes
// are those of any other implementation of these steps.
//
// Bound by memory: q, k and v come in once and q goes out once (the cache's 9/16
// of a byte per element is small beside them). A thread owns eight pairs of one
// token: their cosines and sines stay in registers over the heads of its group,
// so the table is read once per group and not once per head. A turned key head
// goes through LDS, because the pairs (j, j + rot/2) of one thread lie in two
// quantization blocks.
#pragma clang fp contract(off)

#include "kv_common.hpp"

namespace nvfp4 {

static constexpr int kAppendThreads = 256;

struct AppendArgs {
  KvView kv;
  const uint16_t *k, *v, *q;
  uint16_t *q_out;
  int64_t k_t, k_h, v_t, v_h, q_t, q_h, o_t, o_h;
  int64_t tokens;
  const int64_t *slots;
  const float *cos, *sin;
  const int32_t *positions;
  const uint8_t *axis_of;
  int64_t max_pos, position_stride;
  int32_t q_heads, rot, interleaved, axes;
  int32_t per_group;        // heads that one workgroup handles
  int32_t q_groups, kv_groups;
  int32_t turn_chunks;      // threads of a token that turn eight pairs each
  int32_t chunks;           // threads of a token, with those that pass elements on
};

// The scale byte and codes of one block; NaN anywhere in it makes the scale NaN.
__device__ __forceinline__ u32x2_t kv_quantize_block(const float (&x)[16], float g, uint32_t *sbyte) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; i++) top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);   // ordered as |x|, NaN last
  u32x2_t out = {0u, 0u};
  *sbyte = 0u;
  if (top > 0x7F800000u) {
    *sbyte = 0x7Fu;
    return out;
  }
  if (top == 0u) return out;
  const float t = __uint_as_float(top) / 6.0f;
  const uint32_t sb = e4m3_rne_sat(t * g);
  *sbyte = sb;
  if (sb != 0u) {
    const float r = g / e4m3_value(sb);
#define NVFP4_KV_CVT(D, B) \
  out[D] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out[D], x[8 * D + 2 * B] * r, x[8 * D + 2 * B + 1] * r, 1.0f, B)
    NVFP4_KV_CVT(0, 0); NVFP4_KV_CVT(0, 1); NVFP4_KV_CVT(0, 2); NVFP4_KV_CVT(0, 3);
    NVFP4_KV_CVT(1, 0); NVFP4_KV_CVT(1, 1); NVFP4_KV_CVT(1, 2); NVFP4_KV_CVT(1, 3);
#undef NVFP4_KV_CVT
  }
  return out;
}

// Where a token's slot lies: the page's base, and the place in it; false outside the pool.
__device__ __forceinline__ bool find_slot(const KvView &kv, int64_t slot, uint8_t **page, uint32_t *at) {
  const int64_t p = slot >> kv.log_p;
  if (slot < 0 || p >= kv.num_pages) return false;
  *page = kv.pages + p * kv.page_stride;
  *at = (uint32_t)slot & (kv.P() - 1u);
  return true;
}

// The elements a thread turns or passes on: a[j], b[j] of pair 8 c + j, or (c past the turned
// ones) sixteen consecutive elements. VEC: rot is a multiple of 16, every access 16 bytes wide.
template <bool F16, bool VEC>
__device__ __forceinline__ void load_pairs(const uint16_t *x, int c, int D, int rot, int turn_chunks, bool inter,
                                           float (&a)[8], float (&b)[8]) {
  const int half = rot / 2;
  const bool turn = c < turn_chunks;
  if (VEC) {
    const int ea = !turn ? rot + 16 * (c - turn_chunks) : inter ? 16 * c : 8 * c;
    const int eb = (turn && !inter) ? half + 8 * c : ea + 8;
    float lo[8], hi[8];
    unpack8<F16>(*reinterpret_cast<const u32x4_t *>(x + ea), lo);
    unpack8<F16>(*reinterpret_cast<const u32x4_t *>(x + eb), hi);
    if (turn && inter) {
#pragma unroll
      for (int j = 0; j < 4; j++) {
        a[j] = lo[2 * j], b[j] = lo[2 * j + 1];
        a[j + 4] = hi[2 * j], b[j + 4] = hi[2 * j + 1];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) a[j] = lo[j], b[j] = hi[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const int p = 8 * c + j, e = rot + 16 * (c - turn_chunks) + j;
      const int ia = !turn ? e : inter ? 2 * p : p;
      const int ib = !turn ? e + 8 : inter ? 2 * p + 1 : p + half;
      const bool fa = turn ? p < half : e < D, fb = turn ? p < half : e + 8 < D;
      a[j] = fa ? unpack1<F16>(x[ia]) : 0.0f;
      b[j] = fb ? unpack1<F16>(x[ib]) : 0.0f;
    }
  }
}

// Calls put(element, value) or put8(first element, eight values) for what load_pairs read.
template <bool VEC, typename Put, typename Put8>
__device__ __forceinline__ void store_pairs(int c, int D, int rot, int turn_chunks, bool inter, const float (&a)[8],
                                            const float (&b)[8], Put put, Put8 put8) {
  const int half = rot / 2;
  const bool turn = c < turn_chunks;
  if (VEC) {
    const int ea = !turn ? rot + 16 * (c - turn_chunks) : inter ? 16 * c : 8 * c;
    const int eb = (turn && !inter) ? half + 8 * c : ea + 8;
    if (turn && inter) {
      float lo[8], hi[8];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        lo[2 * j] = a[j], lo[2 * j + 1] = b[j];
        hi[2 * j] = a[j + 4], hi[2 * j + 1] = b[j + 4];
      }
      put8(ea, lo);
      put8(eb, hi);
    } else {
      put8(ea, a);
      put8(eb, b);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const int p = 8 * c + j, e = rot + 16 * (c - turn_chunks) + j;
      if (turn) {
        if (p < half) {
          put(inter ? 2 * p : p, a[j]);
          put(inter ? 2 * p + 1 : p + half, b[j]);
        }
      } else {
        if (e < D) put(e, a[j]);
        if (e + 8 < D) put(e + 8, b[j]);
      }
    }
  }
}

template <bool F16, bool VEC>
__global__ __launch_bounds__(kAppendThreads) void append_kernel(const AppendArgs A) {
  extern __shared__ float turned[];                  // [tokens of the workgroup][D], keys only
  const KvView &kv = A.kv;
  const int D = kv.D, blocks = D / 16;
  const int per_wg = kAppendThreads / A.chunks;      // tokens of a workgroup
  const int64_t first = (int64_t)blockIdx.x * per_wg;
  int group = blockIdx.y;

  if (group >= A.q_groups + A.kv_groups) {           // values: a thread per block
    group -= A.q_groups + A.kv_groups;
    const int tl = threadIdx.x / blocks, blk = threadIdx.x % blocks;
    const int64_t t = first + tl;
    if (tl >= per_wg || t >= A.tokens) return;
    uint8_t *page;
    uint32_t at;
    if (!find_slot(kv, A.slots[t], &page, &at)) return;
    const int h1 = min(kv.heads, (group + 1) * A.per_group);
    for (int h = group * A.per_group; h < h1; h++) {
      const uint16_t *x = A.v + t * A.v_t + h * A.v_h + blk * 16;
      float lo[8], hi[8], all[16];
      unpack8<F16>(*reinterpret_cast<const u32x4_t *>(x), lo);
      unpack8<F16>(*reinterpret_cast<const u32x4_t *>(x + 8), hi);
#pragma unroll
      for (int j = 0; j < 8; j++) all[j] = lo[j], all[j + 8] = hi[j];
      uint32_t sb;
      const u32x2_t codes = kv_quantize_block(all, kv.v_g ? kv.v_g[h] : 1.0f, &sb);
      uint8_t *head = page + (uint64_t)h * kv.head_bytes();
      uint32_t *to = reinterpret_cast<uint32_t *>(head + kv.v_codes() + ((at >> 2) * (uint32_t)(D / 8) + 2 * blk) * 16 +
                                                  (at & 3u) * 4);
      to[0] = codes[0];
      to[4] = codes[1];
      head[kv.v_scales() + ((uint32_t)blk << kv.log_p) + at] = (uint8_t)sb;
    }
    return;
  }

  const bool is_q = group < A.q_groups;
  const int tl = threadIdx.x / A.chunks, c = threadIdx.x % A.chunks;
  const int64_t t = first + tl;
  const bool active = tl < per_wg && t < A.tokens;
  const int half = A.rot / 2;
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; j++) cs[j] = 1.0f, sn[j] = 0.0f;
  if (active && c < A.turn_chunks) {
    const float nan = __builtin_nanf("");
    if (VEC && !A.axis_of) {
      const int64_t pos = A.positions[t];
      const bool in = pos >= 0 && pos < A.max_pos;
      const int64_t row = (in ? pos : 0) * half + 8 * c;
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const u32x4_t cw = *reinterpret_cast<const u32x4_a4 *>(A.cos + row + 4 * i);
        const u32x4_t sw = *reinterpret_cast<const u32x4_a4 *>(A.sin + row + 4 * i);
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const uint32_t u = cw[j], w = sw[j];
          cs[4 * i + j] = in ? __uint_as_float(u) : nan;
          sn[4 * i + j] = in ? __uint_as_float(w) : nan;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int p = 8 * c + j;
        if (p < half) {
          const int axis = A.axis_of ? min((int)A.axis_of[p], A.axes - 1) : 0;
          const int64_t pos = A.positions[axis * A.position_stride + t];
          const bool in = pos >= 0 && pos < A.max_pos;
          const int64_t at = (in ? pos : 0) * half + p;
          cs[j] = in ? A.cos[at] : nan;
          sn[j] = in ? A.sin[at] : nan;
        }
      }
    }
  }

  if (is_q) {
    if (!active) return;
    const int h1 = min(A.q_heads, (group + 1) * A.per_group);
    for (int h = group * A.per_group; h < h1; h++) {
      float a[8], b[8];
      load_pairs<F16, VEC>(A.q + t * A.q_t + h * A.q_h, c, D, A.rot, A.turn_chunks, A.interleaved, a, b);
      if (c < A.turn_chunks) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float x = a[j] * cs[j] - b[j] * sn[j];
          const float y = b[j] * cs[j] + a[j] * sn[j];
          a[j] = x, b[j] = y;
        }
      }
      uint16_t *o = A.q_out + t * A.o_t + h * A.o_h;
      store_pairs<VEC>(c, D, A.rot, A.turn_chunks, A.interleaved, a, b, [&](int e, float x) { o[e] = pack1<F16>(x); },
                       [&](int e, const float(&x)[8]) { *reinterpret_cast<u32x4_t *>(o + e) = pack8<F16>(x); });
    }
    return;
  }

  group -= A.q_groups;
  const int qt = threadIdx.x / blocks, blk = threadIdx.x % blocks;    // the block that this thread quantizes
  const int64_t t2 = first + qt;
  uint8_t *page = nullptr;
  uint32_t at = 0;
  const bool keep = qt < per_wg && t2 < A.tokens && find_slot(kv, A.slots[t2], &page, &at);
  const int h1 = min(kv.heads, (group + 1) * A.per_group);
  for (int h = group * A.per_group; h < h1; h++) {
    if (active) {
      float a[8], b[8];
      load_pairs<F16, VEC>(A.k + t * A.k_t + h * A.k_h, c, D, A.rot, A.turn_chunks, A.interleaved, a, b);
      if (c < A.turn_chunks) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float x = a[j] * cs[j] - b[j] * sn[j];
          const float y = b[j] * cs[j] + a[j] * sn[j];
          a[j] = x, b[j] = y;
        }
      }
      float *row = turned + tl * D;
      store_pairs<VEC>(c, D, A.rot, A.turn_chunks, A.interleaved, a, b, [&](int e, float x) { row[e] = x; },
                       [&](int e, const float(&x)[8]) {
                         *reinterpret_cast<f32x4_t *>(row + e) = f32x4_t{x[0], x[1], x[2], x[3]};
                         *reinterpret_cast<f32x4_t *>(row + e + 4) = f32x4_t{x[4], x[5], x[6], x[7]};
                       });
    }
    __syncthreads();
    if (keep) {
      float all[16];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const f32x4_t w = *reinterpret_cast<const f32x4_t *>(turned + qt * D + blk * 16 + 4 * i);
        all[4 * i] = w[0], all[4 * i + 1] = w[1], all[4 * i + 2] = w[2], all[4 * i + 3] = w[3];
      }
      uint32_t sb;
      const u32x2_t codes = kv_quantize_block(all, kv.k_g ? kv.k_g[h] : 1.0f, &sb);
      uint8_t *head = page + (uint64_t)h * kv.head_bytes();
      *reinterpret_cast<u32x2_t *>(head + at * (uint32_t)(D / 2) + blk * 8) = codes;
      head[kv.k_scales() + at * (uint32_t)blocks + blk] = (uint8_t)sb;
    }
    __syncthreads();
  }
}

// fl32(code * scale / g) of a block of 16: the product is exact, the division rounds.
__device__ __forceinline__ void kv_block_values(uint32_t w0, uint32_t w1, uint32_t sbyte, float g, float (&lo)[8],
                                                float (&hi)[8]) {
  const float s = e4m3x2_to_f32(sbyte)[0];
#define NVFP4_KV_VAL(X, W, B)                                              \
  {                                                                        \
    const f32x2_t q = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(W, 1.0f, B); \
    X[2 * B] = (q[0] * s) / g;                                             \
    X[2 * B + 1] = (q[1] * s) / g;                                         \
  }
  NVFP4_KV_VAL(lo, w0, 0) NVFP4_KV_VAL(lo, w0, 1) NVFP4_KV_VAL(lo, w0, 2) NVFP4_KV_VAL(lo, w0, 3)
  NVFP4_KV_VAL(hi, w1, 0) NVFP4_KV_VAL(hi, w1, 1) NVFP4_KV_VAL(hi, w1, 2) NVFP4_KV_VAL(hi, w1, 3)
#undef NVFP4_KV_VAL
}

struct ReadArgs {
  KvView kv;
  const int64_t *slots;
  int64_t tokens;
  void *k, *v;
  int64_t k_t, k_h, v_t, v_h;
};

template <int TYPE>
__device__ __forceinline__ void store16(void *base, int64_t at, const float (&lo)[8], const float (&hi)[8]) {
  if (TYPE == NVFP4_F32) {
    f32x4_t *o = reinterpret_cast<f32x4_t *>((float *)base + at);
    o[0] = f32x4_t{lo[0], lo[1], lo[2], lo[3]};
    o[1] = f32x4_t{lo[4], lo[5], lo[6], lo[7]};
    o[2] = f32x4_t{hi[0], hi[1], hi[2], hi[3]};
    o[3] = f32x4_t{hi[4], hi[5], hi[6], hi[7]};
  } else {
    u32x4_t *o = reinterpret_cast<u32x4_t *>((uint16_t *)base + at);
    o[0] = pack8<TYPE == NVFP4_F16>(lo);
    o[1] = pack8<TYPE == NVFP4_F16>(hi);
  }
}

// A thread per (token, head, block of 16), both sides.
template <int TYPE>
__global__ __launch_bounds__(256) void read_kernel(const ReadArgs A) {
  const KvView &kv = A.kv;
  const int D = kv.D, blocks = D / 16;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / blocks;
  const int blk = (int)(i - row * blocks);
  const int64_t t = row / kv.heads;
  const int h = (int)(row - t * kv.heads);
  if (t >= A.tokens) return;
  uint8_t *page;
  uint32_t at;
  float lo[8], hi[8];
  const bool in = find_slot(kv, A.slots[t], &page, &at);
#pragma unroll
  for (int j = 0; j < 8; j++) lo[j] = 0.0f, hi[j] = 0.0f;
  const uint8_t *head = in ? page + (uint64_t)h * kv.head_bytes() : nullptr;
  if (in) {
    const u32x2_t w = *reinterpret_cast<const u32x2_t *>(head + at * (uint32_t)(D / 2) + blk * 8);
    kv_block_values(w[0], w[1], head[kv.k_scales() + at * (uint32_t)blocks + blk], kv.k_g ? kv.k_g[h] : 1.0f, lo, hi);
  }
  store16<TYPE>(A.k, t * A.k_t + h * A.k_h + blk * 16, lo, hi);
  if (in) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(
        head + kv.v_codes() + ((at >> 2) * (uint32_t)(D / 8) + 2 * blk) * 16 + (at & 3u) * 4);
    kv_block_values(w[0], w[4], head[kv.v_scales() + ((uint32_t)blk << kv.log_p) + at], kv.v_g ? kv.v_g[h] : 1.0f, lo,
                    hi);
  }
  store16<TYPE>(A.v, t * A.v_t + h * A.v_h + blk * 16, lo, hi);
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_kv_page_bytes(int32_t page_size, int32_t kv_heads, int32_t head_dim) {
  if (!kv_geometry_ok(page_size, kv_heads, head_dim)) return 0;
  return (size_t)kv_page_bytes_of(page_size, kv_heads, head_dim);
}

nvfp4_status nvfp4_kv_append(const nvfp4_kv_cache *cache, nvfp4_rows k, nvfp4_rows v, nvfp4_rows q, nvfp4_rows q_out,
                             int dtype, int64_t tokens, int32_t q_heads, const int64_t *slots,
                             const nvfp4_rope *rope, void *stream) {
  if (dtype != NVFP4_BF16 && dtype != NVFP4_F16) return NVFP4_ERR_DTYPE;
  AppendArgs A = {};
  nvfp4_status st = kv_view(cache, &A.kv);
  if (st != NVFP4_OK) return st;
  const int D = A.kv.D;
  const bool with_q = q.base != nullptr;
  if (tokens < 0 || (with_q && (q_heads < 1 || q_heads > 65535))) return NVFP4_ERR_SHAPE;
  if (rope) {
    if (rope->rot_dim < 0 || rope->rot_dim > D || rope->rot_dim % 2 != 0) return NVFP4_ERR_SHAPE;
    if (rope->rot_dim > 0) {
      if (rope->max_pos < 1 || rope->max_pos > 0x7FFFFFFF || rope->axes < 1 || rope->axes > 255 ||
          (rope->axes > 1 && rope->position_stride < tokens))
        return NVFP4_ERR_SHAPE;
      if (rope->interleaved != 0 && rope->interleaved != 1) return NVFP4_ERR_VALUE;
    }
  }
  if (tokens == 0) return NVFP4_OK;
  if (!k.base || !v.base || !slots || (with_q && !q_out.base)) return NVFP4_ERR_NULL;
  if (rope && rope->rot_dim > 0 && (!rope->cos || !rope->sin || !rope->positions)) return NVFP4_ERR_NULL;
  if (!kv_rows_aligned(k) || !kv_rows_aligned(v) || (with_q && (!kv_rows_aligned(q) || !kv_rows_aligned(q_out))) ||
      !aligned(slots, 8))
    return NVFP4_ERR_ALIGN;
  if (rope && rope->rot_dim > 0 &&
      (!aligned(rope->cos, 4) || !aligned(rope->sin, 4) || !aligned(rope->positions, 4)))
    return NVFP4_ERR_ALIGN;
  DeviceInfo d;
  st = device_info(&d);
  if (st != NVFP4_OK) return st;

  A.k = (const uint16_t *)k.base, A.k_t = k.token_stride, A.k_h = k.head_stride;
  A.v = (const uint16_t *)v.base, A.v_t = v.token_stride, A.v_h = v.head_stride;
  A.q = (const uint16_t *)q.base, A.q_t = q.token_stride, A.q_h = q.head_stride;
  A.q_out = (uint16_t *)q_out.base, A.o_t = q_out.token_stride, A.o_h = q_out.head_stride;
  A.tokens = tokens;
  A.slots = slots;
  A.q_heads = with_q ? q_heads : 0;
  if (rope && rope->rot_dim > 0) {
    A.cos = rope->cos, A.sin = rope->sin, A.positions = rope->positions, A.axis_of = rope->axis_of;
    A.max_pos = rope->max_pos, A.position_stride = rope->position_stride;
    A.rot = rope->rot_dim, A.interleaved = rope->interleaved, A.axes = rope->axes;
  }
  A.turn_chunks = (A.rot / 2 + 7) / 8;
  A.chunks = A.turn_chunks + (D - A.rot + 15) / 16;
  const int per_wg = kAppendThreads / A.chunks;
  const int64_t wgs = (tokens + per_wg - 1) / per_wg;
  if (wgs > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  A.per_group = 8;
  A.q_groups = (A.q_heads + A.per_group - 1) / A.per_group;
  A.kv_groups = (A.kv.heads + A.per_group - 1) / A.per_group;
  const dim3 grid((unsigned)wgs, (unsigned)(A.q_groups + 2 * A.kv_groups));
  const size_t lds = (size_t)per_wg * D * 4;
  const bool vec = A.rot % 16 == 0;
  hipStream_t s = (hipStream_t)stream;
  if (dtype == NVFP4_F16) {
    if (vec) hipLaunchKernelGGL((append_kernel<true, true>), grid, dim3(kAppendThreads), lds, s, A);
    else hipLaunchKernelGGL((append_kernel<true, false>), grid, dim3(kAppendThreads), lds, s, A);
  } else {
    if (vec) hipLaunchKernelGGL((append_kernel<false, true>), grid, dim3(kAppendThreads), lds, s, A);
    else hipLaunchKernelGGL((append_kernel<false, false>), grid, dim3(kAppendThreads), lds, s, A);
  }
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

nvfp4_status nvfp4_kv_read(const nvfp4_kv_cache *cache, const int64_t *slots, int64_t tokens, int dtype, nvfp4_rows k,
                           nvfp4_rows v, void *stream) {
  if (dtype != NVFP4_F32 && dtype != NVFP4_BF16 && dtype != NVFP4_F16) return NVFP4_ERR_DTYPE;
  ReadArgs A = {};
  nvfp4_status st = kv_view(cache, &A.kv);
  if (st != NVFP4_OK) return st;
  if (tokens < 0) return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  if (!slots || !k.base || !v.base) return NVFP4_ERR_NULL;
  if (!kv_rows_aligned(k) || !kv_rows_aligned(v) || !aligned(slots, 8)) return NVFP4_ERR_ALIGN;
  const int64_t per_token = (int64_t)A.kv.heads * (A.kv.D / 16);
  if (tokens > ((int64_t)0x7FFFFFFF * 256) / per_token) return NVFP4_ERR_SHAPE;
  DeviceInfo d;
  st = device_info(&d);
  if (st != NVFP4_OK) return st;
  A.slots = slots, A.tokens = tokens;
  A.k = k.base, A.k_t = k.token_stride, A.k_h = k.head_stride;
  A.v = v.base, A.v_t = v.token_stride, A.v_h = v.head_stride;
  const dim3 grid((unsigned)((tokens * per_token + 255) / 256));
  hipStream_t s = (hipStream_t)stream;
  if (dtype == NVFP4_F32) hipLaunchKernelGGL(read_kernel<NVFP4_F32>, grid, dim3(256), 0, s, A);
  else if (dtype == NVFP4_BF16) hipLaunchKernelGGL(read_kernel<NVFP4_BF16>, grid, dim3(256), 0, s, A);
  else hipLaunchKernelGGL(read_kernel<NVFP4_F16>, grid, dim3(256), 0, s, A);
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

}  // extern "C"
