// Append to and read from the NVFP4 key/value cache.
//
// Append: a query or key head of D elements turns in pairs (a, b) by the angle
// of its position,  a' = a cos - b sin,  b' = b cos + a sin,  and a key or value
// block of 16 is held as  s = E4M3(amax / 6 * g),  code = E2M1(x * (g / s)).
// Every step is one IEEE FP32 operation (no contraction), so the cache's bytes
// are those of any other implementation of these steps.
//
// Bound by memory: q, k and v come in once and q goes out once (the cache's 9/16
// of a byte per element is small beside them): 8192 tokens of 40 + 2 x 4 heads of
// 128 (195 MB) take 41.5 us, 4.7 TB/s, the rate of a large copy; 64 tokens (1.5 MB)
// 4.7 us and a read-back of them 4.6, a launch each. Where rot is no multiple of 16, elements
// move two bytes at a time: 8192 tokens of 48 heads of 80, 40 of them turned (119 MB), take 117 us,
// 1.0 TB/s. A thread owns eight pairs of one
// token: their cosines and sines stay in registers over the heads of its group,
// so the table is read once per group and not once per head. A turned key head
// goes through LDS, because the pairs (j, j + rot/2) of one thread lie in two
// quantization blocks.
#pragma clang fp contract(off)

#include "e4m3.hpp"
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

// The elements that a thread turns or passes on: a[j], b[j] of pair 8 c + j, or (c past the turned
// ones) sixteen consecutive elements. As loaded, 16 bytes wide (VEC: rot is a multiple of 16), or
// one by one.
struct Part {
  u32x4_t lo, hi;
};

template <bool INTER>
__device__ __forceinline__ void part_at(int c, int D, int rot, int turn_chunks, int j, int *ea, int *eb, bool *fa, bool *fb) {
  const int half = rot / 2, p = 8 * c + j, e = rot + 16 * (c - turn_chunks) + j;
  const bool turn = c < turn_chunks;
  *ea = !turn ? e : INTER ? 2 * p : p;
  *eb = !turn ? e + 8 : INTER ? 2 * p + 1 : p + half;
  *fa = turn ? p < half : e < D;
  *fb = turn ? p < half : e + 8 < D;
}

template <bool INTER>
__device__ __forceinline__ void first_of(int c, int rot, int turn_chunks, int *ea, int *eb) {
  const bool turn = c < turn_chunks;
  *ea = !turn ? rot + 16 * (c - turn_chunks) : INTER ? 16 * c : 8 * c;
  *eb = (turn && !INTER) ? rot / 2 + 8 * c : *ea + 8;
}

template <bool VEC, bool INTER>
__device__ __forceinline__ Part load_part(const uint16_t *x, int c, int D, int rot, int turn_chunks) {
  Part r;
  if (VEC) {
    int ea, eb;
    first_of<INTER>(c, rot, turn_chunks, &ea, &eb);
    r.lo = *reinterpret_cast<const u32x4_t *>(x + ea);
    r.hi = *reinterpret_cast<const u32x4_t *>(x + eb);
  } else {
    uint16_t a[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      int ea, eb;
      bool fa, fb;
      part_at<INTER>(c, D, rot, turn_chunks, j, &ea, &eb, &fa, &fb);
      a[j] = fa ? x[ea] : 0;
      b[j] = fb ? x[eb] : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      r.lo[i] = a[2 * i] | ((uint32_t)a[2 * i + 1] << 16);
      r.hi[i] = b[2 * i] | ((uint32_t)b[2 * i + 1] << 16);
    }
  }
  return r;
}

// Turns a part: x[0..7] and y[0..7] in the order in which they are stored (VEC: at first_of's two
// places; else a and b of part_at).
template <bool F16, bool VEC, bool INTER>
__device__ __forceinline__ void turn_part(const Part &r, bool turn, const float (&cs)[8], const float (&sn)[8],
                                          float (&x)[8], float (&y)[8]) {
  unpack8<F16>(r.lo, x);
  unpack8<F16>(r.hi, y);
  if (!turn) return;
  if (VEC && INTER) {              // pairs lie side by side: 0..3 in x, 4..7 in y
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const float a = x[2 * j], b = x[2 * j + 1];
      x[2 * j] = a * cs[j] - b * sn[j];
      x[2 * j + 1] = b * cs[j] + a * sn[j];
      const float d = y[2 * j], e = y[2 * j + 1];
      y[2 * j] = d * cs[j + 4] - e * sn[j + 4];
      y[2 * j + 1] = e * cs[j + 4] + d * sn[j + 4];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float a = x[j], b = y[j];
      x[j] = a * cs[j] - b * sn[j];
      y[j] = b * cs[j] + a * sn[j];
    }
  }
}

template <bool F16, bool VEC, bool INTER>
__global__ __launch_bounds__(kAppendThreads) void append_kernel(const AppendArgs A) {
  extern __shared__ float turned[];                  // [tokens of the workgroup][D], keys only
  constexpr int BATCH = 2;                           // heads whose loads are in flight together
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
    const uint16_t *x = A.v + t * A.v_t + blk * 16;
    const int h0 = group * A.per_group, h1 = min(kv.heads, h0 + A.per_group);
    uint8_t *page;
    uint32_t at;
    const bool keep = find_slot(kv, A.slots[t], &page, &at);
    for (int hb = h0; hb < h1; hb += BATCH) {
      u32x4_t lo[BATCH], hi[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; i++) {
        const uint16_t *from = x + min(hb + i, h1 - 1) * A.v_h;
        lo[i] = *reinterpret_cast<const u32x4_t *>(from);
        hi[i] = *reinterpret_cast<const u32x4_t *>(from + 8);
      }
      if (!keep) return;
#pragma unroll
      for (int i = 0; i < BATCH; i++) {
        const int h = hb + i;
        if (h >= h1) break;
        float a[8], b[8], all[16];
        unpack8<F16>(lo[i], a);
        unpack8<F16>(hi[i], b);
#pragma unroll
        for (int j = 0; j < 8; j++) all[j] = a[j], all[j + 8] = b[j];
        uint32_t sb;
        const u32x2_t codes = kv_quantize_block(all, kv.v_g ? kv.v_g[h] : 1.0f, &sb);
        uint8_t *head = page + (uint64_t)h * kv.head_bytes();
        uint32_t *to = reinterpret_cast<uint32_t *>(head + kv.v_codes() + ((at >> 2) * (uint32_t)(D / 8) + 2 * blk) * 16 +
                                                    (at & 3u) * 4);
        to[0] = codes[0];
        to[4] = codes[1];
        head[kv.v_scales() + ((uint32_t)blk << kv.log_p) + at] = (uint8_t)sb;
      }
    }
    return;
  }

  const bool is_q = group < A.q_groups;
  const int tl = threadIdx.x / A.chunks, c = threadIdx.x % A.chunks;
  const int64_t t = first + tl;
  const bool active = tl < per_wg && t < A.tokens, turn = c < A.turn_chunks;
  const int half = A.rot / 2;
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; j++) cs[j] = 1.0f, sn[j] = 0.0f;
  if (active && turn) {
    const float nan = __builtin_nanf("");
    // the eight pairs' axes; where they are the same one, their angles lie side by side in the table
    uint64_t axes = 0;
    if (VEC && A.axis_of) __builtin_memcpy(&axes, A.axis_of + 8 * c, 8);
    if (VEC && axes == (axes & 0xFFu) * 0x0101010101010101ull) {
      const int axis = min((int)(axes & 0xFFu), A.axes - 1);
      const int64_t pos = A.positions[axis * A.position_stride + t];
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
    const uint16_t *src = A.q + t * A.q_t;
    uint16_t *dst = A.q_out + t * A.o_t;
    const int h0 = group * A.per_group, h1 = min(A.q_heads, h0 + A.per_group);
    for (int hb = h0; hb < h1; hb += BATCH) {
      Part r[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; i++)
        r[i] = load_part<VEC, INTER>(src + min(hb + i, h1 - 1) * A.q_h, c, D, A.rot, A.turn_chunks);
#pragma unroll
      for (int i = 0; i < BATCH; i++) {
        if (hb + i >= h1) break;
        float x[8], y[8];
        turn_part<F16, VEC, INTER>(r[i], turn, cs, sn, x, y);
        uint16_t *o = dst + (hb + i) * A.o_h;
        if (VEC) {
          int ea, eb;
          first_of<INTER>(c, A.rot, A.turn_chunks, &ea, &eb);
          *reinterpret_cast<u32x4_t *>(o + ea) = pack8<F16>(x);
          *reinterpret_cast<u32x4_t *>(o + eb) = pack8<F16>(y);
        } else {
#pragma unroll
          for (int j = 0; j < 8; j++) {
            int ea, eb;
            bool fa, fb;
            part_at<INTER>(c, D, A.rot, A.turn_chunks, j, &ea, &eb, &fa, &fb);
            if (fa) o[ea] = pack1<F16>(x[j]);
            if (fb) o[eb] = pack1<F16>(y[j]);
          }
        }
      }
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
      float x[8], y[8];
      turn_part<F16, VEC, INTER>(load_part<VEC, INTER>(A.k + t * A.k_t + h * A.k_h, c, D, A.rot, A.turn_chunks), turn,
                                 cs, sn, x, y);
      float *row = turned + tl * D;
      if (VEC) {
        int ea, eb;
        first_of<INTER>(c, A.rot, A.turn_chunks, &ea, &eb);
        *reinterpret_cast<f32x4_t *>(row + ea) = f32x4_t{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<f32x4_t *>(row + ea + 4) = f32x4_t{x[4], x[5], x[6], x[7]};
        *reinterpret_cast<f32x4_t *>(row + eb) = f32x4_t{y[0], y[1], y[2], y[3]};
        *reinterpret_cast<f32x4_t *>(row + eb + 4) = f32x4_t{y[4], y[5], y[6], y[7]};
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
          int ea, eb;
          bool fa, fb;
          part_at<INTER>(c, D, A.rot, A.turn_chunks, j, &ea, &eb, &fa, &fb);
          if (fa) row[ea] = x[j];
          if (fb) row[eb] = y[j];
        }
      }
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

template <bool F16, bool VEC, bool INTER>
static void launch_append(const AppendArgs &A, dim3 grid, size_t lds, hipStream_t s) {
  hipLaunchKernelGGL((append_kernel<F16, VEC, INTER>), grid, dim3(kAppendThreads), lds, s, A);
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
  if (wgs > kMostWorkgroups) return NVFP4_ERR_SHAPE;
  DeviceInfo d;
  st = device_info(&d);
  if (st != NVFP4_OK) return st;
  // Sixteen heads to a group share one read of the table (8192 tokens of 48 heads, replayed in a graph:
  // 33.3 us, 35.3 with eight); with few tokens, fewer heads to a group fill the CUs instead (64 tokens:
  // 4.3 us with one, 5.8 with two, 8.8 with four to sixteen).
  int groups;
  for (A.per_group = 16;; A.per_group /= 2) {
    A.q_groups = (A.q_heads + A.per_group - 1) / A.per_group;
    A.kv_groups = (A.kv.heads + A.per_group - 1) / A.per_group;
    groups = A.q_groups + 2 * A.kv_groups;
    if (A.per_group == 1 || wgs * groups >= 2 * d.num_cus) break;
  }
  if (groups > 65535) return NVFP4_ERR_SHAPE;
  const dim3 grid((unsigned)wgs, (unsigned)groups);
  const size_t lds = (size_t)per_wg * D * 4;
  const bool vec = A.rot % 16 == 0, f16 = dtype == NVFP4_F16;
  hipStream_t s = (hipStream_t)stream;
  if (vec && A.interleaved) f16 ? launch_append<true, true, true>(A, grid, lds, s) : launch_append<false, true, true>(A, grid, lds, s);
  else if (vec) f16 ? launch_append<true, true, false>(A, grid, lds, s) : launch_append<false, true, false>(A, grid, lds, s);
  else if (A.interleaved) f16 ? launch_append<true, false, true>(A, grid, lds, s) : launch_append<false, false, true>(A, grid, lds, s);
  else f16 ? launch_append<true, false, false>(A, grid, lds, s) : launch_append<false, false, false>(A, grid, lds, s);
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
  if (tokens > kMostWorkgroups * 256 / per_token) return NVFP4_ERR_SHAPE;
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
