// Quantization into FP8 with a scale for each block of 128 columns: E4M3 codes
// and FP32 scales, per row for activations, per 128 x 128 block for weights.
//
//   scale = max(amax, 2^-100) / 448,   code = E4M3_RNE(x / scale)
//
// both divisions in IEEE FP32, so |x / scale| <= 448 (1 + 2^-23) and nothing
// saturates. A block that holds a NaN or an infinity gets scale NaN and NaN
// codes. The maxima are taken over the bits of |x| as whole numbers, whose
// order is that of the values, with NaN above infinity.
//
// Everything is read once and written once: the kernels are bound by HBM. The
// codes' divisions would cost ten instructions each; with r = RN(1 / scale),
//   q = RN(x r),  q' = RN(q + r RN(x - q scale))
// is the correctly rounded quotient (Markstein's theorem: r correctly rounded,
// q within an ulp, the remainder exact), in three. The remainder is inexact
// only where it underflows, far below E4M3's smallest code.
#include "common.hpp"
#include "kv_common.hpp"
#include "launch.hpp"

namespace nvfp4 {
namespace fp8 {

constexpr float kTop = 448.0f;
constexpr uint32_t kLeastBits = 0x0D800000u;      // 2^-100
constexpr uint32_t kInfBits = 0x7F800000u;

// Inputs of over 64 MB (FAR) are read, and codes always written, past the caches
// (nontemporal): a large input has mostly left them, and what it would push out
// is worth more. A weight of 17408 x 5120 55 -> 50 us then; 8192 gated rows of 2 x 17408
// after a kernel that wrote them 248 -> 200; of inputs, 84 MB gain 8 % by it, 36 MB
// lose 3 to 7 %. Codes so written are read back by the next kernel as fast.
constexpr int64_t kNear = int64_t(64) << 20;

template <bool FAR, typename U>
__device__ __forceinline__ U fetch(const U *p) {
  return FAR ? __builtin_nontemporal_load(p) : *p;
}

// Eight consecutive elements of a row as FP32 values (exact); rows start at any element.
template <int DT, bool FAR>
__device__ __forceinline__ void load8(const void *p, float (&x)[8]) {
  if constexpr (DT == NVFP4_F32) {
    typedef f32x4_t U __attribute__((aligned(4)));
    const f32x4_t a = fetch<FAR>(static_cast<const U *>(p)), b = fetch<FAR>(static_cast<const U *>(p) + 1);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  } else {
    typedef u32x4_t U __attribute__((aligned(2)));
    const u32x4_t w = fetch<FAR>(static_cast<const U *>(p));
    unpack8<DT == NVFP4_F16>(w, x);
  }
}

// The largest |x| of eight as bits; a NaN if one is there (v_maximum3 keeps it).
__device__ __forceinline__ uint32_t max8(const float (&x)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) asm("v_maximum3_f32 %0, |%1|, |%2|, %0" : "+v"(m) : "v"(x[i]), "v"(x[i + 1]));
  return __float_as_uint(m) & 0x7FFFFFFFu;
}

// The largest of 16 lanes' (a row of the cross-lane network, turned by 8, 4, 2, 1), in each of them.
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xF, 0xF, false));
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x121, 0xF, 0xF, false));
}

// The scale of a block whose largest |x| has these bits, and its reciprocal.
struct Scale {
  float s, r;
};
__device__ __forceinline__ Scale block_scale(uint32_t top) {
  Scale k;
  if (top >= kInfBits) {
    k.s = k.r = __uint_as_float(0x7FC00000u);
  } else {
    k.s = __uint_as_float(max(top, kLeastBits)) / kTop;
    k.r = 1.0f / k.s;
  }
  return k;
}

// RN(x / s) for |x| <= 448 s (or a NaN where s is one). With the remainder taken
// from -x and negated, a remainder of zero is a zero of x's sign where x is one.
__device__ __forceinline__ float quotient(float x, Scale k) {
  const float q = x * k.r;
  return __builtin_fmaf(-__builtin_fmaf(q, k.s, -x), k.r, q);
}

__device__ __forceinline__ void store8(uint8_t *to, const float (&x)[8], Scale k) {
  u32x2_t c;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(x[4 * h], k), quotient(x[4 * h + 1], k), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(x[4 * h + 2], k), quotient(x[4 * h + 3], k), w, true);
    c[h] = (uint32_t)w;
  }
  __builtin_nontemporal_store(c, reinterpret_cast<u32x2_t *>(to));
}

// silu(g) u = g / (1 + e^-g) u for |g| <= 87. With t = RN(-g log2 e) and what that
// rounding lost, l (exact but for 2^-48 of t), e^-g = 2^t (1 + l ln 2), which is
// below 2^126, so the reciprocal of 1 + e^-g is a normal number. The quotient q by
// a reciprocal good to an ulp has the remainder g - q - q e, where g - q is exact
// for g > 0 (q is half of g at least), so the sum 1 + e need not be; remainder and
// q meet in the one multiply-add that rounds the result. Scales are 3.7e-8 off in
// the mean; 5.5e-8, and a quarter more codes on the other side of a tie, where the
// quotient is rounded before it meets u. The arithmetic counts here: 2048 rows of
// 2 x 17408 BF16 columns take 32 us, two less without that, 47.6 with the library's
// expf, a corrected reciprocal and a long division for each block's row.
constexpr float kLog2e = 0x1.715476p+0f, kLog2eRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
constexpr uint32_t kGateBits = 0x42AE0000u;      // 87

__device__ __forceinline__ float silu_mul(float g, float u) {
  const float t = g * -kLog2e;
  const float l = __builtin_fmaf(g, -kLog2eRest, __builtin_fmaf(g, -kLog2e, -t));
  const float p = __builtin_amdgcn_exp2f(t), e = __builtin_fmaf(p, l * kLn2, p);
  const float r = __builtin_amdgcn_rcpf(1.0f + e);
  const float q = g * r;
  return __builtin_fmaf(q, u, __builtin_fmaf(-q, e, g - q) * r * u);
}

// The same for any g. From 87 on, 1 + e^-g is 1 in FP32, and below -87 it is e^-g, so
// the result is g u or g e^g u. There e^g may be under FP32's range and u still bring
// the product back into it: e^g is taken times 2^160 (t + 160 is exact), u times
// 2^-60, and the rest follows at the end. g is taken as -180 where it is less: the
// largest u then gives 4e-38, a code of 0 under the smallest scale, and so does
// everything below. An infinite g leaves a NaN (-infinity times e to that), as a NaN does.
__device__ __forceinline__ float silu_mul_any(float g, float u) {
  if (!(fabsf(g) > 87.0f)) return silu_mul(g, u);
  if (g > 0.0f) return g * u;
  if (__float_as_uint(g) == 0xFF800000u) return __uint_as_float(0x7FC00000u);
  const float c = fmaxf(g, -180.0f), t = c * kLog2e;
  const float l = __builtin_fmaf(c, kLog2eRest, __builtin_fmaf(c, kLog2e, -t));
  const float p = __builtin_amdgcn_exp2f(t + 160.0f), e = __builtin_fmaf(p, l * kLn2, p);
  return __builtin_ldexpf(c * e * (u * 0x1p-60f), -100);
}

struct RowsArgs {
  const void *x;
  int64_t ldx;
  int64_t units;         // rows * blocks of a row
  int64_t K;
  int32_t blocks;        // of a row
  uint64_t inverse;      // 2^64 / blocks, rounded up (blocks > 1)
  uint32_t small;        // 2^16 / blocks + 1
  uint8_t *codes;
  float *scales;
};

// Sixteen lanes have a block of 128 columns, eight columns each; a thread has
// kRowBlocks blocks, whose loads are all in flight before the first is used (two:
// one, three and four are 1 to 8 % slower). K % 16 == 0: a lane's eight columns
// are all there or none is. Bound by HBM: 2048 rows of 34816 BF16 columns, 214 MB
// read and written, take 35 us (6.1 TB/s); gated into 17408, 178 MB, 32 (5.6).
constexpr int kThreads = 256, kRowBlocks = 2;

template <int DT, bool GATED, bool FAR>
__global__ __launch_bounds__(kThreads) void rows_kernel(RowsArgs a) {
  constexpr int ES = DT == NVFP4_F32 ? 4 : 2, U = kRowBlocks;
  const int l = threadIdx.x & 15, group = threadIdx.x >> 4;
  // The row of the workgroup's first block by one long product on the scalar unit (exact: units times blocks stay below
  // 2^64), its other blocks' from there: at most one row further, or by a short product where rows have few blocks.
  const uint64_t unit0 = (uint64_t)row_workgroup() * (kThreads / 16 * U), row0 = a.blocks > 1 ? __umul64hi(unit0, a.inverse) : unit0;
  const uint32_t block0 = (uint32_t)(unit0 - row0 * (uint32_t)a.blocks);
  const uint8_t *src = static_cast<const uint8_t *>(a.x) + row0 * a.ldx * ES;
  uint8_t *dst = a.codes + row0 * a.K;
  float x[U][8], up[GATED ? U : 1][8];
  uint64_t at[U];        // of the lane's columns in dst
  bool in[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    const uint32_t b = block0 + u * (kThreads / 16) + group;
    const uint32_t down = a.blocks >= kThreads / 16 * U ? (uint32_t)(b >= (uint32_t)a.blocks) : (b * a.small) >> 16;
    const uint32_t c = (b - down * (uint32_t)a.blocks) * 128 + l * 8;
    in[u] = unit0 + u * (kThreads / 16) + group < (uint64_t)a.units && c < a.K;
    at[u] = (uint64_t)down * (uint32_t)a.K + c;
    // Lanes past the end or past the row's last column: eight columns that there are, which count as zeros.
    const uint8_t *p = in[u] ? src + ((uint64_t)down * (uint32_t)a.ldx + c) * ES : static_cast<const uint8_t *>(a.x);
    load8<DT, FAR>(p, x[u]);
    if (GATED) load8<DT, FAR>(p + a.K * ES, up[u]);
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    if (GATED) {
      // The short form where it holds for every gate of the wave (four instructions to see; NaN counts as too large).
      if (__ballot(max8(x[u]) > kGateBits) == 0) {
#pragma unroll
        for (int i = 0; i < 8; i++) x[u][i] = silu_mul(x[u][i], up[u][i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++) x[u][i] = silu_mul_any(x[u][i], up[u][i]);
      }
    }
    const Scale k = block_scale(max16(in[u] ? max8(x[u]) : 0));
    if (in[u]) {
      store8(dst + at[u], x[u], k);
      if (l == 0) a.scales[unit0 + u * (kThreads / 16) + group] = k.s;
    }
  }
}

struct WeightArgs {
  const void *w;
  int64_t ldw, expert_stride, N, K;
  uint32_t count;        // of all blocks
  int32_t row_blocks, blocks;
  uint8_t *codes;
  float *scales;
};

// A workgroup has one block: 16 rows at a time, sixteen lanes to a row, the
// whole block in registers between the maximum and the codes. Bound by HBM:
// 17408 x 5120 of BF16, 267 MB, take 46 us (5.8 TB/s).
template <int DT, bool FAR>
__global__ __launch_bounds__(kThreads) void weight_kernel(WeightArgs a) {
  constexpr int ES = DT == NVFP4_F32 ? 4 : 2;
  __shared__ uint32_t tops[kThreads / 64];
  const int64_t b = row_workgroup();
  if (b >= a.count) return;
  const int64_t cb = b % a.blocks, rb = b / a.blocks % a.row_blocks, e = b / a.blocks / a.row_blocks;
  const int64_t c = cb * 128 + (threadIdx.x & 15) * 8;
  const int64_t r0 = rb * 128 + (threadIdx.x >> 4);
  // Past the last row or column: that row, the last eight columns. They are the block's own and leave its maximum alone.
  const uint8_t *src = static_cast<const uint8_t *>(a.w) + (e * a.expert_stride + min(c, a.K - 8)) * ES;
  float x[8][8];
#pragma unroll
  for (int i = 0; i < 8; i++) load8<DT, FAR>(src + min(r0 + 16 * i, a.N - 1) * a.ldw * ES, x[i]);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) m = max(m, max8(x[i]));
#pragma unroll
  for (int d = 1; d < 64; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; i++) m = max(m, tops[i]);
  const Scale k = block_scale(m);
  uint8_t *dst = a.codes + e * a.N * a.K + c;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int64_t r = r0 + 16 * i;
    if (r < a.N && c < a.K) store8(dst + r * a.K, x[i], k);
  }
  if (threadIdx.x == 0) a.scales[b] = k.s;
}

static int64_t element_bytes(int dtype) { return dtype == NVFP4_F32 ? 4 : 2; }
static bool dtype_ok(int dtype) { return dtype == NVFP4_F32 || dtype == NVFP4_BF16 || dtype == NVFP4_F16; }

}  // namespace fp8
}  // namespace nvfp4

using namespace nvfp4;
using namespace nvfp4::fp8;

#define FP8_DISPATCH(dtype, far, CALL)                                                                \
  switch (dtype) {                                                                                    \
    case NVFP4_F32: if (far) { CALL(NVFP4_F32, true); } else { CALL(NVFP4_F32, false); } break;        \
    case NVFP4_BF16: if (far) { CALL(NVFP4_BF16, true); } else { CALL(NVFP4_BF16, false); } break;     \
    default: if (far) { CALL(NVFP4_F16, true); } else { CALL(NVFP4_F16, false); } break;               \
  }

extern "C" nvfp4_status nvfp4_fp8_quantize(const void *x, int dtype, int64_t rows, int64_t K, int64_t ldx, int gated,
                                           uint8_t *codes, float *scales, void *stream) {
  if (!dtype_ok(dtype)) return NVFP4_ERR_DTYPE;
  if (gated != 0 && gated != 1) return NVFP4_ERR_VALUE;
  if (rows < 0 || K <= 0 || K % 16 != 0 || K > (1 << 28) || ldx < (gated ? 2 * K : K) || ldx > (int64_t(1) << 30) ||
      rows > (int64_t(1) << 31))
    return NVFP4_ERR_SHAPE;
  if (rows == 0) return NVFP4_OK;
  if (!x || !codes || !scales) return NVFP4_ERR_NULL;
  if (!aligned(x, element_bytes(dtype)) || !aligned(codes, 16) || !aligned(scales, 4)) return NVFP4_ERR_ALIGN;
  RowsArgs a;
  a.x = x;
  a.ldx = ldx;
  a.blocks = (int32_t)((K + 127) / 128);
  a.units = rows * a.blocks;
  a.inverse = ~0ull / (uint64_t)a.blocks + 1;
  a.small = (1u << 16) / (uint32_t)a.blocks + 1;
  a.K = K;
  a.codes = codes;
  a.scales = scales;
  const int64_t grid = (a.units + kThreads / 16 * kRowBlocks - 1) / (kThreads / 16 * kRowBlocks);
  if (grid > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  nvfp4_status st = device_info(nullptr);
  if (st != NVFP4_OK) return st;
  const bool far = rows * K * (gated ? 2 : 1) * element_bytes(dtype) > kNear;
#define ROWS(DT, FAR)                                                                                                     \
  if (gated)                                                                                                              \
    hipLaunchKernelGGL((rows_kernel<DT, true, FAR>), row_grid(grid), dim3(kThreads), 0, (hipStream_t)stream, a);          \
  else                                                                                                                    \
    hipLaunchKernelGGL((rows_kernel<DT, false, FAR>), row_grid(grid), dim3(kThreads), 0, (hipStream_t)stream, a)
  FP8_DISPATCH(dtype, far, ROWS)
#undef ROWS
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

extern "C" nvfp4_status nvfp4_fp8_quantize_weight(const void *w, int dtype, int64_t experts, int64_t N, int64_t K,
                                                  int64_t ldw, int64_t expert_stride, uint8_t *codes, float *scales,
                                                  void *stream) {
  if (!dtype_ok(dtype)) return NVFP4_ERR_DTYPE;
  if (experts < 0 || N <= 0 || K <= 0 || K % 16 != 0 || K > (1 << 28) || N > (1 << 28) || ldw < K ||
      ldw > (int64_t(1) << 30) || experts > (1 << 20) || expert_stride < 0 || expert_stride > (int64_t(1) << 40))
    return NVFP4_ERR_SHAPE;
  if (experts == 0) return NVFP4_OK;
  if (!w || !codes || !scales) return NVFP4_ERR_NULL;
  if (!aligned(w, element_bytes(dtype)) || !aligned(codes, 16) || !aligned(scales, 4)) return NVFP4_ERR_ALIGN;
  WeightArgs a;
  a.w = w;
  a.ldw = ldw;
  a.expert_stride = expert_stride;
  a.N = N;
  a.K = K;
  a.row_blocks = (int32_t)((N + 127) / 128);
  a.blocks = (int32_t)((K + 127) / 128);
  a.codes = codes;
  a.scales = scales;
  const int64_t per = (int64_t)a.row_blocks * a.blocks;
  if (per > 0x7FFFFFFF / experts) return NVFP4_ERR_SHAPE;
  a.count = (uint32_t)(per * experts);
  nvfp4_status st = device_info(nullptr);
  if (st != NVFP4_OK) return st;
  const bool far = experts * N * K * element_bytes(dtype) > kNear;
#define WEIGHT(DT, FAR) \
  hipLaunchKernelGGL((weight_kernel<DT, FAR>), row_grid(a.count), dim3(kThreads), 0, (hipStream_t)stream, a)
  FP8_DISPATCH(dtype, far, WEIGHT)
#undef WEIGHT
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}
