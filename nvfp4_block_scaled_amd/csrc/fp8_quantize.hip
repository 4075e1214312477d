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

namespace nvfp4 {
namespace fp8 {

constexpr float kTop = 448.0f;
constexpr uint32_t kLeastBits = 0x0D800000u;      // 2^-100
constexpr uint32_t kInfBits = 0x7F800000u;

// Eight consecutive elements of a row as FP32 values (exact); rows start at any element.
template <int DT>
__device__ __forceinline__ void load8(const void *p, float (&x)[8]) {
  if constexpr (DT == NVFP4_F32) {
    typedef f32x4_t U __attribute__((aligned(4)));
    const f32x4_t a = static_cast<const U *>(p)[0], b = static_cast<const U *>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  } else {
    typedef u32x4_t U __attribute__((aligned(2)));
    const u32x4_t w = *static_cast<const U *>(p);
    unpack8<DT == NVFP4_F16>(w, x);
  }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t max8(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) m = max(m, abs_bits(x[i]));
  return m;
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

// RN(x / s) for |x| <= 448 s (or a NaN where s is one), a zero's sign kept.
__device__ __forceinline__ float quotient(float x, Scale k) {
  const float q = x * k.r;
  return __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-q, k.s, x), k.r, q), x);
}

__device__ __forceinline__ u32x2_t codes8(const float (&x)[8], Scale k) {
  u32x2_t c;
#pragma unroll
  for (int h = 0; h < 2; h++) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(x[4 * h], k), quotient(x[4 * h + 1], k), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(x[4 * h + 2], k), quotient(x[4 * h + 3], k), w, true);
    c[h] = (uint32_t)w;
  }
  return c;
}

// silu(g) u = g / (1 + e^-g) u. With t = RN(-g log2 e) and what that rounding
// lost, l (exact but for 2^-48 of t), e^-g = 2^t (1 + l ln 2). g is taken within
// -87 .. 104 there: above, 1 + e^-g is 1; below, the result is under 2^-119
// either way, less than the smallest scale. The reciprocal is good to an ulp and
// the quotient, after one step with its remainder, to hardly more than half of
// one. The arithmetic counts here: with the library's expf and a division by a
// corrected reciprocal, 2048 rows of 2 x 17408 BF16 columns took 47.6 us, now 41.
__device__ __forceinline__ float silu_mul(float g, float u) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  const float c = __builtin_amdgcn_fmed3f(g, -87.0f, 104.0f);
  const float t = c * -kLog2e;
  const float l = __builtin_fmaf(c, -kLog2eRest, __builtin_fmaf(c, -kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  const float d = 1.0f + __builtin_fmaf(e, l * kLn2, e);
  const float r = __builtin_amdgcn_rcpf(d);
  const float q = g * r;
  return __builtin_fmaf(__builtin_fmaf(-q, d, g), r, q) * u;
}

struct RowsArgs {
  const void *x;
  int64_t ldx;
  int64_t units;         // rows * blocks of a row
  int64_t K;
  int32_t blocks;        // of a row
  uint8_t *codes;
  float *scales;
};

// Sixteen lanes have a block of 128 columns, eight columns each; a thread has U
// blocks, whose loads are all in flight before the first is used (two: one, three
// and four are 1 to 8 % slower). K % 16 == 0: a lane's eight columns are all
// there or none is. Bound by HBM: 2048 rows of 34816 BF16 columns, 214 MB read
// and written, take 40 us (5.3 TB/s); gated into 17408, 178 MB, 41 us (4.3).
constexpr int kThreads = 256;

template <int DT, bool GATED, int U>
__global__ __launch_bounds__(kThreads) void rows_kernel(RowsArgs a) {
  constexpr int ES = DT == NVFP4_F32 ? 4 : 2;
  const int l = threadIdx.x & 15;
  const int64_t first = (int64_t)blockIdx.x * (kThreads / 16 * U) + (threadIdx.x >> 4);
  float x[U][8], up[GATED ? U : 1][8];
  int64_t at[U];         // of the lane's columns in codes, or -1
#pragma unroll
  for (int u = 0; u < U; u++) {
    const int64_t unit = first + u * (kThreads / 16);
    const int64_t row = unit / a.blocks;
    const int64_t c = (unit - row * a.blocks) * 128 + l * 8;
    const bool in = unit < a.units && c < a.K;
    at[u] = in ? row * a.K + c : -1;
#pragma unroll
    for (int i = 0; i < 8; i++) x[u][i] = 0.0f;
    if (GATED) {
#pragma unroll
      for (int i = 0; i < 8; i++) up[u][i] = 0.0f;
    }
    if (in) {
      const uint8_t *p = static_cast<const uint8_t *>(a.x) + (row * a.ldx + c) * ES;
      load8<DT>(p, x[u]);
      if (GATED) load8<DT>(p + a.K * ES, up[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    if (GATED) {
#pragma unroll
      for (int i = 0; i < 8; i++) x[u][i] = silu_mul(x[u][i], up[u][i]);
    }
    uint32_t m = max8(x[u]);
#pragma unroll
    for (int d = 1; d < 16; d *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    const Scale k = block_scale(m);
    if (at[u] >= 0) {
      *reinterpret_cast<u32x2_t *>(a.codes + at[u]) = codes8(x[u], k);
      if (l == 0) a.scales[first + u * (kThreads / 16)] = k.s;
    }
  }
}

struct WeightArgs {
  const void *w;
  int64_t ldw, expert_stride, N, K;
  int32_t row_blocks, blocks;
  uint8_t *codes;
  float *scales;
};

// A workgroup has one block: 16 rows at a time, sixteen lanes to a row, the
// whole block in registers between the maximum and the codes. Bound by HBM:
// 17408 x 5120 of BF16, 267 MB, take 55 us (4.8 TB/s).
template <int DT>
__global__ __launch_bounds__(kThreads) void weight_kernel(WeightArgs a) {
  constexpr int ES = DT == NVFP4_F32 ? 4 : 2;
  __shared__ uint32_t tops[kThreads / 64];
  const int64_t b = blockIdx.x;
  const int64_t cb = b % a.blocks, rb = b / a.blocks % a.row_blocks, e = b / a.blocks / a.row_blocks;
  const int64_t c = cb * 128 + (threadIdx.x & 15) * 8;
  const int64_t r0 = rb * 128 + (threadIdx.x >> 4);
  const uint8_t *src = static_cast<const uint8_t *>(a.w) + (e * a.expert_stride + c) * ES;
  float x[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int64_t r = r0 + 16 * i;
#pragma unroll
    for (int j = 0; j < 8; j++) x[i][j] = 0.0f;
    if (r < a.N && c < a.K) load8<DT>(src + r * a.ldw * ES, x[i]);
  }
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
    if (r < a.N && c < a.K) *reinterpret_cast<u32x2_t *>(dst + r * a.K) = codes8(x[i], k);
  }
  if (threadIdx.x == 0) a.scales[b] = k.s;
}

static bool dtype_ok(int dtype) { return dtype == NVFP4_F32 || dtype == NVFP4_BF16 || dtype == NVFP4_F16; }

}  // namespace fp8
}  // namespace nvfp4

using namespace nvfp4;
using namespace nvfp4::fp8;

extern "C" nvfp4_status nvfp4_fp8_quantize(const void *x, int dtype, int64_t rows, int64_t K, int64_t ldx, int gated,
                                           uint8_t *codes, float *scales, void *stream) {
  if (!dtype_ok(dtype)) return NVFP4_ERR_DTYPE;
  if (gated != 0 && gated != 1) return NVFP4_ERR_VALUE;
  if (rows < 0 || K <= 0 || K % 16 != 0 || K > (1 << 28) || ldx < (gated ? 2 * K : K) || ldx > (int64_t(1) << 30) ||
      rows > (int64_t(1) << 31))
    return NVFP4_ERR_SHAPE;
  if (rows == 0) return NVFP4_OK;
  if (!x || !codes || !scales) return NVFP4_ERR_NULL;
  if (!aligned(x, dtype == NVFP4_F32 ? 4 : 2) || !aligned(codes, 16) || !aligned(scales, 4)) return NVFP4_ERR_ALIGN;
  RowsArgs a;
  a.x = x;
  a.ldx = ldx;
  a.blocks = (int32_t)((K + 127) / 128);
  a.units = rows * a.blocks;
  a.K = K;
  a.codes = codes;
  a.scales = scales;
  constexpr int U = 2;
  const int64_t grid = (a.units + kThreads / 16 * U - 1) / (kThreads / 16 * U);
  if (grid > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  nvfp4_status st = device_info(nullptr);
  if (st != NVFP4_OK) return st;
#define ROWS(DT)                                                                                                       \
  if (gated)                                                                                                           \
    hipLaunchKernelGGL((rows_kernel<DT, true, U>), dim3((unsigned)grid), dim3(kThreads), 0, (hipStream_t)stream, a);   \
  else                                                                                                                 \
    hipLaunchKernelGGL((rows_kernel<DT, false, U>), dim3((unsigned)grid), dim3(kThreads), 0, (hipStream_t)stream, a)
  switch (dtype) {
    case NVFP4_F32: ROWS(NVFP4_F32); break;
    case NVFP4_BF16: ROWS(NVFP4_BF16); break;
    default: ROWS(NVFP4_F16); break;
  }
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
  if (!aligned(w, dtype == NVFP4_F32 ? 4 : 2) || !aligned(codes, 16) || !aligned(scales, 4)) return NVFP4_ERR_ALIGN;
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
  const unsigned grid = (unsigned)(per * experts);
  nvfp4_status st = device_info(nullptr);
  if (st != NVFP4_OK) return st;
  switch (dtype) {
    case NVFP4_F32:
      hipLaunchKernelGGL((weight_kernel<NVFP4_F32>), dim3(grid), dim3(kThreads), 0, (hipStream_t)stream, a);
      break;
    case NVFP4_BF16:
      hipLaunchKernelGGL((weight_kernel<NVFP4_BF16>), dim3(grid), dim3(kThreads), 0, (hipStream_t)stream, a);
      break;
    default:
      hipLaunchKernelGGL((weight_kernel<NVFP4_F16>), dim3(grid), dim3(kThreads), 0, (hipStream_t)stream, a);
  }
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}
