// FP8 products with block scales for gfx950:
//
//   out[m][n] = sum_b  sa[m][b] sw[n / 128][b]  sum_{k in block b} A[m][k] W[n][k]
//
// A [M][K] and W [N][K] in E4M3, blocks of 128 along K, FP32 sums; dense, and
// with the rows of A sorted by expert against a stack of weights.
//
// The inner sum is one v_mfma_f32_16x16x128_f8f6f4, whose 128 products are a
// whole block: it starts from zero and its result meets the block's two scales
// in one FP32 multiply-add a value (the matrix core adds eight products at a
// time with 2^-13 of the largest of them as the last bit kept, and those sums
// in FP32; measured on gaussian rows that is 1.3e-5 of the result, a hundredth
// of the rounding to BF16, which is why no FP32 output is offered). W is the
// instruction's first operand, so a lane holds four consecutive columns of one
// row: one scale a lane, and 8-byte stores.
//
// Order of K inside a block: lane group g = lane / 16 has the 16-byte units g
// and g + 4 of its row. A and W use the same order, so each product is met once.
#include "common.hpp"

namespace nvfp4 {
namespace fp8 {

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;

struct GemmArgs {
  const uint8_t *a, *w;
  const float *a_scales, *w_scales;
  void *out;
  int64_t M, N, K, ldo;
  int32_t blocks;             // of K
  int32_t tiles_m, tiles_n;   // dense: the tile grid; grouped: tiles_n alone
  // grouped
  const int32_t *offsets;     // [experts + 1]
  const int32_t *rows;        // row of A of each sorted row, or null: its own number
  int64_t a_rows;             // rows of A
  int32_t experts;
};

// 64 lanes x 16 bytes (or 4) from global memory to consecutive bytes of LDS,
// with no register between. The compiler does not see the load: every reader
// waits for vmcnt and passes a barrier first.
__device__ __forceinline__ void to_lds16(const uint8_t *src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "m0", "memory");
}
__device__ __forceinline__ void to_lds4(const float *src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(src) : "m0", "memory");
}

__device__ __forceinline__ v8i_t join(u32x4_t a, u32x4_t b) {
  return v8i_t{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// The tile of a workgroup: rows [m0, m1) of out against columns from n0 of the
// weight `expert`. Workgroups of one XCD (ids congruent mod 8) get consecutive
// tiles, so that what they share meets in that XCD's L2.
struct Tile {
  int64_t m0, m1, n0;
  int32_t expert;
};

__device__ __forceinline__ bool xcd_order(uint32_t b, uint32_t total, uint32_t *t) {
  const uint32_t per = (total + 7) / 8;
  *t = (b & 7) * per + (b >> 3);
  return (b >> 3) < per && *t < total;
}

constexpr int kBand = 8;     // tile rows of a band: within one, tiles go down the columns

__device__ __forceinline__ void band_order(uint32_t t, uint32_t rows, uint32_t cols, uint32_t *m, uint32_t *n) {
  const uint32_t band = t / (kBand * cols), first = band * kBand, w = t - band * kBand * cols;
  const uint32_t tall = min((uint32_t)kBand, rows - first);
  *m = first + w % tall;
  *n = w / tall;
}

// The workgroup's tile among those of the experts that have rows, expert by
// expert; every workgroup counts them all (the host does not know the rows).
// Offsets are taken within 0 .. M, an end below its start as no rows.
template <int BM, int THREADS>
__device__ __forceinline__ bool grouped_tile(const GemmArgs &a, uint32_t b, int32_t *sh, Tile *tile) {
  // sh[0 .. WAVES): sums of waves; then the answer
  constexpr int WAVES = THREADS / 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t total = 0;
  if (tid == 0) sh[WAVES] = -1;
  for (int pass = 0; pass < 2; pass++) {
    uint32_t t = 0;
    if (pass == 1 && !xcd_order(b, total * (uint32_t)a.tiles_n, &t)) return false;
    uint32_t base = 0;                           // m tiles of the experts before this round's
    for (int e0 = 0; e0 < a.experts; e0 += THREADS) {
      const int e = e0 + tid;
      int32_t lo = 0, hi = 0;
      if (e < a.experts) {
        lo = max(0, min(a.offsets[e], (int32_t)a.M));
        hi = max(lo, min(a.offsets[e + 1], (int32_t)a.M));
      }
      const uint32_t mine = ((uint32_t)(hi - lo) + BM - 1) / BM;
      uint32_t run = mine;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const uint32_t v = __shfl_up(run, d);
        if (lane >= d) run += v;
      }
      __syncthreads();
      if (lane == 63) sh[wave] = (int32_t)run;
      __syncthreads();
      uint32_t before = base + run - mine;
#pragma unroll
      for (int w = 0; w < WAVES; w++) {
        if (w < wave) before += (uint32_t)sh[w];
        base += (uint32_t)sh[w];
      }
      if (pass == 1 && mine > 0 && t >= before * (uint32_t)a.tiles_n && t < (before + mine) * (uint32_t)a.tiles_n) {
        const uint32_t w = t - before * (uint32_t)a.tiles_n;       // within the expert: down the rows, then across
        sh[WAVES] = e;
        sh[WAVES + 1] = lo + (int32_t)(w % mine) * BM;
        sh[WAVES + 2] = hi;
        sh[WAVES + 3] = (int32_t)(w / mine);
      }
    }
    if (pass == 0) total = base;
  }
  __syncthreads();
  tile->expert = __builtin_amdgcn_readfirstlane(sh[WAVES]);
  if (tile->expert < 0) return false;
  tile->m0 = __builtin_amdgcn_readfirstlane(sh[WAVES + 1]);
  tile->m1 = __builtin_amdgcn_readfirstlane(sh[WAVES + 2]);
  tile->n0 = __builtin_amdgcn_readfirstlane(sh[WAVES + 3]);
  return true;
}

// WM x WN waves share a BM x BN tile; a wave has TM x TN tiles of 16 x 16.
// STAGES blocks of K lie in LDS at a time, rows of 128 bytes whose 16-byte
// units are exchanged by the low bits of the row (unit u of row r lies at
// u ^ (r & 7)), so that neither the loads nor the fragments' reads meet in a bank.
template <int BM, int BN, int WM, int WN, int STAGES, bool GROUPED, bool F16>
__global__ __launch_bounds__(64 * WM * WN, 2) void tile_kernel(GemmArgs p) {
  constexpr int WAVES = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
  constexpr int SCALES = BM < 64 ? 256 : BM * 4;            // a wave's load brings 64 scales
  constexpr int STAGE = (BM + BN) * 128 + SCALES;
  constexpr int LOADS_A = BM / 8 / WAVES, LOADS_W = BN / 8 / WAVES;
  static_assert(LOADS_A * 8 * WAVES == BM && LOADS_W * 8 * WAVES == BN, "whole loads for every wave");
  static_assert(BN / WN <= 128 && 128 % (BN / WN) == 0, "a wave's columns have one scale");
  static_assert(STAGES == 2, "the wait at the top of a step is for everything in flight");
  __shared__ __attribute__((aligned(128))) uint8_t lds[STAGES * STAGE];
  __shared__ int32_t found[WAVES + 4];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4, wm = wave / WN, wn = wave % WN;

  Tile t;
  if constexpr (GROUPED) {
    if (!grouped_tile<BM, 64 * WAVES>(p, blockIdx.x, found, &t)) return;
    t.n0 *= BN;
  } else {
    uint32_t id, tm, tn;
    if (!xcd_order(blockIdx.x, (uint32_t)p.tiles_m * (uint32_t)p.tiles_n, &id)) return;
    band_order(id, p.tiles_m, p.tiles_n, &tm, &tn);
    t.m0 = (int64_t)tm * BM;
    t.m1 = p.M;
    t.n0 = (int64_t)tn * BN;
    t.expert = 0;
  }

  // The row of A that row m of out multiplies (clamped into A: what it gives is not stored).
  auto a_row = [&](int64_t m) -> int64_t {
    m = min(m, t.m1 - 1);
    if (GROUPED && p.rows) {
      const int64_t at = p.rows[m];
      return at < 0 || at >= p.a_rows ? 0 : at;
    }
    return m;
  };

  // Addresses of this lane's part of each load: row lane / 8 of eight, unit
  // (lane % 8) ^ (row % 8) of its 128 bytes.
  const int unit = ((lane & 7) ^ ((lane >> 3) & 7)) * 16;
  const uint8_t *src[LOADS_A + LOADS_W];
#pragma unroll
  for (int i = 0; i < LOADS_A; i++) src[i] = p.a + a_row(t.m0 + (wave * LOADS_A + i) * 8 + (lane >> 3)) * p.K + unit;
  const int64_t w_base = (int64_t)t.expert * p.N;
#pragma unroll
  for (int i = 0; i < LOADS_W; i++) {
    const int64_t n = min(t.n0 + (wave * LOADS_W + i) * 8 + (lane >> 3), p.N - 1);
    src[LOADS_A + i] = p.w + (w_base + n) * p.K + unit;
  }
  constexpr int SCALE_CHUNKS = (BM + 63) / 64;
  const int chunk = wave % SCALE_CHUNKS;                    // waves beyond the chunks bring the same values again
  const float *src_s = p.a_scales + a_row(t.m0 + min(chunk * 64 + lane, BM - 1)) * p.blocks;
  const float *sw = p.w_scales + ((int64_t)t.expert * ((p.N + 127) / 128) + min(t.n0 + wn * (BN / WN), p.N - 1) / 128) * p.blocks;

  const uint32_t base = (uint32_t)(uintptr_t)(lds_u8 *)lds;
  auto load = [&](int kb) {
    const uint32_t at = base + (kb & 1) * STAGE;
    const int64_t k0 = (int64_t)kb * 128;
    // units past the end of a row: its last unit in their place (masked below)
    const int over = (int)max((int64_t)0, k0 + unit + 16 - p.K);
    const int64_t off = k0 - over;
#pragma unroll
    for (int i = 0; i < LOADS_A; i++) to_lds16(src[i] + off, at + (wave * LOADS_A + i) * 1024);
#pragma unroll
    for (int i = 0; i < LOADS_W; i++) to_lds16(src[LOADS_A + i] + off, at + BM * 128 + (wave * LOADS_W + i) * 1024);
    to_lds4(src_s + kb, at + (BM + BN) * 128 + chunk * 256);
  };

  f32x4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; i++)
#pragma unroll
    for (int j = 0; j < TN; j++) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  const uint32_t lo = (uint32_t)(r * 128 + ((g ^ (r & 7)) * 16)), hi = lo ^ 64;
  auto step = [&](int kb, float s, int valid) {           // valid: 16-byte units of the block
    const uint8_t *st = lds + (kb & 1) * STAGE;
    const uint8_t *fa = st + wm * (BM / WM) * 128, *fw = st + BM * 128 + wn * (BN / WN) * 128;
    const float *sc = reinterpret_cast<const float *>(st + (BM + BN) * 128) + wm * (BM / WM);
    auto fragment = [&](const uint8_t *at) {
      u32x4_t x = *reinterpret_cast<const u32x4_t *>(at + lo), y = *reinterpret_cast<const u32x4_t *>(at + hi);
      if (valid < 8) {
        const u32x4_t z = {0u, 0u, 0u, 0u};
        if (g >= valid) x = z;
        if (g + 4 >= valid) y = z;
      }
      return join(x, y);
    };
    v8i_t w[TN];
#pragma unroll
    for (int j = 0; j < TN; j++) w[j] = fragment(fw + j * 2048);
#pragma unroll
    for (int i = 0; i < TM; i++) {
      const v8i_t x = fragment(fa + i * 2048);
      const float sa = sc[i * 16 + r] * s;
#pragma unroll
      for (int j = 0; j < TN; j++) {
        const f32x4_t d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[j], x, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0,
                                                                          0, 0, 0);
#pragma unroll
        for (int q = 0; q < 4; q++) acc[i][j][q] = __builtin_fmaf(sa, d[q], acc[i][j][q]);
      }
    }
  };

  load(0);
  for (int kb = 0; kb < p.blocks; kb++) {
    const float s = sw[kb];
    // everything in flight has arrived and, past the barrier, everybody's; nobody reads the other stage any more
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (kb + 1 < p.blocks) load(kb + 1);
    const int64_t left = p.K - (int64_t)kb * 128;
    if (left >= 128) step(kb, s, 8);
    else step(kb, s, (int)(left / 16));
  }

  // Lane (r, g) has columns 4 g .. 4 g + 3 of row r of each 16 x 16 tile.
  typedef u32x2_t U __attribute__((aligned(2)));
#pragma unroll
  for (int i = 0; i < TM; i++) {
    const int64_t m = t.m0 + wm * (BM / WM) + i * 16 + r;
    bool stored = m < t.m1;
    if (GROUPED && p.rows && stored) stored = p.rows[m] >= 0 && p.rows[m] < p.a_rows;
    if (!stored) continue;
    uint16_t *row = static_cast<uint16_t *>(p.out) + m * p.ldo;
#pragma unroll
    for (int j = 0; j < TN; j++) {
      const int64_t n = t.n0 + wn * (BN / WN) + j * 16 + g * 4;
      uint16_t h[4];
#pragma unroll
      for (int q = 0; q < 4; q++) {
        if (F16) {
          const _Float16 v = (_Float16)acc[i][j][q];
          __builtin_memcpy(&h[q], &v, 2);
        } else {
          h[q] = f32_to_bf16_rne(acc[i][j][q]);
        }
      }
      if (n + 4 <= p.N) {
        const u32x2_t v = {(uint32_t)h[0] | ((uint32_t)h[1] << 16), (uint32_t)h[2] | ((uint32_t)h[3] << 16)};
        *reinterpret_cast<U *>(row + n) = v;
      } else {
#pragma unroll
        for (int q = 0; q < 4; q++)
          if (n + q < p.N) row[n + q] = h[q];
      }
    }
  }
}

template <int BM, int BN, int WM, int WN, bool GROUPED>
static nvfp4_status launch_tiles(GemmArgs a, int dtype, hipStream_t s) {
  a.tiles_n = (int32_t)((a.N + BN - 1) / BN);
  int64_t tm;
  if (GROUPED) {
    tm = a.M / BM + a.experts;            // every expert may end in a partial tile
    if (tm > a.M) tm = a.M;
  } else {
    tm = (a.M + BM - 1) / BM;
  }
  a.tiles_m = (int32_t)tm;
  const int64_t tiles = tm * a.tiles_n;
  if (tiles > 0x7FFFFF00) return NVFP4_ERR_SHAPE;
  const unsigned grid = (unsigned)((tiles + 7) / 8 * 8);
  if (dtype == NVFP4_F16)
    hipLaunchKernelGGL((tile_kernel<BM, BN, WM, WN, 2, GROUPED, true>), dim3(grid), dim3(64 * WM * WN), 0, s, a);
  else
    hipLaunchKernelGGL((tile_kernel<BM, BN, WM, WN, 2, GROUPED, false>), dim3(grid), dim3(64 * WM * WN), 0, s, a);
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

template <bool GROUPED>
static nvfp4_status launch(const GemmArgs &a, int dtype, hipStream_t s) {
  return launch_tiles<128, 128, 2, 2, GROUPED>(a, dtype, s);
}

static bool gemm_sizes_ok(int64_t M, int64_t N, int64_t K, int64_t ldo) {
  return M >= 0 && M <= 0x7FFFFFFF && N > 0 && N <= (1 << 28) && K > 0 && K % 16 == 0 && K <= (1 << 28) && ldo >= N &&
         ldo <= (int64_t(1) << 30);
}

}  // namespace fp8
}  // namespace nvfp4

using namespace nvfp4;
using namespace nvfp4::fp8;

extern "C" size_t nvfp4_fp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) { return 0; }

extern "C" nvfp4_status nvfp4_fp8_gemm(const uint8_t *a, const float *a_scales, const uint8_t *w, const float *w_scales,
                                       int64_t M, int64_t N, int64_t K, void *out, int dtype, int64_t ldo, void *ws,
                                       size_t ws_bytes, void *stream) {
  if (dtype != NVFP4_BF16 && dtype != NVFP4_F16) return NVFP4_ERR_DTYPE;
  if (!gemm_sizes_ok(M, N, K, ldo)) return NVFP4_ERR_SHAPE;
  if (M == 0) return NVFP4_OK;
  if (!a || !a_scales || !w || !w_scales || !out) return NVFP4_ERR_NULL;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scales, 4) || !aligned(w_scales, 4) || !aligned(out, 2))
    return NVFP4_ERR_ALIGN;
  const size_t need = nvfp4_fp8_gemm_workspace_bytes(M, N, K);
  if (need > 0) {
    if (!ws || ws_bytes < need) return NVFP4_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return NVFP4_ERR_ALIGN;
  }
  nvfp4_status st = device_info(nullptr);
  if (st != NVFP4_OK) return st;
  GemmArgs p{};
  p.a = a;
  p.w = w;
  p.a_scales = a_scales;
  p.w_scales = w_scales;
  p.out = out;
  p.M = M;
  p.N = N;
  p.K = K;
  p.ldo = ldo;
  p.blocks = (int32_t)((K + 127) / 128);
  p.a_rows = M;
  return launch<false>(p, dtype, (hipStream_t)stream);
}

extern "C" nvfp4_status nvfp4_fp8_gemm_grouped(const uint8_t *a, const float *a_scales, int64_t a_rows,
                                               const int32_t *rows, const uint8_t *w, const float *w_scales,
                                               int32_t experts, const int32_t *offsets, int64_t M, int64_t N, int64_t K,
                                               void *out, int dtype, int64_t ldo, void *stream) {
  if (dtype != NVFP4_BF16 && dtype != NVFP4_F16) return NVFP4_ERR_DTYPE;
  if (!gemm_sizes_ok(M, N, K, ldo) || a_rows < 0 || a_rows > 0x7FFFFFFF || experts < 1 || experts > 1024 ||
      (!rows && a_rows < M))
    return NVFP4_ERR_SHAPE;
  if (M == 0 || a_rows == 0) return NVFP4_OK;
  if (!a || !a_scales || !w || !w_scales || !offsets || !out) return NVFP4_ERR_NULL;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scales, 4) || !aligned(w_scales, 4) || !aligned(out, 2) ||
      !aligned(offsets, 4) || !aligned(rows, 4))
    return NVFP4_ERR_ALIGN;
  nvfp4_status st = device_info(nullptr);
  if (st != NVFP4_OK) return st;
  GemmArgs p{};
  p.a = a;
  p.w = w;
  p.a_scales = a_scales;
  p.w_scales = w_scales;
  p.out = out;
  p.M = M;
  p.N = N;
  p.K = K;
  p.ldo = ldo;
  p.blocks = (int32_t)((K + 127) / 128);
  p.offsets = offsets;
  p.rows = rows;
  p.a_rows = a_rows;
  p.experts = experts;
  return launch<true>(p, dtype, (hipStream_t)stream);
}
