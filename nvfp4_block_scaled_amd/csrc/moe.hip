// Tokens to experts and back: the sort of (token, choice) pairs by expert, the
// gather of the tokens' rows in that order, the weighted sum of the rows back
// to their tokens, and the gradients of both.
//
// A pair (t, j) with expert id e in 0 .. experts - 1 gets the place
//   offsets[e] + (pairs of expert e before it in t * top + j)
// in the sorted order. Everything that follows needs the places only:
//   gather    rows[place(t, j)] = x[t]                  gradient: x' [t] = sum_j rows'[place(t, j)]
//   combine   out[t] = sum_j w[t, j] y[place(t, j)]     gradient: y' [place(t, j)] = w[t, j] out'[t],
//                                                                 w' [t, j] = out'[t] . y[place(t, j)]
// All four read and write token by token, so a token's row is read once however
// many experts it goes to, sums run over j in order in FP32 (no atomics: the
// same bits on every call), and only rows that a place names are written.
#include "common.hpp"
#include "kv_common.hpp"
#include "launch.hpp"

namespace nvfp4 {
namespace moe {

// ------------------------------------------------------------------- sort
//
// A chunk of consecutive pairs belongs to one workgroup. A wave ranks 64 pairs
// at a time among each other with one ballot per bit of the expert id: the
// lanes that agree in every bit are the pair's fellows, those before it in the
// wave its rank, and the first of them adds their number to the wave's own
// histogram, whose old value counts the fellows of the wave's earlier rounds.
// Sums over waves, chunks and experts do the rest. Ranks come from positions
// alone, so the order is stable and the same on every call.
constexpr int kMaxExperts = 1024;
constexpr int kRounds = 4;               // pairs of a thread in one pass over the histograms

struct SortArgs {
  const void *ids;
  uint32_t pairs, top;
  int32_t experts;
  int32_t bits;             // of the largest id
  int32_t *offsets, *tokens, *places;
  int32_t *counts;          // [chunks][experts] (more than one chunk)
  uint32_t chunk;           // pairs of a chunk
  int32_t chunks;
};

// The expert of pair i, or -1.
template <bool WIDE>
__device__ __forceinline__ int load_id(const SortArgs &a, uint32_t i, uint32_t end) {
  if (i >= end) return -1;
  if (WIDE) {
    const int64_t v = static_cast<const int64_t *>(a.ids)[i];
    return v >= 0 && v < a.experts ? (int)v : -1;
  }
  const int32_t v = static_cast<const int32_t *>(a.ids)[i];
  return v >= 0 && v < a.experts ? v : -1;
}

template <bool WIDE>
__global__ __launch_bounds__(256) void count_kernel(SortArgs a) {
  extern __shared__ int32_t hist[];
  for (int e = threadIdx.x; e < a.experts; e += 256) hist[e] = 0;
  __syncthreads();
  const uint32_t from = blockIdx.x * a.chunk, end = min(a.pairs, from + a.chunk);
  for (uint32_t i = from + threadIdx.x; i < end; i += 256) {
    const int e = load_id<WIDE>(a, i, end);
    if (e >= 0) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += 256) a.counts[(int64_t)blockIdx.x * a.experts + e] = hist[e];
}

// LDS: per-wave histograms [waves][experts], then next[experts]: where the
// chunk's next pair of each expert goes.
template <int THREADS, bool WIDE, bool ONE>
__global__ __launch_bounds__(THREADS) void place_kernel(SortArgs a) {
  constexpr int WAVES = THREADS / 64;
  extern __shared__ int32_t lds[];
  __shared__ int32_t sums[WAVES];
  int32_t *next = lds + WAVES * a.experts;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const uint32_t from = ONE ? 0 : blockIdx.x * a.chunk, end = ONE ? a.pairs : min(a.pairs, from + a.chunk);
  const int E = a.experts;

  // Exclusive sum over the experts of total[e], with `before[e]` added: next[]
  // and, for the first workgroup, the offsets. Thread t has experts PER t .. PER t + PER - 1.
  constexpr int PER = kMaxExperts / THREADS;
  auto scan = [&](const int (&total)[PER], const int (&before)[PER]) {
    int sum = 0;
#pragma unroll
    for (int q = 0; q < PER; q++) sum += total[q];
    int run = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(run, d);
      if (lane >= d) run += v;
    }
    if (lane == 63) sums[wave] = run;
    __syncthreads();
    int base = run - sum;
    for (int w = 0; w < wave; w++) base += sums[w];
#pragma unroll
    for (int q = 0; q < PER; q++) {
      const int e = PER * tid + q;
      if (e < E) {
        next[e] = base + before[q];
        if (ONE || blockIdx.x == 0) a.offsets[e] = base;
        if (e == E - 1) {
          if (ONE || blockIdx.x == 0) a.offsets[E] = base + total[q];
          next[E] = base + total[q];
        }
      }
      base += total[q];
    }
    __syncthreads();
  };

  if (!ONE) {   // what the chunks before this one, and all of them, have of each expert
    int total[PER], before[PER];
#pragma unroll
    for (int q = 0; q < PER; q++) total[q] = before[q] = 0;
    if (PER * tid < E) {
#pragma unroll 16
      for (int c = 0; c < a.chunks; c++) {
#pragma unroll
        for (int q = 0; q < PER; q++) {
          const int e = PER * tid + q;
          const int n = e < E ? a.counts[(int64_t)c * E + e] : 0;
          total[q] += n;
          if (c < (int)blockIdx.x) before[q] += n;
        }
      }
    }
    scan(total, before);
  }

  // One pass takes THREADS * kRounds pairs: each wave kRounds runs of 64.
  int e[kRounds], rank[kRounds];
  auto pass = [&](uint32_t at) {
    for (int i = tid; i < WAVES * E; i += THREADS) lds[i] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; r++) e[r] = load_id<WIDE>(a, at + (wave * kRounds + r) * 64 + lane, end);
#pragma unroll
    for (int r = 0; r < kRounds; r++) {
      uint64_t same = __ballot(e[r] >= 0);
      for (int b = 0; b < a.bits; b++) {
        const uint64_t set = __ballot((e[r] >> b) & 1);
        same &= (e[r] >> b) & 1 ? set : ~set;
      }
      const int ahead = __popcll(same & ((1ull << lane) - 1));
      int old = 0;
      if (e[r] >= 0) {
        old = lds[wave * E + e[r]];                       // every fellow reads it before the first adds
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (ahead == 0) lds[wave * E + e[r]] = old + __popcll(same);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      rank[r] = old + ahead;
    }
    __syncthreads();
  };
  auto place = [&](uint32_t at) {      // histograms to first places, then every pair to its own
    for (int x = tid; x < E; x += THREADS) {
      int run = next[x];
      for (int w = 0; w < WAVES; w++) {
        const int n = lds[w * E + x];
        lds[w * E + x] = run;
        run += n;
      }
      next[x] = run;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; r++) {
      const uint32_t i = at + (wave * kRounds + r) * 64 + lane;
      if (i < end) {
        int p = -1;
        if (e[r] >= 0) {
          p = lds[wave * E + e[r]] + rank[r];
          a.tokens[p] = (int32_t)(i / a.top);
        }
        a.places[i] = p;
      }
    }
    __syncthreads();
  };

  if (ONE) {      // at most one pass
    pass(0);
    int total[PER], none[PER];
#pragma unroll
    for (int q = 0; q < PER; q++) {
      const int x = PER * tid + q;
      total[q] = none[q] = 0;
      for (int w = 0; w < WAVES; w++) total[q] += x < E ? lds[w * E + x] : 0;
    }
    scan(total, none);
    place(0);
  } else {
    for (uint32_t at = from; at < end; at += THREADS * kRounds) {
      pass(at);
      place(at);
    }
  }
  const uint32_t used = (uint32_t)next[E];    // pairs that some expert has; no token behind them
  for (uint32_t i = from + tid; i < end; i += THREADS)
    if (i >= used) a.tokens[i] = -1;
}

// ------------------------------------------------------- rows of 16 bytes a lane
//
// A row is read and written in units of 16 bytes whatever its alignment (the
// hardware takes 16-byte accesses at any element boundary; rows that start at
// one cost it a second cache line per unit at most); the last, partial unit of
// an odd width goes element by element.
//
// FAR: the sorted rows together are more than the memory-side cache of 256 MB
// holds, so the next reader finds none of them there, and they pass it by
// (nontemporal): 32768 rows of 5120 BF16, gather 74.8 -> 65.5 us (5.8 TB/s),
// sum 73.9 -> 65.0, combine's gradient 146.8 -> 134.4 (5.3). Below, a gather and
// the sum of the same rows lose by it: 12000 rows 47.7 -> 49.2, 4096 17.0 -> 17.7.
constexpr int64_t kNear = int64_t(256) << 20;

template <int DT>
struct Elem;
template <>
struct Elem<NVFP4_F32> {
  typedef float T;
  typedef u32x4_t U __attribute__((aligned(4)));
  static constexpr int N = 4;
};
template <>
struct Elem<NVFP4_BF16> {
  typedef uint16_t T;
  typedef u32x4_t U __attribute__((aligned(2)));
  static constexpr int N = 8;
};
template <>
struct Elem<NVFP4_F16> {
  typedef uint16_t T;
  typedef u32x4_t U __attribute__((aligned(2)));
  static constexpr int N = 8;
};

template <int DT, bool FAR = false>
__device__ __forceinline__ u32x4_t load_unit(const void *row, int64_t at, int left) {
  typedef typename Elem<DT>::T T;
  typedef typename Elem<DT>::U U;
  const T *p = static_cast<const T *>(row) + at;
  if (left >= Elem<DT>::N) return FAR ? __builtin_nontemporal_load(reinterpret_cast<const U *>(p)) : *reinterpret_cast<const U *>(p);
  u32x4_t v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < Elem<DT>::N; i++) {
    if (i < left) {
      if (DT == NVFP4_F32) {
        uint32_t b;
        __builtin_memcpy(&b, p + i, 4);
        v[i & 3] = b;
      } else {
        uint16_t b;
        __builtin_memcpy(&b, p + i, 2);
        v[i / 2] |= (uint32_t)b << (16 * (i & 1));
      }
    }
  }
  return v;
}

template <int DT, bool FAR = false>
__device__ __forceinline__ void store_unit(void *row, int64_t at, int left, u32x4_t v) {
  typedef typename Elem<DT>::T T;
  typedef typename Elem<DT>::U U;
  T *p = static_cast<T *>(row) + at;
  if (left >= Elem<DT>::N) {
    if (FAR) __builtin_nontemporal_store(v, reinterpret_cast<U *>(p));
    else *reinterpret_cast<U *>(p) = v;
    return;
  }
#pragma unroll
  for (int i = 0; i < Elem<DT>::N; i++) {
    if (i < left) {
      if (DT == NVFP4_F32) {
        const uint32_t b = v[i & 3];
        __builtin_memcpy(p + i, &b, 4);
      } else {
        const uint16_t b = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
        __builtin_memcpy(p + i, &b, 2);
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ void unpack(const u32x4_t v, float (&x)[Elem<DT>::N]) {
  if constexpr (DT == NVFP4_F32) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint32_t u = v[i];
      x[i] = __uint_as_float(u);
    }
  } else {
    unpack8<DT == NVFP4_F16>(v, x);
  }
}

template <int DT>
__device__ __forceinline__ u32x4_t pack(const float (&x)[Elem<DT>::N]) {
  if constexpr (DT == NVFP4_F32) {
    u32x4_t v;
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = __float_as_uint(x[i]);
    return v;
  } else {
    return pack8<DT == NVFP4_F16>(x);
  }
}

struct RowArgs {
  const void *x;            // tokens' rows
  const void *y;            // sorted rows
  void *out;
  int64_t ldx, ldy, ldo;    // row strides in elements
  int64_t tokens, pairs;
  int32_t top, width;
  const int32_t *places;
  const float *weights;
  float *grad_weights;
  int32_t parts;            // workgroups of a token (gather, combine)
};

constexpr int kRowThreads = 256;
constexpr int kAhead = 8;        // choices of a token whose rows are in flight at once

// The sorted rows of a token's choices j0 .. j0 + kAhead - 1, -1 for none, and their weights: one load brings them, a lane
// for each, and every lane of the wave has them from there (all lanes come here together). A load for each choice is a
// latency for each: 33 tokens by 8, gather 3.7 -> 3.0 us, combine 3.5 -> 3.1, its gradients 9.4 -> 9.0.
__device__ __forceinline__ void choices(const RowArgs &a, int64_t t, int j0, int64_t (&p)[kAhead]) {
  const int lane = threadIdx.x & 63;
  const int32_t mine = lane < kAhead && j0 + lane < a.top ? a.places[t * a.top + j0 + lane] : -1;
#pragma unroll
  for (int j = 0; j < kAhead; j++) {
    const int32_t at = __builtin_amdgcn_readlane(mine, j);
    p[j] = at >= 0 && at < a.pairs ? at : -1;
  }
}
__device__ __forceinline__ void choices(const RowArgs &a, int64_t t, int j0, int64_t (&p)[kAhead], float (&w)[kAhead]) {
  const int lane = threadIdx.x & 63;
  const float mine = lane < kAhead && j0 + lane < a.top ? a.weights[t * a.top + j0 + lane] : 0.0f;
  choices(a, t, j0, p);
#pragma unroll
  for (int j = 0; j < kAhead; j++) w[j] = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(mine), j));
}

// One unit of a token, kept in registers while it goes to each of its places.
template <int DT, bool FAR>
__global__ __launch_bounds__(kRowThreads) void gather_kernel(RowArgs a) {
  constexpr int N = Elem<DT>::N, ES = sizeof(typename Elem<DT>::T);
  const uint32_t at = row_workgroup();
  const int64_t t = at / a.parts;
  if (t >= a.tokens) return;
  const int c = ((int)(at % a.parts) * kRowThreads + (int)threadIdx.x) * N, left = a.width - c;
  u32x4_t v;
  if (left > 0) v = load_unit<DT>(static_cast<const uint8_t *>(a.x) + t * a.ldx * ES, c, left);
  for (int j0 = 0; j0 < a.top; j0 += kAhead) {
    int64_t p[kAhead];
    choices(a, t, j0, p);
#pragma unroll
    for (int j = 0; j < kAhead; j++)
      if (p[j] >= 0 && left > 0) store_unit<DT, FAR>(static_cast<uint8_t *>(a.out) + p[j] * a.ldo * ES, c, left, v);
  }
}

// Up to eight rows of a token are in flight at once; they are added in order.
template <int DT, bool WEIGHTS, bool FAR>
__global__ __launch_bounds__(kRowThreads) void combine_kernel(RowArgs a) {
  constexpr int N = Elem<DT>::N, ES = sizeof(typename Elem<DT>::T);
  const uint32_t at = row_workgroup();
  const int64_t t = at / a.parts;
  if (t >= a.tokens) return;
  const int c = ((int)(at % a.parts) * kRowThreads + (int)threadIdx.x) * N, left = a.width - c;
  float sum[N];
#pragma unroll
  for (int i = 0; i < N; i++) sum[i] = 0.0f;
  for (int j0 = 0; j0 < a.top; j0 += kAhead) {
    u32x4_t v[kAhead];
    int64_t p[kAhead];
    float w[kAhead];
    if constexpr (WEIGHTS) choices(a, t, j0, p, w);
    else choices(a, t, j0, p);
#pragma unroll
    for (int j = 0; j < kAhead; j++)
      if (p[j] >= 0 && left > 0) v[j] = load_unit<DT, FAR>(static_cast<const uint8_t *>(a.y) + p[j] * a.ldy * ES, c, left);
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      if (p[j] < 0) continue;
      float x[N];
      unpack<DT>(v[j], x);
#pragma unroll
      for (int i = 0; i < N; i++) sum[i] = WEIGHTS ? __builtin_fmaf(w[j], x[i], sum[i]) : sum[i] + x[i];
    }
  }
  if (left > 0) store_unit<DT>(static_cast<uint8_t *>(a.out) + t * a.ldo * ES, c, left, pack<DT>(sum));
}

// A workgroup has one token: its gradient is read once for up to eight choices,
// whose rows of y meet it and whose rows of y's gradient leave on the way.
template <int DT, bool FAR>
__global__ __launch_bounds__(kRowThreads) void combine_backward_kernel(RowArgs a) {
  constexpr int N = Elem<DT>::N, ES = sizeof(typename Elem<DT>::T), WAVES = kRowThreads / 64;
  __shared__ float part[WAVES][kAhead];
  const int64_t t = row_workgroup();
  if (t >= a.tokens) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const uint8_t *grad = static_cast<const uint8_t *>(a.x) + t * a.ldx * ES;
  for (int j0 = 0; j0 < a.top; j0 += kAhead) {
    float dot[kAhead], w[kAhead];
    int64_t p[kAhead];
    choices(a, t, j0, p, w);
#pragma unroll
    for (int j = 0; j < kAhead; j++) dot[j] = 0.0f;
    for (int c = tid * N; c < a.width; c += kRowThreads * N) {
      const int left = a.width - c;
      const u32x4_t gv = load_unit<DT>(grad, c, left);
      u32x4_t v[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; j++)
        if (p[j] >= 0) v[j] = load_unit<DT, FAR>(static_cast<const uint8_t *>(a.y) + p[j] * a.ldy * ES, c, left);
      float g[N];
      unpack<DT>(gv, g);
#pragma unroll
      for (int j = 0; j < kAhead; j++) {
        if (p[j] < 0) continue;
        float x[N], o[N];
        unpack<DT>(v[j], x);
#pragma unroll
        for (int i = 0; i < N; i++) {
          dot[j] = __builtin_fmaf(g[i], x[i], dot[j]);
          o[i] = w[j] * g[i];
        }
        store_unit<DT, FAR>(static_cast<uint8_t *>(a.out) + p[j] * a.ldo * ES, c, left, pack<DT>(o));
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
#pragma unroll
      for (int d = 32; d >= 1; d /= 2) dot[j] += __shfl_xor(dot[j], d);
      if (lane == 0) part[wave][j] = dot[j];
    }
    __syncthreads();
    if (tid < kAhead && j0 + tid < a.top) {
      float sum = 0.0f;
      for (int i = 0; i < WAVES; i++) sum += part[i][tid];
      a.grad_weights[t * a.top + j0 + tid] = sum;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- host side

// How the pairs are cut: one workgroup of 1024 threads for what it places in one
// pass (and as many experts as its 16 histograms fit in 64 KB of LDS with), else
// chunks of whole passes of 256 threads, at most kMaxChunks of them. One
// workgroup against two launches, 64 experts: 136 pairs 4.9 and 5.9 us, 4096
// 6.9 and 7.3; with a second pass, 8192, 16.6 and 9.3. 262144 pairs take 31 us:
// latency, of the counts' read and of four passes a chunk.
constexpr int64_t kOnePairs = 1024 * kRounds, kOneExperts = 896;
constexpr int kMaxChunks = 256;

static bool one_workgroup(int64_t pairs, int64_t experts) { return pairs <= kOnePairs && experts <= kOneExperts; }

static void cut(int64_t pairs, int64_t *chunk, int64_t *chunks) {
  const int64_t pass = 256 * kRounds;
  int64_t c = (pairs + kMaxChunks - 1) / kMaxChunks;
  c = c < 1 ? pass : (c + pass - 1) / pass * pass;
  *chunk = c;
  *chunks = pairs < 1 ? 1 : (pairs + c - 1) / c;
}

static bool sort_sizes_ok(int64_t tokens, int64_t top, int64_t experts) {
  return tokens >= 0 && top >= 1 && experts >= 1 && experts <= kMaxExperts && top <= 0x7FFFFFFF &&
         tokens <= 0x7FFFFFFF / top;
}

static size_t sort_workspace(int64_t pairs, int64_t experts) {
  if (one_workgroup(pairs, experts)) return 0;
  int64_t chunk, chunks;
  cut(pairs, &chunk, &chunks);
  return (size_t)(chunks * experts * 4 + 15) / 16 * 16;
}

template <bool WIDE>
static nvfp4_status launch_sort(SortArgs a, hipStream_t s) {
  if (one_workgroup(a.pairs, a.experts)) {
    hipLaunchKernelGGL((place_kernel<1024, WIDE, true>), dim3(1), dim3(1024), (size_t)(17 * a.experts + 1) * 4, s, a);
    NVFP4_LAUNCH_CHECK();
    return NVFP4_OK;
  }
  hipLaunchKernelGGL((count_kernel<WIDE>), dim3(a.chunks), dim3(256), (size_t)a.experts * 4, s, a);
  NVFP4_LAUNCH_CHECK();
  hipLaunchKernelGGL((place_kernel<256, WIDE, false>), dim3(a.chunks), dim3(256), (size_t)(4 * a.experts + a.experts + 1) * 4,
                     s, a);
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

static bool dtype_ok(int dtype) { return dtype == NVFP4_F32 || dtype == NVFP4_BF16 || dtype == NVFP4_F16; }
static size_t dtype_bytes(int dtype) { return dtype == NVFP4_F32 ? 4 : 2; }

// Sizes that the row kernels take: 32-bit columns, pairs that fit a place, byte offsets in 63 bits.
static bool rows_ok(int64_t tokens, int64_t top, int64_t width) {
  return tokens >= 0 && top >= 1 && top <= 0x7FFFFFFF && tokens <= 0x7FFFFFFF / top && width >= 1 && width <= (1 << 28);
}
static bool far_rows(const RowArgs &a, size_t es) { return a.pairs * (int64_t)a.width * (int64_t)es > kNear; }
static bool ld_ok(int64_t ld, int64_t width) { return ld >= width && ld <= (int64_t(1) << 30); }

}  // namespace moe
}  // namespace nvfp4

using namespace nvfp4;
using namespace nvfp4::moe;

#define MOE_DISPATCH(dtype, far, CALL)                                                    \
  switch (dtype) {                                                                        \
    case NVFP4_F32: if (far) CALL(NVFP4_F32, true); else CALL(NVFP4_F32, false); break;    \
    case NVFP4_BF16: if (far) CALL(NVFP4_BF16, true); else CALL(NVFP4_BF16, false); break; \
    default: if (far) CALL(NVFP4_F16, true); else CALL(NVFP4_F16, false); break;           \
  }

extern "C" size_t nvfp4_moe_sort_workspace_bytes(int64_t tokens, int64_t top, int32_t experts) {
  if (!sort_sizes_ok(tokens, top, experts)) return 0;
  return sort_workspace(tokens * top, experts);
}

extern "C" nvfp4_status nvfp4_moe_sort(const void *ids, int id_bytes, int64_t tokens, int64_t top, int32_t experts,
                                       int32_t *offsets, int32_t *sorted_tokens, int32_t *places, void *ws,
                                       size_t ws_bytes, void *stream) {
  if (id_bytes != 4 && id_bytes != 8) return NVFP4_ERR_DTYPE;
  if (!sort_sizes_ok(tokens, top, experts)) return NVFP4_ERR_SHAPE;
  const int64_t pairs = tokens * top;
  if (!offsets || (pairs > 0 && (!ids || !sorted_tokens || !places))) return NVFP4_ERR_NULL;
  if (!aligned(offsets, 4) || !aligned(ids, id_bytes) || !aligned(sorted_tokens, 4) || !aligned(places, 4))
    return NVFP4_ERR_ALIGN;
  const size_t need = sort_workspace(pairs, experts);
  if (need > 0) {
    if (!ws || ws_bytes < need) return NVFP4_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return NVFP4_ERR_ALIGN;
  }
  nvfp4_status st = device_info(nullptr);
  if (st != NVFP4_OK) return st;
  SortArgs a;
  a.ids = ids;
  a.pairs = (uint32_t)pairs;
  a.top = (uint32_t)top;
  a.experts = experts;
  a.bits = experts > 1 ? 32 - __builtin_clz((unsigned)(experts - 1)) : 0;
  a.offsets = offsets;
  a.tokens = sorted_tokens;
  a.places = places;
  a.counts = static_cast<int32_t *>(ws);
  int64_t chunk = 0, chunks = 0;
  if (need > 0) cut(pairs, &chunk, &chunks);
  a.chunk = (uint32_t)chunk;
  a.chunks = (int32_t)chunks;
  return id_bytes == 8 ? launch_sort<true>(a, (hipStream_t)stream) : launch_sort<false>(a, (hipStream_t)stream);
}

extern "C" nvfp4_status nvfp4_moe_gather(const void *x, int dtype, int64_t ldx, const int32_t *places, int64_t tokens,
                                         int64_t top, int64_t width, void *out, int64_t ldo, void *stream) {
  if (!dtype_ok(dtype)) return NVFP4_ERR_DTYPE;
  if (!rows_ok(tokens, top, width) || !ld_ok(ldx, width) || !ld_ok(ldo, width)) return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  if (!x || !places || !out) return NVFP4_ERR_NULL;
  const size_t es = dtype_bytes(dtype);
  if (!aligned(x, es) || !aligned(out, es) || !aligned(places, 4)) return NVFP4_ERR_ALIGN;
  const int64_t per = kRowThreads * (int64_t)(16 / es);
  const int64_t parts = (width + per - 1) / per;
  if (parts * tokens > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  nvfp4_status st = device_info(nullptr);
  if (st != NVFP4_OK) return st;
  RowArgs a{};
  a.x = x;
  a.out = out;
  a.ldx = ldx;
  a.ldo = ldo;
  a.tokens = tokens;
  a.pairs = tokens * top;
  a.top = (int32_t)top;
  a.width = (int32_t)width;
  a.places = places;
  a.parts = (int32_t)parts;
#define GATHER(DT, FAR) \
  hipLaunchKernelGGL((gather_kernel<DT, FAR>), row_grid(parts * tokens), dim3(kRowThreads), 0, (hipStream_t)stream, a)
  MOE_DISPATCH(dtype, far_rows(a, es), GATHER)
#undef GATHER
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

extern "C" nvfp4_status nvfp4_moe_combine(const void *y, int dtype, int64_t ldy, const int32_t *places,
                                          const float *weights, int64_t tokens, int64_t top, int64_t width, void *out,
                                          int64_t ldo, void *stream) {
  if (!dtype_ok(dtype)) return NVFP4_ERR_DTYPE;
  if (!rows_ok(tokens, top, width) || !ld_ok(ldy, width) || !ld_ok(ldo, width)) return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  if (!y || !places || !out) return NVFP4_ERR_NULL;
  const size_t es = dtype_bytes(dtype);
  if (!aligned(y, es) || !aligned(out, es) || !aligned(places, 4) || !aligned(weights, 4)) return NVFP4_ERR_ALIGN;
  const int64_t per = kRowThreads * (int64_t)(16 / es);
  const int64_t parts = (width + per - 1) / per;
  if (parts * tokens > 0x7FFFFFFF) return NVFP4_ERR_SHAPE;
  nvfp4_status st = device_info(nullptr);
  if (st != NVFP4_OK) return st;
  RowArgs a{};
  a.y = y;
  a.out = out;
  a.ldy = ldy;
  a.ldo = ldo;
  a.tokens = tokens;
  a.pairs = tokens * top;
  a.top = (int32_t)top;
  a.width = (int32_t)width;
  a.places = places;
  a.weights = weights;
  a.parts = (int32_t)parts;
  const dim3 grid = row_grid(parts * tokens);
#define COMBINE(DT, FAR) \
  hipLaunchKernelGGL((combine_kernel<DT, true, FAR>), grid, dim3(kRowThreads), 0, (hipStream_t)stream, a)
#define SUM(DT, FAR) \
  hipLaunchKernelGGL((combine_kernel<DT, false, FAR>), grid, dim3(kRowThreads), 0, (hipStream_t)stream, a)
  if (weights) {
    MOE_DISPATCH(dtype, far_rows(a, es), COMBINE)
  } else {
    MOE_DISPATCH(dtype, far_rows(a, es), SUM)
  }
#undef SUM
#undef COMBINE
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

extern "C" nvfp4_status nvfp4_moe_combine_backward(const void *grad, int64_t ldg, const void *y, int64_t ldy, int dtype,
                                                   const int32_t *places, const float *weights, int64_t tokens,
                                                   int64_t top, int64_t width, void *grad_y, int64_t ldo,
                                                   float *grad_weights, void *stream) {
  if (!dtype_ok(dtype)) return NVFP4_ERR_DTYPE;
  if (!rows_ok(tokens, top, width) || !ld_ok(ldg, width) || !ld_ok(ldy, width) || !ld_ok(ldo, width))
    return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  if (!grad || !y || !places || !weights || !grad_y || !grad_weights) return NVFP4_ERR_NULL;
  const size_t es = dtype_bytes(dtype);
  if (!aligned(grad, es) || !aligned(y, es) || !aligned(grad_y, es) || !aligned(places, 4) || !aligned(weights, 4) ||
      !aligned(grad_weights, 4))
    return NVFP4_ERR_ALIGN;
  nvfp4_status st = device_info(nullptr);
  if (st != NVFP4_OK) return st;
  RowArgs a{};
  a.x = grad;
  a.y = y;
  a.out = grad_y;
  a.ldx = ldg;
  a.ldy = ldy;
  a.ldo = ldo;
  a.tokens = tokens;
  a.pairs = tokens * top;
  a.top = (int32_t)top;
  a.width = (int32_t)width;
  a.places = places;
  a.weights = weights;
  a.grad_weights = grad_weights;
#define BACK(DT, FAR) \
  hipLaunchKernelGGL((combine_backward_kernel<DT, FAR>), row_grid(tokens), dim3(kRowThreads), 0, (hipStream_t)stream, a)
  MOE_DISPATCH(dtype, far_rows(a, es), BACK)
#undef BACK
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}
