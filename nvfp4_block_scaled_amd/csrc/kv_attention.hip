// Attention over the NVFP4 key/value cache.
//
// For a query row q and the keys it sees,  t_j = scale * q . k_j,
//   out = sum_j e^(t_j - m) v_j / sum_j e^(t_j - m),   lse = m + ln sum_j e^(t_j - m),
// in one pass over the keys with a running reference m: when a tile's largest
// t passes m by more than a factor 2^8, the sums so far are scaled down to the
// new m. Any m gives the same quotient, so m need not be the exact maximum.
//
// The rows of one KV head are its queries times the query heads of its group:
// row r is query r / G, head r % G of the group. Both products run on the
// matrix cores transposed, S^T = K Q^T and O^T = V^T P^T, in FP16 steps of
// 16 x 16 x 32 (few rows) or 32 x 32 x 16 (many): a column of S^T and of O^T is one query row and stays in the same
// lanes, so the softmax's scaling of O needs no exchange between lanes, and
// P^T leaves the exponential already in the layout that the second product
// takes (the order of its 32 keys is free as long as V's matches).
//
// Precision. code * scale has 6 significant bits and lies in [2^-10, 2688], so
// it is exact in FP16. Each query row is scaled by a power of two to a largest
// magnitude in [2^8, 2^9), which keeps every bit of a BF16 or FP16 element down
// to 2^-22 of the row's largest. P is rounded to FP16 (11 bits, where BF16
// would keep 8) after a factor 2^6, which puts its range at 2^14 .. 2^-24 under
// the lazy reference; the row sums use the unrounded FP32 values. All
// accumulators, maxima and sums are FP32; global scales enter in FP32 at the
// end (k_g into the softmax's factor, v_g into the last division).
#include <math.h>

#include <type_traits>

#include "kv_common.hpp"

namespace nvfp4 {

static constexpr int kWaves = 4;
static constexpr int kTile = 32;                       // keys of one wave's step
static constexpr int kStep = kWaves * kTile;           // keys of one workgroup's step
static constexpr int kBlockRows = 128;                 // query rows of a workgroup of block_kernel
static constexpr float kHeadroom = 8.0f;               // log2 of how far a value may pass the reference
static constexpr float kOffset = 6.0f;                 // log2 of the factor on P

struct AttnArgs {
  KvView kv;
  const uint16_t *q;
  uint16_t *out;
  float *lse;
  int64_t q_t, q_h, o_t, o_h;
  int64_t total_q, table_stride;
  const int32_t *table, *lens, *q_start;
  const uint8_t *mask;
  int64_t mask_stride;
  float scale;
  int32_t batch, max_pages, max_q, window;
  int32_t group;             // query heads of a KV head
  int32_t causal;
  int32_t target;            // workgroups per KV head to split into
  int32_t slots;             // pieces that the workspace holds for each KV head
  float *part_o;             // workspace: partial sums [slot][row][D], then [slot][row][2] of (m, l)
  float *part_ml;
  int32_t *join_count;       // workspace: how many row tiles are joined, and of each its first row,
  int32_t *joins_at;         // its rows, its first slot and its pieces
  int32_t joins;             // row tiles that the workspace has room for
};

// Asks for the arguments' cache lines before the first is needed: left alone, each line is a wait of
// its own, some of them at the kernel's end (256 queries on 32000 keys: 220.3 -> 218.6 us, 64 for each of 16
// sequences of 8000: 279.9 -> 276.5; drafted trees and single tokens: no difference).
template <typename T>
__device__ __forceinline__ void touch(T v) {
  asm volatile("" ::"s"(v));
}
__device__ __forceinline__ void touch_args(const AttnArgs &A) {
  touch(A.q); touch(A.out); touch(A.lse); touch(A.q_t); touch(A.o_t); touch(A.table); touch(A.lens); touch(A.mask);
  touch(A.scale); touch(A.part_o); touch(A.joins_at); touch(A.kv.pages);
}

// ------------------------------------------------------------------- plan

// One sequence's share of the work: rows in tiles of RT, keys in steps of kStep.
struct Seq {
  int len, queries, first;   // keys, queries, row of the first one
  int row_tiles, steps;      // steps: the most that one row tile has
};

template <int RT>
__device__ __forceinline__ Seq sequence(const AttnArgs &A, int b) {
  Seq s;
  const int64_t most = (int64_t)A.max_pages << A.kv.log_p;
  const int n = A.lens[b];
  s.len = n < 0 ? 0 : (int64_t)n > most ? (int)most : n;
  int q0 = b, q1 = b + 1;
  if (A.q_start) {
    const int total = (int)A.total_q;
    q0 = min(max(A.q_start[b], 0), total);
    q1 = min(max(A.q_start[b + 1], q0), total);
  }
  s.first = q0;
  s.queries = q1 - q0;                        // of which the first max_q are computed
  const int used = min(s.queries, A.max_q);
  s.row_tiles = (used * A.group + RT - 1) / RT;
  int span = s.len;
  if (A.window) span = min(span, A.window + (RT + A.group - 2) / A.group + kStep / 2);
  s.steps = (span + kStep - 1) / kStep;
  return s;
}

// Inclusive prefix sum over a wave: shifts inside rows of 16 lanes, then the rows' last lanes.
// The sums over sequences are unsigned: those of a q_start that does not ascend may pass 32 bits, and
// then wrap to numbers that the bounds checks behind them (has_work, join_kernel) turn away.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false);   // row_shr:1
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false);
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);   // row_bcast:15 into rows 1 and 3
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);   // row_bcast:31 into rows 2 and 3
  return v;
}

__device__ __forceinline__ uint32_t lane_of(uint32_t v, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); }
__device__ __forceinline__ uint32_t last_lane(uint32_t v) { return lane_of(v, 63); }

// A workgroup's unit: one row tile of one sequence, and one of the `splits` pieces of its keys.
struct Unit {
  int b, tile, split, splits;
  uint32_t slot;
  Seq s;
};

// False only with sequences that overlap in q_start.
__device__ __forceinline__ bool has_work(const AttnArgs &A, const Unit &u) {
  return (uint32_t)u.tile < (uint32_t)u.s.row_tiles && (u.splits == 1 || u.slot < (uint32_t)A.slots);
}

// A lane's sequences from `base` on, PER each: one where a wave's lanes are enough, else four, whose
// lengths are then on their way together (one token for each of 1024 sequences of 128 keys: 51.8 us, 54.5
// with one to a lane, 58.0 with eight; 128 sequences of up to 4096: 24.6, 24.1, 26.3).
template <int RT, int PER>
__device__ __forceinline__ void shares(const AttnArgs &A, int base, Seq (&s)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; i++) {
    const int b = base + (threadIdx.x & 63) * PER + i;
    s[i] = sequence<RT>(A, min(b, A.batch - 1));
    if (b >= A.batch) s[i].row_tiles = s[i].steps = 0;
  }
}

// How many steps a piece has: the call's steps over the workgroups to fill. For block_kernel, whose
// workgroups are long, half a workgroup for each row tile is set aside, so that all pieces run in one
// round, short last ones included (256 queries on 32000 keys: 299 us without, 219 with half, 223 with a
// whole one; 32 drafted trees with heads of 256: 85, 69, 94; 64 queries on each of 16 sequences of 8000
// keys: 277, 277, 309). rows_kernel's are short and many (64 ragged sequences: 22.2 us without, 23.6 with;
// three queries for each of 16: 23.5, 24.8; 128 ragged sequences: 24.6, 22.8). With more row tiles than
// workgroups only those several times longer than the average are split. s0: the first 64 PER sequences.
template <int RT, int PER>
__device__ __forceinline__ uint32_t piece_steps(const AttnArgs &A, Seq (&s0)[PER]) {
  shares<RT, PER>(A, 0, s0);
  if (A.joins == 0) return 1u << 30;
  uint32_t total = 0, tiles = 0;
#pragma unroll
  for (int i = 0; i < PER; i++) total += s0[i].row_tiles * s0[i].steps, tiles += s0[i].row_tiles;
  for (int base = 64 * PER; base < A.batch; base += 64 * PER) {
    Seq s[PER];
    shares<RT, PER>(A, base, s);
#pragma unroll
    for (int i = 0; i < PER; i++) total += s[i].row_tiles * s[i].steps, tiles += s[i].row_tiles;
  }
  total = last_lane(wave_scan(total)), tiles = last_lane(wave_scan(tiles));
  const uint32_t room = RT < kBlockRows ? A.target : max(A.target - (int)(tiles / 2), max(1, A.target / 4));
  return max(1u, (total + room - 1) / room);
}

__device__ __forceinline__ uint32_t pieces_of(const Seq &s, uint32_t chunk) { return max(1u, (s.steps + chunk - 1) / chunk); }

// Finds unit `unit`; false past the last. Every wave does it for itself with no exchange through memory:
// a prefix sum over the sequences' pieces says whose piece it is. REVERSE: of a sequence under the
// causal mask, the last row tile comes first: it sees the most keys.
template <int RT, bool REVERSE, int PER>
__device__ __forceinline__ bool find_unit_per(const AttnArgs &A, int unit, Unit *out) {
  Seq s[PER];
  const uint32_t chunk = piece_steps<RT, PER>(A, s), u = unit;
  uint32_t units = 0, slots = 0;
  for (int base = 0; base < A.batch; base += 64 * PER) {
    if (base > 0) shares<RT, PER>(A, base, s);
    uint32_t n[PER], mine = 0, part = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) {
      n[i] = pieces_of(s[i], chunk);
      mine += s[i].row_tiles * n[i];
      part += n[i] > 1 ? s[i].row_tiles * n[i] : 0;
    }
    const uint32_t to = units + wave_scan(mine), slot_to = slots + wave_scan(part);
    const uint64_t hit = __ballot(u < to);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      uint32_t first = lane_of(to - mine, at), slot = lane_of(slot_to - part, at);
      bool found = false;
#pragma unroll
      for (int i = 0; i < PER; i++) {
        const uint32_t tiles = lane_of(s[i].row_tiles, at), splits = lane_of(n[i], at);
        const uint32_t count = tiles * splits;
        if (!found && (i == PER - 1 || u < first + count)) {
          found = true;
          const uint32_t tile = (u - first) / splits;
          out->b = base + at * PER + i;
          out->splits = splits;
          out->tile = tile;
          out->split = (u - first) - tile * splits;
          out->slot = slot + u - first;
          out->s.len = lane_of(s[i].len, at);
          out->s.queries = lane_of(s[i].queries, at);
          out->s.first = lane_of(s[i].first, at);
          out->s.row_tiles = tiles;
          out->s.steps = lane_of(s[i].steps, at);
          if (REVERSE && A.causal) out->tile = tiles - 1 - tile;
        }
        first += count;
        if (splits > 1) slot += count;
      }
      return true;
    }
    units = last_lane(to), slots = last_lane(slot_to);
  }
  return false;
}

template <int RT, bool REVERSE>
__device__ __forceinline__ bool find_unit(const AttnArgs &A, int u, Unit *out) {
  return A.batch <= 64 ? find_unit_per<RT, REVERSE, 1>(A, u, out) : find_unit_per<RT, REVERSE, 4>(A, u, out);
}

// Pieces of nearly the same length: piece i of `steps` begins at step begin(i).
struct Pieces {
  int each, longer;          // the first `longer` have one step more
  __device__ __forceinline__ Pieces(int steps, int n) : each(steps / n), longer(steps - steps / n * n) {}
  __device__ __forceinline__ int begin(int i) const { return each * i + min(i, longer); }
};

// Query and head of a row tile's rows: row k of the tile is query first + (rest + k) / G. Below 2^21 a
// product with 1 / G tells (x + 1/2) / G from the next integer; a division is five times as long.
struct RowQuery {
  int first, rest, G;
  float per;
  __device__ __forceinline__ RowQuery(int row0, int g)
      : first(row0 / g), rest(row0 - row0 / g * g), G(g), per(__builtin_amdgcn_rcpf((float)g)) {}
  __device__ __forceinline__ int offset(int k) const { return (int)(((float)(rest + k) + 0.5f) * per); }
  __device__ __forceinline__ int query(int k) const { return first + offset(k); }
  __device__ __forceinline__ int head(int k) const { return rest + k - offset(k) * G; }
};

// What join_kernel has to know of the split row tiles: a workgroup of its own (the grid's first)
// lists them, the same prefix sums again.
template <int RT, bool REVERSE>
__device__ __forceinline__ void list_joins(const AttnArgs &A) {
  if (threadIdx.x >= 64) return;
  const int lane = threadIdx.x;
  Seq one[1];
  const uint32_t chunk = piece_steps<RT, 1>(A, one);
  uint32_t slots = 0, joins = 0;
  for (int base = 0; base < A.batch; base += 64) {
    if (base > 0) shares<RT, 1>(A, base, one);
    const Seq &s = one[0];
    const uint32_t n = pieces_of(s, chunk);
    const int tiles = n > 1 ? s.row_tiles : 0;
    const uint32_t slot_to = slots + wave_scan(tiles * n), join_to = joins + wave_scan(tiles);
    const int rows = min(s.queries, A.max_q) * A.group;
    for (int i = 0; i < tiles; i++) {
      const uint32_t j = join_to - tiles + i;
      const int tile = REVERSE && A.causal ? tiles - 1 - i : i;
      if (j >= (uint32_t)A.joins) break;
      A.joins_at[4 * j] = s.first * A.group + tile * RT;          // (query, head of the group) row
      A.joins_at[4 * j + 1] = min(rows - tile * RT, RT);
      A.joins_at[4 * j + 2] = slot_to - tiles * n + i * n;
      A.joins_at[4 * j + 3] = n;
    }
    slots = last_lane(slot_to), joins = last_lane(join_to);
  }
  if (lane == 0) *A.join_count = min(joins, (uint32_t)A.joins);
}

// The keys that query i of a sequence sees: [lo, hi) (under a tree mask, those before the new ones).
struct Range {
  int lo, hi;
};

__device__ __forceinline__ Range keys_of(const AttnArgs &A, const Seq &s, int i) {
  Range r;
  r.lo = 0;
  r.hi = s.len;
  if (A.mask) {
    r.hi = max(0, s.len - s.queries);
  } else if (A.causal) {
    const int pos = s.len - s.queries + i;
    r.hi = max(0, min(s.len, pos + 1));
    if (A.window) r.lo = min(r.hi, max(0, pos + 1 - A.window));
  }
  return r;
}

// ------------------------------------------------------------------ tiles

// 32 keys of one wave as they lie in the cache. Lane (g = lane / 16, m = lane % 16) holds, for
// each half of 16 keys, key m's codes of elements [g * DP / 4, (g + 1) * DP / 4) with their
// scales, and the codes of values m * VD .. m * VD + VD - 1 of keys 4 g .. 4 g + 3 with theirs.
template <int DP, bool ODD>
struct Tile {
  static constexpr int KS = DP / 32;                   // products of 32 along a key's elements
  static constexpr int NB = DP / 64;                   // scale blocks of a lane's key elements
  static constexpr int VD = DP / 16;                   // value elements of a lane
  static constexpr int NU = DP == 256 ? 2 : 1;         // octets of value elements that a lane loads
  uint32_t kw[2][KS];
  // as loaded: widening here would wait for the load
  typename std::conditional<NB == 4 && !ODD, uint32_t, typename std::conditional<NB == 2 && !ODD, uint16_t, uint8_t>::type>::type
      ks[2][ODD ? NB : 1];
  u32x4_t vw[2][NU];
  uint32_t vs[2];
};

// What does not change from tile to tile: byte offsets of a lane in a head's part of a page.
struct LaneOffsets {
  uint32_t k, ks, v, vs;
};

template <int DP>
__device__ __forceinline__ LaneOffsets lane_offsets(const KvView &kv) {
  const uint32_t lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const uint32_t D = kv.D, octets = D / 8, blocks = D / 16;
  LaneOffsets o;
  // Lanes past the head's elements read some in-page bytes that are multiplied by zero: a key
  // row may be overrun by up to 56 bytes, which the sections behind it always hold.
  o.k = m * (D / 2) + g * (DP / 8);
  o.ks = kv.k_scales() + m * blocks + min(g * (DP / 64), blocks - 1);
  const uint32_t octet = DP == 64 ? m / 2 : DP == 128 ? m : 2 * m;
  o.v = kv.v_codes() + g * (D * 2) + min(octet, octets - (DP == 256 ? 2 : 1)) * 16;
  o.vs = kv.v_scales() + (min(octet / 2, blocks - 1) << kv.log_p) + 4 * g;
  return o;
}

// One head's part of a page as a buffer: a uniform base with 32-bit offsets per lane (no 64-bit
// address registers), and reads past the part return zero.
typedef __amdgpu_buffer_rsrc_t Buffer;

__device__ __forceinline__ Buffer head_buffer(const KvView &kv, int page, int64_t head_at) {
  const uint8_t *p = kv.pages + (int64_t)page * kv.page_stride + head_at;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, kv.head_bytes(), 0x00027000);
}

// A pair of scales, at any byte.
__device__ __forceinline__ uint32_t load_pair(const uint8_t *p) {
  uint16_t h;
  __builtin_memcpy(&h, p, 2);
  return h;
}

// ODD: the scales of a lane do not lie at a multiple of their size (D is no multiple of DP / 4).
template <int DP, bool ODD>
__device__ __forceinline__ void load_half(const KvView &kv, const LaneOffsets &o, Buffer head, uint32_t at, Tile<DP, ODD> &t,
                                          int st) {
  constexpr int NB = Tile<DP, ODD>::NB;
  const uint32_t codes = at * (uint32_t)(kv.D / 2), ks = at * (uint32_t)(kv.D / 16);
#pragma unroll
  for (int i = 0; i < Tile<DP, ODD>::KS / 4; i++) {
    const u32x4_t w = __builtin_amdgcn_raw_buffer_load_b128(head, o.k + 16 * i, codes, 0);
#pragma unroll
    for (int j = 0; j < 4; j++) t.kw[st][4 * i + j] = w[j];
  }
  if (Tile<DP, ODD>::KS == 2) {
    const u32x2_t w = __builtin_amdgcn_raw_buffer_load_b64(head, o.k, codes, 0);
    t.kw[st][0] = w[0], t.kw[st][1] = w[1];
  }
  if constexpr (NB == 1 || ODD) {
#pragma unroll
    for (int i = 0; i < NB; i++) t.ks[st][i] = __builtin_amdgcn_raw_buffer_load_b8(head, o.ks + i, ks, 0);
  } else if constexpr (NB == 2) {
    t.ks[st][0] = __builtin_amdgcn_raw_buffer_load_b16(head, o.ks, ks, 0);
  } else {
    t.ks[st][0] = __builtin_amdgcn_raw_buffer_load_b32(head, o.ks, ks, 0);
  }
#pragma unroll
  for (int u = 0; u < Tile<DP, ODD>::NU; u++) t.vw[st][u] = __builtin_amdgcn_raw_buffer_load_b128(head, o.v + 16 * u, codes, 0);
  t.vs[st] = __builtin_amdgcn_raw_buffer_load_b32(head, o.vs, at, 0);
}

// The scale bytes of a lane's key elements in a half, as one word.
template <int DP, bool ODD>
__device__ __forceinline__ uint32_t key_scales(const Tile<DP, ODD> &t, int st) {
  uint32_t w = t.ks[st][0];
  if (ODD)
#pragma unroll
    for (int i = 1; i < Tile<DP, ODD>::NB; i++) w |= (uint32_t)t.ks[st][i] << (8 * i);
  return w;
}

// Page ids of a tile's two halves. They come through the scalar cache (the table is constant while
// a kernel runs): their waits are counted apart from those of the vector loads, so asking for the
// next tile's page does not wait for the present tile's bytes.
typedef const __attribute__((address_space(4))) int32_t *ConstInts;

struct Ids {
  int id[2];             // as in the table: looked at only when the tile is loaded
};

__device__ __forceinline__ Ids load_ids(const KvView &kv, ConstInts row, int cols, int base) {
  Ids r;
#pragma unroll
  for (int st = 0; st < 2; st++) r.id[st] = row[min((base + 16 * st) >> kv.log_p, cols - 1)];
  return r;
}

// Loads the 32 keys from `base` on. Returns bit st: half st has keys and lies in a page of the pool
// (where not, the bytes are those of the first page).
template <int DP, bool ODD>
__device__ __forceinline__ uint32_t load_tile(const KvView &kv, const LaneOffsets &o, const Ids &ids, int cols,
                                              int64_t head_at, int base, Tile<DP, ODD> &t) {
  uint32_t ok = 0;
#pragma unroll
  for (int st = 0; st < 2; st++) {
    const int key = base + 16 * st;
    // column < cols and 0 <= id < num_pages, by sign bits: it stays on the scalar unit
    const int id = ids.id[st];
    const uint32_t in = (uint32_t)(((key >> kv.log_p) - cols) & ~id & (id - kv.num_pages)) >> 31;
    ok |= in << st;
    load_half<DP, ODD>(kv, o, head_buffer(kv, (int)in * id, head_at), (uint32_t)key & (kv.P() - 1u), t, st);
  }
  return ok;
}

// The eight codes of one dword with the scale pair {s, s} -> eight exact FP16 products.
__device__ __forceinline__ half8_t dequant_dword(uint32_t w, half2_t sc) {
  const half2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0) * sc;
  const half2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1) * sc;
  const half2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2) * sc;
  const half2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3) * sc;
  return half8_t{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// Values of two keys (a, b: the same octet of each) paired for the product over keys: element
// e of the octet as {a_e, b_e}. Swapping nibbles between the two dwords puts a_e and b_e into one
// byte, which one conversion turns into the pair: four bit operations for sixteen elements.
__device__ __forceinline__ uint32_t even_pairs(uint32_t a, uint32_t b) { return (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u); }
__device__ __forceinline__ uint32_t odd_pairs(uint32_t a, uint32_t b) { return ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u); }

template <int BYTE>
__device__ __forceinline__ half2_t pair_value(uint32_t w, half2_t sc) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, BYTE) * sc;
}

__device__ __forceinline__ half8_t join4(half2_t a, half2_t b, half2_t c, half2_t d) {
  return half8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ f32x4_t mfma(half8_t a, half8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Bytes of a scale dword that are NaN, as 0x80 in each; and those as 0xFF.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t s) { return ((s & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t spread(uint32_t top) { return (top >> 7) * 0xFFu; }

// The power of two that brings a query row with largest magnitude `top` into [2^8, 2^9), and its
// inverse (returned). Rows of zeros and rows with an infinity stay as they are.
__device__ __forceinline__ float query_scale(float top, float *up) {
  int e = (int)((__float_as_uint(top) >> 23) & 255u) - 127;      // 2^e <= top < 2^(e+1)
  if (e == 128 || top == 0.0f) e = 8;
  e = max(e, -100);
  *up = __uint_as_float((uint32_t)(127 + 8 - e) << 23);
  return __uint_as_float((uint32_t)(127 - 8 + e) << 23);
}

// ------------------------------------------------------- few rows per head

// Decoding and drafted tokens: up to 16 * NT rows a workgroup. The four waves take the tiles of
// the workgroup's keys in turn, each with its own softmax state and all rows, and join at the end;
// nothing is shared on the way, so there is no barrier in the loop. A key's and a value's bytes
// are read once by one wave, 20 registers a tile at D = 128, the next tile's in flight while the
// present one is computed.
//
// Bound by the cache's bytes where there are many: one token on 262139 keys (151 MB, 4 heads of 128):
// 32.5 us here and 6.0 in join_kernel, 4.6 TB/s of the 6.0 that a plain read reaches; one token for each
// of 64 ragged sequences (54 MB): 18.8 + 4.8 us, of which about ten pass before the first tile is there and
// after the last one. A single sequence of 731 keys (0.4 MB): 9.6 us, all latency; a launch that does
// nothing but find no unit takes 5.6. 8 or 16 waves a workgroup, non-temporal loads and contiguous
// shares of the waves measured slower or the same.
template <int DP, int NT, bool F16, bool ODD>
__global__ __launch_bounds__(256, NT == 1 && DP <= 128 ? 3 : 2) void rows_kernel(const AttnArgs A) {
  constexpr int RT = 16 * NT, KS = Tile<DP, ODD>::KS, NB = Tile<DP, ODD>::NB, VD = Tile<DP, ODD>::VD, NU = Tile<DP, ODD>::NU;
  constexpr int OS = DP + 4;                             // row stride of the join buffer
  __shared__ float join_o[kWaves * 16 * OS];
  __shared__ float join_ml[kWaves][16][2];
  const KvView &kv = A.kv;
  int block = blockIdx.x;
  if (A.joins > 0 && --block < 0) {
    list_joins<RT, false>(A);
    return;
  }
  const int head = block % kv.heads, u = block / kv.heads;
  touch_args(A);
  const float kg = kv.k_g ? kv.k_g[head] : 1.0f, vg = kv.v_g ? kv.v_g[head] : 1.0f;
  Unit unit;
  if (!find_unit<RT, false>(A, u, &unit)) return;
  const Seq &s = unit.s;
  if (!has_work(A, unit)) return;
  const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int D = kv.D, G = A.group;
  const int rows = min(s.queries, A.max_q) * G, row0 = unit.tile * RT;
  const int last_row = min(rows, row0 + RT) - 1;

  // keys of the tile's rows: all see [all_lo, all_hi), none sees outside [lo, hi)
  const RowQuery rq(row0, G);
  const Range ra = keys_of(A, s, rq.first), rb = keys_of(A, s, rq.query(last_row - row0));
  const int lo = ra.lo, hi = A.mask ? s.len : rb.hi, all_lo = rb.lo, all_hi = ra.hi;
  const int base0 = lo & ~(kTile - 1);
  const int steps = (max(0, hi - base0) + kStep - 1) / kStep;
  const Pieces pieces(steps, unit.splits);
  const int step0 = pieces.begin(unit.split), step1 = pieces.begin(unit.split + 1);

  const LaneOffsets off = lane_offsets<DP>(kv);
  const ConstInts row = (ConstInts)(uintptr_t)(A.table + (int64_t)unit.b * A.table_stride);
  const int cols = (int)(((int64_t)s.len + kv.P() - 1) >> kv.log_p);     // table entries that hold keys
  const int64_t head_at = (int64_t)head * kv.head_bytes();
  // this wave's tiles: wave, wave + 4, ... of the piece; the first is on its way while the queries load
  const int first = base0 + step0 * kStep + wave * kTile, end = min(hi, base0 + step1 * kStep);
  Tile<DP, ODD> ta, tb;
  Ids ib = {{0, 0}};
  uint32_t oka = 0;
  if (first < end) {
    const Ids ia = load_ids(kv, row, cols, first);
    ib = load_ids(kv, row, cols, first + kStep);
    oka = load_tile<DP, ODD>(kv, off, ia, cols, head_at, first, ta);
  }

  // this lane's column of S^T in each row tile: its query row, scaled by a power of two
  half8_t q[NT][KS];
  float c[NT], ref[NT], sum[NT];
  int klo[NT], khi[NT];
  const uint8_t *mrow[NT];
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    const int r = min(16 * nt + m, last_row - row0);
    const int i = rq.query(r), gh = rq.head(r);
    const Range kr = keys_of(A, s, i);
    klo[nt] = kr.lo, khi[nt] = kr.hi;
    mrow[nt] = A.mask ? A.mask + (int64_t)(s.first + i) * A.mask_stride : nullptr;
    const uint16_t *src = A.q + (int64_t)(s.first + i) * A.q_t + (int64_t)(head * G + gh) * A.q_h;
    float x[KS][8];
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; k++) {
      const int d = g * (DP / 4) + 8 * k;
      u32x4_t w = {0u, 0u, 0u, 0u};
      if (d < D) w = *reinterpret_cast<const u32x4_t *>(src + d);
      unpack8<F16>(w, x[k]);
#pragma unroll
      for (int j = 0; j < 8; j++) top = fmaxf(top, fabsf(x[k][j]));
    }
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    float up;
    c[nt] = A.scale * 1.44269504088896f / kg * query_scale(top, &up);
#pragma unroll
    for (int k = 0; k < KS; k++)
#pragma unroll
      for (int j = 0; j < 8; j++) q[nt][k][j] = (_Float16)(x[k][j] * up);
    ref[nt] = -INFINITY;
    sum[nt] = 0.0f;
  }
  f32x4_t acc[NT][VD];
#pragma unroll
  for (int nt = 0; nt < NT; nt++)
#pragma unroll
    for (int d = 0; d < VD; d++) acc[nt][d] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // scales of lanes past the head's elements are forced to zero
  uint32_t k_keep = 0;
#pragma unroll
  for (int i = 0; i < NB; i++)
    if (g * NB + i < D / 16) k_keep |= 0xFFu << (8 * i);
  const uint32_t v_keep = m * VD < D ? 0xFFFFFFFFu : 0u;

  auto compute = [&](const Tile<DP, ODD> &t, int base, uint32_t ok) {
    const bool whole = ok == 3u && base >= all_lo && base + kTile <= all_hi;      // every row sees every key
    // scores
    f32x4_t st[NT][2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int nt = 0; nt < NT; nt++) st[nt][h] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      const uint32_t ksb = key_scales<DP, ODD>(t, h) & k_keep;
#pragma unroll
      for (int k = 0; k < KS; k++) {
        const half2_t two = e4m3x2_to_f16(k / 2 >= 2 ? ksb >> 16 : ksb);
        const _Float16 sc = two[(k / 2) & 1];
        const half8_t a = dequant_dword(t.kw[h][k], half2_t{sc, sc});
#pragma unroll
        for (int nt = 0; nt < NT; nt++) st[nt][h] = mfma(a, q[nt][k], st[nt][h]);
      }
    }
    uint32_t vs[2] = {t.vs[0] & v_keep, t.vs[1] & v_keep};
    uint32_t nans[2] = {0u, 0u};
    bool any_nan = false;
    if (!whole) {
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const bool in = (ok >> h) & 1u;
        // register i holds key at + i: compared as i with what is left of it
        const int at = base + 16 * h + 4 * g, v_from = lo - at, v_to = hi - at;
        const int past = min(s.len, s.len - s.queries + A.max_q) - at;
        uint32_t keep = 0;
#pragma unroll
        for (int i = 0; i < 4; i++) {
          if (in && i >= v_from && i < v_to) keep |= 0xFFu << (8 * i);
#pragma unroll
          for (int nt = 0; nt < NT; nt++) {
            bool see = i >= klo[nt] - at && i < khi[nt] - at;
            if (A.mask && i >= khi[nt] - at && i < past) see = mrow[nt][at - (s.len - s.queries) + i] != 0;
            st[nt][h][i] = see && in ? st[nt][h][i] : -INFINITY;
          }
        }
        // values that no row sees count as zero; NaN ones that only some rows see go another way
        vs[h] &= keep;
        nans[h] = nan_bytes(vs[h]);
        vs[h] &= ~spread(nans[h]);
      }
      any_nan = __ballot((nans[0] | nans[1]) != 0u) != 0ull;
    }
    // softmax
    half8_t p[NT];
    half8_t seen[NT];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      if (any_nan) {
#pragma unroll
        for (int j = 0; j < 8; j++) seen[nt][j] = st[nt][j >> 2][j & 3] == -INFINITY ? (_Float16)0.0f : (_Float16)1.0f;
      }
      float top = fmaxf(fmaxf(fmaxf(st[nt][0][0], st[nt][0][1]), fmaxf(st[nt][0][2], st[nt][0][3])),
                        fmaxf(fmaxf(st[nt][1][0], st[nt][1][1]), fmaxf(st[nt][1][2], st[nt][1][3])));
      top *= c[nt];
      if (__ballot(top > ref[nt] + kHeadroom) != 0ull) {
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float to = fmaxf(ref[nt], top);
        const float f = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(ref[nt] - to);
        ref[nt] = to;
        sum[nt] *= f;
#pragma unroll
        for (int d = 0; d < VD; d++) acc[nt][d] *= f;
      }
      const float shift = kOffset - (ref[nt] == -INFINITY ? 0.0f : ref[nt]);
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(st[nt][j >> 2][j & 3], c[nt], shift));
        sum[nt] += e[j];
        p[nt][j] = (_Float16)e[j];
      }
    }
    // values
    half2_t sc[2][2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      sc[h][0] = e4m3x2_to_f16(vs[h]);
      sc[h][1] = e4m3x2_to_f16(vs[h] >> 16);
    }
#pragma unroll
    for (int u2 = 0; u2 < NU; u2++) {
      uint32_t ev[2][2], od[2][2];
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int pr = 0; pr < 2; pr++) {
          const uint32_t wa = t.vw[h][u2][2 * pr], wb = t.vw[h][u2][2 * pr + 1];
          ev[h][pr] = even_pairs(wa, wb);
          od[h][pr] = odd_pairs(wa, wb);
          if (DP == 64) {                          // half an octet per lane
            ev[h][pr] >>= 16 * (m & 1);
            od[h][pr] >>= 16 * (m & 1);
          }
        }
#define NVFP4_KV_VALUE(B)                                                                                      \
  if (2 * B < (DP == 64 ? 4 : 8)) {                                                                            \
    const half8_t ve = join4(pair_value<B>(ev[0][0], sc[0][0]), pair_value<B>(ev[0][1], sc[0][1]),             \
                             pair_value<B>(ev[1][0], sc[1][0]), pair_value<B>(ev[1][1], sc[1][1]));            \
    const half8_t vo = join4(pair_value<B>(od[0][0], sc[0][0]), pair_value<B>(od[0][1], sc[0][1]),             \
                             pair_value<B>(od[1][0], sc[1][0]), pair_value<B>(od[1][1], sc[1][1]));            \
    _Pragma("unroll") for (int nt = 0; nt < NT; nt++) {                                                        \
      acc[nt][(8 * u2 + 2 * B) % VD] = mfma(ve, p[nt], acc[nt][(8 * u2 + 2 * B) % VD]);                        \
      acc[nt][(8 * u2 + 2 * B + 1) % VD] = mfma(vo, p[nt], acc[nt][(8 * u2 + 2 * B + 1) % VD]);                \
    }                                                                                                          \
  }
      NVFP4_KV_VALUE(0) NVFP4_KV_VALUE(1) NVFP4_KV_VALUE(2) NVFP4_KV_VALUE(3)
#undef NVFP4_KV_VALUE
    }
    if (any_nan) {
      // A row that sees a NaN value gets NaN in that value's block, and no other row does: the
      // product of "is NaN" and "is seen" counts them.
      half8_t bad;
#pragma unroll
      for (int j = 0; j < 8; j++) bad[j] = (nans[j >> 2] >> (8 * (j & 3))) & 0x80u ? (_Float16)1.0f : (_Float16)0.0f;
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
        const f32x4_t n = mfma(bad, seen[nt], f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
        for (int d = 0; d < VD; d++)
#pragma unroll
          for (int i = 0; i < 4; i++) acc[nt][d][i] = n[i] > 0.0f ? __builtin_nanf("") : acc[nt][d][i];
      }
    }
  };

  for (int base = first; base < end; base += 2 * kStep) {
    const bool more = base + kStep < end;
    uint32_t okb = 0;
    if (more) okb = load_tile<DP, ODD>(kv, off, ib, cols, head_at, base + kStep, tb);
    const Ids ia = load_ids(kv, row, cols, base + 2 * kStep);
    compute(ta, base, oka);
    if (!more) break;
    if (base + 2 * kStep < end) oka = load_tile<DP, ODD>(kv, off, ia, cols, head_at, base + 2 * kStep, ta);
    ib = load_ids(kv, row, cols, base + 3 * kStep);
    compute(tb, base + kStep, okb);
  }

  // join the four waves, 16 rows at a time
  const bool final = unit.splits == 1;
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    sum[nt] += __shfl_xor(sum[nt], 16, 64);
    sum[nt] += __shfl_xor(sum[nt], 32, 64);
    if (g == 0) {
      join_ml[wave][m][0] = ref[nt];
      join_ml[wave][m][1] = sum[nt];
    }
    __syncthreads();
    float top = join_ml[0][m][0];
#pragma unroll
    for (int w = 1; w < kWaves; w++) top = fmaxf(top, join_ml[w][m][0]);
    const float f = ref[nt] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(ref[nt] - top);
    float *o = join_o + (wave * 16 + m) * OS + 4 * g * VD;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int d = 0; d < VD; d += 4)
        *reinterpret_cast<f32x4_t *>(o + i * VD + d) =
            f32x4_t{acc[nt][d][i] * f, acc[nt][d + 1][i] * f, acc[nt][d + 2][i] * f, acc[nt][d + 3][i] * f};
    __syncthreads();
    constexpr int PER_ROW = DP / 8;                     // threads of a row, eight elements each
#pragma unroll
    for (int it = threadIdx.x; it < 16 * PER_ROW; it += 256) {
      const int n = it / PER_ROW, d = (it % PER_ROW) * 8;
      const int r = row0 + 16 * nt + n;
      if (r > last_row || d >= D) continue;
      float tot = join_ml[0][n][0], l = 0.0f;
#pragma unroll
      for (int w = 1; w < kWaves; w++) tot = fmaxf(tot, join_ml[w][n][0]);
      float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kWaves; w++) {
        const float mw = join_ml[w][n][0];
        const float lw = join_ml[w][n][1];                 // 0 or NaN where no score was a number
        l += mw == -INFINITY ? lw : lw * __builtin_amdgcn_exp2f(mw - tot);
        const f32x4_t y0 = *reinterpret_cast<const f32x4_t *>(join_o + (w * 16 + n) * OS + d);
        const f32x4_t y1 = *reinterpret_cast<const f32x4_t *>(join_o + (w * 16 + n) * OS + d + 4);
#pragma unroll
        for (int j = 0; j < 4; j++) x[j] += y0[j], x[j + 4] += y1[j];
      }
      if (final) {
        const int i = rq.query(16 * nt + n), gh = rq.head(16 * nt + n);
        const int64_t t = s.first + i;
        const int h = head * G + gh;
        const float inv = l == 0.0f ? 0.0f : 1.0f / (l * vg);
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] *= inv;
        *reinterpret_cast<u32x4_t *>(A.out + t * A.o_t + h * A.o_h + d) = pack8<F16>(x);
        if (A.lse && d == 0)
          A.lse[t * (kv.heads * G) + h] = tot == -INFINITY && l == 0.0f
                                              ? -INFINITY
                                              : (tot - kOffset + __builtin_amdgcn_logf(l)) * 0.693147180559945f;
      } else {
        const int64_t at = ((int64_t)unit.slot * kv.heads + head) * RT + 16 * nt + n;
        float *po = A.part_o + at * D + d;
        *reinterpret_cast<f32x4_t *>(po) = f32x4_t{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<f32x4_t *>(po + 4) = f32x4_t{x[4], x[5], x[6], x[7]};
        if (d == 0) {
          A.part_ml[2 * at] = tot;
          A.part_ml[2 * at + 1] = l;
        }
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------ many rows per head

// Prefill chunks and larger sets of drafted tokens: 128 rows a workgroup, 32 a wave, in 32 x 32 x 16
// steps. What rows_kernel does for each wave, dequantizing, the four waves do together here: a tile
// of KT keys goes once to LDS as FP16, already in the order in which the matrix cores take it (a
// fragment of 64 lanes x 16 bytes is contiguous: neither writes nor reads conflict), and every wave
// reads all of it. Two tiles are kept: while one is multiplied, the next one's codes are on their
// way into registers, and they are dequantized into the other buffer before the one barrier of a
// tile.
//
// Chunks of up to 2048 queries of 40 heads on 4 sequences of up to 8192 keys (508 GFLOP): 591 to 606 us,
// 0.84 to 0.86 PFLOP/s (a plain 8192^3 product: 1.27). No unit is full: the matrix cores are busy a
// third of the cycles, the vector units 56 % (350 instructions a wave and tile, of which a third is
// the softmax and a quarter dequantizing), LDS 31 %; the two waves of a SIMD wait for data, barriers
// and each other for the rest. Measured and not better: the next tile's dequantizing among the first
// product's steps (620 against 605), fragments read ahead in the second product too (640 against 636),
// codes two tiles ahead (600 against 606, for twice the code), tiles of 32 keys with three waves a SIMD
// (834 against 600). At D > 128 a lane's sums and queries take 192 registers; two waves a SIMD spill 51
// of 256, and win nothing by it (2048 queries of 8 heads of 256 on 4 x 8192 keys, 481 GFLOP: 921 us with one
// workgroup a CU, 912 with two; 256 on 32000 keys 146 and 144; 32 drafted trees 68.4 and 68.8): one is kept.
template <int DP>
struct Block {
  static constexpr int KT = DP == 256 ? 32 : 64;       // keys of a tile (LDS: 64 KiB at D >= 128)
  static constexpr int KG = KT / 32;                   // 32-key rows of S^T
  static constexpr int KS = DP / 16;                   // products of 16 along a key's elements
  static constexpr int PARTS = DP / 64;                // 32-element parts of a half key
  static constexpr int DT = DP / 32;                   // 32-element columns of V
  static constexpr int T16 = KT / 16;                  // products of 16 along the keys
  static constexpr int OCTETS = DP / 8;
  static constexpr int K_WAVES = KG * PARTS;           // waves that dequantize keys: 2, 4, 4
  static constexpr int V_FIRST = DP == 64 ? 2 : 0;     // first wave that dequantizes values
};

__device__ __forceinline__ f32x16_t mfma32(half8_t a, half8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// Order of a straight stretch of N matrix steps that each take one LDS fragment: AHEAD fragments are
// on their way before the first step, and each step is followed by the read of a later step's. Left
// alone, the compiler reads one or two right before the step that waits for them.
template <int N, int AHEAD>
__device__ __forceinline__ void pace() {
  __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);              // LDS reads
#pragma unroll
  for (int i = 0; i < N; i++) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);                  // a matrix instruction
    if (i < N - AHEAD) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
}

// A thread's part of a tile as it lies in the cache: 32 elements of one key, eight of four values. vm: all
// ones, or zero where the values' page id lies outside the pool (block_kernel's drop_scales).
struct Raw {
  u32x4_t kw, vw;
  uint32_t ks, vs, vm;
};

template <int DP, bool F16>
__global__ __launch_bounds__(256, DP == 256 ? 1 : 2) void block_kernel(const AttnArgs A) {
  using B = Block<DP>;
  constexpr int RT = kBlockRows, KT = B::KT, KG = B::KG, KS = B::KS, DT = B::DT, T16 = B::T16;
  __shared__ u32x4_t kbuf[2][KG * KS * 64];
  __shared__ u32x4_t vbuf[2][DT * T16 * 64];
  const KvView &kv = A.kv;
  int block = blockIdx.x;
  if (A.joins > 0 && --block < 0) {
    list_joins<RT, true>(A);
    return;
  }
  const int head = block % kv.heads, u = block / kv.heads;
  touch_args(A);
  const float gk = kv.k_g ? kv.k_g[head] : 1.0f, vg = kv.v_g ? kv.v_g[head] : 1.0f;
  Unit unit;
  if (!find_unit<RT, true>(A, u, &unit)) return;
  const Seq &s = unit.s;
  if (!has_work(A, unit)) return;
  const int lane = threadIdx.x & 63, m = lane & 31, hi = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int D = kv.D, G = A.group;
  const int rows = min(s.queries, A.max_q) * G, row0 = unit.tile * RT, last_row = min(rows, row0 + RT) - 1;
  const RowQuery rq(row0, G);
  const Range ra = keys_of(A, s, rq.first), rb = keys_of(A, s, rq.query(last_row - row0));
  const int lo = ra.lo, end = A.mask ? s.len : rb.hi, all_lo = rb.lo, all_hi = ra.hi;
  // this wave's rows (the last ones again where there are fewer)
  const int w0 = min(32 * wave, last_row - row0), w1 = min(32 * wave + 31, last_row - row0);
  const bool working = row0 + 32 * wave <= last_row;
  const Range wa = keys_of(A, s, rq.query(w0)), wb = keys_of(A, s, rq.query(w1));
  const int w_lo = wa.lo, w_hi = A.mask ? s.len : wb.hi;
  const int base0 = lo & ~(kStep - 1);
  const int steps = (max(0, end - base0) + kStep - 1) / kStep;
  const Pieces pieces(steps, unit.splits);
  const int first = base0 + pieces.begin(unit.split) * kStep;
  const int last = min(end, base0 + pieces.begin(unit.split + 1) * kStep);

  // this lane's column of S^T: its query row, scaled by a power of two
  const int r = min(32 * wave + m, last_row - row0);
  const int qi = rq.query(r), gh = rq.head(r);
  const Range mine = keys_of(A, s, qi);
  const uint8_t *mrow = A.mask ? A.mask + (int64_t)(s.first + qi) * A.mask_stride : nullptr;
  half8_t q[KS];
  float c;
  {
    const uint16_t *src = A.q + (int64_t)(s.first + qi) * A.q_t + (int64_t)(head * G + gh) * A.q_h;
    u32x4_t w[KS];
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; k++) {
      const int d = hi * (DP / 2) + 8 * k;
      w[k] = u32x4_t{0u, 0u, 0u, 0u};
      if (d < D) w[k] = *reinterpret_cast<const u32x4_t *>(src + d);
    }
#pragma unroll
    for (int k = 0; k < KS; k++) {
      float x[8];
      unpack8<F16>(w[k], x);
#pragma unroll
      for (int j = 0; j < 8; j++) top = fmaxf(top, fabsf(x[j]));
    }
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    float up;
    c = A.scale * 1.44269504088896f / gk * query_scale(top, &up);
#pragma unroll
    for (int k = 0; k < KS; k++) {
      float x[8];
      unpack8<F16>(w[k], x);
#pragma unroll
      for (int j = 0; j < 8; j++) q[k][j] = (_Float16)(x[j] * up);
    }
  }

  // which part of a tile this thread dequantizes
  const bool k_task = B::K_WAVES == kWaves || wave < B::K_WAVES, v_task = B::V_FIRST == 0 || wave >= B::V_FIRST;
  const int kg = k_task ? wave / B::PARTS : 0, part = k_task ? wave % B::PARTS : 0;
  const int kd0 = hi * (DP / 2) + part * 32;             // first element of its key part
  const int vw = wave - B::V_FIRST;
  const int octet = DP == 64 ? lane & 7 : DP == 128 ? lane & 15 : (lane & 15) + 16 * (vw & 1);
  const int tg = DP == 64 ? vw * 8 + (lane >> 3) : DP == 128 ? vw * 4 + (lane >> 4) : (vw >> 1) * 4 + (lane >> 4);
  const uint32_t octets = D / 8, blocks = D / 16;
  const uint32_t oc = min((uint32_t)octet, octets - 1);
  const uint32_t k_keep = (kd0 < D ? 0xFFu : 0u) | (kd0 + 16 < D ? 0xFF00u : 0u);
  const uint32_t v_keep = 8 * octet < D ? 0xFFFFFFFFu : 0u;
  const int32_t *row = A.table + (int64_t)unit.b * A.table_stride;
  const int cols = (int)(((int64_t)s.len + kv.P() - 1) >> kv.log_p);     // table entries that hold keys
  const int64_t head_at = (int64_t)head * kv.head_bytes();
  // (a key row may be overrun inside its page, as in lane_offsets; the scale pair of a part past the
  // head's elements is taken from the last two bytes)
  const uint32_t k_off = kd0 / 2, ks_off = kv.k_scales() + (blocks < 2 ? 0u : min((uint32_t)kd0 / 16, blocks - 1));
  const uint32_t v_off = kv.v_codes() + oc * 16, vs_off = kv.v_scales() + ((oc / 2) << kv.log_p);

  // page ids of a tile's groups of 16 keys, one lane each
  auto load_ids = [&](int base) {
    const int col = (base + 16 * lane) >> kv.log_p;
    return lane < T16 && col < cols ? row[col] : -1;
  };
  auto page_at = [&](int ids, int group) {
    const int id = __builtin_amdgcn_readlane(ids, group);
    return kv.pages + (int64_t)(id >= 0 && id < kv.num_pages ? id : 0) * kv.page_stride + head_at;
  };
  // Which of a tile's groups of 16 keys lie in a page of the pool, as bits.
  constexpr uint32_t ALL = (1u << T16) - 1u;
  auto inside = [&](int ids) { return (uint32_t)__ballot(ids >= 0 && ids < kv.num_pages) & ALL; };
  auto load_raw = [&](int ids, int base, Raw &t) {
    if (k_task) {
      const int key = base + 32 * kg + m;
      const uint8_t *p0 = page_at(ids, 2 * kg), *p1 = page_at(ids, 2 * kg + 1);
      const uint8_t *p = m < 16 ? p0 : p1;
      const uint32_t at = (uint32_t)key & (kv.P() - 1u);
      t.kw = *reinterpret_cast<const u32x4_a4 *>(p + at * (uint32_t)(D / 2) + k_off);
      t.ks = load_pair(p + at * blocks + ks_off);
    }
    if (v_task) {
      const int token = base + 4 * tg;
      const uint8_t *p = DP == 64 ? ((tg >> 2) & 1 ? page_at(ids, 2 * vw + 1) : page_at(ids, 2 * vw))
                                  : page_at(ids, DP == 128 ? vw : vw >> 1);
      const uint32_t at = (uint32_t)token & (kv.P() - 1u);
      t.vw = *reinterpret_cast<const u32x4_t *>(p + at * (uint32_t)(D / 2) + v_off);
      t.vs = *reinterpret_cast<const uint32_t *>(p + at + vs_off);
      t.vm = 0xFFFFFFFFu;
      if (DP == 128) {
        const int id = __builtin_amdgcn_readlane(ids, vw);
        t.vm = id >= 0 && id < kv.num_pages ? 0xFFFFFFFFu : 0u;
      }
    }
  };
  // For an id outside the pool page_at gives the first page, whose owner may hold NaN there, and a zero
  // probability does not cancel NaN: the values of such a group become zero. Where a wave's values lie in
  // one page (D = 128) by a scalar mask on their scales, where they lie in two (64) by a select behind a
  // branch, and at 256, where a wave has the fewest registers to spare, in LDS, by each wave that
  // multiplies the tile, ahead of its own reads. Each costs the least of the three there: chunks of 64-,
  // 128- and 256-wide heads took 401, 592 and 986 us with none of them, 395, 592 and 923 with these, 430,
  // 597 and 1016 with masks, 418, 598 and 926 all in LDS.
  auto drop_scales = [&](Raw &t, int ids) {
    const uint32_t ok = inside(ids);
    if (DP == 64 && ok != ALL) t.vs = (ok >> ((tg >> 2) & (T16 - 1))) & 1u ? t.vs : 0u;
  };
  auto drop_values = [&](int buf, uint32_t ok) {
#pragma nounroll
    for (int f = 0; f < DT * T16; f++)
      if (!((ok >> (f % T16)) & 1u)) vbuf[buf][f * 64 + lane] = u32x4_t{0u, 0u, 0u, 0u};
  };
  // Clears the scales of values that no row sees and, in a tile that some rows see only in part, of
  // NaN values (the rows that see those are mended by themselves); true if there was one.
  auto clear_unseen = [&](Raw &t, int base) {
    const int at = base + 4 * tg, from = lo - at, to = end - at;
    uint32_t keep = 0;
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (i >= from && i < to) keep |= 0xFFu << (8 * i);
    const uint32_t bad = nan_bytes(t.vs & keep & v_keep);
    t.vs &= keep & ~spread(bad);
    return v_task && bad != 0u;
  };
  auto edge = [&](int base) { return base < all_lo || base + KT > all_hi; };
  // Dequantizes this thread's part of a tile into buffer `buf`.
  auto store_tile = [&](const Raw &t, int buf) {
    if (k_task) {
      const half2_t sc = e4m3x2_to_f16(t.ks & k_keep);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const _Float16 f = sc[i >> 1];
        const half8_t w = dequant_dword(t.kw[i], half2_t{f, f});
        u32x4_t o;
        __builtin_memcpy(&o, &w, 16);
        kbuf[buf][(kg * KS + 4 * part + i) * 64 + lane] = o;
      }
    }
    if (v_task) {
      const uint32_t vs = t.vs & v_keep & t.vm;
      const half2_t s01 = e4m3x2_to_f16(vs), s23 = e4m3x2_to_f16(vs >> 16);
      const uint32_t e01 = even_pairs(t.vw[0], t.vw[1]), o01 = odd_pairs(t.vw[0], t.vw[1]);
      const uint32_t e23 = even_pairs(t.vw[2], t.vw[3]), o23 = odd_pairs(t.vw[2], t.vw[3]);
      // element e of the octet: column e % DT, lane octet + OCTETS * (e / DT); four tokens are half
      // of the eight that a lane holds, the other half and the other half wave by the token group
      uint8_t *to = reinterpret_cast<uint8_t *>(vbuf[buf]) + ((tg >> 2) * 64 + (tg & 1) * 32 + octet) * 16 + ((tg >> 1) & 1) * 8;
#define NVFP4_KV_PUT(E, X, Y)                                                                             \
  {                                                                                                       \
    const half2_t a = X, b = Y;                                                                           \
    const uint32_t ua = __builtin_bit_cast(uint32_t, a), ub = __builtin_bit_cast(uint32_t, b);            \
    *reinterpret_cast<u32x2_t *>(to + ((E % DT) * T16 * 64 + B::OCTETS * (E / DT)) * 16) = u32x2_t{ua, ub}; \
  }
      NVFP4_KV_PUT(0, pair_value<0>(e01, s01), pair_value<0>(e23, s23))
      NVFP4_KV_PUT(1, pair_value<0>(o01, s01), pair_value<0>(o23, s23))
      NVFP4_KV_PUT(2, pair_value<1>(e01, s01), pair_value<1>(e23, s23))
      NVFP4_KV_PUT(3, pair_value<1>(o01, s01), pair_value<1>(o23, s23))
      NVFP4_KV_PUT(4, pair_value<2>(e01, s01), pair_value<2>(e23, s23))
      NVFP4_KV_PUT(5, pair_value<2>(o01, s01), pair_value<2>(o23, s23))
      NVFP4_KV_PUT(6, pair_value<3>(e01, s01), pair_value<3>(e23, s23))
      NVFP4_KV_PUT(7, pair_value<3>(o01, s01), pair_value<3>(o23, s23))
#undef NVFP4_KV_PUT
    }
  };

  float ref = -INFINITY, sum = 0.0f;
  f32x16_t acc[DT];
#pragma unroll
  for (int d = 0; d < DT; d++)
#pragma unroll
    for (int i = 0; i < 16; i++) acc[d][i] = 0.0f;

  // Which keys of a tile this lane's row sees, register by register of S^T: key 32 g + o (o a constant
  // of the register, less this half wave's 4 hi) when from <= 32 g + o < to; new keys under a tree
  // mask from `to` up to `past`.
  auto seen = [&](int base, uint32_t ok, auto put) {
    const int at = base + 4 * hi, from = mine.lo - at, to = mine.hi - at, past = min(s.len, s.len - s.queries + A.max_q) - at;
    const uint8_t *mk = A.mask ? mrow + (at - (s.len - s.queries)) : nullptr;
#pragma unroll
    for (int g = 0; g < KG; g++)
#pragma unroll
      for (int i = 0; i < 16; i++) {
        const int o = 32 * g + 8 * (i >> 2) + (i & 3);
        bool see = o >= from && o < to;
        if (A.mask && o >= to && o < past) see = mk[o] != 0;
        put(g, i, see && ((ok >> (2 * g + (i >> 3))) & 1u));
      }
  };
  // A row that sees a NaN value gets NaN in that value's block, and no other row does: the product of
  // "is NaN" and "is seen" counts them. (All of a lane's elements lie in one block.)
  auto nan_rows = [&](int base, int ids, uint32_t ok) {
    f32x16_t n;
#pragma unroll
    for (int i = 0; i < 16; i++) n[i] = 0.0f;
    half8_t see[T16];
    seen(base, ok, [&](int g, int i, bool is) { see[2 * g + (i >> 3)][i & 7] = is ? (_Float16)1.0f : (_Float16)0.0f; });
#pragma unroll
    for (int t = 0; t < T16; t++) {
      const uint8_t *page = page_at(ids, t);
      const uint32_t at = (uint32_t)(base + 16 * t + 4 * hi) & (kv.P() - 1u);
      const uint32_t blk = min((uint32_t)(m % B::OCTETS) / 2, blocks - 1);
      half8_t bad;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const uint32_t vs = page[kv.v_scales() + (blk << kv.log_p) + at + 8 * (j >> 2) + (j & 3)];
        bad[j] = (vs & 0x7Fu) == 0x7Fu && (ok >> t) & 1u ? (_Float16)1.0f : (_Float16)0.0f;
      }
      n = mfma32(bad, see[t], n);
    }
#pragma unroll
    for (int d = 0; d < DT; d++)
#pragma unroll
      for (int i = 0; i < 16; i++) acc[d][i] = n[i] > 0.0f ? __builtin_nanf("") : acc[d][i];
  };

  // While tile t is multiplied, tile t + 1 is on its way into registers; it is dequantized into the
  // other buffer before the one barrier of a tile.
  bool nan_now = false;
  int ids = 0, ids1 = 0;
  Raw raw = {};
  if (first < last) {
    ids = load_ids(first);
    load_raw(ids, first, raw);
    ids1 = load_ids(first + KT);
    drop_scales(raw, ids);
    if (edge(first)) nan_now = clear_unseen(raw, first);
    store_tile(raw, 0);
  }
  nan_now = __syncthreads_or(nan_now);
  int buf = 0;
  for (int base = first; base < last; base += KT, buf ^= 1) {
    const bool more = base + KT < last;
    int ids2 = 0;
    if (more) {
      load_raw(ids1, base + KT, raw);
      ids2 = load_ids(base + 2 * KT);
    }
    if (working && base < w_hi && base + KT > w_lo) {
      f32x16_t st[KG];
#pragma unroll
      for (int g = 0; g < KG; g++) {
#pragma unroll
        for (int i = 0; i < 16; i++) st[g][i] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; k++) {
          const u32x4_t w = kbuf[buf][(g * KS + k) * 64 + lane];
          half8_t a;
          __builtin_memcpy(&a, &w, 16);
          st[g] = mfma32(a, q[k], st[g]);
        }
      }
      pace<KG * KS, 4>();
      const uint32_t ok = inside(ids);
      if (ok != ALL || base < wb.lo || base + KT > wa.hi) {
        seen(base, ok, [&](int g, int i, bool is) { st[g][i] = is ? st[g][i] : -INFINITY; });
        if (DP == 256 && __builtin_expect(ok != ALL, 0)) drop_values(buf, ok);
      }
      float top = st[0][0];
#pragma unroll
      for (int g = 0; g < KG; g++)
#pragma unroll
        for (int i = 0; i < 16; i++) top = fmaxf(top, st[g][i]);
      top *= c;
      if (__ballot(top > ref + kHeadroom) != 0ull) {
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float to = fmaxf(ref, top);
        const float f = to == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(ref - to);
        ref = to;
        sum *= f;
#pragma unroll
        for (int d = 0; d < DT; d++)
#pragma unroll
          for (int i = 0; i < 16; i++) acc[d][i] *= f;
      }
      const float shift = kOffset - (ref == -INFINITY ? 0.0f : ref);
#pragma unroll
      for (int t = 0; t < T16; t++) {
        half8_t p;
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(st[t >> 1][8 * (t & 1) + j], c, shift));
          sum += e;
          p[j] = (_Float16)e;
        }
#pragma unroll
        for (int d = 0; d < DT; d++) {
          const u32x4_t w = vbuf[buf][(d * T16 + t) * 64 + lane];
          half8_t a;
          __builtin_memcpy(&a, &w, 16);
          acc[d] = mfma32(a, p, acc[d]);
        }
      }
      if (nan_now) nan_rows(base, ids, ok);
    }
    bool nan_next = false;
    const bool next_edge = more && edge(base + KT);
    if (next_edge) nan_next = clear_unseen(raw, base + KT);
    if (more) {
      drop_scales(raw, ids1);
      store_tile(raw, buf ^ 1);
    }
    // (only tiles that some rows see in part look at values one by one)
    if (next_edge) nan_now = __syncthreads_or(nan_next);
    else {
      __syncthreads();
      nan_now = false;
    }
    ids = ids1, ids1 = ids2;
  }
  if (!working) return;

  sum += __shfl_xor(sum, 32, 64);
  const bool final = unit.splits == 1;
  const int64_t slot_row = ((int64_t)unit.slot * kv.heads + head) * RT + 32 * wave;
  const int h = head * G + gh;
  if (hi == 0 && row0 + 32 * wave + m <= last_row) {
    if (!final) {
      A.part_ml[2 * (slot_row + m)] = ref, A.part_ml[2 * (slot_row + m) + 1] = sum;
    } else if (A.lse) {
      A.lse[(int64_t)(s.first + qi) * (kv.heads * G) + h] =
          ref == -INFINITY && sum == 0.0f ? -INFINITY
                                          : (ref - kOffset + __builtin_amdgcn_logf(sum)) * 0.693147180559945f;
    }
  }
  // A lane holds elements of one row: stored from there, 64 lanes write to 64 places. The wave's rows go
  // through its quarter of the tiles' LDS (nobody reads tiles any more), 128 columns at a time, and leave
  // in whole rows. Unit u of row m lies at u ^ m, so neither side conflicts.
  constexpr int COLS = DP < 128 ? DP : 128, UNITS = COLS / 4, PHASES = DP / COLS;
  static_assert(sizeof(kbuf) == 2 * 32 * UNITS * 16 && sizeof(vbuf) == sizeof(kbuf), "two waves' rows each");
  f32x4_t *stage = reinterpret_cast<f32x4_t *>(wave < 2 ? &kbuf[0][0] : &vbuf[0][0]) + (wave & 1) * 32 * UNITS;
  const float by = !final ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / (sum * vg);
  const int64_t out_at = (int64_t)(s.first + qi) * A.o_t + (int64_t)h * A.o_h;
#pragma unroll
  for (int ph = 0; ph < PHASES; ph++) {
    // element d of column dt in register i: see store_tile for which it is
#pragma unroll
    for (int i = 16 / PHASES * ph; i < 16 / PHASES * (ph + 1); i++) {
      const int mm = 8 * (i >> 2) + 4 * hi + (i & 3);
      const int unit4 = (8 * (mm % B::OCTETS) + DT * (mm / B::OCTETS) - COLS * ph) / 4;
      if constexpr (DT >= 4) {
#pragma unroll
        for (int j = 0; j < DT; j += 4)
          stage[m * UNITS + ((unit4 + j / 4) ^ (m & (UNITS - 1)))] =
              f32x4_t{acc[j][i] * by, acc[j + 1][i] * by, acc[j + 2][i] * by, acc[j + 3][i] * by};
      } else {
        float *at = reinterpret_cast<float *>(stage + m * UNITS + (unit4 ^ (m & (UNITS - 1))));
        *reinterpret_cast<f32x2_t *>(at + (DT * (mm / B::OCTETS)) % 4) = f32x2_t{acc[0][i] * by, acc[1][i] * by};
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    if (final) {
      constexpr int PER = COLS / 8;                       // lanes of a row
#pragma unroll
      for (int n0 = 0; n0 < 32; n0 += 64 / PER) {
        const int n = n0 + lane / PER, d = (lane % PER) * 8, at = d / 4;
        const int64_t to = __shfl((long long)out_at, n, 64);
        const f32x4_t y0 = stage[n * UNITS + (at ^ (n & (UNITS - 1)))], y1 = stage[n * UNITS + ((at + 1) ^ (n & (UNITS - 1)))];
        const float x[8] = {y0[0], y0[1], y0[2], y0[3], y1[0], y1[1], y1[2], y1[3]};
        if (row0 + 32 * wave + n <= last_row && COLS * ph + d < D)
          *reinterpret_cast<u32x4_t *>(A.out + to + COLS * ph + d) = pack8<F16>(x);
      }
    } else {
#pragma unroll
      for (int n0 = 0; n0 < 32; n0 += 64 / UNITS) {
        const int n = n0 + lane / UNITS, at = lane % UNITS;
        const f32x4_t y = stage[n * UNITS + (at ^ (n & (UNITS - 1)))];
        if (row0 + 32 * wave + n <= last_row && COLS * ph + 4 * at < D)
          *reinterpret_cast<f32x4_t *>(A.part_o + (slot_row + n) * D + COLS * ph + 4 * at) = y;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// ---------------------------------------------------------------- joining

// Joins the pieces of a split row tile: with m_s, l_s, O_s of piece s and m = max m_s,
// out = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s. DP / 4 threads hold a row (four elements
// each) and are a slice; ROWS rows share a workgroup, and the slices of a row take its pieces in
// turn, eight loads in flight, and are added in order: the result does not depend on timing. 5 to 6 us,
// the latency of two dependent loads and a launch; a workgroup that joins the pieces when it is the last
// to finish saves the launch, but its device-scope fences cost 10 to 25 us.
template <int DP, int RT, int ROWS, bool F16>
__global__ __launch_bounds__(256) void join_kernel(const AttnArgs A, int groups) {
  constexpr int TH = DP / 4, SL = 256 / TH / ROWS;      // threads of a slice, slices of a row
  static_assert(SL >= 1, "too many rows");
  __shared__ f32x4_t sm_o[ROWS * SL * TH];
  __shared__ float sm_ml[ROWS * SL][2];
  const KvView &kv = A.kv;
  const int group = blockIdx.x % groups, rest = blockIdx.x / groups;
  const int head = rest % kv.heads, j = rest / kv.heads;
  // (read beside the count, not after it: past the count it is whatever was there, and not used)
  const int count = *A.join_count;
  const int row0 = A.joins_at[4 * j], rows = A.joins_at[4 * j + 1], slot = A.joins_at[4 * j + 2], splits = A.joins_at[4 * j + 3];
  if (j >= count) return;
  // (the second only with sequences that overlap in q_start)
  if (group * ROWS >= rows || (uint32_t)slot >= (uint32_t)A.slots || splits > A.slots - slot) return;
  const int D = kv.D, G = A.group;
  const int sl = threadIdx.x / TH, d = (threadIdx.x % TH) * 4;
  const int n = group * ROWS + sl / SL, part = sl % SL;
  float m = -INFINITY, l = 0.0f;
  f32x4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (d < D && n < rows) {
    const int64_t at0 = ((int64_t)slot * kv.heads + head) * RT + n, step = (int64_t)kv.heads * RT;
    for (int i0 = part; i0 < splits; i0 += 8 * SL) {
      float mi[8], li[8];
      f32x4_t oi[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int piece = i0 + i * SL;
        const int64_t at = at0 + min(piece, splits - 1) * step;
        const f32x2_t ml = *reinterpret_cast<const f32x2_t *>(A.part_ml + 2 * at);
        oi[i] = *reinterpret_cast<const f32x4_t *>(A.part_o + at * D + d);
        mi[i] = piece < splits ? ml[0] : -INFINITY;
        li[i] = piece < splits ? ml[1] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; i++) {
        if (mi[i] == -INFINITY && li[i] == 0.0f) continue;         // a piece without keys
        const float to = fmaxf(m, mi[i]);
        const float fa = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - to);
        const float fb = mi[i] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(mi[i] - to);
        m = to;
        l = l * fa + li[i] * fb;
        o = o * fa + oi[i] * fb;
      }
    }
  }
  if (SL > 1) {
    sm_o[threadIdx.x] = o;
    if (d == 0) sm_ml[sl][0] = m, sm_ml[sl][1] = l;
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int i = 1; i < SL; i++) {
        const float mi = sm_ml[sl + i][0], li = sm_ml[sl + i][1];
        if (mi == -INFINITY && li == 0.0f) continue;
        const float to = fmaxf(m, mi);
        const float fa = m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - to);
        const float fb = mi == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(mi - to);
        m = to;
        l = l * fa + li * fb;
        o = o * fa + sm_o[threadIdx.x + i * TH] * fb;
      }
    }
  }
  if (part != 0 || d >= D || n >= rows) return;
  const float vg = kv.v_g ? kv.v_g[head] : 1.0f;
  const float inv = l == 0.0f ? 0.0f : 1.0f / (l * vg);
  const int r = row0 + n, h = head * G + r % G;
  const int64_t t = r / G;
  uint16_t *to = A.out + t * A.o_t + h * A.o_h + d;
  const uint32_t w0 = (uint32_t)pack1<F16>(o[0] * inv) | ((uint32_t)pack1<F16>(o[1] * inv) << 16);
  const uint32_t w1 = (uint32_t)pack1<F16>(o[2] * inv) | ((uint32_t)pack1<F16>(o[3] * inv) << 16);
  *reinterpret_cast<u32x2_t *>(to) = u32x2_t{w0, w1};
  if (A.lse && d == 0)
    A.lse[t * (kv.heads * G) + h] = m == -INFINITY && l == 0.0f
                                        ? -INFINITY
                                        : (m - kOffset + __builtin_amdgcn_logf(l)) * 0.693147180559945f;
}

// ------------------------------------------------------------------- host

struct Launch {
  int nt;                    // row tiles of 16 nt rows in rows_kernel; 8: block_kernel's 128
  int target;
  int64_t units, joins, slots;
  bool few;
  int rows;                  // rows of a row tile that can be there, in whole workgroups of join_kernel
};

// Sizes of a call from what the host knows of it (the lengths are on the device): pieces per KV
// head are at most `target` + one for each row tile; row tiles that are split at most `target`,
// with at most 2 `target` pieces together (each has more steps than a piece, and the steps of all
// are at most `target` pieces long).
static bool plan_launch(const KvView &kv, int64_t total_q, int32_t q_heads, int64_t batch, int64_t max_pages,
                        int64_t max_q, int cus, Launch *L) {
  const int64_t G = q_heads / kv.heads, most_rows = max_q * G;
  // One token for each of 64 sequences (10 rows): 22.2 us with 16 rows a workgroup, 33.1 with 32. Three
  // for each of 16 sequences of 4000 keys (30 rows): 23.5 with 32, 32.6 in block_kernel. Three to eight for
  // each of 32 (80 rows): 32.6 in block_kernel, 209 with 96 rows in rows_kernel, which spills.
  L->nt = most_rows <= 16 ? 1 : most_rows <= 32 && kv.D <= 128 ? 2 : 8;
  const int64_t RT = 16 * L->nt;
  const int64_t by_seq = batch * ((most_rows + RT - 1) / RT), by_rows = total_q * G / RT + batch;
  const int64_t tiles = by_seq < by_rows ? by_seq : by_rows;
  // Two workgroups for each CU (64 ragged sequences, 262139 keys: 22.2 and 33.3 us; one: 24.7 and 37.2;
  // three: 24.7 and 35.8; four: 24.3 and 38.4); one where only one is resident (256 queries of 8 heads of 256
  // on 32000 keys: 146 us against 155, 32 drafted trees 69 against 74).
  const int wgs = L->nt == 8 && kv.D > 128 ? cus : 2 * cus;
  L->target = wgs / kv.heads > 0 ? wgs / kv.heads : 1;
  const int64_t steps = ((max_pages << kv.log_p) + kStep - 1) / kStep;
  // Up to 1024 keys are not worth splitting for rows_kernel, whose second launch costs the host 2 us (a
  // token on 731 keys: 10.5 us a call in one workgroup a head, 12.7 in pieces; one for each of 1024
  // sequences of 128 keys: 51.8, 71.7). The table's width stands for the keys: the lengths are on the device.
  if (steps > (L->nt < 8 ? 8 : 1)) {
    L->joins = tiles < L->target ? tiles : L->target;
    const int64_t most = tiles * steps, slots = 2 * (int64_t)L->target;
    L->slots = most < slots ? most : slots;
    L->units = most < L->target + tiles ? most : L->target + tiles;
  } else {
    L->joins = L->slots = 0;
    L->units = tiles;
  }
  // A workgroup of join_kernel takes eight rows (at D = 128) where there are many row tiles of few
  // pieces, two with four times as many pieces in flight where there are few of many (one sequence of
  // 8000 keys and 8 queries, 63 pieces: 21.2 us against 28.2; 32 drafted trees: 36.0 against 32.6).
  const int DP = kv.D <= 64 ? 64 : kv.D <= 128 ? 128 : 256;
  L->few = L->joins * kv.heads <= 32;
  const int in_join = L->nt < 8 ? 1 : (L->few ? 256 : 1024) / DP;
  L->rows = (int)(((most_rows < RT ? most_rows : RT) + in_join - 1) / in_join * in_join);
  return L->units * kv.heads < kMostWorkgroups && L->joins * RT * kv.heads <= kMostWorkgroups && steps * tiles <= 0x3FFFFFFF;
}

// Partial sums, (m, l), and the list of what is joined.
static size_t workspace_of(const KvView &kv, const Launch &L) {
  if (L.joins == 0) return 0;
  return (size_t)(L.slots * kv.heads * 16 * L.nt) * (kv.D + 2) * 4 + 16 * (size_t)(L.joins + 1);
}

static nvfp4_status check_sizes(const KvView &kv, int64_t total_q, int32_t q_heads, int64_t batch, int64_t max_pages,
                                int64_t max_q) {
  if (q_heads < 1 || q_heads > 65535 || q_heads % kv.heads != 0) return NVFP4_ERR_SHAPE;
  if (total_q < 0 || total_q > 0x3FFFFFFF / q_heads || batch < 0 || batch > (1 << 20) || max_q < 1 ||
      max_q > 0x7FFFFFFF)
    return NVFP4_ERR_SHAPE;
  // (key numbers are 32-bit, and run some tiles past the last key)
  if (max_pages < 0 || max_pages > (0x7FFFFFFF >> kv.log_p) - 64) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

template <int DP, int NT, int ROWS, bool F16>
static void launch_join(const AttnArgs &A, const Launch &L, hipStream_t s) {
  hipLaunchKernelGGL((join_kernel<DP, 16 * NT, ROWS, F16>), dim3((unsigned)(L.joins * A.kv.heads * (L.rows / ROWS))),
                     dim3(256), 0, s, A, L.rows / ROWS);
}

template <int DP, int NT, bool F16>
static void launch(const AttnArgs &A, const Launch &L, hipStream_t s) {
  const dim3 grid((unsigned)(L.units * A.kv.heads + (L.joins ? 1 : 0)));
  if constexpr (NT == 8) {
    hipLaunchKernelGGL((block_kernel<DP, F16>), grid, dim3(256), 0, s, A);
    if (L.joins && L.few) launch_join<DP, NT, 256 / DP, F16>(A, L, s);
    else if (L.joins) launch_join<DP, NT, 1024 / DP, F16>(A, L, s);
  } else {
    if (A.kv.D % (DP / 4) != 0) hipLaunchKernelGGL((rows_kernel<DP, NT, F16, true>), grid, dim3(256), 0, s, A);
    else hipLaunchKernelGGL((rows_kernel<DP, NT, F16, false>), grid, dim3(256), 0, s, A);
    if (L.joins) launch_join<DP, NT, 1, F16>(A, L, s);
  }
}

template <int DP>
static void launch_dim(const AttnArgs &A, const Launch &L, bool f16, hipStream_t s) {
  if (L.nt == 1) f16 ? launch<DP, 1, true>(A, L, s) : launch<DP, 1, false>(A, L, s);
  else if (L.nt == 8) f16 ? launch<DP, 8, true>(A, L, s) : launch<DP, 8, false>(A, L, s);
  else if constexpr (DP <= 128) f16 ? launch<DP, 2, true>(A, L, s) : launch<DP, 2, false>(A, L, s);
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

size_t nvfp4_kv_attention_workspace_bytes(const nvfp4_kv_cache *cache, int64_t total_q, int32_t q_heads, int64_t batch,
                                          int64_t max_pages, int64_t max_q) {
  KvView kv;
  Launch L;
  if (kv_view(cache, &kv) != NVFP4_OK || check_sizes(kv, total_q, q_heads, batch, max_pages, max_q) != NVFP4_OK) return 0;
  if (max_q > total_q) max_q = total_q > 0 ? total_q : 1;         // as the call does
  if (!plan_launch(kv, total_q, q_heads, batch, max_pages, max_q, device_cus_or_default(), &L)) return 0;
  return workspace_of(kv, L);
}

nvfp4_status nvfp4_kv_attention(const nvfp4_kv_cache *cache, nvfp4_rows q, int dtype, int64_t total_q, int32_t q_heads,
                                const int32_t *table, int64_t table_stride, int64_t max_pages, const int32_t *lens,
                                const int32_t *q_start, int64_t batch, int64_t max_q, const nvfp4_kv_mask *mask,
                                nvfp4_rows out, float *lse, void *ws, size_t ws_bytes, void *stream) {
  if (dtype != NVFP4_BF16 && dtype != NVFP4_F16) return NVFP4_ERR_DTYPE;
  AttnArgs A = {};
  nvfp4_status st = kv_view(cache, &A.kv);
  if (st != NVFP4_OK) return st;
  if ((st = check_sizes(A.kv, total_q, q_heads, batch, max_pages, max_q)) != NVFP4_OK) return st;
  if (batch > 1 && table_stride < max_pages) return NVFP4_ERR_SHAPE;
  if (!q_start && total_q != batch) return NVFP4_ERR_SHAPE;
  if (!mask) return NVFP4_ERR_NULL;
  if (!isfinite(mask->scale) || !(mask->scale > 0.0f)) return NVFP4_ERR_VALUE;
  if ((mask->causal != 0 && mask->causal != 1) || mask->window < 0) return NVFP4_ERR_VALUE;
  if (mask->window > 0 && (!mask->causal || mask->mask)) return NVFP4_ERR_VALUE;
  if (mask->mask && total_q > 1 && mask->mask_stride < max_q) return NVFP4_ERR_SHAPE;
  if (total_q == 0 || batch == 0) return NVFP4_OK;
  if (!q.base || !out.base || !lens || (!table && max_pages > 0)) return NVFP4_ERR_NULL;
  if (!kv_rows_aligned(q) || !kv_rows_aligned(out) || !aligned(lens, 4) || !aligned(table, 4) || !aligned(q_start, 4) ||
      !aligned(lse, 4))
    return NVFP4_ERR_ALIGN;
  if (max_q > total_q) max_q = total_q;
  DeviceInfo d;
  const nvfp4_status on_device = device_info(&d);       // (asked once; arguments are checked without a device too)
  Launch L;
  if (!plan_launch(A.kv, total_q, q_heads, batch, max_pages, max_q, on_device == NVFP4_OK ? d.num_cus : 256, &L))
    return NVFP4_ERR_SHAPE;
  const size_t need = workspace_of(A.kv, L);
  if (need > 0 && (!ws || ws_bytes < need)) return NVFP4_ERR_WORKSPACE;
  if (need > 0 && !aligned(ws, 16)) return NVFP4_ERR_ALIGN;
  if (on_device != NVFP4_OK) return on_device;
  A.q = (const uint16_t *)q.base, A.q_t = q.token_stride, A.q_h = q.head_stride;
  A.out = (uint16_t *)out.base, A.o_t = out.token_stride, A.o_h = out.head_stride;
  A.lse = lse;
  A.total_q = total_q;
  A.table = table, A.table_stride = table_stride, A.max_pages = (int32_t)max_pages;
  A.lens = lens, A.q_start = q_start;
  A.mask = mask->mask, A.mask_stride = mask->mask_stride;
  A.scale = mask->scale;
  A.causal = mask->causal;
  // (a window as long as a sequence can be hides nothing)
  A.window = mask->window >= max_pages << A.kv.log_p ? 0 : (int32_t)mask->window;
  A.batch = (int32_t)batch, A.max_q = (int32_t)max_q;
  A.group = q_heads / A.kv.heads;
  A.target = L.target;
  A.slots = (int32_t)L.slots;
  A.part_o = (float *)ws;
  const int64_t part_rows = L.slots * A.kv.heads * 16 * L.nt;
  A.part_ml = A.part_o + part_rows * A.kv.D;
  A.join_count = (int32_t *)(A.part_ml + 2 * part_rows);
  A.joins_at = A.join_count + 4;
  A.joins = (int32_t)L.joins;
  const bool f16 = dtype == NVFP4_F16;
  if (A.kv.D <= 64) launch_dim<64>(A, L, f16, (hipStream_t)stream);
  else if (A.kv.D <= 128) launch_dim<128>(A, L, f16, (hipStream_t)stream);
  else launch_dim<256>(A, L, f16, (hipStream_t)stream);
  NVFP4_LAUNCH_CHECK();
  return NVFP4_OK;
}

}  // extern "C"
