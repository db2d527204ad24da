// What the attention kernels share (attn_tile.hip: many query rows against
// shared key tiles; attn_wave.hip: few query rows, each wave its own keys).
//
// Rows.  A kv head's query rows of a sequence are (new token, query head of
// the group): row r is token r / G, head r % G, G = n_heads / n_kv_heads.  A
// key tile then serves all G heads at once.  Over selected tokens the rows
// of a unit are one token's G heads.
//
// Both kernels form S^T = K Q^T, so a lane of the result holds one query row's
// scores (16 or 8 of a tile's keys): the softmax needs almost no lane
// exchange, the output's rescaling is one factor per lane, and the weights
// are already laid out as the second operand of O^T = V^T P^T, up to an order
// of the keys that V's reads follow.
//
// LDS tiles hold bf16 rows in 16-byte pieces, piece c of row r at position
// c ^ swizzle(r): K rows are then read 16 at a time, and V four rows at a time
// by gfx950's transposing read, without more lanes per bank than the read's
// size needs.
#pragma once

#include <math.h>

#include "misa_common.h"
#include "misa_launch.h"

namespace misa {

constexpr float kLn2 = 0.6931471805599453f;
// The outputs are rescaled only when a row's maximum has grown by more than this
// (log2) since the last time: weights stay below 2^8, well inside bf16 and fp32.
constexpr float kGrow = 8.f;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_void;
typedef const __attribute__((address_space(1))) void* global_void;

// piece position of row r (D elements a row, D / 8 pieces)
template <int D>
__device__ __forceinline__ int swizzle(int r) {
  return D == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
}

// gfx950's transposing LDS read: lanes 4j .. 4j+3 of a 16-lane group name 4
// consecutive elements each of row j (j = 0..3); lane i of the group receives
// element i of the four rows.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 lds_read_tr(const unsigned char* p) {
  typedef __attribute__((address_space(3))) s16x4* ptr;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)p));
}

// The same for bytes: lanes 2j, 2j + 1 name 8 consecutive bytes each of row j (j =
// 0..7); lane i receives byte i of the eight rows.
__device__ __forceinline__ uint2 lds_read_tr8(const unsigned char* p) {
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) i32x2* ptr;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((ptr)p));
}

// 16 bytes a lane, global -> LDS (dst: the wave's 1 KB, lane order)
__device__ __forceinline__ void load_lds16(const void* src, unsigned char* dst) {
  __builtin_amdgcn_global_load_lds((global_void)src, (lds_void)dst, 16, 0, 0);
}

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

// max over the two halves of a wave / over its four 16-lane rows
__device__ __forceinline__ float max_halves(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float max_rows(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max_halves(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
}
__device__ __forceinline__ float sum_halves(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

// Entry of the block table for token t of sequence b (entries clamped, see
// misa_kv_pages), and the pool row it makes
__device__ __forceinline__ int table_entry(const AttnArgs& a, int b, int t) {
  const uint32_t p = a.page_shift >= 0 ? (uint32_t)t >> a.page_shift : (uint32_t)t / (uint32_t)a.page_keys;
  return a.table[(int64_t)b * a.max_pages + p];
}
__device__ __forceinline__ int pool_row(const AttnArgs& a, int entry, int t) {
  const uint32_t in = a.page_shift >= 0 ? (uint32_t)t & (uint32_t)(a.page_keys - 1) : (uint32_t)t % (uint32_t)a.page_keys;
  const int e = min(max(entry, 0), a.n_pages - 1);
  return e * a.page_keys + (int)in;   // below 2^31: the ABI bounds the pool
}

// Sequence b's new tokens t0 .. t0+m-1 (m: those within n_tokens), the position
// of the first, and its readable length.
struct SeqSpan {
  int t0, m;
  int64_t pos0;
  int len;
};
__device__ __forceinline__ SeqSpan make_span(const AttnArgs& a, int64_t s, int64_t e, int kv_len) {
  const int64_t n = a.n_tokens;
  const int64_t kv = max(kv_len, 0);
  SeqSpan r;
  const int64_t t0 = min(max(s, (int64_t)0), n);
  r.t0 = (int)t0;
  r.m = (int)max((int64_t)0, min(e, n) - t0);
  r.pos0 = kv - (e - s);
  r.len = (int)min(kv, a.max_pages * a.page_keys);
  return r;
}
__device__ __forceinline__ SeqSpan seq_span(const AttnArgs& a, int b) {
  return make_span(a, a.q_start[b], a.q_start[b + 1], a.kv_lens[b]);
}

// The sequence of token t, its span, or false where t is no sequence's token.
// Up to 64 sequences are looked over in one go, so that the search and the
// span's own loads are one trip to memory; more are narrowed 64-fold at a time.
// Uniform.
__device__ __forceinline__ bool seq_of_token(const AttnArgs& a, int64_t t, int lane, int* b_out, SeqSpan* out) {
  int lo = 0, n = a.n_seq;   // the answer is in [lo, lo + n)
  while (n > kWave) {
    const int step = (n + kWave - 1) / kWave;
    const int at = lo + min(lane * step, n - 1);
    const uint64_t m = __ballot(lane * step < n && a.q_start[at] <= t);
    const int j = 63 - (int)__builtin_clzll(m | 1);   // last probe at or before t
    n = min(step, n - j * step);
    lo += j * step;
  }
  const int b = lo + min(lane, n - 1);
  const int64_t s = a.q_start[b], e = a.q_start[b + 1];
  const int kv = a.kv_lens[b];
  const uint64_t m = __ballot(lane < n && s <= t && t < e);
  if (m == 0) return false;
  const int src = (int)__builtin_ctzll(m);
  const int64_t s0 = __builtin_amdgcn_readlane((int)s, src), e0 = __builtin_amdgcn_readlane((int)e, src);
  *b_out = lo + src;
  *out = make_span(a, s0, e0, __builtin_amdgcn_readlane(kv, src));
  return true;
}

// Entry j of token t's list, -1 behind its end (always one load: a load behind
// a branch makes the compiler wait for everything under way)
__device__ __forceinline__ int pick(const AttnArgs& a, int64_t t, int j) {
  const int v = a.idx[t * a.topk + min(j, a.topk - 1)];
  return j < a.topk ? v : -1;
}

// -scale is folded into the sign of q, so that a maximum of scores is a maximum
// of scaled scores
__device__ __forceinline__ bf16x8 load_q(const uint16_t* p, uint32_t flip) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  return as_bf16x8(make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip));
}

// Workgroups of attn_wave that a CU holds, and so waves of a SIMD: what the LDS
// lets in over bf16 pages (128 KB of tiles at head_dim 128), the registers over
// e4m3 pages.  With 32 rows of 128 two waves spill some registers: over selected
// tokens, bound by the vector unit, they are better all the same (1000 x 2048
// picks, 64 / 2 heads: 196 us, alone 246), in decodes one is (64 of 8..16K keys:
// 119 us, with two 133).
constexpr int wave_groups(int D, bool fp8, bool sel, int RT) {
  if (!fp8) return D == 64 ? 2 : 1;
  if (D == 64) return RT == 1 ? 3 : 2;
  return sel || RT == 1 ? 2 : 1;
}

// What a launch adds to the arguments
struct AttnLaunch {
  int n_units;      // row tiles (attn_tile), or sequences / tokens (attn_wave)
  int n_splits;     // key splits of a unit, at most
  int slots;        // workgroups that the GPU holds at a time
  int rows_min;     // dense: attn_tile takes sequences with more rows than this, attn_wave the others
  int rows;         // of a unit, at most
  // n_splits > 1: unnormalised outputs [D], and (maximum, sum), of every row and
  // split.  Dense: [kv head][part_rows x n_splits], where a unit has the places
  // that its rows have in the batch (packed: row r of first token t is t G + r), or
  // `rows` of its own, whichever takes less: padded units cost nothing, nor do
  // rows that are the other kernel's.
  int packed;
  int64_t part_rows;
  float* part_o;
  float2* part_ml;
  // dense: where a unit's rows are, for the join: (first token, first row, rows in all, splits in use)
  int4* unit_info;
};

// Where a unit's part for kv head g begins, and what is between its splits (in
// rows): the splits of a unit are side by side, as the join reads them.  Selected:
// units have as many rows each and stand in their order (placed by the batch's
// rows like the others, 64 tokens x 64 heads took 22.2 us instead of 21.8).
struct PartPlace {
  int64_t begin;
  int step;
};
template <bool SEL>
__device__ __forceinline__ PartPlace part_place(const AttnLaunch& L, int kv_heads, int G, int rows, int g, int unit,
                                                int tok0, int r0, int nrows) {
  if (SEL) return PartPlace{((int64_t)unit * kv_heads + g) * L.n_splits * rows, rows};
  return PartPlace{(g * L.part_rows + (L.packed ? (int64_t)tok0 * G + r0 : (int64_t)unit * rows)) * L.n_splits,
                   min(rows, nrows - r0)};
}

// What a dense launch's lengths are, for one kv head, and the split made of them
struct DenseScan {
  float steps;   // key tiles of all units together
  int units;
  int longest;   // key tiles of one unit, at most
  int per;       // key tiles of a split (0: not scanned)
};

// Key tiles of a split.  Lengths differ within a batch, and a unit's share of the
// splits should follow its own, so all splits are about equally long.
//
// attn_wave, bound by the card's reading: two splits to each workgroup that the
// GPU holds.  No splits where the units are one full round of nearly equal
// length (they would only add rounds), or so many that they balance by
// themselves.
__device__ __forceinline__ int wave_per(const DenseScan& w, const AttnLaunch& L, int kv_heads) {
  const float fair = w.steps * (float)kv_heads / (float)L.slots;
  const float units = (float)w.units * (float)kv_heads;
  int p = max(16, (int)ceilf(fair * 0.5f));
  if (((float)w.longest <= 1.25f * fair && units <= 1.05f * (float)L.slots) || units >= 6.f * (float)L.slots)
    p = max(p, w.longest);
  return p;
}

// attn_tile, bound by each CU's own arithmetic: what counts is the CU with the
// most tiles.  Some ways of cutting the longest unit are weighed, in tiles of a
// CU: splits of p tiles make g workgroups, of which a CU gets ceil(g / 256), and
// works at less than its full rate where fewer of them are resident than it
// holds; a start costs about 2.5 us (1.6 tiles at head_dim 128, 4 at 64), and a
// split's part is written, read and joined, about a hundredth of a tile of every
// CU's time.  g is exact where the units are about equally long (one chunk, a
// batch of equal ones); else the remainders count as half a split a unit, and
// the CUs even out but for half a split.
constexpr int kCuts = 9;
template <int D>
__device__ __forceinline__ int tile_per(const DenseScan& w, const AttnLaunch& L, int kv_heads) {
  constexpr int cut[kCuts] = {1, 2, 3, 4, 5, 6, 8, 14, 32};
  constexpr float start = D == 64 ? 4.f : 1.6f, cus = 256.f, held = D == 64 ? 3.f : 2.f;
  constexpr float one = D == 64 ? 1 / 0.45f : 1 / 0.7f, two = D == 64 ? 2 / 0.8f : 2.f;   // tiles' time beside 1, 2
  const int least = max(8, (w.longest + L.n_splits - 1) / L.n_splits);
  const float heads = (float)kv_heads, longest = (float)w.longest, units = (float)w.units * heads;
  const float fair = w.steps * heads / cus;
  const bool alike = w.steps > 0.9f * (float)w.units * longest;
  float best = longest, lowest = INFINITY;
#pragma unroll
  for (int j = 0; j < kCuts; ++j) {
    const float per = fminf(longest, fmaxf((float)least, ceilf(longest * (1.f / cut[j]) - 1e-3f)));
    const float inv = 1.f / fmaxf(per, 1.f);
    float g, cost;
    if (alike) {
      g = units * ceilf(longest * inv - 1e-3f);
      const float m = ceilf(g * (1.f / cus)), full = held * floorf(m * (1.f / held) + 1e-3f), rest = m - full;
      cost = (full + (rest < 0.5f ? 0.f : rest < 1.5f ? one : two)) * (per + start);
    } else {
      g = j == 0 ? units : w.steps * heads * inv + 0.5f * units;
      cost = fmaxf(fair + g * (start / cus) + 0.5f * per, one * (per + start));
    }
    if (per < longest) cost += g * 0.01f + start;
    if (cost < lowest) {
      lowest = cost;
      best = per;
    }
  }
  return __builtin_amdgcn_readfirstlane((int)best);
}

// Key tiles of each of a unit's splits (the last may have fewer), n in all
__device__ __forceinline__ int split_tiles(const DenseScan& w, const AttnLaunch& L, int n, int* in_use) {
  int per = n;
  if (L.n_splits > 1) per = max(w.per, (n + L.n_splits - 1) / L.n_splits);   // no scan: even shares
  per = max(per, 1);
  *in_use = max(1, (n + per - 1) / per);
  return per;
}

// Up to this many sequences a workgroup sums them all; more share their splits evenly
constexpr int kScanSeqs = 4096;

// Dense units.  TILES: row tiles of BM rows, numbered over the sequences with
// more than rows_min rows; finds unit's sequence, span and first row (false: no
// such tile).  Else unit is the sequence (false: not attn_wave's).  Fills
// `scan` over the sequences of the launch's kind where splits need it.
// Uniform.
template <bool TILES, int KEYS, int D>
__device__ __forceinline__ bool find_unit(const AttnArgs& a, const AttnLaunch& L, int G, int BM, int unit, int lane,
                                          SeqSpan* span, int* b_out, int* r0_out, DenseScan* scan) {
  const bool sums = L.n_splits > 1 && a.n_seq <= kScanSeqs;
  bool found = false;
  int64_t base = 0;
  float steps = 0.f;
  int longest = 0, units = 0;
  const int first = TILES || sums ? 0 : unit / 256 * 256;
  for (int b0 = first; b0 < a.n_seq; b0 += 256) {
    int c[4], sum = 0, s[5], kv[4];
#pragma unroll
    for (int i = 0; i < 5; ++i) s[i] = a.q_start[min(b0 + lane * 4 + i, a.n_seq)];
#pragma unroll
    for (int i = 0; i < 4; ++i) kv[i] = a.kv_lens[min(b0 + lane * 4 + i, a.n_seq - 1)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const SeqSpan sp = make_span(a, s[i], s[i + 1], kv[i]);
      const int64_t rows = (int64_t)sp.m * G;
      const bool in = b0 + lane * 4 + i < a.n_seq && rows > 0 && (rows > L.rows_min) == TILES;
      c[i] = in ? (TILES ? (int)((rows + BM - 1) / BM) : 1) : 0;
      sum += c[i];
      const int n = in ? (sp.len + KEYS - 1) / KEYS : 0;
      steps += (float)c[i] * (float)n;
      longest = max(longest, n);
    }
    units += sum;
    int src = -1, i = 0, left = 0;
    if (TILES) {
      int inc = sum;
#pragma unroll
      for (int o = 1; o < kWave; o <<= 1) {
        const int x = __shfl_up(inc, o);
        if (lane >= o) inc += x;
      }
      const int total = __builtin_amdgcn_readlane(inc, 63);
      if (!found && unit < base + total) {
        const int rel = (int)(unit - base);
        src = (int)__builtin_ctzll(__ballot(inc > rel));
        left = rel - (inc - sum);   // valid on lane src
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (i == k && left >= c[k]) {
            left -= c[k];
            i = k + 1;
          }
        i = __builtin_amdgcn_readlane(i, src);
        left = __builtin_amdgcn_readlane(left, src);
      }
      base += total;
    } else if (unit >= b0 && unit < b0 + 256) {
      src = (unit - b0) / 4;
      i = (unit - b0) % 4;
      // not ours?  (c is 0 there)
      int ci = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i == k) ci = c[k];
      if (__builtin_amdgcn_readlane(ci, src) == 0) return false;
    }
    if (src >= 0) {
      int si = 0, ei = 0, ki = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i == k) {
          si = s[k];
          ei = s[k + 1];
          ki = kv[k];
        }
      *span = make_span(a, __builtin_amdgcn_readlane(si, src), __builtin_amdgcn_readlane(ei, src),
                        __builtin_amdgcn_readlane(ki, src));
      *b_out = b0 + src * 4 + i;
      *r0_out = left * BM;
      found = true;
    }
    if (found && !sums) break;
  }
  if (!found) return false;
  if (sums) {
#pragma unroll
    for (int x = 32; x >= 1; x >>= 1) {
      steps += __shfl_xor(steps, x);
      longest = max(longest, __shfl_xor(longest, x));
      units += __shfl_xor(units, x);
    }
    *scan = DenseScan{steps, units, longest, 0};
    scan->per = TILES ? tile_per<D>(*scan, L, a.n_kv_heads) : wave_per(*scan, L, a.n_kv_heads);
  } else {
    *scan = DenseScan{0.f, 0, 0, 0};
  }
  return true;
}

// Workgroup -> (unit, kv head, split).  Workgroup i runs on XCD i mod 8, and the
// units of one (kv head, split) read the same keys: where there are a
// multiple of 8 such pairs, each goes to one XCD, whose L2 then holds the keys
// for all its units; else neighbours go round the XCDs.  Where an XCD would get
// some splits only, of which a dense unit uses the first ones, the pairs move on
// an XCD every 2^turn units, so that all XCDs get as many splits in use (8 x 256
// tokens over 2700 keys, 20 / 4 heads of 128, three of four splits in use: 117 -> 98
// us).
struct Place {
  int unit, g, split;
};
__device__ __forceinline__ Place place_of(const AttnLaunch& L, int kv_heads, uint32_t i, int turn) {
  const uint32_t n = (uint32_t)L.n_units, pairs = (uint32_t)(kv_heads * L.n_splits);
  uint32_t pair, unit;
  if (pairs % 8 == 0) {
    const uint32_t j = i / 8;
    unit = j % n;
    pair = 8 * (j / n) + ((i + (kv_heads % 8 == 0 ? 0 : unit >> turn)) & 7);
  } else {
    pair = i / n;
    unit = i % n;
  }
  return Place{(int)unit, (int)(pair % (uint32_t)kv_heads), (int)(pair / (uint32_t)kv_heads)};
}

}  // namespace misa
