// Host side of the attention calls: which kernel takes which rows, how the keys
// are split, and the workspace the splits need.
//
// The lengths live on the GPU, so the plan is made from what the host knows:
// the tokens, the heads, the table's width and the caller's bound on a
// sequence's new tokens.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_device.h"

namespace misa {

hipError_t launch_attn_tile(const AttnArgs& a, const AttnLaunch& L, int D, bool fp8, int NW, bool halves, hipStream_t st);
hipError_t launch_attn_wave(const AttnArgs& a, const AttnLaunch& L, int D, bool fp8, int RT, hipStream_t st);

namespace {

// The joins of a call's launches in one: workgroups below n_tile join
// attn_tile's units (BM rows each), the others attn_wave's (16 RT rows).  D / 4
// lanes take a row, 16 bytes of every split each, and go through the splits four
// or eight at a time with a running maximum: each lane forms the row's weights
// by itself, so lanes exchange nothing.  (46k rows of two to four splits: 6 us;
// splits side by side on lanes that then sum by shuffles took 16.)
template <int D, bool SEL>
__global__ void __launch_bounds__(256) k_attn_join(const AttnArgs a, const AttnLaunch tile, const AttnLaunch wave,
                                                   uint32_t n_tile) {
  constexpr int LR = D / 4, RW = 256 / LR;   // lanes of a row, rows of a workgroup
  const bool is_tile = blockIdx.x < n_tile;
  const AttnLaunch& S = is_tile ? tile : wave;
  const uint32_t i = is_tile ? blockIdx.x : blockIdx.x - n_tile;
  const int G = a.n_heads / a.n_kv_heads;
  const uint32_t per = (uint32_t)S.rows / RW;   // workgroups of a unit and kv head
  // attn_tile's parts lie as pieces of 16 bytes, [piece][row], attn_wave's as rows
  const int rr = (int)(i % per) * RW + (is_tile ? (int)threadIdx.x % RW : (int)threadIdx.x / LR);
  const int piece = is_tile ? (int)threadIdx.x / RW : (int)threadIdx.x % LR;
  const int g = (int)(i / per % (uint32_t)a.n_kv_heads), unit = (int)(i / per / (uint32_t)a.n_kv_heads);
  int r0, nrows, tok0, n = S.n_splits;
  if (SEL) {
    const int sub = is_tile ? (G + S.rows - 1) / S.rows : 1;
    tok0 = unit / sub;
    r0 = (unit % sub) * S.rows;
    if (tok0 >= a.q_start[a.n_seq] || tok0 < a.q_start[0]) return;   // no sequence's token: nothing was written
    nrows = G;
  } else {
    const int4 u = S.unit_info[unit];
    tok0 = u.x;
    r0 = u.y;
    nrows = u.z;
    n = u.w;
  }
  const int r = r0 + rr;
  if (n <= 1 || r >= nrows) return;   // written by the unit itself, or no row
  const PartPlace part = part_place<SEL>(S, a.n_kv_heads, G, S.rows, g, unit, tok0, r0, nrows);
  const int64_t pr = part.begin + rr;
  const float2* const ml = S.part_ml + pr;
  const float* const po = S.part_o + (is_tile ? part.begin * D + (piece * part.step + rr) * 4 : pr * D + piece * 4);
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  float top = -INFINITY, sum = 0.f;
  auto some = [&](int s0, auto count) __attribute__((always_inline)) {
    constexpr int U = decltype(count)::value;
    float2 x[U];
    f32x4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) x[k] = ml[(int64_t)min(s0 + k, n - 1) * part.step];
#pragma unroll
    for (int k = 0; k < U; ++k) v[k] = *reinterpret_cast<const f32x4*>(po + (int64_t)min(s0 + k, n - 1) * part.step * D);
    float most = top;
#pragma unroll
    for (int k = 0; k < U; ++k) most = fmaxf(most, x[k].y != 0.f ? x[k].x : -INFINITY);
    const float keep = top == -INFINITY ? 0.f : exp2_raw(top - most);   // (nothing to keep before the first)
    top = most;
    o *= keep;
    sum *= keep;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      // An empty split wrote no output: whatever is there is not used.  Any other
      // takes part however little it weighs, so that its NaN shows.
      const bool in = s0 + k < n && x[k].y != 0.f;
      const float w = exp2_raw(x[k].x - most);
      sum = in ? __builtin_fmaf(w, x[k].y, sum) : sum;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = in ? __builtin_fmaf(w, v[k][e], o[e]) : o[e];
    }
  };
  if (n <= 4)
    some(0, std::integral_constant<int, 4>{});
  else
    for (int s0 = 0; s0 < n; s0 += 8) some(s0, std::integral_constant<int, 8>{});
  const int qi = SEL ? 0 : r / G, qh = g * G + (SEL ? r : r - qi * G);
  const int64_t out_row = ((int64_t)tok0 + qi) * a.n_heads + qh;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  *reinterpret_cast<uint2*>(a.out + out_row * D + piece * 4) =
      make_uint2(pk_bf16(o[0] * inv, o[1] * inv), pk_bf16(o[2] * inv, o[3] * inv));
  if (a.lse != nullptr && piece == 0) a.lse[out_row] = sum != 0.f ? (top + __log2f(sum)) * kLn2 : -INFINITY;
}

struct AttnPlan {
  int RT = 0, wave_units = 0, wave_splits = 1, wave_slots = 0;   // RT = 0: attn_wave does not run
  int NW = 0, tile_units = 0, tile_splits = 1, tile_slots = 0;   // NW = 0: attn_tile does not run
  int BM = 0;            // rows of an attn_tile unit
  bool halves = false;   // its waves: two for each 32 rows
  int rows_min = 0;
  int64_t wave_part = 0, tile_part = 0;   // rows of a kv head's part, a split
  size_t wave_o = 0, wave_ml = 0, wave_info = 0, tile_o = 0, tile_ml = 0, tile_info = 0, total = 0;
  int64_t groups = 0;   // workgroups of the larger launch
};

inline size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// Key splits of `units` workgroups that walk `steps` tiles each, `slots` of them
// resident.
// Selected tokens (exact): units are all alike, so the splits are those of the
// least rounds of workgroups times a round's length, which is its share of the
// tiles and about 4 tiles' time to start, plus the join, which reads every
// split's rows again.
// Dense: the lengths are known to the GPU only, which decides how many of the
// splits a unit uses (split_tiles); this is the bound, two to a slot, by the
// widest the table allows.
int choose_splits(int64_t units, int64_t slots, int64_t steps, int most, bool exact) {
  if (!exact) {
    const int64_t s = units >= 2 * slots ? 1 : (2 * slots + units - 1) / units;
    return (int)std::max<int64_t>(1, std::min<int64_t>({s, most, steps / 4}));
  }
  int best = 1;
  double least = 0;
  for (int s = 1; s <= most && (s == 1 || steps / s >= 2); ++s) {
    const double rounds = (double)((units * s + slots - 1) / slots);
    const double cost = rounds * ((double)((steps + s - 1) / s) + 4.0) + (s > 1 ? 4.0 + (double)(units * s) / 1024 : 0.0);
    if (s == 1 || cost < 0.95 * least) {   // (a split more has to earn its workspace)
      best = s;
      least = cost;
    }
  }
  return best;
}

AttnPlan make_plan(const misa_attn_shape& s, const misa_kv_pages& pg, int topk, bool tree) {
  AttnPlan p;
  const int64_t G = s.n_heads / s.n_kv_heads, T = s.n_tokens, KH = s.n_kv_heads;
  const int64_t ctx = topk > 0 ? topk : pg.max_pages * pg.page_keys;
  if (T == 0) return p;
  int64_t wave_units = 0, tile_units = 0;
  if (topk > 0) {
    if (G <= 32) {
      p.RT = G <= 16 ? 1 : 2;
      wave_units = T;
    } else {
      p.NW = G <= 64 ? 2 : 4;
      p.BM = p.NW * 32;
      tile_units = T * ((G + p.BM - 1) / p.BM);
    }
  } else {
    const int64_t new_max = s.max_new > 0 ? std::min<int64_t>(s.max_new, T) : T;
    const int64_t rows = new_max * G;
    if (rows <= 32) {
      p.RT = rows <= 16 ? 1 : 2;
    } else {
      // one sequence of many rows needs attn_tile alone
      if (s.n_seq > 1 && G <= 32) p.RT = G <= 16 ? 1 : 2;
      p.halves = tree && rows <= 64;   // (a chunk keeps its two waves, and with them the order of its sums)
      p.NW = rows <= 64 && !p.halves ? 2 : 4;
      p.BM = p.halves ? 64 : p.NW * 32;
    }
    p.rows_min = 16 * p.RT;
    if (p.RT > 0) wave_units = s.n_seq;
    if (p.NW > 0) {
      // n sequences with rows r: sum ceil(r / BM) = sum floor((r - 1) / BM) + n, at most.  (A workgroup without rows
      // ends at once, but the one dispatched after it shares a CU: one unit too many of three cost 64 tokens over 8192 keys
      // 32.1 us instead of 26.7.)
      const int64_t n = std::min<int64_t>(s.n_seq, T * G / (p.rows_min + 1));
      tile_units = (T * G - n) / p.BM + n;
    }
  }
  p.groups = std::max(wave_units, tile_units) * KH;
  if (p.groups > ((int64_t)1 << 23)) return p;   // refused by the caller
  p.wave_units = (int)wave_units;
  p.tile_units = (int)tile_units;
  if (p.RT > 0) {
    p.wave_slots = 256 * wave_groups(s.head_dim, pg.kdtype == MISA_K_FP8_E4M3, topk > 0, p.RT);
    p.wave_splits = choose_splits(wave_units * KH, p.wave_slots, (ctx + 127) / 128, 64, topk > 0);
  }
  if (p.NW > 0) {
    const int64_t BM = p.BM;
    const int64_t est = topk > 0 ? tile_units : (T * G + BM - 1) / BM;
    p.tile_slots = s.head_dim == 64 ? 768 : 512;   // LDS, and registers at head_dim 64
    p.tile_splits = choose_splits(est * KH, p.tile_slots, (ctx + 63) / 64, 32, topk > 0);
  }
  p.groups = std::max(wave_units * p.wave_splits, tile_units * p.tile_splits) * KH;
  size_t off = 0;
  // (see AttnLaunch)
  p.wave_part = (int64_t)p.wave_units * 16 * p.RT;
  p.tile_part = (int64_t)p.tile_units * p.BM;
  if (topk == 0) {
    p.wave_part = std::min<int64_t>(T * G, p.wave_part);
    p.tile_part = std::min<int64_t>(T * G, p.tile_part);
  }
  if (p.RT > 0 && p.wave_splits > 1) {
    const size_t rows = (size_t)p.wave_part * KH * p.wave_splits;
    p.wave_o = off;
    off += align_up(rows * s.head_dim * sizeof(float));
    p.wave_ml = off;
    off += align_up(rows * sizeof(float2));
    p.wave_info = off;
    off += align_up((size_t)p.wave_units * sizeof(int4));
  }
  if (p.NW > 0 && p.tile_splits > 1) {
    const size_t rows = (size_t)p.tile_part * KH * p.tile_splits;
    p.tile_o = off;
    off += align_up(rows * s.head_dim * sizeof(float));
    p.tile_ml = off;
    off += align_up(rows * sizeof(float2));
    p.tile_info = off;
    off += align_up((size_t)p.tile_units * sizeof(int4));
  }
  p.total = off;
  return p;
}

}  // namespace

bool attn_fits(const misa_attn_shape& s, const misa_kv_pages& pg, int topk, bool tree) {
  return make_plan(s, pg, topk, tree).groups <= ((int64_t)1 << 23);
}

size_t attn_workspace_bytes(const misa_attn_shape& s, const misa_kv_pages& pg, int topk, bool tree) {
  return make_plan(s, pg, topk, tree).total;
}

hipError_t launch_attention(const misa_attn_shape& s, const misa_kv_pages& pg, const uint16_t* q,
                            const int32_t* q_start, const int32_t* kv_lens, const int32_t* idx, int topk,
                            const uint32_t* tree, int tree_words, uint16_t* out, float* lse, void* ws, hipStream_t st) {
  const AttnPlan p = make_plan(s, pg, topk, tree != nullptr);
  const bool pow2 = (pg.page_keys & (pg.page_keys - 1)) == 0;
  const AttnArgs a{q, s.q_stride_token, s.q_stride_head, pg.k, pg.v, pg.k_scale, pg.v_scale, pg.block_table,
                   pg.max_pages, (int)pg.n_pages, pg.page_keys, pow2 ? __builtin_ctz((unsigned)pg.page_keys) : -1, q_start,
                   kv_lens, idx, topk, out, lse, s.scale * 1.4426950408889634f, s.n_seq, s.n_heads, s.n_kv_heads,
                   s.n_tokens, tree, tree_words};
  const bool fp8 = pg.kdtype == MISA_K_FP8_E4M3;
  char* base = static_cast<char*>(ws);
  const int64_t all = s.n_tokens * (s.n_heads / s.n_kv_heads);   // rows of a kv head
  const AttnLaunch T{p.tile_units, p.tile_splits, p.tile_slots, p.rows_min, p.BM, p.tile_part == all, p.tile_part,
                     reinterpret_cast<float*>(base + p.tile_o), reinterpret_cast<float2*>(base + p.tile_ml),
                     reinterpret_cast<int4*>(base + p.tile_info)};
  const AttnLaunch W{p.wave_units, p.wave_splits, p.wave_slots, p.rows_min, 16 * p.RT, p.wave_part == all, p.wave_part,
                     reinterpret_cast<float*>(base + p.wave_o), reinterpret_cast<float2*>(base + p.wave_ml),
                     reinterpret_cast<int4*>(base + p.wave_info)};
  hipError_t e = hipSuccess;
  if (p.NW > 0) e = launch_attn_tile(a, T, s.head_dim, fp8, p.NW, p.halves, st);
  if (e == hipSuccess && p.RT > 0) e = launch_attn_wave(a, W, s.head_dim, fp8, p.RT, st);
  const int lanes = s.head_dim / 4;   // of a row
  const int64_t n_tile = p.NW > 0 && p.tile_splits > 1 ? (int64_t)p.tile_units * s.n_kv_heads * p.BM * lanes / 256 : 0;
  const int64_t n_wave = p.RT > 0 && p.wave_splits > 1 ? (int64_t)p.wave_units * s.n_kv_heads * p.RT * 16 * lanes / 256 : 0;
  if (e != hipSuccess || n_tile + n_wave == 0) return e;
  const dim3 grid((unsigned)(n_tile + n_wave));
  const uint32_t nt = (uint32_t)n_tile;
  const bool sel = idx != nullptr;
  if (s.head_dim == 128) {
    if (sel) hipLaunchKernelGGL((k_attn_join<128, true>), grid, dim3(256), 0, st, a, T, W, nt);
    else hipLaunchKernelGGL((k_attn_join<128, false>), grid, dim3(256), 0, st, a, T, W, nt);
  } else {
    if (sel) hipLaunchKernelGGL((k_attn_join<64, true>), grid, dim3(256), 0, st, a, T, W, nt);
    else hipLaunchKernelGGL((k_attn_join<64, false>), grid, dim3(256), 0, st, a, T, W, nt);
  }
  return hipGetLastError();
}

}  // namespace misa
