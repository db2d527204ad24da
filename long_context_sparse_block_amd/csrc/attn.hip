// Host side of the attention calls: which kernel takes which rows, how the keys
// are split, and the workspace the splits need.
//
// The lengths live on the GPU, so the plan is made from what the host knows:
// the tokens, the heads, the table's width and the caller's bound on a
// sequence's new tokens.
#include <algorithm>
#include <cmath>

#include "attn_device.h"

namespace misa {

hipError_t launch_attn_tile(const AttnArgs& a, const AttnLaunch& L, int D, bool fp8, int NW, hipStream_t st);
hipError_t launch_attn_wave(const AttnArgs& a, const AttnLaunch& L, int D, bool fp8, int RT, hipStream_t st);

namespace {

struct AttnPlan {
  int RT = 0, wave_units = 0, wave_splits = 1, wave_slots = 0;   // RT = 0: attn_wave does not run
  int NW = 0, tile_units = 0, tile_splits = 1, tile_slots = 0;   // NW = 0: attn_tile does not run
  int rows_min = 0;
  size_t wave_o = 0, wave_ml = 0, tile_o = 0, tile_ml = 0, tile_info = 0, total = 0;
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
// splits a unit uses (split_tiles); this is the bound, three to a slot, by the
// widest the table allows.
int choose_splits(int64_t units, int64_t slots, int64_t steps, int most, bool exact) {
  if (!exact) {
    const int64_t s = units >= 3 * slots ? 1 : (3 * slots + units - 1) / units;
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

AttnPlan make_plan(const misa_attn_shape& s, const misa_kv_pages& pg, int topk) {
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
      tile_units = T * ((G + p.NW * 32 - 1) / (p.NW * 32));
    }
  } else {
    const int64_t new_max = s.max_new > 0 ? std::min<int64_t>(s.max_new, T) : T;
    const int64_t rows = new_max * G;
    if (rows <= 32) {
      p.RT = rows <= 16 ? 1 : 2;
    } else {
      // one sequence of many rows needs attn_tile alone
      if (s.n_seq > 1 && G <= 32) p.RT = G <= 16 ? 1 : 2;
      p.NW = rows <= 64 ? 2 : 4;
    }
    p.rows_min = 16 * p.RT;
    if (p.RT > 0) wave_units = s.n_seq;
    if (p.NW > 0) tile_units = T * G / (p.NW * 32) + std::min<int64_t>(s.n_seq, T * G / (p.rows_min + 1));
  }
  p.groups = std::max(wave_units, tile_units) * KH;
  if (p.groups > ((int64_t)1 << 23)) return p;   // refused by the caller
  p.wave_units = (int)wave_units;
  p.tile_units = (int)tile_units;
  if (p.RT > 0) {
    // resident workgroups a CU: what their LDS lets in (128 KB of bf16 tiles at head_dim 128)
    p.wave_slots = 256 * (pg.kdtype == MISA_K_FP8_E4M3 ? 2 : 1) * (s.head_dim == 64 ? 2 : 1);
    p.wave_splits = choose_splits(wave_units * KH, p.wave_slots, (ctx + 127) / 128, 64, topk > 0);
  }
  if (p.NW > 0) {
    const int64_t BM = p.NW * 32;
    const int64_t est = topk > 0 ? tile_units : (T * G + BM - 1) / BM;
    p.tile_slots = s.head_dim == 64 ? 768 : 512;   // LDS, and registers at head_dim 64
    p.tile_splits = choose_splits(est * KH, p.tile_slots, (ctx + 63) / 64, 32, topk > 0);
  }
  p.groups = std::max(wave_units * p.wave_splits, tile_units * p.tile_splits) * KH;
  size_t off = 0;
  if (p.RT > 0 && p.wave_splits > 1) {
    const size_t rows = (size_t)p.wave_units * KH * p.wave_splits * 16 * p.RT;
    p.wave_o = off;
    off += align_up(rows * s.head_dim * sizeof(float));
    p.wave_ml = off;
    off += align_up(rows * sizeof(float2));
  }
  if (p.NW > 0 && p.tile_splits > 1) {
    const size_t rows = (size_t)p.tile_units * KH * p.tile_splits * 32 * p.NW;
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

bool attn_fits(const misa_attn_shape& s, const misa_kv_pages& pg, int topk) {
  return make_plan(s, pg, topk).groups <= ((int64_t)1 << 23);
}

size_t attn_workspace_bytes(const misa_attn_shape& s, const misa_kv_pages& pg, int topk) {
  return make_plan(s, pg, topk).total;
}

hipError_t launch_attention(const misa_attn_shape& s, const misa_kv_pages& pg, const uint16_t* q,
                            const int32_t* q_start, const int32_t* kv_lens, const int32_t* idx, int topk,
                            uint16_t* out, float* lse, void* ws, hipStream_t st) {
  const AttnPlan p = make_plan(s, pg, topk);
  const bool pow2 = (pg.page_keys & (pg.page_keys - 1)) == 0;
  const AttnArgs a{q, s.q_stride_token, s.q_stride_head, pg.k, pg.v, pg.k_scale, pg.v_scale, pg.block_table,
                   pg.max_pages, (int)pg.n_pages, pg.page_keys, pow2 ? __builtin_ctz((unsigned)pg.page_keys) : -1, q_start,
                   kv_lens, idx, topk, out, lse, s.scale * 1.4426950408889634f, s.n_seq, s.n_heads, s.n_kv_heads,
                   s.n_tokens};
  const bool fp8 = pg.kdtype == MISA_K_FP8_E4M3;
  char* base = static_cast<char*>(ws);
  hipError_t e = hipSuccess;
  if (p.NW > 0) {
    const AttnLaunch L{p.tile_units, p.tile_splits, p.tile_slots, p.rows_min,
                       reinterpret_cast<float*>(base + p.tile_o), reinterpret_cast<float2*>(base + p.tile_ml),
                       reinterpret_cast<int4*>(base + p.tile_info)};
    e = launch_attn_tile(a, L, s.head_dim, fp8, p.NW, st);
  }
  if (e == hipSuccess && p.RT > 0) {
    const AttnLaunch L{p.wave_units, p.wave_splits, p.wave_slots, p.rows_min,
                       reinterpret_cast<float*>(base + p.wave_o), reinterpret_cast<float2*>(base + p.wave_ml), nullptr};
    e = launch_attn_wave(a, L, s.head_dim, fp8, p.RT, st);
  }
  return e;
}

}  // namespace misa
