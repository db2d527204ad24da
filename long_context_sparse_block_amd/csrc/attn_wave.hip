// Attention of few query rows (at most 16 RT of a kv head): decodes, a few
// speculated tokens, or one token's heads over its selected tokens.  Bound by
// the reading of K and V.
//
// Each of a workgroup's 4 waves walks its own 32-key tiles (every fourth of
// the workgroup's key range) with its own LDS, so no barrier stands between a
// wave and its loads; the waves' results join in LDS at the end, and the key
// splits of a unit in a second small kernel.  bf16 tiles go straight to LDS,
// one tile ahead; e4m3 codes pass through registers, where they become bf16.
//
// A tile of a wave is 8 RT + 2 * 8 RT (D = 128) v_mfma_f32_16x16x32_bf16.  The
// softmax weights enter the second product as two bf16 parts (the rounded
// weight and what the rounding left): the matrix cores are idle here anyway,
// and the weights keep 16 bits.
#include "attn_device.h"

namespace misa {

namespace {
constexpr int kWT = 32;      // keys of a wave's tile
constexpr int kWaves = 4;
}  // namespace

template <int D, bool FP8, bool SEL, int RT>
__global__ void __launch_bounds__(kWaves * kWave, FP8 ? 2 : 1) k_attn_wave(const AttnArgs a, const AttnLaunch L) {
  constexpr int RB = D * 2, P = D / 8, RPI = kWave / P;
  constexpr int KS = D / 32, DB = D / 16;
  constexpr int ROWS = 16 * RT;
  constexpr int kTile = kWT * RB;             // bytes of a tile's K (or V) in LDS
  constexpr int kLoads = kWT / RPI;
  constexpr int PC = D / 16, kLoads8 = kWT * PC / kWave;   // e4m3: 16-byte pieces of a row, a lane's loads
  constexpr int kBuf = 2 * kWaves * kTile;    // K and V of the four waves
  __shared__ __attribute__((aligned(16))) unsigned char s_a[kBuf];
  __shared__ __attribute__((aligned(16))) unsigned char s_b[FP8 ? 16 : kBuf];
  __shared__ __attribute__((aligned(16))) float s_sc[FP8 ? 2 * kWaves * kWT : 4];
  __shared__ float s_m[kWaves][ROWS], s_l[kWaves][ROWS];
  static_assert(kBuf >= kWaves * ROWS * D * 4, "the waves' outputs join in the first buffer");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g4 = lane >> 4, c16 = lane & 15;
  const int G = a.n_heads / a.n_kv_heads;

  const Place at = place_of(L, a.n_kv_heads, blockIdx.x);
  const int split = at.split, g = at.g, unit = at.unit;
  int b, tok0, nrows, kend, kfull;   // sequence, first token, rows; keys some row sees, keys every row sees
  int64_t pos0;
  int jt0, jt1;                      // this wave's tiles: jt0, jt0 + 4, ... below jt1
  int in_use = 1;                    // the unit's splits in use
  auto range = [&](const DenseScan& w) {
    const int n = (kend + kWT - 1) / kWT;
    const int per = max(1, L.n_splits == 1 ? n : split_tiles(w, L, a.n_kv_heads, n, 4 * kWaves));
    in_use = max(1, (n + per - 1) / per);
    jt0 = split * per + wave;
    jt1 = min(n, (split + 1) * per);
  };
  const int k32 = lane & 31;
  int pick0 = 0, pick1 = 0, pick2 = 0, pick3 = 0;   // SEL: this lane's listed tokens of the first tiles
  if (SEL) {
    tok0 = unit;
    nrows = G;
    kend = a.topk;
    range(DenseScan{0.f, 0, 0});
    // on their way while the sequence is looked up
    pick0 = pick(a, tok0, jt0 * kWT + k32);
    pick1 = pick(a, tok0, (jt0 + kWaves) * kWT + k32);
    pick2 = pick(a, tok0, (jt0 + 2 * kWaves) * kWT + k32);
    pick3 = pick(a, tok0, (jt0 + 3 * kWaves) * kWT + k32);
    SeqSpan sp;
    if (!seq_of_token(a, tok0, lane, &b, &sp)) return;
    pos0 = sp.pos0 + (tok0 - sp.t0);
    kfull = (int)max((int64_t)0, min((int64_t)sp.len, pos0 + 1));   // tokens the row may list
    if (kfull == 0) jt1 = jt0;
  } else {
    SeqSpan sp;
    DenseScan scan;
    int none;
    if (!find_unit<false, kWT>(a, L, G, 1, unit, lane, &sp, &b, &none, &scan)) return;
    tok0 = sp.t0;
    nrows = sp.m * G;
    pos0 = sp.pos0;
    kend = (int)max((int64_t)0, min((int64_t)sp.len, pos0 + sp.m));
    kfull = (int)max((int64_t)0, min((int64_t)sp.len, pos0 + 1));
    range(scan);
    if (split >= in_use) {   // the join finds an empty split
      const int64_t part = (((int64_t)unit * a.n_kv_heads + g) * L.n_splits + split) * ROWS;
      if (tid < nrows) L.part_ml[part + tid] = make_float2(-INFINITY, 0.f);
      return;
    }
  }

  int vis[RT];
  bf16x8 qf[RT][KS];
  const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
  const float sc = fmaxf(fabsf(a.scale_log2), 1e-30f);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int rc = min(rt * 16 + c16, nrows - 1);
    const int qi = SEL ? 0 : rc / G, qh = g * G + (SEL ? rc : rc - qi * G);
    vis[rt] = SEL ? 0 : (int)max((int64_t)-1, min((int64_t)kend, pos0 + qi + 1));
    const uint16_t* src = a.q + ((int64_t)tok0 + qi) * a.q_st + qh * a.q_sh + g4 * 8;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) qf[rt][ks] = load_q(src + ks * 32, flip);
  }

  unsigned char* const ka = s_a + wave * 2 * kTile;
  unsigned char* const kb_ = s_b + (FP8 ? 0 : wave * 2 * kTile);
  float* const sks = s_sc + (FP8 ? wave * 2 * kWT : 0);
  const int64_t row_stride = (int64_t)a.n_kv_heads * D;
  auto token_at = [&](int jt) -> int {
    const int j = jt * kWT + k32;
    return SEL ? pick(a, tok0, j) : min(j, kend - 1);
  };
  auto seen = [&](int t) -> bool { return t >= 0 && t < kfull; };
  auto clamp_tok = [&](int t) -> int { return SEL ? (seen(t) ? t : 0) : t; };

  // a tile's K and V towards LDS: bf16 straight there, e4m3 codes into
  // registers, from which land() widens them
  struct Codes {
    uint4 k[FP8 ? kLoads8 : 1], v[FP8 ? kLoads8 : 1];
    float scale;
  };
  auto issue = [&](int row_of, unsigned char* dst, Codes& r8) {
    if constexpr (!FP8) {
      int64_t off[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int row = u * RPI + lane / P;
        off[u] = ((int64_t)__shfl(row_of, row) * row_stride + g * D) * 2 + ((lane % P) ^ swizzle<D>(row)) * 16;
      }
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        load_lds16(static_cast<const char*>(a.k) + off[u], dst + u * RPI * RB);
        load_lds16(static_cast<const char*>(a.v) + off[u], dst + kTile + u * RPI * RB);
      }
    } else {
#pragma unroll
      for (int u = 0; u < kLoads8; ++u) {
        const int i = u * kWave + lane;
        const int64_t off = (int64_t)__shfl(row_of, i / PC) * row_stride + g * D + (i % PC) * 16;
        r8.k[u] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.k) + off);
        r8.v[u] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.v) + off);
      }
      r8.scale = (lane < kWT ? a.k_scale : a.v_scale)[(int64_t)row_of * a.n_kv_heads + g];
    }
  };
  auto land = [&](unsigned char* dst, const Codes& r8) {
    if constexpr (FP8) {
#pragma unroll
      for (int u = 0; u < kLoads8; ++u) {
        const int i = u * kWave + lane, row = i / PC, c = 2 * (i % PC);
        const int f = swizzle<D>(row);
        auto put = [&](unsigned char* d, uint4 x) {
          const uint2 w0 = e4m3x4_to_bf16x4(x.x), w1 = e4m3x4_to_bf16x4(x.y);
          const uint2 w2 = e4m3x4_to_bf16x4(x.z), w3 = e4m3x4_to_bf16x4(x.w);
          *reinterpret_cast<uint4*>(d + row * RB + ((c ^ f) << 4)) = make_uint4(w0.x, w0.y, w1.x, w1.y);
          *reinterpret_cast<uint4*>(d + row * RB + (((c + 1) ^ f) << 4)) = make_uint4(w2.x, w2.y, w3.x, w3.y);
        };
        put(dst, r8.k[u]);
        put(dst + kTile, r8.v[u]);
      }
      sks[lane] = r8.scale;   // 32 key scales, 32 value scales
    }
  };

  f32x4 o[RT][DB];
  float m[RT], l[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    m[rt] = -INFINITY;
    l[rt] = 0.f;
#pragma unroll
    for (int db = 0; db < DB; ++db) o[rt][db] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int k_base = c16 * RB + ((g4 ^ swizzle<D>(c16)) << 4);
  const int vr = 4 * g4 + (c16 >> 2);
  const int v_base = vr * RB + ((((lane & 3) >> 1) ^ swizzle<D>(vr)) << 4) + (lane & 1) * 8;

  auto compute = [&](const unsigned char* sk, int jt, uint32_t mask) {
    const unsigned char* sv = sk + kTile;
    f32x4 s[RT][2];   // s[rt][kb][i]: key kb 16 + 4 g4 + i of row rt 16 + c16
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const bf16x8 kf = as_bf16x8(*reinterpret_cast<const uint4*>(sk + kb * 16 * RB + (k_base ^ (ks << 6))));
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) s[rt][kb] = mfma16(kf, qf[rt][ks], s[rt][kb]);
      }
    f32x4 wk[2], wv[2];
    if constexpr (FP8) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        wk[kb] = *reinterpret_cast<const f32x4*>(sks + kb * 16 + 4 * g4);
        wv[kb] = *reinterpret_cast<const f32x4*>(sks + kWT + kb * 16 + 4 * g4);
      }
    }
    bf16x8 ph[RT], pl[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float p[8];
      const int lim = vis[rt] - jt * kWT;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = s[rt][kb][i];
          if constexpr (FP8) x *= wk[kb][i];
          const int key = kb * 16 + 4 * g4 + i;
          const bool ok = SEL ? (mask >> key) & 1 : key < lim;
          p[kb * 4 + i] = ok ? x : -INFINITY;
        }
      float top = p[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, p[e]);
      top = max_rows(top) * sc;
      const float mn = fmaxf(m[rt], top);
      if (__any(mn > m[rt])) {
        const float keep = mn == -INFINITY ? 1.f : exp2_raw(m[rt] - mn);
        m[rt] = mn;
        l[rt] *= keep;
#pragma unroll
        for (int db = 0; db < DB; ++db) o[rt][db] *= keep;
      }
      const float mu = m[rt] == -INFINITY ? 0.f : m[rt];
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = exp2_raw(__builtin_fmaf(p[e], sc, -mu));
      l[rt] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
      if constexpr (FP8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] *= wv[e >> 2][e & 3];
      }
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        hi[e] = pk_bf16(p[2 * e], p[2 * e + 1]);
        lo[e] = pk_bf16(p[2 * e] - __uint_as_float(hi[e] << 16), p[2 * e + 1] - __uint_as_float(hi[e] & 0xFFFF0000u));
      }
      ph[rt] = as_bf16x8(make_uint4(hi[0], hi[1], hi[2], hi[3]));
      pl[rt] = as_bf16x8(make_uint4(lo[0], lo[1], lo[2], lo[3]));
    }
#pragma unroll
    for (int db = 0; db < DB; ++db) {
      const uint2 v0 = lds_read_tr(sv + (v_base ^ (db << 5))), v1 = lds_read_tr(sv + 16 * RB + (v_base ^ (db << 5)));
      const bf16x8 vf = as_bf16x8(make_uint4(v0.x, v0.y, v1.x, v1.y));
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) o[rt][db] = mfma16(vf, pl[rt], mfma16(vf, ph[rt], o[rt][db]));
    }
  };

  if (jt0 < jt1) {
    const int last = jt1 - 1;
    auto look = [&](int t, uint32_t& mask) -> int {
      if (SEL) mask = (uint32_t)__ballot(seen(t));
      return clamp_tok(t);
    };
    auto next = [&](int i) { return min(jt0 + i * kWaves, last); };
    uint32_t m0 = 0, m1 = 0, m2 = 0;   // of this tile and the next two
    const int t0 = look(SEL ? pick0 : token_at(jt0), m0);
    const int t1 = look(SEL ? pick1 : token_at(next(1)), m1);
    const int e0 = table_entry(a, b, t0), e1 = table_entry(a, b, t1);
    if constexpr (FP8) {
      // codes two tiles ahead in registers; they land right before their use
      // (one tile ahead, a wave spent most of its time waiting for gathers).
      // Loads return in order, so a step's look-ups go out before its codes:
      // waiting for them then waits for no codes but the oldest.
      Codes ra, rb;
      int tok_n = look(SEL ? pick2 : token_at(next(2)), m2);
      int ent_n = table_entry(a, b, tok_n);
      int tok_nn = SEL ? pick3 : token_at(next(3));
      issue(pool_row(a, e0, t0), ka, ra);
      issue(pool_row(a, e1, t1), ka, rb);
      auto step = [&](int jt, Codes& r) {
        land(ka, r);
        uint32_t m3 = 0;
        if (jt + 2 * kWaves < jt1) {
          const int row = pool_row(a, ent_n, tok_n);
          tok_n = look(tok_nn, m3);
          ent_n = table_entry(a, b, tok_n);
          tok_nn = token_at(min(jt + 4 * kWaves, last));
          issue(row, ka, r);
        }
        compute(ka, jt, m0);
        m0 = m1;
        m1 = m2;
        m2 = m3;
      };
      for (int jt = jt0; jt < jt1; jt += 2 * kWaves) {
        step(jt, ra);
        if (jt + kWaves < jt1) step(jt + kWaves, rb);
      }
    } else {
      Codes none;
      issue(pool_row(a, e0, t0), ka, none);
      int tok_n = t1, ent_n = e1, tok_nn = SEL ? pick2 : token_at(next(2));
      auto step = [&](int jt, unsigned char* cur, unsigned char* nxt) {
        __builtin_amdgcn_s_waitcnt(0);   // the tile, and the look-ups of the next ones
        if (jt + kWaves < jt1) {
          issue(pool_row(a, ent_n, tok_n), nxt, none);
          tok_n = look(tok_nn, m2);
          ent_n = table_entry(a, b, tok_n);
          tok_nn = token_at(min(jt + 3 * kWaves, last));
        }
        compute(cur, jt, m0);
        m0 = m1;
        m1 = m2;
      };
      for (int jt = jt0; jt < jt1; jt += 2 * kWaves) {
        step(jt, ka, kb_);
        if (jt + kWaves < jt1) step(jt + kWaves, kb_, ka);
      }
    }
  }

  // the four waves' results, relative to their joint maximum, through LDS
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    l[rt] = sum_rows(l[rt]);
    if (g4 == 0) {
      s_m[wave][rt * 16 + c16] = m[rt];
      s_l[wave][rt * 16 + c16] = l[rt];
    }
  }
  __syncthreads();   // (all waves are done with their tiles too)
  float* const so = reinterpret_cast<float*>(s_a);   // [wave][row][D]
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int row = rt * 16 + c16;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_m[w][row]);
    const float f = m[rt] == -INFINITY ? 0.f : exp2_raw(m[rt] - top);
#pragma unroll
    for (int db = 0; db < DB; ++db)
      *reinterpret_cast<f32x4*>(so + (wave * ROWS + row) * D + ((db * 4 + g4) ^ (row & 7)) * 4) = o[rt][db] * f;
  }
  __syncthreads();
  const int64_t part = (((int64_t)unit * a.n_kv_heads + g) * L.n_splits + split) * ROWS;
  for (int i = tid; i < ROWS * (D / 4); i += kWaves * kWave) {
    const int row = i / (D / 4), c = i % (D / 4);
    if (row >= nrows) break;   // (rows ascend with i)
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_m[w][row]);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      sum += s_m[w][row] == -INFINITY ? 0.f : s_l[w][row] * exp2_raw(s_m[w][row] - top);
      acc += *reinterpret_cast<const f32x4*>(so + (w * ROWS + row) * D + (c ^ (row & 7)) * 4);
    }
    if (L.n_splits > 1) {
      if (c == 0) L.part_ml[part + row] = make_float2(top, sum);
      if (sum > 0.f) *reinterpret_cast<f32x4*>(L.part_o + (part + row) * D + c * 4) = acc;
      continue;
    }
    const int qi = SEL ? 0 : row / G, qh = g * G + (SEL ? row : row - qi * G);
    const int64_t orow = ((int64_t)tok0 + qi) * a.n_heads + qh;
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    *reinterpret_cast<uint2*>(a.out + orow * D + c * 4) =
        make_uint2(pk_bf16(acc[0] * inv, acc[1] * inv), pk_bf16(acc[2] * inv, acc[3] * inv));
    if (a.lse != nullptr && c == 0) a.lse[orow] = sum > 0.f ? (top + __log2f(sum)) * kLn2 : -INFINITY;
  }
}

template <int D, bool SEL>
__global__ void __launch_bounds__(256) k_attn_wave_join(const AttnArgs a, const AttnLaunch L, int ROWS) {
  const int lane = threadIdx.x & 63;
  const int unit = blockIdx.x, g = blockIdx.y;
  const int G = a.n_heads / a.n_kv_heads;
  const int row = blockIdx.z * 4 + (threadIdx.x >> 6);
  int tok0, nrows;
  if (SEL) {
    tok0 = unit;
    if (tok0 >= a.q_start[a.n_seq] || tok0 < a.q_start[0]) return;   // no sequence's token: nothing was written
    nrows = G;
  } else {
    const SeqSpan sp = seq_span(a, unit);
    if ((int64_t)sp.m * G > L.rows_min) return;
    tok0 = sp.t0;
    nrows = sp.m * G;
  }
  if (row >= nrows) return;
  const int qi = SEL ? 0 : row / G, qh = g * G + (SEL ? row : row - qi * G);
  join_row<D>(a, L, L.n_splits, (((int64_t)unit * a.n_kv_heads + g) * L.n_splits) * ROWS + row, ROWS,
              ((int64_t)tok0 + qi) * a.n_heads + qh, lane);
}

template <int D, bool FP8, bool SEL>
static hipError_t launch_rt(const AttnArgs& a, const AttnLaunch& L, int RT, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)L.n_units * L.n_splits * a.n_kv_heads));
  if (RT == 1) hipLaunchKernelGGL((k_attn_wave<D, FP8, SEL, 1>), grid, dim3(256), 0, st, a, L);
  else hipLaunchKernelGGL((k_attn_wave<D, FP8, SEL, 2>), grid, dim3(256), 0, st, a, L);
  if (L.n_splits > 1)
    hipLaunchKernelGGL((k_attn_wave_join<D, SEL>), dim3(L.n_units, a.n_kv_heads, RT * 4), dim3(256), 0, st, a, L, RT * 16);
  return hipGetLastError();
}

hipError_t launch_attn_wave(const AttnArgs& a, const AttnLaunch& L, int D, bool fp8, int RT, hipStream_t st) {
  const bool sel = a.idx != nullptr;
  if (D == 128) {
    if (fp8) return sel ? launch_rt<128, true, true>(a, L, RT, st) : launch_rt<128, true, false>(a, L, RT, st);
    return sel ? launch_rt<128, false, true>(a, L, RT, st) : launch_rt<128, false, false>(a, L, RT, st);
  }
  if (fp8) return sel ? launch_rt<64, true, true>(a, L, RT, st) : launch_rt<64, true, false>(a, L, RT, st);
  return sel ? launch_rt<64, false, true>(a, L, RT, st) : launch_rt<64, false, false>(a, L, RT, st);
}

}  // namespace misa
