// Attention of few query rows (at most 16 RT of a kv head): decodes, a few
// speculated tokens, or one token's heads over its selected tokens.  Bound by
// the reading of K and V.
//
// Each of a workgroup's 4 waves walks its own 32-key tiles (every fourth of
// the workgroup's key range) with its own LDS, so no barrier stands between a
// wave and its loads; the waves' results join in LDS at the end, and the key
// splits of a unit in a second small kernel.
//
// bf16 tiles go straight to LDS, one tile ahead.  e4m3 codes are in registers
// almost two tiles ahead (a load straight into LDS is a flat instruction and
// would make the compiler wait for all loads under way at the first result that
// it needs), pass through LDS as they are and are widened as operands: K read
// as rows, V by the transposing read.  (Widened before LDS they made it the
// bound, 71% of the time.  K loaded in the operand's own layout, without LDS,
// was no faster: its lanes are neighbours in different rows, and the load unit
// takes one row a clock, 15 bytes a clock and CU; neighbours in the same row
// make 28 to 44.)
//
// A tile of a wave is 8 RT + 16 RT (D = 128) v_mfma_f32_16x16x32_bf16: the softmax
// weights enter the second product as two bf16 parts (the rounded weight and
// what the rounding left), so the weights keep 16 bits.  The reading leaves the
// other units room for it; one part alone took the same time for decodes (64 of
// 8..16K keys, e4m3: 363 us) and 3% less over selected tokens (1000 x 2048,
// e4m3: 243 to 249 us), but few rows with a few heavy keys average a weight's
// rounding out too little.
//
// Measured: 64 decodes over 8..16K keys, 32 / 8 heads of 128: bf16 577-599 us by card
// (3.2 GB, 5.4 TB/s), e4m3 346-363 us; one token over 32K keys 37 us; 1000 tokens x
// 2048 picks, 32 / 4 heads, e4m3: 249-253 us (2.1 GB of gathered rows; vector unit
// 51%, LDS 30%, MFMA 18%), bf16 490 us.
#include "attn_device.h"

namespace misa {

namespace {
constexpr int kWT = 32;      // keys of a wave's tile
constexpr int kWaves = 4;
}  // namespace

template <int D, bool FP8, bool SEL, int RT>
__global__ void __launch_bounds__(kWaves * kWave, wave_groups(D, FP8, SEL, RT)) k_attn_wave(const AttnArgs a, const AttnLaunch L) {
  constexpr int RB = D * 2, P = D / 8, RPI = kWave / P;    // bf16: bytes and 16-byte pieces of a row, rows of a load
  constexpr int PC = D / 16, RPC = kWave / PC;              // e4m3: pieces of a row, rows of a load
  constexpr int KS = D / 32, DB = D / 16;
  constexpr int ROWS = 16 * RT;
  constexpr int kTile = kWT * RB;                           // bytes of a tile's K (or V) in LDS
  constexpr int kTile8 = kWT * D;                           // of a tile's K (or V) codes
  constexpr int kLoads = kWT / RPI, kLoads8 = kWT / RPC;
  constexpr int kBuf = FP8 ? kWaves * 2 * kTile8 : kWaves * 2 * kTile;
  constexpr int kJoin = 2 * RT * DB * kWave * 16;           // two waves' outputs
  // separate arrays: the compiler then knows which of them a load into LDS fills
  __shared__ __attribute__((aligned(16))) unsigned char s_a[kBuf > kJoin ? kBuf : kJoin];
  __shared__ __attribute__((aligned(16))) unsigned char s_b[FP8 ? 16 : kBuf];
  __shared__ __attribute__((aligned(16))) float s_sc[FP8 ? 2 * kWaves * kWT : 4];
  __shared__ float s_m[kWaves][ROWS], s_l[kWaves][ROWS];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g4 = lane >> 4, c16 = lane & 15;
  const int G = a.n_heads / a.n_kv_heads;

  const Place at = place_of(L, a.n_kv_heads, blockIdx.x, SEL ? 31 : 0);
  const int split = at.split, g = at.g, unit = at.unit;
  int b, tok0, nrows, kend, kfull;   // sequence, first token, rows; keys some row sees, keys every row sees
  int64_t pos0;
  int jt0, jt1;                      // this wave's tiles: jt0, jt0 + 4, ... below jt1
  int in_use = 1;                    // the unit's splits in use
  auto range = [&](const DenseScan& w) __attribute__((always_inline)) {
    const int n = (kend + kWT - 1) / kWT;
    const int per = split_tiles(w, L, n, &in_use);
    jt0 = split * per + wave;
    jt1 = min(n, (split + 1) * per);
  };
  const int k32 = lane & 31;
  const int k_mine = min(lane, 31);   // the key a lane looks up: a load takes a clock for every four lanes apart
  int pick0 = 0, pick1 = 0, pick2 = 0, pick3 = 0;   // SEL: this lane's listed tokens of the first tiles
  if (SEL) {
    tok0 = unit;
    nrows = G;
    kend = a.topk;
    range(DenseScan{0.f, 0, 0, 0});
    // on their way while the sequence is looked up
    pick0 = pick(a, tok0, jt0 * kWT + k_mine);
    pick1 = pick(a, tok0, (jt0 + kWaves) * kWT + k_mine);
    pick2 = pick(a, tok0, (jt0 + 2 * kWaves) * kWT + k_mine);
    pick3 = pick(a, tok0, (jt0 + 3 * kWaves) * kWT + k_mine);
    SeqSpan sp;
    if (!seq_of_token(a, tok0, lane, &b, &sp)) return;
    pos0 = sp.pos0 + (tok0 - sp.t0);
    kfull = (int)max((int64_t)0, min((int64_t)sp.len, pos0 + 1));   // tokens the row may list
    if (kfull == 0) jt1 = jt0;
  } else {
    SeqSpan sp;
    DenseScan scan;
    int none;
    if (!find_unit<false, kWT, D>(a, L, G, 1, unit, lane, &sp, &b, &none, &scan)) {
      if (L.n_splits > 1 && split == 0 && g == 0 && tid == 0) L.unit_info[unit] = make_int4(0, 0, 0, 0);
      return;
    }
    tok0 = sp.t0;
    nrows = sp.m * G;
    pos0 = sp.pos0;
    kend = (int)max((int64_t)0, min((int64_t)sp.len, pos0 + sp.m));
    kfull = (int)max((int64_t)0, min((int64_t)sp.len, pos0 + 1));
    range(scan);
    if (L.n_splits > 1 && split == 0 && g == 0 && tid == 0) L.unit_info[unit] = make_int4(tok0, 0, nrows, in_use);
    if (split >= in_use) return;
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
    // e4m3: step ks of a product takes values 64 (ks / 2) + 16 g4 + 8 (ks % 2) .. +7 of the row, as K's codes come
    const uint16_t* src = a.q + ((int64_t)tok0 + qi) * a.q_st + qh * a.q_sh + g4 * (FP8 ? 16 : 8);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) qf[rt][ks] = load_q(src + (FP8 ? ks / 2 * 64 + ks % 2 * 8 : ks * 32), flip);
  }

  float* const sks = s_sc + (FP8 ? wave * 2 * kWT : 0);   // e4m3: the tile's key scales, then its value scales
  const int64_t row_bytes = (int64_t)a.n_kv_heads * D * (FP8 ? 1 : 2);
  const char* const kg = static_cast<const char*>(a.k) + g * D * (FP8 ? 1 : 2);
  const char* const vg = static_cast<const char*>(a.v) + g * D * (FP8 ? 1 : 2);
  auto token_at = [&](int jt) __attribute__((always_inline)) -> int {
    const int j = jt * kWT + k_mine;
    return SEL ? pick(a, tok0, j) : min(j, kend - 1);
  };
  auto seen = [&](int t) __attribute__((always_inline)) -> bool { return t >= 0 && t < kfull; };
  // Lane k < 32 knows where key k's pool row starts (bytes); others fetch it there
  auto fetch = [&](int64_t off, int from) __attribute__((always_inline)) -> int64_t {
    const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)off, from), hi = (uint32_t)__shfl((int)(off >> 32), from);
    return (int64_t)(((uint64_t)hi << 32) | lo);
  };
  struct Codes {   // e4m3: pieces of K's and V's rows, a scale
    u32x4 k[FP8 ? kLoads8 : 1], v[FP8 ? kLoads8 : 1];
    float scale;
  };
  // where pieces of code rows lie in LDS (piece c of row r at c ^ swz(r)): 16 rows' pieces of a row
  // read, and 8 rows' of a transposing read, are on as many bank groups
  auto swzk = [](int r) { return D == 128 ? (r >> 1) & 7 : (r >> 2) & 3; };
  auto swzv = [](int r) { return D == 128 ? ((r >> 1) & 3) | ((r >> 4) & 1) << 2 : ((r >> 2) & 1) | ((r >> 4) & 1) << 1; };
  auto issue = [&](int row_of, unsigned char* dst, Codes& r8) __attribute__((always_inline)) {
    const int64_t mine = (int64_t)row_of * row_bytes;
    if constexpr (!FP8) {
      int64_t off[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int row = u * RPI + lane / P;
        off[u] = fetch(mine, row) + ((lane % P) ^ swizzle<D>(row)) * 16;
      }
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        load_lds16(kg + off[u], dst + u * RPI * RB);
        load_lds16(vg + off[u], dst + kTile + u * RPI * RB);
      }
    } else {
      int64_t off[kLoads8];
#pragma unroll
      for (int u = 0; u < kLoads8; ++u) off[u] = fetch(mine, u * RPC + lane / PC) + (lane % PC) * 16;
#pragma unroll
      for (int u = 0; u < kLoads8; ++u) r8.k[u] = *reinterpret_cast<const u32x4*>(kg + off[u]);
#pragma unroll
      for (int u = 0; u < kLoads8; ++u) r8.v[u] = *reinterpret_cast<const u32x4*>(vg + off[u]);
      r8.scale = (lane < kWT ? a.k_scale : a.v_scale)[(int64_t)__shfl(row_of, k32) * a.n_kv_heads + g];
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
  // e4m3: the transposing read takes rows 4 g4 .. +3 and 16 + 4 g4 .. +3, two lanes each
  const int vr8 = 16 * (c16 >> 3) + 4 * g4 + ((c16 >> 1) & 3);
  const int v_base8 = vr8 * D + (swzv(vr8) << 4) + (lane & 1) * 8;
  const int k_base8 = c16 * D + ((g4 ^ swzk(c16)) << 4);   // (rows c16 and 16 + c16 are swizzled alike)

  // sk: the tile's K, then its V
  auto compute = [&](const unsigned char* sk, int jt, uint32_t mask) __attribute__((always_inline)) {
    const unsigned char* sv = sk + (FP8 ? kTile8 : kTile);
    uint4 kc[2][FP8 ? D / 64 : 1];   // e4m3: pieces g4 and g4 + 4 of the lane's rows
    if constexpr (FP8) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          kc[kb][i] = *reinterpret_cast<const uint4*>(sk + kb * 16 * D + (k_base8 ^ (i << 6)));
    }
    f32x4 s[RT][2];   // s[rt][kb][i]: key kb 16 + 4 g4 + i of row rt 16 + c16
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        bf16x8 kf;
        if constexpr (FP8) {
          const uint4 c = kc[kb][ks / 2];
          const uint2 lo = e4m3x4_to_bf16x4(ks & 1 ? c.z : c.x), hi = e4m3x4_to_bf16x4(ks & 1 ? c.w : c.y);
          kf = as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y));
        } else {
          kf = as_bf16x8(*reinterpret_cast<const uint4*>(sk + kb * 16 * RB + (k_base ^ (ks << 6))));
        }
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
    // (uniform: most tiles are seen whole by every row)
    const bool whole = SEL ? mask == 0xFFFFFFFFu : (jt + 1) * kWT <= kfull;
    bf16x8 ph[RT], pl[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = s[rt][e >> 2][e & 3];
        if constexpr (FP8) p[e] *= wk[e >> 2][e & 3];
      }
      if (!whole) {
        const int lim = vis[rt] - jt * kWT;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int key = (e >> 2) * 16 + 4 * g4 + (e & 3);
          p[e] = (SEL ? (mask >> key) & 1 : key < lim) ? p[e] : -INFINITY;
        }
      }
      float top = p[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) top = fmaxf(top, p[e]);
      top = max_rows(top) * sc;
      if (__any(top > m[rt] + kGrow)) {   // (m = -inf at first)
        const float mn = fmaxf(m[rt], top);
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
      bf16x8 vf;
      if constexpr (FP8) {
        const uint2 c = lds_read_tr8(sv + (v_base8 ^ (db << 4)));
        const uint2 lo = e4m3x4_to_bf16x4(c.x), hi = e4m3x4_to_bf16x4(c.y);
        vf = as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y));
      } else {
        const uint2 v0 = lds_read_tr(sv + (v_base ^ (db << 5))), v1 = lds_read_tr(sv + 16 * RB + (v_base ^ (db << 5)));
        vf = as_bf16x8(make_uint4(v0.x, v0.y, v1.x, v1.y));
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        o[rt][db] = mfma16(vf, ph[rt], o[rt][db]);
        o[rt][db] = mfma16(vf, pl[rt], o[rt][db]);
      }
    }
  };

  if (jt0 < jt1) {
    const int last = jt1 - 1;
    // An absent entry (a weight of 0) reads the tile's first listed token instead,
    // whose value the row sees anyway; a tile without one is skipped.
    auto look = [&](int t, uint32_t& mask) __attribute__((always_inline)) -> int {
      if (!SEL) return t;
      const bool in = seen(t);
      mask = (uint32_t)__ballot(in);
      const int first = mask != 0 ? __builtin_amdgcn_readlane(t, (int)__builtin_ctz(mask)) : 0;
      return in ? t : first;
    };
    auto next = [&](int i) __attribute__((always_inline)) { return min(jt0 + i * kWaves, last); };
    uint32_t m0 = 0, m1 = 0, m2 = 0;   // of this tile and the next two
    const int t0 = look(SEL ? pick0 : token_at(jt0), m0);
    const int t1 = look(SEL ? pick1 : token_at(next(1)), m1);
    const int e0 = table_entry(a, b, t0), e1 = table_entry(a, b, t1);
    if constexpr (FP8) {
      // Loads return in order: a step's look-ups go out before its codes, so
      // that waiting for them waits for no codes but the oldest.  Near the end
      // the last tile is loaded again (from the cache): loads behind a branch
      // would make the compiler wait for all of them.
      unsigned char* const ka = s_a + wave * 2 * kTile8;
      Codes ra, rb;
      int tok_n = look(SEL ? pick2 : token_at(next(2)), m2);
      int ent_n = table_entry(a, b, tok_n);
      int tok_nn = SEL ? pick3 : token_at(next(3));
      issue(pool_row(a, e0, t0), nullptr, ra);
      __builtin_amdgcn_sched_barrier(0);   // in this order
      issue(pool_row(a, e1, t1), nullptr, rb);
      __builtin_amdgcn_sched_barrier(0);
      auto step = [&](int jt, Codes& r) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kLoads8; ++u) {
          const int row = u * RPC + lane / PC, c = lane % PC;
          *reinterpret_cast<u32x4*>(ka + row * D + ((c ^ swzk(row)) << 4)) = r.k[u];
          *reinterpret_cast<u32x4*>(ka + kTile8 + row * D + ((c ^ swzv(row)) << 4)) = r.v[u];
        }
        sks[lane] = r.scale;
        uint32_t m3 = 0;
        const int row = pool_row(a, ent_n, tok_n);
        tok_n = look(tok_nn, m3);
        ent_n = table_entry(a, b, tok_n);
        tok_nn = token_at(min(jt + 4 * kWaves, last));
        issue(row, nullptr, r);
        if (!SEL || m0 != 0) compute(ka, jt, m0);
        m0 = m1;
        m1 = m2;
        m2 = m3;
      };
      for (int jt = jt0;;) {   // (one way back to the top, for the compiler's count of loads under way)
        step(jt, ra);
        if ((jt += kWaves) >= jt1) break;
        step(jt, rb);
        if ((jt += kWaves) >= jt1) break;
      }
    } else {
      unsigned char* const ka = s_a + wave * 2 * kTile;
      unsigned char* const kb_ = s_b + wave * 2 * kTile;
      Codes none;
      issue(pool_row(a, e0, t0), ka, none);
      int tok_n = t1, ent_n = e1, tok_nn = SEL ? pick2 : token_at(next(2));
      auto step = [&](int jt, unsigned char* cur, unsigned char* nxt) __attribute__((always_inline)) {
        __builtin_amdgcn_s_waitcnt(0);   // the tile, and the look-ups of the next ones
        if (jt + kWaves < jt1) {
          issue(pool_row(a, ent_n, tok_n), nxt, none);
          tok_n = look(tok_nn, m2);
          ent_n = table_entry(a, b, tok_n);
          tok_nn = token_at(min(jt + 3 * kWaves, last));
        }
        if (!SEL || m0 != 0) compute(cur, jt, m0);
        m0 = m1;
        m1 = m2;
      };
      for (int jt = jt0; jt < jt1; jt += 2 * kWaves) {
        step(jt, ka, kb_);
        if (jt + kWaves < jt1) step(jt + kWaves, kb_, ka);
      }
    }
  }

  // the four waves' results, relative to their joint maximum, through LDS:
  // waves 2 and 3 onto 0 and 1, then 1 onto 0
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    l[rt] = sum_rows(l[rt]);
    if (g4 == 0) {
      s_m[wave][rt * 16 + c16] = m[rt];
      s_l[wave][rt * 16 + c16] = l[rt];
    }
  }
  __builtin_amdgcn_s_waitcnt(0);   // (no load into LDS is under way any more)
  __syncthreads();
  f32x4* const so = reinterpret_cast<f32x4*>(s_a);   // [2][RT DB][lane]
  float top[RT], sum[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int row = rt * 16 + c16;
    top[rt] = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top[rt] = fmaxf(top[rt], s_m[w][row]);
    sum[rt] = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
      sum[rt] += s_l[w][row] == 0.f ? 0.f : s_l[w][row] * exp2_raw(s_m[w][row] - top[rt]);
    const float f = m[rt] == -INFINITY ? 0.f : exp2_raw(m[rt] - top[rt]);
#pragma unroll
    for (int db = 0; db < DB; ++db) o[rt][db] *= f;
  }
  auto put = [&](int slot) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RT * DB; ++i) so[(slot * RT * DB + i) * kWave + lane] = o[i / DB][i % DB];
  };
  auto add = [&](int slot) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RT * DB; ++i) o[i / DB][i % DB] += so[(slot * RT * DB + i) * kWave + lane];
  };
  if (wave >= 2) put(wave - 2);
  __syncthreads();
  if (wave < 2) add(wave);
  if (wave == 1) put(1);
  __syncthreads();
  if (wave != 0) return;
  add(1);
  const PartPlace place = part_place<SEL>(L, a.n_kv_heads, G, ROWS, g, unit, tok0, 0, nrows);
  const int64_t part = place.begin + split * place.step;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int row = rt * 16 + c16;
    if (row >= nrows) continue;
    // o[rt][db][i]: element db 16 + 4 g4 + i
    if (in_use > 1) {
      if (g4 == 0) L.part_ml[part + row] = make_float2(top[rt], sum[rt]);
      if (sum[rt] != 0.f)
#pragma unroll
        for (int db = 0; db < DB; ++db)
          *reinterpret_cast<f32x4*>(L.part_o + (part + row) * D + db * 16 + 4 * g4) = o[rt][db];
      continue;
    }
    const int qi = SEL ? 0 : row / G, qh = g * G + (SEL ? row : row - qi * G);
    const int64_t orow = ((int64_t)tok0 + qi) * a.n_heads + qh;
    const float inv = sum[rt] != 0.f ? 1.f / sum[rt] : 0.f;
#pragma unroll
    for (int db = 0; db < DB; ++db)
      *reinterpret_cast<uint2*>(a.out + orow * D + db * 16 + 4 * g4) =
          make_uint2(pk_bf16(o[rt][db][0] * inv, o[rt][db][1] * inv), pk_bf16(o[rt][db][2] * inv, o[rt][db][3] * inv));
    if (a.lse != nullptr && g4 == 0) a.lse[orow] = sum[rt] != 0.f ? (top[rt] + __log2f(sum[rt])) * kLn2 : -INFINITY;
  }
}

template <int D, bool FP8, bool SEL>
static hipError_t launch_rt(const AttnArgs& a, const AttnLaunch& L, int RT, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)L.n_units * L.n_splits * a.n_kv_heads));
  if (RT == 1) hipLaunchKernelGGL((k_attn_wave<D, FP8, SEL, 1>), grid, dim3(256), 0, st, a, L);
  else hipLaunchKernelGGL((k_attn_wave<D, FP8, SEL, 2>), grid, dim3(256), 0, st, a, L);
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
