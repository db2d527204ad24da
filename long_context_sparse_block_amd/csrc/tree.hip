// Trees of drafted tokens: which of a sequence's new tokens descends from which
// (misa_plan_tree), and the move of an accepted path's rows to where the cached
// prefix goes on (misa_keep_path).  What attention makes of the tree is in
// attn_tile.hip and attn_wave.hip.
//
// Both move a few KB: what bounds them is the launch and a chain of dependent
// loads (lengths, then parents or path and table, then the rows).  Measured: the plan
// of 64 trees of 32 3.4 us, of 500 trees of up to 256 7.2 to 8.6 us (a walk of some 60 steps);
// kept paths of up to 8 of 32 nodes, 64 sequences, 8 + 8 heads of 128 5.4-6.2 us, of up to
// 12 of 64, 500 sequences' index keys 5.8-6.5 us.
#include <algorithm>

#include "misa_common.h"
#include "misa_launch.h"

namespace misa {

namespace {
constexpr int kPlanThreads = 256;
constexpr int kLdsNodes = 2048;   // a tree's parents that a workgroup keeps in LDS
}  // namespace

// `slices` workgroups take a sequence, a thread a token: it walks from the token to the root
// and collects its ancestors, a word of bits at a time (parents come before their
// children, so the walk goes through the words from the last to the first).  A step
// is a read of LDS that the next one waits for, some 40 ns, more when many waves
// of a CU walk: a slice for every 256 tokens that the words hold (4 trees of 2048
// tokens, walks of 800 steps, 316 us in one slice, 69 in eight; one of 1024 85, 34).
__global__ void __launch_bounds__(kPlanThreads) k_plan_tree(int n_seq, const int32_t* parents, const int32_t* q_start,
                                                            const int32_t* kv_lens, int64_t n_tokens, int words,
                                                            uint32_t* mask, int32_t* positions) {
  __shared__ int s_up[kLdsNodes];
  const int tid = threadIdx.x;
  const int b = blockIdx.x, slice = blockIdx.y, slices = gridDim.y;
  if (b >= n_seq) {   // rows of no sequence: in front of the first one, behind the last
    const int64_t lo = min(max((int64_t)q_start[0], (int64_t)0), n_tokens);
    const int64_t hi = min(max((int64_t)q_start[n_seq], lo), n_tokens), rows = lo + n_tokens - hi;
    const int64_t step = (int64_t)(gridDim.x - n_seq) * slices * kPlanThreads;
    const int64_t at = ((int64_t)(b - n_seq) * slices + slice) * kPlanThreads + tid;
    for (int64_t i = at; i < rows * words; i += step) mask[i < lo * words ? i : i + (hi - lo) * words] = 0;
    for (int64_t i = at; i < rows; i += step) positions[i < lo ? i : i + (hi - lo)] = -1;
    return;
  }
  const int64_t s = q_start[b], e = q_start[b + 1];
  const int64_t t0 = min(max(s, (int64_t)0), n_tokens);
  const int m = (int)max((int64_t)0, min(e, n_tokens) - t0);
  const int64_t pos0 = (int64_t)max(kv_lens[b], 0) - (e - s);
  const int32_t* const up = parents + t0;
  // an entry that does not name a token before its own makes that a root
  auto parent = [&](int i) __attribute__((always_inline)) {
    const int p = up[i];
    return p < i ? max(p, -1) : -1;
  };
  const int in_lds = min(m, kLdsNodes);
  for (int i = tid; i < in_lds; i += kPlanThreads) s_up[i] = parent(i);
  __syncthreads();
  for (int i = slice * kPlanThreads + tid; i < m; i += slices * kPlanThreads) {
    uint32_t* const row = mask + (t0 + i) * words;
    int j = i, depth = 0;
    for (int w = words - 1; w >= 0; --w) {
      uint32_t bits = 0;
      for (; j >= 32 * w; ++depth) {   // (j falls with every step)
        if ((j >> 5) == w) bits |= 1u << (j & 31);
        j = j < kLdsNodes ? s_up[j] : parent(j);
      }
      row[w] = bits;
    }
    positions[t0 + i] = (int32_t)(pos0 + depth - 1);
  }
}

hipError_t launch_plan_tree(int n_seq, const int32_t* parents, const int32_t* q_start, const int32_t* kv_lens,
                            int64_t n_tokens, int words, uint32_t* mask, int32_t* positions, hipStream_t st) {
  const int slices = (words + 7) / 8;
  const int64_t pad = std::min<int64_t>((256 + slices - 1) / slices, (n_tokens * words + 65535) / 65536);   // for rows of no sequence
  hipLaunchKernelGGL(k_plan_tree, dim3((unsigned)(n_seq + pad), (unsigned)slices), dim3(kPlanThreads), 0, st, n_seq, parents,
                     q_start, kv_lens, n_tokens, words, mask, positions);
  return hipGetLastError();
}

// Which entry of a path a lane reads for entry i: itself, or, where the path has none, its first or last one, whose
// value the lane does not use
__host__ __device__ constexpr int path_entry(int i, int max_path) { return i < 0 ? 0 : i < max_path ? i : max_path - 1; }
// in the path for every lane's entry and the one before it, of paths of one entry too
constexpr bool path_entries_inside(int max_path) {
  for (int i = -1; i < (max_path + 63) / 64 * 64; ++i) {
    const int at = path_entry(i, max_path);
    if (at < 0 || at >= max_path || (i >= 0 && i < max_path && at != i)) return false;
  }
  return true;
}
static_assert(path_entries_inside(1) && path_entries_inside(2) && path_entries_inside(63) && path_entries_inside(64) &&
              path_entries_inside(65) && path_entries_inside(130), "a path's loads stay in it");

// A workgroup takes a sequence (and, of wide rows, some of their pieces), a thread
// a piece of every row: 16 (or 8) bytes of the keys or values, or one scale.  Row i
// of the kept ones comes from place path[i] >= i, and path rises, so a thread that
// goes through the rows in order, reading a few and then writing them, reads
// every row before anything is written there: no other thread touches its pieces.
template <typename Piece>
__global__ void __launch_bounds__(256) k_keep_path(const KeepArgs a) {
  constexpr int U = 8;   // rows under way
  const int lane = threadIdx.x & 63, b = blockIdx.x;
  const int64_t s = a.q_start[b], e = a.q_start[b + 1];
  const int m = (int)min(max(e - s, (int64_t)0), (int64_t)0x7fffffff);
  const int64_t first = (int64_t)max(a.kv_lens[b], 0) - m;
  const int pieces = a.row_bytes / (int)sizeof(Piece);
  const int kv = a.v != nullptr ? 2 : 1;
  // this thread's piece of the K rows, the V rows, their scales
  const int item = blockIdx.y * blockDim.x + threadIdx.x;
  const bool is_row = item < kv * pieces;
  const int sc = item - kv * pieces;
  const bool is_scale = !is_row && a.k_scale != nullptr && sc < kv * a.n_heads;
  char* const base = item < pieces ? a.k : a.v;
  const int64_t col = (int64_t)(item < pieces ? item : item - pieces) * (int)sizeof(Piece);
  float* const sbase = sc < a.n_heads ? a.k_scale : a.v_scale;
  const int scol = sc < a.n_heads ? sc : sc - a.n_heads;
  // pool row of token t (below 2^31: the ABI bounds the pool), -1 where it has none
  auto slot = [&](int64_t t) __attribute__((always_inline)) -> int {
    const uint32_t u = (uint32_t)t, p = u / (uint32_t)a.page_keys;
    if (t < 0 || t > 0x7fffffff || p >= a.max_pages) return -1;
    const int entry = a.table[b * a.max_pages + p];
    return entry < 0 || entry >= a.n_pages ? -1 : entry * a.page_keys + (int)(u - p * (uint32_t)a.page_keys);
  };
  int kept = 0;
  for (int i0 = 0; i0 < a.max_path; i0 += 64) {
    const int i = i0 + lane;
    const int32_t* const path = a.path + (int64_t)b * a.max_path;
    const int node = path[path_entry(i, a.max_path)];
    const int last = path[path_entry(i - 1, a.max_path)], before = i > 0 ? last : -1;
    const bool ok = i < a.max_path && node > before && node >= 0 && node < m;
    const uint64_t gone = ~__ballot(ok);
    const int n = gone == 0 ? 64 : (int)__builtin_ctzll(gone);   // kept ones of these 64
    kept += n;
    // a row that stays, or has no place in the pages, moves nothing
    int src = -1, dst = -1;
    if (lane < n && node != i) {
      src = slot(first + node);
      dst = slot(first + i);
    }
    uint64_t moves = __ballot(src >= 0 && dst >= 0);
    while (moves != 0) {
      // (behind the last one it is read again: loads behind a branch would be waited for one by one)
      int from[U], to[U], l = 0, count = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (moves != 0) {
          l = (int)__builtin_ctzll(moves);
          moves &= moves - 1;
          ++count;
        }
        from[u] = __builtin_amdgcn_readlane(src, l);
        to[u] = __builtin_amdgcn_readlane(dst, l);
      }
      if (is_row) {
        Piece x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = *reinterpret_cast<const Piece*>(base + (int64_t)from[u] * a.row_bytes + col);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < count) *reinterpret_cast<Piece*>(base + (int64_t)to[u] * a.row_bytes + col) = x[u];
      } else if (is_scale) {
        float x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = sbase[(int64_t)from[u] * a.n_heads + scol];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < count) sbase[(int64_t)to[u] * a.n_heads + scol] = x[u];
      }
    }
    if (n < 64) break;
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) a.kept_lens[b] = (int32_t)max((int64_t)0, first + kept);
}

template <typename Piece>
static hipError_t launch_keep(int n_seq, const KeepArgs& a, hipStream_t st) {
  const int items = (a.v != nullptr ? 2 : 1) * (a.row_bytes / (int)sizeof(Piece) + (a.k_scale != nullptr ? a.n_heads : 0));
  const int threads = items <= 64 ? 64 : items <= 128 ? 128 : 256;
  hipLaunchKernelGGL(k_keep_path<Piece>, dim3((unsigned)n_seq, (unsigned)((items + threads - 1) / threads)), dim3(threads), 0,
                     st, a);
  return hipGetLastError();
}

hipError_t launch_keep_path(int n_seq, const KeepArgs& a, hipStream_t st) {
  return a.row_bytes % 16 == 0 ? launch_keep<uint4>(n_seq, a, st) : launch_keep<uint2>(n_seq, a, st);
}

}  // namespace misa
