// Block tables and slot maps from request lengths (misa_plan_pages).
//
// Everything follows from two exclusive sums over the sequences: the new
// tokens (q_start) and the new pages (the offset into the free list).  One
// launch does it all: every workgroup forms both sums for itself (n_seq
// lengths are a few KB that the L2 holds), because the alternative, a scan
// launch before the fill, costs a second launch on a call whose whole work is
// shorter than one.
//
// Sums: thread i sums a run of ceil(n_seq / 256) sequences, the 256 run sums
// are scanned by wave shuffles and kept in LDS (s_tok, s_page: first token and
// first page of each run).  A token finds its run by a binary search in LDS (8
// steps) and its sequence by walking the run; with up to 256 sequences a run
// is one sequence and the walk is empty.  Past 1024 sequences the runs are 256
// long and scanned into LDS in their turn (k_plan_many).
// Sums are 64-bit: n_seq lengths of up to 2^31 pass 32 bits.
//
// Bound by the chain lengths -> sums -> search -> free list -> slots, not by bytes:
// 3.7 us for 64 decodes, 6.9 us for 500 prompts of 1..1024 tokens (3.1 MB; four
// tokens a thread 9.1), a call's 17.6 us for 2000 of them and 78 us for 60000
// sequences of 1..16 (walking longer runs: 28 and 482).
#include <algorithm>

#include "misa_common.h"
#include "misa_launch.h"

namespace misa {

namespace {
constexpr int kThreads = 256;

struct SeqPages {
  int64_t cached, fresh;   // token counts, negative ones taken as 0
  int32_t have, need;      // pages owned, pages to take (both within the table)
};

__device__ __forceinline__ SeqPages seq_pages(const int32_t* cached, const int32_t* fresh, int b, uint32_t P,
                                              int64_t max_pages) {
  SeqPages r;
  r.cached = max(cached[b], 0);
  r.fresh = max(fresh[b], 0);
  // ceil(x / P) of x < 2^32 in 32-bit arithmetic
  const uint32_t c = (uint32_t)r.cached, e = c + (uint32_t)r.fresh;
  const int64_t have = min((int64_t)(c / P + (c % P != 0)), max_pages);
  const int64_t end = min((int64_t)(e / P + (e % P != 0)), max_pages);
  r.have = (int32_t)have;
  r.need = (int32_t)(end - have);
  return r;
}

// last i in [0, 256) with s[i] <= x (s ascending, s[0] <= x)
__device__ __forceinline__ int run_of(const int64_t* s, int64_t x) {
  int lo = 0;
#pragma unroll
  for (int step = kThreads / 2; step >= 1; step >>= 1)
    if (s[lo + step] <= x) lo += step;
  return lo;
}

// Exclusive sums over the workgroup's threads, and the totals
struct Sums {
  int64_t tok, page, all_tok, all_page;
};
__device__ __forceinline__ Sums scan(int64_t tok, int64_t page, int64_t (*s_wave)[kThreads / kWave]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t tok_in = tok, page_in = page;   // inclusive over the wave
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int64_t a = __shfl_up(tok_in, o), c = __shfl_up(page_in, o);
    if (lane >= o) {
      tok_in += a;
      page_in += c;
    }
  }
  if (lane == kWave - 1) {
    s_wave[0][wave] = tok_in;
    s_wave[1][wave] = page_in;
  }
  __syncthreads();
  Sums r{tok_in - tok, page_in - page, 0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / kWave; ++w) {
    if (w < wave) {
      r.tok += s_wave[0][w];
      r.page += s_wave[1][w];
    }
    r.all_tok += s_wave[0][w];
    r.all_page += s_wave[1][w];
  }
  return r;
}

struct PlanArgs {
  int n_seq;
  const int32_t *cached_lens, *new_lens;
  uint32_t P;
  const int32_t* free_pages;
  int n_free;
  int32_t* block_table;
  int64_t max_pages;
  int32_t *q_start, *kv_lens;
  int64_t* slots;
  int32_t* positions;
  int64_t n_tokens;
  int32_t* n_taken;

  __device__ __forceinline__ SeqPages seq(int b) const { return seq_pages(cached_lens, new_lens, b, P, max_pages); }
  __device__ __forceinline__ int32_t taken(int64_t r) const { return r < n_free ? free_pages[r] : -1; }

  // Slot and position of new token i of sequence b, whose first page taken is pfirst.
  // Page ids come from the free list itself (or the row's old entries), never
  // from entries another workgroup may be writing.
  __device__ __forceinline__ void token(int64_t t, int b, const SeqPages& sp, int64_t i, int64_t pfirst) const {
    const uint32_t p = (uint32_t)sp.cached + (uint32_t)i;
    const uint32_t pg = p / P;
    int32_t id = -1;
    if ((int64_t)pg < sp.have) id = block_table[(int64_t)b * max_pages + pg];
    else if ((int64_t)pg < (int64_t)sp.have + sp.need) id = taken(pfirst + pg - sp.have);
    slots[t] = id >= 0 ? (int64_t)id * P + (p - pg * P) : -1;
    positions[t] = (int32_t)min(p, (uint32_t)INT32_MAX);
  }
  __device__ __forceinline__ void lengths(int b, int64_t first, const SeqPages& sp) const {
    q_start[b] = (int32_t)min(first, (int64_t)INT32_MAX);
    kv_lens[b] = (int32_t)min(sp.cached + sp.fresh, (int64_t)INT32_MAX);
  }
  __device__ __forceinline__ void totals(const Sums& all) const {
    q_start[n_seq] = (int32_t)min(all.all_tok, (int64_t)INT32_MAX);
    n_taken[0] = (int32_t)min(all.all_page, (int64_t)INT32_MAX);
  }
};
}  // namespace

// NT: tokens a thread
template <int NT>
__global__ void __launch_bounds__(kThreads) k_plan_pages(const PlanArgs a) {
  __shared__ int64_t s_tok[kThreads], s_page[kThreads];
  __shared__ int64_t s_wave[2][kThreads / kWave];
  const int tid = threadIdx.x;
  const int run = (a.n_seq + kThreads - 1) / kThreads;
  const int b0 = min(tid * run, a.n_seq), b1 = min(b0 + run, a.n_seq);

  int64_t tok = 0, page = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqPages sp = a.seq(b);
    tok += sp.fresh;
    page += sp.need;
  }
  const Sums at = scan(tok, page, s_wave);
  s_tok[tid] = at.tok;
  s_page[tid] = at.page;
  __syncthreads();

  if (blockIdx.x == 0) {
    int64_t t = at.tok;
    for (int b = b0; b < b1; ++b) {
      const SeqPages sp = a.seq(b);
      a.lengths(b, t, sp);
      t += sp.fresh;
    }
    if (tid == 0) a.totals(at);
  }

  // the new table entries
  for (int64_t r = (int64_t)blockIdx.x * kThreads + tid; r < at.all_page; r += (int64_t)gridDim.x * kThreads) {
    const int u = run_of(s_page, r);
    int64_t first = s_page[u];
    for (int b = u * run; b < min((u + 1) * run, a.n_seq); ++b) {
      const SeqPages sp = a.seq(b);
      if (r < first + sp.need) {
        a.block_table[(int64_t)b * a.max_pages + sp.have + (r - first)] = a.taken(r);
        break;
      }
      first += sp.need;
    }
  }

  // the tokens
  const int64_t t0 = (int64_t)blockIdx.x * (kThreads * NT) + tid;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t t = t0 + i * kThreads;
    if (t >= a.n_tokens) break;
    if (t >= at.all_tok) {
      a.slots[t] = -1;
      a.positions[t] = -1;
      continue;
    }
    const int u = run_of(s_tok, t);
    int64_t first = s_tok[u], pfirst = s_page[u];
    for (int b = u * run; b < min((u + 1) * run, a.n_seq); ++b) {
      const SeqPages sp = a.seq(b);
      if (t < first + sp.fresh) {
        a.token(t, b, sp, t - first, pfirst);
        break;
      }
      first += sp.fresh;
      pfirst += sp.need;
    }
  }
}

// More sequences: runs of 256, whose sums the waves form side by side; a workgroup
// writes the lengths and table entries of whole runs, and goes through the runs
// that its tokens lie in, each scanned into LDS first.
__global__ void __launch_bounds__(kThreads) k_plan_many(const PlanArgs a) {
  __shared__ int64_t s_tok[kThreads], s_page[kThreads];   // first token and page of each run
  __shared__ int64_t r_tok[kThreads], r_page[kThreads];   // of each sequence of a run
  __shared__ int64_t s_wave[2][kThreads / kWave];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n_runs = (a.n_seq + kThreads - 1) / kThreads;   // at most 256: n_seq < 65536
  for (int u = wave; u < n_runs; u += kThreads / kWave) {
    int64_t tok = 0, page = 0;
#pragma unroll
    for (int i = 0; i < kThreads / kWave; ++i) {
      const int b = u * kThreads + i * kWave + lane;
      const SeqPages sp = a.seq(min(b, a.n_seq - 1));
      tok += b < a.n_seq ? sp.fresh : 0;
      page += b < a.n_seq ? sp.need : 0;
    }
#pragma unroll
    for (int x = kWave / 2; x >= 1; x >>= 1) {
      tok += __shfl_xor(tok, x);
      page += __shfl_xor(page, x);
    }
    if (lane == 0) {
      r_tok[u] = tok;
      r_page[u] = page;
    }
  }
  __syncthreads();
  const Sums at = scan(tid < n_runs ? r_tok[tid] : 0, tid < n_runs ? r_page[tid] : 0, s_wave);
  s_tok[tid] = at.tok;
  s_page[tid] = at.page;
  auto end_of = [&](const int64_t* s, int u, int64_t all) { return u + 1 < kThreads ? s[u + 1] : all; };
  auto load_run = [&](int u) {   // this thread's sequence of run u, and all of the run's first tokens and pages in LDS
    __syncthreads();
    const int b = u * kThreads + tid;
    SeqPages sp = a.seq(min(b, a.n_seq - 1));
    if (b >= a.n_seq) sp.fresh = sp.need = 0;
    const Sums in = scan(sp.fresh, sp.need, s_wave);
    r_tok[tid] = s_tok[u] + in.tok;
    r_page[tid] = s_page[u] + in.page;
    __syncthreads();
    return sp;
  };

  for (int u = blockIdx.x; u < n_runs; u += gridDim.x) {
    const SeqPages sp = load_run(u);
    if (u * kThreads + tid < a.n_seq) a.lengths(u * kThreads + tid, r_tok[tid], sp);
    const int64_t end = end_of(s_page, u, at.all_page);
    for (int64_t r = s_page[u] + tid; r < end; r += kThreads) {
      const int i = run_of(r_page, r), b = u * kThreads + i;
      a.block_table[(int64_t)b * a.max_pages + a.seq(b).have + (r - r_page[i])] = a.taken(r);
    }
  }
  if (blockIdx.x == 0 && tid == 0) a.totals(at);

  constexpr int NT = 4;
  const int64_t t0 = (int64_t)blockIdx.x * (kThreads * NT);
  const int64_t t1 = min(t0 + kThreads * NT, a.n_tokens), live = min(t1, at.all_tok);
  for (int64_t t = max(live, t0) + tid; t < t1; t += kThreads) {
    a.slots[t] = -1;
    a.positions[t] = -1;
  }
  __syncthreads();   // (s_tok)
  if (t0 >= live) return;
  const int last = run_of(s_tok, live - 1);
  for (int u = run_of(s_tok, t0); u <= last; ++u) {
    const int64_t first = s_tok[u], end = min(end_of(s_tok, u, at.all_tok), live);
    if (first >= end) continue;
    load_run(u);
    for (int64_t t = t0 + tid; t < end; t += kThreads) {
      if (t < first) continue;
      const int i = run_of(r_tok, t), b = u * kThreads + i;
      a.token(t, b, a.seq(b), t - r_tok[i], r_page[i]);
    }
  }
}

hipError_t launch_plan_pages(int n_seq, const int32_t* cached_lens, const int32_t* new_lens, int page_keys,
                             const int32_t* free_pages, int n_free, int32_t* block_table, int64_t max_pages,
                             int32_t* q_start, int32_t* kv_lens, int64_t* slots, int32_t* positions, int64_t n_tokens,
                             int32_t* n_taken, hipStream_t st) {
  const PlanArgs a{n_seq, cached_lens, new_lens, (uint32_t)page_keys, free_pages, n_free, block_table, max_pages,
                   q_start, kv_lens, slots, positions, n_tokens, n_taken};
  // Up to 1024 sequences a thread sums its run of at most four by itself.  A token
  // is a chain of dependent reads, so one a thread while the GPU holds all
  // workgroups at a time; beyond that fewer workgroups, which repeat the sums.
  const bool many = n_seq > 4 * kThreads;
  const int nt = !many && n_tokens <= (int64_t)2048 * kThreads ? 1 : 4;
  const int64_t per = (int64_t)kThreads * nt;
  int64_t blocks = std::max<int64_t>(1, (n_tokens + per - 1) / per);
  if (many) blocks = std::max<int64_t>(blocks, (n_seq + kThreads - 1) / kThreads);
  const auto kernel = many ? k_plan_many : nt == 1 ? k_plan_pages<1> : k_plan_pages<4>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace misa
