// Block tables, slot maps and the split-KV plan, made on the GPU.
//
// All of it is integer bookkeeping over B requests (tens to thousands) whose
// answers the host would otherwise compute and copy every step: what a step
// costs is latency, so each job is one launch of one block of 1024 threads
// with block-wide scans, and only a slot map of many tokens gets a second,
// wide launch (bound by writing 8 bytes per token).  From a graph: tables 4.5 us and
// plan 5.2 for 32 requests with one new token each; tables 16.1 us for 509 requests
// with about a million new tokens (their 8500 page entries go through the one block),
// and the plan of their 1018 rows 9.9.
#include "block_scan.cuh"
#include "mla_internal.h"
#include "plan_device.cuh"
#include "plan_format.h"
#include "ptx.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kThreads = 1024;
constexpr int kPage = 64;

__device__ __forceinline__ void report(int32_t* status, int bits) {
  if (status) atomicOr(status, bits);
}

struct TablesParams {
  int B, max_blocks, n_free, num_blocks, max_new;
  const int32_t* cached;
  const int32_t* fresh;
  int32_t* table;
  int32_t* held;   // pages that the rows of the table hold, or null (then those of the cached tokens)
  const int32_t* free_blocks;
  const int32_t* head_in;
  int32_t* seq_lens;
  int32_t* cu_new;
  int32_t* slots;
  int32_t* positions;
  int32_t* head_out;
  int32_t* status;
  int fill;   // non-zero: this launch writes the slot map too
};

// One block.  Requests are taken 1024 at a time, one thread each, with running
// totals of the new pages and new tokens before them; then the block's threads
// take the chunk's new pages, and its new tokens, one each (the owner by a
// binary search over the chunk's sums in shared memory), so that one long
// prompt does not make one thread loop.
__global__ void __launch_bounds__(kThreads)
build_tables_kernel(const TablesParams p) {
  __shared__ long long ws[32];
  __shared__ int s_pages[kThreads], s_tokens[kThreads];       // inclusive sums over the chunk, admitted requests
  __shared__ int s_held[kThreads], s_cached[kThreads];
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x;
  const int head_raw = *p.head_in;
  const int head = head_raw < 0 || head_raw > p.n_free ? p.n_free : head_raw;
  if (head != head_raw && t == 0) report(p.status, MLA_STATUS_NO_SPACE);
  long long pages_before = 0;                     // of the requests that are valid, admitted or not
  long long asked_before = 0;                     // of those that get their pages
  int used = head, tokens_before = 0;             // admitted ones
  if (t == 0) p.cu_new[0] = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + t;
    const int old = b < p.B ? p.cached[b] : 0, add = b < p.B ? p.fresh[b] : 0;
    const int in_row = p.held && b < p.B ? p.held[b] : 0;
    const bool valid = old >= 0 && add >= 0 && (long long)old + add <= (long long)p.max_blocks * kPage && in_row <= p.max_blocks;
    const int held = valid ? max(in_row, (old + kPage - 1) / kPage) : 0;
    const int need = valid ? max((old + add + kPage - 1) / kPage - held, 0) : 0;
    const int want = valid ? add : 0;
    long long pages_all, asked_all;
    const long long pages_incl = pages_before + block_scan<long long>(need, ws, &pages_all);
    // (a request refused for its blocks asks for no room in the slot map)
    const bool has_pages = valid && (need == 0 || head + pages_incl <= p.n_free);
    const long long asked_incl = asked_before + block_scan<long long>(has_pages ? want : 0, ws, &asked_all);
    const bool admitted = has_pages && (want == 0 || asked_incl <= p.max_new);
    if (b < p.B && !admitted) report(p.status, MLA_STATUS_NO_SPACE);
    int pages_sum = (int)(pages_incl - pages_before), tokens_sum = (int)(asked_incl - asked_before);
    int pages_now = (int)pages_all, tokens_now = (int)asked_all;
    if (!__syncthreads_and(admitted || want == 0)) {   // some request does not fit: sums of those that do
      long long a, c;
      pages_sum = (int)block_scan<long long>(admitted ? need : 0, ws, &a);
      tokens_sum = (int)block_scan<long long>(admitted ? want : 0, ws, &c);
      pages_now = (int)a;
      tokens_now = (int)c;
    }
    s_pages[t] = pages_sum;
    s_tokens[t] = tokens_sum;
    s_held[t] = held;
    s_cached[t] = old;
    if (b < p.B) {
      p.cu_new[b + 1] = tokens_before + tokens_sum;
      p.seq_lens[b] = admitted ? old + add : max(old, 0);
      if (p.held && admitted) p.held[b] = held + need;
    }
    __syncthreads();
    // Pages, then tokens: one each per thread, or four neighbours when there are more
    // than threads, so that a search finds the request of the first and the
    // others' follow by stepping on.
    const int per_p = pages_now > kThreads ? 4 : 1;
    for (int e0 = t * per_p; e0 < pages_now; e0 += kThreads * per_p) {
      int i = find_owner(s_pages, kThreads, e0);
      int blk[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) blk[u] = u < per_p && e0 + u < pages_now ? p.free_blocks[used + e0 + u] : -1;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = e0 + u;
        if (u >= per_p || e >= pages_now) break;
        while (s_pages[i] <= e) ++i;
        if (blk[u] < 0 || blk[u] >= p.num_blocks) report(p.status, MLA_STATUS_BAD_BLOCK);
        p.table[(size_t)(b0 + i) * p.max_blocks + s_held[i] + e - (i > 0 ? s_pages[i - 1] : 0)] = blk[u];
      }
    }
    __syncthreads();   // the new table entries are read below
    if (p.fill) {
      const int per_t = tokens_now > kThreads ? 4 : 1;
      for (int e0 = t * per_t; e0 < tokens_now; e0 += kThreads * per_t) {
        int i = find_owner(s_tokens, kThreads, e0);
        int blk[4], pos[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int e = e0 + u;
          if (u >= per_t || e >= tokens_now) break;
          while (s_tokens[i] <= e) ++i;
          pos[u] = s_cached[i] + e - (i > 0 ? s_tokens[i - 1] : 0);
          blk[u] = __ldcg(p.table + (size_t)(b0 + i) * p.max_blocks + pos[u] / kPage);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int e = e0 + u;
          if (u >= per_t || e >= tokens_now) break;
          const bool ok = blk[u] >= 0 && blk[u] < p.num_blocks;
          if (!ok) report(p.status, MLA_STATUS_BAD_BLOCK);
          p.slots[tokens_before + e] = ok ? blk[u] * kPage + pos[u] % kPage : -1;
          if (p.positions) p.positions[tokens_before + e] = pos[u];
        }
      }
    }
    pages_before += pages_all;
    asked_before += asked_all;
    used += pages_now;
    tokens_before += tokens_now;
    __syncthreads();   // the chunk's sums are rewritten next
  }
  if (t == 0) *p.head_out = used;
  if (p.fill) {
    for (int e = tokens_before + t; e < p.max_new; e += kThreads) {
      p.slots[e] = -1;
      if (p.positions) p.positions[e] = -1;
    }
  }
}

// The slot map of many tokens: a block takes 2048 of them, 8 per thread.  The
// requests of its first and last token come from two rounds of one comparison
// per thread and a count over the block (stride B / 256, then one by one), since a
// binary search would put ten dependent reads in front of everything; within
// that range a token's request is found by a short search.
constexpr int kFillThreads = 256, kFillTokens = 8;

__global__ void __launch_bounds__(kFillThreads)
fill_slots_kernel(const TablesParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x;
  const int first = blockIdx.x * (kFillThreads * kFillTokens);
  const int total = p.cu_new[p.B];
  const int last = min(first + kFillThreads * kFillTokens, total) - 1;
  int lo = 0, hi = 0;
  if (first < total) {   // (block-uniform) requests that end at or before a token come before its own
    const int step = (p.B + kFillThreads - 1) / kFillThreads;
    const int end = (t + 1) * step <= p.B ? p.cu_new[(t + 1) * step] : INT32_MAX;
    const int lo0 = __syncthreads_count(end <= first) * step, hi0 = __syncthreads_count(end <= last) * step;
    const int end_lo = t < step && lo0 + t < p.B ? p.cu_new[lo0 + t + 1] : INT32_MAX;
    const int end_hi = t < step && hi0 + t < p.B ? p.cu_new[hi0 + t + 1] : INT32_MAX;
    lo = lo0 + __syncthreads_count(end_lo <= first);
    hi = hi0 + __syncthreads_count(end_hi <= last);
  }
#pragma unroll 4
  for (int i = 0; i < kFillTokens; ++i) {
    const int e = first + i * kFillThreads + t;
    if (e >= p.max_new) break;
    int slot = -1, pos = -1;
    if (e < total) {
      int b = lo, z = hi;
      while (b < z) {
        const int mid = (b + z) >> 1;
        if (p.cu_new[mid + 1] > e) z = mid; else b = mid + 1;
      }
      pos = p.seq_lens[b] + e - p.cu_new[b + 1];
      const int blk = p.table[(size_t)b * p.max_blocks + pos / kPage];
      if (blk >= 0 && blk < p.num_blocks) slot = blk * kPage + pos % kPage;
      else report(p.status, MLA_STATUS_BAD_BLOCK);
    }
    p.slots[e] = slot;
    if (p.positions) p.positions[e] = pos;
  }
}

// ---------------------------------------------------------------- the plan
// Keys of row (T, qi); 0 for a padded or inconsistent row.
__device__ __forceinline__ int row_keys(const PlanShape& p, int T, int qi, bool* bad) {
  if (T == 0) return 0;
  if (T < p.s_q || (long long)T > (long long)p.max_blocks * kPage) {
    *bad = true;
    return 0;
  }
  return p.causal ? T - p.s_q + 1 + qi : T;
}

__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const PlanShape p, const int32_t* seq_lens, int32_t* plan, int32_t* status) {
  __shared__ PlanScratch scratch;
  griddep_wait();
  griddep_launch_dependents();
  bool bad = false;
  make_plan(p, scratch, plan, [&](int n) { return row_keys(p, seq_lens[n / p.s_q], n % p.s_q, &bad); });
  if (bad) report(status, MLA_STATUS_BAD_SEQLEN);
}

}  // namespace

// Slot maps up to this many tokens are written by the one block that makes the
// tables (7 tokens per thread); longer ones by a launch of their own.  32 requests, from a
// graph, in one block against two launches: 32 tokens 3.7 against 5.0 us, 2048
// 5.5 against 9.7, 8192 9.7 against 8.1, 16384 15.5 against 7.9, 131072 93 against 7.7.
constexpr int kOneBlockTokens = 7168;

mla_status_t launch_build_tables(int B, const int32_t* cached_lens, const int32_t* new_lens, int max_blocks,
                                 int32_t* block_table, int32_t* held_pages, const int32_t* free_blocks, int n_free,
                                 const int32_t* free_head, int num_blocks, int max_new, int32_t* seq_lens,
                                 int32_t* cu_new, int32_t* slots, int32_t* positions, int32_t* free_head_out,
                                 int32_t* status, void* stream) {
  TablesParams p = {B, max_blocks, n_free, num_blocks, max_new, cached_lens, new_lens, block_table, held_pages,
                    free_blocks, free_head, seq_lens, cu_new, slots, positions, free_head_out, status,
                    max_new <= kOneBlockTokens ? 1 : 0};
  cudaError_t e = launch_pdl(build_tables_kernel, dim3(1), dim3(kThreads), 0, stream, p);
  if (e == cudaSuccess && !p.fill) {
    const int per_block = kFillThreads * kFillTokens;
    e = launch_pdl(fill_slots_kernel, dim3((unsigned)(((long long)max_new + per_block - 1) / per_block)),
                   dim3(kFillThreads), 0, stream, p);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(MLA_ERR_CUDA, "build_tables launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

mla_status_t launch_plan(const mla_dims_t& d, const int32_t* seq_lens, int num_clusters, int32_t* plan,
                         int32_t* status, void* stream) {
  const PlanShape p = {d.B, d.s_q, d.n_heads, d.max_blocks_per_seq, d.causal, num_clusters,
                       (int)plan_words_upper_bound(num_clusters, d.B * d.s_q)};
  cudaError_t e = launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p, seq_lens, plan, status);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(MLA_ERR_CUDA, "plan launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

}  // namespace mla
