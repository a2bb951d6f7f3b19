// Block tables, slot maps and the split-KV plan, made on the GPU.
//
// All of it is integer bookkeeping over B requests (tens to thousands) whose
// answers the host would otherwise compute and copy every step: what a step
// costs is latency, so each job is one launch of one block of 1024 threads
// with block-wide scans, and only a slot map of many tokens gets a second,
// wide launch (bound by writing 8 bytes per token).
#include "block_scan.cuh"
#include "mla_internal.h"
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

// First index in [0, n) whose inclusive sum exceeds e (sums[n - 1] > e).
__device__ __forceinline__ int find_owner(const int* sums, int n, int e) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] > e) hi = mid; else lo = mid + 1;
  }
  return lo;
}

struct TablesParams {
  int B, max_blocks, n_free, num_blocks, max_new;
  const int32_t* cached;
  const int32_t* fresh;
  int32_t* table;
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
  long long pages_before = 0, asked_before = 0;   // of the requests that are valid, admitted or not
  int used = head, tokens_before = 0;             // admitted ones
  if (t == 0) p.cu_new[0] = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    const int b = b0 + t;
    const int old = b < p.B ? p.cached[b] : 0, add = b < p.B ? p.fresh[b] : 0;
    const bool valid = old >= 0 && add >= 0 && (long long)old + add <= (long long)p.max_blocks * kPage;
    const int held = valid ? (old + kPage - 1) / kPage : 0;
    const int need = valid ? (old + add + kPage - 1) / kPage - held : 0;
    const int want = valid ? add : 0;
    long long pages_all, asked_all;
    const long long pages_incl = pages_before + block_scan<long long>(need, ws, &pages_all);
    const long long asked_incl = asked_before + block_scan<long long>(want, ws, &asked_all);
    const bool admitted = valid && (want == 0 || ((need == 0 || head + pages_incl <= p.n_free) && asked_incl <= p.max_new));
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
    }
    __syncthreads();
    for (int e = t; e < pages_now; e += kThreads) {
      const int i = find_owner(s_pages, kThreads, e);
      const int rank = e - (i > 0 ? s_pages[i - 1] : 0);
      const int blk = p.free_blocks[used + e];
      if (blk < 0 || blk >= p.num_blocks) report(p.status, MLA_STATUS_BAD_BLOCK);
      p.table[(size_t)(b0 + i) * p.max_blocks + s_held[i] + rank] = blk;
    }
    __syncthreads();   // the new table entries are read below
    if (p.fill) {
      for (int e = t; e < tokens_now; e += kThreads) {
        const int i = find_owner(s_tokens, kThreads, e);
        const int pos = s_cached[i] + e - (i > 0 ? s_tokens[i - 1] : 0);
        const int blk = __ldcg(p.table + (size_t)(b0 + i) * p.max_blocks + pos / kPage);
        const bool ok = blk >= 0 && blk < p.num_blocks;
        if (!ok) report(p.status, MLA_STATUS_BAD_BLOCK);
        p.slots[tokens_before + e] = ok ? blk * kPage + pos % kPage : -1;
        if (p.positions) p.positions[tokens_before + e] = pos;
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

// The slot map of many tokens: a thread per token and 8 tokens per thread, the
// block's range of requests found once (the offsets are read through L1).
constexpr int kFillThreads = 256, kFillTokens = 8;

__global__ void __launch_bounds__(kFillThreads)
fill_slots_kernel(const TablesParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int first = blockIdx.x * (kFillThreads * kFillTokens);
  const int total = p.cu_new[p.B];
  const int last = min(first + kFillThreads * kFillTokens, total) - 1;
  auto owner = [&](int e, int lo, int hi) {   // request of token e, known to lie in [lo, hi]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (p.cu_new[mid + 1] > e) hi = mid; else lo = mid + 1;
    }
    return lo;
  };
  int lo = 0, hi = 0;
  if (first < total) {
    lo = owner(first, 0, p.B - 1);
    hi = owner(last, lo, p.B - 1);
  }
#pragma unroll 4
  for (int i = 0; i < kFillTokens; ++i) {
    const int e = first + i * kFillThreads + threadIdx.x;
    if (e >= p.max_new) break;
    int slot = -1, pos = -1;
    if (e < total) {
      const int b = owner(e, lo, hi);
      const int begin = p.cu_new[b], end = p.cu_new[b + 1];
      pos = p.seq_lens[b] - (end - begin) + (e - begin);
      const int blk = p.table[(size_t)b * p.max_blocks + pos / kPage];
      if (blk >= 0 && blk < p.num_blocks) slot = blk * kPage + pos % kPage;
      else report(p.status, MLA_STATUS_BAD_BLOCK);
    }
    p.slots[e] = slot;
    if (p.positions) p.positions[e] = pos;
  }
}

// ---------------------------------------------------------------- the plan
// The rule of the host planner (plan.cpp), word for word: the rows of a group
// laid end to end, each behind kItemCostPages virtual pages, cut at
// floor(c P / G).  With P >= G every range holds a unit, so a row's pieces are
// the ranges between those of its first and last page; with P < G every unit
// is a range of its own.  The range that holds unit u is the largest c with
// floor(c P / G) <= u, that is floor(((u + 1) G - 1) / P).
//
// One block: (1) the groups' totals; (2) rows in (group, row) order, 1024 at a
// time: offsets by a scan, pieces, items (that order is also the order by
// cluster); (3) partial slots in row order; (4) slots into the items; (5) the
// clusters' first items.  Rows of length 0 (a padded batch) get no item: their
// outputs are left as they are.
struct PlanParams {
  int B, s_q, n_heads, max_blocks, causal, num_clusters;
  const int32_t* seq_lens;
  int32_t* plan;
  int words;          // plan_words_upper_bound
  int32_t* status;
};

// Keys of row (T, qi); 0 for a padded or inconsistent row.
__device__ __forceinline__ int row_keys(const PlanParams& p, int T, int qi, bool* bad) {
  if (T == 0) return 0;
  if (T < p.s_q || (long long)T > (long long)p.max_blocks * kPage) {
    *bad = true;
    return 0;
  }
  return p.causal ? T - p.s_q + 1 + qi : T;
}

__global__ void __launch_bounds__(kThreads)
plan_kernel(const PlanParams p) {
  extern __shared__ int s_cl[];                       // [num_clusters + 1] items per cluster, then their begins
  __shared__ long long ws[32];
  __shared__ int wi[32];
  __shared__ long long s_total[8];
  __shared__ long long s_r0[kThreads];
  __shared__ int s_first[kThreads], s_sum[kThreads], s_row[kThreads], s_pages[kThreads], s_kv[kThreads];
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x;
  const int N = p.B * p.s_q;
  const int groups = p.num_clusters >= p.s_q ? p.s_q : 1;
  const long long G = p.num_clusters / groups;
  const int per_group = groups == 1 ? N : p.B;        // rows of a group
  int32_t* plan = p.plan;
  const int off_cluster = kPlanHeaderWords, off_items = off_cluster + p.num_clusters + 1;
  int32_t* items = plan + off_items;
  // pieces of row n, kept behind the last word that this plan can use until the
  // row section, whose place follows from the item count, is written over it
  // (each row's entry is read before any entry at or above it is overwritten)
  int32_t* pieces_of = plan + p.words - (N + 1);
  for (int c = t; c <= p.num_clusters; c += kThreads) s_cl[c] = 0;
  if (t < 8) s_total[t] = 0;
  __syncthreads();
  // (1)
  bool bad = false;
  for (int g = 0; g < groups; ++g) {
    long long sum = 0;
    for (int k = t; k < per_group; k += kThreads) {
      const int n = groups == 1 ? k : k * p.s_q + g;
      const int kv = row_keys(p, p.seq_lens[n / p.s_q], n % p.s_q, &bad);
      if (kv > 0) sum += kItemCostPages + (kv + kPage - 1) / kPage;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if ((t & 31) == 0 && sum > 0) atomicAdd(reinterpret_cast<unsigned long long*>(&s_total[g]), (unsigned long long)sum);
  }
  if (bad) report(p.status, MLA_STATUS_BAD_SEQLEN);
  __syncthreads();
  // (2)
  int items_before = 0;
  for (int g = 0; g < groups; ++g) {
    const long long P = s_total[g];
    long long line_before = 0;
    for (int k0 = 0; k0 < per_group; k0 += kThreads) {
      const int k = k0 + t;
      const int n = groups == 1 ? k : k * p.s_q + g;
      const int kv = k < per_group ? row_keys(p, p.seq_lens[n / p.s_q], n % p.s_q, &bad) : 0;
      const int pages = (kv + kPage - 1) / kPage;
      const int cost = pages > 0 ? pages + kItemCostPages : 0;
      long long line_all;
      const long long r1 = line_before + block_scan<long long>(cost, ws, &line_all);
      const long long r0 = r1 - pages;
      int first = 0, pieces = 0;
      if (pages > 0) {
        first = (int)(((r0 + 1) * G - 1) / P);
        pieces = P >= G ? (int)((r1 * G - 1) / P) - first + 1 : pages;
      }
      int pieces_all;
      const int sum = block_scan<int>(pieces, wi, &pieces_all);
      s_first[t] = first;
      s_sum[t] = sum;
      s_row[t] = n;
      s_pages[t] = pages;
      s_kv[t] = kv;
      s_r0[t] = r0;
      if (k < per_group) pieces_of[n] = pieces;
      __syncthreads();
      for (int e = t; e < pieces_all; e += kThreads) {
        const int i = find_owner(s_sum, kThreads, e);
        const int j = e - (i > 0 ? s_sum[i - 1] : 0);
        const long long a0 = s_r0[i], a1 = a0 + s_pages[i];
        const long long c = P >= G ? (long long)s_first[i] + j : ((a0 + j + 1) * G - 1) / P;
        const long long lo = c * P / G, hi = (c + 1) * P / G;
        const long long a = lo > a0 ? lo : a0, z = hi < a1 ? hi : a1;
        const int cluster = g * (int)G + (int)c;
        int32_t* w = items + (size_t)(items_before + e) * kItemWords;
        w[kItB] = s_row[i] / p.s_q;
        w[kItQi] = s_row[i] % p.s_q;
        w[kItPageBegin] = (int)(a - a0);
        w[kItPageEnd] = (int)(z - a0);
        w[kItKvLen] = s_kv[i];
        w[kItSlot] = j;                               // its place among the row's pieces, for now
        w[kItRow] = s_row[i];
        w[kItRow + 1] = 0;
        atomicAdd(&s_cl[cluster + 1], 1);
      }
      items_before += pieces_all;
      line_before += line_all;
      __syncthreads();
    }
  }
  const int I = items_before;
  const int off_rows = off_items + I * kItemWords;
  int32_t* rows = plan + off_rows;
  // (3)
  int slots_before = 0;
  for (int n0 = 0; n0 < N; n0 += kThreads) {
    const int n = n0 + t;
    const int pieces = n < N ? pieces_of[n] : 0;
    const int own = pieces > 1 ? pieces : 0;
    int all;
    const int sum = block_scan<int>(own, wi, &all);   // (its barriers also order the read above before the writes below)
    if (n < N) rows[n] = slots_before + sum - own;
    slots_before += all;
  }
  if (t == 0) rows[N] = slots_before;
  __syncthreads();
  // (4) a row is split if its slots differ from the next row's
  for (int e = t; e < I; e += kThreads) {
    int32_t* w = items + (size_t)e * kItemWords;
    const int n = w[kItRow];
    const int begin = rows[n];
    w[kItSlot] = rows[n + 1] > begin ? begin + w[kItSlot] : -1;
  }
  for (int c = off_rows + N + 1 + t; c < p.words; c += kThreads) plan[c] = 0;
  // (5)
  int cl_before = 0;
  for (int c0 = 0; c0 <= p.num_clusters; c0 += kThreads) {
    const int c = c0 + t;
    int all;
    const int sum = block_scan<int>(c <= p.num_clusters ? s_cl[c] : 0, wi, &all);
    if (c <= p.num_clusters) plan[off_cluster + c] = cl_before + sum;
    cl_before += all;
  }
  if (t < kPlanHeaderWords) {
    int v = 0;
    switch (t) {
      case kHdrMagic: v = kPlanMagic; break;
      case kHdrNumClusters: v = p.num_clusters; break;
      case kHdrNumItems: v = I; break;
      case kHdrNumSlots: v = slots_before; break;
      case kHdrNumRows: v = N; break;
      case kHdrHeads: v = p.n_heads; break;
      case kHdrSq: v = p.s_q; break;
      case kHdrB: v = p.B; break;
      case kHdrOffCluster: v = off_cluster; break;
      case kHdrOffItems: v = off_items; break;
      case kHdrOffRows: v = off_rows; break;
      case kHdrTotalWords: v = off_rows + N + 1; break;
      case kHdrMaxBlocks: v = p.max_blocks; break;
      case kHdrCausal: v = p.causal ? 1 : 0; break;
      default: break;
    }
    plan[t] = v;
  }
}

}  // namespace

// Slot maps up to this many tokens are written by the one block that makes the
// tables (16 tokens per thread); longer ones by a launch of their own.
constexpr int kOneBlockTokens = 16384;

mla_status_t launch_build_tables(int B, const int32_t* cached_lens, const int32_t* new_lens, int max_blocks,
                                 int32_t* block_table, const int32_t* free_blocks, int n_free,
                                 const int32_t* free_head, int num_blocks, int max_new, int32_t* seq_lens,
                                 int32_t* cu_new, int32_t* slots, int32_t* positions, int32_t* free_head_out,
                                 int32_t* status, void* stream) {
  TablesParams p = {B, max_blocks, n_free, num_blocks, max_new, cached_lens, new_lens, block_table, free_blocks,
                    free_head, seq_lens, cu_new, slots, positions, free_head_out, status,
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
  PlanParams p = {d.B, d.s_q, d.n_heads, d.max_blocks_per_seq, d.causal, num_clusters, seq_lens, plan,
                  (int)plan_words_upper_bound(num_clusters, d.B * d.s_q), status};
  cudaError_t e = launch_pdl(plan_kernel, dim3(1), dim3(kThreads), (size_t)(num_clusters + 1) * sizeof(int), stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(MLA_ERR_CUDA, "plan launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

}  // namespace mla
