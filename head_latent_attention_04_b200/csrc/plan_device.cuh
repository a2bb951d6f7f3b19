// The split-KV planner on the device: the rule of plan.cpp, word for word.
//
// The rows of a group (a query position, when there are clusters enough for
// every position) are laid end to end, each behind kItemCostPages virtual pages, and
// the line of P units is cut at floor(c P / G).  The range that holds unit u is the
// largest c with floor(c P / G) <= u, that is floor(((u + 1) G - 1) / P).  With
// P >= G every range holds a unit, so a row's pieces are the ranges between
// those of its first and last page; with P < G every unit is a range of its own.
// Rows without keys (a padded batch) have no units and get no item.
//
// One block of 1024 threads; what it costs is latency (scans, divisions and
// barriers one after the other).  Up to 1024 rows (plan_rows) a thread owns a row, and all
// between the lengths and the plan stays in registers and shared memory, with 32-bit
// arithmetic when the products fit; more rows (plan_many_rows) are taken 1024
// at a time in three passes.
#pragma once
#include "block_scan.cuh"
#include "plan_format.h"

#include <cuda_runtime.h>
#include <stdint.h>

namespace mla {

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxClusters = 4096;

struct PlanShape {
  int B, s_q, n_heads, max_blocks, causal, num_clusters;
  int words;   // plan_words_upper_bound
};

struct PlanScratch {
  long long warp_sums[32];
  int warp_ints[32];
  long long line[kPlanThreads];   // line position of the row's end / its first page
  int sum[kPlanThreads];          // pieces up to and with this row
  int first[kPlanThreads];        // range of its first page
  int kv[kPlanThreads];
  int slot[kPlanThreads + 1];
  int cluster[kPlanMaxClusters + 1];
};

// First index in [0, n) whose inclusive sum exceeds e (sums[n - 1] > e).
__device__ __forceinline__ int find_owner(const int* sums, int n, int e) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] > e) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ void plan_header(const PlanShape& p, int32_t* plan, int items, int slots) {
  const int t = threadIdx.x, N = p.B * p.s_q;
  const int off_items = kPlanHeaderWords + p.num_clusters + 1, off_rows = off_items + items * kItemWords;
  if (t < kPlanHeaderWords) {
    int v = 0;
    switch (t) {
      case kHdrMagic: v = kPlanMagic; break;
      case kHdrNumClusters: v = p.num_clusters; break;
      case kHdrNumItems: v = items; break;
      case kHdrNumSlots: v = slots; break;
      case kHdrNumRows: v = N; break;
      case kHdrHeads: v = p.n_heads; break;
      case kHdrSq: v = p.s_q; break;
      case kHdrB: v = p.B; break;
      case kHdrOffCluster: v = kPlanHeaderWords; break;
      case kHdrOffItems: v = off_items; break;
      case kHdrOffRows: v = off_rows; break;
      case kHdrTotalWords: v = off_rows + N + 1; break;
      case kHdrMaxBlocks: v = p.max_blocks; break;
      case kHdrCausal: v = p.causal ? 1 : 0; break;
      default: break;
    }
    plan[t] = v;
  }
  for (int c = off_rows + N + 1 + t; c < p.words; c += kPlanThreads) plan[c] = 0;
}

// cluster[c + 1] holds the items of cluster c: their begins, into the plan.
__device__ __forceinline__ void plan_clusters(const PlanShape& p, PlanScratch& s, int32_t* plan) {
  int before = 0;
  for (int c0 = 0; c0 <= p.num_clusters; c0 += kPlanThreads) {
    const int c = c0 + threadIdx.x;
    int all;
    const int sum = block_scan<int>(c <= p.num_clusters ? s.cluster[c] : 0, s.warp_ints, &all);
    if (c <= p.num_clusters) plan[kPlanHeaderWords + c] = before + sum;
    before += all;
  }
}

// Writes the words of one item; `line` is the line position of the row's first page.
template <typename I>
__device__ __forceinline__ void plan_item(const PlanShape& p, PlanScratch& s, int32_t* w, int n, int kv, I line, int j,
                                          int first, int group, I P, I G, int slot) {
  const I end = line + (kv + 63) / 64;
  const I c = P >= G ? (I)(first + j) : ((line + j + 1) * G - 1) / P;
  const I lo = c * P / G, hi = (c + 1) * P / G;
  const I a = lo > line ? lo : line, z = hi < end ? hi : end;
  w[kItB] = n / p.s_q;
  w[kItQi] = n % p.s_q;
  w[kItPageBegin] = (int)(a - line);
  w[kItPageEnd] = (int)(z - line);
  w[kItKvLen] = kv;
  w[kItSlot] = slot;
  w[kItRow] = n;
  w[kItRow + 1] = 0;
  atomicAdd(&s.cluster[group * (int)G + (int)c + 1], 1);
}

// At most 1024 rows.  keys(n): the row's key count, 0 for none.
template <typename I, typename Keys>
__device__ void plan_rows(const PlanShape& p, PlanScratch& s, int32_t* plan, Keys keys) {
  const int t = threadIdx.x, N = p.B * p.s_q;
  const int groups = p.num_clusters >= p.s_q ? p.s_q : 1;
  const I G = p.num_clusters / groups;
  const int per_group = N / groups;
  // thread t: row t of the (group, row) order, which is also the items' order
  const int g = t / per_group;
  const int n = groups == 1 ? t : (t - g * per_group) * p.s_q + g;
  const int kv = t < N ? keys(n) : 0;
  for (int c = t; c <= p.num_clusters; c += kPlanThreads) s.cluster[c] = 0;
  const int pages = (kv + 63) / 64;
  I line_all;
  const I end = block_scan<I>(pages > 0 ? (I)(pages + kItemCostPages) : (I)0, reinterpret_cast<I*>(s.warp_sums), &line_all);
  s.line[t] = end;
  s.kv[t] = kv;
  __syncthreads();
  I line = 0, P = 0;
  int first = 0, pieces = 0;
  if (t < N) {
    const I base = g > 0 ? (I)s.line[g * per_group - 1] : (I)0;
    P = (I)s.line[(g + 1) * per_group - 1] - base;
    line = end - base - pages;
    if (pages > 0) {
      first = (int)(((line + 1) * G - 1) / P);
      pieces = P >= G ? (int)(((line + pages) * G - 1) / P) - first + 1 : pages;
    }
    s.slot[n] = pieces > 1 ? pieces : 0;
  }
  int items;
  s.sum[t] = block_scan<int>(pieces, s.warp_ints, &items);   // (its barriers order s.slot too)
  const int own = t < N ? s.slot[t] : 0;
  int slots;
  const int slot_end = block_scan<int>(own, s.warp_ints, &slots);
  if (t < N) s.slot[t] = slot_end - own;                     // (t indexes rows here)
  if (t == 0) s.slot[N] = slots;
  s.first[t] = first;
  __syncthreads();
  const int off_items = kPlanHeaderWords + p.num_clusters + 1;
  int32_t* rows = plan + off_items + items * kItemWords;
  for (int i = t; i <= N; i += kPlanThreads) rows[i] = s.slot[i];
  for (int e = t; e < items; e += kPlanThreads) {
    const int k = find_owner(s.sum, kPlanThreads, e);
    const int j = e - (k > 0 ? s.sum[k - 1] : 0);
    const int group = k / per_group;
    const int row = groups == 1 ? k : (k - group * per_group) * p.s_q + group;
    const I base = group > 0 ? (I)s.line[group * per_group - 1] : (I)0;
    const I Pg = (I)s.line[(group + 1) * per_group - 1] - base;
    const int begin = s.slot[row];
    plan_item<I>(p, s, plan + off_items + e * kItemWords, row, s.kv[k], (I)s.line[k] - base - (s.kv[k] + 63) / 64, j,
                 s.first[k], group, Pg, G, s.slot[row + 1] > begin ? begin + j : -1);
  }
  __syncthreads();
  plan_clusters(p, s, plan);
  plan_header(p, plan, items, slots);
}

// Any number of rows.
template <typename Keys>
__device__ void plan_many_rows(const PlanShape& p, PlanScratch& s, int32_t* plan, Keys keys) {
  const int t = threadIdx.x, N = p.B * p.s_q;
  const int groups = p.num_clusters >= p.s_q ? p.s_q : 1;
  const long long G = p.num_clusters / groups;
  const int per_group = N / groups;
  const int off_items = kPlanHeaderWords + p.num_clusters + 1;
  int32_t* items = plan + off_items;
  // pieces of row n, kept behind the last word that this plan can use until the
  // row section, whose place follows from the item count, is written over it
  // (each row's entry is read before any entry at or above it is overwritten)
  int32_t* pieces_of = plan + p.words - (N + 1);
  for (int c = t; c <= p.num_clusters; c += kPlanThreads) s.cluster[c] = 0;
  // (1) rows in (group, row) order: pieces and items; an item's slot word holds
  // its place among the row's pieces for now
  int items_before = 0;
  for (int g = 0; g < groups; ++g) {
    long long P = 0;
    for (int k0 = 0; k0 < per_group; k0 += kPlanThreads) {
      const int k = k0 + t;
      const int kv = k < per_group ? keys(groups == 1 ? k : k * p.s_q + g) : 0;
      long long all;
      block_scan<long long>(kv > 0 ? kItemCostPages + (kv + 63) / 64 : 0, s.warp_sums, &all);
      P += all;
    }
    long long line_before = 0;
    for (int k0 = 0; k0 < per_group; k0 += kPlanThreads) {
      const int k = k0 + t;
      const int n = groups == 1 ? k : k * p.s_q + g;
      const int kv = k < per_group ? keys(n) : 0;
      const int pages = (kv + 63) / 64;
      long long line_all;
      const long long line =
          line_before + block_scan<long long>(pages > 0 ? pages + kItemCostPages : 0, s.warp_sums, &line_all) - pages;
      int first = 0, pieces = 0;
      if (pages > 0) {
        first = (int)(((line + 1) * G - 1) / P);
        pieces = P >= G ? (int)(((line + pages) * G - 1) / P) - first + 1 : pages;
      }
      int pieces_all;
      s.sum[t] = block_scan<int>(pieces, s.warp_ints, &pieces_all);
      s.first[t] = first;
      s.kv[t] = kv;
      s.line[t] = line;
      if (k < per_group) pieces_of[n] = pieces;
      __syncthreads();
      for (int e = t; e < pieces_all; e += kPlanThreads) {
        const int i = find_owner(s.sum, kPlanThreads, e);
        const int j = e - (i > 0 ? s.sum[i - 1] : 0);
        const int row = groups == 1 ? k0 + i : (k0 + i) * p.s_q + g;
        plan_item<long long>(p, s, items + (size_t)(items_before + e) * kItemWords, row, s.kv[i], s.line[i], j,
                             s.first[i], g, P, G, j);
      }
      items_before += pieces_all;
      line_before += line_all;
      __syncthreads();
    }
  }
  int32_t* rows = items + (size_t)items_before * kItemWords;
  // (2) partial slots in row order
  int slots_before = 0;
  for (int n0 = 0; n0 < N; n0 += kPlanThreads) {
    const int n = n0 + t;
    const int pieces = n < N ? pieces_of[n] : 0;
    const int own = pieces > 1 ? pieces : 0;
    int all;
    const int sum = block_scan<int>(own, s.warp_ints, &all);   // (its barriers also order the read above before the writes below)
    if (n < N) rows[n] = slots_before + sum - own;
    slots_before += all;
  }
  if (t == 0) rows[N] = slots_before;
  __syncthreads();
  // (3) into the items: a row is split if its slots end behind where they begin
  for (int e = t; e < items_before; e += kPlanThreads) {
    int32_t* w = items + (size_t)e * kItemWords;
    const int begin = rows[w[kItRow]];
    w[kItSlot] = rows[w[kItRow] + 1] > begin ? begin + w[kItSlot] : -1;
  }
  plan_clusters(p, s, plan);
  plan_header(p, plan, items_before, slots_before);
}

// keys(n) is called by every thread for its rows, more than once.
template <typename Keys>
__device__ __forceinline__ void make_plan(const PlanShape& p, PlanScratch& s, int32_t* plan, Keys keys) {
  const int N = p.B * p.s_q;
  if (N > kPlanThreads) plan_many_rows(p, s, plan, keys);
  // (line + 1) G <= (N (max_blocks + cost) + 1) num_clusters: does it fit 31 bits?
  else if (((long long)N * (p.max_blocks + kItemCostPages) + 1) * p.num_clusters <= INT32_MAX) plan_rows<int>(p, s, plan, keys);
  else plan_rows<long long>(p, s, plan, keys);
}

}  // namespace mla
