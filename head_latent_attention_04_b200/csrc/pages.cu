// Page summaries and the choice of the pages that a query attends to.
//
// Attention over a long cache spends its time on keys that carry no weight.  A
// page (64 tokens) is summarised by the mean of its rows, m = mean_t [c_KV | k_rope],
// kept in 8 bits: scale = amax / 127, code = rint(127 m / amax).  A query
// row's heads are put in the same form, and the page's score is
//   score = fp32( max_h ( (qcode_h . pcode) * qscale_h ) * pscale ):
// the largest mean logit of any head, since all heads share the cache and a
// page that one head needs is needed.  The first n_first and last n_recent
// pages of a query are always taken, then the best scores up to k pages, ties
// to the lowest page.
//
// Everything up to the last rounding is exact, so that a selection does not
// depend on tiles, batch or order of summation: the row sums are kept in
// fp64 (sums of 64 bf16 values, exact unless they span more than 2^40), the
// dot products are integers (|.| <= 576 x 127^2 < 2^24), and the product with
// qscale is kept as an unevaluated fp32 pair.
#include "block_scan.cuh"
#include "fp4_format.h"
#include "mla_internal.h"
#include "ptx.cuh"

#include <cuda_bf16.h>
#include <math_constants.h>

#include <atomic>

namespace mla {
namespace {

using namespace ptx;

constexpr int kPage = 64;
constexpr int kDim = 576;                    // bytes of a summary's codes
constexpr int kRowChunks = kDim / 8;         // 8-column chunks of a cache row

__device__ __forceinline__ void report(int32_t* status, int bits) {
  if (status) atomicOr(status, bits);
}

// ---------------------------------------------------------------- summaries
// One block per page: thread = (8 columns, 16 of the 64 rows), partial sums
// joined through shared memory.  Bound by reading the page; the widening to
// fp64 is done on the bits (the conversion instruction runs at a quarter of the
// rate of the integer operations that replace it): the exponent and mantissa of
// a bf16, fp16 or E2M1 value placed in a double's fields without correcting the
// bias read as the value times a power of two, subnormals included.  All kinds
// end in units of 2^896.
constexpr int kSumThreads = kRowChunks * 4;

enum class Cache { kBf16, kFp8, kFp4 };
constexpr int kF8Row = 656, kF8ScaleOff = 512, kF8RopeOff = 528;

__device__ __forceinline__ double from_hi(uint32_t hi) { return __hiloint2double((int)hi, 0); }

// acc[i] += 2^-896 x (bf16 value i of the 16 bytes)
__device__ __forceinline__ void add_bf16x8(const uint4& v, double (&acc)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] += from_hi(((w[i] << 16) & 0x80000000u) | ((w[i] & 0x7FFFu) << 13));
    acc[2 * i + 1] += from_hi((w[i] & 0x80000000u) | ((w[i] & 0x7FFF0000u) >> 3));
  }
}

template <Cache kind>
__global__ void __launch_bounds__(kSumThreads)
summarize_pages_kernel(const uint8_t* __restrict__ pool, const int32_t* __restrict__ blocks, int num_blocks,
                       int8_t* __restrict__ codes, float* __restrict__ scales, int32_t* status) {
  constexpr int kRowBytes = kind == Cache::kBf16 ? 1152 : kind == Cache::kFp8 ? kF8Row : kF4Row;
  constexpr int kRope = kind == Cache::kBf16 ? 1024 : kind == Cache::kFp8 ? kF8RopeOff : kF4RopeOff;
  constexpr int kRows = kPage / 4;
  __shared__ double s_sum[4][kDim];
  __shared__ unsigned long long s_max[kSumThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int blk = blocks[blockIdx.x];
  if (blk < 0 || blk >= num_blocks) {
    if (blk != -1 && threadIdx.x == 0) report(status, MLA_STATUS_BAD_BLOCK);
    return;
  }
  const int c = threadIdx.x % kRowChunks, part = threadIdx.x / kRowChunks;
  const uint8_t* row = pool + ((size_t)blk * kPage + part * kRows) * kRowBytes;
  double acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (kind == Cache::kBf16 || c >= 64) {
    const uint8_t* src = kind == Cache::kBf16 ? row + 16 * c : row + kRope + 16 * (c - 64);
#pragma unroll 8
    for (int r = 0; r < kRows; ++r) add_bf16x8(__ldg(reinterpret_cast<const uint4*>(src + r * kRowBytes)), acc);
  } else if (kind == Cache::kFp8) {
#pragma unroll 8
    for (int r = 0; r < kRows; ++r) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + r * kRowBytes) + c);
      const float s = __ldg(reinterpret_cast<const float*>(row + r * kRowBytes + kF8ScaleOff) + (c >> 4));
      const double sd = (double)s * 0x1p112;
      uint32_t h[4];
      dequant_e4m3x4_f16(v.x, 0x3C003C00u, h[0], h[1]);   // codes as fp16 (times 1), exact
      dequant_e4m3x4_f16(v.y, 0x3C003C00u, h[2], h[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] += sd * from_hi(((h[i] << 16) & 0x80000000u) | ((h[i] & 0x7FFFu) << 10));
        acc[2 * i + 1] += sd * from_hi((h[i] & 0x80000000u) | ((h[i] & 0x7FFF0000u) >> 6));
      }
    }
  } else {
#pragma unroll 8
    for (int r = 0; r < kRows; ++r) {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(row + r * kRowBytes) + c);
      const uint32_t h = __ldg(reinterpret_cast<const uint16_t*>(row + r * kRowBytes + kF4ScaleOff) + (c >> 2));
      // fp16 scale x 2^(112 - 1008), then x 2^1022: the product below is then in units of 2^896
      const double sd = from_hi((h & 0x7FFFu) << 10) * 0x1p1000 * 0x1p134;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t sign = (i == 7 ? w : w << (28 - 4 * i)) & 0x80000000u;
        const uint32_t mag = (4 * i <= 19 ? w << (19 - 4 * i) : w >> (4 * i - 19)) & 0x00380000u;
        acc[i] += sd * from_hi(sign | mag);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    *reinterpret_cast<double2*>(&s_sum[part][8 * c + i]) = make_double2(acc[i], acc[i + 1]);
  __syncthreads();
  const int col = 2 * threadIdx.x;
  double sum[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    sum[i] = (s_sum[0][col + i] + s_sum[1][col + i]) + (s_sum[2][col + i] + s_sum[3][col + i]);
  // (magnitudes of doubles compare as integers)
  unsigned long long m = max((unsigned long long)__double_as_longlong(fabs(sum[0])),
                             (unsigned long long)__double_as_longlong(fabs(sum[1])));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x / 32] = m;
  __syncthreads();
  m = s_max[0];
#pragma unroll
  for (int i = 1; i < kSumThreads / 32; ++i) m = max(m, s_max[i]);
  const double amax = __longlong_as_double((long long)m);
  int q[2] = {0, 0};
  if (amax > 0.0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) q[i] = __double2int_rn(sum[i] * 127.0 / amax);
  }
  reinterpret_cast<char2*>(codes + (size_t)blk * kDim)[threadIdx.x] = make_char2((signed char)q[0], (signed char)q[1]);
  if (threadIdx.x == 0) scales[blk] = (float)(amax * 0x1p890 / 127.0);   // 2^896 / 64
}

// ---------------------------------------------------------------- scores
// One block per (query row, run of 128-page tiles), tensor cores in 8-bit
// integers: D[page][head] = pcode . qcode, M = 128 pages, N = 128 heads, K = 576
// in 18 steps of 32.  The row's heads are quantised once into shared memory (B,
// K-major); a tile's summaries are gathered through the block table by
// 16-byte asynchronous copies (A, K-major).  Bound by latency at the sizes of
// a decode step (4 rows x 2048 pages are 4.8 MB and 1.2 GFLOP), so the grid
// cuts a row into as many runs as fill the card and the blocks of many rows
// walk a whole row, reusing its quantised heads.
constexpr int kScoreThreads = 512;
constexpr int kTile = 128;
constexpr int kChunkBytes = kTile * 128;          // 128 rows x 128 K-bytes (SW128)
constexpr int kTailBytes = kTile * 64;            // 128 rows x the last 64 K-bytes (SW64)
constexpr int kOperandBytes = 4 * kChunkBytes + kTailBytes;   // 72 KB
constexpr int kMaxHeads = 128;

struct ScoreShared {
  float qscale[kMaxHeads];
  float2 best[4][kTile];
  int block[kTile];
  uint64_t done;
  uint32_t tmem;
  int ok;
};
constexpr int kScoreSmem = 2 * kOperandBytes + (int)sizeof(ScoreShared) + 1024;

struct SelectParams {
  const __nv_bfloat16* q_lat;
  const __nv_bfloat16* q_rope;
  const int8_t* codes;
  const float* scales;
  const int32_t* table;
  const int32_t* seq_lens;
  float* scores;
  int32_t* sel_table;
  int32_t* sel_lens;
  int32_t* sel_pages;
  int32_t* status;
  int s_q, causal, n_heads, max_blocks, num_blocks, k, n_first, n_recent;
};

// Keys that query row n attends (0 for a padded or inconsistent row).
__device__ __forceinline__ int select_keys(const SelectParams& p, int n, bool* bad) {
  const int T = p.seq_lens[n / p.s_q];
  if (T == 0) return 0;
  if (T < p.s_q || (long long)T > (long long)p.max_blocks * kPage) {
    *bad = true;
    return 0;
  }
  return p.causal ? T - p.s_q + 1 + n % p.s_q : T;
}

// Byte offset of 16-byte chunk c (of 36) of row r in an operand.
__device__ __forceinline__ uint32_t operand_off(int r, int c) {
  return c < 32 ? (uint32_t)((c >> 3) * kChunkBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4))
                : (uint32_t)(4 * kChunkBytes + r * 64 + (((c - 32) ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, signed 8-bit operands, 32-bit integer D; K = 32 per MMA.
__device__ __forceinline__ void mma_ss_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
constexpr uint32_t kIdescI8 = (2u << 4)            // D format s32
                              | (1u << 7)          // A format s8
                              | (1u << 10)         // B format s8
                              | ((kMaxHeads >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);

// rint(127 x / amax) with r = 127 / amax: the product is within 2^-23 of the
// quotient (relative); a quotient half-way between two integers has at most
// 8 significant bits and any other is at least 2^-16 away from it (x and amax
// have 8 significant bits), so rounding to 19 bits first puts the exact ties
// back onto the tie and moves nothing across one.
__device__ __forceinline__ int code_of(float x, float r) {
  const float y = __uint_as_float((__float_as_uint(x * r) + 0x10u) & ~0x1Fu);
  return __float2int_rn(y);
}

__global__ void __launch_bounds__(kScoreThreads, 1)
score_pages_kernel(const SelectParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_a = smem;
  uint8_t* s_b = smem + kOperandBytes;
  ScoreShared* sh = reinterpret_cast<ScoreShared*>(smem + 2 * kOperandBytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    mbar_init(&sh->done, 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sh->tmem, 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  griddep_wait();
  griddep_launch_dependents();

  const int n = blockIdx.x;
  bool bad = false;
  const int kv = select_keys(p, n, &bad);
  const int pages = (kv + kPage - 1) / kPage;
  const int scored = pages > p.k ? pages - p.n_recent : 0;   // pages [n_first, scored) compete
  const int tiles = (scored + kTile - 1) / kTile;
  const int32_t* row = p.table + (size_t)(n / p.s_q) * p.max_blocks;
  const uint32_t a_addr = smem_u32(s_a), b_addr = smem_u32(s_b);

  // A: gathers tile t (asynchronous; rows past the last page and rows of bad
  // blocks keep whatever they held, their scores are not used)
  auto load_tile = [&](int t) {
    if (threadIdx.x < kTile) {
      const int pg = t * kTile + threadIdx.x;
      int blk = pg < scored ? row[pg] : -1;
      if (pg < scored && (blk < 0 || blk >= p.num_blocks)) {
        report(p.status, MLA_STATUS_BAD_BLOCK);
        blk = -1;
      }
      sh->block[threadIdx.x] = blk;
    }
    __syncthreads();
#pragma unroll
    for (int i = threadIdx.x; i < kTile * 36; i += kScoreThreads) {
      const int r = i / 36, c = i - 36 * r;
      const int blk = sh->block[r];
      if (blk >= 0) cp_async16(a_addr + operand_off(r, c), p.codes + (size_t)blk * kDim + 16 * c);
    }
  };

  if ((int)blockIdx.y < tiles) {
    load_tile(blockIdx.y);
    // B: a warp quantises eight heads; lane l takes the 8-column chunks l, l + 32 and (l < 8) l + 64
#pragma unroll 1
    for (int hh = 0; hh < kMaxHeads / 16; hh += 4) {
      uint4 v[4][3];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int h = warp * 8 + hh + j;
        const size_t at = (size_t)n * p.n_heads + h;
        const bool in = h < p.n_heads;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        v[j][0] = in ? __ldg(reinterpret_cast<const uint4*>(p.q_lat + at * 512) + lane) : zero;
        v[j][1] = in ? __ldg(reinterpret_cast<const uint4*>(p.q_lat + at * 512) + 32 + lane) : zero;
        v[j][2] = in && lane < 8 ? __ldg(reinterpret_cast<const uint4*>(p.q_rope + at * 64) + lane) : zero;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int h = warp * 8 + hh + j;
        float x[24];
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          const uint32_t w[4] = {v[j][e].x, v[j][e].y, v[j][e].z, v[j][e].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[8 * e + 2 * i] = __uint_as_float(w[i] << 16);
            x[8 * e + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
          }
        }
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 24; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        if (lane == 0) sh->qscale[h] = amax / 127.f;
        const float up = amax < 0x1p-60f ? 0x1p80f : 1.f;   // keeps 127 / amax finite
        const float r = amax > 0.f ? 127.f / (amax * up) : 0.f;
#pragma unroll
        for (int e = 0; e < 3; ++e) {
          if (e == 2 && lane >= 8) break;
          uint32_t o[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float* xe = x + 8 * e + 4 * i;
            o[i] = (uint32_t)(code_of(xe[0] * up, r) & 255) | (uint32_t)(code_of(xe[1] * up, r) & 255) << 8 |
                   (uint32_t)(code_of(xe[2] * up, r) & 255) << 16 | (uint32_t)(code_of(xe[3] * up, r) & 255) << 24;
          }
          const int chunk8 = lane + 32 * e;   // 8 bytes of codes: half of a 16-byte chunk
          *reinterpret_cast<uint2*>(s_b + operand_off(h, chunk8 >> 1) + 8 * (chunk8 & 1)) = make_uint2(o[0], o[1]);
        }
      }
    }
  }
  int it = 0;
  bool ok = true;
  for (int t = blockIdx.y; t < tiles; t += gridDim.y, ++it) {
    cp_async_wait_all();
    fence_proxy_async_smem();
    __syncthreads();
    if (threadIdx.x == 0) {
      tc_fence_after();
      const uint64_t ad = sdesc(a_addr, 16, 1024, kSwizzle128B), bd = sdesc(b_addr, 16, 1024, kSwizzle128B);
#pragma unroll
      for (int s = 0; s < 16; ++s) {
        const uint64_t off = (uint64_t)(((s >> 2) * kChunkBytes + (s & 3) * 32) >> 4);
        mma_ss_i8(tmem, ad + off, bd + off, kIdescI8, s != 0);
      }
      const uint64_t at = sdesc(a_addr + 4 * kChunkBytes, 16, 512, kSwizzle64B);
      const uint64_t bt = sdesc(b_addr + 4 * kChunkBytes, 16, 512, kSwizzle64B);
#pragma unroll
      for (int s = 0; s < 2; ++s) mma_ss_i8(tmem, at + 2 * s, bt + 2 * s, kIdescI8, 1);
      mma_commit(&sh->done);
      sh->ok = mbar_drain(&sh->done, it & 1);
    }
    const int blk = threadIdx.x < kTile ? sh->block[threadIdx.x] : -1;
    __syncthreads();
    ok = sh->ok != 0;   // block-uniform
    if (!ok) break;
    tc_fence_after();
    if (t + (int)gridDim.y < tiles) load_tile(t + gridDim.y);
    // thread = (page, 32 heads): the largest dot x qscale as an exact pair hi + lo
    const int quarter = warp & 3, group = warp >> 2;
    uint32_t d[32];
    tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + 32 * group, d);
    tmem_ld_wait();
    tc_fence_before();
    float hi = -CUDART_INF_F, lo = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float f = (float)(int)d[i], s = sh->qscale[32 * group + i];
      const float h = f * s, l = __fmaf_rn(f, s, -h);
      const bool better = (h > hi || (h == hi && l > lo)) && 32 * group + i < p.n_heads;
      hi = better ? h : hi;
      lo = better ? l : lo;
    }
    sh->best[group][quarter * 32 + lane] = make_float2(hi, lo);
    __syncthreads();
    if (threadIdx.x < kTile) {
      float2 b = sh->best[0][threadIdx.x];
#pragma unroll
      for (int g = 1; g < 4; ++g) {
        const float2 o = sh->best[g][threadIdx.x];
        if (o.x > b.x || (o.x == b.x && o.y > b.y)) b = o;
      }
      const int pg = t * kTile + threadIdx.x;
      if (pg < scored)
        p.scores[(size_t)n * p.max_blocks + pg] =
            blk >= 0 ? (float)(((double)b.x + (double)b.y) * (double)p.scales[blk]) : -CUDART_INF_F;
    }
  }
  if (!ok && threadIdx.x == 0) report(p.status, MLA_STATUS_TIMEOUT);
  cp_async_wait_all();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 128);
}

// ---------------------------------------------------------------- selection
// One block per query row: the k-th best score by a radix search on its
// ordered bits (11, 11 and 10 of them, histograms in shared memory), then one
// ordered pass that writes the pages above it, and the first of those equal to
// it, in page order.  Latency: three histogram passes over the row's scores.
constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;

__device__ __forceinline__ uint32_t order_key(float score) {
  const uint32_t u = __float_as_uint(score + 0.f);   // -0 and +0 are equal
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads)
select_pages_kernel(const SelectParams p) {
  __shared__ int s_hist[kBins];
  __shared__ int s_warp[32];
  __shared__ int s_digit, s_above;
  griddep_wait();
  griddep_launch_dependents();
  const int n = blockIdx.x, t = threadIdx.x;
  bool bad = false;
  const int kv = select_keys(p, n, &bad);
  if (bad && t == 0) report(p.status, MLA_STATUS_BAD_SEQLEN);
  const int pages = (kv + kPage - 1) / kPage;
  const int taken = min(pages, p.k);
  const int32_t* row = p.table + (size_t)(n / p.s_q) * p.max_blocks;
  int32_t* out_table = p.sel_table + (size_t)n * p.k;
  int32_t* out_pages = p.sel_pages ? p.sel_pages + (size_t)n * p.k : nullptr;
  auto put = [&](int at, int page) {
    out_table[at] = page >= 0 ? row[page] : -1;
    if (out_pages) out_pages[at] = page;
  };
  if (t == 0) p.sel_lens[n] = taken > 0 ? kv - (pages - taken) * kPage : 0;
  if (pages <= p.k) {
    for (int i = t; i < p.k; i += kSelThreads) put(i, i < pages ? i : -1);
    return;
  }
  for (int i = t; i < p.n_first; i += kSelThreads) put(i, i);
  for (int i = t; i < p.n_recent; i += kSelThreads) put(p.k - p.n_recent + i, pages - p.n_recent + i);
  int want = p.k - p.n_first - p.n_recent;
  if (want == 0) return;
  const int begin = p.n_first, end = pages - p.n_recent;   // end - begin > want
  const float* scores = p.scores + (size_t)n * p.max_blocks;

  // key bits found so far; after the last digit the threshold itself
  uint32_t prefix = 0;
  const int shifts[3] = {21, 10, 0}, widths[3] = {11, 11, 10};
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const int shift = shifts[d], bins = 1 << widths[d];
    for (int i = t; i < bins; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
    for (int i = begin + t; i < end; i += kSelThreads) {
      const uint32_t key = order_key(scores[i]);
      if (d == 0 || (key >> (shift + widths[d])) == prefix) atomicAdd(&s_hist[(key >> shift) & (bins - 1)], 1);
    }
    __syncthreads();
    // thread t holds the bins (from the top) 2t and 2t + 1
    const int per = bins / kSelThreads;   // 2 or 1
    const int top = bins - 1 - per * t;
    const int c0 = s_hist[top], c1 = per == 2 ? s_hist[top - 1] : 0;
    int all;
    const int incl = block_scan<int>(c0 + c1, s_warp, &all);
    const int before = incl - c0 - c1;
    if (before < want && incl >= want) {
      const bool second = before + c0 < want;
      s_digit = second ? top - 1 : top;
      s_above = second ? before + c0 : before;
    }
    __syncthreads();
    prefix = (prefix << widths[d]) | (uint32_t)s_digit;
    want -= s_above;      // still to take among the keys with this prefix
    __syncthreads();
  }
  // `want` of the pages equal to the threshold, in page order
  int above_before = 0, equal_before = 0;
  for (int i0 = begin; i0 < end; i0 += kSelThreads) {
    const int i = i0 + t;
    const uint32_t key = i < end ? order_key(scores[i]) : 0;
    const bool above = i < end && key > prefix, equal = i < end && key == prefix;
    int all;
    const int incl = block_scan<int>((above ? 1 : 0) | (equal ? 1 << 16 : 0), s_warp, &all);
    const int a = above_before + (incl & 0xFFFF) - (above ? 1 : 0);
    const int e = equal_before + (incl >> 16) - (equal ? 1 : 0);
    if (above || (equal && e < want)) put(p.n_first + a + min(e, want), i);
    above_before += all & 0xFFFF;
    equal_before += all >> 16;
  }
}

cudaError_t score_smem_attr() {   // once per device (outside a capture if the first call is)
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(score_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kScoreSmem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace

mla_status_t launch_summarize_pages(const void* kv_pool, int kind, const int32_t* blocks, int n, int num_blocks,
                                    void* codes, float* scales, int32_t* status, void* stream) {
  auto pool = static_cast<const uint8_t*>(kv_pool);
  auto c = static_cast<int8_t*>(codes);
  auto kernel = kind == MLA_CACHE_BF16  ? summarize_pages_kernel<Cache::kBf16>
                : kind == MLA_CACHE_FP8 ? summarize_pages_kernel<Cache::kFp8>
                                        : summarize_pages_kernel<Cache::kFp4>;
  cudaError_t e = launch_pdl(kernel, dim3(n), dim3(kSumThreads), 0, stream, pool, blocks, num_blocks, c, scales, status);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(MLA_ERR_CUDA, "summarize_pages launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

mla_status_t launch_select_pages(const mla_dims_t& d, const void* q_lat, const void* q_rope, const void* codes,
                                 const float* scales, const int32_t* block_table, const int32_t* seq_lens, int k,
                                 int n_first, int n_recent, float* scores, int32_t* sel_table, int32_t* sel_lens,
                                 int32_t* sel_pages, int32_t* status, void* stream) {
  SelectParams p = {static_cast<const __nv_bfloat16*>(q_lat), static_cast<const __nv_bfloat16*>(q_rope),
                    static_cast<const int8_t*>(codes), scales, block_table, seq_lens, scores, sel_table, sel_lens,
                    sel_pages, status, d.s_q, d.causal, d.n_heads, d.max_blocks_per_seq, d.num_blocks, k, n_first,
                    n_recent};
  const int N = d.B * d.s_q;
  cudaError_t e = cudaSuccess;
  if (d.max_blocks_per_seq > k && k > n_first + n_recent) {   // some row may have pages to choose from
    int dev = 0, sms = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = score_smem_attr();
    const int tiles = (d.max_blocks_per_seq + kTile - 1) / kTile;
    // one block per SM: as many runs of a row as leave no SM idle, one if the rows fill the card
    const int runs = sms / N < 1 ? 1 : (sms / N < tiles ? sms / N : tiles);
    if (e == cudaSuccess)
      e = launch_pdl(score_pages_kernel, dim3(N, runs), dim3(kScoreThreads), kScoreSmem, stream, p);
  }
  if (e == cudaSuccess) e = launch_pdl(select_pages_kernel, dim3(N), dim3(kSelThreads), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(MLA_ERR_CUDA, "select_pages launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

}  // namespace mla
