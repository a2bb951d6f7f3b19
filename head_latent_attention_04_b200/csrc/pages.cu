// Page summaries and the choice of the pages that a query attends to.
//
// Attention over a long cache spends its time on keys that carry no weight.  A
// page (64 tokens) is summarised by the mean of its rows, m = mean_t [c_KV | k_rope],
// kept in 8 bits: scale = amax / 127, code = rint(127 m / amax).  A query
// row's heads are put in the same form, and the page's score is
//   score = fp32( max_h ( (qcode_h . pcode) * qscale_h ) * pscale ):
// the largest mean logit of any head, since all heads share the pages.  It compares raw
// logits: a head whose mean logits are high on every page outranks the others, although a
// constant per head changes nothing in its softmax, and a page that only a head with small
// logits needs may be left out.  The first n_first and last n_recent
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
#include "plan_device.cuh"
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
// joined through shared memory.  The floor is reading the page (8192 pages: bf16 92 us, FP8
// 52, 4-bit 33 at the measured copy rate); it takes 107, 109 and 75 us (106, 102 and 75
// without looking for Inf and NaN), the smaller rows because what a value costs after it is read
// weighs more.  So the widening to fp64 is done
// on the bits: the exponent and mantissa of a bf16, fp16 or E2M1 value placed in a
// double's fields without correcting the bias read as the value times a power of two,
// subnormals included (all kinds end in units of 2^896), and the 4-bit rows are summed in
// fp32 where that is exact.  (8192 4-bit pages: 128 us with every product in fp64, 108 with
// fp32 sums, 88 with eight rows' codes in registers at a time and one division per
// thread, 75 with k_rope in a warp of its own and four blocks per SM.)
constexpr int kSumThreads = kRowChunks * 4;

enum class Cache { kBf16, kFp8, kFp4 };
constexpr int kF8Row = 656, kF8ScaleOff = 512, kF8RopeOff = 528;

__device__ __forceinline__ double from_hi(uint32_t hi) { return __hiloint2double((int)hi, 0); }

// acc[i] += 2^-896 x (bf16 value i of the 16 bytes).  An Inf or a NaN is seen in `special` (not_finite): as
// the largest magnitudes of the pairs of values, their signs meaningless, NaN above all (kMax: one
// instruction a pair, but one chain), or as bits 15 and 31, into which an exponent of all ones
// carries (short chains, which the one warp that reads k_rope alone needs).
template <bool kMax>
__device__ __forceinline__ void add_bf16x8(const uint4& v, double (&acc)[8], uint32_t& special) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t carry[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kMax) asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(special) : "r"(w[i]));
    else carry[i] = (w[i] & 0x7F807F80u) + 0x00800080u;
    acc[2 * i] += from_hi(((w[i] << 16) & 0x80000000u) | ((w[i] & 0x7FFFu) << 13));
    acc[2 * i + 1] += from_hi((w[i] & 0x80000000u) | ((w[i] & 0x7FFF0000u) >> 3));
  }
  if (!kMax) special |= (carry[0] | carry[1]) | (carry[2] | carry[3]);
}
template <bool kMax>
__device__ __forceinline__ bool not_finite(uint32_t special) {
  return kMax ? max(special & 0x7FFFu, (special >> 16) & 0x7FFFu) >= 0x7F80u : (special & 0x80008000u) != 0;
}

// Four E4M3 codes (byte i = code i) -> two fp16 pairs, exact (NaN codes become 0x7FFF).
__device__ __forceinline__ void cvt_e4m3x4_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 c01, c23;\n\tmov.b32 {c01, c23}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, c01;\n\tcvt.rn.f16x2.e4m3x2 %1, c23;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

template <Cache kind>
__global__ void __launch_bounds__(kSumThreads, 4)
summarize_pages_kernel(const uint8_t* pool, const int32_t* blocks, int num_blocks,
                       int8_t* codes, float* scales, int32_t* status) {
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
  // eight warps take c_KV (chunks 0 .. 63), the ninth k_rope (64 .. 71): no warp has both
  const int t = threadIdx.x;
  const int c = t < 256 ? t % 64 : 64 + t % 8, part = t < 256 ? t / 64 : (t - 256) / 8;
  const uint8_t* row = pool + ((size_t)blk * kPage + part * kRows) * kRowBytes;
  double acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  bool finite = true;   // what this thread read
  if (kind == Cache::kBf16 || c >= 64) {
    const uint8_t* src = kind == Cache::kBf16 ? row + 16 * c : row + kRope + 16 * (c - 64);
    uint32_t special = 0;
#pragma unroll 8
    for (int r = 0; r < kRows; ++r)
      add_bf16x8<kind == Cache::kBf16>(__ldcg(reinterpret_cast<const uint4*>(src + r * kRowBytes)), acc, special);
    finite = !not_finite<kind == Cache::kBf16>(special);
  } else if (kind == Cache::kFp8) {
    uint32_t nan_codes = 0;   // bit 7 of a byte: a code was 0x7F or 0xFF
#pragma unroll 8
    for (int r = 0; r < kRows; ++r) {
      const uint2 v = __ldcg(reinterpret_cast<const uint2*>(row + r * kRowBytes) + c);
      const float s = __ldcg(reinterpret_cast<const float*>(row + r * kRowBytes + kF8ScaleOff) + (c >> 4));
      const double sd = (double)s * 0x1p112;
      nan_codes |= ((v.x & 0x7F7F7F7Fu) + 0x01010101u) | ((v.y & 0x7F7F7F7Fu) + 0x01010101u);
      uint32_t h[4];
      cvt_e4m3x4_f16(v.x, h[0], h[1]);
      cvt_e4m3x4_f16(v.y, h[2], h[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] += sd * from_hi(((h[i] << 16) & 0x80000000u) | ((h[i] & 0x7FFFu) << 10));
        acc[2 * i + 1] += sd * from_hi((h[i] & 0x80000000u) | ((h[i] & 0x7FFF0000u) >> 6));
      }
    }
    // (a scale that is not finite makes every sum so: 0 times it is NaN)
    finite = fabs(acc[0]) < CUDART_INF && (nan_codes & 0x80808080u) == 0;
  } else {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(row) + c;
    uint32_t h[kRows], top = 0, low = 31;   // the rows' fp16 scales, their largest and smallest exponent
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      h[r] = __ldcg(reinterpret_cast<const uint16_t*>(row + r * kRowBytes + kF4ScaleOff) + (c >> 2));
    uint32_t w[kRows / 2];                  // eight rows' codes at a time
#pragma unroll
    for (int r = 0; r < kRows / 2; ++r) w[r] = __ldcg(src + r * (kF4Row / 4));
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      top = max(top, h[r] >> 10);
      if (h[r] != 0) low = min(low, h[r] >> 10);
    }
    if (low >= 1 && top <= 30 && top - low <= 5) {
      // Normal scales within 2^5 of one another, nearly always: code x scale is a multiple
      // of 2^(low - 26) and 16 of them stay below 2^(top - 7), 24 bits apart at most, so
      // fp32 sums of the exact products are exact.
      float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const uint32_t codes8 = w[r % (kRows / 2)];
        if (r < kRows / 2) w[r] = __ldcg(src + (r + kRows / 2) * (kF4Row / 4));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = cvt_f16x2_e2m1x2((codes8 >> (8 * k)) & 0xFFu);
          asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
              "fma.rn.f32.f16 %0, lo, %3, %0;\n\tfma.rn.f32.f16 %1, hi, %3, %1;\n\t}"
              : "+f"(f[2 * k]), "+f"(f[2 * k + 1])
              : "r"(x), "h"((uint16_t)h[r]));
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = (double)f[i] * 0x1p-896;
    } else {
#pragma unroll 1
      for (int r = 0; r < kRows; ++r) {
        const uint32_t codes8 = __ldcg(src + r * (kF4Row / 4));
        const uint32_t scale = __ldcg(reinterpret_cast<const uint16_t*>(row + r * kRowBytes + kF4ScaleOff) + (c >> 2));
        // fp16 scale x 2^-1008, then x 2^1134: times the codes' 2^-1022 the product is in units of 2^896
        const double sd = from_hi((scale & 0x7FFFu) << 10) * 0x1p1000 * 0x1p134;
        finite &= (scale & 0x7C00u) != 0x7C00u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t sign = (i == 7 ? codes8 : codes8 << (28 - 4 * i)) & 0x80000000u;
          const uint32_t mag = (4 * i <= 19 ? codes8 << (19 - 4 * i) : codes8 >> (4 * i - 19)) & 0x00380000u;
          acc[i] += sd * from_hi(sign | mag);
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {   // (neighbours start at different pairs: fewer bank conflicts)
    const int i = (k + c) & 3;
    const double2 v = i == 0   ? make_double2(acc[0], acc[1])
                      : i == 1 ? make_double2(acc[2], acc[3])
                      : i == 2 ? make_double2(acc[4], acc[5])
                               : make_double2(acc[6], acc[7]);
    *reinterpret_cast<double2*>(&s_sum[part][8 * c + 2 * i]) = v;
  }
  __syncthreads();
  const int col = 2 * threadIdx.x;
  double sum[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    sum[i] = (s_sum[0][col + i] + s_sum[1][col + i]) + (s_sum[2][col + i] + s_sum[3][col + i]);
  // (magnitudes of doubles compare as integers: high words, then low words of the highest)
  const double big = fabs(sum[0]) > fabs(sum[1]) ? fabs(sum[0]) : fabs(sum[1]);
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)__double2hiint(big));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)__double2hiint(big) == hi ? (uint32_t)__double2loint(big) : 0u);
  const bool warp_finite = __all_sync(0xffffffffu, finite);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x / 32] = warp_finite ? (unsigned long long)hi << 32 | lo : ~0ull;
  __syncthreads();
  unsigned long long m = s_max[0];
#pragma unroll
  for (int i = 1; i < kSumThreads / 32; ++i) m = max(m, s_max[i]);
  const bool usable = m != ~0ull;   // no Inf or NaN in the page
  const double amax = __longlong_as_double((long long)m);
  int q[2] = {0, 0};
  if (amax > 0.0 && usable) {
    // rint(127 sum / amax) by a multiplication, good to 2^-44 absolute; closer than 2^-40 to
    // half-way the quotient itself decides
    const double up = amax < 0x1p-900 ? 0x1p200 : 1.0;   // (sums below 2^-4: 127 / amax stays finite)
    const double top = amax * up, r = 127.0 / top;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const double x = sum[i] * up, y = x * r;
      q[i] = __double2int_rn(y);
      if (fabs(fabs(y - (double)q[i]) - 0.5) < 0x1p-40) q[i] = __double2int_rn(x * 127.0 / top);
    }
  }
  reinterpret_cast<char2*>(codes + (size_t)blk * kDim)[threadIdx.x] = make_char2((signed char)q[0], (signed char)q[1]);
  if (threadIdx.x == 0) {
    scales[blk] = usable ? (float)(amax * 0x1p890 / 127.0) : CUDART_NAN_F;   // 2^896 / 64
    if (!usable) report(status, MLA_STATUS_CACHE_RANGE);
  }
}

// ---------------------------------------------------------------- scores
// One block per (query row, run of 128-page tiles), tensor cores in 8-bit
// integers: D[page][head] = pcode . qcode, M = 128 pages, N = 128 heads, K = 576
// in 18 steps of 32.  The row's heads are quantised once into shared memory (B,
// K-major); a tile's summaries are gathered through the block table by
// 16-byte asynchronous copies (A, K-major; two buffers, and two in tensor
// memory), so that a tile's product and the next tile's copies run under the
// maxima of the tile before.  At one tile a block (4 rows of 2048 pages on 148
// SMs) it is all latency: 7.9 us, of which 2.5 are dependent reads and the issue of the
// copies, 3.4 the quantisation of 147 KB of queries, 1.1 the wait for the copies
// and the product, 0.9 the maxima; where a block walks its row a further tile costs
// 2.1 us, mostly waiting for its 74 KB.  With the selection behind it: 14.7 us for
// 4 rows of 2048 pages, 28.4 for 122 rows of up to 1024.  The grid cuts a row into as many runs as fill the card.
constexpr int kScoreThreads = 512;
constexpr int kTile = 128;
constexpr int kChunkBytes = kTile * 128;          // 128 rows x 128 K-bytes (SW128)
constexpr int kTailBytes = kTile * 64;            // 128 rows x the last 64 K-bytes (SW64)
constexpr int kOperandBytes = 4 * kChunkBytes + kTailBytes;   // 72 KB
constexpr int kMaxHeads = 128;

struct ScoreShared {
  float qscale[kMaxHeads];
  float2 best[4][kTile];
  float scale[kTile];      // of the current tile's summaries, negative for a bad block
  uint64_t done[2];
  uint32_t tmem;
  int ok;
};
constexpr int kScoreSmem = 3 * kOperandBytes + (int)sizeof(ScoreShared) + 1024;

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
  int32_t* plan;   // plan of the selection, or null
  PlanShape shape;
  int N, s_q, causal, n_heads, max_blocks, num_blocks, k, n_first, n_recent;
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

// rint(127 x / amax) in one multiply-add per element: x r + 1.5 x 2^23, with the
// product unrounded, leaves the rounded integer (ties to even) in the low bits.
// For the exact quotients' codes r = 127 / amax must not move a half-way case.  x and amax
// have 8 significant bits, so a quotient 127 x / amax that is not half-way between
// two integers is at least 2^-16 (relative) away from it, far more than r's error.
// Half-way cases: 254 x = (2k + 1) amax.  127 is prime, so it divides amax's significand (254:
// r is then exact) or 2k + 1 = 127, which is x = amax / 2, half-way between 63
// and 64 and due at 64: an inexact r is taken above 127 / amax, which sends it there.
constexpr float kRound = 12582912.f;
__device__ __forceinline__ float code_factor(float amax) {
  const float r = 127.f / amax;
  return __fmaf_rn(r, amax, -127.f) == 0.f ? r : r * (1.f + 0x1p-22f);
}
// Codes of the four bf16 values of two words; `up` is a power of two that both x and r's amax carry.
__device__ __forceinline__ uint32_t code_word(uint32_t w0, uint32_t w1, float r, float up) {
  const float x[4] = {__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xFFFF0000u), __uint_as_float(w1 << 16),
                      __uint_as_float(w1 & 0xFFFF0000u)};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = __float_as_uint(__fmaf_rn(x[i] * up, r, kRound));
  return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

__global__ void __launch_bounds__(kScoreThreads, 1)
score_pages_kernel(const SelectParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_b = smem + 2 * kOperandBytes;
  ScoreShared* sh = reinterpret_cast<ScoreShared*>(smem + 3 * kOperandBytes);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    mbar_init(&sh->done[0], 1);
    mbar_init(&sh->done[1], 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sh->tmem, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  griddep_wait();
  griddep_launch_dependents();

  const int n = blockIdx.x;
  const int32_t* row = p.table + (size_t)(n / p.s_q) * p.max_blocks;
  const uint32_t a_addr = smem_u32(smem), b_addr = smem_u32(s_b);
  // A warp gathers eight rows of a tile.  Its block ids (lanes 0 .. 7) are read before
  // it is known whether the row is that long (the table has max_blocks columns
  // whatever its length).
  auto read_id = [&](int t) {
    const long long pg = (long long)t * kTile + 8 * warp + lane;
    return lane < 8 && pg < p.max_blocks ? row[pg] : -1;
  };
  const int step = gridDim.y;
  int tile = blockIdx.y;
  int id_next = read_id(tile);
  bool bad = false;
  const int kv = select_keys(p, n, &bad);
  const int pages = (kv + kPage - 1) / kPage;
  const int scored = pages > p.k ? pages - p.n_recent : 0;   // pages [n_first, scored) compete
  const int tiles = (scored + kTile - 1) / kTile;

  // Takes the ids of tile t (read earlier) and starts its gather into A buffer b;
  // returns the summary scale of lane l's row (l < 8), -1 for a bad block.  Rows behind the
  // last page and rows of bad blocks keep whatever they held, their scores are not used.
  auto gather = [&](int t, int b, int id) {
    float scale = -1.f;
    if (lane < 8) {
      if (t * kTile + 8 * warp + lane >= scored) id = -1;
      else if (id < 0 || id >= p.num_blocks) {
        report(p.status, MLA_STATUS_BAD_BLOCK);
        id = -1;
      }
      if (id >= 0) scale = __ldcg(p.scales + id);
    }
    // chunks 0 .. 31 of row j go through lanes 0 .. 31, the last four of all eight rows together
    const uint32_t a = a_addr + b * kOperandBytes;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int blk = __shfl_sync(0xffffffffu, id, j);
      if (blk >= 0) cp_async16(a + operand_off(8 * warp + j, lane), p.codes + (size_t)blk * kDim + 16 * lane);
    }
    const int blk = __shfl_sync(0xffffffffu, id, lane >> 2);
    if (blk >= 0)
      cp_async16(a + operand_off(8 * warp + (lane >> 2), 32 + (lane & 3)),
                 p.codes + (size_t)blk * kDim + 512 + 16 * (lane & 3));
    asm volatile("cp.async.commit_group;" ::: "memory");
    return scale;
  };
  auto multiply = [&](int b, bool one_more_in_flight) {
    if (one_more_in_flight) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      const uint32_t a = a_addr + b * kOperandBytes, d = tmem + 128 * b;
      const uint64_t ad = sdesc(a, 16, 1024, kSwizzle128B), bd = sdesc(b_addr, 16, 1024, kSwizzle128B);
#pragma unroll
      for (int s = 0; s < 16; ++s) {
        const uint64_t off = (uint64_t)(((s >> 2) * kChunkBytes + (s & 3) * 32) >> 4);
        mma_ss_i8(d, ad + off, bd + off, kIdescI8, s != 0);
      }
      const uint64_t at = sdesc(a + 4 * kChunkBytes, 16, 512, kSwizzle64B);
      const uint64_t bt = sdesc(b_addr + 4 * kChunkBytes, 16, 512, kSwizzle64B);
#pragma unroll
      for (int s = 0; s < 2; ++s) mma_ss_i8(d, at + 2 * s, bt + 2 * s, kIdescI8, 1);
      mma_commit(&sh->done[b]);
    }
  };

  float scale[2] = {-1.f, -1.f};
  if (tile < tiles) {
    // B: a warp quantises eight heads; lane l takes the 8-column chunks l, l + 32
    // and (l < 8) l + 64 of each
    uint4 v[8][3];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const size_t at = (size_t)n * p.n_heads + 8 * warp + j;
      const bool in = 8 * warp + j < p.n_heads;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      v[j][0] = in ? __ldcg(reinterpret_cast<const uint4*>(p.q_lat + at * 512) + lane) : zero;
      v[j][1] = in ? __ldcg(reinterpret_cast<const uint4*>(p.q_lat + at * 512) + 32 + lane) : zero;
      v[j][2] = in && lane < 8 ? __ldcg(reinterpret_cast<const uint4*>(p.q_rope + at * 64) + lane) : zero;
    }
    scale[0] = gather(tile, 0, id_next);
    id_next = tile + step < tiles ? read_id(tile + step) : -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int h = 8 * warp + j;
      uint32_t m = 0;   // largest magnitudes, a pair of bf16 (their signs come out meaningless)
#pragma unroll
      for (int e = 0; e < 3; ++e) {
        const uint32_t w[4] = {v[j][e].x, v[j][e].y, v[j][e].z, v[j][e].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
      }
      m = max(m & 0x7FFFu, (m >> 16) & 0x7FFFu);       // (as integers they order like the values)
      m = __reduce_max_sync(0xffffffffu, m);
      float amax = __uint_as_float(m << 16);
      if (lane == 0) sh->qscale[h] = amax / 127.f;
      const float up = amax < 0x1p-60f ? 0x1p80f : 1.f;   // keeps 127 / amax finite
      const float r = m > 0 ? code_factor(amax * up) : 0.f;
#pragma unroll
      for (int e = 0; e < 3; ++e) {
        if (e == 2 && lane >= 8) break;
        const int chunk8 = lane + 32 * e;   // 8 bytes of codes: half of a 16-byte chunk
        *reinterpret_cast<uint2*>(s_b + operand_off(h, chunk8 >> 1) + 8 * (chunk8 & 1)) =
            make_uint2(code_word(v[j][e].x, v[j][e].y, r, up), code_word(v[j][e].z, v[j][e].w, r, up));
      }
    }
    const bool more = tile + step < tiles;
    if (more) {
      scale[1] = gather(tile + step, 1, id_next);
      id_next = tile + 2 * step < tiles ? read_id(tile + 2 * step) : -1;
    }
    multiply(0, more);
  }
  bool ok = true;
#pragma unroll 1
  for (int it = 0; tile < tiles; tile += step, ++it) {
    const int b = it & 1;
    if (tid == 0) sh->ok = mbar_drain(&sh->done[b], (it >> 1) & 1);
    __syncthreads();
    ok = sh->ok != 0;   // block-uniform
    if (!ok) break;
    tc_fence_after();
    if (lane < 8) sh->scale[8 * warp + lane] = b ? scale[1] : scale[0];
    if (tile + step < tiles) multiply(b ^ 1, false);   // the next tile's copies are the only ones in flight
    if (tile + 2 * step < tiles) {
      const float s = gather(tile + 2 * step, b, id_next);
      if (b) scale[1] = s; else scale[0] = s;
      id_next = tile + 3 * step < tiles ? read_id(tile + 3 * step) : -1;
    }
    // thread = (page, 32 heads): the largest dot x qscale as an exact pair.  hi is the
    // largest rounded product; the largest product itself rounds to it, so it is
    // hi plus the largest of fma(dot, qscale, -hi), exact for the products that round to hi.
    const int quarter = warp & 3, group = warp >> 2;
    const int heads = min(p.n_heads - 32 * group, 32);
    float hi = -CUDART_INF_F, lo = -CUDART_INF_F;
    if (heads > 0) {
      uint32_t d[32];
      tmem_ld32(tmem + 128 * b + ((uint32_t)(quarter * 32) << 16) + 32 * group, d);
      tmem_ld_wait();
      tc_fence_before();
      const float4* qs = reinterpret_cast<const float4*>(sh->qscale + 32 * group);
      if (heads == 32) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 s = qs[i / 4];
          hi = fmaxf(fmaxf(hi, fmaxf((float)(int)d[i] * s.x, (float)(int)d[i + 1] * s.y)),
                     fmaxf((float)(int)d[i + 2] * s.z, (float)(int)d[i + 3] * s.w));
        }
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 s = qs[i / 4];
          lo = fmaxf(fmaxf(lo, fmaxf(__fmaf_rn((float)(int)d[i], s.x, -hi), __fmaf_rn((float)(int)d[i + 1], s.y, -hi))),
                     fmaxf(__fmaf_rn((float)(int)d[i + 2], s.z, -hi), __fmaf_rn((float)(int)d[i + 3], s.w, -hi)));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < heads) hi = fmaxf(hi, (float)(int)d[i] * sh->qscale[32 * group + i]);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < heads) lo = fmaxf(lo, __fmaf_rn((float)(int)d[i], sh->qscale[32 * group + i], -hi));
      }
    }
    sh->best[group][quarter * 32 + lane] = make_float2(hi, lo);
    __syncthreads();
    if (tid < kTile) {
      float2 best = sh->best[0][tid];
#pragma unroll
      for (int g = 1; g < 4; ++g) {
        const float2 o = sh->best[g][tid];
        if (o.x > best.x || (o.x == best.x && o.y > best.y)) best = o;
      }
      const int pg = tile * kTile + tid;
      const float scale_of = sh->scale[tid];
      if (pg < scored)
        p.scores[(size_t)n * p.max_blocks + pg] =
            scale_of >= 0.f ? (float)(((double)best.x + (double)best.y) * (double)scale_of) : -CUDART_INF_F;
    }
  }
  if (!ok) {
    if (tid == 0) report(p.status, MLA_STATUS_TIMEOUT);
    cp_async_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 256);
}

// ---------------------------------------------------------------- selection
// One block per query row: the k-th best score by a radix search on its
// ordered bits (11, 11 and 10 of them, histograms in shared memory), then one
// ordered pass that writes the pages above it, and the first of those equal to
// it, in page order.  Latency: three histogram passes over the row's scores.  How
// many pages and keys a row gets follows from its length alone, so one more block
// makes the attention's split-KV plan meanwhile.
constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;

__device__ __forceinline__ uint32_t order_key(float score) {
  const uint32_t u = __float_as_uint(score + 0.f);   // -0 and +0 are equal
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads)
select_pages_kernel(const SelectParams p) {
  __shared__ union {
    int hist[3][kBins];
    PlanScratch plan;
  } sh;
  __shared__ int s_warp[32];
  __shared__ int s_digit, s_above;
  for (int i = threadIdx.x; i < 3 * kBins; i += kSelThreads) sh.hist[0][i] = 0;
  griddep_wait();
  griddep_launch_dependents();
  const int n = blockIdx.x, t = threadIdx.x;
  bool bad = false;
  if (n == p.N) {   // the last block: the plan of the selection, whose lengths need no scores
    __syncthreads();   // (the zeroes above lie where the plan's scratch does)
    make_plan(p.shape, sh.plan, p.plan, [&](int i) {
      const int kv = select_keys(p, i, &bad);
      const int pages = (kv + kPage - 1) / kPage;
      return kv - (pages - min(pages, p.k)) * kPage;
    });
    return;
  }
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
  // up to 4096 candidates stay in registers from here on; more are read again in each pass
  constexpr int kHeld = 4;
  const bool held = end - begin <= kHeld * kSelThreads;
  uint32_t key[kHeld];
#pragma unroll
  for (int h = 0; h < kHeld; ++h) {
    const int i = begin + h * kSelThreads + t;
    key[h] = held && i < end ? order_key(scores[i]) : 0;
  }
  __syncthreads();   // the histograms are zero

  // key bits found so far; after the last digit the threshold itself
  uint32_t prefix = 0;
#pragma unroll
  for (int d = 0; d < 3; ++d) {
    const int width = d == 2 ? 10 : 11, shift = d == 0 ? 21 : d == 1 ? 10 : 0, bins = 1 << width;
    int* hist = sh.hist[d];
    auto count = [&](uint32_t k) {
      if (d == 0 || (k >> ((shift + width) & 31)) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
    };
    if (held) {
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
        if (begin + h * kSelThreads + t < end) count(key[h]);
    } else {
      for (int i = begin + t; i < end; i += kSelThreads) count(order_key(scores[i]));
    }
    __syncthreads();
    // thread t holds the bins (from the top) 2t and 2t + 1, or t of the last digit's 1024
    const int per = bins / kSelThreads;
    const int top = bins - 1 - per * t;
    const int c0 = hist[top], c1 = per == 2 ? hist[top - 1] : 0;
    int all;
    const int incl = block_scan<int>(c0 + c1, s_warp, &all);
    const int before = incl - c0 - c1;
    if (before < want && incl >= want) {
      const bool second = before + c0 < want;
      s_digit = second ? top - 1 : top;
      s_above = second ? before + c0 : before;
    }
    __syncthreads();
    prefix = (prefix << width) | (uint32_t)s_digit;
    want -= s_above;      // still to take among the keys with this prefix
    __syncthreads();
  }
  // `want` of the pages equal to the threshold, in page order
  int above_before = 0, equal_before = 0;
  auto take = [&](int i, uint32_t k) {
    const bool above = i < end && k > prefix, equal = i < end && k == prefix;
    int all;
    const int incl = block_scan<int>((above ? 1 : 0) | (equal ? 1 << 16 : 0), s_warp, &all);
    const int a = above_before + (incl & 0xFFFF) - (above ? 1 : 0);
    const int e = equal_before + (incl >> 16) - (equal ? 1 : 0);
    if (above || (equal && e < want)) put(p.n_first + a + min(e, want), i);
    above_before += all & 0xFFFF;
    equal_before += all >> 16;
  };
  if (held) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (begin + h * kSelThreads < end) take(begin + h * kSelThreads + t, key[h]);
  } else {
    for (int i0 = begin; i0 < end; i0 += kSelThreads) {
      const int i = i0 + t;
      take(i, i < end ? order_key(scores[i]) : 0);
    }
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
                                 int32_t* sel_pages, int num_clusters, int32_t* plan, int32_t* status, void* stream) {
  const int N = d.B * d.s_q;
  const PlanShape shape = {N, 1, d.n_heads, k, 1, num_clusters,
                           plan ? (int)plan_words_upper_bound(num_clusters, N) : 0};
  SelectParams p = {static_cast<const __nv_bfloat16*>(q_lat), static_cast<const __nv_bfloat16*>(q_rope),
                    static_cast<const int8_t*>(codes), scales, block_table, seq_lens, scores, sel_table, sel_lens,
                    sel_pages, status, plan, shape, N, d.s_q, d.causal, d.n_heads, d.max_blocks_per_seq, d.num_blocks, k, n_first,
                    n_recent};
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
  if (e == cudaSuccess) e = launch_pdl(select_pages_kernel, dim3(plan ? N + 1 : N), dim3(kSelThreads), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(MLA_ERR_CUDA, "select_pages launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

}  // namespace mla
