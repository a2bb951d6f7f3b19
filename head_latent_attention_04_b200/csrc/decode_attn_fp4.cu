// Absorbed MLA decode attention over a 4-bit latent cache (rows of fp4_format.h)
// on sm_100a: tcgen05, TMEM, TMA and 2-CTA clusters.
//
// The mathematics is that of decode_attn.cu, per query row (token n, head h) over keys t < kv_len:
//   logit_t = scale * (q_lat . c_KV[t] + q_rope . k_rope[t]),  o_lat = sum_t softmax(logit)_t c_KV[t],
// with c_KV[t, j] = code[t, j] * s[t, j / 32], one pass over the keys with a running
// reference maximum and sum, and partial results merged by mla_combine where the plan
// splits a row.
//
// What bounds it.  A token is 416 bytes, so at 128 heads its 2 x 128 x 1088 operations
// take 2.7 times as long at the measured tensor rate as its bytes at the measured copy
// rate: the floor is the tensor cores' (4 x 128K tokens: 89 us).  The products do not run
// on the 4-bit codes: q_lat and P stay in 16 bits and the scales are fp16, which no
// block-scaled product takes, and along the keys, which P . c_KV sums over, the scales change with every
// key.  So every half page is widened to fp16 in shared memory.  No unit is saturated (tensor pipe 32 %, issue
// slots 46 %, shared memory 45 % on 32 x 4096 tokens): the kernel is bound by the
// serial chains of its warps, and three of them turn once per 64-key page in about 2400 cycles
// each, of which the tensor pipe needs 1088: the sender warps (two stages' waits,
// widening 570, the scores' wait, conversion and store 700), the softmax warps (2500), and the exchange (a copy
// takes 1050, the answer that the tile is free and the next copy's start as long again).
// 4 x 128K tokens: 144.5 us launched from a graph, 165 us launched back to back for a second, where the
// card's power limit holds the SM clock at 1.6 of 1.965 GHz; in that loop the bf16
// cache's kernel takes 179 us, the FP8 cache's 187 (32 x 4096 tokens: 48.5 against 54
// and 57).  So the 4-bit cache holds 2.8 times the tokens of bf16 and is a little faster.
//
// Why this shape (as in decode_attn.cu).  O for 128 heads x 512 columns in fp32 is
// one SM's whole tensor memory, so a cluster of two CTAs splits the latent
// dimension: CTA r owns latent columns [256r, 256r + 256) and RoPE columns [32r, 32r + 32),
// computes partial scores over its 288 columns and exchanges them through
// distributed shared memory in log2 units, rounded to fp16 (16 KB per page
// each way, one bulk copy counted on the receiver's mbarrier), and both CTAs add the
// two in fp32.  fp16, because a tile of fp32 each way does not fit beside the rings and
// doubles the exchange.  What it costs: a logit moves by at most 2^-11 (|p0| + |p1|) in
// log2 units, p0 and p1 its two partials, so a weight by that times ln 2 (partials of 16:
// 1 % at worst); two halves that cancel are rounded at their own size.  Measured on 4096
// random keys, relative Frobenius error of o_lat, of which the output's own rounding is
// 1.7e-3: logits up to 9 1.8e-3, to 26 2.1e-3, to 84 3.5e-3, to 244 3.6e-3 (with the sum
// rounded to fp16 as well 2.0e-3, 2.7e-3, 5.3e-3, 4.3e-3, and 1.5 % less time).
//
// Two rings, because the cache's bytes are few: four raw half pages (13 KB each:
// 8 KB of codes, 1 KB of scales, 4 KB of RoPE columns, which the QK product reads there)
// hide the TMA's latency, and a stage of 32 KB holds the widened page from its QK to its PV product.
// A single ring widened in place, as for the FP8 cache, holds its stage for the TMA's
// latency too.
//
// TMEM (512 columns): O [0, 256) fp32, S [256, 320) fp32 (free once the sender has read
// it), two P buffers [320, 352) and [352, 384) in fp16 (page g uses buffer g & 1),
// q_lat half [384, 512) in fp16 pairs.
//
// Warps (640 threads): 0 TMA; 1 QK issuer, owner of the tensor memory; 2 PV issuer;
// 3-6 and 16-19 query loader, widening and score sender; 7-14 softmax, correction, epilogue
// (16 rows each, two threads per row); 15 copies score tiles to the peer.
// Steps (4 x 128K tokens, from a graph): four sender warps with a ring of its own for
// the raw pages 160 us; a query's loads 16 at a time 157; the scores read
// when the own tile is free, their registers not live across that wait, 149; the wait for a P
// buffer at the start of a page 148; a row's two softmax threads in one warp, joined by
// a shuffle instead of a barrier, 145; eight sender warps 143.5, which read and free S before they wait
// for the own tile 142; scores added in fp32 and the stores into tensor memory behind their
// fences, which is what they should compute and order, 144.5.  Measured and not kept: a group of warps for the
// widening alone 144 to 181 us; two softmax groups taking pages in turn with one thread
// per row 198; two tiles for the peer's scores (and three raw stages) 145; two or three barriers polled at once
// 141.5 to 144; one wait for two barriers by different lanes 181 to 262; one lane waiting for its warp
// 480; test_wait before try_wait 157; widening two pages ahead 174; codes widened by byte permutes instead of the
// conversion instruction 203.
//
// Failure: every wait is bounded (200 ms by default, mla_set_wait_limit_ns); a role that
// gives up sets MLA_STATUS_TIMEOUT, stops its peer, drains the copies and products it
// issued and returns without trapping.
#include "fp4_format.h"
#include "mla_internal.h"
#include "plan_format.h"
#include "ptx.cuh"
#include "tmap.h"

#include <cuda_bf16.h>
#include <math_constants.h>

#include <atomic>

namespace mla {
namespace {

using namespace ptx;

constexpr int kPage = 64;
constexpr int kRows = 128;
constexpr int kStages = 4;                                   // widened half pages
constexpr int kRawStages = 4;                                // half pages as they are in the cache
constexpr int kChunkBytes = kPage * 128;                     // 64 keys x 64 latent cols in fp16 (SW128)
constexpr int kStageBytes = 4 * kChunkBytes;                 // 32 KB
// Raw stage: this CTA's 128 bytes of codes per key (SW128), its 32 RoPE columns
// (SW64, the QK product reads them there) and its 16 bytes of scales per key.
constexpr int kRawCodes = 0;
constexpr int kRawRope = kRawCodes + kPage * 128;
constexpr int kRawScales = kRawRope + kPage * 64;
constexpr int kRawBytes = kRawScales + kPage * 16;           // 13 KB of HBM per half page
constexpr int kXRow = 64 * 2;                                // fp16 score row, 16B chunks XOR (row & 7)
constexpr int kXBytes = kRows * kXRow;                       // one score tile (16 KB)

constexpr int kOffKV = 0;
constexpr int kOffRaw = kOffKV + kStages * kStageBytes;
constexpr int kOffXPeer = kOffRaw + kRawStages * kRawBytes;  // peer's partial scores (one tile)
constexpr int kOffXOwn = kOffXPeer + kXBytes;                // own partial scores (fp16, one tile)
constexpr int kOffQRope = kOffXOwn + kXBytes;                // bf16 q_rope half, 128 rows x 64 B (SW64, A of QK)
constexpr int kOffBar = kOffQRope + kRows * 64;

constexpr int kThreads = 640;            // 20 warps
constexpr int kSoftWarp0 = 7, kCopyWarp = 15, kSendWarp1 = 16;   // senders are warps 3 .. 6 and 16 .. 19
constexpr int kSoftWarps = 8, kSendWarps = 8;

constexpr uint32_t kTmemO = 0, kTmemS = 256, kTmemP = 320, kTmemQ = 384, kTmemCols = 512;   // P: two 32-column buffers
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;   // log2 units: rescale O only when the max grows by > 2^8

struct DecodeParams {
  const __nv_bfloat16* q_lat;   // [N][H][512]
  const __nv_bfloat16* q_rope;  // [N][H][64]
  const int32_t* block_table;   // [B][max_blocks]
  const int32_t* seq_lens;      // [B]
  const int32_t* plan;
  float* o_part;                // [slots][H][512]
  float* lse_part;              // [slots][H]
  __nv_bfloat16* o_lat;         // [N][H][512]
  float* lse_out;               // [N][H] or null
  int32_t* status;
  int n_heads, max_blocks, num_blocks, s_q, causal, B, n_rows, num_clusters;
  PlanRoom room;
  float scale_log2;             // scale * log2(e)
  uint64_t wait_ns;             // limit of every protocol wait (drains of issued work use the default)
  uint32_t zero;                // 0, read at run time (see the release of the peer tile)
};

struct Bars {
  uint64_t raw_full[kRawStages];    // the TMA has landed
  uint64_t raw_empty[kRawStages];   // its QK product is complete (it was widened before that)
  uint64_t kv_conv[kStages];        // widened to fp16 (8 sender warps)
  uint64_t kv_empty[kStages];       // its PV product is complete
  uint64_t q_full, q_empty;
  uint64_t s_full;       // QK product of the current page is in S
  uint64_t s_read;       // the sender has read S (the next QK may overwrite it)
  uint64_t own_full;     // own fp16 partial-score tile written (8 sender warps)
  uint64_t own_free;     // own tile read by the softmax (8 warps) and by its bulk copy (1)
  uint64_t x_recv;       // peer's fp16 partial scores landed in the peer tile (1 arrival + 16 KB tx)
  uint64_t x_sendok;     // peer has read its peer tile, which this CTA may refill (8 remote arrivals)
  // P written (O rescaled if needed), 8 softmax warps.  One per P buffer, as o_full: the softmax writes
  // page g + 2's P only after page g's product, so no phase passes before the PV issuer has seen
  // it (with one barrier for both, pages g and g + 1 could).
  uint64_t p_full[2];
  uint64_t o_full[2];     // PV product of a page complete, per P buffer (page g uses buffer g & 1)
  uint64_t o_done;        // every PV product of the current item complete (epilogue)
  uint64_t o_free, qk_done, pv_done;
  uint32_t tmem_base;    // TMEM allocation
  uint32_t sent_count;   // score tiles this CTA has copied to its peer
  WaitCtl wc;            // abort flag and wait limit of every role
};
constexpr int kSmemBytes = kOffBar + (int)sizeof(Bars) + 1024;

__device__ __forceinline__ void report(int32_t* status, int bits) {
  if (status) atomicOr(status, bits);
}

// Suspend-time hint of the pipeline waits: a waiting warp takes no issue slots, and
// the waits, which stand inlined in every role's loop, are half as long as without it
// (4 x 128K tokens: 149 us against 165).
constexpr uint32_t kWaitHintNs = 1000;

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile WaitCtl* wc) {
  return __all_sync(0xffffffffu, mbar_wait<false, kWaitHintNs>(bar, parity, wc));
}
// For data the peer CTA's bulk copy wrote: its complete_tx releases at cluster
// scope, so the waiter must acquire at cluster scope to see the bytes.
__device__ __forceinline__ bool warp_wait_cluster(uint64_t* bar, uint32_t parity, volatile WaitCtl* wc) {
  return __all_sync(0xffffffffu, mbar_wait<true, kWaitHintNs>(bar, parity, wc));
}

// The plan fixes each row's key count (kv_len) from the host seq_lens it was
// made with.  True if the device seq_lens (T of the item's sequence) now give
// another count: the softmax then masks every key of the item, so the row is
// written as zeros with LSE -inf, and MLA_STATUS_BAD_SEQLEN is reported.
__device__ __forceinline__ bool item_stale(const int32_t* w, int T, const DecodeParams& p) {
  const int want = p.causal ? T - p.s_q + 1 + w[kItQi] : T;
  return want != w[kItKvLen];
}

// Keys of the item's last page that are attended (1 .. 64).  When fewer than
// 64, that page is loaded shifted: its first `attended` keys land in stage
// rows [64 - attended, 64) and the rows above them are the TMA's zero fill
// (a negative row coordinate), so no stale or non-finite cache row past the
// key count ever reaches the P.c_KV product (where 0 * Inf would be NaN).
__device__ __forceinline__ int last_page_keys(const int32_t* w) {
  return w[kItKvLen] - (w[kItPageEnd] - 1) * kPage;
}

// Tensor-memory access of 16 lanes (taddr's lane .. + 15): threads 0-15 at taddr, threads 16-31
// (the same lanes again) kSplit columns on; N consecutive columns each.
template <int kSplit>
__device__ __forceinline__ void tmem_ld16x2_32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32], %33;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr), "n"(kSplit));
}
template <int kSplit>
__device__ __forceinline__ void tmem_st16x2_32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x32bx2.x32.b32 [%0], %1, "
      "{%2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33};" ::"r"(taddr),
      "n"(kSplit), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
template <int kSplit>
__device__ __forceinline__ void tmem_st16x2_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], %1, "
      "{%2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17};" ::"r"(taddr),
      "n"(kSplit), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// (a.lo + c) + b.lo and the same of the high halves in fp32, for fp16 pairs a and b: the
// mixed-precision add takes the fp16 operand exactly and rounds the sum once.
__device__ __forceinline__ void add_f16x2_to_f32(uint32_t a, uint32_t b, float c, float& lo, float& hi) {
  asm("{\n\t.reg .f16 a0, a1, b0, b1;\n\t.reg .f32 x, y;\n\t"
      "mov.b32 {a0, a1}, %2;\n\tmov.b32 {b0, b1}, %3;\n\t"
      "add.rn.f32.f16 x, a0, %4;\n\tadd.rn.f32.f16 y, a1, %4;\n\t"
      "add.rn.f32.f16 %0, b0, x;\n\tadd.rn.f32.f16 %1, b1, y;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(a), "r"(b), "f"(c));
}

// Three-input maximum and packed fp32 addition.
__device__ __forceinline__ float max3f(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
mla_decode_fp4_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_rope,
                      const __grid_constant__ CUtensorMap tm_scale, const DecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_kv = smem + kOffKV;
  uint8_t* s_raw = smem + kOffRaw;
  uint8_t* s_xpeer = smem + kOffXPeer;
  uint8_t* s_xown = smem + kOffXOwn;
  uint8_t* s_qrope = smem + kOffQRope;
  Bars* bars = reinterpret_cast<Bars*>(smem + kOffBar);
  uint32_t* tmem_slot = &bars->tmem_base;
  volatile WaitCtl* wc = &bars->wc;
  volatile uint32_t* sent_count = &bars->sent_count;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank(), peer = rank ^ 1u;
  const int cid = (int)cluster_id_x();
  // A role that gives up stops both CTAs of the pair (the peer would otherwise
  // wait for score tiles that never come): it raises its own flag and the
  // peer's, so after the final cluster barrier both flags tell the same story.
  auto give_up = [&]() {
    wc->abort = 1;
    st_cluster_u32(mapa(smem_u32((const void*)&wc->abort), peer), 1u);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRawStages; ++s) {
      mbar_init(&bars->raw_full[s], 1);
      mbar_init(&bars->raw_empty[s], 1);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->kv_conv[s], kSendWarps);
      mbar_init(&bars->kv_empty[s], 1);
    }
    mbar_init(&bars->q_full, kSendWarps);
    mbar_init(&bars->q_empty, 1);
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->s_read, kSendWarps);
    mbar_init(&bars->own_full, kSendWarps);
    mbar_init(&bars->own_free, kSoftWarps + 1);
    mbar_init(&bars->x_recv, 1);
    mbar_init(&bars->x_sendok, kSoftWarps);
    mbar_init(&bars->p_full[0], kSoftWarps);
    mbar_init(&bars->p_full[1], kSoftWarps);
    mbar_arrive_expect_tx(&bars->x_recv, kXBytes);   // armed for page 0
    mbar_init(&bars->o_full[0], 1);
    mbar_init(&bars->o_full[1], 1);
    mbar_init(&bars->o_done, 1);
    mbar_init(&bars->o_free, kSoftWarps);
    mbar_init(&bars->qk_done, 1);
    mbar_init(&bars->pv_done, 1);
    wc->abort = 0;
    wc->limit_ns = p.wait_ns;
    *sent_count = 0;
    fence_mbar_init();
    prefetch_tmap(&tm_codes);
    prefetch_tmap(&tm_rope);
    prefetch_tmap(&tm_scale);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // peer barriers and flags initialised before any remote access
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();   // set-up above overlaps the previous kernel; global memory only from here
  griddep_launch_dependents();

  // The section offsets follow from the cluster count, so the cluster's item
  // range is read without first waiting for the header (checked alongside).
  // The plan must match the launch (uniform over the grid).
  const int32_t* plan = p.plan;
  const int off_cluster = kPlanHeaderWords, off_items = kPlanHeaderWords + p.num_clusters + 1;
  const int32_t* items = plan + off_items;
  const int it_begin_raw = plan[off_cluster + cid], it_end_raw = plan[off_cluster + cid + 1];
  // (no short-circuit: the words are read together, not one after the other)
  const bool plan_ok = (plan[kHdrMagic] == kPlanMagic) & (plan[kHdrNumClusters] == p.num_clusters) &
                       (plan[kHdrNumRows] == p.n_rows) & (plan[kHdrHeads] == p.n_heads) &
                       (plan[kHdrB] == p.B) & (plan[kHdrSq] == p.s_q) &
                       (plan[kHdrMaxBlocks] == p.max_blocks) & (plan[kHdrCausal] == (p.causal ? 1 : 0)) &
                       (plan[kHdrOffCluster] == off_cluster) & (plan[kHdrOffItems] == off_items) &
                       (plan[kHdrTotalWords] <= p.room.plan_words) & (plan[kHdrNumSlots] <= p.room.part_slots);
  const int it_begin = plan_ok ? it_begin_raw : 0;
  const int it_end = plan_ok ? it_end_raw : 0;
  if (!plan_ok && threadIdx.x == 0 && rank == 0 && cid == 0) report(p.status, MLA_STATUS_BAD_PLAN);

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    // Lane 0 waits and issues; the whole warp fetches block ids 32 pages at a
    // time with one coalesced load, so a page's TMA never waits on its own
    // block-table read.  (An L2 prefetch of the blocks a few pages ahead was
    // measured slower at distances 2 to 12.)
    int g = 0;
    bool fail = false;
    for (int it = it_begin; it < it_end && !fail; ++it) {
      if (__any_sync(0xffffffffu, wc->abort != 0)) break;   // warp-uniform
      const int32_t* w = items + (size_t)it * kItemWords;
      const int b = w[kItB], pb = w[kItPageBegin], pe = w[kItPageEnd];
      const int shift = kPage - min(last_page_keys(w), kPage);   // zero-filled rows of the last page
      int my_blk = pb + lane < pe ? p.block_table[(size_t)b * p.max_blocks + pb + lane] : 0;
      if (lane == 0 && it + 1 < it_end) {   // the next item's query rows, so that its loaders read them from L2
        const size_t nrow = (size_t)items[(size_t)(it + 1) * kItemWords + kItRow];
        bulk_prefetch_l2(p.q_lat + nrow * p.n_heads * 512, (uint32_t)p.n_heads * 1024u);
        bulk_prefetch_l2(p.q_rope + nrow * p.n_heads * 64, (uint32_t)p.n_heads * 128u);
      }
      for (int pg = pb; pg < pe && !fail; ++pg, ++g) {
        const int rel = pg - pb;
        if ((rel & 31) == 0 && rel > 0) {
          const int q = pg + lane;
          my_blk = q < pe ? p.block_table[(size_t)b * p.max_blocks + q] : 0;
        }
        int blk = __shfl_sync(0xffffffffu, my_blk, rel & 31);
        if (lane == 0) {
          const int s = g % kRawStages;
          if (g >= kRawStages &&
              !mbar_wait<false, kWaitHintNs>(&bars->raw_empty[s], ((g / kRawStages) - 1) & 1, wc)) {
            fail = true;
          } else {
            if (blk < 0 || blk >= p.num_blocks) {
              report(p.status, MLA_STATUS_BAD_BLOCK);
              blk = 0;
            }
            uint8_t* st = s_raw + s * kRawBytes;
            const int y = pg + 1 == pe ? -shift : 0;   // first row of the block to load
            mbar_arrive_expect_tx(&bars->raw_full[s], kRawBytes);   // zero-filled bytes count too
            tma_load_3d(st + kRawCodes, &tm_codes, &bars->raw_full[s], 128 * rank, y, blk);
            tma_load_3d(st + kRawScales, &tm_scale, &bars->raw_full[s], 16 * rank, y, blk);
            tma_load_3d(st + kRawRope, &tm_rope, &bars->raw_full[s], 32 * rank, y, blk);
          }
        }
        fail = __shfl_sync(0xffffffffu, fail, 0);
        if (fail) break;   // this page was not issued
      }
    }
    if (lane == 0) {
      if (fail) {
        give_up();
        report(p.status, MLA_STATUS_TIMEOUT);
      }
      // every issued load must land before the CTA may exit
      for (int k = g - 1; k >= 0 && k >= g - kRawStages; --k)
        mbar_drain(&bars->raw_full[k % kRawStages], (k / kRawStages) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ QK issuer
    // S = [q_lat | q_rope] . [c_KV | k_rope]^T over this CTA's 288 columns:
    // M = 128 rows, N = 64 keys, 16 MMAs with A = q_lat and 2 with A = q_rope,
    // from TMEM and shared memory.  S is single-buffered; the sender frees it (s_read) as
    // soon as it has copied the product out.  The whole warp runs the loop
    // (descriptors stay warp-uniform) and one elected lane issues.
    const uint32_t idesc_qk = idesc_bf16(128, 64, 0, 0);                                // RoPE half
    const uint32_t idesc_lat = idesc_f16(128, 64, 0, 0);                                // latent half
    const uint64_t kv_desc0 = sdesc(smem_u32(s_kv), 16, 1024, kSwizzle128B);
    const uint64_t kr_desc0 = sdesc(smem_u32(s_raw) + kRawRope, 16, 512, kSwizzle64B);
    const uint64_t qr_desc = sdesc(smem_u32(s_qrope), 16, 512, kSwizzle64B);
    bool ok = true;
    int g = 0;
    for (int it = it_begin; ok && it < it_end; ++it) {
      const int32_t* w = items + (size_t)it * kItemWords;
      const int n = w[kItPageEnd] - w[kItPageBegin];
      if (!warp_wait(&bars->q_full, (it - it_begin) & 1, wc)) { ok = false; break; }
      for (int j = 0; j < n; ++j, ++g) {
        const int s = g % kStages, sr = g % kRawStages;
        if (!warp_wait(&bars->raw_full[sr], (g / kRawStages) & 1, wc) ||
            !warp_wait(&bars->kv_conv[s], (g / kStages) & 1, wc) ||
            (g > 0 && !warp_wait(&bars->s_read, (g - 1) & 1, wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t kvd = kv_desc0 + (uint64_t)((s * kStageBytes) >> 4);
        const uint64_t krd = kr_desc0 + (uint64_t)((sr * kRawBytes) >> 4);
#pragma unroll
        for (int t = 0; t < 16; ++t)   // latent half: K = 256 in steps of 16, A = q_lat from TMEM
          mma_ts_elect(tmem + kTmemS, tmem + kTmemQ + 8 * t,
                       kvd + (uint64_t)(((t >> 2) * kChunkBytes + (t & 3) * 32) >> 4), idesc_lat, t != 0);
#pragma unroll
        for (int t = 0; t < 2; ++t)    // RoPE half: K = 32, A = q_rope from shared memory
          mma_ss_elect(tmem + kTmemS, qr_desc + (uint64_t)(t * 2), krd + (uint64_t)(t * 2), idesc_qk, 1);
        mma_commit_elect(&bars->s_full);
        mma_commit_elect(&bars->raw_empty[sr]);
      }
      if (ok) mma_commit_elect(&bars->q_empty);   // q_lat and q_rope (TMEM) may be replaced
    }
    if (!ok && lane == 0) {
      give_up();
      report(p.status, MLA_STATUS_TIMEOUT);
    }
    __syncwarp();
    mma_commit_elect(&bars->qk_done);
    mbar_drain(&bars->qk_done, 0);   // no MMA may still write TMEM at dealloc
  } else if (warp == 2) {
    // ------------------------------------------------------------ PV issuer
    // O += P . c_KV: M = 128 rows, N = 256 latent columns, K = 64 keys in 4
    // MMAs, A = P (fp16 pairs) from TMEM buffer g & 1, B = the stage's c_KV
    // half (MN-major).  Warp-wide loop, one elected lane issues.
    const uint32_t idesc_pv = idesc_f16(128, 256, 0, 1);
    const uint64_t v_desc0 = sdesc(smem_u32(s_kv), kChunkBytes, 1024, kSwizzle128B);
    bool ok = true;
    int g = 0;
    for (int it = it_begin; ok && it < it_end; ++it) {
      const int32_t* w = items + (size_t)it * kItemWords;
      const int n = w[kItPageEnd] - w[kItPageBegin];
      const int ii = it - it_begin;
      for (int j = 0; j < n; ++j, ++g) {
        const int s = g % kStages;
        if (!warp_wait(&bars->p_full[g & 1], (g >> 1) & 1, wc) ||
            (j == 0 && ii > 0 && !warp_wait(&bars->o_free, (ii - 1) & 1, wc))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t vd = v_desc0 + (uint64_t)((s * kStageBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)   // 64 keys in steps of 16; P (fp16 pairs) from TMEM
          mma_ts_elect(tmem + kTmemO, tmem + kTmemP + 32 * (g & 1) + 8 * kk, vd + (uint64_t)(kk * (2048 >> 4)),
                       idesc_pv, (j | kk) != 0);
        mma_commit_elect(&bars->kv_empty[s]);
        mma_commit_elect(&bars->o_full[g & 1]);
      }
      // o_full alone cannot tell the last page's completion from the one before
      // (a parity wait sees one phase at a time), so the epilogue waits on this
      if (ok) mma_commit_elect(&bars->o_done);
    }
    if (!ok && lane == 0) {
      give_up();
      report(p.status, MLA_STATUS_TIMEOUT);
    }
    __syncwarp();
    mma_commit_elect(&bars->pv_done);
    mbar_drain(&bars->pv_done, 0);
  } else if (warp < kSoftWarp0 || warp >= kSendWarp1) {
    // ------------------------------------------------------------ query loader, widening, score sender (8 warps)
    // Two warps per TMEM lane quarter, thread = (row r, half).  At each item start
    // it copies half of row r's 256 q_lat columns into TMEM and (half 0) its 32
    // q_rope columns into shared memory (A operands of the QK product) once the
    // previous item's last QK has completed; the producer has prefetched those
    // rows into L2.  Per page it reads 32 keys of this CTA's partial scores
    // as soon as the QK product lands, frees S, rounds to fp16 into
    // the own tile, and the copy warp pushes that tile to the peer's tile with a
    // bulk copy that completes on the peer's x_recv (16-byte chunks XOR-swizzled
    // by row & 7).
    const int quarter = warp & 3;
    const int half = warp >= kSendWarp1 ? 1 : 0;
    const int r = quarter * 32 + lane;
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const float sl2 = p.scale_log2;
    // Widens page gg to fp16.  Thread = (key cr, 64 of this CTA's 256 columns):
    // 32 bytes of codes, two groups of 32 columns, each 16 bytes with one scale;
    // a group's codes become fp16 by the conversion instruction, exactly, and are
    // multiplied by the scale, one rounding.  Page g + 1 is widened before page
    // g's scores are awaited (pages 0 and 1 before page 0's), that is, right after
    // page g - 1's scores have gone out: neither the score exchange nor the next
    // QK product waits for it.
    auto widen = [&](int gg) -> bool {
      const int s = gg % kStages, sr = gg % kRawStages;
      if (!warp_wait(&bars->raw_full[sr], (gg / kRawStages) & 1, wc) ||
          (gg >= kStages && !warp_wait(&bars->kv_empty[s], ((gg / kStages) - 1) & 1, wc)))
        return false;
      const int ch = lane >> 3;
      // (recomputed per call: kept live across the sender loop they cost registers)
      int cr;
      asm volatile("mov.b32 %0, %1;" : "=r"(cr) : "r"(8 * (4 * half + (warp - 3) % 13) + (lane & 7)));
      const uint32_t raw = smem_u32(s_raw + sr * kRawBytes);
      const uint32_t codes = raw + kRawCodes + cr * 128;
      uint32_t s01;   // the scales of the two groups
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(s01) : "r"(raw + kRawScales + cr * 16 + ch * 4) : "memory");
      const uint32_t row = smem_u32(s_kv + s * kStageBytes) + ch * kChunkBytes + cr * 128;
      uint4 raw_codes[2];   // (all reads before the first write: their latencies overlap)
#pragma unroll
      for (int gi = 0; gi < 2; ++gi) raw_codes[gi] = ld_shared_v4(codes + (((2 * ch + gi) ^ (cr & 7)) << 4));
#pragma unroll
      for (int gi = 0; gi < 2; ++gi) {
        const uint4 v = raw_codes[gi];
        const uint32_t sc2 = __byte_perm(s01, 0, gi ? 0x3232 : 0x1010);
        const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {   // 8 codes -> one 16-byte chunk
          uint32_t o[4];
          dequant_e2m1x8_f16(wd[k], sc2, o);
          st_shared_v4(row + (((4 * gi + k) ^ (cr & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
        }
      }
      fence_proxy_async_smem();   // read by the tensor cores
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->kv_conv[s]);
      return true;
    };
    int g = 0;
    int pages_total = 0, widened = 0;   // this cluster's pages, and those widened so far
    for (int it = it_begin; it < it_end; ++it)
      pages_total += items[(size_t)it * kItemWords + kItPageEnd] - items[(size_t)it * kItemWords + kItPageBegin];
    for (int it = it_begin; it < it_end; ++it) {
      const int32_t* w = items + (size_t)it * kItemWords;
      const int ii = it - it_begin;
      if (ii > 0 && !warp_wait(&bars->q_empty, (ii - 1) & 1, wc)) goto sender_fail;
      tc_fence_after();   // q_lat is written after the last item's products have read it
      {
        if (half == 0) {
          const uint4* rsrc = reinterpret_cast<const uint4*>(p.q_rope + ((size_t)w[kItRow] * p.n_heads + r) * 64 +
                                                             32 * rank);
          // row r of the K-major A tile, 64 bytes: 16-byte chunk k at (k ^ ((r >> 1) & 3))
          // (the 64-byte swizzle the MMA descriptor names)
          uint4 q[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) q[k] = r < p.n_heads ? rsrc[k] : make_uint4(0, 0, 0, 0);
          const uint32_t dst = smem_u32(s_qrope) + r * 64;
#pragma unroll
          for (int k = 0; k < 4; ++k) st_shared_v4(dst + ((k ^ ((r >> 1) & 3)) << 4), q[k]);
          fence_proxy_async_smem();   // read by the tensor cores
        }
        const uint4* src = reinterpret_cast<const uint4*>(p.q_lat + ((size_t)w[kItRow] * p.n_heads + r) * 512 +
                                                          256 * rank);
        // the latent products take fp16 operands (plain loads: the eight pieces of a
        // line that a row's thread reads one after the other come from L1; through
        // L2 alone an item started 6 us later)
#pragma unroll 1
        for (int hh = 2 * half; hh < 2 * half + 2; ++hh) {
          uint32_t v[32];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint4 q = r < p.n_heads ? src[8 * hh + k] : make_uint4(0, 0, 0, 0);
            v[4 * k] = q.x; v[4 * k + 1] = q.y; v[4 * k + 2] = q.z; v[4 * k + 3] = q.w;
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = bf16x2_to_f16x2(v[k]);
          tmem_st32(tmem + lane_addr + kTmemQ + 32 * hh, v);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->q_full);
      }
      const int n = w[kItPageEnd] - w[kItPageBegin];
      for (int j = 0; j < n; ++j, ++g) {
        // pages up to g + 1: at g = 0 pages 0 and 1, then one per page
        for (; widened < min(g + 2, pages_total); ++widened)
          if (!widen(widened)) goto sender_fail;
        uint32_t v[32];
        if (!warp_wait(&bars->s_full, g & 1, wc)) goto sender_fail;
        tc_fence_after();
        tmem_ld32(tmem + lane_addr + kTmemS + 32 * half, v);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->s_read);
        uint32_t hv[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)   // scaled to log2 units, then rounded to fp16
          hv[k] = pack_f16(__uint_as_float(v[2 * k]) * sl2, __uint_as_float(v[2 * k + 1]) * sl2);
        // single tile: page g - 1's own tile must have been read by the softmax and the copy
        if (g >= 1 && !warp_wait(&bars->own_free, (g - 1) & 1, wc)) goto sender_fail;
        {
          uint8_t* own = s_xown + r * kXRow;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(own + (((4 * half + k) ^ (r & 7)) << 4)) =
                make_uint4(hv[4 * k], hv[4 * k + 1], hv[4 * k + 2], hv[4 * k + 3]);
        }
        fence_proxy_async_smem();   // the copy warp's bulk copy reads the tile through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->own_full);
      }
    }
    goto sender_done;
  sender_fail:
    give_up();
    if (lane == 0) report(p.status, MLA_STATUS_TIMEOUT);
  sender_done:;
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------ score copy (one thread)
    // Per page: one bulk copy of the own fp16 tile to the peer's tile,
    // completing on the peer's x_recv, once the 8 sender warps have written
    // it and the peer has read page g - 1 out of its tile.  The own tile may
    // be rewritten once the copy has read it (own_free).  A warp of its own,
    // so that waiting for the copy never holds back the next page's score read.
    if (lane == 0) {
      const uint32_t x_peer = mapa(smem_u32(s_xpeer), peer);
      const uint32_t x_recv_peer = mapa(smem_u32(&bars->x_recv), peer);
      uint32_t sent = 0;
      bool ok = true;
      int g = 0;
      for (int it = it_begin; ok && it < it_end; ++it) {
        const int32_t* w = items + (size_t)it * kItemWords;
        const int n = w[kItPageEnd] - w[kItPageBegin];
        for (int j = 0; j < n; ++j, ++g) {
          if ((g >= 1 && !mbar_wait<true, kWaitHintNs>(&bars->x_sendok, (g - 1) & 1, wc)) ||
              !mbar_wait<false, kWaitHintNs>(&bars->own_full, g & 1, wc)) {
            ok = false;
            break;
          }
          bulk_copy_to_peer(x_peer, smem_u32(s_xown), kXBytes, x_recv_peer);
          bulk_commit();
          *sent_count = ++sent;
          bulk_wait_read<0>();
          mbar_arrive(&bars->own_free);
        }
      }
      if (!ok) {
        give_up();
        report(p.status, MLA_STATUS_TIMEOUT);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax / epilogue (8 warps)
    // A warp has 16 rows, half of its TMEM lane quarter, and two threads per row, lanes
    // l and l + 16: thread = (row r, key half c), keys [32c, 32c + 32) of each page and output
    // columns [128c, 128c + 128) of this CTA's 256.  A row's maximum and sum are joined
    // by one shuffle.
    const int c = lane >> 4;
    const int row0 = 32 * (warp & 3) + 16 * ((warp - kSoftWarp0) >> 2);   // the warp's rows
    const int r = row0 + (lane & 15);
    const int tid = threadIdx.x - kSoftWarp0 * 32;    // 0 .. 255
    const uint32_t lane_addr = (uint32_t)row0 << 16;
    const uint32_t x_sendok_peer = mapa(smem_u32(&bars->x_sendok), peer);
    bool out_of_range = false;   // fp16 partials overflowed: a reference max of +Inf or -Inf, or a NaN sum
    // The sequence length of the next item is loaded one item ahead, so that
    // the stale-plan check never waits for memory at an item boundary.
    int T_next = it_begin < it_end ? p.seq_lens[items[(size_t)it_begin * kItemWords + kItB]] : 0;
    int g = 0;
    for (int it = it_begin; it < it_end; ++it) {
      const int32_t* w = items + (size_t)it * kItemWords;
      const int row = w[kItRow], slot = w[kItSlot], pb = w[kItPageBegin];
      const int n = w[kItPageEnd] - pb;
      const int ii = it - it_begin;
      const bool stale = item_stale(w, T_next, p);
      if (it + 1 < it_end) T_next = p.seq_lens[items[(size_t)(it + 1) * kItemWords + kItB]];
      if (stale && tid == 0 && rank == 0) report(p.status, MLA_STATUS_BAD_SEQLEN);
      // keys masked in the item's last page: the zero-filled rows of its shifted load
      const int shift_last = kPage - min(last_page_keys(w), kPage);

      float m_ref = -CUDART_INF_F, l_run = 0.f;
      float nb = 0.f;   // -m_ref, or 0 as long as no key was seen
      for (int j = 0; j < n; ++j) {
        const int gj = g + j;
        // full score = fp16(own partial) + fp16(peer partial), identical in both CTAs.
        // The own tile is read (and released) first: it lands before the peer's.
        // P buffer gj & 1 is free once the PV product of page gj - 2 has completed
        if (gj >= 2 && !warp_wait(&bars->o_full[gj & 1], ((gj >> 1) - 1) & 1, wc)) goto softmax_fail;
        uint4 po[4], pr[4];
        const uint32_t off_base = (uint32_t)(4 * c);
        if (!warp_wait(&bars->own_full, gj & 1, wc)) goto softmax_fail;
        {
          const uint8_t* orow = s_xown + r * kXRow;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            po[k] = *reinterpret_cast<const uint4*>(orow + (((off_base + k) ^ (r & 7)) << 4));
          uint32_t bar_addr = smem_u32(&bars->own_free);
          // arrive only after the own tile was read (one word of each 16-byte load)
          asm volatile("" : "+r"(bar_addr) : "r"(po[0].x ^ po[1].x ^ po[2].x ^ po[3].x));
          __syncwarp();
          if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar_addr) : "memory");
        }
        if (!warp_wait_cluster(&bars->x_recv, gj & 1, wc)) goto softmax_fail;
        {
          const uint8_t* xrow = s_xpeer + r * kXRow;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            pr[k] = *reinterpret_cast<const uint4*>(xrow + (((off_base + k) ^ (r & 7)) << 4));
          // The peer tile is consumed: re-arm x_recv for page gj + 1, then let the peer refill it.
          // Its next copy must come after every lane's reads.  A release at cluster scope would say
          // so, but it waits for all that the CTA has in flight (4 x 128K tokens: 151 -> 209 us); the
          // arrive instead depends on what was read: its address takes in a vote over all four loads
          // of every lane (p.zero is 0, which the compiler does not know), so it cannot be
          // issued before they have returned.
          const uint32_t read = (pr[0].x ^ pr[1].x ^ pr[2].x ^ pr[3].x) & p.zero;
          const uint32_t ok_addr = x_sendok_peer + __ballot_sync(0xffffffffu, read != 0);
          if (lane == 0) {
            if (warp == kSoftWarp0) mbar_arrive_expect_tx(&bars->x_recv, kXBytes);
            mbar_arrive_relaxed_cluster(ok_addr);
          }
        }
        // Scores in log2 units above the row's reference maximum, (fp16(own) - m_ref) + fp16(peer) in
        // fp32: the partials' roundings to fp16 are the only ones that count.  (The pair's CTAs
        // add in different orders, so their references may differ in the last bit: each
        // normalises its own columns by its own sum.)
        float sc[32];
        {
          const uint32_t* ow = reinterpret_cast<const uint32_t*>(po);
          const uint32_t* pw = reinterpret_cast<const uint32_t*>(pr);
#pragma unroll
          for (int k = 0; k < 16; ++k) add_f16x2_to_f32(ow[k], pw[k], nb, sc[2 * k], sc[2 * k + 1]);
        }
        // masked keys [0, lo) of this page (-inf): the last page's zero fill, or
        // all of them when the device seq_lens disagree with the plan
        const int lo = stale ? kPage : (j == n - 1 ? shift_last : 0);
        if (lo > 32 * c) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (32 * c + k < lo) sc[k] = -CUDART_INF_F;
        }
        float mloc;
        {
          float t[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            t[k] = max3f(sc[8 * k], sc[8 * k + 1], sc[8 * k + 2]);
            t[k] = max3f(t[k], sc[8 * k + 3], sc[8 * k + 4]);
            t[k] = max3f(t[k], sc[8 * k + 5], sc[8 * k + 6]);
          }
          t[0] = max3f(t[0], sc[7], sc[15]);
          t[1] = max3f(t[1], sc[23], sc[31]);
          mloc = fmaxf(max3f(t[0], t[1], t[2]), t[3]);
        }
        const float mx = fmaxf(mloc, __shfl_xor_sync(0xffffffffu, mloc, 16));

        // lazy reference max (log2 domain): move it only when the row max grows by > 2^8
        const bool first = m_ref == -CUDART_INF_F;
        const bool move = first ? mx != -CUDART_INF_F : mx > kRescaleThreshold;
        float alpha = 1.f;
        if (__any_sync(0xffffffffu, move)) {
          const float d = move ? -mx : 0.f;
          if (move) {
            alpha = first ? 0.f : ex2(-mx);
            m_ref = first ? mx : m_ref + mx;
            nb = -m_ref;
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 x = add2(make_float2(sc[2 * k], sc[2 * k + 1]), make_float2(d, d));
            sc[2 * k] = x.x;
            sc[2 * k + 1] = x.y;
          }
        }
        uint32_t pk[16];
        float2 ps[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 e = make_float2(ex2(sc[2 * k]), ex2(sc[2 * k + 1]));
          pk[k] = pack_f16(e.x, e.y);
          ps[k & 1] = add2(ps[k & 1], e);
        }
        l_run = l_run * alpha + ((ps[0].x + ps[0].y) + (ps[1].x + ps[1].y));

        if (__any_sync(0xffffffffu, move && j > 0)) {
          // rescaling O: the PV product of page gj - 1 (same item) must have landed
          if (!warp_wait(&bars->o_full[(gj - 1) & 1], ((gj - 1) >> 1) & 1, wc)) goto softmax_fail;
          tc_fence_after();
          const float a = (move && j > 0) ? alpha : 1.f;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t o[32];
            tmem_ld16x2_32<128>(tmem + lane_addr + kTmemO + 32 * q, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
            tmem_st16x2_32<128>(tmem + lane_addr + kTmemO + 32 * q, o);
          }
          tmem_st_wait();
        }
        tc_fence_after();   // after the product that read this buffer (awaited above)
        tmem_st16x2_16<16>(tmem + lane_addr + kTmemP + 32 * (gj & 1), pk);   // keys [32c, 32c+32), fp16 pairs
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[gj & 1]);
      }

      // epilogue: O / l  ->  o_lat (whole row) or the row's partial slot.  A
      // stale item has P = 0 throughout: its row is written as zeros.
      {
        if (!warp_wait(&bars->o_done, ii & 1, wc)) goto softmax_fail;
        tc_fence_after();
        {   // the same order in both threads of a row
          const float other = __shfl_xor_sync(0xffffffffu, l_run, 16);
          l_run = c == 0 ? l_run + other : other + l_run;
        }
        // (every item attends a key, so no score above -Inf means that all of them left fp16 downwards; a
        // key here and there that does so has no weight either way, and looking for it in every
        // page costs 2.3 %)
        out_of_range |= (m_ref == CUDART_INF_F) | (l_run != l_run) | (!stale & (m_ref == -CUDART_INF_F));
        const float inv_l = l_run > 0.f ? 1.f / l_run : 0.f;
        const bool valid = r < p.n_heads;
        const bool o_lat_32b = (reinterpret_cast<uintptr_t>(p.o_lat) & 31) == 0;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t o[32];
          tmem_ld16x2_32<128>(tmem + lane_addr + kTmemO + 32 * q, o);
          tmem_ld_wait();
          if (!valid) continue;
          const int col = 256 * rank + 128 * c + 32 * q;
          if (slot < 0) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k)
              pk[k] = pack_bf16(__uint_as_float(o[2 * k]) * inv_l, __uint_as_float(o[2 * k + 1]) * inv_l);
            __nv_bfloat16* dst = p.o_lat + ((size_t)row * p.n_heads + r) * 512 + col;
            if (o_lat_32b) {   // one full 32-byte sector per store
              st_global_v8(dst, pk[0], pk[1], pk[2], pk[3], pk[4], pk[5], pk[6], pk[7]);
              st_global_v8(dst + 16, pk[8], pk[9], pk[10], pk[11], pk[12], pk[13], pk[14], pk[15]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                reinterpret_cast<uint4*>(dst)[k] = make_uint4(pk[4 * k], pk[4 * k + 1], pk[4 * k + 2], pk[4 * k + 3]);
            }
          } else {
            // column-group-major partials, 8 columns (32 bytes) per group: a warp's
            // 32 rows of one group are 1 KB contiguous, and a reader of one row
            // gets whole 32-byte sectors
            float* dst = p.o_part + (((size_t)slot * 64 + col / 8) * p.n_heads + r) * 8;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(__uint_as_float(o[8 * k + e]) * inv_l);
              st_global_v8(dst + (size_t)k * p.n_heads * 8, v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]);
            }
          }
        }
        if (valid && rank == 0 && c == 0) {
          const float lse = (l_run > 0.f) ? (m_ref + __log2f(l_run)) * kLn2 : -CUDART_INF_F;
          if (slot >= 0) p.lse_part[(size_t)slot * p.n_heads + r] = lse;
          else if (p.lse_out) p.lse_out[(size_t)row * p.n_heads + r] = lse;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->o_free);
      }
      g += n;
    }
    goto softmax_done;
  softmax_fail:
    give_up();
    if (lane == 0) report(p.status, MLA_STATUS_TIMEOUT);
  softmax_done:
    if (__any_sync(0xffffffffu, out_of_range) && lane == 0 && rank == 0) report(p.status, MLA_STATUS_SCORE_RANGE);
  }

  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
  __syncwarp();
  cluster_sync();   // no CTA leaves while its peer may still write into its shared memory
  // After a give-up, roles may have left their loops with the peer's last
  // score tile still on its way here.  A give-up raises both CTAs' flags
  // before its CTA reaches the barrier above, so after it both flags agree
  // and both CTAs take the same branch.  A copy is only sent after the
  // receiver consumed the previous one, so at most the peer's last copy is
  // outstanding: wait (default limit) for its phase, which lands because it
  // was issued, then meet the peer once more.
  {
    // (addresses recomputed here rather than kept live through the roles)
    Bars* b = reinterpret_cast<Bars*>(((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023)) + kOffBar);
    if (*reinterpret_cast<volatile int*>(&b->wc.abort) != 0) {
      if (threadIdx.x == 0) {
        const uint32_t sent_by_peer = ld_cluster_u32(mapa(smem_u32(&b->sent_count), cluster_ctarank() ^ 1u));
        if (sent_by_peer > 0) mbar_drain<true>(&b->x_recv, (sent_by_peer - 1) & 1);
      }
      __syncwarp();
      cluster_sync();
    }
  }
}

std::atomic<uint64_t> g_wait_limit_ns{kWaitLimitNs};

// Once per device, so that later launches can be captured in a CUDA graph.
cudaError_t decode_smem_attr() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(mla_decode_fp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace

mla_status_t launch_decode_attn_fp4cache(const mla_dims_t& d, const void* q_lat, const void* q_rope,
                                         const void* kv_pool_fp4, const int32_t* block_table,
                                         const int32_t* seq_lens, const int32_t* plan_dev, int32_t num_clusters,
                                         float* o_part, float* lse_part, PlanRoom room, void* o_lat, float* lse_out,
                                         int32_t* status, void* stream) {
  // The pool as (byte or column, row within the block, block): a box may start
  // at a negative row, which the TMA fills with zeros (the shifted last page).
  CUtensorMap tm_codes, tm_rope, tm_scale;
  const uint8_t* pool = static_cast<const uint8_t*>(kv_pool_fp4);
  const uint64_t stride[2] = {kF4Row, (uint64_t)kPage * kF4Row};
  const uint64_t cdims[3] = {256, (uint64_t)kPage, (uint64_t)d.num_blocks};
  const uint32_t cbox[3] = {128, kPage, 1};
  mla_status_t st = encode_tmap_u8(&tm_codes, pool, 3, cdims, stride, cbox, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != MLA_OK) return st;
  const uint64_t sdims[3] = {32, (uint64_t)kPage, (uint64_t)d.num_blocks};
  const uint32_t sbox[3] = {16, kPage, 1};
  st = encode_tmap_u8(&tm_scale, pool + kF4ScaleOff, 3, sdims, stride, sbox, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (st != MLA_OK) return st;
  const uint64_t rdims[3] = {64, (uint64_t)kPage, (uint64_t)d.num_blocks};
  const uint32_t rbox[3] = {32, kPage, 1};
  st = encode_tmap_bf16(&tm_rope, pool + kF4RopeOff, 3, rdims, stride, rbox, CU_TENSOR_MAP_SWIZZLE_64B);
  if (st != MLA_OK) return st;

  DecodeParams p;
  p.q_lat = static_cast<const __nv_bfloat16*>(q_lat);
  p.q_rope = static_cast<const __nv_bfloat16*>(q_rope);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.plan = plan_dev;
  p.o_part = o_part;
  p.lse_part = lse_part;
  p.o_lat = static_cast<__nv_bfloat16*>(o_lat);
  p.lse_out = lse_out;
  p.status = status;
  p.n_heads = d.n_heads;
  p.max_blocks = d.max_blocks_per_seq;
  p.num_blocks = d.num_blocks;
  p.s_q = d.s_q;
  p.causal = d.causal;
  p.B = d.B;
  p.n_rows = d.B * d.s_q;
  p.num_clusters = num_clusters;
  p.room = room;
  p.scale_log2 = d.scale * 1.4426950408889634f;
  p.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  p.zero = 0;

  cudaError_t e = decode_smem_attr();
  if (e == cudaSuccess) {
    e = launch_pdl(mla_decode_fp4_kernel, dim3(2 * num_clusters), dim3(kThreads), kSmemBytes, stream, tm_codes,
                   tm_rope, tm_scale, p);
    if (e == cudaSuccess) e = cudaGetLastError();
  }
  if (e != cudaSuccess) return set_error(MLA_ERR_CUDA, "decode launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

void set_decode_fp4_wait_limit_ns(int64_t ns) {
  g_wait_limit_ns.store(ns > 0 ? (uint64_t)ns : kWaitLimitNs, std::memory_order_relaxed);
}

}  // namespace mla
