// Rows of the 4-bit latent cache: the writer and the reader.
//
// A cached token is [c_KV (512) | k_rope (64)].  The 4-bit row keeps c_KV in
// sixteen groups of 32 columns, each with one fp16 scale, and k_rope in bf16:
//   bytes [0, 256)    E2M1 codes, column 2i in the low nibble of byte i
//   bytes [256, 288)  sixteen fp16 scales, c[t, j] = code[j] * s_{j / 32}
//   bytes [288, 416)  k_rope in bf16
// with s = fp16(amax / 6) and code = E2M1(c / s), rounded to nearest even and
// saturated at 6 (E2M1: 0, .5, 1, 1.5, 2, 3, 4, 6).  The scale is fp16 so that
// the attention kernel, whose operands are fp16, multiplies by it as it is; a
// group is 32 columns because the scales then cost 6 % of the row (16-column
// groups: 14 %).
//
// Both kernels are copies with a little arithmetic, bound by HBM: 1152 bytes in
// and 416 out per row (and the reverse).  A thread owns 8 columns (16 bytes of
// bf16, 4 bytes of codes), 72 threads a row, so that every load and store of a
// warp is contiguous; the four threads of a group combine their maxima by
// shuffles.  16301 rows, from a graph: written in 7.2 us, read in 5.0 (3.9 us each at
// the measured copy rate); 65536 rows 25.6 and 22.2 (15.7 each); 32 rows 1.5 and 1.5.  The
// writer's distance is no tail: a row's scales are sixteen 2-byte stores, and each
// wave's first loads are exposed.  Reads go to L2 (__ldcg): the kernel before, whose end this one waits for
// after its blocks have started, may have written what is read.
#include "fp4_format.h"
#include "mla_internal.h"
#include "ptx.cuh"

#include <cuda_bf16.h>

namespace mla {
namespace {

using namespace ptx;

constexpr int kRowChunks = 72;               // 16-byte chunks of a bf16 row: 64 of c_KV, 8 of k_rope
constexpr int kLatChunks = 64;
constexpr int kRowsPerBlock = 4;
constexpr int kThreads = kRowChunks * kRowsPerBlock;

__device__ __forceinline__ void report(int32_t* status, int bits) {
  if (status) atomicOr(status, bits);
}

// fma(x, r, 48) - 48 of a pair, each step rounded to nearest.
__device__ __forceinline__ float2 to_grid(float2 x, float r) {
  float2 y;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 c, {%6, %6};\n\tadd.rn.f32x2 a, a, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(x.x), "f"(x.y), "f"(r), "f"(48.f), "f"(-48.f));
  return y;
}

// One thread's part of a row: 8 columns of c_KV, or 16 bytes of k_rope (c >= kLatChunks).
// `live` is the same for the four threads of a group.
__device__ __forceinline__ void quantize_chunk(uint4 v, int c, bool live, uint8_t* dst, int32_t* status) {
  float x[8];
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;   // largest magnitudes, a pair of bf16 (their signs come out meaningless)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
  }
  m = max(m & 0x7FFFu, (m >> 16) & 0x7FFFu);   // (as integers magnitudes order like the values, NaN above all)
  const uint32_t group = 0xFu << (threadIdx.x & 28);   // the lanes of this group of 32 columns
  m = max(m, __shfl_xor_sync(group, m, 1));
  m = max(m, __shfl_xor_sync(group, m, 2));
  if (!live) return;
  if (c >= kLatChunks) {
    reinterpret_cast<uint4*>(dst + kF4RopeOff)[c - kLatChunks] = v;
    return;
  }
  // The largest usable scale: beyond it 6 s leaves fp16.  A group with a larger value or a
  // NaN is written with that scale and flagged.
  const float amax = __uint_as_float(m << 16);
  const bool out_of_range = !(amax <= 65504.f);
  const __half s16 = __float2half_rn(out_of_range ? kF4MaxScale : amax / 6.f);
  const float s = __half2float(s16);
  const float r = s > 0.f ? 1.f / s : 0.f;
  // x r is within 2^-22 of x / s (relative).  A quotient that is not half-way
  // between two grid values is at least 2^-13 away from it (x has 8 significant bits,
  // s 11, a half-way point 3), and |x / s| <= 9 unless the row is flagged (a subnormal s may be two
  // thirds of amax / 6), so adding and taking off 48 (a grid of 2^-18) moves only the exact ties, onto the
  // tie: the codes are those of the exact quotient.  The sum loses the sign of what becomes 0: a
  // code keeps the sign of its value (8 is -0).
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = to_grid(make_float2(x[2 * i], x[2 * i + 1]), r);
    codes |= cvt_e2m1x2(copysignf(y.x, x[2 * i]), copysignf(y.y, x[2 * i + 1])) << (8 * i);
  }
  reinterpret_cast<uint32_t*>(dst)[c] = codes;
  if ((c & 3) == 0) {
    reinterpret_cast<__half*>(dst + kF4ScaleOff)[c >> 2] = s16;
    if (out_of_range) report(status, MLA_STATUS_CACHE_RANGE);
  }
}

// kRows rows per thread, all loads in flight before the first is used: rows
// blockIdx.x * 4 kRows + 4 i + threadIdx.x / 72.
template <int kRows>
__global__ void __launch_bounds__(kThreads)
kv_quantize_fp4_kernel(const uint4* kv, const int32_t* slots, long long n,
                       uint8_t* pool, long long pool_rows, int32_t* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = threadIdx.x % kRowChunks;
  const long long row0 = (long long)blockIdx.x * (kRowsPerBlock * kRows) + threadIdx.x / kRowChunks;
  uint4 v[kRows];
  long long slot[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const long long row = row0 + kRowsPerBlock * i;
    slot[i] = row < n ? (long long)__ldcg(slots + row) : -1;
    v[i] = row < n ? __ldcg(kv + row * kRowChunks + c) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    // (no early return: the shuffles of a group's four threads, which share a row)
    const bool live = slot[i] >= 0 && slot[i] < pool_rows;
    if (!live && slot[i] != -1 && c == 0) report(status, MLA_STATUS_BAD_BLOCK);
    quantize_chunk(v[i], c, live, pool + slot[i] * kF4Row, status);
  }
}

template <int kRows>
__global__ void __launch_bounds__(kThreads)
kv_dequantize_fp4_kernel(const uint8_t* pool, const int32_t* slots, long long n,
                         uint4* out, long long pool_rows, int32_t* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = threadIdx.x % kRowChunks;
  const long long row0 = (long long)blockIdx.x * (kRowsPerBlock * kRows) + threadIdx.x / kRowChunks;
  long long slot[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const long long row = row0 + kRowsPerBlock * i;
    slot[i] = row < n ? (long long)__ldcg(slots + row) : -1;
    if (slot[i] < 0 || slot[i] >= pool_rows) {
      if (slot[i] != -1 && c == 0) report(status, MLA_STATUS_BAD_BLOCK);
      slot[i] = -1;
    }
  }
  if (c >= kLatChunks) {
    uint4 v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (slot[i] >= 0) v[i] = __ldcg(reinterpret_cast<const uint4*>(pool + slot[i] * kF4Row + kF4RopeOff) + (c - kLatChunks));
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (slot[i] >= 0) out[(row0 + kRowsPerBlock * i) * kRowChunks + c] = v[i];
    return;
  }
  uint32_t codes[kRows];
  __half scale[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (slot[i] < 0) continue;
    const uint8_t* src = pool + slot[i] * kF4Row;
    codes[i] = __ldcg(reinterpret_cast<const uint32_t*>(src) + c);
    scale[i] = __ldcg(reinterpret_cast<const __half*>(src + kF4ScaleOff) + (c >> 2));
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (slot[i] < 0) continue;
    const float s = __half2float(scale[i]);
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {   // code x scale is exact in fp32 (2 + 11 bits); one rounding to bf16
      const float2 f = unpack_f16x2(cvt_f16x2_e2m1x2((codes[i] >> (8 * k)) & 0xFFu));
      o[k] = pack_bf16(f.x * s, f.y * s);
    }
    out[(row0 + kRowsPerBlock * i) * kRowChunks + c] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// Rows per thread: one while the blocks of that are at most two per place on the card (a
// step's rows: latency counts), else four (a prompt's: bytes in flight count).  One
// against four, from a graph, writing / reading: 32 rows 1.5 / 1.5 against 2.5 / 2.2 us,
// 4096 2.6 / 2.3 against 3.2 / 2.7, 8192 4.3 / 3.7 against 4.7 / 3.6, 16301 7.3 / 5.9
// against 7.2 / 5.0, 65536 28.2 / 32.7 against 25.6 / 22.2.
mla_status_t grid_of(long long n, bool* many, unsigned* blocks) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return set_error(MLA_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
  *many = n > 2LL * sms * (2048 / kThreads) * kRowsPerBlock;
  const long long per = *many ? 4 * kRowsPerBlock : kRowsPerBlock;
  const long long g = (n + per - 1) / per;
  if (g > INT32_MAX) return set_error(MLA_ERR_UNSUPPORTED, "too many rows in one call");
  *blocks = (unsigned)g;
  return MLA_OK;
}

}  // namespace

mla_status_t launch_kv_quantize_fp4(const void* kv, const int32_t* slots, long long n, void* pool_fp4,
                                    long long pool_rows, int32_t* status, void* stream) {
  bool many = false;
  unsigned blocks = 0;
  mla_status_t st = grid_of(n, &many, &blocks);
  if (st != MLA_OK) return st;
  cudaError_t e = launch_pdl(many ? kv_quantize_fp4_kernel<4> : kv_quantize_fp4_kernel<1>, dim3(blocks), dim3(kThreads), 0, stream,
                             static_cast<const uint4*>(kv), slots, n, static_cast<uint8_t*>(pool_fp4), pool_rows,
                             status);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(MLA_ERR_CUDA, "kv_quantize_fp4 launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

mla_status_t launch_kv_dequantize_fp4(const void* pool_fp4, const int32_t* slots, long long n, void* out,
                                      long long pool_rows, int32_t* status, void* stream) {
  bool many = false;
  unsigned blocks = 0;
  mla_status_t st = grid_of(n, &many, &blocks);
  if (st != MLA_OK) return st;
  cudaError_t e = launch_pdl(many ? kv_dequantize_fp4_kernel<4> : kv_dequantize_fp4_kernel<1>, dim3(blocks), dim3(kThreads), 0, stream,
                             static_cast<const uint8_t*>(pool_fp4), slots, n, static_cast<uint4*>(out), pool_rows,
                             status);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(MLA_ERR_CUDA, "kv_dequantize_fp4 launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

}  // namespace mla
