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
// shuffles.
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

__global__ void __launch_bounds__(kThreads)
kv_quantize_fp4_kernel(const uint4* __restrict__ kv, const int32_t* __restrict__ slots, long long n,
                       uint8_t* __restrict__ pool, long long pool_rows, int32_t* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = threadIdx.x % kRowChunks;
  const long long row = (long long)blockIdx.x * kRowsPerBlock + threadIdx.x / kRowChunks;
  // (no early return: the four threads of a group share a row, so a shuffle
  // needs only the threads of its own group, which all take the same way)
  const bool in = row < n;
  const long long slot = in ? (long long)slots[row] : -1;
  const bool live = slot >= 0 && slot < pool_rows;
  if (in && !live && slot != -1 && c == 0) report(status, MLA_STATUS_BAD_BLOCK);
  const uint4 v = live ? __ldg(kv + row * kRowChunks + c) : make_uint4(0, 0, 0, 0);
  float x[8];
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    amax = fmaxf(amax, fabsf(x[i]));
    nan |= x[i] != x[i];
  }
  const uint32_t group = 0xFu << (threadIdx.x & 28);   // the lanes of this group of 32 columns
  amax = fmaxf(amax, __shfl_xor_sync(group, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(group, amax, 2));
  nan = __any_sync(group, nan);
  if (!live) return;
  uint8_t* dst = pool + slot * kF4Row;
  if (c >= kLatChunks) {
    reinterpret_cast<uint4*>(dst + kF4RopeOff)[c - kLatChunks] = v;
    return;
  }
  // The largest usable scale: beyond it 6 s leaves fp16.  Such a row is written
  // with that scale and flagged.
  __half s16 = __float2half_rn(fminf(amax, 65504.f) / 6.f);
  bool out_of_range = nan;
  if (!(__half2float(s16) <= kF4MaxScale)) {
    s16 = __float2half_rn(kF4MaxScale);
    out_of_range = true;
  }
  if (amax > 65504.f) out_of_range = true;
  const float s = __half2float(s16);
  const float r = s > 0.f ? 1.f / s : 0.f;
  // y = x / s is within 2^-22 of the quotient (relative).  A quotient that is not
  // half-way between two grid values is at least 2^-13 away from it (x has 8
  // significant bits, s 11, a half-way point 3), and |y| < 8.5 unless the row is
  // flagged, so adding and taking off 48 (a grid of 2^-18) moves only the exact
  // ties, onto the tie: the codes are those of the exact quotient.
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y0 = __fsub_rn(__fadd_rn(x[2 * i] * r, 48.f), 48.f);
    const float y1 = __fsub_rn(__fadd_rn(x[2 * i + 1] * r, 48.f), 48.f);
    codes |= cvt_e2m1x2(copysignf(y0, x[2 * i]), copysignf(y1, x[2 * i + 1])) << (8 * i);
  }
  reinterpret_cast<uint32_t*>(dst)[c] = codes;
  if ((c & 3) == 0) {
    reinterpret_cast<__half*>(dst + kF4ScaleOff)[c >> 2] = s16;
    if (out_of_range) report(status, MLA_STATUS_CACHE_RANGE);
  }
}

__global__ void __launch_bounds__(kThreads)
kv_dequantize_fp4_kernel(const uint8_t* __restrict__ pool, const int32_t* __restrict__ slots, long long n,
                         uint4* __restrict__ out, long long pool_rows, int32_t* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = threadIdx.x % kRowChunks;
  const long long row = (long long)blockIdx.x * kRowsPerBlock + threadIdx.x / kRowChunks;
  if (row >= n) return;
  const long long slot = slots[row];
  if (slot < 0 || slot >= pool_rows) {
    if (slot != -1 && c == 0) report(status, MLA_STATUS_BAD_BLOCK);
    return;
  }
  const uint8_t* src = pool + slot * kF4Row;
  if (c >= kLatChunks) {
    out[row * kRowChunks + c] = __ldg(reinterpret_cast<const uint4*>(src + kF4RopeOff) + (c - kLatChunks));
    return;
  }
  const uint32_t codes = __ldg(reinterpret_cast<const uint32_t*>(src) + c);
  const float s = __half2float(__ldg(reinterpret_cast<const __half*>(src + kF4ScaleOff) + (c >> 2)));
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // code x scale is exact in fp32 (2 + 11 bits); one rounding to bf16
    const float2 f = unpack_f16x2(cvt_f16x2_e2m1x2((codes >> (8 * i)) & 0xFFu));
    o[i] = pack_bf16(f.x * s, f.y * s);
  }
  out[row * kRowChunks + c] = make_uint4(o[0], o[1], o[2], o[3]);
}

mla_status_t grid_of(long long n, unsigned* blocks) {
  const long long g = (n + kRowsPerBlock - 1) / kRowsPerBlock;
  if (g > INT32_MAX) return set_error(MLA_ERR_UNSUPPORTED, "too many rows in one call");
  *blocks = (unsigned)g;
  return MLA_OK;
}

}  // namespace

mla_status_t launch_kv_quantize_fp4(const void* kv, const int32_t* slots, long long n, void* pool_fp4,
                                    long long pool_rows, int32_t* status, void* stream) {
  unsigned blocks = 0;
  mla_status_t st = grid_of(n, &blocks);
  if (st != MLA_OK) return st;
  cudaError_t e = launch_pdl(kv_quantize_fp4_kernel, dim3(blocks), dim3(kThreads), 0, stream,
                             static_cast<const uint4*>(kv), slots, n, static_cast<uint8_t*>(pool_fp4), pool_rows,
                             status);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(MLA_ERR_CUDA, "kv_quantize_fp4 launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

mla_status_t launch_kv_dequantize_fp4(const void* pool_fp4, const int32_t* slots, long long n, void* out,
                                      long long pool_rows, int32_t* status, void* stream) {
  unsigned blocks = 0;
  mla_status_t st = grid_of(n, &blocks);
  if (st != MLA_OK) return st;
  cudaError_t e = launch_pdl(kv_dequantize_fp4_kernel, dim3(blocks), dim3(kThreads), 0, stream,
                             static_cast<const uint8_t*>(pool_fp4), slots, n, static_cast<uint4*>(out), pool_rows,
                             status);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return set_error(MLA_ERR_CUDA, "kv_dequantize_fp4 launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

}  // namespace mla
