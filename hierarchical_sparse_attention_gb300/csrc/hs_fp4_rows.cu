// 4-bit MLA rows written from bf16 tokens (pack) and read back as bf16 (unpack), a warp per token.
//
// pack, per block of 16 latent dims x, with y = x / latent_scale (exact: a power of two):
//   scale = e4m3(max |y| / 6), saturating;  code_i = e2m1(y_i / scale), saturating, 0 if scale = 0
// both to nearest, ties to even; 6 is the largest e2m1 magnitude. In 32 bits this is what exact
// arithmetic gives: y has 8 significant bits, scale 4 and a point halfway between two codes 3, so a
// quotient that is not halfway is at least 2^-8 (relative) away from halfway (see `quotients`), and
// likewise max |y| / 6 and the scale's halfway points. A block with a NaN or an infinity gets the
// scale NaN (0x7F) and zero codes, so that it reads back as NaN. RoPE values are copied.
//
// What bounds them: memory. Measured for 32,768 tokens written and 65,536 read back, one after the
// other: 30.8 us, 155 MB, 0.74 of a copy's bandwidth (launches and the first loads' latency are a
// fifth of so short a pass). On the way, when that was 29.7: 37.8 us with a division per code and the loads after the
// row's number; two or four tokens of a warp at a time 29.1 and 33.3 us (and 1 and 2.5 us more for
// 32 tokens).
#include "hs_fp4.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

namespace hs {
namespace {

constexpr int kRowsThreads = 256;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float e4m3_value(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// The quotients x r of a pair of bf16 values, r = 1 / (latent_scale scale) rounded to nearest, each
// put on a grid of 2^-11 (that is what adding and taking away 1.5 x 2^12 does) with x's sign: in e2m1
// they round as the exact quotients do. One that is halfway between two codes (at least 1/4, a multiple
// of 1/4) is off by less than 2^-20 before and lands on the halfway point; one that is not is at least
// 2^-8 of it, so 2^-10, away and stays on its side.
__device__ __forceinline__ float2 quotients(uint32_t w, float r) {
  constexpr float kGrid = 6144.f;
  const float a = __fadd_rn(__fmaf_rn(bf16_lo(w), r, kGrid), -kGrid), b = __fadd_rn(__fmaf_rn(bf16_hi(w), r, kGrid), -kGrid);
  return make_float2(__uint_as_float((__float_as_uint(a) & 0x7FFFFFFFu) | (w << 16 & 0x80000000u)),
                     __uint_as_float((__float_as_uint(b) & 0x7FFFFFFFu) | (w & 0x80000000u)));
}

__global__ void __launch_bounds__(kRowsThreads) fp4_pack_kernel(const Fp4RowsArgs a, uint32_t* __restrict__ err) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t i = ((int64_t)blockIdx.x * kRowsThreads + threadIdx.x) >> 5;
  if (i >= a.n) return;  // whole warps
  // (a token that is skipped is read all the same, so that its values need not wait for its row's number)
  const int32_t row = a.rows[i];
  const uint16_t* src = a.kv + i * a.kv_stride;
  const uint4 v0 = *reinterpret_cast<const uint4*>(src + 16 * lane);
  const uint4 v1 = *reinterpret_cast<const uint4*>(src + 16 * lane + 8);
  const uint32_t rope = *reinterpret_cast<const uint32_t*>(src + kFp4Latent + 2 * lane);
  if (row < 0 || row >= a.pool_rows) {
    if (row >= 0 && lane == 0) atomicOr(err, HS_FLAG_DEVROW);
    return;
  }
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  uint32_t top = 0;  // the largest magnitude as bf16 bits, two lanes of 16
#pragma unroll
  for (int k = 0; k < 8; ++k) top = __vmaxu2(top, w[k] & 0x7FFF7FFFu);
  top = max(top & 0xFFFFu, top >> 16);
  const float inv = 1.f / a.latent_scale;
  uint8_t scale = 0x7F;
  uint32_t c[2] = {0u, 0u};
  if (top < 0x7F80u) {
    scale = __nv_cvt_float_to_fp8(__uint_as_float(top << 16) * inv / 6.f, __NV_SATFINITE, __NV_E4M3);
    const float s = e4m3_value(scale);
    if (s > 0.f) {
      const float r = inv * __frcp_rn(s);  // (inv is a power of two)
#pragma unroll
      for (int k = 0; k < 8; ++k)
        c[k >> 2] |= (uint32_t)__nv_cvt_float2_to_fp4x2(quotients(w[k], r), __NV_E2M1, cudaRoundNearest) << (8 * (k & 3));
    }
  }
  uint8_t* dst = a.pool + (int64_t)row * kFp4Row;
  *reinterpret_cast<uint2*>(dst + 8 * lane) = make_uint2(c[0], c[1]);
  dst[kFp4Scales + lane] = scale;
  *reinterpret_cast<uint32_t*>(dst + kFp4RopeAt + 4 * lane) = rope;
  // hs_backup may be the next kernel of the stream: it starts as a programmatic dependent and reads
  // rows before its wait, so each row is made visible before its writer exits
  __threadfence();
}

__global__ void __launch_bounds__(kRowsThreads) fp4_unpack_kernel(const Fp4RowsArgs a, uint32_t* __restrict__ err) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t i = ((int64_t)blockIdx.x * kRowsThreads + threadIdx.x) >> 5;
  if (i >= a.n) return;
  const int32_t row = a.rows[i];
  uint32_t w[8] = {}, rope = 0;
  if (row >= 0 && row < a.pool_rows) {
    const uint8_t* src = a.pool + (int64_t)row * kFp4Row;
    const uint2 c = *reinterpret_cast<const uint2*>(src + 8 * lane);
    const float s = e4m3_value(src[kFp4Scales + lane]) * a.latent_scale;  // exact: a power of two
    rope = *reinterpret_cast<const uint32_t*>(src + kFp4RopeAt + 4 * lane);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = ((k < 4 ? c.x : c.y) >> (8 * (k & 3))) & 0xFFu;
      const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)b, __NV_E2M1);
      const float2 v = __half22float2(__half2(h));
      // exact unless latent_scale takes the value out of bf16's range
      const __nv_bfloat162 o = __floats2bfloat162_rn(v.x * s, v.y * s);
      w[k] = *reinterpret_cast<const uint32_t*>(&o);
    }
  } else if (row >= a.pool_rows && lane == 0) {
    atomicOr(err, HS_FLAG_DEVROW);
  }
  uint16_t* dst = a.kv + i * a.kv_stride;
  *reinterpret_cast<uint4*>(dst + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(dst + 16 * lane + 8) = make_uint4(w[4], w[5], w[6], w[7]);
  *reinterpret_cast<uint32_t*>(dst + kFp4Latent + 2 * lane) = rope;
}

unsigned blocks(int32_t n) { return (unsigned)(((int64_t)n * 32 + kRowsThreads - 1) / kRowsThreads); }

}  // namespace

cudaError_t launch_fp4_pack(const Fp4RowsArgs& a, uint32_t* err, cudaStream_t stream) {
  return launch(fp4_pack_kernel, dim3(blocks(a.n)), kRowsThreads, 0, stream, a, err);
}

cudaError_t launch_fp4_unpack(const Fp4RowsArgs& a, uint32_t* err, cudaStream_t stream) {
  return launch(fp4_unpack_kernel, dim3(blocks(a.n)), kRowsThreads, 0, stream, a, err);
}

}  // namespace hs
