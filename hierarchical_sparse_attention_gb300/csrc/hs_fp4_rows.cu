// 4-bit MLA rows written from bf16 tokens (pack) and read back as bf16 (unpack), a warp per token.
//
// pack, per block of 16 latent dims x, with y = x / latent_scale (exact: a power of two):
//   scale = e4m3(max |y| / 6), saturating;  code_i = e2m1(y_i / scale), saturating, 0 if scale = 0
// both to nearest, ties to even; 6 is the largest e2m1 magnitude. In 32 bits this is what exact
// arithmetic gives: y has 8 significant bits and scale 4, so a quotient that is not halfway
// between two codes is at least 2^-8 (relative) away from halfway, and one that is comes out of
// the division exactly; likewise max |y| / 6 and the scale's halfway points. A block with a NaN or
// an infinity gets the scale NaN (0x7F) and zero codes, so that it reads back as NaN.
// RoPE values are copied.
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

__global__ void __launch_bounds__(kRowsThreads) fp4_pack_kernel(const Fp4RowsArgs a, uint32_t* __restrict__ err) {
  const int lane = threadIdx.x & 31;
  const int64_t i = ((int64_t)blockIdx.x * kRowsThreads + threadIdx.x) >> 5;
  if (i < a.n) {  // whole warps
    const int32_t row = a.rows[i];
    if (row >= 0 && row < a.pool_rows) {
      const uint16_t* src = a.kv + i * a.kv_stride;
      uint8_t* dst = a.pool + (int64_t)row * kFp4Row;
      const uint4 v0 = *reinterpret_cast<const uint4*>(src + 16 * lane);
      const uint4 v1 = *reinterpret_cast<const uint4*>(src + 16 * lane + 8);
      const uint32_t rope = *reinterpret_cast<const uint32_t*>(src + kFp4Latent + 2 * lane);
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
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 y = make_float2(__fdiv_rn(bf16_lo(w[k]) * inv, s), __fdiv_rn(bf16_hi(w[k]) * inv, s));
            c[k >> 2] |= (uint32_t)__nv_cvt_float2_to_fp4x2(y, __NV_E2M1, cudaRoundNearest) << (8 * (k & 3));
          }
        }
      }
      *reinterpret_cast<uint2*>(dst + 8 * lane) = make_uint2(c[0], c[1]);
      dst[kFp4Scales + lane] = scale;
      *reinterpret_cast<uint32_t*>(dst + kFp4RopeAt + 4 * lane) = rope;
      // hs_backup may be the next kernel of the stream: it starts as a programmatic dependent and
      // reads rows before its wait, so each row is made visible before its writer exits
      __threadfence();
    } else if (row >= a.pool_rows && lane == 0) {
      atomicOr(err, HS_FLAG_DEVROW);
    }
  }
}

__global__ void __launch_bounds__(kRowsThreads) fp4_unpack_kernel(const Fp4RowsArgs a, uint32_t* __restrict__ err) {
  const int lane = threadIdx.x & 31;
  const int64_t i = ((int64_t)blockIdx.x * kRowsThreads + threadIdx.x) >> 5;
  if (i >= a.n) return;
  const int32_t row = a.rows[i];
  uint32_t w[8] = {}, rope = 0;
  if (row >= 0 && row < a.pool_rows) {
    const uint8_t* src = a.pool + (int64_t)row * kFp4Row;
    const uint2 c = *reinterpret_cast<const uint2*>(src + 8 * lane);
    const float s = e4m3_value(src[kFp4Scales + lane]);
    rope = *reinterpret_cast<const uint32_t*>(src + kFp4RopeAt + 4 * lane);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = ((k < 4 ? c.x : c.y) >> (8 * (k & 3))) & 0xFFu;
      const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)b, __NV_E2M1);
      const float2 v = __half22float2(__half2(h));
      // exact unless latent_scale takes the value out of bf16's range
      const __nv_bfloat162 o = __floats2bfloat162_rn(v.x * s * a.latent_scale, v.y * s * a.latent_scale);
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
  return launch(fp4_pack_kernel, dim3(blocks(a.n)), kRowsThreads, stream, false, a, err);
}

cudaError_t launch_fp4_unpack(const Fp4RowsArgs& a, uint32_t* err, cudaStream_t stream) {
  return launch(fp4_unpack_kernel, dim3(blocks(a.n)), kRowsThreads, stream, false, a, err);
}

}  // namespace hs
