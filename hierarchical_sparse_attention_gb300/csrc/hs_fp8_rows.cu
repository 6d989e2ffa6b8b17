// fp8 MLA rows written from bf16 tokens (pack: root-mean-square norm, rotary positions, quantisation) and read back as
// bf16 (unpack), a warp per token.
//
// pack, over a token's 512 latent values x:  y = x w / sqrt(mean x^2 + eps); per 128 dims scale = the least power of two
// with max |y| <= 448 scale; code = e4m3(y / scale). RoPE pairs (a, b): a cos - b sin, a sin + b cos.
//
// The codes are those of exact arithmetic (but for y within 2^-44 of a border between two codes): the sum of squares and
// the root are kept as sums of two floats, and y, a product of the exact x w with them, is rounded to odd at 24 bits, so
// that the hardware's rounding to e4m3 and the scale's comparison see which side of a border y is on. Rounded to nearest
// at 24 bits instead, one code of some 300,000 falls on the other side, by a whole step (2^-3 of the value).
//
// What bounds them, at 32,768 tokens written and 65,536 read back (42.9 us in a row; the bytes take 27.5): reading back, memory
// (20.5 us, 5.9 TB/s); writing, the instructions of exact rounding (25.5 us, 74 % of the issue slots; its bytes take 10).
// Tried: tokens in a loop, the next one's loads ahead (26.6); in 32 bits first, and exactly where values 2^-20 lower and
// higher have other codes (25 to 27: the second conversion costs what it saves).
#include "hs_chunk.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace hs {
namespace {

constexpr int kRowsThreads = 256;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A sum of two floats, hi the nearest to it.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
  float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));  // s + e = a.hi + b.hi
  e = __fadd_rn(e, __fadd_rn(a.lo, b.lo));
  Pair r;
  r.hi = __fadd_rn(s, e);
  r.lo = __fsub_rn(e, __fsub_rn(r.hi, s));
  return r;
}

// v r.hi + v r.lo, rounded to odd: cut to 24 bits, the last one set where anything was cut off.
__device__ __forceinline__ float times_odd(float v, Pair r) {
  const float c = __fmul_rn(v, r.lo), q = __fmaf_rz(v, r.hi, c);
  const float left = __fadd_rn(__fmaf_rn(v, r.hi, -q), c);
  // (r > 0: the sign is v's, a zero's too)
  return __uint_as_float(__float_as_uint(q) | (__float_as_uint(v) & 0x80000000u) | (left != 0.f && fabsf(q) < INFINITY ? 1u : 0u));
}

__global__ void __launch_bounds__(kRowsThreads) fp8_pack_kernel(const Fp8RowsArgs a, uint32_t* __restrict__ err) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t i = ((int64_t)blockIdx.x * kRowsThreads + threadIdx.x) >> 5;
  if (i >= a.n) return;  // whole warps
  // (a token that is skipped is read all the same, so that its values need not wait for its row's number)
  const int32_t row = a.rows[i];
  const int32_t pos = a.rope_table ? a.positions[i] : 0;
  const uint16_t* src = a.kv + i * a.kv_stride;
  const uint4 v0 = *reinterpret_cast<const uint4*>(src + 16 * lane);
  const uint4 v1 = *reinterpret_cast<const uint4*>(src + 16 * lane + 8);
  uint32_t rope = *reinterpret_cast<const uint32_t*>(src + kFp8Latent + 2 * lane);
  const bool bad_row = row >= a.pool_rows, bad_pos = a.rope_table && (pos < 0 || pos >= a.rope_positions);
  if (row < 0 || bad_row || bad_pos) {
    if (row >= 0 && lane == 0) atomicOr(err, bad_row ? HS_FLAG_DEVROW : HS_FLAG_SEQLEN);
    return;
  }
  float cosine = 1.f, sine = 0.f;  // (on their way while the latents are worked on)
  if (a.rope_table) {
    const float* t = a.rope_table + (int64_t)pos * kFp8Rope + lane;
    cosine = __ldg(t);
    sine = __ldg(t + kFp8Rope / 2);
  }
  const uint32_t xs[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  float y[16];
  if (a.norm_weight) {
    const uint4 w0 = __ldg(reinterpret_cast<const uint4*>(a.norm_weight + 16 * lane));
    const uint4 w1 = __ldg(reinterpret_cast<const uint4*>(a.norm_weight + 16 * lane + 8));
    const uint32_t ws[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    // all of it over a power of two near the largest of |x| and sqrt(eps), so that squares neither overflow nor vanish
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = __vmaxu2(top, xs[k] & 0x7FFF7FFFu);
    top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
    const bool finite = top < 0x7F80u;
    const int down = min(max(max((int)(top >> 7), (int)(__float_as_uint(sqrtf(a.norm_eps)) >> 23)) - 127, -125), 125);
    const float unit = __uint_as_float((uint32_t)(127 - down) << 23);
    // A lane's 16 squares (below 4, of 16 bits, exact in the product): their sum from 4 on, which no square is larger than, so that
    // what each addition rounds off is what the square is over the difference, exactly. It is summed by itself.
    float total = 4.f, off = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      y[k] = __fmul_rn(k & 1 ? bf16_hi(xs[k >> 1]) : bf16_lo(xs[k >> 1]), unit);
      const float more = __fmaf_rn(y[k], y[k], total);
      off = __fadd_rn(off, __fmaf_rn(y[k], y[k], -__fsub_rn(more, total)));
      total = more;
    }
    Pair sum = add({total - 4.f, 0.f}, {off, 0.f});
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const Pair other = {__shfl_xor_sync(0xffffffffu, sum.hi, d), __shfl_xor_sync(0xffffffffu, sum.lo, d)};
      sum = add(sum, other);
    }
    const Pair mean = add({sum.hi * (1.f / kFp8Latent), sum.lo * (1.f / kFp8Latent)}, {a.norm_eps * unit * unit, 0.f});
    // 1 / sqrt(mean) by one Newton step in two floats from the nearest float (each lane the same)
    Pair r;
    r.hi = __frsqrt_rn(mean.hi);
    const float rr = __fmul_rn(r.hi, r.hi), rr_lo = __fmaf_rn(r.hi, r.hi, -rr);
    float left = __fmaf_rn(-mean.hi, rr, 1.f);
    left = __fmaf_rn(-mean.hi, rr_lo, left);
    left = __fmaf_rn(-mean.lo, rr, left);
    r.lo = finite ? 0.5f * r.hi * left : __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[2 * k] = times_odd(__fmul_rn(y[2 * k], bf16_lo(ws[k])), r);  // (x w is exact)
      y[2 * k + 1] = times_odd(__fmul_rn(y[2 * k + 1], bf16_hi(ws[k])), r);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      y[2 * k] = bf16_lo(xs[k]);
      y[2 * k + 1] = bf16_hi(xs[k]);
    }
  }
  uint32_t top = 0;  // of the block's magnitudes, as bits; eight lanes have a block
#pragma unroll
  for (int k = 0; k < 16; ++k) top = max(top, __float_as_uint(y[k]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
  float scale = __uint_as_float(0x7FC00000u);
  uint32_t c[4] = {0u, 0u, 0u, 0u};
  if (top < 0x7F800000u) {
    // 448 = 1.75 x 2^8; biased exponents: the scale's is at least 1, and at most 247
    const int e = max((int)(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u), 1);
    scale = __uint_as_float((uint32_t)e << 23);
    const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      c[k >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y[2 * k] * inv, y[2 * k + 1] * inv), __NV_SATFINITE, __NV_E4M3)
                   << (16 * (k & 1));
  }
  if (a.rope_table) {
    // each product's rounding error goes into the sum, so that cancellation does not show it
    const float x = bf16_lo(rope), z = bf16_hi(rope);
    const float zs = __fmul_rn(z, sine), zc = __fmul_rn(z, cosine);
    const float u = __fsub_rn(__fmaf_rn(x, cosine, -zs), __fmaf_rn(z, sine, -zs));
    const float v = __fadd_rn(__fmaf_rn(x, sine, zc), __fmaf_rn(z, cosine, -zc));
    const __nv_bfloat162 h = __floats2bfloat162_rn(u, v);
    rope = *reinterpret_cast<const uint32_t*>(&h);
  }
  uint8_t* dst = a.pool + (int64_t)row * kFp8Row;
  *reinterpret_cast<uint4*>(dst + 16 * lane) = make_uint4(c[0], c[1], c[2], c[3]);
  if ((lane & 7) == 0) *reinterpret_cast<float*>(dst + kFp8Scales + lane / 2) = scale;
  *reinterpret_cast<uint32_t*>(dst + kFp8RopeAt + 4 * lane) = rope;
  // hs_backup may be the next kernel of the stream: it starts as a programmatic dependent and reads
  // rows before its wait, so each row is made visible before its writer exits
  __threadfence();
}

__global__ void __launch_bounds__(kRowsThreads) fp8_unpack_kernel(const Fp8RowsArgs a, uint32_t* __restrict__ err) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t i = ((int64_t)blockIdx.x * kRowsThreads + threadIdx.x) >> 5;
  if (i >= a.n) return;
  const int32_t row = a.rows[i];
  uint32_t w[8] = {}, rope = 0;
  if (row >= 0 && row < a.pool_rows) {
    const uint8_t* src = a.pool + (int64_t)row * kFp8Row;
    const uint4 v = *reinterpret_cast<const uint4*>(src + 16 * lane);
    const float s = *reinterpret_cast<const float*>(src + kFp8Scales + 4 * (lane >> 3));
    rope = *reinterpret_cast<const uint32_t*>(src + kFp8RopeAt + 4 * lane);
    const uint32_t c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c[k >> 1] >> (16 * (k & 1))), __NV_E4M3);
      const float2 x = __half22float2(__half2(h));
      const __nv_bfloat162 o = __floats2bfloat162_rn(x.x * s, x.y * s);
      w[k] = *reinterpret_cast<const uint32_t*>(&o);
    }
  } else if (row >= a.pool_rows && lane == 0) {
    atomicOr(err, HS_FLAG_DEVROW);
  }
  uint16_t* dst = a.kv + i * a.kv_stride;
  *reinterpret_cast<uint4*>(dst + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(dst + 16 * lane + 8) = make_uint4(w[4], w[5], w[6], w[7]);
  *reinterpret_cast<uint32_t*>(dst + kFp8Latent + 2 * lane) = rope;
}

unsigned blocks(int32_t n) { return (unsigned)(((int64_t)n * 32 + kRowsThreads - 1) / kRowsThreads); }

}  // namespace

cudaError_t launch_fp8_pack(const Fp8RowsArgs& a, uint32_t* err, cudaStream_t stream) {
  return launch(fp8_pack_kernel, dim3(blocks(a.n)), kRowsThreads, 0, stream, a, err);
}

cudaError_t launch_fp8_unpack(const Fp8RowsArgs& a, uint32_t* err, cudaStream_t stream) {
  return launch(fp8_unpack_kernel, dim3(blocks(a.n)), kRowsThreads, 0, stream, a, err);
}

}  // namespace hs
