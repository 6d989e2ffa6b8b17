// MLA decode attention over 4-bit rows: through a row table (hs_fp4_sparse_mla_decode) or through
// a page table for the tokens of a sliding window and its sinks (hs_fp4_window_mla_decode).
//
// Per query (request r, query i, head h) over the rows j that it sees:
//   s_j = sm_scale (q[:512] . latent_j + q[512:] . rope_j),   o = softmax(s) . latent,
//   lse = log sum_j exp s_j
// One CTA per query and head; each warp takes every eighth row and keeps the running maximum m,
// the sum l and the output of what it has seen: a new maximum m' scales l and the output by
// exp(m - m'). The warps' parts are joined in shared memory. All sums are in 32 bits.
#include "hs_fp4.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

namespace hs {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;

__global__ void __launch_bounds__(kThreads) fp4_mla_kernel(const Fp4MlaArgs a, uint32_t* __restrict__ err) {
  __shared__ float s_o[kWarps][kFp4Latent], s_m[kWarps], s_l[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, i = blockIdx.x % a.num_queries, r = blockIdx.x / a.num_queries;
  int64_t n = 0, sinks = 0, start = 0;  // rows seen; the first `sinks` are tokens 0 .., the rest from `start`
  if (a.seq_lens == nullptr) {
    n = a.top_k;
  } else {
    const int64_t S = a.seq_lens[r];
    if (S < 0 || S > (int64_t)a.max_pages * a.page_size) {
      if (threadIdx.x == 0) atomicOr(err, HS_FLAG_SEQLEN);
    } else if (S - a.num_queries + i >= 0) {
      const int64_t p = S - a.num_queries + i;
      sinks = min((int64_t)a.sinks, p + 1);
      start = max(sinks, p + 1 - a.window);
      n = sinks + p + 1 - start;
    }
  }
  const size_t at = ((size_t)r * a.num_queries + i) * a.num_heads + h;
  float q[16], q_rope[2];
#pragma unroll
  for (int k = 0; k < 16; ++k) q[k] = __uint_as_float((uint32_t)a.q[at * kFp4Dims + 16 * lane + k] << 16);
#pragma unroll
  for (int k = 0; k < 2; ++k) q_rope[k] = __uint_as_float((uint32_t)a.q[at * kFp4Dims + kFp4Latent + 2 * lane + k] << 16);
  float m = -INFINITY, l = 0.f, o[16] = {};
  for (int64_t j = warp; j < n; j += kWarps) {
    int64_t row;
    if (a.seq_lens == nullptr) {
      row = a.out_rows[(size_t)r * a.top_k + j];
    } else {
      const int64_t t = j < sinks ? j : start + j - sinks;
      const int32_t page = a.pages[(size_t)r * a.max_pages + t / a.page_size];
      row = page < 0 ? -1 : (int64_t)page * a.page_size + t % a.page_size;
      if ((row < 0 || row >= a.pool_rows) && lane == 0) atomicOr(err, HS_FLAG_DEVROW);
    }
    if (row < 0 || row >= a.pool_rows) continue;
    const uint8_t* rec = a.pool + row * kFp4Row;
    const uint2 c = *reinterpret_cast<const uint2*>(rec + 8 * lane);
    const float sc = __half2float(__half(__nv_cvt_fp8_to_halfraw(rec[kFp4Scales + lane], __NV_E4M3))) * a.latent_scale;
    const uint32_t rope = *reinterpret_cast<const uint32_t*>(rec + kFp4RopeAt + 4 * lane);
    float v[16], s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t b = ((k < 4 ? c.x : c.y) >> (8 * (k & 3))) & 0xFFu;
      const float2 x = __half22float2(__half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)b, __NV_E2M1)));
      v[2 * k] = x.x * sc;
      v[2 * k + 1] = x.y * sc;
      s += q[2 * k] * v[2 * k] + q[2 * k + 1] * v[2 * k + 1];
    }
    s += q_rope[0] * __uint_as_float(rope << 16) + q_rope[1] * __uint_as_float(rope & 0xFFFF0000u);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.sm_scale;
    const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : expf(m - mn), p = s == -INFINITY ? 0.f : expf(s - mn);
    l = l * f + p;
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = o[k] * f + p * v[k];
    m = mn;
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) s_o[warp][16 * lane + k] = o[k];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  for (int w = 0; w < kWarps; ++w) sum += s_m[w] == -INFINITY && s_l[w] == 0.f ? 0.f : s_l[w] * expf(s_m[w] - top);
  for (int d = threadIdx.x; d < kFp4Latent; d += kThreads) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += s_m[w] == -INFINITY && s_l[w] == 0.f ? 0.f : s_o[w][d] * expf(s_m[w] - top);
    const __nv_bfloat16 b = __float2bfloat16_rn(sum == 0.f ? 0.f : x / sum);
    a.o[at * kFp4Latent + d] = *reinterpret_cast<const uint16_t*>(&b);
  }
  if (threadIdx.x == 0) a.lse[at] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

int32_t fp4_mla_splits(int32_t, int32_t, int32_t, int64_t) { return 1; }
size_t fp4_mla_workspace_bytes(int32_t num_requests, int32_t num_heads, int32_t num_queries, int32_t splits) {
  return splits == 1 ? 0 : (size_t)splits * num_requests * num_queries * num_heads * (kFp4Latent + 1) * sizeof(float);
}

cudaError_t launch_fp4_mla(const Fp4MlaArgs& a, int32_t num_requests, float* part, uint32_t* err,
                           cudaStream_t stream) {
  (void)part;
  return launch(fp4_mla_kernel, dim3((unsigned)num_requests * a.num_queries, (unsigned)a.num_heads), kThreads, stream,
                false, a, err);
}

}  // namespace hs
