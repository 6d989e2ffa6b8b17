// Steps with several new tokens of a sequence: the batch's plan, fp8 MLA rows, attention of chunks. What the
// kernels are told, their launch interface, and what they share.
//
// An fp8 record is 656 B: 512 B of e4m3 codes, four fp32 scales (scale b for dims 128 b .. 128 b + 127), 128 B of
// bf16 RoPE values.
#pragma once

#include "hs_fp4.h"

namespace hs {

constexpr int kFp8Latent = 512, kFp8Rope = 64, kFp8Dims = kFp8Latent + kFp8Rope;
constexpr int kFp8Block = 128;             // dims per scale
constexpr int kFp8Scales = kFp8Latent;     // byte offsets in a record
constexpr int kFp8RopeAt = kFp8Scales + 4 * (kFp8Latent / kFp8Block);
constexpr int kFp8Row = kFp8RopeAt + 2 * kFp8Rope;
static_assert(kFp8Row == HS_FP8_ROW_BYTES, "the record and the header agree");

struct BatchArgs {
  int32_t n, num_requests, max_pages, page_size, max_tokens, max_blocks;
  int64_t pool_rows;
  const int32_t *requests, *old_lens, *new_lens;  // [n]
  const int32_t* pages;                           // [num_requests, max_pages]
  int32_t* token_offsets;                         // [n + 1]
  int32_t* seq_lens;                              // [n] or NULL
  int32_t *entries, *positions, *rows;            // [max_tokens] or NULL
  int32_t* block_tables;                          // [n, max_blocks] or NULL
};
cudaError_t launch_batch_plan(const BatchArgs& a, uint32_t* err, cudaStream_t stream);

struct Fp8RowsArgs {
  int32_t n;
  uint16_t* kv;  // [n, kv_stride] bf16, 576 used (read by pack, written by unpack)
  int64_t kv_stride;
  const int32_t* rows;  // [n]
  uint8_t* pool;
  int64_t pool_rows;
  // pack
  const uint16_t* norm_weight;  // [512] bf16, or NULL
  float norm_eps;
  const int32_t* positions;  // [n], or NULL
  const float* rope_table;   // [rope_positions, 64]: 32 cosines, 32 sines; or NULL
  int32_t rope_positions;
};
cudaError_t launch_fp8_pack(const Fp8RowsArgs& a, uint32_t* err, cudaStream_t stream);
cudaError_t launch_fp8_unpack(const Fp8RowsArgs& a, uint32_t* err, cudaStream_t stream);

struct ChunkArgs {
  int32_t n, num_heads, max_tokens;
  const int32_t* token_offsets;  // [n + 1]
  const int32_t* seq_lens;       // [n]
  const uint16_t* q;             // [max_tokens, num_heads, 576] bf16
  const uint8_t* pool;           // [pool_rows, 656]
  int64_t pool_rows;
  int32_t page_size, max_blocks;
  const int32_t* block_tables;  // [n, max_blocks]
  float sm_scale;
  uint16_t* o;  // [max_tokens, num_heads, 512] bf16
  float* lse;   // [max_tokens, num_heads]
  int64_t max_kv_tokens;
};
size_t chunk_workspace_bytes(int32_t n, int32_t num_heads, int32_t max_tokens, int64_t max_kv_tokens);
cudaError_t launch_chunk_mla(const ChunkArgs& a, void* workspace, uint32_t* err, cudaStream_t stream);

// Exclusive prefix sums of N values over the CTA's kThreads threads; total gets the sums. Called by every thread. Sums
// are 64-bit.
template <int kThreads, int N>
__device__ __forceinline__ void cta_prefix(int64_t (&v)[N], int64_t (&total)[N]) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kThreads % 32 == 0, "whole warps");
  __shared__ int64_t s_warp[N][kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = v[i];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x[i], d);
      if (lane >= d) x[i] += y;
    }
  __syncthreads();  // the last call's readers are done with s_warp
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane == 31) s_warp[i][warp] = x[i];
  __syncthreads();
  // every thread sums the warps before its own (few: no second scan and barrier)
#pragma unroll
  for (int i = 0; i < N; ++i) {
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int64_t y = s_warp[i][w];
      before += w < warp ? y : 0;
      all += y;
    }
    total[i] = all;
    v[i] = before + x[i] - v[i];
  }
}

}  // namespace hs
