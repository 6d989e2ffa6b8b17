// 4-bit MLA rows: the record, what the kernels are told of it, and its launch interface.
//
// A record is 416 B: 256 B of e2m1 codes (latent dim 2i in the low nibble of byte i, dim 2i + 1 in
// its high nibble), 32 B of e4m3 scales (scale b for dims 16b .. 16b + 15), 128 B of bf16 RoPE
// values. 416 B is 13 sectors of 32 B, so a row of a 32-byte aligned pool shares no sector with
// its neighbours. A latent value is code x scale x latent_scale: at most 2 + 4 significant bits and
// latent_scale a power of two, so code x scale is exact in f16 (|.| <= 6 x 448, >= 2^-10) and
// code x scale x latent_scale in bf16.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "hs.h"

namespace hs {

constexpr int kFp4Latent = 512, kFp4Rope = 64, kFp4Dims = kFp4Latent + kFp4Rope;
constexpr int kFp4Block = 16;                            // dims per scale
constexpr int kFp4Scales = kFp4Latent / 2;               // byte offsets in a record
constexpr int kFp4RopeAt = kFp4Scales + kFp4Latent / kFp4Block;
constexpr int kFp4Row = kFp4RopeAt + 2 * kFp4Rope;
static_assert(kFp4Row == HS_FP4_ROW_BYTES, "the record and the header agree");

// A launch as a programmatic dependent of the kernel before it, which saves the gap between the two:
// every kernel launched so begins with pdl_wait(), in every thread. Returns its own error
// (cudaGetLastError could hand back another call's).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

struct Fp4RowsArgs {
  int32_t n;
  uint16_t* kv;  // [n, kv_stride] bf16, 576 used (read by pack, written by unpack)
  int64_t kv_stride;
  const int32_t* rows;  // [n]
  float latent_scale;
  uint8_t* pool;
  int64_t pool_rows;
};

// One attention call: the tiles' rows come from a row table (out_rows) or, with seq_lens, from
// the tokens that a window and sinks leave visible, through a page table.
struct Fp4MlaArgs {
  const uint16_t* q;  // [R, num_queries, num_heads, 576] bf16
  const uint8_t* pool;
  int64_t pool_rows;
  int32_t num_heads, num_queries, splits;
  float sm_scale, latent_scale;
  uint16_t* o;  // [R, num_queries, num_heads, 512] bf16
  float* lse;   // [R, num_queries, num_heads]
  const int32_t* out_rows;  // row table [R, top_k], -1: none
  int32_t top_k;
  const int32_t* seq_lens;  // window: lengths [R], each with its last num_queries tokens the queries'
  const int32_t* pages;     // [R, max_pages], -1: not on the device
  int32_t page_size, max_pages, window, sinks;
  uint32_t page_mul, page_shift, pool_pages;  // filled in by launch_fp4_mla
};

cudaError_t launch_fp4_pack(const Fp4RowsArgs& a, uint32_t* err, cudaStream_t stream);
cudaError_t launch_fp4_unpack(const Fp4RowsArgs& a, uint32_t* err, cudaStream_t stream);
int32_t fp4_mla_splits(int32_t num_requests, int32_t num_heads, int32_t num_queries, int64_t rows);
size_t fp4_mla_workspace_bytes(int32_t num_requests, int32_t num_heads, int32_t num_queries, int32_t splits);
// part: the splits' partial outputs and log-sum-exps (NULL for one split).
cudaError_t launch_fp4_mla(const Fp4MlaArgs& a, int32_t num_requests, float* part, uint32_t* err,
                           cudaStream_t stream);

// Pages (hs_pages.cu): the caller's descriptor and the widest piece its pools can be copied in.
struct PageArgs {
  hs_page_pool p;
  int32_t vec;  // 16, 4 or 1
};
size_t pages_workspace_bytes(int32_t num_requests, int32_t num_pages);
cudaError_t launch_pages_init(const PageArgs& a, cudaStream_t stream);
cudaError_t launch_pages_extend(const PageArgs& a, int32_t n, const int32_t* requests, const int32_t* old_lens,
                                const int32_t* new_lens, int32_t* granted, cudaStream_t stream);
cudaError_t launch_pages_fork(const PageArgs& a, int32_t n, const int32_t* parents, const int32_t* children,
                              const int32_t* lens, int32_t* granted, cudaStream_t stream);
cudaError_t launch_pages_free(const PageArgs& a, int32_t n, const int32_t* requests, const int32_t* first_pages,
                              const int32_t* end_pages, cudaStream_t stream);
cudaError_t launch_pages_compact(const PageArgs& a, cudaStream_t stream);

}  // namespace hs
