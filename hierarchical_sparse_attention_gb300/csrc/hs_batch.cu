// The batch of a step: flat tokens, their positions and pool rows, and block tables, from the requests' lengths and
// the page table.
//
//   token_offsets = exclusive prefix sums of the accepted entries' new - old;  flat token k of entry i (the last one
//   with token_offsets[i] <= k): position p = old_i + k - token_offsets[i], row = page(p / page_size) page_size +
//   p % page_size
//
// Every CTA goes over all entries (three words each) in runs of its threads, with the run's prefix sums in shared
// memory, and writes its share of the run's tokens and table rows: one launch, no workspace, nothing handed from CTA to
// CTA. A step has tens to a thousand entries; up to kThreads of them are one run.
//
// What bounds it: the host. A call is 9 us of the caller's thread (19 arguments, one launch), the kernel 4 to 5 us of
// dependent loads and barriers for 32 entries as for 1,024 with 47,000 tokens and 4 MB of block tables.
#include "hs_chunk.h"

namespace hs {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kColumns = 256;  // of a block table's row: a warp's share at a time

__global__ void __launch_bounds__(kThreads) batch_plan_kernel(const BatchArgs a, uint32_t* __restrict__ err) {
  __shared__ uint32_t s_once[HS_MAX_PAGE_REQUESTS / 32], s_twice[HS_MAX_PAGE_REQUESTS / 32];
  __shared__ int32_t s_at[kThreads];  // the run's tokens before each entry
  __shared__ int32_t s_req[kThreads], s_old[kThreads], s_new[kThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first_cta = blockIdx.x == 0;
  for (int i = tid; i < (a.num_requests + 31) / 32; i += kThreads) s_once[i] = s_twice[i] = 0;
  pdl_wait();
  __syncthreads();
  for (int i = tid; i < a.n; i += kThreads) {
    const int32_t r = a.requests[i];
    if (r >= 0 && r < a.num_requests && (atomicOr(&s_once[r >> 5], 1u << (r & 31)) >> (r & 31) & 1u))
      atomicOr(&s_twice[r >> 5], 1u << (r & 31));
  }
  __syncthreads();
  int64_t most = (int64_t)a.max_pages * a.page_size;
  if (a.block_tables) most = min(most, (int64_t)a.max_blocks * a.page_size);
  int64_t asked = 0;  // by the entries so far
  int32_t taken = 0;  // by those that got their tokens
  uint32_t flags = 0;
  for (int base = 0; base < a.n; base += kThreads) {
    const int i = base + tid, here = min(kThreads, a.n - base);
    int32_t r = -1, from = 0, to = 0;
    if (i < a.n) {
      r = a.requests[i];
      from = a.old_lens[i];
      to = a.new_lens[i];
      uint32_t flag = 0;
      if (r < 0) {  // a padding entry
      } else if (r >= a.num_requests) {
        flag = HS_FLAG_TOKEN;
      } else if (s_twice[r >> 5] >> (r & 31) & 1u) {
        flag = HS_FLAG_DUP;
      } else if (from < 0 || to < from || to > most) {
        flag = HS_FLAG_SEQLEN;
      }
      if (r < 0 || flag) r = -1, from = to = 0;
      flags |= flag;
    }
    int64_t at[1] = {to - from}, sums[1];
    cta_prefix<kThreads>(at, sums);
    const int64_t before = asked + at[0];
    asked += sums[0];
    if (to > from && before + (to - from) > a.max_tokens) {
      flags |= HS_FLAG_FULL;
      r = -1;
      from = to = 0;
    }
    at[0] = to - from;
    cta_prefix<kThreads>(at, sums);
    const int64_t sum = sums[0];
    s_at[tid] = (int32_t)at[0];
    s_req[tid] = r;
    s_old[tid] = from;
    s_new[tid] = to;
    if (first_cta && i < a.n) {
      a.token_offsets[i] = taken + (int32_t)at[0];
      if (a.seq_lens) a.seq_lens[i] = to;
    }
    __syncthreads();
    // the run's tokens
    if (a.entries || a.positions || a.rows) {
      for (int64_t k = (int64_t)blockIdx.x * kThreads + tid; k < sum; k += (int64_t)gridDim.x * kThreads) {
        int lo = 0, hi = here - 1;  // the last entry whose prefix is <= k
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_at[mid] <= (int32_t)k) lo = mid;
          else hi = mid - 1;
        }
        const int32_t pos = s_old[lo] + ((int32_t)k - s_at[lo]);
        const int64_t to_slot = taken + k;
        if (a.entries) a.entries[to_slot] = base + lo;
        if (a.positions) a.positions[to_slot] = pos;
        if (a.rows) {
          const int32_t b = pos / a.page_size;
          const int32_t page = a.pages[(int64_t)s_req[lo] * a.max_pages + b];
          const int64_t row = (int64_t)page * a.page_size + (pos - b * a.page_size);
          const bool there = page >= 0 && row < a.pool_rows;
          if (!there) flags |= HS_FLAG_DEVROW;
          a.rows[to_slot] = there ? (int32_t)row : -1;
        }
      }
    }
    // the run's table rows, kColumns of an entry to a warp
    if (a.block_tables) {
      const int parts = (a.max_blocks + kColumns - 1) / kColumns;
      for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < (int64_t)here * parts; u += (int64_t)gridDim.x * kWarps) {
        const int e = (int)(u / parts), c0 = (int)(u - (int64_t)e * parts) * kColumns;
        const int held = (int)(((int64_t)s_new[e] + a.page_size - 1) / a.page_size);  // (no larger than max_pages)
        const int32_t* src = a.pages + (int64_t)max(s_req[e], 0) * a.max_pages;
        int32_t* dst = a.block_tables + (int64_t)(base + e) * a.max_blocks;
        int32_t v[kColumns / 32];
#pragma unroll
        for (int j = 0; j < kColumns / 32; ++j) {
          const int c = c0 + 32 * j + lane;
          v[j] = c < held ? src[c] : -1;
        }
#pragma unroll
        for (int j = 0; j < kColumns / 32; ++j) {
          const int c = c0 + 32 * j + lane;
          if (c < a.max_blocks) dst[c] = v[j];
        }
      }
    }
    taken += (int32_t)sum;
    __syncthreads();  // (before the next run's entries)
  }
  if (first_cta && tid == 0) a.token_offsets[a.n] = taken;
  for (int64_t k = taken + (int64_t)blockIdx.x * kThreads + tid; k < a.max_tokens; k += (int64_t)gridDim.x * kThreads) {
    if (a.entries) a.entries[k] = -1;
    if (a.positions) a.positions[k] = -1;
    if (a.rows) a.rows[k] = -1;
  }
  if (flags) atomicOr(err, flags);
}

}  // namespace

cudaError_t launch_batch_plan(const BatchArgs& a, uint32_t* err, cudaStream_t stream) {
  const int64_t tokens = (a.max_tokens + kThreads - 1) / kThreads;
  const int64_t tables = a.block_tables ? ((int64_t)a.n * ((a.max_blocks + kColumns - 1) / kColumns) + kWarps - 1) / kWarps : 1;
  const int64_t ctas = tokens > tables ? tokens : tables;
  return launch(batch_plan_kernel, dim3((unsigned)(ctas < 1 ? 1 : ctas > 152 ? 152 : ctas)), kThreads, 0, stream, a, err);
}

}  // namespace hs
