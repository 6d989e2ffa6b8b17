// Attention of a step's new tokens over the fp8 pages of their sequences, causal.
//
// Per query head of the token at position p, over the tokens t <= p of its sequence:
//   s_t = sm_scale (q[:512] . latent_t + q[512:] . rope_t),  o = softmax(s) . latent,  lse = log sum_t exp s_t
//
// A first kernel lists the entries with queries; the second has a warp per query head, which goes over its sequence in
// blocks of 32 rows (values in 32 bits in shared memory) with the running maximum and sum of a softmax.
#include "hs_chunk.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace hs {
namespace {

constexpr int MH = 128;  // query heads of a tile: all heads of as many tokens of an entry as fit
constexpr int DQK = kFp8Dims, DL = kFp8Latent;
constexpr int kListThreads = 512;

// An entry with queries.
struct Entry {
  int32_t q0, nq, seq;  // first flat token, queries, tokens (0: they see nothing)
  int32_t table;        // its number: the block table's row
  int32_t tile0;        // tiles of the entries before it
};
struct Work {
  int32_t* count;  // entries listed
  int32_t* tiles;
  Entry* entries;  // [n]
};
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
size_t work_of(Work* w, void* workspace, int32_t n) {
  uint8_t* at = static_cast<uint8_t*>(workspace);
  w->count = reinterpret_cast<int32_t*>(at);
  w->tiles = w->count + 1;
  w->entries = reinterpret_cast<Entry*>(at + 256);
  return 256 + up256((size_t)n * sizeof(Entry));
}

__global__ void __launch_bounds__(kListThreads) chunk_list_kernel(const ChunkArgs a, const Work w, uint32_t* __restrict__ err) {
  pdl_wait();
  const int tid = threadIdx.x, per_tile = MH / a.num_heads;
  int64_t blocks = 0, listed = 0, tiles = 0;
  uint32_t flags = 0;
  for (int base = 0; base < a.n; base += kListThreads) {
    const int i = base + tid;
    int32_t q0 = 0, nq = 0, seq = 0;
    if (i < a.n) {
      q0 = a.token_offsets[i];
      const int32_t q1 = a.token_offsets[i + 1];
      seq = a.seq_lens[i];
      if (q0 < 0 || q1 < q0 || q1 > a.max_tokens) flags |= HS_FLAG_SEQLEN;
      else nq = q1 - q0;
      if (nq > 0 && (seq < 0 || seq > (int64_t)a.max_blocks * a.page_size)) {
        flags |= HS_FLAG_SEQLEN;
        seq = 0;
      }
    }
    const int64_t need = nq > 0 ? (seq + 63) / 64 : 0;
    int64_t sum;
    const int64_t before = blocks + cta_prefix<kListThreads>(need, &sum);
    blocks += sum;
    if (need > 0 && (before + need) * 64 > a.max_kv_tokens) {
      flags |= HS_FLAG_FULL;
      seq = 0;
    }
    const int64_t slot = listed + cta_prefix<kListThreads>(nq > 0, &sum);
    listed += sum;
    const int64_t tile0 = tiles + cta_prefix<kListThreads>((nq + per_tile - 1) / per_tile, &sum);
    tiles += sum;
    if (nq > 0) w.entries[slot] = {q0, nq, seq, i, (int32_t)tile0};
  }
  if (flags) atomicOr(err, flags);
  if (tid == 0) {
    *w.count = (int32_t)listed;
    *w.tiles = (int32_t)tiles;
  }
}

constexpr int kWarps = 8, BJ = 32, KS = DQK + 1;
constexpr size_t kSmem = (size_t)(BJ * KS + kWarps * DQK + BJ) * 4;

__global__ void __launch_bounds__(kWarps * 32) chunk_plain_kernel(const ChunkArgs a, const Work w, uint32_t* __restrict__ err) {
  extern __shared__ float smem[];
  float* k = smem;                                         // [BJ][KS]
  float* qs = smem + BJ * KS;                              // [kWarps][DQK]
  int* there = reinterpret_cast<int*>(qs + kWarps * DQK);  // [BJ]
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per_tile = MH / a.num_heads;
  const int count = *w.count, groups = MH / kWarps;
  for (int64_t u = blockIdx.x; u < (int64_t)*w.tiles * groups; u += gridDim.x) {
    const int tile = (int)(u / groups);
    int lo = 0, hi = count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (w.entries[mid].tile0 <= tile) lo = mid;
      else hi = mid - 1;
    }
    const Entry e = w.entries[lo];
    const int first = (tile - e.tile0) * per_tile, tokens = min(per_tile, e.nq - first);
    const int m = (int)(u % groups) * kWarps + warp;
    const bool live = m < tokens * a.num_heads;
    const int64_t row = ((int64_t)e.q0 + first) * a.num_heads + m;
    const int64_t end = (int64_t)e.seq - e.nq + first + tokens;  // past the last position that some query of the tile sees
    const int64_t mine = (int64_t)e.seq - e.nq + first + m / a.num_heads + 1;
    __syncthreads();
    if (live)
      for (int d = lane; d < DQK; d += 32) qs[warp * DQK + d] = __uint_as_float((uint32_t)a.q[row * DQK + d] << 16);
    float top = -INFINITY, sum = 0.f, o[DL / 32] = {};
    for (int64_t j0 = 0; j0 < end; j0 += BJ) {
      __syncthreads();
      for (int j = warp; j < BJ; j += kWarps) {
        const int64_t t = j0 + j;
        int64_t r = -1;
        if (t < end) {
          const int32_t page = a.block_tables[(int64_t)e.table * a.max_blocks + t / a.page_size];
          r = (int64_t)page * a.page_size + t % a.page_size;
          if (page < 0 || r >= a.pool_rows) {
            r = -1;
            if (lane == 0) atomicOr(err, HS_FLAG_DEVROW);
          }
        }
        if (lane == 0) there[j] = r >= 0;
        const uint8_t* src = a.pool + max(r, (int64_t)0) * kFp8Row;
        for (int d = lane; d < DQK; d += 32) {
          float v = 0.f;
          if (r < 0) {
          } else if (d < DL) {
            v = __half2float(__half(__nv_cvt_fp8_to_halfraw(src[d], __NV_E4M3))) *
                reinterpret_cast<const float*>(src + kFp8Scales)[d / kFp8Block];
          } else {
            v = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(src + kFp8RopeAt)[d - DL] << 16);
          }
          k[j * KS + d] = v;
        }
      }
      __syncthreads();
      if (live) {
        float s = 0.f;
        for (int d = 0; d < DQK; ++d) s += qs[warp * DQK + d] * k[lane * KS + d];
        const bool sees = j0 + lane < mine && there[lane];
        s = sees ? s * a.sm_scale : -INFINITY;
        float bm = s;
        for (int d = 16; d > 0; d >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, d));
        const float m_new = fmaxf(top, bm), ref = m_new == -INFINITY ? 0.f : m_new;
        const float keep = expf(top - ref), p = expf(s - ref);
        float z = p;
        for (int d = 16; d > 0; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
        top = m_new;
        sum = sum * keep + z;
        for (int i = 0; i < DL / 32; ++i) o[i] *= keep;
        for (int j = 0; j < BJ; ++j) {
          const float pj = __shfl_sync(0xffffffffu, p, j);
          if (pj == 0.f) continue;  // (a row that is not seen may hold a NaN)
          for (int i = 0; i < DL / 32; ++i) o[i] += pj * k[j * KS + 32 * i + lane];
        }
      }
    }
    if (live) {
      for (int i = 0; i < DL / 32; ++i) {
        const __nv_bfloat16 h = __float2bfloat16(sum == 0.f ? 0.f : o[i] / sum);
        a.o[row * DL + 32 * i + lane] = *reinterpret_cast<const uint16_t*>(&h);
      }
      if (lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : top + logf(sum);
    }
  }
}

}  // namespace

size_t chunk_workspace_bytes(int32_t n, int32_t num_heads, int32_t max_tokens, int64_t max_kv_tokens) {
  Work w;
  return work_of(&w, nullptr, n);
}

cudaError_t launch_chunk_mla(const ChunkArgs& a, void* workspace, uint32_t* err, cudaStream_t stream) {
  Work w;
  work_of(&w, workspace, a.n);
  cudaError_t e = cudaFuncSetAttribute(chunk_plain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e == cudaSuccess) e = launch(chunk_list_kernel, dim3(1), kListThreads, 0, stream, a, w, err);
  if (e == cudaSuccess) e = launch(chunk_plain_kernel, dim3(152 * 2), kWarps * 32, kSmem, stream, a, w, err);
  return e;
}

}  // namespace hs
