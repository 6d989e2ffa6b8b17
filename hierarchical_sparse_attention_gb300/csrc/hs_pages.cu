// Pages of a cache: tables of pages per request, reference counts, a stack of free pages, and the
// page copies of a fork and of a compaction, in every layer's pool.
//
// State (the caller's, on the device): resident_pages [num_requests, max_pages] (page or -1),
// page_refs [num_pages] (table entries that hold the page), free_pages [num_pages] with free_count
// (the stack's entries 0 .. free_count - 1, its top last). Every result is a function of the
// arguments and the state alone: grants go by prefix sums over the entries in their order, pages
// are pushed and packed in the order of their numbers, and the atomics only add, clear or set.
//
// What bounds the calls: extend, fork and free are chains of dependent loads and barriers of one CTA
// over little data, 4 to 10 us a kernel for 4 as for 200 entries (7.5 us extend, 7.2 and 3.8 us fork's two
// kernels, 7 to 10 us free's; from a host that launches them one by one its launches take as
// long); compact is bound by memory once it moves more than some hundred pages (58 us for 379 MB).
#include "hs_fp4.h"
#include "hs_tcgen05.cuh"

namespace hs {
namespace {

constexpr int kPlanThreads = 1024;  // the one-CTA plans
constexpr int kPageThreads = 256;
constexpr int kMaxRequests = HS_MAX_PAGE_REQUESTS;

// Workspace: a header, then per page a bit (freed by this call; zero between calls) and the
// compaction's lists, then per entry of a fork what the plan found and gave.
struct PageWork {
  uint32_t* ticket;    // CTAs of a fork's check or of a free that are done; zero between calls
  int32_t* moves;      // pages that the compaction moves
  int32_t* live;       // live pages
  uint32_t* freed;     // [ceil(num_pages / 32)]
  int32_t *src, *dst;  // [num_pages] the compaction's moves
  int32_t* rank;       // [num_pages] of a page past the live count: its move, or -1
  int32_t* used;       // [num_requests] entry i: its child's row holds a page
  int32_t* fresh;      // [num_requests] entry i: its copy's page; -1 none needed; -2 refused
};

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

PageWork work_of(const hs_page_pool& p) {
  uint8_t* at = static_cast<uint8_t*>(p.workspace);
  auto take = [&](size_t bytes) {
    uint8_t* r = at;
    at += up256(bytes);
    return r;
  };
  PageWork w;
  uint32_t* head = reinterpret_cast<uint32_t*>(take(256));
  w.ticket = head;
  w.moves = reinterpret_cast<int32_t*>(head + 1);
  w.live = reinterpret_cast<int32_t*>(head + 2);
  w.freed = reinterpret_cast<uint32_t*>(take(((size_t)p.num_pages + 31) / 32 * 4));
  w.src = reinterpret_cast<int32_t*>(take((size_t)p.num_pages * 4));
  w.dst = reinterpret_cast<int32_t*>(take((size_t)p.num_pages * 4));
  w.rank = reinterpret_cast<int32_t*>(take((size_t)p.num_pages * 4));
  w.used = reinterpret_cast<int32_t*>(take((size_t)p.num_requests * 4));
  w.fresh = reinterpret_cast<int32_t*>(take((size_t)p.num_requests * 4));
  return w;
}

// At the end of a kernel that changes tables or rows: hs_backup may be the next kernel of the
// stream, and it reads both before its wait (a programmatic dependent), so each thread makes what
// it wrote visible before it exits.
__device__ __forceinline__ void show_writes() { __threadfence(); }

// Exclusive prefix sum of v over the CTA's threads; *total gets the sum. Called by every thread; sums
// are 64-bit (entries x pages passes 32).
template <int kThreads>
__device__ int64_t block_prefix(int64_t v, int64_t* total) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int64_t s_warp[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // the last call's readers are done with s_warp
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t t = lane < kWarps ? s_warp[lane] : 0;
#pragma unroll
    for (int d = 1; d < kWarps; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t += y;
    }
    if (lane < kWarps) s_warp[lane] = t;
  }
  __syncthreads();
  *total = s_warp[kWarps - 1];
  return x - v + (warp ? s_warp[warp - 1] : 0);
}

// In every thread of a CTA that has written what the grid's last CTA reads: is this that CTA? (With
// __ldcg it sees what the others wrote. It leaves the ticket zero for the next call.)
__device__ bool last_cta(uint32_t* ticket) {
  __shared__ uint32_t s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(ticket, 1u) == gridDim.x * gridDim.y - 1;
    if (s_last) *ticket = 0;
    __threadfence();
  }
  __syncthreads();
  return s_last;
}

// The stack's height, kept inside its array whatever the state holds.
__device__ __forceinline__ int32_t stack_height(const hs_page_pool& p) {
  const int32_t c = *p.free_count;
  if (c < 0 || c > p.num_pages) {
    if (threadIdx.x == 0) atomicOr(p.error_flags, HS_FLAG_STATE);
    return c < 0 ? 0 : p.num_pages;
  }
  return c;
}
// The k-th page from the top of a stack of `height` (k < height), taken into use; -1 if the stack
// holds no page there.
__device__ __forceinline__ int32_t pop(const hs_page_pool& p, int32_t height, int64_t k) {
  const int32_t page = p.free_pages[height - 1 - k];
  if (page < 0 || page >= p.num_pages || atomicCAS(&p.page_refs[page], 0, 1) != 0) {
    atomicOr(p.error_flags, HS_FLAG_STATE);
    return -1;
  }
  return page;
}

__global__ void pages_init_kernel(const hs_page_pool p, const PageWork w) {
  pdl_wait();
  const int64_t step = (int64_t)gridDim.x * blockDim.x, t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  for (int64_t i = t; i < (int64_t)p.num_requests * p.max_pages; i += step) p.resident_pages[i] = -1;
  for (int64_t i = t; i < p.num_pages; i += step) {
    p.page_refs[i] = 0;
    p.free_pages[i] = p.num_pages - 1 - (int32_t)i;  // page 0 on top
  }
  for (int64_t i = t; i < ((int64_t)p.num_pages + 31) / 32; i += step) w.freed[i] = 0;
  if (t == 0) {
    *p.free_count = p.num_pages;
    *w.ticket = 0;
  }
  show_writes();
}

// One CTA. Entry i asks for the pages [ceil(old / page_size), ceil(new / page_size)) of its
// request; it gets all of them if the running sum of what the entries ask for is within the stack.
__global__ void __launch_bounds__(kPlanThreads)
    pages_extend_kernel(const hs_page_pool p, int32_t n, const int32_t* __restrict__ requests,
                        const int32_t* __restrict__ old_lens, const int32_t* __restrict__ new_lens,
                        int32_t* __restrict__ granted) {
  __shared__ uint32_t s_once[kMaxRequests / 32], s_twice[kMaxRequests / 32];
  __shared__ int64_t s_at[kPlanThreads];                         // the chunk's prefix sums
  __shared__ int32_t s_req[kPlanThreads], s_first[kPlanThreads];  // and where its pages go
  __shared__ uint8_t s_bad[kPlanThreads];
  const int tid = threadIdx.x;
  const int words = (p.num_requests + 31) / 32;
  for (int i = tid; i < words; i += kPlanThreads) s_once[i] = s_twice[i] = 0;
  pdl_wait();
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int32_t r = requests[i];
    if (r >= 0 && r < p.num_requests && (atomicOr(&s_once[r >> 5], 1u << (r & 31)) >> (r & 31) & 1u))
      atomicOr(&s_twice[r >> 5], 1u << (r & 31));
  }
  __syncthreads();
  const int32_t height = stack_height(p);
  const int64_t most = (int64_t)p.max_pages * p.page_size;
  int64_t asked = 0, taken = 0;  // by the entries so far
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + tid;
    int64_t need = 0, first = 0;
    int32_t r = -1;
    uint32_t flag = 0;
    if (i < n) {
      r = requests[i];
      const int64_t a = old_lens[i], b = new_lens[i];
      if (r < 0) {  // a padding entry
      } else if (r >= p.num_requests) {
        flag = HS_FLAG_TOKEN;
      } else if (s_twice[r >> 5] >> (r & 31) & 1u) {
        flag = HS_FLAG_DUP;
      } else if (a < 0 || b < a || b > most) {
        flag = HS_FLAG_SEQLEN;
      } else {
        first = (a + p.page_size - 1) / p.page_size;
        need = (b + p.page_size - 1) / p.page_size - first;
      }
    }
    // the pages asked for, spread over the threads: is any of them there already?
    int64_t sum;
    s_at[tid] = block_prefix<kPlanThreads>(need, &sum);
    s_req[tid] = r;
    s_first[tid] = (int32_t)first;
    s_bad[tid] = 0;
    __syncthreads();
    auto entry_of = [&](int64_t k) {  // the last entry whose prefix is <= k
      int lo = 0, hi = kPlanThreads - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_at[mid] <= k) lo = mid;
        else hi = mid - 1;
      }
      return lo;
    };
    for (int64_t k = tid; k < sum; k += kPlanThreads) {
      const int e = entry_of(k);
      if (p.resident_pages[(size_t)s_req[e] * p.max_pages + s_first[e] + (k - s_at[e])] != -1) s_bad[e] = 1;
    }
    __syncthreads();
    if (s_bad[tid]) {
      flag = HS_FLAG_STATE;
      need = 0;
    }
    const int64_t before = asked + block_prefix<kPlanThreads>(need, &sum);
    asked += sum;
    const bool got = need == 0 || before + need <= height;
    if (i < n) {
      if (flag) atomicOr(p.error_flags, flag);
      if (!got) atomicOr(p.error_flags, HS_FLAG_NOPAGE);
      if (granted) granted[i] = flag || !got ? -1 : (int32_t)need;
    }
    const int64_t mine = block_prefix<kPlanThreads>(got ? need : 0, &sum);
    s_at[tid] = mine;
    __syncthreads();
    for (int64_t k = tid; k < sum; k += kPlanThreads) {
      const int e = entry_of(k);
      p.resident_pages[(size_t)s_req[e] * p.max_pages + s_first[e] + (k - s_at[e])] = pop(p, height, taken + k);
    }
    taken += sum;
    __syncthreads();
  }
  if (tid == 0) *p.free_count = height - (int32_t)taken;
  show_writes();
}

// A CTA per entry looks whether the child's row holds a page; the last one done plans every
// entry: which are refused, and the page of each copy.
__global__ void __launch_bounds__(kPlanThreads)
    pages_fork_plan_kernel(const hs_page_pool p, const PageWork w, int32_t n, const int32_t* __restrict__ parents,
                           const int32_t* __restrict__ children, const int32_t* __restrict__ lens,
                           int32_t* __restrict__ granted) {
  __shared__ uint32_t s_once[kMaxRequests / 32], s_twice[kMaxRequests / 32], s_parent[kMaxRequests / 32];
  const int tid = threadIdx.x;
  pdl_wait();
  {
    const int32_t c = children[blockIdx.x];
    int held = 0;
    if (c >= 0 && c < p.num_requests)
      for (int i = tid; i < p.max_pages; i += kPlanThreads)
        held |= p.resident_pages[(size_t)c * p.max_pages + i] != -1;
    held = __syncthreads_or(held);
    if (tid == 0) w.used[blockIdx.x] = held;
    if (!last_cta(w.ticket)) return;
  }
  const int words = (p.num_requests + 31) / 32;
  for (int i = tid; i < words; i += kPlanThreads) s_once[i] = s_twice[i] = s_parent[i] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const int32_t c = children[i], q = parents[i];
    if (c < 0 || q < 0) continue;  // a padding entry
    if (c < p.num_requests && (atomicOr(&s_once[c >> 5], 1u << (c & 31)) >> (c & 31) & 1u))
      atomicOr(&s_twice[c >> 5], 1u << (c & 31));
    if (q < p.num_requests) atomicOr(&s_parent[q >> 5], 1u << (q & 31));
  }
  __syncthreads();
  const int32_t height = stack_height(p);
  const int64_t most = (int64_t)p.max_pages * p.page_size;
  int64_t asked = 0, taken = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + tid;
    int64_t need = 0;
    uint32_t flag = 0;
    bool padding = true;
    if (i < n) {
      const int32_t c = children[i], q = parents[i];
      const int64_t len = lens[i];
      padding = c < 0 || q < 0;
      if (padding) {
      } else if (c >= p.num_requests || q >= p.num_requests) {
        flag = HS_FLAG_TOKEN;
      } else if ((s_twice[c >> 5] | s_parent[c >> 5]) >> (c & 31) & 1u) {
        flag = HS_FLAG_DUP;
      } else if (len < 0 || len > most) {
        flag = HS_FLAG_SEQLEN;
      } else if (__ldcg(&w.used[i])) {
        flag = HS_FLAG_STATE;
      } else if (len % p.page_size) {
        const int32_t page = p.resident_pages[(size_t)q * p.max_pages + len / p.page_size];
        if (page >= p.num_pages || page < -1) flag = HS_FLAG_STATE;
        else need = page >= 0;
      }
    }
    int64_t sum;
    const int64_t before = asked + block_prefix<kPlanThreads>(need, &sum);
    asked += sum;
    const bool got = need == 0 || before + need <= height;
    const int64_t mine = block_prefix<kPlanThreads>(got ? need : 0, &sum);
    if (i < n) {
      if (flag) atomicOr(p.error_flags, flag);
      if (!got) atomicOr(p.error_flags, HS_FLAG_NOPAGE);
      const bool refused = flag || !got;
      w.fresh[i] = refused || padding ? -2 : need ? pop(p, height, taken + mine) : -1;
      if (granted) granted[i] = refused ? -1 : (int32_t)need;
    }
    taken += sum;
  }
  if (tid == 0) *p.free_count = height - (int32_t)taken;
}

// `bytes` from src to dst by the CTA, in pieces of `vec` bytes (both start on a multiple of it).
template <typename V>
__device__ __forceinline__ void copy_span_as(const uint8_t* src, uint8_t* dst, int64_t bytes) {
  const V* s = reinterpret_cast<const V*>(src);
  V* d = reinterpret_cast<V*>(dst);
  const int64_t n = bytes / (int64_t)sizeof(V);
  int64_t i = threadIdx.x;
  for (; i + 3 * kPageThreads < n; i += 4 * kPageThreads) {
    V x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = s[i + u * kPageThreads];
#pragma unroll
    for (int u = 0; u < 4; ++u) d[i + u * kPageThreads] = x[u];
  }
  for (; i < n; i += kPageThreads) d[i] = s[i];
}
__device__ __forceinline__ void copy_span(const uint8_t* src, uint8_t* dst, int64_t bytes, int vec) {
  if (vec == 16) copy_span_as<uint4>(src, dst, bytes);
  else if (vec == 4) copy_span_as<uint32_t>(src, dst, bytes);
  else copy_span_as<uint8_t>(src, dst, bytes);
}

// Per entry: blockIdx.y 0 gives the child its parent's whole pages and the copy's page, 1 + l
// copies the rows of the page that is not full in layer l.
__global__ void __launch_bounds__(kPageThreads)
    pages_fork_kernel(const PageArgs a, const PageWork w, const int32_t* __restrict__ parents,
                      const int32_t* __restrict__ children, const int32_t* __restrict__ lens) {
  pdl_wait();
  const hs_page_pool& p = a.p;
  const int i = blockIdx.x;
  const int32_t fresh = w.fresh[i];
  if (fresh == -2) return;
  const int32_t* src = p.resident_pages + (size_t)parents[i] * p.max_pages;
  const int32_t full = lens[i] / p.page_size, rest = lens[i] % p.page_size;
  if (blockIdx.y == 0) {
    int32_t* dst = p.resident_pages + (size_t)children[i] * p.max_pages;
    for (int k = threadIdx.x; k < full; k += kPageThreads) {
      int32_t page = src[k];
      if (page >= p.num_pages || page < -1) {
        atomicOr(p.error_flags, HS_FLAG_STATE);
        page = -1;
      }
      if (page >= 0) atomicAdd(&p.page_refs[page], 1);
      dst[k] = page;
    }
    if (threadIdx.x == 0 && fresh >= 0) dst[full] = fresh;
  } else if (fresh >= 0) {
    uint8_t* pool = static_cast<uint8_t*>(p.device_pools[blockIdx.y - 1]);
    const int64_t page = (int64_t)p.page_size * p.row_bytes;
    copy_span(pool + src[full] * page, pool + fresh * page, (int64_t)rest * p.row_bytes, a.vec);
  }
  show_writes();
}

// The marked pages onto the stack, the lowest on top, and the marks away, by one CTA of kPlanThreads: a
// word of marks to a thread for their ranks, then a bit to a thread.
__device__ void push_freed(const hs_page_pool& p, const PageWork& w) {
  __shared__ uint32_t s_bits[kPlanThreads];
  __shared__ int64_t s_rank[kPlanThreads];
  const int tid = threadIdx.x, lane = tid & 31;
  const int32_t height = stack_height(p);
  const int words = (int)(((int64_t)p.num_pages + 31) / 32);
  int64_t total = 0;
#pragma unroll 4
  for (int i = tid; i < words; i += kPlanThreads) total += __popc(__ldcg(w.freed + i));
  block_prefix<kPlanThreads>(total, &total);
  if (total == 0) return;
  int64_t rank = 0;  // marked pages below this chunk's
  for (int base = 0; base < words; base += kPlanThreads) {
    const uint32_t bits = base + tid < words ? __ldcg(w.freed + base + tid) : 0u;
    int64_t sum;
    s_rank[tid] = rank + block_prefix<kPlanThreads>(__popc(bits), &sum);
    s_bits[tid] = bits;
    rank += sum;
    if (bits) w.freed[base + tid] = 0;
    __syncthreads();
    for (int k = tid >> 5; sum > 0 && k < min(kPlanThreads, words - base); k += kPlanThreads / 32) {
      const uint32_t x = s_bits[k];
      if (!(x >> lane & 1u)) continue;
      const int64_t place = height + total - 1 - s_rank[k] - __popc(x & ((1u << lane) - 1));
      if (place < p.num_pages) p.free_pages[place] = 32 * (base + k) + lane;
      else atomicOr(p.error_flags, HS_FLAG_STATE);  // more pages than the pool has
    }
  }
  if (tid == 0) *p.free_count = (int32_t)min((int64_t)p.num_pages, height + total);
}

// Every entry of the ranges: out of the table, its page's count down by one; a page that nobody
// holds any more is marked. An entry is taken out by one thread however often the call names it. The
// last CTA puts the marked pages onto the stack.
__global__ void __launch_bounds__(kPlanThreads)
    pages_free_kernel(const hs_page_pool p, const PageWork w, const int32_t* __restrict__ requests,
                      const int32_t* __restrict__ first_pages, const int32_t* __restrict__ end_pages) {
  pdl_wait();
  const int i = blockIdx.x;
  const int32_t r = requests[i];
  if (r >= p.num_requests && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.error_flags, HS_FLAG_TOKEN);
  if (r >= 0 && r < p.num_requests) {
    const int32_t lo = first_pages ? max(first_pages[i], 0) : 0;
    const int32_t hi = end_pages ? min(end_pages[i], p.max_pages) : p.max_pages;
    int32_t* row = p.resident_pages + (size_t)r * p.max_pages;
    for (int64_t k = lo + (int64_t)blockIdx.y * kPlanThreads + threadIdx.x; k < hi; k += (int64_t)gridDim.y * kPlanThreads) {
      if (row[k] == -1) continue;
      const int32_t page = atomicExch(&row[k], -1);
      if (page == -1) continue;
      if (page < 0 || page >= p.num_pages) {
        atomicOr(p.error_flags, HS_FLAG_STATE);
        continue;
      }
      const int32_t held = atomicSub(&p.page_refs[page], 1);
      if (held == 1) {
        atomicOr(&w.freed[page >> 5], 1u << (page & 31));
      } else if (held <= 0) {  // the count did not cover this entry
        atomicAdd(&p.page_refs[page], 1);
        atomicOr(p.error_flags, HS_FLAG_STATE);
      }
    }
  }
  show_writes();
  if (last_cta(w.ticket)) push_freed(p, w);
  show_writes();
}

// One CTA, a strip of pages per warp: the live pages are counted, those past the live count get
// the free pages among the first ones, both in the order of their numbers.
__global__ void __launch_bounds__(kPlanThreads) pages_compact_plan_kernel(const hs_page_pool p, const PageWork w) {
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t strip = ((int64_t)p.num_pages + kPlanThreads - 1) / kPlanThreads * 32;
  const int64_t lo = min(warp * strip, (int64_t)p.num_pages), hi = min(lo + strip, (int64_t)p.num_pages);
  const uint32_t below = (1u << lane) - 1;
  int64_t count = 0;
#pragma unroll 8  // (the loads of a batch go out together)
  for (int64_t b = lo; b < hi; b += 32) count += __popc(__ballot_sync(~0u, b + lane < hi && p.page_refs[b + lane] > 0));
  int64_t live;
  int64_t before = block_prefix<kPlanThreads>(lane == 0 ? count : 0, &live);  // live pages below the strip
  before = __shfl_sync(~0u, before, 0);
  // live pages among the first `live`: the rest of those are holes, as many as there are pages to move
  count = 0;
#pragma unroll 8
  for (int64_t b = lo; b < min(hi, live); b += 32)
    count += __popc(__ballot_sync(~0u, b + lane < min(hi, live) && p.page_refs[b + lane] > 0));
  int64_t kept;
  block_prefix<kPlanThreads>(lane == 0 ? count : 0, &kept);
  for (int64_t b = lo; b < hi; b += 32) {
    const int64_t page = b + lane;
    const bool in = page < hi, used = in && p.page_refs[page] > 0;
    const uint32_t m = __ballot_sync(~0u, used);
    const int64_t k = before + __popc(m & below);  // live pages below this one
    if (in && page < live && !used) w.dst[page - k] = (int32_t)page;
    if (in && page >= live) {
      w.rank[page] = used ? (int32_t)(k - kept) : -1;
      if (used) w.src[k - kept] = (int32_t)page;
    }
    before += __popc(m);
  }
  if (threadIdx.x == 0) {
    *w.moves = (int32_t)(live - kept);
    *w.live = (int32_t)live;
  }
}

// Bytes of a page that are copied at a time, and the spans of a CTA's ring, two CTAs to an SM: 78 to 80 us for a
// step that moves 379 MB (read and written) of 26-KB pages. Beside 77: spans of 16 KB and rings of 6 79 us, of 8
// and 12 83, one CTA with a ring of 12 to an SM 83, 256 threads that load and store 64 bytes each in
// turn 96.
constexpr int kSpan = 32768;
constexpr int kRing = 3;

// The copies of a compaction: span k of all of them.
struct Span {
  const uint8_t* src;
  uint8_t* dst;
  int bytes;
};
__device__ __forceinline__ Span span_of(const hs_page_pool& p, const PageWork& w, int64_t k) {
  const int64_t page = (int64_t)p.page_size * p.row_bytes;
  const int spans = (int)((page + kSpan - 1) / kSpan);
  const int64_t at = k % spans * kSpan, rest = k / spans, m = rest / p.num_layers;
  uint8_t* pool = static_cast<uint8_t*>(p.device_pools[rest % p.num_layers]);
  return {pool + w.src[m] * page + at, pool + w.dst[m] * page + at, (int)min((int64_t)kSpan, page - at)};
}

// A warp's share of them through a ring in shared memory, by bulk copies in and out: nothing but
// their issue costs instructions, and two of a ring's spans are always on their way in.
__device__ __forceinline__ void copy_through_ring(const hs_page_pool& p, const PageWork& w, uint8_t* ring, uint64_t* full,
                                                  volatile int* abort, int64_t tasks, int lane) {
  if (blockIdx.x >= tasks) return;
  const int64_t n = (tasks - blockIdx.x + gridDim.x - 1) / gridDim.x;
  int64_t loaded = 0;
  Span ahead{};                    // lane l: span 32 (loaded / 32) + l of this CTA's
  uint8_t* dst = nullptr;          // lane l: where the span in slot l goes
  int bytes = 0;
  auto load = [&](int64_t upto) {  // the loads of the spans before `upto`
    for (; loaded < n && loaded < upto; ++loaded) {
      const int from = (int)(loaded & 31), slot = (int)(loaded % kRing);
      if (from == 0 && loaded + lane < n) ahead = span_of(p, w, blockIdx.x + (loaded + lane) * gridDim.x);
      const uint64_t s = __shfl_sync(~0u, (uint64_t)ahead.src, from), d = __shfl_sync(~0u, (uint64_t)ahead.dst, from);
      const int b = __shfl_sync(~0u, ahead.bytes, from);
      if (lane == slot) {
        dst = (uint8_t*)d;
        bytes = b;
      }
      if (lane == 0) {
        tc::bar_arrive_tx(&full[slot], (uint32_t)b);
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         tc::smem_u32(ring + slot * kSpan)),
                     "l"(s), "r"(b), "r"(tc::smem_u32(&full[slot]))
                     : "memory");
      }
    }
  };
  load(kRing);
  for (int64_t i = 0; i < n; ++i) {
    const int slot = (int)(i % kRing);
    const bool here = __all_sync(~0u, tc::pipe_wait(&full[slot], 1, (int)(i / kRing & 1), abort));
    const uint64_t d = __shfl_sync(~0u, (uint64_t)dst, slot);
    const int b = __shfl_sync(~0u, bytes, slot);
    if (!here) break;
    if (lane == 0) {
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(d), "r"(tc::smem_u32(ring + slot * kSpan)), "r"(b)
                   : "memory");
      // the span before has been read out of its slot, which takes the next one
      asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 1;" ::: "memory");
    }
    __syncwarp();
    load(i + kRing);  // (of slot (i - 1) % kRing, at most)
  }
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  if (*abort) {  // never met: the waits are bounded so that a kernel always ends
    if (lane == 0) atomicOr(p.error_flags, HS_FLAG_TIMEOUT);
    __syncwarp();
    *abort = 0;
    __syncwarp();
    for (int64_t i = max((int64_t)0, loaded - kRing); i < loaded; ++i)  // copies in flight get one more bound
      tc::pipe_wait(&full[i % kRing], 1, (int)(i / kRing & 1), abort);
  }
  __syncwarp();
}

// Pages move, their counts with them; every table entry that names a moved page names its new
// one; the stack holds the pages past the live ones, the lowest on top. kBulk: pools and rows on
// 16-byte boundaries; the first warp has the copies, the others the tables.
template <bool kBulk>
__global__ void __launch_bounds__(kPageThreads) pages_compact_kernel(const PageArgs a, const PageWork w) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(8) uint64_t full[kRing];
  __shared__ int s_abort;
  if (kBulk && threadIdx.x == 0) {
    for (int k = 0; k < kRing; ++k) tc::bar_init(&full[k], 1);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  const hs_page_pool& p = a.p;
  const int32_t moves = *w.moves, live = *w.live;
  const int64_t page = (int64_t)p.page_size * p.row_bytes;
  const int64_t tasks = (page + kSpan - 1) / kSpan * moves * p.num_layers;
  int first = 0;  // the first thread of those that have the tables
  if (kBulk) {
    first = 32;
    if (threadIdx.x < 32) {
      __syncwarp();
      copy_through_ring(p, w, ring, full, &s_abort, tasks, threadIdx.x);
      show_writes();
      return;
    }
  } else {
    for (int64_t k = blockIdx.x; k < tasks; k += gridDim.x) {
      const Span s = span_of(p, w, k);
      copy_span(s.src, s.dst, s.bytes, a.vec);
    }
  }
  const int64_t step = (int64_t)gridDim.x * (kPageThreads - first), t = (int64_t)blockIdx.x * (kPageThreads - first) + threadIdx.x - first;
  for (int64_t k = t; k < moves; k += step) {
    p.page_refs[w.dst[k]] = p.page_refs[w.src[k]];
    p.page_refs[w.src[k]] = 0;
  }
  for (int64_t k = t; k < (int64_t)p.num_requests * p.max_pages; k += step) {
    const int32_t old = p.resident_pages[k];
    if (old < live) continue;
    const int32_t m = old < p.num_pages ? w.rank[old] : -1;
    if (m >= 0) p.resident_pages[k] = w.dst[m];
    else atomicOr(p.error_flags, HS_FLAG_STATE);  // a page that nobody counted
  }
  for (int64_t k = t; k < p.num_pages - live; k += step) p.free_pages[k] = p.num_pages - 1 - (int32_t)k;
  if (t == 0) *p.free_count = p.num_pages - live;
  show_writes();
}

cudaError_t sm_count(int* n) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
}

}  // namespace

size_t pages_workspace_bytes(int32_t num_requests, int32_t num_pages) {
  return 256 + up256(((size_t)num_pages + 31) / 32 * 4) + 3 * up256((size_t)num_pages * 4) +
         2 * up256((size_t)num_requests * 4);
}

cudaError_t launch_pages_init(const PageArgs& a, cudaStream_t stream) {
  const int64_t n = (int64_t)a.p.num_requests * a.p.max_pages;
  const int64_t most = n > a.p.num_pages ? n : a.p.num_pages;
  const unsigned grid = (unsigned)((most + kPageThreads - 1) / kPageThreads < 1216 ? (most + kPageThreads - 1) / kPageThreads : 1216);
  return launch(pages_init_kernel, dim3(grid), kPageThreads, 0, stream, a.p, work_of(a.p));
}

cudaError_t launch_pages_extend(const PageArgs& a, int32_t n, const int32_t* requests, const int32_t* old_lens,
                                const int32_t* new_lens, int32_t* granted, cudaStream_t stream) {
  return launch(pages_extend_kernel, dim3(1), kPlanThreads, 0, stream, a.p, n, requests, old_lens, new_lens, granted);
}

cudaError_t launch_pages_fork(const PageArgs& a, int32_t n, const int32_t* parents, const int32_t* children,
                              const int32_t* lens, int32_t* granted, cudaStream_t stream) {
  const PageWork w = work_of(a.p);
  const cudaError_t e = launch(pages_fork_plan_kernel, dim3((unsigned)n), kPlanThreads, 0, stream, a.p, w, n, parents,
                               children, lens, granted);
  if (e != cudaSuccess) return e;
  return launch(pages_fork_kernel, dim3((unsigned)n, 1u + (unsigned)a.p.num_layers), kPageThreads, 0, stream, a, w,
                parents, children, lens);
}

cudaError_t launch_pages_free(const PageArgs& a, int32_t n, const int32_t* requests, const int32_t* first_pages,
                              const int32_t* end_pages, cudaStream_t stream) {
  const PageWork w = work_of(a.p);
  const int chunks = (a.p.max_pages + kPlanThreads - 1) / kPlanThreads;
  return launch(pages_free_kernel, dim3((unsigned)n, (unsigned)(chunks < 64 ? chunks : 64)), kPlanThreads, 0, stream, a.p, w,
                requests, first_pages, end_pages);
}

cudaError_t launch_pages_compact(const PageArgs& a, cudaStream_t stream) {
  const PageWork w = work_of(a.p);
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  if ((e = launch(pages_compact_plan_kernel, dim3(1), kPlanThreads, 0, stream, a.p, w)) != cudaSuccess) return e;
  if (a.vec < 16) return launch(pages_compact_kernel<false>, dim3(4u * (unsigned)sms), kPageThreads, 0, stream, a, w);
  e = cudaFuncSetAttribute(pages_compact_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing * kSpan);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return e;
  }
  return launch(pages_compact_kernel<true>, dim3(2u * (unsigned)sms), kPageThreads, kRing * kSpan, stream, a, w);
}

}  // namespace hs
