// Attention of a step's new tokens over the fp8 pages of their sequences, causal, on the 5th-generation tensor cores
// (tcgen05, accumulators in tensor memory).
//
// Per query head of the token at position p, over the tokens t <= p of its sequence:
//   s_t = sm_scale (q[:512] . latent_t + q[512:] . rope_t),  o = softmax(s) . latent,  lse = log sum_t exp s_t
//
// Three kernels (four for more than 1,024 entries):
//   - chunk_rows: the list of the entries with queries and the work dealt out evenly; and every sequence's rows once, from their pages, as f16 in blocks of 64 rows laid out as the tensor cores
//     read them, so that the attention brings a block in with one bulk copy and no arithmetic;
//   - chunk_mla: tiles of 128 query heads (all heads of as many tokens of an entry as fit) over their blocks;
//   - chunk_merge: joins the parts of tiles that were cut.
//
// chunk_mla. The work of a call is one line: the entries' tiles, one after the other, each as long as its blocks. It is cut
// into as many equal pieces as there are pairs of CTAs, so that every pair ends at the same time whatever the lengths are;
// a piece's first and last tile may be parts, whose results (in 32 bits) chunk_merge joins. A pair, on two SMs, because Q
// (288 columns), S and O (512) do not fit one tensor memory, nor K, V, Q and P one shared memory, takes a tile's blocks of
// 64 rows in turn:
//   - the S-CTA (even rank) holds Q in tensor memory and computes S = Q . K^T of each block into one of three buffers; its
//     three softmax warpgroups (a block each in turn, a query head per thread) run the online softmax and write P as f16
//     into the O-CTA's shared memory;
//   - the O-CTA holds O (128 x 512 in 32 bits, all of its tensor memory) and adds P . V; its corrector rescales O in the
//     rare blocks that raise a head's reference maximum.
// The roles hand blocks over through mbarriers with bounded waits, and run on from tile to tile: Q comes through the ring of
// K's slots (a slot holds a block of 64 rows of 576 values, or half of Q), V through a ring of half blocks.
//
// What bounds it (256 tokens x 128 heads behind 48,000: 1.95 ms, 1,760 TFLOP/s, 0.91 of cuBLAS's bf16 burst and above what it
// sustains): a block takes a pair 0.77 us, 1,400 clocks at the 1.8 GHz that the power limit leaves, of which the S-CTA's 36 MMAs are
// 1,150 and the O-CTA's 8 are 1,024. Then a tile's change, 3.7 us (the last S 0.9, Q's copy and its way to tensor memory 2.4,
// K's ring, which Q has taken, full again), a third of a first chunk's time. What each part brought
// (256 tokens behind 48,000, or a first chunk of 2,048):
//   P stored 512 bytes a warp instead of 16 bytes a line (see pdesc)       2,712 -> 2,025 us
//   S with an issuer per buffer: a commit holds its thread up, 500 clocks with a block's MMAs queued before it, and the waits
//   for the next block 300 more, in which another thread's MMAs keep the tensor core busy    2,744 -> 2,712
//   P . V with an issuer per half of O, K's slots in two parts, four P buffers, blocks in order    2,051 -> 1,966
//   Q brought by the issuing warps while the softmax is at the tile before    650 -> 531
//   the read-out by eight warps, halves of O handed back as they are read, the corrector at the next tile    531 -> 485
//   a block's MMAs issued in one go, a tile's own cost of six blocks    471 -> 444
// Tried, not kept: rows fetched into L2 six blocks ahead (2,470 us); a look at a barrier and a branch between a block's MMAs
// (2,640: their operands leave the uniform registers); slots in three parts (no change); rows of short batches brought by
// the pair itself, through the O-CTA's reading-out warps (a decode step 68 -> 142 us; loads kept four tasks ahead: 180).
//
// Precision. Latents (e4m3 x scale) and RoPE values go through f16: exact where the scale is a power of two, else off by 2^-11
// of themselves, and by 2^-25 where they are below 2^-14. Q goes through f16, over a power of two where its head's
// largest value is below 1 or above 65504, which goes into its scores' scale: off by 2^-25 of the head's largest. P, whose
// reference weighs 2^7, is rounded to f16: by up to 2^-11 of a weight, and by 2^-32 of the largest weight where it is below
// 2^-21 of that; its sum takes weights unrounded, so lse does not see it. Scores, maxima, sums and O are in 32 bits.
//
// NaN, infinities and values that f16 does not hold. A row that a query does not see gets P = 0, and 0 x NaN must not reach O:
// such values are zeros in the blocks, and a mark for their row makes its score NaN for the queries that see it, and so
// their outputs, and only theirs.
#include "hs_chunk.h"
#include "hs_tcgen05.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>
#include <climits>
#include <type_traits>

namespace hs {

using namespace tc;

namespace {

constexpr int T = 512;   // threads per CTA: 16 warps
constexpr int MH = 128;  // MMA M: query heads of a tile (what is there of the next tokens fills it up)
constexpr int BJ = 64;   // rows per block
constexpr int DQK = kFp8Dims, DL = kFp8Latent;
constexpr int QATOMS = DQK / 64, ATOMS = DL / 64;  // swizzle atoms of 64 values in a block of K and of V
constexpr int NS = 3;    // S buffers and softmax warpgroups: a block each in turn
constexpr int NP = 4;    // P buffers
constexpr int NK = 3, NV = 4;  // slots of the S-CTA's ring (a block, or half of Q) and of the O-CTA's (half of V's block)
// Barriers of V's slots: two to a slot in turn, as a use of an odd slot count is the other half's use before, whose issuer
// waits on the other barrier: so each issuer waits on every phase of its own.
constexpr int NVF = 2 * NV;
constexpr uint32_t TMEM_COLS = 512, Q_COL = 0, S_COL = 288;
static_assert(S_COL + NS * BJ <= TMEM_COLS, "Q and the S buffers fit tensor memory");
// S-CTA warps: 0-11 softmax, 12-14 issuers, 15 copies, and 12-15 bring Q; O-CTA: 0-3 corrector, 4-11 read out, 12 and 13
// issuers, 15 copies.
// S has an issuer per buffer, P . V one per half of O.
constexpr int ISSUER = 12, COPIER = 15, OUT = 4, NOUT = 2;  // NOUT warps read out a quarter of the heads

constexpr uint32_t ATOM = BJ * 128, BLOCK = QATOMS * ATOM, HALF_V = ATOMS / 2 * ATOM;
constexpr uint32_t S_RING = 0;
// A slot of K is filled and handed back in two parts (values 0 - 319, and the rest), so that the next block's copies start while
// the tensor core is at the second: three slots cover a copy's way (860 clocks from a commit to the copy's start, 1,680 to
// its end) and a block's MMAs (1,150) only so.
constexpr uint32_t PART = 5 * ATOM;
constexpr uint32_t S_REF = NK * BLOCK;             // the reference maxima, handed from block to block
constexpr uint32_t S_UP = S_REF + MH * 4;          // what a head's Q was divided by, of the last NQ tiles
// A softmax warpgroup that is at a block may find S computed up to five blocks on (its next one and the two after that), and
// so, of tiles of one block each, Q set six tiles on: it looks at those tiles' barriers later, each before its
// next use.
constexpr int NQ = 8;
constexpr uint32_t S_END = S_UP + NQ * MH * 4;
constexpr uint32_t O_RING = 0;
constexpr uint32_t O_P = NV * HALF_V;
constexpr uint32_t P_BUF = MH * BJ * 2, P_BYTES = P_BUF + MH * 4;  // P and the rescale factors of a block
constexpr uint32_t FIN_WG = 2 * MH * 4;            // a softmax warpgroup's sums and references of a tile
constexpr uint32_t O_ALPHA = O_P + NP * P_BUF;
constexpr int NF = NP + 1;  // tiles whose totals are kept: P's buffers let the S-CTA be four tiles ahead, of one block each
constexpr uint32_t FIN = NS * FIN_WG + MH * 4;     // of a tile: the warpgroups', and what a unit of a score is
constexpr uint32_t O_FIN = O_ALPHA + NP * MH * 4;
constexpr uint32_t O_END = O_FIN + NF * FIN;
constexpr uint32_t SMEM_BYTES = S_END > O_END ? S_END : O_END;
constexpr uint32_t STATIC_BYTES = 1024;  // barriers and flags, one block of a tile's alignment
static_assert(STATIC_BYTES + SMEM_BYTES <= 227 * 1024, "shared memory of a CTA");
static_assert(BLOCK % 1024 == 0 && HALF_V % 1024 == 0 && O_P % 1024 == 0, "the swizzle's alignment");
// P of a score that equals its reference is 2^7, and a reference stays until it is passed by 2^8.9, so that
// P < 2^15.91 = 61,500 in f16, which then keeps a weight to 2^-11 of itself down to 2^-21 of the reference's.
constexpr float kRefLog2 = 7.f, kRescaleLog2 = 8.9f;
constexpr uint32_t kIdescQK = idesc(BJ, MH, false);
constexpr uint32_t kIdescPV = idesc(256, MH, true);

// How the work is dealt out, in blocks: what a tile takes besides its blocks, and the least part of a tile.
constexpr int kTileCost = 6, kLeastPart = 4;
constexpr int kPairs = 76;  // of CTAs, at most
constexpr int kListThreads = 512;
constexpr int kRowsThreads = 192, HB = BJ / 2;  // chunk_rows: a CTA has half a block at a time
constexpr int kFoldEntries = 1024;  // up to so many entries each CTA of chunk_rows goes over them itself
static_assert(kPairs < kRowsThreads && kPairs < kListThreads, "a thread per pair");

// An entry with queries.
struct __align__(16) Entry {
  int32_t q0, nq, seq;  // first flat token, queries, tokens (0: they see nothing)
  int32_t table;        // its number: the block table's row
  int64_t cost;         // of the entries before it, in tokens (64 to a block)
  int32_t block;        // its first block of rows in the workspace
  int32_t none;
};
static_assert(sizeof(Entry) == 32, "two loads");
struct Pos {
  int32_t ent, tile, blk, none;
};
struct Work {
  int32_t* count;   // entries listed
  int32_t* blocks;  // blocks of their sequences
  Pos* starts;      // [kPairs + 1] where a pair's work begins
  Entry* entries;   // [n]
  uint4* state;     // [blocks] two words of rows that exist, two of rows with a value that f16 does not hold
  uint8_t* kv;      // [blocks] x BLOCK bytes
  float* part_lse;  // [2 kPairs, MH] of a pair's first tile, where that began before, and of one that goes on after it
  float* part_o;    // [2 kPairs, MH, DL]
};
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
size_t work_of(Work* w, void* workspace, int32_t n, int64_t max_kv_tokens) {
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    uint8_t* r = workspace == nullptr ? nullptr : static_cast<uint8_t*>(workspace) + at;
    at += up256(bytes);
    return r;
  };
  const size_t blocks = (size_t)(max_kv_tokens / BJ);
  w->count = reinterpret_cast<int32_t*>(take(8));
  w->blocks = w->count + 1;
  w->starts = reinterpret_cast<Pos*>(take((kPairs + 1) * sizeof(Pos)));
  w->entries = reinterpret_cast<Entry*>(take((size_t)n * sizeof(Entry)));
  w->state = reinterpret_cast<uint4*>(take(blocks * sizeof(uint4)));
  w->kv = take(blocks * BLOCK);
  w->part_lse = reinterpret_cast<float*>(take((size_t)2 * kPairs * MH * 4));
  w->part_o = reinterpret_cast<float*>(take((size_t)2 * kPairs * MH * DL * 4));
  return at;
}

// P's descriptor: no swizzle, chunk c (8 values) of row m at 16 (128 c + m), so that a warp's stores of a chunk are 512
// consecutive bytes. (Between two SMs' shared memories 16 KB of P take 860 clocks so, 1,600 to 2,000 where each lane's 16
// bytes go to a line of their own, as rows of 128 bytes want it, and a block's MMAs 1,150.)
__device__ __forceinline__ uint64_t pdesc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)((MH * 16) >> 4) << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}

// 64 accumulator columns of this thread's row.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[BJ]) {
#pragma unroll
  for (int h = 0; h < BJ; h += 16) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v + h);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr + h));
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- the list

// What tiles 0 .. t - 1 of an entry cost, in tokens: tile i reads the `before` tokens before the entry's queries and
// (i + 1) per_tile of these (a little more than it does where the last tile is not full, or before is negative).
__device__ __forceinline__ int64_t cost_of(int64_t before, int per_tile, int64_t t) {
  return (max(before, (int64_t)0) + kTileCost * BJ) * t + per_tile * (t * (t + 1) / 2);
}
__device__ __forceinline__ int blocks_of(int64_t tokens) { return tokens > 0 ? (int)((tokens + BJ - 1) / BJ) : 0; }

// What the call says of entry i: its first flat token, queries, and tokens.
__device__ __forceinline__ uint32_t look_up(const ChunkArgs& a, int i, int32_t& q0, int32_t& nq, int32_t& seq) {
  nq = seq = q0 = 0;
  if (i >= a.n) return 0;
  q0 = a.token_offsets[i];
  const int32_t q1 = a.token_offsets[i + 1];
  seq = a.seq_lens[i];
  if (q0 < 0 || q1 < q0 || q1 > a.max_tokens) return HS_FLAG_SEQLEN;
  nq = q1 - q0;
  if (nq == 0 || (seq >= 0 && seq <= (int64_t)a.max_blocks * a.page_size)) return 0;
  seq = 0;
  return HS_FLAG_SEQLEN;
}

// The list, by a CTA of kThreads threads.
template <int kThreads>
__device__ __forceinline__ void list_entries(const ChunkArgs& a, const Work& w, int pairs, uint32_t* __restrict__ err) {
  const int tid = threadIdx.x, per_tile = MH / a.num_heads;
  __shared__ Entry s_entry[kThreads];  // the first ones
  int64_t blocks = 0, listed = 0, cost = 0;
  uint32_t flags = 0;
  for (int base = 0; base < a.n; base += kThreads) {
    const int i = base + tid;
    int32_t q0, nq, seq;
    flags |= look_up(a, i, q0, nq, seq);
    // blocks asked for, and entries, in one sum: up to 2^41 and 2^10
    constexpr int kBits = 20;
    static_assert(kThreads < (1 << kBits), "the entries of a run");
    const int64_t need = nq > 0 ? blocks_of(seq) : 0;
    // (an entry that does not fit is given its cost all the same: which ones fit is not known yet)
    int64_t at[2] = {need << kBits | (nq > 0), nq > 0 ? cost_of((int64_t)seq - nq, per_tile, (nq + per_tile - 1) / per_tile) : 0};
    int64_t sum[2];
    cta_prefix<kThreads>(at, sum);
    const int64_t before = blocks + (at[0] >> kBits), slot = listed + (at[0] & ((1 << kBits) - 1));
    if (need > 0 && (before + need) * BJ > a.max_kv_tokens) {
      flags |= HS_FLAG_FULL;
      seq = 0;
    }
    if (nq > 0) {
      const Entry e = {q0, nq, seq, i, cost + at[1], (int32_t)min(before, a.max_kv_tokens / BJ), 0};
      w.entries[slot] = e;
      if (slot < kThreads) s_entry[slot] = e;
    }
    blocks += sum[0] >> kBits;
    listed += sum[0] & ((1 << kBits) - 1);
    cost += sum[1];
  }
  if (flags) atomicOr(err, flags);
  if (tid == 0) {
    *w.count = (int32_t)listed;
    *w.blocks = (int32_t)min(blocks, a.max_kv_tokens / BJ);
  }
  __syncthreads();  // (the entries, which any thread reads now)
  if (tid > pairs) return;
  const auto entry = [&](int i) -> Entry { return i < kThreads ? s_entry[i] : w.entries[i]; };
  const int used = (int)max(min((int64_t)pairs, cost / (kLeastPart * BJ)), (int64_t)1);  // pairs that get anything
  Pos at = {(int32_t)listed, 0, 0, 0};
  if (tid < used && listed > 0) {
    const int64_t x = cost / used * tid + cost % used * tid / used;
    int lo = 0, hi = (int)listed - 1;  // the last entry that begins at or before x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (entry(mid).cost <= x) lo = mid;
      else hi = mid - 1;
    }
    const Entry e = entry(lo);
    const int tiles = (e.nq + per_tile - 1) / per_tile;
    const int64_t before = (int64_t)e.seq - e.nq, y = x - e.cost;
    // the last tile that begins at or before y: the root of the cost, a quadratic, put right by what rounding took
    const float b = (float)(max(before, (int64_t)0) + kTileCost * BJ) + 0.5f * per_tile;
    int64_t t = (int64_t)(2.f * (float)y / (b + sqrtf(b * b + 2.f * per_tile * (float)y)));
    t = min(max(t, (int64_t)0), (int64_t)tiles - 1);
    while (t > 0 && cost_of(before, per_tile, t) > y) --t;
    while (t < tiles - 1 && cost_of(before, per_tile, t + 1) <= y) ++t;
    const int all = blocks_of(before + min((t + 1) * per_tile, (int64_t)e.nq));
    int64_t blk = max((y - cost_of(before, per_tile, t)) / BJ - kTileCost, (int64_t)0);
    if (blk < kLeastPart) blk = 0;
    if (blk > 0 && all - blk < kLeastPart) blk = 0, ++t;
    if (tid == 0) t = blk = 0;
    at.ent = lo;
    at.tile = (int)t;
    at.blk = (int)blk;
    if (t == tiles) at = {lo + 1, 0, 0, 0};
  }
  w.starts[tid] = at;
}

// (a call of many entries: otherwise a CTA of chunk_rows does it)
__global__ void __launch_bounds__(kListThreads) chunk_list_kernel(const ChunkArgs a, const Work w, int pairs, uint32_t* __restrict__ err) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  pdl_wait();
  list_entries<kListThreads>(a, w, pairs, err);
}

// ---------------------------------------------------------------- the rows

// Pairs of f16 values: those that are not finite become zeros.
__device__ __forceinline__ uint32_t without_bad(uint32_t x) {
  if ((x & 0x7C00u) == 0x7C00u) x &= 0xFFFF0000u;
  if ((x & 0x7C000000u) == 0x7C000000u) x &= 0x0000FFFFu;
  return x;
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// A CTA takes a run of half blocks (32 rows), one after the other. A thread has 32 values of a row, a warp eight rows of 128 (or 16
// of 64) at a time. Within 32 values, chunk j of four takes pair j of each, the order of columns that the read-out of O
// wants (and Q's values have); the place of chunk c of row x of a line's eight is c ^ x, so that a thread's four chunks are
// half a line, two whole sectors. A scale that f16 holds (a power of two, say) multiplies in f16, which rounds the exact
// product; others in 32 bits.
// Bound by memory: 656 bytes read and 1,152 written a row. (Blocks of 64 rows through shared memory and a bulk copy each
// were bound by their way, at 4.2 TB/s.)
// kFold: the entries are not listed yet. The last CTA lists them, and the others find the run's in the call's arrays: the same few
// loads as from a list, and a launch less (4 us of a call).
template <bool kFold>
__global__ void __launch_bounds__(kRowsThreads, 5) chunk_rows_kernel(const ChunkArgs a, const Work w, int pairs, uint32_t* __restrict__ err) {
  __shared__ int s_entry;
  __shared__ int32_t s_first[kFold ? kFoldEntries : 1], s_seq[kFold ? kFoldEntries : 1];  // first blocks, tokens
  __shared__ int32_t s_row[2][HB];
  __shared__ uint32_t s_there[2], s_bad[2];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (kFold && blockIdx.x == gridDim.x - 1) {
    list_entries<kRowsThreads>(a, w, pairs, err);
    return;
  }
  const int ctas = gridDim.x - (kFold ? 1 : 0);
  int count, total;  // entries (kFold: of the call), half blocks (below 2^26)
  if (kFold) {
    int64_t blocks = 0;
    for (int base = 0; base < a.n; base += kRowsThreads) {
      const int i = base + tid;
      int32_t q0, nq, seq;
      look_up(a, i, q0, nq, seq);
      const int64_t need = nq > 0 ? blocks_of(seq) : 0;
      int64_t before[1] = {need}, sum[1];
      cta_prefix<kRowsThreads>(before, sum);
      before[0] += blocks;
      blocks += sum[0];
      if (i < a.n) {
        s_first[i] = (int32_t)min(before[0], a.max_kv_tokens / BJ);
        s_seq[i] = nq > 0 && (before[0] + need) * BJ <= a.max_kv_tokens ? seq : 0;
      }
    }
    __syncthreads();
    count = a.n;
    total = 2 * (int)min(blocks, a.max_kv_tokens / BJ);
  } else {
    count = *w.count;
    total = 2 * *w.blocks;
  }
  const int from = (int)((int64_t)total * blockIdx.x / ctas), end = (int)((int64_t)total * (blockIdx.x + 1) / ctas);
  if (from >= end) return;
  const auto first_of = [&](int i) { return i >= count ? INT_MAX : kFold ? s_first[i] : w.entries[i].block; };
  // the last entry whose first block is at or before the run's
  int at = 0;
  if (kFold) {
    for (int hi = count - 1; at < hi;) {
      const int mid = (at + hi + 1) >> 1;
      if (s_first[mid] <= from >> 1) at = mid;
      else hi = mid - 1;
    }
  } else {
    for (int n = count; n > 1;) {
      const int step = (n + kRowsThreads - 1) / kRowsThreads, i = at + tid * step;
      if (i < at + n && first_of(i) <= from >> 1 && (i + step >= at + n || first_of(i + step) > from >> 1)) s_entry = i;
      __syncthreads();
      n = min(step, at + n - s_entry);
      at = s_entry;
      __syncthreads();
    }
  }
  struct Run {
    int block, seq, table;
  };
  const auto run_of = [&](int i) -> Run {
    if (kFold) return {s_first[i], s_seq[i], i};
    const Entry e = w.entries[i];
    return {e.block, e.seq, e.table};
  };
  Run e = run_of(at);
  int next = first_of(at + 1);  // the entry's end
  // the pool row of lane's row of half block h (-1: none; -2: none, where one should be)
  const auto row_of = [&](int h) -> int32_t {
    while (h >> 1 >= next) {
      e = run_of(++at);
      next = first_of(at + 1);
    }
    const int64_t t = (int64_t)(h - 2 * e.block) * HB + lane;
    if (t >= e.seq) return -1;
    const int32_t p = (int32_t)t / a.page_size, page = a.block_tables[(int64_t)e.table * a.max_blocks + p];
    const int64_t r = (int64_t)page * a.page_size + ((int32_t)t - p * a.page_size);
    return page >= 0 && r < a.pool_rows ? (int32_t)r : -2;
  };
  uint32_t* state = reinterpret_cast<uint32_t*>(w.state);  // of half block h: words 4 (h / 2) + h % 2, and two after it
  int32_t mine = warp == 0 ? row_of(from) : -1;
  bool missing = false;
  for (int h = from; h < end; ++h) {
    const int turn = h & 1;
    if (warp == 0) {
      s_row[turn][lane] = mine;
      missing |= mine == -2;
      const uint32_t there = __ballot_sync(0xffffffffu, mine >= 0);
      if (lane == 0) {
        s_there[turn] = there;
        s_bad[turn] = 0;
      }
      if (h + 1 < end) mine = row_of(h + 1);
    }
    __syncthreads();
    if (tid == 0 && h > from) {
      state[4 * ((h - 1) >> 1) + (turn ^ 1)] = s_there[turn ^ 1];
      state[4 * ((h - 1) >> 1) + (turn ^ 1) + 2] = s_bad[turn ^ 1];
    }
    // the codes of a thread's three tasks are on their way at once
    uint32_t c[3][8];
    float s[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int task = warp + k * (kRowsThreads / 32);
      if (task >= 16) break;
      // latents: rows 8 (task / 4) .., 128 values of scale task % 4
      const int32_t r = s_row[turn][8 * (task >> 2) + (lane & 7)];
      const uint8_t* src = a.pool + (int64_t)max(r, 0) * kFp8Row;
      const uint4* codes = reinterpret_cast<const uint4*>(src + 32 * (4 * (task & 3) + (lane >> 3)));
      const uint4 zero = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(c[k]) = r >= 0 ? __ldg(codes) : zero;
      *reinterpret_cast<uint4*>(c[k] + 4) = r >= 0 ? __ldg(codes + 1) : zero;
      s[k] = r >= 0 ? __ldg(reinterpret_cast<const float*>(src + kFp8Scales) + (task & 3)) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int task = warp + k * (kRowsThreads / 32);
      __half2 top = __float2half2_rn(0.f);
      uint32_t x[4][4];
      int row, g;
      if (task < 16) {
        row = 8 * (task >> 2) + (lane & 7);
        g = 4 * (task & 3) + (lane >> 3);
        const __half one = __float2half_rn(s[k]);
        const bool in_f16 = __half2float(one) == s[k];
        const __half2 pair = __half2half2(one);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const __half2_raw q = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c[k][2 * u + (j >> 1)] >> (16 * (j & 1))), __NV_E4M3);
            __half2 v = __hmul2(__half2(q), pair);
            if (!in_f16) {
              const float2 f = __half22float2(__half2(q));
              v = __floats2half2_rn(f.x * s[k], f.y * s[k]);
            }
            top = __hmax2_nan(top, __habs2(v));
            x[j][u] = bits(v);
          }
      } else {  // RoPE: 16 rows, 64 values
        row = 16 * (task - 16) + 8 * (lane >> 4) + (lane & 7);
        g = 16 + ((lane >> 3) & 1);
        const int32_t r = s_row[turn][row];
        uint32_t y[16] = {};
        if (r >= 0) {
          const uint4* src = reinterpret_cast<const uint4*>(a.pool + (int64_t)r * kFp8Row + kFp8RopeAt + 64 * (g - 16));
#pragma unroll
          for (int u = 0; u < 4; ++u) *reinterpret_cast<uint4*>(y + 4 * u) = __ldg(src + u);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const __half2 v = __floats2half2_rn(__uint_as_float(y[4 * u + j] << 16), __uint_as_float(y[4 * u + j] & 0xFFFF0000u));
            top = __hmax2_nan(top, __habs2(v));
            x[j][u] = bits(v);
          }
      }
      if (without_bad(bits(top)) != bits(top)) {  // few
        atomicOr(&s_bad[turn], 1u << row);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int u = 0; u < 4; ++u) x[j][u] = without_bad(x[j][u]);
      }
      uint8_t* line = w.kv + (size_t)(h >> 1) * BLOCK + (g >> 1) * ATOM + turn * (HB * 128) + row * 128;
#pragma unroll
      for (int j = 0; j < 4; j += 2) {  // two chunks: a sector
        const int place = ((g & 1) * 4 + j) ^ (row & 7);
        const bool swap = row & 1;
        uint32_t y[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          y[u] = swap ? x[j + 1][u] : x[j][u];
          y[4 + u] = swap ? x[j][u] : x[j + 1][u];
        }
        store8(reinterpret_cast<uint32_t*>(line + (place & 6) * 16), y, true);
      }
    }
  }
  __syncthreads();
  if (tid == 0) {
    const int h = end - 1;
    state[4 * (h >> 1) + (h & 1)] = s_there[h & 1];
    state[4 * (h >> 1) + (h & 1) + 2] = s_bad[h & 1];
  }
  if (missing) atomicOr(err, HS_FLAG_DEVROW);
}
static_assert(kRowsThreads / 32 * 3 == 16 + HB / 16, "three tasks a warp");

// ---------------------------------------------------------------- the attention

struct Barriers {
  uint64_t k_full[2][NK], k_free[2][NK];  // S-CTA: each part of a ring slot: its bytes are there; it has been read
  uint64_t v_full[NVF], v_free[NV];       // O-CTA: the same of a slot
  uint64_t q_full[NQ], q_done;     // S-CTA: Q in tensor memory; the tile's last S is done
  // per softmax warpgroup, so that whoever waits on one waits on every phase of it (parities repeat):
  uint64_t s_full[NS], s_free[NS]; // S-CTA: S written; S read
  uint64_t s_next[NS];             // S-CTA: the block's MMAs have been issued
  uint64_t m_set[NS][4];           // S-CTA: the block's reference maxima of a warp's heads are set
  uint64_t p_free[NP];             // both, arrived by the O-CTA's issuers: P . V of the block is done
  uint64_t p_full[NP];             // O-CTA, completed by the S-CTA's stores
  uint64_t pv_go[NP];              // O-CTA: O is ready for P . V of the block
  uint64_t fin[NF];                // O-CTA: the S-CTA's totals of a tile are here
  uint64_t o_full, o_free[2];      // O-CTA: a tile's last P . V is done; a half of O has been read
};
static_assert(NP == NS + 1, "softmax's waits for P's buffers");

struct __align__(STATIC_BYTES) Control {
  Barriers bs;
  uint32_t taddr;
  int abort;
  int issued[NS];  // blocks whose MMAs each issuer started (the last commit to wait for)
  int requested;   // ring slots (S-CTA: parts of them) whose copies were started
};
static_assert(sizeof(Control) == STATIC_BYTES, "one block");

// A tile, or a part of one: what a pair does next. Every role computes it by itself.
struct Unit {
  int nblk;        // its blocks
  int first, kv;   // the first one's number in its sequence, and in the workspace
  int live;        // query heads of the tile
  size_t row0;     // the first one's row of q, o and lse
  int64_t seen;    // tokens that the tile's first query sees
  bool whole;
};
struct Walk {
  Pos at, end;
  Entry e;
  int held;  // the entry that e is
};
__device__ __forceinline__ bool next_unit(const ChunkArgs& a, const Work& w, int per_tile, Walk& k, Unit& u) {
  if (k.at.ent == k.end.ent && k.at.tile == k.end.tile && k.at.blk == k.end.blk) return false;
  if (k.held != k.at.ent) {
    k.e = w.entries[k.at.ent];
    k.held = k.at.ent;
  }
  const int first = k.at.tile * per_tile, tokens = min(per_tile, k.e.nq - first);
  u.seen = (int64_t)k.e.seq - k.e.nq + first + 1;
  const int all = blocks_of(u.seen + tokens - 1);
  const bool cut = k.at.ent == k.end.ent && k.at.tile == k.end.tile;
  u.first = k.at.blk;
  u.nblk = (cut ? k.end.blk : all) - u.first;
  u.kv = k.e.block + u.first;
  u.live = tokens * a.num_heads;
  u.row0 = ((size_t)k.e.q0 + first) * a.num_heads;
  u.whole = u.first == 0 && !cut;
  if (cut) {
    k.at = k.end;
  } else {
    k.at.blk = 0;
    if (first + tokens >= k.e.nq) {
      ++k.at.ent;
      k.at.tile = 0;
    } else {
      ++k.at.tile;
    }
  }
  return true;
}

// What a unit of q . row is in log2 units.
__device__ __forceinline__ float score_log2(const ChunkArgs& a) { return fabsf(a.sm_scale * 1.4426950408889634f); }

__global__ void __launch_bounds__(T, 1)
    chunk_mla_kernel(const ChunkArgs a, const Work w, const __grid_constant__ CUtensorMap tm_q, uint32_t* __restrict__ err) {
  // (what is static fills a block of the tiles' alignment, and the rest begins after it)
  extern __shared__ __align__(STATIC_BYTES) uint8_t base[];
  __shared__ __align__(STATIC_BYTES) Control ctl;
  Barriers& bs = ctl.bs;
  if ((smem_u32(base) & (STATIC_BYTES - 1)) != 0) {  // (never: the tiles' swizzle wants it)
    if (threadIdx.x == 0) atomicOr(err, HS_FLAG_TIMEOUT);
    return;
  }
  volatile int* abort = &ctl.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = blockIdx.x & 1u, partner = rank ^ 1u;  // 0: S-CTA, 1: O-CTA
  const int pair = blockIdx.x >> 1;

  if (tid == 0) {
    for (int k = 0; k < 2 * NK; ++k) {
      bar_init(&bs.k_full[0][k], 1);
      bar_init(&bs.k_free[0][k], 1);
    }
    for (int k = 0; k < NVF; ++k) bar_init(&bs.v_full[k], 1);
    for (int k = 0; k < NV; ++k) bar_init(&bs.v_free[k], 1);
    for (int k = 0; k < NQ; ++k) bar_init(&bs.q_full[k], 4);  // one arrival per warp that brings Q
    bar_init(&bs.q_done, NS);
    for (int k = 0; k < NS; ++k) {
      bar_init(&bs.s_full[k], 1);
      bar_init(&bs.s_next[k], 1);
      bar_init(&bs.s_free[k], 4);  // the warps of the block's softmax warpgroup
      for (int x = 0; x < 4; ++x) bar_init(&bs.m_set[k][x], 1);
    }
    for (int k = 0; k < NP; ++k) {
      bar_init(&bs.p_free[k], 2);
      bar_init(&bs.p_full[k], 1);  // the O-CTA's expect_tx; the S-CTA's stores complete it
      bar_init(&bs.pv_go[k], 4);
    }
    for (int k = 0; k < NF; ++k) bar_init(&bs.fin[k], 1);  // the same
    bar_init(&bs.o_full, 2);
    for (int k = 0; k < 2; ++k) bar_init(&bs.o_free[k], 4 * NOUT);
    ctl.abort = 0;
    for (int k = 0; k < NS; ++k) ctl.issued[k] = 0;
    ctl.requested = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (rank == 1)
      for (int k = 0; k < NP; ++k) bar_arrive_tx(&bs.p_full[k], P_BYTES);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.taddr)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  // both CTAs' barriers are initialised before either arrives on the other's
  asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  // the merge kernel may launch where SMs come free; it waits for this grid's completion before reading
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  pdl_wait();
  asm volatile("fence.proxy.async;" ::: "memory");  // what the kernels before wrote, before this one's bulk copies of it
  const uint32_t tbase = ctl.taddr;
  const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
  const int head = (warp & 3) * 32 + lane;  // this thread's row of the tile = its tensor-memory lane
  const int per_tile = MH / a.num_heads, token = head / a.num_heads;
  Walk walk;
  walk.at = w.starts[pair];
  walk.end = w.starts[pair + 1];
  walk.held = -1;

  // The units of this pair, one after the other. Each role goes through them by itself: what the roles
  // hand each other carries on from unit to unit.
  bool ok = true;
  int done = 0, full = 0;  // blocks, and units with blocks, before this one
  Unit un;
#pragma unroll 1
  for (; __all_sync(0xffffffffu, next_unit(a, w, per_tile, walk, un)); done += un.nblk, full += un.nblk > 0) {
    un.nblk = __reduce_max_sync(0xffffffffu, un.nblk);
    const int nblk = un.nblk;
    const int use0 = done + 2 * full;  // the S-CTA's ring: Q's two slots, then a slot per block
    if (rank == 0) {
      // ================================ S-CTA ================================
      if (nblk == 0) continue;
      if (warp < 4 * NS) {
        const int wg = warp >> 2;
        ok = __all_sync(0xffffffffu, ready_or_wait(bs.q_full, NQ, full, abort));
        if (!ok) break;
        const float up = reinterpret_cast<const float*>(base + S_UP)[full % NQ * MH + head];
        // Warpgroup wg takes the blocks whose number g = done + b has g % NS = wg, a query head per
        // thread. From one block to the next only the reference maximum goes over, from warp to warp
        // (the warps of the same heads): it is known once a block's scores have been read, so the
        // warpgroups' exponentials overlap. Each keeps the sum of its own blocks under the reference of
        // its last one. References are
        // scores as S holds them, and a weight's exponent is the difference, scaled: a score times the scale
        // is rounded by whole units from 2^24 on.
        float m_own = -INFINITY, l_own = 0.f;  // the sum of this thread's blocks, under this reference
        float* s_ref = reinterpret_cast<float*>(base + S_REF);
        const uint32_t pbuf0 = remote(base + O_P + 16 * head, partner);
        const uint32_t alpha0 = remote(base + O_ALPHA + 4 * head, partner), rbar0 = remote(&bs.p_full[0], partner);
        // what a unit of S is; a scale of zero stays above it, so that -inf stays -inf
        const float sl2 = fminf(fmaxf(score_log2(a) * up, 1e-37f), 3e38f);
        const uint32_t s_at = tbase + lane_off + S_COL + BJ * wg;
        const int64_t sees_to = un.seen + token - (int64_t)un.first * BJ;  // rows of the unit that this query sees
        int b = wg - done % NS;
        if (b < 0) b += NS;
        const bool mine = b < nblk, last = (done + nblk - 1) % NS == wg;
        uint32_t turn = (uint32_t)((done + b) / NS) & 1u;  // of this warpgroup: its barriers' phase
        uint4 state = {};
        if (mine) state = __ldcg(w.state + un.kv + b);
#pragma unroll 1
        for (; ok && b < nblk; b += NS, turn ^= 1u) {
          const int g = done + b;
          const int64_t left = sees_to - (int64_t)b * BJ;
          const int to = (int)min(max(left, (int64_t)0), (int64_t)BJ);
          const uint32_t sees0 = state.x & bit_range(0, to), sees1 = state.y & bit_range(0, to - 32);
          const uint32_t nan0 = state.z, nan1 = state.w;
          if (b + NS < nblk) state = __ldcg(w.state + un.kv + b + NS);
          ok = __all_sync(0xffffffffu, ready_or_wait(&bs.s_full[wg], 1, (int)turn, abort));
          if (!ok) break;
          tc_after();
          const bool every = __all_sync(0xffffffffu, (sees0 & sees1) == 0xFFFFFFFFu && (nan0 | nan1) == 0u);
          float t[BJ];  // the scores; -inf where this query does not look
          tmem_ld64(s_at, t);
          tc_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&bs.s_free[wg]);  // S has been read
          if (!every) {
#pragma unroll
            for (int i = 0; i < BJ; ++i) {
              const uint32_t sees = i < 32 ? sees0 : sees1, nan = i < 32 ? nan0 : nan1;
              t[i] = ((sees >> (i & 31)) & 1u) ? (((nan >> (i & 31)) & 1u) ? __uint_as_float(0x7FC00000u) : t[i]) : -INFINITY;
            }
          }
          float x0 = t[0], x1 = t[1], x2 = t[2], x3 = t[3];
#pragma unroll
          for (int i = 4; i < BJ; i += 4) {
            x0 = fmaxf(x0, t[i]);
            x1 = fmaxf(x1, t[i + 1]);
            x2 = fmaxf(x2, t[i + 2]);
            x3 = fmaxf(x3, t[i + 3]);
          }
          const float bm = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
          float m_run = -INFINITY;
          if (g > 0) {
            // (the block before is the last warpgroup's block of this turn, or of the turn before)
            const int before = wg == 0 ? NS - 1 : wg - 1;
            ok = __all_sync(0xffffffffu, ready_or_wait(&bs.m_set[before][warp & 3], 1, (int)(wg == 0 ? turn ^ 1u : turn), abort));
            if (!ok) break;
            if (b > 0) m_run = s_ref[head];
          }
          // Lazy rescale: a head keeps its reference until a block's maximum passes it by 2^kRescaleLog2,
          // and O is rescaled only on those rare jumps. (NaN scores leave it alone.)
          const float m_new = (bm - m_run) * sl2 > kRescaleLog2 || m_run == -INFINITY ? fmaxf(m_run, bm) : m_run;
          s_ref[head] = m_new;
          __syncwarp();
          if (lane == 0) bar_arrive(&bs.m_set[wg][warp & 3]);
          const float alpha = m_new == -INFINITY ? 1.f : ex2((m_run - m_new) * sl2);  // m_run = -inf: O is still 0
          const float ref = m_new == -INFINITY ? 0.f : m_new;  // a NaN score stays one, an unseen row's weight is 0
          l_own *= m_new == -INFINITY ? 1.f : ex2((m_own - m_new) * sl2);
          m_own = m_new;
          // the O-CTA's P buffer is free once P . V of block g - NP is done (that of g - 2 NP is known to be: the warpgroup
          // of block g - NP = g - 1 - NS has waited for it and was then at block g - 1, whose m_set has been seen)
          ok = __all_sync(0xffffffffu, g < NP || ready_or_wait<true>(bs.p_free, NP, g - NP, abort));
          if (!ok) break;
          const uint32_t pbuf = pbuf0 + (g % NP) * P_BUF, rbar = rbar0 + (g % NP) * 8;
          st_async_f32(alpha0 + (g % NP) * (MH * 4), alpha, rbar);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int q = 0; q < BJ / 8; ++q) {  // 16-B chunks of 8 f16
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float2 e = fma2(add2(make_float2(t[8 * q + 2 * i], t[8 * q + 2 * i + 1]), make_float2(-ref, -ref)),
                              make_float2(sl2, sl2), make_float2(kRefLog2, kRefLog2));
              e = make_float2(ex2(e.x), ex2(e.y));
              const __half2 pb = __floats2half2_rn(e.x, e.y);
              sum = add2(sum, e);
              v[i] = *reinterpret_cast<const uint32_t*>(&pb);
            }
            st_async16(pbuf + q * (MH * 16), make_uint4(v[0], v[1], v[2], v[3]), rbar);
          }
          l_own += sum.x + sum.y;
        }
        // its sum, under the reference of its last block, to the O-CTA
        if (ok && mine) {
          const uint32_t fin = remote(base + O_FIN, partner) + (full % NF) * FIN;
          const uint32_t bar = remote(&bs.fin[full % NF], partner);
          st_async_f32(fin + wg * FIN_WG + 4 * head, l_own, bar);
          st_async_f32(fin + wg * FIN_WG + 4 * (MH + head), m_own, bar);
          if (last) st_async_f32(fin + NS * FIN_WG + 4 * head, sl2, bar);
        }
      } else {
        const uint64_t k0 = mdesc(smem_u32(base + S_RING), 16, 1024);
        const auto copy = [&](int i) {  // one thread: half of Q (64 rows, in boxes of 64 values), or a block
          const int use = use0 + i;
#pragma unroll 1
          for (int part = 0; part < 2; ++part) {
            if (use >= NK && !ready_or_wait(bs.k_free[part], NK, use - NK, abort)) return false;
            uint64_t* bar = &bs.k_full[part][use % NK];
            const uint32_t from = part ? PART : 0, size = part ? BLOCK - PART : PART;
            const uint32_t dst = smem_u32(base + S_RING + (use % NK) * BLOCK) + from;
            bar_arrive_tx(bar, size);
            ctl.requested = 2 * use + part + 1;
            if (i < 2) {
              for (uint32_t at = 0; at < size; at += ATOM)
                asm volatile(
                    "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                        dst + at),
                    "l"(&tm_q), "r"((int)((from + at) / ATOM) * 64), "r"((int)un.row0 + BJ * i), "r"(smem_u32(bar))
                    : "memory");
            } else {
              asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                           "l"(w.kv + (size_t)(un.kv + i - 2) * BLOCK + from), "r"(size), "r"(smem_u32(bar))
                           : "memory");
            }
          }
          return true;
        };
        bool go = true;
        if (warp == COPIER) {  // Q and the first block, as far as the ring goes before Q has left it
          for (int i = 0; lane == 0 && go && i < NK; ++i) go = copy(i);
          go = __shfl_sync(0xffffffffu, (int)go, 0) != 0;
        }
        // Q into tensor memory, a head per thread, column c holding the values of places 2c, 2c + 1 of a row, over a power
        // of two that brings the head's largest to 2^14 .. 2^15 where it is below 1 or above 65504. The tile before may still
        // be in the softmax: it needs its S only, all of which is done.
        go = go && (full == 0 || ready_or_wait(&bs.q_done, 1, full - 1, abort));
        const int q_use = use0 + (head >> 6);
        go = go && ready_or_wait(bs.k_full[0], NK, q_use, abort) && ready_or_wait(bs.k_full[1], NK, q_use, abort);
        go = __all_sync(0xffffffffu, go);
        if (go) {
          tc_after();
          const uint8_t* src = base + S_RING + (q_use % NK) * BLOCK + (head & 63) * 128;
          // It is taken as it is first, and once more where some head's values want a divisor.
          const auto take = [&](auto scaled, float mul) {  // the largest magnitude in f16
            constexpr bool kScaled = decltype(scaled)::value;
            __half2 top = __float2half2_rn(0.f);
#pragma unroll 3
            for (int h = 0; h < 2 * QATOMS; ++h) {  // 32 values: 16 columns
              uint32_t x[16], y[16];
#pragma unroll
              for (int u = 0; u < 4; ++u)
                *reinterpret_cast<uint4*>(x + 4 * u) =
                    *reinterpret_cast<const uint4*>(src + (h >> 1) * ATOM + ((((h & 1) * 4 + u) ^ (head & 7)) << 4));
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const float lo = __uint_as_float(x[4 * u + j] << 16), hi = __uint_as_float(x[4 * u + j] & 0xFFFF0000u);
                  const __half2 f = kScaled ? __floats2half2_rn(lo * mul, hi * mul) : __floats2half2_rn(lo, hi);
                  if (!kScaled) top = __hmax2(top, __habs2(f));
                  y[4 * j + u] = *reinterpret_cast<const uint32_t*>(&f);
                }
              asm volatile(
                  "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
                      tbase + lane_off + Q_COL + 16 * h),
                  "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7]), "r"(y[8]), "r"(y[9]),
                  "r"(y[10]), "r"(y[11]), "r"(y[12]), "r"(y[13]), "r"(y[14]), "r"(y[15])
                  : "memory");
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            return fmaxf(__low2float(top), __high2float(top));
          };
          float up = 1.f;
          const float largest = take(std::false_type{}, 1.f);
          if (__any_sync(0xffffffffu, head < un.live && !(largest >= 1.f && largest < 65504.f)) || a.sm_scale < 0.f) {
            uint32_t top = 0;
#pragma unroll 1
            for (int c = 0; c < 8 * QATOMS; ++c) top = max_bf16x2(top, *reinterpret_cast<const uint4*>(src + (c >> 3) * ATOM + ((c & 7) << 4)));
            top = max(top & 0xFFFFu, top >> 16);
            const int down = top == 0 ? 127 : min(127 + 14 + 127 - (int)(top >> 7), 253);  // biased
            const float mul = __uint_as_float((uint32_t)down << 23);
            up = __uint_as_float((uint32_t)(254 - down) << 23);
            take(std::true_type{}, a.sm_scale < 0.f ? -mul : mul);  // (negative, so that scores scale by a positive factor)
          }
          reinterpret_cast<float*>(base + S_UP)[full % NQ * MH + head] = up;
          tc_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&bs.q_full[full % NQ]);
        }
        if (warp == COPIER) {
#pragma unroll 1
          for (int i = NK; lane == 0 && go && i < 2 + nblk; ++i) go = copy(i);
          go = __shfl_sync(0xffffffffu, (int)go, 0) != 0;
        } else {
          // (tensor memory starts at 0: all of it is allocated here)
          const int wg = warp - ISSUER;
          const bool one = elected();
          go = __all_sync(0xffffffffu, go && ready_or_wait(bs.q_full, NQ, full, abort));
          if (go && one && wg == 0) {  // Q has left its slots
            for (int k = 0; k < 4; ++k) bar_arrive(&bs.k_free[k & 1][(use0 + (k >> 1)) % NK]);
          }
          tc_after();
          int b = wg - done % NS;
          if (b < 0) b += NS;
          if (go && one && b >= nblk) bar_arrive(&bs.q_done);  // nothing of this unit
          int turn = (done + b) / NS;  // of this buffer
#pragma unroll 1
          for (; go && b < nblk; b += NS, ++turn) {
            const int use = use0 + 2 + b;
            go = ready_or_wait(bs.k_full[0], NK, use, abort) && ready_or_wait(bs.k_full[1], NK, use, abort);
            go = go && (turn == 0 || ready_or_wait(&bs.s_free[wg], 1, turn - 1, abort));
            // blocks in their order: issued side by side, two would take as long as both and leave their slots together
            const int before = done + b - 1;
            go = go && (before < 0 || ready_or_wait(bs.s_next, NS, before, abort));
            go = __all_sync(0xffffffffu, go);
            if (!go) break;
            tc_after();
            const uint64_t dk0 = k0 + (uint64_t)((use % NK) * (BLOCK >> 4));
            const uint32_t d = S_COL + BJ * wg;
            const auto mmas = [&](auto first, auto end) {
#pragma unroll
              for (int kk = decltype(first)::value; kk < decltype(end)::value; ++kk)
                mma_ta(d, Q_COL + 8 * kk, dk0 + (uint64_t)(((kk >> 2) * ATOM + (kk & 3) * 32) >> 4), kIdescQK, kk > 0);
            };
            using First = std::integral_constant<int, 0>;
            using Middle = std::integral_constant<int, PART / ATOM * 4>;
            using End = std::integral_constant<int, QATOMS * 4>;
            if (one) {
              ctl.issued[wg] = turn + 1;
              mmas(First{}, Middle{});
              commit(&bs.k_free[0][use % NK]);
              mmas(Middle{}, End{});
              bar_arrive(&bs.s_next[wg]);
              commit(&bs.s_full[wg]);
              commit(&bs.k_free[1][use % NK]);
              if (b + NS >= nblk) commit(&bs.q_done);
            }
            __syncwarp();
          }
        }
        ok = go;
      }
    } else {
      // ================================ O-CTA ================================
      const float* alpha_buf = reinterpret_cast<const float*>(base + O_ALPHA);
      if (warp < 4) {
        // corrector: where a reference maximum of the warp's heads rose, rescale O once P . V of the
        // block before is done
#pragma unroll 1
        for (int b = 0; ok && b < nblk; ++b) {
          const int g = done + b;
          ok = __all_sync(0xffffffffu, ready_or_wait<true>(bs.p_full, NP, g, abort));
          if (!ok) break;
          const float f = alpha_buf[g % NP * MH + head];
          // this buffer's next phase is block g + NP: its bytes come only after P . V of block g
          if (tid == 0) bar_arrive_tx(&bs.p_full[g % NP], P_BYTES);
          if (__any_sync(0xffffffffu, b > 0 && f != 1.f)) {
            ok = __all_sync(0xffffffffu, ready_or_wait(bs.p_free, NP, g - 1, abort));
            if (!ok) break;
            tc_after();
#pragma unroll 1
            for (int c = 0; c < DL; c += 16) {
              float v[16];
              tmem_ld16(tbase + lane_off + c, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] *= f;
              tmem_st16(tbase + lane_off + c, v);
            }
            tc_before();
          }
          __syncwarp();
          if (lane == 0) bar_arrive(&bs.pv_go[g % NP]);
        }
      } else if (warp == ISSUER || warp == ISSUER + 1) {
        const int nh = warp - ISSUER;  // this issuer's 256 columns
        const bool one = elected();
        const uint64_t p0 = pdesc(smem_u32(base + O_P)), v0 = mdesc(smem_u32(base + O_RING), ATOM, 1024);
#pragma unroll 1
        for (int b = 0; ok && b < nblk; ++b) {
          const int g = done + b, use = 2 * g + nh;
          bool go = ready_or_wait(bs.pv_go, NP, g, abort);
          if (b == 0) go = go && (full == 0 || ready_or_wait(&bs.o_free[nh], 1, full - 1, abort));
          go = go && ready_or_wait(bs.v_full, NVF, use, abort);
          ok = __all_sync(0xffffffffu, go);
          if (!ok) break;
          tc_after();
          fence_async_smem();  // P's writes, seen through their barrier, before the tensor core's reads
          const uint64_t dp0 = p0 + (uint64_t)((g % NP) * (P_BUF >> 4)), dv0 = v0 + (uint64_t)((use % NV) * (HALF_V >> 4));
          if (one) {
#pragma unroll
            for (int kk = 0; kk < BJ / 16; ++kk)
              mma_ss(256 * nh, dp0 + (uint64_t)((kk * 2 * MH * 16) >> 4), dv0 + (uint64_t)((kk * 2048) >> 4), kIdescPV,
                     (b > 0 || kk > 0) ? 1u : 0u);
            commit(&bs.v_free[use % NV]);
            commit_multicast(&bs.p_free[g % NP], (uint16_t)3);
            if (b == nblk - 1) commit(&bs.o_full);
            ctl.issued[nh] = g + 1;
          }
          __syncwarp();
        }
      } else if (warp == COPIER) {
#pragma unroll 1
        for (int i = 0; lane == 0 && ok && i < 2 * nblk; ++i) {
          const int use = 2 * done + i;
          ok = use < NV || ready_or_wait(bs.v_free, NV, use - NV, abort);
          if (!ok) break;
          uint64_t* bar = &bs.v_full[use % NVF];
          bar_arrive_tx(bar, HALF_V);
          ctl.requested = use + 1;
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                           smem_u32(base + O_RING + (use % NV) * HALF_V)),
                       "l"(w.kv + (size_t)(un.kv + (i >> 1)) * BLOCK + (i & 1) * HALF_V), "r"(HALF_V), "r"(smem_u32(bar))
                       : "memory");
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      }
      if (warp < ISSUER) {
        // The read-out. Warps w and w + 4 have a quarter of the heads, as tensor memory has it, and every
        // second 32 columns. The columns are ordered so that a lane's fragments are eight consecutive dims of each of
        // four rows, and four lanes have 32 dims of a row. The warps that have nothing else to do wait at a barrier of
        // the hardware, not at the mbarriers; the corrector meets them there and goes on to the next tile.
        ok = sync_and(ok, 32 * ISSUER);
        if (!ok) break;  // (all of them: one that gave up further down comes here once more)
        if (warp < OUT) continue;
        const int set = (warp - OUT) >> 2;
        float l = 0.f, m = -INFINITY, sl2 = 0.f;
        if (nblk > 0) {
          const int k = full % NF;
          if (tid == 32 * OUT) bar_arrive_tx(&bs.fin[k], min(nblk, NS) * FIN_WG + MH * 4);
          ok = ready_or_wait<true>(bs.fin, NF, full, abort) && ready_or_wait(&bs.o_full, 1, full, abort);
          ok = __all_sync(0xffffffffu, ok);
          tc_after();
          // the warpgroups' sums, from the reference of each to the last block's
          const float* fin = reinterpret_cast<const float*>(base + O_FIN + k * FIN) + head;
          sl2 = fin[NS * (FIN_WG / 4)];
          m = fin[(done + nblk - 1) % NS * (FIN_WG / 4) + MH];
          for (int b = 0; b < min(nblk, NS); ++b) {
            const float* of = fin + (done + nblk - 1 - b) % NS * (FIN_WG / 4);
            l += of[MH] == -INFINITY ? of[0] : of[0] * ex2((of[MH] - m) * sl2);  // (no score: 0, or NaN)
          }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;  // l is NaN where a weight is
        const int part = 2 * pair + (un.first > 0 ? 0 : 1);
        const size_t out0 = un.whole ? un.row0 : (size_t)part * MH;
        const int row = (warp & 3) * 32 + (lane >> 2);  // and 8, 16, 24 after it
        const size_t at = (out0 + row) * DL + 8 * (lane & 3);
#pragma unroll 1
        for (int i = set; ok && i < DL / 32; i += 2 * NOUT) {  // two of the set's 32 columns at a time
          float v[2][2][16] = {};
          const bool two = i + NOUT < DL / 32;
          if (nblk > 0) {
            tmem_ld_frag(tbase + lane_off + 32 * i, v[0]);
            if (two) tmem_ld_frag(tbase + lane_off + 32 * (i + NOUT), v[1]);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
            // the columns below 256, or all, are in registers
            tc_before();
            __syncwarp();
            if (lane == 0 && i < DL / 64 && i + 2 * NOUT >= DL / 64) bar_arrive(&bs.o_free[0]);
            if (lane == 0 && i + 2 * NOUT >= DL / 32) bar_arrive(&bs.o_free[1]);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c = 32 * (i + e * NOUT);
            if (e == 1 && !two) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // rows 8 k after the first
              const float f = __shfl_sync(0xffffffffu, inv, 8 * k + (lane >> 2));
              uint32_t x[8];
#pragma unroll
              for (int q = 0; q < 8; ++q) x[q] = __float_as_uint(v[e][k >> 1][4 * (q >> 1) + 2 * (k & 1) + (q & 1)] * f);
              if (row + 8 * k >= un.live) {  // no query head
              } else if (un.whole) {
                uint32_t h[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(x[2 * q]), __uint_as_float(x[2 * q + 1]));
                  h[q] = *reinterpret_cast<const uint32_t*>(&y);
                }
                *reinterpret_cast<uint4*>(a.o + at + 8 * k * DL + c) = make_uint4(h[0], h[1], h[2], h[3]);
              } else {
                store8(reinterpret_cast<uint32_t*>(w.part_o + at + 8 * k * DL + c), x, true);
              }
            }
          }
        }
        if (ok && set == 0 && head < un.live)
          (un.whole ? a.lse : w.part_lse)[out0 + head] = l == 0.f ? -INFINITY : (m * sl2 + (log2f(l) - kRefLog2)) * 0.6931471805599453f;
        __syncwarp();
      }
      if (!ok && warp >= ISSUER) break;
    }
    if (!ok && rank == 0) break;
  }

  __syncthreads();
  // MMAs and their arrivals in this CTA are over, and the S-CTA has the O-CTA's last P-buffer releases
  if (ok && done > 0) {
    if (rank == 0) {
      for (int k = max(done + 2 * full - NK, 0); k < done + 2 * full; ++k)
        ok = ok && ready_or_wait(bs.k_free[0], NK, k, abort) && ready_or_wait(bs.k_free[1], NK, k, abort);
      ok = ok && ready_or_wait(&bs.q_done, 1, full - 1, abort);
      for (int b = done >= NP ? done - NP : 0; b < done; ++b) ok = ok && ready_or_wait<true>(bs.p_free, NP, b, abort);
    } else {
      ok = ready_or_wait(bs.v_free, NV, 2 * done - 2, abort) && ready_or_wait(bs.v_free, NV, 2 * done - 1, abort) &&
           ready_or_wait(bs.p_free, NP, done - 1, abort);
    }
  }
  ok = __syncthreads_and(ok && !*abort);
  if (!ok) {
    // outputs are not valid: flag it, and give copies and MMAs still in flight one more bound before
    // the shared and tensor memory are released
    if (tid == 0) atomicOr(err, HS_FLAG_TIMEOUT);
    __syncthreads();
    if (tid == 0) ctl.abort = 0;
    __syncthreads();
    const int m = ctl.requested;
    if (rank == 0) {
      for (int k = m >= 2 * NK ? m - 2 * NK : 0; k < m; ++k) pipe_wait(bs.k_full[k & 1], NK, k >> 1, abort);
      for (int k = 0; k < NS; ++k)
        if (ctl.issued[k] > 0) pipe_wait(&bs.s_full[k], 1, ctl.issued[k] - 1, abort);
    } else {
      for (int k = m >= NV ? m - NV : 0; k < m; ++k) pipe_wait(bs.v_full, NVF, k, abort);
      // (each issuer's last block; a block that only one of them issued completes no phase: its slot's does)
      for (int k = 0; k < 2; ++k)
        if (ctl.issued[k] > 0) pipe_wait(bs.v_free, NV, 2 * (ctl.issued[k] - 1) + k, abort);
    }
  }
  tc_before();
  __syncthreads();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(TMEM_COLS) : "memory");
  cluster_sync_all();  // the partner no longer reads or arrives on this CTA's shared memory
  if (!ok && tid == 0) stay();
}

// ---------------------------------------------------------------- the join

// The parts of a tile that pair blockIdx.y began and did not end, joined in their order, weighed by their log-sum-exps.
// A CTA has kMergeRows query heads, a thread eight output dims of one; what it asks of memory it asks for at once (parts
// one after the other, each found from the one before, took 47 us where a tile has 32).
constexpr int kMergeRows = 4, kMergeThreads = kMergeRows * DL / 8;
static_assert(kMergeThreads > kPairs, "a thread per pair");
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const ChunkArgs a, const Work w, int pairs) {
  __shared__ Pos s_start[kPairs + 1];
  __shared__ int s_slot[kPairs];
  __shared__ float s_lse[kMergeRows][kPairs], s_weight[kMergeRows][kPairs];
  pdl_wait();
  const int p = blockIdx.y, tid = threadIdx.x;
  const Pos from = w.starts[p], cut = w.starts[p + 1];
  if (cut.blk == 0 || (from.ent == cut.ent && from.tile == cut.tile && from.blk > 0)) return;
  if (tid <= pairs) s_start[tid] = w.starts[tid];
  const Entry e = w.entries[cut.ent];
  __syncthreads();
  // pair q > p has a part if its work begins inside the tile and is not nothing: so many before it, in order
  int n = 1;
  {
    bool part = false;
    if (tid > p && tid < pairs) {
      const Pos b = s_start[tid], c = s_start[tid + 1];
      part = b.ent == cut.ent && b.tile == cut.tile && b.blk > 0 && !(b.ent == c.ent && b.tile == c.tile && b.blk == c.blk);
    }
    int at = 1;
#pragma unroll
    for (int k = 0; k < (kPairs + 31) / 32; ++k) {
      const int here = __syncthreads_count(part && tid >> 5 == k);
      if (tid >> 5 > k) at += here;
      n += here;
    }
    at += __popc(__ballot_sync(0xffffffffu, part) & ((1u << (tid & 31)) - 1u));
    if (part) s_slot[at] = 2 * tid;
    if (tid == 0) s_slot[0] = 2 * p + 1;
  }
  __syncthreads();
  const int per_tile = MH / a.num_heads, first = cut.tile * per_tile, live = min(per_tile, e.nq - first) * a.num_heads;
  const int r = tid / (DL / 8), c8 = tid % (DL / 8), m = blockIdx.x * kMergeRows + r;
  if (m < live)
    for (int k = c8; k < n; k += DL / 8) s_lse[r][k] = w.part_lse[s_slot[k] * MH + m];
  __syncthreads();
  float top = -INFINITY;  // (a NaN leaves the maximum alone)
  for (int k = 0; k < n; ++k) top = fmaxf(top, s_lse[r][k]);
  const float ref = top == -INFINITY ? 0.f : top;
  for (int k = c8; k < n; k += DL / 8) s_weight[r][k] = expf(s_lse[r][k] - ref);
  __syncthreads();
  if (m >= live) return;
  float acc[8] = {}, z = 0.f;
#pragma unroll 4
  for (int k = 0; k < n; ++k) {
    const float4* src = reinterpret_cast<const float4*>(w.part_o + ((size_t)s_slot[k] * MH + m) * DL) + 2 * c8;
    const float4 u = src[0], v = src[1];
    const float f = s_weight[r][k];
    z += f;
    acc[0] += f * u.x;
    acc[1] += f * u.y;
    acc[2] += f * u.z;
    acc[3] += f * u.w;
    acc[4] += f * v.x;
    acc[5] += f * v.y;
    acc[6] += f * v.z;
    acc[7] += f * v.w;
  }
  const float inv = z == 0.f ? 0.f : 1.f / z;
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    h[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  const size_t row = ((size_t)e.q0 + first) * a.num_heads + m;
  *reinterpret_cast<uint4*>(a.o + row * DL + 8 * c8) = make_uint4(h[0], h[1], h[2], h[3]);
  if (c8 == 0) a.lse[row] = z == 0.f ? -INFINITY : top + logf(z);
}

// Q ([rows][576] bf16) as a 2-D tensor read in boxes of 64 rows x 64 dims, its 16-B chunks XOR-ed
// with the row % 8; rows past the end read as zeros.
cudaError_t q_map(CUtensorMap* m, const uint16_t* q, int64_t rows) {
  EncodeTiled fn = encoder();
  if (fn == nullptr) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)DQK, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)DQK * 2};
  const cuuint32_t box[2] = {64u, (cuuint32_t)BJ};
  const cuuint32_t elem[2] = {1u, 1u};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<uint16_t*>(q), dims, strides, box, elem,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// CTA pairs that the current device holds at once: a CTA takes an SM. What a device is asked is kept, and the kernels are
// set up for it on the way.
constexpr int kDevices = 64;
cudaError_t pairs_resident(int* pairs) {
  static std::atomic<int> known[kDevices];
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < kDevices && (*pairs = known[dev].load(std::memory_order_acquire)) > 0) return e;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(chunk_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  *pairs = sms / 2 < 1 ? 1 : sms / 2 < kPairs ? sms / 2 : kPairs;
  if (e != cudaSuccess)
    (void)cudaGetLastError();
  else if (dev < kDevices)
    known[dev].store(*pairs, std::memory_order_release);
  return e;
}

}  // namespace

size_t chunk_workspace_bytes(int32_t n, int32_t num_heads, int32_t max_tokens, int64_t max_kv_tokens) {
  Work w;
  return work_of(&w, nullptr, n, max_kv_tokens);
}

cudaError_t launch_chunk_mla(const ChunkArgs& a, void* workspace, uint32_t* err, cudaStream_t stream) {
  Work w;
  work_of(&w, workspace, a.n, a.max_kv_tokens);
  int pairs = 1;
  cudaError_t e = pairs_resident(&pairs);
  CUtensorMap tm_q;
  if (e == cudaSuccess) e = q_map(&tm_q, a.q, (int64_t)a.max_tokens * a.num_heads);
  const bool fold = a.n <= kFoldEntries;
  const int64_t blocks = a.max_kv_tokens / HB, ctas = 10 * (int64_t)pairs;
  const unsigned rows_ctas = (unsigned)(blocks < ctas ? blocks : ctas);
  if (e == cudaSuccess && !fold) e = launch(chunk_list_kernel, dim3(1), kListThreads, 0, stream, a, w, pairs, err);
  if (e == cudaSuccess && (fold || rows_ctas > 0))
    e = launch(fold ? chunk_rows_kernel<true> : chunk_rows_kernel<false>, dim3(rows_ctas + (fold ? 1 : 0)), kRowsThreads, 0, stream, a, w, pairs, err);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)pairs);
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, chunk_mla_kernel, a, w, tm_q, err);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return e;
  }
  // a tile that has less than two of the least parts is not cut
  constexpr int64_t kWhole = (2 * kLeastPart - 1) * BJ;
  if ((int64_t)a.max_blocks * a.page_size <= kWhole || a.max_kv_tokens <= kWhole) return cudaSuccess;
  const int rows = MH / a.num_heads * a.num_heads;
  return launch(chunk_merge_kernel, dim3((unsigned)((rows + kMergeRows - 1) / kMergeRows), (unsigned)pairs),
                kMergeThreads, 0, stream, a, w, pairs);
}

}  // namespace hs
