// MLA decode attention over 4-bit rows on the 5th-generation tensor cores (tcgen05, accumulators in
// tensor memory): through a row table (hs_fp4_sparse_mla_decode) or through a page table for the
// tokens of a sliding window and its sinks (hs_fp4_window_mla_decode).
//
// Per query head over the rows j that it sees:
//   s_j = sm_scale (q[:512] . latent_j + q[512:] . rope_j),  o = softmax(s) . latent,
//   lse = log sum_j exp s_j
//
// Tiles. The 128 rows of an MMA are query heads of one request: all heads of as many of its queries
// as fit (one query of 65 heads or more, eight of 16). A pair of CTAs in a cluster takes units (tile,
// split of the tile's rows), one after the other, and walks each in blocks of 64 rows:
//   - the S-CTA (even rank) holds Q in tensor memory and computes S = Q . K^T of each block into one
//     of three buffers; its softmax warpgroups (a block each in turn, a query head per thread) run the
//     online softmax and write P as f16 into the O-CTA's shared memory;
//   - the O-CTA holds O (128 x 512 in 32 bits, all of its tensor memory) and adds P . V; its
//     corrector rescales O in the rare blocks that raise a head's reference maximum.
// In each CTA eight dequantisation warps bring the records they own (eight rows of each block) into
// shared memory with 16-byte asynchronous copies, two blocks ahead (the O-CTA, whose rows are in L2 by
// then, one), each in a ring of its own that no other warp touches, and write them as f16 into the CTA's tiles. The roles hand blocks over through
// mbarriers with bounded waits. The two halves are on two SMs because Q (288 columns), S and O (512) do
// not fit one tensor memory, nor K, V, Q and P one shared memory; both read every row, the second one
// from L2.
//
// What bounds it (256 requests, 128 heads, 2,048 rows: 159 us, against 42 for its bytes and 74 for its
// operations): a block takes a pair 1.1 us, 0.63 of them the S-CTA's MMAs. The rest is hand-overs: a K
// tile's round (written 0.5 us, handed over 0.3, multiplied 0.63, released 0.2) is 0.85 us a block with
// two tiles, S's and P's 0.8 with three buffers, and shared memory has no room for more; they do not
// overlap perfectly. Timed with parts left out: 155 us instead of 155 (a long window) with a quarter of
// the MMAs, 141 with a quarter of the tiles' writes, 152 with all rows in L2. A unit has ~4 us around its
// blocks (Q, the first block's way through the pipeline, the read-out), 8 us for a first one, 5 more
// with the merge of splits.
//
// Why these copies: a row is 416 bytes anywhere in the pool. Measured per SM, rows from HBM / L2:
// four-row tensor gathers 16 / 24 GB/s from one warp and 20 / 33 from four, a bulk copy per row 24 /
// 31 from four warps (the copy engine's requests in flight bound them), 16-byte asynchronous copies
// 56 / 88 (76 SMs at once). Loads into registers blocks ahead are no faster than the gathers: a
// thread's outstanding loads share a few scoreboards, so that waiting for a block waits for the next.
//
// Precision. code x scale is exact in f16, so K and V hold the latents' exact values but for
// latent_scale, which goes into the scores' scale and the outputs instead. Q's latent part goes
// from bf16 to f16: exact but for values below 2^-14, off by at most 2^-25, which is 2^-19 of the head's
// largest; a head whose largest is below 2^-6 or above 65504 is divided by a power of two, which goes
// into its scores' scale (the values are exact then down to 2^-32 of the largest). RoPE values
// meet Q's in bf16, exact (Q's divided by latent_scale, a power of two), in MMAs of their own type
// that add to the same sums. P, the one operand that has to be rounded, is rounded to f16: by up to
// 2^-11 of a weight (bf16 would cost 2^-8, as much as the output's rounding), and, as f16 has no more
// than 40 binades, by up to 2^-32 of the largest weight where a weight is smaller than 2^-21 of it
// (kRefLog2). Over N such rows, as behind a sink that outweighs each of them, the output may be off
// by N 2^-32 of their latents; split rows have a largest weight per split. The weights' sum takes
// them unrounded, so lse does not see it. Scores, maxima, sums and O are in 32 bits.
//
// NaN and infinities. A row that a query does not see gets P = 0, and 0 x NaN must not reach O: V
// holds zero for a block whose scale is NaN, while K keeps the NaN, which makes the score, the
// weight and so the output NaN for the queries that see the row, and only for them.
#include "hs_fp4.h"
#include "hs_tcgen05.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <atomic>
#include <type_traits>

namespace hs {

using namespace tc;

namespace {

constexpr int T = 736;          // threads per CTA: 23 warps
constexpr int MH = 128;         // MMA M: query heads of a tile (padded with zero rows)
constexpr int BJ = 64;          // rows per block
constexpr int DQK = kFp4Dims, DL = kFp4Latent;
constexpr int QATOMS = DQK / 64, ATOMS = DL / 64;  // swizzle atoms of 64 values in Q and in a tile of latents
constexpr int NT = 2;           // tiles in flight
constexpr int S_ND = 3, O_ND = 2;  // blocks of records in a dequantisation warp's ring: one read, the others on their way
constexpr int NS = 3;           // S buffers, softmax warpgroups and P buffers: a block each in turn
constexpr uint32_t TMEM_COLS = 512, Q_COL = 0, S_COL = 288;
static_assert(S_COL + NS * BJ <= TMEM_COLS, "Q and the S buffers fit tensor memory");
// S-CTA warps: 0-11 softmax, 12 issuer, 13-22 dequantisation; O-CTA: 0-3 corrector, 4 issuer, 5-14
// dequantisation, 15-22 and the corrector's read out. Dequantisation leaves out the warps w % 4 = 0: an
// issuer whose MMAs wait for the tensor core holds up the shared-memory instructions of the warps on its
// scheduler (a window of 8,192 rows took 173 us instead of 155 with one of the S-CTA's eight there, 182
// with two).
constexpr int S_ISSUER = 12, S_DEQ0 = 13;
constexpr int O_ISSUER = 4, O_DEQ0 = 5, O_OUT0 = 15, NOUT = 3;  // NOUT warps read out a quarter of the heads
static_assert(4 + T / 32 - O_OUT0 == 4 * NOUT, "the warps that meet at the read-out's barrier");
constexpr int NDEQ = 8, RW = BJ / NDEQ;  // dequantisation warps of each CTA, eight rows of a block each
constexpr int MASKS = 16;       // blocks whose row masks are kept (the copies are at most 8 ahead of the softmax)

constexpr uint32_t KV_ATOM = BJ * 128, TILE = ATOMS * KV_ATOM;
constexpr uint32_t QBOX = MH * 128;
constexpr int REC = kFp4RopeAt;                    // bytes of a record that go through the rings: codes and scales
constexpr uint32_t S_RING = S_ND * RW * REC, O_RING = O_ND * RW * REC;  // a dequantisation warp's ring
constexpr uint32_t S_TILES = 0;                    // latents of K; Q's are staged over them before the first block
// RoPE values are copied straight to their tiles: a block's copies start when the tensor core is known to
// be done with the block five before it. (Measured when 256 requests took 176 us so: 182 through the rings
// like the rest, 183 with four tiles and so later copies.)
constexpr int NR = 5;
constexpr uint32_t S_ROPE = NT * TILE;             // (Q's are staged over two of them)
constexpr uint32_t S_RAW = S_ROPE + NR * KV_ATOM;
static_assert(ATOMS * QBOX <= NT * TILE && QBOX == 2 * KV_ATOM, "Q's staging");
constexpr uint32_t S_REF = S_RAW + NDEQ * S_RING;  // the reference maxima, handed from block to block
constexpr uint32_t S_MASK = S_REF + MH * 4;     // a byte per block and dequantisation warp: which of its rows exist
constexpr uint32_t S_QTOP = S_MASK + MASKS * NDEQ;  // a head's largest latent in each third of Q, and RoPE value
constexpr uint32_t S_END = S_QTOP + (NS + 1) * MH * 2;
constexpr uint32_t O_TILES = 0, O_RAW = NT * TILE;
constexpr uint32_t O_P = (O_RAW + NDEQ * O_RING + 1023u) & ~1023u;
constexpr uint32_t P_BUF = MH * BJ * 2, P_BYTES = P_BUF + MH * 4;  // P and the rescale factors of a block
constexpr uint32_t FIN_WG = 2 * MH * 4;          // a softmax warpgroup's sums and references of a unit
constexpr uint32_t O_ALPHA = O_P + NS * P_BUF;
constexpr uint32_t O_FIN = O_ALPHA + NS * MH * 4;
constexpr int NF = NS + 1;  // units whose totals are kept: P's buffers let the S-CTA be three units ahead, of one block each
constexpr uint32_t O_END = O_FIN + NF * NS * FIN_WG;
constexpr uint32_t SMEM_BYTES = S_END > O_END ? S_END : O_END;
constexpr uint32_t STATIC_BYTES = 1024;  // barriers and flags, one block of a tile's alignment
static_assert(STATIC_BYTES + SMEM_BYTES <= 227 * 1024, "shared memory of a CTA");
// P of a score that equals its reference is 2^7, and a reference stays until it is passed by 2^8.9, so that
// P < 2^15.91 = 61,500 in f16, which then keeps a weight to 2^-11 of itself down to 2^-21 of the
// reference's, and to 2^-32 of the reference's below that. Room below the reference is taken from the room
// above it, where too little costs rescales, ~2 us each (us, 256 requests of 2,048 rows / a window of
// 8,192): 161 / 156 with 0 and 15, 160 / 158 with 7 and 8.9, 167 / 162 with 8 and 7, 220 / 191 with 10 and 5.
constexpr float kRefLog2 = 7.f, kRescaleLog2 = 8.9f;
constexpr uint32_t kIdescQK = idesc(BJ, MH, false);                              // f16 latents
constexpr uint32_t kIdescRope = kIdescQK | (1u << 7) | (1u << 10);               // bf16 RoPE
constexpr uint32_t kIdescPV = idesc(256, MH, true);

struct Barriers {
  uint64_t tile_full[NT], tile_free[NT];  // dequantisation <-> issuer
  uint64_t q_raw[NS], q_full;             // S-CTA: a third of Q staged; Q in tensor memory
  // per softmax warpgroup, so that whoever waits on one waits on every phase of it (parities repeat):
  uint64_t s_full[NS], s_free[NS];        // S-CTA: S written; S read
  uint64_t m_set[NS][4];                  // S-CTA: the block's reference maxima of a warp's heads are set
  uint64_t p_free[NS];                    // S-CTA, arrived by the O-CTA: P . V of the block is done
  uint64_t p_full[NS];                    // O-CTA, completed by the S-CTA's stores
  uint64_t pv_go[NS];                     // O-CTA: O is ready for P . V of the block
  uint64_t fin[NF];                       // O-CTA: the S-CTA's totals of a unit are here
  uint64_t o_full, o_free;                // O-CTA: a unit's last P . V is done; O has been read out
};

struct __align__(STATIC_BYTES) Control {
  Barriers bs;
  uint32_t taddr;
  int abort;
  int issued;     // blocks whose MMAs the issuer started (the last commit to wait for)
  int requested;  // units whose Q was requested
};
static_assert(sizeof(Control) == STATIC_BYTES, "one block");

// What a unit of a score without its scales is in log2 units.
__device__ __forceinline__ float score_log2(const Fp4MlaArgs& a) {
  return fabsf(a.sm_scale * a.latent_scale * 1.4426950408889634f);
}
// The power of two that a head's Q is divided by, given the bf16 bits of its largest latent and RoPE value. 1 where f16
// holds its latents: none over 65504, and what is lost (2^-25 of values below 2^-14) at most 2^-19 of the largest.
// Otherwise the largest becomes 2^15 .. 65280. RoPE values are divided too, in bf16, and over latent_scale >= 2^-32: so
// that none of them overflows, the divisor is at least 2^-75 of the largest one, which takes room from latents
// only where RoPE values are more than 2^60 times as large, and at least 2^-95.
__device__ __forceinline__ float q_divisor(uint32_t top, uint32_t rope) {
  if (top == 0 || (top >= 0x3C80u && top < 0x4780u)) return 1.f;  // 2^-6, 2^16
  return __uint_as_float((uint32_t)max(max((int)(top >> 7) - 15, (int)(rope >> 7) - 75), 127 - 95) << 23);
}
// The rows of a tile's split, j = 0 .. n - 1, and who sees them.
template <bool kWin>
struct Rows {
  const int32_t* table;  // the request's rows, or its pages
  uint32_t pool_rows, pool_pages;  // below 2^31; window: pages that begin inside the pool
  int n, j0;  // rows of this split; the split's first row in the tile's list (j unsigned: past n it may pass 2^31)
  // window: the list is tokens 0 .. kept - 1, then from `start`
  int kept, start, page_size;
  uint32_t page_mul, page_shift;  // t / page_size = t page_mul >> page_shift for 0 <= t < 2^31

  __device__ __forceinline__ int token(uint32_t j) const {
    const int i = (int)((uint32_t)j0 + j);
    return i < kept ? i : (int)((uint32_t)start + (uint32_t)(i - kept));
  }
  __device__ __forceinline__ int page_of(int t) const { return (int)((uint64_t)(uint32_t)t * page_mul >> page_shift); }
  // what the table holds for row j (loaded ahead), and the pool row that it means (-1: none)
  __device__ __forceinline__ int32_t raw(uint32_t j) const {
    if (j >= (uint32_t)n) return -1;
    return __ldg(table + (kWin ? page_of(token(j)) : j0 + (int)j));
  }
  __device__ __forceinline__ int32_t row(int32_t raw, uint32_t j) const {
    if (!kWin) return (uint32_t)raw < pool_rows ? raw : -1;
    const int t = token(j), page = page_of(t);
    const uint32_t r = (uint32_t)(raw - page) * (uint32_t)page_size + (uint32_t)t;  // below 2^32 for a page inside
    return (uint32_t)raw < pool_pages && r < pool_rows ? (int32_t)r : -1;
  }
};

// Four bytes of codes (a pair of dims each, low nibble first) to four f16 pairs.
__device__ __forceinline__ uint4 codes_to_f16(uint32_t w) {
  uint4 h;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h.x), "=r"(h.y), "=r"(h.z), "=r"(h.w)
      : "r"(w));
  return h;
}
__device__ __forceinline__ uint4 times(uint4 v, __half2 s) {
  uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&x[i]), s);
    x[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// A dequantisation warp's copies of a block: its eight rows' codes and scales into a slot of its ring,
// eight lanes of 16 bytes to a row, four rows at a time: 128 consecutive bytes of each, which meet
// every bank once, and addresses that are one register and a constant. In the S-CTA the RoPE values go
// straight to their places in their tile, chunk c of row x of eight at c ^ x. Rows that do not exist
// become zeros. y: lane l has row l % 8 (-1: none); dst, rope: this lane's places.
template <bool kS>
__device__ __forceinline__ void copy_rows(uint32_t dst, uint32_t rope, int32_t y, const uint8_t* __restrict__ pool, int lane) {
  const auto copy16 = [](uint32_t to, const uint8_t* from, int size) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(size) : "memory");
  };
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int32_t row = __shfl_sync(0xffffffffu, y, 4 * g + (lane >> 3));
    const uint8_t* src = pool + (int64_t)max(row, 0) * kFp4Row + 16 * (lane & 7);
    const int size = row >= 0 ? 16 : 0;
    copy16(dst + 4 * g * REC, src, size);
    copy16(dst + 4 * g * REC + 128, src + 128, size);
    if ((lane & 7) < 2) copy16(dst + 4 * g * REC + 256, src + 256, size);
    if (kS) copy16(g ? (rope ^ 64u) + 512u : rope, src + kFp4RopeAt, size);
  }
}

// What a lane reads of its warp's eight rows. Step s covers four rows (4 (s / 2) ..) and half of
// their latent dims: lane = (row of the four, 32 dims `it`), placed so that the eight lanes of a load
// or store phase have four rows and both halves of a line: the reads (rows 288 bytes apart) and,
// through the tile's swizzle, the writes then meet every bank once.
struct Held {
  uint4 codes[4];
  uint16_t scales[4];
};
__device__ __forceinline__ Held read_rows(const uint8_t* slot, int lane) {
  Held h;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint8_t* rec = slot + (4 * (s >> 1) + ((lane >> 1) & 3)) * REC;
    const int it = (lane & 1) + 2 * (lane >> 3) + 8 * (s & 1);
    h.codes[s] = *reinterpret_cast<const uint4*>(rec + 16 * it);
    h.scales[s] = *reinterpret_cast<const uint16_t*>(rec + kFp4Scales + 2 * it);
  }
  return h;
}

// Writes them into the tile, as f16, at the warp's group of eight rows. The place of chunk c of row x
// of a line's eight is c ^ x: of a lane's four chunks it is one address with two bits flipped.
template <bool kS>
__device__ __forceinline__ void write_rows(const Held& h, uint8_t* group, int lane) {
  const int in4 = (lane >> 1) & 3;
  const uint32_t at0 = smem_u32(group) + (lane >> 3) * KV_ATOM + in4 * 128 + (lane & 1) * 64 + in4 * 16;
  const uint32_t at1 = (at0 ^ 64u) + 512u;
  uint32_t scales[4] = {h.scales[0], h.scales[1], h.scales[2], h.scales[3]};
  if (!kS) {  // V: zeros for NaN (0x7F, 0xFF; see above), which are few: one look at all of them. K keeps it
    const uint32_t x = (((scales[0] | scales[1] << 16) & 0x7F7F7F7Fu) + 0x01010101u) |
                       (((scales[2] | scales[3] << 16) & 0x7F7F7F7Fu) + 0x01010101u);
    if (x & 0x80808080u)
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if ((scales[s] & 0x7Fu) == 0x7Fu) scales[s] &= 0xFF00u;
        if ((scales[s] & 0x7F00u) == 0x7F00u) scales[s] &= 0xFFu;
      }
  }
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint32_t w[4] = {h.codes[s].x, h.codes[s].y, h.codes[s].z, h.codes[s].w};
    const __half2_raw raw = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)scales[s], __NV_E4M3);  // of 16 dims each
    const __half2 pair = raw, sc[2] = {__low2half2(pair), __high2half2(pair)};
    uint4 v[4];  // the lane's 32 dims, a chunk of eight each
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = times(codes_to_f16(w[u]), sc[u >> 1]);
    if (!kS) {  // V: chunk j takes pair j of each, the order of columns that the read-out wants
      const uint4 a = v[0], b = v[1], c = v[2], d = v[3];
      v[0] = make_uint4(a.x, b.x, c.x, d.x);
      v[1] = make_uint4(a.y, b.y, c.y, d.y);
      v[2] = make_uint4(a.z, b.z, c.z, d.z);
      v[3] = make_uint4(a.w, b.w, c.w, d.w);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(((s >> 1 ? at1 : at0) ^ (uint32_t)(u << 4)) + (s & 1) * 4 * KV_ATOM),
                   "r"(v[u].x), "r"(v[u].y), "r"(v[u].z), "r"(v[u].w)
                   : "memory");
  }
}

// A dequantisation warp's loop over a unit's blocks: block b is written while the rows of the next
// ND - 1 blocks are on their way, and two more blocks' row numbers. `done`: blocks of the units before
// (places in rings go on from unit to unit). In the S-CTA it waits, before its first tile write, until Q
// has left the staging area, and tells the softmax which of its rows exist. A block's copies start once
// the tensor core has read the block five before it, whose RoPE tile they go to.
template <bool kS, bool kWin>
__device__ __forceinline__ bool run_dequant(const Rows<kWin>& rows, const uint8_t* __restrict__ pool, int nblk, int done,
                                            uint32_t q_phase, uint8_t* ring, uint8_t* rope, uint8_t* masks, uint8_t* tiles,
                                            Barriers& bs, int wq, int lane, uint32_t* err, volatile int* abort) {
  constexpr int ND = kS ? S_ND : O_ND;
  const uint32_t own = RW * wq + (lane & 7);
  auto of_block = [own](int b) { return (uint32_t)b * BJ + own; };  // this lane's row
  bool missing = false, ok = true;
  // slots of the ring: the next one to fill, and the next one to read
  const uint32_t ring0 = smem_u32(ring) + (lane >> 3) * REC + 16 * (lane & 7), ring_end = ring0 + ND * RW * REC;
  const uint32_t rope0 = kS ? smem_u32(rope) + RW * wq * 128 + (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4) : 0u;
  uint32_t fill = ring0, rope_fill = rope0 + done % NR * KV_ATOM;
  const uint8_t* read = ring;
  auto start = [&](int32_t raw, int b) {  // the copies of block b (one group of copies, empty past the end)
    if (b < nblk) {
      const uint32_t j = of_block(b);
      const int32_t y = rows.row(raw, j);
      if (kS) {
        if (kWin) missing |= j < (uint32_t)rows.n && y < 0;
        const uint32_t mask = __ballot_sync(0xffffffffu, y >= 0);
        if (lane == 0) masks[((done + b) % MASKS) * NDEQ + wq] = (uint8_t)mask;
      }
      copy_rows<kS>(fill, rope_fill, y, pool, lane);
      rope_fill += KV_ATOM;
      if (rope_fill == rope0 + NR * KV_ATOM) rope_fill = rope0;
      fill += RW * REC;
      if (fill == ring_end) fill = ring0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  static_assert(NT == 2 && NR >= S_ND + NT, "a block's RoPE tile is free when its copies start");
  static_assert(S_ND == 3 && O_ND == 2, "so many blocks' copies are started here");
  const int32_t t0 = rows.raw(of_block(0)), t1 = kS ? rows.raw(of_block(1)) : -1;
  int32_t t2 = rows.raw(of_block(ND - 1)), t3 = rows.raw(of_block(ND));  // the two blocks' after these
  start(t0, 0);
  if (kS) start(t1, 1);
#pragma unroll 1
  for (int b = 0; b < nblk; ++b) {
    const int g = done + b;
    start(t2, b + ND - 1);  // into the slot that block b - 1 was read from
    t2 = t3;
    t3 = rows.raw(of_block(b + ND + 1));
    asm volatile("cp.async.wait_group %0;" ::"n"(ND - 1) : "memory");
    __syncwarp();
    const Held held = read_rows(read, lane);
    read = read + RW * REC == ring + ND * RW * REC ? ring : read + RW * REC;
    if (kS && b == 0) ok = ready_or_wait(&bs.q_full, 1, (int)q_phase, abort);
    if (g >= NT) ok = ok && ready_or_wait(bs.tile_free, NT, g - NT, abort);
    ok = __all_sync(0xffffffffu, ok);  // (and the slot has been read)
    if (!ok) break;
    write_rows<kS>(held, tiles + (g % NT) * TILE + wq * 1024, lane);
    __syncwarp();  // (the issuer has the proxy fence: here it would wait for the copies in flight too)
    if (lane == 0) bar_arrive(&bs.tile_full[g % NT]);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // none is left in flight at the end
  __syncwarp();
  if (kS && kWin && __any_sync(0xffffffffu, missing) && lane == 0) atomicOr(err, HS_FLAG_DEVROW);
  return ok;
}

// The dequantisation warp that CTA warp w is, of those that begin with warp `first` (first % 4 = 1);
// -1 if none.
__device__ __forceinline__ int deq_warp(int w, int first) {
  const int i = w - first, q = 3 * (i >> 2) + (i & 3);
  return i >= 0 && (i & 3) != 3 && q < NDEQ ? q : -1;
}

// The tiles' numbers: the first `whole` tiles are a unit each, the others, whose query heads begin with
// row `split_row` of q, o and lse and are `split_rows`, a unit per split.
struct Tiles {
  int per_request, queries;  // of a request; of a tile
  int units, whole, split_row, split_rows;
};

// A unit of work: a tile or one of its splits. Every thread of a pair computes it from its number.
template <bool kWin>
struct Unit {
  Rows<kWin> rows;
  int nblk;          // blocks of this split
  int live;          // query heads of the tile
  size_t row0;       // the first one's row of q, o and lse
  int splits, p;     // the tile's, and this one
  int first_query;
  int64_t seq_len;   // window
};
template <bool kWin>
__device__ __forceinline__ Unit<kWin> unit_of(const Fp4MlaArgs& a, const Tiles& ts, int u, bool flag, uint32_t* err) {
  Unit<kWin> x;
  // (divisions are long: none where there is nothing to divide)
  int tile = u;
  x.splits = 1;
  x.p = 0;
  if (u >= ts.whole) {
    const int v = u - ts.whole, q = v / a.splits;
    x.splits = a.splits;
    x.p = v - q * a.splits;
    tile = ts.whole + q;
  }
  int r = tile;
  x.first_query = 0;
  if (ts.per_request > 1) {
    r = tile / ts.per_request;
    x.first_query = (tile - r * ts.per_request) * ts.queries;
  }
  const int nq = min(ts.queries, a.num_queries - x.first_query);
  x.live = nq * a.num_heads;
  x.row0 = ((size_t)r * a.num_queries + x.first_query) * a.num_heads;
  // the tile's rows: every row that some query of the tile sees
  x.rows.pool_rows = (uint32_t)a.pool_rows;
  int total;
  if (kWin) {
    x.rows.table = a.pages + (size_t)r * a.max_pages;
    x.rows.page_size = a.page_size;
    x.rows.pool_pages = a.pool_pages;
    x.rows.page_mul = a.page_mul;
    x.rows.page_shift = a.page_shift;
    x.seq_len = a.seq_lens[r];
    const bool bad = x.seq_len < 0 || x.seq_len > (int64_t)a.max_pages * a.page_size;
    if (bad && flag) atomicOr(err, HS_FLAG_SEQLEN);
    // tokens up to the tile's last query, from the first one of its first query
    const int64_t at = x.seq_len - a.num_queries + x.first_query;
    const int64_t end = bad ? 0 : max((int64_t)0, at + nq), first = max((int64_t)0, at);
    x.rows.kept = (int)min((int64_t)a.sinks, end);
    x.rows.start = (int)max((int64_t)x.rows.kept, first + 1 - a.window);
    total = x.rows.kept + (int)max((int64_t)0, end - x.rows.start);
  } else {
    x.rows.table = a.out_rows + (size_t)r * a.top_k;
    total = a.top_k;
  }
  const int all = (int)(((int64_t)total + BJ - 1) / BJ), per = x.splits == 1 ? all : (all + x.splits - 1) / x.splits;
  x.nblk = max(0, min(per, all - x.p * per));
  x.rows.j0 = x.p * per * BJ;
  x.rows.n = x.nblk > 0 ? (int)min((int64_t)total - x.rows.j0, (int64_t)x.nblk * BJ) : 0;
  return x;
}

// Where half a box of Q (64 rows of 64 dims) is staged: the latents' over the K tiles, the RoPE values'
// over the RoPE tiles of two of the unit's blocks (g0: the number of its first one), whose copies start
// when Q is in tensor memory: those of the first S_ND blocks may be on their way before.
static_assert(NR >= S_ND + 2, "Q's two staged tiles are none of those that a unit's first copies go to");
__device__ __forceinline__ uint32_t q_stage(int bx, int half, int g0) {
  return bx < ATOMS ? S_TILES + bx * QBOX + half * KV_ATOM : S_ROPE + (g0 + S_ND + half) % NR * KV_ATOM;
}
// Q's 128 rows from row0 as tensor boxes of 64 rows and dims, a third of the dims to a barrier (rows past
// the tile's are not used).
__device__ __forceinline__ void request_q(const CUtensorMap* tm_q, size_t row0, int g0, uint8_t* base, Barriers& bs) {
  fence_async_smem();  // earlier generic accesses of the staging area and the barriers, before the copies
  for (int g = 0; g < NS; ++g) {
    bar_arrive_tx(&bs.q_raw[g], QATOMS / NS * QBOX);
    for (int i = 2 * (QATOMS / NS) * g; i < 2 * (QATOMS / NS) * (g + 1); ++i)
      asm volatile(
          "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
              smem_u32(base + q_stage(i >> 1, i & 1, g0))),
          "l"(tm_q), "r"(64 * (i >> 1)), "r"((int)row0 + BJ * (i & 1)), "r"(smem_u32(&bs.q_raw[g]))
          : "memory");
  }
}

// The same boxes into L2, a unit ahead.
__device__ __forceinline__ void prefetch_q(const CUtensorMap* tm_q, size_t row0) {
  for (int i = 0; i < 2 * QATOMS; ++i)
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(tm_q), "r"(64 * (i >> 1)), "r"((int)row0 + BJ * (i & 1))
                 : "memory");
}

template <bool kWin>
__global__ void __launch_bounds__(T, 1)
    fp4_mla_kernel(const Fp4MlaArgs a, const Tiles ts,
                   const __grid_constant__ CUtensorMap tm_q, float* __restrict__ part_o, float* __restrict__ part_lse,
                   uint32_t* __restrict__ err) {
  // (what is static fills a block of the tiles' alignment, and the rest begins after it)
  extern __shared__ __align__(STATIC_BYTES) uint8_t base[];
  __shared__ __align__(STATIC_BYTES) Control ctl;
  Barriers& bs = ctl.bs;
  uint32_t& s_taddr = ctl.taddr;
  int &s_abort = ctl.abort, &s_issued = ctl.issued, &s_requested = ctl.requested;
  if ((smem_u32(base) & (STATIC_BYTES - 1)) != 0) {  // (never: the tiles' swizzle wants it)
    if (threadIdx.x == 0) atomicOr(err, HS_FLAG_TIMEOUT);
    return;
  }
  volatile int* abort = &s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = blockIdx.x & 1u, partner = rank ^ 1u;  // 0: S-CTA, 1: O-CTA
  const int pairs = gridDim.x >> 1;

  if (tid == 0) {
    for (int k = 0; k < NT; ++k) {
      bar_init(&bs.tile_full[k], NDEQ);
      bar_init(&bs.tile_free[k], 1);
    }
    for (int k = 0; k < NS; ++k) {
      bar_init(&bs.q_raw[k], 1);
      bar_init(&bs.s_full[k], 1);
      bar_init(&bs.s_free[k], 4);  // the warps of the block's softmax warpgroup
      for (int w = 0; w < 4; ++w) bar_init(&bs.m_set[k][w], 1);
      bar_init(&bs.p_free[k], 1);
    }
    bar_init(&bs.q_full, 4 * NS);  // one arrival per softmax warp
    for (int k = 0; k < NS; ++k) {
      bar_init(&bs.p_full[k], 1);  // the O-CTA's expect_tx; the S-CTA's stores complete it
      bar_init(&bs.pv_go[k], 4);
    }
    for (int k = 0; k < NF; ++k) bar_init(&bs.fin[k], 1);  // the same
    bar_init(&bs.o_full, 1);
    bar_init(&bs.o_free, 4 * NOUT);
    s_abort = 0;
    s_issued = 0;
    s_requested = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_wait();
    if (rank == 0) {
      const Unit<kWin> first = unit_of<kWin>(a, ts, blockIdx.x >> 1, false, err);
      if (first.nblk > 0) {
        request_q(&tm_q, first.row0, 0, base, bs);
        s_requested = 1;
      }
    } else {
      for (int k = 0; k < NS; ++k) bar_arrive_tx(&bs.p_full[k], P_BYTES);
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_taddr)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  // both CTAs' barriers are initialised before either arrives on the other's (the initialiser's fence
  // makes them visible: the barrier itself need not wait for anything)
  asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  pdl_wait();
  const uint32_t tbase = s_taddr;
  const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
  const int head = (warp & 3) * 32 + lane;  // this thread's row of the tile = its tensor-memory lane
  uint8_t* masks = base + S_MASK;

  // The units of this pair, one after the other. Each role goes through them by itself: what the roles
  // hand each other carries on from unit to unit, so that a unit's first blocks are brought in while
  // the last one's end is computed and read out.
  bool ok = true;
  int done = 0, full = 0;  // blocks, and units with blocks, before this one
#pragma unroll 1
  for (int u = blockIdx.x >> 1; u < ts.units; u += pairs) {
    const Unit<kWin> un = unit_of<kWin>(a, ts, u, tid == 0, err);
    const int nblk = un.nblk;
    if (rank == 0) {
      // ================================ S-CTA ================================
      uint8_t* tiles = base + S_TILES;
      const uint32_t q_phase = (uint32_t)full & 1u;
      float m_own = -INFINITY, l_own = 0.f;  // softmax: the sum of this thread's blocks, under this reference
      if (warp < 4 * NS) {
        const int wg = warp >> 2;
        float up = 1.f;  // what this head's Q is divided by
        if (nblk > 0) {
          // Q into tensor memory (warpgroup wg the columns [96 wg, 96 wg + 96)), column c holding dims
          // 2c, 2c + 1: the latent part as f16, the RoPE part as bf16 over latent_scale. Q has landed
          // only after the last unit's MMAs, which read the columns. It is taken as it is first, and once
          // more where some head's latents do not fit f16 so (3 us more a unit; the look costs nothing that shows).
          ok = __all_sync(0xffffffffu, ready_or_wait(&bs.q_raw[wg], 1, (int)q_phase, abort));
          tc_after();
          const bool live = ok && head < un.live;
          const uint32_t sign = a.sm_scale < 0.f ? 0x80008000u : 0u;  // so that scores scale by a positive factor
          const auto box = [&](int bx) { return base + q_stage(bx, head >> 6, done) + (head & 63) * 128; };
          const auto take = [&](auto divide, float down) {  // the largest magnitude in f16 of this third's latents
            constexpr bool kDivide = decltype(divide)::value;
            const float inv = down / a.latent_scale;
            __half2 top = __float2half2_rn(0.f);
#pragma unroll 1
            for (int bx = QATOMS / NS * wg; bx < QATOMS / NS * (wg + 1); ++bx) {
              const uint8_t* src = box(bx);
#pragma unroll
              for (int h = 0; h < 4; ++h) {  // two 16-B chunks: 16 dims, 8 columns
                uint32_t x[8] = {};
                if (live) {
                  *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(src + (((2 * h) ^ (head & 7)) << 4));
                  *reinterpret_cast<uint4*>(x + 4) = *reinterpret_cast<const uint4*>(src + (((2 * h + 1) ^ (head & 7)) << 4));
                }
                if (bx < ATOMS) {
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    const float lo = __uint_as_float(x[i] << 16), hi = __uint_as_float(x[i] & 0xFFFF0000u);
                    const __half2 v = kDivide ? __floats2half2_rn(lo * down, hi * down) : __floats2half2_rn(lo, hi);
                    if (!kDivide) top = __hmax2(top, __habs2(v));
                    x[i] = *reinterpret_cast<const uint32_t*>(&v) ^ sign;
                  }
                } else {
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    const __nv_bfloat162 v =
                        __floats2bfloat162_rn(__uint_as_float(x[i] << 16) * inv, __uint_as_float(x[i] & 0xFFFF0000u) * inv);
                    x[i] = *reinterpret_cast<const uint32_t*>(&v) ^ sign;
                  }
                }
                asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                                 tbase + lane_off + Q_COL + 32 * bx + 8 * h),
                             "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                             : "memory");
              }
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            return fmaxf(__low2float(top), __high2float(top));
          };
          const float top = take(std::false_type{}, 1.f);
          // a third that is too large, or so small that the head may be: all of it is looked at (every softmax warp
          // comes to these barriers, whether its wait ended well or not)
          if (sync_or<2>(live && !(top >= 0x1p-6f && top < 65504.f), 4 * NS * 32)) {
            uint16_t* tops = reinterpret_cast<uint16_t*>(base + S_QTOP) + head;
            uint32_t lat = 0, rope = 0;  // two lanes of 16 bits
#pragma unroll 1
            for (int bx = QATOMS / NS * wg; bx < QATOMS / NS * (wg + 1); ++bx)
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                const uint4 x = *reinterpret_cast<const uint4*>(box(bx) + ((c ^ (head & 7)) << 4));
                if (bx < ATOMS) lat = max_bf16x2(lat, x);
                else rope = max_bf16x2(rope, x);
              }
            tops[MH * wg] = (uint16_t)max(lat & 0xFFFFu, lat >> 16);
            if (wg == NS - 1) tops[MH * NS] = (uint16_t)max(rope & 0xFFFFu, rope >> 16);
            sync_n<2>(4 * NS * 32);
            up = q_divisor(max(max((uint32_t)tops[0], (uint32_t)tops[MH]), (uint32_t)tops[2 * MH]), tops[3 * MH]);
            if (__any_sync(0xffffffffu, live && up != 1.f)) take(std::true_type{}, 1.f / up);
          }
          tc_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&bs.q_full);
        }
        // window: this query sees the list's rows [0, see_kept) and [see_lo, see_hi)
        int see_kept = 0, see_lo = 0, see_hi = 0;
        if (kWin) {
          const int64_t at = un.seq_len - a.num_queries + un.first_query + head / a.num_heads;  // its token
          see_kept = (int)min((int64_t)un.rows.kept, at + 1) - un.rows.j0;
          see_lo = (int)(un.rows.kept + max((int64_t)0, at + 1 - a.window - un.rows.start)) - un.rows.j0;
          see_hi = (int)(un.rows.kept + max((int64_t)0, at + 1 - un.rows.start)) - un.rows.j0;
        }
        // Warpgroup wg takes the blocks whose number g = done + b has g % NS = wg, a query head per
        // thread. From one block to the next only the reference maximum goes over, from warp to warp
        // (the warps of the same heads): it is known once a block's scores have been read, so the
        // warpgroups' exponentials overlap. Each keeps the sum of its own blocks under the reference of
        // its last one. The scores are read twice, for the maximum and for the weights. References are
        // scores as S holds them, and a weight's exponent is the difference, scaled: a score times the scale
        // is rounded by whole units from 2^24 on, so that scaled scores less a scaled reference made a
        // weight of its own reference 2^16 or 0 instead of 1.
        float* s_ref = reinterpret_cast<float*>(base + S_REF);
        const uint32_t pbuf = remote(base + O_P + wg * P_BUF, partner);  // (block g's buffer is g % NS = wg)
        const uint32_t r_alpha = remote(base + O_ALPHA + 4 * (wg * MH + head), partner), rbar = remote(&bs.p_full[wg], partner);
        // what a unit of S is; a scale of zero stays above it, so that -inf stays -inf
        const float sl2 = fminf(fmaxf(score_log2(a) * up, 1e-37f), 3e38f);
        const uint32_t s_at = tbase + lane_off + S_COL + BJ * wg;
        int b = wg - done % NS;
        if (b < 0) b += NS;
        const bool mine = b < nblk;  // it has a block of this unit
        uint32_t turn = (uint32_t)((done + b) / NS) & 1u;  // of this warpgroup: its barriers' phase
#pragma unroll 1
        for (; ok && b < nblk; b += NS, turn ^= 1u) {
          const int g = done + b;
          ok = __all_sync(0xffffffffu, ready_or_wait(&bs.s_full[wg], 1, (int)turn, abort));
          if (!ok) break;
          tc_after();
          // the rows that exist, and that this query sees
          const volatile uint32_t* at = reinterpret_cast<const volatile uint32_t*>(masks + (g % MASKS) * NDEQ);
          uint32_t sees0 = at[0], sees1 = at[1];
          if (kWin) {
            const int j = BJ * b;
            sees0 &= bit_range(0, see_kept - j) | bit_range(see_lo - j, see_hi - j);
            sees1 &= bit_range(0, see_kept - j - 32) | bit_range(see_lo - j - 32, see_hi - j - 32);
          }
          const bool every = __all_sync(0xffffffffu, (sees0 & sees1) == 0xFFFFFFFFu);
          const auto scores = [&](int c, float (&t)[32]) {  // 32 c .. 32 c + 31 of the block, -inf where it does not look
            tmem_ld32(s_at + 32 * c, t);
            if (!every) {
              const uint32_t sees = c ? sees1 : sees0;
#pragma unroll
              for (int i = 0; i < 32; ++i) t[i] = ((sees >> i) & 1u) ? t[i] : -INFINITY;
            }
          };
          float bm = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < BJ / 32; ++c) {
            float t[32];
            scores(c, t);
            float x0 = t[0], x1 = t[1];
#pragma unroll
            for (int i = 2; i < 32; i += 2) {
              x0 = fmaxf(x0, t[i]);
              x1 = fmaxf(x1, t[i + 1]);
            }
            bm = fmaxf(bm, fmaxf(x0, x1));
          }
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
          // the O-CTA's P buffer is free once P . V of block g - 3 is done
          ok = __all_sync(0xffffffffu, g < NS || ready_or_wait<true>(bs.p_free, NS, g - NS, abort));
          if (!ok) break;
          st_async_f32(r_alpha, alpha, rbar);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int c = 0; c < BJ / 32; ++c) {
            float t[32];
            scores(c, t);
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // four 16-B chunks of 8 f16
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float2 e = fma2(add2(make_float2(t[8 * q + 2 * i], t[8 * q + 2 * i + 1]), make_float2(-ref, -ref)),
                                make_float2(sl2, sl2), make_float2(kRefLog2, kRefLog2));
                e = make_float2(ex2(e.x), ex2(e.y));
                const __half2 pb = __floats2half2_rn(e.x, e.y);
                sum = add2(sum, e);
                w[i] = *reinterpret_cast<const uint32_t*>(&pb);
              }
              st_async16(pbuf + sw128(head, 32 * c + 8 * q), make_uint4(w[0], w[1], w[2], w[3]), rbar);
            }
          }
          tc_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&bs.s_free[wg]);  // S has been read
          l_own += sum.x + sum.y;
        }
        // its sum, under the reference of its last block, to the O-CTA
        if (ok && mine) {
          const uint32_t fin = remote(base + O_FIN, partner) + ((full % NF) * NS + wg) * FIN_WG;
          const uint32_t bar = remote(&bs.fin[full % NF], partner);
          st_async_f32(fin + 4 * head, l_own, bar);
          st_async_f32(fin + 4 * (MH + head), m_own * up, bar);  // a score again, exact
        }
      } else if (warp == S_ISSUER) {
        // (tensor memory starts at 0: all of it is allocated here)
        const bool one = elected();
        const uint64_t k0 = mdesc(smem_u32(base + S_TILES), 16, 1024), r0 = mdesc(smem_u32(base + S_ROPE), 16, 1024);
        const bool more = u + pairs < ts.units;
        Unit<kWin> next;
        next.nblk = 0;
        if (more) next = unit_of<kWin>(a, ts, u + pairs, false, err);
        if (one && next.nblk > 0) prefetch_q(&tm_q, next.row0);
        bool go = __all_sync(0xffffffffu, nblk == 0 || ready_or_wait(&bs.q_full, 1, (int)q_phase, abort));
#pragma unroll 1
        for (int b = 0; go && b < nblk; ++b) {
          const int g = done + b;
          go = ready_or_wait(bs.tile_full, NT, g, abort);
          go = go && (g < NS || ready_or_wait(bs.s_free, NS, g - NS, abort));
          go = __all_sync(0xffffffffu, go);
          if (!go) break;
          tc_after();
          fence_async_smem();  // the tile's generic writes, seen through its barrier, before the tensor core's reads
          const uint64_t dk0 = k0 + (uint64_t)((g % NT) * (TILE >> 4)), dr0 = r0 + (uint64_t)((g % NR) * (KV_ATOM >> 4));
          const uint32_t d = S_COL + BJ * (g % NS);
          if (one) {
#pragma unroll
            for (int kk = 0; kk < QATOMS * 4; ++kk)
              mma_ta(d, Q_COL + 8 * kk,
                     kk < DL / 16 ? dk0 + (uint64_t)(((kk >> 2) * KV_ATOM + (kk & 3) * 32) >> 4) : dr0 + (uint64_t)(((kk & 3) * 32) >> 4),
                     kk < DL / 16 ? kIdescQK : kIdescRope, kk > 0);
            commit(&bs.s_full[g % NS]);
            commit(&bs.tile_free[g % NT]);
            s_issued = g + 1;
          }
          __syncwarp();
        }
        // the next unit's Q, once this one's MMAs have read the tiles that it is staged over
        if (go && next.nblk > 0) {
          const int last = done + nblk - 1;
          go = __all_sync(0xffffffffu, last < 0 || ready_or_wait(bs.tile_free, NT, last, abort));
          if (go && one) {
            request_q(&tm_q, next.row0, done + nblk, base, bs);
            ++s_requested;
          }
          __syncwarp();
        }
        ok = go;
      } else if (const int wq = deq_warp(warp, S_DEQ0); wq >= 0) {
        ok = run_dequant<true, kWin>(un.rows, a.pool, nblk, done, q_phase, base + S_RAW + wq * S_RING, base + S_ROPE, masks, tiles, bs, wq,
                                     lane, err, abort);
      }
    } else {
      // ================================ O-CTA ================================
      uint8_t* tiles = base + O_TILES;
      const float* alpha_buf = reinterpret_cast<const float*>(base + O_ALPHA);
      const bool out_warp = warp < 4 || warp >= O_OUT0;
      if (warp < 4) {
        // corrector: where a reference maximum of the warp's heads rose, rescale O once P . V of the
        // block before is done
#pragma unroll 1
        for (int b = 0; ok && b < nblk; ++b) {
          const int g = done + b;
          ok = __all_sync(0xffffffffu, ready_or_wait<true>(bs.p_full, NS, g, abort));
          if (!ok) break;
          const float f = alpha_buf[g % NS * MH + head];
          // this buffer's next phase is block g + 3: its bytes come only after P . V of block g
          if (tid == 0) bar_arrive_tx(&bs.p_full[g % NS], P_BYTES);
          if (__any_sync(0xffffffffu, b > 0 && f != 1.f)) {
            ok = __all_sync(0xffffffffu, ready_or_wait(bs.tile_free, NT, g - 1, abort));
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
          if (lane == 0) bar_arrive(&bs.pv_go[g % NS]);
        }
      } else if (warp == O_ISSUER) {
        const bool one = elected();
        const uint64_t p0 = mdesc(smem_u32(base + O_P), 16, 1024), v0 = mdesc(smem_u32(base + O_TILES), KV_ATOM, 1024);
#pragma unroll 1
        for (int b = 0; b < nblk; ++b) {
          const int g = done + b;
          bool go = ready_or_wait(bs.tile_full, NT, g, abort);
          go = go && ready_or_wait(bs.pv_go, NS, g, abort);
          if (b == 0) go = go && (full == 0 || ready_or_wait(&bs.o_free, 1, full - 1, abort));
          ok = __all_sync(0xffffffffu, go);
          if (!ok) break;
          tc_after();
          fence_async_smem();  // V's and P's writes, seen through their barriers, before the tensor core's reads
          const uint64_t dp0 = p0 + (uint64_t)((g % NS) * (P_BUF >> 4)), dv0 = v0 + (uint64_t)((g % NT) * (TILE >> 4));
          if (one) {
#pragma unroll
            for (int kk = 0; kk < BJ / 16; ++kk)
#pragma unroll
              for (int nh = 0; nh < 2; ++nh)
                mma_ss(256 * nh, dp0 + (uint64_t)((kk * 32) >> 4), dv0 + (uint64_t)((nh * 4 * KV_ATOM + kk * 2048) >> 4),
                       kIdescPV, (b > 0 || kk > 0) ? 1u : 0u);
            commit(&bs.tile_free[g % NT]);
            commit_multicast(&bs.p_free[g % NS], (uint16_t)(1u << partner));
            if (b == nblk - 1) commit(&bs.o_full);
            s_issued = g + 1;
          }
          __syncwarp();
        }
      } else if (const int wq = deq_warp(warp, O_DEQ0); wq >= 0) {
        ok = run_dequant<false, kWin>(un.rows, a.pool, nblk, done, 0u, base + O_RAW + wq * O_RING, nullptr, masks, tiles, bs, wq, lane,
                                 err, abort);
      }
      if (out_warp) {
        // The read-out. Warps 0 - 3, 16 - 19 and (20, 21, 22, 15) have a quarter of the heads each, by
        // their number % 4 as tensor memory has it, and every third 32 columns. The columns of V's tile
        // are ordered so that a lane's fragments are eight consecutive dims of each of four rows, and
        // four lanes have 32 dims of a row (a thread a row made the stores take twice as long). The
        // warps that have nothing else to do wait at a barrier of the hardware, not at the mbarriers:
        // their looks slowed the others down (about 1 us more from P to P . V).
        ok = sync_and(ok, 32 * 4 * NOUT);
        if (!ok) break;  // (all of them: one that gave up further down comes here once more)
        const int set = warp < 4 ? 0 : warp >= 16 && warp < 20 ? 1 : 2;
        const bool direct = un.splits == 1;
        const float sl2 = score_log2(a);
        float l = 0.f, m = -INFINITY;
        if (nblk > 0) {
          const int k = full % NF;
          if (tid == 0 && ok) bar_arrive_tx(&bs.fin[k], min(nblk, NS) * FIN_WG);
          ok = ok && ready_or_wait<true>(bs.fin, NF, full, abort) && ready_or_wait(&bs.o_full, 1, full, abort);
          ok = __all_sync(0xffffffffu, ok);
          tc_after();
          // the warpgroups' sums, from the reference of each to the last block's
          const float* fin = reinterpret_cast<const float*>(base + O_FIN) + (size_t)k * NS * (FIN_WG / 4) + head;
          m = fin[(done + nblk - 1) % NS * (FIN_WG / 4) + MH];
          for (int b = 0; b < min(nblk, NS); ++b) {
            const float* of = fin + (done + nblk - 1 - b) % NS * (FIN_WG / 4);
            l += of[MH] == -INFINITY ? of[0] : of[0] * ex2((of[MH] - m) * sl2);  // (no score: 0, or NaN)
          }
        }
        const float inv = l == 0.f ? 0.f : a.latent_scale / l;  // l is NaN where a weight is
        const size_t out0 = direct ? un.row0 : un.row0 - ts.split_row + (size_t)un.p * ts.split_rows;
        const int row = (warp & 3) * 32 + (lane >> 2);  // and 8, 16, 24 after it
        const size_t at = (out0 + row) * DL + 8 * (lane & 3);
        const bool aligned = ((uintptr_t)part_o & 31u) == 0;
#pragma unroll 1
        for (int c = 32 * set; ok && c < DL; c += 32 * NOUT) {
          float v[2][16] = {};
          if (nblk > 0) {
            tmem_ld_frag(tbase + lane_off + c, v);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {  // rows 8 k after the first
            const float f = __shfl_sync(0xffffffffu, inv, 8 * k + (lane >> 2));
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[k >> 1][4 * (i >> 1) + 2 * (k & 1) + (i & 1)] * f);
            if (row + 8 * k >= un.live) {  // no query head
            } else if (direct) {
              uint32_t h[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
                h[i] = *reinterpret_cast<const uint32_t*>(&x);
              }
              *reinterpret_cast<uint4*>(a.o + at + 8 * k * DL + c) = make_uint4(h[0], h[1], h[2], h[3]);
            } else {
              store8(reinterpret_cast<uint32_t*>(part_o + at + 8 * k * DL + c), w, aligned);
            }
          }
          __syncwarp();
        }
        if (ok && set == 0 && head < un.live)
          (direct ? a.lse : part_lse)[out0 + head] = l == 0.f ? -INFINITY : (m * sl2 + (log2f(l) - kRefLog2)) * 0.6931471805599453f;
        __syncwarp();
        if (nblk > 0 && ok) {
          tc_before();
          if (lane == 0) bar_arrive(&bs.o_free);
        }
      }
      if (!ok && !out_warp) break;
    }
    if (!ok && rank == 0) break;
    done += nblk;
    full += nblk > 0;
  }

  __syncthreads();
  // the S-CTA's MMAs are done (the O-CTA's are, unit by unit), and it has the O-CTA's last P-buffer
  // releases (its last arrivals here)
  if (rank == 0 && ok) {
    ok = done == 0 || pipe_wait(bs.tile_free, NT, done - 1, abort);
    for (int b = done >= NS ? done - NS : 0; b < done; ++b) ok = ok && pipe_wait<true>(bs.p_free, NS, b, abort);
  }
  ok = __syncthreads_and(ok && !*abort);
  if (!ok) {
    // outputs are not valid: flag it, and give copies and MMAs still in flight one more bound before
    // the shared and tensor memory are released
    if (tid == 0) atomicOr(err, HS_FLAG_TIMEOUT);
    __syncthreads();
    if (tid == 0) s_abort = 0;
    __syncthreads();
    const int n = s_issued, q = s_requested;
    for (int g = 0; rank == 0 && q > 0 && g < NS; ++g) pipe_wait(&bs.q_raw[g], 1, q - 1, abort);
    if (n > 0) {
      // (of a ring as deep as blocks can be in flight, so that the parity is block n - 1's and no earlier one's)
      if (rank == 0)
        pipe_wait(bs.s_full, NS, n - 1, abort);
      else
        pipe_wait(bs.tile_free, NT, n - 1, abort);
    }
  }
  tc_before();
  __syncthreads();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(TMEM_COLS) : "memory");
  // the merge kernel (if any) may launch; it waits for this grid's completion before reading
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  cluster_sync_all();  // the partner no longer reads or arrives on this CTA's shared memory
  if (!ok && tid == 0) stay();
}

// The splits of query heads row0 .. row0 + rows - 1 joined, in split order, as an online softmax over their log-sum-exps
// (one pass, and the loads of two splits go out together). A thread per eight output dims.
constexpr int COMBINE_T = 256;
__global__ void __launch_bounds__(COMBINE_T)
    fp4_combine_kernel(const Fp4MlaArgs a, int row0, int rows, const float* __restrict__ part_o, const float* __restrict__ part_lse) {
  pdl_wait();
  const int64_t g = (int64_t)blockIdx.x * COMBINE_T + threadIdx.x;
  const int64_t row = g / (DL / 8);
  const int c8 = (int)(g % (DL / 8));
  if (row >= rows) return;
  float acc[8] = {}, z = 0.f, m = -INFINITY;
#pragma unroll 2
  for (int p = 0; p < a.splits; ++p) {
    const float x = __ldg(part_lse + (size_t)p * rows + row);
    const float4* src = reinterpret_cast<const float4*>(part_o + ((size_t)p * rows + row) * DL) + 2 * c8;
    const float4 u = __ldg(src), v = __ldg(src + 1);
    const float mx = fmaxf(m, x), ref = mx == -INFINITY ? 0.f : mx;  // (a NaN leaves the maximum alone)
    const float keep = expf(m - ref), w = expf(x - ref);
    m = mx;
    z = z * keep + w;
    acc[0] = acc[0] * keep + w * u.x;
    acc[1] = acc[1] * keep + w * u.y;
    acc[2] = acc[2] * keep + w * u.z;
    acc[3] = acc[3] * keep + w * u.w;
    acc[4] = acc[4] * keep + w * v.x;
    acc[5] = acc[5] * keep + w * v.y;
    acc[6] = acc[6] * keep + w * v.z;
    acc[7] = acc[7] * keep + w * v.w;
  }
  const float inv = z == 0.f ? 0.f : 1.f / z;
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    h[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  reinterpret_cast<uint4*>(a.o + (size_t)(row0 + row) * DL)[c8] = make_uint4(h[0], h[1], h[2], h[3]);
  if (c8 == 0) a.lse[row0 + row] = z == 0.f ? -INFINITY : m + logf(z);
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

// CTA pairs that the current device holds at once: a CTA takes an SM. What a device is asked is kept, and
// the kernels are set up for it on the way (both take host time as long as a quarter of a launch).
constexpr int kDevices = 64;
cudaError_t pairs_resident(int* pairs) {
  static std::atomic<int> known[kDevices];
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < kDevices && (*pairs = known[dev].load(std::memory_order_acquire)) > 0) return e;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(fp4_mla_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(fp4_mla_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  *pairs = sms > 3 ? sms / 2 : 1;
  if (e != cudaSuccess)
    (void)cudaGetLastError();
  else if (dev < kDevices)
    known[dev].store(*pairs, std::memory_order_release);
  return e;
}

// Queries of one request whose heads share a tile, and the tiles that its queries make.
int queries_per_tile(int num_heads, int num_queries) {
  const int fit = MH / num_heads;
  return fit < num_queries ? (fit > 1 ? fit : 1) : num_queries;
}
int tiles_per_request(int num_heads, int num_queries) {
  const int g = queries_per_tile(num_heads, num_queries);
  return (num_queries + g - 1) / g;
}

}  // namespace

// Tiles that are not split: all, or the rounds in which every pair takes one. (A round's units end
// together, so that splitting them would only add partial outputs: 64 requests of 2,048 rows 50 us whole,
// 63 in 2; it is the last, partly filled round that splits fill.)
static int whole_tiles(int64_t tiles, int splits, int slots) { return (int)(splits == 1 ? tiles : tiles / slots * slots); }

// In tenths of a block's time (1.2 us): a round of units takes their blocks and 5 blocks' time around
// them; splitting at all adds 4 (partial outputs in 32 bits, the merge kernel and its launch), and 4
// more per unit and pair for the partials' traffic. Measured (us, 128 heads, 2,048 rows): one request
// 48 whole, 25 in 4 splits, 20 in 16; 16 requests 49, 27 in 4, 38 in 6 (two rounds); 32 requests 49,
// 36 in 2, 50 in 3 (two rounds). Of 512 rows: 8 requests 20.5, 18 in 4; 32 requests 21, 22 in 2.
int32_t fp4_mla_splits(int32_t num_requests, int32_t num_heads, int32_t num_queries, int64_t rows) {
  int slots = 0;
  if (pairs_resident(&slots) != cudaSuccess) return 1;
  const int64_t tiles = (int64_t)num_requests * tiles_per_request(num_heads, num_queries);
  const int64_t blocks = (rows + BJ - 1) / BJ;
  int64_t best = 1, best_cost = INT64_MAX;
  for (int64_t s = 1; s <= HS_MAX_MLA_SPLITS && s <= blocks; ++s) {
    const int64_t whole = whole_tiles(tiles, (int)s, slots), units = (tiles - whole) * s;
    if (s > 1 && units == 0) break;
    const int64_t rounds = (whole + slots - 1) / slots, more = (units + slots - 1) / slots;
    const int64_t cost = 10 * (rounds * (blocks + 5) + more * ((blocks + s - 1) / s + 5)) + (s > 1 ? 40 + 40 * units / slots : 0);
    if (cost < best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return (int32_t)best;
}

// (Fewer tiles are split than there are pairs.)
size_t fp4_mla_workspace_bytes(int32_t num_requests, int32_t num_heads, int32_t num_queries, int32_t splits) {
  if (splits == 1) return 0;
  size_t rows = (size_t)num_requests * num_queries * num_heads;
  int pairs = 0;
  if (pairs_resident(&pairs) == cudaSuccess && rows > (size_t)pairs * MH) rows = (size_t)pairs * MH;
  return splits * rows * (DL + 1) * sizeof(float);
}

cudaError_t launch_fp4_mla(const Fp4MlaArgs& args, int32_t num_requests, float* part, uint32_t* err,
                           cudaStream_t stream) {
  // division by the page size as a product: with 2^(s - 1) < d <= 2^s and m = floor(2^(31 + s) / d) + 1,
  // m d is above 2^(31 + s) by at most d <= 2^s, so that t m / 2^(31 + s) is above t / d by less than
  // 1 / d for every t < 2^31
  Fp4MlaArgs a = args;
  if (a.seq_lens != nullptr) {
    a.pool_pages = (uint32_t)((a.pool_rows + a.page_size - 1) / a.page_size);
    a.page_shift = 31;
    while (((int64_t)1 << (a.page_shift - 31)) < a.page_size) ++a.page_shift;
    a.page_mul = (uint32_t)(((uint64_t)1 << a.page_shift) / (uint64_t)a.page_size + 1);
  }
  const bool win = a.seq_lens != nullptr;
  const auto kernel = win ? fp4_mla_kernel<true> : fp4_mla_kernel<false>;
  const int rows = num_requests * a.num_queries * a.num_heads;
  int pairs = 1;
  cudaError_t e = pairs_resident(&pairs);
  CUtensorMap tm_q;
  if (e == cudaSuccess) e = q_map(&tm_q, a.q, rows);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return e;
  }
  Tiles ts;
  ts.per_request = tiles_per_request(a.num_heads, a.num_queries);
  ts.queries = queries_per_tile(a.num_heads, a.num_queries);
  const int tiles = num_requests * ts.per_request;
  ts.whole = whole_tiles(tiles, a.splits, pairs);
  ts.units = ts.whole + (tiles - ts.whole) * a.splits;
  ts.split_row = (ts.whole / ts.per_request * a.num_queries + ts.whole % ts.per_request * ts.queries) * a.num_heads;
  ts.split_rows = rows - ts.split_row;
  float* part_lse = part ? part + (size_t)a.splits * ts.split_rows * DL : nullptr;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)(ts.units < pairs ? ts.units : pairs));
  cfg.blockDim = dim3(T);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, a, ts, tm_q, part, part_lse, err);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return e;
  }
  if (ts.whole == tiles) return cudaSuccess;
  return launch(fp4_combine_kernel, dim3((unsigned)(((int64_t)ts.split_rows * (DL / 8) + COMBINE_T - 1) / COMBINE_T)), COMBINE_T,
                0, stream, a, ts.split_row, ts.split_rows, (const float*)part, (const float*)part_lse);
}

}  // namespace hs
