// Tensor-core (tcgen05) split kernel over a 4-bit latent cache (kv4.cuh).
//
// The split kernel's job and orientation are those of split_tc.cuh: a group of
// NQ query rows of one request lies on the MMA's N, 128 keys per tile on its M;
// a partial is a normalised O and an LSE per row, for the merge kernel.  What
// differs is the operand type.  A 4-bit value with a power-of-two scale is an
// exact e5m2 float, so a tile is expanded to 8 bits, not 16: 80 KB for 128
// keys, half the stores, and K = 32 per MMA.  The bf16 queries and the fp32
// weights P become pairs of 8-bit floats:
//
//   q * 2^x = q_hi + q_lo / 32     (x per row: the row's largest |q| in [128, 256))
//   S^T     = K . [q_hi | q_lo]^T  one MMA chain with N = 2 NQ; s = (S_hi + S_lo / 32) * c,
//             c = 2^-x * sm_scale * log2(e)
//   p       = p_hi + p_lo          O^T += V^T . p_hi, V^T . p_lo
//
// e4m3 carries 4 significant bits, so q_hi takes a bf16 value's upper four and
// q_lo the other four exactly, down to 2^-14 of the row's largest value; smaller
// ones are off by at most 2^-22 of it.  The products and sums are fp32.  A single e4m3 P instead of the
// pair would take a quarter off the MMAs and 3 % off the call (64k keys, NQ = 64),
// for four significant bits in place of seven or eight.
//
// What P keeps.  In a column's scale a weight p >= 2^-6 is off by at most 2^-8 of
// itself (2^-9 for NQ <= 32) and 2^-11 from its way through a half; a smaller one
// by at most 2^-14 (2^-15), however small it is: 8-bit floats end there, a bf16 P
// would not.  Many small weights below one large one -- a sink above a long tail,
// as language models have it -- would so lose what they are together, which l,
// summed from p itself, still counts.  So the scale follows them: now and then a
// column's mean weight so far is looked at, and where it is below 2^-5 the scale
// is raised until the tile's maximum maps to 2^6, O^T and l with it (fp32 has room
// for 2^80).  What all the small ones lose is then at most 2^-8 of l (2^-9):
// n keys lose n * 2^-14.  They are weighed a tile after they were looked at, so
// where a mean of 2^-5 was found after k tiles, the next verdict is a tile after
// the next look, and the sum is at least 8, the first maximum, by then:
//   k        1              3                5                9 ...
//   verdict  512 / 2^14     768 / 2^14       1280 / 2^14      1792 / 2^14
//   of       8              12               20               36
// each 2^-8 or less.  A maximum just mapped to 2^6 faces six tiles at most:
// 2^-10.4.  A sink 11 above a tail of 32,767 equal keys: 0.1 % off in O; with a
// scale from the maximum alone (2^2 to 2^8) up to 31 % (NQ <= 32) and 5 %.  It costs 2 to 4 % of the call (64k keys 111.0 -> 114.9 us,
// 185k 75.2 -> 77.8, 16 ragged requests 291 -> 297, decode 43.2 -> 44.2), nearly all
// of it in the rescales that the smaller headroom brings.  Maxima at 2^4 and 2^6
// would cost 7 % at 64k keys; 2^2 and 2^4 with a mean of 2^-6 1.5 %, for a
// bound of 2^-6.
//
// The RoPE residual codes are 64 more K columns against the same q_rope, so a
// key is 640 codes: five blocks of 128, 20 k-steps of 32.
//
// p_lo.  NQ <= 32: p_hi and 32 * p_lo (both e4m3) sit side by side on N and O^T
// keeps both halves in tensor memory (4 x 2 NQ columns), added at the end.  An
// M = 128 MMA costs 32 + N/4 cycles, most of it for reading its 4 KB A operand
// from shared memory, so the second half is nearly free.  NQ = 48 and 64: p_lo
// is e5m2 and accumulates into the same O^T, a second MMA (tensor memory holds
// 512 columns).
//
// Work.  With nsplit = 0 the grid is one CTA per SM.  All row groups' tiles,
// each group with kKv4SegCost tiles more for its start and end, form one axis
// that is cut into equal pieces; a CTA works through the segments of its piece
// (kv4::Schedule).  Lengths are read on the device, so a captured graph follows
// them.  With nsplit >= 1 a CTA takes one chunk of one row group.
//
// Warp roles (CG = NQ / 16 column groups; registers are dealt out by role):
//   4 CG warps     softmax: a thread owns one key and 16 columns.  They also
//                  turn a segment's queries into q_hi, q_lo, and write O out.
//   1 + 1 warps    MMAs of S^T and of O^T, and the tensor memory
//   2 warps        segments, row ids, mask words, a ring of 4 tiles ahead
//   8 or 16 warps  expansion.  A thread owns quarter q (32 codes) of each block
//                  of one key (NQ <= 32) or two.  It loads the next tile's
//                  codes into registers as it finishes this tile's blocks, so a
//                  load has a whole tile's time to land and no packed staging
//                  passes through shared memory.
//
// Slots.  Two sets of four 16 KB slots (128 keys x 128 channels, 8 bits, in the
// 128-byte-swizzle atom of 8 keys x 128 bytes), by tile parity, take the value
// blocks; the RoPE block has its own slot (NQ <= 48), or goes through block 0's
// slot first (NQ = 64; shared memory is full).  The same bytes are the K-major
// A operand of S^T and the MN-major A operand of O^T.  The RoPE block is free
// after S^T, value block m after O^T block m.
//
// P^T is written MN-major (a thread owns one key, its columns are contiguous:
// 16-byte stores), in the unswizzled layout of 16 columns x 8 keys cores.
//
// What bounds it (GB300).  576 rows over 64k keys, NQ = 64: 115 us per call, 0.72
// PFLOP/s of the bf16-equivalent work; the tensor pipe is 47 % busy, the ALUs 54 %,
// shared memory 84 % (46 % loads and stores, 38 % MMA operands).  No unit is
// the limit alone.  Measured when the scale of P came from the maximum alone (110
// us): a tile takes ~5500 cycles, its expansion ~4700 of them, and a slot set's
// round -- expand, S^T, softmax, O^T -- twice that.  Timed without the
// exponentials and conversions it took 107 us, without the softmax's meeting
// 104, with half the expansion 109.7, with all of these cut 100.  Neither polling
// in place of suspended waits, nor a first pass over the expansion's code while it
// waits for row ids, nor asking for the next slot a block ahead gained anything
// (113, 115 and 118 us against 111).
// Decode (16 requests, NQ = 16): 44 us, 2.0 TB/s; ~8 us are start-up (three
// dependent reads: lengths, row ids, rows) and 4 the merge.
//
// Waits are bounded as in split_tc.cuh.
#pragma once

#include "kv4.cuh"
#include "tc_ptx.cuh"

namespace mlav {

// Base 2.  A column's scale of p: the first maximum it sees maps to 2^kKv4First
// (scores usually grow for a while), one that would pass 2^kKv4Limit (e4m3 ends
// at 448) lowers the scale until it maps to 2^kKv4Top, and a mean weight below
// kKv4MeanP raises it until the tile's maximum does (What P keeps, above).
constexpr float kKv4First = 3.0f, kKv4Top = 6.0f, kKv4Limit = 8.0f;
constexpr float kKv4MeanP = 0.03125f;
constexpr float kKv4MaxSum = 1.2e24f;  // 2^80: a sum that the raised scale may not pass
// Whether the mean is looked at after so many tiles of a segment: 1, 3, 5, 9, 13, ...  (Not after two in a row: the
// sums of one look are read in the tile in which the next ones would be written.)
__device__ __forceinline__ bool kv4_looks_at_mean(int done) {
  return (done & 3) == 1 || done == 3;
}
constexpr float kQLoScale = 32.f;
constexpr float kPLoScale = 32.f;  // concatenated halves only

template <int NQ>
struct Kv4Cfg {
  static_assert(NQ == 16 || NQ == 32 || NQ == 48 || NQ == 64, "row-group sizes built");
  static constexpr bool kConcat = NQ <= 32;
  static constexpr int kKeys = kKeysPerTile;
  static constexpr int kHC = 16;  // query columns per softmax thread
  static constexpr int kCG = NQ / kHC;
  static constexpr int kSoftmaxWarps = 4 * kCG;
  static constexpr int kSoftmaxThreads = 32 * kSoftmaxWarps;
  static constexpr int kMmaWarp = kSoftmaxWarps;           // S^T, and the next one O^T
  static constexpr int kIndexWarp = kSoftmaxWarps + 2;     // the other two of that warpgroup
  static constexpr int kIndexWarps = 2;
  static constexpr int kIndexRing = 4;                     // tiles of row ids and mask words in flight
  static constexpr int kExpandWarp = kSoftmaxWarps + 4;
  static constexpr int kOwnKeys = kCG <= 2 ? 1 : 2;              // keys of a tile per expansion thread
  static constexpr int kExpandWarps = 16 / kOwnKeys;
  static constexpr int kThreads = 32 * (kExpandWarp + kExpandWarps);
  // Registers per thread by role.  A block starts with 65536 / kThreads rounded down to what all its warps can
  // have; the shares together are at most the start's, or the last warps would wait for ever.
  static constexpr int kWarpgroups = kThreads / 128;
  static constexpr int kRegsStart = 65536 / kThreads / 8 * 8 > 128 ? 128 : 65536 / kThreads / 8 * 8;
  static constexpr int kRegsMma = 48;
  static constexpr int kRegsSoftmax = kCG == 1 ? 96 : kCG == 2 ? 88 : kCG == 3 ? 80 : 72;
  static constexpr int kRegsExpand = kCG == 1 ? 80 : kCG == 2 ? 64 : kCG == 3 ? 96 : 80;
  static_assert(kCG * kRegsSoftmax + kRegsMma + (kExpandWarps / 4) * kRegsExpand <= kWarpgroups * kRegsStart,
                "register shares");
  static constexpr int kQBlock = 2 * NQ * 128;  // one 128-channel block of q_hi rows, then q_lo rows
  static constexpr int kQRope = 2 * NQ * 64;    // RoPE channels, once: the residual codes meet the same bytes
  static constexpr int kQBytes = 4 * kQBlock + kQRope;
  static constexpr int kPCore = kKeys * 16;     // 16 query columns x 128 keys of P^T
  static constexpr int kPBytes = 2 * NQ * kKeys;
  static constexpr int kPBufs = NQ >= 48 ? 1 : 2;
  static constexpr int kSlotBytes = kKeys * 128;
  // With one key per expansion thread a block is short work beside its wait, signal and loads: the value blocks then go
  // two at a time (GB300, 16-row groups, 16 decode requests: 44.2 -> 43.1 us per call; 32-row groups, 16 ragged
  // requests: 478 -> 446).  With two keys single blocks are better (48 rows, 185k keys: 78.9 against 84.1 us; 64 rows,
  // 64k keys: 110.8 against 113.3): S^T starts sooner.
  static constexpr bool kPairs = kOwnKeys == 1;
  // Blocks are handed on in runs that end at last(u), the u-th block's run.
  __host__ __device__ static constexpr int last(int u) { return kPairs && u > 0 ? (u + 1) / 2 * 2 : u; }
  __host__ __device__ static constexpr bool opens_run(int u) { return u == 0 || last(u - 1) != last(u); }
  static constexpr bool kRopeSlot = NQ <= 48;
  static constexpr int kSlots = kRopeSlot ? 9 : 8;
  // Slot of the u-th block of tile t, and the parity of its fill there.
  __host__ __device__ static constexpr int slot(int t, int u) {
    return u == 0 && kRopeSlot ? 8 : 4 * (t & 1) + (u & 3);
  }
  __host__ __device__ static constexpr uint32_t fill(int t, int u) {
    return !kRopeSlot && (u & 3) == 0 ? (u == 4 ? 1u : 0u) : kRopeSlot && u == 0 ? t & 1u : (t >> 1) & 1u;
  }
  static constexpr int kOffP = kQBytes;
  static constexpr int kOffRing = kOffP + kPBufs * kPBytes;
  static constexpr int kOffCtl = kOffRing + kSlots * kSlotBytes;
  static constexpr int kOStride = kConcat ? 2 * NQ : NQ;  // tensor-memory columns per O^T block
  static constexpr int kColS = 4 * kOStride;              // two S^T buffers of 2 NQ columns
  static_assert(kColS + 4 * NQ <= 512, "tensor memory budget");
  static_assert(kOffRing % 1024 == 0, "slots are 1024-byte aligned");
};

// What a CTA does: segments, each a range of tiles of one row group of one
// request, one after the other.  nt = 0 ends the list.
struct Kv4Segment {
  int32_t nt;          // tiles
  int32_t tile0;       // the first one
  int32_t rot;         // tile t of the segment is tile0 + (t + rot) % nt
  int32_t n_tokens;    // its query tokens
  int32_t i0, ntok;    // tokens the row group spans
  int32_t r0, nrows;   // its rows within the request
  int32_t keys;        // L: keys of the request
  int32_t prefix;      // P
  int32_t kv0;         // its place in kv_indices
  int32_t mask0;       // its place in the mask (bits)
  int64_t q0;          // first token row of the request
  int64_t prow;        // row of the partial outputs
};
struct Kv4Request {
  int32_t n, keys, kv0, mask0, groups, q0;
};
// Where the hand-out of segments stands (kv4::next_segment).
struct Kv4Cursor {
  int64_t x, x_end, piece;  // own piece of the axis
  int64_t carry;            // axis before request `base`
  int32_t base;             // the 32 requests in `req` and `end`
  int32_t done;
  Kv4Request req[32];
  int64_t end[32];          // inclusive scan of their lengths on the axis, from `carry`
};
constexpr uint32_t kTileFirst = 1, kTileEnd = 2;  // first tile of a segment; no tile, the end of all

template <int NQ>
struct Kv4Ctl {
  uint64_t full[Kv4Cfg<NQ>::kSlots];
  uint64_t empty[Kv4Cfg<NQ>::kSlots];
  // Two of each, by tile parity: the column groups and the MMAs may be a tile apart.
  uint64_t s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t idx_full[Kv4Cfg<NQ>::kIndexRing], idx_empty[Kv4Cfg<NQ>::kIndexRing];
  uint64_t seg_full[2], seg_empty[2];
  uint64_t q_full, sm_sync, mma_idle[2];
  uint32_t tmem_base;
  int abort;
  int flag[Kv4Cfg<NQ>::kSoftmaxWarps];
  alignas(16) float cscale[NQ];  // raw score -> base-2 score
  alignas(16) float nmu[NQ];     // what turns a score into log2 p; +inf before any visible key
  alignas(16) float alpha[NQ];   // rescale factor of the tile; 1/l in the epilogue
  alignas(16) float red[4][NQ];
  alignas(16) float sum[4][NQ];  // sums of p where the mean is looked at
  uint16_t colmask[kMaxQLen][Kv4Cfg<NQ>::kCG];  // per token: which of a column group's columns are its
  Kv4Segment seg[2];
  Kv4Cursor cursor;
  uint32_t tile[Kv4Cfg<NQ>::kIndexRing];                     // kTile* bits
  int32_t row_id[Kv4Cfg<NQ>::kIndexRing][kKeysPerTile];      // pool row of each key, 0 where there is none
  uint32_t see[Kv4Cfg<NQ>::kIndexRing][4][kMaxQLen];         // per 32 keys and token: which keys it sees
  uint32_t see_all[Kv4Cfg<NQ>::kIndexRing][4];               // every token sees all 32
};

template <int NQ>
constexpr int kv4_smem_bytes() {
  return Kv4Cfg<NQ>::kOffCtl + (int)sizeof(Kv4Ctl<NQ>);
}

namespace kv4 {

// kind::f8f6f4, fp32 accumulator: bits 4-5 D (1 = f32) | 7-9 A, 10-12 B format
// (0 = e4m3, 1 = e5m2) | 15, 16 A, B major (1 = MN) | 17-22 N>>3 | 24-28 M>>4
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int afmt, int bfmt, bool a_mn, bool b_mn) {
  return (1u << 4) | ((uint32_t)afmt << 7) | ((uint32_t)bfmt << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
constexpr int kE4M3 = 0, kE5M2 = 1;
constexpr uint64_t kSwizzle64B = 4;

__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Two floats -> two 8-bit floats (a in the low byte) and back to halves.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float a, float b) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));
  return d;
}
__device__ __forceinline__ uint32_t cvt_e4m3x2_f16x2(uint32_t h2) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(h2));
  return d;
}
__device__ __forceinline__ uint32_t cvt_e5m2x2_f16x2(uint32_t h2) {
  uint16_t d;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(d) : "r"(h2));
  return d;
}
__device__ __forceinline__ uint32_t cvt_f16x2_e4m3x2(uint32_t v) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)v));
  return d;
}
__device__ __forceinline__ uint32_t cvt_f16x2(float a, float b) {  // a in the low half
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Pairs of fp32 in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Barrier of `nthreads` threads that tells each whether any of them said yes.
__device__ __forceinline__ bool bar_any(int id, int nthreads, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)mine), "r"(id), "r"(nthreads)
      : "memory");
  return any != 0;
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int kFrom, int kTo>
__device__ __forceinline__ void regs_to() {
  if constexpr (kTo > kFrom) regs_inc<kTo>();
  if constexpr (kTo < kFrom) regs_dec<kTo>();
}

__device__ __forceinline__ uint4 ldg128(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Bytes of (a, b) chosen by the four nibbles of the low half of sel, each 0..7
// (a plain permute: __byte_perm would mask the nibbles once more).
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// One word of 8 codes -> two words of 4 e5m2 values.  lo, hi: the eight
// magnitudes times the group's scale, one byte each.
__device__ __forceinline__ void expand8(uint32_t w, uint32_t lo, uint32_t hi, uint32_t& o0, uint32_t& o1) {
  const uint32_t sel = w & 0x77777777u;
  o0 = prmt(lo, hi, sel) | (w & 0x80808080u);
  o1 = prmt(lo, hi, sel >> 16) | ((w << 4) & 0x80808080u);
}

// The scaled magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6 as e5m2 bytes: exponent
// field + e for all but the zero.  The scale byte is a valid one.
__device__ __forceinline__ void scale_table(uint32_t scale_byte, uint32_t& lo, uint32_t& hi) {
  lo = scale_byte * 0x04040400u + (0x3E3C3800u - 127u * 0x04040400u);
  hi = scale_byte * 0x04040404u + (0x46444240u - 127u * 0x04040404u);
}

// The ten scale bytes of a quarter row: x, y and the low half of z.  A row that
// was never stored may hold bytes outside the format; they are clamped to it, so
// that every code expands to a finite value.  The check of all at once is a
// third of what clamping each as it is used would cost.
__device__ __forceinline__ bool scales_valid(const uint4& s) {
  // valid: byte - 114 is 0 .. 26 (the first byte that is not spoils the ones after it, no matter)
  const uint32_t x = s.x - 0x72727272u, y = s.y - 0x72727272u, z = ((s.z & 0xFFFFu) | 0x72720000u) - 0x72727272u;
  return (((x | (x + 0x05050505u)) | (y | (y + 0x05050505u)) | (z | (z + 0x05050505u))) & 0xE0E0E0E0u) == 0;
}
__device__ __forceinline__ uint32_t clamp_scales(uint32_t w) {
  uint32_t r = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) r |= (uint32_t)(kv4_exponent((w >> (8 * k)) & 0xFFu) + 127) << (8 * k);
  return r;
}
__device__ __forceinline__ void make_valid(uint4& s) {
  if (scales_valid(s)) return;
  s.x = clamp_scales(s.x);
  s.y = clamp_scales(s.y);
  s.z = clamp_scales(s.z);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Slots.  Tile t's value blocks 0..3 stay in slots 4(t%2) .. 4(t%2)+3 until O^T
// is done with them.  The RoPE block, which only S^T reads, has slot 8 where
// shared memory has room for nine; else it passes through slot 0 of the tile's
// set before block 0 does.  Order of expansion and of S^T: RoPE, 1, 2, 3, 0.
__host__ __device__ constexpr int block_of(int u) { return u == 0 ? 4 : u & 3; }

// Bounded wait for phase `parity` of `bar`: at most kWaitTries tries, each of
// which the hardware suspends for at most 20 us (mbar_try_wait), 2.6 s in all.
// Gives up as well once another thread of the CTA has raised *abort, and raises
// it when it gives up.  Short code on purpose: it stands at many places, and
// what the roles' loops take of the instruction cache counts (see below).
constexpr int kWaitTries = 1 << 17;
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
#pragma unroll 1
  for (int tries = kWaitTries; tries > 0; --tries) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
  }
  *abort = 1;
  return false;
}

// Sum of v[0..15] over the warp, index by index: lane l returns that of index l / 2.
__device__ __forceinline__ float reduce16(float (&v)[16], int lane) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool upper = (lane & (2 * o)) != 0;
#pragma unroll
    for (int m = 0; m < o; ++m) {
      const float send = upper ? v[m] : v[m + o];
      const float keep = upper ? v[m + o] : v[m];
      v[m] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * o);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

__device__ __forceinline__ float warp_max(float x) {
  float d;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(x));
  return d;
}

// Max (or sum) of each of the 16 columns over the warp, to dst.
template <bool kMax>
__device__ __forceinline__ void columns_to_smem(const float (&x)[16], float* dst, int lane) {
  if constexpr (kMax) {
    float r = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float m = warp_max(x[k]);
      r = lane == k ? m : r;
    }
    if (lane < 16) dst[lane] = r;
  } else {
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = x[k];
    const float r = reduce16(v, lane);
    if ((lane & 1) == 0) dst[lane >> 1] = r;
  }
}

// Hands a CTA its segments (one full warp calls it).
//
// Flat (a.seg_table set): the work of the call -- for each request and row group
// seg_cost units of start and end, then one per tile -- lies on one axis, and
// the CTAs take equal pieces of it, so they end together whatever the requests'
// lengths are.  A piece that ends inside a row group's keys leaves a partial;
// the partials of group g of request b are numbered from (CTA that has its
// first tile) + b * groups_max + g on, by CTA, which no two segments share.
// Otherwise: one chunk of one row group per CTA (the grid), or none.
struct Schedule {
  // Request b and its length on the axis (none past the batch).
  static __device__ __forceinline__ int64_t request(const SplitArgs& a, int nq, int b, Kv4Request& r) {
    r = {};
    if (b >= a.batch) return 0;
    const RequestTokens rq = request_tokens(a, b);
    r.kv0 = a.kv_indptr[b];
    r.mask0 = a.mask_indptr[b];
    r.q0 = (int)rq.q0;
    r.n = rq.n;
    r.keys = a.kv_indptr[b + 1] - r.kv0 + rq.n;
    r.groups = (rq.n * a.H + nq - 1) / nq;
    return (int64_t)r.groups * ((r.keys + kKeysPerTile - 1) / kKeysPerTile + a.seg_cost);
  }
  static __device__ __forceinline__ int64_t scan(int64_t v, int lane) {  // inclusive, over the warp
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    return v;
  }
  // (numbers below 2^31, as a rule: a tenth of the 64-bit division's time)
  static __device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {
    return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
  }
  // Requests base .. base+31 into the cursor; returns the axis after them.
  static __device__ __forceinline__ int64_t fetch(const SplitArgs& a, int nq, int lane, int base, int64_t carry,
                                                  Kv4Cursor& c) {
    Kv4Request r;
    const int64_t incl = carry + scan(request(a, nq, base + lane, r), lane);
    __syncwarp();  // every lane has read what is replaced (shuffles order no memory)
    c.req[lane] = r;
    c.end[lane] = incl;
    if (lane == 0) {
      c.base = base;
      c.carry = carry;
    }
    __syncwarp();
    return __shfl_sync(0xffffffffu, incl, 31);
  }

  static __device__ __forceinline__ void start(const SplitArgs& a, int nq, int lane, Kv4Cursor& c) {
    int64_t total = 0, piece = 1;
    if (a.seg_table) {
#pragma unroll 1
      for (int b = 0; b < a.batch; b += 32) total = fetch(a, nq, lane, b, total, c);
      piece = divide(total + gridDim.x - 1, gridDim.x);
      piece = piece < 1 ? 1 : piece;
      if (a.batch > 32) fetch(a, nq, lane, 0, 0, c);
    } else {
      fetch(a, nq, lane, blockIdx.z, 0, c);  // (only its own request counts)
    }
    if (lane == 0) {
      const int64_t x = blockIdx.x * piece;
      c.x = x;
      c.x_end = x + piece < total ? x + piece : total;
      c.piece = piece;
      c.done = 0;
    }
    __syncwarp();
  }

  static __device__ __forceinline__ void rows(const SplitArgs& a, int nq, int g, const Kv4Request& r, Kv4Segment& s) {
    s.q0 = r.q0;
    s.n_tokens = r.n;
    s.keys = r.keys;
    s.prefix = r.keys - r.n;
    s.kv0 = r.kv0;
    s.mask0 = r.mask0;
    s.r0 = g * nq;
    s.nrows = r.n * a.H - s.r0 < nq ? r.n * a.H - s.r0 : nq;
    s.i0 = s.r0 / a.H;
    s.ntok = (s.r0 + s.nrows - 1) / a.H - s.i0 + 1;
  }

  // The next segment, or one of no tiles (the whole warp calls it, lane 0 writes s).
  static __device__ __forceinline__ void next(const SplitArgs& a, int nq, int lane, Kv4Cursor& c, Kv4Segment& s) {
    if (!a.seg_table) {
      const Kv4Request& r = c.req[0];
      const int g = blockIdx.x;
      const bool none = c.done || g >= r.groups;
      __syncwarp();
      if (lane == 0) {
        c.done = 1;
        s.nt = 0;
      }
      if (none) return;
      // chunk_len, in tiles
      const int tiles = (r.keys + kKeysPerTile - 1) / kKeysPerTile;
      const int per = (int)(((uint32_t)r.keys + (uint32_t)a.nsplit - 1u) / (uint32_t)a.nsplit);
      int chunk = (per + kKeysPerTile - 1) / kKeysPerTile;
      chunk = chunk < a.min_chunk / kKeysPerTile ? a.min_chunk / kKeysPerTile : chunk;
      const int64_t t0 = (int64_t)blockIdx.y * chunk;
      const int64_t prow = (int64_t)blockIdx.y * a.rows_max + (int64_t)r.q0 * a.H + g * nq;
      if (t0 >= tiles) {  // an empty chunk
        const int nrows = r.n * a.H - g * nq;
        for (int n = lane; n < nrows && n < nq; n += 32) a.part_lse[prow + n] = -INFINITY;
        return;
      }
      if (lane == 0) {
        rows(a, nq, g, r, s);
        s.prow = prow;
        s.tile0 = (int)t0;
        s.nt = tiles - s.tile0 < chunk ? tiles - s.tile0 : chunk;
        // The row groups of a chunk read the same keys; staggered they read them
        // from L2 one after the other.
        s.rot = g % s.nt;
      }
      return;
    }
    int64_t x = c.x;
    const int64_t x_end = c.x_end;
    __syncwarp();
#pragma unroll 1
    while (x < x_end) {
      const uint32_t past = __ballot_sync(0xffffffffu, c.end[lane] > x);
      if (!past) {
        fetch(a, nq, lane, c.base + 32, c.end[31], c);
        continue;
      }
      const int l = __ffs(past) - 1;
      const Kv4Request& r = c.req[l];
      const int tiles = (r.keys + kKeysPerTile - 1) / kKeysPerTile;
      const int64_t from = l ? c.end[l - 1] : c.carry;  // the request's place on the axis
      const int g = (int)divide(x - from, tiles + a.seg_cost);
      const int64_t first = from + (int64_t)g * (tiles + a.seg_cost) + a.seg_cost;  // the group's first tile
      const int64_t end = first + tiles;
      const int64_t t0 = x > first ? x - first : 0;
      x = x_end < end ? x_end : end;
      if (x - first <= t0) continue;  // only of the group's start
      if (lane == 0) {
        const int slot = (c.base + l) * a.groups_max + g;
        rows(a, nq, g, r, s);
        s.prow = (int64_t)(blockIdx.x + slot) * nq;
        s.tile0 = (int)t0;
        s.nt = (int)(x - first - t0);
        s.rot = 0;
        // where the merge finds the group's partials, and how many
        if (t0 == 0)
          a.seg_table[slot] = make_int2(blockIdx.x + slot, (int)divide(end - 1, c.piece) - (int)blockIdx.x + 1);
        c.x = x;
      }
      __syncwarp();
      return;
    }
    if (lane == 0) s.nt = 0;
  }
};

}  // namespace kv4

template <int NQ>
__global__ void __launch_bounds__(Kv4Cfg<NQ>::kThreads, 1) split_kv4_kernel(const __grid_constant__ SplitArgs a) {
  using Cfg = Kv4Cfg<NQ>;
  constexpr int kKeys = Cfg::kKeys;
  constexpr int S = Cfg::kSlots;
  constexpr int HC = Cfg::kHC;
  constexpr int CG = Cfg::kCG;
  constexpr int kSoftmaxWarps = Cfg::kSoftmaxWarps;
  constexpr int kSoftmaxThreads = Cfg::kSoftmaxThreads;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  extern __shared__ __align__(1024) uint8_t kv4_smem[];  // the swizzle atoms are 1024-byte aligned
  const uint32_t sQ = smem_u32(kv4_smem), sP = sQ + Cfg::kOffP, sRing = sQ + Cfg::kOffRing;
  Kv4Ctl<NQ>& ctl = *reinterpret_cast<Kv4Ctl<NQ>*>(kv4_smem + Cfg::kOffCtl);

  // ---- set-up ---------------------------------------------------------------
  if (tid == 0) {
    for (int k = 0; k < S; ++k) {
      mbar_init(&ctl.full[k], Cfg::kExpandWarps);
      mbar_init(&ctl.empty[k], 1);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&ctl.s_full[k], 1);
      mbar_init(&ctl.s_free[k], kSoftmaxWarps);
      mbar_init(&ctl.p_full[k], kSoftmaxWarps);
      mbar_init(&ctl.pv_done[k], 1);
      mbar_init(&ctl.seg_full[k], 1);
      mbar_init(&ctl.seg_empty[k], kSoftmaxWarps + Cfg::kIndexWarps);
      mbar_init(&ctl.mma_idle[k], 1);
    }
    for (int k = 0; k < Cfg::kIndexRing; ++k) {
      mbar_init(&ctl.idx_full[k], 1);
      mbar_init(&ctl.idx_empty[k], kSoftmaxWarps + Cfg::kExpandWarps + 2);
    }
    mbar_init(&ctl.q_full, kSoftmaxWarps);
    mbar_init(&ctl.sm_sync, kSoftmaxWarps);
    ctl.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == Cfg::kMmaWarp) {
    tc::tmem_alloc(&ctl.tmem_base, 512);
    tc::tmem_relinquish();
  }
  // (its loads' latency passes beside the rest of the set-up)
  if (warp == Cfg::kIndexWarp) kv4::Schedule::start(a, NQ, lane, ctl.cursor);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;
  // Tiles are counted through all segments (t below, in the rings and their
  // parities), so no role waits for the others at a segment's end: the rings
  // just go on, with only the queries and O^T changing hands.
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, kv4::wait(bar, parity, &ctl.abort));
  };

  if (warp >= Cfg::kExpandWarp) {
    // =========================== expansion ===================================
    // Thread (warp w, lane) owns codes 32q..32q+31 of each block of key 8w +
    // lane/4 (and of 64 + that, with 8 warps), q = lane % 4: a warp's load of one
    // block covers 8 rows x 64 contiguous bytes, and its 16-byte stores reach
    // all 32 banks (8 lanes = 2 keys x 4 chunks of opposite parity).
    kv4::regs_to<Cfg::kRegsStart, Cfg::kRegsExpand>();
    const int w = warp - Cfg::kExpandWarp;
    const int q = lane & 3;
    const int key0 = 8 * w + (lane >> 2);
    const uint32_t off0 = key0 * 128 + (((2 * q) ^ (key0 & 7)) << 4);
    const uint32_t off1 = key0 * 128 + (((2 * q + 1) ^ (key0 & 7)) << 4);
    constexpr int K = Cfg::kOwnKeys;
    int32_t row[K] = {}, id[K] = {};  // pool rows of the tile being loaded, and of the one after
    uint4 code[K][kKv4Blocks], scale[K];
    bool ok = true, more = true;
    auto at = [&](int h, int byte) { return a.kv4_pool + 16 * q + byte + (uint64_t)(uint32_t)row[h] * kKv4RowBytes; };
    // Pool rows of the own keys of tile t, if there is one.  (A key without a
    // row reads row 0: its weight is 0, and a 4-bit value is finite whatever the
    // bytes.)
    auto read_ids = [&](int t) {
      const int r = t % Cfg::kIndexRing;
      ok = wait_warp(&ctl.idx_full[r], (t / Cfg::kIndexRing) & 1);
      more = ok && !(ctl.tile[r] & kTileEnd);
#pragma unroll
      for (int h = 0; h < K; ++h) id[h] = more ? ctl.row_id[r][key0 + 64 * h] : 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.idx_empty[r]);
    };
    read_ids(0);
    if (more) {
#pragma unroll
      for (int h = 0; h < K; ++h) {
        row[h] = id[h];
        scale[h] = kv4::ldg128(at(h, kKv4ScaleOff));
#pragma unroll
        for (int u = 0; u < kKv4Blocks; ++u)
          code[h][kv4::block_of(u)] = kv4::ldg128(at(h, 64 * kv4::block_of(u)));
      }
    }
    bool have = more;
    if (have) read_ids(1);
#pragma unroll 1
    for (int t = 0; have && ok; ++t) {
      // Loads of tile t+1 follow the use of their registers in tile t; after the
      // last tile they read row 0.
      uint4 next_scale[K];
#pragma unroll
      for (int h = 0; h < K; ++h) {
        kv4::make_valid(scale[h]);
        row[h] = id[h];
        next_scale[h] = kv4::ldg128(at(h, kKv4ScaleOff));
      }
#pragma unroll
      for (int u = 0; u < kKv4Blocks; ++u) {
        const int m = kv4::block_of(u), sl = Cfg::slot(t, u);
        // (O^T frees the value blocks' slots in the order 0, 1, 2, 3: the wait for
        // the run's highest block covers the other)
        if (Cfg::opens_run(u)) {
          const int z = Cfg::last(u) == kKv4Blocks - 1 ? u : Cfg::last(u);
          ok = ok && wait_warp(&ctl.empty[Cfg::slot(t, z)], Cfg::fill(t, z) ^ 1);
        }
        if (ok) {
          // (one copy of the code for both keys: the roles' loops share the
          // instruction cache)
#pragma unroll 1
          for (int h = 0; h < K; ++h) {
            const uint4 c = h ? code[K - 1][m] : code[0][m];
            const uint4 sc = h ? scale[K - 1] : scale[0];
            const uint32_t sw = m < 2 ? sc.x : m < 4 ? sc.y : sc.z;
            uint32_t lo[2], hi[2], o[8];
            kv4::scale_table((sw >> (16 * (m & 1))) & 0xFFu, lo[0], hi[0]);
            kv4::scale_table((sw >> (16 * (m & 1) + 8)) & 0xFFu, lo[1], hi[1]);
            kv4::expand8(c.x, lo[0], hi[0], o[0], o[1]);
            kv4::expand8(c.y, lo[0], hi[0], o[2], o[3]);
            kv4::expand8(c.z, lo[1], hi[1], o[4], o[5]);
            kv4::expand8(c.w, lo[1], hi[1], o[6], o[7]);
            const uint32_t dst = sRing + sl * Cfg::kSlotBytes + h * 64 * 128;
            kv4::sts128(dst + off0, o[0], o[1], o[2], o[3]);
            kv4::sts128(dst + off1, o[4], o[5], o[6], o[7]);
          }
          if (u == Cfg::last(u)) {
            __syncwarp();
            if (lane == 0 && !(a.test_stall && t + u == 0)) mbar_arrive(&ctl.full[sl]);
#pragma unroll
            for (int b = 0; b < kKv4Blocks; ++b) {
              if (Cfg::last(b) != u) continue;
#pragma unroll
              for (int h = 0; h < K; ++h) code[h][kv4::block_of(b)] = kv4::ldg128(at(h, 64 * kv4::block_of(b)));
            }
          }
        }
      }
      have = more;
      if (ok && more) read_ids(t + 2);
#pragma unroll
      for (int h = 0; h < K; ++h) scale[h] = next_scale[h];
    }
  } else if (warp >= Cfg::kMmaWarp) {
    // ============================ MMA issue ==================================
    // Two warps, one for each product, so that neither waits behind the other:
    // the tensor core takes their MMAs as they come.  The whole warp runs the
    // loop and one elected lane issues: the loop's values then stay
    // warp-uniform, where an MMA takes its descriptors from.  With a single
    // thread running it every MMA cost ~160 cycles to issue, against 32 + N/4
    // (N <= 128) that the tensor core needs for one.  The writers' generic
    // stores are ordered before the MMAs' reads by a proxy fence here, after
    // the wait: at the writers it held each block up until its stores landed.
    kv4::regs_to<Cfg::kRegsStart, Cfg::kRegsMma>();
    if (warp < Cfg::kIndexWarp) {
      const bool leader = kv4::elect_one();
      auto wait_mma = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool ok = wait_warp(bar, parity);
        fence_proxy_async_smem();
        tc::fence_after_sync();
        return ok;
      };
      // Bits of tile t; kTileEnd after a wait that gave up.
      auto tile_bits = [&](int t) -> uint32_t {
        const int r = t % Cfg::kIndexRing;
        if (!wait_warp(&ctl.idx_full[r], (t / Cfg::kIndexRing) & 1)) return kTileEnd;
        const uint32_t bits = ctl.tile[r];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.idx_empty[r]);
        return bits;
      };
      if (warp == Cfg::kMmaWarp) {
        constexpr uint32_t idesc = kv4::idesc_f8(kKeys, 2 * NQ, kv4::kE5M2, kv4::kE4M3, false, false);
        const uint64_t desc_k = tc::smem_desc(sRing, 16, 1024, tc::kSwizzle128B);
        const uint64_t desc_q = tc::smem_desc(sQ, 16, 1024, tc::kSwizzle128B);
        const uint64_t desc_r = tc::smem_desc(sQ + 4 * Cfg::kQBlock, 16, 512, kv4::kSwizzle64B);  // RoPE part
        uint32_t q_phase = 0;
#pragma unroll 1
        for (int t = 0;; ++t) {
          const uint32_t bits = tile_bits(t);
          if (bits & kTileEnd) break;
          if (bits & kTileFirst) {
            if (!wait_mma(&ctl.q_full, q_phase)) break;
            q_phase ^= 1;
          }
          if (t >= 2 && !wait_mma(&ctl.s_free[t & 1], ((t - 2) >> 1) & 1)) break;
          const uint32_t d = tmem + Cfg::kColS + (t & 1) * 2 * NQ;
          bool ok = true;
#pragma unroll 1
          for (int u = 0; u < kKv4Blocks; ++u) {
            const int slot = Cfg::slot(t, u);
            if (Cfg::opens_run(u)) {
              const int z = Cfg::last(u);
              if (!(ok = wait_mma(&ctl.full[Cfg::slot(t, z)], Cfg::fill(t, z)))) break;
            }
            const uint64_t ad = desc_k + (uint32_t)(slot * (Cfg::kSlotBytes >> 4));
            if (leader && u == 0) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                kv4::mma_f8_ss(d, ad + 2 * k, desc_r + 2 * (k & 1), idesc, k == 0 ? 0u : 1u);
              tc::mma_commit(&ctl.empty[slot]);  // only S^T reads the RoPE block
            } else if (leader) {
              const uint64_t bd = desc_q + (uint32_t)(kv4::block_of(u) * (Cfg::kQBlock >> 4));
#pragma unroll
              for (int k = 0; k < 4; ++k) kv4::mma_f8_ss(d, ad + 2 * k, bd + 2 * k, idesc, 1u);
              if (u == kKv4Blocks - 1) tc::mma_commit(&ctl.s_full[t & 1]);
            }
            __syncwarp();
          }
          if (!ok) break;
        }
      } else {
        constexpr uint32_t idesc =
            kv4::idesc_f8(128, Cfg::kConcat ? 2 * NQ : NQ, kv4::kE5M2, kv4::kE4M3, true, true);
        constexpr uint32_t idesc_lo = kv4::idesc_f8(128, NQ, kv4::kE5M2, kv4::kE5M2, true, true);
        const uint64_t desc_v = tc::smem_desc(sRing, Cfg::kSlotBytes, 1024, tc::kSwizzle128B);
        const uint64_t desc_p = tc::smem_desc(sP, 128, Cfg::kPCore, 0);
#pragma unroll 1
        for (int t = 0;; ++t) {
          const uint32_t bits = tile_bits(t);
          if (bits & kTileEnd) break;
          // (P^T(t) was written after S^T(t), so its value blocks are there too,
          // and after the last segment's O^T was read out)
          if (!wait_mma(&ctl.p_full[t & 1], (t >> 1) & 1)) break;
          const uint64_t pd = desc_p + (uint32_t)((t % Cfg::kPBufs) * (Cfg::kPBytes >> 4));
#pragma unroll 1
          for (int m = 0; m < 4; ++m) {
            const int slot = 4 * (t & 1) + m;
            const uint64_t ad = desc_v + (uint32_t)(slot * (Cfg::kSlotBytes >> 4));
            const uint32_t d = tmem + m * Cfg::kOStride;
            if (leader) {
#pragma unroll
              for (int k = 0; k < kKeys / 32; ++k) {
                kv4::mma_f8_ss(d, ad + k * (4096 >> 4), pd + k * (512 >> 4), idesc,
                               k == 0 && (bits & kTileFirst) ? 0u : 1u);
                if (!Cfg::kConcat)
                  kv4::mma_f8_ss(d, ad + k * (4096 >> 4), pd + (((NQ / 16) * Cfg::kPCore + k * 512) >> 4), idesc_lo,
                                 1u);
              }
              tc::mma_commit(&ctl.empty[slot]);
              if (m == 3) tc::mma_commit(&ctl.pv_done[t & 1]);
            }
            __syncwarp();
          }
        }
      }
      // Every MMA this warp issued has completed before tensor memory is freed.
      if (leader) {
        tc::mma_commit(&ctl.mma_idle[warp - Cfg::kMmaWarp]);
        int never = 0;  // (also after an abort)
        kv4::wait(&ctl.mma_idle[warp - Cfg::kMmaWarp], 0, &never);
      }
      __syncwarp();
    } else {
      // ================= segments, row ids and mask words =====================
      // The first warp hands out the segments; the two take turns at the tiles:
      // the pool rows of the tile's keys, and per 32 keys and token the mask's
      // bits, less keys that have no row.
      const int iw = warp - Cfg::kIndexWarp;
      uint32_t bad = 0;
      int t_seg = 0;  // first tile of the segment in the count of all
      bool ok = true;
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        if (iw == 0) {
          if (!(ok = wait_warp(&ctl.seg_empty[k & 1], ((k >> 1) & 1) ^ 1))) break;
          kv4::Schedule::next(a, NQ, lane, ctl.cursor, ctl.seg[k & 1]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.seg_full[k & 1]);
        }
        if (!(ok = wait_warp(&ctl.seg_full[k & 1], (k >> 1) & 1))) break;
        const Kv4Segment& sg = ctl.seg[k & 1];
        const int nt = sg.nt;
        if (nt == 0) {
          // the end, as one more tile
          const int r = t_seg % Cfg::kIndexRing;
          if (t_seg % Cfg::kIndexWarps == iw &&
              wait_warp(&ctl.idx_empty[r], ((t_seg / Cfg::kIndexRing) & 1) ^ 1) && lane == 0) {
            ctl.tile[r] = kTileEnd;
            mbar_arrive(&ctl.idx_full[r]);
          }
          break;
        }
        const int tile0 = sg.tile0, rot = sg.rot, i0 = sg.i0, ntok = sg.ntok, L = sg.keys, n_tok = sg.n_tokens;
        const int P = sg.prefix;
        const int32_t* pre_ids = a.kv_indices + sg.kv0;
        const int32_t* new_ids = a.out_cache_loc + sg.q0 - P;
        const int64_t block0 = sg.mask0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.seg_empty[k & 1]);
        const uint8_t* mask_lo = a.mask + (block0 >> 3);  // the request's mask block, in whole bytes
        const uint8_t* mask_hi = a.mask + ((block0 + (int64_t)n_tok * L + 7) >> 3);
#pragma unroll 1
        for (int i = (iw - t_seg) & (Cfg::kIndexWarps - 1); i < nt; i += Cfg::kIndexWarps) {
          const int t = t_seg + i;
          const int r = t % Cfg::kIndexRing;
          const int key0 = (tile0 + (i + rot < nt ? i + rot : i + rot - nt)) * kKeys;
          // all the tile's loads first: one latency
          int32_t id[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = key0 + 32 * j + lane;
            const int32_t* p = key < P ? pre_ids + key : new_ids + key;
            id[j] = key < L ? __ldg(p) : -1;
          }
          uint32_t w[5], valid[4], blind = 0;  // blind: bit j, some token does not see all of the j-th 32 keys
          int shift;
          auto load_mask = [&](int tok) {
            const int64_t bit = block0 + (int64_t)(i0 + tok) * L + key0;
            const uintptr_t byte = reinterpret_cast<uintptr_t>(a.mask + (bit >> 3));
            const uint8_t* p = reinterpret_cast<const uint8_t*>(byte & ~(uintptr_t)3);
            shift = 8 * (int)(byte & 3) + (int)(bit & 7);
            w[0] = w[1] = w[2] = w[3] = w[4] = 0;
            if (tok >= ntok) return;
            if (p >= mask_lo && p + 20 <= mask_hi) {
#pragma unroll
              for (int j = 0; j < 5; ++j) w[j] = __ldg(reinterpret_cast<const uint32_t*>(p) + j);
            } else {  // at an end of the mask block: only its own bytes are read
#pragma unroll 1
              for (int n = 0; n < 20; ++n) {
                const uint32_t v = p + n >= mask_lo && p + n < mask_hi ? __ldg(p + n) : 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(w[j], w[j + 1], 8);
                w[4] = (w[4] >> 8) | (v << 24);
              }
            }
          };
          int tok = lane;
          load_mask(tok);
          if (!(ok = wait_warp(&ctl.idx_empty[r], ((t / Cfg::kIndexRing) & 1) ^ 1))) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool in = id[j] >= 0 && id[j] < a.pool_rows;
            if (!in && key0 + 32 * j + lane < L) bad = 1;  // left out, and reported
            valid[j] = __ballot_sync(0xffffffffu, in);
            ctl.row_id[r][32 * j + lane] = in ? id[j] : 0;
          }
#pragma unroll 1
          for (;; load_mask(tok)) {
            if (tok < ntok) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t v = __funnelshift_r(w[j], w[j + 1], shift) & valid[j];
                ctl.see[r][j][tok] = v;
                if (v != 0xffffffffu) blind |= 1u << j;
              }
            }
            tok += 32;
            if (tok - lane >= ntok) break;
          }
          blind = __reduce_or_sync(0xffffffffu, blind);
          if (lane < 4) ctl.see_all[r][lane] = !((blind >> lane) & 1);
          if (lane == 0) ctl.tile[r] = i == 0 ? kTileFirst : 0u;
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.idx_full[r]);
        }
        t_seg += nt;
      }
      if (bad) atomicOr(a.status, kStatusBadRow);
    }
  } else {
    // ============================ softmax ====================================
    kv4::regs_to<Cfg::kRegsStart, Cfg::kRegsSoftmax>();
    const int quad = warp & 3;
    const int half = warp >> 2;      // column group
    const int j = 32 * quad + lane;  // key within the tile == TMEM lane
    const int c0 = half * HC;        // first query column of this thread
    const int bar_id = 2 + half;     // the group's four warps (quads) share its columns
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quad) << 16);
    int t = 0;  // tiles of all segments
    bool my_abort = false;
    // All softmax warps meet here, but a column group may have given up and left:
    // so this wait is bounded too, and each group then decides as one.
    uint32_t sync_phase = 0;
    auto meet = [&](bool ok) -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.sm_sync);
      ok = wait_warp(&ctl.sm_sync, sync_phase) && ok;
      sync_phase ^= 1;
      return !kv4::bar_any(bar_id, 128, !ok);
    };
#pragma unroll 1
    for (int k = 0;; ++k) {
      // (every warp is done with the last segment's tables)
      if (!meet(wait_warp(&ctl.seg_full[k & 1], (k >> 1) & 1))) break;
      const Kv4Segment& sg = ctl.seg[k & 1];
      if (sg.nt == 0) break;
      const int nrows = sg.nrows;
      const int64_t grow0 = sg.q0 * a.H + sg.r0;  // global row of the group's first row
      const int t_end = t + sg.nt;
      const int ntok = sg.ntok;
      for (int n = tid; n < NQ; n += kSoftmaxThreads) ctl.nmu[n] = INFINITY;
      for (int i = tid; i < ntok * CG; i += kSoftmaxThreads) {
        const int tok = i / CG, h = i % CG;
        // rows (tok + i0) * H .. + H of the request, as columns of the group
        const int first = (sg.i0 + tok) * a.H - sg.r0 - h * HC;
        const int lo = first < 0 ? 0 : first;
        int hi = first + a.H < HC ? first + a.H : HC;
        hi = nrows - h * HC < hi ? nrows - h * HC : hi;
        ctl.colmask[tok][h] = (uint16_t)(hi > lo ? (0xFFFFu >> (HC - (hi - lo))) << lo : 0u);
      }
      // Queries: warp w turns rows w, w + warps, ... into q_hi and q_lo, two at
      // a time so that their loads overlap.  Lane l holds channels 8l..8l+7 and
      // 256+8l.., lanes 0-7 also RoPE channels 8l...  (The last segment's S^T
      // is complete: this warp has read it.)
      constexpr int kRowsAtOnce = 2;
      static_assert(NQ % (kSoftmaxWarps * kRowsAtOnce) == 0, "whole rounds of query rows");
#pragma unroll 1
      for (int base = warp; base < NQ; base += kSoftmaxWarps * kRowsAtOnce) {
        uint4 v[kRowsAtOnce][3];
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i) {
          const int n = base + i * kSoftmaxWarps;
          v[i][0] = v[i][1] = v[i][2] = make_uint4(0, 0, 0, 0);
          if (n < nrows) {
            const uint4* qn = reinterpret_cast<const uint4*>(a.q_nope + (grow0 + n) * kDLatent);
            v[i][0] = __ldg(qn + lane);
            v[i][1] = __ldg(qn + 32 + lane);
            if (lane < 8) v[i][2] = __ldg(reinterpret_cast<const uint4*>(a.q_rope + (grow0 + n) * kDRope) + lane);
          }
        }
#pragma unroll
        for (int i = 0; i < kRowsAtOnce; ++i) {
          const int n = base + i * kSoftmaxWarps;
          uint32_t top = 0;  // largest |q| as bits: bf16 magnitudes order as integers
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            const uint32_t u[4] = {v[i][c].x, v[i][c].y, v[i][c].z, v[i][c].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, max(u[e] & 0x7FFFu, (u[e] >> 16) & 0x7FFFu));
          }
          top = __reduce_max_sync(0xffffffffu, top);
          const int ex = (int)(top >> 7);  // biased exponent of the largest value
          // 2^x brings it into [128, 256); rows of zeros or denormals use the largest x
          int x = 7 + 127 - ex;
          x = x > 126 ? 126 : x;
          const float up = pow2f(x);
          // a row with an infinity or a NaN scores NaN
          if (lane == 0) ctl.cscale[n] = ex == 255 ? NAN : a.scale_log2 * pow2f(-x);
          // 8 channels -> 8 bytes of q_hi (at `at`) and of q_lo (`lo_off` further on)
          auto put = [&](uint32_t at, uint32_t lo_off, const uint4& bits) {
            const uint32_t u[4] = {bits.x, bits.y, bits.z, bits.w};
            uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float f0 = __uint_as_float(u[e] << 16) * up, f1 = __uint_as_float(u[e] & 0xFFFF0000u) * up;
              const uint32_t h = kv4::cvt_e4m3x2(f0, f1);
              const uint32_t hf = kv4::cvt_f16x2_e4m3x2(h);
              const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hf));
              const uint32_t l = kv4::cvt_e4m3x2((f0 - back.x) * kQLoScale, (f1 - back.y) * kQLoScale);
              hi[e >> 1] |= h << (16 * (e & 1));
              lo[e >> 1] |= l << (16 * (e & 1));
            }
            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at), "r"(hi[0]), "r"(hi[1]) : "memory");
            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(at + lo_off), "r"(lo[0]), "r"(lo[1]) : "memory");
          };
          static_assert(NQ % 8 == 0, "q_lo row n swizzles as q_hi row n");
          const uint32_t in_block = (((lane & 15) >> 1) ^ (n & 7)) << 4;  // 16-byte chunk, 128-byte swizzle
          const uint32_t at = sQ + (lane >> 4) * Cfg::kQBlock + n * 128 + in_block + 8 * (lane & 1);
          put(at, NQ * 128, v[i][0]);
          put(at + 2 * Cfg::kQBlock, NQ * 128, v[i][1]);
          if (lane < 8)  // RoPE: rows of 64 bytes, 64-byte swizzle
            put(sQ + 4 * Cfg::kQBlock + n * 64 + (((lane >> 1) ^ ((n >> 1) & 3)) << 4) + 8 * (lane & 1), NQ * 64,
                v[i][2]);
        }
      }
      if (!meet(true)) break;  // the tables are written
      if (lane == 0) mbar_arrive(&ctl.q_full);

      float acc[HC];  // sum of p over this thread's keys
#pragma unroll
      for (int c = 0; c < HC; ++c) acc[c] = 0.f;
      const int t_first = t;
#pragma unroll 1
      for (; t < t_end; ++t) {
        // Which of its columns see this thread's key.
        uint32_t vis = 0xffffffffu;
        const int r = t % Cfg::kIndexRing;
        if (!my_abort) my_abort = !kv4::wait(&ctl.idx_full[r], (t / Cfg::kIndexRing) & 1, &ctl.abort);
        const bool all_vis = ctl.see_all[r][quad] != 0;
        if (!all_vis) {
          vis = 0;
          for (int tl = 0; tl < ntok; ++tl)
            if ((ctl.see[r][quad][tl] >> lane) & 1u) vis |= ctl.colmask[tl][half];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.idx_empty[r]);
        const uint32_t t_s = t_lane + Cfg::kColS + (t & 1) * 2 * NQ + c0;

        if (!my_abort) my_abort = !kv4::wait(&ctl.s_full[t & 1], (t >> 1) & 1, &ctl.abort);
        // (asked now, so that the answer is there by the time P^T is written)
        const bool p_free = t < Cfg::kPBufs ||
                            mbar_test_wait(&ctl.pv_done[(t - Cfg::kPBufs) & 1], ((t - Cfg::kPBufs) >> 1) & 1);
        my_abort = __any_sync(0xffffffffu, my_abort);  // tcgen05.ld below is warp-collective
        tc::fence_after_sync();
        // x = base-2 score + nmu (or the score alone), -inf where masked
        float x[HC];
        auto load_scores = [&](bool with_mu) {
          float lo[HC];
          kv4::tmem_ld16(t_s, x);
          kv4::tmem_ld16(t_s + NQ, lo);
          const float4* cs4 = reinterpret_cast<const float4*>(&ctl.cscale[c0]);
          const float4* nm4 = reinterpret_cast<const float4*>(&ctl.nmu[c0]);
          tc::tmem_wait_ld();
#pragma unroll
          for (int k4 = 0; k4 < HC / 4; ++k4) {
            const float4 cs = cs4[k4];
            const float4 nm = with_mu ? nm4[k4] : make_float4(0.f, 0.f, 0.f, 0.f);
            const float2 inv = make_float2(1.f / kQLoScale, 1.f / kQLoScale);
            float* xs = &x[4 * k4];
            const float* ls = &lo[4 * k4];
            float2 u = kv4::fma2(make_float2(ls[0], ls[1]), inv, make_float2(xs[0], xs[1]));
            float2 v = kv4::fma2(make_float2(ls[2], ls[3]), inv, make_float2(xs[2], xs[3]));
            u = kv4::fma2(u, make_float2(cs.x, cs.y), make_float2(nm.x, nm.y));
            v = kv4::fma2(v, make_float2(cs.z, cs.w), make_float2(nm.z, nm.w));
            xs[0] = u.x;
            xs[1] = u.y;
            xs[2] = v.x;
            xs[3] = v.y;
          }
          if (!all_vis) {
#pragma unroll
            for (int c = 0; c < HC; ++c) x[c] = ((vis >> c) & 1u) ? x[c] : -INFINITY;
          }
        };
        const bool first = t == t_first;  // there is no maximum yet
        bool need = false;
        const int done = t - t_first;
        // The sums so far: written in one tile, weighed up in the next, with its
        // meeting in between.  Lane c of each warp weighs column c0 + c; one that has
        // seen no key, or is no row, asks for nothing.
        if (kv4_looks_at_mean(done)) kv4::columns_to_smem<false>(acc, &ctl.sum[quad][c0], lane);
        float l = 0.f;
        bool small = false;
        if (kv4_looks_at_mean(done - 1) && lane < HC) {
          const int n = c0 + lane;
          l = (ctl.sum[0][n] + ctl.sum[1][n]) + (ctl.sum[2][n] + ctl.sum[3][n]);
          small = l > 0.f && l < (float)(done - 1) * (kKeys * kKv4MeanP) && n < nrows;
          need = small;
        }
        if (!my_abort && !first) {
          load_scores(true);
          float top = fmaxf(x[0], x[1]);
#pragma unroll
          for (int c = 2; c < HC; c += 2) top = kv4::max3(top, x[c], x[c + 1]);
          need = need || top > kKv4Limit;
        } else if (my_abort) {
#pragma unroll
          for (int c = 0; c < HC; ++c) x[c] = -INFINITY;
        }
        bool rescale = false;
        if (first || kv4::bar_any(bar_id, 128, need || my_abort || ctl.abort)) {
          // Rare but for a segment's first tile: a score passed the running max
          // by too much, a column saw its first key, its weights have become
          // small, or a wait gave up.
          const bool ab = __any_sync(0xffffffffu, my_abort) || ctl.abort;
          if (lane == 0) ctl.flag[warp] = ab ? 1 : 0;
          if (!my_abort) load_scores(false);
          kv4::columns_to_smem<true>(x, &ctl.red[quad][c0], lane);
          named_bar_sync(bar_id, 128);
          my_abort =
              (ctl.flag[4 * half] | ctl.flag[4 * half + 1] | ctl.flag[4 * half + 2] | ctl.flag[4 * half + 3]) != 0;
          if (my_abort) break;
          bool raised = false;
          if (j < HC) {
            const int n = c0 + j;
            const float cm = fmaxf(fmaxf(ctl.red[0][n], ctl.red[1][n]), fmaxf(ctl.red[2][n], ctl.red[3][n]));
            const float old = ctl.nmu[n];
            float al = 1.f;
            if (small && cm + old < kKv4Top) {
              const float up = ex2_approx(kKv4Top - cm - old);  // (cm = -inf: +inf)
              if (l * up < kKv4MaxSum) {
                al = up;
                ctl.nmu[n] = kKv4Top - cm;
                raised = true;
              }
            }
            if (cm + old > kKv4Limit) {  // old = +inf: the first visible key (cm = -inf gives NaN, no)
              const float nm = (old == INFINITY ? kKv4First : kKv4Top) - cm;
              al = old == INFINITY ? 0.f : ex2_approx(nm - old);
              ctl.nmu[n] = nm;
              raised = true;
            }
            ctl.alpha[n] = al;
          }
          rescale = kv4::bar_any(bar_id, 128, raised) && t > t_first;
#pragma unroll
          for (int c = 0; c < HC; ++c) {
            acc[c] *= ctl.alpha[c0 + c];
            x[c] += ctl.nmu[c0 + c] == INFINITY ? 0.f : ctl.nmu[c0 + c];
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.s_free[t & 1]);  // the S^T buffer may be overwritten
        // P^T(t) overwrites what O^T(t - kPBufs) read; a rescale of O^T needs all of them done.
        if (!p_free)
          my_abort = !kv4::wait(&ctl.pv_done[(t - Cfg::kPBufs) & 1], ((t - Cfg::kPBufs) >> 1) & 1, &ctl.abort);
        if (Cfg::kPBufs > 1 && rescale && !my_abort)
          my_abort = !kv4::wait(&ctl.pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1, &ctl.abort);
        my_abort = __any_sync(0xffffffffu, my_abort);
        tc::fence_after_sync();
        if (!my_abort && rescale) {
#pragma unroll 1
          for (int m = 0; m < 4 * (Cfg::kConcat ? 2 : 1); ++m) {
            const uint32_t col = Cfg::kConcat ? (m >> 1) * Cfg::kOStride + (m & 1) * NQ : m * Cfg::kOStride;
#pragma unroll 1
            for (int c = 0; c < HC; c += 8) {
              float v[8];
              tc::tmem_ld8(t_lane + col + c0 + c, v);
              tc::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] *= ctl.alpha[c0 + c + e];
              tc::tmem_st8(t_lane + col + c0 + c, v);
            }
          }
          tc::tmem_wait_st();
        }
        if (!my_abort) {
          const uint32_t dst = sP + (t % Cfg::kPBufs) * Cfg::kPBytes + j * 16 + half * Cfg::kPCore;
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const float p0 = ex2_approx(x[4 * k4 + 0]);  // x = -inf (masked) gives 0
            const float p1 = ex2_approx(x[4 * k4 + 1]);
            const float p2 = ex2_approx(x[4 * k4 + 2]);
            const float p3 = ex2_approx(x[4 * k4 + 3]);
            const float2 a01 = kv4::add2(make_float2(acc[4 * k4], acc[4 * k4 + 1]), make_float2(p0, p1));
            const float2 a23 = kv4::add2(make_float2(acc[4 * k4 + 2], acc[4 * k4 + 3]), make_float2(p2, p3));
            acc[4 * k4 + 0] = a01.x;
            acc[4 * k4 + 1] = a01.y;
            acc[4 * k4 + 2] = a23.x;
            acc[4 * k4 + 3] = a23.y;
            // through halves: 11 bits, far finer than the 8 to 9 kept
            const uint32_t h01 = kv4::cvt_f16x2(p0, p1), h23 = kv4::cvt_f16x2(p2, p3);
            const uint32_t u01 = kv4::cvt_e4m3x2_f16x2(h01), u23 = kv4::cvt_e4m3x2_f16x2(h23);
            uint32_t r01 = kv4::sub_f16x2(h01, kv4::cvt_f16x2_e4m3x2(u01));
            uint32_t r23 = kv4::sub_f16x2(h23, kv4::cvt_f16x2_e4m3x2(u23));
            hi[k4] = u01 | (u23 << 16);
            if constexpr (Cfg::kConcat) {
              r01 = kv4::mul_f16x2(r01, 0x50005000u);  // 32: kPLoScale
              r23 = kv4::mul_f16x2(r23, 0x50005000u);
              lo[k4] = kv4::cvt_e4m3x2_f16x2(r01) | (kv4::cvt_e4m3x2_f16x2(r23) << 16);
            } else {
              lo[k4] = kv4::cvt_e5m2x2_f16x2(r01) | (kv4::cvt_e5m2x2_f16x2(r23) << 16);
            }
          }
          kv4::sts128(dst, hi[0], hi[1], hi[2], hi[3]);
          kv4::sts128(dst + (NQ / 16) * Cfg::kPCore, lo[0], lo[1], lo[2], lo[3]);
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0 && !my_abort) mbar_arrive(&ctl.p_full[t & 1]);
      }

      // ---- the segment's end: l, LSE, O = O^T / l -----------------------------
      named_bar_sync(bar_id, 128);  // (a raise of the last tile has read red)
      kv4::columns_to_smem<false>(acc, &ctl.red[quad][c0], lane);
      if (!my_abort) my_abort = !kv4::wait(&ctl.pv_done[(t_end - 1) & 1], ((t_end - 1) >> 1) & 1, &ctl.abort);
      tc::fence_after_sync();
      if (kv4::bar_any(bar_id, 128, my_abort || ctl.abort)) {
        my_abort = true;
        break;
      }
      if (j < HC) {
        const int n = c0 + j;
        const float l = (ctl.red[0][n] + ctl.red[1][n]) + (ctl.red[2][n] + ctl.red[3][n]);
        ctl.alpha[n] = l == 0.f ? 0.f : 1.f / l;
        // A row that is not a number gets +inf: the largest of its LSEs in any merge,
        // where its weight exp(inf - inf) makes the row NaN.  (A NaN would be passed
        // over by their maxima, and the row would read as one that sees nothing.)
        if (n < nrows)
          a.part_lse[sg.prow + n] = l == 0.f ? -INFINITY
                                    : l != l ? INFINITY
                                             : (__log2f(l) - ctl.nmu[n]) * 0.69314718055994530942f;
      }
      named_bar_sync(bar_id, 128);
      // Thread (quad, lane) holds latent column 128m + j of rows c0..c0+HC: a
      // warp store writes 128 contiguous bytes of one row.  Rows with nothing
      // visible are not written (their LSE is -inf).
      float* ocol = a.part_o + (sg.prow + c0) * kDLatent + j;
#pragma unroll 1
      for (int m = 0; m < 4; ++m, ocol += 128) {
        float v[16];
        kv4::tmem_ld16(t_lane + m * Cfg::kOStride + c0, v);
        if constexpr (Cfg::kConcat) {
          float lo[16];
          kv4::tmem_ld16(t_lane + m * Cfg::kOStride + NQ + c0, lo);
          tc::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] = fmaf(lo[c], 1.f / kPLoScale, v[c]);
        } else {
          tc::tmem_wait_ld();
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float inv = ctl.alpha[c0 + c];
          if (c0 + c < nrows && inv != 0.f) ocol[c * kDLatent] = v[c] * inv;
        }
      }
      tc::fence_before_sync();  // O^T may be overwritten once P^T of the next tile is written
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.seg_empty[k & 1]);
    }
  }

  // ---- teardown ---------------------------------------------------------------
  __syncthreads();
  if (tid == 0 && ctl.abort) atomicOr(a.status, kStatusTimeout);
  if (warp == Cfg::kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int NQ>
cudaError_t launch_split_kv4_nq(const SplitArgs& a, dim3 grid, cudaStream_t stream) {
  constexpr int smem = kv4_smem_bytes<NQ>();
  static_assert(smem <= 232448, "shared memory budget exceeded");
  cudaError_t e = cudaFuncSetAttribute(split_kv4_kernel<NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  split_kv4_kernel<NQ><<<grid, Kv4Cfg<NQ>::kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mlav
