// Tensor-core (tcgen05) attention for requests that share prefixes, by pairs of
// CTAs (a cluster of two).
//
// A pair takes a row group -- up to 128 query rows (token, head pairs; of all the
// requests of a group, or of one request) -- and a run of 64-key tiles, and
// leaves the group's partial softmax statistics for the merge.  Query rows sit on
// the MMA's M = 128, so an fp32 O of 512 latent columns would fill tensor memory
// (128 lanes x 512 columns).  The pair shares the work of a tile: CTA c takes the
// scores and the softmax of 32 of its keys, and half of O's columns,
//   S_c[128 x 32]   = Q[128 x 576] . K_c^T             (36 MMAs, K = 16, N = 32)
//   O_c[128 x 256] += P[128 x 64] . V[64 x 256 of 512] (4 MMAs, K = 16, N = 256)
// and sends its half of P to the other CTA: 64 bytes per row and tile.  (Splitting
// the latent columns in both products was built first.  It gathers a quarter less
// and its MMAs are 1.3 times shorter, but it sends scores, 256 bytes per row and
// tile: between two CTAs pass about 19 bytes per clock, and stores on their way
// there hold up every other shared-memory access.  128k keys x 2048 rows took
// 859 us so.)
//
// Even and odd tiles of a row group go to two sets of four softmax warps, a thread
// per query row and 32 keys, each with places of its own for scores and weights:
// one set's chain -- scores, weights, the other CTA's half, about 3,000 cycles --
// overlaps the other's.  A set keeps, per row, a reference for its weights,
// p = 2^(s - m); the CTA keeps one for O, M, handed from tile to tile.  References
// are 16 + a multiple of 32, so they are mostly the same one, and where they are
// not the weights change from one to the other exactly.
//
// Three warps issue MMAs: even tiles' scores, odd tiles' scores, values.  (A warp
// that has issued MMAs and a commit gets to its next wait only when they are nearly
// done, and then needs 400 to 500 cycles up to its next MMA: one warp for all kept
// the tensor pipe at 60 %; 128k keys x 2048 rows took 582 us.)
//
// A operands in tensor memory spare shared memory: with A there an MMA with N = 32
// takes 16 cycles, with A in shared memory 40.  What fits is Q's first 384
// channels (192 columns of bf16 pairs); the other 192 channels and P are in shared
// memory (with N = 256 an MMA takes 128 cycles either way).  Tensor memory: O
// 0..255, Q 256..447, S 448..479 (even tiles) and 480..511 (odd).
//
// Shared memory, in blocks of 64 columns (128 bytes) of keys or query rows, 128-byte
// swizzled -- the K-major layout of the score product and the MN-major one of the
// value product's B: Q's three blocks; a ring of what only the scores read (of this
// CTA's 32 keys the other CTA's half of the latent, and the RoPE columns), which
// the score product reads first; rings of values (this CTA's half) of its own keys
// and of the other CTA's.  Weights, both CTAs', stand in pieces of eight keys by all
// rows, K-major and not swizzled, so that a warp sends 512 bytes in a row: 16-byte
// pieces of a swizzled row go between CTAs at a quarter of that rate.
//
// Warps: 0-7 softmax (they also bring Q in and take O out of tensor memory), 8, 9
// and 11 issue the MMAs, 10 gathers the other CTA's keys, 12-15 own keys, with
// 16-byte cp.async.
//
// Work in equal pieces: the row groups of all groups' shared parts, then of all
// requests' own parts, each as long as its tiles and what its start and end cost,
// form an axis; pair w takes the w-th of equal pieces (every CTA sums up the lengths
// itself).  Pairs at the same prefix go through it in step, so that its rows come
// from L2 for all but the first.  Row group with first row R (0 .. rows_max for
// shared parts, rows_max .. for own ones) leaves pair w's partial at row R + 128 w,
// and the table's entry R says which pairs have one.
//
// What bounds it: shared memory and the tensor pipe.  A tile takes 1,650 to 1,750
// cycles of a CTA; its MMAs alone 1,376, its 200 KB of shared-memory traffic (48 of
// it Q, 52 the gather's) 1,560 at 128 bytes per cycle.  A row group's start and end
// cost 20,000 cycles: Q in, the first scores, the last exchange, 131 KB of O out.
// 2048 rows behind 128k shared keys: 440 us, 1.35 PFLOP/s (0.71 of the measured
// peak); 9216 rows behind 8k, 161 us; 512 rows behind 32k, 66 us.
//
// Every wait is bounded; on a timeout the CTA raises the status bit and drains,
// and the other CTA of the pair runs into its own limit.
#include <cooperative_groups.h>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace mlav {
namespace {

namespace cg = cooperative_groups;

constexpr int kRows = kSharedRows, kKeys = kSharedKeys;
constexpr int kOwnKeys = kKeys / 2;             // a CTA's keys of a tile
constexpr int kHalfLatent = kDLatent / 2;
constexpr int kBlockBytes = kOwnKeys * 128;     // 64 columns of 32 keys
constexpr int kQBlock = kRows * 128;            // 64 columns of Q
constexpr int kQSteps = 24;                     // k-steps of 16 channels with Q in tensor memory (6 blocks)
// Rings.  Of this CTA's keys: the half of the latent that only the scores read, with the RoPE columns, and the half
// that the values need too; of the other CTA's keys the latter half.
constexpr int kScoreStages = 2, kScoreBytes = 5 * kBlockBytes;
constexpr int kOwnStages = 4, kOtherStages = 2, kValueBytes = 4 * kBlockBytes;
constexpr int kPPiece = kRows * 16;               // eight keys' weights of all rows
constexpr int kPBytes = 2 * (kOwnKeys / 8) * kPPiece;  // a CTA's weights of two tiles
constexpr int kSoftmaxWarps = 8;
constexpr int kMmaWarp = kSoftmaxWarps;                      // and the next: issue the score products
constexpr int kOtherWarp = kMmaWarp + 2, kOtherWarps = 1;    // gathers the other CTA's keys
constexpr int kValueWarp = kMmaWarp + 3;                     // issues the value products
constexpr int kGatherWarp = kMmaWarp + 4, kGatherWarps = 4;  // gather own keys (a warpgroup of their own: registers)
constexpr int kThreads = 32 * (kGatherWarp + kGatherWarps);
// Registers per thread by warpgroup; together at most the 4 x 128 of the launch.
constexpr int kRegsSoftmax = 144, kRegsMma = 112, kRegsGather = 112;
static_assert(kThreads == 512 && 2 * kRegsSoftmax + kRegsMma + kRegsGather <= 512, "register shares");
constexpr int kKeysPerWarp = kOwnKeys / kGatherWarps;  // own keys gathered by a warp
constexpr int kColO = 0, kColQ = 256, kColS = 448;  // (S: 32 columns for even tiles, 32 for odd ones)
// Base 2, before a reference is raised.  Weights and O are floating numbers, so a
// reference far below the maximum costs no precision; what it must not do is overflow.
constexpr float kRowHeadroom = 16.0f, kOutHeadroom = 32.0f;
// References are 16 + a multiple of 32: those of both CTAs, and of O, are mostly the same one.  (Above 2^23: the largest score.)
constexpr float kRefStep = 32.0f, kRefOffset = 16.0f;
// Start and end of a row group, in tiles: so much and so much per 32 rows.
constexpr int kSegCost = 5, kQuadCost = 2;
constexpr int kMaxSpans = 2 * kMaxSharedBatch;
constexpr int64_t kAxisEnd = 0xFFFFFFFF;  // (2^32 tiles would take half a day)

struct Ctl {
  uint64_t full[kOwnStages], empty_own[kOwnStages], empty_score[kScoreStages];
  uint64_t full_other[kOtherStages], empty_other[kOtherStages];
  uint64_t q_full, s_full[2], s_free[2], p_full[2], pv_done[2], x_full[2], l_full, mma_idle;  // [2]: even, odd tiles
  uint64_t m_set[2][4];  // by quarter of the rows: a tile's M stands in m_row
  uint32_t tmem_base;
  int abort;
  alignas(4) uint8_t valid[kOwnStages][kGatherWarps];  // own keys of a tile that exist, 8 bits per gather warp
  float m_row[kRows];                  // reference of O
  float x_ref[2][kRows];               // the other CTA's references, with its weights
  float sum[2][3][kRows];              // at the end of a row group: references and sums of even and odd tiles,
  alignas(16) float4 x_sum[2][kRows];  // and the other CTA's
  uint32_t some[kMaxSpans / 32];  // which spans of the axis have a length
  int64_t warp_sum[kThreads / 32];
};

constexpr int kOffScore = 3 * kQBlock;
constexpr int kOffOwn = kOffScore + kScoreStages * kScoreBytes;
constexpr int kOffOther = kOffOwn + kOwnStages * kValueBytes;
constexpr int kOffP = kOffOther + kOtherStages * kValueBytes;
constexpr int kOffX = kOffP + kPBytes;
constexpr int kOffCtl = kOffX + kPBytes;
constexpr int kOffEnds = kOffScore;  // the axis, while it is set up
constexpr int kSmem = kOffCtl + (int)sizeof(Ctl) + 1024;  // (alignment slack)
static_assert(kMaxSpans * 4 <= kOffP - kOffEnds && kGatherWarps == 4, "places in shared memory");

// ---- wider TMEM accesses ------------------------------------------------------
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// D = A*B (+ D): A from tensor memory, B from shared memory.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// mbar_wait_spin by a whole warp, with no look at the clock for the first polls.
__device__ __forceinline__ bool wait_spin(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
#pragma unroll 1
  for (int it = 0; it < 64; ++it)
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, abort, status));
}

// mbar_wait by a whole warp: one test where the phase is over already, as it mostly is.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

// ---- the other CTA of the pair -------------------------------------------------
// Arrive once on `bar` of the other CTA when every MMA issued before by this thread completes.
__device__ __forceinline__ void commit_to(uint64_t* bar, uint32_t rank) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)(1u << rank))
      : "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// 16 bytes into the other CTA's shared memory, counted by its barrier.
__device__ __forceinline__ void send16(uint32_t dst, uint32_t bar, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(dst), "r"(a), "r"(b),
      "r"(c), "r"(d), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void send4(uint32_t dst, uint32_t bar, float a) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(dst),
               "r"(__float_as_uint(a)), "r"(bar)
               : "memory");
}
// 2^(a - b) of whole numbers (a = -inf: 0).
__device__ __forceinline__ float ratio(float a, float b) {
  const float d = a - b;
  return d >= -126.f ? __int_as_float(((int)fminf(d, 127.f) + 127) << 23) : 0.f;
}
// Weights from one reference to another (an exact product).
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t w, uint32_t f) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(f));
  return r;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// A row's 32 weights in shared memory, by a power of two.
__device__ __forceinline__ void scale_weights(uint32_t at, float by) {
  const uint32_t f = __float_as_uint(by) >> 16, f2 = f | f << 16;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t x[4];
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(at + c * kPPiece)
                 : "memory");
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = scale_bf16x2(x[k], f2);
    sts128(at + c * kPPiece, x[0], x[1], x[2], x[3]);
  }
}

template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// ---- the axis --------------------------------------------------------------------
// Span e: the shared part of group e, or the own part of request e - groups.
struct Span {
  int64_t kv0;     // first entry of its index array
  int64_t q0;      // first token row
  int64_t mask0;   // own parts: first mask bit
  int64_t keys;
  int64_t prefix;  // keys in the index array (the rest: drafts)
  int ntok;
  bool own;
};

__device__ __forceinline__ void token_range(const SharedArgs& a, int r0, int r1, int64_t& q0, int& n) {
  int64_t most = (int64_t)(r1 - r0) * a.T;
  if (most < 0) most = 0;
  q0 = (int64_t)r0 * a.T;
  int64_t m = most;
  if (a.qo_indptr) {
    q0 = a.qo_indptr[r0];
    m = (int64_t)a.qo_indptr[r1 > r0 ? r1 : r0] - q0;
  }
  // (what the contract gives; rows outside the partials would be written otherwise)
  const int64_t all = (int64_t)a.batch * a.T;
  if (q0 < 0 || q0 > all) q0 = all;
  if (m > most) m = most;
  if (m > all - q0) m = all - q0;
  n = m < 0 ? 0 : (int)m;
}

__device__ __forceinline__ Span span_of(const SharedArgs& a, int e) {
  Span s;
  s.own = e >= a.groups;
  if (!s.own) {
    auto clip = [&](int r) { return r < 0 ? 0 : r > a.batch ? a.batch : r; };
    const int r0 = e == 0 ? 0 : clip(a.group_indptr[e]);
    const int r1 = e == a.groups - 1 ? a.batch : clip(a.group_indptr[e + 1]);
    token_range(a, r0, r1, s.q0, s.ntok);
    s.kv0 = a.shared_indptr[e];
    s.prefix = a.shared_indptr[e + 1] - s.kv0;
    s.prefix = s.prefix < 0 ? 0 : s.prefix;
    s.keys = s.prefix;
    s.mask0 = 0;
  } else {
    const int b = e - a.groups;
    token_range(a, b, b + 1, s.q0, s.ntok);
    s.kv0 = a.kv_indptr[b];
    s.prefix = a.kv_indptr[b + 1] - s.kv0;
    s.prefix = s.prefix < 0 ? 0 : s.prefix;
    s.keys = s.prefix + s.ntok;
    s.mask0 = a.mask_indptr[b];
  }
  return s;
}
__device__ __forceinline__ int64_t groups_of(const SharedArgs& a, const Span& s) {
  return ((int64_t)s.ntok * a.H + kRows - 1) / kRows;
}
__device__ __forceinline__ int seg_cost(const SharedArgs& a, const Span& s) {
  const int64_t rows = (int64_t)s.ntok * a.H;
  return kSegCost + kQuadCost * (rows < kRows ? (int)(rows + 31) / 32 : 4);
}
__device__ __forceinline__ int64_t tiles_of(const Span& s) { return (s.keys + kKeys - 1) / kKeys; }

// Where a pair is on the axis; every role of its CTAs walks it by itself.
struct Cursor {
  const uint32_t* some;  // bit e: span e has a length
  int spans, e;
  int64_t start;  // of span e
  int64_t x, x_end, piece;
  int pair;
};
struct Segment {
  Span s;
  int64_t row0;   // first row (of all tokens' rows)
  int64_t place;  // of the row group: row0, or rows_max + row0
  int r0;         // first row within the span
  int nrows;
  int64_t tile0;
  int nt;
  int turn;       // of a shared part: the run starts this many tiles behind tile0, and ends before it
  int64_t first_pair;
  int pairs;  // that have a partial of it
  __device__ __forceinline__ int tile(int t) const { return t + turn < nt ? t + turn : t + turn - nt; }
};

// Row id of key `key` + tiles of the segment; -1 where there is no such key.
__device__ __forceinline__ int32_t load_id(const SharedArgs& a, const Segment& g, int64_t key, int t) {
  const int64_t j = key + (int64_t)g.tile(t) * kKeys;
  if (t >= g.nt || j >= g.s.keys) return -1;
  return j < g.s.prefix ? __ldg((g.s.own ? a.kv_indices : a.shared_indices) + g.s.kv0 + j)
                        : __ldg(a.out_cache_loc + g.s.q0 + (j - g.s.prefix));
}

// First span with a length from span e on.
__device__ __forceinline__ int next_span(const Cursor& c, int e) {
  while (e < c.spans) {
    const uint32_t w = c.some[e >> 5] >> (e & 31);
    if (w) return e + __ffs(w) - 1;
    e = (e | 31) + 1;
  }
  return c.spans;
}

// The next row group and run of tiles of the pair; false at the end of its piece.
__device__ __forceinline__ bool next_segment(const SharedArgs& a, Cursor& c, Segment& g) {
  while (c.x < c.x_end) {
    if (c.e >= c.spans) return false;
    g.s = span_of(a, c.e);
    const int cost = seg_cost(a, g.s);
    const int64_t tiles = tiles_of(g.s), len = tiles + cost, all = groups_of(a, g.s) * len;
    if (c.start + all <= c.x) {
      c.start += all;
      c.e = next_span(c, c.e + 1);
      continue;
    }
    // (the axis has less than 2^32 tiles)
    const int64_t i = (uint32_t)(c.x - c.start) / (uint32_t)len, e0 = c.start + i * len, e1 = e0 + len;
    g.r0 = (int)(i * kRows);
    const int64_t left = (int64_t)g.s.ntok * a.H - g.r0;
    g.nrows = left < kRows ? (int)left : kRows;
    g.row0 = g.s.q0 * a.H + g.r0;
    g.place = g.row0 + (g.s.own ? a.rows_max : 0);
    const int64_t stop = c.x_end < e1 ? c.x_end : e1;
    int64_t t0 = c.x - e0 - cost, t1 = stop - e0 - cost;
    t0 = t0 < 0 ? 0 : t0;
    const bool heads = c.x == e0;  // this pair has the row group's start on the axis
    c.x = stop;
    g.tile0 = t0;
    g.nt = t1 > t0 ? (int)(t1 - t0) : 0;
    // Pairs at the same prefix read the same keys at the same time, as far as it goes: at its tile u a pair is at tile u
    // modulo the piece.  (Each starting with its first tile, a prefix larger than L2 came from memory for every pair.)
    g.turn = 0;
    if (!g.s.own) {
      const int64_t u = e0 + cost + t0 - c.pair * c.piece;
      const int64_t off = (u - t0) % c.piece, turn = off < 0 ? off + c.piece : off;
      if (turn < g.nt) g.turn = (int)turn;
    }
    g.first_pair = (uint32_t)(e0 + cost) / (uint32_t)c.piece;
    g.pairs = tiles ? (int)((uint32_t)(e1 - 1) / (uint32_t)c.piece - g.first_pair + 1) : 0;
    if (g.nt > 0 || heads) return true;
  }
  return false;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    split_shared_kernel(const __grid_constant__ SharedArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  const uint32_t pad = ((raw_addr + 1023u) & ~1023u) - raw_addr;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_addr + pad;
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + kOffCtl);
  uint32_t* ends = reinterpret_cast<uint32_t*>(smem + kOffEnds);
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- set-up: barriers, tensor memory, the axis ------------------------------------
  if (tid == 0) {
    for (int k = 0; k < kOwnStages; ++k) {
      mbar_init(&ctl.full[k], kGatherWarps * 33);  // every lane's copies and, per warp, its valid bits
      mbar_init(&ctl.empty_own[k], 1);
    }
    for (int k = 0; k < kOtherStages; ++k) {
      mbar_init(&ctl.full_other[k], kOtherWarps * 32);
      mbar_init(&ctl.empty_other[k], 1);
    }
    for (int k = 0; k < kScoreStages; ++k) mbar_init(&ctl.empty_score[k], 1);
    mbar_init(&ctl.q_full, kSoftmaxWarps);
    for (int k = 0; k < 2; ++k) {
      mbar_init(&ctl.s_full[k], 2);  // the product, and the issuing lane (which has seen the tile's valid bits)
      mbar_init(&ctl.s_free[k], kSoftmaxWarps / 2);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(&ctl.p_full[k], kSoftmaxWarps / 2);
      mbar_init(&ctl.pv_done[k], 2);  // of both CTAs
      mbar_init(&ctl.x_full[k], 1);
      for (int q = 0; q < 4; ++q) mbar_init(&ctl.m_set[k][q], 1);
    }
    mbar_init(&ctl.l_full, 1 + kSoftmaxWarps);
    mbar_init(&ctl.mma_idle, 3);
    ctl.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&ctl.tmem_base, 512);
    tc::tmem_relinquish();
  }
  Cursor cur;
  cur.some = ctl.some;
  cur.spans = a.groups + a.batch;
  {
    int64_t carry = 0;
    for (int base = 0; base < cur.spans; base += kThreads) {
      const int e = base + tid;
      int64_t v = 0;
      if (e < cur.spans) {
        const Span s = span_of(a, e);
        v = groups_of(a, s) * (tiles_of(s) + seg_cost(a, s));
      }
      const int64_t len = v;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      if (lane == 31) ctl.warp_sum[warp] = v;
      const uint32_t some = __ballot_sync(0xffffffffu, len > 0);
      if (lane == 0 && e < kMaxSpans) ctl.some[e >> 5] = some;
      __syncthreads();
      int64_t before = carry;
      for (int w = 0; w < warp; ++w) before += ctl.warp_sum[w];
      if (e < cur.spans) ends[e] = (uint32_t)(before + v < kAxisEnd ? before + v : kAxisEnd);
      for (int w = 0; w < kThreads / 32; ++w) carry += ctl.warp_sum[w];
      __syncthreads();
    }
    carry = carry < kAxisEnd ? carry : kAxisEnd;
    const int64_t pairs = a.clusters;
    cur.piece = (carry + pairs - 1) / pairs;
    cur.piece = cur.piece < 1 ? 1 : cur.piece;
    cur.pair = blockIdx.x >> 1;
    cur.x = cur.pair * cur.piece;
    cur.x_end = cur.x + cur.piece < carry ? cur.x + cur.piece : carry;
    int lo = 0, hi = cur.spans;  // first span that ends behind x
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ends[mid] <= cur.x)
        lo = mid + 1;
      else
        hi = mid;
    }
    cur.e = lo;
    cur.start = lo ? ends[lo - 1] : 0;
  }
  tc::fence_before_sync();
  cluster.sync();
  tc::fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;

  if (warp >= kGatherWarp) {
    fewer_registers<kRegsGather>();
    // ============================ gather ================================================
    // Own keys: warp gw fills eight of the 32.  An instruction copies 128 bytes of four keys, a lane 16 bytes of key
    // lane/8 or lane/8 + 4; a row's pieces then differ by constants.
    const int gw = warp - kGatherWarp;
    uint32_t bad = 0;
    uint32_t tt = 0, sa = 0, pa = 1, so = 0, po = 1;  // tiles so far; places in the two rings and their parities
    bool stop = false;
    Segment g;
    const int sub = lane >> 3, chunk = lane & 7;
    // (the swizzle takes the key's last three bits: those of keys sub and sub + 4 of the eight)
    const uint32_t to = (gw * kKeysPerWarp + sub) * 128, to_a = to + ((chunk ^ sub) << 4),
                   to_b = to + 512 + ((chunk ^ (sub + 4)) << 4);
    while (!stop && next_segment(a, cur, g)) {
      const int64_t key0 = g.tile0 * kKeys + kOwnKeys * rank + gw * kKeysPerWarp + chunk;  // (the lanes hold them four times)
      int32_t id0 = load_id(a, g, key0, 0), id1 = load_id(a, g, key0, 1);
#pragma unroll 1
      for (int t = 0; t < g.nt; ++t, ++tt) {
        int32_t row = id0;
        id0 = id1;
        id1 = load_id(a, g, key0, t + 2);
        const bool ok = row >= 0 && row < a.pool_rows;
        if (!ok && key0 + (int64_t)g.tile(t) * kKeys < g.s.keys) bad = 1;
        row = ok ? row : -1;
        const uint32_t valid = __ballot_sync(0xffffffffu, ok) & 0xFFu;
        const __nv_bfloat16* src[2];
        uint32_t n[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int32_t r = __shfl_sync(0xffffffffu, row, 4 * k + sub);
          n[k] = r < 0 ? 0u : 16u;
          src[k] = a.kv_pool + (int64_t)(r < 0 ? 0 : r) * kDRow + chunk * 8;
        }
        if (!wait_warp(&ctl.empty_score[sa], pa, &ctl.abort, a.status) ||
            !wait_warp(&ctl.empty_own[so], po, &ctl.abort, a.status)) {
          stop = true;
          break;
        }
        if (!(a.test_stall && tt == 0)) {  // test only: the first tile never lands
          if (lane == 0) ctl.valid[so][gw] = (uint8_t)valid;
          const uint32_t score = sbase + kOffScore + sa * kScoreBytes, value = sbase + kOffOwn + so * kValueBytes;
          const uint32_t half[2] = {rank == 0 ? value : score, rank == 0 ? score : value};
#pragma unroll
          for (int blk = 0; blk < 8; ++blk) {
            const uint32_t dst = half[blk >> 2] + (blk & 3) * kBlockBytes;
            cp_async16(dst + to_a, src[0] + 64 * blk, n[0]);
            cp_async16(dst + to_b, src[1] + 64 * blk, n[1]);
          }
          cp_async16(score + 4 * kBlockBytes + to_a, src[0] + kDLatent, n[0]);
          cp_async16(score + 4 * kBlockBytes + to_b, src[1] + kDLatent, n[1]);
          cp_async_arrive(&ctl.full[so]);
          if (lane == 0) mbar_arrive(&ctl.full[so]);
        }
        if (++sa == kScoreStages) {
          sa = 0;
          pa ^= 1u;
        }
        if (++so == kOwnStages) {
          so = 0;
          po ^= 1u;
        }
      }
    }
    cp_async_wait_all();
    if (bad) atomicOr(a.status, kStatusBadRow);
  } else if (warp >= kMmaWarp) {
    fewer_registers<kRegsMma>();
    if (warp != kOtherWarp) {
      // ============================ MMA issue ==============================================
      // Two warps issue the score products, of even and of odd tiles, one the value products: each waits for its own
      // operands, and the tensor pipe has another one's to do meanwhile.  A whole warp walks the loop and one elected lane
      // issues, so that what an MMA takes its descriptors from stays warp-uniform.
      const bool leader = elect_one();
      bool ok = true;
      Segment g;
      if (warp != kValueWarp) {
        const int h = warp - kMmaWarp;
        constexpr uint32_t idesc = tc::idesc_bf16_f32(kRows, kOwnKeys, false, false);
        const uint64_t desc_q = tc::smem_desc(sbase, 16, 1024, tc::kSwizzle128B);
        const uint64_t desc_s = tc::smem_desc(sbase + kOffScore, 16, 1024, tc::kSwizzle128B);
        const uint64_t desc_k = tc::smem_desc(sbase + kOffOwn, 16, 1024, tc::kSwizzle128B);
        const uint32_t d_s = tmem + kColS + 32 * h;
        uint32_t before = 0, seg = 0, uses = 0;  // tiles of the row groups before; tiles of this parity so far
        while (ok && next_segment(a, cur, g)) {
          if (g.nt == 0) continue;
          ok = wait_spin(&ctl.q_full, seg & 1u, &ctl.abort, a.status);
          ++seg;
          for (int t = h; ok && t < g.nt; t += 2, ++uses) {
            const uint32_t tile = before + t;
            if (uses > 0) ok = wait_spin(&ctl.s_free[h], (uses - 1) & 1u, &ctl.abort, a.status);
            ok = ok && wait_spin(&ctl.full[tile % kOwnStages], tile / kOwnStages & 1u, &ctl.abort, a.status);
            if (!ok) break;
            fence_proxy_async_smem();
            tc::fence_after_sync();
            const uint64_t ds = desc_s + (tile % kScoreStages) * (uint32_t)(kScoreBytes >> 4),
                           dv = desc_k + (tile % kOwnStages) * (uint32_t)(kValueBytes >> 4);
            if (leader) {
              // What only the scores read goes first, so that its place is free for the next tile but one sooner.
              const bool low = rank == 0;  // the values' half of the latent is channels 0..255
              auto product = [&](uint64_t keys, int k, uint32_t accumulate) {  // latent channels 16 k .. + 15
                const uint64_t d = keys + (uint32_t)((((k >> 2) & 3) * kBlockBytes + (k & 3) * 32) >> 4);
                if (k < kQSteps)
                  mma_bf16_ts(d_s, tmem + kColQ + 8 * k, d, idesc, accumulate);
                else
                  tc::mma_bf16_ss(d_s, desc_q + (uint32_t)((((k - kQSteps) >> 2) * kQBlock + (k & 3) * 32) >> 4), d, idesc,
                                  accumulate);
              };
              if (low) {
#pragma unroll
                for (int k = 16; k < 32; ++k) product(ds, k, k > 16);
              } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) product(ds, k, k > 0);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc::mma_bf16_ss(d_s, desc_q + (uint32_t)((2 * kQBlock + k * 32) >> 4),
                                ds + (uint32_t)((4 * kBlockBytes + k * 32) >> 4), idesc, 1u);
              tc::mma_commit(&ctl.empty_score[tile % kScoreStages]);
              if (low) {
#pragma unroll
                for (int k = 0; k < 16; ++k) product(dv, k, 1u);
              } else {
#pragma unroll
                for (int k = 16; k < 32; ++k) product(dv, k, 1u);
              }
              tc::mma_commit(&ctl.s_full[h]);
              mbar_arrive(&ctl.s_full[h]);
            }
          }
          before += g.nt;
        }
      } else {
        constexpr uint32_t idesc = tc::idesc_bf16_f32(kRows, kHalfLatent, false, true);
        const uint64_t desc_v = tc::smem_desc(sbase + kOffOwn, kBlockBytes, 1024, tc::kSwizzle128B);
        const uint64_t desc_o = tc::smem_desc(sbase + kOffOther, kBlockBytes, 1024, tc::kSwizzle128B);
        // (weights, not swizzled: eight keys of eight rows in 128 bytes, the rows' next eight behind them)
        const uint64_t desc_p = tc::smem_desc(sbase + kOffP, kPPiece, 128, 0);
        const uint64_t desc_x = tc::smem_desc(sbase + kOffX, kPPiece, 128, 0);
        uint32_t tile = 0, uses0 = 0, uses1 = 0;
        while (ok && next_segment(a, cur, g)) {
          for (int t = 0; ok && t < g.nt; ++t, ++tile) {
            const uint32_t h = t & 1;
            ok = wait_spin(&ctl.full_other[tile % kOtherStages], tile / kOtherStages & 1u, &ctl.abort, a.status) &&
                 wait_spin(&ctl.p_full[h], (h ? uses1 : uses0) & 1u, &ctl.abort, a.status);
            if (!ok) break;
            uses0 += h ^ 1u;
            uses1 += h;
            fence_proxy_async_smem();
            tc::fence_after_sync();
            const uint64_t dv = desc_v + (tile % kOwnStages) * (uint32_t)(kValueBytes >> 4),
                           dx = desc_o + (tile % kOtherStages) * (uint32_t)(kValueBytes >> 4);
            if (leader) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {  // own keys, then the other CTA's
                tc::mma_bf16_ss(tmem + kColO, (k < 2 ? desc_p : desc_x) + (4 * h + 2 * (k & 1)) * (uint32_t)(kPPiece >> 4),
                                (k < 2 ? dv : dx) + (uint32_t)((k & 1) * 2048 >> 4), idesc, t > 0 || k > 0);
                if (k == 1) tc::mma_commit(&ctl.empty_own[tile % kOwnStages]);
              }
              tc::mma_commit(&ctl.pv_done[h]);
              commit_to(&ctl.pv_done[h], rank ^ 1u);
              tc::mma_commit(&ctl.empty_other[tile % kOtherStages]);
            }
          }
        }
      }
      // Drain: every MMA of the three warps has completed before tensor memory is freed.
      if (leader) tc::mma_commit(&ctl.mma_idle);
      const uint64_t t0 = global_timer_ns();
      for (uint32_t it = 0; it < (1u << 30); ++it)
        if (mbar_try_wait(&ctl.mma_idle, 0) || ((it & 63u) == 63u && global_timer_ns() - t0 > kWaitLimitNs)) break;
      __syncwarp();
    } else {
      // ==================== gather: the other CTA's keys, this CTA's half of the latent ====================
      // 128 bytes of four keys per instruction.
      const int sub = lane >> 3, chunk = lane & 7;
      uint32_t so = 0, po = 1;
      bool stop = false;
      Segment g;
      const uint32_t to_a = sub * 128 + ((chunk ^ sub) << 4), to_b = sub * 128 + ((chunk ^ (sub + 4)) << 4);
      while (!stop && next_segment(a, cur, g)) {
        const int64_t key0 = g.tile0 * kKeys + kOwnKeys * (rank ^ 1u) + lane;
        int32_t id0 = load_id(a, g, key0, 0), id1 = load_id(a, g, key0, 1);
#pragma unroll 1
        for (int t = 0; t < g.nt; ++t) {
          const int32_t row = id0 >= 0 && id0 < a.pool_rows ? id0 : -1;  // (the CTA that they belong to reports bad ones)
          id0 = id1;
          id1 = load_id(a, g, key0, t + 2);
          if (!wait_warp(&ctl.empty_other[so], po, &ctl.abort, a.status)) {
            stop = true;
            break;
          }
          const uint32_t value = sbase + kOffOther + so * kValueBytes;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int32_t r = __shfl_sync(0xffffffffu, row, 4 * k + sub);
            const __nv_bfloat16* src = a.kv_pool + (int64_t)(r < 0 ? 0 : r) * kDRow + rank * kHalfLatent + chunk * 8;
#pragma unroll
            for (int blk = 0; blk < 4; ++blk)
              cp_async16(value + blk * kBlockBytes + 512 * k + (k & 1 ? to_b : to_a), src + 64 * blk, r < 0 ? 0u : 16u);
          }
          cp_async_arrive(&ctl.full_other[so]);
          if (++so == kOtherStages) {
            so = 0;
            po ^= 1u;
          }
        }
      }
      cp_async_wait_all();
    }
  } else {
    more_registers<kRegsSoftmax>();
    // ============================ softmax ================================================
    const int quad = warp & 3, half = warp >> 2;
    const int r = 32 * quad + lane;  // query row in the group = TMEM lane
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quad) << 16);
    // Scores are kept unscaled, as S or, for a negative scale, -S; a scale of 0 becomes one that no difference survives.
    const float scale = fmaxf(fabsf(a.scale_log2), 1e-30f);
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
    const uint64_t scale2 = pair(scale, scale);
    const uint32_t other = rank ^ 1u;
    const uint32_t p_own = sbase + kOffP + 4 * half * kPPiece + r * 16, x_own = p_own + (kOffX - kOffP);
    const uint32_t x_peer = peer_addr(x_own, other);
    const uint32_t ref_peer = peer_addr(smem_u32(&ctl.x_ref[half][r]), other);
    const uint32_t sum_peer = peer_addr(smem_u32(&ctl.x_sum[half][r]), other);
    const uint32_t bar_peer = peer_addr(smem_u32(&ctl.x_full[half]), other);
    const uint32_t l_bar_peer = peer_addr(smem_u32(&ctl.l_full), other);
    uint32_t uses = 0, uses_other = 0, tile = 0, seg = 0;  // tiles of this warp's parity so far, of the other one, of both
    bool stop = false;
    Segment g;
    while (!stop && next_segment(a, cur, g)) {
      const bool row_in = r < g.nrows;
      if (rank == 0 && half == 0 && row_in && g.tile0 == 0) a.table[g.place + r] = make_int2((int)g.first_pair, g.pairs);
      if (g.nt == 0) continue;
      const bool active = 32 * quad < g.nrows;  // this warp's quarter has rows at all
      const uint32_t quads = (g.nrows + 31) / 32;
      // ---- Q: channels 0..383 into tensor memory, the others into shared memory ----------------------------------
      // Whole sectors of a row by neighbouring lanes.  (A row is a lane of tensor memory; with each lane reading its own
      // row, 16 bytes at a time, this took 11,000 to 15,000 cycles.)
      if (active) {
        // 16-byte piece c of 72 of a row (rows behind the last one: that one)
        const auto piece = [&](int row, int c) -> const uint4* {
          row = row < g.nrows ? row : g.nrows - 1;
          return c < 64 ? reinterpret_cast<const uint4*>(a.q_nope + (g.row0 + row) * kDLatent) + c
                        : reinterpret_cast<const uint4*>(a.q_rope + (g.row0 + row) * kDRope) + c - 64;
        };
        // Channels 384 .. 575 of 16 of the rows: 128 bytes of four rows per instruction.
        const int own_row = 32 * quad + 16 * half + (lane >> 3);
        const auto place = [&](int k) {
          const int row = own_row + 4 * (k & 3);
          return sbase + (k >> 2) * kQBlock + row * 128 + (((lane & 7) ^ (row & 7)) << 4);
        };
#pragma unroll
        for (int k = 0; k < 12; ++k) cp_async16(place(k), piece(own_row + 4 * (k & 3), 48 + 8 * (k >> 2) + (lane & 7)), 16u);
        // Channels 192 * half .. + 191 of the quarter's rows: 64 bytes of eight rows per instruction, turned around in the
        // place of this CTA's weights, which nobody uses between two row groups.
        const uint32_t turn = sbase + kOffP + warp * 2048;
#pragma unroll 1
        for (int j = 0; j < 3; ++j) {
          uint4 y[2][4];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) y[i][k] = __ldg(piece(32 * quad + 8 * k + (lane >> 2), 24 * half + 8 * j + 4 * i + (lane & 3)));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            __syncwarp();  // (the last ones have been read)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = 8 * k + (lane >> 2);
              sts128(turn + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4), y[i][k].x ^ flip, y[i][k].y ^ flip,
                     y[i][k].z ^ flip, y[i][k].w ^ flip);
            }
            __syncwarp();
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(w[4 * c]), "=r"(w[4 * c + 1]), "=r"(w[4 * c + 2]), "=r"(w[4 * c + 3])
                           : "r"(turn + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4))
                           : "memory");
            tmem_st16(t_lane + kColQ + 96 * half + 32 * j + 16 * i, w);
          }
        }
        cp_async_wait_all();
        if (flip) {
#pragma unroll 1
          for (int k = 0; k < 12; ++k) {
            uint32_t x, y, z, w;
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x), "=r"(y), "=r"(z), "=r"(w) : "r"(place(k)) : "memory");
            sts128(place(k), x ^ flip, y ^ flip, z ^ flip, w ^ flip);
          }
        }
        fence_proxy_async_smem();
        tc::tmem_wait_st();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.q_full);

      const int token = row_in ? (g.r0 + r) / a.H : 0;
      const int64_t mask_row = g.s.mask0 + (int64_t)token * g.s.keys;
      float m = -INFINITY;  // reference of the row's weights in this CTA's tiles of this parity
      // of this thread's keys: sums of the weights as P has them, and before rounding (even and odd keys)
      uint64_t l_round = 0, l_full = 0;
      bool saw = false;  // any of this thread's keys at all
      // Warps 0-3 take the row group's even tiles, 4-7 the odd ones.
#pragma unroll 1
      for (int t = half; t < g.nt; t += 2, ++uses) {
        if (lane == 0 && quad == 0) tma::arrive_expect_tx(&ctl.x_full[half], quads * (32 * kOwnKeys * 2 + 32 * 4));
        // which of the 32 keys this row sees
        uint32_t sees = 0xFFFFFFFFu;
        if (g.s.own) {
          sees = 0;
          const int64_t key0 = (g.tile0 + t) * kKeys + kOwnKeys * rank;
          const int64_t left = g.s.keys - key0 < kOwnKeys ? g.s.keys - key0 : kOwnKeys;
          if (row_in && left > 0) {
            const int64_t bit = mask_row + key0;
            const uint8_t* p = a.mask + (bit >> 3);
            const int shift = (int)(bit & 7), bytes = (int)((shift + left + 7) >> 3);
            uint64_t v = 0;
#pragma unroll
            for (int i = 0; i < 5; ++i)
              if (i < bytes) v |= (uint64_t)__ldg(p + i) << (8 * i);
            sees = (uint32_t)(v >> shift);
          }
        }
        // ---- the scores of this CTA's 32 keys, and their weights --------------------------
        if (!wait_warp(&ctl.s_full[half], uses & 1u, &ctl.abort, a.status)) {
          stop = true;
          break;
        }
        tc::fence_after_sync();
        float n[32];
        if (active) {
          tmem_ld32(t_lane + kColS + 32 * half, n);
          tc::tmem_wait_ld();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.s_free[half]);
        uint32_t w[16];
        if (active) {
          sees &= *reinterpret_cast<const uint32_t*>(ctl.valid[(tile + t) % kOwnStages]);
          saw |= sees != 0;
          if (sees != 0xFFFFFFFFu) {
#pragma unroll
            for (int k = 0; k < 32; ++k) n[k] = (sees >> k) & 1u ? n[k] : -INFINITY;
          }
          float t4[4] = {n[0], n[1], n[2], n[3]};
#pragma unroll
          for (int k = 4; k < 32; ++k) t4[k & 3] = fmaxf(t4[k & 3], n[k]);
          const float most = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])), top = most * scale;
          const bool large = fabsf(top) >= 0x1p23f && fabsf(top) < INFINITY;
          if (top > m + kRowHeadroom) {  // (m = -inf: any key that is seen)
            // (from 2^23 on floats are whole numbers, and too far apart for steps of 32)
            const float up = large ? top : fmaf(kRefStep, ceilf((top - kRefOffset) * (1.f / kRefStep)), kRefOffset),
                        alpha = ratio(m, up);
            const uint64_t alpha2 = pair(alpha, alpha);
            l_round = fma2(l_round, alpha2, 0);
            l_full = fma2(l_full, alpha2, 0);
            m = up;
          }
          float mu = m == -INFINITY ? 0.f : -m;
          if (large) {  // (what rounding the largest one's product by itself leaves out may be far from 0)
#pragma unroll
            for (int k = 0; k < 32; ++k) n[k] -= most;
            mu += top;
          }
          const uint64_t mu2 = pair(mu, mu);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float p0, p1;
            unpair(fma2(pair(n[2 * k], n[2 * k + 1]), scale2, mu2), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
            w[k] = *reinterpret_cast<const uint32_t*>(&h);
            l_full = add2(l_full, pair(p0, p1));
            l_round = add2(l_round, pair(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u)));
          }
        }
        // ---- to both CTAs, whose MMAs have read the weights of two tiles ago ----------------
        // (warps without rows wait too: none may arrive twice in one phase of p_full)
        if (uses > 0 && !wait_warp(&ctl.pv_done[half], (uses - 1) & 1u, &ctl.abort, a.status)) {
          stop = true;
          break;
        }
        if (active) {
#pragma unroll
          for (int c = 0; c < 4; ++c) send16(x_peer + c * kPPiece, bar_peer, w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
          send4(ref_peer, bar_peer, m);
#pragma unroll
          for (int c = 0; c < 4; ++c) sts128(p_own + c * kPPiece, w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
          // ---- one reference for both, and for the tiles before -----------------------------
          bool ok = wait_warp(&ctl.x_full[half], uses & 1u, &ctl.abort, a.status);
          const uint32_t before = uses_other + (half ? (t >> 1) : (t >> 1) - 1);  // tile t - 1 among those of its parity
          if (t > 0) ok = ok && wait_warp(&ctl.m_set[half ^ 1][quad], before & 1u, &ctl.abort, a.status);
          if (!ok) {
            stop = true;
            break;
          }
          const float mx = *reinterpret_cast<volatile float*>(&ctl.x_ref[half][r]);
          const float old = t > 0 ? *reinterpret_cast<volatile float*>(&ctl.m_row[r]) : -INFINITY;
          const float high = fmaxf(m, mx);
          const bool lift = high > old + kOutHeadroom;  // (old = -inf: the first key that either CTA sees)
          const float M = lift ? high : old;
          if (__any_sync(0xffffffffu, lift && old != -INFINITY)) {
            if (!wait_warp(&ctl.pv_done[half ^ 1], before & 1u, &ctl.abort, a.status)) {
              stop = true;
              break;
            }
            tc::fence_after_sync();
            const float alpha = lift ? ratio(old, M) : 1.f;
#pragma unroll 1
            for (int c = 0; c < 32; ++c) {
              float v[8];
              tc::tmem_ld8(t_lane + kColO + 8 * c, v);
              tc::tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] *= alpha;
              tc::tmem_st8(t_lane + kColO + 8 * c, v);
            }
            tc::tmem_wait_st();
          }
          if (lift || t == 0) ctl.m_row[r] = M;
          // (a reference of -inf goes with weights of 0)
          if ((m != M && m != -INFINITY) || (mx != M && mx != -INFINITY)) {
            scale_weights(p_own, ratio(m, M));
            scale_weights(x_own, ratio(mx, M));
          }
          fence_proxy_async_smem();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl.p_full[half]);
          mbar_arrive(&ctl.m_set[half][quad]);
        }
      }
      // Sums go where the last row group's stood: all warps of both CTAs have read those once a tile of this one has been
      // through.  Warps without a tile wait for the other parity's.
      if (half == 1 && g.nt == 1 && active && !stop)
        stop = !wait_warp(&ctl.m_set[0][quad], uses_other & 1u, &ctl.abort, a.status);
      if (stop) break;
      tile += g.nt;
      uses_other += half ? (g.nt + 1) >> 1 : g.nt >> 1;
      // ---- the row group's partial -----------------------------------------------------
      if (tid == 0) tma::arrive_expect_tx(&ctl.l_full, quads * 2 * 32 * 16);
      if (active) {
        float even, odd;
        unpair(l_round, even, odd);
        float lr = even + odd;
        unpair(l_full, even, odd);
        float lf = even + odd;
        // A query with an infinity may score -inf with every key: 0 over 0.
        if (saw && m == -INFINITY) lr = lf = __int_as_float(0x7FFFFFFF);
        send16(sum_peer, l_bar_peer, __float_as_uint(m), __float_as_uint(lr), __float_as_uint(lf), 0u);
        ctl.sum[half][0][r] = m;
        ctl.sum[half][1][r] = lr;
        ctl.sum[half][2][r] = lf;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.l_full);
      // The last value products of both parities; with them the other CTA's last arrivals here are in: none comes after
      // this CTA has left.
      stop = !wait_warp(&ctl.l_full, seg & 1u, &ctl.abort, a.status) ||
             (uses > 0 && !wait_warp(&ctl.pv_done[half], (uses - 1) & 1u, &ctl.abort, a.status)) ||
             (uses_other > 0 && !wait_warp(&ctl.pv_done[half ^ 1], (uses_other - 1) & 1u, &ctl.abort, a.status));
      if (stop) break;
      ++seg;
      tc::fence_after_sync();
      if (active) {
        const float M = ctl.m_row[r];
        float lr = 0.f, lf = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float f = ratio(ctl.sum[k][0][r], M);
          lr += ctl.sum[k][1][r] * f;
          lf += ctl.sum[k][2][r] * f;
          const float4 v = ctl.x_sum[k][r];
          const float fx = ratio(v.x, M);
          lr += v.y * fx;
          lf += v.z * fx;
        }
        const int64_t at = g.place + (int64_t)kRows * cur.pair + r;
        const bool seen = !(lr <= 0.f);  // (a NaN is passed on)
        const float inv = 1.f / lr;
        if (rank == 0 && half == 0 && row_in)
          a.part_lse[at] = seen ? (M + __log2f(lf)) * 0.69314718055994530942f : -INFINITY;
        float* out = a.part_o + at * kDLatent + rank * kHalfLatent + half * 128;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float v[32];
          tmem_ld32(t_lane + kColO + half * 128 + 32 * c, v);
          tc::tmem_wait_ld();
          if (row_in && seen) {
#pragma unroll
            for (int k = 0; k < 32; k += 8)
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out + 32 * c + k),
                           "r"(__float_as_uint(v[k] * inv)), "r"(__float_as_uint(v[k + 1] * inv)),
                           "r"(__float_as_uint(v[k + 2] * inv)), "r"(__float_as_uint(v[k + 3] * inv)),
                           "r"(__float_as_uint(v[k + 4] * inv)), "r"(__float_as_uint(v[k + 5] * inv)),
                           "r"(__float_as_uint(v[k + 6] * inv)), "r"(__float_as_uint(v[k + 7] * inv))
                           : "memory");
          }
        }
      }
      tc::fence_before_sync();
    }
    if (stop) {  // what was sent to the other CTA has long landed before it may leave
      const uint64_t t0 = global_timer_ns();
      for (uint32_t it = 0; it < (1u << 20) && global_timer_ns() - t0 < 200000ull; ++it) {}
    }
  }

  // ---- teardown ---------------------------------------------------------------------------
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
  cluster.sync();
}

}  // namespace

int split_shared_smem() { return kSmem; }

cudaError_t launch_split_shared(const SharedArgs& a, cudaStream_t stream) {
  static_assert(kSmem <= 232448, "shared memory budget exceeded");
  cudaError_t e = cudaFuncSetAttribute(split_shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  split_shared_kernel<<<2 * a.clusters, kThreads, kSmem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mlav
