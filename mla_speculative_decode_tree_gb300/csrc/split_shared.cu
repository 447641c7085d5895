// Tensor-core (tcgen05) attention for requests that share prefixes, by pairs of
// CTAs (a cluster of two).
//
// A pair takes a row group -- up to 128 query rows (token, head pairs; of all the
// requests of a group, or of one request) -- and a run of 64-key tiles, and
// leaves the group's partial softmax statistics for the merge.  Query rows sit on
// the MMA's M = 128, so an fp32 O of 512 latent columns would fill tensor memory
// (128 lanes x 512 columns).  The pair splits the latent columns instead: CTA c
// owns latent columns 256c .. 256c+255 and RoPE columns 32c .. 32c+31, of the keys
// as of the queries, and
//   S_c[128 x 64]   = Q_c[128 x 288] . K_c^T        (18 MMAs, K = 16, N = 64)
//   S               = S_0 + S_1                      (each half sent to the other CTA)
//   O_c[128 x 256] += P[128 x 64] . V_c[64 x 256]    (4 MMAs, K = 16, N = 256)
// so each key lands once per pair and each CTA gathers half of its row.  Both
// CTAs hold the same S bit for bit (the sum of two commutes) and do the same
// softmax; 64 exponentials per row and tile are cheaper than another exchange.
//
// Q_c (as 144 columns of bf16 pairs) and P (32 columns) are A operands in tensor
// memory, so shared memory feeds the B operands only, 64 bytes per clock at full
// rate: with A there too the score product would take 1.5 times as long.
// Tensor memory: O 0..255, Q 256..399, S 400..463, P 464..495.
//
// Shared memory: kStages tiles of K_c in five blocks of 64 keys x 128 bytes (four
// latent blocks and one of which the first half is used), 128-byte swizzled: that
// atom is the K-major layout of the score product's B and the MN-major layout of
// the value product's; and two buffers for the other CTA's S (32 KB each).
//
// Warps: 0-7 softmax (thread = a query row and 32 of the tile's keys; it also
// brings its row's Q into tensor memory and takes O out of it), 8 issues the MMAs,
// 9-12 gather rows with 16-byte cp.async.  In the steady state the issuing thread
// runs QK(t+1), PV(t), QK(t+2), ...: S is read out of tensor memory at once, so
// one S buffer is enough for the tensor pipe to have QK(t+1) to do while the
// softmax of tile t runs.
//
// Work in equal pieces: the row groups of all groups' shared parts, then of all
// requests' own parts, each as long as its tiles and kSegCost more, form an axis;
// pair w takes the w-th of equal pieces (every CTA sums up the lengths itself).
// Row group with first row R (0 .. rows_max for shared parts, rows_max .. for own
// ones) leaves pair w's partial at row R + 128 w, and the table's entry R says
// which pairs have one.
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
constexpr int kHalfLatent = kDLatent / 2, kHalfRope = kDRope / 2;
constexpr int kStages = 3;
constexpr int kBlockBytes = kKeys * 128;        // 64 columns of a tile
constexpr int kStageBytes = 5 * kBlockBytes;
constexpr int kXBytes = kRows * kKeys * 4;      // the other CTA's S
constexpr int kSoftmaxWarps = 8;
constexpr int kMmaWarp = kSoftmaxWarps;
constexpr int kGatherWarp = kMmaWarp + 1, kGatherWarps = 4;
constexpr int kThreads = 32 * (kGatherWarp + kGatherWarps);
constexpr int kKeysPerWarp = kKeys / kGatherWarps;  // gathered by a warp
constexpr int kColO = 0, kColQ = 256, kColS = 400, kColP = 464;
constexpr float kHeadroom = 8.0f;  // base 2, before the running maximum is raised
// Start and end of a row group, in tiles.
constexpr int kSegCost = 5;
constexpr int kMaxSpans = 2 * kMaxSharedBatch;

struct Ctl {
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full, s_full, s_free, p_full, pv_done, x_full[2], mma_idle;
  uint32_t tmem_base;
  int abort;
  int64_t total;
  uint16_t valid[kStages][kGatherWarps];  // keys of a tile that exist, 16 bits per gather warp
  int failed[2][4];                       // softmax warps that gave up, by half of the keys and quarter of the rows
  float red[2][kRows];                    // per half of the keys: row maxima, sums
  float red2[2][kRows];
  int64_t warp_sum[kThreads / 32];
};

constexpr int kOffX = kStages * kStageBytes;
constexpr int kOffCtl = kOffX + 2 * kXBytes;
constexpr int kOffEnds = (kOffCtl + (int)sizeof(Ctl) + 15) / 16 * 16;
constexpr int kSmem = kOffEnds + 1024;  // + the axis (8 bytes per group and request) + alignment slack

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
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
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

// ---- the other CTA of the pair -------------------------------------------------
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// 16 bytes into the other CTA's shared memory, counted by its barrier.
__device__ __forceinline__ void send16(uint32_t dst, uint32_t bar, float a, float b, float c, float d) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(dst),
      "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(__float_as_uint(c)), "r"(__float_as_uint(d)), "r"(bar)
      : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
// mbar_wait for bytes from the other CTA.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1; it < (1u << 30); ++it) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) break;
    }
  }
  *abort = 1;
  atomicOr(status, kStatusTimeout);
  return false;
}
__device__ __forceinline__ bool or_sync(int id, bool p) {  // over the 64 threads that share rows
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbarrier.cta.red.or.pred b, %2, 64, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(p ? 1u : 0u), "r"(id)
      : "memory");
  return r != 0;
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
__device__ __forceinline__ int64_t tiles_of(const Span& s) { return (s.keys + kKeys - 1) / kKeys; }

// Where a pair is on the axis; every role of its CTAs walks it by itself.
struct Cursor {
  const int64_t* ends;  // shared memory: end of each span on the axis
  int spans, e;
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
  int64_t first_pair;
  int pairs;  // that have a partial of it
};

// The next row group and run of tiles of the pair; false at the end of its piece.
__device__ __forceinline__ bool next_segment(const SharedArgs& a, Cursor& c, Segment& g) {
  while (c.x < c.x_end) {
    while (c.e < c.spans && c.ends[c.e] <= c.x) ++c.e;
    if (c.e >= c.spans) return false;
    g.s = span_of(a, c.e);
    const int64_t start = c.e ? c.ends[c.e - 1] : 0;
    const int64_t tiles = tiles_of(g.s), len = tiles + kSegCost;
    const int64_t i = (c.x - start) / len, e0 = start + i * len, e1 = e0 + len;
    g.r0 = (int)(i * kRows);
    const int64_t left = (int64_t)g.s.ntok * a.H - g.r0;
    g.nrows = left < kRows ? (int)left : kRows;
    g.row0 = g.s.q0 * a.H + g.r0;
    g.place = g.row0 + (g.s.own ? a.rows_max : 0);
    const int64_t stop = c.x_end < e1 ? c.x_end : e1;
    int64_t t0 = c.x - e0 - kSegCost, t1 = stop - e0 - kSegCost;
    t0 = t0 < 0 ? 0 : t0;
    const bool heads = c.x == e0;  // this pair has the row group's start on the axis
    c.x = stop;
    g.tile0 = t0;
    g.nt = t1 > t0 ? (int)(t1 - t0) : 0;
    g.first_pair = (e0 + kSegCost) / c.piece;
    g.pairs = tiles ? (int)((e1 - 1) / c.piece - g.first_pair + 1) : 0;
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
  int64_t* ends = reinterpret_cast<int64_t*>(smem + kOffEnds);
  cg::cluster_group cluster = cg::this_cluster();
  const uint32_t rank = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // ---- set-up: barriers, tensor memory, the axis ------------------------------------
  if (tid == 0) {
    for (int k = 0; k < kStages; ++k) {
      mbar_init(&ctl.full[k], kGatherWarps * 33);  // every lane's copies and, per warp, its valid bits
      mbar_init(&ctl.empty[k], 1);
    }
    mbar_init(&ctl.q_full, kSoftmaxWarps);
    mbar_init(&ctl.s_full, 1);
    mbar_init(&ctl.s_free, kSoftmaxWarps);
    mbar_init(&ctl.p_full, kSoftmaxWarps);
    mbar_init(&ctl.pv_done, 1);
    mbar_init(&ctl.x_full[0], 1);
    mbar_init(&ctl.x_full[1], 1);
    mbar_init(&ctl.mma_idle, 1);
    ctl.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&ctl.tmem_base, 512);
    tc::tmem_relinquish();
  }
  Cursor cur;
  cur.ends = ends;
  cur.spans = a.groups + a.batch;
  {
    int64_t carry = 0;
    for (int base = 0; base < cur.spans; base += kThreads) {
      const int e = base + tid;
      int64_t v = 0;
      if (e < cur.spans) {
        const Span s = span_of(a, e);
        v = groups_of(a, s) * (tiles_of(s) + kSegCost);
      }
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      if (lane == 31) ctl.warp_sum[warp] = v;
      __syncthreads();
      int64_t before = carry;
      for (int w = 0; w < warp; ++w) before += ctl.warp_sum[w];
      if (e < cur.spans) ends[e] = before + v;
      for (int w = 0; w < kThreads / 32; ++w) carry += ctl.warp_sum[w];
      __syncthreads();
    }
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
  }
  tc::fence_before_sync();
  cluster.sync();
  tc::fence_after_sync();
  const uint32_t tmem = ctl.tmem_base;

  if (warp >= kGatherWarp) {
    // ============================ gather ================================================
    // Warp gw fills keys 16 gw .. 16 gw + 15 of each tile: per key one instruction of 32 lanes x 16 bytes for this
    // CTA's 512 latent bytes, and one for the 64 RoPE bytes of eight keys.
    const int gw = warp - kGatherWarp;
    uint32_t bad = 0;
    int64_t tt = 0;  // tiles so far
    bool stop = false;
    Segment g;
    while (!stop && next_segment(a, cur, g)) {
      const int32_t* index = g.s.own ? a.kv_indices : a.shared_indices;
      auto load_id = [&](int t) -> int32_t {  // of this lane's key of tile t (lanes 0..15)
        const int64_t j = (g.tile0 + t) * kKeys + gw * kKeysPerWarp + (lane & 15);
        if (t >= g.nt || j >= g.s.keys) return -1;  // no such key
        return j < g.s.prefix ? __ldg(index + g.s.kv0 + j) : __ldg(a.out_cache_loc + g.s.q0 + (j - g.s.prefix));
      };
      int32_t id0 = load_id(0), id1 = load_id(1);
#pragma unroll 1
      for (int t = 0; t < g.nt; ++t, ++tt) {
        int32_t row = id0;
        id0 = id1;
        id1 = load_id(t + 2);
        const bool ok = row >= 0 && row < a.pool_rows;
        if (!ok && (g.tile0 + t) * kKeys + gw * kKeysPerWarp + (lane & 15) < g.s.keys) bad = 1;
        row = ok ? row : -1;
        const uint32_t valid = __ballot_sync(0xffffffffu, ok) & 0xFFFFu;
        const int stage = (int)(tt % kStages);
        const bool got = mbar_wait(&ctl.empty[stage], ((uint32_t)(tt / kStages) & 1u) ^ 1u, &ctl.abort, a.status);
        if (!__all_sync(0xffffffffu, got)) {
          stop = true;
          break;
        }
        if (a.test_stall && tt == 0) continue;  // test only: the first tile never lands
        if (lane == 0) ctl.valid[stage][gw] = (uint16_t)valid;
        const uint32_t dst = sbase + stage * kStageBytes;
        const int blk = lane >> 3, chunk = lane & 7;
        const __nv_bfloat16* src = a.kv_pool + rank * kHalfLatent + lane * 8;
#pragma unroll
        for (int k = 0; k < kKeysPerWarp; ++k) {
          const int key = gw * kKeysPerWarp + k;
          const int32_t r = __shfl_sync(0xffffffffu, row, k);
          cp_async16(dst + blk * kBlockBytes + key * 128 + ((chunk ^ (key & 7)) << 4),
                     src + (int64_t)(r < 0 ? 0 : r) * kDRow, r < 0 ? 0u : 16u);
        }
#pragma unroll
        for (int k = 0; k < kKeysPerWarp; k += 8) {
          const int key = gw * kKeysPerWarp + k + (lane >> 2);
          const int32_t r = __shfl_sync(0xffffffffu, row, k + (lane >> 2));
          cp_async16(dst + 4 * kBlockBytes + key * 128 + (((lane & 3) ^ (key & 7)) << 4),
                     a.kv_pool + (int64_t)(r < 0 ? 0 : r) * kDRow + kDLatent + rank * kHalfRope + (lane & 3) * 8,
                     r < 0 ? 0u : 16u);
        }
        cp_async_arrive(&ctl.full[stage]);
        if (lane == 0) mbar_arrive(&ctl.full[stage]);
      }
    }
    cp_async_wait_all();
    if (bad) atomicOr(a.status, kStatusBadRow);
  } else if (warp == kMmaWarp) {
    // ============================ MMA issue ==============================================
    if (lane == 0) {
      constexpr uint32_t idesc_qk = tc::idesc_bf16_f32(kRows, kKeys, false, false);
      constexpr uint32_t idesc_pv = tc::idesc_bf16_f32(kRows, kHalfLatent, false, true);
      bool ok = true;
      int64_t tt = 0;  // tiles whose scores have been issued
      uint32_t seg = 0;
      Segment g;
      auto qk = [&]() {  // scores of tile tt
        const int stage = (int)(tt % kStages);
        ok = mbar_wait_spin(&ctl.full[stage], (uint32_t)(tt / kStages) & 1u, &ctl.abort, a.status);
        if (ok && tt > 0) ok = mbar_wait_spin(&ctl.s_free, (uint32_t)(tt - 1) & 1u, &ctl.abort, a.status);
        if (!ok) return;
        fence_proxy_async_smem();
        tc::fence_after_sync();
        const uint32_t base = sbase + stage * kStageBytes;
#pragma unroll
        for (int k = 0; k < 18; ++k)
          mma_bf16_ts(tmem + kColS, tmem + kColQ + 8 * k,
                      tc::smem_desc(base + (k >> 2) * kBlockBytes + (k & 3) * 32, 16, 1024, tc::kSwizzle128B), idesc_qk,
                      k > 0);
        tc::mma_commit(&ctl.s_full);
        ++tt;
      };
      auto pv = [&](int64_t u, bool first) {  // O += P V of tile u
        ok = mbar_wait_spin(&ctl.p_full, (uint32_t)u & 1u, &ctl.abort, a.status);
        if (!ok) return;
        tc::fence_after_sync();
        const int stage = (int)(u % kStages);
        const uint32_t base = sbase + stage * kStageBytes;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_bf16_ts(tmem + kColO, tmem + kColP + 8 * k,
                      tc::smem_desc(base + k * 2048, kBlockBytes, 1024, tc::kSwizzle128B), idesc_pv, !(first && k == 0));
        tc::mma_commit(&ctl.empty[stage]);
        tc::mma_commit(&ctl.pv_done);
      };
      while (ok && next_segment(a, cur, g)) {
        if (g.nt == 0) continue;
        ok = mbar_wait_spin(&ctl.q_full, seg & 1u, &ctl.abort, a.status);
        tc::fence_after_sync();
        ++seg;
        if (ok) qk();
#pragma unroll 1
        for (int t = 0; t < g.nt && ok; ++t) {
          if (t + 1 < g.nt) qk();
          if (ok) pv(t + 1 < g.nt ? tt - 2 : tt - 1, t == 0);
        }
      }
      // Drain: every MMA this thread issued has completed before tensor memory is freed.
      tc::mma_commit(&ctl.mma_idle);
      const uint64_t t0 = global_timer_ns();
      for (uint32_t it = 0; it < (1u << 30); ++it)
        if (mbar_try_wait(&ctl.mma_idle, 0) || ((it & 63u) == 63u && global_timer_ns() - t0 > kWaitLimitNs)) break;
    }
    __syncwarp();
  } else {
    // ============================ softmax ================================================
    const int quad = warp & 3, half = warp >> 2;
    const int r = 32 * quad + lane;  // query row in the group = TMEM lane
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quad) << 16);
    const float scale = a.scale_log2;
    const uint32_t other = rank ^ 1u;
    const uint32_t x_own = sbase + kOffX + half * 8 * kRows * 16 + r * 16;
    const uint32_t x_peer = peer_addr(x_own, other);
    const uint32_t bar_peer[2] = {peer_addr(smem_u32(&ctl.x_full[0]), other), peer_addr(smem_u32(&ctl.x_full[1]), other)};
    int64_t tt = 0;
    bool stop = false, fail = false;
    Segment g;
    while (!stop && next_segment(a, cur, g)) {
      const bool row_in = r < g.nrows;
      if (rank == 0 && half == 0 && row_in && (g.tile0 == 0))
        a.table[g.place + r] = make_int2((int)g.first_pair, g.pairs);
      if (g.nt == 0) continue;
      const bool active = 32 * quad < g.nrows;  // this warp's quarter has rows at all
      const int quads = (g.nrows + 31) / 32;
      // ---- Q: this thread's half of the row's slice --------------------------------------
      if (active) {
        const __nv_bfloat16* qn = a.q_nope + (g.row0 + (row_in ? r : 0)) * kDLatent + rank * kHalfLatent + half * 128;
        const __nv_bfloat16* qr = a.q_rope + (g.row0 + (row_in ? r : 0)) * kDRope + rank * kHalfRope + half * 16;
        uint4 v[18];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = __ldg(reinterpret_cast<const uint4*>(qn) + k);
        v[16] = __ldg(reinterpret_cast<const uint4*>(qr));
        v[17] = __ldg(reinterpret_cast<const uint4*>(qr) + 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t w[16] = {v[4 * k].x,     v[4 * k].y,     v[4 * k].z,     v[4 * k].w,
                                  v[4 * k + 1].x, v[4 * k + 1].y, v[4 * k + 1].z, v[4 * k + 1].w,
                                  v[4 * k + 2].x, v[4 * k + 2].y, v[4 * k + 2].z, v[4 * k + 2].w,
                                  v[4 * k + 3].x, v[4 * k + 3].y, v[4 * k + 3].z, v[4 * k + 3].w};
          tmem_st16(t_lane + kColQ + half * 64 + 16 * k, w);
        }
        const uint32_t w[8] = {v[16].x, v[16].y, v[16].z, v[16].w, v[17].x, v[17].y, v[17].z, v[17].w};
        tmem_st8u(t_lane + kColQ + 128 + half * 8, w);
        tc::tmem_wait_st();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.q_full);

      const int token = row_in ? (g.r0 + r) / a.H : 0;
      const int64_t mask_row = g.s.mask0 + (int64_t)token * g.s.keys;
      float m = -INFINITY;              // running maximum, base 2
      float l_round = 0.f, l_full = 0.f;  // of this thread's keys: sums of the weights as P has them, and before rounding
#pragma unroll 1
      for (int t = 0; t < g.nt; ++t, ++tt) {
        const int stage = (int)(tt % kStages);
        const int buf = (int)(tt & 1);
        if (tid == 0) tma::arrive_expect_tx(&ctl.x_full[buf], (uint32_t)quads * 2u * 32u * 128u);
        // which of the 32 keys this row sees
        const int64_t key0 = (g.tile0 + t) * kKeys + 32 * half;
        uint32_t sees = 0xFFFFFFFFu;
        if (g.s.own) {
          sees = 0;
          const int64_t n = g.s.keys - key0 < 32 ? g.s.keys - key0 : 32;
          if (row_in && n > 0) {
            const int64_t bit = mask_row + key0;
            const uint8_t* p = a.mask + (bit >> 3);
            const int shift = (int)(bit & 7), bytes = (int)((shift + n + 7) >> 3);
            uint64_t w = 0;
#pragma unroll
            for (int i = 0; i < 5; ++i)
              if (i < bytes) w |= (uint64_t)__ldg(p + i) << (8 * i);
            sees = (uint32_t)(w >> shift);
          }
        }
        bool got = mbar_wait(&ctl.full[stage], (uint32_t)(tt / kStages) & 1u, &ctl.abort, a.status);
        sees &= (uint32_t)ctl.valid[stage][2 * half] | ((uint32_t)ctl.valid[stage][2 * half + 1] << 16);
        got = got && mbar_wait(&ctl.s_full, (uint32_t)tt & 1u, &ctl.abort, a.status);
        fail |= !__all_sync(0xffffffffu, got);
        tc::fence_after_sync();
        float s[32];
        if (active) {
          tmem_ld32(t_lane + kColS + 32 * half, s);
          tc::tmem_wait_ld();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.s_free);
        if (active) {
          const uint32_t off = buf * kXBytes;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            send16(x_peer + off + c * kRows * 16, bar_peer[buf], s[4 * c], s[4 * c + 1], s[4 * c + 2], s[4 * c + 3]);
        }
        got = mbar_wait_cluster(&ctl.x_full[buf], (uint32_t)(tt >> 1) & 1u, &ctl.abort, a.status);
        fail |= !__all_sync(0xffffffffu, got);
        bool raise = false;
        float top = -INFINITY;
        if (active) {
          const uint32_t off = buf * kXBytes;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float x[4];
            asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                         : "r"(x_own + off + c * kRows * 16)
                         : "memory");
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * c + i] = (s[4 * c + i] + x[i]) * scale;
          }
          if (sees != 0xFFFFFFFFu) {
#pragma unroll
            for (int k = 0; k < 32; ++k) s[k] = (sees >> k) & 1u ? s[k] : -INFINITY;
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) top = fmaxf(top, s[k]);
          raise = top > m + kHeadroom;  // (m = -inf: any key that is seen)
          // The two warps of a quarter stay together: they leave the loop in the same place.
          raise = or_sync(1 + quad, raise || fail);
          if (raise) {
            ctl.red[half][r] = top;
            if (lane == 0) ctl.failed[half][quad] = fail ? 1 : 0;
            named_bar_sync(1 + quad, 64);
            top = fmaxf(top, ctl.red[half ^ 1][r]);
            fail |= ctl.failed[half ^ 1][quad] != 0;
            named_bar_sync(1 + quad, 64);  // (read before the next raise writes)
          }
        }
        if (fail) {
          stop = true;
          break;
        }
        // P(t) overwrites what PV(t-1) reads, and a rescaled O needs it complete.
        if (t > 0) {
          got = mbar_wait(&ctl.pv_done, (uint32_t)(tt - 1) & 1u, &ctl.abort, a.status);
          fail |= !__all_sync(0xffffffffu, got);  // (left at the next meeting)
        }
        tc::fence_after_sync();
        if (active) {
          if (raise) {
            float alpha = 1.f;
            if (top > m + kHeadroom) {
              alpha = m == -INFINITY ? 0.f : ex2_approx(m - top);
              m = top;
            }
            l_round *= alpha;
            l_full *= alpha;
            if (t > 0) {
#pragma unroll 1
              for (int c = 0; c < 16; ++c) {
                float v[8];
                tc::tmem_ld8(t_lane + kColO + half * 128 + 8 * c, v);
                tc::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] *= alpha;
                tc::tmem_st8(t_lane + kColO + half * 128 + 8 * c, v);
              }
            }
          }
          const float mu = m == -INFINITY ? 0.f : m;
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float p0 = ex2_approx(s[2 * k] - mu), p1 = ex2_approx(s[2 * k + 1] - mu);
            const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
            w[k] = *reinterpret_cast<const uint32_t*>(&h);
            l_full += p0 + p1;
            l_round += __uint_as_float(w[k] << 16) + __uint_as_float(w[k] & 0xFFFF0000u);
          }
          tmem_st16(t_lane + kColP + 16 * half, w);
          tc::tmem_wait_st();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.p_full);
      }
      if (stop) break;
      // ---- the row group's partial -----------------------------------------------------
      const bool got = mbar_wait(&ctl.pv_done, (uint32_t)(tt - 1) & 1u, &ctl.abort, a.status);
      fail |= !__all_sync(0xffffffffu, got);
      stop = active ? or_sync(1 + quad, fail) : fail;
      if (stop) break;
      tc::fence_after_sync();
      if (active) {
        ctl.red[half][r] = l_round;
        ctl.red2[half][r] = l_full;
        named_bar_sync(1 + quad, 64);
        const float lr = ctl.red[0][r] + ctl.red[1][r], lf = ctl.red2[0][r] + ctl.red2[1][r];
        named_bar_sync(1 + quad, 64);
        const int64_t at = g.place + (int64_t)kRows * cur.pair + r;
        const float inv = lr > 0.f ? 1.f / lr : 0.f;
        if (rank == 0 && half == 0 && row_in)
          a.part_lse[at] = lr > 0.f ? (m + __log2f(lf)) * 0.69314718055994530942f : -INFINITY;
        float* out = a.part_o + at * kDLatent + rank * kHalfLatent + half * 128;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float v[32];
          tmem_ld32(t_lane + kColO + half * 128 + 32 * c, v);
          tc::tmem_wait_ld();
          if (row_in && lr > 0.f) {
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

int split_shared_smem() { return kSmem + (int)sizeof(int64_t) * kMaxSpans; }

cudaError_t launch_split_shared(const SharedArgs& a, cudaStream_t stream) {
  const int smem = kSmem + (int)sizeof(int64_t) * (a.groups + a.batch);
  static_assert(kSmem + sizeof(int64_t) * kMaxSpans <= 232448, "shared memory budget exceeded");
  cudaError_t e = cudaFuncSetAttribute(split_shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       split_shared_smem());
  if (e != cudaSuccess) return e;
  split_shared_kernel<<<2 * a.clusters, kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mlav
