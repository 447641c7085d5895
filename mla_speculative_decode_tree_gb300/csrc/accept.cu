// Draft trees verified against the target's probabilities (speculative
// sampling on trees), one thread-block cluster per request, one launch.
//
// The definition is in whole numbers, so it does not depend on the order of any
// sum: probabilities are w = round(p * 2^38), random numbers k = floor(u *
// 2^24).  At a node, r = w(target row) and Z = 2^38.  Each child c (token x), in
// ascending order:  s = w(draft row) * Z >> 38, or without draft rows Z at x and
// 0 elsewhere;  accepted when k[c] * s(x) < r(x) * 2^24, else Z -= sum min(r, s)
// and r = max(r - s, 0).  With r the node's remaining mass the next token is the
// first one at which the running sum of r exceeds floor(k * sum(r) / 2^24).
//
// What has to be read is little: of a node on the path one value per child, and
// whole rows only where the walk ends (the target row, and the draft row after a
// rejection) or where a second child is tried after a rejection.  So what bounds
// a request is latency -- tree -> the children's probabilities, fetched for all
// nodes at once -> one pass over a row for its sum -> the search in the part that
// holds the token, about 5 us -- and, where children are rejected, the arithmetic
// of the passes.  The walk runs on shared memory, in every CTA alike; the CTAs of
// a cluster only exchange sums (about 1 us).
//
// A pass adds w(p) without 64-bit conversions, which this GPU does slowly: p *
// 2^19 rounded to a whole number h by adding 2^23, and what that leaves, exact in
// fp32, times 2^19 rounded the same way; w = h * 2^19 + l, since h * 2^19 is even
// and so moves no tie.  As w never falls where p grows, min(w(p), w(q)) = w(min(p,
// q)), and after a node's first rejection max(w(p) - w(q), 0) = w(p) - w(q) where
// p > q: both sums need no 64-bit arithmetic per entry either.  After the first
// rejection only entries with p > q count: each warp keeps theirs in shared memory,
// and later rejections' passes run on those, r = w(p) less the sum of the s.
//
// 16 requests, trees of 9, 131,072 tokens: 17.7 us (10 us for a request with one
// rejection and a child behind it, 15 us with two); 64 requests, trees of up to 16,
// 150,001 tokens: 45 us, of which the rows' 77 MB take 11.3.  In 64 bits throughout
// these took 50.6 and 199 us, with 19-bit parts 29.8 and 97.8; what is kept, clusters
// of 16 and a search by the whole CTA did the rest.
#include <cooperative_groups.h>

#include "common.cuh"

namespace mlav {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;  // two CTAs per SM (of 1024 or 256 threads: no faster)
constexpr int kOne = 38;
constexpr int kMaxCluster = 16;
constexpr int kUnroll = 2;

// (a NaN, a negative probability: 0; above 1: 1)
__device__ __forceinline__ float clip(float p) { return __saturatef(p); }

// Sums of at most kMost weights in two parts of 19 bits.  Each part is the lower bits of a float with a constant on top;
// what the constants add up to, modulo 2^32, comes off at the end.
template <int kMost>
struct Sum {
  static_assert(kMost <= 2048, "the parts' sums have to fit 31 bits");
  uint32_t high = 0, low = 0;
  __device__ __forceinline__ void add(float p) {
    const float t = fmaf(p, 524288.f, 8388608.f);             // 2^23 + h
    const float rest = fmaf(p, 524288.f, -(t - 8388608.f));   // exact, at most half
    high += __float_as_uint(t);
    low += __float_as_uint(fmaf(rest, 524288.f, 12582912.f));
  }
  // Two weights at once, in pairs of floats.
  __device__ __forceinline__ void add(float p, float q) {
    const uint64_t v = pair(p, q), up = pair(524288.f, 524288.f);
    const uint64_t t = fma2(v, up, pair(8388608.f, 8388608.f));
    const uint64_t minus = fma2(t, pair(-1.f, -1.f), pair(8388608.f, 8388608.f));  // (exact)
    const uint64_t low2 = fma2(fma2(v, up, minus), up, pair(12582912.f, 12582912.f));
    high += (uint32_t)t + (uint32_t)(t >> 32);
    low += (uint32_t)low2 + (uint32_t)(low2 >> 32);
  }
  // of exactly n weights
  __device__ __forceinline__ int64_t value(uint32_t n) const {
    return ((int64_t)(high - n * 0x4B000000u) << 19) + (int32_t)(low - n * 0x4B400000u);
  }
};
__device__ __forceinline__ int64_t weight(float p) {
  Sum<1> s;
  s.add(clip(p));
  return s.value(1);
}
__device__ __forceinline__ int64_t random24(float u) {
  return (int64_t)fminf(fmaxf(floorf(u * 16777216.f), 0.f), 16777215.f);
}
// w * Z >> 38, both at most 2^38
__device__ __forceinline__ int64_t scaled(int64_t w, int64_t Z) {
  return (int64_t)((__umul64hi((uint64_t)w, (uint64_t)Z) << (64 - kOne)) | (((uint64_t)w * (uint64_t)Z) >> kOne));
}

// A weight of an entry in [0, 1] as m * 2^e, m below 2^24: what a float holds.  (From 2^-15 on the weight is the float's
// own whole number, below a sum with 2^23 rounds it.)  Products with Z then fit 64 bits.
struct Weight {
  uint32_t m;
  int e;
  explicit __device__ __forceinline__ Weight(float p) {
    const uint32_t bits = __float_as_uint(p);
    const bool whole = p >= 0x1p-15f;
    m = whole ? (bits & 0x7FFFFFu) | 0x800000u : __float_as_uint(fmaf(p, 0x1p38f, 8388608.f)) - 0x4B000000u;
    e = whole ? (int)(bits >> 23) - 112 : 0;
  }
  __device__ __forceinline__ int64_t value() const { return (int64_t)((uint64_t)m << e); }
  __device__ __forceinline__ int64_t times(int64_t Z) const { return (int64_t)(((uint64_t)Z * m) >> (kOne - e)); }
};

// Four neighbouring entries of a row; `at` is the first one's index, `fast`
// says that their address is a multiple of 16 bytes.
__device__ __forceinline__ float4 load4(const float* row, int at, int vocab, bool fast) {
  if (fast && at >= 0 && at + 4 <= vocab) return __ldg(reinterpret_cast<const float4*>(row + at));
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = at + i >= 0 && at + i < vocab ? __ldg(row + at + i) : 0.f;
  return make_float4(v[0], v[1], v[2], v[3]);
}

// Every CTA of the cluster has started: arrive first thing, wait before the first access to another CTA's shared memory.
__device__ __forceinline__ void started_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void started_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Shared {
  int32_t token[kMaxQLen];
  int64_t k[kMaxQLen], wp[kMaxQLen], wq[kMaxQLen];  // of each node's token in its parent's rows
  int64_t z[kMaxQLen];                              // Z at each rejection of the node that the walk is at
  int32_t rejected[kMaxQLen];                       // and the tokens
  int32_t path[kMaxQLen];
  int64_t part[kWarps];
  int64_t all[2][kMaxCluster];  // the CTAs' sums; two in turn, so that an exchange needs one cluster barrier
  int cur, num, tried, last;    // the walk's state; last: the last child looked at
  int64_t Z;
  int ask;  // 1: the walk needs sum min(r, s) for its next child, 0: it has ended
};

// What a warp keeps, in shared memory, of a node's entries after the first rejection: p and q of those that still have r >
// 0 (p > q).  Vectors from `from` on found no room and are read again by every pass.
struct Kept {
  float2* entry;
  int room, n, from;
};

// What a pass adds up, per entry.
enum class What { kLeft, kTaken };  // r as it is now; min(r, s) of the last rejection

template <bool kDraft>
struct Node {
  const float* p;
  const float* q;
  int vocab, off;  // off: entries from the last 16-byte boundary to the target row's start
  bool q_fast;
  int tried;
  const int64_t* z;
  const int32_t* token;

  // r of one entry.
  __device__ __forceinline__ int64_t left(float pv, float qv, int x) const {
    int64_t r = Weight(clip(pv)).value();
    if (kDraft) {
      if (tried > 0) {
        const Weight w(clip(qv));
        r -= w.value();  // (Z is 2^38 at first)
        for (int j = 1; j < tried; ++j) r -= w.times(z[j]);
        r = r > 0 ? r : 0;
      }
    } else {
      for (int j = 0; j < tried; ++j) r = token[j] == x ? (r > z[j] ? r - z[j] : 0) : r;
    }
    return r;
  }
  // Vector k covers entries 4k - off .. 4k - off + 3.
  __device__ __forceinline__ float4 target(int k) const { return load4(p, 4 * k - off, vocab, true); }
  __device__ __forceinline__ float4 draft(int k) const { return load4(q, 4 * k - off, vocab, q_fast); }

  // The first rejection's sum min(w(p), w(q)) over vectors begin .. end - 1, by a whole warp; what is left is kept.
  __device__ __forceinline__ int64_t first(int begin, int end, int lane, Kept& kept) const {
    int64_t t = 0;
    int n = 0, from = end;
    bool keep = kept.room > 0;
    const uint32_t below = (1u << lane) - 1;
    if (!keep) from = begin;
#pragma unroll 1
    for (int k0 = begin; k0 < end; k0 += 32 * kUnroll) {
      float4 pv[kUnroll], qv[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int k = k0 + 32 * u + lane;
        pv[u] = qv[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < end) {
          pv[u] = target(k);
          qv[u] = draft(k);
        }
      }
      Sum<4 * kUnroll> less;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const float a[4] = {clip(pv[u].x), clip(pv[u].y), clip(pv[u].z), clip(pv[u].w)},
                    b[4] = {clip(qv[u].x), clip(qv[u].y), clip(qv[u].z), clip(qv[u].w)};
        less.add(fminf(a[0], b[0]), fminf(a[1], b[1]));
        less.add(fminf(a[2], b[2]), fminf(a[3], b[3]));
        if (keep) {
          int at = n;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t more = __ballot_sync(0xffffffffu, a[i] > b[i]);
            const int place = at + __popc(more & below);
            if (a[i] > b[i] && place < kept.room) kept.entry[place] = make_float2(a[i], b[i]);
            at += __popc(more);
          }
          if (at > kept.room) {
            keep = false;
            from = min(k0 + 32 * u, end);
          } else {
            n = at;
          }
        }
      }
      t += less.value(4 * kUnroll);
    }
    kept.n = n;
    kept.from = from;
    __syncwarp();
    return t;
  }
  // The same sums as below after two rejections or more, of the kept entries.
  template <What kWhat>
  __device__ __forceinline__ int64_t later(int lane, const Kept& kept) const {
    const int n = kWhat == What::kTaken ? tried - 1 : tried;
    const int64_t z1 = n > 1 ? z[1] : 0, zn = kWhat == What::kTaken ? z[n] : 0;
    int64_t t = 0;
#pragma unroll 2
    for (int i = lane; i < kept.n; i += 32) {
      const float2 v = kept.entry[i];
      const Weight w(v.y);
      int64_t r = Weight(v.x).value() - w.value() - w.times(z1);
      for (int j = 2; j < n; ++j) r -= w.times(z[j]);
      r = r > 0 ? r : 0;
      if (kWhat == What::kTaken) {
        const int64_t last = w.times(zn);
        r = r < last ? r : last;
      }
      t += r;
    }
    return t;
  }

  // Sum over vectors first, first + 32, ... below end (kTaken: of the second rejection or a later one).
  template <What kWhat>
  __device__ __forceinline__ int64_t sum(int first, int end) const {
    const int n = kWhat == What::kTaken ? tried - 1 : tried;  // rejections before
    const bool simple = kWhat == What::kLeft && n <= 1;
    const bool both = kDraft && n > 0;
    int64_t t = 0;
#pragma unroll 1
    for (int k = first; k < end; k += 32 * kUnroll) {
      float4 pv[kUnroll], qv[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        pv[u] = qv[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k + 32 * u < end) {
          pv[u] = target(k + 32 * u);
          if (both) qv[u] = draft(k + 32 * u);
        }
      }
      Sum<4 * kUnroll> more, less;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const float a[4] = {clip(pv[u].x), clip(pv[u].y), clip(pv[u].z), clip(pv[u].w)};
        if (!both) {
          more.add(a[0], a[1]);
          more.add(a[2], a[3]);
          continue;
        }
        const float b[4] = {clip(qv[u].x), clip(qv[u].y), clip(qv[u].z), clip(qv[u].w)};
        if (simple) {  // max(w(p) - w(q), 0) = w(p) - min(w(p), w(q))
          more.add(a[0], a[1]);
          more.add(a[2], a[3]);
          less.add(fminf(a[0], b[0]), fminf(a[1], b[1]));
          less.add(fminf(a[2], b[2]), fminf(a[3], b[3]));
          continue;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // r is what the sum of the s leaves of w(p): an r that has reached 0 stays there.
          const Weight w(b[i]);
          int64_t r = Weight(a[i]).value() - w.value();
          for (int j = 1; j < n; ++j) r -= w.times(z[j]);
          r = r > 0 ? r : 0;
          if (kWhat == What::kTaken) {
            const int64_t last = w.times(z[n]);
            r = r < last ? r : last;
          }
          t += r;
        }
      }
      if (!both)
        t += more.value(4 * kUnroll);
      else if (simple)
        t += more.value(4 * kUnroll) - less.value(4 * kUnroll);
    }
    return t;
  }
};

template <bool kDraft>
__global__ void __launch_bounds__(kThreads, 2) accept_kernel(AcceptArgs a) {
  __shared__ Shared s;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t q0 = a.qo_indptr ? (int64_t)a.qo_indptr[b] : (int64_t)b * a.T;
  int n = a.qo_indptr ? a.qo_indptr[b + 1] - (int)q0 : a.T;
  n = n < 0 ? 0 : n > a.T ? a.T : n;
  if (n == 0) {  // (the whole cluster)
    if (rank == 0) {
      for (int j = tid; j < a.T; j += kThreads) a.accepted[(int64_t)b * a.T + j] = -1;
      if (tid == 0) {
        a.num_accepted[b] = 0;
        a.next_tokens[b] = -1;
      }
    }
    return;
  }
  if (C > 1) started_arrive();
  const float u_next = a.u_next[b];
  int parent[2] = {-1, -1};  // of nodes lane, lane + 32; -1: none that the walk can come from
  if (warp < 2 && tid < n && tid > 0) {
    const int c = tid, from = a.parents[q0 + c], x = a.tokens[q0 + c];
    const float u = a.u[q0 + c];
    if (from >= 0 && from < c && x >= 0 && x < a.vocab) {
      s.wp[c] = weight(__ldg(a.target + (q0 + from) * a.target_stride + x));
      s.wq[c] = kDraft ? weight(__ldg(a.draft + (q0 + from) * a.draft_stride + x)) : 0;
      parent[0] = from;
    }
    s.token[c] = x;
    s.k[c] = random24(u);
    s.rejected[c] = parent[0];  // (on its way to the walking warp)
  }
  if (tid == 0) {
    s.rejected[0] = -1;
    s.cur = s.tried = s.last = 0;
    s.path[0] = 0;
    s.num = 1;
    s.Z = (int64_t)1 << kOne;
  }
  __syncthreads();
  if (warp == 0) {
    parent[0] = lane < n ? s.rejected[lane] : -1;
    parent[1] = lane + 32 < n ? s.rejected[lane + 32] : -1;
    __syncwarp();
  }

  extern __shared__ float2 room[];
  Kept kept;
  kept.room = kDraft ? a.keep : 0;  // entries per warp
  kept.entry = room + warp * kept.room;
  kept.n = kept.from = 0;
  int kept_node = -1;
  Node<kDraft> node;
  node.vocab = a.vocab;
  node.z = s.z;
  node.token = s.rejected;
  int round = 0, w0 = 0, w1 = 0;  // this warp's vectors
  const auto w_first = [&](int w) {
    const int vectors = (node.off + a.vocab + 3) / 4, per = (vectors + C - 1) / C, v0 = min(rank * per, vectors);
    return min(v0 + w * ((per + kWarps - 1) / kWarps), min(v0 + per, vectors));
  };
  const auto w_end = [&](int w) {
    const int vectors = (node.off + a.vocab + 3) / 4, per = (vectors + C - 1) / C, v0 = min(rank * per, vectors);
    return min(w_first(w) + (per + kWarps - 1) / kWarps, min(v0 + per, vectors));
  };
  // A sum over the row by warps' parts (s.part) and CTAs (s.all), all of them known to all CTAs.
  auto pass = [&](auto&& f) -> int64_t {
    w0 = w_first(warp);
    w1 = w_end(warp);
    const int64_t t = warp_sum(f());
    if (lane == 0) s.part[warp] = t;
    if (C > 1 && round == 0) started_wait();
    __syncthreads();
    ++round;
    if (warp == 0) {
      const int64_t x = warp_sum(lane < kWarps ? s.part[lane] : 0);
      if (lane < C) *cluster.map_shared_rank(&s.all[round & 1][rank], lane) = x;
    }
    if (C > 1)
      cluster.sync();
    else
      __syncthreads();
    return warp_sum(lane < C ? s.all[round & 1][lane] : 0);
  };

  // ---- the walk, by the first warp ----------------------------------------------------
#pragma unroll 1
  for (;;) {
    if (warp == 0) {
      int cur = s.cur, tried = s.tried, last = s.last, num = s.num, ask = 0;
      int64_t Z = s.Z;
#pragma unroll 1
      for (;;) {
        const uint32_t lo = __ballot_sync(0xffffffffu, parent[0] == cur && lane > last);
        const uint32_t hi = __ballot_sync(0xffffffffu, parent[1] == cur && lane + 32 > last);
        if (!(lo | hi)) break;
        const int c = lo ? __ffs(lo) - 1 : __ffs(hi) + 31;  // the next child
        if (kDraft && Z < 0) {  // Z after the last rejection is not known yet
          ask = 1;
          break;
        }
        last = c;
        const int x = s.token[c];
        int64_t r = s.wp[c];
        for (int j = 0; j < tried; ++j) {
          const int64_t sj = kDraft ? scaled(s.wq[c], s.z[j]) : (s.rejected[j] == x ? s.z[j] : 0);
          r = r > sj ? r - sj : 0;
        }
        const int64_t sx = kDraft ? scaled(s.wq[c], Z) : Z;
        __syncwarp();
        if ((uint64_t)s.k[c] * (uint64_t)sx < (uint64_t)r << 24) {
          cur = c;
          if (lane == 0) s.path[num] = c;
          ++num;
          tried = 0;
          Z = (int64_t)1 << kOne;
        } else {
          if (lane == 0) {
            s.z[tried] = Z;
            s.rejected[tried] = x;
          }
          ++tried;
          Z = kDraft ? -1 : Z - (r < sx ? r : sx);
        }
        __syncwarp();
      }
      if (lane == 0) {
        s.cur = cur;
        s.tried = tried;
        s.last = last;
        s.num = num;
        s.Z = Z;
        s.ask = ask;
      }
    }
    __syncthreads();
    node.p = a.target + (q0 + s.cur) * a.target_stride;
    node.q = kDraft ? a.draft + (q0 + s.cur) * a.draft_stride : nullptr;
    node.off = (int)((reinterpret_cast<uintptr_t>(node.p) >> 2) & 3);
    node.q_fast = kDraft && (int)((reinterpret_cast<uintptr_t>(node.q) >> 2) & 3) == node.off;
    node.tried = s.tried;
    if (!kDraft || !s.ask) break;
    const int64_t z = s.z[s.tried - 1];
    const int64_t taken = pass([&]() -> int64_t {
      if constexpr (kDraft) {
        if (node.tried == 1) {
          kept_node = s.cur;
          return node.first(w0, w1, lane, kept);
        }
        const int64_t t = node.template later<What::kTaken>(lane, kept);
        return t + node.template sum<What::kTaken>(kept.from + lane, w1);
      }
      return 0;
    });
    if (tid == 0) s.Z = z > taken ? z - taken : 0;
    __syncthreads();
  }

  // ---- the next token -------------------------------------------------------------
  auto left_sum = [&]() -> int64_t {
    int64_t t = 0;
    if (kDraft && kept_node == s.cur && node.tried > 1) {
      t = node.template later<What::kLeft>(lane, kept);
      t += node.template sum<What::kLeft>(kept.from + lane, w1);
    } else {
      t = node.template sum<What::kLeft>(w0 + lane, w1);
    }
    if (!kDraft) {
      // Rejected tokens in this warp's part: what they lack (each token once).
      for (int j = lane; j < node.tried; j += 32) {
        const int x = s.rejected[j], k = (x + node.off) >> 2;
        bool first = k >= w0 && k < w1;
        for (int i = 0; i < j; ++i) first = first && s.rejected[i] != x;
        if (first) {
          const float pv = __ldg(node.p + x);
          t += node.left(pv, 0.f, x) - weight(pv);
        }
      }
    }
    return t;
  };
  int64_t sum = pass(left_sum);
  if (sum == 0 && node.tried > 0) {  // nothing is left (roundings only): the target itself
    node.tried = 0;
    sum = pass(left_sum);
  }
  if (rank == 0) {
    for (int j = tid; j < a.T; j += kThreads) a.accepted[(int64_t)b * a.T + j] = j < s.num ? s.path[j] : -1;
    if (tid == 0) {
      a.num_accepted[b] = s.num;
      if (sum == 0) a.next_tokens[b] = -1;
    }
  }
  const int64_t aim = (int64_t)__umul64hi((uint64_t)random24(u_next) << 40, (uint64_t)sum);
  int64_t mine = warp_sum(lane < rank ? s.all[round & 1][lane] : 0);
  if (sum == 0 || aim < mine || aim >= mine + s.all[round & 1][rank]) return;
  // A warp's part in this CTA holds the token; all of the CTA looks through that part, a vector a thread.
  const auto scan = [&](int64_t v) -> int64_t {  // over the lanes, each with those before it
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    return v;
  };
  int64_t parts = lane < kWarps ? s.part[lane] : 0, upto = scan(parts);
  const int part = min(__ffs(__ballot_sync(0xffffffffu, mine + upto > aim)) - 1, kWarps - 1);
  mine += __shfl_sync(0xffffffffu, upto - parts, part);
  w0 = w_first(part);
  w1 = w_end(part);
#pragma unroll 1
  for (int k0 = w0; k0 < w1; k0 += kThreads) {
    const int k = k0 + tid, x = 4 * k - node.off;
    int64_t r[4] = {0, 0, 0, 0};
    if (k < w1) {
      const float4 p4 = node.target(k), q4 = kDraft && node.tried > 0 ? node.draft(k) : make_float4(0.f, 0.f, 0.f, 0.f);
      r[0] = node.left(p4.x, q4.x, x);
      r[1] = node.left(p4.y, q4.y, x + 1);
      r[2] = node.left(p4.z, q4.z, x + 2);
      r[3] = node.left(p4.w, q4.w, x + 3);
    }
    const int64_t own = (r[0] + r[1]) + (r[2] + r[3]);
    upto = scan(own);
    __syncthreads();  // (the parts have been read)
    if (lane == 31) s.part[warp] = upto;
    __syncthreads();
    parts = lane < kWarps ? s.part[lane] : 0;
    const int64_t to = scan(parts), before = mine + __shfl_sync(0xffffffffu, to - parts, warp),
                  all = __shfl_sync(0xffffffffu, to, 31);
    if (before + upto - own <= aim && aim < before + upto) {
      int64_t at = before + upto - own;
      int i = 0;
      while (i < 3 && (at += r[i]) <= aim) ++i;
      a.next_tokens[b] = x + i;
    }
    mine += all;
    if (mine > aim) return;
  }
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs& a, int sms, cudaStream_t stream) {
  // CTAs per request.  A batch is as slow as its request with the most rejections, whose passes are bound by arithmetic:
  // up to 16 while each has 3500 entries (16 requests, 131,072 tokens: clusters of 4 / 8 / 16 take 38 / 21.5 / 18.7 us).
  // But no more than twice what the GPU has room for at once, or requests queue up for their start, dependent reads of 2
  // us (64 requests, 150,001 tokens: 8 / 16 take 46 / 56 us).  And enough of them to keep the entries of a request that is
  // half rejected (256 requests, 131,072 tokens: 2 / 4 take 150 / 117 us).
  const int64_t resident = 2 * (int64_t)sms;
  int C = 1;
  while (C < kMaxCluster &&
         ((a.draft && a.vocab > 32768 * C) || (a.vocab >= 7000 * C && a.batch * C <= resident)))
    C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.batch * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Shared memory for what is kept, of half an SM.
  const size_t room = a.draft ? 104u * 1024u : 0;
  AcceptArgs args = a;
  args.keep = (int)(room / sizeof(float2)) / kWarps;
  cfg.dynamicSmemBytes = room;
  auto kernel = a.draft ? accept_kernel<true> : accept_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && room) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)room);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, args);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mlav
