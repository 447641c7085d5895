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
// it is latency: tree -> the children's probabilities, fetched for all nodes at
// once -> one pass over a row for its sum -> the search in the part that holds
// the token.  The walk runs on shared memory, in every CTA alike; the CTAs of a
// cluster only exchange sums.
//
// A pass adds w(p) without 64-bit conversions, which this GPU does slowly: p *
// 2^19 rounded to a whole number h by adding 2^23, and what that leaves, exact in
// fp32, times 2^19 rounded the same way; w = h * 2^19 + l, since h * 2^19 is even
// and so moves no tie.  As w never falls where p grows, min(w(p), w(q)) = w(min(p,
// q)), and after a node's first rejection max(w(p) - w(q), 0) = w(p) - w(q) where
// p > q: both sums need no 64-bit arithmetic per entry either.  Later rejections
// of a node take the general way.  16 requests, trees of 9, 131,072 tokens: 50.6 ->
// 29.8 us; 64 requests, trees of up to 16, 150,001 tokens: 199 -> 97.8.
#include <cooperative_groups.h>

#include "common.cuh"

namespace mlav {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxWarps = 32;
constexpr int kOne = 38;
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 4;

// (a NaN, a negative probability: 0; above 1: 1)
__device__ __forceinline__ float clip(float p) { return fminf(fmaxf(p, 0.f), 1.f); }

// Sums of weights in two parts of 19 bits; flushed before they overflow.
struct Sum {
  uint32_t high = 0;
  int32_t low = 0;
  static __device__ __forceinline__ void split(float p, uint32_t& h, int32_t& l) {
    const float t = fmaf(p, 524288.f, 8388608.f);             // 2^23 + h
    const float rest = fmaf(p, 524288.f, -(t - 8388608.f));   // exact, at most half
    h = __float_as_uint(t) - 0x4B000000u;
    l = (int32_t)(__float_as_uint(fmaf(rest, 524288.f, 12582912.f)) - 0x4B400000u);
  }
  __device__ __forceinline__ void add(float p) {
    uint32_t h;
    int32_t l;
    split(p, h, l);
    high += h;
    low += l;
  }
  __device__ __forceinline__ int64_t flush() {
    const int64_t v = ((int64_t)high << 19) + low;
    high = 0;
    low = 0;
    return v;
  }
};
__device__ __forceinline__ int64_t weight(float p) {
  Sum s;
  s.add(clip(p));
  return s.flush();
}
__device__ __forceinline__ int64_t random24(float u) {
  return (int64_t)fminf(fmaxf(floorf(u * 16777216.f), 0.f), 16777215.f);
}
// w * Z >> 38, both at most 2^38
__device__ __forceinline__ int64_t scaled(int64_t w, int64_t Z) {
  return (int64_t)((__umul64hi((uint64_t)w, (uint64_t)Z) << (64 - kOne)) | (((uint64_t)w * (uint64_t)Z) >> kOne));
}

// The same of w = h * 2^19 + l: each shift drops what a floor drops.
__device__ __forceinline__ int64_t scaled(uint32_t h, int32_t l, int64_t Z) {
  const int32_t zh = (int32_t)(Z >> 19), zl = (int32_t)(Z & 0x7FFFF);
  const int64_t mid = (int64_t)(int32_t)h * zl + (int64_t)l * zh + (((int64_t)l * zl) >> 19);
  return (int64_t)(int32_t)h * zh + (mid >> 19);
}

// Four neighbouring entries of a row; `at` is the first one's index, `fast`
// says that their address is a multiple of 16 bytes.
__device__ __forceinline__ float4 load4(const float* row, int at, int vocab, bool fast) {
  if (fast && at >= 0 && at + 4 <= vocab) return __ldg(reinterpret_cast<const float4*>(row + at));
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = at + i >= 0 && at + i < vocab ? __ldg(row + at + i) : 0.f;
  return make_float4(v[0], v[1], v[2], v[3]);
}

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
  int64_t part[kMaxWarps];
  int64_t all[2][kMaxCluster];  // the CTAs' sums; two in turn, so that an exchange needs one cluster barrier
  int cur, num, tried, last;    // the walk's state; last: the last child looked at
  int64_t Z;
  int ask;  // 1: the walk needs sum min(r, s) for its next child, 0: it has ended
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
    int64_t r = weight(pv);
    const int64_t w = kDraft && tried > 0 ? weight(qv) : 0;
    for (int j = 0; j < tried; ++j) {
      const int64_t s = kDraft ? (j == 0 ? w : scaled(w, z[j])) : (token[j] == x ? z[j] : 0);  // (Z is 2^38 at first)
      r = r > s ? r - s : 0;
    }
    return r;
  }
  // Vector k covers entries 4k - off .. 4k - off + 3.
  __device__ __forceinline__ float4 target(int k) const { return load4(p, 4 * k - off, vocab, true); }
  __device__ __forceinline__ float4 draft(int k) const { return load4(q, 4 * k - off, vocab, q_fast); }

  // Sum over vectors first, first + 32, ... below end.
  template <What kWhat>
  __device__ __forceinline__ int64_t sum(int first, int end) const {
    const int n = kWhat == What::kTaken ? tried - 1 : tried;  // rejections before
    const bool simple = !kDraft || n == 0 || (n == 1 && kWhat == What::kLeft);
    const bool both = kDraft && (kWhat == What::kTaken || n > 0);
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
      Sum more, less;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const float a[4] = {pv[u].x, pv[u].y, pv[u].z, pv[u].w}, b[4] = {qv[u].x, qv[u].y, qv[u].z, qv[u].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = clip(a[i]);
          if (!both) {
            more.add(x);
            continue;
          }
          const float y = clip(b[i]);
          if (simple) {
            if (kWhat == What::kTaken) {
              more.add(fminf(x, y));
            } else {
              more.add(x > y ? x : 0.f);
              less.add(x > y ? y : 0.f);
            }
          } else {
            // r is what the sum of the s leaves of w(p): an r that has reached 0 stays there.
            uint32_t h;
            int32_t l;
            Sum::split(y, h, l);
            int64_t s = ((int64_t)h << 19) + l;
            for (int j = 1; j < n; ++j) s += scaled(h, l, z[j]);
            int64_t r = weight(x) - s;
            r = r > 0 ? r : 0;
            if (kWhat == What::kTaken) {
              s = scaled(h, l, z[n]);
              r = r < s ? r : s;
            }
            t += r;
          }
        }
      }
      t += more.flush() - less.flush();
    }
    return t;
  }
};

template <bool kDraft, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) accept_kernel(AcceptArgs a) {
  constexpr int kWarps = kThreads / 32;
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

  Node<kDraft> node;
  node.vocab = a.vocab;
  node.z = s.z;
  node.token = s.rejected;
  int round = 0, w0 = 0, w1 = 0;
  // A sum over the row by warps' parts (s.part) and CTAs (s.all), all of them known to all CTAs.
  auto pass = [&](auto&& f) -> int64_t {
    const int vectors = (node.off + a.vocab + 3) / 4;
    const int per = (vectors + C - 1) / C;
    const int v0 = min(rank * per, vectors), v1 = min(v0 + per, vectors);
    const int per_warp = (per + kWarps - 1) / kWarps;
    w0 = min(v0 + warp * per_warp, v1);
    w1 = min(w0 + per_warp, v1);
    const int64_t t = warp_sum(f());
    if (lane == 0) s.part[warp] = t;
    __syncthreads();
    ++round;
    if (tid < C) {
      int64_t x = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) x += s.part[w];
      *cluster.map_shared_rank(&s.all[round & 1][rank], tid) = x;
    }
    if (C > 1)
      cluster.sync();
    else
      __syncthreads();
    int64_t x = 0;
    for (int c = 0; c < C; ++c) x += s.all[round & 1][c];
    return x;
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
    const int64_t taken = pass([&] { return node.template sum<What::kTaken>(w0 + lane, w1); });
    if (tid == 0) s.Z = z > taken ? z - taken : 0;
    __syncthreads();
  }

  // ---- the next token -------------------------------------------------------------
  auto left_sum = [&]() -> int64_t {
    int64_t t = node.template sum<What::kLeft>(w0 + lane, w1);
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
  int64_t mine = 0;
  for (int c = 0; c < rank; ++c) mine += s.all[round & 1][c];
  for (int w = 0; w < warp; ++w) mine += s.part[w];
  if (sum == 0 || aim < mine || aim >= mine + s.part[warp]) return;
  // This warp's part holds the token.
#pragma unroll 1
  for (int k0 = w0; k0 < w1; k0 += 32 * kUnroll) {
    float4 pv[kUnroll], qv[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = k0 + 32 * u + lane;
      pv[u] = qv[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < w1) {
        pv[u] = node.target(k);
        if (kDraft && node.tried > 0) qv[u] = node.draft(k);
      }
    }
#pragma unroll 1
    for (int u = 0; u < kUnroll; ++u) {
      const int k = k0 + 32 * u + lane, x = 4 * k - node.off;
      float4 p4 = pv[0], q4 = qv[0];
#pragma unroll
      for (int i = 1; i < kUnroll; ++i) {
        if (i == u) {
          p4 = pv[i];
          q4 = qv[i];
        }
      }
      const int64_t r[4] = {node.left(p4.x, q4.x, x), node.left(p4.y, q4.y, x + 1), node.left(p4.z, q4.z, x + 2),
                            node.left(p4.w, q4.w, x + 3)};
      const int64_t own = (r[0] + r[1]) + (r[2] + r[3]);
      int64_t upto = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, mine + upto > aim);
      if (past) {
        if (lane == __ffs(past) - 1) {
          int64_t at = mine + upto - own;
          int i = 0;
          while (i < 3 && (at += r[i]) <= aim) ++i;
          a.next_tokens[b] = x + i;
        }
        return;
      }
      mine += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs& a, cudaStream_t stream) {
  // As many CTAs per request as a cluster has, while each has 4096 entries: a batch is as slow as its request with the
  // most rejections (64 requests, up to 16 nodes, 150,001 tokens: clusters of 2 / 4 / 8 take 170 / 119 / 98 us).  1024
  // threads where a CTA has its SM to itself, else two CTAs of 512 (16 requests: 30 against 38 us; 64: 120 against 98).
  int C = 1;
  while (C < kMaxCluster && a.vocab > 4096 * C) C *= 2;
  const bool alone = (int64_t)a.batch * C <= 152;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.batch * C));
  cfg.blockDim = dim3(alone ? 1024 : 512);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = a.draft ? (alone ? accept_kernel<true, 1024> : accept_kernel<true, 512>)
                        : (alone ? accept_kernel<false, 1024> : accept_kernel<false, 512>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mlav
