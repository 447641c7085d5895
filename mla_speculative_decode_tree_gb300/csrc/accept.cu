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
// the token.  The walk itself runs on shared memory, in every CTA alike; the
// CTAs of a cluster only exchange sums.
#include <cooperative_groups.h>

#include "common.cuh"

namespace mlav {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kOne = 38;
constexpr int kMaxCluster = 8;
constexpr int kUnroll = 4;

__device__ __forceinline__ int64_t weight(float p) {
  // (a NaN, a negative probability: 0; above 1: 1)
  return __float2ll_rn(fminf(fmaxf(p, 0.f), 1.f) * 274877906944.f);
}
__device__ __forceinline__ int64_t random24(float u) {
  return (int64_t)fminf(fmaxf(floorf(u * 16777216.f), 0.f), 16777215.f);
}
// w * Z >> 38, both at most 2^38
__device__ __forceinline__ int64_t scaled(int64_t w, int64_t Z) {
  return (int64_t)((__umul64hi((uint64_t)w, (uint64_t)Z) << (64 - kOne)) | (((uint64_t)w * (uint64_t)Z) >> kOne));
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

// The remaining mass at a node after `tried` rejections.
template <bool kDraft>
struct Node {
  const float* p;
  const float* q;
  int vocab, off;  // off: entries from the last 16-byte boundary to the target row's start
  bool q_fast;
  int tried;
  const int64_t* z;      // Z at each rejection
  const int32_t* token;  // the rejected tokens

  __device__ __forceinline__ int64_t left(float pv, float qv, int x) const {
    int64_t r = weight(pv);
    if (tried == 0) return r;
    if (kDraft) {
      const int64_t w = weight(qv);
      r -= w;  // Z is 2^38 at the first
      r = r < 0 ? 0 : r;
      for (int j = 1; j < tried; ++j) {
        r -= scaled(w, z[j]);
        r = r < 0 ? 0 : r;
      }
    } else {
      for (int j = 0; j < tried; ++j)
        if (token[j] == x) {
          r -= z[j];
          r = r < 0 ? 0 : r;
        }
    }
    return r;
  }
  // Vector k covers entries 4k - off .. 4k - off + 3.
  __device__ __forceinline__ void values(int k, float4& a, float4& b) const {
    a = load4(p, 4 * k - off, vocab, true);
    b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (kDraft && tried > 0) b = load4(q, 4 * k - off, vocab, q_fast);
  }
  __device__ __forceinline__ void lefts(int k, const float4& a, const float4& b, int64_t (&r)[4]) const {
    const int x = 4 * k - off;
    r[0] = left(a.x, b.x, x);
    r[1] = left(a.y, b.y, x + 1);
    r[2] = left(a.z, b.z, x + 2);
    r[3] = left(a.w, b.w, x + 3);
  }
};

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Shared {
  int32_t parent[kMaxQLen], token[kMaxQLen];
  int64_t k[kMaxQLen], wp[kMaxQLen], wq[kMaxQLen];  // of each node's token in its parent's rows
  int64_t z[kMaxQLen];
  int32_t rejected[kMaxQLen];
  int32_t path[kMaxQLen];
  int64_t part[kWarps];
  int64_t total[2];  // this CTA's sum; two in turn, so that one exchange needs one cluster barrier
  int64_t all[kMaxCluster];
  int cur, num, tried, next;  // the walk's state; next: the next node to look at
  int64_t Z;
  int ask;  // 1: the walk needs sum min(r, s) for its next child, 0: it has ended
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
  if (tid < n) {
    const int c = tid, parent = c == 0 ? -1 : a.parents[q0 + c], x = a.tokens[q0 + c];
    s.parent[c] = parent;
    s.token[c] = x;
    s.k[c] = random24(a.u[q0 + c]);
    int64_t wp = -1, wq = 0;  // -1: cannot be accepted
    if (parent >= 0 && parent < c && x >= 0 && x < a.vocab) {
      wp = weight(__ldg(a.target + (q0 + parent) * a.target_stride + x));
      if (kDraft) wq = weight(__ldg(a.draft + (q0 + parent) * a.draft_stride + x));
    }
    s.wp[c] = wp;
    s.wq[c] = wq;
  }
  if (tid == 0) {
    s.cur = s.tried = 0;
    s.path[0] = 0;
    s.num = s.next = 1;
    s.Z = (int64_t)1 << kOne;
  }
  __syncthreads();

  Node<kDraft> node;
  node.vocab = a.vocab;
  node.z = s.z;
  node.token = s.rejected;
  int round = 0;
  int64_t sum = 0, mine = 0;
  int v0 = 0, v1 = 0, w0 = 0, w1 = 0;
  // Sums f over the row in this CTA's slice, by warp (s.part), and exchanges
  // the CTAs' sums (s.all); returns the row's sum.
  auto pass = [&](auto&& f) -> int64_t {
    const int vectors = (node.off + a.vocab + 3) / 4;
    const int per = (vectors + C - 1) / C;
    v0 = min(rank * per, vectors);
    v1 = min(v0 + per, vectors);
    const int per_warp = (per + kWarps - 1) / kWarps;
    w0 = min(v0 + warp * per_warp, v1);
    w1 = min(w0 + per_warp, v1);
    int64_t t = 0;
#pragma unroll 1
    for (int k = w0 + lane; k < w1; k += 32 * kUnroll) {
      float4 pv[kUnroll], qv[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (k + 32 * u < w1) node.values(k + 32 * u, pv[u], qv[u]);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (k + 32 * u < w1) t += f(k + 32 * u, pv[u], qv[u]);
    }
    t = warp_sum(t);
    if (lane == 0) s.part[warp] = t;
    __syncthreads();
    if (tid == 0) {
      int64_t x = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) x += s.part[w];
      s.total[round & 1] = x;
    }
    cluster.sync();
    if (tid < C) s.all[tid] = *cluster.map_shared_rank(&s.total[round & 1], tid);
    ++round;
    __syncthreads();
    int64_t x = 0;
    for (int c = 0; c < C; ++c) x += s.all[c];
    return x;
  };
  auto at_node = [&]() {
    node.p = a.target + (q0 + s.cur) * a.target_stride;
    node.q = kDraft ? a.draft + (q0 + s.cur) * a.draft_stride : nullptr;
    node.off = (int)((reinterpret_cast<uintptr_t>(node.p) >> 2) & 3);
    node.q_fast = kDraft && (int)((reinterpret_cast<uintptr_t>(node.q) >> 2) & 3) == node.off;
    node.tried = s.tried;
  };

  // ---- the walk ----------------------------------------------------------------
#pragma unroll 1
  for (;;) {
    if (tid == 0) {
      int cur = s.cur, tried = s.tried, c = s.next;
      int64_t Z = s.Z;
      int ask = 0;
#pragma unroll 1
      for (; c < n; ++c) {
        if (s.parent[c] != cur) continue;
        if (s.wp[c] < 0) continue;  // no such token: nothing to accept or to take away
        if (kDraft && tried > 0 && Z < 0) {  // Z after the last rejection is not known yet
          ask = 1;
          break;
        }
        const int x = s.token[c];
        int64_t r = s.wp[c], sx;
        if (kDraft) {
          for (int j = 0; j < tried; ++j) {
            r -= scaled(s.wq[c], s.z[j]);
            r = r < 0 ? 0 : r;
          }
          sx = scaled(s.wq[c], Z);
        } else {
          for (int j = 0; j < tried; ++j)
            if (s.rejected[j] == x) {
              r -= s.z[j];
              r = r < 0 ? 0 : r;
            }
          sx = Z;
        }
        if ((uint64_t)s.k[c] * (uint64_t)sx < (uint64_t)r << 24) {
          cur = c;
          s.path[s.num++] = c;
          tried = 0;
          Z = (int64_t)1 << kOne;
        } else {
          s.z[tried] = Z;
          s.rejected[tried++] = x;
          Z = kDraft ? -1 : Z - (r < sx ? r : sx);
        }
      }
      s.cur = cur;
      s.tried = tried;
      s.next = c;
      s.Z = Z;
      s.ask = ask;
    }
    __syncthreads();
    at_node();
    if (!s.ask) break;
    // Z -= sum min(r, s), r and s as they were at the last rejection
    node.tried = s.tried - 1;
    const int64_t z = s.z[s.tried - 1];
    const bool both = node.tried == 0;
    const int64_t gone = pass([&](int k, const float4& pv, const float4& qv) {
      float4 qx = qv;
      if (both) qx = load4(node.q, 4 * k - node.off, a.vocab, node.q_fast);
      int64_t r[4];
      node.lefts(k, pv, qx, r);
      const float w[4] = {qx.x, qx.y, qx.z, qx.w};
      int64_t t = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t sv = scaled(weight(w[i]), z);
        t += r[i] < sv ? r[i] : sv;
      }
      return t;
    });
    if (tid == 0) s.Z = z - gone < 0 ? 0 : z - gone;
    __syncthreads();
  }

  // ---- the next token -------------------------------------------------------------
  auto left_sum = [&](int k, const float4& pv, const float4& qv) {
    int64_t r[4];
    node.lefts(k, pv, qv, r);
    return (r[0] + r[1]) + (r[2] + r[3]);
  };
  sum = pass(left_sum);
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
  const int64_t aim = (int64_t)__umul64hi((uint64_t)random24(a.u_next[b]) << 40, (uint64_t)sum);
  for (int c = 0; c < rank; ++c) mine += s.all[c];
  if (sum > 0 && aim >= mine && aim < mine + s.all[rank]) {
    for (int w = 0; w < warp; ++w) mine += s.part[w];
    if (aim >= mine && aim < mine + s.part[warp]) {  // this warp's part holds the token
#pragma unroll 1
      for (int k0 = w0; k0 < w1; k0 += 32) {
        const int k = k0 + lane;
        int64_t r[4] = {0, 0, 0, 0};
        if (k < w1) {
          float4 pv, qv;
          node.values(k, pv, qv);
          node.lefts(k, pv, qv, r);
        }
        int64_t upto = (r[0] + r[1]) + (r[2] + r[3]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, mine + upto > aim);
        if (past) {
          if (lane == __ffs(past) - 1) {
            int64_t x = mine + upto - ((r[0] + r[1]) + (r[2] + r[3]));
            int i = 0;
            while (i < 3 && (x += r[i]) <= aim) ++i;
            a.next_tokens[b] = 4 * k - node.off + i;
          }
          break;
        }
        mine += __shfl_sync(0xffffffffu, upto, 31);
      }
    }
  }
  cluster.sync();  // nobody leaves while its sums are read
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs& a, cudaStream_t stream) {
  int C = 1;
  while (C < kMaxCluster && (int64_t)a.batch * C * 2 <= 304 && a.vocab > 4096 * C) C *= 2;
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, a.draft ? accept_kernel<true> : accept_kernel<false>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mlav
