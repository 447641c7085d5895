// The cache between steps: accepted rows moved to the front of a step's new
// ones, the list of free pages, requests forked and released.
//
// Pages carry reference counts: how many requests hold them.  A page that a
// step took and only rejected drafts used never gets one, so it is free again
// by itself.  Every result is the same for any order of the blocks: counts are
// added, lists are in ascending or in the caller's order.
//
// All of it moves few bytes through dependent reads (lengths -> table -> rows),
// so the kernels are written for latency: lists are read whole, the moved rows
// with many 16-byte loads in flight, and each operator is one launch.
#include <cooperative_groups.h>

#include "common.cuh"

namespace mlav {
namespace {

namespace cg = cooperative_groups;

// Pool row of position pos of a request, -1 where its page has none.
__device__ __forceinline__ int64_t row_of(int32_t page, int64_t within, int page_size, int64_t pool_rows) {
  const int64_t r = (int64_t)page * page_size + within;
  return page >= 0 && r < pool_rows ? r : -1;
}

// Copies row src[j] to row dst[j], j < n, of one layer, by a warp.  Up to kAhead
// rows are read before any of them is written, and in ascending j: a source that
// is an earlier row's destination has been read by then when src is ascending
// and dst[j] <= src[j] in the same order.
constexpr int kAhead = 4;
__device__ __forceinline__ void move_rows(uint8_t* layer, int row_bytes, const int32_t* src, const int32_t* dst, int n,
                                          int lane) {
  const int pieces = row_bytes / 16;
#pragma unroll 1
  for (int j0 = 0; j0 < n; j0 += kAhead) {
    uint4 v[kAhead][3];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (j0 + u >= n) continue;
      const uint4* from = reinterpret_cast<const uint4*>(layer + (int64_t)src[j0 + u] * row_bytes);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (lane + 32 * k < pieces) v[u][k] = __ldcs(from + lane + 32 * k);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (j0 + u >= n) continue;
      uint4* to = reinterpret_cast<uint4*>(layer + (int64_t)dst[j0 + u] * row_bytes);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (lane + 32 * k < pieces) to[lane + 32 * k] = v[u][k];
    }
  }
}

// ---- commit --------------------------------------------------------------------
// Block (x, b): request b's rows in layers x, x + gridDim.x * warps, ... (a warp
// per layer); block (0, b) also its length and pages.
constexpr int kCommitThreads = 128;

__global__ void __launch_bounds__(kCommitThreads) commit_kernel(CommitArgs a) {
  __shared__ int32_t slot[kMaxQLen], path[kMaxQLen], src[kMaxQLen], dst[kMaxQLen];
  __shared__ int kept, moved;
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t q0 = a.qo_indptr ? (int64_t)a.qo_indptr[b] : (int64_t)b * a.T;
  int T = a.qo_indptr ? a.qo_indptr[b + 1] - (int)q0 : a.T;
  T = T < 0 ? 0 : T > a.T ? a.T : T;
  int n = a.num_accepted[b];
  bool bad = n < 0 || n > T;
  n = n < 0 ? 0 : n > T ? T : n;
  // Read before the barriers: new_seq_lens may be seq_lens, and thread 0 writes it while other warps still move rows.
  const int64_t P = a.seq_lens[b] > 0 ? a.seq_lens[b] : 0;
  if (tid < T) {
    slot[tid] = a.out_cache_loc[q0 + tid];
    path[tid] = a.accepted[(int64_t)b * a.T + tid];
  }
  __syncthreads();
  if (warp == 0) {
    // The path up to the first entry that does not ascend within the tree, and
    // of it the rows that move.
    int n_ok = n, m = 0;
#pragma unroll
    for (int h = 0; h < kMaxQLen; h += 32) {
      const int j = h + lane;
      const bool ok = j >= n || (path[j] >= (j == 0 ? 0 : path[j - 1] + 1) && path[j] < T);
      const uint32_t no = __ballot_sync(0xffffffffu, !ok);
      if (no && n_ok > h + __ffs(no) - 1) n_ok = h + __ffs(no) - 1;
      const bool in = j < n_ok && path[j] != j;
      const int32_t from = in ? slot[path[j]] : 0, to = in ? slot[j] : 0;
      const bool rows_ok = from >= 0 && from < a.pool.rows && to >= 0 && to < a.pool.rows;
      bad |= in && !rows_ok;
      const uint32_t moves = __ballot_sync(0xffffffffu, in && rows_ok);
      if (in && rows_ok) {
        const int at = m + __popc(moves & ((1u << lane) - 1u));
        src[at] = from;
        dst[at] = to;
      }
      m += __popc(moves);
    }
    bad |= n_ok < n;
    if (lane == 0) {
      kept = n_ok;
      moved = m;
    }
  }
  __syncthreads();
  for (int layer = blockIdx.x * (kCommitThreads / 32) + warp; layer < a.pool.layers;
       layer += gridDim.x * (kCommitThreads / 32))
    move_rows(a.pool.base + layer * a.pool.layer_stride, a.pool.row_bytes, src, dst, moved, lane);
  if (blockIdx.x != 0) return;
  const int64_t L = P + kept;
  if (tid == 0) a.new_seq_lens[b] = (int32_t)(L > 0x7FFFFFFF ? 0x7FFFFFFF : L);
  if (a.block_table) {
    const int64_t c0 = (P + a.page_size - 1) / a.page_size;
    int64_t c1 = (L + a.page_size - 1) / a.page_size;
    c1 = c1 < a.max_pages ? c1 : a.max_pages;
    for (int64_t c = c0 + tid; c < c1; c += kCommitThreads) {
      const int32_t page = a.block_table[(int64_t)b * a.max_pages + c];
      if (page >= 0 && page < a.num_pages)
        a.page_refs[page] = 1;
      else
        bad = true;
    }
  }
  if (bad) atomicOr(a.status, kStatusBadRow);
}

// ---- free list -----------------------------------------------------------------
// The pages whose count is 0, in ascending order, then -1 up to the end.  One
// cluster: a CTA turns its part of the counts into bits and their running
// counts in shared memory, the CTAs exchange their sums, then a warp writes the
// pages of a word of bits with one store.  8,193 / 100,000 / 1,000,000 pages: 6.0 / 8.1 / 31.5 us.
constexpr int kFreeThreads = 1024;
constexpr int kFreeWarps = kFreeThreads / 32;
constexpr int kFreeWords = 8192;  // words of 32 pages per CTA and round
constexpr int kFreeUnroll = 8;
constexpr int kFreeCluster = 8;

__global__ void __launch_bounds__(kFreeThreads, 1)
    list_free_kernel(const int32_t* refs, int num_pages, int32_t* free_pages, int32_t* num_free) {
  extern __shared__ uint32_t mem[];
  uint32_t* const bits = mem;
  uint32_t* const before = mem + kFreeWords;
  __shared__ uint32_t warp_sum[kFreeWarps];
  __shared__ uint32_t totals[2];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool wide = (reinterpret_cast<uintptr_t>(refs) & 15) == 0;
  uint32_t carry = 0;
  int round = 0;
  const int64_t all_words = ((int64_t)num_pages + 31) / 32;
  for (int64_t base = 0; base < all_words; base += (int64_t)C * kFreeWords, ++round) {
    const int64_t left = all_words - base;
    const int64_t per = left < (int64_t)C * kFreeWords ? ((left + C - 1) / C + 3) / 4 * 4 : kFreeWords;  // whole quads
    const int64_t first = base + rank * per;
    const int words = (int)(first >= all_words ? 0 : all_words - first < per ? all_words - first : per);
    // A warp reads 128 counts at a time: lane l four of them, eight lanes a word.
#pragma unroll 1
    for (int w = 4 * warp; w < words; w += 4 * kFreeWarps * kFreeUnroll) {
      uint32_t nib[kFreeUnroll];
#pragma unroll
      for (int u = 0; u < kFreeUnroll; ++u) {
        const int64_t page = (first + w + 4 * kFreeWarps * u) * 32 + 4 * lane;
        nib[u] = 0;
        if (w + 4 * kFreeWarps * u < words) {
          if (wide && page + 4 <= num_pages) {
            const int4 v = __ldg(reinterpret_cast<const int4*>(refs + page));
            nib[u] = (v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3;
          } else {
            for (int i = 0; i < 4; ++i)
              if (page + i < num_pages && __ldg(refs + page + i) == 0) nib[u] |= 1u << i;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kFreeUnroll; ++u) {
        const int at = w + 4 * kFreeWarps * u;
        uint32_t x = nib[u] << (4 * (lane & 7));
        x |= __shfl_xor_sync(0xffffffffu, x, 1);
        x |= __shfl_xor_sync(0xffffffffu, x, 2);
        x |= __shfl_xor_sync(0xffffffffu, x, 4);
        if ((lane & 7) == 0 && at + (lane >> 3) < words) bits[at + (lane >> 3)] = x;
      }
    }
    __syncthreads();
    // Running counts: thread t holds words per_t * t ..
    const int per_t = (words + kFreeThreads - 1) / kFreeThreads;
    uint32_t mine = 0;
    for (int i = 0; i < per_t; ++i) {
      const int w = per_t * tid + i;
      if (w < words) mine += __popc(bits[w]);
    }
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    uint32_t ws = warp_sum[lane], wu = ws;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, wu, o);
      if (lane >= o) wu += y;
    }
    uint32_t at = __shfl_sync(0xffffffffu, wu - ws, warp) + upto - mine;
    const uint32_t total = __shfl_sync(0xffffffffu, wu, 31);
    for (int i = 0; i < per_t; ++i) {
      const int w = per_t * tid + i;
      if (w < words) {
        before[w] = at;
        at += __popc(bits[w]);
      }
    }
    if (tid == 0) totals[round & 1] = total;
    cluster.sync();
    uint32_t below = carry, sum = 0;
    for (int c = 0; c < C; ++c) {
      const uint32_t t = *cluster.map_shared_rank(&totals[round & 1], c);
      below += c < rank ? t : 0;
      sum += t;
    }
    carry += sum;
    for (int w = warp; w < words; w += kFreeWarps) {
      const uint32_t x = bits[w];
      if (x >> lane & 1u)
        free_pages[(int64_t)below + before[w] + __popc(x & ((1u << lane) - 1u))] = (int32_t)((first + w) * 32 + lane);
    }
    __syncthreads();
  }
  if (rank == 0 && tid == 0) *num_free = (int32_t)carry;
  for (int64_t i = (int64_t)carry + rank * kFreeThreads + tid; i < num_pages; i += (int64_t)C * kFreeThreads)
    free_pages[i] = -1;
  cluster.sync();  // nobody leaves while its sums are read
}

// The same of at most kFewPages pages, by one CTA with eight counts per thread: no bits, no cluster.  2048 pages: 4.9 ->
// 3.0 us, of which an empty launch is 1.5.
constexpr int kFewPages = 8 * kFreeThreads;

__global__ void __launch_bounds__(kFreeThreads, 1)
    list_free_few_kernel(const int32_t* refs, int num_pages, int32_t* free_pages, int32_t* num_free) {
  __shared__ uint32_t warp_sum[kFreeWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool wide = (reinterpret_cast<uintptr_t>(refs) & 15) == 0;
  uint32_t bits = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int page = 8 * tid + 4 * k;
    if (wide && page + 4 <= num_pages) {
      const int4 v = __ldg(reinterpret_cast<const int4*>(refs + page));
      bits |= ((v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3) << (4 * k);
    } else {
      for (int i = 0; i < 4; ++i)
        if (page + i < num_pages && __ldg(refs + page + i) == 0) bits |= 1u << (4 * k + i);
    }
  }
  const uint32_t mine = __popc(bits);
  uint32_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  uint32_t ws = warp_sum[lane], wu = ws;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, wu, o);
    if (lane >= o) wu += y;
  }
  int at = (int)(__shfl_sync(0xffffffffu, wu - ws, warp) + upto - mine);
  const int total = (int)__shfl_sync(0xffffffffu, wu, 31);
  for (; bits; bits &= bits - 1) free_pages[at++] = 8 * tid + __ffs(bits) - 1;
  for (int i = total + tid; i < num_pages; i += kFreeThreads) free_pages[i] = -1;
  if (tid == 0) *num_free = total;
}

// ---- fork ----------------------------------------------------------------------
// Block (x, i): fork i's share of table entries and of rows; block (0, i) its length.
constexpr int kForkThreads = 256;

__device__ __forceinline__ bool in_range(int r, int n) { return (uint32_t)r < (uint32_t)n; }

__global__ void __launch_bounds__(kForkThreads) fork_kernel(ForkArgs a) {
  const int i = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t status = 0;
  // Tokens of fork j's source; -1: it names a request that is not there, or itself.
  auto length = [&](int j) -> int64_t {
    const int s = a.src[j], d = a.dst[j];
    if (!in_range(s, a.requests) || !in_range(d, a.requests) || s == d) return -1;
    const int64_t P = a.seq_lens[s];
    return P < 0 ? 0 : P;
  };
  // Fresh pages go to the forks in order; a request that is forked into twice, or
  // from as well, is left alone (every block of it finds the same).
  int rank = 0, clash = 0;
  const int dst = a.dst[i];
  for (int j = tid; j < a.n; j += kForkThreads) {
    if (j < i) {
      const int64_t P = length(j);
      rank += P > 0 && P % a.page_size != 0 ? 1 : 0;
    }
    clash |= (j < i && a.dst[j] == dst) || (j != i && a.src[j] == dst);
  }
  __shared__ int ranks;
  if (tid == 0) ranks = 0;
  __syncthreads();
  if (rank) atomicAdd(&ranks, rank);
  clash = __syncthreads_or(clash);
  rank = ranks;
  const int64_t P = length(i);
  const int64_t full = P > 0 ? P / a.page_size : 0;
  const int tail = P > 0 ? (int)(P % a.page_size) : 0;
  // The entries that the forks went through; the list may end before them.  (The last of them is read now, used at the end.)
  const bool counts = blockIdx.x == 0 && i == a.n - 1 && tid == 0;
  int used = 0, last_entry = 0;
  if (counts) {
    used = rank + (tail ? 1 : 0);
    used = used < a.num_free ? used : a.num_free;
    if (used > 0) last_entry = a.free_pages[used - 1];
  }
  const auto count = [&]() {
    if (counts) *a.pages_used = last_entry < 0 ? list_end(a.free_pages, used) : used;
  };
  if (P < 0 || clash) {
    if (tid == 0 && blockIdx.x == 0) atomicOr(a.status, kStatusBadRow);
    count();
    return;
  }
  const int32_t* from = a.block_table + (int64_t)a.src[i] * a.max_pages;
  int32_t* to = a.block_table + (int64_t)dst * a.max_pages;
  for (int64_t c = (int64_t)blockIdx.x * kForkThreads + tid; c < full && c < a.max_pages;
       c += (int64_t)gridDim.x * kForkThreads) {
    const int32_t page = from[c];
    to[c] = page;
    if (in_range(page, a.num_pages))
      atomicAdd(a.page_refs + page, 1);
    else
      status |= kStatusBadRow;
  }
  if (full + (tail ? 1 : 0) > a.max_pages) status |= kStatusNoPage;
  int64_t len = P;
  if (tail) {
    int32_t fresh = rank < a.num_free && full < a.max_pages ? a.free_pages[rank] : -1;
    if (!in_range(fresh, a.num_pages) || row_of(fresh, tail - 1, a.page_size, a.pool.rows) < 0) {
      fresh = -1;
      status |= kStatusNoPage;
      len = full * a.page_size;  // what the shared pages hold
    }
    const int32_t old = full < a.max_pages ? from[full] : -1;
    if (blockIdx.x == 0 && tid == 0 && full < a.max_pages) {
      to[full] = fresh;
      if (fresh >= 0) a.page_refs[fresh] = 1;
    }
    if (fresh >= 0 && in_range(old, a.num_pages) && row_of(old, tail - 1, a.page_size, a.pool.rows) >= 0) {
      // The tail's rows lie together in both pages, so a layer's part is one run of
      // 16-byte pieces.
      const int64_t pieces = (int64_t)tail * a.pool.row_bytes / 16;
      const int64_t o0 = (int64_t)old * a.page_size * a.pool.row_bytes, n0 = (int64_t)fresh * a.page_size * a.pool.row_bytes;
      constexpr int kRun = 32 * 8;  // pieces per warp and step
      const int64_t runs = (pieces + kRun - 1) / kRun, warps = (int64_t)gridDim.x * (kForkThreads / 32);
      for (int64_t w = (int64_t)blockIdx.x * (kForkThreads / 32) + warp; w < runs * a.pool.layers; w += warps) {
        const int64_t layer = w / runs, p0 = (w - layer * runs) * kRun + lane;
        uint8_t* base = a.pool.base + layer * a.pool.layer_stride;
        const uint4* s = reinterpret_cast<const uint4*>(base + o0);
        uint4* d = reinterpret_cast<uint4*>(base + n0);
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (p0 + 32 * k < pieces) v[k] = __ldcs(s + p0 + 32 * k);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (p0 + 32 * k < pieces) d[p0 + 32 * k] = v[k];
      }
    } else if (fresh >= 0) {
      status |= kStatusBadRow;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    const int64_t most = (int64_t)a.max_pages * a.page_size;
    a.seq_lens[dst] = (int32_t)(len < most ? len : most);
  }
  count();
  if (status) atomicOr(a.status, status);
}

// ---- release -------------------------------------------------------------------
// A cluster per entry: its CTAs share the request's pages.
constexpr int kReleaseThreads = 512;
constexpr int kReleaseCluster = 8;

__global__ void __launch_bounds__(kReleaseThreads) release_kernel(ReleaseArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int i = blockIdx.x / C, tid = threadIdx.x;
  const int b = a.which[i];
  uint32_t status = 0;
  // (an entry that an earlier one repeats has been counted there)
  int again = 0;
  for (int j = tid; j < i; j += kReleaseThreads) again |= a.which[j] == b;
  again = __syncthreads_or(again);
  const bool is = in_range(b, a.requests);
  if (is && !again) {
    const int64_t P = a.seq_lens[b];
    int64_t pages = P > 0 ? (P + a.page_size - 1) / a.page_size : 0;
    if (pages > a.max_pages) pages = a.max_pages;
    for (int64_t c = (int64_t)rank * kReleaseThreads + tid; c < pages; c += (int64_t)C * kReleaseThreads) {
      const int32_t page = a.block_table[(int64_t)b * a.max_pages + c];
      if (in_range(page, a.num_pages)) {
        if (atomicSub(a.page_refs + page, 1) <= 0) {  // it had none: the count stays
          atomicAdd(a.page_refs + page, 1);
          status |= kStatusBadRow;
        }
      } else {
        status |= kStatusBadRow;
      }
    }
  }
  if (!is) status |= kStatusBadRow;
  cluster.sync();  // every CTA has read the length
  if (is && !again && rank == 0 && tid == 0) a.seq_lens[b] = 0;
  if (status) atomicOr(a.status, status);
}

template <typename Kernel, typename... Args>
cudaError_t launch_cluster(Kernel kernel, int blocks, int threads, int cluster, size_t smem, cudaStream_t stream,
                           Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_commit(const CommitArgs& a, cudaStream_t stream) {
  const int x = (a.pool.layers + kCommitThreads / 32 - 1) / (kCommitThreads / 32);
  commit_kernel<<<dim3(x < 1 ? 1 : x, a.batch), kCommitThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_list_free(const int32_t* page_refs, int num_pages, int32_t* free_pages, int32_t* num_free,
                             cudaStream_t stream) {
  if (num_pages <= kFewPages) {
    list_free_few_kernel<<<1, kFreeThreads, 0, stream>>>(page_refs, num_pages, free_pages, num_free);
    return cudaGetLastError();
  }
  constexpr size_t smem = 2 * kFreeWords * sizeof(uint32_t);
  cudaError_t e = cudaFuncSetAttribute(list_free_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  int C = 2;
  while (C < kFreeCluster && (int64_t)C * 8192 < num_pages) C *= 2;
  return launch_cluster(list_free_kernel, C, kFreeThreads, C, smem, stream, page_refs, num_pages, free_pages, num_free);
}

cudaError_t launch_fork(const ForkArgs& a, cudaStream_t stream) {
  // Enough blocks per fork for its table entries and for the rows of a full page
  // in all layers, 4 KB of row data (a step of the copy loop) per warp.
  const int64_t bytes = (int64_t)a.pool.layers * (a.page_size - 1) * a.pool.row_bytes;
  const int64_t by_rows = (bytes + 4096 * (kForkThreads / 32) - 1) / (4096 * (kForkThreads / 32));
  const int64_t by_pages = (a.max_pages + 4 * kForkThreads - 1) / (4 * kForkThreads);
  int64_t x = by_rows > by_pages ? by_rows : by_pages;
  x = x < 1 ? 1 : x > 128 ? 128 : x;
  fork_kernel<<<dim3((unsigned)x, (unsigned)a.n), kForkThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_release(const ReleaseArgs& a, cudaStream_t stream) {
  int C = 1;
  while (C < kReleaseCluster && C * 2 * kReleaseThreads < a.max_pages) C *= 2;
  return launch_cluster(release_kernel, a.n * C, kReleaseThreads, C, 0, stream, a);
}

}  // namespace mlav
