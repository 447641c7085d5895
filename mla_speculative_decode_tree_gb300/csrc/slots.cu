// Block tables and slot maps of a step, built on the device from the
// requests' lengths: the index arrays that a verify call, a store and a mask
// build read, without a host round trip, so the whole step fits one CUDA
// graph.
//
// Request b holds P_b = seq_lens[b] cached tokens in ceil(P_b / page) pages
// and takes T_b new ones.  It needs F_b = ceil((P_b + T_b) / page) -
// ceil(P_b / page) fresh pages, taken from free_pages in request order.
//   kv_indptr = scan(P_b), qo_indptr = scan(T_b), pages_used = sum F_b
//   row(b, pos) = table[b, pos / page] * page + pos % page
//   kv_indices[kv_indptr[b] + j]    = row(b, j),        j < P_b
//   out_cache_loc[qo_indptr[b] + t] = row(b, P_b + t),  t < T_b
//
// Every block scans the lengths of all requests itself (at most 4096: 32 KB
// from L2), so no block waits on another and one launch does everything; a
// row in a fresh page reads the free list, not the table entry another block
// writes.  The three exclusive scans stay in shared memory, and an output
// element finds its request by binary search there.
#include "common.cuh"

namespace mlav {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 4;  // outputs per thread and pass, 32 apart within a warp's 128

struct SlotsDev {
  SlotsArgs a;
  int32_t* kv;     // shared: exclusive scans, [batch + 1] each
  int32_t* qo;
  int32_t* fresh;

  __device__ __forceinline__ int seq_len(int b) const {
    const int v = a.seq_lens[b];
    return v > 0 ? v : 0;
  }
  __device__ __forceinline__ int new_len(int b) const {
    const int v = a.new_lens ? a.new_lens[b] : a.q_len;
    return v > 0 ? v : 0;
  }
  __device__ __forceinline__ int64_t page_of(int64_t pos) const {
    return a.page_shift >= 0 ? pos >> a.page_shift : (int64_t)((uint64_t)pos / (uint32_t)a.page_size);
  }
  __device__ __forceinline__ int64_t pages(int64_t tokens) const { return page_of(tokens + a.page_size - 1); }

  // The last b with scan[b] <= x (requests without entries are skipped).
  __device__ __forceinline__ int owner(const int32_t* scan, int64_t x) const {
    int lo = 0, hi = a.batch - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (scan[mid] <= x)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }

  // Pool row of position pos of request b, -1 where there is none.
  __device__ __forceinline__ int32_t row(int b, int64_t pos, uint32_t& status) const {
    const int64_t c = page_of(pos);
    const int64_t have = pages(kv[b + 1] - kv[b]);
    int64_t page = -1;
    if (c >= a.max_pages) {
      status |= kStatusNoPage;
    } else if (c < have) {
      page = a.block_table[(int64_t)b * a.max_pages + c];
      if (page < 0) status |= kStatusBadRow;
    } else {
      const int64_t f = (int64_t)fresh[b] + (c - have);
      if (f < a.num_free) {
        page = a.free_pages[f];
        if (page < 0) status |= kStatusBadRow;
      } else {
        status |= kStatusNoPage;
      }
    }
    if (page < 0) return -1;
    const int64_t r = page * a.page_size + (pos - c * a.page_size);
    if (r >= a.pool_rows) {
      status |= kStatusBadRow;
      return -1;
    }
    return (int32_t)r;
  }
};

// Exclusive scan of value(b), b < batch, into out[0 .. batch], by the block;
// sums saturate at 2^31 - 1.
template <typename F>
__device__ __forceinline__ void block_scan(int batch, int32_t* out, uint32_t* warp_sum, F value) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto add = [](uint32_t x, uint32_t y) {
    const uint32_t s = x + y;  // both at most 2^31 - 1
    return s > 0x7FFFFFFFu ? 0x7FFFFFFFu : s;
  };
  uint32_t carry = 0;
  for (int base = 0; base < batch; base += kThreads) {
    const int b = base + threadIdx.x;
    const uint32_t v = b < batch ? (uint32_t)value(b) : 0u;
    uint32_t x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x = add(x, y);
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    uint32_t before = carry;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
      if (w < warp) before = add(before, warp_sum[w]);
    if (b < batch) out[b + 1] = (int32_t)add(before, x);
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) carry = add(carry, warp_sum[w]);
    __syncthreads();
  }
  if (threadIdx.x == 0) out[0] = 0;
}

__global__ void __launch_bounds__(kThreads) slots_kernel(SlotsArgs args) {
  extern __shared__ int32_t scans[];
  __shared__ uint32_t warp_sum[kThreads / 32];
  const int n1 = args.batch + 1;
  const SlotsDev d{args, scans, scans + n1, scans + 2 * n1};
  const SlotsArgs& a = d.a;
  block_scan(a.batch, d.kv, warp_sum, [&](int b) { return d.seq_len(b); });
  block_scan(a.batch, d.qo, warp_sum, [&](int b) { return d.new_len(b); });
  block_scan(a.batch, d.fresh, warp_sum, [&](int b) {
    const int64_t P = d.seq_len(b);
    return (int32_t)(d.pages(P + d.new_len(b)) - d.pages(P));
  });
  __syncthreads();

  uint32_t status = 0;
  const int64_t K = d.kv[a.batch], N = d.qo[a.batch], F = d.fresh[a.batch];
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b <= a.batch; b += kThreads) {
      a.kv_indptr[b] = d.kv[b];
      a.qo_indptr[b] = d.qo[b];
    }
    if (threadIdx.x == 0) {
      *a.pages_used = (int32_t)(F < a.num_free ? F : a.num_free);
      if (F > a.num_free) status |= kStatusNoPage;
      if (K > a.kv_capacity || N > a.loc_capacity) status |= kStatusCapacity;
    }
  }
  const int64_t n_kv = K < a.kv_capacity ? K : a.kv_capacity;
  const int64_t n_loc = N < a.loc_capacity ? N : a.loc_capacity;
  const int64_t warp0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int64_t warps = ((int64_t)gridDim.x * kThreads) >> 5;
  const int lane = threadIdx.x & 31;
  // One pass over both maps: chunks of 128 entries, the prefixes' first.
  const int64_t c_kv = (n_kv + 127) / 128, c_loc = (n_loc + 127) / 128;
  for (int64_t c = warp0; c < c_kv + c_loc; c += warps) {
    const bool pre = c < c_kv;
    const int32_t* scan = pre ? d.kv : d.qo;
    int32_t* out = pre ? a.kv_indices : a.out_cache_loc;
    const int64_t n = pre ? n_kv : n_loc;
    const int64_t x0 = (pre ? c : c - c_kv) * 128 + lane;
    int32_t r[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      const int64_t x = x0 + 32 * k;
      r[k] = -1;
      if (x < n) {
        const int b = d.owner(scan, x);
        const int64_t pos = x - scan[b] + (pre ? 0 : d.kv[b + 1] - d.kv[b]);
        r[k] = d.row(b, pos, status);
      }
    }
#pragma unroll
    for (int k = 0; k < kPerThread; ++k)
      if (x0 + 32 * k < n) out[x0 + 32 * k] = r[k];
  }
  // The fresh pages' table entries.
  for (int64_t f = (int64_t)blockIdx.x * kThreads + threadIdx.x; f < F; f += (int64_t)gridDim.x * kThreads) {
    const int b = d.owner(d.fresh, f);
    const int64_t c = d.pages(d.kv[b + 1] - d.kv[b]) + (f - d.fresh[b]);
    if (c < a.max_pages) a.block_table[(int64_t)b * a.max_pages + c] = f < a.num_free ? a.free_pages[f] : -1;
  }
  if (status) atomicOr(a.status, status);
}

}  // namespace

cudaError_t launch_slots(const SlotsArgs& a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int smem = 3 * (a.batch + 1) * (int)sizeof(int32_t);
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  // The totals are on the device; the arrays' capacities bound them.
  const int64_t want = (a.kv_capacity + a.loc_capacity + kThreads * kPerThread - 1) / (kThreads * kPerThread);
  const int64_t cap = (int64_t)sms * 4;
  const int grid = (int)(want < 1 ? 1 : want < cap ? want : cap);
  slots_kernel<<<grid, kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mlav
