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
// writes.  The three exclusive scans and P_b stay in shared memory.  A warp takes 128
// output entries; their request is found by a warp-wide search there, and a
// chunk inside one request's prefix -- nearly all -- then needs two table
// entries per thread and one 16-byte store.
//
// Its traffic is small (512 requests with 2.1 M cached tokens: 8.4 MB, 1.3 us);
// what bounds it is latency -- launch, lengths, scan, a table entry -- and
// instructions: 8.6 us (GB300), of which ~4 are what 16 requests take as well.
// One block of 1024 threads per SM beats two of 512 (8.8 us: the scan is done
// twice) and four (12); chunks of neighbouring warps beat a run of chunks per
// warp (16).
#include "common.cuh"

namespace mlav {
namespace {

constexpr int kThreads = 1024;  // one block per SM: the scans are done once there
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = 4;  // consecutive outputs per thread: a warp's chunk is 128

// kPow2: pages of 2^page_shift rows.
template <bool kPow2>
struct SlotsDev {
  SlotsArgs a;
  int32_t* kv;     // shared: exclusive scans, [batch + 1] each
  int32_t* qo;
  int32_t* fresh;
  int32_t* cached;  // P_b (the scan's sums stop at 2^31 - 1, so its differences are not it)

  __device__ __forceinline__ int seq_len(int b) const {
    const int v = a.seq_lens[b];
    return v > 0 ? v : 0;
  }
  __device__ __forceinline__ int new_len(int b) const {
    const int v = a.new_lens ? a.new_lens[b] : a.q_len;
    return v > 0 ? v : 0;
  }
  __device__ __forceinline__ int64_t page_of(int64_t pos) const {
    if (kPow2) return pos >> a.page_shift;
    if ((pos >> 32) == 0) return (uint32_t)pos / (uint32_t)a.page_size;
    return (int64_t)((uint64_t)pos / (uint32_t)a.page_size);
  }
  __device__ __forceinline__ int page_of_entry(int pos) const {
    return kPow2 ? pos >> a.page_shift : (int)((uint32_t)pos / (uint32_t)a.page_size);
  }
  __device__ __forceinline__ int64_t pages(int64_t tokens) const { return page_of(tokens + a.page_size - 1); }

  // The last b of lo..hi with scan[b] <= x (requests without entries are skipped).
  __device__ __forceinline__ int owner(const int32_t* scan, int32_t x, int lo, int hi) const {
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (scan[mid] <= x)
        lo = mid;
      else
        hi = mid - 1;
    }
    return lo;
  }

  // The same for the warp's common x: 32 probes at a time.
  __device__ __forceinline__ int owner_warp(const int32_t* scan, int32_t x, int lane) const {
    int lo = 0, n = a.batch;
    while (n > 1) {
      const int step = (n + 31) >> 5, i = lane * step;
      const uint32_t below = __ballot_sync(0xffffffffu, i < n && (i == 0 || scan[lo + i] <= x));
      const int last = (31 - __clz(below)) * step;
      lo += last;
      n = n - last < step ? n - last : step;
    }
    return lo;
  }

  // Pool row of position pos, which lies on `page`, the request's c-th; -1 where there is none
  // (fresh: a page of the free list, which an entry of -1 ends).
  __device__ __forceinline__ int32_t row_on(int32_t page, int64_t c, int64_t pos, uint32_t& status, bool fresh = false) const {
    const int64_t r = (int64_t)page * a.page_size + (pos - c * a.page_size);
    if (page >= 0 && r < a.pool_rows) return (int32_t)r;
    status |= fresh && page < 0 ? kStatusNoPage : kStatusBadRow;
    return -1;
  }

  // Where the page of position pos of request b is written, its c-th page; null where there is none.
  __device__ __forceinline__ const int32_t* page_at(int b, int64_t pos, int64_t& c, bool& is_fresh) const {
    c = page_of(pos);
    const int64_t have = pages(cached[b]);
    is_fresh = c >= have;
    if (c >= a.max_pages) return nullptr;
    if (c < have) return a.block_table + (int64_t)b * a.max_pages + c;
    const int64_t f = (int64_t)fresh[b] + (c - have);
    return f < a.num_free ? a.free_pages + f : nullptr;
  }

  // Rows of cached positions pos .. pos+3 of request b.
  __device__ __forceinline__ int4 rows4(int b, int pos, uint32_t& status) const {
    const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
    if (a.page_size >= kPerThread) {
      // they lie on two pages at most, both whole in the pool as a rule
      const int c0 = page_of_entry(pos), c1 = page_of_entry(pos + 3);
      if (c1 < a.max_pages) {
        const uint32_t p0 = (uint32_t)table[c0], p1 = (uint32_t)table[c1];
        if (p0 < a.whole_pages && p1 < a.whole_pages) {
          const int x = (int)(p0 - c0) * a.page_size + pos, y = (int)(p1 - c1) * a.page_size + pos;
          const int next = c1 * a.page_size - pos;  // from here on the second page
          return make_int4(0 < next ? x : y, (1 < next ? x : y) + 1, (2 < next ? x : y) + 2, (3 < next ? x : y) + 3);
        }
      }
    }
    int32_t r[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      const int c = page_of_entry(pos + k);
      r[k] = -1;
      if (c < a.max_pages)
        r[k] = row_on(table[c], c, pos + k, status);
      else
        status |= kStatusNoPage;
    }
    return make_int4(r[0], r[1], r[2], r[3]);
  }
};

__device__ __forceinline__ uint32_t add_sat(uint32_t x, uint32_t y) {  // both at most 2^31 - 1
  const uint32_t s = x + y;
  return s > 0x7FFFFFFFu ? 0x7FFFFFFFu : s;
}

// Inclusive scans of three values over the warp.
__device__ __forceinline__ void scan3(uint32_t (&x)[3], int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x[k], off);
      if (lane >= off) x[k] = add_sat(x[k], y);
    }
  }
}

// The three exclusive scans, by the block: kThreads requests at a time, all
// three sums together; sums stop at 2^31 - 1.
template <bool kPow2>
__device__ __forceinline__ void scan_requests(const SlotsDev<kPow2>& d) {
  __shared__ uint32_t warp_sum[3][kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t carry[3] = {0, 0, 0};
#pragma unroll 1
  for (int base = 0; base < d.a.batch; base += kThreads) {
    const int b = base + threadIdx.x;
    uint32_t x[3] = {0, 0, 0};
    if (b < d.a.batch) {
      const int P = d.seq_len(b), T = d.new_len(b);
      d.cached[b] = P;
      x[0] = (uint32_t)P;
      x[1] = (uint32_t)T;
      x[2] = (uint32_t)(d.pages((int64_t)P + T) - d.pages(P));
    }
    if (base + 32 * warp < d.a.batch) scan3(x, lane);
    if (lane == 31) {
#pragma unroll
      for (int k = 0; k < 3; ++k) warp_sum[k][warp] = x[k];
    }
    __syncthreads();
    uint32_t sum[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) sum[k] = warp_sum[k][lane];
    scan3(sum, lane);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t before = __shfl_sync(0xffffffffu, sum[k], warp > 0 ? warp - 1 : 0);
      int32_t* const out = k == 0 ? d.kv : k == 1 ? d.qo : d.fresh;
      if (b < d.a.batch) out[b + 1] = (int32_t)add_sat(add_sat(carry[k], warp > 0 ? before : 0u), x[k]);
      carry[k] = add_sat(carry[k], __shfl_sync(0xffffffffu, sum[k], 31));
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) d.kv[0] = d.qo[0] = d.fresh[0] = 0;
  __syncthreads();
}

template <bool kPow2>
__global__ void __launch_bounds__(kThreads) slots_kernel(SlotsArgs args) {
  extern __shared__ int32_t scans[];
  const int n1 = args.batch + 1;
  const SlotsDev<kPow2> d{args, scans, scans + n1, scans + 2 * n1, scans + 3 * n1};
  const SlotsArgs& a = d.a;
  scan_requests(d);

  uint32_t status = 0;
  const int64_t K = d.kv[a.batch], N = d.qo[a.batch], F = d.fresh[a.batch];
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b <= a.batch; b += kThreads) {
      a.kv_indptr[b] = d.kv[b];
      a.qo_indptr[b] = d.qo[b];
    }
    if (threadIdx.x == 0) {
      if (F == 0 || a.num_free == 0) *a.pages_used = 0;  // (else whoever writes the last page's table entry)
      if (F > a.num_free) status |= kStatusNoPage;
      if (K > a.kv_capacity || N > a.loc_capacity) status |= kStatusCapacity;
    }
  }
  // (the scans stop at 2^31 - 1: 32 bits count the entries)
  const int n_kv = (int)(K < a.kv_capacity ? K : a.kv_capacity);
  const int n_loc = (int)(N < a.loc_capacity ? N : a.loc_capacity);
  const int warps = gridDim.x * kWarps;
  const int lane = threadIdx.x & 31;
  // One pass over both maps: chunks of 128 entries, the prefixes' first.
  const int c_kv = (int)(((uint32_t)n_kv + 127) / 128), c_all = c_kv + (int)(((uint32_t)n_loc + 127) / 128);
  const bool wide = (reinterpret_cast<uintptr_t>(a.kv_indices) & 15) == 0;
  for (int c = (threadIdx.x >> 5) * gridDim.x + blockIdx.x; c < c_all; c += warps) {  // few chunks go to all SMs
    const bool pre = c < c_kv;
    const int32_t* scan = pre ? d.kv : d.qo;
    int32_t* out = pre ? a.kv_indices : a.out_cache_loc;
    const int n = pre ? n_kv : n_loc;
    const int first = (pre ? c : c - c_kv) * 128;
    // The chunk's first entry finds its request for the warp, in a chunk of
    // several requests the last one too.
    const int left = n - first;
    const int b0 = d.owner_warp(scan, first, lane);
    if (pre && left >= 128 && scan[b0 + 1] - first >= 128) {
      const int x0 = first + kPerThread * lane;
      const int4 r = d.rows4(b0, x0 - scan[b0], status);
      if (wide) {
        *reinterpret_cast<int4*>(out + x0) = r;
      } else {
        out[x0] = r.x;
        out[x0 + 1] = r.y;
        out[x0 + 2] = r.z;
        out[x0 + 3] = r.w;
      }
      continue;
    }
    const int b1 = d.owner_warp(scan, first + (left < 128 ? left : 128) - 1, lane);
    const int32_t* at[kPerThread];
    int64_t pos[kPerThread], page_no[kPerThread];
    bool fresh[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      at[k] = nullptr;
      fresh[k] = false;
      if (lane + 32 * k < left) {
        const int x = first + lane + 32 * k;
        const int b = d.owner(scan, x, b0, b1);
        pos[k] = (int64_t)(x - scan[b]) + (pre ? 0 : d.cached[b]);
        at[k] = d.page_at(b, pos[k], page_no[k], fresh[k]);
        if (!at[k]) status |= kStatusNoPage;
      }
    }
    int32_t page[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) page[k] = at[k] ? *at[k] : -1;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      if (lane + 32 * k < left)
        out[first + lane + 32 * k] = at[k] ? d.row_on(page[k], page_no[k], pos[k], status, fresh[k]) : -1;
    }
  }
  // The fresh pages' table entries (the last warps have the fewest chunks).
  const int64_t last = (F < a.num_free ? F : a.num_free) - 1;
  for (int64_t f = (int64_t)(kThreads - 1 - threadIdx.x) * gridDim.x + blockIdx.x; f < F;
       f += (int64_t)gridDim.x * kThreads) {
    const int b = d.owner(d.fresh, f, 0, a.batch - 1);
    const int64_t c = d.pages(d.cached[b]) + (f - d.fresh[b]);
    const int32_t page = f < a.num_free ? a.free_pages[f] : -1;
    if (c < a.max_pages) a.block_table[(int64_t)b * a.max_pages + c] = page;
    if (f == last) {  // (the list may end before it)
      const int used = page < 0 ? list_end(a.free_pages, (int)f) : (int)f + 1;
      *a.pages_used = used;
      if (used < F) status |= kStatusNoPage;
    }
  }
  if (status) atomicOr(a.status, status);
}

}  // namespace

cudaError_t launch_slots(const SlotsArgs& a, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  auto kernel = a.page_shift >= 0 ? slots_kernel<true> : slots_kernel<false>;
  const int smem = (4 * a.batch + 3) * (int)sizeof(int32_t);
  if (smem > 47 * 1024) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  // The totals are on the device; the arrays' capacities bound them.
  const int64_t want = (a.kv_capacity + a.loc_capacity + 511) / 512;  // at least four chunks for a block
  const int64_t cap = (int64_t)sms;
  const int grid = (int)(want < 1 ? 1 : want < cap ? want : cap);
  kernel<<<grid, kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mlav
