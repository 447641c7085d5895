// Merge kernel: combines the nsplit partials of every query row by
// log-sum-exp -- the second reduction kernel of the split-K verify
// [Custom sm_120 Verify Kernel, §"Building the Custom Kernel: From Occupancy
// Starvation to Flash-Decode"].  The per-row arithmetic is merge_row_half or
// merge_row_quarter (merge_row.cuh), bit for bit that of the split kernel's
// fused merge.
#include "merge_row.cuh"

namespace mlav {
namespace {

// Two layouts.  Many rows (the grid spans several waves): two warps per row,
// one per half of the 512 latent columns, four rows per block -- more bytes in
// flight per thread for a merge bound by reading the partials.  At most one
// wave of rows: four warps per row, one per quarter of the columns, two rows
// per block -- shorter per-row latency for a merge bound by its round trips.
// Both compute the same bits (merge_row.cuh).
constexpr int kHalfRowsPerBlock = 4;
constexpr int kQuarterRowsPerBlock = 2;

__global__ void __launch_bounds__(64 * kHalfRowsPerBlock) merge_half_kernel(MergeArgs a) {
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    // The split kernels of this call have finished (stream order): hand their
    // status bits to the "last call" word and reset the accumulator.
    const uint32_t st = a.status[0];
    if (st) atomicOr(a.status + 1, st);
    a.status[0] = 0u;
  }
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kHalfRowsPerBlock + (warp >> 1);
  const int half = warp & 1;
  if (row >= a.rows) return;
  if (a.qo_indptr && (int64_t)row >= (int64_t)a.qo_indptr[a.batch] * a.H) return;  // past the call's tokens
  merge_row_half<false>(a.part_lse, a.part_o, a.rows_max, a.nsplit, row, half, lane, a.o, a.lse);
}

template <bool kSpec>
__global__ void __launch_bounds__(128 * kQuarterRowsPerBlock, 2) merge_quarter_kernel(MergeArgs a) {
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    const uint32_t st = a.status[0];
    if (st) atomicOr(a.status + 1, st);
    a.status[0] = 0u;
  }
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int row = blockIdx.x * kQuarterRowsPerBlock + (warp >> 2);
  const int quarter = warp & 3;
  if (row >= a.rows) return;
  if (a.qo_indptr && (int64_t)row >= (int64_t)a.qo_indptr[a.batch] * a.H) return;  // past the call's tokens
  merge_row_quarter<kSpec>(a.part_lse, a.part_o, a.rows_max, a.nsplit, row, quarter, lane, a.o, a.lse);
}

// Partials of work in equal pieces (split_kv4.cuh): row group g of request b
// has the partials that seg_table[b * groups_max + g] names, nq rows each, from
// one (many short requests) to one per SM (a single long one).  A block merges
// rows_per_block rows of a request, at most 4: a warp per row where the row
// groups have few partials, else one row after the other with the partials
// dealt out to the warps.  Lane l owns columns 128 k + 4 l .. + 3.  Sums run in
// a fixed order.  An LSE of +inf makes the row NaN.
//
// What bounds it is the chain of reads: lengths, table, LSEs and partials.  A
// warp per quarter or half row, as in the merges above, left a single long
// request to a few SMs: 72 rows of ~76 partials took 16.5 us, here 10.9; 9216
// rows of two or three, 22 against 13 (cold caches).  Eight warps per row gain
// 1.6 us at 72 rows and cost 1.7 us at 576, whose blocks then take two waves;
// a block per half row gains 0.3 us at 72.
constexpr int kPieceWarps = 4;
constexpr int kFewPartials = 4;
constexpr int kAtOnce = 3;

// Largest LSE of a row's n partials, `stride` apart, and the sum of their weights.
__device__ __forceinline__ void merge_weights(const float* lse, int n, int64_t stride, int lane, float& M, float& W) {
  M = -INFINITY;
  for (int s = lane; s < n; s += 32) M = fmaxf(M, lse[s * stride]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  W = 0.f;
  if (M == -INFINITY) return;
  for (int s = lane; s < n; s += 32) W += expf(lse[s * stride] - M);  // (-inf gives 0)
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) W += __shfl_xor_sync(0xffffffffu, W, off);
}

// M and W of a row, and in acc the weighted sum of its partials first, first +
// step, ... below n.  kAtOnce partials are read at a time, the first ones before
// the LSEs are known; what has weight 0 was never written and is dropped.
__device__ __forceinline__ void merge_partials(const float* lse, const float* part, int first, int step, int n,
                                               int64_t stride, int lane, float& M, float& W, float (&acc)[16]) {
  float w[kAtOnce];
  float4 v[kAtOnce][4];
  auto load = [&](int s0) {
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int s = s0 + u * step;
      w[u] = -INFINITY;
      if (s < n) {
        w[u] = lse[s * stride];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[u][k] = *reinterpret_cast<const float4*>(part + s * stride * kDLatent + 128 * k);
      }
    }
  };
  load(first);
  merge_weights(lse, n, stride, lane, M, W);
#pragma unroll
  for (int k = 0; k < 16; ++k) acc[k] = 0.f;
#pragma unroll 1
  for (int s0 = first; s0 < n;) {
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (w[u] == -INFINITY) continue;
      const float x = expf(w[u] - M);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc[4 * k + 0] = fmaf(x, v[u][k].x, acc[4 * k + 0]);
        acc[4 * k + 1] = fmaf(x, v[u][k].y, acc[4 * k + 1]);
        acc[4 * k + 2] = fmaf(x, v[u][k].z, acc[4 * k + 2]);
        acc[4 * k + 3] = fmaf(x, v[u][k].w, acc[4 * k + 3]);
      }
    }
    s0 += kAtOnce * step;
    load(s0);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__global__ void __launch_bounds__(32 * kPieceWarps, 5) merge_pieces_kernel(MergeArgs a) {
  __shared__ float4 sums[kPieceWarps][kDLatent / 4];
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    const uint32_t st = a.status[0];
    if (st) atomicOr(a.status + 1, st);
    a.status[0] = 0u;
  }
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int blocks = (a.T * a.H + a.rows_per_block - 1) / a.rows_per_block;  // of a request
  const int b = blockIdx.x / blocks;
  const int r0 = (blockIdx.x - b * blocks) * a.rows_per_block;  // row within the request
  const int64_t q0 = a.qo_indptr ? (int64_t)a.qo_indptr[b] : (int64_t)b * a.T;
  const int64_t n_tok = a.qo_indptr ? (int64_t)a.qo_indptr[b + 1] - q0 : a.T;
  const int left = (int)(n_tok < a.T ? n_tok : a.T) * a.H - r0;
  if (left <= 0) return;
  const int rows = left < a.rows_per_block ? left : a.rows_per_block;
  const int64_t stride = a.nq;  // rows from one partial of a group to the next
  const int2* table = a.seg_table + b * a.groups_max;
  const int g0 = r0 / a.nq;  // the rows lie in two groups at most
  // A split CTA that gave up has not written the entries of its later row groups:
  // they hold what stood there, and one that points out of the workspace counts
  // as no partials.
  auto entry = [&](int g) -> int2 {
    const int2 s = table[g];
    const bool in = s.x >= 0 && s.y >= 0 && s.y <= a.partials && s.x <= a.partials - s.y;
    return in ? s : make_int2(0, 0);
  };
  const int2 seg0 = entry(g0);
  const int2 seg1 = (r0 + rows - 1) / a.nq != g0 ? entry(g0 + 1) : seg0;
  auto place = [&](int r, int& n) -> int64_t {  // first partial's row of row r0 + r, and how many
    const int2 seg = (r0 + r) / a.nq == g0 ? seg0 : seg1;
    n = seg.y;
    return (int64_t)seg.x * a.nq + (r0 + r) % a.nq;
  };
  float acc[16];
  float M, W;
  int n;
  if (max(seg0.y, seg1.y) <= kFewPartials) {
    if (warp >= rows) return;
    const int64_t prow = place(warp, n), row = q0 * a.H + r0 + warp;
    const float* part = a.part_o + prow * kDLatent + 4 * lane;
    merge_partials(a.part_lse + prow, part, 0, 1, n, stride, lane, M, W, acc);
    const float inv = W == 0.f ? 0.f : 1.f / W;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      *reinterpret_cast<uint2*>(a.o + row * kDLatent + 128 * k + 4 * lane) =
          make_uint2(pack_bf16(acc[4 * k] * inv, acc[4 * k + 1] * inv),
                     pack_bf16(acc[4 * k + 2] * inv, acc[4 * k + 3] * inv));
    if (lane == 0) a.lse[row] = M + logf(W);  // (nothing visible: -inf)
    return;
  }
#pragma unroll 1
  for (int r = 0; r < rows; ++r) {
    const int64_t prow = place(r, n), row = q0 * a.H + r0 + r;
    const float* part = a.part_o + prow * kDLatent + 4 * lane;
    merge_partials(a.part_lse + prow, part, warp, kPieceWarps, n, stride, lane, M, W, acc);
    if (r > 0) __syncthreads();  // the last row's sums have been read
#pragma unroll
    for (int k = 0; k < 4; ++k)
      sums[warp][32 * k + lane] = make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
    __syncthreads();
    const float inv = W == 0.f ? 0.f : 1.f / W;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kPieceWarps; ++w) {
      const float4 y = sums[w][threadIdx.x];
      t.x += y.x;
      t.y += y.y;
      t.z += y.z;
      t.w += y.w;
    }
    reinterpret_cast<uint2*>(a.o + row * kDLatent)[threadIdx.x] =
        make_uint2(pack_bf16(t.x * inv, t.y * inv), pack_bf16(t.z * inv, t.w * inv));
    if (threadIdx.x == 0) a.lse[row] = M + logf(W);
  }
}

}  // namespace

// Rows per block: up to 4 while that still leaves four blocks per SM.
int merge_pieces_rows(int64_t rows, int sms) {
  const int64_t r = rows / (4 * (int64_t)sms);
  return r < 1 ? 1 : r > kPieceWarps ? kPieceWarps : (int)r;
}

cudaError_t launch_merge_pieces(const MergeArgs& a, cudaStream_t stream) {
  const int grid = (a.T * a.H + a.rows_per_block - 1) / a.rows_per_block * a.batch;
  merge_pieces_kernel<<<grid, 32 * kPieceWarps, 0, stream>>>(a);
  return cudaGetLastError();
}

int merge_blocks(int rows, bool quarter) {
  const int per = quarter ? kQuarterRowsPerBlock : kHalfRowsPerBlock;
  return (rows + per - 1) / per;
}

// Quarter layout while its blocks (two rows each, two per SM) fit one wave.
bool merge_quarter_fits(int64_t rows, int sms) {
  return (rows + kQuarterRowsPerBlock - 1) / kQuarterRowsPerBlock <= 2 * (int64_t)sms;
}

cudaError_t launch_merge(const MergeArgs& a, cudaStream_t stream) {
  const int blocks = merge_blocks(a.rows, a.quarter != 0);
  if (blocks == 0) return cudaSuccess;
  if (!a.quarter)
    merge_half_kernel<<<blocks, 64 * kHalfRowsPerBlock, 0, stream>>>(a);
  else if (a.speculative)
    merge_quarter_kernel<true><<<blocks, 128 * kQuarterRowsPerBlock, 0, stream>>>(a);
  else
    merge_quarter_kernel<false><<<blocks, 128 * kQuarterRowsPerBlock, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mlav
