// C ABI of the operators around a verify step (declared in
// include/mla_verify.h): attention over shared prefixes, the drafts'
// verification, and the cache's rows and pages between steps.
#include <algorithm>
#include <cmath>

#include "plan.cuh"

namespace mlav {

// Workspace of a shared plan.  Tensor-core kernel: a table entry per query row
// for the shared and for the own part, then partials: a row group's partial of
// pair w stands 128 * w rows behind the group's own place, so a row has one
// place per part and 128 more per pair.  CUDA-core kernel: the chunks' partials.
void plan_shared(mla_verify_plan_s* pl, int sms) {
  auto round_up = [](size_t x, size_t a) { return (x + a - 1) / a * a; };
  size_t rows;
  pl->fused = false;
  pl->resident = pl->kernel == 1;
  if (pl->kernel) {
    pl->nq = kSharedRows;
    pl->pieces = sms / 2 > 1 ? sms / 2 : 1;
    pl->splits = 1;
    pl->smem = split_shared_smem();
    rows = 2 * (size_t)pl->rows_max + (size_t)kSharedRows * pl->pieces;
    pl->off_lse = round_up(kWsHeader + sizeof(int2) * 2 * (size_t)pl->rows_max, 256);
  } else {
    pl->shared_splits = 8;
    pl->own_splits = 4;
    pl->splits = pl->shared_splits + pl->own_splits;
    pl->min_chunk = kMinChunk;
    pl->chunk_granule = kKeysPerTile;
    rows = (size_t)pl->splits * (size_t)pl->rows_max;
    pl->off_lse = kWsHeader;
  }
  pl->off_o = round_up(pl->off_lse + sizeof(float) * rows, 256);
  pl->ws_bytes = pl->off_o + sizeof(float) * rows * kDLatent;
}

namespace {

// The shared and the own part on CUDA cores, and the ordinary merge of all
// their chunks.
cudaError_t run_shared_simt(const mla_verify_plan_s* pl, const SharedArgs& s, cudaStream_t st) {
  SplitArgs a = {};
  a.q_nope = s.q_nope;
  a.q_rope = s.q_rope;
  a.kv_pool = s.kv_pool;
  a.out_cache_loc = s.out_cache_loc;
  a.mask = s.mask;
  a.mask_indptr = s.mask_indptr;
  a.qo_indptr = s.qo_indptr;
  a.H = s.H;
  a.T = s.T;
  a.min_chunk = pl->min_chunk;
  a.chunk_granule = pl->chunk_granule;
  a.pool_rows = s.pool_rows;
  a.rows_max = s.rows_max;
  a.scale_log2 = s.scale_log2;
  a.status = s.status;
  a.part_lse = s.part_lse;
  a.part_o = s.part_o;

  a.group_indptr = s.group_indptr;
  a.requests = s.batch;
  a.batch = s.groups;
  a.kv_indptr = s.shared_indptr;
  a.kv_indices = s.shared_indices;
  a.nsplit = pl->shared_splits;
  const int64_t rows = (int64_t)s.batch * s.T * s.H;
  cudaError_t e = launch_split_simt(
      a, dim3((unsigned)((rows + kSimtRowsPerCta - 1) / kSimtRowsPerCta), a.nsplit, a.batch), st);
  if (e != cudaSuccess) return e;
  a.group_indptr = nullptr;
  a.batch = s.batch;
  a.kv_indptr = s.kv_indptr;
  a.kv_indices = s.kv_indices;
  a.nsplit = pl->own_splits;
  a.part_lse += (size_t)pl->shared_splits * s.rows_max;
  a.part_o += (size_t)pl->shared_splits * s.rows_max * kDLatent;
  e = launch_split_simt(a, dim3((s.T * s.H + kSimtRowsPerCta - 1) / kSimtRowsPerCta, a.nsplit, a.batch), st);
  if (e != cudaSuccess) return e;
  MergeArgs m = {};
  m.rows = (int)rows;
  m.qo_indptr = s.qo_indptr;
  m.batch = s.batch;
  m.H = s.H;
  m.nsplit = pl->splits;
  m.rows_max = s.rows_max;
  m.part_lse = s.part_lse;
  m.part_o = s.part_o;
  m.o = s.o;
  m.lse = s.lse;
  m.status = s.status;
  return launch_merge(m, st);
}

int check_pool(const mla_verify_plan_s* pl, const void* kv_pool, int32_t layers, int64_t layer_stride) {
  if (!kv_pool || !aligned(kv_pool, 16) || layers < 1 || layer_stride < 0 || layer_stride % 16) return MLA_VERIFY_EINVAL;
  const int64_t bytes = pl->p.pool_rows * (pl->kv4 ? kKv4RowBytes : kRowBytes);
  return layers > 1 && layer_stride < bytes ? MLA_VERIFY_EINVAL : MLA_VERIFY_OK;
}

PoolLayers pool_layers(const mla_verify_plan_s* pl, void* kv_pool, int32_t layers, int64_t layer_stride) {
  return {static_cast<uint8_t*>(kv_pool), layer_stride, layers, pl->kv4 ? kKv4RowBytes : kRowBytes, pl->p.pool_rows};
}

template <typename... P>
bool words(const P*... p) {  // all there, 4-byte aligned
  const void* all[] = {p...};
  for (const void* x : all)
    if (!x || !aligned(x, 4)) return false;
  return true;
}

int done(cudaError_t e) { return e == cudaSuccess ? MLA_VERIFY_OK : record_cuda_error(e); }

}  // namespace
}  // namespace mlav

extern "C" {

int mla_verify_run_shared(mla_verify_plan_t pl, const void* q_nope_absorbed, const void* q_rope, const void* kv_pool,
                          const int32_t* group_indptr, const int32_t* shared_indptr, const int32_t* shared_indices,
                          const int32_t* kv_indptr, const int32_t* kv_indices, const int32_t* qo_indptr,
                          const int32_t* out_cache_loc, const uint8_t* custom_mask, const int32_t* mask_indptr,
                          int32_t batch, int32_t num_groups, float sm_scale, void* workspace, size_t workspace_bytes,
                          void* o, float* lse, void* stream) {
  if (!pl || !pl->shared || batch < 0 || batch > pl->p.max_batch) return MLA_VERIFY_EINVAL;
  if (batch == 0) return MLA_VERIFY_OK;
  if (num_groups < 1 || num_groups > pl->p.max_batch) return MLA_VERIFY_EINVAL;
  // shared_indices may be NULL only when every shared prefix is empty.
  if (!words(group_indptr, shared_indptr) || (shared_indices && !aligned(shared_indices, 4)) ||
      (qo_indptr && !aligned(qo_indptr, 4)) || !o || !lse || !aligned(o, 16) || !aligned(lse, 4))
    return MLA_VERIFY_EINVAL;
  int rc = check_inputs(q_nope_absorbed, q_rope, kv_pool, kv_indptr, kv_indices, out_cache_loc, custom_mask,
                        mask_indptr, sm_scale);
  if (rc != MLA_VERIFY_OK) return rc;
  if ((rc = check_workspace(pl, workspace, workspace_bytes)) != MLA_VERIFY_OK) return rc;
  if ((rc = check_device()) != MLA_VERIFY_OK) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SharedArgs a = {};
  a.q_nope = static_cast<const __nv_bfloat16*>(q_nope_absorbed);
  a.q_rope = static_cast<const __nv_bfloat16*>(q_rope);
  a.kv_pool = static_cast<const __nv_bfloat16*>(kv_pool);
  a.group_indptr = group_indptr;
  a.shared_indptr = shared_indptr;
  a.shared_indices = shared_indices;
  a.kv_indptr = kv_indptr;
  a.kv_indices = kv_indices;
  a.out_cache_loc = out_cache_loc;
  a.mask = custom_mask;
  a.mask_indptr = mask_indptr;
  a.qo_indptr = qo_indptr;
  a.batch = batch;
  a.groups = num_groups;
  a.H = pl->p.num_heads;
  a.T = pl->p.q_len;
  a.clusters = pl->pieces;
  a.test_stall = (pl->p.flags & MLA_VERIFY_TEST_STALL_GATHER) ? 1 : 0;
  a.pool_rows = pl->p.pool_rows;
  a.rows_max = pl->rows_max;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.table = reinterpret_cast<int2*>(ws + kWsHeader);
  a.part_lse = reinterpret_cast<float*>(ws + pl->off_lse);
  a.part_o = reinterpret_cast<float*>(ws + pl->off_o);
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!pl->kernel) return done(run_shared_simt(pl, a, st));
  const cudaError_t e = launch_split_shared(a, st);
  return e != cudaSuccess ? done(e) : done(launch_merge_shared(a, st));
}

int mla_verify_accept_drafts(mla_verify_plan_t pl, const float* target_probs, int64_t target_stride,
                             const float* draft_probs, int64_t draft_stride, int32_t vocab, const int32_t* draft_tokens,
                             const int32_t* parents, const int32_t* qo_indptr, const float* uniform,
                             const float* uniform_next, int32_t batch, int32_t* accepted, int32_t* num_accepted,
                             int32_t* next_tokens, void* workspace, size_t workspace_bytes, void* stream) {
  if (!pl || batch < 0 || batch > pl->p.max_batch) return MLA_VERIFY_EINVAL;
  if (batch == 0) return MLA_VERIFY_OK;
  if (vocab < 1 || vocab > (1 << 30) || target_stride < vocab || (draft_probs && draft_stride < vocab) ||
      !words(target_probs, draft_tokens, parents, uniform, uniform_next, accepted, num_accepted, next_tokens) ||
      (draft_probs && !aligned(draft_probs, 4)) || (qo_indptr && !aligned(qo_indptr, 4)))
    return MLA_VERIFY_EINVAL;
  int rc;
  if ((rc = check_workspace(pl, workspace, workspace_bytes)) != MLA_VERIFY_OK) return rc;
  if ((rc = check_device()) != MLA_VERIFY_OK) return rc;
  AcceptArgs a = {target_probs, draft_probs, target_stride, draft_stride, draft_tokens, parents, qo_indptr, uniform,
                  uniform_next, batch, pl->p.q_len, vocab, accepted, num_accepted, next_tokens};
  return done(launch_accept(a, pl->sms, static_cast<cudaStream_t>(stream)));
}

int mla_verify_commit_drafts(mla_verify_plan_t pl, void* kv_pool, int32_t num_layers, int64_t layer_stride,
                             const int32_t* qo_indptr, const int32_t* out_cache_loc, const int32_t* accepted,
                             const int32_t* num_accepted, int32_t batch, const int32_t* seq_lens,
                             int32_t* new_seq_lens, int32_t page_size, const int32_t* block_table, int32_t max_pages,
                             int32_t* page_refs, int32_t num_pages, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (!pl || batch < 0 || batch > pl->p.max_batch || batch > 65535) return MLA_VERIFY_EINVAL;
  if (batch == 0) return MLA_VERIFY_OK;
  int rc;
  if ((rc = check_pool(pl, kv_pool, num_layers, layer_stride)) != MLA_VERIFY_OK) return rc;
  if (!words(out_cache_loc, accepted, num_accepted, seq_lens, new_seq_lens) || (qo_indptr && !aligned(qo_indptr, 4)))
    return MLA_VERIFY_EINVAL;
  if (block_table || page_refs) {
    if (!words(block_table, page_refs) || page_size < 1 || max_pages < 1 || num_pages < 0) return MLA_VERIFY_EINVAL;
  }
  if ((rc = check_workspace(pl, workspace, workspace_bytes)) != MLA_VERIFY_OK) return rc;
  if ((rc = check_device()) != MLA_VERIFY_OK) return rc;
  CommitArgs a = {pool_layers(pl, kv_pool, num_layers, layer_stride), qo_indptr, out_cache_loc, accepted, num_accepted,
                  batch, pl->p.q_len, page_size, max_pages, seq_lens, new_seq_lens, block_table, page_refs, num_pages,
                  static_cast<uint32_t*>(workspace)};
  return done(launch_commit(a, static_cast<cudaStream_t>(stream)));
}

int mla_verify_list_free_pages(mla_verify_plan_t pl, const int32_t* page_refs, int32_t num_pages, int32_t* free_pages,
                               int32_t* num_free, void* stream) {
  if (!pl || num_pages < 0 || !words(num_free) || (num_pages > 0 && !words(page_refs, free_pages)))
    return MLA_VERIFY_EINVAL;
  int rc;
  if ((rc = check_device()) != MLA_VERIFY_OK) return rc;
  return done(launch_list_free(page_refs, num_pages, free_pages, num_free, static_cast<cudaStream_t>(stream)));
}

int mla_verify_fork(mla_verify_plan_t pl, void* kv_pool, int32_t num_layers, int64_t layer_stride, const int32_t* src,
                    const int32_t* dst, int32_t n, int32_t page_size, int32_t* block_table, int32_t num_requests,
                    int32_t max_pages, int32_t* seq_lens, int32_t* page_refs, int32_t num_pages,
                    const int32_t* free_pages, int32_t num_free, int32_t* pages_used, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!pl || n < 0 || n > kMaxForks) return MLA_VERIFY_EINVAL;
  if (n == 0) return MLA_VERIFY_OK;
  int rc;
  if ((rc = check_pool(pl, kv_pool, num_layers, layer_stride)) != MLA_VERIFY_OK) return rc;
  if (!words(src, dst, block_table, seq_lens, page_refs, pages_used) || (num_free > 0 && !words(free_pages)) ||
      page_size < 1 || num_requests < 1 || max_pages < 1 || num_pages < 1 || num_free < 0)
    return MLA_VERIFY_EINVAL;
  if ((rc = check_workspace(pl, workspace, workspace_bytes)) != MLA_VERIFY_OK) return rc;
  if ((rc = check_device()) != MLA_VERIFY_OK) return rc;
  ForkArgs a = {pool_layers(pl, kv_pool, num_layers, layer_stride), src, dst, n, page_size, max_pages, num_requests,
                num_pages, num_free, block_table, seq_lens, page_refs, free_pages, pages_used,
                static_cast<uint32_t*>(workspace)};
  return done(launch_fork(a, static_cast<cudaStream_t>(stream)));
}

int mla_verify_release(mla_verify_plan_t pl, const int32_t* requests, int32_t n, int32_t page_size,
                       const int32_t* block_table, int32_t num_requests, int32_t max_pages, int32_t* seq_lens,
                       int32_t* page_refs, int32_t num_pages, void* workspace, size_t workspace_bytes, void* stream) {
  if (!pl || n < 0 || n > kMaxForks) return MLA_VERIFY_EINVAL;
  if (n == 0) return MLA_VERIFY_OK;
  if (!words(requests, block_table, seq_lens, page_refs) || page_size < 1 || num_requests < 1 || max_pages < 1 ||
      num_pages < 1)
    return MLA_VERIFY_EINVAL;
  int rc;
  if ((rc = check_workspace(pl, workspace, workspace_bytes)) != MLA_VERIFY_OK) return rc;
  if ((rc = check_device()) != MLA_VERIFY_OK) return rc;
  ReleaseArgs a = {requests, n, page_size, max_pages, num_requests, num_pages, block_table, seq_lens, page_refs,
                   static_cast<uint32_t*>(workspace)};
  return done(launch_release(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
