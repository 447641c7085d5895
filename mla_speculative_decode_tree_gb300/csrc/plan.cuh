// The host-side plan and the checks that the entry points' translation units
// share (defined in api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/mla_verify.h"
#include "kv4.cuh"

using namespace mlav;

struct mla_verify_plan_s {
  mla_verify_params p;
  int kernel;  // 1 = tcgen05, 0 = CUDA cores
  int sms;     // of the device that the plan was made on
  int nq;      // query rows per split CTA
  bool resident;  // tensor-core kernel in resident-tile mode (each key lands once per CTA)
  int groups;  // row groups per request
  int64_t rows_max;
  bool fused;  // the split kernel merges (MLA_VERIFY_FUSED_MERGE on the tensor-core kernel)
  int splits;  // KV chunks per request = grid dimension = partials per row (nsplit, or the plan's count)
  int min_chunk;  // shortest chunk of any request (keys)
  int chunk_granule;  // chunk lengths are multiples of it (keys)
  size_t off_cnt, off_lse, off_o, ws_bytes;  // [0, off_lse) must be zero between calls
  int merge_blocks;
  bool merge_quarter;  // merge with four warps per row (at most one wave of rows)
  int smem;
  bool kv4;  // the pool holds 4-bit rows (MLA_VERIFY_KV4)
  int pieces;  // > 0: the 4-bit kernel's CTAs, which take the work in equal pieces (nsplit = 0)
  int seg_cost;  // its start and end of a row group, in tiles
  int merge_rows;  // rows per merge block then
  bool shared;  // requests in groups with shared prefixes (MLA_VERIFY_SHARED)
  int shared_splits, own_splits;  // its CUDA-core kernel: KV chunks of a shared and of an own part
};

namespace mlav {
// Records the text of a CUDA error for mla_verify_strerror and returns MLA_VERIFY_ECUDA.
int record_cuda_error(cudaError_t e);
// MLA_VERIFY_OK on an sm_103 device (cached per device).
int check_device();
// The input arrays of a split launch (everything but the workspace).
int check_inputs(const void* q_nope_absorbed, const void* q_rope, const void* kv_pool, const int32_t* kv_indptr,
                 const int32_t* kv_indices, const int32_t* out_cache_loc, const uint8_t* custom_mask,
                 const int32_t* mask_indptr, float sm_scale);
// The workspace of a call that only reports into its status word.
int check_workspace(const mla_verify_plan_s* pl, const void* workspace, size_t workspace_bytes);
// Sizes of a plan with MLA_VERIFY_SHARED (api_step.cu).
void plan_shared(mla_verify_plan_s* pl, int sms);
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
}  // namespace mlav
