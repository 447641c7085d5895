// Store and load of 4-bit cache rows (format: kv4.cuh).
//
// Store: token i's 512 latent and 64 RoPE bf16 values are coded and written
// to pool row slots[i]; load is the reverse, a gather of rows back to bf16.
// Both are bound by HBM (1152 + 384 bytes per row; the arithmetic is ~20
// operations per value).  One warp per row: lane l codes channels 16l..16l+15
// -- one scale group, so the group's maximum needs no shuffle -- and lanes
// 0..3 code the RoPE groups (value and residual) as well.
#include "kv4.cuh"

namespace mlav {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack8(uint4 u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// Codes 16 values: two words; returns the exponent.  With `rest`, what the
// code leaves out replaces the values (exact in fp32: the code's value has at
// most two significant bits at or above the value's own).
__device__ __forceinline__ int encode16(float (&x)[16], uint32_t (&w)[2], bool rest) {
  float a = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) a = fmaxf(a, fabsf(x[k]));  // fmaxf drops NaN
  const int e = kv4_exponent_of(a);
  const float down = pow2f(-e), up = pow2f(e);
  w[0] = w[1] = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const uint32_t c = kv4_magnitude(fabsf(x[k]) * down);
    const uint32_t neg = (x[k] < 0.f && c) ? 1u : 0u;
    w[k >> 3] |= (c << (4 * (k & 7))) | (neg << kv4_sign_bit(k & 7));
    if (rest) x[k] -= kv4_value(c, neg, up);
  }
  return e;
}

__global__ void __launch_bounds__(kThreads) store_kernel(const __nv_bfloat16* latent, int64_t latent_stride,
                                                         const __nv_bfloat16* rope, int64_t rope_stride,
                                                         const int32_t* slots, int64_t n, uint8_t* pool,
                                                         int64_t pool_rows, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  if (i >= n) return;
  const int64_t slot = slots[i];
  if (slot < 0 || slot >= pool_rows) {
    if (slot != -1 && lane == 0) atomicOr(status, kStatusBadRow);
    return;
  }
  uint8_t* row = pool + slot * kKv4RowBytes;
  float x[16];
  const uint4* src = reinterpret_cast<const uint4*>(latent + i * latent_stride) + 2 * lane;
  unpack8(src[0], x);
  unpack8(src[1], x + 8);
  uint32_t w[2];
  int e = encode16(x, w, false);
  reinterpret_cast<uint2*>(row)[lane] = make_uint2(w[0], w[1]);
  row[kv4_scale_at(16 * lane)] = (uint8_t)(e + 127);
  if (lane < 4) {
    const uint4* rs = reinterpret_cast<const uint4*>(rope + i * rope_stride) + 2 * lane;
    unpack8(rs[0], x);
    unpack8(rs[1], x + 8);
    e = encode16(x, w, true);
    reinterpret_cast<uint2*>(row)[32 + lane] = make_uint2(w[0], w[1]);
    row[kv4_scale_at(512 + 16 * lane)] = (uint8_t)(e + 127);
    e = encode16(x, w, false);
    reinterpret_cast<uint2*>(row)[36 + lane] = make_uint2(w[0], w[1]);
    row[kv4_scale_at(576 + 16 * lane)] = (uint8_t)(e + 127);
  } else if (lane < 16) {  // the 24 bytes that hold no scale
    const int q = (lane - 4) / 3, k = (lane - 4) % 3;
    *reinterpret_cast<uint16_t*>(row + kKv4ScaleOff + 16 * q + 10 + 2 * k) = 0;
  }
}

__global__ void __launch_bounds__(kThreads) load_kernel(const uint8_t* pool, int64_t pool_rows, const int32_t* slots,
                                                        int64_t n, __nv_bfloat16* latent, int64_t latent_stride,
                                                        __nv_bfloat16* rope, int64_t rope_stride, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  if (i >= n) return;
  const int64_t slot = slots[i];
  const bool ok = slot >= 0 && slot < pool_rows;
  if (!ok && slot != -1 && lane == 0) atomicOr(status, kStatusBadRow);
  const uint8_t* row = pool + (ok ? slot : 0) * kKv4RowBytes;
  auto group = [&](int code, float (&f)[16]) {
    const uint2 w = ok ? reinterpret_cast<const uint2*>(row)[code / 16] : make_uint2(0, 0);
    const float s = ok ? pow2f(kv4_exponent(row[kv4_scale_at(code)])) : 1.f;
    float lo[8], hi[8];
    kv4_decode8(w.x, s, lo);
    kv4_decode8(w.y, s, hi);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[k] = lo[k];
      f[8 + k] = hi[k];
    }
  };
  auto put = [](__nv_bfloat16* dst, const float (&f)[16]) {
    uint32_t p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
      p[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(p[0], p[1], p[2], p[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(p[4], p[5], p[6], p[7]);
  };
  float f[16];
  group(16 * lane, f);
  put(latent + i * latent_stride + 16 * lane, f);
  if (lane < 4) {
    float r[16];
    group(512 + 16 * lane, f);
    group(576 + 16 * lane, r);
#pragma unroll
    for (int k = 0; k < 16; ++k) f[k] += r[k];
    put(rope + i * rope_stride + 16 * lane, f);
  }
}

}  // namespace

cudaError_t launch_store_kv4(const void* latent, int64_t latent_stride, const void* rope, int64_t rope_stride,
                             const int32_t* slots, int64_t n, void* pool, int64_t pool_rows, uint32_t* status,
                             cudaStream_t stream) {
  if (n <= 0) return cudaSuccess;
  const int64_t blocks = (n * 32 + kThreads - 1) / kThreads;
  store_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(latent), latent_stride, static_cast<const __nv_bfloat16*>(rope), rope_stride,
      slots, n, static_cast<uint8_t*>(pool), pool_rows, status);
  return cudaGetLastError();
}

cudaError_t launch_load_kv4(const void* pool, int64_t pool_rows, const int32_t* slots, int64_t n, void* latent,
                            int64_t latent_stride, void* rope, int64_t rope_stride, uint32_t* status,
                            cudaStream_t stream) {
  if (n <= 0) return cudaSuccess;
  const int64_t blocks = (n * 32 + kThreads - 1) / kThreads;
  load_kernel<<<(unsigned)blocks, kThreads, 0, stream>>>(
      static_cast<const uint8_t*>(pool), pool_rows, slots, n, static_cast<__nv_bfloat16*>(latent), latent_stride,
      static_cast<__nv_bfloat16*>(rope), rope_stride, status);
  return cudaGetLastError();
}

}  // namespace mlav
