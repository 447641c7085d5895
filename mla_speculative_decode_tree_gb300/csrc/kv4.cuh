// The 4-bit latent cache row and its arithmetic (device side).
//
// A row is 384 bytes: 640 codes of 4 bits in five blocks of 128 -- 512 latent
// channels, 64 RoPE channels, the 64 RoPE channels' residuals -- and one
// power-of-two scale per 16 codes.  A code is a sign and a magnitude of
// {0, 0.5, 1, 1.5, 2, 3, 4, 6} (the e2m1 numbers); the value is code * 2^e.
//
//   bytes 64m .. 64m+63   codes of block m, 8 channels per 32-bit word
//   byte  320+16q+2m+h    scale byte e + 127 of codes 128m + 32q + 16h .. +15
//                         (q = 0..3, m = 0..4, h = 0, 1; the other 24 bytes are 0)
//
// In a word of 8 channels the magnitude of channel i is bits 4i..4i+2, the
// signs of channels 0..3 are bits 7, 15, 23, 31 and those of channels 4..7
// bits 3, 11, 19, 27.  A byte permute indexed by the magnitudes of four
// channels then gives four 8-bit floats whose signs already sit in place (or
// one shift away): 7 instructions per 8 values, against 11 with the signs
// next to their magnitudes.  A thread that holds quarter q of every block
// reads all its scales with one 16-byte load.
//
// Scales are held in [-13, 13], so every value (1 or 2 significant bits times
// 2^e) is an exact, normal 8-bit e5m2 float as well as an exact bf16: the
// tensor cores take it without rounding.
//
// 16 codes per scale, not 32: a power of two alone wastes up to one bit of
// the 4-bit range, the smaller group wins half of it back, and 384 bytes are
// three whole 128-byte lines either way.  RoPE keys carry the positions and
// are the smaller part, so their residual is coded as well (about 6 bits);
// the residual multiplies the same query values, so to the score product it
// is 64 further channels.
#pragma once

#include "common.cuh"

namespace mlav {

constexpr int kKv4Blocks = 5;
constexpr int kKv4RowBytes = 384;
constexpr int kKv4ScaleOff = 320;
constexpr int kKv4EMin = -13, kKv4EMax = 13;

#if defined(__CUDACC__)

// Scale byte -> the exponent it stands for; a byte outside the format (a row
// that was never stored) is clamped, so no code decodes to infinity or NaN.
__device__ __forceinline__ int kv4_exponent(uint32_t byte) {
  int e = (int)byte - 127;
  e = e < kKv4EMin ? kKv4EMin : e;
  return e > kKv4EMax ? kKv4EMax : e;
}

__device__ __forceinline__ int kv4_scale_at(int code) {  // byte offset of the scale of a code index
  return kKv4ScaleOff + 16 * ((code & 127) >> 5) + 2 * (code >> 7) + ((code & 31) >> 4);
}

// Value of magnitude c (0..7) with 2^e: e2m1 c = (exponent c >> 1, mantissa
// c & 1), exponent 0 meaning 0 or one half.
__device__ __forceinline__ float kv4_value(uint32_t c, uint32_t neg, float scale) {
  const float mag = c < 2 ? 0.5f * (float)c : (1.0f + 0.5f * (float)(c & 1)) * (float)(1 << ((c >> 1) - 1));
  return (neg ? -mag : mag) * scale;
}

// The 8 channels of one word.
__device__ __forceinline__ void kv4_decode8(uint32_t w, float scale, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t neg = (w >> (i < 4 ? 8 * i + 7 : 8 * (i - 4) + 3)) & 1u;
    f[i] = kv4_value((w >> (4 * i)) & 7u, neg, scale);
  }
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Scale exponent of 16 values with largest magnitude a: the least e with
// a <= 6 * 2^e, held in the format's range (a beyond it saturates).  With
// a = m * 2^x, m in [1, 2): 6 * 2^e = 1.5 * 2^(e+2), so e = x - 2, or x - 1
// when m > 1.5.
__device__ __forceinline__ int kv4_exponent_of(float a) {
  const uint32_t bits = __float_as_uint(a);
  int e = (int)(bits >> 23) - 127 - 2 + ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  e = e < kKv4EMin ? kKv4EMin : e;
  return e > kKv4EMax ? kKv4EMax : e;
}

#endif  // __CUDACC__

cudaError_t launch_store_kv4(const void* latent, int64_t latent_stride, const void* rope, int64_t rope_stride,
                             const int32_t* slots, int64_t n, void* pool, int64_t pool_rows, uint32_t* status,
                             cudaStream_t stream);
cudaError_t launch_load_kv4(const void* pool, int64_t pool_rows, const int32_t* slots, int64_t n, void* latent,
                            int64_t latent_stride, void* rope, int64_t rope_stride, uint32_t* status,
                            cudaStream_t stream);

}  // namespace mlav
