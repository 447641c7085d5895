// Store and load of 4-bit cache rows (format: kv4.cuh).
//
// Store: token i's 512 latent and 64 RoPE bf16 values are coded and written
// to pool row slots[i]; load is the reverse, a gather of rows back to bf16.
// Both are bound by HBM: 1152 bytes of bf16 and 384 of codes per row.
//
// A lane takes one group of 16 latent channels of a row: 32 bytes of bf16 in
// one 256-bit access, so a warp moves a whole row of latents and the group's
// maximum needs no shuffle.  The RoPE channels are only four groups, so with
// many rows a warp takes four rows and codes their RoPE parts together, a group
// per lane; with few it takes one, and more SMs share the work (see many()).
// 65,536 rows (GB300): store 23.2 us (4.35 TB/s), load 17.9 us (5.6 TB/s); a
// plain copy of as many bytes takes 15.  What the store has beside its traffic
// is coding: its ALU pipe is 68 % busy.
//
// Coding a group: the largest magnitude by 16-bit integer maxima (bf16
// magnitudes order as integers), the exponent from its bits, then the
// hardware's conversion to e2m1 -- which rounds to nearest, ties to the even
// code, and stops at 6, the format's own rule -- and a few bit moves that put
// the signs where the expansion of kv4.cuh wants them.  Decoding: two byte
// permutes give the high and low bytes of four bf16 values.
#include "kv4.cuh"

namespace mlav {
namespace {

// Warps need no company: small blocks leave a finer tail (32,768 rows stored and read back at 256 / 128 / 64 / 32 threads: store
// 22.0 / 21.3 / 20.9 / 20.9 us).
constexpr int kThreads = 64;
constexpr int kManyRows = 4;  // rows per warp when there are enough

struct Vec32 {
  uint32_t w[8];
};
// 32 bytes, 32-byte aligned (wide) or 16-byte aligned.
__device__ __forceinline__ Vec32 load32(const void* p, bool wide) {
  Vec32 v;
  if (wide) {
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]),
                   "=r"(v.w[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldg(static_cast<const uint4*>(p)), b = __ldg(static_cast<const uint4*>(p) + 1);
    v = {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  }
  return v;
}
__device__ __forceinline__ void store32(void* p, const Vec32& v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]),
                 "r"(v.w[3]), "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v.w[4], v.w[5], v.w[6], v.w[7]);
  }
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Four values to e2m1, the first in the low nibble of the low half.
__device__ __forceinline__ uint32_t cvt_e2m1x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b8 lo, hi, z;\n\tcvt.rn.satfinite.e2m1x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi, lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r & 0xFFFFu;
}

// Eight e2m1 nibbles in channel order -> the row's word: magnitudes stay, the
// sign of channel i moves to its place, that of a zero is dropped.
__device__ __forceinline__ uint32_t place_signs(uint32_t n) {
  const uint32_t mag = n & 0x77777777u;
  const uint32_t sign = n & (mag + 0x77777777u) & 0x88888888u;  // bit 3 of a sum: the magnitude is not 0
  // nibble k of a half -> bit 3 of byte k
  auto spread = [](uint32_t t) {
    t = (t | (t << 8)) & 0x00880088u;
    return (t | (t << 4)) & 0x08080808u;
  };
  return mag | (spread(sign & 0xFFFFu) << 4) | spread(sign >> 16);
}

// The group's exponent from its largest bf16 magnitude (a NaN counts as none).
__device__ __forceinline__ int exponent_of_bits(uint32_t mag16) { return kv4_exponent_of(__uint_as_float(mag16 << 16)); }

// Codes the 16 values of v; returns the exponent.
__device__ __forceinline__ int encode16(const Vec32& v, uint32_t (&w)[2]) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max_u16x2(top, v.w[k] & 0x7FFF7FFFu);
  uint32_t m = max(top & 0xFFFFu, top >> 16);
  Vec32 x = v;
  if (m > 0x7F80u) {  // a NaN: 0 in its place
    m = 0;
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
      if ((x.w[k] & 0x7FFFu) > 0x7F80u) x.w[k] &= 0xFFFF0000u;
      if ((x.w[k] & 0x7FFF0000u) > 0x7F800000u) x.w[k] &= 0xFFFFu;
      m = max(m, max(x.w[k] & 0x7FFFu, (x.w[k] >> 16) & 0x7FFFu));
    }
  }
  const int e = exponent_of_bits(m);
  const float down = pow2f(-e);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t n[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t a = x.w[4 * h + 2 * i], b = x.w[4 * h + 2 * i + 1];
      n[i] = cvt_e2m1x4(__uint_as_float(a << 16) * down, __uint_as_float(a & 0xFFFF0000u) * down,
                        __uint_as_float(b << 16) * down, __uint_as_float(b & 0xFFFF0000u) * down);
    }
    w[h] = place_signs(n[0] | (n[1] << 16));
  }
  return e;
}

// 16 codes (two words) with 2^e -> 16 bf16 values.  The eight magnitudes as
// bf16 are 0 and base[c] + (e << 7); their high and low bytes make two permute tables.
__device__ __forceinline__ Vec32 decode16(uint2 codes, int e) {
  const uint32_t add = (uint32_t)e << 7;
  const uint32_t t01 = (0x3F00u + add) << 16;                                         // 0, 0.5
  const uint32_t add2 = (add & 0xFFFFu) * 0x10001u;
  const uint32_t t23 = __vadd2(0x3FC03F80u, add2), t45 = __vadd2(0x40404000u, add2), t67 = __vadd2(0x40C04080u, add2);
  const uint32_t hi0 = __byte_perm(t01, t23, 0x7531), hi1 = __byte_perm(t45, t67, 0x7531);
  const uint32_t lo0 = __byte_perm(t01, t23, 0x6420), lo1 = __byte_perm(t45, t67, 0x6420);
  Vec32 v;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w = h ? codes.y : codes.x;
    const uint32_t sel = w & 0x77777777u;
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // channels 4k .. 4k+3 of the word
      const uint32_t s4 = k ? sel >> 16 : sel;
      const uint32_t sign = (k ? w << 4 : w) & 0x80808080u;
      const uint32_t hi = __byte_perm(hi0, hi1, s4) | sign, lo = __byte_perm(lo0, lo1, s4);
      v.w[4 * h + 2 * k] = __byte_perm(lo, hi, 0x5140);
      v.w[4 * h + 2 * k + 1] = __byte_perm(lo, hi, 0x7362);
    }
  }
  return v;
}

// RoPE: codes 16 values and then what the code leaves out of them (exact in
// fp32: the code's value is one or two bits at or above the value's own).
__device__ __forceinline__ void encode16_twice(const Vec32& v, uint32_t (&w)[2], int& e, uint32_t (&rw)[2], int& re) {
  e = encode16(v, w);
  const Vec32 coded = decode16(make_uint2(w[0], w[1]), e);
  float x[16], a = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[2 * k] = __uint_as_float(v.w[k] << 16) - __uint_as_float(coded.w[k] << 16);
    x[2 * k + 1] = __uint_as_float(v.w[k] & 0xFFFF0000u) - __uint_as_float(coded.w[k] & 0xFFFF0000u);
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    x[k] = x[k] == x[k] ? x[k] : 0.f;  // a NaN was coded as 0
    a = fmaxf(a, fabsf(x[k]));
  }
  re = kv4_exponent_of(a);
  const float down = pow2f(-re);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* y = x + 8 * h;
    rw[h] = place_signs(cvt_e2m1x4(y[0] * down, y[1] * down, y[2] * down, y[3] * down) |
                        (cvt_e2m1x4(y[4] * down, y[5] * down, y[6] * down, y[7] * down) << 16));
  }
}

// The pool row a warp's r-th token names, or -1 (also for a slot outside the
// pool other than -1, which raises the status bit).
template <int R>
__device__ __forceinline__ int32_t own_slot(const int32_t* slots, int64_t i0, int64_t n, int64_t pool_rows, int lane,
                                            uint32_t* status) {
  int32_t s = -1;
  if (lane < R && i0 + lane < n) {
    s = __ldg(slots + i0 + lane);
    if (s != -1 && (s < 0 || s >= pool_rows)) {
      atomicOr(status, kStatusBadRow);
      s = -1;
    }
  }
  return s;
}

// R rows per warp.
template <int R>
__global__ void __launch_bounds__(kThreads) store_kernel(const __nv_bfloat16* latent, int64_t latent_stride,
                                                         const __nv_bfloat16* rope, int64_t rope_stride,
                                                         const int32_t* slots, int64_t n, uint8_t* pool,
                                                         int64_t pool_rows, bool wide, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t i0 = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) * R;
  if (i0 >= n) return;
  Vec32 x[R], xr = {};
  const int rr = lane >> 2;  // RoPE: row of this lane's group
  if (rr < R && i0 + rr < n) xr = load32(rope + (i0 + rr) * rope_stride + 16 * (lane & 3), wide);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    x[r] = {};
    if (i0 + r < n) x[r] = load32(latent + (i0 + r) * latent_stride + 16 * lane, wide);
  }
  const int32_t own = own_slot<R>(slots, i0, n, pool_rows, lane, status);
  uint32_t w[2], rw[2];
  int e, re;
  encode16_twice(xr, w, e, rw, re);
  {
    // Lane (row rr, group g) writes its two groups' codes and bytes 8..15 of scale
    // slot q = g: the scales of RoPE groups 2q, 2q+1 (q < 2) or of residual groups
    // 2q-4, 2q-3, and the six unused bytes.
    const int g = lane & 3;
    const uint32_t own_scales = (uint32_t)(e + 127) | ((uint32_t)(re + 127) << 16);
    const uint32_t s0 = __shfl_sync(0xffffffffu, own_scales, (lane & ~3) | ((2 * g) & 3));
    const uint32_t s1 = __shfl_sync(0xffffffffu, own_scales, (lane & ~3) | ((2 * g + 1) & 3));
    const int32_t slot = __shfl_sync(0xffffffffu, own, rr < R ? rr : 0);
    if (rr < R && slot >= 0) {
      uint2* row = reinterpret_cast<uint2*>(pool + (int64_t)slot * kKv4RowBytes);
      row[32 + g] = make_uint2(w[0], w[1]);
      row[36 + g] = make_uint2(rw[0], rw[1]);
      const uint32_t shift = g < 2 ? 0 : 16;
      row[kKv4ScaleOff / 8 + 2 * g + 1] = make_uint2(((s0 >> shift) & 0xFFu) | (((s1 >> shift) & 0xFFu) << 8), 0u);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int32_t slot = __shfl_sync(0xffffffffu, own, r);
    e = encode16(x[r], w);
    if (slot >= 0) {
      uint8_t* row = pool + (int64_t)slot * kKv4RowBytes;
      reinterpret_cast<uint2*>(row)[lane] = make_uint2(w[0], w[1]);
      row[kv4_scale_at(16 * lane)] = (uint8_t)(e + 127);
    }
  }
}

template <int R>
__global__ void __launch_bounds__(kThreads) load_kernel(const uint8_t* pool, int64_t pool_rows, const int32_t* slots,
                                                        int64_t n, __nv_bfloat16* latent, int64_t latent_stride,
                                                        __nv_bfloat16* rope, int64_t rope_stride, bool wide,
                                                        uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t i0 = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) * R;
  if (i0 >= n) return;
  const int32_t own = own_slot<R>(slots, i0, n, pool_rows, lane, status);
  uint2 code[R], rc[2];
  uint32_t scale[R], rs[2];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int32_t slot = __shfl_sync(0xffffffffu, own, r);
    code[r] = make_uint2(0, 0);
    scale[r] = 127;
    if (slot >= 0) {
      const uint8_t* row = pool + (int64_t)slot * kKv4RowBytes;
      code[r] = __ldg(reinterpret_cast<const uint2*>(row) + lane);
      scale[r] = __ldg(row + kv4_scale_at(16 * lane));
    }
  }
  const int rr = lane >> 2;  // RoPE: row of this lane's group
  {
    const int32_t slot = __shfl_sync(0xffffffffu, own, rr < R ? rr : 0);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      rc[k] = make_uint2(0, 0);
      rs[k] = 127;
      if (rr < R && slot >= 0) {
        const uint8_t* row = pool + (int64_t)slot * kKv4RowBytes;
        rc[k] = __ldg(reinterpret_cast<const uint2*>(row) + 32 + 4 * k + (lane & 3));
        rs[k] = __ldg(row + kv4_scale_at(512 + 64 * k + 16 * (lane & 3)));
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (i0 + r < n)
      store32(latent + (i0 + r) * latent_stride + 16 * lane, decode16(code[r], kv4_exponent(scale[r])), wide);
  if (rr < R && i0 + rr < n) {
    const Vec32 a = decode16(rc[0], kv4_exponent(rs[0])), b = decode16(rc[1], kv4_exponent(rs[1]));
    Vec32 s;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const __nv_bfloat162 h =
          __floats2bfloat162_rn(__uint_as_float(a.w[k] << 16) + __uint_as_float(b.w[k] << 16),
                                __uint_as_float(a.w[k] & 0xFFFF0000u) + __uint_as_float(b.w[k] & 0xFFFF0000u));
      s.w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    store32(rope + (i0 + rr) * rope_stride + 16 * (lane & 3), s, wide);
  }
}

bool is_wide(const void* a, int64_t a_stride, const void* b, int64_t b_stride) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | (uint64_t)(2 * a_stride) |
           (uint64_t)(2 * b_stride)) & 31) == 0;
}

// Four rows per warp from 2048 rows on (GB300, us per call, one against four
// rows: store of 1000 rows 2.3 / 3.0, 4000 4.4 / 3.1, 65536 43.8 / 24.3; load
// 2.0 / 2.5, 2.9 / 2.6, 24.0 / 18.4).  Eight are within 5 % of four.
bool many(int64_t n) { return n >= 2048; }

unsigned blocks_for(int64_t n, int rows) {
  const int64_t warps = (n + rows - 1) / rows;
  return (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
}

}  // namespace

cudaError_t launch_store_kv4(const void* latent, int64_t latent_stride, const void* rope, int64_t rope_stride,
                             const int32_t* slots, int64_t n, void* pool, int64_t pool_rows, uint32_t* status,
                             cudaStream_t stream) {
  if (n <= 0) return cudaSuccess;
  const bool wide = is_wide(latent, latent_stride, rope, rope_stride);
  const int rows = many(n) ? kManyRows : 1;
  auto kernel = rows == 1 ? store_kernel<1> : store_kernel<kManyRows>;
  kernel<<<blocks_for(n, rows), kThreads, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(latent), latent_stride, static_cast<const __nv_bfloat16*>(rope), rope_stride,
      slots, n, static_cast<uint8_t*>(pool), pool_rows, wide, status);
  return cudaGetLastError();
}

cudaError_t launch_load_kv4(const void* pool, int64_t pool_rows, const int32_t* slots, int64_t n, void* latent,
                            int64_t latent_stride, void* rope, int64_t rope_stride, uint32_t* status,
                            cudaStream_t stream) {
  if (n <= 0) return cudaSuccess;
  const bool wide = is_wide(latent, latent_stride, rope, rope_stride);
  const int rows = many(n) ? kManyRows : 1;
  auto kernel = rows == 1 ? load_kernel<1> : load_kernel<kManyRows>;
  kernel<<<blocks_for(n, rows), kThreads, 0, stream>>>(
      static_cast<const uint8_t*>(pool), pool_rows, slots, n, static_cast<__nv_bfloat16*>(latent), latent_stride,
      static_cast<__nv_bfloat16*>(rope), rope_stride, wide, status);
  return cudaGetLastError();
}

}  // namespace mlav
