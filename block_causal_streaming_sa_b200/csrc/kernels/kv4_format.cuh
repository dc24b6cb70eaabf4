// The 4-bit row format: e2m1 codes with one 8-bit scale per 16 values of D.
//
// A scale byte b is the fp16 with bits b << 7: five exponent bits and three
// fraction bits, so turning it into a number is one shift. A value is code * scale
// with 2 and 4 significant bits, at most 6: the fp16 product is exact as long as
// it stays in range, which scales up to 10240 (6 * 10240 = 61440) and down to
// 2^-17 (half of it is 2^-18, fp16 reaches 2^-24) guarantee. So products over
// dequantised K and V start from exactly the stored values.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../sa_internal.h"
#include "ptx.cuh"

namespace sa {

constexpr unsigned kMaxScaleByte = 226;   // 10240 = 1.25 * 2^13
constexpr float kMaxStored = 61440.0f;    // 6 * 10240

// Launches may begin while the kernel before them on the stream drains (the host asks
// for that): every kernel lets the next one begin early and waits, in every block,
// until the kernel before it has finished and its writes can be seen.
__device__ __forceinline__ void begin_early() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One cache as the kernels see it (include/sa.h: sa_kv4_cache).
struct Kv4 {
  int B, H, N;  // sequences, KV heads, capacity in rows
  uint8_t *k_codes, *v_codes, *k_scales, *v_scales;
  int32_t* pos;
  float* weight;
  int32_t* seq;      // [4][B]
  unsigned* status;  // status word, ticket of the append kernel
};

// seq rows.
constexpr int kSeqHeld = 0, kSeqTotal = 1, kSeqLast = 2, kSeqTail = 3;

struct Kv4Rows {
  void* data;
  long long sb, st, sh;
};

// Rows held by sequence b. seq is the caller's memory: whatever it holds, no row
// index leaves the planes.
__device__ __forceinline__ int rows_held(const Kv4& c, int b) {
  return min(max(c.seq[kSeqHeld * c.B + b], 0), c.N);
}

__device__ __forceinline__ int tokens_of(const int32_t* counts, int b, int T) {
  return counts == nullptr ? T : min(max(counts[b], 0), T);
}

// The scale byte of a block whose largest magnitude is amax (finite, <= 65504 is
// not required): the smallest scale >= amax / 6. The division is IEEE, so that
// amax = 6 s gives s itself: amax has at most 11 significant bits, so a quotient
// that is not a scale differs from every scale by more than its rounding.
__device__ __forceinline__ unsigned scale_byte(float amax) {
  const float u = __fdiv_rn(amax, 6.0f);
  if (!(u < 10240.0f)) return kMaxScaleByte;
  if (u < 6.103515625e-5f)  // below 2^-14: multiples of 2^-17
    return static_cast<unsigned>(ceilf(u * 131072.0f));
  // keep three fraction bits, rounding up; exponent bias 127 -> 15
  return ((__float_as_uint(u) + 0xFFFFFu) >> 20) - ((127u - 15u) << 3);
}

__device__ __forceinline__ float scale_value(unsigned byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// x * inv of a pair (inv = 1 / scale) moved to the nearest multiple of 2^-16: a quotient
// that equals a midpoint between two codes comes out as that midpoint whatever
// inv's rounding did (error < 2^-20), and no other quotient can reach it (x and
// midpoint * scale have at most 11 significant bits, so they differ by 2^-13 of
// the code range or more). Ties then go to the even code as in exact arithmetic.
__device__ __forceinline__ void snap2(float2& x, float inv) {
  ptx::ffma2(x.x, x.y, x.x, x.y, inv, inv, 192.0f, 192.0f);
  ptx::fadd2(x.x, x.y, x.x, x.y, -192.0f, -192.0f);
}

// Eight codes (e2m1, nearest even, saturating) of eight values into one word.
__device__ __forceinline__ uint32_t e2m1x8(float2 a, float2 b, float2 c, float2 d) {
  uint32_t w;
  asm("{\n\t.reg .b8 p, q, r, s;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n\t"
      "mov.b32 %0, {p, q, r, s};\n\t}"
      : "=r"(w)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return w;
}

// The eight codes of one word as four fp16 pairs, unscaled.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// A scale byte as an fp16 pair, and two as the halves of one (multiplications: the
// pipe that shifts and selects is the one the conversions load).
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t byte) { return byte * 0x00800080u; }
__device__ __forceinline__ uint32_t scales_f16x2(uint32_t lo, uint32_t hi) {
  return hi * 0x00800000u + lo * 0x80u;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A pair of stored 16-bit input values as floats, and back (dtype: SA_DTYPE_*).
template <int kDtype>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (kDtype == SA_DTYPE_FP16) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  } else {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
}

template <int kDtype>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (kDtype == SA_DTYPE_FP16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace sa
