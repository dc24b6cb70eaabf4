// Appending rows to a 4-bit cache (quantisation) and reading them back.
//
// Append reads 4 D bytes a row and head and writes D + D / 8 + 8, read the reverse: HBM is
// their floor (10800 rows x 12 heads, D 128, 86 MB: 13 us). Read takes 18 us (4.8 TB/s), append
// 24 (3.6 TB/s): it has the conversion to codes, and a fence and a counter at each block's end,
// on top. A thread owns one block of 16 values of K and
// the same block of V: two 16-byte loads each, one 8-byte and one 1-byte store.
// The threads of a warp cover consecutive blocks of consecutive tokens of one
// head, so loads are whole lines of the input rows and the stores of a head's
// tokens are contiguous in its plane.
#pragma once

#include "kv4_format.cuh"

namespace sa {

struct Kv4AppendParams {
  Kv4 c;
  Kv4Rows k, v;
  const int32_t* counts;
  int T, replace;
};

// Largest magnitude of both halves of two words; NaN if any is.
template <int kDtype>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (kDtype == SA_DTYPE_FP16)
    asm("{\n\t.reg .b32 x, y;\n\tabs.f16x2 x, %1;\n\tabs.f16x2 y, %2;\n\t"
        "max.NaN.f16x2 %0, x, y;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
  else
    asm("{\n\t.reg .b32 x, y;\n\tabs.bf16x2 x, %1;\n\tabs.bf16x2 y, %2;\n\t"
        "max.NaN.bf16x2 %0, x, y;\n\t}"
        : "=r"(r)
        : "r"(a), "r"(b));
  return r;
}

template <int kDtype>
__device__ __forceinline__ void quantise_block(const uint4 (&in)[2], uint2* codes, uint8_t* scale,
                                               bool& bad) {
  const uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
  // the maximum on packed pairs, two words an instruction
  uint32_t m = max_abs2<kDtype>(w[0], w[1]);
#pragma unroll
  for (int i = 2; i < 8; i += 2)
    m = max_abs2<kDtype>(m, max_abs2<kDtype>(w[i], w[i + 1]));
  const float2 m2 = unpack2<kDtype>(max_abs2<kDtype>(m, (m >> 16) | (m << 16)));
  float amax = m2.x;
  float2 x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = unpack2<kDtype>(w[i]);
  if (!(amax <= kMaxStored)) {  // some value is not finite or beyond the largest stored one
    bad = true;
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // clamps infinities; fminf / fmaxf turn a NaN into the bound
      x[i].x = fmaxf(fminf(x[i].x, kMaxStored), -kMaxStored);
      x[i].y = fmaxf(fminf(x[i].y, kMaxStored), -kMaxStored);
      amax = fmaxf(amax, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
    }
  }
  const unsigned byte = scale_byte(amax);
  const float inv = byte != 0 ? __fdiv_rn(1.0f, scale_value(byte)) : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) snap2(x[i], inv);
  *codes = make_uint2(e2m1x8(x[0], x[1], x[2], x[3]), e2m1x8(x[4], x[5], x[6], x[7]));
  *scale = static_cast<uint8_t>(byte);
}

// grid: (ceil(T * D / 16 / 256), H, B). The last block to finish moves seq on;
// every block has read it by then.
template <int D, int kDtype>
__global__ void __launch_bounds__(256)
    kv4_append_kernel(const __grid_constant__ Kv4AppendParams p) {
  constexpr int NB = D / 16;
  const Kv4& c = p.c;
  const int b = blockIdx.z, h = blockIdx.y;
  begin_early();
  wait_for_previous();
  const int held = rows_held(c, b);
  const int last = p.replace ? min(max(c.seq[kSeqLast * c.B + b], 0), held) : 0;
  const int base = held - last;
  const int total = c.seq[kSeqTotal * c.B + b] - last;
  const int n = min(tokens_of(p.counts, b, p.T), c.N - base);
  const long long item = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const int t = static_cast<int>(item / NB), blk = static_cast<int>(item % NB);
  bool bad = false;
  if (t < n) {
    uint4 kin[2], vin[2];
    const uint16_t* ks = static_cast<const uint16_t*>(p.k.data) + b * p.k.sb + t * p.k.st +
                         h * p.k.sh + blk * 16;
    const uint16_t* vs = static_cast<const uint16_t*>(p.v.data) + b * p.v.sb + t * p.v.st +
                         h * p.v.sh + blk * 16;
    kin[0] = __ldcg(reinterpret_cast<const uint4*>(ks));
    kin[1] = __ldcg(reinterpret_cast<const uint4*>(ks) + 1);
    vin[0] = __ldcg(reinterpret_cast<const uint4*>(vs));
    vin[1] = __ldcg(reinterpret_cast<const uint4*>(vs) + 1);
    const size_t row = (static_cast<size_t>(b) * c.H + h) * c.N + base + t;
    quantise_block<kDtype>(kin, reinterpret_cast<uint2*>(c.k_codes + row * (D / 2)) + blk,
                           c.k_scales + row * NB + blk, bad);
    quantise_block<kDtype>(vin, reinterpret_cast<uint2*>(c.v_codes + row * (D / 2)) + blk,
                           c.v_scales + row * NB + blk, bad);
    if (blk == 0) {
      c.pos[row] = total + t;
      c.weight[row] = 0.f;
    }
  }
  if (bad) atomicOr(c.status, kDevWarnSaturated);
  __shared__ bool s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    const unsigned all = gridDim.x * gridDim.y * gridDim.z;
    s_last = atomicAdd(c.status + 1, 1u) == all - 1;
  }
  __syncthreads();
  if (!s_last) return;
  for (int i = threadIdx.x; i < c.B; i += 256) {
    const int hi = rows_held(c, i);
    const int li = p.replace ? min(max(c.seq[kSeqLast * c.B + i], 0), hi) : 0;
    const int want = tokens_of(p.counts, i, p.T);
    const int got = min(want, c.N - (hi - li));
    if (got < want) atomicOr(c.status, kDevErrFull);
    c.seq[kSeqHeld * c.B + i] = hi - li + got;
    c.seq[kSeqTotal * c.B + i] += got - li;
    c.seq[kSeqLast * c.B + i] = got;
    c.seq[kSeqTail * c.B + i] += got - li;
  }
  if (threadIdx.x == 0) c.status[1] = 0;  // ready for the next launch
}

struct Kv4ReadParams {
  Kv4 c;
  Kv4Rows k, v;
  int first, T;  // first = SA_KV4_LAST: the rows of the last append
};

template <int kDtype>
__device__ __forceinline__ void dequantise_block(uint2 codes, unsigned scale, uint4* out) {
  const uint32_t s = scale_f16x2(scale);
  uint32_t h[8];
  uint32_t a[4];
  codes_to_f16(codes.x, a);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = mul_f16x2(a[i], s);
  codes_to_f16(codes.y, a);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[4 + i] = mul_f16x2(a[i], s);
  if constexpr (kDtype == SA_DTYPE_BF16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = unpack2<SA_DTYPE_FP16>(h[i]);
      h[i] = pack2<SA_DTYPE_BF16>(f.x, f.y);
    }
  }
  out[0] = make_uint4(h[0], h[1], h[2], h[3]);
  out[1] = make_uint4(h[4], h[5], h[6], h[7]);
}

template <int D, int kDtype>
__global__ void __launch_bounds__(256) kv4_read_kernel(const __grid_constant__ Kv4ReadParams p) {
  constexpr int NB = D / 16;
  const Kv4& c = p.c;
  const int b = blockIdx.z, h = blockIdx.y;
  begin_early();
  wait_for_previous();
  const int held = rows_held(c, b);
  int base = p.first, n = p.T;
  if (p.first < 0) {
    const int last = min(max(c.seq[kSeqLast * c.B + b], 0), held);
    base = held - last;
    n = min(n, last);
  }
  const long long item = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const int t = static_cast<int>(item / NB), blk = static_cast<int>(item % NB);
  if (t >= n || t >= held - base) return;
  const size_t row = (static_cast<size_t>(b) * c.H + h) * c.N + base + t;
  const uint2 kc = reinterpret_cast<const uint2*>(c.k_codes + row * (D / 2))[blk];
  const uint2 vc = reinterpret_cast<const uint2*>(c.v_codes + row * (D / 2))[blk];
  const unsigned ks = c.k_scales[row * NB + blk], vs = c.v_scales[row * NB + blk];
  dequantise_block<kDtype>(
      kc, ks,
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.k.data) + b * p.k.sb + t * p.k.st +
                               h * p.k.sh + blk * 16));
  dequantise_block<kDtype>(
      vc, vs,
      reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.v.data) + b * p.v.sb + t * p.v.st +
                               h * p.v.sh + blk * 16));
}

}  // namespace sa
