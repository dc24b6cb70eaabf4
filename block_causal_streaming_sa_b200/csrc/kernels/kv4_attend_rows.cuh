// Attention over a 4-bit cache, one warp per query row: a plain form that is right
// for every size. Scores take a key row per lane, outputs D / 32 values per lane.
#pragma once

#include "kv4_params.cuh"

namespace sa {

template <int D, int kDtype>
__global__ void __launch_bounds__(128) kv4_attend_rows_kernel(
    const __grid_constant__ Kv4AttendParams p) {
  const Kv4& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, hq = blockIdx.y, h = hq / p.group;
  const int t = blockIdx.x * 4 + warp;
  const int held = rows_held(c, b), n_tok = tokens_of(p.counts, b, p.T);
  __shared__ float sq[4][D];
  if (t >= n_tok) return;
  if (p.causal && n_tok > 1 && n_tok > c.seq[kSeqTail * c.B + b] && lane == 0)
    atomicOr(c.status, kDevErrOrder);
  const uint16_t* qr =
      static_cast<const uint16_t*>(p.q.data) + b * p.q.sb + t * p.q.st + hq * p.q.sh;
  for (int d = 2 * lane; d < D; d += 64) {
    const float2 v = unpack2<kDtype>(*reinterpret_cast<const uint32_t*>(qr + d));
    sq[warp][d] = v.x;
    sq[warp][d + 1] = v.y;
  }
  __syncwarp();
  const size_t plane = (static_cast<size_t>(b) * c.H + h) * c.N;
  const int n = rows_seen(p, held, n_tok, t);
  float m = -INFINITY, l = 0.f;
  float o[D / 32];
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    if (j < n) {
      s = 0.f;
      for (int blk = 0; blk < D / 16; ++blk) {
        const uint2 w = *(reinterpret_cast<const uint2*>(c.k_codes + (plane + j) * (D / 2)) + blk);
        const float sc = scale_value(c.k_scales[(plane + j) * (D / 16) + blk]);
        uint32_t f[8], g[4];
        codes_to_f16(w.x, g);
        for (int i = 0; i < 4; ++i) f[i] = g[i];
        codes_to_f16(w.y, g);
        for (int i = 0; i < 4; ++i) f[4 + i] = g[i];
        for (int i = 0; i < 8; ++i) {
          const float2 v = unpack2<SA_DTYPE_FP16>(f[i]);
          s = fmaf(v.x * sc, sq[warp][blk * 16 + 2 * i], s);
          s = fmaf(v.y * sc, sq[warp][blk * 16 + 2 * i + 1], s);
        }
      }
      s *= p.scale_log2;
    }
    float mx = s;
    for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, k));
    const float mn = fmaxf(m, mx);
    const float a = exp2f(m - mn);
    const float pr = j < n ? exp2f(s - mn) : 0.f;
    m = mn;
    l = l * a + pr;
    for (int i = 0; i < D / 32; ++i) o[i] *= a;
    const int cnt = min(32, n - j0);
    for (int k = 0; k < cnt; ++k) {
      const float pk = __shfl_sync(~0u, pr, k);
      const size_t row = plane + j0 + k;
      for (int i = 0; i < D / 64; ++i) {
        const int d = i * 64 + 2 * lane;
        const unsigned byte = c.v_codes[row * (D / 2) + d / 2];
        const float sc = scale_value(c.v_scales[row * (D / 16) + d / 16]);
        uint32_t g[4];
        codes_to_f16(byte * 0x01010101u, g);
        const float2 v = unpack2<SA_DTYPE_FP16>(g[0]);
        o[2 * i] = fmaf(pk, v.x * sc, o[2 * i]);
        o[2 * i + 1] = fmaf(pk, v.y * sc, o[2 * i + 1]);
      }
    }
  }
  for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(~0u, l, k);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t* orow = static_cast<uint16_t*>(p.o.data) + b * p.o.sb + t * p.o.st + hq * p.o.sh;
  for (int i = 0; i < D / 64; ++i)
    *reinterpret_cast<uint32_t*>(orow + i * 64 + 2 * lane) =
        pack2<kDtype>(o[2 * i] * inv, o[2 * i + 1] * inv);
  if (lane == 0) {
    const size_t at = (static_cast<size_t>(b) * p.heads + hq) * p.T + t;
    const float l2 = l > 0.f ? m + log2f(l) : -INFINITY;
    if (p.lse != nullptr) p.lse[at] = l2 * 0.69314718055994531f;
    p.scores[at] = l2;
  }
}

// weight[j] += the probabilities of row j: a thread per row, queries in order.
template <int D, int kDtype>
__global__ void __launch_bounds__(128) kv4_weight_rows_kernel(
    const __grid_constant__ Kv4AttendParams p) {
  const Kv4& c = p.c;
  const int b = blockIdx.z, h = blockIdx.y;
  const int held = rows_held(c, b), n_tok = tokens_of(p.counts, b, p.T);
  const int j = blockIdx.x * 128 + threadIdx.x;
  if (j >= held) return;
  const size_t row = (static_cast<size_t>(b) * c.H + h) * c.N + j;
  float k[D];
  for (int blk = 0; blk < D / 16; ++blk) {
    const uint2 w = *(reinterpret_cast<const uint2*>(c.k_codes + row * (D / 2)) + blk);
    const float sc = scale_value(c.k_scales[row * (D / 16) + blk]);
    uint32_t f[4];
    codes_to_f16(w.x, f);
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2<SA_DTYPE_FP16>(f[i]);
      k[blk * 16 + 2 * i] = v.x * sc;
      k[blk * 16 + 2 * i + 1] = v.y * sc;
    }
    codes_to_f16(w.y, f);
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2<SA_DTYPE_FP16>(f[i]);
      k[blk * 16 + 8 + 2 * i] = v.x * sc;
      k[blk * 16 + 8 + 2 * i + 1] = v.y * sc;
    }
  }
  float sum = 0.f;
  for (int g = 0; g < p.group; ++g) {
    const int hq = h * p.group + g;
    for (int t = 0; t < n_tok; ++t) {
      if (j >= rows_seen(p, held, n_tok, t)) continue;
      const uint16_t* qr =
          static_cast<const uint16_t*>(p.q.data) + b * p.q.sb + t * p.q.st + hq * p.q.sh;
      float s = 0.f;
#pragma unroll
      for (int d = 0; d < D; d += 2) {
        const float2 v = unpack2<kDtype>(__ldg(reinterpret_cast<const uint32_t*>(qr + d)));
        s = fmaf(v.x, k[d], s);
        s = fmaf(v.y, k[d + 1], s);
      }
      const float l2 = p.scores[(static_cast<size_t>(b) * p.heads + hq) * p.T + t];
      sum += exp2f(s * p.scale_log2 - l2);
    }
  }
  c.weight[row] += sum;
}

}  // namespace sa
