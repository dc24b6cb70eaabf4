// Weights drawn by many query rows: a thread per cache row, queries in order.
#pragma once

#include "kv4_params.cuh"

namespace sa {

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
      const float l2 = p.row_lse[((static_cast<size_t>(b) * c.H + h) * p.q_tiles) * 128 +
                               t * p.group + g];
      sum += exp2f(s * p.scale_log2 - l2);
    }
  }
  c.weight[row] += sum;
}

}  // namespace sa
