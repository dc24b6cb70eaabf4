// Eviction from a 4-bit cache by accumulated attention weight.
//
// Per (sequence, KV head) with more than `keep` rows: the keep-th largest key is
// found by radix selection over 32-bit ordered keys (four passes of eight bits,
// histogram in shared memory), then one ordered pass numbers the evicted rows
// below `keep` (holes) and the kept rows from `keep` on (movers); hole j takes
// mover j. Only rows that have to move do: one per evicted row at most, instead
// of a shift of everything behind the first evicted row. Writes go below `keep`,
// reads come from `keep` on, so the moves need no order among themselves.
#pragma once

#include "kv4_format.cuh"

namespace sa {

struct Kv4EvictParams {
  Kv4 c;
  int keep, first, recent;
  int32_t* n_moves;  // [B][H]
  int32_t* lists;    // [B][H][N]: holes from the front, movers from N / 2
};

// Order of a row among its head's: protected rows above every weight, NaN below,
// equal numbers (both zeros among them) equal.
__device__ __forceinline__ unsigned evict_key(float w, int pos, int first, int keep_from) {
  if (pos < first || pos >= keep_from) return 0xFFFFFFFFu;
  if (isnan(w)) return 0u;
  const unsigned u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(1024) kv4_evict_select_kernel(
    const __grid_constant__ Kv4EvictParams p) {
  const Kv4& c = p.c;
  const int h = blockIdx.x, b = blockIdx.y;
  const int n = rows_held(c, b);
  const size_t plane = (static_cast<size_t>(b) * c.H + h) * c.N;
  int32_t* n_moves = p.n_moves + static_cast<size_t>(b) * c.H + h;
  if (n <= p.keep) {
    if (threadIdx.x == 0) *n_moves = 0;
    return;
  }
  const int keep_from = c.seq[kSeqTotal * c.B + b] - p.recent;
  auto key_of = [&](int j) {
    return evict_key(c.weight[plane + j], c.pos[plane + j], p.first, keep_from);
  };
  __shared__ int hist[256];
  __shared__ unsigned s_prefix;
  __shared__ int s_left;
  unsigned prefix = 0;
  int left = p.keep;  // rows still to be found among those that match the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += 1024) hist[i] = 0;
    __syncthreads();
    const unsigned mask = shift == 24 ? 0u : ~0u << (shift + 8);
    for (int j = threadIdx.x; j < n; j += 1024) {
      const unsigned k = key_of(j);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int l = left, i = 255;
      while (l > hist[i]) l -= hist[i--];
      s_prefix = prefix | (static_cast<unsigned>(i) << shift);
      s_left = l;
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
    __syncthreads();
  }
  // prefix: the keep-th largest key; the first `left` rows that equal it stay
  __shared__ int warp_sum[3][32];
  int base_eq = 0, base_hole = 0, base_move = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t* holes = p.lists + plane;
  int32_t* movers = holes + c.N / 2;
  auto block_scan = [&](int which, bool flag, int& total) {
    const unsigned bal = __ballot_sync(~0u, flag);
    if (lane == 0) warp_sum[which][warp] = __popc(bal);
    __syncthreads();
    int before = 0;
    total = 0;
    for (int i = 0; i < 32; ++i) {
      const int v = warp_sum[which][i];
      if (i < warp) before += v;
      total += v;
    }
    __syncthreads();
    return before + __popc(bal & ((1u << lane) - 1));
  };
  for (int j0 = 0; j0 < n; j0 += 1024) {
    const int j = j0 + threadIdx.x;
    const unsigned k = j < n ? key_of(j) : 0u;
    const bool eq = j < n && k == prefix;
    int total;
    const int rank = base_eq + block_scan(0, eq, total);
    base_eq += total;
    const bool kept = j < n && (k > prefix || (eq && rank < left));
    const bool hole = j < p.keep && !kept, mover = j >= p.keep && kept;
    const int at_h = base_hole + block_scan(1, hole, total);
    base_hole += total;
    const int at_m = base_move + block_scan(2, mover, total);
    base_move += total;
    if (hole) holes[at_h] = j;
    if (mover) movers[at_m] = j;
  }
  if (threadIdx.x == 0) *n_moves = base_move;
}

// One row per 16 lanes: 16-byte pieces of codes, then scales, position and weight.
// Block (0, 0, 0) sets seq, which no block reads here.
template <int D>
__global__ void __launch_bounds__(256) kv4_evict_move_kernel(
    const __grid_constant__ Kv4EvictParams p) {
  const Kv4& c = p.c;
  const int h = blockIdx.y, b = blockIdx.z;
  const size_t plane = (static_cast<size_t>(b) * c.H + h) * c.N;
  const int n = p.n_moves[static_cast<size_t>(b) * c.H + h];
  const int32_t* holes = p.lists + plane;
  const int32_t* movers = holes + c.N / 2;
  constexpr int kPieces = D / 32;  // 16-byte pieces of one code row
  const int sub = threadIdx.x & 15;
  for (int i = blockIdx.x * 16 + (threadIdx.x >> 4); i < n; i += gridDim.x * 16) {
    const size_t to = plane + holes[i], from = plane + movers[i];
    if (sub < kPieces) {
      reinterpret_cast<uint4*>(c.k_codes + to * (D / 2))[sub] =
          reinterpret_cast<const uint4*>(c.k_codes + from * (D / 2))[sub];
    } else if (sub < 2 * kPieces) {
      reinterpret_cast<uint4*>(c.v_codes + to * (D / 2))[sub - kPieces] =
          reinterpret_cast<const uint4*>(c.v_codes + from * (D / 2))[sub - kPieces];
    } else if (sub < 2 * kPieces + D / 64) {
      const int s = sub - 2 * kPieces;
      reinterpret_cast<uint32_t*>(c.k_scales + to * (D / 16))[s] =
          reinterpret_cast<const uint32_t*>(c.k_scales + from * (D / 16))[s];
    } else if (sub < 2 * kPieces + D / 32) {
      const int s = sub - 2 * kPieces - D / 64;
      reinterpret_cast<uint32_t*>(c.v_scales + to * (D / 16))[s] =
          reinterpret_cast<const uint32_t*>(c.v_scales + from * (D / 16))[s];
    } else if (sub == 14) {
      c.pos[to] = c.pos[from];
    } else if (sub == 15) {
      c.weight[to] = c.weight[from];
    }
  }
  if (blockIdx.x == 0 && h == 0 && b == 0) {
    for (int i = threadIdx.x; i < c.B; i += 256) {
      const int held = rows_held(c, i);
      if (held > p.keep) {
        c.seq[kSeqHeld * c.B + i] = p.keep;
        c.seq[kSeqLast * c.B + i] = 0;
        c.seq[kSeqTail * c.B + i] = 0;
      }
    }
  }
}

}  // namespace sa
