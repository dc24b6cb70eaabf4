// Parameters and index arithmetic shared by the attention kernels over a 4-bit cache.
#pragma once

#include "kv4_format.cuh"
#include "ptx.cuh"

namespace sa {

// Query rows of one (sequence, KV head): row r is token r / group, query head
// h * group + r % group. Rows of one token are neighbours, so a tile of rows spans
// few tokens and, under a causal mask, ends early.
struct Kv4AttendParams {
  Kv4 c;
  Kv4Rows q, o;
  const int32_t* counts;
  float* lse;  // [B][heads][T] or null
  int heads, group, T, causal, add_weight;
  float scale_log2;  // softmax scale * log2 e
  // few query rows (kv4_decode.cuh)
  int row_blocks;  // blocks of query rows per (sequence, KV head)
  float* part_o;   // [slot][rows of a block][D], not normalised
  float2* part_ml; // [slot][rows of a block]: maximum (base 2), sum
  float* scores;   // [B][H][N][score_rows], base 2
  int score_rows;
  // many query rows (kv4_chunk.cuh)
  int q_tiles, pairs;  // tiles of 128 query rows per (sequence, KV head), and pairs of them
  uint8_t* q_img;      // [B][H][q_tiles] shared memory images of the fp16 query tiles
  float* row_scale;    // [B][H][q_tiles * 128]: score factor of a staged row
  float* row_lse;      // the same: base-2 log-sum-exp, +inf where no weight is drawn
  long long* line;     // [B + 1]
  int* pre;            // [B][pairs + 1]
};

// Rows that query token t of sequence b reads.
__device__ __forceinline__ int rows_seen(const Kv4AttendParams& p, int held, int n_tok, int t) {
  return p.causal ? max(min(held - n_tok + t + 1, held), 0) : held;
}

// Report a causal call whose rows an eviction put out of order.
__device__ __forceinline__ void check_order(const Kv4AttendParams& p, int b, int n_tok) {
  if (p.causal && n_tok > 1 && n_tok > p.c.seq[kSeqTail * p.c.B + b])
    atomicOr(p.c.status, kDevErrOrder);
}

// The power of two that brings a row whose largest magnitude is amax to [1, 2):
// bf16 has a wider range than the fp16 that enters the products. Values below
// 2^-14 of the largest lose bits, 2^-25 of it at most. Rows that are zero or not
// finite stay as they are (NaN and infinities then reach their own outputs only).
__device__ __forceinline__ float row_factor(float amax) {
  const unsigned e = __float_as_uint(amax) >> 23;
  if (!(amax > 0.f) || e >= 255u) return 1.f;
  return __uint_as_float((254u - min(max(e, 1u), 253u)) << 23);
}

}  // namespace sa
