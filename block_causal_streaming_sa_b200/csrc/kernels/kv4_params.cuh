// Parameters and index arithmetic shared by the attention kernels over a 4-bit cache.
#pragma once

#include "kv4_format.cuh"
#include "ptx.cuh"

namespace sa {

// 2^x of two values on the FMA and integer pipes, for a share of the exponentials that
// the exponential unit alone would hold up: x = n + f, n = round(x), 2^f on [-1/2, 1/2]
// by a degree-5 polynomial (minimax in relative error, 2.4e-7 evaluated in fp32;
// fit_exp2_poly.py), n added to the exponent. From -127 down the result is a subnormal's last
// bit, for the caller to flush. Sums that rank rows come from these values, hence a
// polynomial as exact as the unit (2^-22). A NaN comes out as if it were -127: an exponent
// added to a NaN would leave a finite number as well.
__device__ __forceinline__ void exp2_fma2(float& y0, float& y1, float x0, float x1) {
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23
  constexpr float c0 = 1.0000001192092896f, c1 = 0.6931469440460205f, c2 = 0.24022120237350464f;
  constexpr float c3 = 0.05550713092088699f, c4 = 0.009675540961325169f;
  constexpr float c5 = 0.0013276472454890609f;
  x0 = fmaxf(x0, -127.0f);
  x1 = fmaxf(x1, -127.0f);
  float t0, t1, f0, f1, q0, q1;
  ptx::fadd2(t0, t1, x0, x1, kRound, kRound);
  ptx::fadd2(f0, f1, t0, t1, -kRound, -kRound);  // n
  ptx::ffma2(f0, f1, f0, f1, -1.0f, -1.0f, x0, x1);
  ptx::ffma2(q0, q1, f0, f1, c5, c5, c4, c4);
  ptx::ffma2(q0, q1, q0, q1, f0, f1, c3, c3);
  ptx::ffma2(q0, q1, q0, q1, f0, f1, c2, c2);
  ptx::ffma2(q0, q1, q0, q1, f0, f1, c1, c1);
  ptx::ffma2(q0, q1, q0, q1, f0, f1, c0, c0);
  y0 = __int_as_float(__float_as_int(q0) + (__float_as_int(t0) << 23));
  y1 = __int_as_float(__float_as_int(q1) + (__float_as_int(t1) << 23));
}

// P = 2^(score - reference) enters the second product as fp16. The reference follows the
// running maximum from kRefBelow below it, and is raised once a score exceeds it by more
// than kRefTop: P stays below 2^15 (fp16 reaches 2^16), and what is kRefBelow + 14 powers of
// two below the maximum still has all eleven bits, what is kRefBelow + 25 below it some.
// Behind a row that dominates (the first of a sequence often does) everything else lies
// far below the maximum, and its roundings add up over a long cache instead of cancelling:
// with the reference at the maximum, whatever lay 17 nats below it lost its share of O. Five
// powers of two between the two bounds keep the raises rare: 8, 5, 4, 3 of them take 788, 784,
// 798, 849 us (6120 x 24480 rows, 12 heads, scores of a deviation of 1.1 nats).
constexpr float kRefBelow = 10.0f, kRefTop = 15.0f;

// What a staged row's scores are multiplied with. Kept above zero: a masked score is
// -inf, and 0 * -inf is not.
__device__ __forceinline__ float score_factor(const float scale_log2, float row_factor) {
  return fmaxf(scale_log2 / row_factor, 1.17549435e-38f);
}

// Work of many unequal items laid out as one line of steps and cut into equal ranges,
// one a block: sequence by sequence, KV head by KV head, item by item. Heads of a
// sequence have the same items.
struct StepLine {
  long long* begin;  // [B + 1]: steps before sequence b
  int* pre;          // [B][items + 2]: steps of one head of b before each of its items and
                     // after the last; at the end the number of its items
  int items;         // at most
  __device__ __forceinline__ int* row(int b) const {
    return pre + static_cast<size_t>(b) * (items + 2);
  }
};

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
  float2* part_ml; // [slot][rows of a block]: reference (base 2), sum
  float* scores;   // [B][H][N][score_rows], base 2
  int score_rows;
  // many query rows (kv4_chunk.cuh, kv4_weights.cuh)
  int q_tiles;           // tiles of 128 query rows per (sequence, KV head)
  uint8_t* q_img;        // [B][H][q_tiles] shared memory images of the fp16 query tiles
  float* row_scale;      // [B][H][q_tiles * 128]: score factor of a staged row
  float* row_nlse;       // the same: minus its base-2 log-sum-exp, -inf if it draws no weight
  StepLine line;         // steps of the attention: items of 512 query rows x key tiles
  StepLine weight_line;  // steps of the weights: key tiles x query tiles
  float* part_w;         // [slot][128]: partial sums of weights
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

// Fills `line` from count(b), the items of sequence b, and steps(b, item): one block of
// 256 threads, a sequence per warp.
template <typename F, typename G>
__device__ __forceinline__ void lay_line(const StepLine& line, int B, int H, F count, G steps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b = warp; b < B; b += 8) {
    int* pre = line.row(b);
    const int n = min(count(b), line.items);
    int sum = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int v = i0 + lane < n ? steps(b, i0 + lane) : 0;
      int x = v;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int y = __shfl_up_sync(~0u, x, k);
        if (lane >= k) x += y;
      }
      if (i0 + lane < n) pre[i0 + lane] = sum + x - v;
      sum += __shfl_sync(~0u, x, 31);
    }
    if (lane == 0) {
      pre[n] = sum;
      pre[line.items + 1] = n;
      line.begin[b + 1] = static_cast<long long>(sum) * H;
    }
  }
  __syncthreads();
  if (warp == 0) {
    if (lane == 0) line.begin[0] = 0;
    long long sum = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      long long x = b0 + lane < B ? line.begin[b0 + lane + 1] : 0;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const long long y = __shfl_up_sync(~0u, x, k);
        if (lane >= k) x += y;
      }
      if (b0 + lane < B) line.begin[b0 + lane + 1] = sum + x;
      sum += __shfl_sync(~0u, x, 31);
    }
  }
}

// A walk along a range of a line: its items, each with its steps [t0, t1) of n.
struct LineWalk {
  long long at, stop;
  int b, h, item;
  int t0, t1, n;

  __device__ __forceinline__ void start(long long from, long long to) {
    at = from;
    stop = to;
    b = h = item = t0 = t1 = n = 0;
  }
  // The next item of the range of a line over B sequences; false at its end.
  __device__ __forceinline__ bool next(const StepLine& line, int B) {
    if (at >= stop) return false;
    int lo = b, hi = B;  // begin[lo] <= at < begin[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (line.begin[mid] <= at)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;  // of sequences without steps that share a start, the last is the one with steps
    const int* pre = line.row(b);
    const int items = pre[line.items + 1], per_head = pre[items];
    const long long in_b = at - line.begin[b];
    h = static_cast<int>(in_b / per_head);
    const int in_h = static_cast<int>(in_b % per_head);
    lo = 0;
    hi = items;  // pre[lo] <= in_h < pre[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (pre[mid] <= in_h)
        lo = mid;
      else
        hi = mid;
    }
    // of items without steps that share a start, the last is the one with steps
    item = lo;
    n = pre[item + 1] - pre[item];
    t0 = in_h - pre[item];
    t1 = static_cast<int>(min(static_cast<long long>(n), t0 + (stop - at)));
    at += t1 - t0;
    return true;
  }
};

__device__ __forceinline__ long long line_share(const StepLine& line, int B, int blocks) {
  return (line.begin[B] + blocks - 1) / blocks;
}

// Range `block` of `blocks` of the line.
__device__ __forceinline__ LineWalk line_range(const StepLine& line, int B, int block, int blocks) {
  const long long share = line_share(line, B, blocks), total = line.begin[B];
  LineWalk w;
  w.start(min(block * share, total), min((block + 1) * share, total));
  return w;
}

// Where a block leaves the partial result of an item: a range that begins inside one
// (t0 > 0) can do so once, a range that ends inside one it began (t0 = 0) too.
__device__ __forceinline__ size_t partial_slot(int block, int t0) {
  return 2 * static_cast<size_t>(block) + (t0 > 0 ? 0 : 1);
}

// An item that lies in several blocks' ranges, found from the one boundary (block
// ranges `boundary` and `boundary` + 1) that has to merge it: the first inside it.
struct SplitItem {
  LineWalk w;
  int first, last;  // blocks that have a part

  __device__ __forceinline__ bool find(const StepLine& line, int B, int blocks, int boundary) {
    const long long share = line_share(line, B, blocks), total = line.begin[B];
    const long long from = (boundary + 1) * share;
    if (from >= total) return false;
    w.start(from, total);
    w.next(line, B);
    const long long begin = from - w.t0, end = begin + w.n;
    if (w.t0 == 0 || from - share > begin) return false;
    first = static_cast<int>(begin / share);
    last = static_cast<int>((end - 1) / share);
    return true;
  }
  __device__ __forceinline__ size_t slot(int block) const {
    return partial_slot(block, block == first ? 0 : 1);
  }
};

}  // namespace sa
