// Attention of few query rows over a 4-bit cache: one generated token, some drafts.
//
// Bound by reading the cache: D + D / 8 bytes a row and KV head. What a row costs on
// an SM apart from that is its dequantisation, so the products go to the register
// matrix instruction (mma m16n8k16): its operands come from shared memory straight
// into the registers the codes are unpacked in, while tcgen05 operands would have to
// be written back to shared memory at 16 bits and read again (1 KB a row and head
// against 288 bytes), more than the shared memory of an SM carries at HBM speed;
// the tensor core itself is idle either way (8 useful query rows of the tile).
//
//  * S^T = K Q^T: 16 cache rows x 8 query rows x 16 values. The order of the values
//    along D is free as long as both operands agree, so a lane's K registers are the
//    codes of one aligned 16-byte (D = 64: 8-byte) piece of a row, in order.
//  * O^T = V^T P^T: 16 values x 8 query rows x 16 cache rows. A lane owns D / 8
//    consecutive values of four rows; two rows' codes are merged into bytes before
//    the conversion, which then yields pairs of rows. P^T comes from S^T by
//    transposing 8 x 8 blocks (movmatrix); both keep query rows on the same lanes, so
//    the softmax statistics never move.
//  * The reference of a query row (kRefBelow) is raised only when a score exceeds it by
//    more than kRefTop (checked by one vote a tile): no reduction across lanes otherwise.
//    l and O are fp32.
//  * Each warp streams tiles of 32 rows through a ring of its own (a bulk copy by
//    each of four lanes, an mbarrier a stage), so warps never wait for one another.
//  * The rows of all sequences and heads are one line of tiles, cut into equal
//    ranges, one a block, whatever the lengths: long rows are split over blocks and
//    short ones share one. A range that crosses heads leaves one partial result per
//    head; (block + head) numbers them without gaps growing beyond blocks + heads.
//    kv4_join_kernel merges them in that order.
//
// Measured: 4 x 131071 rows, 8 heads, D 128, 8 query rows: 125 us, 4.8 TB/s (the copies
// alone, without arithmetic, 91 us; the rest is unpacking at the 1.3 GHz held under
// this load). 700 rows, 8 heads: 10 us, launches and dependent loads. With 20 query rows
// (8 sequences of up to 8000 rows, 8 heads, D 64: 23 us) it is latency: eight warps an SM, whose
// registers allow no more, fill 41 % of the issue slots and 24 % of the matrix unit.
#pragma once

#include "kv4_params.cuh"

namespace sa {

// The reference before any score: finite, so that a masked score (-inf) minus it is -inf,
// and below every score.
constexpr float kNoScore = -3.402823466e38f;

// Blocks an SM of kv4_decode_kernel for 8 nt query rows, by its registers and shared memory;
// the workspace is laid out for as many.
__host__ __device__ constexpr int decode_blocks_per_sm(int nt) {
  return nt == 1 ? 4 : nt == 2 ? 3 : 2;
}

template <int D, int NT>
struct DecodeShape {
  static constexpr int kWarps = 4;
  static constexpr int kRows = 8 * NT;  // query rows of a block
  static constexpr int kTile = 32;      // cache rows of a warp's tile
  static constexpr int kCodes = kTile * D / 2, kScales = kTile * D / 16;
  static constexpr int kStageBytes = 2 * (kCodes + kScales);
  static constexpr int kStages = D == 128 ? 3 : 4;  // 55 KB (D 128): four blocks an SM
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kMergeStride = D + 4;
  static constexpr int kMerge = kWarps * kRows * kMergeStride * 4;
  static constexpr int kData = kRing > kMerge ? kRing : kMerge;
  static constexpr int kOffMl = kData;                             // float2 [warp][row]
  static constexpr int kOffQ = kOffMl + kWarps * kRows * 8;        // fragments, NT > 1
  static constexpr int kOffSl = kOffQ + (NT > 1 ? kRows * D * 2 : 0);
  static constexpr int kOffBar = kOffSl + kRows * 4;
  static constexpr int kSmem = kOffBar + kWarps * kStages * 8 + 16;
  static constexpr int kBlocksPerSm = decode_blocks_per_sm(NT);
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

// Cache row, within 16, of row r of the matrix tiles: an order in which neither the
// K loads (lanes of equal r / 4: neighbours in r) nor the V loads (every second r)
// meet the same banks more often than their bytes make necessary.
template <int D>
__device__ __forceinline__ int tile_row(int r) {
  if constexpr (D == 128) return r ^ ((r >> 1) & 1);
  constexpr unsigned order = 0x57463120u;  // 0 2 1 3 6 4 7 5
  return (r & 8) | static_cast<int>((order >> ((r & 7) * 4)) & 7u);
}

// The tiles of all (sequence, head, row block) units lie on one line. Every warp derives
// what it needs from the lengths, a sequence a lane.
struct Line {
  int share;  // tiles of a block: at least 4, so that every warp has one
  int total;
};

// Tiles of one unit of sequence b.
__device__ __forceinline__ int unit_tiles(const Kv4AttendParams& p, int b, int tile) {
  if (b >= p.c.B || tokens_of(p.counts, b, p.T) == 0) return 0;
  return (rows_held(p.c, b) + tile - 1) / tile;
}

__device__ __forceinline__ int scan_lanes(int x, int lane) {
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int y = __shfl_up_sync(~0u, x, k);
    if (lane >= k) x += y;
  }
  return x;
}

__device__ __forceinline__ Line line_of(const Kv4AttendParams& p, int blocks, int tile, int lane) {
  int sum = 0;
  for (int b = lane; b < p.c.B; b += 32) sum += unit_tiles(p, b, tile);
  Line l;
  l.total = __reduce_add_sync(~0u, sum) * p.c.H * p.row_blocks;
  l.share = max((l.total + blocks - 1) / blocks, 4);
  return l;
}

// The sequence that holds tile `at` of the line (at < total), its first tile and the
// tiles of one of its units.
__device__ __forceinline__ void find_sequence(const Kv4AttendParams& p, int at, int tile, int lane,
                                              int& b, int& begin, int& per_unit) {
  const int units = p.c.H * p.row_blocks;
  int base = 0;
  for (int b0 = 0;; b0 += 32) {
    const int n = unit_tiles(p, b0 + lane, tile);
    const int end = base + scan_lanes(n * units, lane);
    const unsigned past = __ballot_sync(~0u, at < end);
    if (past != 0 || b0 + 32 >= p.c.B) {
      const int hit = past != 0 ? __ffs(past) - 1 : 31;
      b = b0 + hit;
      begin = __shfl_sync(~0u, end - n * units, hit);
      per_unit = __shfl_sync(~0u, n, hit);
      return;
    }
    base = __shfl_sync(~0u, end, 31);
  }
}

// Tiles of the line before sequence `upto`.
__device__ __forceinline__ int tiles_before(const Kv4AttendParams& p, int upto, int tile,
                                            int lane) {
  int sum = 0;
  for (int b = lane; b < upto; b += 32) sum += unit_tiles(p, b, tile);
  return __reduce_add_sync(~0u, sum) * p.c.H * p.row_blocks;
}

// A lane's quarter of a query row as the fragments of S^T = K Q^T: lane (g, tig) of
// step k holds values 4 k .. 4 k + 3 of its D / 4 consecutive ones of row g. Scaled to
// fp16 by a power of two per row; returns what the row's scores are multiplied with.
template <int D, int kDtype>
__device__ __forceinline__ float query_fragments(const uint4 (&w)[D / 32], float scale_log2,
                                                 uint32_t (&frag)[D / 16][2]) {
  float2 v[D / 8];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    v[4 * i] = unpack2<kDtype>(w[i].x);
    v[4 * i + 1] = unpack2<kDtype>(w[i].y);
    v[4 * i + 2] = unpack2<kDtype>(w[i].z);
    v[4 * i + 3] = unpack2<kDtype>(w[i].w);
  }
#pragma unroll
  for (int i = 0; i < D / 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
  amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
  const float f = row_factor(amax);
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    frag[k][0] = pack2<SA_DTYPE_FP16>(v[2 * k].x * f, v[2 * k].y * f);
    frag[k][1] = pack2<SA_DTYPE_FP16>(v[2 * k + 1].x * f, v[2 * k + 1].y * f);
  }
  return score_factor(scale_log2, f);
}

// This lane's quarter of query row `row` of (sequence b, KV head h); zeros if not there.
template <int D>
__device__ __forceinline__ void load_query(const Kv4AttendParams& p, int b, int h, int row,
                                           bool there, int tig, uint4 (&w)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  if (!there) return;
  const uint16_t* q = static_cast<const uint16_t*>(p.q.data) + b * p.q.sb +
                      (row / p.group) * p.q.st + (h * p.group + row % p.group) * p.q.sh +
                      tig * (D / 4);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) w[i] = reinterpret_cast<const uint4*>(q)[i];
}

// A warp tile's K codes as operand registers: [word][16-row half][rows g, g + 8][pair].
// `kc`, `ksc`: the tile's codes and scales in shared memory.
template <int D>
struct KeyWords {
  uint32_t w[2][2][D / 32], s[2][2];
  __device__ __forceinline__ void load(uint32_t kc, uint32_t ksc, int g, int tig) {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        const int row = sub * 16 + tile_row<D>(g + 8 * hi);
        if constexpr (D == 128) {
          const uint4 x = lds128(kc + row * 64 + tig * 16);
          w[sub][hi][0] = x.x;
          w[sub][hi][1] = x.y;
          w[sub][hi][D / 32 - 2] = x.z;
          w[sub][hi][D / 32 - 1] = x.w;
          s[sub][hi] = lds16(ksc + row * 8 + tig * 2);
        } else {
          const uint2 x = lds64(kc + row * 32 + tig * 8);
          w[sub][hi][0] = x.x;
          w[sub][hi][D / 32 - 1] = x.y;
          s[sub][hi] = lds8(ksc + row * 4 + tig);
        }
      }
  }
  // Word `i` (two steps of 16 values): a[half][rows g, g + 8][pair], scaled.
  __device__ __forceinline__ void convert(int i, uint32_t (&a)[2][2][4]) const {
#pragma unroll
    for (int sub = 0; sub < 2; ++sub)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        codes_to_f16(w[sub][hi][i], a[sub][hi]);
        const uint32_t sc =
            scale_f16x2(D == 128 ? (s[sub][hi] >> (8 * (i >> 1))) & 255u : s[sub][hi]);
#pragma unroll
        for (int k = 0; k < 4; ++k) a[sub][hi][k] = mul_f16x2(a[sub][hi][k], sc);
      }
  }
};

template <int D, int NT, int kDtype, bool kScores>
__global__ void __launch_bounds__(128, DecodeShape<D, NT>::kBlocksPerSm)
    kv4_decode_kernel(const __grid_constant__ Kv4AttendParams p) {
  using S = DecodeShape<D, NT>;
  constexpr int KS = D / 16;       // steps along D of S^T = tiles of values of O^T
  constexpr int KW = D / 32;       // words of K codes of a lane and row
  constexpr int VW = D / 64;       // words of V codes of a lane and row
  extern __shared__ __align__(128) uint8_t smem[];
  const Kv4& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tig = lane & 3;
  const uint32_t sbase = ptx::smem_addr(smem);
  const uint32_t ring = sbase + warp * S::kStages * S::kStageBytes;
  const uint32_t bars = sbase + S::kOffBar + warp * S::kStages * 8;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kSmem - 16);
  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < S::kStages; ++s) ptx::mbar_init(bars + 8 * s, 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  // In this order: the join reads the lengths before it waits for this kernel, so it
  // must not begin before the kernel that wrote them (an append) has finished.
  wait_for_previous();
  begin_early();

  const Line line = line_of(p, gridDim.x, S::kTile, lane);
  int at = min(static_cast<long long>(blockIdx.x) * line.share,
               static_cast<long long>(line.total));
  const int stop = min(at + line.share, line.total);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < c.B; b += 128) check_order(p, b, tokens_of(p.counts, b, p.T));
  if (at >= stop) return;

  int b, b0, per_unit;  // the sequence of tile `at`, its first tile, tiles of a unit
  find_sequence(p, at, S::kTile, lane, b, b0, per_unit);
  int st = 0, pending = 0;  // stage in turn; copies under way or not used yet
  uint32_t phase = 0;
  bool ok = true;
  const int copy_at = lane == 0   ? 0
                      : lane == 1 ? S::kCodes
                      : lane == 2 ? 2 * S::kCodes
                                  : 2 * S::kCodes + S::kScales;

  while (at < stop) {
    // one unit: tiles [t0, t1) of sequence b, KV head h, query rows row0 ..
    if (at >= b0 + per_unit * c.H * p.row_blocks)
      find_sequence(p, at, S::kTile, lane, b, b0, per_unit);
    const int unit_in_b = (at - b0) / per_unit;
    const int t0 = at - b0 - unit_in_b * per_unit;
    const int t1 = min(per_unit, t0 + (stop - at));
    const int h = unit_in_b / p.row_blocks, rb = unit_in_b % p.row_blocks;
    const int unit = b * c.H * p.row_blocks + unit_in_b;
    const int held = rows_held(c, b), n_tok = tokens_of(p.counts, b, p.T);
    const int n_rows = n_tok * p.group, row0 = rb * S::kRows;
    const size_t plane = (static_cast<size_t>(b) * c.H + h) * c.N;

    // Lanes 0 .. 3 each issue one of a tile's four copies, from `src` on.
    const int copy_bytes = lane < 2 ? S::kCodes : S::kScales;
    const uint8_t* src = (lane == 0   ? c.k_codes
                          : lane == 1 ? c.v_codes
                          : lane == 2 ? c.k_scales
                                      : c.v_scales) +
                         plane * (lane < 2 ? D / 2 : D / 16);
    auto fill = [&](int tile, int stage) {
      const uint32_t bar = bars + 8 * stage;
      if (lane == 0) ptx::mbar_arrive_expect_tx(bar, S::kStageBytes);
      __syncwarp();
      if (lane < 4)
        bulk_load(ring + stage * S::kStageBytes + copy_at,
                  src + static_cast<size_t>(tile) * copy_bytes, copy_bytes, bar);
    };
    // The query row of this lane is asked for before the ring is filled: behind 200 KB of
    // copies an SM it would come microseconds later. Warps share the rows of NT > 1.
    const int my_nt = NT == 1 ? 0 : warp, q_row = row0 + my_nt * 8 + g;
    const bool has_row = my_nt < NT && q_row < n_rows;
    uint4 qw[D / 32];
    load_query<D>(p, b, h, q_row, has_row, tig, qw);
    int next = t0 + warp;  // next tile to load; the ring is empty here
    for (int s = 0; s < S::kStages && ok && next < t1; ++s, next += S::kWarps, ++pending)
      fill(next, st + s < S::kStages ? st + s : st + s - S::kStages);

    uint32_t qf[KS][2];  // the lane's own row; with NT > 1 all rows are in shared memory
    float sl[NT][2];     // scale * log2 e / row factor of this lane's query columns
    float* s_sl = reinterpret_cast<float*>(smem + S::kOffSl);
    if constexpr (NT > 1) __syncthreads();  // the previous unit is done with them
    if (my_nt < NT) {
      const float scale = query_fragments<D, kDtype>(qw, p.scale_log2, qf);
      if constexpr (NT == 1) {  // lane 4 n (or any of its four) holds row n's
        sl[0][0] = __shfl_sync(~0u, scale, 8 * tig);
        sl[0][1] = __shfl_sync(~0u, scale, 8 * tig + 4);
      } else {
#pragma unroll
        for (int k = 0; k < KS; ++k)
          *reinterpret_cast<uint2*>(smem + S::kOffQ + ((k * NT + my_nt) * 32 + lane) * 8) =
              make_uint2(qf[k][0], qf[k][1]);
        if (tig == 0) s_sl[my_nt * 8 + g] = scale;
      }
    }
    if constexpr (NT > 1) {
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        sl[nt][0] = s_sl[nt * 8 + 2 * tig];
        sl[nt][1] = s_sl[nt * 8 + 2 * tig + 1];
      }
    }

    float o[KS][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[k][nt][i] = 0.f;
      m[nt][0] = m[nt][1] = kNoScore;
      l[nt][0] = l[nt][1] = 0.f;
    }
    // rows before this see no mask
    const int open = p.causal ? max(held - n_tok + 1, 0) : held;

    for (int t = t0 + warp; ok && t < t1; t += S::kWarps) {
      ok = __all_sync(~0u, ptx::mbar_wait(bars + 8 * st, phase, abort_flag, c.status));
      if (!ok) break;
      --pending;
      const uint32_t kc = ring + st * S::kStageBytes, vc = kc + S::kCodes;
      const uint32_t ksc = vc + S::kCodes, vsc = ksc + S::kScales;
      const int j0 = t * S::kTile;
      const bool edge = j0 + S::kTile > open;

      // ---- S^T
      float s[2][NT][4];
      KeyWords<D> kw;
      kw.load(kc, ksc, g, tig);
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[sub][nt][i] = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {  // a word is two steps
        uint32_t a[2][2][4];
        kw.convert(w, a);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int k = 2 * w + half;
            uint32_t b0, b1;
            if constexpr (NT == 1) {
              b0 = qf[k][0];
              b1 = qf[k][1];
            } else {
              const uint2 f = lds64(sbase + S::kOffQ + ((k * NT + nt) * 32 + lane) * 8);
              b0 = f.x;
              b1 = f.y;
            }
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
              mma_16816(s[sub][nt], a[sub][0][2 * half], a[sub][1][2 * half],
                        a[sub][0][2 * half + 1], a[sub][1][2 * half + 1], b0, b1);
          }
      }

      // ---- softmax: s[sub][nt] = rows g, g, g + 8, g + 8; queries 2 tig, 2 tig + 1, ..
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = row0 + nt * 8 + 2 * tig + (i & 1);
            const int end = rows_seen(p, held, n_tok, r / p.group);
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
              if (j0 + sub * 16 + tile_row<D>(g + (i & 2) * 4) >= end)
                s[sub][nt][i] = -INFINITY;
          }
      }
      if constexpr (kScores) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = row0 + nt * 8 + 2 * tig;
          if (r < p.score_rows)
#pragma unroll
            for (int sub = 0; sub < 2; ++sub)
#pragma unroll
              for (int hi = 0; hi < 2; ++hi) {
                const size_t row = plane + j0 + sub * 16 + tile_row<D>(g + 8 * hi);
                *reinterpret_cast<float2*>(p.scores + row * p.score_rows + r) =
                    make_float2(s[sub][nt][2 * hi] * sl[nt][0], s[sub][nt][2 * hi + 1] * sl[nt][1]);
              }
        }
      }
      float x[2][NT][4];
      auto subtract = [&]() {
        float top = -INFINITY;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[sub][nt][i] = fmaf(s[sub][nt][i], sl[nt][i & 1], -m[nt][i & 1]);
              top = fmaxf(top, x[sub][nt][i]);
            }
        return top;
      };
      if (__any_sync(~0u, subtract() > kRefTop)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float mx = fmaxf(fmaxf(s[0][nt][i], s[0][nt][i + 2]),
                             fmaxf(s[1][nt][i], s[1][nt][i + 2]));
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, k));
            mx = fmaxf(mx * sl[nt][i] - kRefBelow, m[nt][i]);
            const float a = mx > m[nt][i] ? ptx::ex2(m[nt][i] - mx) : 1.f;
            m[nt][i] = mx;
            l[nt][i] *= a;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[k][nt][i] *= a;
              o[k][nt][i + 2] *= a;
            }
          }
        subtract();
      }
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int sub = 0; sub < 2; ++sub) {
          const float p0 = ptx::ex2(x[sub][nt][0]), p1 = ptx::ex2(x[sub][nt][1]);
          const float p2 = ptx::ex2(x[sub][nt][2]), p3 = ptx::ex2(x[sub][nt][3]);
          l[nt][0] += p0 + p2;
          l[nt][1] += p1 + p3;
          pb[sub][nt][0] = transpose_8x8(pack2<SA_DTYPE_FP16>(p0, p1));
          pb[sub][nt][1] = transpose_8x8(pack2<SA_DTYPE_FP16>(p2, p3));
        }

      // ---- O^T: a lane's rows are 2 tig, 2 tig + 1, and those + 8; its values
      // D / 8 g .. (matrix rows g and g + 8 of tile k are values 2 k and 2 k + 1)
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        uint32_t vw[4][VW], byte[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = sub * 16 + tile_row<D>(2 * tig + (e & 1) + 8 * (e >> 1));
          if constexpr (D == 128) {
            const uint2 w = lds64(vc + row * 64 + g * 8);
            vw[e][0] = w.x;
            vw[e][VW - 1] = w.y;
            byte[e] = lds8(vsc + row * 8 + g);
          } else {
            vw[e][0] = lds32(vc + row * 32 + g * 4);
            byte[e] = lds8(vsc + row * 4 + (g >> 1));
          }
          // rows not held may hold any bytes: a scale that is NaN must not meet P = 0
          if (edge && j0 + row >= held) byte[e] = 0;
        }
        const uint32_t sc[2] = {scales_f16x2(byte[0], byte[1]), scales_f16x2(byte[2], byte[3])};
#pragma unroll
        for (int w = 0; w < VW; ++w) {
          // Two rows' codes of one value into a byte, so that the conversion leaves
          // them as a pair: [rows 0 and 1, rows 2 and 3][even, odd values].
          uint32_t v[2][2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t x = vw[2 * e][w], y = vw[2 * e + 1][w];
            codes_to_f16((x & 0x0F0F0F0Fu) | ((y * 16u) & 0xF0F0F0F0u), v[e][0]);
            codes_to_f16(((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), v[e][1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = mul_f16x2(v[0][0][i], sc[0]), a1 = mul_f16x2(v[0][1][i], sc[0]);
            const uint32_t a2 = mul_f16x2(v[1][0][i], sc[1]), a3 = mul_f16x2(v[1][1][i], sc[1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_16816(o[4 * w + i][nt], a0, a1, a2, a3, pb[sub][nt][0], pb[sub][nt][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (next < t1) {  // the ring was full: this stage is the next to fill
        fill(next, st);
        next += S::kWarps;
        ++pending;
      }
      if (++st == S::kStages) {
        st = 0;
        phase ^= 1u;
      }
    }
    // (after an abort the blocks' barriers below are still met; the result is void)

    // ---- merge the four warps in shared memory (the rings are empty now)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) l[nt][i] += __shfl_xor_sync(~0u, l[nt][i], k);
    __syncthreads();
    float2* s_ml = reinterpret_cast<float2*>(smem + S::kOffMl);
    float* s_o = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = nt * 8 + 2 * tig + i;
        if (g == 0) s_ml[warp * S::kRows + r] = make_float2(m[nt][i], l[nt][i]);
        float* dst = s_o + (warp * S::kRows + r) * S::kMergeStride + g * (D / 8);
#pragma unroll
        for (int k = 0; k < KS; k += 2)
          *reinterpret_cast<float4*>(dst + 2 * k) =
              make_float4(o[k][nt][i], o[k][nt][i + 2], o[k + 1][nt][i], o[k + 1][nt][i + 2]);
      }
    }
    __syncthreads();
    const size_t slot = static_cast<size_t>(blockIdx.x) + unit;
    for (int i = threadIdx.x; i < S::kRows * (D / 4); i += 128) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      if (row0 + r >= n_rows) break;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < S::kWarps; ++w) mx = fmaxf(mx, s_ml[w * S::kRows + r].x);
      const float ref = mx == -INFINITY ? 0.f : mx;
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < S::kWarps; ++w) {
        const float2 ml = s_ml[w * S::kRows + r];
        const float a = ptx::ex2(ml.x - ref);
        const float4 x =
            *reinterpret_cast<float4*>(s_o + (w * S::kRows + r) * S::kMergeStride + d);
        sum += ml.y * a;
        acc.x += x.x * a;
        acc.y += x.y * a;
        acc.z += x.z * a;
        acc.w += x.w * a;
      }
      *reinterpret_cast<float4*>(p.part_o + (slot * S::kRows + r) * D + d) = acc;
      if (d == 0) p.part_ml[slot * S::kRows + r] = make_float2(mx, sum);
    }
    at += t1 - t0;
    // the copies of the next unit go through the asynchronous proxy into memory that
    // was just read and written here
    __syncthreads();
    ptx::fence_proxy_async_smem();
  }
  // after an abort: copies still under way land before the block's memory goes
  if (!ok) {
    volatile int none = 0;
    for (; pending > 0; --pending) {
      ptx::mbar_wait(bars + 8 * st, phase, &none, c.status);
      if (++st == S::kStages) {
        st = 0;
        phase ^= 1u;
      }
    }
  }
}

// Merge of the partial results of kv4_decode_kernel, W warps per query row, and, where
// that left the scores (up to 8 query rows), the rows' weights. Blocks below
// join_blocks merge; the others add weights, a range of rows of one (sequence, KV
// head) each, kJoinKeys at a time: they derive the log-sum-exp of its query rows from the same partial
// results, so no order among blocks is needed.
constexpr int kJoinKeys = 512;

template <int D, int kRows, int W, int kDtype>
__global__ void __launch_bounds__(128)
    kv4_join_kernel(const __grid_constant__ Kv4AttendParams p, int blocks, int join_blocks,
                    int parts) {
  const Kv4& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool joins = static_cast<int>(blockIdx.x) < join_blocks;
  // join: block = (unit, 4 / W rows of it); weights (8 query rows or fewer): block =
  // (head plane, one of `parts` ranges of its rows)
  constexpr int kGroups = kRows * W / 4;
  const int id = joins ? blockIdx.x / kGroups : (blockIdx.x - join_blocks) / parts;
  const int units_b = c.H * p.row_blocks;
  const int b = joins ? id / units_b : id / c.H;
  // The lengths were there before the decode kernel let this one begin: the schedule
  // needs no wait, only that this SM's L1 holds no older ones.
  __threadfence();
  const int held = rows_held(c, b), n_tok = tokens_of(p.counts, b, p.T);
  const int n_rows = n_tok * p.group;
  const int part_rows = ((held + parts - 1) / parts + 127) / 128 * 128;
  const int j0 = joins ? 0 : static_cast<int>((blockIdx.x - join_blocks) % parts) * part_rows;
  const bool idle = n_rows == 0 || (!joins && j0 >= held);
  Line line = {1, 0};
  int b0 = 0, per_unit = 0;
  if (!idle) {
    line = line_of(p, blocks, 32, lane);
    b0 = tiles_before(p, b, 32, lane);
    per_unit = unit_tiles(p, b, 32);
  }
  begin_early();
  wait_for_previous();
  if (idle) return;

  // Partial results of one query row: `n` slots from `first` on.
  auto slots_of = [&](int unit_in_b, size_t& first, int& n) {
    const int u0 = b0 + unit_in_b * per_unit;
    first = static_cast<size_t>(u0 / line.share) + static_cast<size_t>(b) * units_b + unit_in_b;
    n = per_unit == 0 ? 0 : (u0 + per_unit - 1) / line.share - u0 / line.share + 1;
  };

  if (joins) {
    const int unit_in_b = id % units_b;
    const int h = unit_in_b / p.row_blocks, rb = unit_in_b % p.row_blocks;
    const int part = warp % W;  // slots part, part + W, ..
    const int r = (blockIdx.x % kGroups) * (4 / W) + warp / W;
    const int row = rb * kRows + r;
    if (W == 1 && row >= n_rows) return;
    size_t first;
    int n;
    slots_of(unit_in_b, first, n);
    if (W > 1 && row >= n_rows) return;  // the whole block: a row
    constexpr int V = D / 32;
    float acc[V], mx = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    // 32 slots' statistics at a time, a slot a lane; eight rows of loads under way
    const int mine = (n - part + W - 1) / W;
    for (int s0 = 0; s0 < mine; s0 += 32) {
      const int cnt = min(mine - s0, 32);
      const size_t base = first + part + static_cast<size_t>(s0) * W;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < cnt) ml = p.part_ml[(base + static_cast<size_t>(lane) * W) * kRows + r];
      float m_new = ml.x;
#pragma unroll
      for (int k = 16; k; k >>= 1) m_new = fmaxf(m_new, __shfl_xor_sync(~0u, m_new, k));
      m_new = fmaxf(m_new, mx);
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      const float old = ptx::ex2(mx - ref), a = ptx::ex2(ml.x - ref);
      mx = m_new;
      float add = ml.y * a;
#pragma unroll
      for (int k = 16; k; k >>= 1) add += __shfl_xor_sync(~0u, add, k);
      sum = sum * old + add;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] *= old;
      for (int k0 = 0; k0 < cnt; k0 += 8) {
        float x[8][V];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const size_t at = (base + static_cast<size_t>(min(k0 + k, cnt - 1)) * W) * kRows + r;
          const float* src = p.part_o + at * D + lane * V;
          if constexpr (V == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            x[k][0] = v.x;
            x[k][1] = v.y;
            x[k][V - 2] = v.z;
            x[k][V - 1] = v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            x[k][0] = v.x;
            x[k][1] = v.y;
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float ak = __shfl_sync(~0u, a, k0 + k & 31);
          if (k0 + k < cnt)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(x[k][i], ak, acc[i]);
        }
      }
    }
    if constexpr (W > 1) {  // the warps' parts, in order
      __shared__ float s_acc[W][D];
      __shared__ float2 s_ml[W];
#pragma unroll
      for (int i = 0; i < V; ++i) s_acc[warp][lane * V + i] = acc[i];
      if (lane == 0) s_ml[warp] = make_float2(mx, sum);
      __syncthreads();
      if (warp != 0) return;
#pragma unroll
      for (int w = 1; w < W; ++w) mx = fmaxf(mx, s_ml[w].x);
      const float ref = mx == -INFINITY ? 0.f : mx;
      sum = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float a = ptx::ex2(s_ml[w].x - ref);
        sum += s_ml[w].y * a;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(s_acc[w][lane * V + i], a, acc[i]);
      }
    }
    // a sum that is NaN (a query that is not finite) must stay NaN
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int t = row / p.group, hq = h * p.group + row % p.group;
    uint16_t* dst = static_cast<uint16_t*>(p.o.data) + b * p.o.sb + t * p.o.st + hq * p.o.sh +
                    lane * V;
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack2<kDtype>(acc[0] * inv, acc[1] * inv),
                     pack2<kDtype>(acc[V - 2] * inv, acc[V - 1] * inv));
    else
      *reinterpret_cast<uint32_t*>(dst) = pack2<kDtype>(acc[0] * inv, acc[1] * inv);
    if (lane == 0) {
      const float lse2 = sum == 0.f ? -INFINITY : mx + log2f(sum);
      if (p.lse != nullptr)
        p.lse[(static_cast<size_t>(b) * p.heads + hq) * p.T + t] = lse2 * 0.69314718055994531f;
      if (kRows > 8 && p.add_weight)
        p.row_nlse[(static_cast<size_t>(b) * c.H + h) * p.score_rows + row] =
            sum == 0.f ? -INFINITY : -lse2;
    }
    return;
  }

  // ---- weights of rows j0 .. of KV head h. Scores and weights are asked for first: the
  // log-sum-exps are a chain of dependent loads of their own (ragged batch of 16, 8
  // heads, 1.4 M rows in all: 69 us against 71; long ranges, few blocks: 66).
  const int h = id % c.H;
  const size_t plane = (static_cast<size_t>(b) * c.H + h) * c.N;
  constexpr int kKeys = kJoinKeys / 128;
  const int j1 = min(j0 + part_rows, held);
  float2 x[kKeys][4];
  float w[kKeys];
  auto load = [&](int from) {
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
      const int j = from + k * 128 + threadIdx.x;
      const float* src = p.scores + (plane + j) * p.score_rows;
#pragma unroll
      for (int r = 0; r < 4; ++r) x[k][r] = make_float2(-INFINITY, -INFINITY);
      if (j < j1) {
        if ((p.score_rows & 3) == 0) {
#pragma unroll
          for (int r = 0; r < 4; r += 2)
            if (2 * r < p.score_rows) {
              const float4 v = reinterpret_cast<const float4*>(src)[r / 2];
              x[k][r] = make_float2(v.x, v.y);
              x[k][r + 1] = make_float2(v.z, v.w);
            }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (2 * r < p.score_rows) x[k][r] = reinterpret_cast<const float2*>(src)[r];
        }
      }
      w[k] = j < j1 ? c.weight[plane + j] : 0.f;
    }
  };
  load(j0);
  __shared__ float2 s_lse[4];  // of 8 query rows, and the rows each sees
  __shared__ int2 s_end[4];
  for (int row = warp; row < 8; row += 4) {
    float mx = -INFINITY, sum = 0.f;
    if (row < n_rows) {
      size_t first;
      int n;
      slots_of(h * p.row_blocks + row / kRows, first, n);
      const float2* ml = p.part_ml + first * kRows + row % kRows;
      for (int s = lane; s < n; s += 32) mx = fmaxf(mx, ml[static_cast<size_t>(s) * kRows].x);
#pragma unroll
      for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, k));
      const float ref = mx == -INFINITY ? 0.f : mx;
      for (int s = lane; s < n; s += 32) {
        const float2 v = ml[static_cast<size_t>(s) * kRows];
        sum += v.y * ptx::ex2(v.x - ref);
      }
#pragma unroll
      for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(~0u, sum, k);
    }
    if (lane == 0) {
      reinterpret_cast<float*>(s_lse)[row] = sum != 0.f ? mx + log2f(sum) : INFINITY;
      reinterpret_cast<int*>(s_end)[row] =
          row < n_rows ? rows_seen(p, held, n_tok, row / p.group) : 0;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int from = j0; from < j1; from += kJoinKeys) {
    if (from > j0) load(from);
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
      const int j = from + k * 128 + threadIdx.x;
      float sum = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float2 lse = s_lse[r];
        const int2 end = s_end[r];
        // (by its place, not by its score of -inf: the lse may be NaN)
        if (2 * r < p.score_rows)
          sum += (j < end.x ? ptx::ex2(x[k][r].x - lse.x) : 0.f) +
                 (j < end.y ? ptx::ex2(x[k][r].y - lse.y) : 0.f);
      }
      if (j < j1) c.weight[plane + j] = w[k] + sum;
    }
  }
}

// Weights drawn by 9 to 64 query rows: one more pass over K, its scores now against
// known log-sum-exps. Reads D / 2 + D / 16 bytes a cache row, where leaving the scores
// for the join moves 8 bytes a cache row per query row (32 rows, 8 x 8 x 32768: 306 us
// in all against 200). A warp owns its cache rows, so there are no atomics.
template <int D>
struct DecodeWeightShape {
  static constexpr int kTile = 32, kWarps = 4, kStages = 4, kNt = 8;
  static constexpr int kCodes = kTile * D / 2, kScales = kTile * D / 16;
  static constexpr int kStageBytes = kCodes + kScales;
  static constexpr int kOffQ = kWarps * kStages * kStageBytes;  // fragments of 64 rows
  static constexpr int kOffSl = kOffQ + 64 * D * 2;             // score factor, -lse
  static constexpr int kOffBar = kOffSl + 64 * 8;
  static constexpr int kSmem = kOffBar + kWarps * kStages * 8 + 16;
  static constexpr int kBlocksPerSm = 4;
};

template <int D, int kDtype>
__global__ void __launch_bounds__(128, 4)
    kv4_decode_weight_kernel(const __grid_constant__ Kv4AttendParams p) {
  using S = DecodeWeightShape<D>;
  constexpr int KS = D / 16, KW = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  const Kv4& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tig = lane & 3;
  const uint32_t sbase = ptx::smem_addr(smem);
  const uint32_t ring = sbase + warp * S::kStages * S::kStageBytes;
  const uint32_t bars = sbase + S::kOffBar + warp * S::kStages * 8;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kSmem - 16);
  float2* s_row = reinterpret_cast<float2*>(smem + S::kOffSl);
  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < S::kStages; ++s) ptx::mbar_init(bars + 8 * s, 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  __threadfence();  // the lengths: as in the join
  const Line line = line_of(p, gridDim.x, S::kTile, lane);
  int at = min(static_cast<long long>(blockIdx.x) * line.share,
               static_cast<long long>(line.total));
  const int stop = min(at + line.share, line.total);
  int b = 0, b0 = 0, per_unit = 1;
  if (at < stop) find_sequence(p, at, S::kTile, lane, b, b0, per_unit);
  begin_early();
  wait_for_previous();  // the join's log-sum-exps
  int st = 0, pending = 0;
  uint32_t phase = 0;
  bool ok = true;

  while (at < stop) {
    if (at >= b0 + per_unit * c.H) find_sequence(p, at, S::kTile, lane, b, b0, per_unit);
    const int h = (at - b0) / per_unit;
    const int t0 = at - b0 - h * per_unit;
    const int t1 = min(per_unit, t0 + (stop - at));
    const int held = rows_held(c, b), n_tok = tokens_of(p.counts, b, p.T);
    const int n_rows = n_tok * p.group, n_nt = (n_rows + 7) / 8;
    const size_t plane = (static_cast<size_t>(b) * c.H + h) * c.N;
    auto fill = [&](int tile, int stage) {
      const uint32_t bar = bars + 8 * stage;
      if (lane == 0) ptx::mbar_arrive_expect_tx(bar, S::kStageBytes);
      __syncwarp();
      const size_t row = plane + static_cast<size_t>(tile) * S::kTile;
      if (lane < 2)
        bulk_load(ring + stage * S::kStageBytes + (lane == 0 ? 0 : S::kCodes),
                  lane == 0 ? c.k_codes + row * (D / 2) : c.k_scales + row * (D / 16),
                  lane == 0 ? S::kCodes : S::kScales, bar);
    };
    int next = t0 + warp;
    for (int s = 0; s < S::kStages && ok && next < t1; ++s, next += S::kWarps, ++pending)
      fill(next, st + s < S::kStages ? st + s : st + s - S::kStages);
    __syncthreads();  // the previous unit is done with the queries
    for (int nt = warp; nt < n_nt; nt += S::kWarps) {
      const int row = nt * 8 + g;
      uint4 qw[D / 32];
      uint32_t qf[KS][2];
      load_query<D>(p, b, h, row, row < n_rows, tig, qw);
      const float scale = query_fragments<D, kDtype>(qw, p.scale_log2, qf);
#pragma unroll
      for (int k = 0; k < KS; ++k)
        *reinterpret_cast<uint2*>(smem + S::kOffQ + ((nt * KS + k) * 32 + lane) * 8) =
            make_uint2(qf[k][0], qf[k][1]);
      if (tig == 0)  // rows that are not there draw nothing
        s_row[row] = make_float2(
            scale, row < n_rows
                       ? p.row_nlse[(static_cast<size_t>(b) * c.H + h) * p.score_rows + row]
                       : -INFINITY);
    }
    __syncthreads();
    const int open = p.causal ? max(held - n_tok + 1, 0) : held;

    for (int t = t0 + warp; ok && t < t1; t += S::kWarps) {
      const int j0 = t * S::kTile;
      // the weights so far, asked for ahead: lane (g, 0) owns rows g, g + 8 of each half
      float w[2][2];
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          const int j = j0 + sub * 16 + tile_row<D>(g + 8 * hi);
          w[sub][hi] = tig == 0 && j < held ? c.weight[plane + j] : 0.f;
        }
      ok = __all_sync(~0u, ptx::mbar_wait(bars + 8 * st, phase, abort_flag, c.status));
      if (!ok) break;
      --pending;
      const uint32_t kc = ring + st * S::kStageBytes;
      KeyWords<D> kw;
      kw.load(kc, kc + S::kCodes, g, tig);
      uint32_t a[KW][2][2][4];
#pragma unroll
      for (int i = 0; i < KW; ++i) kw.convert(i, a[i]);
      __syncwarp();  // every lane has read the stage
      if (next < t1) {
        fill(next, st);
        next += S::kWarps;
        ++pending;
      }
      if (++st == S::kStages) {
        st = 0;
        phase ^= 1u;
      }
      const bool edge = j0 + S::kTile > open;
      float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 1
      for (int nt = 0; nt < n_nt; ++nt) {
        float s[2][4];
#pragma unroll
        for (int sub = 0; sub < 2; ++sub)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[sub][i] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint2 f = lds64(sbase + S::kOffQ + ((nt * KS + k) * 32 + lane) * 8);
          const int i = k >> 1, half = k & 1;
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
            mma_16816(s[sub], a[i][sub][0][2 * half], a[i][sub][1][2 * half],
                      a[i][sub][0][2 * half + 1], a[i][sub][1][2 * half + 1], f.x, f.y);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = nt * 8 + 2 * tig + i;
          const float2 row = s_row[r];
          const int end = edge ? rows_seen(p, held, n_tok, r / p.group) : held;
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
              const float e = ptx::ex2(fmaf(s[sub][2 * hi + i], row.x, row.y));
              const int j = j0 + sub * 16 + tile_row<D>(g + 8 * hi);
              sum[sub][hi] += edge && j >= end ? 0.f : e;
            }
        }
      }
#pragma unroll
      for (int sub = 0; sub < 2; ++sub)
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          float x = sum[sub][hi];
          x += __shfl_xor_sync(~0u, x, 1);
          x += __shfl_xor_sync(~0u, x, 2);
          const int j = j0 + sub * 16 + tile_row<D>(g + 8 * hi);
          if (tig == 0 && j < held) c.weight[plane + j] = w[sub][hi] + x;
        }
    }
    at += t1 - t0;
  }
  // after an abort: copies still under way land before the block's memory goes
  volatile int none = 0;
  for (; pending > 0; --pending) {
    ptx::mbar_wait(bars + 8 * st, phase, &none, c.status);
    if (++st == S::kStages) {
      st = 0;
      phase ^= 1u;
    }
  }
}

}  // namespace sa
