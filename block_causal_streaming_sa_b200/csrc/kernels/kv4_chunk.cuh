// Attention of many query rows over a 4-bit cache: chunks and prompts.
//
// Bound by the matrix and exponential units and by what feeds them: 4 D flop and one
// exponential per (query row, cache row). The design is the chunk-cache attention's
// (query tiles of 128 rows ping-pong over every K / V tile, S and O in tensor memory,
// P written over S), with these differences:
//  * Two SMs work as a pair (cta_group::2, tiles of 256 query rows): each holds half of
//    every K tile (64 of its 128 rows) and of every V tile (half the columns), which the
//    tensor cores of both read. Alone, an SM's products read 192 KB of shared memory per
//    step against the 2048 cycles they take, all that shared memory delivers, and
//    the conversion's 64 KB came on top (3700 cycles a step measured); paired they read
//    128 KB and write 32.
//  * A key tile's scores come as two halves of 64 rows in the two halves of a query
//    tile's 128 columns. Softmax goes through them one after the other and puts P where
//    half a's scores were; the next tile's half a goes where half b's were as soon as
//    they have been read, and its half b over P once P V is done. So there are always
//    scores to work on: with whole tiles, a tile's softmax (2100 cycles) and its products
//    (1280 with their latencies) took turns, 3400 a step where each pipe needs 2048.
//  * K and V arrive as codes. A warpgroup of its own reads them from global memory
//    one tile ahead into registers, converts and scales them (exact in fp16) and
//    stores them in the swizzled layout the products read. Converting on the fly reads
//    288 bytes a row and head instead of the 512 + 800 that a 16-bit copy made ahead
//    would move, and needs no copy of the cache.
//  * Queries are staged once per call (kv4_stage_kernel): scaled to fp16 by a power
//    of two per row and stored as the 128-row tiles' shared memory images, so a tile
//    is one bulk copy whatever the tensor's strides are. They are double-buffered: the
//    next item's arrive while this one is worked on.
//  * Work is one line of (512 query rows, key tile) steps cut into equal ranges, one
//    a pair of SMs, so neither causal masks, ragged lengths nor the last round leave
//    SMs idle. A pair writes whole items to O; of an item that lies in several ranges
//    each pair leaves an fp32 partial result, at most two a pair, which
//    kv4_chunk_join_kernel merges in the order of the ranges.
//  * Registers: 512 threads launched at 128; softmax warpgroups 192, conversion 72,
//    the issuing warpgroup 56 (their sum is the launch's).
//
// Measured, replayed: 6120 x 24480 rows, 12 heads, D 128: 0.72 ms (1280 TFLOP/s) on a part that
// was idle, 0.78 ms (1180) once its clock has settled under this load; 3100 cycles a step, of
// which the softmax warps work 2750.
#pragma once

#include <type_traits>

#include "kv4_params.cuh"

namespace sa {

constexpr int kItemRows = 512;  // query rows of an item: two tiles of 256, each over two SMs

template <int D>
struct ChunkShape {
  static constexpr int BN = 128;            // cache rows of a key tile
  static constexpr int kTile = 128 * D * 2; // bytes of a query tile's rows in one SM
  static constexpr int kBox = 128 * 128;    // bytes of 64 columns of 128 rows
  static constexpr int kHalf = 128 * D;     // bytes of half a K or V tile
  static constexpr int NSTAGE = 6;          // K0 K1 V0 K2 V1 ..: K runs one tile ahead
  static constexpr int kThreads = 512;
  static constexpr int kRegsSoftmax = 192, kRegsConvert = 72, kRegsIssue = 56;
  static_assert(2 * kRegsSoftmax + kRegsConvert + kRegsIssue <= 512, "launched at 128 each");
  static constexpr int kOffQ = 0;           // [buffer][tile]
  static constexpr int kOffKV = 4 * kTile;
  static constexpr int kOffBar = kOffKV + NSTAGE * kHalf;
  static constexpr int kSmem = kOffBar + 256 + 1024;  // + alignment slack
  static constexpr int kTmemCols = 512;
  static constexpr uint32_t kIdescQK = ptx::idesc_f32acc(256, 64, 0, 0);  // fp16
  static constexpr uint32_t kIdescPV = ptx::idesc_f32acc(256, D, 0, 1);   // fp16, V MN-major
  // Tensor memory: per query tile two 64-column halves for scores and P, and O.
  __host__ __device__ static constexpr int col_x(int i, int half) { return i * 128 + half * 64; }
  __host__ __device__ static constexpr int col_o(int i) { return 256 + i * D; }
  // Barriers: the leader's (block 0 of the pair) collect arrivals of both blocks, the
  // others are each block's own.
  __host__ __device__ static constexpr int FULL(int s) { return s; }  // leader
  __host__ __device__ static constexpr int EMPTY(int s) { return NSTAGE + s; }
  __host__ __device__ static constexpr int SA(int i) { return 2 * NSTAGE + i; }
  __host__ __device__ static constexpr int SB(int i) { return 2 * NSTAGE + 2 + i; }
  __host__ __device__ static constexpr int READ(int i) { return 2 * NSTAGE + 4 + i; }   // leader
  __host__ __device__ static constexpr int PFULL(int i) { return 2 * NSTAGE + 6 + i; }  // leader
  __host__ __device__ static constexpr int OFINAL(int i) { return 2 * NSTAGE + 8 + i; }
  __host__ __device__ static constexpr int QLOAD(int q) { return 2 * NSTAGE + 10 + q; }
  __host__ __device__ static constexpr int QREADY(int q) { return 2 * NSTAGE + 12 + q; }  // leader
  __host__ __device__ static constexpr int QEMPTY(int q) { return 2 * NSTAGE + 14 + q; }
  __host__ __device__ static constexpr int DRAIN() { return 2 * NSTAGE + 16; }
  static_assert((2 * NSTAGE + 17) * 8 <= 240, "barrier area");
  static_assert(kSmem <= 232448, "shared memory");
};

// Offset of 16-byte piece c of row r in a 128-byte-swizzled K-major tile of 128 rows.
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
  return static_cast<uint32_t>((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z,
                                       uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z),
               "r"(w)
               : "memory");
}

// Products of a pair of SMs. Shared memory descriptors are given by their low words:
// the high word (stride between groups of eight rows, version 1, swizzle) is the
// same for all tiles of a kind, and 64-bit descriptors kept ready would not fit the
// issuing warp's registers.
constexpr uint32_t kDescHi128 = 64u | 1u << 14 | 2u << 29;  // 1024 bytes, 128-byte swizzle
constexpr uint32_t kDescHi64 = 32u | 1u << 14 | 4u << 29;   // 512 bytes, 64-byte swizzle

__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo_bytes) {
  return ((addr >> 4) & 0x3FFFu) | (lbo_bytes >> 4) << 16;
}

__device__ __forceinline__ void umma2_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                         bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(kDescHi128)
      : "memory");
}

__device__ __forceinline__ void umma2_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t b_hi,
                                         uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(b_hi)
      : "memory");
}

// Arrive on this barrier of both blocks when all earlier products have finished.
__device__ __forceinline__ void umma2_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// The leader's copy of a barrier, and an arrival on it from either block. What is handed
// over stays on the arriving SM: its shared memory (written, then fenced for the
// asynchronous proxy) and tensor memory (ordered by tcgen05.wait and the fence before
// the arrival) are read by that SM's own tensor core. So the release is the block's
// (the default); one for the cluster took ~1000 cycles, between every P and its product.
__device__ __forceinline__ uint32_t leader_addr(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void arrive_leader(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// True in one lane of the (whole) warp, the same one at every call.
__device__ __forceinline__ bool ptx_elect() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Bounded wait on a barrier that the other block may arrive on.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity,
                                             volatile int* abort_flag, unsigned* status) {
  auto done = [&]() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (done()) return true;
  const long long t0 = clock64();
  while (true) {
    if (done()) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > ptx::kWaitCycles) {
      *abort_flag = 1;
      atomicOr(status, kDevErrTimeout);
      return false;
    }
  }
}

// Key tiles that item `item` (query rows 512 item ..) of sequence b goes through.
__device__ __forceinline__ int item_tiles(const Kv4AttendParams& p, int held, int n_tok, int item) {
  const int n_rows = n_tok * p.group;
  if (kItemRows * item >= n_rows) return 0;
  const int last = min(kItemRows * (item + 1), n_rows) - 1;
  return (rows_seen(p, held, n_tok, last / p.group) + 127) / 128;
}

// Query tiles that draw weight from key tile `kt`: from the tile of the first token
// that sees one of its rows on. `from` is that tile.
__device__ __forceinline__ int weight_steps(const Kv4AttendParams& p, int held, int n_tok, int kt,
                                            int& from) {
  from = 0;
  if (kt * 128 >= held) return 0;
  const int tiles = (n_tok * p.group + 127) / 128;
  if (p.causal) from = max(kt * 128 - (held - n_tok), 0) * p.group / 128;
  return max(tiles - from, 0);
}

// Queries to fp16 tiles, per-row scales, and the lines of steps. Block (x, h, b)
// stages tile x; blocks (q_tiles, 0, 0) and (q_tiles + 1, 0, 0) lay the lines.
template <int D, int kDtype>
__global__ void __launch_bounds__(256)
    kv4_stage_kernel(const __grid_constant__ Kv4AttendParams p) {
  constexpr int C = D / 8;  // 16-byte pieces of a row
  const Kv4& c = p.c;
  // In this order: the next kernel takes all of an SM's tensor memory as soon as it begins,
  // which a kernel in front of this one that lets its successor begin early may still be
  // about to allocate; each would wait for the other.
  wait_for_previous();
  begin_early();
  if (static_cast<int>(blockIdx.x) >= p.q_tiles) {
    if (blockIdx.y != 0 || blockIdx.z != 0) return;
    if (static_cast<int>(blockIdx.x) == p.q_tiles) {
      for (int b = threadIdx.x; b < c.B; b += 256)
        check_order(p, b, tokens_of(p.counts, b, p.T));
      lay_line(
          p.line, c.B, c.H,
          [&](int b) {
            return (tokens_of(p.counts, b, p.T) * p.group + kItemRows - 1) / kItemRows;
          },
          [&](int b, int i) {
            return item_tiles(p, rows_held(c, b), tokens_of(p.counts, b, p.T), i);
          });
    } else {
      lay_line(
          p.weight_line, c.B, c.H, [&](int b) { return (rows_held(c, b) + 127) / 128; },
          [&](int b, int i) {
            int from;
            return weight_steps(p, rows_held(c, b), tokens_of(p.counts, b, p.T), i, from);
          });
    }
    return;
  }
  const int b = blockIdx.z, h = blockIdx.y, tile = blockIdx.x;
  const int held = rows_held(c, b), n_tok = tokens_of(p.counts, b, p.T);
  const int n_rows = n_tok * p.group;
  if (tile * 128 >= n_rows) return;
  // no block goes to an item without tiles
  const bool empty = item_tiles(p, held, n_tok, tile * 128 / kItemRows) == 0;
  const size_t tile_id = (static_cast<size_t>(b) * c.H + h) * p.q_tiles + tile;
  uint8_t* dst = p.q_img + tile_id * (128 * D * 2);
  constexpr int kAhead = 4;  // loads under way a thread
  static_assert(128 * C % (256 * kAhead) == 0);
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < 128 * C; i0 += 256 * kAhead) {
    uint4 in[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * 256, row = tile * 128 + i / C;
      const int t = row / p.group, hq = h * p.group + row % p.group;
      in[k] = make_uint4(0u, 0u, 0u, 0u);
      if (row < n_rows)
        in[k] = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q.data) +
                                               b * p.q.sb + t * p.q.st + hq * p.q.sh)[i % C];
    }
#pragma unroll
    for (int step = 0; step < kAhead; ++step) {
      const int i = i0 + step * 256, r = i / C, piece = i % C, row = tile * 128 + r;
      const int t = row / p.group, hq = h * p.group + row % p.group;
      const uint4 w = in[step];
      const float2 v[4] = {unpack2<kDtype>(w.x), unpack2<kDtype>(w.y), unpack2<kDtype>(w.z),
                           unpack2<kDtype>(w.w)};
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) amax = fmaxf(amax, fmaxf(fabsf(v[k].x), fabsf(v[k].y)));
#pragma unroll
      for (int k = 1; k < C; k <<= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, k));
      const float f = row_factor(amax);
      uint32_t x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = pack2<SA_DTYPE_FP16>(v[k].x * f, v[k].y * f);
      *reinterpret_cast<uint4*>(dst + tile_offset(r, piece)) = make_uint4(x[0], x[1], x[2], x[3]);
      if (piece == 0)
        p.row_scale[tile_id * 128 + r] = row < n_rows ? score_factor(p.scale_log2, f) : 0.f;
      if (row >= n_rows) {
        if (piece == 0) p.row_nlse[tile_id * 128 + r] = -INFINITY;  // such rows draw no weight
      } else if (empty) {
        uint16_t* o = static_cast<uint16_t*>(p.o.data) + b * p.o.sb + t * p.o.st + hq * p.o.sh;
        *reinterpret_cast<uint4*>(o + piece * 8) = make_uint4(0u, 0u, 0u, 0u);
        if (piece == 0) {
          if (p.lse != nullptr)
            p.lse[(static_cast<size_t>(b) * p.heads + hq) * p.T + t] = -INFINITY;
          p.row_nlse[tile_id * 128 + r] = -INFINITY;
        }
      }
    }
  }
}

// One query row's result: O / l to its place, or the partial row. A function of its
// own so that its registers do not add to the score loop's.
template <int D, int kDtype>
__device__ __noinline__ void chunk_epilogue(const Kv4AttendParams& p, uint32_t tO, float m,
                                            float lsum, bool whole, size_t slot, int b, int h,
                                            int row, int n_rows) {
  if (!whole) {
    const int r = row % kItemRows;
    float4* dst = reinterpret_cast<float4*>(p.part_o) + slot * (D / 4) * kItemRows + r;
#pragma unroll 1
    for (int j = 0; j < D / 32; ++j) {
      uint32_t o[32];
      ptx::tmem_ld32(tO + j * 32, o);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 32; k += 4)  // [D / 4][512 rows][4]: a warp's stores are contiguous
        dst[static_cast<size_t>(j * 8 + k / 4) * kItemRows] =
            make_float4(__uint_as_float(o[k]), __uint_as_float(o[k + 1]),
                        __uint_as_float(o[k + 2]), __uint_as_float(o[k + 3]));
    }
    p.part_ml[slot * kItemRows + r] = make_float2(m, lsum);
    return;
  }
  const float inv = lsum == 0.f ? 0.f : 1.f / lsum;  // NaN stays NaN
  const int t = row / p.group, hq = h * p.group + row % p.group;
  // 32 columns at a time; four lanes exchange theirs, so that a store covers 64 bytes of
  // 8 rows. With each lane storing its own row the 32 lines of an instruction took 4000
  // of the epilogue's 6000 cycles.
  const int lane = threadIdx.x & 31, piece = lane & 3;
  const long long own = row < n_rows ? b * p.o.sb + t * p.o.st + hq * p.o.sh : -1;
  long long off[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) off[k] = __shfl_sync(~0u, own, (lane & ~3) + k);
  uint16_t* dst = static_cast<uint16_t*>(p.o.data) + piece * 8;
#pragma unroll 1
  for (int j = 0; j < D / 32; ++j) {
    uint32_t o[32];
    ptx::tmem_ld32(tO + j * 32, o);
    ptx::tmem_wait_ld();
    uint32_t v[4][4];  // this row's 16-byte pieces, then piece `piece` of the four rows
#pragma unroll
    for (int k = 0; k < 16; ++k)
      v[k >> 2][k & 3] = pack2<kDtype>(__uint_as_float(o[2 * k]) * inv,
                                       __uint_as_float(o[2 * k + 1]) * inv);
#pragma unroll
    for (int bit = 1; bit < 4; bit <<= 1)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if ((k & bit) == 0)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const bool upper = (lane & bit) != 0;
            const uint32_t got =
                __shfl_xor_sync(~0u, upper ? v[k][w] : v[k | bit][w], bit);
            v[k][w] = upper ? got : v[k][w];
            v[k | bit][w] = upper ? v[k | bit][w] : got;
          }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (off[k] >= 0)
        *reinterpret_cast<uint4*>(dst + off[k] + j * 32) =
            make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
  }
  if (row < n_rows) {
    const float lse2 = lsum == 0.f ? -INFINITY : m + log2f(lsum);
    if (p.lse != nullptr)
      p.lse[(static_cast<size_t>(b) * p.heads + hq) * p.T + t] = lse2 * 0.69314718055994531f;
    p.row_nlse[((static_cast<size_t>(b) * p.c.H + h) * p.q_tiles) * 128 + row] =
        lsum == 0.f ? -INFINITY : -lse2;
  }
}

// Rare steps of the softmax, functions of their own so that their registers do not add
// to the score loop's: scale D columns of fp32, and 32 columns of fp16 pairs.
template <int D>
__device__ __noinline__ void chunk_scale_columns(uint32_t tO, float alpha) {
#pragma unroll 1
  for (int j = 0; j < D / 32; ++j) {
    uint32_t o[32];
    ptx::tmem_ld32(tO + j * 32, o);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
    ptx::tmem_st32(tO + j * 32, o);
  }
  ptx::tmem_wait_st();
}

__device__ __noinline__ void chunk_scale_p(uint32_t tP, float alpha) {
  uint32_t v[32];
  ptx::tmem_ld32(tP, v);
  ptx::tmem_wait_ld();
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const float2 f = unpack2<SA_DTYPE_FP16>(v[k]);
    v[k] = pack2<SA_DTYPE_FP16>(f.x * alpha, f.y * alpha);
  }
  ptx::tmem_st32(tP, v);
  ptx::tmem_wait_st();
}

// Codes of a thread's part of a tile, read ahead: 16-byte pieces (32 codes), piece
// i * 128 + thread of `P` a row, with their two scales.
template <int N>
struct ConvertRegs {
  uint4 w[N];
  uint32_t sc[N];
};

// Pieces piece0 .. piece0 + P - 1 of rows row0 + key(row).
template <int D, int P, int N, typename F>
__device__ __forceinline__ void convert_load(ConvertRegs<N>& x, const uint8_t* codes,
                                             const uint8_t* scales, size_t row0, int piece0,
                                             int tid, F key) {
  const uint4* src = reinterpret_cast<const uint4*>(codes + row0 * (D / 2)) + piece0;
  const uint16_t* sc = reinterpret_cast<const uint16_t*>(scales + row0 * (D / 16)) + piece0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = (i * 128 + tid) / P, piece = (i * 128 + tid) % P;
    x.w[i] = src[key(row) * (D / 32) + piece];
    x.sc[i] = sc[key(row) * (D / 32) + piece];
  }
}

// Into a tile in shared memory, `offset(row, 16-byte piece)` from `tile`; cache rows
// from `valid` on become zeros (what lies there may be anything, and a scale may be NaN).
template <int P, int N, typename F, typename G>
__device__ __forceinline__ void convert_store(const ConvertRegs<N>& x, uint32_t tile, int tid,
                                              int valid, F key, G offset) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = (i * 128 + tid) / P, piece = (i * 128 + tid) % P;
    const uint32_t bytes = key(row) < valid ? x.sc[i] : 0u;
    const uint32_t s0 = scale_f16x2(bytes & 255u), s1 = scale_f16x2(bytes >> 8);
    const uint32_t w[4] = {x.w[i].x, x.w[i].y, x.w[i].z, x.w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h[4];
      codes_to_f16(w[j], h);
      const uint32_t s = j < 2 ? s0 : s1;
      sts128(tile + offset(row, piece * 4 + j), mul_f16x2(h[0], s), mul_f16x2(h[1], s),
             mul_f16x2(h[2], s), mul_f16x2(h[3], s));
    }
  }
}

template <int D, int kDtype>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(512, 1)
    kv4_chunk_kernel(const __grid_constant__ Kv4AttendParams p) {
  using S = ChunkShape<D>;
  extern __shared__ uint8_t smem_raw[];
  const Kv4& c = p.c;
  const uint32_t raw = ptx::smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t sbase = ptx::smem_addr(smem);  // the same offset in both blocks
  auto bar = [&](int i) { return sbase + S::kOffBar + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffBar + 240);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffBar + 248);
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x & 1;  // 0: the leader, which issues the products
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::NSTAGE; ++s) {
      ptx::mbar_init(bar(S::FULL(s)), 8);  // four converting warps of each block
      ptx::mbar_init(bar(S::EMPTY(s)), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(S::SA(i)), 1);
      ptx::mbar_init(bar(S::SB(i)), 1);
      ptx::mbar_init(bar(S::READ(i)), 8);  // four warps of each block
      ptx::mbar_init(bar(S::PFULL(i)), 8);
      ptx::mbar_init(bar(S::OFINAL(i)), 1);
      ptx::mbar_init(bar(S::QLOAD(i)), 1);
      ptx::mbar_init(bar(S::QREADY(i)), 2);
      ptx::mbar_init(bar(S::QEMPTY(i)), 1);
    }
    ptx::mbar_init(bar(S::DRAIN()), 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     ptx::smem_addr(tmem_slot)),
                 "r"(S::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  ptx::tc_fence_before();
  __syncthreads();
  cluster_sync();  // both blocks' barriers are there
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  wait_for_previous();  // staged queries and schedule

  LineWalk walk = line_range(p.line, c.B, pair, pairs);
  auto wait = [&](int which, uint32_t parity) {
    return wait_cluster(bar(which), parity, abort_flag, c.status);
  };
  // Tiles of 256 query rows of the walk's item: 1 or 2.
  auto item_halves = [&]() {
    return tokens_of(p.counts, walk.b, p.T) * p.group > walk.item * kItemRows + 256 ? 2 : 1;
  };

  if (warp >= 12) {
    ptx::setmaxnreg_dec<S::kRegsIssue>();
    if (warp == 12 && rank == 0) {
      // ------------------------------------------------------------ MMA issuer (leader)
      // The whole warp goes through the loop, so that the compiler sees uniform values and
      // keeps them in uniform registers, which the product instructions take their
      // operands from; one lane issues. A single thread's loop had to move every
      // operand there (92 cycles a product instead of the 64 it runs).
      const bool issues = ptx_elect();
      int stage = 0, item = 0;
      uint32_t phase = 0, sm_phase[2] = {0u, 0u};
      bool ok = true;
      auto all_wait = [&](int which, uint32_t parity) {
        return __all_sync(~0u, wait(which, parity)) != 0;
      };
      auto take = [&](int& s_out) -> bool {
        s_out = stage;
        const bool r = all_wait(S::FULL(stage), phase);
        if (++stage == S::NSTAGE) {
          stage = 0;
          phase ^= 1u;
        }
        return r;
      };
      // Scores of half `b` of a key tile (32 of each block's 64 rows) into half `x`.
      auto issue_s = [&](auto tile, int sk, int b, int x) {
        constexpr int i = decltype(tile)::value;
        const uint32_t qa = desc_lo(sbase + S::kOffQ + ((item & 1) * 2 + i) * S::kTile, 16);
        const uint32_t kb = desc_lo(sbase + S::kOffKV + sk * S::kHalf + b * 32 * 128, 16);
        if (issues) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)  // 64 columns: a box of 128 (Q) or 64 (K) rows
            umma2_ss(tmem + S::col_x(i, 0) + x * 64,
                     qa + (((kk >> 2) * S::kBox + (kk & 3) * 32) >> 4),
                     kb + (((kk >> 2) * (S::kBox / 2) + (kk & 3) * 32) >> 4), S::kIdescQK,
                     kk > 0);
          umma2_commit(bar(b == 0 ? S::SA(i) : S::SB(i)));
        }
      };
      auto issue_pv = [&](auto tile, int sv, int x, bool accumulate) {
        constexpr int i = decltype(tile)::value;
        // D / 2 columns of V a block: rows of 128 (D 64: 64) bytes
        const uint32_t vb = desc_lo(sbase + S::kOffKV + sv * S::kHalf, 16);
        if (issues) {
#pragma unroll
          for (int kk = 0; kk < S::BN / 16; ++kk)
            umma2_ts(tmem + S::col_o(i), tmem + S::col_x(i, 0) + x * 64 + kk * 8,
                     vb + (kk * 16 * D >> 4),
                     D == 128 ? kDescHi128 : kDescHi64, S::kIdescPV, accumulate || kk > 0);
        }
      };
      auto commit = [&](int which) {
        if (issues) umma2_commit(bar(which));
      };
      constexpr std::integral_constant<int, 0> tile0;
      constexpr std::integral_constant<int, 1> tile1;
      while (ok && walk.next(p.line, c.B)) {
        const bool two = item_halves() == 2;
        const int t0 = __shfl_sync(~0u, walk.t0, 0), t1 = __shfl_sync(~0u, walk.t1, 0);
        int sk = 0, sv = 0;
        ok = all_wait(S::QREADY(item & 1), (item >> 1) & 1) && take(sk);
        if (!ok) break;
        ptx::tc_fence_after();
        issue_s(tile0, sk, 0, 0);
        issue_s(tile0, sk, 1, 1);
        if (two) {
          issue_s(tile1, sk, 0, 0);
          issue_s(tile1, sk, 1, 1);
        }
        commit(S::EMPTY(sk));
        int x = 0;  // half of P (and of half a's scores) of this tile
        for (int t = t0; ok && t < t1; ++t, x ^= 1) {
          const bool more = t + 1 < t1;
          if (!more) commit(S::QEMPTY(item & 1));  // its last products are issued
          ok = (!more || take(sk)) && take(sv);
          // One query tile: half a of the next scores, P V, half b of the next scores.
          auto step = [&](auto tile, bool last) {
            constexpr int i = decltype(tile)::value;
            ok = ok && all_wait(S::READ(i), sm_phase[i]);
            if (!ok) return;
            ptx::tc_fence_after();
            if (more) issue_s(tile, sk, 0, x ^ 1);
            ok = all_wait(S::PFULL(i), sm_phase[i]);
            if (!ok) return;
            sm_phase[i] ^= 1u;
            ptx::tc_fence_after();
            issue_pv(tile, sv, x, t > t0);
            if (last) commit(S::EMPTY(sv));
            if (more)
              issue_s(tile, sk, 1, x);
            else
              commit(S::OFINAL(i));
          };
          step(tile0, !two);
          if (two) step(tile1, true);
          if (ok && more) commit(S::EMPTY(sk));
        }
        ++item;
      }
      commit(S::DRAIN());
    }
    if (warp == 13 && lane == 0) {
      // ------------------------------------------------------------ query tiles
      uint32_t item = 0;
      bool ok = true;
      volatile int none = 0;
      while (ok && walk.next(p.line, c.B)) {
        const int q = item & 1, n_rows = tokens_of(p.counts, walk.b, p.T) * p.group;
        ok = wait(S::QEMPTY(q), ((item >> 1) & 1) ^ 1u);
        if (!ok) break;
        // tiles rank and 2 + rank of the item's four, as far as they have rows
        const int first = walk.item * 4 + rank;
        const int tiles = n_rows > (first + 2) * 128 ? 2 : n_rows > first * 128 ? 1 : 0;
        ptx::mbar_arrive_expect_tx(bar(S::QLOAD(q)), tiles * S::kTile);
        for (int i = 0; i < tiles; ++i)
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, "
              "[%3];" ::"r"(sbase + S::kOffQ + (q * 2 + i) * S::kTile),
              "l"(p.q_img + ((static_cast<size_t>(walk.b) * c.H + walk.h) * p.q_tiles + first +
                             2 * i) *
                                S::kTile),
              "r"(S::kTile), "r"(bar(S::QLOAD(q)))
              : "memory");
        // (also after an abort: the copies land before the block can end)
        ok = ptx::mbar_wait(bar(S::QLOAD(q)), (item >> 1) & 1, &none, c.status);
        ptx::fence_proxy_async_smem();
        arrive_leader(leader_addr(bar(S::QREADY(q))));
        ++item;
      }
    }
  } else if (warp >= 8) {
    ptx::setmaxnreg_dec<S::kRegsConvert>();
    // ------------------------------------------------------------ conversion
    // K: rows 32 rank .. of each half of the tile, all columns; V: all rows, columns
    // D / 2 rank ..
    constexpr int PK = D / 32, PV = D / 64, N = D / 64;
    const int tid = threadIdx.x - 256;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    auto publish = [&](const ConvertRegs<N>& x, int valid, auto store) {
      if (!__all_sync(~0u, wait(S::EMPTY(stage), phase ^ 1u))) {
        ok = false;
        return;
      }
      store(x, sbase + S::kOffKV + stage * S::kHalf, valid);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_leader(leader_addr(bar(S::FULL(stage))));
      if (++stage == S::NSTAGE) {
        stage = 0;
        phase ^= 1u;
      }
    };
    auto key_k = [&](int r) { return r + rank * 32 + (r & 32); };
    auto key_v = [](int r) { return r; };
    auto store_k = [&](const ConvertRegs<N>& x, uint32_t tile, int valid) {
      convert_store<PK>(x, tile, tid, valid, key_k, [](int r, int c) {  // boxes of 64 rows
        return static_cast<uint32_t>((c >> 3) * (64 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
      });
    };
    auto store_v = [&](const ConvertRegs<N>& x, uint32_t tile, int valid) {
      convert_store<PV>(x, tile, tid, valid, key_v, [](int r, int c) {
        if constexpr (D == 128) return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
        return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
      });
    };
    while (ok && walk.next(p.line, c.B)) {
      const int held = rows_held(c, walk.b);
      const size_t plane = (static_cast<size_t>(walk.b) * c.H + walk.h) * c.N;
      ConvertRegs<N> kx, vx;
      auto load_k = [&](int t) {
        convert_load<D, PK>(kx, c.k_codes, c.k_scales, plane + t * 128, 0, tid, key_k);
      };
      auto load_v = [&](int t) {
        convert_load<D, PV>(vx, c.v_codes, c.v_scales, plane + t * 128, rank * PV, tid, key_v);
      };
      load_k(walk.t0);
      load_v(walk.t0);
      publish(kx, held - walk.t0 * 128, store_k);
      if (walk.t0 + 1 < walk.t1) load_k(walk.t0 + 1);
      for (int t = walk.t0; ok && t < walk.t1; ++t) {
        if (t + 1 < walk.t1) {
          publish(kx, held - (t + 1) * 128, store_k);
          if (!ok) break;
          if (t + 2 < walk.t1) load_k(t + 2);
        }
        publish(vx, held - t * 128, store_v);
        if (t + 1 < walk.t1) load_v(t + 1);
      }
    }
  } else {
    ptx::setmaxnreg_inc<S::kRegsSoftmax>();
    // ------------------------------------------------------------ softmax
    const int i = warp >> 2;       // query tile of this warpgroup
    const int quarter = warp & 3;  // tensor memory lanes this warp may access
    const int r = quarter * 32 + lane;
    const uint32_t t_lane = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tX = tmem + t_lane + S::col_x(i, 0);
    const uint32_t tO = tmem + t_lane + S::col_o(i);
    const uint32_t read = leader_addr(bar(S::READ(i))), p_full = leader_addr(bar(S::PFULL(i)));
    uint32_t s_phase = 0, items = 0;
    bool ok = true;
    while (ok && walk.next(p.line, c.B)) {
      const int held = rows_held(c, walk.b), n_tok = tokens_of(p.counts, walk.b, p.T);
      const int n_rows = n_tok * p.group;
      if (i >= item_halves()) continue;
      const int tile = walk.item * 4 + 2 * i + rank, row = tile * 128 + r;
      const bool used = tile * 128 < n_rows;  // else this block's rows are not there
      const int end = row < n_rows ? rows_seen(p, held, n_tok, row / p.group) : held;
      const float sl = used ? p.row_scale[((static_cast<size_t>(walk.b) * c.H + walk.h) *
                                           p.q_tiles) * 128 + row]
                            : 0.f;
      float m = -INFINITY, lsum = 0.f;
      for (int t = walk.t0, x = 0; t < walk.t1; ++t, x ^= 1) {
        uint32_t sr[2][32];  // a half's scores
        const uint32_t tA = tX + x * 64, tB = tX + (x ^ 1) * 64;  // a, then P; b
        auto load = [&](int half, uint32_t from) {
          ptx::tc_fence_after();
          if (!used) return;
          ptx::tmem_ld32(from, sr[0]);
          ptx::tmem_ld32(from + 32, sr[1]);
          ptx::tmem_wait_ld();
          const int hi = end - t * 128 - half * 64;
          if (hi < 64) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (j * 32 + k >= hi) sr[j][k] = __float_as_uint(-INFINITY);
          }
        };
        auto row_max = [&]() {  // of the scaled scores
          float mx[8];
#pragma unroll
          for (int a = 0; a < 8; ++a) mx[a] = __uint_as_float(sr[0][a]);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 32; k += 2)
              if (j > 0 || k >= 8)
                mx[(k >> 1) & 7] = ptx::fmax3(mx[(k >> 1) & 7], __uint_as_float(sr[j][k]),
                                              __uint_as_float(sr[j][k + 1]));
          return fmaxf(ptx::fmax3(mx[0], mx[1], mx[2]),
                       fmaxf(ptx::fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]))) *
                 sl;
        };
        // P = 2^(s * scale - m) of a half, m the reference (kRefBelow); returns the row's sum
        auto exponentials = [&](uint32_t to) {
          // a row can meet keys wholly behind its last one before any it sees
          const float nm = m == -INFINITY ? 0.f : -m;
          float rs[8];
#pragma unroll
          for (int a = 0; a < 8; ++a) rs[a] = 0.f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float x0, x1;
              ptx::ffma2(x0, x1, __uint_as_float(sr[j][2 * k]), __uint_as_float(sr[j][2 * k + 1]),
                         sl, sl, nm, nm);
              const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
              const int a = (k & 3) * 2;
              ptx::fadd2(rs[a], rs[a + 1], rs[a], rs[a + 1], p0, p1);
              pk[k] = pack2<SA_DTYPE_FP16>(p0, p1);
            }
            ptx::tmem_st16(to + j * 16, pk);
          }
          return ((rs[0] + rs[1]) + (rs[2] + rs[3])) + ((rs[4] + rs[5]) + (rs[6] + rs[7]));
        };
        // Raises the reference where the half's largest score mx asks for it; returns what
        // the sum and O so far scale with.
        auto raise = [&](float mx) {
          float alpha = 1.f;
          if (mx > m + kRefTop) {
            alpha = ptx::ex2(m - (mx - kRefBelow));
            m = mx - kRefBelow;
          }
          lsum *= alpha;
          if (t > walk.t0) chunk_scale_columns<D>(tO, alpha);  // the first P V overwrites O
          return alpha;
        };

        bool have_b = false;
        auto wait_b = [&]() {
          if (!have_b) ok = __all_sync(~0u, wait(S::SB(i), s_phase));
          have_b = true;
        };
        ok = __all_sync(~0u, wait(S::SA(i), s_phase));
        if (!ok) break;
        load(0, tA);
        float rs = 0.f;
        if (used) {
          const float mx = row_max();
          if (__any_sync(~0u, mx > m + kRefTop)) {
            // half b is issued behind the last P V: with it O stands still
            wait_b();
            if (!ok) break;
            ptx::tc_fence_after();
            raise(mx);
          }
          rs = exponentials(tA);
        }
        wait_b();
        if (!ok) break;
        load(1, tB);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(read);
        if (used) {
          const float mx = row_max();
          if (__any_sync(~0u, mx > m + kRefTop)) {
            // half a's P is scaled too (its second rounding to fp16, in the few tiles where
            // a maximum grows that much)
            ptx::tmem_wait_st();
            const float alpha = raise(mx);
            rs *= alpha;
            chunk_scale_p(tA, alpha);
          }
          lsum += rs + exponentials(tA + 32);
          ptx::tmem_wait_st();
        }
        s_phase ^= 1u;
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(p_full);
      }
      if (!ok) break;
      if (!__all_sync(~0u, wait(S::OFINAL(i), items & 1))) break;
      ++items;
      ptx::tc_fence_after();
      if (used)
        chunk_epilogue<D, kDtype>(p, tO, m, lsum, walk.t0 == 0 && walk.t1 == walk.n,
                                  partial_slot(pair, walk.t0), walk.b, walk.h, row, n_rows);
      ptx::tc_fence_before();
    }
  }

  // Every product has finished before either block gives up its memory.
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    volatile int none = 0;
    wait_cluster(bar(S::DRAIN()), 0, &none, c.status);
  }
  __syncthreads();
  cluster_sync();
  ptx::tc_fence_after();
  if (warp == 12)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(S::kTmemCols)
                 : "memory");
}

// Merge of the items that lie in several ranges, one boundary (blockIdx.x) and 32 of the
// 512 query rows (blockIdx.y) a block.
template <int D, int kDtype>
__global__ void __launch_bounds__(128)
    kv4_chunk_join_kernel(const __grid_constant__ Kv4AttendParams p, int blocks) {
  begin_early();
  wait_for_previous();
  const Kv4& c = p.c;
  SplitItem split;
  if (!split.find(p.line, c.B, blocks, blockIdx.x)) return;
  const LineWalk& w = split.w;
  const int n_tok = tokens_of(p.counts, w.b, p.T), n_rows = n_tok * p.group;
  // four threads a row, D / 4 values each: r = row in the pair
  const int r = blockIdx.y * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  const int row = w.item * kItemRows + r;
  if (row >= n_rows) return;
  float mx = -INFINITY;
  for (int k = split.first; k <= split.last; ++k)
    mx = fmaxf(mx, p.part_ml[split.slot(k) * kItemRows + r].x);
  const float ref = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f;
  constexpr int V = D / 16;  // float4 of a thread
  float4 acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = split.first; k <= split.last; ++k) {
    const size_t slot = split.slot(k);
    const float2 ml = p.part_ml[slot * kItemRows + r];
    const float a = ptx::ex2(ml.x - ref);
    sum += ml.y * a;
    const float4* src = reinterpret_cast<const float4*>(p.part_o) +
                        slot * (D / 4) * kItemRows + part * V * kItemRows + r;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float4 x = src[j * kItemRows];
      acc[j].x = fmaf(x.x, a, acc[j].x);
      acc[j].y = fmaf(x.y, a, acc[j].y);
      acc[j].z = fmaf(x.z, a, acc[j].z);
      acc[j].w = fmaf(x.w, a, acc[j].w);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int t = row / p.group, hq = w.h * p.group + row % p.group;
  uint16_t* dst = static_cast<uint16_t*>(p.o.data) + w.b * p.o.sb + t * p.o.st + hq * p.o.sh +
                  part * (D / 4);
#pragma unroll
  for (int j = 0; j < V; j += 2)
    *reinterpret_cast<uint4*>(dst + 4 * j) =
        make_uint4(pack2<kDtype>(acc[j].x * inv, acc[j].y * inv),
                   pack2<kDtype>(acc[j].z * inv, acc[j].w * inv),
                   pack2<kDtype>(acc[j + 1].x * inv, acc[j + 1].y * inv),
                   pack2<kDtype>(acc[j + 1].z * inv, acc[j + 1].w * inv));
  if (part == 0) {
    const float lse2 = sum == 0.f ? -INFINITY : mx + log2f(sum);
    if (p.lse != nullptr)
      p.lse[(static_cast<size_t>(w.b) * p.heads + hq) * p.T + t] = lse2 * 0.69314718055994531f;
    p.row_nlse[((static_cast<size_t>(w.b) * c.H + w.h) * p.q_tiles) * 128 + row] =
        sum == 0.f ? -INFINITY : -lse2;
  }
}

}  // namespace sa
