// Eviction from a 4-bit cache by accumulated attention weight.
//
// Reads a weight and a position (8 bytes) a row and moves at most one row per evicted
// one: kept rows from `keep` on go into the places of evicted rows below it, instead
// of everything behind the first evicted row moving up. Small next to an attention
// over the same rows in bytes, so what counts is the chain of dependent steps; all of
// it is one launch:
//  * a cluster of 1 to 8 blocks per (sequence, KV head) keeps the rows' keys (ordered
//    32-bit images of the weights) in shared memory, read once;
//  * the keep-th largest key by radix selection, 10 + 11 + 11 bits: a histogram a
//    block, searched over the cluster through distributed shared memory by every block
//    alike, so a pass costs one cluster barrier. The search goes through sums of 32 or
//    64 bins first: reading all 2048 bins of 8 blocks took 12 K cycles a pass, the two
//    steps 2 K. In the first pass weights crowd into a few exponents: neighbouring
//    lanes count in eight copies (one copy: 6 K cycles for 4096 rows);
//  * rows are numbered in order: each warp owns consecutive rows and counts, by
//    ballots, those above and equal to that key on both sides of `keep`; two scans over
//    the warps and arithmetic give the places of its holes and movers;
//  * the j-th hole takes the j-th mover. Writes go below `keep`, reads come from `keep`
//    on, so the moves need no order among themselves.
//
// Measured: 54000 rows down to 43200, 12 heads, D 128: 25 to 33 us; one row of 4097, 64
// heads: 12 us (a first version, a block a head and a launch for the moves: 280 and 45);
// 32768 rows down to 24576, D 64: 32 heads 31 us, 64 heads 60.
#pragma once

#include <cooperative_groups.h>

#include <type_traits>

#include "kv4_format.cuh"

namespace sa {

struct Kv4EvictParams {
  Kv4 c;
  int keep, first, recent;
  int smem_keys;   // keys a block keeps in shared memory; rows beyond are read again
  int32_t* lists;  // [B][H][N]: holes from the front, movers from N / 2
};

constexpr int kEvictCopies = 8;
constexpr int kEvictHist = (kEvictCopies + 1) * 1024 + 2 * 2048;
constexpr int kEvictFixedSmem = (kEvictHist + 96 + 64) * 4 + 2 * 32 * 8;

// Order of a row among its head's: protected rows above every weight, NaN below,
// equal numbers (both zeros among them) equal.
__device__ __forceinline__ unsigned evict_key(float w, int pos, int first, int keep_from) {
  if (pos < first || pos >= keep_from) return 0xFFFFFFFFu;
  if (isnan(w)) return 0u;
  const unsigned u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// grid (cluster, H, B), 1024 threads.
template <int D>
__global__ void __launch_bounds__(1024, 1)
    kv4_evict_kernel(const __grid_constant__ Kv4EvictParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ int smem_ints[];
  int* copies = smem_ints;                   // [kEvictCopies][1024], the first pass
  int* hist = copies + kEvictCopies * 1024;  // 1024 bins, then twice 2048
  int* coarse = smem_ints + kEvictHist;      // [3][32]: sums of 32 (64) bins
  int* s_pick = coarse + 96;                 // bin, rows left; holes, movers of this block
  long long* s_warp = reinterpret_cast<long long*>(s_pick + 64);  // [2][32]
  unsigned* s_key = reinterpret_cast<unsigned*>(s_warp + 64);
  const Kv4& c = p.c;
  const int h = blockIdx.y, b = blockIdx.z;
  const int rank = static_cast<int>(cluster.block_rank());
  const int blocks = static_cast<int>(cluster.num_blocks());
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned below_lane = (1u << lane) - 1;
  begin_early();
  wait_for_previous();
  const int n = rows_held(c, b);
  const size_t plane = (static_cast<size_t>(b) * c.H + h) * c.N;

  // A barrier of all of the head's blocks (the cluster's takes 1500 cycles even for one).
  auto sync_head = [&]() {
    if (blocks > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  // Sum over the head's blocks of their copies of a counter.
  auto sum_over_blocks = [&](const int* mine) {
    if (blocks == 1) return *mine;
    int sum = 0;
    for (int r = 0; r < blocks; ++r) sum += *cluster.map_shared_rank(mine, r);
    return sum;
  };

  // The warps' ordered scan of a pair of counts (low and high word): the sum over lower
  // warps, and the block's total. `buffer`: 0 and 1 in turn, so one barrier does.
  auto scan_warps = [&](int buffer, long long mine, long long& total) {
    if (lane == 0) s_warp[buffer * 32 + warp] = mine;
    __syncthreads();
    long long x = s_warp[buffer * 32 + lane];
    const long long own = x;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long y = __shfl_up_sync(~0u, x, k);
      if (lane >= k) x += y;
    }
    total = __shfl_sync(~0u, x, 31);
    return __shfl_sync(~0u, x - own, warp);
  };

  if (n > p.keep) {
    const int keep_from = c.seq[kSeqTotal * c.B + b] - p.recent;
    // rows of a warp, a multiple of 32 so that loads start on whole lines
    const int per_warp = ((n + blocks * 32 - 1) / (blocks * 32) + 31) / 32 * 32;
    const int j0 = min((rank * 32 + warp) * per_warp, n);
    const int j1 = min(j0 + per_warp, n);
    auto compute_key = [&](int j) {
      return evict_key(c.weight[plane + j], c.pos[plane + j], p.first, keep_from);
    };
    const int slot0 = warp * per_warp - j0;  // key slot of row j: slot0 + j
    auto key_of = [&](int j) {
      return slot0 + j < p.smem_keys ? s_key[slot0 + j] : compute_key(j);
    };
    // four loads of each kind under way at a time
    const int in_smem = min(j1, p.smem_keys - slot0);
    for (int j = j0 + lane; j < in_smem; j += 128) {
      float w[4];
      int at[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + 32 * k < in_smem) {
          w[k] = c.weight[plane + j + 32 * k];
          at[k] = c.pos[plane + j + 32 * k];
        }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (j + 32 * k < in_smem)
          s_key[slot0 + j + 32 * k] = evict_key(w[k], at[k], p.first, keep_from);
    }
    for (int i = threadIdx.x; i < kEvictHist; i += 1024) smem_ints[i] = 0;
    __syncthreads();

    unsigned prefix = 0;
    int left = p.keep;  // rows still to find among those that match the prefix
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 22 : pass == 1 ? 11 : 0;
      const int above = pass == 1 ? 22 : 11;
      int* mine = hist + (pass == 0 ? 0 : 1024 + (pass - 1) * 2048);
      int* count = pass == 0 ? copies + (lane & (kEvictCopies - 1)) * 1024 : mine;
      for (int j = j0 + lane; j < j1; j += 32) {
        const unsigned k = key_of(j);
        if (pass == 0 || k >> above == prefix) atomicAdd(&count[(k >> shift) & 2047u], 1);
      }
      __syncthreads();
      int sum = 0;  // of 32 (64) bins, one sum a warp
      if (pass == 0) {
#pragma unroll
        for (int k = 0; k < kEvictCopies; ++k) sum += copies[k * 1024 + threadIdx.x];
        mine[threadIdx.x] = sum;
      } else {
        sum = mine[warp * 64 + lane] + mine[warp * 64 + 32 + lane];
      }
#pragma unroll
      for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(~0u, sum, k);
      if (lane == 0) coarse[pass * 32 + warp] = sum;
      sync_head();
      if (warp == 0) {
        // Counts from the top, `PER` bins a lane: the bin in which the left-th row from the
        // top lies, and how many of it are wanted.
        int need = left;
        auto search = [&](const int* counts, int from, auto per_lane) {
          constexpr int PER = decltype(per_lane)::value;
          int v[PER], x = 0;
          const int top = from + 32 * PER - 1 - lane * PER;
#pragma unroll
          for (int k = 0; k < PER; ++k) x += v[k] = sum_over_blocks(counts + top - k);
          const int own = x;
#pragma unroll
          for (int k = 1; k < 32; k <<= 1) {
            const int y = __shfl_up_sync(~0u, x, k);
            if (lane >= k) x += y;
          }
          // (there are at least `need` rows: some lane reaches it)
          const int at = max(__ffs(__ballot_sync(~0u, x >= need)) - 1, 0);
          int bin = top, rest = need - (x - own);
          if (PER == 2 && rest > v[0]) {
            bin = top - 1;
            rest -= v[0];
          }
          need = __shfl_sync(~0u, rest, at);
          return __shfl_sync(~0u, bin, at);
        };
        constexpr std::integral_constant<int, 1> one;
        constexpr std::integral_constant<int, 2> two;
        const int block = search(coarse + pass * 32, 0, one);
        const int bin = pass == 0 ? search(mine, block * 32, one) : search(mine, block * 64, two);
        if (lane == 0) {
          s_pick[0] = bin;
          s_pick[1] = need;
        }
      }
      __syncthreads();
      prefix = (prefix << 11) | static_cast<unsigned>(s_pick[0]);
      left = s_pick[1];
    }
    // prefix: the keep-th largest key; the first `left` rows that equal it stay.
    int equal_before = 0;  // such rows in lower blocks: their last histograms tell
    for (int r = 0; r < rank; ++r)
      equal_before += *cluster.map_shared_rank(hist + 3072 + (prefix & 2047u), r);
    int more[2] = {0, 0}, equal[2] = {0, 0};  // below `keep` and from it on
    for (int j = j0; j < j1; j += 32) {
      const bool in = j + lane < j1;
      const unsigned k = in ? key_of(j + lane) : 0u;
      const unsigned gt = __ballot_sync(~0u, in && k > prefix);
      const unsigned eq = __ballot_sync(~0u, in && k == prefix);
      const int split = min(max(p.keep - j, 0), 32);  // lanes below `keep`
      const unsigned low = split == 32 ? ~0u : (1u << split) - 1;
      more[0] += __popc(gt & low);
      more[1] += __popc(gt & ~low);
      equal[0] += __popc(eq & low);
      equal[1] += __popc(eq & ~low);
    }
    long long total;
    equal_before += static_cast<int>(scan_warps(0, equal[0] + equal[1], total));
    const int stay0 = min(max(left - equal_before, 0), equal[0]);
    const int stay1 = min(max(left - equal_before - equal[0], 0), equal[1]);
    const int my_holes = min(max(p.keep - j0, 0), j1 - j0) - more[0] - stay0;
    const int my_movers = more[1] + stay1;
    const long long below =
        scan_warps(1, static_cast<long long>(my_movers) << 32 | my_holes, total);
    int holes = static_cast<int>(below), movers = static_cast<int>(below >> 32);
    if (threadIdx.x == 0) {
      s_pick[2] = static_cast<int>(total);
      s_pick[3] = static_cast<int>(total >> 32);
    }
    sync_head();
    int moves = s_pick[3];
    if (blocks > 1) {
      moves = 0;
      for (int r = 0; r < blocks; ++r) {
        const int* other = cluster.map_shared_rank(s_pick, r);
        if (r < rank) {
          holes += other[2];
          movers += other[3];
        }
        moves += other[3];
      }
    }
    int32_t* hole_list = p.lists + plane;
    int32_t* mover_list = hole_list + c.N / 2;
    if (my_holes + my_movers > 0) {
      int seen = equal_before;
      for (int j = j0; j < j1; j += 32) {
        const bool in = j + lane < j1, low = j + lane < p.keep;
        const unsigned k = in ? key_of(j + lane) : 0u;
        const unsigned eq = __ballot_sync(~0u, in && k == prefix);
        const bool kept =
            in && (k > prefix || (k == prefix && seen + __popc(eq & below_lane) < left));
        seen += __popc(eq);
        const unsigned hole = __ballot_sync(~0u, in && low && !kept);
        const unsigned mover = __ballot_sync(~0u, !low && kept);
        if (hole >> lane & 1u) hole_list[holes + __popc(hole & below_lane)] = j + lane;
        if (mover >> lane & 1u) mover_list[movers + __popc(mover & below_lane)] = j + lane;
        holes += __popc(hole);
        movers += __popc(mover);
      }
    }
    sync_head();  // lists written; no block reads another's shared memory from here

    // 16 threads a row: 16-byte pieces of codes, 4-byte ones of scales, position and
    // weight; four rows of each under way at a time.
    constexpr int kPieces = D / 32, kScaleWords = D / 64;
    const int sub = threadIdx.x & 15;
    uint8_t* base = nullptr;  // this thread's array, its piece and bytes of a row
    int row_bytes = 0, piece = 0;
    if (sub < 2 * kPieces) {
      base = sub < kPieces ? c.k_codes : c.v_codes;
      row_bytes = D / 2;
      piece = sub % kPieces * 16;
    } else if (sub < 2 * kPieces + 2 * kScaleWords) {
      const int s = sub - 2 * kPieces;
      base = s < kScaleWords ? c.k_scales : c.v_scales;
      row_bytes = D / 16;
      piece = s % kScaleWords * 4;
    } else if (sub >= 14) {
      base = reinterpret_cast<uint8_t*>(sub == 14 ? static_cast<void*>(c.pos) : c.weight);
      row_bytes = 4;
    }
    base += plane * row_bytes + piece;
    for (int i = rank * 64 + (threadIdx.x >> 4); i < moves; i += blocks * 256) {
      int from[4], to[4];
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int at = i + k * blocks * 64;
        from[k] = at < moves ? mover_list[at] : -1;
        to[k] = at < moves ? hole_list[at] : -1;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (from[k] >= 0 && row_bytes != 0) {
          const uint8_t* src = base + static_cast<size_t>(from[k]) * row_bytes;
          if (sub < 2 * kPieces)
            v[k] = *reinterpret_cast<const uint4*>(src);
          else
            v[k].x = *reinterpret_cast<const uint32_t*>(src);
        }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (from[k] >= 0 && row_bytes != 0) {
          uint8_t* dst = base + static_cast<size_t>(to[k]) * row_bytes;
          if (sub < 2 * kPieces)
            *reinterpret_cast<uint4*>(dst) = v[k];
          else
            *reinterpret_cast<uint32_t*>(dst) = v[k].x;
        }
    }
  }

  // the last block to finish moves seq on: every block has read it by then
  __shared__ bool s_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(c.status + 2, 1u) == gridDim.x * gridDim.y * gridDim.z - 1;
  }
  __syncthreads();
  if (!s_last) return;
  for (int i = threadIdx.x; i < c.B; i += 1024)
    if (rows_held(c, i) > p.keep) {
      c.seq[kSeqHeld * c.B + i] = p.keep;
      c.seq[kSeqLast * c.B + i] = 0;
      c.seq[kSeqTail * c.B + i] = 0;
    }
  if (threadIdx.x == 0) c.status[2] = 0;  // ready for the next launch
}

}  // namespace sa
