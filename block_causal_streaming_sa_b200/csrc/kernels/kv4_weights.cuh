// Attention weight drawn by the rows of a 4-bit cache from many query rows:
//   weight[j] += sum over queries l of 2^(s_lj - lse_l)
// after the attention has left every query's log-sum-exp.
//
// One product and one exponential per (query row, cache row): 128 x 128 exponentials
// take twice the cycles of their product. A quarter of them goes to the FMA pipe; more there is
// slower (3/8: 1.65 ms in the measurement below), and halving the operands' shared memory
// traffic by pairs of SMs gains nothing (1.58). No unit is full then: issue slots 73 %,
// exponential unit 61 %, shared memory 52 %, tensor core 41 % of the active cycles; what
// remains are waits of the twelve warps that sum, for tensor memory and for one another.
// Transposed scores S^T = K Q^T put a cache row on a thread, so its sum stays in the
// thread's registers over all queries: no reduction across threads and no atomics,
// the same bits on every run. K is converted once per key tile; query tiles stream
// past it as bulk copies of the staged images, with the rows' scales and
// log-sum-exps. Storing the attention's own probabilities instead would move 2 bytes
// per pair, more than the product costs.
//
//  * Steps (key tile, query tile) are cut evenly over the blocks like the attention's.
//  * One warp loads query tiles into a ring of four stages; one issues the products into
//    the four tensor memory buffers of the same numbers; three warpgroups take the steps
//    in turn; one converts key tiles, one ahead.
//
// Measured: 10800 x 43200 rows, 12 heads, D 128: 1.57 ms.
#pragma once

#include "kv4_chunk.cuh"

namespace sa {

// Packed sums that take subnormals as zero: exponentials below 2^-126 add nothing, whichever
// way they are taken.
__device__ __forceinline__ void fadd2_ftz(float& d0, float& d1, float x0, float x1) {
  asm("{\n\t.reg .b64 ra, rb;\n\t"
      "mov.b64 ra, {%0, %1};\n\tmov.b64 rb, {%2, %3};\n\t"
      "add.rn.ftz.f32x2 ra, ra, rb;\n\tmov.b64 {%0, %1}, ra;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(x0), "f"(x1));
}

template <int D>
struct WeightShape {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kStages = 4;
  static constexpr int kGroups = 3;  // warpgroups that take steps in turn
  static constexpr int kThreads = 128 * (kGroups + 1) + 64;
  static constexpr int kOffK = 0;                              // two key tiles
  static constexpr int kOffQ = 2 * kTile;                      // query tiles
  static constexpr int kOffRow = kOffQ + kStages * kTile;      // [stage][scale | -lse][128]
  static constexpr int kOffAcc = kOffRow + kStages * 1024;     // [2][kGroups - 1][128]
  static constexpr int kOffBar = kOffAcc + 1024 * (kGroups - 1);
  static constexpr int kSmem = kOffBar + 256 + 1024;           // + alignment slack
  static constexpr uint32_t kIdesc = ptx::idesc_f32acc(128, 128, 0, 0);
  __host__ __device__ static constexpr int QFULL(int s) { return s; }
  __host__ __device__ static constexpr int SFULL(int s) { return kStages + s; }
  __host__ __device__ static constexpr int EMPTY(int s) { return 2 * kStages + s; }
  __host__ __device__ static constexpr int KFULL(int i) { return 3 * kStages + i; }
  __host__ __device__ static constexpr int KEMPTY(int i) { return 3 * kStages + 2 + i; }
  __host__ __device__ static constexpr int DRAIN() { return 3 * kStages + 4; }
  static_assert(kSmem <= 232448, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(WeightShape<D>::kThreads, 1)
    kv4_weight_kernel(const __grid_constant__ Kv4AttendParams p) {
  using S = WeightShape<D>;
  extern __shared__ uint8_t smem_raw[];
  const Kv4& c = p.c;
  const uint32_t raw = ptx::smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t sbase = ptx::smem_addr(smem);
  auto bar = [&](int i) { return sbase + S::kOffBar + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffBar + 240);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffBar + 248);
  const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      ptx::mbar_init(bar(S::QFULL(s)), 1);
      ptx::mbar_init(bar(S::SFULL(s)), 1);
      ptx::mbar_init(bar(S::EMPTY(s)), 4);  // the four warps that read the step
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(S::KFULL(i)), 4);  // the four converting warps
      ptx::mbar_init(bar(S::KEMPTY(i)), 1);
    }
    ptx::mbar_init(bar(S::DRAIN()), 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  constexpr int kConvert = 4 * S::kGroups, kIssue = kConvert + 4;  // first warps of the roles
  if (warp == kIssue) {
    ptx::tmem_alloc(ptx::smem_addr(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  wait_for_previous();  // the attention's log-sum-exps

  LineWalk walk = line_range(p.weight_line, c.B, blockIdx.x, gridDim.x);
  auto wait = [&](int which, uint32_t parity) {
    return ptx::mbar_wait(bar(which), parity, abort_flag, c.status);
  };
  // Query tile of step t of the walk's item.
  auto first_tile = [&]() {
    int from;
    weight_steps(p, rows_held(c, walk.b), tokens_of(p.counts, walk.b, p.T), walk.item, from);
    return from + walk.t0;
  };

  if (warp == kIssue + 1) {
    // -------------------------------------------------------------- query tiles
    if (lane == 0) {
      uint32_t step = 0;
      bool ok = true;
      while (ok && walk.next(p.weight_line, c.B)) {
        const size_t tile0 =
            (static_cast<size_t>(walk.b) * c.H + walk.h) * p.q_tiles + first_tile();
        for (int t = 0; t < walk.t1 - walk.t0; ++t, ++step) {
          const int s = step % S::kStages;
          ok = wait(S::EMPTY(s), ((step / S::kStages) & 1) ^ 1u);
          if (!ok) break;
          const uint32_t full = bar(S::QFULL(s)), row = sbase + S::kOffRow + s * 1024;
          ptx::mbar_arrive_expect_tx(full, S::kTile + 1024);
          auto load = [&](uint32_t dst, const void* src, uint32_t bytes) {
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], "
                "%2, [%3];" ::"r"(dst),
                "l"(src), "r"(bytes), "r"(full)
                : "memory");
          };
          load(sbase + S::kOffQ + s * S::kTile, p.q_img + (tile0 + t) * S::kTile, S::kTile);
          load(row, p.row_scale + (tile0 + t) * 128, 512);
          load(row + 512, p.row_nlse + (tile0 + t) * 128, 512);
        }
      }
      // copies under way land before the block can end
      volatile int none = 0;
      for (uint32_t k = step > S::kStages ? step - S::kStages : 0; k < step; ++k)
        ptx::mbar_wait(bar(S::QFULL(k % S::kStages)), (k / S::kStages) & 1, &none, c.status);
    }
  } else if (warp == kIssue) {
    // -------------------------------------------------------------- MMA issuer
    // (the whole warp, for uniform values; see kv4_chunk_kernel)
    const bool issues = ptx_elect();
    auto all_wait = [&](int which, uint32_t parity) {
      return __all_sync(~0u, wait(which, parity)) != 0;
    };
    uint32_t step = 0, unit = 0;
    bool ok = true;
    while (ok && walk.next(p.weight_line, c.B)) {
      const int kb = unit & 1, steps = __shfl_sync(~0u, walk.t1 - walk.t0, 0);
      ok = all_wait(S::KFULL(kb), (unit >> 1) & 1);
      for (int t = 0; ok && t < steps; ++t, ++step) {
        const int s = step % S::kStages;
        ok = all_wait(S::QFULL(s), (step / S::kStages) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t ka = sbase + S::kOffK + kb * S::kTile;
        const uint32_t qb = sbase + S::kOffQ + s * S::kTile;
        if (issues) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
            ptx::umma_ss(tmem + s * 128, ptx::smem_desc_sw128(ka + off, 16, 1024),
                         ptx::smem_desc_sw128(qb + off, 16, 1024), S::kIdesc, kk > 0 ? 1u : 0u);
          }
          ptx::umma_commit(bar(S::SFULL(s)));
        }
      }
      if (ok && issues) ptx::umma_commit(bar(S::KEMPTY(kb)));
      ++unit;
    }
    if (issues) {
      volatile int none = 0;
      ptx::umma_commit(bar(S::DRAIN()));
      ptx::mbar_wait(bar(S::DRAIN()), 0, &none, c.status);
    }
  } else if (warp >= kConvert) {
    // -------------------------------------------------------------- conversion
    const int tid = threadIdx.x - 32 * kConvert;
    uint32_t unit = 0;
    while (walk.next(p.weight_line, c.B)) {
      const int kb = unit & 1;
      const size_t row0 = (static_cast<size_t>(walk.b) * c.H + walk.h) * c.N +
                          static_cast<size_t>(walk.item) * 128;
      constexpr int P = D / 32;
      ConvertRegs<P> x;
      auto key = [](int r) { return r; };
      convert_load<D, P>(x, c.k_codes, c.k_scales, row0, 0, tid, key);
      if (!__all_sync(~0u, wait(S::KEMPTY(kb), ((unit >> 1) & 1) ^ 1u))) break;
      convert_store<P>(x, sbase + S::kOffK + kb * S::kTile, tid,
                       rows_held(c, walk.b) - walk.item * 128, key, tile_offset);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(S::KFULL(kb)));
      ++unit;
    }
  } else {
    // -------------------------------------------------------------- sums
    const int wg = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float* s_acc = reinterpret_cast<float*>(smem + S::kOffAcc);
    uint32_t step = 0, unit = 0;
    bool ok = true;
    while (walk.next(p.weight_line, c.B)) {
      const int held = rows_held(c, walk.b), n_tok = tokens_of(p.counts, walk.b, p.T);
      const int j = walk.item * 128 + r;
      // first query row that sees row j
      const int row_min = p.causal ? max(j - (held - n_tok), 0) * p.group : 0;
      const int tile0 = first_tile();
      float acc[8];
#pragma unroll
      for (int a = 0; a < 8; ++a) acc[a] = 0.f;
      for (int t = 0; t < walk.t1 - walk.t0; ++t, ++step) {
        if (step % S::kGroups != static_cast<uint32_t>(wg)) continue;
        const int s = step % S::kStages;
        ok = ok && __all_sync(~0u, wait(S::SFULL(s), (step / S::kStages) & 1));
        if (!ok) continue;  // the barrier below is still met
        ptx::tc_fence_after();
        const int hidden = row_min - (tile0 + t) * 128;  // columns before this see nothing
        const float* scale = reinterpret_cast<const float*>(smem + S::kOffRow + s * 1024);
        uint32_t x[2][32];
        ptx::tmem_ld32(t_lane + s * 128, x[0]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          ptx::tmem_wait_ld();
          if (q < 3) ptx::tmem_ld32(t_lane + s * 128 + (q + 1) * 32, x[(q + 1) & 1]);
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const float4 sl = *reinterpret_cast<const float4*>(scale + q * 32 + k);
            const float4 nl = *reinterpret_cast<const float4*>(scale + 128 + q * 32 + k);
            const uint32_t* v = x[q & 1] + k;
            float e0, e1, e2, e3;
            ptx::ffma2(e0, e1, __uint_as_float(v[0]), __uint_as_float(v[1]), sl.x, sl.y, nl.x,
                       nl.y);
            ptx::ffma2(e2, e3, __uint_as_float(v[2]), __uint_as_float(v[3]), sl.z, sl.w, nl.z,
                       nl.w);
            e0 = ptx::ex2(e0);
            e1 = ptx::ex2(e1);
            if (k % 8 == 4) {  // a quarter, see above
              exp2_fma2(e2, e3, e2, e3);
            } else {
              e2 = ptx::ex2(e2);
              e3 = ptx::ex2(e3);
            }
            if (hidden > 0) {
              const int col = q * 32 + k;
              e0 = col < hidden ? 0.f : e0;
              e1 = col + 1 < hidden ? 0.f : e1;
              e2 = col + 2 < hidden ? 0.f : e2;
              e3 = col + 3 < hidden ? 0.f : e3;
            }
            const int a = (k & 4);
            fadd2_ftz(acc[a], acc[a + 1], e0, e1);
            fadd2_ftz(acc[a + 2], acc[a + 3], e2, e3);
          }
        }
        // A query whose log-sum-exp is NaN gives NaN to every row it sees; the polynomial
        // dropped it. One vote over the tile's 128, each looked at only if it hits.
        const float4 nl = *reinterpret_cast<const float4*>(scale + 128 + lane * 4);
        if (__any_sync(~0u, isnan((nl.x + nl.y) + (nl.z + nl.w)))) {
#pragma unroll 1
          for (int col = max(hidden, 0); col < 128; ++col)
            if (isnan(scale[128 + col])) acc[0] += scale[128 + col];
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(S::EMPTY(s)));
      }
      const float sum = ((acc[0] + acc[1]) + (acc[2] + acc[3])) +
                        ((acc[4] + acc[5]) + (acc[6] + acc[7]));
      // the warpgroups' sums, always in the same order
      float* others = s_acc + (unit & 1) * (S::kGroups - 1) * 128 + r;
      if (wg > 0) others[(wg - 1) * 128] = sum;
      asm volatile("bar.sync 1, %0;" ::"n"(128 * S::kGroups) : "memory");
      if (wg == 0 && ok) {
        float both = sum;
#pragma unroll
        for (int k = 0; k < S::kGroups - 1; ++k) both += others[k * 128];
        if (walk.t0 > 0 || walk.t1 < walk.n) {
          p.part_w[partial_slot(blockIdx.x, walk.t0) * 128 + r] = both;
        } else if (j < held) {
          float* w = c.weight + (static_cast<size_t>(walk.b) * c.H + walk.h) * c.N + j;
          *w += both;
        }
      }
      ++unit;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kIssue) ptx::tmem_dealloc(tmem, 512);
}

// Weights of key tiles that lie in several blocks' ranges, summed in their order.
__global__ void __launch_bounds__(128)
    kv4_weight_join_kernel(const __grid_constant__ Kv4AttendParams p, int blocks) {
  begin_early();
  wait_for_previous();
  const Kv4& c = p.c;
  SplitItem split;
  if (!split.find(p.weight_line, c.B, blocks, blockIdx.x)) return;
  const LineWalk& w = split.w;
  const int j = w.item * 128 + threadIdx.x;
  if (j >= rows_held(c, w.b)) return;
  float sum = 0.f;
  for (int k = split.first; k <= split.last; ++k)
    sum += p.part_w[split.slot(k) * 128 + threadIdx.x];
  c.weight[(static_cast<size_t>(w.b) * c.H + w.h) * c.N + j] += sum;
}

}  // namespace sa
