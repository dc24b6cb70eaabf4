// Host side of the 4-bit KV cache (include/sa.h: sa_kv4_*): argument checks,
// workspace layout and kernel launches. Nothing is kept between calls.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <initializer_list>
#include <string>
#include <utility>

#include "host_common.h"
#include "kernels/kv4_chunk.cuh"
#include "kernels/kv4_decode.cuh"
#include "kernels/kv4_evict.cuh"
#include "kernels/kv4_rows.cuh"
#include "kernels/kv4_weights.cuh"

using sa::aligned16;
using sa::device_memory;
using sa::g_error;
using sa::Kv4;
using sa::Kv4Rows;
using sa::NvtxRange;

namespace {

constexpr int kMaxGridYZ = 65535;
// Rows of a sequence: a pass of one block of queries over as many stays within the
// kernels' bounded waits (a second), and all row counts within 32 bits.
constexpr int kMaxCapacity = 1 << 26;

int refuse(int code, const std::string& why) {
  g_error = "kv4: " + why;
  return code;
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Makes `device` current for the call's launches and puts the caller's back.
class DeviceGuard {
 public:
  explicit DeviceGuard(int device) {
    if (cudaGetDevice(&before_) != cudaSuccess) before_ = -1;
    if (before_ >= 0 && device >= 0 && device != before_)
      changed_ = cudaSetDevice(device) == cudaSuccess;
  }
  ~DeviceGuard() {
    if (changed_) cudaSetDevice(before_);
  }
  DeviceGuard(const DeviceGuard&) = delete;
  DeviceGuard& operator=(const DeviceGuard&) = delete;

 private:
  int before_ = -1;
  bool changed_ = false;
};

int check_sizes(const sa_kv4_cache* c) {
  if (c == nullptr) return refuse(SA_ERR_INVALID_ARG, "cache is NULL");
  if (c->batch < 1 || c->kv_heads < 1 || c->capacity < 1)
    return refuse(SA_ERR_INVALID_ARG, "batch, kv_heads and capacity must be >= 1");
  if (c->head_dim != 64 && c->head_dim != 128)
    return refuse(SA_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (c->capacity % 128 != 0)
    return refuse(SA_ERR_INVALID_ARG, "capacity must be a multiple of 128");
  if (c->batch > kMaxGridYZ || c->kv_heads > kMaxGridYZ ||
      1LL * c->batch * c->kv_heads > (1LL << 24) || c->capacity > kMaxCapacity)
    return refuse(SA_ERR_UNSUPPORTED, "too many sequences, heads or rows");
  return SA_OK;
}

// Sizes, pointers and the device they lie on (-1: managed memory).
int check_cache(const sa_kv4_cache* c, Kv4* out, int* device) {
  if (int rc = check_sizes(c); rc != SA_OK) return rc;
  const void* const ptr[8] = {c->k_codes, c->v_codes, c->k_scales, c->v_scales,
                              c->pos,     c->weight,  c->seq,      c->status};
  static const char* const name[8] = {"k_codes", "v_codes", "k_scales", "v_scales",
                                      "pos",     "weight",  "seq",      "status"};
  for (int i = 0; i < 8; ++i)
    if (ptr[i] == nullptr || !aligned16(ptr[i]))
      return refuse(SA_ERR_INVALID_ARG,
                    std::string(name[i]) + " must be non-NULL and 16-byte aligned");
  std::string why;
  *device = -1;
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, c->k_codes) == cudaSuccess) {
    if (a.type == cudaMemoryTypeDevice) *device = a.device;
  } else {
    cudaGetLastError();
  }
  for (int i = 0; i < 8; ++i)
    if (!device_memory(ptr[i], *device, name[i], &why)) return refuse(SA_ERR_INVALID_ARG, why);
  out->B = c->batch;
  out->H = c->kv_heads;
  out->N = c->capacity;
  out->k_codes = c->k_codes;
  out->v_codes = c->v_codes;
  out->k_scales = c->k_scales;
  out->v_scales = c->v_scales;
  out->pos = c->pos;
  out->weight = c->weight;
  out->seq = c->seq;
  out->status = c->status;
  return SA_OK;
}

// Rows [B, T, heads, D]; `written`: no two rows may overlap.
int check_rows(const sa_rows* r, const char* name, int B, int T, int heads, int D, bool written,
               int device, Kv4Rows* out) {
  if (r == nullptr || (r->data == nullptr && T > 0) || !aligned16(r->data))
    return refuse(SA_ERR_INVALID_ARG,
                  std::string(name) + " must be non-NULL and 16-byte aligned");
  for (int64_t s : {r->stride_b, r->stride_t, r->stride_h})
    if (s < 0 || s % 8 != 0)
      return refuse(SA_ERR_INVALID_ARG,
                    std::string(name) + ": strides must be multiples of 8 and >= 0");
  if (written) {
    // from the smallest stride up, each has to step over all that lies below it
    std::pair<int64_t, int> dim[3] = {{r->stride_b, B}, {r->stride_t, T}, {r->stride_h, heads}};
    std::sort(dim, dim + 3);
    int64_t span = D;
    for (const auto& d : dim) {
      if (d.second <= 1) continue;
      if (d.first < span)
        return refuse(SA_ERR_INVALID_ARG, std::string(name) + ": rows that are written overlap");
      span += d.first * (d.second - 1);
    }
  }
  std::string why;
  if (!device_memory(r->data, device, name, &why)) return refuse(SA_ERR_INVALID_ARG, why);
  out->data = r->data;
  out->sb = r->stride_b;
  out->st = r->stride_t;
  out->sh = r->stride_h;
  return SA_OK;
}

int check_call(int dtype, int T, int max_T, const int32_t* counts, int device) {
  if (dtype != SA_DTYPE_BF16 && dtype != SA_DTYPE_FP16)
    return refuse(SA_ERR_INVALID_ARG, "dtype must be SA_DTYPE_BF16 or SA_DTYPE_FP16");
  if (T < 0) return refuse(SA_ERR_INVALID_ARG, "T must be >= 0");
  if (T > max_T) return refuse(SA_ERR_UNSUPPORTED, "T is too large");
  if (reinterpret_cast<uintptr_t>(counts) & 3u)
    return refuse(SA_ERR_INVALID_ARG, "counts must be 4-byte aligned");
  std::string why;
  if (!device_memory(counts, device, "counts", &why)) return refuse(SA_ERR_INVALID_ARG, why);
  return SA_OK;
}

int check_workspace(const void* ws, size_t bytes, size_t need, int device) {
  if (need == 0) return SA_OK;
  if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || bytes < need)
    return refuse(SA_ERR_INVALID_ARG,
                  "workspace must be 256-byte aligned and hold the bytes asked for");
  std::string why;
  if (!device_memory(ws, device, "workspace", &why)) return refuse(SA_ERR_INVALID_ARG, why);
  return SA_OK;
}

// Launch that may begin while the kernel before it on the stream drains; the kernel
// itself waits until that one has finished (wait_for_previous, in every block).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                         A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The result of a call from that of its launches. Kernels take what the ones before them
// left in the workspace for granted, so the first launch that fails is a call's last.
int launched(const char* what, cudaError_t e) {
  if (e == cudaSuccess) return SA_OK;
  cudaGetLastError();
  return refuse(SA_ERR_CUDA, std::string(what) + " launch: " + cudaGetErrorString(e));
}

constexpr int kMaxTokens = 1 << 24;

int check_heads(const sa_kv4_cache* c, int heads, int T) {
  if (heads < 1 || heads % c->kv_heads != 0)
    return refuse(SA_ERR_INVALID_ARG, "heads must be a multiple of kv_heads");
  const long long rows = 1LL * (heads / c->kv_heads) * T;
  if (heads > kMaxGridYZ || rows > (1LL << 30) ||
      (rows + 127) / 128 * (c->capacity / 128) > INT32_MAX ||
      1LL * c->batch * c->kv_heads * (c->capacity / 32) > INT32_MAX / 4)
    return refuse(SA_ERR_UNSUPPORTED, "too many query rows");
  return SA_OK;
}

constexpr int kMaxDevices = 64;

// Number of SMs of the current device (asked once a device).
int sm_count() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
      n = 148;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Lets `kernel` use its dynamic shared memory on the current device. regs > 0: the
// register count its split between warpgroups assumes; with fewer at launch a
// warpgroup would wait for registers that do not exist, so such a build is refused.
template <auto kernel>
bool allow_smem(int bytes, int regs = 0) {
  static std::atomic<bool> done[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  if (done[dev].load(std::memory_order_relaxed)) return true;
  cudaFuncAttributes fa;
  if (regs > 0 && (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess || fa.numRegs != regs))
    return false;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
      cudaSuccess)
    return false;
  done[dev].store(true, std::memory_order_relaxed);
  return true;
}

// How an attention is run: sizes that follow from the shape alone, so that the
// workspace can be asked for ahead.
struct AttendPlan {
  bool few;        // few query rows: kv4_decode.cuh
  int nt;          // query rows of a block / 8
  int row_blocks;  // blocks of query rows per (sequence, KV head)
  int score_rows;
  long long blocks;  // of the decode kernel, at most
  size_t off_o, off_ml, off_scores;
  // many query rows: kv4_chunk.cuh
  int q_tiles, items;
  size_t off_q, off_scale, off_nlse, off_begin[2], off_pre[2], off_w;
  size_t total;
};

constexpr int kFewRows = 64;
constexpr int kMostSms = 160;  // the workspace covers a grid of any GPU of this kind

AttendPlan plan_attend(const sa_kv4_cache* c, int heads, int T, bool weights) {
  AttendPlan a{};
  if (T == 0) return a;  // nothing runs
  const int rows = heads / c->kv_heads * T, D = c->head_dim;
  const size_t planes = static_cast<size_t>(c->batch) * c->kv_heads;
  a.few = rows <= kFewRows;
  size_t off = 0;
  if (a.few) {
    // blocks of at most 32 query rows, as even as multiples of 8 allow
    const int n8 = std::max((rows + 7) / 8, 1);
    a.row_blocks = (n8 + 3) / 4;
    a.nt = (n8 + a.row_blocks - 1) / a.row_blocks;
    a.blocks = static_cast<long long>(kMostSms) * sa::decode_blocks_per_sm(a.nt);
    const size_t slots = a.blocks + planes * a.row_blocks;
    a.off_o = off;
    off += align_up(slots * 8 * a.nt * D * sizeof(float), 256);
    a.off_ml = off;
    off += align_up(slots * 8 * a.nt * sizeof(float2), 256);
    a.score_rows = (rows + 1) / 2 * 2;
    // for the weights: every score, or with more than 8 query rows their log-sum-exps
    a.off_scores = off;
    if (weights)
      off += align_up((a.nt == 1 ? planes * c->capacity : planes) * a.score_rows * sizeof(float),
                      256);
  } else {
    auto take = [&](size_t bytes) {
      const size_t at = off;
      off += align_up(bytes, 256);
      return at;
    };
    a.q_tiles = (rows + 127) / 128;
    a.items = (rows + sa::kItemRows - 1) / sa::kItemRows;
    const size_t q_rows = planes * a.q_tiles * 128;
    a.off_q = take(q_rows * D * 2);
    a.off_scale = take(q_rows * sizeof(float));
    a.off_nlse = take(q_rows * sizeof(float));
    const int items[2] = {a.items, c->capacity / 128};
    for (int i = 0; i < (weights ? 2 : 1); ++i) {
      a.off_begin[i] = take((c->batch + 1) * sizeof(long long));
      a.off_pre[i] = take(static_cast<size_t>(c->batch) * (items[i] + 2) * sizeof(int));
    }
    if (weights) a.off_w = take(2ull * kMostSms * 128 * sizeof(float));
    // two partial results of 512 rows a pair of SMs
    a.off_o = take(1ull * kMostSms * sa::kItemRows * D * sizeof(float));
    a.off_ml = take(1ull * kMostSms * sa::kItemRows * sizeof(float2));
  }
  a.total = off;
  return a;
}

template <int D, int NT, int kDtype, bool kScores>
cudaError_t launch_decode(const sa::Kv4AttendParams& p, cudaStream_t s) {
  using S = sa::DecodeShape<D, NT>;
  using W = sa::DecodeWeightShape<D>;
  const bool second_pass = p.add_weight && !kScores;
  if (!allow_smem<sa::kv4_decode_kernel<D, NT, kDtype, kScores>>(S::kSmem) ||
      (second_pass && !allow_smem<sa::kv4_decode_weight_kernel<D, kDtype>>(W::kSmem)))
    return cudaErrorInvalidConfiguration;
  const int blocks = std::min(sm_count(), kMostSms) * S::kBlocksPerSm;
  cudaError_t e = launch_after(sa::kv4_decode_kernel<D, NT, kDtype, kScores>, dim3(blocks),
                               dim3(128), S::kSmem, s, p);
  if (e != cudaSuccess) return e;
  const int units = p.c.B * p.c.H * p.row_blocks;
  // weights: as many blocks as run at once (six an SM), twice, since lengths differ; of
  // 512 rows or more
  const int parts = std::max(std::min(2 * 6 * std::min(sm_count(), kMostSms) / (p.c.B * p.c.H),
                                      (p.c.N + sa::kJoinKeys - 1) / sa::kJoinKeys),
                             1);
  // Long rows leave many partial results: a block merges one query row's. With 8 or
  // fewer a warp a row is enough.
  auto join = [&](auto kernel, int warps) {
    const int merge = units * (S::kRows * warps / 4);
    return launch_after(kernel, dim3(merge + (kScores ? p.c.B * p.c.H * parts : 0)), dim3(128), 0,
                        s, p, blocks, merge, parts);
  };
  e = blocks > 8 * units ? join(sa::kv4_join_kernel<D, S::kRows, 4, kDtype>, 4)
                         : join(sa::kv4_join_kernel<D, S::kRows, 1, kDtype>, 1);
  if (e != cudaSuccess || !second_pass) return e;
  sa::Kv4AttendParams q = p;
  q.row_blocks = 1;  // a unit has all query rows
  return launch_after(sa::kv4_decode_weight_kernel<D, kDtype>,
                      dim3(std::min(sm_count(), kMostSms) * W::kBlocksPerSm), dim3(128), W::kSmem,
                      s, q);
}

template <int D, int kDtype>
cudaError_t launch_decode_nt(const sa::Kv4AttendParams& p, int nt, cudaStream_t s) {
  if (nt == 1)
    return p.add_weight ? launch_decode<D, 1, kDtype, true>(p, s)
                        : launch_decode<D, 1, kDtype, false>(p, s);
  return nt == 2   ? launch_decode<D, 2, kDtype, false>(p, s)
         : nt == 3 ? launch_decode<D, 3, kDtype, false>(p, s)
                   : launch_decode<D, 4, kDtype, false>(p, s);
}

template <int D, int kDtype>
cudaError_t launch_chunk(const sa::Kv4AttendParams& p, cudaStream_t s) {
  using S = sa::ChunkShape<D>;
  using W = sa::WeightShape<D>;
  if (!allow_smem<sa::kv4_chunk_kernel<D, kDtype>>(S::kSmem, 128) ||
      (p.add_weight && !allow_smem<sa::kv4_weight_kernel<D>>(W::kSmem)))
    return cudaErrorInvalidConfiguration;
  const int blocks = std::min(sm_count(), kMostSms), pairs = std::max(blocks / 2, 1);
  cudaError_t e = launch_after(sa::kv4_stage_kernel<D, kDtype>,
                               dim3(p.q_tiles + (p.add_weight ? 2 : 1), p.c.H, p.c.B), dim3(256),
                               0, s, p);
  if (e == cudaSuccess)
    e = launch_after(sa::kv4_chunk_kernel<D, kDtype>, dim3(2 * pairs), dim3(S::kThreads), S::kSmem,
                     s, p);
  if (e == cudaSuccess && pairs > 1)
    e = launch_after(sa::kv4_chunk_join_kernel<D, kDtype>, dim3(pairs - 1, sa::kItemRows / 32),
                     dim3(128), 0, s, p, pairs);
  if (e == cudaSuccess && p.add_weight)
    e = launch_after(sa::kv4_weight_kernel<D>, dim3(blocks), dim3(W::kThreads), W::kSmem, s, p);
  if (e == cudaSuccess && p.add_weight && blocks > 1)
    e = launch_after(sa::kv4_weight_join_kernel, dim3(blocks - 1), dim3(128), 0, s, p, blocks);
  return e;
}

size_t evict_bytes(const sa_kv4_cache* c) {
  return align_up(static_cast<size_t>(c->batch) * c->kv_heads * c->capacity * sizeof(int32_t), 256);
}

constexpr int kMostKeys = 40960;  // keys in an eviction block's shared memory (160 KB)

template <int D>
cudaLaunchConfig_t evict_config(dim3 grid, int keys, cudaLaunchAttribute (&at)[2]) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(1024);
  cfg.dynamicSmemBytes = sa::kEvictFixedSmem + keys * 4;
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = grid.x;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters of `n` eviction blocks that run at once on the current device: one block an SM (its
// threads fill the registers), and a cluster within a group of SMs that does not divide by
// it, so the device is asked (once a size).
template <int D>
int evict_clusters_at_once(int n) {
  static std::atomic<int> known[kMaxDevices][4];
  int dev = 0, count = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::atomic<int>& slot = known[dev][n == 8 ? 3 : n / 2];
  if ((count = slot.load(std::memory_order_relaxed)) > 0) return count;
  cudaLaunchAttribute at[2];
  const cudaLaunchConfig_t cfg = evict_config<D>(dim3(n, 1, 1), kMostKeys, at);
  if (cudaOccupancyMaxActiveClusters(&count, sa::kv4_evict_kernel<D>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return sm_count() / n;
  }
  slot.store(count, std::memory_order_relaxed);
  return count;
}

// Blocks that share one head's rows: as many as leave each 4096 rows or more while all heads
// still run at once, and in any case enough for the keys to fit their shared memory. Heads x
// rows, us with this rule and with the next larger (smaller) cluster: 32 x 32768 31 (65, 46),
// 64 x 32768 61 (73, 93), 16 x 65536 48 (61, 81), 96 x 32768 100 (115), 148 x 131072 554
// (607, 731).
template <int D>
int evict_cluster(const Kv4& c) {
  int n = 1;
  while (n < 8) {
    const int at_once = evict_clusters_at_once<D>(n * 2);
    const bool keys_fit = c.N <= n * kMostKeys;
    if (at_once < 1 ||  // (part of a device may hold none; keys that do not fit are read again)
        (keys_fit && (n * 2 * 4096 > c.N || 1LL * c.B * c.H > at_once)))
      break;
    n *= 2;
  }
  return n;
}

template <int D>
cudaError_t launch_evict(sa::Kv4EvictParams p, cudaStream_t s) {
  if (!allow_smem<sa::kv4_evict_kernel<D>>(sa::kEvictFixedSmem + kMostKeys * 4))
    return cudaErrorInvalidConfiguration;
  const int cluster = evict_cluster<D>(p.c);
  const int per_block = ((p.c.N + cluster * 32 - 1) / (cluster * 32) + 31) / 32 * 32 * 32;
  p.smem_keys = std::min(per_block, kMostKeys);
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = evict_config<D>(dim3(cluster, p.c.H, p.c.B), p.smem_keys, at);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, sa::kv4_evict_kernel<D>, p);
}

}  // namespace

extern "C" {

SA_API int sa_kv4_reset(const sa_kv4_cache* c, sa_stream stream) {
  NvtxRange range_("sa_kv4_reset");
  Kv4 k;
  int device;
  if (int rc = check_cache(c, &k, &device); rc != SA_OK) return rc;
  DeviceGuard guard(device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(k.seq, 0, sizeof(int32_t) * 4 * k.B, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(k.status, 0, 16, s);
  if (e != cudaSuccess)
    return refuse(SA_ERR_CUDA, std::string("reset: ") + cudaGetErrorString(e));
  return SA_OK;
}

SA_API int sa_kv4_append(const sa_kv4_cache* c, const sa_rows* K, const sa_rows* V, int dtype,
                         int T, const int32_t* counts, int replace, sa_stream stream) {
  NvtxRange range_("sa_kv4_append");
  sa::Kv4AppendParams p;
  int device;
  if (int rc = check_cache(c, &p.c, &device); rc != SA_OK) return rc;
  if (int rc = check_call(dtype, T, kMaxTokens, counts, device); rc != SA_OK) return rc;
  const int D = c->head_dim;
  if (int rc = check_rows(K, "K", p.c.B, T, p.c.H, D, false, device, &p.k); rc != SA_OK) return rc;
  if (int rc = check_rows(V, "V", p.c.B, T, p.c.H, D, false, device, &p.v); rc != SA_OK) return rc;
  p.counts = counts;
  p.T = T;
  p.replace = replace != 0;
  DeviceGuard guard(device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const long long items = 1LL * T * (D / 16);
  const dim3 grid(static_cast<unsigned>(items > 0 ? (items + 255) / 256 : 1), p.c.H, p.c.B);
  const bool half = dtype == SA_DTYPE_FP16;
  auto* kernel = D == 128 ? (half ? sa::kv4_append_kernel<128, SA_DTYPE_FP16>
                                  : sa::kv4_append_kernel<128, SA_DTYPE_BF16>)
                          : (half ? sa::kv4_append_kernel<64, SA_DTYPE_FP16>
                                  : sa::kv4_append_kernel<64, SA_DTYPE_BF16>);
  return launched("append", launch_after(kernel, grid, dim3(256), 0, s, p));
}

SA_API int sa_kv4_read(const sa_kv4_cache* c, int first, const sa_rows* K, const sa_rows* V,
                       int dtype, int T, sa_stream stream) {
  NvtxRange range_("sa_kv4_read");
  sa::Kv4ReadParams p;
  int device;
  if (int rc = check_cache(c, &p.c, &device); rc != SA_OK) return rc;
  if (int rc = check_call(dtype, T, kMaxTokens, nullptr, device); rc != SA_OK) return rc;
  if (first < 0 && first != SA_KV4_LAST)
    return refuse(SA_ERR_INVALID_ARG, "first must be >= 0 or SA_KV4_LAST");
  const int D = c->head_dim;
  if (int rc = check_rows(K, "K", p.c.B, T, p.c.H, D, true, device, &p.k); rc != SA_OK) return rc;
  if (int rc = check_rows(V, "V", p.c.B, T, p.c.H, D, true, device, &p.v); rc != SA_OK) return rc;
  if (T == 0) return SA_OK;
  if (K->data == V->data) return refuse(SA_ERR_INVALID_ARG, "K and V must not be the same");
  p.first = first;
  p.T = T;
  DeviceGuard guard(device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>((1LL * T * (D / 16) + 255) / 256), p.c.H, p.c.B);
  const bool half = dtype == SA_DTYPE_FP16;
  auto* kernel = D == 128 ? (half ? sa::kv4_read_kernel<128, SA_DTYPE_FP16>
                                  : sa::kv4_read_kernel<128, SA_DTYPE_BF16>)
                          : (half ? sa::kv4_read_kernel<64, SA_DTYPE_FP16>
                                  : sa::kv4_read_kernel<64, SA_DTYPE_BF16>);
  return launched("read", launch_after(kernel, grid, dim3(256), 0, s, p));
}

SA_API size_t sa_kv4_attend_bytes(const sa_kv4_cache* c, int heads, int T, int add_weight) {
  if (check_sizes(c) != SA_OK || T < 0 || T > kMaxTokens || check_heads(c, heads, T) != SA_OK)
    return 0;
  return plan_attend(c, heads, T, add_weight != 0).total;
}

SA_API int sa_kv4_attend(const sa_kv4_cache* c, const sa_rows* Q, const sa_rows* O, int dtype,
                         int heads, int T, const int32_t* counts, int causal, float scale,
                         float* lse, int add_weight, void* workspace, size_t workspace_bytes,
                         sa_stream stream) {
  NvtxRange range_("sa_kv4_attend");
  sa::Kv4AttendParams p;
  int device;
  if (int rc = check_cache(c, &p.c, &device); rc != SA_OK) return rc;
  if (int rc = check_call(dtype, T, kMaxTokens, counts, device); rc != SA_OK) return rc;
  if (int rc = check_heads(c, heads, T); rc != SA_OK) return rc;
  const int D = c->head_dim;
  if (int rc = check_rows(Q, "Q", p.c.B, T, heads, D, false, device, &p.q); rc != SA_OK) return rc;
  if (int rc = check_rows(O, "O", p.c.B, T, heads, D, true, device, &p.o); rc != SA_OK) return rc;
  if (T > 0 && O->data == Q->data) return refuse(SA_ERR_INVALID_ARG, "O must not alias Q");
  if (!std::isfinite(scale)) return refuse(SA_ERR_INVALID_ARG, "scale must be finite");
  std::string why;
  if (reinterpret_cast<uintptr_t>(lse) & 3u)
    return refuse(SA_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  if (!device_memory(lse, device, "lse", &why)) return refuse(SA_ERR_INVALID_ARG, why);
  const AttendPlan plan = plan_attend(c, heads, T, add_weight != 0);
  if (int rc = check_workspace(workspace, workspace_bytes, plan.total, device); rc != SA_OK)
    return rc;
  if (T == 0) return SA_OK;
  p.counts = counts;
  p.lse = lse;
  p.heads = heads;
  p.group = heads / p.c.H;
  p.T = T;
  p.causal = causal != 0;
  p.scale_log2 = (scale > 0.f ? scale : 1.f / std::sqrt(static_cast<float>(D))) * 1.44269504f;
  p.add_weight = add_weight != 0;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.row_blocks = plan.row_blocks;
  p.part_o = reinterpret_cast<float*>(ws + plan.off_o);
  p.part_ml = reinterpret_cast<float2*>(ws + plan.off_ml);
  p.scores = reinterpret_cast<float*>(ws + plan.off_scores);
  p.row_nlse = p.scores;
  p.score_rows = plan.score_rows;
  DeviceGuard guard(device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool half = dtype == SA_DTYPE_FP16;
  if (plan.few)
    return launched("attention",
                    D == 128 ? (half ? launch_decode_nt<128, SA_DTYPE_FP16>(p, plan.nt, s)
                                     : launch_decode_nt<128, SA_DTYPE_BF16>(p, plan.nt, s))
                             : (half ? launch_decode_nt<64, SA_DTYPE_FP16>(p, plan.nt, s)
                                     : launch_decode_nt<64, SA_DTYPE_BF16>(p, plan.nt, s)));
  p.q_tiles = plan.q_tiles;
  p.q_img = ws + plan.off_q;
  p.row_scale = reinterpret_cast<float*>(ws + plan.off_scale);
  p.row_nlse = reinterpret_cast<float*>(ws + plan.off_nlse);
  p.part_w = reinterpret_cast<float*>(ws + plan.off_w);
  auto line = [&](int i, int items) {
    return sa::StepLine{reinterpret_cast<long long*>(ws + plan.off_begin[i]),
                        reinterpret_cast<int*>(ws + plan.off_pre[i]), items};
  };
  p.line = line(0, plan.items);
  p.weight_line = line(1, p.c.N / 128);
  return launched("attention", D == 128 ? (half ? launch_chunk<128, SA_DTYPE_FP16>(p, s)
                                                : launch_chunk<128, SA_DTYPE_BF16>(p, s))
                                        : (half ? launch_chunk<64, SA_DTYPE_FP16>(p, s)
                                                : launch_chunk<64, SA_DTYPE_BF16>(p, s)));
}

SA_API size_t sa_kv4_evict_bytes(const sa_kv4_cache* c) {
  return check_sizes(c) == SA_OK ? evict_bytes(c) : 0;
}

SA_API int sa_kv4_evict(const sa_kv4_cache* c, int keep, int first, int recent, void* workspace,
                        size_t workspace_bytes, sa_stream stream) {
  NvtxRange range_("sa_kv4_evict");
  sa::Kv4EvictParams p;
  int device;
  if (int rc = check_cache(c, &p.c, &device); rc != SA_OK) return rc;
  if (keep < 1 || first < 0 || recent < 0 || 1LL * first + recent > keep)
    return refuse(SA_ERR_INVALID_ARG, "need keep >= 1, first, recent >= 0, first + recent <= keep");
  if (int rc = check_workspace(workspace, workspace_bytes, evict_bytes(c), device); rc != SA_OK)
    return rc;
  if (keep >= p.c.N) return SA_OK;  // nothing can be above it
  p.keep = keep;
  p.first = first;
  p.recent = recent;
  p.lists = static_cast<int32_t*>(workspace);
  DeviceGuard guard(device);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched("eviction",
                  c->head_dim == 128 ? launch_evict<128>(p, s) : launch_evict<64>(p, s));
}

SA_API int sa_kv4_get_status(const sa_kv4_cache* c, sa_stream stream) {
  Kv4 k;
  int device;
  if (int rc = check_cache(c, &k, &device); rc != SA_OK) return rc;
  DeviceGuard guard(device);
  unsigned word = 0;
  cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaSuccess) e = cudaMemcpy(&word, k.status, sizeof(word), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess)
    return refuse(SA_ERR_CUDA, std::string("status: ") + cudaGetErrorString(e));
  if (word & sa::kDevErrTimeout) return SA_ERR_TIMEOUT;
  if (word & sa::kDevErrFull) return SA_ERR_FULL;
  if (word & sa::kDevErrOrder) return SA_ERR_STATE;
  if (word & sa::kDevWarnSaturated) return SA_ERR_RANGE;
  return SA_OK;
}

}  // extern "C"
