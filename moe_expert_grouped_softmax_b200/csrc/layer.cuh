// Host side of include/moe_layer.h: argument checks, tensor maps and launches
// of the residual norm, the dense gated feed-forward block and dropout.
// Part of moe_lora.cu (one translation unit, one device status word).
#pragma once

#include "dense_pair.cuh"
#include "dense_split.cuh"
#include "dropout.cuh"
#include "ffn_rows.cuh"
#include "moe_layer.h"
#include "norm.cuh"

namespace {

// Current device's number, and its SM count from the first call on it (a small
// call's launches cost about as much host time as its kernels take).
constexpr int kMaxDevices = 64;
int current_device() {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kMaxDevices ? dev : -1;
}
int layer_sms() {
  static std::atomic<int> sms[kMaxDevices];
  const int dev = current_device();
  if (dev < 0) return num_sms();
  int n = sms[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    n = num_sms();
    sms[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Raises a kernel's shared-memory limit once per device; `Key` is one type
// per kernel instance.
template <class Key, typename K>
bool allow_smem(K kern, int bytes) {
  static std::atomic<uint64_t> done{0};
  const int dev = current_device();
  if (dev >= 0 && ((done.load(std::memory_order_relaxed) >> dev) & 1)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return false;
  if (dev >= 0) done.fetch_or(uint64_t{1} << dev, std::memory_order_relaxed);
  return true;
}
template <auto Kern>
struct KernelKey {};

inline bool aligned_to(const void* p, size_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}
inline bool aligned16(const void* p) { return aligned_to(p, 16); }
constexpr int kLayerMaxT = 1 << 30;
constexpr int kNormMaxH = 16384;

inline bool row_type_ok(int dtype) {
  return dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_FP16 || dtype == MOE_DTYPE_FP32;
}
inline int chunk_elems(int dtype) { return dtype == MOE_DTYPE_FP32 ? 4 : 8; }
// whether every tensor lies at a multiple of its element's size
template <typename... P>
bool whole_elems(int dtype, P... p) {
  return (aligned_to(p, dtype == MOE_DTYPE_FP32 ? 4 : 2) && ...);
}

// p in [0, 1]: threshold round(p 2^32) on the 32 random bits of an element
bool drop_args(double p, const int64_t* rng, DropArgs* d) {
  *d = DropArgs{};
  if (!(p >= 0.0 && p <= 1.0)) return false;
  if (p == 0.0) return true;
  if (!rng || !aligned_to(rng, 8)) return false;
  const double thr = std::nearbyint(p * 4294967296.0);
  d->rng = rng;
  d->all = thr > 4294967295.0;  // from p = 1 - 2^-33 on no word reaches it
  d->threshold = d->all ? 0u : static_cast<uint32_t>(thr);
  d->scale = d->all ? 0.f : static_cast<float>(1.0 / (1.0 - p));
  return true;
}

// ------------------------------------------------------------ residual norm
// Blocks of one row each: threads hold VPT chunks.  One chunk per thread up
// to max_threads, then two, four, and (fp32 rows over 8192) eight.
struct NormShape {
  int vpt, threads;
};
NormShape norm_shape(int H, int dtype, int max_threads) {
  const int chunks = (H + chunk_elems(dtype) - 1) / chunk_elems(dtype);
  int vpt = 1;
  while (vpt < 8 && (chunks + vpt - 1) / vpt > max_threads) vpt *= 2;
  const int threads = ((chunks + vpt - 1) / vpt + 31) / 32 * 32;
  return NormShape{vpt, threads};
}

// The backward: 8 elements a thread up to rows of 7168 (896 threads of 72
// registers), 16 up to 8192, 32 beyond.  Eight against sixteen, us for 8192
// rows, add + norm / with post norm, channel gate and dropout too:
//           bf16                         fp32
//   3600    87 : 66    164 : 138         103 : 86    229 : 199
//   4096    87 : 68    166 : 142         105 : 96    234 : 199
//   4608    93 : 104   185 : 220         137 : 166   280 : 369
//   5120    95 : 105   190 : 226         120 : 136   246 : 319
//   6144   103 : 109   219 : 245         163 : 189   311 : 392
//   7168   111 : 118   248 : 272         153 : 172   368 : 421
// and 114 : 122 at 2880 with all parts.  From 3585 to 4096 sixteen, of which
// two blocks fit an SM, is the faster one: the rule does not follow that yet.
// Rows that are not 16-byte aligned want eight throughout (4097 bf16, add +
// norm: 183 : 290).
struct NormBwdShape {
  int elems, threads, blocks_per_sm;
};
NormBwdShape norm_bwd_shape(int H, int dtype) {
  NormBwdShape s;
  s.elems = H <= 7168 ? 8 : H <= 8192 ? 16 : 32;
  const int vpt = s.elems / chunk_elems(dtype);
  const int chunks = (H + chunk_elems(dtype) - 1) / chunk_elems(dtype);
  s.threads = ((chunks + vpt - 1) / vpt + 31) / 32 * 32;
  s.blocks_per_sm = std::min(8, std::max(1, (s.elems == 8 ? 896 : 512) / s.threads));
  return s;
}
// Blocks of the backward (each leaves one partial row per sum over tokens); a
// B200's SMs, so that the workspace's size does not depend on a device
int norm_bwd_blocks(int T, int H, int dtype) {
  return std::min(T, 148 * norm_bwd_shape(H, dtype).blocks_per_sm);
}

// Rows in flight of a ring of n tensors, for blocks_per_sm blocks an SM; 0 if
// not one fits.
int ring_stages(size_t row_bytes, int n, int blocks_per_sm) {
  const size_t room = (static_cast<size_t>(kSmemOptin) - 4096) / blocks_per_sm - 2048;
  return static_cast<int>(std::min<size_t>(RowRing::kMaxStages, room / (n * row_bytes)));
}
template <auto Kern, typename A>
moe_status_t launch_rows_ring(A a, int n, int blocks_per_sm, size_t row_bytes, int grid,
                              int threads, bool ring, cudaStream_t st) {
  size_t smem = 0;
  a.stages = 1;
  a.wait_ns = g_wait_limit_ns;
  a.stall_test = g_stall_test;
  if (ring) {
    a.stages = ring_stages(row_bytes, n, blocks_per_sm);
    smem = a.stages * n * row_bytes;
    // one limit for every row length: calls at once may differ in theirs
    if (a.stages < 1 || !allow_smem<KernelKey<Kern>>(Kern, kSmemOptin - 4096)) return MOE_ERR_CUDA;
  }
  launch_k(Kern, grid, threads, smem, st, a);
  count_launch();
  return launch_status();
}

template <int DT, bool AL>
moe_status_t launch_norm_fwd(const NormArgs& a, cudaStream_t st) {
  const int sms = std::max(1, layer_sms());
  const size_t row = static_cast<size_t>(a.H) * Chunk<DT>::SIZE;
  const int n = 1 + (a.res ? 1 : 0) + (a.gate_kind == MOE_GATE_ELEMENT ? 1 : 0);
  ProfScope prof(MOE_PROF_NORM_FWD, st);
  // few rows: a chunk per thread up to 1024 of them, each row its own block
  NormShape s = norm_shape(a.H, DT, 1024);
  if (s.vpt == 1 && a.T <= 2 * sms)
    return launch_rows_ring<norm_fwd_kernel<DT, AL, 1, false>>(a, n, 1, row, a.T, s.threads, false,
                                                               st);
  // else at most 512 threads, 64 registers each: 1024 threads an SM
  s = norm_shape(a.H, DT, 512);
  const int per_sm = std::min(16, std::max(1, 1024 / s.threads));
  const int grid = static_cast<int>(std::min<long long>(a.T, 1ll * sms * per_sm));
  // one or two chunks a thread: aligned rows by the ring (three tensors' rows
  // of 16 KB fit twice for each of two blocks), others by the threads
  if (s.vpt == 1)
    return launch_rows_ring<norm_fwd_kernel<DT, AL, 1, AL>>(a, n, per_sm, row, grid, s.threads, AL,
                                                            st);
  if (s.vpt == 2)
    return launch_rows_ring<norm_fwd_kernel<DT, AL, 2, AL>>(a, n, per_sm, row, grid, s.threads, AL,
                                                            st);
  if constexpr (DT == kRowFp32) {
    if (s.vpt == 8)
      return launch_rows_ring<norm_fwd_kernel<DT, AL, 8, false>>(a, n, per_sm, row, grid,
                                                                 s.threads, false, st);
  }
  return launch_rows_ring<norm_fwd_kernel<DT, AL, 4, false>>(a, n, per_sm, row, grid, s.threads,
                                                             false, st);
}

template <int DT, bool AL, int ELEMS, int MAXT, bool RING>
moe_status_t launch_norm_bwd_t(const NormBwdArgs& a, const NormBwdShape& s, int grid,
                               cudaStream_t st) {
  const int n = (a.w_pre ? 2 : 0) + (a.dr ? 1 : 0) + (a.dy ? 1 : 0) +
                (a.dy && a.gate_kind == MOE_GATE_ELEMENT ? 1 : 0);
  return launch_rows_ring<norm_bwd_kernel<DT, AL, ELEMS / Chunk<DT>::CH, MAXT, RING>>(
      a, n, s.blocks_per_sm, static_cast<size_t>(a.H) * Chunk<DT>::SIZE, grid, s.threads, RING, st);
}

template <int DT, bool AL>
moe_status_t launch_norm_bwd(const NormBwdArgs& a, void* dw_post, void* dw_pre, void* dgate_c,
                             cudaStream_t st) {
  const NormBwdShape s = norm_bwd_shape(a.H, DT);
  const int grid = norm_bwd_blocks(a.T, a.H, DT);
  moe_status_t stt = MOE_OK;
  ProfScope prof(MOE_PROF_NORM_BWD, st);
  if (a.T > 0) {
    // rows over 8192 do not fit twice: their threads load for themselves
    stt = a.H <= 3584    ? launch_norm_bwd_t<DT, AL, 8, 448, AL>(a, s, grid, st)
          : s.elems == 8 ? launch_norm_bwd_t<DT, AL, 8, 896, AL>(a, s, grid, st)
          : s.elems == 16 ? launch_norm_bwd_t<DT, AL, 16, 512, AL>(a, s, grid, st)
                          : launch_norm_bwd_t<DT, AL, 32, 512, false>(a, s, grid, st);
    if (stt != MOE_OK) return stt;
  }
  if (dw_post || dw_pre || dgate_c) {
    launch_k(norm_sums_kernel<DT>, dim3((a.H + 127) / 128, 3), 1024, 0, st,
             static_cast<const float*>(a.part), a.T > 0 ? grid : 0, a.H, dw_post, dw_pre,
             dgate_c);
    count_launch();
    stt = launch_status();
  }
  return stt;
}

template <template <int, bool> class F, typename... A>
moe_status_t by_row_type(int dtype, bool al, A&&... args) {
  switch (dtype) {
    case MOE_DTYPE_BF16: return al ? F<kRowBf16, true>::run(args...) : F<kRowBf16, false>::run(args...);
    case MOE_DTYPE_FP16: return al ? F<kRowFp16, true>::run(args...) : F<kRowFp16, false>::run(args...);
    default: return al ? F<kRowFp32, true>::run(args...) : F<kRowFp32, false>::run(args...);
  }
}
template <int DT, bool AL>
struct NormFwd {
  static moe_status_t run(const NormArgs& a, cudaStream_t st) {
    return launch_norm_fwd<DT, AL>(a, st);
  }
};
template <int DT, bool AL>
struct NormBwd {
  static moe_status_t run(const NormBwdArgs& a, void* p, void* q, void* g, cudaStream_t st) {
    return launch_norm_bwd<DT, AL>(a, p, q, g, st);
  }
};
template <int DT, bool AL>
struct Dropout {
  static moe_status_t run(const void* x, void* out, int T, int H, const DropArgs& d,
                          cudaStream_t st) {
    const long long chunks = static_cast<long long>(T) * ((H + Chunk<DT>::CH - 1) / Chunk<DT>::CH);
    const int grid = static_cast<int>(
        std::min<long long>((chunks + 255) / 256,
                            static_cast<long long>(std::max(1, layer_sms())) * kDropBlocksPerSM));
    ProfScope prof(MOE_PROF_DROPOUT, st);
    const bool wide = AL && H % (2 * Chunk<DT>::CH) == 0 &&
                      ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & 31) == 0;
    if constexpr (AL) {
      if (wide) launch_k(dropout_kernel<DT, true, 2>, grid, 256, 0, st, x, out, T, H, d);
    }
    if (!wide) launch_k(dropout_kernel<DT, AL, 1>, grid, 256, 0, st, x, out, T, H, d);
    count_launch();
    return launch_status();
  }
};

template <typename... P>
bool all_aligned(int H, int dtype, P... p) {
  return H % chunk_elems(dtype) == 0 && (aligned16(p) && ...);
}

// ------------------------------------------------------------- gated FFN
bool ffn_shape_ok(int T, int H, int I, int dtype, int act) {
  if (T < 0 || T > kLayerMaxT) return false;
  if (H < 64 || I < 64 || (H % 16) || (I % 16) || H > (1 << 24) || I > (1 << 24)) return false;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return false;
  return act == MOE_ACT_SILU || act == MOE_ACT_GELU_TANH;
}

// fp32 map of 32 x 32 boxes (128-byte swizzle)
bool tmap_f32(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer,
              uint64_t pitch_bytes) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {pitch_bytes};
  cuuint32_t box[2] = {32, 32};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launches on `st`, in clusters of `cluster` CTAs where that is over 1 (a
// kernel with __cluster_dims__ needs 1); `dependent`: may start while the
// stream's preceding kernel still runs (the kernel waits for it itself).
template <typename... KArgs, typename... Args>
void launch_dep(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, int cluster,
                bool dependent, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  cudaLaunchKernelEx(&cfg, kern, args...);
  count_launch();
}

// One GEMM's operands: A is [M, K] (or [K, M] with a_mn), B is [N, K] (or
// [K, N] with B_MN; for kDenseGlu [2N, K]), 16-bit elements, the rows dense.
struct DenseOp {
  const void *A, *B;
  DenseArgs args;
  void* out;
};

// n GEMMs in one launch on CTA pairs.  Z: kDenseGlu: written where given;
// kDenseGluBwd: read.
template <int DT, int EPI, bool B_MN>
moe_status_t launch_dense_pair(const DenseOp* ops, int n, float* Z, bool dependent,
                               int prof_kind, cudaStream_t st) {
  using C = DensePairCfg<EPI>;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  // in decreasing order of K
  const DenseOp* order[3];
  for (int i = 0; i < n; ++i) {
    int j = i;
    for (; j > 0 && order[j - 1]->args.K < ops[i].args.K; --j) order[j] = order[j - 1];
    order[j] = &ops[i];
  }
  DenseMaps maps;
  DenseBatch batch{};
  batch.n = n;
  long long tiles = 0;
  for (int i = 0; i < n; ++i) {
    DenseArgs& args = batch.prob[i];
    args = order[i]->args;
    const void *A = order[i]->A, *B = order[i]->B;
    void* out = order[i]->out;
    const uint64_t M = args.M, N = args.N, K = args.K;
    if (args.K == batch.prob[0].K) batch.n_long = i + 1;
    args.tile_n = (EPI == kDenseGlu || B_MN) ? 256 : pair_tile_n(args.N, false);
    args.m_tiles = (args.M + 255) / 256;
    args.n_tiles = EPI == kDenseGlu ? (args.N + 127) / 128
                                    : (args.N + args.tile_n - 1) / args.tile_n;
    args.out = out;
    tiles += static_cast<long long>(args.m_tiles) * args.n_tiles;
    bool ok = args.a_mn ? tmap_2d(&maps.a[i], A, M, K, M * 2, 64, 64, sw)
                        : tmap_2d(&maps.a[i], A, K, M, K * 2, 64, 128, sw);
    if (B_MN) ok = ok && tmap_2d(&maps.b[i], B, N, K, N * 2, 64, 64, sw);
    else if (EPI == kDenseGlu) ok = ok && tmap_2d(&maps.b[i], B, K, 2 * N, K * 2, 64, 64, sw);
    else ok = ok && tmap_2d(&maps.b[i], B, K, N, K * 2, 64, args.tile_n / 2, sw);
    const uint64_t ld = (EPI == kDenseGluBwd ? 2 * N : N) * 2;
    ok = ok && tmap_2d(&maps.o[i], out, N, M, ld, 64, 32, sw);
    if (EPI == kDenseGluBwd)
      ok = ok && tmap_2d(&maps.o2, static_cast<uint16_t*>(out) + N, N, M, ld, 64, 32, sw) &&
           tmap_f32(&maps.o3, Z, 2 * N, M, 2 * N * 4);
    if (EPI == kDenseGlu && Z) {
      ok = ok && tmap_f32(&maps.o2, Z, N, M, 2 * N * 4) &&
           tmap_f32(&maps.o3, Z + N, N, M, 2 * N * 4);
      args.save_z = 1;
    }
    if (!ok) return MOE_ERR_CUDA;
  }
  for (int i = n; i < 3; ++i) {
    maps.a[i] = maps.a[0];
    maps.b[i] = maps.b[0];
    maps.o[i] = maps.o[0];
  }
  if (EPI == kDenseStore || (EPI == kDenseGlu && !Z)) maps.o2 = maps.o[0];
  if (EPI == kDenseStore || !Z) maps.o3 = maps.o[0];
  constexpr auto kern = dense_pair_kernel<DT, EPI, B_MN>;
  if (!allow_smem<KernelKey<kern>>(kern, C::SMEM_BYTES)) return MOE_ERR_CUDA;
  if (tiles >= (1ll << 30)) return MOE_ERR_UNSUPPORTED;
  const int pairs = static_cast<int>(std::min<long long>(layer_sms() / 2, tiles));
  if (pairs <= 0) return MOE_ERR_CUDA;
  ProfScope prof(prof_kind, st);
  launch_dep(kern, dim3(2 * pairs), C::THREADS, C::SMEM_BYTES, 1, dependent, st, maps, batch,
             g_wait_limit_ns, g_stall_test);
  return launch_status();
}

// How a dense GEMM runs: splits = 0 on CTA pairs (256 x 256 tiles), else as
// 128 x bn tiles of `splits` CTAs each: the least of the estimated times (us),
//   pair   6 + rounds of 74 tiles, 0.28 per 64 of K each, + one epilogue;
//   split  2 + rounds of 148 CTAs (clusters that share SMs cost most of a
//          round more), each 3, 2 + splits / 4 for the exchange, 0.20 or 0.26
//          per 64 of K and the epilogue's share.
// The counts are a B200's 148 SMs, not the device's: an estimate for this one
// chip, the same wherever it is asked for.  Fitted to cold-weight graph
// timings; forward of one block, pair against the chosen split: 60 / 31 us at
// 64 x 7168 x 2048 (T x H x I), 44 / 24 us at 64 x 2880 x 2880, 33 / 21 us at
// 1021 x 2048 x 768, 22 / 9 us at 512 x 256 x 512; weight gradients of 128 x
// 7168 x 2048: pair 36 us, the best split 66 us.
struct DensePlan {
  int bn, splits;
  double us;
};
DensePlan dense_plan(int M, int N, int K, int epi) {
  const int cols = epi == kDenseGlu ? 2 * N : N;  // accumulator columns
  const int k = (K + 63) / 64;
  const double pair_epi = epi == kDenseGluBwd ? 6.0 : 3.5;
  const long long pair_tiles = ((M + 255ll) / 256) * ((cols + 255) / 256);
  const long long pair_rounds = (pair_tiles + 73) / 74;
  double best = 6.0 + pair_rounds * 0.28 * k + pair_epi +
                (pair_rounds - 1) * std::max(0.0, pair_epi - 0.28 * k);
  DensePlan plan{256, 0, best};
  if ((M + 127ll) / 128 > 65535) return plan;  // m-tiles are the grid's y
  for (int bn = 64; bn <= 128; bn *= 2)
    for (int sp = 1; sp <= 4 && sp <= k; sp *= 2) {
      const long long ctas = ((M + 127ll) / 128) * ((cols + bn - 1) / bn) * sp;
      const double rounds = ctas <= 148 ? 1.0 : sp == 1 ? ctas / 148.0 : (ctas + 147) / 148 * 0.85;
      const double t = 2.0 + rounds * (3.0 + (sp > 1 ? 2.0 + 0.25 * sp : 0.0) +
                                       ((k + sp - 1) / sp) * (bn == 128 ? 0.26 : 0.20) +
                                       (epi == kDenseGluBwd ? 4.5 : 1.5) * bn / 128 / sp);
      if (t < best) {
        best = t;
        plan = DensePlan{bn, sp, t};
      }
    }
  return plan;
}

template <int DT, int EPI, bool A_MN, bool B_MN, int BN>
moe_status_t launch_dense_split(const DenseOp& op, float* Z, int splits, bool dependent,
                                int prof_kind, cudaStream_t st) {
  using C = DenseSplitCfg<EPI, A_MN, B_MN, BN>;
  DenseArgs args = op.args;
  const void *A = op.A, *B = op.B;
  const uint64_t M = args.M, N = args.N, K = args.K;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  args.m_tiles = (args.M + 127) / 128;
  args.n_tiles = EPI == kDenseGlu ? (args.N + BN / 2 - 1) / (BN / 2) : (args.N + BN - 1) / BN;
  args.out = op.out;
  args.Z = Z;
  args.wait_ns = g_wait_limit_ns;
  args.stall_test = g_stall_test;
  CUtensorMap ta, tb;
  bool ok = A_MN ? tmap_2d(&ta, A, M, K, M * 2, 64, 64, sw) : tmap_2d(&ta, A, K, M, K * 2, 64, 128, sw);
  if (B_MN) ok = ok && tmap_2d(&tb, B, N, K, N * 2, 64, 64, sw);
  else if (EPI == kDenseGlu) ok = ok && tmap_2d(&tb, B, K, 2 * N, K * 2, 64, BN / 2, sw);
  else ok = ok && tmap_2d(&tb, B, K, N, K * 2, 64, BN, sw);
  if (!ok) return MOE_ERR_CUDA;
  constexpr auto kern = dense_split_kernel<DT, EPI, A_MN, B_MN, BN>;
  const long long ctas = 1ll * args.n_tiles * splits * args.m_tiles;
  const int ns = ctas <= layer_sms() ? C::NS1 : C::NS2;
  if (!allow_smem<KernelKey<kern>>(kern, C::smem_bytes(C::NS1))) return MOE_ERR_CUDA;
  ProfScope prof(prof_kind, st);
  launch_dep(kern, dim3(args.n_tiles * splits, args.m_tiles), C::THREADS, C::smem_bytes(ns), splits,
             dependent, st, ta, tb, args, splits, ns);
  return launch_status();
}

// One dense GEMM.  `dependent`: the kernel before it on the stream is one of
// this call's, which lets it start early; it waits for that one before it
// reads anything but weights.
template <int DT, int EPI, bool A_MN, bool B_MN>
moe_status_t launch_dense(const DensePlan& p, const DenseOp& op, float* Z, bool dependent,
                          int prof_kind, cudaStream_t st) {
  if (p.splits == 0) return launch_dense_pair<DT, EPI, B_MN>(&op, 1, Z, dependent, prof_kind, st);
  if (p.bn == 128)
    return launch_dense_split<DT, EPI, A_MN, B_MN, 128>(op, Z, p.splits, dependent, prof_kind, st);
  return launch_dense_split<DT, EPI, A_MN, B_MN, 64>(op, Z, p.splits, dependent, prof_kind, st);
}

// Tokens up to which the forward runs as two weight streams on the legacy
// MMA (ffn_rows_kernel).
constexpr int kRowsMaxT = 32;

// The plan of one product (MOE_FFN_*) of a call.
DensePlan ffn_plan(int T, int H, int I, int product) {
  switch (product) {
    case MOE_FFN_GATE_UP: return dense_plan(T, I, H, kDenseGlu);
    case MOE_FFN_DOWN: return dense_plan(T, H, I, kDenseStore);
    case MOE_FFN_DH: return dense_plan(T, I, H, kDenseGluBwd);
    case MOE_FFN_DX: return dense_plan(T, H, 2 * I, kDenseStore);
    case MOE_FFN_DW1: return dense_plan(2 * I, H, T, kDenseStore);
    default: return dense_plan(H, I, T, kDenseStore);
  }
}
// dX, dW1 and dW2 (their plans in g): all on CTA pairs in one launch, or each
// as it is best by itself
bool ffn_merged(int T, int H, int I, const DensePlan (&g)[3]) {
  const auto tiles = [](int n) { return (n + 255) / 256; };
  const auto steps = [](int k) { return (k + 63) / 64; };
  const double work = (static_cast<double>(tiles(T)) * tiles(H) * steps(2 * I) +
                       (static_cast<double>(tiles(2 * I)) * tiles(H) +
                        static_cast<double>(tiles(H)) * tiles(I)) * steps(T)) / 74;
  const int k_long = steps(std::max(2 * I, T));
  return 9.5 + 0.28 * std::max<double>(k_long, 1.08 * work) < g[0].us + g[1].us + g[2].us;
}

template <int DT, bool GLU, int NT, int RT>
moe_status_t launch_rows_t(const RowsArgs& a, int prof_kind, cudaStream_t st) {
  const int per = (GLU ? 8 : 16) * RT;
  constexpr auto kern = ffn_rows_kernel<DT, GLU, NT, RT>;
  constexpr int smem = RowsCfg<NT, RT>::SMEM_BYTES;
  if (!allow_smem<KernelKey<kern>>(kern, smem)) return MOE_ERR_CUDA;
  ProfScope prof(prof_kind, st);
  launch_dep(kern, dim3((a.N + per - 1) / per), 32 * kRowsWarps, smem, 1, !GLU, st, a);
  return launch_status();
}
template <int DT, bool GLU>
moe_status_t launch_rows(const RowsArgs& a, int prof_kind, cudaStream_t st) {
  // Over 8 tokens a block takes two row tiles: every block reads all tokens,
  // and with one tile those reads outweigh the weights (24 tokens of 2880 x
  // 2880: 20.1 against 17.9 us; 16 of 7168 x 2048: 22.9 against 20.6).
  if (a.T <= 8) return launch_rows_t<DT, GLU, 1, 1>(a, prof_kind, st);
  if (a.T <= 16) return launch_rows_t<DT, GLU, 2, 2>(a, prof_kind, st);
  if (a.T <= 24) return launch_rows_t<DT, GLU, 3, 2>(a, prof_kind, st);
  return launch_rows_t<DT, GLU, 4, 2>(a, prof_kind, st);
}

template <int DT>
moe_status_t ffn_fwd_t(const void* X, const void* W1, const void* W2, int T, int H, int I,
                       int act, const void* add, void* Y, float* Z, void* h, cudaStream_t st) {
  if (T <= kRowsMaxT) {
    const RowsArgs up{W1, X, nullptr, h, Z, T, I, H, act};
    const moe_status_t s = launch_rows<DT, true>(up, MOE_PROF_FFN_GATE_UP, st);
    if (s != MOE_OK) return s;
    return launch_rows<DT, false>(RowsArgs{W2, h, add, Y, nullptr, T, H, I, act},
                                  MOE_PROF_FFN_DOWN, st);
  }
  DenseOp up{X, W1, {}, h}, down{h, W2, {}, Y};
  up.args.M = T; up.args.N = I; up.args.K = H; up.args.act = act;
  down.args.M = T; down.args.N = H; down.args.K = I; down.args.add = add;
  const moe_status_t s = launch_dense<DT, kDenseGlu, false, false>(
      ffn_plan(T, H, I, MOE_FFN_GATE_UP), up, Z, false, MOE_PROF_FFN_GATE_UP, st);
  if (s != MOE_OK) return s;
  return launch_dense<DT, kDenseStore, false, false>(ffn_plan(T, H, I, MOE_FFN_DOWN), down, nullptr,
                                                     true, MOE_PROF_FFN_DOWN, st);
}

template <int DT>
moe_status_t ffn_bwd_t(const void* dY, const void* X, const void* W1, const void* W2, int T,
                       int H, int I, int act, const float* Z, const void* h, const void* add,
                       void* dX, void* dW1, void* dW2, void* dZ, cudaStream_t st) {
  DenseOp dh{dY, W2, {}, dZ};
  dh.args.M = T; dh.args.N = I; dh.args.K = H; dh.args.act = act;
  moe_status_t s = launch_dense<DT, kDenseGluBwd, false, true>(
      ffn_plan(T, H, I, MOE_FFN_DH), dh, const_cast<float*>(Z), false, MOE_PROF_FFN_DH, st);
  if (s != MOE_OK) return s;
  DenseOp g[3] = {{dZ, W1, {}, dX}, {dZ, X, {}, dW1}, {dY, h, {}, dW2}};
  g[0].args.M = T; g[0].args.N = H; g[0].args.K = 2 * I; g[0].args.add = add;
  g[1].args.M = 2 * I; g[1].args.N = H; g[1].args.K = T; g[1].args.a_mn = 1;
  g[2].args.M = H; g[2].args.N = I; g[2].args.K = T; g[2].args.a_mn = 1;
  DensePlan plan[3] = {ffn_plan(T, H, I, MOE_FFN_DX)};
  if (dW1) {
    plan[1] = ffn_plan(T, H, I, MOE_FFN_DW1);
    plan[2] = ffn_plan(T, H, I, MOE_FFN_DW2);
    if (ffn_merged(T, H, I, plan))
      return launch_dense_pair<DT, kDenseStore, true>(g, 3, nullptr, true, MOE_PROF_FFN_DW, st);
  }
  s = launch_dense<DT, kDenseStore, false, true>(plan[0], g[0], nullptr, true, MOE_PROF_FFN_DX, st);
  for (int i = 1; dW1 && i < 3 && s == MOE_OK; ++i)
    s = launch_dense<DT, kDenseStore, true, true>(plan[i], g[i], nullptr, true, MOE_PROF_FFN_DW, st);
  return s;
}

// Z fp32 [T, 2I], then h 16-bit [T, I]
inline size_t ffn_z_bytes(int T, int I) { return align256(static_cast<size_t>(T) * 2 * I * 4); }

}  // namespace

extern "C" {

// ------------------------------------------------------------ residual norm
moe_status_t moe_residual_norm_fwd(const void* y, const void* res, const void* w_post,
                                   const void* gate, int gate_kind, float scale,
                                   const void* w_pre, float w_offset, float eps, double p,
                                   const int64_t* rng, int T, int H, int dtype, void* r, void* n,
                                   float* stats, moe_stream_t stream) {
  if (!row_type_ok(dtype) || T < 0 || T > kLayerMaxT || H < 1 || H > kNormMaxH)
    return MOE_ERR_UNSUPPORTED;
  if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_ELEMENT) return MOE_ERR_UNSUPPORTED;
  NormArgs a{};
  if (!drop_args(p, rng, &a.drop)) return MOE_ERR_INVALID_ARG;
  if ((gate_kind != MOE_GATE_NONE) != (gate != nullptr)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!y || (!w_pre != !n) || (!r && !n) || ((w_post || w_pre) && !stats))
    return MOE_ERR_INVALID_ARG;
  if (!whole_elems(dtype, y, res, w_post, gate, w_pre, r, n) || !aligned_to(stats, 4))
    return MOE_ERR_INVALID_ARG;
  a.y = y; a.res = res; a.w_post = w_post; a.gate = gate; a.w_pre = w_pre;
  a.r = r; a.n = n; a.stats = stats; a.T = T; a.H = H; a.gate_kind = gate_kind;
  a.eps = eps; a.scale = scale; a.w_offset = w_offset;
  const void* g = gate_kind >= MOE_GATE_CHANNEL ? gate : nullptr;
  return by_row_type<NormFwd>(dtype, all_aligned(H, dtype, y, res, w_post, g, w_pre, r, n), a,
                              stream);
}

size_t moe_residual_norm_bwd_workspace_bytes(int T, int H, int dtype) {
  if (T <= 0 || H <= 0 || H > kNormMaxH || !row_type_ok(dtype)) return 256;
  return align256(static_cast<size_t>(norm_bwd_blocks(T, H, dtype)) * 3 * H * 4);
}

moe_status_t moe_residual_norm_bwd(const void* dr, const void* dn, const void* y, const void* r,
                                   const float* stats, const void* w_post, const void* gate,
                                   int gate_kind, float scale, const void* w_pre, float w_offset,
                                   double p, const int64_t* rng, int T, int H, int dtype,
                                   void* dres, void* dy, void* dgate, void* dw_post, void* dw_pre,
                                   void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!row_type_ok(dtype) || T < 0 || T > kLayerMaxT || H < 1 || H > kNormMaxH)
    return MOE_ERR_UNSUPPORTED;
  if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_ELEMENT) return MOE_ERR_UNSUPPORTED;
  NormBwdArgs a{};
  if (!drop_args(p, rng, &a.drop)) return MOE_ERR_INVALID_ARG;
  if (!w_post != !dw_post || !w_pre != !dw_pre) return MOE_ERR_INVALID_ARG;
  if ((gate_kind != MOE_GATE_NONE) != (gate != nullptr) || !gate != !dgate)
    return MOE_ERR_INVALID_ARG;
  if ((w_post || gate) && !dy) return MOE_ERR_INVALID_ARG;
  if (T > 0) {
    if (!dr && !dn) return MOE_ERR_INVALID_ARG;
    if (!w_pre != !dn || (w_pre && !r) || (dy && !y) || (!dy && !dres)) return MOE_ERR_INVALID_ARG;
    if ((w_post || w_pre) && !stats) return MOE_ERR_INVALID_ARG;
    if (!ws || ws_bytes < moe_residual_norm_bwd_workspace_bytes(T, H, dtype))
      return MOE_ERR_INVALID_ARG;
  }
  if (!whole_elems(dtype, dr, dn, y, r, w_post, gate, w_pre, dres, dy, dgate, dw_post, dw_pre) ||
      !aligned_to(stats, 4) || !aligned_to(ws, 4))
    return MOE_ERR_INVALID_ARG;
  a.dr = dr; a.dn = dn; a.y = y; a.r = r; a.w_post = w_post; a.gate = gate; a.w_pre = w_pre;
  a.stats = stats; a.dres = dres; a.dy = dy; a.dgate = dgate;
  a.part = static_cast<float*>(ws); a.T = T; a.H = H; a.gate_kind = gate_kind;
  a.scale = scale; a.w_offset = w_offset;
  const void* g = gate_kind >= MOE_GATE_CHANNEL ? gate : nullptr;
  void* ge = gate_kind == MOE_GATE_ELEMENT ? dgate : nullptr;
  return by_row_type<NormBwd>(
      dtype, all_aligned(H, dtype, dr, dn, y, r, w_post, g, w_pre, dres, dy, ge), a, dw_post,
      dw_pre, gate_kind == MOE_GATE_CHANNEL ? dgate : nullptr, stream);
}

// ---------------------------------------------------------------- dropout
moe_status_t moe_dropout(const void* x, int T, int H, int dtype, double p, const int64_t* rng,
                         void* out, moe_stream_t stream) {
  if (!row_type_ok(dtype) || T < 0 || T > kLayerMaxT || H < 1 || H > kLayerMaxT)
    return MOE_ERR_UNSUPPORTED;
  DropArgs d;
  if (!rng || !aligned_to(rng, 8) || !drop_args(p, rng, &d)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !out || !whole_elems(dtype, x, out)) return MOE_ERR_INVALID_ARG;
  if (p == 0.0) {  // nothing is dropped: every word is at least 0
    d.rng = rng;
    d.scale = 1.f;
  }
  return by_row_type<Dropout>(dtype, all_aligned(H, dtype, x, out), x, out, T, H, d, stream);
}

// -------------------------------------------------------------- gated FFN
size_t moe_ffn_saved_bytes(int T, int H, int I) {
  (void)H;
  if (T <= 0 || I <= 0) return 256;
  return ffn_z_bytes(T, I) + align256(static_cast<size_t>(T) * I * 2);
}
size_t moe_ffn_workspace_bytes(int T, int H, int I) {
  (void)H;
  if (T <= 0 || I <= 0) return 256;
  return align256(static_cast<size_t>(T) * 2 * I * 2);
}

int moe_ffn_kernel(int T, int H, int I, int product, int need_dw) {
  if (!ffn_shape_ok(T, H, I, MOE_DTYPE_BF16, MOE_ACT_SILU) || T == 0) return -1;
  if (product < MOE_FFN_GATE_UP || product > MOE_FFN_DW2) return -1;
  if (product >= MOE_FFN_DW1 && !need_dw) return -1;
  if (product <= MOE_FFN_DOWN && T <= kRowsMaxT) return MOE_FFN_TOKENS;
  if (product >= MOE_FFN_DX && need_dw) {
    const DensePlan g[3] = {ffn_plan(T, H, I, MOE_FFN_DX), ffn_plan(T, H, I, MOE_FFN_DW1),
                            ffn_plan(T, H, I, MOE_FFN_DW2)};
    if (ffn_merged(T, H, I, g)) return MOE_FFN_PAIRS_MERGED;
  }
  const DensePlan d = ffn_plan(T, H, I, product);
  return d.splits == 0 ? MOE_FFN_PAIRS : d.bn * 16 + d.splits;
}

moe_status_t moe_ffn_fwd(const void* X, const void* W1, const void* W2, int T, int H, int I,
                         int dtype, int act, const void* add, void* Y, void* saved,
                         size_t saved_bytes, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!ffn_shape_ok(T, H, I, dtype, act)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!X || !W1 || !W2 || !Y) return MOE_ERR_INVALID_ARG;
  if (saved ? saved_bytes < moe_ffn_saved_bytes(T, H, I)
            : (!ws || ws_bytes < moe_ffn_workspace_bytes(T, H, I)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(W1) || !aligned16(W2) || !aligned16(Y) || !aligned16(add) ||
      !aligned16(saved) || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  float* Z = static_cast<float*>(saved);
  void* h = saved ? at<void>(saved, ffn_z_bytes(T, I)) : ws;
  return dtype == MOE_DTYPE_BF16
             ? ffn_fwd_t<kBf16>(X, W1, W2, T, H, I, act, add, Y, Z, h, stream)
             : ffn_fwd_t<kFp16>(X, W1, W2, T, H, I, act, add, Y, Z, h, stream);
}

moe_status_t moe_ffn_bwd(const void* dY, const void* X, const void* W1, const void* W2, int T,
                         int H, int I, int dtype, int act, const void* saved, size_t saved_bytes,
                         const void* add, void* dX, void* dW1, void* dW2, void* ws,
                         size_t ws_bytes, moe_stream_t stream) {
  if (!ffn_shape_ok(T, H, I, dtype, act)) return MOE_ERR_UNSUPPORTED;
  if (!dW1 != !dW2) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = stream;
  if (T == 0) {
    const size_t wb = static_cast<size_t>(H) * I * 2;
    if (dW1 && (cudaMemsetAsync(dW1, 0, 2 * wb, st) != cudaSuccess ||
                cudaMemsetAsync(dW2, 0, wb, st) != cudaSuccess))
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!dY || !X || !W1 || !W2 || !saved || !dX || !ws) return MOE_ERR_INVALID_ARG;
  if (saved_bytes < moe_ffn_saved_bytes(T, H, I) || ws_bytes < moe_ffn_workspace_bytes(T, H, I))
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(dY) || !aligned16(X) || !aligned16(W1) || !aligned16(W2) || !aligned16(saved) ||
      !aligned16(add) || !aligned16(dX) || !aligned16(dW1) || !aligned16(dW2) || !aligned16(ws))
    return MOE_ERR_INVALID_ARG;
  const float* Z = static_cast<const float*>(saved);
  const void* h = at<void>(saved, ffn_z_bytes(T, I));
  return dtype == MOE_DTYPE_BF16
             ? ffn_bwd_t<kBf16>(dY, X, W1, W2, T, H, I, act, Z, h, add, dX, dW1, dW2, ws, st)
             : ffn_bwd_t<kFp16>(dY, X, W1, W2, T, H, I, act, Z, h, add, dX, dW1, dW2, ws, st);
}

}  // extern "C"
