// Dense GEMMs of the gated feed-forward block on CTA pairs:
//   kDenseGlu     h[t, i] = act(g) u,  [g | u] = X W1^T        (gate_up forward)
//   kDenseStore   out = A B^T (+ add)                          (down forward, dX, dW1, dW2)
//   kDenseGluBwd  dh = dY W2;  dg = dh u act'(g), du = dh act(g)
//
// One pair of CTAs (two SMs) computes a 256 x Nt tile of the output with
// tcgen05.mma.cta_group::2 (M = 256, N = Nt <= 256): each CTA stages its 128
// rows of A and half of the tile's B columns, 64 of K per stage, and both
// CTAs' copies complete on the leader's barrier.  Either operand may be
// K-major (rows of K contiguous elements) or MN-major (K rows of contiguous
// M or N elements, read in place as 64-column atoms), so no operand is ever
// transposed or copied:
//                 A                        B
//   gate_up fwd   X   [T, H]   K-major     W1 [2I, H]  K-major
//   down fwd      h   [T, I]   K-major     W2 [H, I]   K-major
//   dh            dY  [T, H]   K-major     W2 [H, I]   MN-major
//   dX            dZ1 [T, 2I]  K-major     W1 [2I, H]  MN-major
//   dW1           dZ1 [T, 2I]  MN-major    X  [T, H]   MN-major
//   dW2           dY  [T, H]   MN-major    h  [T, I]   MN-major
// Ragged M, N and K come from the copies' zero fill and the stores' clipping.
// The fp32 accumulators (two sets of 256 TMEM columns, so that a tile's
// epilogue overlaps the next tile's mainloop) are summed over K in one fixed
// order: every result is the same from run to run.
//
// h and dZ are rounded to the 16-bit type on their way out, here and in the
// other forms: they are operands of the next product, and kind::f16 takes both
// operands in one 16-bit type.  Each such rounding is at most half a step of
// a value that is summed over with others of either sign, so the 2-norm of a
// result is off by one more half step beside its own rounding: 0.0023 against
// 0.0017 of a pass in fp32 (bf16, against 64 bits).  In fp32 (as TF32, half
// the rate) or as two 16-bit terms (twice the products) the second GEMM would
// cost twice as much.  The sums before and after stay in fp32, and so do the
// saved g and u: rounded too, dX would be off 1.8 times as far.
//
// The tensor pipe is the bound.  8192 x 7168 x 2048 (T x H x I), bf16, each
// launch by itself: gate_up forward 314 us (1.53 PFLOP/s, 0.90 of the measured
// burst peak), down forward 163 us (1.47), dh 190 us (1.27: 256 tiles are 3.5
// rounds of 74), dX + dW1 + dW2 in one launch 780 us (1.54).  Back to back the
// power limit takes over: the whole pass 1.70 ms, 1.27 PFLOP/s, 0.90 of the
// sustained peak.
//
// Waits are bounded and the teardown is the one of the grouped pair kernel.
#pragma once

#include "gemm_pair.cuh"

namespace moe {

enum DenseEpi { kDenseStore = 0, kDenseGlu = 1, kDenseGluBwd = 2 };
enum DenseAct { kActSilu = 0, kActGeluTanh = 1 };
enum HalfType { kBf16 = 0, kFp16 = 1 };

// One GEMM of a launch.
struct DenseArgs {
  int M, N, K;         // output rows and columns (Glu: N = I), reduction length
  int m_tiles, n_tiles;
  int tile_n;          // MMA columns of a tile (kDenseGlu: 256)
  int a_mn;            // A is MN-major
  const void* add;     // kDenseStore: [M, N] added before the rounding, or null
  void* out;           // kDenseStore: [M, N]
  const float* Z;      // kDenseGluBwd: saved [g | u], fp32 [M, 2N]
  int save_z;          // kDenseGlu: write Z through its tensor maps
  int act;
  uint64_t wait_ns;
  int stall_test;
};

// Programmatic dependent launch: wait until the stream's preceding kernel has
// completed (returns at once in an ordinary launch); let the next one start.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---------------------------------------------------------- 16-bit values
template <int DT>
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
  if constexpr (DT == kBf16) {
    return pack_bf16x2(a, b);
  } else {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}
template <int DT>
__device__ __forceinline__ float2 unpack_h2(uint32_t v) {
  if constexpr (DT == kBf16) {
    return make_float2(bf16_lo(v), bf16_hi(v));
  } else {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
}

// ------------------------------------------------------------ activations
// 1 / (1 + exp(-x)).  The hardware tanh form (absolute error 2^-12) that the
// expert block uses would cost an fp16 result half its last place, and a small
// logistic most of its bits, so this one goes through the hardware's powers of
// two and reciprocal, each documented to a few fp32 steps (2^-22 and 2^-23
// relative); the product x log2(e), rounded, adds |x| 2^-24.  Beside the
// 16-bit rounding of h (2^-11 at least) both are lost.  1 + exp(-x) is in [1,
// inf], and the reciprocal of inf is 0.
__device__ __forceinline__ float logistic(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

// gelu (tanh form): 0.5 x (1 + tanh(k (x + c x^3))) = x sigma(2 k (x + c x^3)).
constexpr float kGelu2K = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_fwd(float x) {
  if constexpr (ACT == kActSilu) return x * logistic(x);
  else return x * logistic(kGelu2K * fmaf(kGeluC * x * x, x, x));
}
// a = act(x), da = act'(x)
template <int ACT>
__device__ __forceinline__ void act_both(float x, float& a, float& da) {
  const float s = logistic(ACT == kActSilu ? x : kGelu2K * fmaf(kGeluC * x * x, x, x));
  a = x * s;
  if constexpr (ACT == kActSilu) da = fmaf(a, 1.f - s, s);
  else da = fmaf(a * (1.f - s), kGelu2K * fmaf(3.f * kGeluC * x, x, 1.f), s);
}
// f with the activation as a constant (the choice is made once for many
// elements)
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  if (act == kActSilu) f(Int<kActSilu>{});
  else f(Int<kActGeluTanh>{});
}

// Instruction descriptor of kind::f16 with the given 16-bit operand type.
template <int DT>
__host__ __device__ constexpr uint32_t idesc_h_f32(int M, int N, bool a_mn, bool b_mn) {
  const uint32_t d = idesc_bf16_f32(M, N, a_mn, b_mn);
  return DT == kBf16 ? d : d & ~((1u << 7) | (1u << 10));  // format 0: fp16
}

// Up to three GEMMs in one launch (the backward's dX, dW1 and dW2), in
// decreasing order of K; the first `n_long` of them have the same K.
struct DenseBatch {
  DenseArgs prob[3];
  int n, n_long;
};
struct DenseMaps {
  CUtensorMap a[3], b[3], o[3];
  CUtensorMap o2, o3;  // kDenseGlu: gate and up halves of Z; kDenseGluBwd: du, Z
};

template <int EPI>
struct DensePairCfg {
  static constexpr int BK = 64;
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int B_BYTES = 128 * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int ATOM = 64 * BK * 2;             // one 64-column MN-major atom
  static constexpr int EPI_WARPS = 4;                  // one per TMEM lane quarter
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int BOX = 4096;                     // 32 rows x 128 bytes
  static constexpr int NBOX = 2;                       // store boxes per epilogue warp
  static constexpr int RING = EPI_WARPS * NBOX * BOX;
  // kDenseGluBwd: per epilogue warp a box of saved gates and one of ups
  static constexpr int ZBUF = EPI == kDenseGluBwd ? EPI_WARPS * 2 * BOX : 0;
  static constexpr int MISC = 512;
  static constexpr int NS = (kSmemOptin - 1024 - RING - ZBUF - MISC) / STAGE_BYTES;
  static constexpr int SMEM_BYTES = 1024 + NS * STAGE_BYTES + RING + ZBUF + MISC;
  static constexpr int TMEM_COLS = 512;
  static constexpr int ACC_STRIDE = 256;
  static_assert(NS >= 4, "stages");
  static_assert((2 * NS + 8 + EPI_WARPS) * 8 + 32 <= MISC, "barrier area");
};

// Tiles in groups of 8 m-tiles, m fastest: the 74 tiles in flight cover
// about 8 x 9 tiles, so that each operand row is read from L2 by several
// pairs at once and a group's B columns stay in L2 over its m-tiles.
__device__ __forceinline__ void dense_tile(const DenseArgs& a, int tile, int& mt, int& nt) {
  constexpr int G = 8;
  const int per = G * a.n_tiles;
  const int g = tile / per, in = tile - g * per;
  const int gm = min(G, a.m_tiles - g * G);
  nt = in / gm;
  mt = g * G + (in - nt * gm);
}

// The tiles of one pair of CTAs, the same sequence in every role.  Long tiles
// (the first n_long problems) go round the pairs; where that leaves `rem`
// pairs one long tile ahead, the others first take as many short tiles as
// make up for it, then short tiles go round all pairs, the less loaded first.
// (One launch against one per GEMM: the 6.05 + 3.03 + 12.1 rounds of the
// 8192 x 7168 x 2048 backward take 7 + 4 + 13.)
struct DenseSchedule {
  int p, P, n_a, n_b, rem, s;
  bool light_first;
  int mine_a, i;

  __device__ __forceinline__ DenseSchedule(const DenseBatch& b, int pair, int pairs)
      : p(pair), P(pairs), n_a(0), n_b(0), i(0) {
    for (int q = 0; q < b.n; ++q)
      (q < b.n_long ? n_a : n_b) += b.prob[q].m_tiles * b.prob[q].n_tiles;
    mine_a = p < n_a ? (n_a - p + P - 1) / P : 0;
    rem = n_a % P;
    s = 0;
    light_first = true;
    if (rem && n_b) {
      const int ka = b.prob[0].K, kb = b.prob[b.n_long].K;
      s = min((ka + kb / 2) / kb, (n_b + P - rem - 1) / (P - rem));
      light_first = ka > s * kb;
    }
  }
  // next tile: its problem and place in it; false after the last
  __device__ __forceinline__ bool next(const DenseBatch& b, int& prob, int& mt, int& nt) {
    int t;
    if (i < mine_a) {
      t = p + i * P;
    } else {
      const int j = i - mine_a;
      const bool light = rem && p >= rem;
      const int L = P - rem;
      if (light && j < s) {
        t = j * L + (p - rem);
      } else {
        const int order = rem && light_first ? (light ? p - rem : p + L) : p;
        t = (rem ? s * L : 0) + (j - (light ? s : 0)) * P + order;
      }
      if (t >= n_b) return false;
      t += n_a;
    }
    ++i;
    prob = 0;
    while (t >= b.prob[prob].m_tiles * b.prob[prob].n_tiles) {
      t -= b.prob[prob].m_tiles * b.prob[prob].n_tiles;
      ++prob;
    }
    dense_tile(b.prob[prob], t, mt, nt);
    return true;
  }
};

// One epilogue warp's ring of staged boxes: 32 rows x 128 bytes, 128-byte
// swizzled, one row per lane.  A box is written with one TMA store, which
// clips what lies outside the tensor.
template <int NBOX>
struct BoxRing {
  uint8_t* base;
  int slot;
  __device__ __forceinline__ uint8_t* open(int lane) {
    uint8_t* box = base + slot * 4096;
    slot = slot + 1 == NBOX ? 0 : slot + 1;
    if (lane == 0) bulk_wait_group_read<NBOX - 1>();  // the slot's last store has read it
    __syncwarp();
    return box;
  }
  __device__ __forceinline__ void close(const CUtensorMap* tm, const uint8_t* box, int x, int y,
                                        uint64_t pol, int lane) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(tm, box, x, y, pol);
      bulk_commit_group();
    }
  }
  // 64 16-bit values per lane, as 32 packed words
  __device__ __forceinline__ void put(const CUtensorMap* tm, const uint32_t* w, int x, int y,
                                      uint64_t pol, int lane) {
    uint8_t* box = open(lane);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<uint4*>(box + swz_offset(lane, c, 128)) =
          make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    close(tm, box, x, y, pol, lane);
  }
  // 32 fp32 values per lane
  __device__ __forceinline__ void put_f32(const CUtensorMap* tm, const float* v, int x, int y,
                                          uint64_t pol, int lane) {
    uint8_t* box = open(lane);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<float4*>(box + swz_offset(lane, c, 128)) =
          make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    close(tm, box, x, y, pol, lane);
  }
};

// maps.a, maps.b: the operands (boxes in the launcher); maps.o: the outputs in
// boxes of 64 columns x 32 rows; kDenseGlu: maps.o2 / maps.o3 = the gate and up
// halves of Z in 32 x 32 fp32 boxes; kDenseGluBwd: maps.o = dg, maps.o2 = du,
// maps.o3 = Z [M, 2N] in 32 x 32 fp32 boxes, which each epilogue warp loads one
// 32-column step ahead, also into its next tile.  (Read by the threads, a row
// each, the 256 KB of Z a CTA's tile needs take the load unit 8.6 us, about a
// mainloop of K = 1536.)
template <int DT, int EPI, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(DensePairCfg<EPI>::THREADS, 1)
    dense_pair_kernel(const __grid_constant__ DenseMaps maps,
                      const __grid_constant__ DenseBatch batch, uint64_t wait_ns,
                      int stall_test) {
  using C = DensePairCfg<EPI>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sStage = smem;
  uint8_t* sRing = sStage + C::NS * C::STAGE_BYTES;
  uint8_t* sZ = sRing + C::RING;
  uint64_t* full = reinterpret_cast<uint64_t*>(sZ + C::ZBUF);
  uint64_t* empty = full + C::NS;
  uint64_t* acc_full = empty + C::NS;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* final_bar = acc_empty + 2;
  uint64_t* peer_done = final_bar + 1;
  uint64_t* drained = peer_done + 1;
  uint64_t* z_full = drained + 1;                      // one per epilogue warp
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(z_full + C::EPI_WARPS);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  int* s_issued = reinterpret_cast<int*>(s_tmem + 4);  // [0] own copies, [2] the peer's

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * C::EPI_WARPS);
    }
    for (int i = 0; i < C::EPI_WARPS; ++i) mbar_init(&z_full[i], 1);
    mbar_init(final_bar, 1);
    mbar_init(peer_done, 1);
    mbar_init(drained, 1);
    for (int i = 0; i < 4; ++i) s_issued[i] = 0;
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < batch.n; ++i) {
      prefetch_tmap(&maps.a[i]);
      prefetch_tmap(&maps.b[i]);
      prefetch_tmap(&maps.o[i]);
    }
    if constexpr (EPI != kDenseStore) {
      prefetch_tmap(&maps.o2);
      prefetch_tmap(&maps.o3);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(s_tmem, C::TMEM_COLS);
    tmem_relinquish_pair();
  }
  // everything above touches only shared memory, TMEM and the kernel's
  // parameters; a launch that may overlap the kernel before it waits here
  pdl_wait();
  pdl_launch();
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  auto lead = [&](const void* p) { return mapa_shared(smem_u32(p), 0); };
  // columns of a tile: MN-major B loads whole 64-column atoms, and a last
  // tile with at most 128 columns runs with N = 128
  auto tile_cols = [&](const DenseArgs& args, int nt) {
    if constexpr (B_MN) return args.N - nt * 256 <= 128 ? 128 : 256;
    else return args.tile_n;
  };
  const uint32_t stage_bytes =
      (EPI == kDenseGlu || B_MN)
          ? static_cast<uint32_t>(C::STAGE_BYTES)
          : static_cast<uint32_t>(C::A_BYTES + batch.prob[0].tile_n * C::BK);
  DenseSchedule sched(batch, blockIdx.x >> 1, gridDim.x >> 1);
  int pi, mt, nt;
  // f with the problem's index as a constant: operands' tensor maps and sizes
  // at fixed parameter addresses (an index in a register cost the producer
  // 10% of a GEMM with MN-major B: dX of 16384 x 2048 x 768 77 us against 70)
  auto with_problem = [](int i, auto f) {
    if (EPI != kDenseStore || !B_MN || i == 0) f(Int<0>{});
    else if (i == 1) f(Int<1>{});
    else f(Int<2>{});
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0, n_st = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && sched.next(batch, pi, mt, nt)) {
        with_problem(pi, [&](auto index) {
          constexpr int I = decltype(index)::value;
          const DenseArgs& args = batch.prob[I];
          const int m0 = mt * 256 + static_cast<int>(rank) * 128;
          const int n0 = EPI == kDenseGlu
                             ? nt * 128 + static_cast<int>(rank) * 64
                             : nt * (B_MN ? 256 : args.tile_n) +
                                   static_cast<int>(rank) * (tile_cols(args, nt) >> 1);
          const int k_iters = (args.K + C::BK - 1) / C::BK;
          [[maybe_unused]] const int up0 = n0 + args.N;  // kDenseGlu: first up row
          auto loads = [&](auto mn) {
            for (int kt = 0; kt < k_iters; ++kt) {
              if (!mbar_wait(&empty[stage], phase ^ 1, s_abort, wait_ns)) { ok = false; break; }
              uint8_t* st = sStage + stage * C::STAGE_BYTES;
              uint8_t* sb = st + C::A_BYTES;
              const int k0 = kt * C::BK;
              const uint32_t fb = lead(&full[stage]);
              if (leader) mbar_arrive_expect_tx(&full[stage], 2 * stage_bytes);
              if constexpr (decltype(mn)::value != 0) {
                tma_load_2d_pair(st, &maps.a[I], fb, m0, k0);
                tma_load_2d_pair(st + C::ATOM, &maps.a[I], fb, m0 + 64, k0);
              } else {
                tma_load_2d_pair(st, &maps.a[I], fb, k0, m0);
              }
              if constexpr (B_MN) {
                tma_load_2d_pair(sb, &maps.b[I], fb, n0, k0);
                tma_load_2d_pair(sb + C::ATOM, &maps.b[I], fb, n0 + 64, k0);
              } else if constexpr (EPI == kDenseGlu) {
                tma_load_2d_pair(sb, &maps.b[I], fb, k0, n0);             // gate rows
                tma_load_2d_pair(sb + C::ATOM, &maps.b[I], fb, k0, up0);  // up rows
              } else {
                tma_load_2d_pair(sb, &maps.b[I], fb, k0, n0);
              }
              ++n_st;
              if (++stage == C::NS) {
                stage = 0;
                phase ^= 1;
              }
            }
          };
          if (EPI == kDenseStore && B_MN && args.a_mn) loads(Int<1>{});
          else loads(Int<0>{});
        });
      }
      s_issued[0] = n_st;
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------------------------------------------------- MMA (leader)
      constexpr uint16_t kBoth = 0x3;
      const uint64_t b_desc0 =
          smem_desc(smem_u32(sStage) + C::A_BYTES, B_MN ? C::ATOM : 16, 1024, kLayoutSW128);
      constexpr uint64_t kStageInc = C::STAGE_BYTES >> 4;
      constexpr uint64_t kBStep = B_MN ? (2048 >> 4) : (32 >> 4);
      int stage = 0, local = 0;
      uint64_t soff = 0;
      uint32_t phase = 0;
      bool ok = true;
      // one tile; A's order is a constant of the loop (descriptor steps held
      // in registers cost the issuing thread 6% of the dX GEMM)
      auto mainloop = [&](auto mn, uint32_t t_acc, int cols, int k_iters) {
        constexpr bool kAMN = decltype(mn)::value != 0;
        constexpr uint64_t kAStep = kAMN ? (2048 >> 4) : (32 >> 4);  // 16 of K
        const uint64_t a_desc0 =
            smem_desc(smem_u32(sStage), kAMN ? C::ATOM : 16, 1024, kLayoutSW128);
        const uint32_t idesc = idesc_h_f32<DT>(256, cols, kAMN, B_MN);
        for (int kt = 0; kt < k_iters; ++kt) {
          if (!warp_wait(&full[stage], phase, s_abort, wait_ns)) return false;
          tc_fence_after();
          const uint64_t da = a_desc0 + soff, db = b_desc0 + soff;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < C::BK / 16; ++kk)
              umma_bf16_pair(t_acc, da + kk * kAStep, db + kk * kBStep, idesc,
                             (kt | kk) ? 1u : 0u);
            umma_commit_pair_mc(&empty[stage], kBoth);
          }
          __syncwarp();
          soff += kStageInc;
          if (++stage == C::NS) {
            stage = 0;
            soff = 0;
            phase ^= 1;
          }
        }
        return true;
      };
      if (stall_test) ok = warp_wait(final_bar, 0, s_abort, wait_ns);
      for (; ok && sched.next(batch, pi, mt, nt); ++local) {
        const DenseArgs& args = batch.prob[pi];
        const int cols = tile_cols(args, nt);
        const int k_iters = (args.K + C::BK - 1) / C::BK;
        const int b = local & 1;
        const uint32_t use = (local >> 1) & 1;
        const uint32_t t_acc = tmem_base + b * C::ACC_STRIDE;
        if (!warp_wait_cluster(&acc_empty[b], use ^ 1, s_abort, wait_ns)) { ok = false; break; }
        tc_fence_after();
        if (EPI == kDenseStore && B_MN && args.a_mn)
          ok = mainloop(Int<1>{}, t_acc, cols, k_iters);
        else
          ok = mainloop(Int<0>{}, t_acc, cols, k_iters);
        if (!ok) break;
        if (elect_one()) umma_commit_pair_mc(&acc_full[b], kBoth);
        __syncwarp();
      }
      if (elect_one()) umma_commit_pair_mc(final_bar, kBoth);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int ew = warp & 3;  // TMEM lane quarter
    const uint32_t lane_base = static_cast<uint32_t>(ew * 32) << 16;
    const uint64_t pol = policy_evict_normal();
    // Z is read again only in the backward: it leaves L2 to h and the operands
    // (forward and dX of 16384 x 2048 x 768, a few passes: 281 -> 263 us)
    [[maybe_unused]] const uint64_t pol_z = policy_evict_first();
    BoxRing<C::NBOX> ring{sRing + (warp - 2) * C::NBOX * C::BOX, 0};
    const int my_row = static_cast<int>(rank) * 128 + ew * 32;  // in the tile
    // kDenseGluBwd: the next 32-column step of saved gates and ups
    uint8_t* zb = sZ + (warp - 2) * 2 * C::BOX;
    uint64_t* zbar = &z_full[warp - 2];
    uint32_t z_phase = 0;
    bool z_pending = false;
    auto fetch_z = [&](int col, int y) {
      if (lane == 0) {
        mbar_arrive_expect_tx(zbar, 2 * C::BOX);
        tma_load_2d(zb, &maps.o3, zbar, col, y);
        tma_load_2d(zb + C::BOX, &maps.o3, zbar, batch.prob[0].N + col, y);
      }
      z_pending = true;
    };
    int pi1 = 0, mt1 = 0, nt1 = 0;  // the tile after this one
    bool more = sched.next(batch, pi, mt, nt);
    if constexpr (EPI == kDenseGluBwd) {
      if (more) fetch_z(nt * 256, mt * 256 + my_row);
    }
    for (int local = 0; more; ++local, pi = pi1, mt = mt1, nt = nt1) {
      more = sched.next(batch, pi1, mt1, nt1);
      const DenseArgs& args = batch.prob[0];
      const int b = local & 1;
      const uint32_t use = (local >> 1) & 1;
      const int y0 = mt * 256 + my_row;
      const int row = y0 + lane;
      const bool rows_any = y0 < args.M;
      const uint32_t t_acc = tmem_base + lane_base + b * C::ACC_STRIDE;
      if (!warp_wait(&acc_full[b], use, s_abort, wait_ns)) break;
      tc_fence_after();
      if constexpr (EPI == kDenseGlu) {
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {  // 64 output columns: [gate 64 | up 64] in TMEM
          const int col = nt * 128 + q * 64;
          if (col >= args.N || !rows_any) break;
          uint32_t hp[32];
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            float g[32], u[32];
            tmem_ld<32>(t_acc + q * 128 + c, g);
            tmem_ld<32>(t_acc + q * 128 + 64 + c, u);
            tmem_ld_wait();
            if (args.save_z && col + c < args.N) {
              ring.put_f32(&maps.o2, g, col + c, y0, pol_z, lane);
              ring.put_f32(&maps.o3, u, col + c, y0, pol_z, lane);
            }
            with_act(args.act, [&](auto act) {
              constexpr int A = decltype(act)::value;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                hp[c / 2 + i] = pack_h2<DT>(act_fwd<A>(g[2 * i]) * u[2 * i],
                                            act_fwd<A>(g[2 * i + 1]) * u[2 * i + 1]);
            });
          }
          ring.put(&maps.o[0], hp, col, y0, pol, lane);
        }
      } else if constexpr (EPI == kDenseGluBwd) {
        const int col0 = nt * 256, hi = min(args.N, col0 + 256);
        bool ok = true;
#pragma unroll 1
        for (int c0 = 0; ok && col0 + c0 < hi; c0 += 64) {
          const int col = col0 + c0;
          uint32_t dgp[32], dup[32];
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            if (col + c >= hi) break;  // a last box of 16 or 32 columns
            if (!warp_wait(zbar, z_phase, s_abort, wait_ns)) { ok = false; break; }
            z_phase ^= 1;
            z_pending = false;
            float g[32], u[32];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 zg = *reinterpret_cast<const float4*>(zb + swz_offset(lane, i, 128));
              const float4 zu =
                  *reinterpret_cast<const float4*>(zb + C::BOX + swz_offset(lane, i, 128));
              g[4 * i] = zg.x; g[4 * i + 1] = zg.y; g[4 * i + 2] = zg.z; g[4 * i + 3] = zg.w;
              u[4 * i] = zu.x; u[4 * i + 1] = zu.y; u[4 * i + 2] = zu.z; u[4 * i + 3] = zu.w;
            }
            // every lane has its row of the boxes before the copies that
            // replace them start (the fence keeps the loads above them)
            fence_proxy_async_smem();
            __syncwarp();
            if (col + c + 32 < hi) fetch_z(col + c + 32, y0);
            else if (more) fetch_z(nt1 * 256, mt1 * 256 + my_row);
            float dh[32];
            tmem_ld<32>(t_acc + c0 + c, dh);
            tmem_ld_wait();
            with_act(args.act, [&](auto act) {
              constexpr int A = decltype(act)::value;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float a0, d0, a1, d1;
                act_both<A>(g[2 * i], a0, d0);
                act_both<A>(g[2 * i + 1], a1, d1);
                dgp[c / 2 + i] = pack_h2<DT>(dh[2 * i] * u[2 * i] * d0,
                                             dh[2 * i + 1] * u[2 * i + 1] * d1);
                dup[c / 2 + i] = pack_h2<DT>(dh[2 * i] * a0, dh[2 * i + 1] * a1);
              }
            });
          }
          if (ok && rows_any) {
            ring.put(&maps.o[0], dgp, col, y0, pol, lane);
            ring.put(&maps.o2, dup, col, y0, pol, lane);
          }
        }
        if (!ok) break;
      } else {
        with_problem(pi, [&](auto index) {
          constexpr int I = decltype(index)::value;
          const DenseArgs& args = batch.prob[I];
          const bool rows_any = y0 < args.M, rvalid = row < args.M;
          const int Nt = tile_cols(args, nt);
          const int col0 = nt * (B_MN ? 256 : args.tile_n);
          const int hi = rows_any ? min(args.N, col0 + Nt) : col0;
#pragma unroll 1
          for (int c0 = 0; col0 + c0 < hi; c0 += 64) {
            const int col = col0 + c0;
            uint4 ad[8];
            const bool has_add = args.add != nullptr;
            if (has_add) {
              const uint4* ap = reinterpret_cast<const uint4*>(
                  static_cast<const uint16_t*>(args.add) +
                  static_cast<size_t>(rvalid ? row : 0) * args.N + col);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                ad[i] = make_uint4(0, 0, 0, 0);
                if (rvalid && col + 8 * i < hi) ad[i] = ap[i];
              }
            }
            uint32_t w[32];
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
              float v[32];
              tmem_ld<32>(t_acc + c0 + c, v);
              tmem_ld_wait();
              if (has_add) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const uint4 q4 = ad[c / 8 + i / 4];
                  const uint32_t aw = (i & 3) == 0 ? q4.x : (i & 3) == 1 ? q4.y
                                      : (i & 3) == 2 ? q4.z : q4.w;
                  const float2 f = unpack_h2<DT>(aw);
                  v[2 * i] += f.x;
                  v[2 * i + 1] += f.y;
                }
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) w[c / 2 + i] = pack_h2<DT>(v[2 * i], v[2 * i + 1]);
            }
            if (col + 64 <= col0 + Nt) {
              ring.put(&maps.o[I], w, col, y0, pol, lane);
            } else if (rvalid) {
              // a tile narrower than whole boxes: the columns past it belong
              // to the next tile
              uint4* op = reinterpret_cast<uint4*>(static_cast<uint16_t*>(args.out) +
                                                   static_cast<size_t>(row) * args.N + col);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (col + 8 * i < hi)
                  op[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            }
          }
        });
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) MOE_ACC_RELEASE(lead(&acc_empty[b]));
    }
    if constexpr (EPI == kDenseGluBwd) {
      if (z_pending && lane == 0) drain_wait(zbar, z_phase, wait_ns);  // after an abort
    }
    if (lane == 0) bulk_wait_group<0>();  // every staged store has been written
    __syncwarp();
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    drain_wait(final_bar, 0, wait_ns);
    if (!leader) {
      st_shared_cluster_s32(lead(&s_issued[2]), s_issued[0]);
      mbar_arrive_cluster(lead(peer_done));
      drain_wait(drained, 0, wait_ns);
    } else {
      drain_wait_cluster(peer_done, 0, wait_ns);
      drain_pair_copies(full, C::NS, stage_bytes, s_issued[0], s_issued[2], wait_ns);
      mbar_arrive_cluster(mapa_shared(smem_u32(drained), 1));
    }
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
  }
}

}  // namespace moe
