// The dense GEMMs of dense_pair.cuh for few rows or small outputs, where
// 256 x 256 tiles would leave most SMs without work: one 128 x BN tile per
// cluster of S CTAs (BN = 64 or 128, S = 1, 2 or 4), each CTA summing its
// share of K (tcgen05, M = 128) and then finishing 1/S of the tile's columns:
// the partial tiles meet in distributed shared memory and are added in rank
// order, so results do not depend on timing.  Same operands, epilogues,
// formulas and roundings as the pair kernel.
//
// Between tens and a few hundred rows the weights' bytes are the floor, and
// what costs is latency, so: all first stages of weights are requested before
// the kernel waits for the one before it (programmatic dependent launch; the
// activations come after the wait), what the epilogue reads is requested
// before the accumulator is awaited, and the epilogue is S times shorter.
// Stages: 192 KB in flight for one CTA an SM; with more CTAs than SMs, 96 KB
// each for two.  A CTA's 32 KB per 64 of K reach it at about 64 bytes a clock,
// which bounds the larger cases.  Forward, cold weights: 128 x 7168 x 2048
// (T x H x I) 30 us, 2.9 TB/s; 1021 x 2048 x 768 22 us, where 9.6 GFLOP take 6
// at the peak; training pass 512 x 256 x 512 fp16 30 us in four launches.
#pragma once

#include "ffn_rows.cuh"

namespace moe {

template <int EPI, bool A_MN, bool B_MN, int BN>
struct DenseSplitCfg {
  static constexpr int BK = 64;
  static constexpr int A_BYTES = 128 * BK * 2;
  static constexpr int B_BYTES = BN * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int ATOM = 64 * BK * 2;
  // stages: 192 KB of them for one CTA an SM, 96 KB each for two
  static constexpr int NS1 = BN == 128 ? 6 : 8, NS2 = NS1 / 2;
  static constexpr int MISC = 256;
  static constexpr int smem_bytes(int ns) { return 1024 + ns * STAGE_BYTES + MISC; }
  static constexpr int THREADS = 192;
  static_assert(NS2 * STAGE_BYTES >= BN * 128 * 4, "the partial tile overlays the stages");
  static_assert(smem_bytes(NS1) <= kSmemOptin && (2 * NS1 + 2) * 8 + 8 <= MISC, "shared memory");
};

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// What a thread's epilogue reads for 32 columns of its row, in 16-byte pieces.
struct EpiIn {
  uint4 v[16];
};

template <int DT, int EPI, bool A_MN, bool B_MN, int BN>
__global__ void __launch_bounds__(192, 2)
    dense_split_kernel(const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmB, const DenseArgs args,
                       int splits, int ns) {
  using C = DenseSplitCfg<EPI, A_MN, B_MN, BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + ns * C::STAGE_BYTES);
  uint64_t* empty = full + ns;
  uint64_t* acc_full = empty + ns;
  uint64_t* never = acc_full + 1;  // stall test: nothing arrives here
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(never + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = splits > 1 ? cluster_ctarank() : 0;
  const int nt = blockIdx.x / splits, mt = blockIdx.y;
  const int m0 = mt * 128;
  const int n0 = nt * (EPI == kDenseGlu ? BN / 2 : BN);
  const int k_all = (args.K + C::BK - 1) / C::BK;
  const int kb = static_cast<int>(static_cast<long long>(k_all) * rank / splits);
  const int ke = static_cast<int>(static_cast<long long>(k_all) * (rank + 1) / splits);
  const uint64_t wait_ns = args.wait_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ns; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(never, 1);
    *s_abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  pdl_launch();

  int issued = 0;  // producer: stages requested
  if (warp == 0) {
    if (lane == 0) {
      auto load_b = [&](int kt, int stage) {
        uint8_t* sb = smem + stage * C::STAGE_BYTES + C::A_BYTES;
        const int k0 = kt * C::BK;
        mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES);
        if constexpr (B_MN) {
#pragma unroll
          for (int i = 0; i < BN / 64; ++i)
            tma_load_2d(sb + i * C::ATOM, &tmB, &full[stage], n0 + 64 * i, k0);
        } else if constexpr (EPI == kDenseGlu) {
          tma_load_2d(sb, &tmB, &full[stage], k0, n0);
          tma_load_2d(sb + BN / 2 * 128, &tmB, &full[stage], k0, n0 + args.N);
        } else {
          tma_load_2d(sb, &tmB, &full[stage], k0, n0);
        }
      };
      auto load_a = [&](int kt, int stage) {
        uint8_t* sa = smem + stage * C::STAGE_BYTES;
        const int k0 = kt * C::BK;
        if constexpr (A_MN) {
          tma_load_2d(sa, &tmA, &full[stage], m0, k0);
          tma_load_2d(sa + C::ATOM, &tmA, &full[stage], m0 + 64, k0);
        } else {
          tma_load_2d(sa, &tmA, &full[stage], k0, m0);
        }
      };
      const int n = ke - kb, ahead = min(n, ns);
      // B is a weight except for the weights' gradients (A_MN)
      if constexpr (!A_MN)
        for (int i = 0; i < ahead; ++i) load_b(kb + i, i);
      pdl_wait();
      for (int i = 0; i < ahead; ++i) {
        if constexpr (A_MN) load_b(kb + i, i);
        load_a(kb + i, i);
      }
      issued = ahead;
      int stage = ahead == ns ? 0 : ahead;
      uint32_t phase = ahead == ns ? 1 : 0;
      for (int i = ahead; i < n; ++i) {
        if (!mbar_wait(&empty[stage], phase ^ 1, s_abort, wait_ns)) break;
        load_b(kb + i, stage);
        load_a(kb + i, stage);
        ++issued;
        if (++stage == ns) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_h_f32<DT>(128, BN, A_MN, B_MN);
    const uint64_t a0 = smem_desc(smem_u32(smem), A_MN ? C::ATOM : 16, 1024, kLayoutSW128);
    const uint64_t b0 =
        smem_desc(smem_u32(smem) + C::A_BYTES, B_MN ? C::ATOM : 16, 1024, kLayoutSW128);
    constexpr uint64_t kAStep = A_MN ? (2048 >> 4) : (32 >> 4);
    constexpr uint64_t kBStep = B_MN ? (2048 >> 4) : (32 >> 4);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    if (args.stall_test) ok = warp_wait(never, 0, s_abort, wait_ns);
    for (int kt = kb; ok && kt < ke; ++kt) {
      if (!warp_wait(&full[stage], phase, s_abort, wait_ns)) { ok = false; break; }
      tc_fence_after();
      if (elect_one()) {
        const uint64_t off = static_cast<uint64_t>(stage) * (C::STAGE_BYTES >> 4);
#pragma unroll
        for (int kk = 0; kk < C::BK / 16; ++kk)
          umma_bf16(tmem, a0 + off + kk * kAStep, b0 + off + kk * kBStep, idesc,
                    (kt > kb || kk) ? 1u : 0u);
        umma_commit(&empty[stage]);
      }
      __syncwarp();
      if (++stage == ns) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (elect_one()) umma_commit(acc_full);
    __syncwarp();
  }

  // ---------------------------------------------------------------- epilogue
  // This CTA's columns of the tile: [c_lo, c_lo + CS) (kDenseGlu: of the
  // tile's BN / 2 outputs).
  constexpr int OUT = EPI == kDenseGlu ? BN / 2 : BN;
  const int CS = OUT / splits, c_lo = static_cast<int>(rank) * CS;
  const bool epi = warp >= 2;
  const int ew = warp & 3, row_t = ew * 32 + lane;
  const int row = m0 + row_t;
  const bool rvalid = epi && row < args.M;
  const size_t N = args.N;
  // requests what 32 columns from tile column c need
  auto fetch = [&](EpiIn& in, int c) {
#pragma unroll
    for (int i = 0; i < 16; ++i) in.v[i] = make_uint4(0, 0, 0, 0);
    if constexpr (EPI == kDenseGluBwd) {
      const float* z = args.Z + static_cast<size_t>(row) * 2 * N + n0 + c;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (rvalid && c + 4 * i < c_lo + CS && n0 + c + 4 * i < args.N) {
          in.v[i] = *reinterpret_cast<const uint4*>(z + 4 * i);
          in.v[8 + i] = *reinterpret_cast<const uint4*>(z + N + 4 * i);
        }
    } else if constexpr (EPI == kDenseStore) {
      if (args.add == nullptr) return;
      const uint16_t* ad =
          static_cast<const uint16_t*>(args.add) + static_cast<size_t>(row) * N + n0 + c;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (rvalid && c + 8 * i < c_lo + CS && n0 + c + 8 * i < args.N)
          in.v[i] = *reinterpret_cast<const uint4*>(ad + 8 * i);
    }
  };
  EpiIn in;
  bool ok = true;
  if (epi) {
    pdl_wait();  // Z and add come from earlier kernels
    fetch(in, c_lo);
    ok = warp_wait(acc_full, 0, s_abort, wait_ns);
    tc_fence_after();
  }
  const uint32_t t_acc = tmem + (static_cast<uint32_t>(ew * 32) << 16);
  float* s_part = reinterpret_cast<float*>(smem);  // [BN][128], over the stages
  if (splits > 1) {
    if (epi && ok) {
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        float v[32];
        tmem_ld<32>(t_acc + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) s_part[(c + i) * 128 + row_t] = v[i];
      }
    }
    cluster_sync_all();
  }
  if (epi && ok) {
    // 8 accumulator columns from tile column c
    auto acc8 = [&](int c, float* v) {
      if (splits == 1) {
        __syncwarp();
        tmem_ld<8>(t_acc + c, v);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
        for (int s = 0; s < splits; ++s) {
          const uint32_t p = mapa_shared(smem_u32(s_part + c * 128 + row_t), s);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += ld_shared_cluster_f32(p + i * 512);
        }
      }
    };
#pragma unroll 1
    for (int c32 = c_lo; c32 < c_lo + CS; c32 += 32) {
      if (c32 != c_lo) fetch(in, c32);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = c32 + 8 * q, col = n0 + c;
        if (c >= c_lo + CS || col >= args.N) break;  // uniform over the warp
        const size_t at = static_cast<size_t>(row) * N + col;
        float v[8];
        acc8(c, v);
        if constexpr (EPI == kDenseGlu) {
          float u[8], h[8];
          acc8(c + BN / 2, u);
          with_act(args.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = act_fwd<decltype(act)::value>(v[i]) * u[i];
          });
          if (rvalid && args.Z) {
            float4* z = reinterpret_cast<float4*>(const_cast<float*>(args.Z) +
                                                  static_cast<size_t>(row) * 2 * N + col);
            z[0] = make_float4(v[0], v[1], v[2], v[3]);
            z[1] = make_float4(v[4], v[5], v[6], v[7]);
            z += N / 4;
            z[0] = make_float4(u[0], u[1], u[2], u[3]);
            z[1] = make_float4(u[4], u[5], u[6], u[7]);
          }
          if (rvalid)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(args.out) + at) =
                make_uint4(pack_h2<DT>(h[0], h[1]), pack_h2<DT>(h[2], h[3]),
                           pack_h2<DT>(h[4], h[5]), pack_h2<DT>(h[6], h[7]));
        } else if constexpr (EPI == kDenseGluBwd) {
          float dg[8], du[8];
          with_act(args.act, [&](auto act) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 zg = in.v[2 * q + i / 4], zu = in.v[8 + 2 * q + i / 4];
            const uint32_t gw = i % 4 == 0 ? zg.x : i % 4 == 1 ? zg.y : i % 4 == 2 ? zg.z : zg.w;
            const uint32_t uw = i % 4 == 0 ? zu.x : i % 4 == 1 ? zu.y : i % 4 == 2 ? zu.z : zu.w;
            float a, da;
            act_both<decltype(act)::value>(__uint_as_float(gw), a, da);
            dg[i] = v[i] * __uint_as_float(uw) * da;
            du[i] = v[i] * a;
          }
          });
          uint16_t* o = static_cast<uint16_t*>(args.out) + static_cast<size_t>(row) * 2 * N + col;
          if (rvalid) {
            *reinterpret_cast<uint4*>(o) =
                make_uint4(pack_h2<DT>(dg[0], dg[1]), pack_h2<DT>(dg[2], dg[3]),
                           pack_h2<DT>(dg[4], dg[5]), pack_h2<DT>(dg[6], dg[7]));
            *reinterpret_cast<uint4*>(o + N) =
                make_uint4(pack_h2<DT>(du[0], du[1]), pack_h2<DT>(du[2], du[3]),
                           pack_h2<DT>(du[4], du[5]), pack_h2<DT>(du[6], du[7]));
          }
        } else {
          if (args.add) {
            const uint32_t aw[4] = {in.v[q].x, in.v[q].y, in.v[q].z, in.v[q].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = unpack_h2<DT>(aw[i]);
              v[2 * i] += f.x;
              v[2 * i + 1] += f.y;
            }
          }
          if (rvalid)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(args.out) + at) =
                make_uint4(pack_h2<DT>(v[0], v[1]), pack_h2<DT>(v[2], v[3]),
                           pack_h2<DT>(v[4], v[5]), pack_h2<DT>(v[6], v[7]));
        }
      }
    }
  }

  // ---------------------------------------------------------------- teardown
  // the other CTAs' reads of this one's partial tile
  if (splits > 1) cluster_sync_all();
  tc_fence_before();
  __syncthreads();
  if (warp == 0 && lane == 0) {
    if (*s_abort) {
      // after a wait that ran out: copies and MMAs in flight
      for (int i = max(0, issued - ns); i < issued; ++i)
        drain_wait(&full[i % ns], (i / ns) & 1, wait_ns);
      drain_wait(acc_full, 0, wait_ns);
    }
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, BN);
  }
}

}  // namespace moe
