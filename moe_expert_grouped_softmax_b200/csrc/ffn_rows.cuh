// Gated feed-forward block for a few tokens (decoding): both products stream
// the weights once, so their bytes are the floor (3 H I elements).
//
// The weights are the M operand of mma.sync m16n8k16 and the tokens its
// N = 8 columns: a 16-row tile of A is 8 gate rows and the 8 up rows of the
// same outputs (gate_up) or 16 rows of W2 (down), so that a lane's four
// accumulators hold gate and up of the same (output, token) pairs and act(g) u
// needs no exchange.  The sum over K may run in any order as long as A and B
// agree on it, so lane c of a row's four takes elements 8c .. 8c + 7 of each
// 32 of K as its part of two MMAs: every operand is a 16-byte piece that one
// lane brings and uses itself.  The pieces come by asynchronous copies into
// shared memory, several steps deep (registers could not hold that many in
// flight), and need no barrier, since no lane reads another's.  A warp takes
// every 8th 64 of K (the block's 8 warps read 1 KB of a row side by side);
// the warps' partial sums meet in shared memory and are added in warp order.
//
// Legacy MMA is enough here: at 8 columns a tile's 4 KFLOP come with 512
// bytes of weights, far below any tensor rate.
//
// Cold weights, forward: one token of 7168 x 2048 19.3 us (88 MB, 4.6 TB/s;
// the floor is 13.7: 256 and 448 blocks on 296 slots, so both launches end with
// part of the chip idle), 23 of 2880 x 2880 18.9 us (floor 7.8: 180 and 90
// blocks on 148 SMs, two steps in flight a warp where one token has four, and
// every block also reads all tokens).  From 25 tokens on a block's two steps
// take 128 KB, so that only one fits an SM.  Held in registers instead of
// shared memory the loads in flight were fewer: 25 us for one token.
#pragma once

#include "dense_pair.cuh"

namespace moe {

struct RowsArgs {
  const void* W;     // gate_up: [2N, K]; down: [N, K]
  const void* X;     // [T, K]
  const void* add;   // down: [T, N] or null
  void* out;         // [T, N]
  float* Z;          // gate_up: [T, 2N] or null
  int T, N, K, act;
};

// 16 bytes global -> shared, zeros where !in (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int DT>
__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (DT == kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int DT>
__device__ __forceinline__ void put_half(void* p, size_t i, float v) {
  if constexpr (DT == kBf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}
template <int DT>
__device__ __forceinline__ float get_half(const void* p, size_t i) {
  if constexpr (DT == kBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else return __half2float(static_cast<const __half*>(p)[i]);
}

constexpr int kRowsWarps = 8;

// Steps of 64 of K in flight per warp: 96 KB a block where that is two or
// more (two blocks an SM), else two (one block an SM).
template <int NT, int RT>
struct RowsCfg {
  static constexpr int PIECES = 4 * RT + 2 * NT;  // 16 bytes each, per lane and step
  static constexpr int THREADS = 32 * kRowsWarps;
  static constexpr int STEP_BYTES = PIECES * 16 * THREADS;
  static constexpr int DEPTH = 98304 / STEP_BYTES < 2 ? 2 : 98304 / STEP_BYTES;
  static constexpr int PART_BYTES = kRowsWarps * RT * NT * 32 * 16;
  static constexpr int SMEM_BYTES =
      DEPTH * STEP_BYTES > PART_BYTES ? DEPTH * STEP_BYTES : PART_BYTES;
};

// GLU: gate_up (8 RT outputs per block), else down (16 RT outputs); NT
// 8-token columns.
template <int DT, bool GLU, int NT, int RT>
__global__ void __launch_bounds__(32 * kRowsWarps, 2) ffn_rows_kernel(const RowsArgs a) {
  using C = RowsCfg<NT, RT>;
  constexpr int D = C::DEPTH;
  extern __shared__ __align__(128) uint8_t s_ring[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int K = a.K, n0 = blockIdx.x * (GLU ? 8 : 16) * RT;
  const uint16_t* W = static_cast<const uint16_t*>(a.W);
  const uint16_t* X = static_cast<const uint16_t*>(a.X);
  // this lane's two rows of each A tile
  const uint16_t* w_lo[RT];
  const uint16_t* w_hi[RT];
  bool live[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = n0 + r * (GLU ? 8 : 16) + g;
    live[r] = (GLU ? row : row + 8) < a.N;  // N is a multiple of 16: whole tiles
    const size_t lo = live[r] ? row : 0, hi = live[r] ? (GLU ? a.N + row : row + 8) : 0;
    w_lo[r] = W + lo * K;
    w_hi[r] = W + hi * K;
  }
  float acc[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][t][i] = 0.f;

  const int steps = (K + 63) / 64;
  const int mine = steps > warp ? (steps - warp + kRowsWarps - 1) / kRowsWarps : 0;
  const uint32_t ring = smem_u32(s_ring) + threadIdx.x * 16;
  auto piece = [&](int slot, int p) -> uint32_t {
    return static_cast<uint32_t>((slot * C::PIECES + p) * C::THREADS * 16);
  };
  auto issue_w = [&](int i, int slot) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = (warp + i * kRowsWarps) * 64 + 32 * q + 8 * c;
      const int kk = k < K ? k : 0;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        copy16(ring + piece(slot, (q * RT + r) * 2), w_lo[r] + kk, k < K && live[r]);
        copy16(ring + piece(slot, (q * RT + r) * 2 + 1), w_hi[r] + kk, k < K && live[r]);
      }
    }
  };
  auto issue_x = [&](int i, int slot) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int k = (warp + i * kRowsWarps) * 64 + 32 * q + 8 * c;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tok = t * 8 + g;
        const bool in = k < K && tok < a.T;
        copy16(ring + piece(slot, 4 * RT + q * NT + t),
               X + (in ? static_cast<size_t>(tok) * K + k : 0), in);
      }
    }
  };
  if constexpr (GLU) {
    pdl_launch();  // the down product may start reading W2
  } else {
    // h comes from the kernel before, W2 does not
#pragma unroll
    for (int i = 0; i < D; ++i)
      if (i < mine) issue_w(i, i);
    pdl_wait();
  }
#pragma unroll
  for (int i = 0; i < D; ++i) {
    if (i < mine) {
      if constexpr (GLU) issue_w(i, i);
      issue_x(i, i);
    }
    copy_commit();
  }
  int slot = 0;
  for (int i = 0; i < mine; ++i) {
    copy_wait<D - 1>();
    const uint8_t* at = s_ring + threadIdx.x * 16;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      uint4 lo[RT], hi[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        lo[r] = *reinterpret_cast<const uint4*>(at + piece(slot, (q * RT + r) * 2));
        hi[r] = *reinterpret_cast<const uint4*>(at + piece(slot, (q * RT + r) * 2 + 1));
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 b = *reinterpret_cast<const uint4*>(at + piece(slot, 4 * RT + q * NT + t));
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          mma16816<DT>(acc[r][t], lo[r].x, hi[r].x, lo[r].y, hi[r].y, b.x, b.y);
          mma16816<DT>(acc[r][t], lo[r].z, hi[r].z, lo[r].w, hi[r].w, b.z, b.w);
        }
      }
    }
    // the MMAs have taken this slot's pieces
    if (i + D < mine) {
      issue_w(i + D, slot);
      issue_x(i + D, slot);
    }
    copy_commit();
    slot = slot + 1 == D ? 0 : slot + 1;
  }
  copy_wait<0>();
  __syncthreads();  // every warp has read its pieces: the partial sums go over them
  float4 (*s_part)[RT * NT][32] = reinterpret_cast<float4 (*)[RT * NT][32]>(s_ring);
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
      s_part[warp][r * NT + t][lane] =
          make_float4(acc[r][t][0], acc[r][t][1], acc[r][t][2], acc[r][t][3]);
  __syncthreads();
  for (int i = warp; i < RT * NT; i += kRowsWarps) {
    float4 v = s_part[0][i][lane];
#pragma unroll
    for (int w = 1; w < kRowsWarps; ++w) {
      const float4 o = s_part[w][i][lane];
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
    const int r = i / NT, tok = (i % NT) * 8 + 2 * c;
    const int n = n0 + r * (GLU ? 8 : 16) + g;
    if ((GLU ? n : n + 8) >= a.N) continue;
    const size_t N = a.N;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (tok + j >= a.T) break;
      const float lo = j ? v.y : v.x, hi = j ? v.w : v.z;
      const size_t row = static_cast<size_t>(tok + j);
      if constexpr (GLU) {
        if (a.Z) {
          a.Z[row * 2 * N + n] = lo;
          a.Z[row * 2 * N + N + n] = hi;
        }
        // h is the next product's operand: 16 bits (see dense_pair.cuh)
        with_act(a.act, [&](auto act) {
          put_half<DT>(a.out, row * N + n, act_fwd<decltype(act)::value>(lo) * hi);
        });
      } else {
        const float x = a.add ? get_half<DT>(a.add, row * N + n) : 0.f;
        const float y = a.add ? get_half<DT>(a.add, row * N + n + 8) : 0.f;
        put_half<DT>(a.out, row * N + n, lo + x);
        put_half<DT>(a.out, row * N + n + 8, hi + y);
      }
    }
  }
}

}  // namespace moe
