// Gated feed-forward block for a few tokens (decoding): both products stream
// the weights once, so their bytes are the floor (3 H I elements).
//
// The weights are the M operand of mma.sync m16n8k16 and the tokens its
// N = 8 columns: a 16-row tile of A is 8 gate rows and the 8 up rows of the
// same outputs (gate_up) or 16 rows of W2 (down), so that a lane's four
// accumulators hold gate and up of the same (output, token) pairs and act(g) u
// needs no exchange.  Operands go from global memory straight to registers,
// 16 bytes per lane: the sum over K may run in any order as long as A and B
// agree on it, so lane c of a row's four takes elements 8c .. 8c + 7 of each
// 32 of K as its part of two MMAs.  A warp takes every 8th 64 of K (the block's
// 8 warps read 1 KB of a row side by side); the warps' partial sums meet in
// shared memory and are added in warp order.
//
// Legacy MMA is enough here: at 8 columns a tile's 4 KFLOP come with 512
// bytes of weights, far below any tensor rate.
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

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// 16 bytes of weights, read once: not kept in L1.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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

// GLU: gate_up (8 RT outputs per block), else down (16 RT outputs); NT
// 8-token columns.
template <int DT, bool GLU, int NT, int RT>
__global__ void __launch_bounds__(32 * kRowsWarps) ffn_rows_kernel(const RowsArgs a) {
  constexpr int U = RT == 1 ? 4 : 2;  // 64-of-K steps in flight per warp
  __shared__ float4 s_part[kRowsWarps][RT * NT][32];
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
    w_lo[r] = W + lo * K + 8 * c;
    w_hi[r] = W + hi * K + 8 * c;
  }
  float acc[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][t][i] = 0.f;

  const int steps = (K + 63) / 64;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if constexpr (GLU) pdl_launch();  // the down product may start reading W2
  bool first = true;
  for (int s0 = warp; s0 < steps; s0 += kRowsWarps * U) {
    uint4 lo[U][RT][2], hi[U][RT][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int k = (s0 + u * kRowsWarps) * 64 + 32 * q;
        const bool in = k + 8 * c < K;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          lo[u][r][q] = in && live[r] ? ld_stream(w_lo[r] + k) : zero;
          hi[u][r][q] = in && live[r] ? ld_stream(w_hi[r] + k) : zero;
        }
      }
    if (first) {
      // down: h comes from the kernel before, W2 does not
      if constexpr (!GLU) pdl_wait();
      first = false;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int k = (s0 + u * kRowsWarps) * 64 + 32 * q + 8 * c;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int tok = t * 8 + g;
          uint4 b = zero;
          if (tok < a.T && k < K)
            b = *reinterpret_cast<const uint4*>(X + static_cast<size_t>(tok) * K + k);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const uint4 l = lo[u][r][q], h = hi[u][r][q];
            mma16816<DT>(acc[r][t], l.x, h.x, l.y, h.y, b.x, b.y);
            mma16816<DT>(acc[r][t], l.z, h.z, l.w, h.w, b.z, b.w);
          }
        }
      }
  }
  if constexpr (!GLU) {
    if (first) pdl_wait();  // a warp without steps
  }
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
        put_half<DT>(a.out, row * N + n, act_fwd(a.act, lo) * hi);
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
