// What the row kernels (residual norm, dropout) share: chunks of 16 bytes of
// a row in any of the three element types, a counter-based generator, and
// block-wide sums in a fixed order.
#pragma once

#include <cuda_fp16.h>

#include "ptx.cuh"

namespace moe {

enum RowType { kRowBf16 = 0, kRowFp16 = 1, kRowFp32 = 2 };

// A chunk: 16 bytes of a row, CH elements (8 of 16 bits, 4 of 32).
template <int DT>
struct Chunk {
  static constexpr int CH = DT == kRowFp32 ? 4 : 8;
  static constexpr int SIZE = DT == kRowFp32 ? 4 : 2;

  static __device__ __forceinline__ void unpack(const uint4& q, float* v) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == kRowFp32) {
        v[i] = __uint_as_float(w[i]);
      } else if constexpr (DT == kRowBf16) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }

  static __device__ __forceinline__ uint4 pack(const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == kRowFp32) {
        w[i] = __float_as_uint(v[i]);
      } else if constexpr (DT == kRowBf16) {
        w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
      } else {
        const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }

  // Columns [c, c + CH) of the row at p; with !ALIGNED element by element,
  // zeros at or past H.
  template <bool ALIGNED>
  static __device__ __forceinline__ uint4 load(const void* row, int c, int H) {
    if constexpr (ALIGNED) {
      return *reinterpret_cast<const uint4*>(static_cast<const char*>(row) + c * SIZE);
    } else if constexpr (DT == kRowFp32) {
      uint32_t w[4];
      const uint32_t* p = static_cast<const uint32_t*>(row) + c;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = c + i < H ? p[i] : 0u;
      return make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      uint32_t w[4];
      const uint16_t* p = static_cast<const uint16_t*>(row) + c;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = c + 2 * i < H ? p[2 * i] : 0u;
        const uint32_t hi = c + 2 * i + 1 < H ? p[2 * i + 1] : 0u;
        w[i] = lo | (hi << 16);
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
  }

  template <bool ALIGNED>
  static __device__ __forceinline__ void store(void* row, int c, int H, const uint4& q) {
    if constexpr (ALIGNED) {
      *reinterpret_cast<uint4*>(static_cast<char*>(row) + c * SIZE) = q;
    } else {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      if constexpr (DT == kRowFp32) {
        uint32_t* p = static_cast<uint32_t*>(row) + c;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < H) p[i] = w[i];
      } else {
        uint16_t* p = static_cast<uint16_t*>(row) + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (c + 2 * i < H) p[2 * i] = static_cast<uint16_t>(w[i] & 0xFFFFu);
          if (c + 2 * i + 1 < H) p[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
        }
      }
    }
  }
};

// Start of row t of a [T, H] tensor (64-bit offsets).
template <int DT>
__device__ __forceinline__ const char* row_at(const void* p, int t, int H) {
  return static_cast<const char*>(p) + static_cast<size_t>(t) * H * Chunk<DT>::SIZE;
}
template <int DT>
__device__ __forceinline__ char* row_at(void* p, int t, int H) {
  return static_cast<char*>(p) + static_cast<size_t>(t) * H * Chunk<DT>::SIZE;
}

// ---------------------------------------------------------------- dropout
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as
// easy as 1, 2, 3", SC11): four 32-bit words for each (counter, key).  The
// bits of element (t, c) are word c % 4 at counter (c / 4, t, offset) and key
// seed, so they depend neither on the launch nor on alignment, and forward
// and backward draw the same ones: the mask is never stored.
__device__ __forceinline__ uint4 philox4x32(uint4 c, uint2 k) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(c.x) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c.z) * 0xCD9E8D57u;
    c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k.x, static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a >> 32) ^ c.w ^ k.y, static_cast<uint32_t>(a));
    k.x += 0x9E3779B9u;
    k.y += 0xBB67AE85u;
  }
  return c;
}

struct DropArgs {
  const int64_t* rng;  // device [2]: seed, offset; null: no dropout
  uint32_t threshold;  // kept: word >= threshold
  int all;             // p == 1: nothing is kept
  float scale;         // 1 / (1 - p)
};

struct DropKey {
  uint2 key;
  uint32_t off_lo, off_hi;
};

__device__ __forceinline__ DropKey drop_key(const DropArgs& d) {
  const uint64_t seed = static_cast<uint64_t>(d.rng[0]), off = static_cast<uint64_t>(d.rng[1]);
  return DropKey{make_uint2(static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32)),
                 static_cast<uint32_t>(off), static_cast<uint32_t>(off >> 32)};
}

// Bit i of the result: column c + i of row t is kept (c a multiple of CH).
template <int CH>
__device__ __forceinline__ uint32_t drop_bits(const DropArgs& d, const DropKey& k, int t, int c) {
  uint32_t m = 0;
#pragma unroll
  for (int q = 0; q < CH / 4; ++q) {
    const uint4 w = philox4x32(make_uint4(static_cast<uint32_t>(c / 4 + q),
                                          static_cast<uint32_t>(t), k.off_lo, k.off_hi),
                               k.key);
    m |= (w.x >= d.threshold ? 1u : 0u) << (4 * q);
    m |= (w.y >= d.threshold ? 2u : 0u) << (4 * q);
    m |= (w.z >= d.threshold ? 4u : 0u) << (4 * q);
    m |= (w.w >= d.threshold ? 8u : 0u) << (4 * q);
  }
  return d.all ? 0u : m;
}

// ------------------------------------------------------------- block sums
// Sum of v over the block, the same value in every thread, added in a fixed
// order.  Two buffers of 32 per sum in flight, taken in turn, so that one
// barrier per sum is enough: a buffer is written again only after the next
// sum's barrier, which every reader of the first has passed.
struct BlockSum {
  float2 (*buf)[32];
  int turn;
  __device__ __forceinline__ float2 operator()(float2 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    float2* b = buf[turn];
    turn ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) b[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < nw ? b[lane] : make_float2(0.f, 0.f);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return v;
  }
  __device__ __forceinline__ float operator()(float v) {
    return (*this)(make_float2(v, 0.f)).x;
  }
};

}  // namespace moe
