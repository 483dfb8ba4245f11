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

  // The elements at columns c, c + step, ... of a row.  ALIGNED: step 1, one
  // 16-byte access; otherwise step 32 (a warp's accesses are contiguous), each
  // element for itself, zeros at or past H; only a row's last 32 CH columns
  // are tested one by one.
  static __device__ __forceinline__ bool inside(int c, int H) {
    return c - static_cast<int>(threadIdx.x & 31) + 32 * CH <= H;  // the warp's columns
  }
  template <bool ALIGNED>
  static __device__ __forceinline__ uint4 load(const void* row, int c, int H) {
    if constexpr (ALIGNED) {
      return *reinterpret_cast<const uint4*>(static_cast<const char*>(row) +
                                             static_cast<size_t>(c) * SIZE);
    } else if constexpr (DT == kRowFp32) {
      uint32_t w[4];
      const uint32_t* p = static_cast<const uint32_t*>(row) + c;
      if (inside(c, H)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = p[32 * i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = c + 32 * i < H ? p[32 * i] : 0u;
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      uint32_t w[4];
      const uint16_t* p = static_cast<const uint16_t*>(row) + c;
      if (inside(c, H)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = p[64 * i] | (static_cast<uint32_t>(p[64 * i + 32]) << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = c + 64 * i < H ? p[64 * i] : 0u;
        const uint32_t hi = c + 64 * i + 32 < H ? p[64 * i + 32] : 0u;
        w[i] = lo | (hi << 16);
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
  }

  template <bool ALIGNED>
  static __device__ __forceinline__ void store(void* row, int c, int H, const uint4& q) {
    if constexpr (ALIGNED) {
      *reinterpret_cast<uint4*>(static_cast<char*>(row) + static_cast<size_t>(c) * SIZE) = q;
    } else {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      if constexpr (DT == kRowFp32) {
        uint32_t* p = static_cast<uint32_t*>(row) + c;
        if (inside(c, H)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) p[32 * i] = w[i];
          return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + 32 * i < H) p[32 * i] = w[i];
      } else {
        uint16_t* p = static_cast<uint16_t*>(row) + c;
        if (inside(c, H)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[64 * i] = static_cast<uint16_t>(w[i] & 0xFFFFu);
            p[64 * i + 32] = static_cast<uint16_t>(w[i] >> 16);
          }
          return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (c + 64 * i < H) p[64 * i] = static_cast<uint16_t>(w[i] & 0xFFFFu);
          if (c + 64 * i + 32 < H) p[64 * i + 32] = static_cast<uint16_t>(w[i] >> 16);
        }
      }
    }
  }

  // First column of chunk n of a row's chunks in thread order (a warp's 32
  // chunks cover the same 32 CH columns either way), and the step to the next.
  template <bool ALIGNED>
  static __device__ __forceinline__ int first(int n) {
    return ALIGNED ? n * CH : (n & ~31) * CH + (n & 31);
  }
  template <bool ALIGNED>
  static constexpr int kStep = ALIGNED ? 1 : 32;
  // whether chunk n holds columns of the row (warp-uniform unless ALIGNED)
  template <bool ALIGNED>
  static __device__ __forceinline__ bool live(int n, int H) {
    return ALIGNED ? n * CH < H : (n & ~31) * CH < H;
  }
};

// 32 bytes at a 32-byte aligned address.
__device__ __forceinline__ void load32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                 "=r"(b.w)
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store32(void* p, uint4 a, uint4 b) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y),
               "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Two fp32 operations in one instruction (each rounded as by itself).
__device__ __forceinline__ void fma2(float* d, const float* a, const float* b, const float* c) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
      "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]), "f"(c[0]), "f"(c[1]));
}
__device__ __forceinline__ void mul2(float* d, const float* a, const float* b) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
__device__ __forceinline__ void add2(float* d, const float* a, const float* b) {
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d[0]), "=f"(d[1])
      : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
// The same for a chunk of N elements; a scalar operand stands for all.
template <int N>
__device__ __forceinline__ void mul_n(float* d, const float* a, const float* b) {
#pragma unroll
  for (int i = 0; i < N; i += 2) mul2(d + i, a + i, b + i);
}
template <int N>
__device__ __forceinline__ void mul_n(float* d, const float* a, float b) {
  const float b2[2] = {b, b};
#pragma unroll
  for (int i = 0; i < N; i += 2) mul2(d + i, a + i, b2);
}
template <int N>
__device__ __forceinline__ void add_n(float* d, const float* a, const float* b) {
#pragma unroll
  for (int i = 0; i < N; i += 2) add2(d + i, a + i, b + i);
}
template <int N>
__device__ __forceinline__ void add_n(float* d, const float* a, float b) {
  const float b2[2] = {b, b};
#pragma unroll
  for (int i = 0; i < N; i += 2) add2(d + i, a + i, b2);
}
// d = a b + c
template <int N>
__device__ __forceinline__ void fma_n(float* d, const float* a, const float* b, const float* c) {
#pragma unroll
  for (int i = 0; i < N; i += 2) fma2(d + i, a + i, b + i, c + i);
}
template <int N>
__device__ __forceinline__ void fma_n(float* d, const float* a, float b, const float* c) {
  const float b2[2] = {b, b};
#pragma unroll
  for (int i = 0; i < N; i += 2) fma2(d + i, a + i, b2, c + i);
}
// s[0], s[1] += sums of a b over even and odd elements
template <int N>
__device__ __forceinline__ void dot_n(float* s, const float* a, const float* b) {
#pragma unroll
  for (int i = 0; i < N; i += 2) fma2(s, a + i, b + i, s);
}

// One contiguous copy global -> shared of `bytes` (addresses and size
// multiples of 16), counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

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
// Q counters run side by side under one key, so that each round's key words
// are formed once for all of them.
template <int Q>
__device__ __forceinline__ void philox4x32(uint4 (&c)[Q], uint2 k) {
#pragma unroll
  for (int r = 0; r < 10; ++r) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const uint64_t a = static_cast<uint64_t>(c[q].x) * 0xD2511F53u;
      const uint64_t b = static_cast<uint64_t>(c[q].z) * 0xCD9E8D57u;
      c[q] = make_uint4(static_cast<uint32_t>(b >> 32) ^ c[q].y ^ k.x, static_cast<uint32_t>(b),
                        static_cast<uint32_t>(a >> 32) ^ c[q].w ^ k.y, static_cast<uint32_t>(a));
    }
    k.x += 0x9E3779B9u;
    k.y += 0xBB67AE85u;
  }
}

struct DropArgs {
  const int64_t* rng;  // device [2]: seed, offset; null: no dropout
  uint32_t threshold;  // kept: word >= threshold
  int all;             // round(p 2^32) is 2^32: nothing is kept
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

// The random words of chunks n[0], ..., n[U - 1] of one row.  A lane draws the
// 4-column groups of its own 16 bytes; where elements lie 32 columns apart it
// fetches the words of its columns from the lanes that drew them (whole warps,
// all lanes here).
template <int CH, int U, bool ALIGNED>
struct DropWords {
  static constexpr int G = CH / 4;
  uint32_t w[U][CH];
  __device__ __forceinline__ void draw(const DropKey& k, int row, const int (&n)[U]) {
    uint4 c[U * G];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int q = 0; q < G; ++q)
        c[u * G + q] =
            make_uint4(static_cast<uint32_t>(ALIGNED ? n[u] * G + q
                                                     : (n[u] & ~31) * G + (n[u] & 31) + 32 * q),
                       static_cast<uint32_t>(row), k.off_lo, k.off_hi);
    philox4x32(c, k.key);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const uint4 v = c[u * G + i / 4];
        if constexpr (ALIGNED) {
          w[u][i] = i % 4 == 0 ? v.x : i % 4 == 1 ? v.y : i % 4 == 2 ? v.z : v.w;
        } else {
          // column base + lane + 32 i: word lane % 4 of group lane / 4 + 8 i
          const int lane = threadIdx.x & 31, src = (lane >> 2) + 8 * (i & 3);
          const uint32_t x = __shfl_sync(0xffffffffu, v.x, src);
          const uint32_t y = __shfl_sync(0xffffffffu, v.y, src);
          const uint32_t z = __shfl_sync(0xffffffffu, v.z, src);
          const uint32_t t = __shfl_sync(0xffffffffu, v.w, src);
          w[u][i] = lane & 2 ? (lane & 1 ? t : z) : (lane & 1 ? y : x);
        }
      }
  }
  __device__ __forceinline__ bool keep(const DropArgs& d, int u, int i) const {
    return w[u][i] >= d.threshold && !d.all;
  }
};

// ------------------------------------------------------------- block sums
// Sum of v over the block, the same value in every thread, added in a fixed
// order.  Two buffers of 32 per sum in flight, taken in turn, so that one
// barrier per sum is enough: a buffer is written again only after the next
// sum's barrier, which every reader of the first has passed.
struct BlockSum {
  float2 (*buf)[32];
  int turn;

  static __device__ __forceinline__ float warp(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
  __device__ __forceinline__ float operator()(float v) {
    v = warp(v);
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (nw == 1) return v;
    float2* b = buf[turn];
    turn ^= 1;
    if (lane == 0) b[threadIdx.x >> 5].x = v;
    __syncthreads();
    return warp(lane < nw ? b[lane].x : 0.f);
  }
  __device__ __forceinline__ float2 operator()(float2 v) {
    v = make_float2(warp(v.x), warp(v.y));
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (nw == 1) return v;
    float2* b = buf[turn];
    turn ^= 1;
    if (lane == 0) b[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < nw ? b[lane] : make_float2(0.f, 0.f);
    return make_float2(warp(v.x), warp(v.y));
  }
};

}  // namespace moe
