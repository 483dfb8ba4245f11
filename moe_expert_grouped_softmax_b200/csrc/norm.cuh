// Residual norm: the norms before and after a block, fused with the block's
// dropout, gate, residual scale and residual add.
//   x^ = x rstd(x),  rstd(x) = 1 / sqrt(mean(x^2) + eps)
//   b  = y^ (o + w_post)            (b = y without w_post)
//   b  = keep b / (1 - p)           (with dropout)
//   r  = res + s gate b
//   n  = r^ (o + w_pre)
// and backward, from dr (of r) and dn (of n):
//   a    = dn (o + w_pre)
//   dres = dr + rstd_r (a - r^ mean(a r^))             (total gradient of r)
//   dgate = s dres b,   db = s gate dres keep / (1 - p)
//   e    = db (o + w_post)
//   dy   = rstd_y (e - y^ mean(e y^))
//   dw_pre = sum_t dn r^,  dw_post = sum_t db y^       (over tokens)
//
// A block works on one row at a time, held in registers between its sums:
// every tensor is read once and written once, so HBM is the bound.
#pragma once

#include "rows.cuh"

namespace moe {

enum GateKind { kGateNone = 0, kGateToken = 1, kGateChannel = 2, kGateElement = 3 };

struct NormArgs {
  const void *y, *res, *w_post, *gate, *w_pre;
  void *r, *n;
  float* stats;  // [2, T]: rstd of y, rstd of r
  int T, H, gate_kind;
  float eps, scale, w_offset;
  DropArgs drop;
};

struct NormBwdArgs {
  const void *dr, *dn, *y, *r, *w_post, *gate, *w_pre;
  const float* stats;
  void *dres, *dy, *dgate;
  float* part;  // [blocks][3][H]: sums over each block's rows (dw_post, dw_pre, dgate)
  int T, H, gate_kind;
  float scale, w_offset;
  DropArgs drop;
};

template <int DT>
__device__ __forceinline__ float elem_at(const void* p, int i) {
  if constexpr (DT == kRowFp32) return static_cast<const float*>(p)[i];
  else if constexpr (DT == kRowBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else return __half2float(static_cast<const __half*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void put_elem(void* p, int i, float v) {
  if constexpr (DT == kRowFp32) static_cast<float*>(p)[i] = v;
  else if constexpr (DT == kRowBf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// Thread i of a block holds chunks i, i + blockDim, ... (VPT of them).
template <int DT, bool ALIGNED, int VPT>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512) norm_fwd_kernel(const NormArgs a) {
  using C = Chunk<DT>;
  constexpr int CH = C::CH;
  __shared__ float2 s_sum[2][32];
  BlockSum block_sum{s_sum, 0};
  griddep_sync();
  const int H = a.H;
  const float inv_h = 1.f / static_cast<float>(H);
  DropKey key{};
  if (a.drop.rng) key = drop_key(a.drop);
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    float v[VPT][CH];
    uint4 res[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = (threadIdx.x + j * blockDim.x) * CH;
      uint4 q = make_uint4(0, 0, 0, 0);
      res[j] = q;
      if (c < H) {
        q = C::template load<ALIGNED>(row_at<DT>(a.y, t, H), c, H);
        if (a.res) res[j] = C::template load<ALIGNED>(row_at<DT>(a.res, t, H), c, H);
      }
      C::unpack(q, v[j]);
    }
    if (a.w_post) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < CH; ++i) ss = fmaf(v[j][i], v[j][i], ss);
      const float rs = rsqrtf(fmaf(block_sum(ss), inv_h, a.eps));
      if (threadIdx.x == 0) a.stats[t] = rs;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = (threadIdx.x + j * blockDim.x) * CH;
        if (c >= H) continue;
        float w[CH];
        C::unpack(C::template load<ALIGNED>(a.w_post, c, H), w);
#pragma unroll
        for (int i = 0; i < CH; ++i) v[j][i] = v[j][i] * rs * (a.w_offset + w[i]);
      }
    }
    const float s = a.gate_kind == kGateToken ? a.scale * elem_at<DT>(a.gate, t) : a.scale;
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = (threadIdx.x + j * blockDim.x) * CH;
      if (c >= H) continue;
      if (a.drop.rng) {
        const uint32_t m = drop_bits<CH>(a.drop, key, t, c);
#pragma unroll
        for (int i = 0; i < CH; ++i) v[j][i] = (m >> i) & 1u ? v[j][i] * a.drop.scale : 0.f;
      }
      float f[CH];
      if (a.gate_kind >= kGateChannel) {
        C::unpack(C::template load<ALIGNED>(
                      a.gate_kind == kGateChannel ? a.gate : row_at<DT>(a.gate, t, H), c, H), f);
#pragma unroll
        for (int i = 0; i < CH; ++i) v[j][i] *= f[i];
      }
      C::unpack(res[j], f);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        v[j][i] = fmaf(s, v[j][i], f[i]);
        if (ALIGNED || c + i < H) ss = fmaf(v[j][i], v[j][i], ss);
      }
      if (a.r) C::template store<ALIGNED>(row_at<DT>(a.r, t, H), c, H, C::pack(v[j]));
    }
    if (a.w_pre) {
      const float rs = rsqrtf(fmaf(block_sum(ss), inv_h, a.eps));
      if (threadIdx.x == 0) a.stats[a.T + t] = rs;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = (threadIdx.x + j * blockDim.x) * CH;
        if (c >= H) continue;
        float w[CH];
        C::unpack(C::template load<ALIGNED>(a.w_pre, c, H), w);
#pragma unroll
        for (int i = 0; i < CH; ++i) v[j][i] = v[j][i] * rs * (a.w_offset + w[i]);
        C::template store<ALIGNED>(row_at<DT>(a.n, t, H), c, H, C::pack(v[j]));
      }
    }
  }
}

// Backward of one row after another; the sums over tokens stay in the
// thread's registers (it keeps the same columns for every row) and leave as
// one partial row per block, added up by norm_sums_kernel in block order.
template <int DT, bool ALIGNED, int VPT>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormBwdArgs a) {
  using C = Chunk<DT>;
  constexpr int CH = C::CH;
  __shared__ float2 s_sum[2][32];
  BlockSum block_sum{s_sum, 0};
  griddep_sync();
  const int H = a.H;
  const float inv_h = 1.f / static_cast<float>(H);
  DropKey key{};
  if (a.drop.rng) key = drop_key(a.drop);
  float acc_post[VPT][CH], acc_pre[VPT][CH], acc_gate[VPT][CH];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < CH; ++i) acc_post[j][i] = acc_pre[j][i] = acc_gate[j][i] = 0.f;

  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    float d[VPT][CH];  // the gradient of r, then of y
    if (a.w_pre) {
      const float rs = a.stats[a.T + t];
      float rh[VPT][CH];
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int c = (threadIdx.x + j * blockDim.x) * CH;
        uint4 qr = make_uint4(0, 0, 0, 0), qn = qr, qw = qr;
        if (c < H) {
          qr = C::template load<ALIGNED>(row_at<DT>(a.r, t, H), c, H);
          qn = C::template load<ALIGNED>(row_at<DT>(a.dn, t, H), c, H);
          qw = C::template load<ALIGNED>(a.w_pre, c, H);
        }
        float w[CH];
        C::unpack(qr, rh[j]);
        C::unpack(qn, d[j]);
        C::unpack(qw, w);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          rh[j][i] *= rs;
          acc_pre[j][i] = fmaf(d[j][i], rh[j][i], acc_pre[j][i]);
          d[j][i] *= a.w_offset + w[i];
          sum = fmaf(d[j][i], rh[j][i], sum);
        }
      }
      const float mean = block_sum(sum) * inv_h;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < CH; ++i) d[j][i] = rs * (d[j][i] - rh[j][i] * mean);
    } else {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < CH; ++i) d[j][i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = (threadIdx.x + j * blockDim.x) * CH;
      if (c >= H) continue;
      if (a.dr) {
        float f[CH];
        C::unpack(C::template load<ALIGNED>(row_at<DT>(a.dr, t, H), c, H), f);
#pragma unroll
        for (int i = 0; i < CH; ++i) d[j][i] += f[i];
      }
      if (a.dres) C::template store<ALIGNED>(row_at<DT>(a.dres, t, H), c, H, C::pack(d[j]));
    }
    if (!a.dy) continue;
    const float rs = a.w_post ? a.stats[t] : 1.f;
    const float g_t = a.gate_kind == kGateToken ? elem_at<DT>(a.gate, t) : 1.f;
    float yh[VPT][CH];
    float2 sum = make_float2(0.f, 0.f);  // e y^ over the row; dgate of the token
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = (threadIdx.x + j * blockDim.x) * CH;
      uint4 q = make_uint4(0, 0, 0, 0);
      if (c < H) q = C::template load<ALIGNED>(row_at<DT>(a.y, t, H), c, H);
      C::unpack(q, yh[j]);
      if (c >= H) continue;
      float w[CH], g[CH];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        w[i] = 1.f;
        g[i] = g_t;
      }
      if (a.w_post) {
        C::unpack(C::template load<ALIGNED>(a.w_post, c, H), w);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          w[i] += a.w_offset;
          yh[j][i] *= rs;
        }
      }
      if (a.gate_kind >= kGateChannel)
        C::unpack(C::template load<ALIGNED>(
                      a.gate_kind == kGateChannel ? a.gate : row_at<DT>(a.gate, t, H), c, H), g);
      const uint32_t m = a.drop.rng ? drop_bits<CH>(a.drop, key, t, c) : 0xFFFFFFFFu;
      const float ks = a.drop.rng ? a.scale * a.drop.scale : a.scale;
      float dg[CH];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const float e = (m >> i) & 1u ? ks * d[j][i] : 0.f;  // s dres keep / (1 - p)
        // a dropped y contributes nothing, whatever it holds
        dg[i] = (m >> i) & 1u ? e * yh[j][i] * w[i] : 0.f;
        const float db = e * g[i];
        if (a.w_post) {
          acc_post[j][i] = fmaf(db, yh[j][i], acc_post[j][i]);
          d[j][i] = db * w[i];
          sum.x = fmaf(d[j][i], yh[j][i], sum.x);
        } else {
          d[j][i] = db;
        }
        acc_gate[j][i] += dg[i];
        sum.y += dg[i];
      }
      if (a.gate_kind == kGateElement)
        C::template store<ALIGNED>(row_at<DT>(a.dgate, t, H), c, H, C::pack(dg));
    }
    if (a.w_post || a.gate_kind == kGateToken) {
      sum = block_sum(sum);
      if (a.gate_kind == kGateToken && threadIdx.x == 0) put_elem<DT>(a.dgate, t, sum.y);
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int c = (threadIdx.x + j * blockDim.x) * CH;
      if (c >= H) continue;
      if (a.w_post) {
        const float mean = sum.x * inv_h;
#pragma unroll
        for (int i = 0; i < CH; ++i) d[j][i] = rs * (d[j][i] - yh[j][i] * mean);
      }
      C::template store<ALIGNED>(row_at<DT>(a.dy, t, H), c, H, C::pack(d[j]));
    }
  }

  float* part = a.part + static_cast<size_t>(blockIdx.x) * 3 * H;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = (threadIdx.x + j * blockDim.x) * CH;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (c + i >= H) continue;
      if (a.w_post) part[c + i] = acc_post[j][i];
      if (a.w_pre) part[H + c + i] = acc_pre[j][i];
      if (a.gate_kind == kGateChannel) part[2 * H + c + i] = acc_gate[j][i];
    }
  }
}

// dw_post, dw_pre and the channel gate's gradient: column sums of the blocks'
// partial rows, in block order, rounded once to the parameter's type.
template <int DT>
__global__ void __launch_bounds__(256) norm_sums_kernel(const float* part, int blocks, int H,
                                                        void* dw_post, void* dw_pre,
                                                        void* dgate) {
  griddep_sync();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  void* out = blockIdx.y == 0 ? dw_post : blockIdx.y == 1 ? dw_pre : dgate;
  if (out == nullptr) return;
  __shared__ float s[8][32];
  float v = 0.f;
  if (c < H)
    for (int b = w; b < blocks; b += 8)
      v += part[(static_cast<size_t>(b) * 3 + blockIdx.y) * H + c];
  s[w][threadIdx.x & 31] = v;
  __syncthreads();
  if (w != 0 || c >= H) return;
  for (int i = 1; i < 8; ++i) v += s[i][threadIdx.x];
  put_elem<DT>(out, c, v);
}

}  // namespace moe
