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
// every tensor is read once and written once, so HBM is the floor.  What keeps
// the kernels from it is that a row's two block-wide sums follow one another:
// with one to four blocks an SM little else runs across their barriers, and
// with all parts on (55 instructions an element forward, 88 backward, 11 of
// them the generator's) 65% and 59% of the issue slots are busy at 3.5 and 2.9
// TB/s, so that neither is full.  bf16, us forward / backward:
//                        add + norm     post norm, channel gate, dropout too
//   8192 x  2880           38 /  57         69 / 113
//   8192 x  4096           50 /  87         84 / 166
//   8192 x  5120           64 /  95         98 / 191
//   8192 x  7168           87 / 111        134 / 247
//   8192 x  8192          101 / 123        148 / 286
//   4096 x 16384          138 / 178        212 / 498
//   4096 x 16383          230 / 396  (element by element)
// fp32, add + norm: 8192 x 7168 163 / 153, 4096 x 16384 178 / 425.  The
// backward of rows over 8192 holds 32 elements a thread and spills (980 to
// 1372 bytes a thread are stored), which is most of its distance from the
// floor.  One row: 3.3 us.
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
  int stages;      // rows in flight (RING)
  int stall_test;
  uint64_t wait_ns;
};

struct NormBwdArgs {
  const void *dr, *dn, *y, *r, *w_post, *gate, *w_pre;
  const float* stats;
  void *dres, *dy, *dgate;
  float* part;  // [blocks][3][H]: sums over each block's rows (dw_post, dw_pre, dgate)
  int T, H, gate_kind;
  float scale, w_offset;
  DropArgs drop;
  int stages;      // rows in flight (RING)
  int stall_test;
  uint64_t wait_ns;
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

// v = keep ? v * scale : 0 for a thread's chunks of row t (two at a time under
// one set of round keys); where `also` is given, also = keep ? also : 0 (a
// dropped y counts as zero, whatever it holds).
template <int DT, int VPT, bool ALIGNED>
__device__ __forceinline__ void drop_row(const DropArgs& d, const DropKey& key, int t,
                                         float scale, float (&v)[VPT][Chunk<DT>::CH],
                                         float (*also)[Chunk<DT>::CH] = nullptr) {
  constexpr int CH = Chunk<DT>::CH, U = VPT < 2 ? 1 : 2;
#pragma unroll
  for (int j = 0; j < VPT; j += U) {
    int n[U];
#pragma unroll
    for (int u = 0; u < U; ++u) n[u] = threadIdx.x + (j + u) * blockDim.x;
    DropWords<CH, U, ALIGNED> words;
    words.draw(key, t, n);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const bool keep = words.keep(d, u, i);
        v[j + u][i] = keep ? v[j + u][i] : 0.f;
        if (also) also[j + u][i] = keep ? also[j + u][i] : 0.f;
      }
#pragma unroll
    for (int u = 0; u < U; ++u) mul_n<CH>(v[j + u], v[j + u], scale);
  }
}

// Rows of up to five tensors, `stages` rows deep, brought to shared memory by
// bulk copies that thread 0 issues ahead of their use.  The block's row i goes
// to stage i % stages, as that stage's use number i / stages.  Thread 0 arms a
// stage again only after its own wait for the row before has succeeded (the
// barrier takes one arrival a phase): once one has run out it issues nothing
// more.  Bit 0 of `phase` is the parity of the stage's use; the bits above it
// are 0, or 1 + the row whose wait ran out first.
struct RowRing {
  static constexpr int kMaxStages = 4;
  uint8_t* base;
  uint64_t* full;
  volatile int* abort;
  uint64_t wait_ns;
  uint32_t row_bytes;
  int stages;
  const void** src;  // shared, thread 0's own
  int n = 0, stage = 0;
  uint32_t phase = 0;

  __device__ __forceinline__ int add(const void* p) {
    if (p == nullptr) return 0;
    if (threadIdx.x == 0) src[n] = p;
    return n++;
  }
  // (stall test: the barriers wait for one more arrival, which only finish()
  // makes)
  __device__ __forceinline__ void init(int stall_test) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1 + stall_test);
      *abort = 0;
      fence_mbar_init();
    }
    __syncthreads();
  }
  __device__ __forceinline__ const uint8_t* at(int slot) const {
    return base + static_cast<size_t>(stage * n + slot) * row_bytes;
  }
  __device__ __forceinline__ void issue(int st, int t) {
    uint64_t* bar = &full[st];
    mbar_arrive_expect_tx(bar, n * row_bytes);
    for (int q = 0; q < n; ++q)
      bulk_load(base + static_cast<size_t>(st * n + q) * row_bytes,
                static_cast<const char*>(src[q]) + static_cast<size_t>(t) * row_bytes, row_bytes,
                bar);
  }
  // The block's first rows t0, t0 + step, ...
  __device__ __forceinline__ void start(int rows, int t0, int step) {
    if (threadIdx.x == 0)
      for (int i = 0; i < min(rows, stages); ++i) issue(i, t0 + i * step);
  }
  // Row k.  On a wait that ran out (recorded) the row is garbage, but every
  // thread still passes the same barriers.
  __device__ __forceinline__ void wait(int k) {
    if (!mbar_wait(&full[stage], phase & 1, abort, wait_ns) && phase < 2) phase |= (k + 1) << 1;
  }
  // Every thread has read the stage: fill it with row t (t < 0: no more) and
  // go on to the next.
  __device__ __forceinline__ void next(int t) {
    if (threadIdx.x == 0 && t >= 0 && phase < 2) issue(stage, t);
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  // After a wait that ran out: let the copies in flight land.
  __device__ __forceinline__ void finish(int rows, int stall_test) {
    if (threadIdx.x == 0 && phase >= 2) {
#pragma unroll 1
      for (int i = 0; stall_test && i < stages; ++i) mbar_arrive(&full[i]);
      const int issued = min(rows, static_cast<int>(phase >> 1) - 1 + stages);
#pragma unroll 1
      for (int i = max(0, issued - stages); i < issued; ++i)
        drain_wait(&full[i % stages], (i / stages) & 1, wait_ns);
    }
    __syncthreads();
  }
};

__device__ __forceinline__ int block_rows(int T) {
  return (T - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) /
         static_cast<int>(gridDim.x);
}

// Thread i of a block holds chunks i, i + blockDim, ... (VPT of them) of one
// row after another.  With RING (16-byte aligned rows, several a block) the
// rows arrive by bulk copies, as many ahead as fit (four at most): with two or
// more stages the loads of later rows run under this row's two block sums,
// with one (the backward in fp32 from four or five tensors, at 1792, 3584 or
// 7168 columns for instance) under its last stores only.  Otherwise each
// thread loads its own.
template <int DT, bool ALIGNED, int VPT, bool RING>
__global__ void __launch_bounds__(VPT == 1 ? 1024 : 512, VPT == 2 ? 2 : 1)
    norm_fwd_kernel(const NormArgs a) {
  using C = Chunk<DT>;
  constexpr int CH = C::CH;
  static_assert(ALIGNED || !RING, "bulk copies take whole 16-byte pieces");
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ float2 s_sum[2][32];
  __shared__ uint64_t s_full[RowRing::kMaxStages];
  __shared__ int s_abort;
  __shared__ const void* s_src[5];
  BlockSum block_sum{s_sum, 0};
  const int H = a.H;
  const float inv_h = 1.f / static_cast<float>(H);
  const int rows = block_rows(a.T);
  RowRing ring{s_ring, s_full, &s_abort, a.wait_ns, static_cast<uint32_t>(H) * C::SIZE, a.stages,
               s_src};
  int q_y = 0, q_res = 0, q_g = 0;
  if constexpr (RING) {
    q_y = ring.add(a.y);
    q_res = ring.add(a.res);
    if (a.gate_kind == kGateElement) q_g = ring.add(a.gate);
    ring.init(a.stall_test);
  }
  griddep_sync();
  DropKey key{};
  if (a.drop.rng) key = drop_key(a.drop);
  if constexpr (RING) ring.start(rows, blockIdx.x, gridDim.x);
  auto load = [&](const void* p, int slot, int t, int c) -> uint4 {
    if constexpr (RING) return *reinterpret_cast<const uint4*>(ring.at(slot) + c * C::SIZE);
    else return C::template load<ALIGNED>(row_at<DT>(p, t, H), c, H);
  };
  int col[VPT];
  bool live[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int n = threadIdx.x + j * blockDim.x;
    col[j] = C::template first<ALIGNED>(n);
    live[j] = C::template live<ALIGNED>(n, H);
  }
  for (int k = 0; k < rows; ++k) {
    const int t = blockIdx.x + k * gridDim.x;
    if constexpr (RING) ring.wait(k);
    float v[VPT][CH];
    uint4 res[VPT], gate[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      uint4 q = make_uint4(0, 0, 0, 0);
      res[j] = gate[j] = q;
      if (live[j]) {
        q = load(a.y, q_y, t, col[j]);
        if (a.res) res[j] = load(a.res, q_res, t, col[j]);
        if (a.gate_kind == kGateElement) gate[j] = load(a.gate, q_g, t, col[j]);
        else if (a.gate_kind == kGateChannel) gate[j] = C::template load<ALIGNED>(a.gate, col[j], H);
      }
      C::unpack(q, v[j]);
    }
    const float s = a.gate_kind == kGateToken ? a.scale * elem_at<DT>(a.gate, t) : a.scale;
    if (a.w_post) {
      float ss[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < VPT; ++j) dot_n<CH>(ss, v[j], v[j]);
      const float rs = rsqrtf(fmaf(block_sum(ss[0] + ss[1]), inv_h, a.eps));
      if (threadIdx.x == 0) a.stats[t] = rs;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (!live[j]) continue;
        float w[CH];
        C::unpack(C::template load<ALIGNED>(a.w_post, col[j], H), w);
        if (a.w_offset != 0.f) add_n<CH>(w, w, a.w_offset);
        mul_n<CH>(v[j], v[j], rs);
        mul_n<CH>(v[j], v[j], w);
      }
    }
    if (a.drop.rng) drop_row<DT, VPT, ALIGNED>(a.drop, key, t, a.drop.scale, v);
    float s2[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (!live[j]) continue;
      float f[CH];
      if (a.gate_kind >= kGateChannel) {
        C::unpack(gate[j], f);
        mul_n<CH>(v[j], v[j], f);
      }
      C::unpack(res[j], f);
      fma_n<CH>(v[j], v[j], s, f);  // zero in columns at or past H
      dot_n<CH>(s2, v[j], v[j]);
      if (a.r) C::template store<ALIGNED>(row_at<DT>(a.r, t, H), col[j], H, C::pack(v[j]));
    }
    const float ss = a.w_pre ? block_sum(s2[0] + s2[1]) : 0.f;
    if constexpr (RING) {
      // every thread has read this row's stage: the block sum's barrier
      if (!a.w_pre || blockDim.x == 32) __syncthreads();
      ring.next(k + a.stages < rows ? t + a.stages * static_cast<int>(gridDim.x) : -1);
    }
    if (a.w_pre) {
      const float rs = rsqrtf(fmaf(ss, inv_h, a.eps));
      if (threadIdx.x == 0) a.stats[a.T + t] = rs;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (!live[j]) continue;
        float w[CH];
        C::unpack(C::template load<ALIGNED>(a.w_pre, col[j], H), w);
        if (a.w_offset != 0.f) add_n<CH>(w, w, a.w_offset);
        mul_n<CH>(v[j], v[j], rs);
        mul_n<CH>(v[j], v[j], w);
        C::template store<ALIGNED>(row_at<DT>(a.n, t, H), col[j], H, C::pack(v[j]));
      }
    }
  }
  if constexpr (RING) ring.finish(rows, a.stall_test);
}

// Backward of one row after another, as the forward's rows; the sums over
// tokens stay in the thread's registers (it keeps the same columns for every
// row) and leave as one partial row per block, added up by norm_sums_kernel.
template <int DT, bool ALIGNED, int VPT, int MAXT, bool RING>
__global__ void __launch_bounds__(MAXT, MAXT == 448 && VPT * Chunk<DT>::CH == 8 ? 2 : 1)
    norm_bwd_kernel(const NormBwdArgs a) {
  using C = Chunk<DT>;
  constexpr int CH = C::CH;
  static_assert(ALIGNED || !RING, "bulk copies take whole 16-byte pieces");
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ float2 s_sum[2][32];
  __shared__ uint64_t s_full[RowRing::kMaxStages];
  __shared__ int s_abort;
  __shared__ const void* s_src[5];
  BlockSum block_sum{s_sum, 0};
  const int H = a.H;
  const float inv_h = 1.f / static_cast<float>(H);
  const int rows = block_rows(a.T);
  RowRing ring{s_ring, s_full, &s_abort, a.wait_ns, static_cast<uint32_t>(H) * C::SIZE, a.stages,
               s_src};
  int q_dn = 0, q_r = 0, q_dr = 0, q_y = 0, q_g = 0;
  if constexpr (RING) {
    if (a.w_pre) {
      q_dn = ring.add(a.dn);
      q_r = ring.add(a.r);
    }
    q_dr = ring.add(a.dr);
    if (a.dy) q_y = ring.add(a.y);
    if (a.dy && a.gate_kind == kGateElement) q_g = ring.add(a.gate);
    ring.init(a.stall_test);
  }
  griddep_sync();
  DropKey key{};
  if (a.drop.rng) key = drop_key(a.drop);
  if constexpr (RING) ring.start(rows, blockIdx.x, gridDim.x);
  auto load = [&](const void* p, int slot, int t, int c) -> uint4 {
    if constexpr (RING) return *reinterpret_cast<const uint4*>(ring.at(slot) + c * C::SIZE);
    else return C::template load<ALIGNED>(row_at<DT>(p, t, H), c, H);
  };
  int col[VPT];
  bool live[VPT];
  float acc_post[VPT][CH], acc_pre[VPT][CH], acc_gate[VPT][CH];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int n = threadIdx.x + j * blockDim.x;
    col[j] = C::template first<ALIGNED>(n);
    live[j] = C::template live<ALIGNED>(n, H);
#pragma unroll
    for (int i = 0; i < CH; ++i) acc_post[j][i] = acc_pre[j][i] = acc_gate[j][i] = 0.f;
  }
  // the row's statistics, read one row ahead
  float st_pre = a.w_pre ? a.stats[a.T + blockIdx.x] : 0.f;
  float st_post = a.w_post ? a.stats[blockIdx.x] : 1.f;

  for (int k = 0; k < rows; ++k) {
    const int t = blockIdx.x + k * gridDim.x;
    const float rs_pre = st_pre, rs_post = st_post;
    if (k + 1 < rows) {
      if (a.w_pre) st_pre = a.stats[a.T + t + gridDim.x];
      if (a.w_post) st_post = a.stats[t + gridDim.x];
    }
    const float g_t = a.gate_kind == kGateToken ? elem_at<DT>(a.gate, t) : 1.f;
    if constexpr (RING) ring.wait(k);
    float d[VPT][CH];  // the gradient of r, then of y
    // without the ring all of a row's loads go out before the first sum
    uint4 pdr[VPT], py[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      pdr[j] = py[j] = make_uint4(0, 0, 0, 0);
      if constexpr (!RING) {
        if (live[j] && a.dr) pdr[j] = load(a.dr, q_dr, t, col[j]);
        if (live[j] && a.dy) py[j] = load(a.y, q_y, t, col[j]);
      }
    }
    if (a.w_pre) {
      float rh[VPT][CH];
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        uint4 qr = make_uint4(0, 0, 0, 0), qn = qr, qw = qr;
        if (live[j]) {
          qr = load(a.r, q_r, t, col[j]);
          qn = load(a.dn, q_dn, t, col[j]);
          qw = C::template load<ALIGNED>(a.w_pre, col[j], H);
        }
        float w[CH];
        C::unpack(qr, rh[j]);
        C::unpack(qn, d[j]);
        C::unpack(qw, w);
        if (a.w_offset != 0.f) add_n<CH>(w, w, a.w_offset);
        mul_n<CH>(rh[j], rh[j], rs_pre);
        fma_n<CH>(acc_pre[j], d[j], rh[j], acc_pre[j]);
        mul_n<CH>(d[j], d[j], w);
        dot_n<CH>(sum, d[j], rh[j]);
      }
      const float mean = block_sum(sum[0] + sum[1]) * inv_h;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        fma_n<CH>(d[j], rh[j], -mean, d[j]);
        mul_n<CH>(d[j], d[j], rs_pre);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < CH; ++i) d[j][i] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (!live[j]) continue;
      if (a.dr) {
        if constexpr (RING) pdr[j] = load(a.dr, q_dr, t, col[j]);
        float f[CH];
        C::unpack(pdr[j], f);
        add_n<CH>(d[j], d[j], f);
      }
      if (a.dres) C::template store<ALIGNED>(row_at<DT>(a.dres, t, H), col[j], H, C::pack(d[j]));
    }
    const bool sum2 = a.dy && (a.w_post || a.gate_kind == kGateToken);
    float yh[VPT][CH];
    float2 sum = make_float2(0.f, 0.f);  // e y^ over the row; dgate of the token
    float e2[2] = {0.f, 0.f};
    if (a.dy) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if constexpr (RING) {
          if (live[j]) py[j] = load(a.y, q_y, t, col[j]);
        }
        C::unpack(py[j], yh[j]);
      }
      // s dres keep / (1 - p)
      if (a.drop.rng) {
        if (a.w_post)
          drop_row<DT, VPT, ALIGNED>(a.drop, key, t, a.scale * a.drop.scale, d);
        else
          drop_row<DT, VPT, ALIGNED>(a.drop, key, t, a.scale * a.drop.scale, d, yh);
      } else {
#pragma unroll
        for (int j = 0; j < VPT; ++j) mul_n<CH>(d[j], d[j], a.scale);
      }
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (!live[j]) continue;
        float w[CH];
        if (a.w_post) {
          C::unpack(C::template load<ALIGNED>(a.w_post, col[j], H), w);
          if (a.w_offset != 0.f) add_n<CH>(w, w, a.w_offset);
          mul_n<CH>(yh[j], yh[j], rs_post);
        } else {
#pragma unroll
          for (int i = 0; i < CH; ++i) w[i] = 1.f;
        }
        if (a.gate_kind != kGateNone) {
          float g[CH], dg[CH];
          if (a.gate_kind == kGateToken) {
#pragma unroll
            for (int i = 0; i < CH; ++i) g[i] = g_t;
          } else if (a.gate_kind == kGateChannel) {
            C::unpack(C::template load<ALIGNED>(a.gate, col[j], H), g);
          } else {
            C::unpack(load(a.gate, q_g, t, col[j]), g);
          }
          mul_n<CH>(dg, d[j], yh[j]);
          mul_n<CH>(dg, dg, w);
          mul_n<CH>(d[j], d[j], g);
          if (a.gate_kind == kGateToken) {
#pragma unroll
            for (int i = 0; i < CH; ++i) sum.y += dg[i];
          } else if (a.gate_kind == kGateChannel) {
            add_n<CH>(acc_gate[j], acc_gate[j], dg);
          } else {
            C::template store<ALIGNED>(row_at<DT>(a.dgate, t, H), col[j], H, C::pack(dg));
          }
        }
        if (a.w_post) {
          fma_n<CH>(acc_post[j], d[j], yh[j], acc_post[j]);
          mul_n<CH>(d[j], d[j], w);
          dot_n<CH>(e2, d[j], yh[j]);
        }
      }
    }
    sum.x = e2[0] + e2[1];
    if (sum2) {
      if (a.gate_kind == kGateToken) sum = block_sum(sum);
      else sum.x = block_sum(sum.x);
    }
    if constexpr (RING) {
      // every thread has read this row's stage: the block sum's barrier
      if (!sum2 || blockDim.x == 32) __syncthreads();
      ring.next(k + a.stages < rows ? t + a.stages * static_cast<int>(gridDim.x) : -1);
    }
    if (!a.dy) continue;
    if (a.gate_kind == kGateToken && threadIdx.x == 0) put_elem<DT>(a.dgate, t, sum.y);
    const float mean = sum.x * inv_h;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (!live[j]) continue;
      if (a.w_post) {
        fma_n<CH>(d[j], yh[j], -mean, d[j]);
        mul_n<CH>(d[j], d[j], rs_post);
      }
      C::template store<ALIGNED>(row_at<DT>(a.dy, t, H), col[j], H, C::pack(d[j]));
    }
  }

  if constexpr (RING) ring.finish(rows, a.stall_test);
  float* part = a.part + static_cast<size_t>(blockIdx.x) * 3 * H;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = col[j] + i * C::template kStep<ALIGNED>;
      if (c >= H) continue;
      if (a.w_post) part[c] = acc_post[j][i];
      if (a.w_pre) part[H + c] = acc_pre[j][i];
      if (a.gate_kind == kGateChannel) part[2 * H + c] = acc_gate[j][i];
    }
  }
}

// dw_post, dw_pre and the channel gate's gradient: column sums of the blocks'
// partial rows, rounded once to the parameter's type.  A block takes 128
// columns of one sum, four per lane; its 32 warps take every 32nd partial row
// and are added in warp order (8 warps: 21 us for 444 rows of 2051).
template <int DT>
__global__ void __launch_bounds__(1024) norm_sums_kernel(const float* part, int blocks, int H,
                                                        void* dw_post, void* dw_pre,
                                                        void* dgate) {
  griddep_sync();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c0 = blockIdx.x * 128 + lane;
  void* out = blockIdx.y == 0 ? dw_post : blockIdx.y == 1 ? dw_pre : dgate;
  if (out == nullptr) return;
  __shared__ float s[32][128];
  float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int b = w; b < blocks; b += 32) {
    const float* p = part + (static_cast<size_t>(b) * 3 + blockIdx.y) * H;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c0 + 32 * i < H) v[i] += p[c0 + 32 * i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[w][lane + 32 * i] = v[i];
  __syncthreads();
  const int c = blockIdx.x * 128 + threadIdx.x;
  if (threadIdx.x >= 128 || c >= H) return;
  float sum = s[0][threadIdx.x];
#pragma unroll
  for (int i = 1; i < 32; ++i) sum += s[i][threadIdx.x];
  put_elem<DT>(out, c, sum);
}

}  // namespace moe
