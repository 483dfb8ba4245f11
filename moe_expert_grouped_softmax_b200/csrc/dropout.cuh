// Dropout: out[t, c] = keep(t, c) x[t, c] / (1 - p), forward and backward
// (the gradient's mask is the same one).  Streams x once; a dropped element
// is written as zero whatever x holds there.
//
// HBM is the floor (2 elements moved: 58 us below); the generator's five 32 x
// 32-bit products an element, at 30 lanes a clock and SM, take 55 of the 16-bit
// types' time and its eleven integer operations about as much on another pipe
// (61% busy).  None is full: a warp loads, draws and stores in turn, and 16
// warps an SM do not cover that.  32768 x 2880 bf16: 88 us, 4.3 TB/s; fp32: 125
// us, 6.0 TB/s.
#pragma once

#include "rows.cuh"

namespace moe {

constexpr int kDropBlocksPerSM = 2;

// A thread takes two pieces of a row an iteration, one grid stride apart, both
// loaded before the generator runs.  A piece is PC chunks (32 bytes where
// rows allow it, PC = 2): its counters share their row, so the first two
// rounds' products of the row and the offset are formed once.  Pieces go by
// their place in the row-major list; (row, piece) steps by (stride / per_row,
// stride % per_row), so that only the first costs a division.  Rows that are
// not 16-byte aligned go by whole warps' pieces (per_row a multiple of 32).
template <int DT, bool ALIGNED, int PC>
__global__ void __launch_bounds__(256, kDropBlocksPerSM) dropout_kernel(const void* x, void* out,
                                                                        int T, int H,
                                                                        const DropArgs drop) {
  using C = Chunk<DT>;
  constexpr int U = 2, CH = C::CH, W = PC * CH;
  griddep_sync();
  const DropKey key = drop_key(drop);
  const int per_row = ALIGNED ? (H + W - 1) / W : (H + 32 * CH - 1) / (32 * CH) * 32;
  const uint64_t stride = static_cast<uint64_t>(gridDim.x) * blockDim.x;
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  int64_t t = static_cast<int64_t>(first / per_row);
  int q = static_cast<int>(first % per_row);
  const int64_t dt = static_cast<int64_t>(stride / per_row);
  const int dq = static_cast<int>(stride % per_row);
  while (t < T) {
    int row[U], n[U];
    bool in[U];
    uint4 v[U][PC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      in[u] = t < T;
      row[u] = static_cast<int>(in[u] ? t : 0);
      n[u] = q * PC;
#pragma unroll
      for (int j = 0; j < PC; ++j) v[u][j] = make_uint4(0, 0, 0, 0);
      if (in[u]) {
        const char* rp = row_at<DT>(x, row[u], H);
        if constexpr (PC == 2) load32(rp + static_cast<size_t>(n[u]) * 16, v[u][0], v[u][1]);
        else v[u][0] = C::template load<ALIGNED>(rp, C::template first<ALIGNED>(n[u]), H);
      }
      t += dt;
      q += dq;
      if (q >= per_row) {
        q -= per_row;
        ++t;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int at[PC];
#pragma unroll
      for (int j = 0; j < PC; ++j) at[j] = n[u] + j;
      DropWords<CH, PC, ALIGNED> words;
      words.draw(key, row[u], at);
#pragma unroll
      for (int j = 0; j < PC; ++j) {
        float f[CH];
        C::unpack(v[u][j], f);
#pragma unroll
        for (int i = 0; i < CH; ++i) f[i] = words.keep(drop, j, i) ? f[i] * drop.scale : 0.f;
        v[u][j] = C::pack(f);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!in[u]) continue;
      char* rp = row_at<DT>(out, row[u], H);
      if constexpr (PC == 2) store32(rp + static_cast<size_t>(n[u]) * 16, v[u][0], v[u][1]);
      else C::template store<ALIGNED>(rp, C::template first<ALIGNED>(n[u]), H, v[u][0]);
    }
  }
}

}  // namespace moe
