// Dropout: out[t, c] = keep(t, c) x[t, c] / (1 - p), forward and backward
// (the gradient's mask is the same one).  Streams x once; a dropped element
// is written as zero whatever x holds there.
#pragma once

#include "rows.cuh"

namespace moe {

// Each thread takes chunks idx, idx + stride, ... of the row-major chunk
// list, stepping (row, chunk) by (stride / per_row, stride % per_row) so that
// only the first costs a division.
template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(256) dropout_kernel(const void* x, void* out, int T, int H,
                                                      const DropArgs drop) {
  using C = Chunk<DT>;
  griddep_sync();
  const DropKey key = drop_key(drop);
  const int per_row = (H + C::CH - 1) / C::CH;
  const uint64_t stride = static_cast<uint64_t>(gridDim.x) * blockDim.x;
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  int64_t t = static_cast<int64_t>(first / per_row);
  int q = static_cast<int>(first % per_row);
  const int64_t dt = static_cast<int64_t>(stride / per_row);
  const int dq = static_cast<int>(stride % per_row);
  while (t < T) {
    const int c = q * C::CH, row = static_cast<int>(t);
    const uint4 v = C::template load<ALIGNED>(row_at<DT>(x, row, H), c, H);
    const uint32_t m = drop_bits<C::CH>(drop, key, row, c);
    float f[C::CH];
    C::unpack(v, f);
#pragma unroll
    for (int i = 0; i < C::CH; ++i) f[i] = (m >> i) & 1u ? f[i] * drop.scale : 0.f;
    C::template store<ALIGNED>(row_at<DT>(out, row, H), c, H, C::pack(f));
    t += dt;
    q += dq;
    if (q >= per_row) {
      q -= per_row;
      ++t;
    }
  }
}

}  // namespace moe
