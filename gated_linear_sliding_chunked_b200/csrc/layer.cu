// What the layer operators share on the host side: the workspace query and
// the fixed-order sum of per-block partials of parameter gradients.
#include "layer.cuh"

namespace lz {
namespace {

constexpr int kCols = 32;

// One block per 32 columns: the row lanes add every kLanes-th row each
// (coalesced across columns), then the lanes' sums are added in order.
template <int kLanes>
__global__ void __launch_bounds__(kCols* kLanes) sum_rows_kernel(SumRowsParams p) {
  __shared__ float red[kLanes][kCols];
  const int c = threadIdx.x % kCols, l = threadIdx.x / kCols;
  const size_t col = (size_t)blockIdx.x * kCols + c, C = p.c0 + p.c1 + p.c2;
  float s = 0.f;
  if (col < C) {
#pragma unroll 4
    for (int r = l; r < p.P; r += kLanes) s += p.part[(size_t)r * p.ld + col];
  }
  red[l][c] = s;
  __syncthreads();
  if (l == 0 && col < C) {
    float t = 0.f;
#pragma unroll
    for (int x = 0; x < kLanes; ++x) t += red[x][c];
    size_t i = col;
    float* out = p.out0;
    if (i >= p.c0) {
      i -= p.c0;
      out = p.out1;
      if (i >= p.c1) {
        i -= p.c1;
        out = p.out2;
      }
    }
    if (out) out[i] = t;
  }
}

}  // namespace

cudaError_t launch_sum_rows(const SumRowsParams& p, cudaStream_t s) {
  const size_t C = p.c0 + p.c1 + p.c2;
  if (C == 0) return cudaSuccess;
  ScopedTiming tm("layer_sum_rows", s);
  const unsigned grid = (unsigned)((C + kCols - 1) / kCols);
  // 1184 partials of 3 x 1024 values: 27 us with 8 lanes, 9.5 to 11 us with 32
  if (p.P > 128) sum_rows_kernel<32><<<grid, kCols * 32, 0, s>>>(p);
  else sum_rows_kernel<8><<<grid, kCols * 8, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace lz

extern "C" size_t lz_layer_workspace_bytes(const void* d, int which) {
  if (!d) return 0;
  switch (which) {
    case LZ_WS_CONV_BWD: return lz::conv_bwd_ws((const lz_conv_dims*)d);
    case LZ_WS_SCAN_FWD:
    case LZ_WS_SCAN_BWD:
    case LZ_WS_SCAN_BWD_SAVED:
    case LZ_WS_SCAN_STATES: return lz::scan_ws((const lz_scan_dims*)d, which);
    case LZ_WS_NORM_BWD: return lz::norm_bwd_ws((const lz_norm_dims*)d);
    default: return 0;
  }
}
