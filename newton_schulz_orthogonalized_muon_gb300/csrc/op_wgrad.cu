// The weight's gradient of a linear layer from its input kept in 8 bits:
//   dw[o][n] = sum over tokens t of dy[t][o] * x[t][n]  (+ add[o][n]),
//   x[t][n] = code[t][n] * 2^(scale[n / 128][t] - 127).
//
// 64 x 64 output tiles, 16 tokens a step through shared memory, 4 x 4 outputs
// a thread, fp32 sums.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "op_common.cuh"

namespace muon {
namespace {

constexpr int WT = 64, WK = 16;

__global__ void __launch_bounds__(256) act8_wgrad_kernel(const WgradParams p) {
  __shared__ float sy[WK][WT], sx[WK][WT];
  const int o0 = blockIdx.y * WT, n0 = blockIdx.x * WT;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (long long t0 = 0; t0 < p.rows; t0 += WK) {
    for (int i = threadIdx.x; i < WK * WT; i += 256) {
      const int k = i / WT, c = i % WT;
      const long long t = t0 + k;
      sy[k][c] = t < p.rows && o0 + c < p.out ? to_f32(p.dy[t * p.ldy + o0 + c]) : 0.f;
      float x = 0.f;
      if (t < p.rows && n0 + c < p.cols) {
        const __half h = __half(__nv_cvt_fp8_to_halfraw(p.codes[t * p.ldc + n0 + c], __NV_E4M3));
        x = to_f32(h) * __int_as_float(p.scales[((n0 + c) >> 7) * p.lds + t] << 23);
      }
      sx[k][c] = x;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WK; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = sy[k][ty * 4 + i];
        b[i] = sx[k][tx * 4 + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 4; ++j) {
      const int o = o0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (o >= p.out || n >= p.cols) continue;
      float v = acc[i][j];
      if (p.add != nullptr) v += load_f32(p.add, o * p.ldadd + n, p.odtype);
      store_from_f32(p.dw, o * p.ldw + n, p.odtype, v);
    }
  }
}

}  // namespace

cudaError_t launch_act8_wgrad(const WgradParams& p, cudaStream_t s) {
  const dim3 grid((p.cols + WT - 1) / WT, (p.out + WT - 1) / WT);
  act8_wgrad_kernel<<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace muon
