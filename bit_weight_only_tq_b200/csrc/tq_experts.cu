// tq_experts.cu -- products of each expert's rows with its packed weights (tq_gemm_experts,
// w4g_gemm_experts of include/tq_moe.h).  The rows of expert e are offsets[e] .. offsets[e + 1] - 1
// of the sorted rows; only the device knows those numbers, so every kernel derives its work from
// them and the host sizes the grid from R, E and N alone.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tq_common.cuh"

namespace tq {

struct ExpertArgs {
  const __half* x;
  const uint8_t* w;        // [E][N][row_bytes]
  const __half* sc;        // ternary [E][N]; W4A16 [E][N][K / 128]
  const uint8_t* zp;       // W4A16 [E][N][K / 128] or null
  const __half* bias;      // [E][N] or null
  __half* y;               // [R][N]
  const int32_t* offsets;  // [E + 1]
  const int32_t* order;    // [R] or null
  int64_t X, R, N, K;
  int E, top_k;
};

// The x row of sorted row r, or -1.
__device__ __forceinline__ int64_t expert_x_row(const ExpertArgs& a, int64_t r) {
  const int64_t t = a.order ? a.order[r] / a.top_k : r;
  return t >= 0 && t < a.X ? t : -1;
}

// ---------------------------------------------------------------------------------------------
// Any shape and alignment: one warp per (row, 32 outputs), lanes over k.  Correct, not fast.
// ---------------------------------------------------------------------------------------------
template <bool kInt4>
__global__ void __launch_bounds__(256) experts_generic_kernel(const ExpertArgs a) {
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31;
  const int64_t nb = (a.N + 31) / 32, total = a.offsets[a.E];
  const int64_t rows = total < a.R ? total : a.R, G = a.K / 128;
  const int64_t row_bytes = kInt4 ? a.K / 2 : (a.K + 3) / 4;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); task < rows * nb; task += step) {
    const int64_t r = task / nb, n0 = (task - r * nb) * 32;
    int lo = 0, hi = a.E;  // the expert: offsets[lo] <= r < offsets[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.offsets[mid] <= r)
        lo = mid;
      else
        hi = mid;
    }
    const int64_t xr = expert_x_row(a, r);
    for (int64_t n = n0; n < n0 + 32 && n < a.N; ++n) {
      const int64_t en = static_cast<int64_t>(lo) * a.N + n;
      const uint8_t* w = a.w + en * row_bytes;
      float acc = 0.0f;
      if (xr >= 0) {
        for (int64_t k = lane; k < a.K; k += 32) {
          const float xv = __half2float(a.x[xr * a.K + k]);
          if (kInt4) {
            const int u = (w[k >> 1] >> (4 * (k & 1))) & 15;
            const int z = a.zp ? a.zp[en * G + (k >> 7)] : 8;
            acc = fmaf(xv, __half2float(a.sc[en * G + (k >> 7)]) * static_cast<float>(u - z), acc);
          } else {
            acc = fmaf(xv, static_cast<float>(((w[k >> 2] >> (2 * (k & 3))) & 3) - 1), acc);
          }
        }
      }
      acc = warp_sum(acc);
      if (lane == 0) {
        if (!kInt4) acc *= __half2float(a.sc[en]);
        if (a.bias) acc += __half2float(a.bias[en]);
        a.y[r * a.N + n] = __float2half_rn(acc);
      }
    }
  }
}

template <bool kInt4>
static cudaError_t launch_experts_generic(const ExpertArgs& a, cudaStream_t s) {
  return launch_pdl(experts_generic_kernel<kInt4>, dim3(row_grid(a.R * ((a.N + 31) / 32), 8, 8)), dim3(256), 0, 1, s, a);
}

cudaError_t launch_gemm_experts(bool int4, int path, const ExpertArgs& a, cudaStream_t s) {
  (void)path;
  return int4 ? launch_experts_generic<true>(a, s) : launch_experts_generic<false>(a, s);
}

}  // namespace tq
