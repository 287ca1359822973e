// tq_dx.cu -- the packed products' gradient for x, dx[m, k] = sum_n dy[m, n] What[n, k] (include/tq_lora.h).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "tq_common.cuh"

namespace tq {

struct DxArgs {
  const __half* dy;
  const uint8_t* w;   // ternary [N][ceil(K / 4)] or W4A16 [N][K / 2] bytes
  const __half* sc;   // ternary [N]; W4A16 [N][K / 128]
  const uint8_t* zp;  // W4A16 zero-points [N][K / 128], or null (symmetric)
  __half* dx;
  int64_t M, N, K;
};

// ---------------------------------------------------------------------------------------------
// Any shape and alignment: a thread per byte (ternary, four columns) or word (INT4, eight columns) of a
// weight row and kDxGenM tokens; a CTA stages dy and the scales of kDxGenN rows in shared memory.
// ---------------------------------------------------------------------------------------------
constexpr int kDxGenThreads = 128;
constexpr int kDxGenM = 8;
constexpr int kDxGenN = 64;

template <bool kInt4>
__global__ void __launch_bounds__(kDxGenThreads) dx_generic_kernel(const DxArgs a) {
  constexpr int kCols = kInt4 ? 8 : 4;
  __shared__ float ds[kDxGenN][kDxGenM];
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int64_t units = (a.K + kCols - 1) / kCols, G = a.K >> 7;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * kDxGenThreads + threadIdx.x;
  for (int64_t m0 = static_cast<int64_t>(blockIdx.y) * kDxGenM; m0 < a.M;
       m0 += static_cast<int64_t>(gridDim.y) * kDxGenM) {
    float acc[kDxGenM][kCols] = {};
    for (int64_t n0 = 0; n0 < a.N; n0 += kDxGenN) {
      __syncthreads();
      for (int i = threadIdx.x; i < kDxGenN * kDxGenM; i += kDxGenThreads) {
        const int n = i % kDxGenN, m = i / kDxGenN;
        ds[n][m] = m0 + m < a.M && n0 + n < a.N ? __half2float(a.dy[(m0 + m) * a.N + n0 + n]) : 0.0f;
      }
      __syncthreads();
      if (u >= units) continue;
      const int cnt = static_cast<int>(a.N - n0 < kDxGenN ? a.N - n0 : kDxGenN);
      for (int i = 0; i < cnt; ++i) {
        const int64_t n = n0 + i;
        uint32_t word;
        float s, z;
        if (kInt4) {
          word = reinterpret_cast<const uint32_t*>(a.w)[n * units + u];
          s = __half2float(a.sc[n * G + (u >> 4)]);
          z = a.zp ? static_cast<float>(a.zp[n * G + (u >> 4)]) : 8.0f;
        } else {
          word = a.w[n * units + u];
          s = __half2float(a.sc[n]);
          z = 1.0f;
        }
        float w[kCols];
#pragma unroll
        for (int e = 0; e < kCols; ++e)
          w[e] = s * (static_cast<float>((word >> ((kInt4 ? 4 : 2) * e)) & (kInt4 ? 15u : 3u)) - z);
#pragma unroll
        for (int m = 0; m < kDxGenM; ++m) {
          const float d = ds[i][m];
#pragma unroll
          for (int e = 0; e < kCols; ++e) acc[m][e] = fmaf(d, w[e], acc[m][e]);
        }
      }
    }
    if (u < units) {
#pragma unroll
      for (int m = 0; m < kDxGenM; ++m)
#pragma unroll
        for (int e = 0; e < kCols; ++e)
          if (m0 + m < a.M && u * kCols + e < a.K) a.dx[(m0 + m) * a.K + u * kCols + e] = __float2half_rn(acc[m][e]);
    }
  }
}

static cudaError_t launch_dx_generic(bool int4, const DxArgs& a, cudaStream_t s) {
  const int64_t units = int4 ? a.K / 8 : (a.K + 3) / 4, mt = (a.M + kDxGenM - 1) / kDxGenM;
  const dim3 grid(static_cast<unsigned>((units + kDxGenThreads - 1) / kDxGenThreads),
                  static_cast<unsigned>(mt < 65535 ? mt : 65535));
  return launch_pdl(int4 ? dx_generic_kernel<true> : dx_generic_kernel<false>, grid, dim3(kDxGenThreads), 0, 1, s, a);
}

bool dx_supported(int64_t N, int64_t K) { return N > 0 && N % 8 == 0 && K % 64 == 0; }

cudaError_t launch_dx(bool int4, int path, const DxArgs& a, cudaStream_t s) { return launch_dx_generic(int4, a, s); }

}  // namespace tq
