// tq_moe.cu -- mixture-of-experts routing and the exchange of rows between tokens and experts
// (include/tq_moe.h): softmax top-k, the stable counting sort of slots by expert, and the row
// kernels (gather, weighted sum, their gradients).  All of them are bound by memory or, at the
// sizes of a decode step, by the latency of one launch.
//
// Every kernel is launched with programmatic dependent launch: it lets the next kernel of the
// stream start its prologue at once and waits for the previous one before its first access.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "tq_common.cuh"

namespace tq {

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 32;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// W consecutive elements as one memory access (W sizeof(T) = 2, 4, 8 or 16 bytes, aligned).
template <typename T, int W>
struct alignas(sizeof(T) * W) Vec {
  T v[W];
};

template <typename... KArgs, typename... Args>
static cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t s,
                              Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// ---------------------------------------------------------------------------------------------
// Router.  One warp per token; lane l holds VPL scores in registers, in groups of W consecutive
// ones (one load each): v -> expert (v / W) 32 W + W l + v % W, increasing in v.  The choices are k
// rounds of a warp-wide maximum over each lane's best; only the lane that held the winner looks
// through its scores again, so that a round costs one reduction (and that rescan: the warp waits for it).
// 8192 tokens, 256 experts, top 8, bf16: 8.5 us, bound by instructions (the ALU 72 % busy), and the gradient
// 5.9 (renormalised 4.4), a chain of shared-memory steps with one token per warp in flight (issue 35 %); their
// bytes take 2.1.  16 tokens: 2.0 us, one launch.
// ---------------------------------------------------------------------------------------------
constexpr int kRouteThreads = 128;

// Order-preserving key of a score: larger score, larger key; -0 and +0 share one; 0 for what may
// not be chosen (-inf, NaN).
__device__ __forceinline__ uint32_t route_key(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float route_unkey(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// The same of a 16-bit score, from its value: a 16-bit key.
__device__ __forceinline__ uint32_t route_bits16(float x, __half) { return __half_as_ushort(__float2half_rn(x)); }
__device__ __forceinline__ uint32_t route_bits16(float x, __nv_bfloat16) { return __float_as_uint(x) >> 16; }
__device__ __forceinline__ uint32_t route_bits16(float, float) { return 0u; }  // not used
__device__ __forceinline__ float route_value16(uint32_t b, __half) {
  return __half2float(__ushort_as_half(static_cast<uint16_t>(b)));
}
__device__ __forceinline__ float route_value16(uint32_t b, __nv_bfloat16) { return __uint_as_float(b << 16); }
__device__ __forceinline__ float route_value16(uint32_t, float) { return 0.0f; }  // not used
template <typename T>
__device__ __forceinline__ uint32_t route_key16(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t u = route_bits16(x + 0.0f, T());
  return (u & 0x8000u) ? ~u & 0xFFFFu : u | 0x8000u;
}
template <typename T>
__device__ __forceinline__ float route_unkey16(uint32_t k) {
  return route_value16((k & 0x8000u) ? k & 0x7FFFu : ~k & 0xFFFFu, T());
}
// exp(x - m) for x <= m; 1 where they are equal, which at m = +inf is the limit.
__device__ __forceinline__ float exp_below(float x, float m) { return x == m ? 1.0f : expf(x - m); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

template <typename T, int VPL, int W>
__device__ __forceinline__ void route_load(const T* row, int E, int lane, float (&x)[VPL]) {
#pragma unroll
  for (int g = 0; g < VPL / W; ++g) {
    const int i0 = (g * 32 + lane) * W;
    if (i0 < E) {  // E % W == 0: whole groups
      const Vec<T, W> t = *reinterpret_cast<const Vec<T, W>*>(row + i0);
#pragma unroll
      for (int c = 0; c < W; ++c) x[g * W + c] = to_f32(t.v[c]);
    } else {
#pragma unroll
      for (int c = 0; c < W; ++c) x[g * W + c] = -INFINITY;
    }
  }
}

template <typename T, int VPL, int W>
__global__ void __launch_bounds__(kRouteThreads)
    moe_route_kernel(const T* __restrict__ logits, float* __restrict__ weights, int32_t* __restrict__ ids, int64_t T_,
                     int E, int k, int renorm) {
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + (threadIdx.x >> 5);
  if (t >= T_) return;
  float x[VPL];
  route_load<T, VPL, W>(logits + t * E, E, lane, x);
  auto expert = [&](int v) { return (v / W) * 32 * W + W * lane + v % W; };
  uint32_t my_key = 0;  // lane j: the j-th choice
  int my_id = -1;
  uint32_t top = 0;
  if (sizeof(T) == 2) {
    // a 16-bit score's key fits the upper half of a word with the expert's complement below it: one
    // maximum finds the largest score and the lowest expert among equals
    uint32_t word[VPL], best = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const uint32_t key = route_key16<T>(x[v]);
      word[v] = key ? (key << 16) | (0xFFFFu - static_cast<uint32_t>(expert(v))) : 0u;
      best = max(best, word[v]);
    }
    for (int j = 0; j < k; ++j) {
      const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
      if (m == 0) break;
      if (j == 0) top = m;
      if (lane == j) my_key = m;
      if (j + 1 < k && best == m) {  // the lane that held it looks for its next
        best = 0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          if (word[v] == m) word[v] = 0;
          best = max(best, word[v]);
        }
      }
    }
    if (my_key) my_id = static_cast<int>(0xFFFFu - (my_key & 0xFFFFu));
  } else {
    uint32_t key[VPL];
    uint32_t bk = 0;
    int bi = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      key[v] = route_key(x[v]);
      if (key[v] > bk) {
        bk = key[v];
        bi = expert(v);
      }
    }
    for (int j = 0; j < k; ++j) {
      const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, bk);
      if (m == 0) break;
      if (j == 0) top = m;
      const int i = __reduce_min_sync(0xFFFFFFFFu, bk == m ? bi : 0x7FFFFFFF);
      if (lane == j) {
        my_key = m;
        my_id = i;
      }
      if (j + 1 < k && bk == m && bi == i) {  // the lane that held it looks for its next
        bk = 0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          if (expert(v) == i) key[v] = 0;
          if (key[v] > bk) {
            bk = key[v];
            bi = expert(v);
          }
        }
      }
    }
  }
  auto value = [](uint32_t m) { return sizeof(T) == 2 ? route_unkey16<T>(m >> 16) : route_unkey(m); };
  const float mx = value(top);
  float e = my_id >= 0 ? exp_below(value(my_key), mx) : 0.0f;
  float sum;
  if (renorm) {
    sum = warp_sum(e);
  } else {
    sum = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      if (x[v] > -INFINITY) sum += exp_below(x[v], mx);
    sum = warp_sum(sum);
  }
  if (lane < k) {
    weights[t * k + lane] = my_id >= 0 ? e / sum : 0.0f;
    ids[t * k + lane] = my_id;
  }
}

template <typename T, int VPL, int W>
__global__ void __launch_bounds__(kRouteThreads)
    moe_route_bwd_kernel(const float* __restrict__ dweights, const T* __restrict__ logits,
                         const float* __restrict__ weights, const int32_t* __restrict__ ids, T* __restrict__ dlogits,
                         int64_t T_, int E, int k, int renorm) {
  __shared__ float rows[kRouteThreads / 32][VPL * 32];
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + warp;
  if (t >= T_) return;
  float* row = rows[warp];
  int id = -1;
  float g = 0.0f, w = 0.0f;
  if (lane < k) {
    id = ids[t * k + lane];
    if (id < 0 || id >= E) {
      id = -1;
    } else {
      g = dweights[t * k + lane];
      w = weights[t * k + lane];
    }
  }
  float x[VPL];
  if (!renorm) route_load<T, VPL, W>(logits + t * E, E, lane, x);
#pragma unroll
  for (int v = 0; v < VPL; ++v) row[v * 32 + lane] = 0.0f;
  const float inner = warp_sum(g * w);
  __syncwarp();
  // distinct ids: one addition per element
  if (id >= 0) atomicAdd(&row[id], renorm ? w * (g - inner) : g);
  __syncwarp();
  float mx = -INFINITY, inv = 0.0f;
  if (!renorm) {
#pragma unroll
    for (int v = 0; v < VPL; ++v) mx = fmaxf(mx, x[v]);  // fmaxf passes over a NaN
    mx = warp_max(mx);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      x[v] = x[v] > -INFINITY ? exp_below(x[v], mx) : 0.0f;
      sum += x[v];
    }
    sum = warp_sum(sum);
    inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  }
#pragma unroll
  for (int q = 0; q < VPL / W; ++q) {
    const int i0 = (q * 32 + lane) * W;
    if (i0 < E) {
      Vec<T, W> o;
#pragma unroll
      for (int c = 0; c < W; ++c) {
        const float r = row[i0 + c];
        o.v[c] = from_f32<T>(renorm ? r : x[q * W + c] * inv * (r - inner));
      }
      *reinterpret_cast<Vec<T, W>*>(dlogits + t * E + i0) = o;
    }
  }
}

// Calls f(VPL, W) with the smallest register count that holds E scores per warp and the widest
// access that the row stride and the pointers allow.
template <typename T, typename F>
static cudaError_t route_dispatch(int64_t E, uintptr_t ptrs, F f) {
  auto vec = [&](int w) { return E % w == 0 && ptrs % (w * sizeof(T)) == 0; };
#define TQ_ROUTE(VPL)                                                                     \
  {                                                                                       \
    constexpr int W = (VPL) < static_cast<int>(16 / sizeof(T)) ? (VPL) : static_cast<int>(16 / sizeof(T)); \
    if (W > 1 && vec(W)) return f(std::integral_constant<int, VPL>(), std::integral_constant<int, W>()); \
    return f(std::integral_constant<int, VPL>(), std::integral_constant<int, 1>());       \
  }
  if (E <= 32) TQ_ROUTE(1)
  if (E <= 64) TQ_ROUTE(2)
  if (E <= 128) TQ_ROUTE(4)
  if (E <= 256) TQ_ROUTE(8)
  if (E <= 512) TQ_ROUTE(16)
  TQ_ROUTE(32)
#undef TQ_ROUTE
}

template <typename T>
static cudaError_t route_t(const void* logits, float* weights, int32_t* ids, int64_t n, int64_t E, int k, int renorm,
                           cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((n + kRouteThreads / 32 - 1) / (kRouteThreads / 32)));
  return route_dispatch<T>(E, reinterpret_cast<uintptr_t>(logits), [&](auto vpl, auto w) {
    return launch_pdl(moe_route_kernel<T, decltype(vpl)::value, decltype(w)::value>, grid, dim3(kRouteThreads), 0, 1, s,
                      static_cast<const T*>(logits), weights, ids, n, static_cast<int>(E), k, renorm);
  });
}

template <typename T>
static cudaError_t route_bwd_t(const float* dw, const void* logits, const float* weights, const int32_t* ids,
                               void* dlogits, int64_t n, int64_t E, int k, int renorm, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((n + kRouteThreads / 32 - 1) / (kRouteThreads / 32)));
  return route_dispatch<T>(
      E, reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits), [&](auto vpl, auto w) {
        return launch_pdl(moe_route_bwd_kernel<T, decltype(vpl)::value, decltype(w)::value>, grid,
                          dim3(kRouteThreads), 0, 1, s, dw, static_cast<const T*>(logits), weights, ids,
                          static_cast<T*>(dlogits), n, static_cast<int>(E), k, renorm);
      });
}

cudaError_t launch_moe_route(const void* logits, int dtype, float* weights, int32_t* ids, int64_t n, int64_t E, int k,
                             int renorm, cudaStream_t s) {
  if (dtype == 0) return route_t<float>(logits, weights, ids, n, E, k, renorm, s);
  if (dtype == 1) return route_t<__half>(logits, weights, ids, n, E, k, renorm, s);
  return route_t<__nv_bfloat16>(logits, weights, ids, n, E, k, renorm, s);
}

cudaError_t launch_moe_route_bwd(const float* dw, const void* logits, int dtype, const float* weights,
                                 const int32_t* ids, void* dlogits, int64_t n, int64_t E, int k, int renorm,
                                 cudaStream_t s) {
  if (dtype == 0) return route_bwd_t<float>(dw, logits, weights, ids, dlogits, n, E, k, renorm, s);
  if (dtype == 1) return route_bwd_t<__half>(dw, logits, weights, ids, dlogits, n, E, k, renorm, s);
  return route_bwd_t<__nv_bfloat16>(dw, logits, weights, ids, dlogits, n, E, k, renorm, s);
}

// ---------------------------------------------------------------------------------------------
// Sort.  One launch of one cluster: CTA c of C and warp w of W own a contiguous run of L slots.
// Each warp counts its run per expert in shared memory; prefix sums over the warps, over the
// CTAs (distributed shared memory) and over the experts give every (warp, expert) its first
// sorted row; each warp then walks its run again, 32 slots at a time, and a slot's row is that
// start plus the number of equal ids before it in the strip (match.any).  Stable and without
// atomics whose order could show: the counting adds are integers.  Latency bounds it; eight CTAs are what
// one portable cluster, and so one launch without a workspace, can have.  us of 128 experts: 104 slots 2.3,
// 2048 7.2 and 8192 13.7 (one CTA), 8193 8.5, 32768 10.5, 131072 25, 524288 82.
// ---------------------------------------------------------------------------------------------
constexpr int kSortMaxWarps = 32;
constexpr int kSortCluster = 8;

__global__ void __launch_bounds__(kSortMaxWarps * 32, 1)
    moe_sort_kernel(const int32_t* __restrict__ ids, int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                    int32_t* __restrict__ pos, int64_t R, int E, int64_t L, int C) {
  extern __shared__ int sort_smem[];
  const int nt = blockDim.x, W = nt >> 5, B = E + 1;  // bin E: slots of no expert
  int* cnt = sort_smem;                               // [W][B]
  int* tot = cnt + W * B;                             // [B] this CTA's counts
  int* start = tot + B;                               // [B] first row of this CTA's slots per bin
  int* scan = start + B;                              // [W]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  pdl_allow_dependents();
  for (int i = tid; i < W * B; i += nt) cnt[i] = 0;
  pdl_wait_prior_grids();
  const int64_t lo = (static_cast<int64_t>(rank) * W + warp) * L;
  const int64_t hi = lo + L < R ? lo + L : R;
  __syncthreads();
  auto bin = [&](int64_t i) {
    const int id = ids[i];
    return id >= 0 && id < E ? id : E;
  };
#pragma unroll 4
  for (int64_t i = lo + lane; i < hi; i += 32) atomicAdd(&cnt[warp * B + bin(i)], 1);
  __syncthreads();
  for (int e = tid; e < B && W <= 8; e += nt) {  // few warps: a thread per bin
    int run = 0;
#pragma unroll 4
    for (int w = 0; w < W; ++w) {
      const int c = cnt[w * B + e];
      cnt[w * B + e] = run;
      run += c;
    }
    tot[e] = run;
  }
  for (int e = warp; e < B && W > 8; e += W) {  // a warp per bin, lane w: warp w's count
    const int c = lane < W ? cnt[lane * B + e] : 0;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane < W) cnt[lane * B + e] = incl - c;
    if (lane == 31) tot[e] = incl;
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  // thread tid: the experts [tid P, tid P + P) of the scan over experts
  const int P = (E + nt - 1) / nt;
  int sum = 0;
  for (int e = tid * P; e < E && e < tid * P + P; ++e) {
    int before = 0, all = tot[e];
    if (C > 1) {
      int v[kSortCluster];
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c)
        v[c] = __float_as_int(ld_shared_cluster_f32(mapa_shared(smem_u32(&tot[e]), static_cast<uint32_t>(c))));
      all = 0;
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c) {
        before += c < rank ? v[c] : 0;
        all += v[c];
      }
    }
    start[e] = sum + before;
    if (rank == 0) offsets[e] = sum;  // completed below
    sum += all;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int base = incl - sum, total = 0;
  for (int w = 0; w < W; ++w) {
    if (w < warp) base += scan[w];
    total += scan[w];
  }
  for (int e = tid * P; e < E && e < tid * P + P; ++e) {
    start[e] += base;
    if (rank == 0) offsets[e] += base;
  }
  if (tid == 0) {
    int before = 0;
    for (int c = 0; c < rank; ++c)
      before += __float_as_int(ld_shared_cluster_f32(mapa_shared(smem_u32(&tot[E]), static_cast<uint32_t>(c))));
    start[E] = total + before;
    if (rank == 0) offsets[E] = total;
  }
  // no CTA leaves while another reads its counts: the wait is at the end
  if (C > 1) cluster_arrive();
  __syncthreads();
  int* mine = cnt + warp * B;
  for (int64_t s0 = lo; s0 < hi; s0 += 32) {
    const int64_t i = s0 + lane;
    const bool in = i < hi;
    const int b = in ? bin(i) : E + 1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, b);
    const int before = __popc(same & ((1u << lane) - 1u));
    int row = 0;
    if (in) row = start[b] + mine[b] + before;
    __syncwarp();
    if (in && before == 0) mine[b] += __popc(same);
    __syncwarp();
    if (in) {
      order[row] = static_cast<int32_t>(i);
      pos[i] = b < E ? row : -1;
    }
  }
  if (C > 1) cluster_wait();
}

cudaError_t launch_moe_sort(const int32_t* ids, int32_t* offsets, int32_t* order, int32_t* pos, int64_t R, int64_t E,
                            cudaStream_t s) {
  // one CTA while its warps walk at most eight strips each; a cluster of eight beyond
  const int C = R <= 8 * 32 * kSortMaxWarps ? 1 : kSortCluster;
  int W = static_cast<int>((R + 31) / 32);
  W = C > 1 || W > kSortMaxWarps ? kSortMaxWarps : (W < 4 ? 4 : W);
  int64_t L = (R + static_cast<int64_t>(C) * W - 1) / (static_cast<int64_t>(C) * W);
  L = (L + 31) / 32 * 32;
  const size_t smem = sizeof(int) * ((static_cast<size_t>(W) + 2) * static_cast<size_t>(E + 1) + static_cast<size_t>(W));
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(moe_sort_kernel), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(moe_sort_kernel, dim3(static_cast<unsigned>(C)), dim3(static_cast<unsigned>(32 * W)), smem, C, s, ids,
                    offsets, order, pos, R, static_cast<int>(E), L, C);
}

// ---------------------------------------------------------------------------------------------
// Rows.  A CTA of 128 threads takes one row (or token) at a time, each thread a 16-byte vector per
// step, with the rows' loads of a step in flight together; 16 CTAs per SM keep enough of them in
// flight for HBM, which bounds these kernels (a warp per segment of a row, with more loads per
// thread and fewer threads, reached half the bandwidth).  With few rows a CTA takes one step of a row.
// 8192 tokens, top 2, 4096 wide, bf16: the sum 31 us (6.5 TB/s), its gradients 54 us (6.2 TB/s).
// 4096 tokens, top 8, 4096 wide, fp16: the gather writes 268 MB in 62 us, where a plain fill of as
// much memory takes 73: writes bound it.  Rows that are no multiple of 16 bytes go element by element: the sum
// 114 us, its gradients 108 (8192 x top 2, 4097 wide), the gather 129 (4096 x top 8).  A token's gradients are one
// CTA's work, since dweights sums over its row: 1 token, top 8, 4096 wide 4.8 us, the sum 1.7.
// ---------------------------------------------------------------------------------------------
constexpr int kRowThreads = 128;

// Grid of a kernel whose CTAs take `tasks` tasks with a stride of the grid.
static unsigned row_grid(int64_t tasks, int tasks_per_cta, int ctas_per_sm) {
  const int64_t want = (tasks + tasks_per_cta - 1) / tasks_per_cta;
  const int64_t cap = static_cast<int64_t>(current_device_info().num_sms) * ctas_per_sm;
  return static_cast<unsigned>(want < cap ? (want > 0 ? want : 1) : cap);
}

// How rows of `steps` steps are cut into tasks: whole rows, or single steps while the rows alone
// would not give every SM a few CTAs.
static int row_parts(int64_t rows, int steps) {
  return rows < 4 * current_device_info().num_sms ? steps : 1;
}

template <typename V>
__global__ void __launch_bounds__(kRowThreads)
    moe_gather_kernel(const V* __restrict__ x, const int32_t* __restrict__ order, const int32_t* __restrict__ offsets,
                      V* __restrict__ rows, int64_t T_, int64_t R, int nv, int parts, int k, int E) {
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int64_t kept = offsets[E] < R ? offsets[E] : R;
  const int part = blockIdx.x % parts, per = (nv + parts - 1) / parts;
  const int v0 = part * per + threadIdx.x, v1 = part * per + per < nv ? part * per + per : nv;
  const int64_t step = gridDim.x / parts;
  int64_t r = blockIdx.x / parts;
  int slot = r < kept ? order[r] : 0;
  for (; r < kept; r += step) {
    const int64_t t = slot >= 0 ? slot / k : T_;
    slot = r + step < kept ? order[r + step] : 0;  // the next row's, a row ahead
    if (t >= T_) continue;
    const V* src = x + t * nv;
    V* dst = rows + r * nv;
    for (int v = v0; v < v1; v += 4 * kRowThreads) {
      V b[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (v + u * kRowThreads < v1) b[u] = src[v + u * kRowThreads];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (v + u * kRowThreads < v1) dst[v + u * kRowThreads] = b[u];
    }
  }
}

cudaError_t launch_moe_gather(const void* x, int elem, const int32_t* order, const int32_t* offsets, void* rows,
                              int64_t n, int64_t H, int k, int64_t E, cudaStream_t s) {
  const int64_t R = n * k, bytes = H * elem;
  const bool vec = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(rows) | static_cast<uintptr_t>(bytes)) & 15u) == 0;
  auto run = [&](auto v) {
    using V = decltype(v);
    const int nv = static_cast<int>(bytes / static_cast<int64_t>(sizeof(V)));
    const int parts = row_parts(R, (nv + kRowThreads - 1) / kRowThreads);
    const unsigned grid = row_grid(R, 1, 16) * static_cast<unsigned>(parts);
    return launch_pdl(moe_gather_kernel<V>, dim3(grid), dim3(kRowThreads), 0, 1, s, static_cast<const V*>(x), order, offsets,
                      static_cast<V*>(rows), n, R, nv, parts, k, static_cast<int>(E));
  };
  if (vec) return run(uint4());
  return elem == 4 ? run(uint32_t()) : run(uint16_t());
}

// out[t] = sum_j w_j y[pos_j], added in the order of j, KB rows at a time.
template <typename T, int VE, int KB>
__global__ void __launch_bounds__(kRowThreads)
    moe_combine_kernel(const T* __restrict__ y, const int32_t* __restrict__ pos, const float* __restrict__ weights,
                       T* __restrict__ out, int64_t T_, int64_t R, int H, int parts, int k) {
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int steps = (H + kRowThreads * VE - 1) / (kRowThreads * VE);
  const int part = blockIdx.x % parts, per = (steps + parts - 1) / parts * kRowThreads * VE;
  const int h1 = part * per + per < H ? part * per + per : H;
  const int64_t step = gridDim.x / parts;
  for (int64_t t = blockIdx.x / parts; t < T_; t += step) {
    int p[KB];
    float w[KB];
    auto take = [&](int j0) {
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        p[j] = j0 + j < k ? pos[t * k + j0 + j] : -1;
        if (p[j] >= R) p[j] = -1;
        w[j] = weights && j0 + j < k ? weights[t * k + j0 + j] : 1.0f;
      }
    };
    take(0);
    for (int h = part * per + threadIdx.x * VE; h < h1; h += kRowThreads * VE) {
      float acc[VE];
#pragma unroll
      for (int c = 0; c < VE; ++c) acc[c] = 0.0f;
      for (int j0 = 0; j0 < k; j0 += KB) {
        if (k > KB) take(j0);
        Vec<T, VE> v[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (p[j] >= 0) v[j] = *reinterpret_cast<const Vec<T, VE>*>(y + static_cast<int64_t>(p[j]) * H + h);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          if (p[j] >= 0) {
#pragma unroll
            for (int c = 0; c < VE; ++c) acc[c] = fmaf(w[j], to_f32(v[j].v[c]), acc[c]);
          }
        }
      }
      Vec<T, VE> o;
#pragma unroll
      for (int c = 0; c < VE; ++c) o.v[c] = from_f32<T>(acc[c]);
      *reinterpret_cast<Vec<T, VE>*>(out + t * H + h) = o;
    }
  }
}

// The gradients of one token by one CTA, KB choices at a time: each thread holds a vector of dout,
// multiplies it into KB rows of y (dweights, reduced over the CTA at the end) and writes KB rows
// of dy; the loads of all KB rows are in flight together.
template <typename T, int VE, int KB>
__global__ void __launch_bounds__(kRowThreads)
    moe_combine_bwd_kernel(const T* __restrict__ dout, const T* __restrict__ y, const int32_t* __restrict__ pos,
                           const float* __restrict__ weights, T* __restrict__ dy, float* __restrict__ dweights,
                           int64_t T_, int64_t R, int64_t H, int k) {
  __shared__ float part[2][kRowThreads / 32][KB];
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int buf = 0;
  for (int64_t t = blockIdx.x; t < T_; t += gridDim.x) {
    for (int j0 = 0; j0 < k; j0 += KB, buf ^= 1) {
      int sp[KB];
      float sw[KB], dot[KB];
#pragma unroll
      for (int j = 0; j < KB; ++j) {
        sp[j] = j0 + j < k ? pos[t * k + j0 + j] : -1;
        if (sp[j] >= R) sp[j] = -1;
        sw[j] = dy && j0 + j < k ? weights[t * k + j0 + j] : 0.0f;
        dot[j] = 0.0f;
      }
      for (int64_t h = static_cast<int64_t>(tid) * VE; h < H; h += kRowThreads * VE) {
        const Vec<T, VE> d = *reinterpret_cast<const Vec<T, VE>*>(dout + t * H + h);
        Vec<T, VE> v[KB];
        if (dweights) {
#pragma unroll
          for (int j = 0; j < KB; ++j)
            if (sp[j] >= 0) v[j] = *reinterpret_cast<const Vec<T, VE>*>(y + static_cast<int64_t>(sp[j]) * H + h);
        }
        if (dy) {
#pragma unroll
          for (int j = 0; j < KB; ++j) {
            if (sp[j] >= 0) {
              Vec<T, VE> o;
#pragma unroll
              for (int c = 0; c < VE; ++c) o.v[c] = from_f32<T>(sw[j] * to_f32(d.v[c]));
              *reinterpret_cast<Vec<T, VE>*>(dy + static_cast<int64_t>(sp[j]) * H + h) = o;
            }
          }
        }
        if (dweights) {
#pragma unroll
          for (int j = 0; j < KB; ++j) {
            if (sp[j] >= 0) {
#pragma unroll
              for (int c = 0; c < VE; ++c) dot[j] = fmaf(to_f32(d.v[c]), to_f32(v[j].v[c]), dot[j]);
            }
          }
        }
      }
      if (dweights) {
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          const float s = warp_sum(dot[j]);
          if (lane == 0) part[buf][warp][j] = s;
        }
        __syncthreads();  // the other buffer's readers are past it when it is written again
        if (tid < KB && j0 + tid < k) {
          float s = 0.0f;
          for (int w = 0; w < kRowThreads / 32; ++w) s += part[buf][w][tid];
          dweights[t * k + j0 + tid] = s;
        }
      }
    }
  }
}

template <typename T>
static bool rows_vectorised(int64_t H, uintptr_t ptrs) {
  return ((ptrs | static_cast<uintptr_t>(H * static_cast<int64_t>(sizeof(T)))) & 15u) == 0;
}

template <typename T>
static cudaError_t combine_t(const void* y, const int32_t* pos, const float* weights, void* out, int64_t n, int64_t R,
                             int64_t H, int k, cudaStream_t s) {
  auto run2 = [&](auto ve, auto kb) {
    constexpr int VE = decltype(ve)::value;
    const int parts = row_parts(n, static_cast<int>((H + kRowThreads * VE - 1) / (kRowThreads * VE)));
    const unsigned grid = row_grid(n, 1, 16) * static_cast<unsigned>(parts);
    return launch_pdl(moe_combine_kernel<T, VE, decltype(kb)::value>, dim3(grid), dim3(kRowThreads), 0, 1, s,
                      static_cast<const T*>(y), pos, weights, static_cast<T*>(out), n, R, static_cast<int>(H), parts, k);
  };
  auto run = [&](auto ve) {
    if (k <= 2) return run2(ve, std::integral_constant<int, 2>());
    if (k <= 4) return run2(ve, std::integral_constant<int, 4>());
    return run2(ve, std::integral_constant<int, 8>());
  };
  if (rows_vectorised<T>(H, reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(out)))
    return run(std::integral_constant<int, 16 / sizeof(T)>());
  return run(std::integral_constant<int, 1>());
}

template <typename T>
static cudaError_t combine_bwd_t(const void* dout, const void* y, const int32_t* pos, const float* weights, void* dy,
                                 float* dweights, int64_t n, int64_t R, int64_t H, int k, cudaStream_t s) {
  auto run2 = [&](auto ve, auto kb) {
    const unsigned grid = row_grid(n, 1, 16);
    return launch_pdl(moe_combine_bwd_kernel<T, decltype(ve)::value, decltype(kb)::value>, dim3(grid),
                      dim3(kRowThreads), 0, 1, s, static_cast<const T*>(dout), static_cast<const T*>(y), pos,
                      weights, static_cast<T*>(dy), dweights, n, R, H, k);
  };
  auto run = [&](auto ve) {
    if (k <= 2) return run2(ve, std::integral_constant<int, 2>());
    if (k <= 4) return run2(ve, std::integral_constant<int, 4>());
    return run2(ve, std::integral_constant<int, 8>());
  };
  if (rows_vectorised<T>(H, reinterpret_cast<uintptr_t>(dout) | reinterpret_cast<uintptr_t>(y) |
                                reinterpret_cast<uintptr_t>(dy)))
    return run(std::integral_constant<int, 16 / sizeof(T)>());
  return run(std::integral_constant<int, 1>());
}

cudaError_t launch_moe_combine(const void* y, int dtype, const int32_t* pos, const float* weights, void* out, int64_t n,
                               int64_t R, int64_t H, int k, cudaStream_t s) {
  if (dtype == 0) return combine_t<float>(y, pos, weights, out, n, R, H, k, s);
  if (dtype == 1) return combine_t<__half>(y, pos, weights, out, n, R, H, k, s);
  return combine_t<__nv_bfloat16>(y, pos, weights, out, n, R, H, k, s);
}

cudaError_t launch_moe_combine_bwd(const void* dout, const void* y, int dtype, const int32_t* pos, const float* weights,
                                   void* dy, float* dweights, int64_t n, int64_t R, int64_t H, int k, cudaStream_t s) {
  if (dtype == 0) return combine_bwd_t<float>(dout, y, pos, weights, dy, dweights, n, R, H, k, s);
  if (dtype == 1) return combine_bwd_t<__half>(dout, y, pos, weights, dy, dweights, n, R, H, k, s);
  return combine_bwd_t<__nv_bfloat16>(dout, y, pos, weights, dy, dweights, n, R, H, k, s);
}

}  // namespace tq
