// tq_lora.cu -- low-rank adapters beside the packed projections (include/tq_lora.h): the kernels that take any
// shape and alignment, and dropout.
//
// Forward and backward are four forms of three sums, over the rows m(r) of the sorted positions r of each adapter l:
//   reduce   V[r, j]   = f sum_c P[m, c] W_l(c, j)               v: P = drop(x), W = A;  dv: P = dy, W = B
//   expand   O[m, c]   = base[m, c] + f sum_j V[r, j] W_l(c, j)  out: V = v, W = B;      dx: V = dv, W = A, the sum dropped
//   wgrad    G_l(c, j) = f sum_r P[m, c] V[r, j]                 dA: P = drop(x), V = dv;  dB: P = dy, V = v
//
// with W(c, j) stored as A [rank, C] (column c of row j) or as B [C, rank].  The factors that do not depend on the
// summation index (scaling, 1 / (1 - p)) are applied to the fp32 sum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "tq_common.cuh"

namespace tq {

constexpr int kLoraMaxRank = 128;

// Dropout of a [rows, width] matrix.  thr = 0: nothing is dropped and rng is not read.
struct DropArgs {
  const int64_t* rng;  // seed, offset
  uint32_t thr;        // 16-bit numbers below it are dropped
  float scale;         // 65536 / (65536 - thr)
};

// One of the sums above.  wc, wj: strides of W_l(c, j) (or of G_l), ws: stride between adapters.
struct LoraArgs {
  const void* P;
  const void* W;
  const void* base;         // expand: may be null
  void* O;                  // expand: O; wgrad: G
  float* V;                 // reduce: written, else read
  const float* scaling;     // [L] or null
  const int32_t* offsets;   // [L + 1]
  const int32_t* order;     // [M] or null
  DropArgs drop;            // of P (reduce, wgrad) or of the sum (expand)
  int64_t M, C;
  int64_t wc, wj, ws;
  int L, rank;
  bool use_scaling;         // f includes scaling[l]
  // tensor-core kernels: rows of P, of W and of base and O in whole, aligned 16-byte vectors (element by element
  // otherwise); wgrad: O aligned to them
  bool pvec, wvec, yvec;
  // Tensor-core reduce: the largest finite magnitude that each CTA of a tile wrote to V (most) and found in V2 (most2),
  // kLoraMostPer slots per tile; null: not wanted
  const float* V2;
  float* most;
  float* most2;
  bool behind;  // tensor-core wgrad: the preceding kernels on the stream are this call's own
  // Tensor-core wgrad: V as hi and lo [M, 2 padded rank], scaled by 1 / inv[l]
  const void* Q;
  const float* inv;
};

constexpr int kLoraMostPer = 8;

// ---------------------------------------------------------------------------------------------
// Philox4x32-10: ten rounds of two 32 x 32 -> 64 bit products, the key advanced by two odd constants
// (Salmon, Moraes, Dror, Shaw, SC 2011).  128 bits per call serve eight elements with 16 bits each: with 32 bits per
// element the integer units, not memory, would bound a kernel that drops as it reads.
// ---------------------------------------------------------------------------------------------
struct PhiloxKey {
  uint32_t k0, k1, o0, o1;
};

__device__ __forceinline__ PhiloxKey philox_key(const DropArgs& d) {
  PhiloxKey k = {0u, 0u, 0u, 0u};
  if (d.thr) {
    const uint64_t seed = static_cast<uint64_t>(d.rng[0]), off = static_cast<uint64_t>(d.rng[1]);
    k.k0 = static_cast<uint32_t>(seed);
    k.k1 = static_cast<uint32_t>(seed >> 32);
    k.o0 = static_cast<uint32_t>(off);
    k.o1 = static_cast<uint32_t>(off >> 32);
  }
  return k;
}

__device__ __forceinline__ uint4 philox(uint64_t group, const PhiloxKey& key) {
  uint32_t c0 = static_cast<uint32_t>(group), c1 = static_cast<uint32_t>(group >> 32), c2 = key.o0, c3 = key.o1;
  uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u, p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(p1);
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Whether element e of the group is kept.
__device__ __forceinline__ bool drop_keeps(const uint4& w, int e, uint32_t thr) {
  const uint32_t word = (e >> 1) == 0 ? w.x : ((e >> 1) == 1 ? w.y : ((e >> 1) == 2 ? w.z : w.w));
  return ((e & 1) ? word : word << 16) >= thr << 16;  // thr <= 65535
}

// Eight 16-bit elements of a group with the dropped ones zero.  (Comparing whole words decides the high halves,
// shifted ones the low halves: 32 cycles of a warp beside the generator's 115; the packed 16-bit comparison takes 45.)
__device__ __forceinline__ uint32_t drop_word16(uint32_t x, uint32_t bits, uint32_t thr) {
  const uint32_t t = thr << 16;
  if (bits < t) x &= 0x0000FFFFu;
  if ((bits << 16) < t) x &= 0xFFFF0000u;
  return x;
}
__device__ __forceinline__ uint4 drop_apply16(const uint4& x, uint64_t group, const PhiloxKey& key, uint32_t thr) {
  const uint4 w = philox(group, key);
  return make_uint4(drop_word16(x.x, w.x, thr), drop_word16(x.y, w.y, thr), drop_word16(x.z, w.z, thr),
                    drop_word16(x.w, w.w, thr));
}

// The adapter of sorted position r, or -1: the last l with offsets[l] <= r, where r < offsets[l + 1].
__device__ __forceinline__ int adapter_of(const int32_t* offsets, int L, int64_t r) {
  int lo = -1, hi = L + 1;  // offsets[lo] <= r < offsets[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo < L ? lo : -1;
}

// The row at sorted position r, or -1.
__device__ __forceinline__ int64_t lora_row(const LoraArgs& a, int64_t r) {
  const int64_t m = a.order ? static_cast<int64_t>(a.order[r]) : r;
  return m >= 0 && m < a.M ? m : -1;
}

__device__ __forceinline__ float lora_factor(const LoraArgs& a, int l) {
  const float f = a.drop.thr ? a.drop.scale : 1.0f;
  return a.use_scaling && a.scaling ? f * a.scaling[l] : f;
}

// ---------------------------------------------------------------------------------------------
// Any shape and alignment (CUDA cores, element by element)
// ---------------------------------------------------------------------------------------------
constexpr int kLoraGenThreads = 256;
constexpr int kLoraGenJ = 4;  // inner columns per warp of the reduction

// A warp per (position, four inner columns); a lane takes groups of eight columns c.
template <typename T>
__global__ void __launch_bounds__(kLoraGenThreads) lora_generic_reduce_kernel(const LoraArgs a) {
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31;
  const int nj = (a.rank + kLoraGenJ - 1) / kLoraGenJ;
  const int64_t groups = (a.C + 7) >> 3;
  const PhiloxKey key = philox_key(a.drop);
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kLoraGenThreads / 32) + (threadIdx.x >> 5); w < a.M * nj;
       w += static_cast<int64_t>(gridDim.x) * (kLoraGenThreads / 32)) {
    const int64_t r = w / nj;
    const int j0 = static_cast<int>(w - r * nj) * kLoraGenJ;
    const int l = adapter_of(a.offsets, a.L, r);
    if (l < 0) continue;
    const int64_t m = lora_row(a, r);
    const T* W = static_cast<const T*>(a.W) + l * a.ws;
    float acc[kLoraGenJ] = {};
    for (int64_t g = lane; m >= 0 && g < groups; g += 32) {
      const T* p = static_cast<const T*>(a.P) + m * a.C + 8 * g;
      const uint4 bits = a.drop.thr ? philox(m * groups + g, key) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t c = 8 * g + e;
        if (c >= a.C) break;
        if (a.drop.thr && !drop_keeps(bits, e, a.drop.thr)) continue;
        const float v = to_f32(p[e]);
#pragma unroll
        for (int i = 0; i < kLoraGenJ; ++i)
          if (j0 + i < a.rank) acc[i] = fmaf(v, to_f32(W[c * a.wc + (j0 + i) * a.wj]), acc[i]);
      }
    }
    const float f = lora_factor(a, l);
#pragma unroll
    for (int i = 0; i < kLoraGenJ; ++i) {
      const float s = warp_sum(acc[i]);
      if (lane == 0 && j0 + i < a.rank) a.V[r * a.rank + j0 + i] = f * s;
    }
  }
}

// A CTA per position; a thread takes groups of eight columns.
template <typename T>
__global__ void __launch_bounds__(kLoraGenThreads) lora_generic_expand_kernel(const LoraArgs a) {
  __shared__ float vs[kLoraMaxRank];
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int64_t groups = (a.C + 7) >> 3;
  const PhiloxKey key = philox_key(a.drop);
  for (int64_t r = blockIdx.x; r < a.M; r += gridDim.x) {
    const int64_t m = lora_row(a, r);
    if (m < 0) continue;
    const int l = adapter_of(a.offsets, a.L, r);
    __syncthreads();
    if (l >= 0 && threadIdx.x < a.rank) vs[threadIdx.x] = a.V[r * a.rank + threadIdx.x];
    __syncthreads();
    const T* base = a.base ? static_cast<const T*>(a.base) + m * a.C : nullptr;
    T* out = static_cast<T*>(a.O) + m * a.C;
    const T* W = static_cast<const T*>(a.W) + (l >= 0 ? l * a.ws : 0);
    const float f = l >= 0 ? lora_factor(a, l) : 0.0f;
    for (int64_t g = threadIdx.x; g < groups; g += kLoraGenThreads) {
      const uint4 bits = a.drop.thr ? philox(m * groups + g, key) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t c = 8 * g + e;
        if (c >= a.C) break;
        float s = 0.0f;
        const bool kept = l >= 0 && !(a.drop.thr && !drop_keeps(bits, e, a.drop.thr));
        if (kept)
          for (int j = 0; j < a.rank; ++j) s = fmaf(vs[j], to_f32(W[c * a.wc + j * a.wj]), s);
        const float b = base ? to_f32(base[c]) : 0.0f;
        out[c] = from_f32<T>(kept ? fmaf(f, s, b) : b);
      }
    }
  }
}

// A thread per (group of eight columns, eight inner columns) of an adapter: it walks the adapter's rows.
template <typename T>
__global__ void __launch_bounds__(128) lora_generic_wgrad_kernel(const LoraArgs a) {
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int64_t groups = (a.C + 7) >> 3;
  const int64_t g = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
  if (g >= groups) return;
  const int j0 = blockIdx.y * 8, l = blockIdx.z;
  const int64_t r0 = max(a.offsets[l], 0), r1 = min(static_cast<int64_t>(a.offsets[l + 1]), a.M);
  const PhiloxKey key = philox_key(a.drop);
  float acc[8][8] = {};
  for (int64_t r = r0; r < r1; ++r) {
    const int64_t m = lora_row(a, r);
    if (m < 0) continue;
    const T* p = static_cast<const T*>(a.P) + m * a.C + 8 * g;
    const uint4 bits = a.drop.thr ? philox(m * groups + g, key) : make_uint4(0u, 0u, 0u, 0u);
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = j0 + i < a.rank ? a.V[r * a.rank + j0 + i] : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (8 * g + e >= a.C || (a.drop.thr && !drop_keeps(bits, e, a.drop.thr))) continue;
      const float v = to_f32(p[e]);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[e][i] = fmaf(v, q[i], acc[e][i]);
    }
  }
  const float f = lora_factor(a, l);
  T* out = static_cast<T*>(a.O) + l * a.ws;
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * g + e < a.C && j0 + i < a.rank) out[(8 * g + e) * a.wc + (j0 + i) * a.wj] = from_f32<T>(f * acc[e][i]);
}

// fn(T()) for the dtype of a call (bf16 or fp16).
template <typename F>
static cudaError_t with_type16(bool bf16, F fn) {
  return bf16 ? fn(__nv_bfloat16()) : fn(__half());
}

static unsigned lora_grid(int64_t tasks, int per_sm) {
  const int64_t most = static_cast<int64_t>(current_device_info().num_sms) * per_sm;
  return static_cast<unsigned>(tasks < 1 ? 1 : (tasks < most ? tasks : most));
}

static cudaError_t lora_generic_reduce(bool bf16, const LoraArgs& a, cudaStream_t s) {
  const int64_t warps = a.M * ((a.rank + kLoraGenJ - 1) / kLoraGenJ);
  return with_type16(bf16, [&](auto t) {
    return launch_pdl(lora_generic_reduce_kernel<decltype(t)>, dim3(lora_grid((warps + 7) / 8, 16)),
                      dim3(kLoraGenThreads), 0, 1, s, a);
  });
}

static cudaError_t lora_generic_expand(bool bf16, const LoraArgs& a, cudaStream_t s) {
  return with_type16(bf16, [&](auto t) {
    return launch_pdl(lora_generic_expand_kernel<decltype(t)>, dim3(lora_grid(a.M, 16)), dim3(kLoraGenThreads), 0, 1, s,
                      a);
  });
}

static cudaError_t lora_generic_wgrad(bool bf16, const LoraArgs& a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((((a.C + 7) >> 3) + 127) / 128), static_cast<unsigned>((a.rank + 7) / 8),
                  static_cast<unsigned>(a.L));
  return with_type16(bf16, [&](auto t) {
    return launch_pdl(lora_generic_wgrad_kernel<decltype(t)>, grid, dim3(128), 0, 1, s, a);
  });
}

// ---------------------------------------------------------------------------------------------
// Dropout
// ---------------------------------------------------------------------------------------------
constexpr int kDropThreads = 256;

// Whole, aligned groups: a thread per group of eight columns.  16384 x 4096 in bf16: 48 us, 0.85 of the copy rate;
// with two groups per thread in flight 54.
template <typename T>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const T* x, T* out, const DropArgs d, int64_t total) {
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const PhiloxKey key = philox_key(d);
  const float f = d.thr ? d.scale : 1.0f;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kDropThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kDropThreads) {
    constexpr int kW = 16 / sizeof(T);  // elements per 16 bytes
    Vec<T, kW> v[8 / kW];
#pragma unroll
    for (int q = 0; q < 8 / kW; ++q) v[q] = reinterpret_cast<const Vec<T, kW>*>(x)[i * (8 / kW) + q];
    const uint4 bits = d.thr ? philox(i, key) : make_uint4(~0u, ~0u, ~0u, ~0u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      T& t = v[e / kW].v[e % kW];
      t = from_f32<T>(drop_keeps(bits, e, d.thr) ? f * to_f32(t) : 0.0f);
    }
#pragma unroll
    for (int q = 0; q < 8 / kW; ++q) reinterpret_cast<Vec<T, kW>*>(out)[i * (8 / kW) + q] = v[q];
  }
}

// Any width and alignment: a warp per 256 columns of a row.  Each lane draws for one group, and the elements are
// taken in the order of memory, their truth values from the lane that drew them.
template <typename T>
__global__ void __launch_bounds__(kDropThreads)
    dropout_any_kernel(const T* x, T* out, const DropArgs d, int64_t M, int64_t K) {
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31;
  const int64_t groups = (K + 7) >> 3, segments = (K + 255) >> 8, total = M * segments;
  const PhiloxKey key = philox_key(d);
  const float f = d.thr ? d.scale : 1.0f;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kDropThreads + threadIdx.x) >> 5; i < total;
       i += (static_cast<int64_t>(gridDim.x) * kDropThreads) >> 5) {
    const int64_t m = i / segments, c0 = (i - m * segments) << 8;
    const T* src = x + m * K + c0;
    T v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c0 + 32 * e + lane < K) v[e] = src[32 * e + lane];
    uint32_t kept = 0xFFu;
    if (d.thr) {
      const uint4 bits = philox(m * groups + (c0 >> 3) + lane, key);
      kept = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) kept |= drop_keeps(bits, e, d.thr) ? 1u << e : 0u;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t k = __shfl_sync(0xFFFFFFFFu, kept, 4 * e + (lane >> 3));
      if (c0 + 32 * e + lane < K)
        out[m * K + c0 + 32 * e + lane] = from_f32<T>((k >> (lane & 7)) & 1u ? f * to_f32(v[e]) : 0.0f);
    }
  }
}

cudaError_t launch_dropout(const void* x, int dtype, void* out, const DropArgs& d, int64_t M, int64_t K,
                           cudaStream_t s) {
  const int64_t groups = M * ((K + 7) >> 3);
  const bool vec = K % 8 == 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
  const dim3 grid(lora_grid((groups + kDropThreads - 1) / kDropThreads, 32));
  auto run = [&](auto t) {
    using T = decltype(t);
    const T* xt = static_cast<const T*>(x);
    T* ot = static_cast<T*>(out);
    if (vec) return launch_pdl(dropout_kernel<T>, grid, dim3(kDropThreads), 0, 1, s, xt, ot, d, groups);
    return launch_pdl(dropout_any_kernel<T>, grid, dim3(kDropThreads), 0, 1, s, xt, ot, d, M, K);
  };
  return dtype == 0 ? run(float()) : (dtype == 1 ? run(__half()) : run(__nv_bfloat16()));
}

}  // namespace tq
