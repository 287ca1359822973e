// tq_lora_fast.cu -- low-rank adapters (include/tq_lora.h): the sums over many rows (reduce, wgrad and expand on
// tcgen05, with 16-byte accesses where rows are made of whole vectors and element by element otherwise) and the
// single launch for few rows.
//
// Work is cut by adapter: a tile is up to 128 sorted positions of one adapter, found on the device from
// the offsets, so that one captured graph serves any plan.
//
// v and dv are fp32.  As operands of a 16-bit product they are split, v s = hi + lo with hi = round(v s), lo =
// round(v s - hi) and s a power of two (fp16 only: bf16 has the exponents of fp32), which keeps them to 2^-22 (fp16) or
// 2^-16 (bf16) of each; hi and lo enter the same fp32 sum, and 1 / s is applied to it, exactly.  s is a row's own in
// expand and in the kernel for few rows.  In wgrad, which sums over rows, it is an adapter's: the last half
// step of lo is 2^-25 beside a largest number of 2^14 or more, so that up to 2^-39 of that one is left out.  A third
// part would keep 24 bits of bf16 too and cost half as many products again; the outputs' own rounding is far above.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "tq_common.cuh"

namespace tq {

constexpr int kLoraTile = 128;  // positions per tile

// ---------------------------------------------------------------------------------------------
// Types
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1, __half) {
  mma_16816(d, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1, __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// cp_async_16 to a shared-memory address.
__device__ __forceinline__ void cp_async_16s(uint32_t smem_dst, const void* gmem_src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_dst), "l"(gmem_src), "r"(src_bytes)
               : "memory");
}

// A bounded wait by a whole warp, with one result for all its lanes: lanes that each went by a result of their own could
// part before an instruction that takes the whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity)) != 0;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(T a, T b) {
  Vec<T, 2> v;
  v.v[0] = a;
  v.v[1] = b;
  return *reinterpret_cast<uint32_t*>(&v);
}

// Two fp32 numbers, already scaled, as hi and lo pairs.  What is not finite has no lo part (infinity less itself is
// NaN).
template <typename T>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const T ha = from_f32<T>(a), hb = from_f32<T>(b);
  float la = a - to_f32(ha), lb = b - to_f32(hb);
  if (!(fabsf(a) <= 3.0e38f)) la = 0.0f;
  if (!(fabsf(b) <= 3.0e38f)) lb = 0.0f;
  hi = pack2<T>(ha, hb);
  lo = pack2<T>(from_f32<T>(la), from_f32<T>(lb));
}

// The power of two that brings `most` to [2^14, 2^15) (fp16), so that the largest value fits and the smallest ones
// keep their bits; 1 for bf16, for zero and for what is not finite.  inv: its inverse.
template <typename T>
__device__ __forceinline__ float split_scale(float most, float& inv) {
  inv = 1.0f;
  if (!std::is_same<T, __half>::value || !(most > 0.0f) || !(most <= 3.0e38f)) return 1.0f;
  int e = 14 - (static_cast<int>(__float_as_uint(most) >> 23) - 127);
  e = e > 126 ? 126 : e;
  inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// The magnitude of a number that is finite, else zero: what an adapter's power of two is made from, since an infinity in
// one inner column must not leave the other columns without one.
__device__ __forceinline__ float finite_abs(float x) { return fabsf(x) <= 3.402823466e38f ? fabsf(x) : 0.0f; }

// Eight consecutive 16-bit elements of which `left` are there (zero past them), one by one; out of line, since what
// runs beside it is slower for the code.
__device__ __noinline__ uint4 load8_any(const uint16_t* p, int64_t left) {
  uint16_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = e < left ? p[e] : static_cast<uint16_t>(0);
  return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
}

// Eight consecutive 16-bit elements of a row of `width` from column c (zero past it); vec: whole and aligned.
__device__ __forceinline__ uint4 load8(const void* row, int64_t c, int64_t width, bool vec) {
  const uint16_t* p = static_cast<const uint16_t*>(row) + c;
  if (c >= width) return make_uint4(0u, 0u, 0u, 0u);
  if (vec) return *reinterpret_cast<const uint4*>(p);
  return load8_any(p, width - c);
}

// ---------------------------------------------------------------------------------------------
// Tiles.  Tile t of a plan: the tiles of adapter 0, of adapter 1, ..., then those of the positions of no adapter (l =
// -1), which are counted on from the ones before offsets[0] to the ones from offsets[L] on.  Run by a whole warp, all
// of whose lanes get the result.  A plan has at most lora_max_tiles(); kTile positions each.
// ---------------------------------------------------------------------------------------------
struct LoraTile {
  int l;        // adapter, -1: none, -2: past the last tile
  int cnt;      // positions
  int64_t pos;  // the first one (l = -1: its number among those of no adapter)
  int first;    // the adapter's first tile
};

__device__ __forceinline__ int64_t clamp_pos(int64_t o, int64_t M) { return o < 0 ? 0 : (o < M ? o : M); }

template <int kTile = kLoraTile>
__device__ __forceinline__ LoraTile lora_tile(const int32_t* offsets, int L, int64_t M, int t) {
  const int lane = threadIdx.x & 31;
  LoraTile r = {-2, 0, 0, 0};
  int done = 0;  // tiles of the adapters seen
  for (int l0 = 0; l0 < L; l0 += 128) {  // four adapters per lane
    int64_t o[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const int l = l0 + 4 * lane + i;
      o[i] = clamp_pos(offsets[l < L ? l : L], M);
    }
    int n[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      n[i] = o[i + 1] > o[i] ? static_cast<int>((o[i + 1] - o[i] + kTile - 1) / kTile) : 0;
      sum += n[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += up;
    }
    const int total = __shfl_sync(0xFFFFFFFFu, incl, 31);
    if (t < done + total) {
      int before = done + incl - sum;
      const bool mine = t >= before && t < before + sum;
      LoraTile f = {-2, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (mine && t >= before && t < before + n[i]) {
          f.l = l0 + 4 * lane + i;
          f.first = before;
          f.pos = o[i] + static_cast<int64_t>(t - before) * kTile;
          f.cnt = static_cast<int>(o[i + 1] - f.pos < kTile ? o[i + 1] - f.pos : kTile);
        }
        before += n[i];
      }
      const int src = __ffs(__ballot_sync(0xFFFFFFFFu, mine)) - 1;
      r.l = __shfl_sync(0xFFFFFFFFu, f.l, src);
      r.cnt = __shfl_sync(0xFFFFFFFFu, f.cnt, src);
      r.pos = __shfl_sync(0xFFFFFFFFu, f.pos, src);
      r.first = __shfl_sync(0xFFFFFFFFu, f.first, src);
      return r;
    }
    done += total;
  }
  const int64_t head = clamp_pos(offsets[0], M), tail = M - clamp_pos(offsets[L], M);
  r.pos = static_cast<int64_t>(t - done) * kTile;
  if (r.pos < head + tail) {
    r.l = -1;
    r.first = done;
    r.cnt = static_cast<int>(head + tail - r.pos < kTile ? head + tail - r.pos : kTile);
  }
  return r;
}

// The number of tiles of a plan; run by a whole warp.
__device__ __forceinline__ int64_t lora_tiles(const int32_t* offsets, int L, int64_t M) {
  int64_t sum = 0;
  for (int l = threadIdx.x & 31; l < L; l += 32) {
    const int64_t n = clamp_pos(offsets[l + 1], M) - clamp_pos(offsets[l], M);
    sum += n > 0 ? (n + kLoraTile - 1) / kLoraTile : 0;
  }
  const int64_t none = clamp_pos(offsets[0], M) + M - clamp_pos(offsets[L], M);
  return warp_sum(sum) + (none + kLoraTile - 1) / kLoraTile;
}

static int64_t lora_max_tiles(int64_t M, int64_t L, int tile = kLoraTile) {
  const int64_t t = M / tile + L + 1;
  return t < M ? t : M;
}

// Tiles to expect of a plan of M rows and L adapters: each adapter that has rows ends in a part-filled one.
static int64_t lora_likely_tiles(int64_t M, int64_t L) {
  return L > 1 ? M / kLoraTile + (L < M ? L : M) : (M + kLoraTile - 1) / kLoraTile;
}

// The smallest padded rank of 16, 32, 64 or 128 (a multiple of an MMA's 16 k).
template <typename F>
static cudaError_t with_rank(int rank, F fn) {
  if (rank <= 16) return fn(std::integral_constant<int, 16>());
  if (rank <= 32) return fn(std::integral_constant<int, 32>());
  if (rank <= 64) return fn(std::integral_constant<int, 64>());
  return fn(std::integral_constant<int, 128>());
}

// ---------------------------------------------------------------------------------------------
// reduce and wgrad on tcgen05: D (128 x up to 256 fp32, tensor memory) += A B^T over stages in shared memory.
//   reduce  D[position, j]  A: the tile's rows of P, 128 x 128 columns (K-major; 64 columns for ranks above 64)
//                           B: W, as A [rank, C] those columns of each j (K-major), as B [C, rank] those rows (MN)
//   wgrad   D[c, j]         A: 64 rows x 128 columns of P (MN-major)
//                           B: 64 rows of V, hi and lo side by side (MN-major); their sums are added at the end
// Both read P once and little else, so HBM bounds them (2 rank FLOPs per element of P leave the tensor pipe idle most
// of the time).  P is fetched row by row through `order` with 16-byte cp.async (a row's 128 or 256 bytes are
// consecutive lanes), which zero-fills too and needs no tensor map, by sixteen loader warps: with eight, or with
// three times the instructions per stage, the latency of a warp's own instructions set the pace, not memory.  With
// dropout each thread masks what it copied before it hands the stage on.
// The summation (columns, rows) is split over a cluster of S CTAs while tiles leave SMs idle; partial sums go through
// distributed shared memory and are added in rank order.
// One CTA per SM (its shared memory keeps every other kernel with tensor memory out), so that none waits for tensor
// memory that a CTA holds which itself waits for a cluster.
// 8192 rows, rank 64, each kernel alone and cold: reduce of 8192 columns 34 us and of 2048 17 (6.1 TB/s between them,
// 12 us of start and end; with dropout 2.3 times that slope: Philox), dv of 4096 23, wgrad of 4096 30, with dropout 44.
// ---------------------------------------------------------------------------------------------
constexpr int kLtcWarps = 16;  // loaders
constexpr int kLtcLoaders = 32 * kLtcWarps;
constexpr int kLtcThreads = kLtcLoaders + 32;
constexpr int kLtcEpiWarps = 8;  // of the loaders, read the sums
enum { kReduceA = 0, kReduceB = 1, kWgrad = 2 };

constexpr int kRowStages = 16;    // wgrad: stages whose rows are fetched together (two such sets are kept)

template <int kMode, int RP>
struct LoraTcLayout {
  static constexpr bool kW = kMode == kWgrad;
  static constexpr int kN = kW ? 2 * RP : RP;                               // MMA columns
  static constexpr int kSub = kW || RP > 64 ? 1 : 2;                        // reduce: planes of 64 columns per stage
  static constexpr int kTileP = kW ? 16384 : kSub * 16384;
  static constexpr int kPlaneW = kMode == kReduceA ? RP * 128 : (kW ? 64 : 64 * kSub) * 128;
  static constexpr int kTileW = kMode == kReduceA ? kSub * kPlaneW : (kN + 63) / 64 * kPlaneW;
  static constexpr int kStage = kTileP + kTileW;
  static constexpr int kRing = 200 * 1024 / kStage < 8 ? 200 * 1024 / kStage : 8;
  static constexpr int kLag = kRing - 2;                                    // stages between request and hand-over
  static constexpr int kChunks = kW ? 16 : 8 * kSub;                        // 16-byte chunks of a row of P per stage
  static constexpr int kStep = kLtcLoaders / kChunks;                       // rows between a thread's chunks
  static constexpr int kPer = (kW ? 64 : 128) / kStep;                      // chunks of P per thread
  static constexpr int kChunksW = kW ? 16 * RP : RP * 8 * kSub;             // chunks of the B operand per stage
  static constexpr int kPerW = (kChunksW + kLtcLoaders - 1) / kLtcLoaders;
  static constexpr int kOffBar = kRing * kStage;                            // full[R], empty[R], accFull, TMEM slot
  static constexpr int kOffRow = kOffBar + (2 * kRing + 2) * 8;
  static constexpr int kOffMost = kOffRow + (kW ? 2 * kRowStages * 64 : 128) * 4;
  static constexpr int kAlloc = kOffMost + 128 + 1024;
  static constexpr uint32_t kTmemCols = kN <= 32 ? 32u : (kN <= 64 ? 64u : (kN <= 128 ? 128u : 256u));
  static_assert(kRing >= 4 && kAlloc > 116 * 1024 && kAlloc <= 227 * 1024, "one CTA per SM");
  static_assert(128 * (RP + 8) * 4 <= kRing * kStage, "partial sums fit");
};

// Shared-memory descriptor of an MN-major operand, 128-byte swizzle: planes of 64 elements along M / N, `plane` bytes
// apart (leading byte offset), each of 128-byte rows of one k, groups of eight rows 1024 bytes apart (stride byte
// offset).
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t smem_addr, uint32_t plane) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(plane >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// The sums of one launch: one, or both weight gradients (the same plan and rank), whose tiles of columns follow each
// other.
struct LoraSums {
  LoraArgs a[2];
  int first;  // wgrad: tiles of columns of a[0]
};

// kVec: all rows in whole, aligned vectors; without it kDrop is decided at run time where it is set.
template <typename T, int kMode, int RP, bool kDrop, bool kVec>
__global__ void __launch_bounds__(kLtcThreads, 1)
lora_tc_kernel(const __grid_constant__ LoraSums sums_of, const int S) {
  using L = LoraTcLayout<kMode, RP>;
  constexpr bool kW = kMode == kWgrad;
  const bool second = kW && static_cast<int>(blockIdx.x) >= sums_of.first;
  const LoraArgs& a = sums_of.a[second ? 1 : 0];
  const bool pvec = kVec || a.pvec, wvec = kVec || a.wvec, yvec = kVec || a.yvec;
  const bool drop = kDrop && (kVec || a.drop.thr != 0);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kOffBar);
  uint64_t* empty = full + L::kRing;
  uint64_t* accFull = empty + L::kRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accFull + 1);
  int* rowbuf = reinterpret_cast<int*>(sm + L::kOffRow);  // reduce: the tile's rows; wgrad: those of two sets of stages
  float* mostbuf = reinterpret_cast<float*>(sm + L::kOffMost);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(blockIdx.z);
  // wgrad follows kernels of the same call, which let it start only after the work before the call had finished: all
  // but Q and inv may be read before the wait.
  if (!kW || !a.behind) pdl_wait_prior_grids();

  // the work of this cluster: positions [pos0, pos0 + cnt) of adapter l; columns from c0 (wgrad); stages [s0, s0 + ns)
  int l, ns_all;
  int64_t pos0, cnt, c0 = 0;
  if (!kW) {
    const LoraTile t = lora_tile(a.offsets, a.L, a.M, blockIdx.x);
    if (t.l < 0) return;  // the whole cluster
    l = t.l;
    pos0 = t.pos;
    cnt = t.cnt;
    ns_all = static_cast<int>((a.C + 64 * L::kSub - 1) / (64 * L::kSub));
  } else {
    l = static_cast<int>(blockIdx.y);
    pos0 = clamp_pos(a.offsets[l], a.M);
    cnt = clamp_pos(a.offsets[l + 1], a.M) - pos0;
    c0 = (static_cast<int64_t>(blockIdx.x) - (second ? sums_of.first : 0)) * 128;
    if (cnt <= 0) {  // no rows: zeros (the whole cluster returns)
      T* out = static_cast<T*>(a.O) + l * a.ws;
      if (rank == 0)
        for (int i = tid; i < 128 * a.rank; i += kLtcThreads) {
          const int64_t c = c0 + (a.wc == 1 ? i & 127 : i / a.rank);
          const int j = a.wc == 1 ? i >> 7 : i % a.rank;
          if (c < a.C) out[c * a.wc + j * a.wj] = from_f32<T>(0.0f);
        }
      if (a.behind) pdl_wait_prior_grids();
      return;
    }
    ns_all = static_cast<int>((cnt + 63) / 64);
  }
  const int s0 = static_cast<int>(static_cast<int64_t>(rank) * ns_all / S);
  const int ns = static_cast<int>(static_cast<int64_t>(rank + 1) * ns_all / S) - s0;  // may be 0

  if (tid == 0) {
    for (int i = 0; i < L::kRing; ++i) {
      mbar_init(&full[i], kLtcWarps);
      mbar_init(&empty[i], 1);
    }
    mbar_init(accFull, 1);
    fence_mbar_init();
  }
  if (warp == kLtcWarps) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  if (!kW && tid < 128) rowbuf[tid] = tid < cnt ? static_cast<int>(lora_row(a, pos0 + tid)) : -1;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  pdl_allow_dependents();
  const uint32_t tmem = *tmem_slot;
  const PhiloxKey key = kDrop ? philox_key(a.drop) : PhiloxKey{0u, 0u, 0u, 0u};
  const int64_t groups = (a.C + 7) >> 3;
  const uint16_t* P = static_cast<const uint16_t*>(a.P);
  float f = lora_factor(a, l);

  // A wait that runs out is recorded, and whoever waited goes on with what there is, waits no more and comes to every
  // barrier like the others: one that left the loop would leave them at a barrier for good, and lanes that went by
  // results of their own would part before an instruction that takes the whole warp.
  bool ok = !(warp == kLtcWarps && skip_x_loads());  // failure-path test hook (no MMA is issued), else true
  if (warp < kLtcWarps) {
    // ------------------------------------------------------------------ loaders
    const int prow = tid / L::kChunks, pch = tid % L::kChunks;  // chunk pch of rows prow + kStep k, k < kPer
    const uint32_t pdst = (pch >> 3) * (kW ? 8192 : 16384) + prow * 128 + (((pch & 7) ^ (prow & 7)) << 4);
    const uint32_t ring0 = smem_u32(sm), ring1 = ring0 + L::kRing * L::kStage;
    int64_t c = kW ? c0 + 8 * pch : static_cast<int64_t>(s0) * 64 * L::kSub + 8 * pch;  // this thread's column
    // reduce: each chunk's address in the first stage (nothing is copied for a position without a row: its sums are
    // not used, and no other sum reads what the stage holds for it)
    const uint16_t* src[kW ? 1 : L::kPer];
    int m[L::kPer];
    if (!kW) {
#pragma unroll
      for (int k = 0; k < L::kPer; ++k) {
        m[k] = rowbuf[prow + L::kStep * k];
        src[k] = P + (m[k] >= 0 ? static_cast<int64_t>(m[k]) * a.C : 0) + c;
      }
    }
    // wgrad: the rows (-1: none) of kRowStages stages at a time, the next set's in registers half a set ahead
    const bool pin = c < a.C;
    const uint16_t* pcol = P + (pin ? c : 0);
    const uint32_t psize = pin ? 16u : 0u;
    constexpr int kRowPer = kRowStages * 64 / kLtcLoaders;
    int rnext[kRowPer];
    auto fetch_rows = [&](int i) {  // of the set that begins with stage i
#pragma unroll
      for (int k = 0; k < kRowPer; ++k) {
        const int64_t r = static_cast<int64_t>(s0 + i) * 64 + tid + kLtcLoaders * k;
        rnext[k] = r < cnt ? static_cast<int>(lora_row(a, pos0 + r)) : -1;
      }
    };
    if (kW && ns > 0) fetch_rows(0);
    // the B operand: chunks tid + 512 k of the stage
    const uint16_t* wsrc[L::kPerW];
    uint32_t wdst[L::kPerW], wsize[L::kPerW];
    int wrow[L::kPerW];  // summation index within the stage, for the zeros past its end
#pragma unroll
    for (int k = 0; k < L::kPerW; ++k) {
      const int q = tid + kLtcLoaders * k;
      const bool mine = q < L::kChunksW;
      int row, ch;
      if (kMode == kReduceA) {  // row: j; 8 kSub chunks of its columns
        row = q / (8 * L::kSub);
        ch = q % (8 * L::kSub);
        wsize[k] = mine && row < a.rank ? 16u : 0u;
        wrow[k] = 8 * ch;
        wsrc[k] = static_cast<const uint16_t*>(a.W) + l * a.ws + (wsize[k] ? row * a.C : 0) +
                  static_cast<int64_t>(s0) * 64 * L::kSub + 8 * ch;
      } else {                  // row: summation index; RP / 8 (wgrad: RP / 4, hi and lo) chunks
        constexpr int kRowChunks = kW ? RP / 4 : RP / 8;
        row = q / kRowChunks;
        ch = q % kRowChunks;
        wsize[k] = mine && (kW || 8 * ch < a.rank) ? 16u : 0u;
        wrow[k] = row;
        wsrc[k] = kW ? static_cast<const uint16_t*>(a.Q) +
                           (pos0 + static_cast<int64_t>(s0) * 64 + row) * (2 * RP) + 8 * ch
                     : static_cast<const uint16_t*>(a.W) + l * a.ws +
                           (static_cast<int64_t>(s0) * 64 * L::kSub + row) * a.rank + 8 * ch;
      }
      wdst[k] = L::kTileP + (ch >> 3) * L::kPlaneW + row * 128 + (((ch & 7) ^ (row & 7)) << 4);
    }
    // what a copy of zeros names: the start of the operand itself, since an address must be a multiple of 16 bytes
    // whatever is read there, and P has only its type's alignment where pvec is false
    const uint16_t* const wzero = static_cast<const uint16_t*>(kW ? a.Q : a.W);
    const int64_t wadvance = kMode == kReduceA ? 64 * L::kSub : (kW ? 64 * 2 * RP : 64 * L::kSub * a.rank);
    // summation indexes left from the current stage on (columns or positions)
    int64_t left = kW ? cnt - static_cast<int64_t>(s0) * 64 : a.C - static_cast<int64_t>(s0) * 64 * L::kSub;
    // One stage; kTail: some of its summation indexes are past the end, and zeros.
    auto request = [&](auto tail, int i, uint32_t st) {
      constexpr bool kTail = decltype(tail)::value;
      if (kW) {
        const int* rows = rowbuf + (i % (2 * kRowStages)) * 64 + prow;
#pragma unroll
        for (int k = 0; k < L::kPer; ++k) {
          const int mk = rows[L::kStep * k];
          const uint32_t dst = st + pdst + k * L::kStep * 128;
          if (pvec)
            cp_async_16s(dst, pcol + static_cast<int64_t>(mk < 0 ? 0 : mk) * a.C, mk < 0 ? 0u : psize);
          else
            *reinterpret_cast<uint4*>(sm + (dst - ring0)) =
                mk < 0 ? make_uint4(0u, 0u, 0u, 0u) : load8(P + static_cast<int64_t>(mk) * a.C, c, a.C, false);
        }
      } else {
        const uint32_t size = !kTail || 8 * pch < left ? 16u : 0u;
#pragma unroll
        for (int k = 0; k < L::kPer; ++k) {
          const uint32_t dst = st + pdst + k * L::kStep * 128;
          if (pvec) {
            if (m[k] >= 0) cp_async_16s(dst, size ? src[k] : P, size);
          } else if (m[k] >= 0) {
            const int64_t ci = c + static_cast<int64_t>(i) * 64 * L::kSub;
            *reinterpret_cast<uint4*>(sm + (dst - ring0)) = load8(src[k] - ci, ci, a.C, false);
          }
          src[k] += 64 * L::kSub;
        }
      }
#pragma unroll
      for (int k = 0; k < L::kPerW; ++k) {
        if (L::kChunksW % kLtcLoaders != 0 && tid + kLtcLoaders * k >= L::kChunksW) continue;
        const uint32_t size = !kTail || wrow[k] < left ? wsize[k] : 0u;
        if (kW || wvec) {
          cp_async_16s(st + wdst[k], size ? wsrc[k] : wzero, size);
        } else {  // from the row's start: wc0 columns (or inner columns) before this chunk
          const int64_t wc0 = kMode == kReduceA ? (static_cast<int64_t>(s0) + i) * 64 * L::kSub + wrow[k]
                                                : 8 * ((tid + kLtcLoaders * k) % (RP / 8));
          *reinterpret_cast<uint4*>(sm + (st - ring0) + wdst[k]) =
              size ? load8(wsrc[k] - wc0, wc0, kMode == kReduceA ? a.C : a.rank, false) : make_uint4(0u, 0u, 0u, 0u);
        }
        wsrc[k] += wadvance;
      }
      left -= kW ? 64 : 64 * L::kSub;
    };
    int hd = 0, hs = 0;  // the stage to hand over and its slot
    auto hand_over = [&]() {
      if (drop) {
        uint8_t* st = sm + hs * L::kStage + pdst;
        const int64_t hc = kW ? c : c + static_cast<int64_t>(hd) * 64 * L::kSub;
        if (hc < a.C)
#pragma unroll
          for (int k = 0; k < L::kPer; ++k) {
            const int64_t mk = kW ? rowbuf[(hd % (2 * kRowStages)) * 64 + prow + L::kStep * k] : m[k];
            uint4* x = reinterpret_cast<uint4*>(st + k * L::kStep * 128);
            if (mk >= 0) *x = drop_apply16(*x, mk * groups + (hc >> 3), key, a.drop.thr);
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[hs]);
      ++hd;
      if (++hs == L::kRing) hs = 0;
    };
    if (kW && a.behind) pdl_wait_prior_grids();
    uint32_t st = ring0, parity = 1u;  // the slot of the stage requested, and the parity of its last release
    uint64_t* release = empty;
    for (int i = 0; i < ns; ++i) {
      if (kW && i % kRowStages == 0) {
        // The set before last is not read any more: a warp is at most a ring ahead of another.
#pragma unroll
        for (int k = 0; k < kRowPer; ++k) rowbuf[(i % (2 * kRowStages)) * 64 + tid + kLtcLoaders * k] = rnext[k];
        __syncwarp();
        named_barrier_sync(1, kLtcLoaders);
      }
      if (kW && i % kRowStages == kRowStages / 2 && i + kRowStages / 2 < ns) fetch_rows(i + kRowStages / 2);
      if (ok && i >= L::kRing) ok = mbar_wait(release, parity);
      if (left >= (kW ? 64 : 64 * L::kSub))
        request(std::false_type(), i, st);
      else
        request(std::true_type(), i, st);
      st += L::kStage;
      ++release;
      if (st == ring1) {
        st = ring0;
        release = empty;
        parity ^= 1u;
      }
      cp_async_commit();
      if (i >= L::kLag) {
        cp_async_wait<L::kLag>();
        hand_over();
      }
    }
    cp_async_wait<0>();
    while (hd < ns) hand_over();
    if (ns > 0) ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(accFull, 0u)) != 0;
  } else if (lane == 0) {
    // ------------------------------------------------------------------ MMA issuer
    constexpr uint32_t kType = std::is_same<T, __half>::value ? 0u : (1u << 7) | (1u << 10);
    constexpr uint32_t kMajor = kMode == kReduceA ? 0u : (kMode == kReduceB ? 1u << 16 : (1u << 15) | (1u << 16));
    constexpr uint32_t kIdesc = idesc_f16_f32(128, L::kN) | kType | kMajor;
    const uint32_t base = smem_u32(sm);
    int s = 0;
    uint32_t parity = 0u;
    // as the loaders do: the limit of a wait is for this kernel's own stages, not for the kernels ahead
    if (kW && a.behind) pdl_wait_prior_grids();
    for (int i = 0; i < ns && ok; ++i) {
      ok = mbar_wait(&full[s], parity);
      if (!ok) break;
      // The stage was written by other threads' cp.async and stores, which the barrier orders before this point; the
      // fence makes them visible to the tensor core, once a stage instead of once a loader.
      fence_proxy_async_smem();
      tc_fence_after_sync();
      const uint32_t pa = base + s * L::kStage, wa = pa + L::kTileP;
#pragma unroll
      for (int p = 0; p < L::kSub; ++p) {
        const uint64_t ad = kW ? sdesc_mnmajor_sw128(pa, 8192u) : sdesc_kmajor_sw128(pa + p * 16384);
        const uint64_t bd = kMode == kReduceA ? sdesc_kmajor_sw128(wa + p * L::kPlaneW)
                                              : sdesc_mnmajor_sw128(wa + p * 8192, L::kPlaneW);
        // 16 of the summation index: 32 bytes of a K-major row, 16 rows of 128 bytes of an MN-major plane
#pragma unroll
        for (int q = 0; q < 4; ++q)
          umma_f16(tmem, ad + (kW ? 128u : 2u) * q, bd + (kMode == kReduceA ? 2u : 128u) * q, kIdesc,
                   (i | p | q) != 0 ? 1u : 0u);
      }
      umma_commit(&empty[s]);
      if (++s == L::kRing) {
        s = 0;
        parity ^= 1u;
      }
    }
    if (ok && ns > 0) umma_commit(accFull);
  }
  __syncwarp();
  tc_fence_after_sync();

  // ------------------------------------------------------------------ sums out of tensor memory
  // Warp w < 8 has lanes 32 (w % 4) .. + 31 (position or column r of the tile) and half w / 4 of the inner columns.
  if (kW) f *= a.inv[l];  // (the loaders have waited for the kernel that wrote it)
  const int r = tid & 127;
  const bool epi = warp < kLtcEpiWarps;
  if (!kW && rowbuf[r] < 0) f = 0.0f;  // a position without a row
  const bool none = !kW && rowbuf[r] < 0;
  float most = 0.0f, most2 = 0.0f;
  auto emit = [&](int j, float v) {
    if (j >= a.rank) return;
    if (kW) {
      if (c0 + r < a.C) (static_cast<T*>(a.O) + l * a.ws)[(c0 + r) * a.wc + j * a.wj] = from_f32<T>(f * v);
    } else if (r < cnt) {
      const int64_t at = (pos0 + r) * a.rank + j;
      const float o = none ? 0.0f : f * v;
      a.V[at] = o;
      most = fmaxf(most, finite_abs(o));
      if (a.most2) most2 = fmaxf(most2, finite_abs(a.V2[at]));
    }
  };
  auto sums = [&](int j0, float (&v)[8]) {
    const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + j0;
    uint32_t x[8], y[8];
    if (ok && ns > 0) {
      tmem_ld_32x32b_x8(at, x);
      if (kW) tmem_ld_32x32b_x8(at + RP, y);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(x[e]) + (kW ? __uint_as_float(y[e]) : 0.0f);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.0f;
    }
  };
  if (S == 1) {
    if (epi)
#pragma unroll 1
      for (int j0 = (warp >> 2) * (RP / 2); j0 < (warp >> 2) * (RP / 2) + RP / 2; j0 += 8) {
        float v[8];
        sums(j0, v);
        if (!kW && (a.rank & 3) == 0) {  // whole float4s of a position's row
          if (r < cnt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (j0 + 4 * h >= a.rank) continue;
              const int64_t at = (pos0 + r) * a.rank + j0 + 4 * h;
              float4 o = make_float4(f * v[4 * h], f * v[4 * h + 1], f * v[4 * h + 2], f * v[4 * h + 3]);
              if (none) o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              *reinterpret_cast<float4*>(a.V + at) = o;
              most = fmaxf(fmaxf(fmaxf(finite_abs(o.x), finite_abs(o.y)), fmaxf(finite_abs(o.z), finite_abs(o.w))), most);
              if (a.most2) {
                const float4 p = *reinterpret_cast<const float4*>(a.V2 + at);
                most2 =
                    fmaxf(fmaxf(fmaxf(finite_abs(p.x), finite_abs(p.y)), fmaxf(finite_abs(p.z), finite_abs(p.w))), most2);
              }
            }
        } else if (kW && a.wj == 1 && (a.rank & 7) == 0 && yvec) {  // dB: eight consecutive elements of a row
          if (c0 + r < a.C && j0 < a.rank) {
            Vec<T, 8> o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o.v[e] = from_f32<T>(f * v[e]);
            *reinterpret_cast<Vec<T, 8>*>(static_cast<T*>(a.O) + l * a.ws + (c0 + r) * a.rank + j0) = o;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) emit(j0 + e, v[e]);
        }
      }
  } else {
    // inner columns [q cpo, (q + 1) cpo) are added up by CTA q: partial sums [source][column][128]
    const int cpo = (RP + S - 1) / S;
    float* red = reinterpret_cast<float*>(sm);
    const uint32_t red_local = smem_u32(red);
    cluster_arrive();  // every CTA of the cluster is past its main loop: the rings are free
    cluster_wait();
    if (epi)
#pragma unroll 1
      for (int j0 = (warp >> 2) * (RP / 2); j0 < (warp >> 2) * (RP / 2) + RP / 2; j0 += 8) {
        float v[8];
        sums(j0, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int q = (j0 + e) / cpo;
          const uint32_t dst = red_local + 4u * static_cast<uint32_t>((rank * cpo + (j0 + e) - q * cpo) * 128 + r);
          st_shared_cluster_f32(mapa_shared(dst, static_cast<uint32_t>(q)), v[e]);
        }
      }
    cluster_arrive();  // all partial sums have landed
    cluster_wait();
    if (warp < kLtcWarps)
      for (int j = tid >> 7; j < cpo && rank * cpo + j < RP; j += kLtcLoaders / 128) {
        float v = 0.0f;
        for (int q = 0; q < S; ++q) v += red[(q * cpo + j) * 128 + r];
        emit(rank * cpo + j, v);
      }
  }
  if (!kW && a.most) {
    most = warp_max(most);
    most2 = warp_max(most2);
    if (lane == 0 && warp < kLtcWarps) {
      mostbuf[warp] = most;
      mostbuf[16 + warp] = most2;
    }
    __syncthreads();
    if (tid < 2) {
      float x = 0.0f;
      for (int i = 0; i < kLtcWarps; ++i) x = fmaxf(x, mostbuf[16 * tid + i]);
      float* to = tid == 0 ? a.most : a.most2;
      if (to) to[static_cast<int64_t>(blockIdx.x) * kLoraMostPer + rank] = x;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kLtcWarps) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

// V [M, rank] fp32 -> hi and lo [M, 2 RP] (zeros past the rank), scaled by the adapter's power of two, whose inverse
// goes to inv[l]: once for all columns of wgrad, which would repeat it for each 128 of them.  A CTA per tile; grid y:
// v and dv.
struct LoraSplitArgs {
  const float* V[2];
  const float* most[2];  // or null (bf16)
  void* Q[2];
  float* inv[2];
  const int32_t* offsets;
  int64_t M;
  int L, rank, most_n;
};

template <typename T, int RP>
__global__ void __launch_bounds__(256) lora_split_kernel(const LoraSplitArgs a) {
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31;
  const bool y = blockIdx.y != 0;
  const float* const V = y ? a.V[1] : a.V[0];
  const float* const tiles = y ? a.most[1] : a.most[0];
  uint4* const Q = static_cast<uint4*>(y ? a.Q[1] : a.Q[0]);
  const LoraTile t = lora_tile(a.offsets, a.L, a.M, blockIdx.x);
  if (t.l < 0) return;
  float scale = 1.0f, inv = 1.0f;
  if (std::is_same<T, __half>::value) {
    const int64_t n = clamp_pos(a.offsets[t.l + 1], a.M) - clamp_pos(a.offsets[t.l], a.M);
    const int64_t slots = (n + kLoraTile - 1) / kLoraTile * a.most_n;
    float most = 0.0f;
    for (int64_t i = lane; i < slots; i += 32) {
      const int64_t k = i / a.most_n;
      most = fmaxf(most, tiles[(t.first + k) * kLoraMostPer + i - k * a.most_n]);
    }
    scale = split_scale<T>(warp_max(most), inv);
  }
  if (threadIdx.x == 0 && static_cast<int>(blockIdx.x) == t.first) (y ? a.inv[1] : a.inv[0])[t.l] = inv;
  const bool vec = (a.rank & 3) == 0;
  for (int q = threadIdx.x; q < t.cnt * (RP / 8); q += 256) {
    const int row = q / (RP / 8), ch = q % (RP / 8);
    const float* src = V + (t.pos + row) * a.rank + 8 * ch;
    float v[8];
    if (vec) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 x = 8 * ch + 4 * h < a.rank ? *reinterpret_cast<const float4*>(src + 4 * h)
                                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        v[4 * h] = x.x;
        v[4 * h + 1] = x.y;
        v[4 * h + 2] = x.z;
        v[4 * h + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 8 * ch + e < a.rank ? src[e] : 0.0f;
    }
    uint4 hi, lo;
    split2<T>(scale * v[0], scale * v[1], hi.x, lo.x);
    split2<T>(scale * v[2], scale * v[3], hi.y, lo.y);
    split2<T>(scale * v[4], scale * v[5], hi.z, lo.z);
    split2<T>(scale * v[6], scale * v[7], hi.w, lo.w);
    uint4* dst = Q + (t.pos + row) * (RP / 4);
    dst[ch] = hi;
    dst[RP / 8 + ch] = lo;
  }
}

// Clusters of S CTAs that can be resident at once (a cluster lies in one GPC, so the GPCs bound them below SMs / S:
// on a B200 148, 74, 45, 33, 26, 22, 15 and 15 for S = 1 .. 8), queried once per device and S.
static int lora_cluster_capacity(const DeviceInfo& di, int S) {
  static std::atomic<int> cache[kPfMaxDevices][kLoraMostPer + 1];
  if (S == 1) return di.num_sms;
  if (di.device < 0 || di.device >= kPfMaxDevices) return di.num_sms / S;
  int n = cache[di.device][S].load(std::memory_order_relaxed);
  if (n > 0) return n;
  auto* kern = lora_tc_kernel<__half, kReduceA, 64, false, true>;
  constexpr int kAlloc = LoraTcLayout<kReduceA, 64>::kAlloc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, static_cast<unsigned>(S));
  cfg.blockDim = dim3(kLtcThreads);
  cfg.dynamicSmemBytes = kAlloc;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 1;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = static_cast<unsigned>(S);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (ensure_smem_attr(reinterpret_cast<const void*>(kern), kAlloc) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
    (void)cudaGetLastError();
    return di.num_sms / S;
  }
  cache[di.device][S].store(n, std::memory_order_relaxed);
  return n;
}

// CTAs per cluster for `tiles` tiles of `stages` stages: a wave costs a CTA its share of the stages, the time of
// about seven for its start and end, and of three more for the exchange between CTAs.
static int lora_split(int64_t tiles, int64_t stages) {
  const DeviceInfo di = current_device_info();
  int best = 1;
  double cost = 0.0;
  for (int S = 1; S <= kLoraMostPer && (S == 1 || S * 2 <= stages); ++S) {
    const int64_t cap = lora_cluster_capacity(di, S);
    const double c = static_cast<double>((tiles + cap - 1) / cap) *
                     (static_cast<double>(stages) / S + (S > 1 ? 10.0 : 7.0));
    if (S == 1 || c < 0.97 * cost) {
      cost = c;
      best = S;
    }
  }
  return best;
}

static int lora_pad_rank(int64_t rank) { return rank <= 16 ? 16 : (rank <= 32 ? 32 : (rank <= 64 ? 64 : 128)); }

template <typename T, int kMode, int RP, bool kDrop>
static cudaError_t launch_lora_tc(const LoraSums& sums, dim3 grid, cudaStream_t s) {
  bool vec = true;
  for (const LoraArgs& a : sums.a) vec = vec && a.pvec && (a.wvec || kMode == kWgrad) && (a.yvec || kMode != kWgrad);
  auto* kern = vec ? lora_tc_kernel<T, kMode, RP, kDrop, true> : lora_tc_kernel<T, kMode, RP, kMode != kReduceB, false>;
  constexpr int kAlloc = LoraTcLayout<kMode, RP>::kAlloc;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), kAlloc);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kLtcThreads);
  cfg.dynamicSmemBytes = kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = grid.z;
  cfg.attrs = attr;
  cfg.numAttrs = grid.z > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, sums, static_cast<int>(grid.z));
}

// CTAs that reduce a tile together (the maxima of a tile have one slot for each).
static int lora_reduce_split(const LoraArgs& a) {
  return lora_split(lora_likely_tiles(a.M, a.L), (a.C + 127) / 128);
}

static cudaError_t lora_fast_reduce(bool bf16, const LoraArgs& a, cudaStream_t s) {
  const LoraSums sums = {{a, a}, 0};
  const dim3 grid(static_cast<unsigned>(lora_max_tiles(a.M, a.L)), 1, static_cast<unsigned>(lora_reduce_split(a)));
  return with_type16(bf16, [&](auto t) {
    using T = decltype(t);
    return with_rank(a.rank, [&](auto rp) {
      constexpr int RP = decltype(rp)::value;
      if (a.wc != 1) return launch_lora_tc<T, kReduceB, RP, false>(sums, grid, s);
      return a.drop.thr ? launch_lora_tc<T, kReduceA, RP, true>(sums, grid, s)
                        : launch_lora_tc<T, kReduceA, RP, false>(sums, grid, s);
    });
  });
}

// b: the other gradient in the same launch, or null.
static cudaError_t lora_fast_wgrad(bool bf16, const LoraArgs& a, const LoraArgs* b, cudaStream_t s) {
  const int64_t first = (a.C + 127) / 128, ct = first + (b ? (b->C + 127) / 128 : 0);
  const LoraSums sums = {{a, b ? *b : a}, static_cast<int>(first)};
  const int64_t some = a.L < a.M ? a.L : (a.M < 1 ? 1 : a.M);
  const int S = lora_split(ct * some, a.M / some / 64);
  const dim3 grid(static_cast<unsigned>(ct), static_cast<unsigned>(a.L), static_cast<unsigned>(S));
  return with_type16(bf16, [&](auto t) {
    using T = decltype(t);
    return with_rank(a.rank, [&](auto rp) {
      constexpr int RP = decltype(rp)::value;
      return a.drop.thr ? launch_lora_tc<T, kWgrad, RP, true>(sums, grid, s)
                        : launch_lora_tc<T, kWgrad, RP, false>(sums, grid, s);
    });
  });
}

// Workspace of the gradients: dv fp32 [M, rank]; the tiles' maxima of v and of dv; the inverse scales; v and dv as hi
// and lo.
struct LoraWorkspace {
  float* dv;
  float* most[2];
  float* inv[2];
  uint16_t* Q[2];
  size_t bytes;
};

LoraWorkspace lora_workspace(void* base, int64_t M, int64_t L, int64_t rank) {
  LoraWorkspace w;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    void* p = static_cast<char*>(base) + at;
    at += (bytes + 15) / 16 * 16;
    return p;
  };
  w.dv = static_cast<float*>(take(static_cast<size_t>(M) * rank * 4));
  for (int i = 0; i < 2; ++i) {
    w.most[i] = static_cast<float*>(take(static_cast<size_t>(lora_max_tiles(M, L)) * kLoraMostPer * 4));
    w.inv[i] = static_cast<float*>(take(static_cast<size_t>(L) * 4));
    w.Q[i] = static_cast<uint16_t*>(take(static_cast<size_t>(M) * 2 * lora_pad_rank(rank) * 2));
  }
  w.bytes = at;
  return w;
}

// hi and lo of v (into Q[0]) and, with `both`, of dv (Q[1]).
cudaError_t launch_lora_split(bool bf16, bool both, const LoraWorkspace& w, const float* v, const int32_t* offsets,
                              int64_t M, int64_t L, int rank, int most_n, cudaStream_t s) {
  LoraSplitArgs a = {};
  a.V[0] = v;
  a.V[1] = w.dv;
  for (int i = 0; i < 2; ++i) {
    a.most[i] = bf16 ? nullptr : w.most[i];
    a.Q[i] = w.Q[i];
    a.inv[i] = w.inv[i];
  }
  a.offsets = offsets;
  a.M = M;
  a.L = static_cast<int>(L);
  a.rank = rank;
  a.most_n = most_n;
  const dim3 grid(static_cast<unsigned>(lora_max_tiles(M, L)), both ? 2 : 1);
  return with_type16(bf16, [&](auto t) {
    using T = decltype(t);
    return with_rank(rank, [&](auto rp) {
      return launch_pdl(lora_split_kernel<T, decltype(rp)::value>, grid, dim3(256), 0, 1, s, a);
    });
  });
}

// ---------------------------------------------------------------------------------------------
// expand on tcgen05: O[m, c] = base[m, c] + f sum_j V[r, j] W_l(c, j).
//   D[position, c] (128 x 128, four buffers in tensor memory) = [hi | lo] of V (shared memory, K-major, kept for the
//   CTA's whole range of columns) x W (four stages of 128 columns)
// Bound by the rows of base and O, each touched once with 16-byte accesses straight between memory and the registers
// that hold the sums.  Sixteen epilogue warps, each with 32 positions and 32 columns of a block, read D in the
// fragment layout of m16n8 (16x256b), which gives a lane columns 2 t, 2 t + 1 of each n8 tile; W's columns are dealt
// to four n8 tiles so that these are eight consecutive ones: column c = 8 u + 2 j + e of a block of 32 is column 2 u
// + e of tile j.  base is requested two blocks ahead.
// At 96 registers the forms with W as A spill where they drop, in bf16 (78 bytes stored and 180 loaded at ranks up to
// 64, 104 and 216 at 128; dx of 8192 x 4096, rank 64, 54 us, and 40 without dropout), and at rank 128 in both types (72
// and 160 without dropout); the other bf16 forms spill 8 bytes, the fp16 ones none up to rank 64.
// Four loader warps bring W: as B [C, rank] a column's 16-byte pieces with cp.async, as A [rank, C] through
// registers, since pairs of columns part ways (4-byte cp.async took 78 cycles an instruction).  Only barriers of
// single stages tie the warps.
// All tiles' blocks in a row are dealt to the CTAs, one per SM, in equal runs, which cross from tile to tile where
// they must: with a CTA per tile and range of columns, SMs were idle for a third of the time (4096 rows, 6 adapters,
// rank 32, 18944 columns: 81 us, now 71).  mma.sync on the same fragments, two CTAs per SM, was bound by the MMA rate
// from rank 64 on (rank 128, 8192 x 8192, no base: 150 us; this 79, rank 64 72 and 50, rank 16 44 and 35, the rate of
// plain writes).
// ---------------------------------------------------------------------------------------------
constexpr int kXpEpi = 16;     // epilogue warps
constexpr int kXpLoad = 4;     // loader warps; the first also issues the MMAs (20 warps: 96 registers a thread, 21: 80)
constexpr int kXpThreads = 32 * (kXpEpi + kXpLoad);
constexpr int kXpCols = 128;   // columns per block (MMA N)
constexpr int kXpRing = 4;     // stages of W, and of D
constexpr int kXpCopy = 8;     // vectors per lane and round where rows of no adapter are copied

template <int RP, bool kWA>
struct LoraXpLayout {
  static constexpr int kPlanesV = 2 * RP <= 64 ? 1 : 2 * RP / 64;     // planes of 64 k: hi then lo
  static constexpr int kTileV = kPlanesV * 16384;
  static constexpr int kPlaneW = kWA ? RP * 128 : kXpCols * 128;      // A: 64 columns x RP k; B: 128 columns x 64 k
  static constexpr int kTileW = kWA ? 2 * kPlaneW : (RP + 63) / 64 * kPlaneW;
  static constexpr int kLag = kWA ? 0 : kXpRing - 2;                  // stages between request and hand-over (B)
  static constexpr int kOffW = kTileV;
  static constexpr int kOffBar = kOffW + kXpRing * kTileW;            // wfull, wempty, dfull, dempty, vfull; TMEM slot
  static constexpr int kOffF = kOffBar + (4 * kXpRing + 2) * 8;       // fp32 factor of each position
  static constexpr int kBytes = kOffF + 2 * 128 * 4 + 1024;
  static constexpr int kAlloc = kBytes > 116 * 1024 + 64 ? kBytes : 116 * 1024 + 64;  // one CTA per SM, as above
  static_assert(kAlloc <= 227 * 1024 && kTileW % 1024 == 0, "shared memory");
};

// 16 lanes x 32 columns of tensor memory in the fragment layout of m16n8: r[4 j + i] is element i of the n8 tile j.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

template <typename T, int RP, bool kWA, bool kDrop, bool kVec>  // kVec, kDrop as in lora_tc_kernel
__global__ void __launch_bounds__(kXpThreads, 1) lora_expand_tc_kernel(const LoraArgs a) {
  using L = LoraXpLayout<RP, kWA>;
  const bool wvec = kVec || a.wvec, yvec = kVec || a.yvec, drop = kDrop && (kVec || a.drop.thr != 0);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* wfull = reinterpret_cast<uint64_t*>(sm + L::kOffBar);
  uint64_t* wempty = wfull + kXpRing;
  uint64_t* dfull = wempty + kXpRing;
  uint64_t* dempty = dfull + kXpRing;
  uint64_t* vfull = dempty + kXpRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(vfull + 1);
  float* rowf = reinterpret_cast<float*>(sm + L::kOffF);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The preceding kernel is this call's reduction (or one behind it), which let this one start only after the work
  // before the call had finished: everything but V may be read at once.
  const int64_t nblk = (a.C + kXpCols - 1) / kXpCols, total = lora_tiles(a.offsets, a.L, a.M) * nblk;
  const int64_t run0 = total * blockIdx.x / gridDim.x, run1 = total * (blockIdx.x + 1) / gridDim.x;
  if (run0 == run1) {
    pdl_wait_prior_grids();  // no CTA ends before the kernels ahead of it: the next takes this grid's end for theirs
    return;
  }
  const T* base = static_cast<const T*>(a.base);
  T* out = static_cast<T*>(a.O);

  if (tid == 0) {
    for (int i = 0; i < kXpRing; ++i) {
      mbar_init(&wfull[i], kXpLoad);
      mbar_init(&wempty[i], 1);
      mbar_init(&dfull[i], 1);
      mbar_init(&dempty[i], kXpEpi);
    }
    mbar_init(vfull, kXpEpi);
    fence_mbar_init();
  }
  if (warp == kXpEpi) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  pdl_allow_dependents();
  const uint32_t tmem = *tmem_slot;

  bool ok = !(warp == kXpEpi && skip_x_loads());  // as in lora_tc_kernel
  if (warp < kXpEpi) {
    // ------------------------------------------------------------------ epilogue
    const int g = lane >> 2, t = lane & 3, r0 = (warp & 3) * 32 + g;
    const PhiloxKey key = kDrop ? philox_key(a.drop) : PhiloxKey{0u, 0u, 0u, 0u};
    const int64_t groups = (a.C + 7) >> 3;
    int s = 0, seg = 0;
    uint32_t parity = 0u;
    bool waited = false;
    for (int64_t run = run0; run < run1;) {
      const int64_t tn = run / nblk, c_begin = (run - tn * nblk) * kXpCols;
      const int nb = static_cast<int>(run1 - run < nblk * (tn + 1) - run ? run1 - run : nblk * (tn + 1) - run);
      const int64_t c_stop = c_begin + static_cast<int64_t>(nb) * kXpCols, c_end = c_stop < a.C ? c_stop : a.C;
      run += nb;
      const LoraTile tile = lora_tile(a.offsets, a.L, a.M, static_cast<int>(tn));
      if (tile.l < 0) {  // rows of no adapter: base alone
        if (base == out) continue;
        const int64_t head = clamp_pos(a.offsets[0], a.M), at = clamp_pos(a.offsets[a.L], a.M);
        const int vecs = static_cast<int>((c_end - c_begin) >> 3);
        for (int i = warp; i < tile.cnt; i += kXpEpi) {
          const int64_t q = tile.pos + i, m = lora_row(a, q < head ? q : q - head + at);
          if (m < 0) continue;
          if (!yvec) {
            for (int64_t c = c_begin + lane; c < c_end; c += 32)
              out[m * a.C + c] = base ? base[m * a.C + c] : from_f32<T>(0.0f);
            continue;
          }
          uint4* dst = reinterpret_cast<uint4*>(out + m * a.C + c_begin);
          const uint4* src = reinterpret_cast<const uint4*>(base + m * a.C + c_begin);
          for (int j = lane; j < vecs; j += 32 * kXpCopy) {  // all loads of a round before its stores
            uint4 x[kXpCopy];
#pragma unroll
            for (int k = 0; k < kXpCopy; ++k)
              x[k] = base && j + 32 * k < vecs ? src[j + 32 * k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int k = 0; k < kXpCopy; ++k)
              if (j + 32 * k < vecs) dst[j + 32 * k] = x[k];
          }
        }
        continue;
      }
      int m[4];  // rows of positions r0 + 8 i
#pragma unroll
      for (int i = 0; i < 4; ++i)
        m[i] = r0 + 8 * i < tile.cnt ? static_cast<int>(lora_row(a, tile.pos + r0 + 8 * i)) : -1;
      int64_t c = c_begin + (warp >> 2) * 32 + 8 * t;  // this lane's eight columns
      uint4 y[2][4];
      auto load_base = [&](uint4 (&to)[4], int64_t at) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          to[i] = base && m[i] >= 0 && at < c_end ? load8(base + static_cast<int64_t>(m[i]) * a.C, at, a.C, yvec)
                                                  : make_uint4(0u, 0u, 0u, 0u);
      };
      load_base(y[0], c);
      load_base(y[1], c + kXpCols);
      {
        // V of the tile as hi and lo, four threads per position (the last run's MMAs have read theirs: this warp has
        // seen their sums)
        const int row = tid >> 2, part = tid & 3;
        constexpr int kE = RP / 4;  // inner columns per thread
        const bool there = row < tile.cnt;
        const float* src = a.V + (tile.pos + row) * a.rank;
        float most = 0.0f;
        float v[kE];
        if (!waited) pdl_wait_prior_grids();
        waited = true;
        if ((a.rank & 3) == 0) {
#pragma unroll
          for (int e = 0; e < kE; e += 4) {
            const int j = part * kE + e;
            const float4 x = there && j < a.rank ? *reinterpret_cast<const float4*>(src + j)
                                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            v[e] = x.x;
            v[e + 1] = x.y;
            v[e + 2] = x.z;
            v[e + 3] = x.w;
          }
        } else {
#pragma unroll
          for (int e = 0; e < kE; ++e) v[e] = there && part * kE + e < a.rank ? src[part * kE + e] : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < kE; ++e) most = fmaxf(most, fabsf(v[e]));
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        float inv;
        const float sc = split_scale<T>(most, inv);
#pragma unroll
        for (int e = 0; e < kE; e += 4) {
          uint2 hi, lo;
          split2<T>(sc * v[e], sc * v[e + 1], hi.x, lo.x);
          split2<T>(sc * v[e + 2], sc * v[e + 3], hi.y, lo.y);
          const int kh = part * kE + e, kl = RP + kh;  // k of hi and of lo
          auto at = [&](int k) {
            return sm + (k >> 6) * 16384 + row * 128 + ((((k >> 3) & 7) ^ (row & 7)) << 4) + (k & 4) * 2;
          };
          *reinterpret_cast<uint2*>(at(kh)) = hi;
          *reinterpret_cast<uint2*>(at(kl)) = lo;
        }
        if (part == 0) rowf[(seg & 1) * 128 + row] = inv * lora_factor(a, tile.l);
        __syncwarp();
        if (lane == 0) mbar_arrive(vfull);
      }
      // rowf, of which there are two, since a warp may be done with a short run before another reads this one's
      named_barrier_sync(1, 32 * kXpEpi);
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = rowf[(seg & 1) * 128 + r0 + 8 * i];
      auto block = [&](uint4 (&yb)[4]) {
        ok = ok && mbar_wait(&dfull[s], parity);  // (a vote here costs registers that the bf16 kernels do not have)
        __syncwarp();
        tc_fence_after_sync();
        const uint32_t at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + s * kXpCols + (warp >> 2) * 32;
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // positions r0 + 16 h and + 8
          uint32_t acc[16];
          tmem_ld_16x256b_x4(at + (static_cast<uint32_t>(16 * h) << 16), acc);
          tmem_ld_wait();
          if (h == 1) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&dempty[s]);
          }
          if (c >= c_end || !ok) continue;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (m[2 * h + i] < 0) continue;
            const int64_t at_row = static_cast<int64_t>(m[2 * h + i]) * a.C + c;
            Vec<T, 8> o = *reinterpret_cast<const Vec<T, 8>*>(&yb[2 * h + i]);
            const uint4 bits = drop ? philox(m[2 * h + i] * groups + (c >> 3), key) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x = __uint_as_float(acc[4 * (e >> 1) + 2 * i + (e & 1)]), z = to_f32(o.v[e]);
              o.v[e] = from_f32<T>(drop && !drop_keeps(bits, e, a.drop.thr) ? z : fmaf(f[2 * h + i], x, z));
            }
            if (yvec) {
              *reinterpret_cast<Vec<T, 8>*>(out + at_row) = o;
            } else {
              for (int e = 0; e < 8 && c + e < a.C; ++e) out[at_row + e] = o.v[e];
            }
          }
        }
        if (++s == kXpRing) {
          s = 0;
          parity ^= 1u;
        }
      };
      for (int b = 0; b < nb; b += 2) {
        block(y[0]);
        load_base(y[0], c + 2 * kXpCols);
        c += kXpCols;
        if (b + 1 < nb) {
          block(y[1]);
          load_base(y[1], c + 2 * kXpCols);
          c += kXpCols;
        }
      }
      ++seg;
    }
    if (!waited) pdl_wait_prior_grids();
  } else {
    // ------------------------------------------------------------------ loaders of W; the first warp also issues the
    // MMAs
    const int w = tid - 32 * kXpEpi;  // 0 .. 127
    constexpr uint32_t kType = std::is_same<T, __half>::value ? 0u : (1u << 7) | (1u << 10);
    constexpr uint32_t kIdesc = idesc_f16_f32(128, kXpCols) | kType | (kWA ? 1u << 16 : 0u);
    const uint32_t base_v = smem_u32(sm);
    int s = 0, hs = 0, seg = 0;
    uint32_t parity = 1u, hparity = 0u;
    int64_t done = 0;  // blocks requested in earlier runs
    // Whatever waits for V, directly or through the stages of W, first waits for the kernels ahead, without a limit.
    bool waited = false;
    auto wait_ahead = [&]() {
      if (!waited) pdl_wait_prior_grids();
      waited = true;
    };
    for (int64_t run = run0; run < run1;) {
      const int64_t tn = run / nblk, c_begin = (run - tn * nblk) * kXpCols;
      const int nb = static_cast<int>(run1 - run < nblk * (tn + 1) - run ? run1 - run : nblk * (tn + 1) - run);
      run += nb;
      const LoraTile tile = lora_tile(a.offsets, a.L, a.M, static_cast<int>(tn));
      if (tile.l < 0) continue;
      const uint16_t* W = static_cast<const uint16_t*>(a.W) + tile.l * a.ws;
      // A: chunk (row j = w / 16 + 8 i, eight columns from 8 (w % 16)) of a block, a block ahead in registers
      constexpr int kPerA = kWA ? RP / 8 : 1;
      uint4 pre[kPerA];
      const int ach = w & 15, aj = w >> 4;
      auto load_a = [&](int b) {
        const int64_t at = c_begin + static_cast<int64_t>(b) * kXpCols + 8 * ach;
#pragma unroll
        for (int i = 0; i < kPerA; ++i)
          pre[i] = at < a.C && aj + 8 * i < a.rank ? load8(W + (aj + 8 * i) * a.C, at, a.C, wvec)
                                                   : make_uint4(0u, 0u, 0u, 0u);
      };
      if (kWA) load_a(0);
      for (int b = 0; b < nb + L::kLag; ++b) {
        if (b < nb) {
          if (done + b >= kXpRing) {
            wait_ahead();
            if (ok) ok = mbar_wait(&wempty[s], parity);
          }
          uint8_t* st = sm + L::kOffW + s * L::kTileW;
          if (kWA) {
            // columns 8 u + 2 j + e of a block of 32 to 8 j + 2 u + e: piece j of the chunk to 16-byte chunk j of the
            // block
            const int hb = ach >> 2;
            uint8_t* dst = st + (hb >> 1) * L::kPlaneW + aj * 128 + 4 * (ach & 3);
#pragma unroll
            for (int i = 0; i < kPerA; ++i) {
              const uint32_t word[4] = {pre[i].x, pre[i].y, pre[i].z, pre[i].w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint32_t*>(dst + i * 1024 + (((4 * (hb & 1) + j) ^ (aj & 7)) << 4)) = word[j];
            }
            if (b + 1 < nb) load_a(b + 1);
          } else {
            // column c of 128 to its place, RP / 8 pieces
            const int64_t c0 = c_begin + static_cast<int64_t>(b) * kXpCols;
            const int c = w, pos = (c & ~31) + 8 * ((c >> 1) & 3) + 2 * ((c >> 3) & 3) + (c & 1);
            const bool there = c0 + c < a.C;
            const uint16_t* src = W + (there ? (c0 + c) * a.rank : 0);
#pragma unroll
            for (int ch = 0; ch < RP / 8; ++ch) {
              uint8_t* dst = st + (ch >> 3) * L::kPlaneW + pos * 128 + (((ch & 7) ^ (pos & 7)) << 4);
              const bool in = there && 8 * ch < a.rank;
              if (wvec)
                cp_async_16(dst, in ? src + 8 * ch : W, in ? 16u : 0u);
              else
                *reinterpret_cast<uint4*>(dst) = in ? load8(src, 8 * ch, a.rank, false) : make_uint4(0u, 0u, 0u, 0u);
            }
          }
          if (++s == kXpRing) {
            s = 0;
            parity ^= 1u;
          }
        }
        if (!kWA) {
          cp_async_commit();
          if (b < L::kLag) continue;
          cp_async_wait<L::kLag>();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&wfull[hs]);
        if (warp == kXpEpi) {
          // the MMAs of the block handed over: four buffers of D keep the epilogue busy while this warp waits
          const int d = b - L::kLag;
          wait_ahead();
          ok = ok && (d > 0 || mbar_wait(vfull, static_cast<uint32_t>(seg & 1))) && mbar_wait(&wfull[hs], hparity) &&
               (done + d < kXpRing || mbar_wait(&dempty[hs], hparity ^ 1u));
          if (lane == 0 && ok) {
            fence_proxy_async_smem();  // for the other warps' copies and stores, which the barriers order before this
            tc_fence_after_sync();
            const uint32_t wa = base_v + L::kOffW + hs * L::kTileW;
#pragma unroll
            for (int part = 0; part < 2; ++part)  // hi, lo
#pragma unroll
              for (int q = 0; q < RP / 16; ++q) {
                const int kv = part * RP + 16 * q;
                const uint64_t ad = sdesc_kmajor_sw128(base_v + (kv >> 6) * 16384) + 2 * ((kv & 63) >> 4);
                const uint64_t bd = kWA ? sdesc_mnmajor_sw128(wa, L::kPlaneW) + 128 * q
                                        : sdesc_kmajor_sw128(wa + (q >> 2) * L::kPlaneW) + 2 * (q & 3);
                umma_f16(tmem + hs * kXpCols, ad, bd, kIdesc, (part | q) != 0 ? 1u : 0u);
              }
            umma_commit(&wempty[hs]);
            umma_commit(&dfull[hs]);
          }
          __syncwarp();
        }
        if (++hs == kXpRing) {
          hs = 0;
          hparity ^= 1u;
        }
      }
      done += nb;
      ++seg;
    }
    cp_async_wait<0>();
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kXpEpi) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int RP, bool kWA, bool kDrop>
static cudaError_t launch_lora_expand_tc(const LoraArgs& a, cudaStream_t s) {
  auto* kern = a.wvec && a.yvec ? lora_expand_tc_kernel<T, RP, kWA, kDrop, true>
                                : lora_expand_tc_kernel<T, RP, kWA, kWA, false>;
  constexpr int kAlloc = LoraXpLayout<RP, kWA>::kAlloc;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), kAlloc);
  if (e != cudaSuccess) return e;
  // a CTA per SM, fewer where that would leave them a single block
  const int64_t sms = current_device_info().num_sms;
  const int64_t runs = (lora_max_tiles(a.M, a.L) * ((a.C + kXpCols - 1) / kXpCols) + 1) / 2;
  return launch_pdl(kern, dim3(static_cast<unsigned>(runs < sms ? runs : sms)), dim3(kXpThreads), kAlloc, 1, s, a);
}

static cudaError_t lora_fast_expand(bool bf16, const LoraArgs& a, cudaStream_t s) {
  return with_type16(bf16, [&](auto t) {
    using T = decltype(t);
    return with_rank(a.rank, [&](auto rp) {
      constexpr int RP = decltype(rp)::value;
      if (a.wc != 1) return launch_lora_expand_tc<T, RP, false, false>(a, s);
      return a.drop.thr ? launch_lora_expand_tc<T, RP, true, true>(a, s)
                        : launch_lora_expand_tc<T, RP, true, false>(a, s);
    });
  });
}

// ---------------------------------------------------------------------------------------------
// Few rows: one launch.  A cluster of eight CTAs takes up to eight positions of one adapter: each CTA sums an eighth
// of the columns of x (m16n8k16: 16 inner columns x 8 positions), the partial sums meet through distributed shared
// memory in rank order, and each CTA then computes an eighth of the columns of out (16 x 8: 8 positions, rows 8 .. 15
// unused, x 8 columns).
// Bound by the latency of this chain and, with many adapters, by reading each one's A and B once from HBM.  So B does
// not wait for the chain: 32 rows of B are one piece of memory, and each warp keeps the next two or three such blocks
// in flight into shared memory of its own by bulk copies from the start on.  (B ahead in registers spilled; asked
// into L2 by prefetches, these held up the warps that made them for up to 6 us.)
// One row, rank 16, 4096 -> 4096: 4.5 us; 61 rows of 32 adapters of rank 64, 4096 -> 14336: 19 us for 66 MB (10 us at
// the copy rate); 250 rows of 100 adapters of rank 8, 3584 -> 512: 11 us.
// Within 32 k, lane t of a quad takes the eight consecutive k = 8 t .. 8 t + 7 (both operands the same, so the order
// within the sum does not matter) in one 16-byte load.
// ---------------------------------------------------------------------------------------------
constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewRows = 8;
constexpr int kFewCluster = 8;

template <int RP>
struct LoraFewLayout {
  static constexpr int kSlots = RP <= 32 ? 3 : 2;       // blocks of B in flight per warp
  static constexpr int kSlot = 32 * RP * 2;
  static constexpr int kOffRed = kFewWarps * kSlots * kSlot;             // the warps' partial sums [column][position]
  static constexpr int kOffPart = kOffRed + kFewWarps * RP * kFewRows * 4;  // of the CTA
  static constexpr int kOffV = kOffPart + RP * kFewRows * 4;             // v [position][inner column]
  static constexpr int kOffBar = kOffV + RP * kFewRows * 4;
  static constexpr int kBytes = kOffBar + kFewWarps * kSlots * 8;
};

struct LoraFewArgs {
  const void* x;
  const void* A;
  const void* B;
  const void* base;
  void* out;
  float* V;  // may be null
  const float* scaling;
  const int32_t* offsets;
  const int32_t* order;
  int64_t M, N, K;
  int L, rank;
};

// kVec: rows of B in whole 16-byte vectors (8-byte ones for RP = 16).
template <typename T, int RP, bool kVec>
__global__ void __launch_bounds__(kFewThreads, RP <= 16 ? 3 : (RP <= 64 ? 2 : 1)) lora_few_kernel(const LoraFewArgs a) {
  using L = LoraFewLayout<RP>;
  constexpr int RT = RP / 16;                 // tiles of 16 inner columns
  constexpr int KG = RP < 32 ? 1 : RP / 32;   // groups of 32 inner columns (RP = 16: one of 16)
  extern __shared__ __align__(128) uint8_t few_smem[];
  uint8_t* sm = few_smem;
  float* part = reinterpret_cast<float*>(sm + L::kOffPart);
  float* vs = reinterpret_cast<float*>(sm + L::kOffV);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  float* red = reinterpret_cast<float*>(sm + L::kOffRed) + warp * RP * kFewRows;
  uint8_t* slots = sm + warp * L::kSlots * L::kSlot;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kOffBar) + warp * L::kSlots;
  if (lane == 0) {
    for (int i = 0; i < L::kSlots; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const bool skip = skip_x_loads();  // failure-path test hook (no block of B is requested): never set in normal use
  const int rank = static_cast<int>(blockIdx.x);  // in the cluster
  const LoraTile chunk = lora_tile<kFewRows>(a.offsets, a.L, a.M, blockIdx.y);
  if (chunk.l == -2) return;  // (the whole cluster, as below)
  const int64_t r = chunk.pos;
  const int l = chunk.l, cnt = chunk.cnt;
  // columns of out of this CTA, in blocks of 32
  const int nblk = static_cast<int>((a.N + 31) / 32);
  const int parts = kFewCluster * static_cast<int>(gridDim.z);
  const int part_id = static_cast<int>(blockIdx.z) * kFewCluster + rank;
  const int b0 = static_cast<int>(static_cast<int64_t>(part_id) * nblk / parts);
  const int b1 = static_cast<int>(static_cast<int64_t>(part_id + 1) * nblk / parts);
  auto row_of = [&](int64_t q) {
    const int64_t m = a.order ? static_cast<int64_t>(a.order[q]) : q;
    return m >= 0 && m < a.M ? m : -1;
  };
  if (l < 0) {  // rows of no adapter: base alone, a warp each
    if (a.base == a.out || warp >= cnt) return;
    const int64_t head = clamp_pos(a.offsets[0], a.M), q = r + warp;
    const int64_t m = row_of(q < head ? q : q - head + clamp_pos(a.offsets[a.L], a.M));
    if (m < 0) return;
    const int c1 = b1 * 32 < a.N ? b1 * 32 : static_cast<int>(a.N);
    for (int c = b0 * 32 + 8 * lane; c < c1; c += 8 * 32)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + m * a.N + c) =
          a.base ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.base) + m * a.N + c)
                 : make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int64_t m = g < cnt ? row_of(r + g) : -1;  // of this lane's position
  const T* A = static_cast<const T*>(a.A) + static_cast<int64_t>(l) * a.rank * a.K;
  const T* B = static_cast<const T*>(a.B) + static_cast<int64_t>(l) * a.rank * a.N;
  // Block blk of B into slot s of this warp (whole 16-byte pieces: N is a multiple of 8); one lane.
  auto request = [&](int blk, int s) {
    const int64_t n0 = static_cast<int64_t>(blk) * 32, n = a.N - n0 < 32 ? a.N - n0 : 32;
    const uint32_t bytes = static_cast<uint32_t>(n * a.rank * 2);
    mbar_arrive_expect_tx(&bars[s], bytes);
    bulk_load_1d(slots + s * L::kSlot, B + n0 * a.rank, bytes, &bars[s]);
  };
  if (lane == 0 && !skip)
    for (int i = 0; i < L::kSlots; ++i)
      if (b0 + warp + kFewWarps * i < b1) request(b0 + warp + kFewWarps * i, i);

  // ---- an eighth of x A^T, groups of 32 columns dealt to the warps.  No load of A depends on a bound: where a row
  // or column is past the end the address is one within the same matrix row, and what is read there meets a zero of x
  // or goes to an unused sum.
  const int K = static_cast<int>(a.K), ng = (K + 31) / 32;
  const int g0 = rank * ng / kFewCluster, g1 = (rank + 1) * ng / kFewCluster;
  {
    float acc[RT][4] = {};
    const T* xrow = static_cast<const T*>(a.x) + (m >= 0 ? m * a.K : 0);
    constexpr int kU = RP <= 32 ? 2 : 1;  // groups whose loads a warp has in flight
    for (int q = g0 + warp; q < g1; q += kFewWarps * kU) {
      uint4 xv[kU], lo[kU][RT], hi[kU][RT];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        int k = 32 * (q + kFewWarps * u) + 8 * t;
        const bool in = m >= 0 && q + kFewWarps * u < g1 && k < K;
        if (k >= K) k = 0;
        xv[u] = make_uint4(0u, 0u, 0u, 0u);
        if (in) xv[u] = *reinterpret_cast<const uint4*>(xrow + k);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const int j = 16 * i + g;
          const uint32_t j0 = static_cast<uint32_t>(j < a.rank ? j : a.rank - 1);
          const uint32_t j1 = static_cast<uint32_t>(j + 8 < a.rank ? j + 8 : a.rank - 1);
          lo[u][i] = *reinterpret_cast<const uint4*>(A + (j0 * static_cast<uint32_t>(K) + static_cast<uint32_t>(k)));
          hi[u][i] = *reinterpret_cast<const uint4*>(A + (j1 * static_cast<uint32_t>(K) + static_cast<uint32_t>(k)));
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          mma16(acc[i], lo[u][i].x, hi[u][i].x, lo[u][i].y, hi[u][i].y, xv[u].x, xv[u].y, T());
          mma16(acc[i], lo[u][i].z, hi[u][i].z, lo[u][i].w, hi[u][i].w, xv[u].z, xv[u].w, T());
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      *reinterpret_cast<float2*>(&red[(16 * i + g) * kFewRows + 2 * t]) = make_float2(acc[i][0], acc[i][1]);
      *reinterpret_cast<float2*>(&red[(16 * i + g + 8) * kFewRows + 2 * t]) = make_float2(acc[i][2], acc[i][3]);
    }
  }

  // ---- base of this warp's first blocks, and the partial sums meet
  constexpr int kY = 2;
  uint4 yv[kY];
  const T* yrow = static_cast<const T*>(a.base) + (m >= 0 ? m * a.N : 0);
  auto load_y = [&](int blk) {
    const int c = 32 * blk + 8 * t;
    uint4 y = make_uint4(0u, 0u, 0u, 0u);
    if (a.base && m >= 0 && blk < b1 && c < a.N) y = *reinterpret_cast<const uint4*>(yrow + c);
    return y;
  };
#pragma unroll
  for (int i = 0; i < kY; ++i) yv[i] = load_y(b0 + warp + kFewWarps * i);
  __syncthreads();
  for (int i = tid; i < RP * kFewRows; i += kFewThreads) {
    const float* p = reinterpret_cast<const float*>(sm + L::kOffRed) + i;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) s += p[w * RP * kFewRows];
    part[i] = s;
  }
  cluster_arrive();
  cluster_wait();
  for (int i = tid; i < RP * kFewRows; i += kFewThreads) {
    const uint32_t at = smem_u32(&part[i]);
    float p[kFewCluster], s = 0.0f;
#pragma unroll
    for (int q = 0; q < kFewCluster; ++q) p[q] = ld_shared_cluster_f32(mapa_shared(at, static_cast<uint32_t>(q)));
#pragma unroll
    for (int q = 0; q < kFewCluster; ++q) s += p[q];
    const int j = i / kFewRows, pos = i % kFewRows;
    vs[pos * RP + j] = s;
    if (a.V && part_id == 0 && pos < cnt && j < a.rank) a.V[(r + pos) * a.rank + j] = s;
  }
  cluster_arrive();  // this CTA has read the others' partial sums; waited for at the end
  __syncthreads();

  // ---- fragments of v: position g, hi and lo, lane's k as in the blocks of B (zeros past the rank)
  const int kc = RP < 32 ? 4 * t : 8 * t;
  uint32_t hi[KG][4], lo[KG][4];
  float f;
  {
    float most = 0.0f, v[KG][8];
#pragma unroll
    for (int q = 0; q < KG; ++q)
#pragma unroll
      for (int e = 0; e < (RP < 32 ? 4 : 8); ++e) {
        const int j = 32 * q + kc + e;
        v[q][e] = j < a.rank ? vs[g * RP + j] : 0.0f;
        most = fmaxf(most, fabsf(v[q][e]));
      }
    most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
    most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
    const float s = split_scale<T>(most, f);
    if (a.scaling) f *= a.scaling[l];
#pragma unroll
    for (int q = 0; q < KG; ++q)
#pragma unroll
      for (int e = 0; e < (RP < 32 ? 2 : 4); ++e) split2<T>(s * v[q][2 * e], s * v[q][2 * e + 1], hi[q][e], lo[q][e]);
  }
  // column 8 (g / 2) + 2 j + g % 2 of a block is column g of tile j, so that a lane ends with eight consecutive ones
  const uint32_t brow = static_cast<uint32_t>(8 * (g >> 1) + (g & 1)) * static_cast<uint32_t>(a.rank);
  T* orow = static_cast<T*>(a.out) + (m >= 0 ? m * a.N : 0);
  int slot = 0;
  uint32_t parity = 0u;
  bool ok = true;
  for (int blk = b0 + warp; blk < b1 && ok; blk += kFewWarps) {
    const T* bs = reinterpret_cast<const T*>(slots + slot * L::kSlot);
    const uint4 ycur = yv[0];
    yv[0] = yv[1];
    yv[1] = load_y(blk + kY * kFewWarps);
    ok = warp_wait(&bars[slot], parity);
    if (!ok) {  // (recorded) this copy and those requested ahead get one more bounded wait each before the CTA may end
      for (int i = 0; i < L::kSlots && blk + kFewWarps * i < b1; ++i) {
        (void)warp_wait(&bars[slot], parity);
        if (++slot == L::kSlots) {
          slot = 0;
          parity ^= 1u;
        }
      }
      break;
    }
    float d[4][4] = {};
#pragma unroll
    for (int q = 0; q < KG; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const T* row = bs + brow + 2 * j * a.rank;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (!kVec) w = load8(row, 32 * q + kc, a.rank, false);
        else if (RP >= 32) w = *reinterpret_cast<const uint4*>(row + (32 * q + kc < a.rank ? 32 * q + kc : 0));
        else *reinterpret_cast<uint2*>(&w) = *reinterpret_cast<const uint2*>(row + (kc < a.rank ? kc : 0));
        mma16(d[j], hi[q][0], 0u, hi[q][1], 0u, w.x, w.y, T());
        mma16(d[j], lo[q][0], 0u, lo[q][1], 0u, w.x, w.y, T());
        if (RP >= 32) {
          mma16(d[j], hi[q][2], 0u, hi[q][3], 0u, w.z, w.w, T());
          mma16(d[j], lo[q][2], 0u, lo[q][3], 0u, w.z, w.w, T());
        }
      }
    __syncwarp();  // the block has been read
    if (lane == 0 && blk + kFewWarps * L::kSlots < b1) request(blk + kFewWarps * L::kSlots, slot);
    if (++slot == L::kSlots) {
      slot = 0;
      parity ^= 1u;
    }
    const int c = 32 * blk + 8 * t;
    if (m >= 0 && c < a.N) {
      Vec<T, 8> y = *reinterpret_cast<const Vec<T, 8>*>(&ycur);
#pragma unroll
      for (int e = 0; e < 8; ++e) y.v[e] = from_f32<T>(fmaf(f, d[e >> 1][e & 1], to_f32(y.v[e])));
      *reinterpret_cast<Vec<T, 8>*>(orow + c) = y;
    }
  }
  cluster_wait();  // the others may still be reading this CTA's partial sums
}

// Rows that one launch of the kernel above may cover (grid y).
constexpr int64_t kLoraFewMaxRows = 65535;

cudaError_t launch_lora_few(bool bf16, const LoraFewArgs& a, cudaStream_t s) {
  const int64_t chunks = lora_max_tiles(a.M, a.L, kFewRows);
  // Few chunks: several clusters each, which all sum x A^T and share the columns of out, while there are SMs for them
  // and a warp has more than a block of columns (one row of rank 64, 4096 -> 14336: 12.5 us by one cluster, 7.7 by
  // four).
  int64_t q = current_device_info().num_sms / (kFewCluster * chunks);
  const int64_t most = (a.N + 32 * 64 - 1) / (32 * 64);
  q = q > most ? most : q;
  const dim3 grid(kFewCluster, static_cast<unsigned>(chunks), static_cast<unsigned>(q < 1 ? 1 : q));
  return with_type16(bf16, [&](auto t) {
    using T = decltype(t);
    return with_rank(a.rank, [&](auto rp) {
      constexpr int RP = decltype(rp)::value;
      auto* kern = a.rank % (RP < 32 ? 4 : 8) == 0 ? lora_few_kernel<T, RP, true> : lora_few_kernel<T, RP, false>;
      constexpr int kBytes = LoraFewLayout<RP>::kBytes;
      const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), kBytes);
      if (e != cudaSuccess) return e;
      return launch_pdl(kern, grid, dim3(kFewThreads), kBytes, kFewCluster, s, a);
    });
  });
}

constexpr int kLoraGeneric = 3;  // TQ_PATH_GENERIC

static bool lora_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static LoraArgs lora_vectors(LoraArgs a) {
  const bool rows = a.C % 8 == 0;
  a.pvec = rows && lora_aligned(a.P);
  a.wvec = (a.wc == 1 ? rows : a.rank % 8 == 0) && lora_aligned(a.W);
  a.yvec = lora_aligned(a.O) && (a.P || (rows && lora_aligned(a.base)));  // (wgrad has P, and only O)
  return a;
}

cudaError_t launch_lora_reduce(bool bf16, int path, const LoraArgs& a, cudaStream_t s) {
  return path == kLoraGeneric ? lora_generic_reduce(bf16, a, s) : lora_fast_reduce(bf16, lora_vectors(a), s);
}
cudaError_t launch_lora_expand(bool bf16, int path, const LoraArgs& a, cudaStream_t s) {
  return path == kLoraGeneric ? lora_generic_expand(bf16, a, s) : lora_fast_expand(bf16, lora_vectors(a), s);
}
cudaError_t launch_lora_wgrad(bool bf16, int path, const LoraArgs& a, cudaStream_t s) {
  return path == kLoraGeneric ? lora_generic_wgrad(bf16, a, s) : lora_fast_wgrad(bf16, lora_vectors(a), nullptr, s);
}
// Both gradients of the weights, no dropout.
cudaError_t launch_lora_wgrad_both(bool bf16, int path, const LoraArgs& a, const LoraArgs& b, cudaStream_t s) {
  if (path == kLoraGeneric) {
    const cudaError_t e = lora_generic_wgrad(bf16, a, s);
    return e != cudaSuccess ? e : lora_generic_wgrad(bf16, b, s);
  }
  const LoraArgs other = lora_vectors(b);
  return lora_fast_wgrad(bf16, lora_vectors(a), &other, s);
}

}  // namespace tq
