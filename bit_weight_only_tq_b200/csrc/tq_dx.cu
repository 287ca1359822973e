// tq_dx.cu -- the packed products' gradient for x, dx[m, k] = sum_n dy[m, n] What[n, k] (include/tq_lora.h).
//
// The products sum over the packed dimension k; this sums over the rows n, so each decoded weight is needed with n,
// not k, running along the tensor core's summation index.  On the tensor-core path What^T is the A operand in tensor
// memory and dy the B operand:
//   D[k, m] (TMEM, fp32) += A[k, n] (TMEM, fp16) * B[m, n]^T (smem, dy tile, K-major)
// A TMEM lane holds one k and its columns hold pairs of n, while a packed word holds 8 (INT4) or 16 (ternary) k of
// one n.  Eight (sixteen) lanes of a decode warp load the words of as many rows n and exchange them by a butterfly
// (three or four shuffles, each followed by a byte permute or a shift and a mask), after which each lane's word holds
// its own k for 8 (16) consecutive n, in order; it is then decoded as in the products.  That costs 8 instructions per
// 8 INT4 weights and 11 per 16 ternary ones, against a load per weight without the exchange, and no shared-memory
// traffic beyond the packed bytes: a decoded tile in shared memory (MN-major, needing no exchange) would be written
// and read again there, and shared memory already carries the dy tile twice at the tensor core's full rate.
//
// Scales run along n here, two per TMEM column: (c - 1) s is exact in fp16 (ternary); fp16((u - z) s) is one rounding
// per INT4 weight, as in the products' tensor-core path.  It shows in the result, 2.7e-4 off relative rms where the fp16
// rounding of dx alone is 2.1e-4.  The scale cannot wait for the sum, which runs over n as it does, and a scale on dy
// would round that instead; exact weights would take a second part and twice the MMAs.
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
  __half* rows;       // [M][dx_padded(N)] copies of dy's rows (tensor cores, rows that TMA cannot address), or null
  int64_t M, N, K;
};

inline int64_t dx_padded(int64_t N) { return (N + 7) / 8 * 8; }

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

// ---------------------------------------------------------------------------------------------
// Tensor cores.  One CTA = 128 columns k x TN tokens x a range of n, in stages of 64 n:
//   warp 0: TMA of the dy tile (TN tokens x 64 n, 128-byte swizzle); warp 2: TMA of the packed weights, 256 rows x 32
//   bytes (ternary) or 64 bytes (INT4) per tile, swizzled so that the decode warps' loads meet no (INT4) or two-way
//   (ternary) bank conflicts; warp 3: the scales (and zero-points) of those 256 rows, as pairs; warp 1: tensor memory
//   and the MMAs; warps 4-11: two groups of four decode warps on alternate stages.  All twelve run the epilogue.
// Every wait is bounded, as in the products; a whole warp's wait has one result (warp_wait).
// 8192 x 14336 -> 4096 ternary: 680 us, 1414 TFLOP/s (tensor pipe 80 % busy, SM clock 1540 MHz at the power limit);
// 4096 x 4096 -> 14336 INT4 with zero-points: 414 us, 1160 TFLOP/s (64 % busy: a stage's decode ends after its MMAs);
// 61 x 1024 -> 4096 INT4: 8.4 us.  Four groups of decode warps (92 registers instead of 128) are 1 to 10 % slower.
// ---------------------------------------------------------------------------------------------
constexpr int kXM = 128;        // columns k per CTA (UMMA M, TMEM lanes)
constexpr int kXN = 64;         // n per stage
constexpr int kXTileN = 256;    // n per packed tile
constexpr int kXSPP = kXTileN / kXN;
constexpr int kXPRing = 3;
constexpr int kXGroups = 2;     // groups of four decode warps
constexpr int kXThreads = 128 * (1 + kXGroups);
constexpr int kXEpiGroups = 1 + kXGroups;

template <bool kInt4, int TN>
struct DxLayout {
  static constexpr int kRowBytes = kInt4 ? 64 : 32;              // packed bytes of 128 k of a row
  static constexpr int kTileD = TN * kXN * 2;
  static constexpr int kTileP = kXTileN * kRowBytes;
  static constexpr int kTileS = kXTileN / 2 * (kInt4 ? 8 : 4);   // per pair of n: {zero pair,} scale pair
  static constexpr int kRing = TN == 256 ? 4 : 8;                // stages: dy tile in shared memory, weights in TMEM
  static constexpr int kOffP = kRing * kTileD;
  static constexpr int kOffS = kOffP + kXPRing * kTileP;
  static constexpr int kOffBar = kOffS + kXPRing * kTileS;
  // barriers: full[R] (dy landed and weights decoded), empty[R], fullP[3], emptyP[3], accFull; then the TMEM slot
  static constexpr int kNumBars = 2 * kRing + 2 * kXPRing + 1;
  static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffTmemSlot + 16;
  // alignment slack; at least 116 KB so that one CTA runs per SM and none waits for another's tensor memory
  static constexpr int kAlloc = kBytes + 1024 > 116 * 1024 ? kBytes + 1024 : 116 * 1024;
  static constexpr uint32_t kColA = TN;
  static constexpr uint32_t kTmemCols = TN + 32 * kRing <= 256 ? 256u : 512u;
  static_assert(TN + 32 * kRing <= 512, "tensor memory");
  static_assert(kXM * TN * 4 <= kOffP + kXPRing * kTileP, "split partials fit in the rings");
  static_assert(kXEpiGroups * 32 * kXM * 2 <= kRing * kTileD, "staging fits in the dy ring");
  static_assert(kOffP % 1024 == 0 && kTileP % 1024 == 0 && kTileS % 16 == 0 && kAlloc <= 227 * 1024, "shared memory");
};

// One step of a transposition of w-bit fields across lanes: of the pair (x, partner's y) the lane keeps the fields of
// its own side.  16 and 8 bits: a byte permute with a selector of the lane's side; 4 and 2 bits: a rotation and a
// select.
__device__ __forceinline__ uint32_t exchange_bytes(uint32_t x, int d, uint32_t sel) {
  return __byte_perm(x, __shfl_xor_sync(0xFFFFFFFFu, x, d), sel);
}
__device__ __forceinline__ uint32_t exchange_bits(uint32_t x, int d, uint32_t rot, uint32_t mask) {
  const uint32_t y = __shfl_xor_sync(0xFFFFFFFFu, x, d);
  return (x & mask) | (__funnelshift_l(y, y, rot) & ~mask);
}

// 8 INT4 codes of consecutive n -> 8 fp16 (u - z) s; zs: {zero pair, scale pair} of each pair of n.
__device__ __forceinline__ void dx_decode_w4(uint32_t w, const uint4& zs0, const uint4& zs1, uint32_t* v) {
  const uint32_t z[4] = {zs0.x, zs0.z, zs1.x, zs1.z}, s[4] = {zs0.y, zs0.w, zs1.y, zs1.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = hmul2_u32(hsub2_u32((byte_to_halves(w, i) & 0x00F0000Fu) | 0x54006400u, z[i]), s[i]);
}

template <bool kInt4, int TN>
__global__ void __launch_bounds__(kXThreads, 1)
    dx_tc_kernel(const __grid_constant__ CUtensorMap tmap_dy, const __grid_constant__ CUtensorMap tmap_w,
                 const DxArgs a, const int S, const int kt0) {
  using L = DxLayout<kInt4, TN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kOffBar);
  uint64_t* empty = full + L::kRing;
  uint64_t* fullP = empty + L::kRing;
  uint64_t* emptyP = fullP + kXPRing;
  uint64_t* accFull = emptyP + kXPRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::kOffTmemSlot);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kt = kt0 + static_cast<int>(blockIdx.x);  // tile of columns
  const int64_t k0 = static_cast<int64_t>(kt) * kXM, m0 = static_cast<int64_t>(blockIdx.y) * TN;
  const int ns_all = static_cast<int>((a.N + kXN - 1) / kXN);
  const int rank = static_cast<int>(blockIdx.z);  // slice of n = rank in the cluster
  const int s0 = static_cast<int>((static_cast<int64_t>(rank) * ns_all) / S);
  const int ns = static_cast<int>((static_cast<int64_t>(rank + 1) * ns_all) / S) - s0;  // >= 1
  const int npt = (ns + kXSPP - 1) / kXSPP;

  pdl_allow_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kRing; ++i) {
      mbar_init(&full[i], 5);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < kXPRing; ++i) {
      mbar_init(&fullP[i], 2);  // the packed tile's bytes, the scales
      mbar_init(&emptyP[i], 4 * kXGroups);
    }
    mbar_init(accFull, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_prior_grids();

  bool ok = true;
  bool acc_flag = false;
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmap_dy);
      const bool skip = skip_x_loads();  // failure-path test hook: never set in normal use
      for (int i = 0; i < ns && ok && !skip; ++i) {
        const int s = i % L::kRing;
        if (i >= L::kRing) {
          ok = mbar_wait(&empty[s], static_cast<uint32_t>((i / L::kRing) - 1) & 1u);
          if (!ok) break;
        }
        mbar_arrive_expect_tx(&full[s], L::kTileD);
        tma_load_2d(sm + s * L::kTileD, &tmap_dy, &full[s], (s0 + i) * kXN, static_cast<int32_t>(m0));
      }
    }
  } else if (warp == 2) {
    if (lane == 0) {
      tma_prefetch_desc(&tmap_w);
      for (int pt = 0; pt < npt && ok; ++pt) {
        const int s = pt % kXPRing;
        if (pt >= kXPRing) {
          ok = mbar_wait(&emptyP[s], static_cast<uint32_t>((pt / kXPRing) - 1) & 1u);
          if (!ok) break;
        }
        mbar_arrive_expect_tx(&fullP[s], L::kTileP);
        tma_load_2d(sm + L::kOffP + s * L::kTileP, &tmap_w, &fullP[s], kt * L::kRowBytes,
                    (s0 + pt * kXSPP) * kXN);
      }
    }
  } else if (warp == 3) {
    // scales of the tile's 256 rows: eight per lane, loaded before the wait for the slot; rows past N get scale zero
    const int64_t G = a.K >> 7, gi = k0 >> 7;
    for (int pt = 0; pt < npt && ok; ++pt) {
      const int s = pt % kXPRing;
      const int64_t n0 = static_cast<int64_t>(s0 + pt * kXSPP) * kXN + 8 * lane;
      uint32_t sc[8], zp[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t n = n0 + i;
        sc[i] = n < a.N ? __half_as_ushort(a.sc[kInt4 ? n * G + gi : n]) : 0u;
        zp[i] = kInt4 && a.zp && n < a.N ? static_cast<uint32_t>(a.zp[n * G + gi]) : 8u;
      }
      if (pt >= kXPRing) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_relaxed(&emptyP[s], static_cast<uint32_t>((pt / kXPRing) - 1) & 1u)) != 0;
        if (!ok) break;
      }
      uint4* dst = reinterpret_cast<uint4*>(sm + L::kOffS + s * L::kTileS);
      uint32_t s2[4], z2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s2[i] = sc[2 * i] | (sc[2 * i + 1] << 16);
        // (1024 + z, 64 + z) in fp16: what the low and the high nibble of a byte stand above
        z2[i] = (0x6400u + zp[2 * i]) | ((0x5400u + 16u * zp[2 * i + 1]) << 16);
      }
      if (kInt4) {
        dst[2 * lane] = make_uint4(z2[0], s2[0], z2[1], s2[1]);
        dst[2 * lane + 1] = make_uint4(z2[2], s2[2], z2[3], s2[3]);
      } else {
        dst[lane] = make_uint4(s2[0], s2[1], s2[2], s2[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&fullP[s]);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_f16_f32(kXM, TN);
      const uint32_t d_base = smem_u32(sm);
      for (int i = 0; i < ns && ok; ++i) {
        const int s = i % L::kRing;
        ok = mbar_wait(&full[s], static_cast<uint32_t>(i / L::kRing) & 1u);
        if (!ok) break;
        tc_fence_after_sync();
        const uint64_t bdesc = sdesc_kmajor_sw128(d_base + s * L::kTileD);
        const uint32_t a_tmem = tmem + L::kColA + 32 * s;
#pragma unroll
        for (int q = 0; q < kXN / 16; ++q)
          umma_f16_ts(tmem, a_tmem + 8 * q, bdesc + 2 * q, idesc, (i | q) != 0 ? 1u : 0u);
        umma_commit(&empty[s]);
      }
      if (ok) umma_commit(accFull);
    }
  } else {
    // ------------------------------------------------------------------ decode warps
    const int dg = (warp >> 2) - 1, w = warp & 3;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(w * 32) << 16);
    // this lane's word of a block of rows, and its selectors in the exchange
    const int b = kInt4 ? lane & 7 : lane & 15, aw = kInt4 ? lane >> 3 : lane >> 4;
    const uint32_t off = kInt4 ? b * 64 + ((w ^ (b >> 1)) << 4) + 4 * aw
                               : b * 32 + (((w >> 1) ^ ((b >> 2) & 1)) << 4) + 8 * (w & 1) + 4 * aw;
    const bool up16 = (lane & (kInt4 ? 4 : 8)) != 0, up8 = (lane & (kInt4 ? 2 : 4)) != 0;
    const bool up4 = (lane & (kInt4 ? 1 : 2)) != 0, up2 = (lane & 1) != 0;
    const uint32_t sel16 = up16 ? 0x3276u : 0x5410u, sel8 = up8 ? 0x3715u : 0x6240u;
    const uint32_t rot4 = up4 ? 28u : 4u, m4 = up4 ? 0xF0F0F0F0u : 0x0F0F0F0Fu;
    const uint32_t rot2 = up2 ? 30u : 2u, m2 = up2 ? 0xCCCCCCCCu : 0x33333333u;
    for (int i = dg; i < ns && ok; i += kXGroups) {
      const int s = i % L::kRing, pt = i / kXSPP, ci = i - pt * kXSPP, ps = pt % kXPRing;
      if (ci == dg) {  // this group's first stage of the packed tile
        ok = warp_wait(&fullP[ps], static_cast<uint32_t>(pt / kXPRing) & 1u);
        if (!ok) break;
      }
      constexpr int kWords = kInt4 ? 8 : 4;          // words per lane and stage, of 8 or 16 n each
      constexpr int kBlock = kInt4 ? 8 * 64 : 16 * 32;  // bytes of a block of rows
      const uint8_t* tile = sm + L::kOffP + ps * L::kTileP + ci * kXN * L::kRowBytes + off;
      const uint4* zs = reinterpret_cast<const uint4*>(sm + L::kOffS + ps * L::kTileS) + ci * (kInt4 ? 16 : 8);
      uint32_t pw[kWords];
#pragma unroll
      for (int j = 0; j < kWords; ++j) pw[j] = *reinterpret_cast<const uint32_t*>(tile + j * kBlock);
      uint32_t v[32];  // column j = fp16 pair (n = 2j, 2j + 1) of this k
#pragma unroll
      for (int j = 0; j < kWords; ++j) {
        uint32_t x = pw[j];
        if (kInt4) {
          x = exchange_bytes(x, 4, sel16);
          x = exchange_bytes(x, 2, sel8);
          x = exchange_bits(x, 1, rot4, m4);
          dx_decode_w4(x, zs[2 * j], zs[2 * j + 1], v + 4 * j);
        } else {
          x = exchange_bytes(x, 8, sel16);
          x = exchange_bytes(x, 4, sel8);
          x = exchange_bits(x, 2, rot4, m4);
          x = exchange_bits(x, 1, rot2, m2);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 d = decode_tq_8(x, h), sc = zs[2 * j + h];
            v[8 * j + 4 * h] = hmul2_u32(d.x, sc.x);
            v[8 * j + 4 * h + 1] = hmul2_u32(d.y, sc.y);
            v[8 * j + 4 * h + 2] = hmul2_u32(d.z, sc.z);
            v[8 * j + 4 * h + 3] = hmul2_u32(d.w, sc.w);
          }
        }
      }
      // done with this packed tile: both groups arrive on every tile but a CTA's last, which no later load waits for
      if (ci + kXGroups >= kXSPP || i + kXGroups >= ns) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&emptyP[ps]);
      }
      if (i >= L::kRing) {
        ok = warp_wait(&empty[s], static_cast<uint32_t>((i / L::kRing) - 1) & 1u);
        if (!ok) break;
        tc_fence_after_sync();
      }
      tmem_st_32x32b_x32(lane_base + L::kColA + 32 * s, v);
      tmem_st_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
    }
    acc_flag = ok && warp_wait(accFull, 0u);
  }

  // ------------------------------------------------------------------ epilogue (all warps)
  // Groups of four warps take 32-token chunks of the accumulator in turn; a warp reads TMEM lanes 32 (warp % 4) .. +
  // 31, i.e. column k0 + threadIdx.x % 128.
  if (threadIdx.x == 128) tmem_slot[1] = acc_flag ? 1u : 0u;
  __syncwarp();
  named_barrier_sync(1 + kXEpiGroups, kXThreads);
  const bool acc_ok = tmem_slot[1] != 0u;
  tc_fence_after_sync();
  {
    const int grp = ((warp >> 2) + kXEpiGroups - 1) % kXEpiGroups;
    const int r = threadIdx.x & (kXM - 1);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // dx[m0 + t0 + t, k0 ..] for t < cnt (<= 32) from this group's staging buffer [cnt][128] fp16; K is a multiple of
    // 64
    auto store_staged = [&](const __half* stage, int t0, int cnt) {
      named_barrier_sync(1 + grp, 128);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int idx = r + 128 * q, tok = idx >> 4, ch = idx & 15;
        const int64_t m = m0 + t0 + tok, kb = k0 + ch * 8;
        if (tok < cnt && m < a.M && kb < a.K)
          *reinterpret_cast<uint4*>(a.dx + m * a.K + kb) = *reinterpret_cast<const uint4*>(stage + tok * kXM + ch * 8);
      }
      named_barrier_sync(1 + grp, 128);
    };
    auto load_chunk = [&](int c, uint32_t (&rr)[32]) {
      if (acc_ok) {
        tmem_ld_32x32b_x32(lane_base + c * 32, rr);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) rr[j] = 0u;
      }
    };
    if (S == 1) {
      __half* stage = reinterpret_cast<__half*>(sm) + grp * 32 * kXM;
#pragma unroll 1
      for (int c = grp; c < TN / 32 && acc_ok; c += kXEpiGroups) {
        uint32_t rr[32];
        load_chunk(c, rr);
#pragma unroll
        for (int j = 0; j < 32; ++j) stage[j * kXM + r] = __float2half_rn(__uint_as_float(rr[j]));
        store_staged(stage, c * 32, 32);
      }
    } else {
      // the tokens are split over the S CTAs of the cluster (TN / S each); each CTA sends its partial sums of the
      // others' tokens into their shared memory, [source rank][token / 4][k][token % 4] fp32, and adds those of its
      // own in rank order
      const int tpo = TN / S, own0 = rank * tpo, own1 = own0 + tpo;
      float* red = reinterpret_cast<float*>(sm);
      const uint32_t red_local = smem_u32(red);
      auto slot = [&](int src, int tl) { return ((src * (tpo >> 2) + (tl >> 2)) * kXM + r) * 4; };
      cluster_arrive();  // every CTA of the cluster is past its main loop: the rings are free
      cluster_wait();
#pragma unroll 1
      for (int c = grp; c < TN / 32; c += kXEpiGroups) {
        if (c * 32 >= own0 && c * 32 + 32 <= own1) continue;
        uint32_t rr[32];
        load_chunk(c, rr);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const int tok = c * 32 + j, q = tok / tpo;
          if (q != rank) {
            const uint32_t dst = red_local + 4u * static_cast<uint32_t>(slot(rank, tok - q * tpo));
            st_shared_cluster_v4_f32(mapa_shared(dst, static_cast<uint32_t>(q)), rr[j], rr[j + 1], rr[j + 2],
                                     rr[j + 3]);
          }
        }
      }
      cluster_arrive();  // all partials have landed
      cluster_wait();
      // group g stages at 8 g KB of the own slot (no CTA writes there), used only with more than g own chunks
      const int oc0 = own0 / 32;
      __half* stage = reinterpret_cast<__half*>(red + static_cast<size_t>(own0) * kXM) + grp * 32 * kXM;
#pragma unroll 1
      for (int c = oc0 + grp; c * 32 < own1; c += kXEpiGroups) {
        const int b0 = max(c * 32, own0), b1 = min(c * 32 + 32, own1);
        uint32_t rr[32];
        load_chunk(c, rr);
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
        for (int src = 0; src < S; ++src) {
          if (src == rank) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += __uint_as_float(rr[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const int tok = c * 32 + j;
              if (tok >= b0 && tok < b1) {
                const float4 p = *reinterpret_cast<const float4*>(red + slot(src, tok - own0));
                v[j] += p.x;
                v[j + 1] += p.y;
                v[j + 2] += p.z;
                v[j + 3] += p.w;
              }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int tok = c * 32 + j;
          if (tok >= b0 && tok < b1 && acc_ok) stage[(tok - b0) * kXM + r] = __float2half_rn(v[j]);
        }
        store_staged(stage, b0, b1 - b0);
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

template <bool kInt4, int TN>
static cudaLaunchConfig_t dx_config(dim3 grid, cudaStream_t s, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kXThreads, 1, 1);
  cfg.dynamicSmemBytes = DxLayout<kInt4, TN>::kAlloc;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = grid.z;
  cfg.attrs = attr;
  cfg.numAttrs = grid.z > 1 ? 2 : 1;
  return cfg;
}

// rows[m, 0 .. padded) = dy[m, 0 .. N), zeros: a warp per 256 elements.
__global__ void __launch_bounds__(256) dx_rows_kernel(const __half* dy, __half* rows, int64_t M, int64_t N,
                                                      int64_t padded) {
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31;
  const int64_t segments = (padded + 255) >> 8;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5; i < M * segments;
       i += (static_cast<int64_t>(gridDim.x) * 256) >> 5) {
    const int64_t m = i / segments, c0 = (i - m * segments) << 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c = c0 + 32 * e + lane;
      if (c < padded) rows[m * padded + c] = c < N ? dy[m * N + c] : __float2half_rn(0.0f);
    }
  }
}

// Clusters of S CTAs that can be resident at once, queried once per device and S; 0 when unknown.
template <bool kInt4, int TN>
static int dx_cluster_capacity(int device, int S) {
  static std::atomic<int> cache[kPfMaxDevices][4];
  if (device < 0 || device >= kPfMaxDevices || S < 2 || S > 8) return 0;
  std::atomic<int>& slot = cache[device][S == 2 ? 1 : (S == 4 ? 2 : 3)];
  int n = slot.load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = dx_config<kInt4, TN>(dim3(1, 1, static_cast<unsigned>(S)), nullptr, attr);
  cfg.attrs = attr + 1;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, dx_tc_kernel<kInt4, TN>, &cfg) != cudaSuccess || n <= 0) {
    (void)cudaGetLastError();
    return 0;
  }
  slot.store(n, std::memory_order_relaxed);
  return n;
}

template <bool kInt4, int TN>
static cudaError_t launch_dx_tc(const DxArgs& a, cudaStream_t s) {
  using L = DxLayout<kInt4, TN>;
  auto* kern = dx_tc_kernel<kInt4, TN>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), L::kAlloc);
  if (e != cudaSuccess) return e;
  const __half* dy = a.rows ? a.rows : a.dy;
  const int64_t width = a.rows ? dx_padded(a.N) : a.N;
  if (a.rows) {
    e = launch_pdl(dx_rows_kernel, dim3(lora_grid((a.M * ((width + 255) >> 8) + 7) / 8, 16)), dim3(256), 0, 1, s, a.dy,
                   a.rows, a.M, a.N, width);
    if (e != cudaSuccess) return e;
  }
  CUtensorMap td, tw;
  const uint64_t kbytes = static_cast<uint64_t>(a.K) / (kInt4 ? 2 : 4);
  if (!make_tmap_2d(&td, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dy, static_cast<uint64_t>(width), static_cast<uint64_t>(a.M),
                    static_cast<uint64_t>(width) * 2, kXN, TN, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, kbytes, static_cast<uint64_t>(a.N), kbytes, L::kRowBytes,
                    kXTileN, kInt4 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B))
    return cudaErrorInvalidValue;
  const DeviceInfo di = current_device_info();
  const int64_t kt = (a.K + kXM - 1) / kXM, mt = (a.M + TN - 1) / TN, ns = (a.N + kXN - 1) / kXN;
  auto capacity = [&](int cs) { return dx_cluster_capacity<kInt4, TN>(di.device, cs); };
  auto run = [&](int64_t first, int64_t last, int S) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = dx_config<kInt4, TN>(
        dim3(static_cast<unsigned>(last - first), static_cast<unsigned>(mt), static_cast<unsigned>(S)), s, attr);
    return cudaLaunchKernelEx(&cfg, kern, td, tw, a, S, static_cast<int>(first));
  };
  // n split over a cluster while the tiles leave SMs idle and all clusters are resident at once, and a nearly empty
  // last wave split off into a launch of its own, as in the products
  int S = 1;
  while (S < 8 && kt * mt * S * 2 <= di.num_sms && S * 2 <= ns) {
    const int cap = capacity(S * 2);
    if (cap > 0 && kt * mt > cap) break;
    S *= 2;
  }
  if (S == 1) {
    const PrefillTailPlan tp = prefill_tail_plan(kt, mt, static_cast<int>(ns), di.num_sms, capacity);
    if (tp.rows_main > 0) {
      e = run(0, tp.rows_main, tp.Sm);
      return e != cudaSuccess ? e : run(tp.rows_main, kt, tp.St);
    }
  }
  return run(0, kt, S);
}

bool dx_supported(int64_t M, int64_t N, int64_t K) {
  return N > 0 && K % 64 == 0 && (M + 63) / 64 <= 65535;
}

// Tiles of 64, 128 or 256 tokens, as in the products: an MMA of fewer columns costs as much as one of 64.
cudaError_t launch_dx(bool int4, int path, const DxArgs& a, cudaStream_t s) {
  if (path != 2) return launch_dx_generic(int4, a, s);
  const int tn = prefill_tile_tokens(a.M);
  if (int4)
    return tn == 64 ? launch_dx_tc<true, 64>(a, s)
                    : (tn == 128 ? launch_dx_tc<true, 128>(a, s) : launch_dx_tc<true, 256>(a, s));
  return tn == 64 ? launch_dx_tc<false, 64>(a, s)
                  : (tn == 128 ? launch_dx_tc<false, 128>(a, s) : launch_dx_tc<false, 256>(a, s));
}

}  // namespace tq
