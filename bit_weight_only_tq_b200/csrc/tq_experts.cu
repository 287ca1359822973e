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
  __half* rows;            // [R][K] scratch, or null (PREFILL with order needs it)
  int64_t X, R, N, K;
  int E, top_k;
};

// A named barrier of whole warps, each converged first (bar.sync is warp-aligned).
__device__ __forceinline__ void warps_barrier(int id, int nthreads) {
  __syncwarp();
  named_barrier_sync(id, nthreads);
}

__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// The x row of sorted row r, or -1.
__device__ __forceinline__ int64_t expert_x_row(const ExpertArgs& a, int64_t r) {
  if (!a.order) return r < a.X ? r : -1;
  const int slot = a.order[r], t = slot / a.top_k;
  return slot >= 0 && t < a.X ? t : -1;
}

// offsets[e], clamped to [0, R].
__device__ __forceinline__ int expert_bound(const ExpertArgs& a, int e) {
  const int64_t o = a.offsets[e];
  return static_cast<int>(o < 0 ? 0 : (o < a.R ? o : a.R));
}

// ---------------------------------------------------------------------------------------------
// Any shape and alignment: one warp per (row, 32 outputs), lanes over k, one output at a time with the weights
// read by bytes: shapes and addresses that the other kernels cannot take (K % 64, unaligned views), and their
// check.  8 experts, 4096 -> 2048, 16 rows: 361 us INT4, 209 us ternary, where DECODE takes 15 and 13.
// ---------------------------------------------------------------------------------------------
template <bool kInt4>
__global__ void __launch_bounds__(256) experts_generic_kernel(const ExpertArgs a) {
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31;
  const int64_t nb = (a.N + 31) / 32, row0 = expert_bound(a, 0);
  const int64_t rows = expert_bound(a, a.E) - row0, G = a.K / 128;
  const int64_t row_bytes = kInt4 ? a.K / 2 : (a.K + 3) / 4;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t task = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); task < rows * nb; task += step) {
    const int64_t r = row0 + task / nb, n0 = task % nb * 32;
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

// rows[r] = x[row(r)] for offsets[0] <= r < offsets[E]: a warp per 2 KB.  Not tq_moe_gather's kernel, which
// leaves the row of a slot outside x as it was: here it has to read as zeros.
__global__ void __launch_bounds__(256) experts_rows_kernel(const ExpertArgs a) {
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int lane = threadIdx.x & 31;
  const int64_t row0 = expert_bound(a, 0), nv = a.K / 8, segs = (nv + 127) / 128;
  const int64_t tasks = (expert_bound(a, a.E) - row0) * segs, step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); w < tasks; w += step) {
    const int64_t r = row0 + w / segs, v0 = w % segs * 128 + lane;
    const int64_t xr = expert_x_row(a, r);
    uint4 b[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      b[u] = xr >= 0 && v0 + 32 * u < nv ? reinterpret_cast<const uint4*>(a.x)[xr * nv + v0 + 32 * u]
                                         : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (v0 + 32 * u < nv) reinterpret_cast<uint4*>(a.rows)[r * nv + v0 + 32 * u] = b[u];
  }
}

static cudaError_t launch_experts_rows(const ExpertArgs& a, cudaStream_t s) {
  const int64_t segs = (a.K / 8 + 127) / 128;
  return launch_pdl(experts_rows_kernel, dim3(row_grid(a.R * segs, 8, 8)), dim3(256), 0, 1, s, a);
}

// ---------------------------------------------------------------------------------------------
// The expert chunks of a launch: expert e's rows are cut into ceil(rows / TM) chunks of up to TM.
// first[e] = chunks of the experts before e (E + 1 entries in shared memory), from the offsets
// clamped to [0, R]; called by all nt threads of the CTA (nt <= 1024), scratch holds nt / 32 ints.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void expert_chunks(const ExpertArgs& a, int TM, int* first, int* scratch, int nt) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = (a.E + nt - 1) / nt;
  const int e0 = tid * P, e1 = e0 + P < a.E ? e0 + P : a.E;
  int sum = 0;
  int prev = e0 < a.E ? expert_bound(a, e0) : 0;
  for (int e = e0; e < e1; ++e) {
    const int next = expert_bound(a, e + 1);
    first[e] = sum;
    sum += next > prev ? (next - prev - 1) / TM + 1 : 0;  // rows + TM - 1 could pass an int
    prev = next;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  int base = incl - sum, total = 0;
  for (int w = 0; w < nt >> 5; ++w) {
    if (w < warp) base += scratch[w];
    total += scratch[w];
  }
  for (int e = e0; e < e1; ++e) first[e] += base;
  if (tid == 0) first[a.E] = total;
  __syncthreads();
}

// Work item `item` of a launch with `tiles` row tiles per expert: an expert's items run over its
// chunks first, so that the chunks which share a weight tile run close together.
struct ExpertItem {
  int e, tile, row0, rows;  // expert, row tile of its weights, first sorted row, number of rows
};
// kEven: an expert's chunks hold about the same number of rows (a multiple of 16), else TM each.
template <bool kEven>
__device__ __forceinline__ ExpertItem expert_item(const ExpertArgs& a, const int* first, int64_t item, int64_t tiles,
                                                  int TM) {
  int lo = 0, hi = a.E;  // first[lo] tiles <= item < first[lo + 1] tiles
  const int chunk_at = (item | tiles) >> 31 == 0
                           ? static_cast<int>(static_cast<uint32_t>(item) / static_cast<uint32_t>(tiles))
                           : static_cast<int>(item / tiles);
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= chunk_at)
      lo = mid;
    else
      hi = mid;
  }
  const int c = first[lo + 1] - first[lo];
  const int local = static_cast<int>(item - first[lo] * tiles);
  ExpertItem it;
  it.e = lo;
  it.tile = local / c;
  const int b0 = expert_bound(a, lo), b1 = expert_bound(a, lo + 1);
  const int size = kEven ? ((b1 - b0 - 1) / c + 16) / 16 * 16 : TM;
  it.row0 = b0 + (local - it.tile * c) * size;
  it.rows = b1 - it.row0 < size ? b1 - it.row0 : size;
  return it;
}

// (v & mask) | base in one instruction: with both constants written out the compiler spends two, and
// constants that it sees as uniform it moves into place for every use.  They come from shared memory.
struct DecodeConsts {  // natural order, from a byte in both halves: see decode_tq_8, w4_zero_pair
  uint32_t mask0, base0, mask1, base1;
};
__device__ __forceinline__ void store_decode_consts(bool int4, uint32_t* c) {  // four words
  c[0] = int4 ? 0x00F0000Fu : 0x000C0003u;
  c[1] = int4 ? 0x54006400u : 0x5C006400u;
  c[2] = 0x00C00030u;
  c[3] = 0x4C005400u;
}
__device__ __forceinline__ DecodeConsts load_decode_consts(const uint32_t* c) {
  const volatile uint32_t* v = c;
  return DecodeConsts{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t base) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(base));
  return r;
}
struct FieldConsts {  // fields i and i + 4 (i + 8) of a word: mask and base of the i-th
  uint32_t mask[4], base[4];
};
__device__ __forceinline__ void store_field_consts(bool int4, uint32_t* c) {  // eight words
  c[0] = int4 ? 0x000F000Fu : 0x00030003u;
  c[1] = int4 ? 0x00F000F0u : 0x000C000Cu;
  c[2] = 0x00300030u;
  c[3] = 0x00C000C0u;
  c[4] = 0x64006400u;                          // 1024: unit in the lowest bits
  c[5] = int4 ? 0x54005400u : 0x5C005C00u;     // 64 (four bits up) or 256 (two)
  c[6] = 0x54005400u;
  c[7] = 0x4C004C00u;                          // 16
}
__device__ __forceinline__ FieldConsts load_field_consts(const uint32_t* c) {
  const volatile uint32_t* v = c;
  return FieldConsts{{v[0], v[1], v[2], v[3]}, {v[4], v[5], v[6], v[7]}};
}

// ---------------------------------------------------------------------------------------------
// Few rows per expert: the packed weights' bytes are the floor.  Persistent CTAs; an item is 128 weight
// rows of one expert times up to 8 of its rows, all of K.  One producer warp keeps a ring
// of stages full: 128 weight rows x 128 packed bytes by TMA (128-byte swizzle) and the rows' x by
// one bulk copy each, running ahead across items.  Consumer warps form KG groups of four that take
// the CTA's stages in turn (the ring is a multiple of KG long, so that a slot has one consumer
// group, which sees every phase of its barriers); warp w of a group takes the weight rows 32 w ..
// 32 w + 31, on mma.sync m16n8k16 with the decoded weights as A (16 weight rows) and x as B (8
// rows of x).
//
// The order of k within a product is free as long as both operands share it.  Lane (g, t) =
// (lane / 4, lane % 4) takes 16 packed bytes of its weight rows -- 32 INT4 or 64 ternary codes of
// consecutive k -- and the same k of x.  A 32-bit word is decoded with masks alone: nibbles (or
// 2-bit codes) i and i + 4 (i + 8) land in the two halves of a register, in a place of the
// fraction where their weight is 1 over a base of 1024, 256, 64 or 16; one fp16x2 subtraction
// takes the base (and the zero-point) off, exactly.  x is brought into the same pairs by byte
// permutes, once per warp for 32 weight rows.
//
// An item may also be 64 weight rows with stages of twice the k (wide): the same bytes per stage, two
// warps on each half of its k, whose sums are added with the groups'.  Half as many stages are in
// flight then, since x takes twice the room.
//
// Bank conflicts: rows of x are 16 bytes apart modulo 128, and lane t's x starts 64 (128) bytes after
// lane t - 1's: two lanes share banks (four, and so the odd ternary lanes take their words in pairs
// the other way round).  Ordering the words of all lanes apart took two selects per MMA, which cost more
// than the shared memory's extra cycles.  Weight row of lane group g is (g / 2) + 4 (g % 2), so that the two
// rows of a quarter-warp access differ in the swizzle's top bit.
//
// One row for each of 8 experts, 4096 -> 14336: INT4 61 us, 4.0 TB/s of packed weights and scales,
// ternary 51 us, 2.3 TB/s; issue 57 and 52 %, ALU 50 and 53 % busy.  No unit is full: the four or so warps
// of a scheduler wait for a stage, then decode at the same time.  Of 6.9 (7.0) warp cycles per instruction 1.2
// (1.2) wait for a barrier, shared or global memory (long scoreboard), 1.2 (1.4) for the ALU, 1.4 (1.3) were
// ready and not selected, 0.8 (0.7) are fixed latencies, 0.6 (0.7) dispatch.  A token's 8 of 64 experts,
// 2048 -> 2816, INT4 with zero-points: 13.2 us, of which the weights' bytes take 3.7: launch, chunk table, first
// loads and the last sums are not overlapped with anything.
// ---------------------------------------------------------------------------------------------
constexpr int kERows = 128;       // weight rows per item
constexpr int kEItems = 4;        // item descriptors in flight

// Two CTAs per SM with KG = 2, or, for few items (a token's experts), one with KG = 4: an item then has
// the warps of the whole SM.
template <bool kInt4, int KG>
struct SkinnyLayout {
  static constexpr int TM = 8;
  static constexpr int kConsumers = 128 * KG;
  static constexpr int kThreads = kConsumers + 32;
  static constexpr int kCtasPerSm = 4 / KG;
  static constexpr int KS = kInt4 ? 256 : 512;         // k per stage
  static constexpr int kLogKS = kInt4 ? 8 : 9;
  static constexpr int kXRow = KS * 2 + 16;            // bytes between rows of x
  static constexpr int kTileW = kERows * 128;
  static constexpr int kTileX = TM * kXRow;
  static constexpr int kPart = TM * 132 * 4;           // one group's sums [TM][132] fp32
  static constexpr int kRing = 2 * KG;                 // stages of an item of 128 weight rows; half for 64
  static constexpr int kLogRing = KG == 4 ? 3 : 2;
  static constexpr bool kWide = KG == 4;
  static constexpr int kOffX = kRing * kTileW;
  static constexpr int kOffPart = kOffX + kRing * kTileX;
  static constexpr int kOffBar = kOffPart + KG * kPart;
  static constexpr int kOffItem = kOffBar + 2 * (kRing + kEItems) * 8;
  static constexpr int kOffScan = kOffItem + kEItems * 32;  // descriptors of 32 bytes
  static constexpr int kOffConst = kOffScan + 32 * 4;       // FieldConsts
  static constexpr int kOffFirst = kOffConst + 32;
  static constexpr int bytes(int E) { return kOffFirst + (E + 1) * 4 + 1024; }  // 1024: alignment
  static_assert(kRing == 1 << kLogRing && kRing % KG == 0, "ring");
  static_assert(!kWide || (kRing / 2 % KG == 0 && kRing / 2 * TM * (2 * KS * 2 + 16) <= kRing * kTileX), "wide items");
  static_assert(kOffFirst + 1025 * 4 + 1024 <= 227 * 1024 / kCtasPerSm, "shared memory");
};

__device__ __forceinline__ uint32_t sel(bool c, uint32_t a, uint32_t b) { return c ? a : b; }

template <bool kInt4, int KG>
__global__ void __launch_bounds__(SkinnyLayout<kInt4, KG>::kThreads, SkinnyLayout<kInt4, KG>::kCtasPerSm)
    experts_skinny_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_h,
                          const ExpertArgs a) {
  using L = SkinnyLayout<kInt4, KG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kOffBar);
  uint64_t* empty = full + L::kRing;
  uint64_t* item_full = empty + L::kRing;
  uint64_t* item_empty = item_full + kEItems;
  int4* items = reinterpret_cast<int4*>(sm + L::kOffItem);  // [kEItems][2]: (e, tile, row0, rows), (row mask, ...)
  int* scan = reinterpret_cast<int*>(sm + L::kOffScan);
  int* first = reinterpret_cast<int*>(sm + L::kOffFirst);
  // values that steer the roles are broadcast, so that the compiler knows them to be warp-uniform
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  pdl_allow_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kRing; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);  // the four warps of the group that takes the stage
    }
    for (int i = 0; i < kEItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], 4 * KG);
    }
    store_field_consts(kInt4, reinterpret_cast<uint32_t*>(sm + L::kOffConst));
    fence_mbar_init();
    tma_prefetch_desc(&tmap_w);
    tma_prefetch_desc(&tmap_h);
  }
  pdl_wait_prior_grids();
  const bool skipx = skip_x_loads();  // failure-path test hook: never set in normal use
  expert_chunks(a, L::TM, first, scan, L::kThreads);
  // Tall items of 128 weight rows, or wide ones of 64 with stages of twice the k, where those end sooner:
  // a round of wide items takes half as long (64 tall items of 14336 k: 34.5 -> 21.8 us INT4, 25.3 ->
  // 15.2 us ternary; 160: 68 -> 57 and 50 -> 43 us).  Not with two CTAs per SM, which share it unevenly where
  // one has an item more (896 items of 4096 k: 65 -> 70 us INT4).  Numbers of items fit 32 bits by far: y has
  // to fit memory.
  const uint32_t chunks = static_cast<uint32_t>(uniform(first[a.E])), n32 = static_cast<uint32_t>(a.N);
  const uint32_t tall = chunks * ((n32 + kERows - 1) / kERows), wides = chunks * ((n32 + kERows / 2 - 1) / (kERows / 2));
  const int wide = L::kWide && uniform((wides + gridDim.x - 1) / gridDim.x < 2 * ((tall + gridDim.x - 1) / gridDim.x));
  const int tile_rows = kERows >> wide, ring = L::kRing >> wide, xrow = wide ? 2 * L::KS * 2 + 16 : L::kXRow;
  const int ks = L::KS << wide;  // k per stage
  const int64_t tiles = (n32 + tile_rows - 1) >> (7 - wide);
  const int64_t total = wide ? wides : tall;
  const int nk = static_cast<int>((static_cast<uint32_t>(a.K) + ks - 1) >> (L::kLogKS + wide));
  bool ok = true;
  // A stage's weights: 128 rows x 128 bytes, or (wide) two boxes of 64 rows side by side.
  auto load_weights = [&](int s, int kb, int wrow) {
    uint8_t* dst = sm + s * L::kTileW;
    if (wide) {
      tma_load_2d(dst, &tmap_h, &full[s], kb * 256, wrow);
      tma_load_2d(dst + L::kTileW / 2, &tmap_h, &full[s], kb * 256 + 128, wrow);
    } else {
      tma_load_2d(dst, &tmap_w, &full[s], kb * 128, wrow);
    }
  };

  if (warp == KG * 4) {
    // ------------------------------------------------------------------ producer
    // The first item's weights are requested before its rows are looked up; their barriers complete
    // with the arrivals that add the rows' bytes.
    int q = 0, n = 0;
    for (int64_t item = blockIdx.x; item < total && ok; item += gridDim.x, ++n) {
      const ExpertItem it = expert_item<false>(a, first, item, tiles, L::TM);
      const int wrow = static_cast<int>(static_cast<int64_t>(it.e) * a.N + static_cast<int64_t>(it.tile) * tile_rows);
      const int early = n == 0 ? (nk < ring ? nk : ring) : 0;
      if (lane < early) {
        mbar_expect_tx(&full[lane], L::kTileW);
        load_weights(lane, lane, wrow);
      }
      __syncwarp();
      int64_t xr = -1;
      if (lane < it.rows) xr = expert_x_row(a, it.row0 + lane);
      const uint32_t mask = __ballot_sync(0xFFFFFFFFu, xr >= 0);
      const uint8_t* src = reinterpret_cast<const uint8_t*>(a.x + (xr >= 0 ? xr * a.K : 0));
      const int d = n % kEItems;
      if (n >= kEItems) ok = mbar_wait_relaxed(&item_empty[d], static_cast<uint32_t>(n / kEItems - 1) & 1u);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      if (lane == 0) {
        items[d * 2] = make_int4(it.e, it.tile, it.row0, it.rows);
        items[d * 2 + 1].x = static_cast<int>(mask);
        mbar_arrive(&item_full[d]);
      }
      for (int kb = 0; kb < nk && ok; ++kb, ++q) {
        const int s = q & (ring - 1), lap = q >> (L::kLogRing - wide);
        if (q >= ring) ok = mbar_wait_relaxed(&empty[s], static_cast<uint32_t>(lap - 1) & 1u);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const int64_t k0 = static_cast<int64_t>(kb) * ks;
        const uint32_t xb = static_cast<uint32_t>((a.K - k0 < ks ? a.K - k0 : ks) * 2);
        if (lane == 0) {
          mbar_arrive_expect_tx(&full[s], (kb >= early ? L::kTileW : 0) + __popc(mask) * xb);
          if (kb >= early) load_weights(s, kb, wrow);
        }
        __syncwarp();
        if (xr >= 0 && !skipx)
          bulk_load_1d(sm + L::kOffX + (s * L::TM + lane) * xrow, src + k0 * 2, xb, &full[s]);
      }
    }
  } else {
    // ------------------------------------------------------------------ consumers
    const int kg = warp >> 2, rg = warp & 3;
    // the warp's first weight row in the tile, and (wide) which half of the stage's k it takes
    const int wr0 = wide ? (rg & 1) * 32 : rg * 32, kh = wide ? rg >> 1 : 0;
    const int g = lane >> 2, t = lane & 3;
    const int pg = (g >> 1) | ((g & 1) << 2);  // weight row of this lane group within 8
    const int64_t G = a.K >> 7;
    const bool odd = (t & 1) != 0;
    // two groups' scales (zero-points) in one load: whole pairs per row, aligned
    const bool pairs = (G & 1) == 0 && (reinterpret_cast<uintptr_t>(a.sc) & 3u) == 0 &&
                       (reinterpret_cast<uintptr_t>(a.zp) & 1u) == 0;
    const FieldConsts fc = load_field_consts(reinterpret_cast<const uint32_t*>(sm + L::kOffConst));
    float* part = reinterpret_cast<float*>(sm + L::kOffPart);
    int q0 = 0, n = 0;  // stages before this item; items before it
    for (int64_t item = blockIdx.x; item < total; item += gridDim.x, ++n, q0 += nk) {
      float acc[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][c] = 0.0f;
      const int d = n % kEItems;
      if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait_warp(&item_full[d], static_cast<uint32_t>(n / kEItems) & 1u));
      const int4 it = items[d * 2];
      const uint32_t rmask = static_cast<uint32_t>(items[d * 2 + 1].x);
      __syncwarp();
      if (lane == 0) mbar_arrive(&item_empty[d]);
      const int64_t n0 = static_cast<int64_t>(it.y) * tile_rows;
      const int64_t en0 = static_cast<int64_t>(it.x) * a.N;
      // the group scales (and zero-points) of this lane's four weight rows, loaded one of the
      // group's stages ahead: two fp16 per register, the eight zero-points as nibbles of one
      const __half* const sct = a.sc + (kInt4 && ok ? (en0 + n0) * G : 0);
      const uint8_t* const zpt = kInt4 && a.zp ? a.zp + (ok ? (en0 + n0) * G : 0) : nullptr;
      int rowG[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = wr0 + 8 * j + pg;
        rowG[j] = ok && n0 + r < a.N ? static_cast<int>(r * G) : 0;  // past N: any scale, not stored
      }
      uint32_t sc[4] = {0u, 0u, 0u, 0u}, zp = 0x88888888u;
      auto load_scales = [&](int kb) {
        const int g0 = 2 * ((kb << wide) + kh);
        if (g0 >= G) return;  // nothing of the stage in this half
        if (pairs) {
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[j] = *reinterpret_cast<const uint32_t*>(sct + rowG[j] + g0);
          if (zpt) {
            zp = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t z = *reinterpret_cast<const uint16_t*>(zpt + rowG[j] + g0);
              zp |= ((z & 15u) | ((z >> 4) & 0xF0u)) << (8 * j);
            }
          }
          return;
        }
        const bool two = g0 + 1 < G;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half* p = sct + rowG[j] + g0;
          sc[j] = __half_as_ushort(p[0]) | (two ? static_cast<uint32_t>(__half_as_ushort(p[1])) << 16 : 0u);
        }
        if (zpt) {
          zp = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint8_t* p = zpt + rowG[j] + g0;
            zp |= (p[0] & 15u) << (8 * j) | (two ? (p[1] & 15u) << (8 * j + 4) : 0u);
          }
        }
      };
      const int kb0 = (kg + KG - q0 % KG) % KG;  // the group's first stage of the item
      if (kInt4 && kb0 < nk) load_scales(kb0);
      for (int kb = kb0; kb < nk && ok; kb += KG) {
        const int q = q0 + kb, s = q & (ring - 1), lap = q >> (L::kLogRing - wide);
        uint32_t sc_now[4];
        const uint32_t zp_now = zp;
        if (kInt4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) sc_now[j] = sc[j];
          if (kb + KG < nk) load_scales(kb + KG);
        }
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_warp(&full[s], static_cast<uint32_t>(lap) & 1u));
        if (!ok) break;
        const uint8_t* wt = sm + s * L::kTileW + (rg * 32 + pg) * 128;  // either way: two boxes of 64 rows
        const uint8_t* xt = sm + L::kOffX + (s * L::TM + g) * xrow + kh * (L::KS * 2);
        // 16-byte chunks of a row that hold weights: all eight but in the last stage
        const int64_t left = a.K - static_cast<int64_t>(kb) * ks - kh * L::KS;
        const int live = left >= L::KS ? 8 : (left > 0 ? static_cast<int>(left / (kInt4 ? 32 : 64)) : 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (4 * i >= live) break;
          const bool in = 4 * i + t < live;  // always for INT4 (whole groups)
          uint4 w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w[j] = *reinterpret_cast<const uint4*>(wt + j * 8 * 128 + (((4 * i + t) ^ pg) << 4));
            if (!kInt4) {  // this lane takes word p ^ (t & 1)
              const uint4 u = w[j];
              w[j] = make_uint4(sel(odd, u.y, u.x), sel(odd, u.x, u.y), sel(odd, u.w, u.z), sel(odd, u.z, u.w));
            }
          }
          float grp[2][4];
          uint32_t zl[4], zh[4];  // 1024 + z and 64 + z
          if (kInt4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t z = ((zp_now >> (8 * j + 4 * i)) & 15u) * 0x00010001u;
              zl[j] = 0x64006400u + z;
              zh[j] = 0x54005400u + (z << 4);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int c = 0; c < 4; ++c) grp[m][c] = 0.0f;
          }
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            uint32_t wd[4] = {(&w[0].x)[p], (&w[1].x)[p], (&w[2].x)[p], (&w[3].x)[p]};
            if (kInt4) {
              uint32_t d[4][4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t v = wd[j], v8 = v >> 8;
                d[j][0] = hsub2_u32(and_or(v, fc.mask[0], fc.base[0]), zl[j]);
                d[j][1] = hsub2_u32(and_or(v, fc.mask[1], fc.base[1]), zh[j]);
                d[j][2] = hsub2_u32(and_or(v8, fc.mask[0], fc.base[0]), zl[j]);
                d[j][3] = hsub2_u32(and_or(v8, fc.mask[1], fc.base[1]), zh[j]);
              }
              const int piece = 4 * (4 * i + t) + p;
              const uint4 x = *reinterpret_cast<const uint4*>(xt + piece * 16);
              const uint32_t b0 = __byte_perm(x.x, x.z, 0x5410), b1 = __byte_perm(x.x, x.z, 0x7632);
              const uint32_t b2 = __byte_perm(x.y, x.w, 0x5410), b3 = __byte_perm(x.y, x.w, 0x7632);
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                mma_16816(grp[m], d[2 * m][0], d[2 * m + 1][0], d[2 * m][1], d[2 * m + 1][1], b0, b1);
                mma_16816(grp[m], d[2 * m][2], d[2 * m + 1][2], d[2 * m][3], d[2 * m + 1][3], b2, b3);
              }
            } else {
              const int piece = 8 * (4 * i + t) + 2 * (p ^ (t & 1));
              const uint8_t* xp = xt + piece * 16;
              const uint4 x0 = in ? *reinterpret_cast<const uint4*>(xp) : make_uint4(0u, 0u, 0u, 0u);
              const uint4 x1 = in ? *reinterpret_cast<const uint4*>(xp + 16) : make_uint4(0u, 0u, 0u, 0u);
              // codes j and j + 8 at bits 2 j and 16 + 2 j: j = 0..3 of v, then 4..7 of v >> 8
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t d[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const uint32_t v = h ? wd[j] >> 8 : wd[j];
                  d[j][0] = hsub2_u32(and_or(v, fc.mask[0], fc.base[0]), 0x64016401u);  // 1024 + c - 1025
                  d[j][1] = hsub2_u32(and_or(v, fc.mask[1], fc.base[1]), 0x5C045C04u);  // 256 + c - 257
                  d[j][2] = hsub2_u32(and_or(v, fc.mask[2], fc.base[2]), 0x54105410u);  // 64 + c - 65
                  d[j][3] = hsub2_u32(and_or(v, fc.mask[3], fc.base[3]), 0x4C404C40u);  // 16 + c - 17
                }
                const uint32_t xa = h ? x0.z : x0.x, xb = h ? x0.w : x0.y;
                const uint32_t ya = h ? x1.z : x1.x, yb = h ? x1.w : x1.y;
                const uint32_t b0 = __byte_perm(xa, ya, 0x5410), b1 = __byte_perm(xa, ya, 0x7632);
                const uint32_t b2 = __byte_perm(xb, yb, 0x5410), b3 = __byte_perm(xb, yb, 0x7632);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                  mma_16816(acc[m], d[2 * m][0], d[2 * m + 1][0], d[2 * m][1], d[2 * m + 1][1], b0, b1);
                  mma_16816(acc[m], d[2 * m][2], d[2 * m + 1][2], d[2 * m][3], d[2 * m + 1][3], b2, b3);
                }
              }
            }
          }
          if (kInt4) {
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const float s0 = __half2float(__ushort_as_half(static_cast<uint16_t>(sc_now[2 * m] >> (16 * i))));
              const float s1 = __half2float(__ushort_as_half(static_cast<uint16_t>(sc_now[2 * m + 1] >> (16 * i))));
              acc[m][0] = fmaf(grp[m][0], s0, acc[m][0]);
              acc[m][1] = fmaf(grp[m][1], s0, acc[m][1]);
              acc[m][2] = fmaf(grp[m][2], s1, acc[m][2]);
              acc[m][3] = fmaf(grp[m][3], s1, acc[m][3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);
      }
      // the groups' sums, added in group order, then y
      warps_barrier(1, L::kConsumers);  // the previous item's sums have been read
      float* mine = part + kg * (L::kPart / 4);
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) mine[(2 * t + (c & 1)) * 132 + rg * 32 + 16 * m + 8 * (c >> 1) + pg] = acc[m][c];
      warps_barrier(1, L::kConsumers);
      if (ok) {
        const int64_t nn = n0 + 4 * lane;
        float es[4] = {1.0f, 1.0f, 1.0f, 1.0f}, eb[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (nn + c < a.N) {
            if (!kInt4) es[c] = __half2float(a.sc[en0 + nn + c]);
            if (a.bias) eb[c] = __half2float(a.bias[en0 + nn + c]);
          }
        }
        for (int r = warp; r < it.w; r += 4 * KG) {
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if ((rmask >> r) & 1u) {  // a row outside x reads as zeros
            v = *reinterpret_cast<const float4*>(part + r * 132 + 4 * lane);
#pragma unroll
            for (int k = 1; k < KG; ++k) {
              const float4 u = *reinterpret_cast<const float4*>(part + k * (L::kPart / 4) + r * 132 + 4 * lane);
              v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
            }
          }
          if (wide) {  // the halves of k: rows 0-63 of the tile in both halves of the columns
            v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, 16);
            v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, 16);
            v.z += __shfl_xor_sync(0xFFFFFFFFu, v.z, 16);
            v.w += __shfl_xor_sync(0xFFFFFFFFu, v.w, 16);
            if (lane >= 16) continue;
          }
          __half o[4] = {__float2half_rn(fmaf(v.x, es[0], eb[0])), __float2half_rn(fmaf(v.y, es[1], eb[1])),
                         __float2half_rn(fmaf(v.z, es[2], eb[2])), __float2half_rn(fmaf(v.w, es[3], eb[3]))};
          __half* dst = a.y + (static_cast<int64_t>(it.z) + r) * a.N + nn;
          if ((a.N & 3) == 0) {
            if (nn < a.N) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(o);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (nn + c < a.N) dst[c] = o[c];
          }
        }
      }
    }
  }
}

template <bool kInt4, int KG>
static cudaError_t launch_experts_skinny_t(const ExpertArgs& a, int64_t items, cudaStream_t s) {
  using L = SkinnyLayout<kInt4, KG>;
  const uint64_t row_bytes = static_cast<uint64_t>(kInt4 ? a.K / 2 : a.K / 4);
  const uint64_t wrows = static_cast<uint64_t>(a.E) * a.N;
  CUtensorMap tw, th;
  if (!make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, row_bytes, wrows, row_bytes, 128, kERows,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&th, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, row_bytes, wrows, row_bytes, 128, kERows / 2,
                    CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto* kern = experts_skinny_kernel<kInt4, KG>;
  const int smem = L::bytes(a.E);
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(row_grid(L::kWide ? 2 * items : items, 1, L::kCtasPerSm)), dim3(L::kThreads), static_cast<size_t>(smem), 1, s, tw,
                    th, a);
}

template <bool kInt4>
static cudaError_t launch_experts_skinny(const ExpertArgs& a, cudaStream_t s) {
  // at most min(R, E + R / 8) chunks
  const int64_t by_rows = a.E + a.R / 8, chunks = a.R < by_rows ? a.R : by_rows;
  const int64_t items = chunks * ((a.N + kERows - 1) / kERows);
  // One CTA per SM where its items run in one round, or, up to twice as many, where they are long (two rounds
  // of short ones pay their fixed cost twice).  `items` counts an expert for every row; rows that share one
  // make fewer, and one round is where the single CTA gains most.  us with two CTAs | one, INT4 / ternary:
  //               120 items                  176                        296
  //   8 stages    11.0 |  9.6 / 15.8 | 12.0  12.0 | 13.3 / 16.8 | 16.6  13.3 | 15.6 / 17.6 | 19.9
  //   16 stages   17.8 | 14.0 / 26.3 | 18.0  19.9 | 22.7 / 29.0 | 28.5  21.9 | 24.7 / 30.3 | 32.3
  //   28 stages   26.7 | 19.9 / 40.0 | 27.4  31.4 | 32.8 / 47.6 | 43.2  33.6 | 36.3 / 48.7 | 50.7
  //   56 stages   42.5 | 34.3 / 63.5 | 49.3  58.6 | 55.5 / 91.1 | 76.9  60.1 | 63.7 / 91.4 | 92.7
  // so that from 16 stages the loss where every row has an expert of its own is 14 % at most and the gain
  // where they share 19 to 32 %.
  const int64_t sms = current_device_info().num_sms, nk = a.K / SkinnyLayout<kInt4, 2>::KS;
  if (items <= sms || (items <= 2 * sms && nk >= 16)) return launch_experts_skinny_t<kInt4, 4>(a, items, s);
  return launch_experts_skinny_t<kInt4, 2>(a, items, s);
}

// ---------------------------------------------------------------------------------------------
// Many rows per expert: a dense contraction, on tcgen05 with the decoded weights as A in tensor
// memory (as in the prefill GEMM) and the sorted rows of x as B in shared memory.  Persistent CTAs,
// one per SM; an item is RT tiles of 128 weight rows of one expert times up to TN of its rows, all of
// K.  The MMA's N is the item's own number of rows rounded up to 16 (an expert's rows are cut
// evenly), so a ragged expert costs its rows and not a full tile.
// RT = 2: a stage of x (128 k) feeds two accumulators, which halves the x that crosses L2 per MMA (512
// rows per expert, 4096 -> 7168: 240 us INT4, 203 us ternary; RT = 1: 311 and 266 us).  RT = 1 serves
// launches whose items would otherwise leave SMs idle.  With few rows per expert the packed weights
// bound it: TN = 64 leaves the shared memory of the wider x tiles to twice the packed tiles in flight.
// 20 warps:
//   warp 0      x by TMA (tiles of 64 k, 128-byte swizzle, boxes of 32 rows);
//   warp 1      the MMAs (with RT = 2 those of one row tile, warp 3 the other's): the whole warp runs
//               the loop and one elected lane issues, so that the operands are warp-uniform values
//               (computed by a single lane they cost about 140 cycles per MMA).  A barrier test costs
//               the issuing warp 200 to 300 cycles whatever its outcome: hence eight MMAs per test,
//               and one warp's tests under the other's MMAs;
//   warp 2      finds the items (a search in the chunk table), hands them to the other warps through
//               a ring of descriptors one item ahead, and loads the packed weights, 128 rows x 128
//               bytes per load (2 INT4 / 4 ternary stages);
//   warps 4-19  four groups of four that decode, a row tile's stages in turn (thread = weight row =
//               tensor memory lane: 128 weights into the group's slot) and, at the start of the next
//               item, read the item's accumulator: row scale and bias, fp16, and rows of y by TMA
//               stores from a staging buffer per warp (all CTAs reach this point together, and plain
//               stores of 9.7 MB at once held the warps up for 2.7 us per item).  INT4 group scales
//               (and zero-points) are loaded a stage ahead.
// One barrier per stage counts the decode warps of the row tiles, one of which waits for the stage's x,
// after the slot, so that the issuing warps test one barrier per stage.  The chain from an MMA's end to
// the next one on the same slot -- barrier wake-ups, tensor memory stores, the test -- takes about 0.8
// us, and each barrier wait of a decode warp 0.1 to 0.2 us: stages of 64 k lost more to it.
//
// 4096 rows, 8 experts, 4096 -> 14336: INT4 402 us (1.20 PFLOP/s), ternary 341 us (1.41); tensor pipe
// 63 and 73 %, issue 70 and 59 % busy.  A decode warp takes about 3100 (2650) cycles per stage, 1270
// (750) of them decoding, the rest in the four waits and the sums; the MMAs ask for 2048.  Measured
// and left out: pairs of CTAs sharing 256 x 256 items (cta_group::2; half the decoding per MMA, but
// barriers across CTAs: 16384 rows 2044 us against 1729), rows copied in the pairs' order so that no
// byte permutes are needed (no change), a warp of its own for x's barrier (ptxas goes from 96 registers to 80 and
// spills; the kernels here spill 32 to 80 bytes, <INT4, 2, 128> the most, and <ternary, 1, *> and <ternary, 2, 64>
// none).
// 16384 rows run at the power limit (990 W, 1440 MHz).
// ---------------------------------------------------------------------------------------------
constexpr int kTBox = 32;        // sorted rows per x load
constexpr int kTK = 128;         // k per stage
constexpr int kTGroups = 4;      // decode groups
constexpr int kTThreads = 32 * (4 + 4 * kTGroups);
constexpr int kTItems = 4;
constexpr int kTMaxRing = 4;

template <bool kInt4, int RT, int TN>
struct ExpertTcLayout {
  static constexpr int SPP = kInt4 ? 2 : 4;    // stages per packed tile
  static constexpr int SG = kTGroups / RT;     // decode groups, and slots, of a row tile
  static constexpr int RX = RT == 2 ? 3 : 4;   // stages of x
  static constexpr int RP = RT == 2 ? (TN == 64 ? 4 : 2) : (TN == 64 ? 7 : 3);  // packed tiles
  // A decode warp tests the barrier of stage q's x knowing that the MMAs of stage q - SG are done, and
  // so that x of stage q - RX, the barrier's previous one, has landed.
  static_assert(RX >= SG && RX <= kTMaxRing, "rings");
  static constexpr int kSubX = TN * 128;       // 64 k of x
  static constexpr int kTileX = 2 * kSubX;
  static constexpr int kTileP = RT * kERows * 128;
  static constexpr int kOffP = RX * kTileX;
  static constexpr int kOffY = kOffP + RP * kTileP;  // per decode warp: 32 rows of y, 32 columns
  static constexpr int kOffBar = kOffY + 4 * kTGroups * 32 * 64;
  // full[SG], empty[SG], fullX[RX], emptyX[RX][2] (by halves of 64 k), fullP[RP], emptyP[RP], accFull[RT],
  // accEmpty[RT], itemFull[I], itemEmpty[I]
  static constexpr int kNumBars = 5 * kTMaxRing + 2 * RP + 4 + 2 * kTItems;
  static constexpr int kOffItem = (kOffBar + kNumBars * 8 + 15) / 16 * 16;
  static constexpr int kOffMisc = kOffItem + kTItems * 16;  // TMEM address, decode constants
  static constexpr int kOffScan = kOffMisc + 32;
  static constexpr int kOffFirst = kOffScan + 32 * 4;
  static constexpr int bytes(int E) { return kOffFirst + (E + 1) * 4 + 1024; }
  static constexpr uint32_t kColA = RT * TN;   // slots of 64 columns: 128 k
  static_assert(RT * TN + 64 * RT * SG <= 512, "tensor memory");
  static_assert(kOffFirst + 1025 * 4 + 1024 <= 227 * 1024 && kOffFirst > 114 * 1024, "one CTA per SM");
};

// 32 INT4 codes -> 16 registers of fp16 pairs (u - z) s, in natural order (as decode_w4_8).  u - z is exact;
// the product with the scale is rounded to fp16, half a step (2^-11) per weight, and overflows from 65520.
// A scale that stayed outside would need the sums of each group of 128 k apart, in fp32: read from tensor
// memory, scaled and added once per stage, 128 sums per weight row where the registers and tensor memory
// of an item are full.  16384 rows, 4096 -> 14336: relative error of y (rms) 2.65e-4, of which its own
// rounding to fp16 is 2.07e-4.
__device__ __forceinline__ void decode_piece_w4(const uint4& c, uint32_t s2, uint32_t zsub, const DecodeConsts& k,
                                                uint32_t* v) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    v[i] = hmul2_u32(hsub2_u32(and_or(byte_to_halves(w[i >> 2], i & 3), k.mask0, k.base0), zsub), s2);
}
// 32 ternary codes -> 16 registers of fp16 pairs c - 1, in natural order (as decode_tq_8).
__device__ __forceinline__ void decode_piece_tq(const uint2& c, const DecodeConsts& k, uint32_t* v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t t = byte_to_halves(i < 4 ? c.x : c.y, i & 3);
    v[2 * i] = hsub2_u32(and_or(t, k.mask0, k.base0), 0x5C046401u);
    v[2 * i + 1] = hsub2_u32(and_or(t, k.mask1, k.base1), 0x4C405410u);
  }
}

template <bool kInt4, int RT, int TN>
__global__ void __launch_bounds__(kTThreads, 1)
    experts_tc_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                      const __grid_constant__ CUtensorMap tmap_y, const ExpertArgs a) {
  using L = ExpertTcLayout<kInt4, RT, TN>;
  constexpr int SG = L::SG, RX = L::RX, RP = L::RP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kOffBar);
  uint64_t* empty = full + kTMaxRing;
  uint64_t* full_x = empty + kTMaxRing;
  uint64_t* empty_x = full_x + kTMaxRing;
  uint64_t* fullP = empty_x + 2 * kTMaxRing;
  uint64_t* emptyP = fullP + RP;
  uint64_t* acc_full = emptyP + RP;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* item_full = acc_empty + 2;
  uint64_t* item_empty = item_full + kTItems;
  int4* items = reinterpret_cast<int4*>(sm + L::kOffItem);  // (e, tile, row0, rows)
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + L::kOffMisc);
  int* first = reinterpret_cast<int*>(sm + L::kOffFirst);
  // values that steer the roles are broadcast, so that the compiler knows them to be warp-uniform
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  pdl_allow_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < SG; ++i) {
      mbar_init(&full[i], 4 * RT);
      mbar_init(&empty[i], RT);
    }
    for (int i = 0; i < RX; ++i) mbar_init(&full_x[i], 2);
    for (int i = 0; i < 2 * RX; ++i) mbar_init(&empty_x[i], RT);
    for (int i = 0; i < RP; ++i) {
      mbar_init(&fullP[i], 1);
      mbar_init(&emptyP[i], 4 * kTGroups);
    }
    for (int i = 0; i < RT; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4 * SG);
    }
    for (int i = 0; i < kTItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], 1 + RT + 4 * kTGroups);
    }
    store_decode_consts(kInt4, misc + 4);
    fence_mbar_init();
    tma_prefetch_desc(&tmap_x);
    tma_prefetch_desc(&tmap_w);
  }
  if (warp == 1) {
    tmem_alloc(misc, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  pdl_wait_prior_grids();
  expert_chunks(a, TN, first, reinterpret_cast<int*>(sm + L::kOffScan), kTThreads);  // synchronises
  tc_fence_after_sync();
  constexpr uint32_t tmem = 0;  // all 512 columns are this CTA's: they start at 0
  const int64_t tiles = (a.N + RT * kERows - 1) / (RT * kERows);
  const int64_t total = static_cast<int64_t>(first[a.E]) * tiles;
  const int nk = static_cast<int>((a.K + kTK - 1) / kTK);  // the last stage may hold 64 k
  const int npt = (nk + L::SPP - 1) / L::SPP;
  // items of this CTA
  const int count = uniform(static_cast<int>(total > blockIdx.x ? (total - blockIdx.x + gridDim.x - 1) / gridDim.x : 0));
  bool ok = true;

  // Waits of a whole warp; the lanes agree on the outcome.  wait_ahead: for the producers.
  auto wait_all = [&](uint64_t* bar, int phase) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_warp(bar, static_cast<uint32_t>(phase) & 1u)) != 0;
  };
  auto wait_ahead = [&](uint64_t* bar, int phase) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_relaxed(bar, static_cast<uint32_t>(phase) & 1u)) != 0;
  };
  // Item n of this CTA; every warp that uses items reads each once and releases it.
  auto take_item = [&](int n, int4* it) {
    const int d = n % kTItems;
    const bool got = wait_all(&item_full[d], n / kTItems);
    *it = items[d];
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[d]);
    return got;
  };

  if (warp == 2) {
    // ------------------------------------------------------------------ items, packed weights
    auto publish = [&](int n) {
      const ExpertItem it = expert_item<true>(a, first, blockIdx.x + static_cast<int64_t>(n) * gridDim.x, tiles, TN);
      const int d = n % kTItems;
      if (n >= kTItems) ok = wait_ahead(&item_empty[d], n / kTItems - 1);
      if (ok && lane == 0) {
        items[d] = make_int4(it.e, it.tile, it.row0, it.rows);
        mbar_arrive(&item_full[d]);
      }
      __syncwarp();
      return static_cast<int>(static_cast<int64_t>(it.e) * a.N + static_cast<int64_t>(it.tile) * (RT * kERows));
    };
    int s = 0, phase = -1, row = 0;  // packed slot; its previous load's phase
    if (count > 0) row = publish(0);
    for (int n = 0; n < count && ok; ++n) {
      const int row_next = n + 1 < count ? publish(n + 1) : 0;
      for (int pt = 0; pt < npt && ok; ++pt) {
        if (phase >= 0) ok = wait_ahead(&emptyP[s], phase);
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&fullP[s], L::kTileP);
#pragma unroll
          for (int h = 0; h < RT; ++h)
            tma_load_2d(sm + L::kOffP + s * L::kTileP + h * kERows * 128, &tmap_w, &fullP[s], pt * 128, row + h * kERows);
        }
        __syncwarp();
        if (++s == RP) {
          s = 0;
          ++phase;
        }
      }
      row = row_next;
    }
  } else if (warp == 1 || (RT == 2 && warp == 3)) {
    // ------------------------------------------------------------------ MMA
    const int h = warp >> 1;  // row tile
    const uint32_t leader = elect_one() ? 1u : 0u;
    const uint64_t xdesc = sdesc_kmajor_sw128(smem_u32(sm));
    int s = 0, phase = 0, sx = 0;
    for (int n = 0; n < count && ok; ++n) {
      int4 it;
      ok = take_item(n, &it);
      if (ok && n >= 1) ok = wait_all(&acc_empty[h], n - 1);
      const uint32_t idesc = idesc_f16_f32(kERows, static_cast<uint32_t>((uniform(it.w) + 15) / 16 * 16));
      for (int kb = 0; kb < nk && ok; ++kb) {
        ok = wait_all(&full[s], phase);
        if (!ok) break;
        tc_fence_after_sync();
        const uint64_t bdesc = xdesc + static_cast<uint64_t>(sx * (L::kTileX >> 4));
        const uint32_t asrc = L::kColA + 64 * (h * SG + s);
        const bool two = a.K - static_cast<int64_t>(kb) * kTK >= kTK;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (q == 0 || two) {
#pragma unroll
            for (int k16 = 0; k16 < 4; ++k16)
              umma_f16_ts_if(leader, h * TN, asrc + 32 * q + 8 * k16, bdesc + q * (L::kSubX >> 4) + 2 * k16, idesc,
                             (kb | q | k16) != 0 ? 1u : 0u);
          }
          umma_commit_if(leader, &empty_x[2 * sx + q]);
        }
        umma_commit_if(leader, &empty[s]);
        if (++s == SG) {
          s = 0;
          phase ^= 1;
        }
        if (++sx == RX) sx = 0;
      }
      if (ok) umma_commit_if(leader, &acc_full[h]);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------------ x
    const bool skipx = skip_x_loads();  // failure-path test hook: never set in normal use
    int s = 0, phase = -1;              // x slot; its previous stage's phase
    for (int n = 0; n < count && ok && warp == 0; ++n) {
      int4 it;
      ok = take_item(n, &it);
      const int boxes = (it.w + kTBox - 1) / kTBox;
      for (int kb = 0; kb < nk && ok && !skipx; ++kb) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (phase >= 0) ok = ok && wait_ahead(&empty_x[2 * s + q], phase);
          if (!ok) break;
          if (q == 0 || a.K - static_cast<int64_t>(kb) * kTK >= kTK) {
            if (lane == 0) mbar_arrive_expect_tx(&full_x[s], boxes * kTBox * 128);
            __syncwarp();
            if (lane < boxes)
              tma_load_2d(sm + s * L::kTileX + q * L::kSubX + lane * kTBox * 128, &tmap_x, &full_x[s], kb * kTK + q * 64,
                          it.z + lane * kTBox);
          } else if (lane == 0) {
            mbar_arrive(&full_x[s]);
          }
        }
        if (++s == RX) {
          s = 0;
          ++phase;
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ decode, epilogue
    const int grp = (warp >> 2) - 1, h = grp / SG, sg = grp % SG;
    const int r = threadIdx.x & (kERows - 1);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t slot = lane_base + L::kColA + 64 * grp;
    uint64_t* const full_s = &full[sg];
    uint64_t* const empty_s = &empty[sg];
    const bool watch_x = h == 0 && (warp & 3) == 0;  // one of the warps that arrive for a stage
    int sx = sg, phase_x = 0;                        // the barrier of x of the group's next stage
    const int64_t G = a.K >> 7;
    const uint8_t* prow0 = sm + L::kOffP + (h * kERows + r) * 128;
    int4 nx = make_int4(0, 0, 0, 0);
    // scales / zero-points of this thread's weight row: one group of k per stage
    const __half* scp = a.sc;
    const uint8_t* zpp = a.zp;
    uint32_t sc_nxt = 0, zp_nxt = 8;
    auto fetch = [&](int kb) {
      sc_nxt = __half_as_ushort(scp[kb]);
      if (zpp) zp_nxt = zpp[kb];
    };
    auto start_item = [&](const int4& it, int kb) {  // the group's first stage of the item is kb
      const int64_t n = static_cast<int64_t>(it.y) * (RT * kERows) + h * kERows + r;
      const int64_t row = (static_cast<int64_t>(it.x) * a.N + (n < a.N ? n : 0)) * G;  // past N: not stored
      scp = a.sc + row;
      if (a.zp) zpp = a.zp + row;
      fetch(kb);
    };
    const DecodeConsts consts = load_decode_consts(misc + 4);
    __half* const stage = reinterpret_cast<__half*>(sm + L::kOffY) + (warp - 4) * 32 * 32;
    const bool vec = (a.N & 7) == 0;  // y itself is 16-byte aligned
    int own = 0;                      // stages that the group has decoded
    int kn = sg;                      // its next stage within the item
    int ps = 0, phase_p = 0;          // packed slot
    bool ready = false;               // the next stage's scale has been fetched

    // 32 weight rows (n0 and on) x up to 32 rows of y (row and on; cnt of them) from packed pairs of rows.
    auto store_chunk = [&](const uint32_t (&out)[16], int n0, int row, int cnt) {
      if (cnt <= 0) return;
      if (vec) {
        if (lane == 0) tma_store_wait_read();  // the buffer's previous stores
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const __half2 p = *reinterpret_cast<const __half2*>(&out[j]);
          stage[(2 * j) * 32 + lane] = __low2half(p);
          stage[(2 * j + 1) * 32 + lane] = __high2half(p);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (cnt >= 16) tma_store_2d(&tmap_y, stage, n0, row);
          if (cnt >= 32) tma_store_2d(&tmap_y, stage + 16 * 32, n0, row + 16);
          tma_store_commit();
        }
        __syncwarp();
      }
      // what no store of 16 whole rows covers
      const int from = vec ? (cnt < 32 ? cnt / 16 * 16 : 32) : 0;
      uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + static_cast<int64_t>(row) * a.N + n0 + lane;
      if (from < cnt && n0 + lane < a.N) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j >= from && j < cnt) y[j * a.N] = static_cast<uint16_t>((j & 1) ? out[j >> 1] >> 16 : out[j >> 1]);
      }
      __syncwarp();
    };
    // The sums of item n: of its 32-row chunks group sg of row tile h takes every SG-th.  Read and
    // rounded into registers, so that the accumulator is free for the next item's MMAs; the second
    // chunk is held there until the group's next stage is done and the first one's stores have been read.
    constexpr int kChunks = TN / 32 > SG ? TN / 32 / SG : 1;
    static_assert(kChunks <= 2, "one chunk is held");
    uint32_t held[16];
    int held_n0 = 0, held_row = 0, held_cnt = 0;
    auto epilogue = [&](int n, const int4& it) {
      const int n0 = it.y * (RT * kERows) + h * kERows + (warp & 3) * 32;  // the warp's weight rows
      const int nr = n0 + lane;
      const int64_t en = static_cast<int64_t>(it.x) * a.N + nr;
      float es = 1.0f, eb = 0.0f;
      if (nr < a.N) {
        if (!kInt4) es = __half2float(a.sc[en]);
        if (a.bias) eb = __half2float(a.bias[en]);
      }
      if (!wait_all(&acc_full[h], n)) return false;
      tc_fence_after_sync();
      uint32_t out[kChunks][16];
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int tok = (c * SG + sg) * 32;
        if (tok < it.w) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(lane_base + h * TN + tok, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const __half2 p = __floats2half2_rn(fmaf(__uint_as_float(v[2 * j]), es, eb),
                                                fmaf(__uint_as_float(v[2 * j + 1]), es, eb));
            out[c][j] = *reinterpret_cast<const uint32_t*>(&p);
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[h]);
      store_chunk(out[0], n0, it.z + sg * 32, it.w - sg * 32);
      if (kChunks == 2) {
#pragma unroll
        for (int j = 0; j < 16; ++j) held[j] = out[kChunks - 1][j];
        held_n0 = n0;
        held_row = it.z + (SG + sg) * 32;
        held_cnt = it.w - (SG + sg) * 32;
      }
      return true;
    };

    // U steps per packed tile, at most one stage of the group in each.  The previous item's sums are
    // read after the group's first stage of the item (its second needs the slot back, and so the MMAs
    // that wait for them), or, by the group whose slot the previous item's last MMAs use, before it.
    // A last round without stages reads the last item's.
    constexpr int U = L::SPP > SG ? L::SPP / SG : 1;
    if (count > 0) ok = take_item(0, &nx);
    int4 it = nx;
    for (int n = 0; n <= count && count > 0 && ok; ++n) {
      const int4 prev = it;
      it = nx;
      const bool more = n + 1 < count;
      if (kInt4 && !ready && n < count && kn < nk) start_item(it, kn);
      ready = false;
      if (more) ok = take_item(n + 1, &nx);
      const int steps = n < count ? npt * U : 0;
      bool owed = n > 0;
      for (int i = owed && (n == count || kn >= SG - 1) ? -1 : 0, u = 0, pt = 0; i < steps && ok; ++i) {
        if (i >= 0) {
          if (u == 0) ok = wait_all(&fullP[ps], phase_p);
          const uint8_t* prow = prow0 + ps * L::kTileP;
          const int end = pt * L::SPP + L::SPP < nk ? pt * L::SPP + L::SPP : nk;
          if (kn < end && ok) {
            const int ci = kn - pt * L::SPP;  // stage within the packed tile
            uint32_t s2 = 0, zsub = 0;
            uint4 pc[kInt4 ? 4 : 2];
#pragma unroll
            for (int c = 0; c < (kInt4 ? 4 : 2); ++c)
              pc[c] = *reinterpret_cast<const uint4*>(prow + ((((kInt4 ? 4 : 2) * ci + c) ^ (r & 7)) << 4));
            if (kInt4) {
              s2 = sc_nxt | (sc_nxt << 16);
              zsub = w4_zero_pair(zp_nxt & 15u);
              if (kn + SG < nk) {
                fetch(kn + SG);
              } else if (more && kn + SG < 2 * nk) {
                start_item(nx, kn + SG - nk);
                ready = true;
              }
            }
            // two halves of 64 k, each decoded before the wait for its half of the slot; in a last stage of
            // 64 k the second is decoded too, and not multiplied
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t v[32];
              if (kInt4) {
                decode_piece_w4(pc[2 * q], s2, zsub, consts, v);
                decode_piece_w4(pc[2 * q + 1], s2, zsub, consts, v + 16);
              } else {
                decode_piece_tq(make_uint2(pc[q].x, pc[q].y), consts, v);
                decode_piece_tq(make_uint2(pc[q].z, pc[q].w), consts, v + 16);
              }
              if (own > 0 && q == 0) ok = ok && wait_all(empty_s, own - 1);
              if (watch_x && q == 0) {
                ok = ok && wait_all(&full_x[sx], phase_x);
                sx += SG;
                if (sx >= RX) {
                  sx -= RX;
                  phase_x ^= 1;
                }
              }
              if (!ok) break;
              tc_fence_after_sync();
              tmem_st_32x32b_x32(slot + 32 * q, v);
            }
            if (!ok) break;
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(full_s);
            ++own;
            kn += SG;
            if (kChunks == 2 && held_cnt > 0 && !owed) {
              store_chunk(held, held_n0, held_row, held_cnt);
              held_cnt = 0;
            }
          }
          if (++u == U) {  // done with the packed tile
            u = 0;
            ++pt;
            __syncwarp();
            if (lane == 0) mbar_arrive(&emptyP[ps]);
            if (++ps == RP) {
              ps = 0;
              phase_p ^= 1;
            }
          }
        }
        if (owed && ok) {
          owed = false;
          if (kChunks == 2) {  // a group without a stage in the item before
            store_chunk(held, held_n0, held_row, held_cnt);
            held_cnt = 0;
          }
          ok = epilogue(n - 1, prev);
        }
      }
      kn -= nk;
    }
    if (kChunks == 2) store_chunk(held, held_n0, held_row, ok ? held_cnt : 0);
    if (lane == 0) tma_store_wait();
  }

  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <bool kInt4>
static cudaError_t launch_experts_tc(const ExpertArgs& a, cudaStream_t s) {
  const uint64_t row_bytes = static_cast<uint64_t>(kInt4 ? a.K / 2 : a.K / 4);
  CUtensorMap tx, tw;
  if (!make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, row_bytes, static_cast<uint64_t>(a.E) * a.N, row_bytes, 128,
                    kERows, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.x, static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.X),
                    static_cast<uint64_t>(a.K) * 2, 64, kTBox, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  CUtensorMap ty = tx;  // not used when rows of y are not 16-byte aligned
  if (a.N % 8 == 0 && !make_tmap_2d(&ty, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.y, static_cast<uint64_t>(a.N),
                                    static_cast<uint64_t>(a.R), static_cast<uint64_t>(a.N) * 2, 32, 16,
                                    CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  auto items = [&](int RT, int TN) {  // at most
    const int64_t by_rows = a.E + a.R / TN, chunks = a.R < by_rows ? a.R : by_rows;
    return chunks * ((a.N + RT * kERows - 1) / (RT * kERows));
  };
  auto run = [&](auto rt, auto tn) {
    constexpr int RT = decltype(rt)::value, TN = decltype(tn)::value;
    auto* kern = experts_tc_kernel<kInt4, RT, TN>;
    const int smem = ExpertTcLayout<kInt4, RT, TN>::bytes(a.E);
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(row_grid(items(RT, TN), 1, 1)), dim3(kTThreads), static_cast<size_t>(smem), 1, s, tx, tw,
                      ty, a);
  };
  // 64 rows per item while uneven routing leaves most experts below that; 256 weight rows per item where such
  // items (at most `items` of them) fill the SMs.  us, INT4 / ternary, rows spread at random:
  //   TN = 64 | 128, RT = 2, 8 experts of 4096 -> 14336: 32 rows per expert 100 | 104 / 79 | 81, 48: 102 | 106 /
  //   83 | 84, 64: 125 | 108 / 99 | 89, 96: 169 | 118 / 134 | 99; 64 experts of 2048 -> 2816 at 48: 73 | 77 /
  //   61 | 63, at 64: 107 | 79 / 86 | 67.
  //   RT = 1 | 2, 8 experts of 4096 -> N, 40 rows each: 104 items at most, 64 there 22.9 | 29.7 / 20.3 | 23.7;
  //   130, 80 there 39.4 | 29.9 / 35.1 | 24.2; 182, 112 there 39.4 | 30.9 / 35.2 | 25.3; 416, 256 there 71 | 57 /
  //   64 | 45: RT = 1 is the better one while its items, twice as many, take one round.
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  const std::integral_constant<int, 64> n64;
  const std::integral_constant<int, 128> n128;
  const int sms = current_device_info().num_sms;
  if (a.R / a.E <= 48) return items(2, 64) >= sms ? run(two, n64) : run(one, n64);
  return items(2, 128) >= sms ? run(two, n128) : run(one, n128);
}

template <bool kInt4>
static cudaError_t launch_experts(int path, const ExpertArgs& a, cudaStream_t s) {
  if (path == 3 || a.X == 0) return launch_experts_generic<kInt4>(a, s);
  if (path == 2) {
    if (!a.order) return launch_experts_tc<kInt4>(a, s);
    // rows read through the order are copied into sorted order first: one pass over them at memory
    // speed, where copies from inside the product's kernel slowed its MMAs by half
    const cudaError_t e = launch_experts_rows(a, s);
    if (e != cudaSuccess) return e;
    ExpertArgs b = a;
    b.x = a.rows;
    b.X = a.R;
    b.order = nullptr;
    return launch_experts_tc<kInt4>(b, s);
  }
  return launch_experts_skinny<kInt4>(a, s);
}

cudaError_t launch_gemm_experts(bool int4, int path, const ExpertArgs& a, cudaStream_t s) {
  return int4 ? launch_experts<true>(path, a, s) : launch_experts<false>(path, a, s);
}

}  // namespace tq
