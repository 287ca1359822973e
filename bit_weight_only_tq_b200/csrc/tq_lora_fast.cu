// tq_lora_fast.cu -- low-rank adapters (include/tq_lora.h) with 16-byte vectors along both widths: the sums over many
// rows (reduce and wgrad on tcgen05, expand on mma.sync) and the single launch for few rows.
//
// Work is cut by adapter: a tile is up to 128 sorted positions of one adapter, found on the device from
// the offsets, so that one captured graph serves any plan.
//
// v and dv are fp32.  As operands of a 16-bit product they are split, v s = hi + lo with hi = round(v s), lo = round(v s - hi) and s
// a power of two (fp16 only: bf16 has the exponents of fp32), which keeps 22 (fp16) or 16 (bf16) bits; hi and lo enter the
// same fp32 sum, and 1 / s is applied to it, exactly.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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

template <typename T>
__device__ __forceinline__ uint32_t pack2(T a, T b) {
  Vec<T, 2> v;
  v.v[0] = a;
  v.v[1] = b;
  return *reinterpret_cast<uint32_t*>(&v);
}

// Two fp32 numbers, already scaled, as hi and lo pairs.  What is not finite has no lo part (infinity less itself is NaN).
template <typename T>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const T ha = from_f32<T>(a), hb = from_f32<T>(b);
  float la = a - to_f32(ha), lb = b - to_f32(hb);
  if (!(fabsf(a) <= 3.0e38f)) la = 0.0f;
  if (!(fabsf(b) <= 3.0e38f)) lb = 0.0f;
  hi = pack2<T>(ha, hb);
  lo = pack2<T>(from_f32<T>(la), from_f32<T>(lb));
}

// The power of two that brings `most` to [2^14, 2^15) (fp16), so that the largest value fits and the smallest ones keep their bits; 1
// for bf16, for zero and for what is not finite.  inv: its inverse.
template <typename T>
__device__ __forceinline__ float split_scale(float most, float& inv) {
  inv = 1.0f;
  if (!std::is_same<T, __half>::value || !(most > 0.0f) || !(most <= 3.0e38f)) return 1.0f;
  int e = 14 - (static_cast<int>(__float_as_uint(most) >> 23) - 127);
  e = e > 126 ? 126 : e;
  inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint4 and4(const uint4& a, const uint4& b) {
  return make_uint4(a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w);
}

// Eight consecutive 16-bit elements of a row of `width` from column c (zero past it); vec: whole and aligned.
__device__ __forceinline__ uint4 load8(const void* row, int64_t c, int64_t width, bool vec) {
  const uint16_t* p = static_cast<const uint16_t*>(row) + c;
  if (c >= width) return make_uint4(0u, 0u, 0u, 0u);
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint16_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = c + e < width ? p[e] : static_cast<uint16_t>(0);
  return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
}

// ---------------------------------------------------------------------------------------------
// Tiles.  Tile t of a plan: the tiles of adapter 0, of adapter 1, ..., then those of the positions of no adapter (l = -1),
// which are counted on from the ones before offsets[0] to the ones from offsets[L] on.  Run by a whole warp, all of
// whose lanes get the result.  A plan has at most lora_max_tiles().
// ---------------------------------------------------------------------------------------------
struct LoraTile {
  int l;        // adapter, -1: none, -2: past the last tile
  int cnt;      // positions
  int64_t pos;  // the first one (l = -1: its number among those of no adapter)
  int first;    // the adapter's first tile
};

__device__ __forceinline__ int64_t clamp_pos(int64_t o, int64_t M) { return o < 0 ? 0 : (o < M ? o : M); }

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
      n[i] = o[i + 1] > o[i] ? static_cast<int>((o[i + 1] - o[i] + kLoraTile - 1) / kLoraTile) : 0;
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
          f.pos = o[i] + static_cast<int64_t>(t - before) * kLoraTile;
          f.cnt = static_cast<int>(o[i + 1] - f.pos < kLoraTile ? o[i + 1] - f.pos : kLoraTile);
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
  r.pos = static_cast<int64_t>(t - done) * kLoraTile;
  if (r.pos < head + tail) {
    r.l = -1;
    r.first = done;
    r.cnt = static_cast<int>(head + tail - r.pos < kLoraTile ? head + tail - r.pos : kLoraTile);
  }
  return r;
}

static int64_t lora_max_tiles(int64_t M, int64_t L) {
  const int64_t t = M / kLoraTile + L + 1;
  return t < M ? t : M;
}

// ---------------------------------------------------------------------------------------------
// expand: O[m, c] = base[m, c] + f sum_j V[r, j] W_l(c, j).
// Bound by the rows of base and O (rank FLOPs per byte moved and column, 16-bit), so each is touched once, with 16-byte accesses
// straight between memory and the registers that hold the sums.  A CTA takes a tile's 128 positions (16 per warp) and a range of
// columns in blocks of 64; V stays in registers as fragments, W goes through two shared-memory buffers.
// m16n8k16 gives a lane columns 2t, 2t + 1 of each n8 tile; W's columns are dealt to four n8 tiles so that these are
// eight consecutive columns: column c = 8 u + 2 j + e of a block of 32 is column 2 u + e of tile j.  W as B [C, rank]: rows are
// picked so in the ldmatrix addresses; W as A [rank, C]: pairs of columns are placed so when they are stored to shared memory.
// ---------------------------------------------------------------------------------------------
constexpr int kExpThreads = 256;
constexpr int kExpCols = 64;

template <typename T, int RP, bool kWA, bool kDrop>
__global__ void __launch_bounds__(kExpThreads) lora_expand_kernel(const LoraArgs a, const int cols_per_cta) {
  constexpr int KT = RP / 16;
  constexpr int kStride = kWA ? kExpCols * 2 + 16 : RP * 2 + 16;  // bytes per row; the 16 keep ldmatrix free of conflicts
  constexpr int kBuf = (kWA ? RP : kExpCols) * kStride;
  constexpr int kChunks = RP * kExpCols / 8;                      // 16-byte chunks of a block of W
  constexpr int kPer = (kChunks + kExpThreads - 1) / kExpThreads;
  __shared__ __align__(16) uint8_t sm[2 * kBuf];
  pdl_allow_dependents();
  pdl_wait_prior_grids();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const LoraTile tile = lora_tile(a.offsets, a.L, a.M, blockIdx.x);
  if (tile.l == -2) return;
  const int64_t c_begin = static_cast<int64_t>(blockIdx.y) * cols_per_cta;
  const int64_t c_end = c_begin + cols_per_cta < a.C ? c_begin + cols_per_cta : a.C;
  const T* base = static_cast<const T*>(a.base);
  T* out = static_cast<T*>(a.O);

  if (tile.l < 0) {  // rows of no adapter: base alone
    if (base == out) return;
    const int64_t head = clamp_pos(a.offsets[0], a.M), at = clamp_pos(a.offsets[a.L], a.M);
    const int vecs = static_cast<int>((c_end - c_begin) >> 3);
    for (int i = warp; i < tile.cnt; i += kExpThreads / 32) {
      const int64_t q = tile.pos + i, m = lora_row(a, q < head ? q : q - head + at);
      if (m < 0) continue;
      uint4* dst = reinterpret_cast<uint4*>(out + m * a.C + c_begin);
      const uint4* src = reinterpret_cast<const uint4*>(base + m * a.C + c_begin);
#pragma unroll 4
      for (int j = lane; j < vecs; j += 32) dst[j] = base ? src[j] : make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }

  const T* W = static_cast<const T*>(a.W) + tile.l * a.ws;
  const bool wvec = kWA || (a.rank & 7) == 0;
  const PhiloxKey key = philox_key(a.drop);
  // the rows of this lane: positions 16 warp + g and + 8 of the tile
  int64_t m[2];
  float f[2];
  uint32_t hi[KT][4], lo[KT][4];
  {
    float v[KT][8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 16 * warp + g + 8 * h;
      m[h] = i < tile.cnt ? lora_row(a, tile.pos + i) : -1;
      const float* row = a.V + (tile.pos + i) * a.rank;
      float most = 0.0f;
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 16 * k + 2 * t + (e & 1) + 8 * (e >> 1);
          const float x = m[h] >= 0 && j < a.rank ? row[j] : 0.0f;
          v[k][4 * h + e] = x;
          most = fmaxf(most, fabsf(x));
        }
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      float inv;
      const float s = split_scale<T>(most, inv);
      f[h] = inv * lora_factor(a, tile.l);
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        split2<T>(s * v[k][4 * h], s * v[k][4 * h + 1], hi[k][h], lo[k][h]);
        split2<T>(s * v[k][4 * h + 2], s * v[k][4 * h + 3], hi[k][2 + h], lo[k][2 + h]);
      }
    }
  }

  uint4 wpre[kPer], ynow[4], ynext[4];
  auto load_w = [&](int64_t c0) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int q = threadIdx.x + kExpThreads * i;
      wpre[i] = make_uint4(0u, 0u, 0u, 0u);
      if (q >= kChunks) continue;
      if (kWA) {
        const int j = q / (kExpCols / 8), ch = q % (kExpCols / 8);
        if (j < a.rank) wpre[i] = load8(W + j * a.C, c0 + 8 * ch, a.C, true);
      } else {
        const int c = q / (RP / 8), ch = q % (RP / 8);
        if (c0 + c < a.C) wpre[i] = load8(W + (c0 + c) * a.rank, 8 * ch, a.rank, wvec);
      }
    }
  };
  auto store_w = [&](uint8_t* buf) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int q = threadIdx.x + kExpThreads * i;
      if (q >= kChunks) continue;
      if (kWA) {
        const int j = q / (kExpCols / 8), ch = q % (kExpCols / 8);
        uint32_t* dst = reinterpret_cast<uint32_t*>(buf + j * kStride + (ch >> 2) * 64 + (ch & 3) * 4);
        dst[0] = wpre[i].x;
        dst[4] = wpre[i].y;
        dst[8] = wpre[i].z;
        dst[12] = wpre[i].w;
      } else {
        const int c = q / (RP / 8), ch = q % (RP / 8);
        *reinterpret_cast<uint4*>(buf + c * kStride + ch * 16) = wpre[i];
      }
    }
  };
  auto load_y = [&](int64_t c0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // i = 2 half + row
      const int64_t c = c0 + 32 * (i >> 1) + 8 * t;
      ynext[i] = base && m[i & 1] >= 0 && c < c_end ? *reinterpret_cast<const uint4*>(base + m[i & 1] * a.C + c)
                                                    : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  load_w(c_begin);
  load_y(c_begin);
  const uint32_t sbase = smem_u32(sm);
  const int mq = lane >> 3, mr = lane & 7;  // matrix and row of this lane's ldmatrix address
  const uint32_t frag = kWA ? ((mq & 1) * 8 + mr) * kStride + (mq >> 1) * 16
                            : (8 * (mr >> 1) + 2 * (mq >> 1) + (mr & 1)) * kStride + (mq & 1) * 16;
  int it = 0;
  for (int64_t c0 = c_begin; c0 < c_end; c0 += kExpCols, ++it) {
    store_w(sm + (it & 1) * kBuf);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) ynow[i] = ynext[i];
    if (c0 + kExpCols < c_end) {
      load_w(c0 + kExpCols);
      load_y(c0 + kExpCols);
    }
    const uint32_t buf = sbase + (it & 1) * kBuf + frag;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float acc[4][4] = {};
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          uint32_t b[4];
          if (kWA)
            ldmatrix_x4_trans(buf + 16 * k * kStride + half * 64 + j * 16, b);
          else
            ldmatrix_x4(buf + (32 * half + 2 * j) * kStride + 32 * k, b);
          mma16(acc[j], hi[k][0], hi[k][1], hi[k][2], hi[k][3], b[0], b[1], T());
          mma16(acc[j + 1], hi[k][0], hi[k][1], hi[k][2], hi[k][3], b[2], b[3], T());
          mma16(acc[j], lo[k][0], lo[k][1], lo[k][2], lo[k][3], b[0], b[1], T());
          mma16(acc[j + 1], lo[k][0], lo[k][1], lo[k][2], lo[k][3], b[2], b[3], T());
        }
      const int64_t c = c0 + 32 * half + 8 * t;
      if (c >= c_end) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (m[h] < 0) continue;
        Vec<T, 8> y = *reinterpret_cast<const Vec<T, 8>*>(&ynow[2 * half + h]);
        const uint4 bits = kDrop ? philox((m[h] * a.C + c) >> 3, key) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float s = acc[e >> 1][2 * h + (e & 1)], b = to_f32(y.v[e]);
          y.v[e] = from_f32<T>(kDrop && !drop_keeps(bits, e, a.drop.thr) ? b : fmaf(f[h], s, b));
        }
        *reinterpret_cast<Vec<T, 8>*>(out + m[h] * a.C + c) = y;
      }
    }
  }
}

// The smallest padded rank of 16, 32, 64 or 128 (a multiple of an MMA's 16 k).
template <typename F>
static cudaError_t with_rank(int rank, F fn) {
  if (rank <= 16) return fn(std::integral_constant<int, 16>());
  if (rank <= 32) return fn(std::integral_constant<int, 32>());
  if (rank <= 64) return fn(std::integral_constant<int, 64>());
  return fn(std::integral_constant<int, 128>());
}

static cudaError_t lora_fast_expand(bool bf16, const LoraArgs& a, cudaStream_t s) {
  const int64_t tiles = lora_max_tiles(a.M, a.L), full = (a.M + kLoraTile - 1) / kLoraTile;
  const int64_t blocks = (a.C + kExpCols - 1) / kExpCols;
  // columns split until the tiles with rows give each SM four CTAs or a CTA is left with two blocks
  int64_t split = (4 * current_device_info().num_sms + full - 1) / full;
  if (split > (blocks + 1) / 2) split = (blocks + 1) / 2;
  if (split < 1) split = 1;
  const int64_t per = (blocks + split - 1) / split;
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((blocks + per - 1) / per));
  const int cols = static_cast<int>(per) * kExpCols;
  return with_type16(bf16, [&](auto t) {
    using T = decltype(t);
    return with_rank(a.rank, [&](auto rp) {
      constexpr int RP = decltype(rp)::value;
      auto* kern = a.wc == 1 ? (a.drop.thr ? lora_expand_kernel<T, RP, true, true> : lora_expand_kernel<T, RP, true, false>)
                             : lora_expand_kernel<T, RP, false, false>;
      return launch_pdl(kern, grid, dim3(kExpThreads), 0, 1, s, a, cols);
    });
  });
}

constexpr int kLoraGeneric = 3;  // TQ_PATH_GENERIC

cudaError_t launch_lora_reduce(bool bf16, int path, const LoraArgs& a, cudaStream_t s) {
  return lora_generic_reduce(bf16, a, s);
}
cudaError_t launch_lora_expand(bool bf16, int path, const LoraArgs& a, cudaStream_t s) {
  return path == kLoraGeneric ? lora_generic_expand(bf16, a, s) : lora_fast_expand(bf16, a, s);
}
cudaError_t launch_lora_wgrad(bool bf16, int path, const LoraArgs& a, cudaStream_t s) {
  return lora_generic_wgrad(bf16, a, s);
}

}  // namespace tq
