// tq_lora_api.cu -- the extern "C" boundary of the adapters' calls (include/tq_lora.h): argument validation
// and dispatch.
#include "../../include/tq_lora.h"
#include "tq_common.cuh"

namespace {

constexpr int64_t kLoraMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kLoraMaxWidth = int64_t(1) << 24;

inline bool dtype16_ok(int d) { return d == TQ_F16 || d == TQ_BF16; }

// The dropout of a call; false: p is not a probability that can be kept.
bool drop_args(double p, const int64_t* rng, tq::DropArgs* d) {
  if (!(p >= 0.0 && p < 1.0)) return false;
  const uint32_t thr = static_cast<uint32_t>(p * 65536.0 + 0.5);
  if (thr > 65535u) return false;
  d->rng = rng;
  d->thr = thr;
  d->scale = static_cast<float>(65536.0 / (65536.0 - thr));
  return true;
}

int check_lora(int dtype, int64_t M, int64_t L, int64_t N, int64_t K, int rank, int path, double p, const int64_t* rng,
               tq::DropArgs* d) {
  if (!dtype16_ok(dtype)) return TQ_ERR_DTYPE;
  if (M < 0 || M > kLoraMaxRows || L < 1 || L > TQ_LORA_MAX_ADAPTERS) return TQ_ERR_SHAPE;
  if (N < 0 || N > kLoraMaxWidth || K < 1 || K > kLoraMaxWidth) return TQ_ERR_SHAPE;
  if (rank < 1 || rank > TQ_LORA_MAX_RANK || !drop_args(p, rng, d)) return TQ_ERR_SHAPE;
  if (path < TQ_PATH_AUTO || path > TQ_PATH_GENERIC) return TQ_ERR_PATH;
  return TQ_OK;
}

// The kernel for few rows takes 16-byte vectors along both widths.
bool lora_few_shape(int64_t M, int64_t N, int64_t K) { return N % 8 == 0 && K % 8 == 0 && M <= tq::kLoraFewMaxRows; }

// The sums of one call, W as A [rank, C] or as B [C, rank].
tq::LoraArgs lora_sum(const void* P, const void* W, bool w_is_a, int64_t C, int rank, int64_t M, int64_t L, float* V,
                      const float* scaling, const int32_t* offsets, const int32_t* order) {
  tq::LoraArgs a = {};
  a.P = P;
  a.W = W;
  a.V = V;
  a.scaling = scaling;
  a.offsets = offsets;
  a.order = order;
  a.M = M;
  a.C = C;
  a.wc = w_is_a ? 1 : rank;
  a.wj = w_is_a ? C : 1;
  a.ws = rank * C;
  a.L = static_cast<int>(L);
  a.rank = rank;
  a.use_scaling = !w_is_a;
  a.drop = tq::DropArgs{nullptr, 0u, 1.0f};
  return a;
}

}  // namespace

extern "C" {

int tq_lora_path(int64_t M, int64_t L, int64_t N, int64_t K, int rank, int dropout, int aligned) {
  if (M < 0 || L < 1 || N < 0 || K < 1 || rank < 1) return TQ_ERR_SHAPE;
  if (M == 0 || N == 0) return TQ_PATH_GENERIC;
  if (dropout || !aligned || !lora_few_shape(M, N, K)) return TQ_PATH_PREFILL;
  // DECODE reads an adapter's weights once per eight rows, PREFILL once per 128 and has two launches' worth of start
  // and end. us of DECODE | PREFILL, rows spread over the adapters at random, fp16:
  //   rows x adapters         256 x 1      512 x 1      1024 x 1     256 x 64     1024 x 64     2048 x 64
  //   4096 -> 4096, 16         7 | 14      13 | 15      19 | 15      13 | 30       27 | 35       43 | 42
  //   4096 -> 14336, 16       11 | 15      20 | 17      33 | 26      23 | 60       44 | 71       71 | 81
  //   14336 -> 4096, 32       13 | 20      23 | 21      44 | 24      29 | 53       57 | 57       95 | 74
  //   4096 -> 4096, 64        14 | 17      26 | 19      46 | 19      29 | 41       57 | 44       96 | 50
  //   4096 -> 14336, 64       16 | 19      31 | 22      60 | 33      41 | 83       79 | 91      135 | 101
  //   4096 -> 4096, 128       30 | 23      50 | 25      89 | 25      62 | 60      120 | 63      204 | 71
  const int64_t some = L < M ? (L < 128 ? L : 128) : M;
  const int64_t most = 32000 + (rank <= 64 ? 800 * (some - 1) : 0);
  return M * (rank + 32) <= most ? TQ_PATH_DECODE : TQ_PATH_PREFILL;
}

int tq_lora(const void* x, int dtype, const void* a, const void* b, const float* scaling, const void* base, void* out,
            float* v, const int32_t* offsets, const int32_t* order, double p, const int64_t* rng, int64_t M, int64_t L,
            int64_t N, int64_t K, int rank, int path, void* stream) {
  tq::DropArgs drop;
  const int st = check_lora(dtype, M, L, N, K, rank, path, p, rng, &drop);
  if (st != TQ_OK || M == 0 || N == 0) return st;
  if (!x || !a || !b || !out || !offsets || (drop.thr && !rng)) return TQ_ERR_NULL;
  const bool al = aligned16(x) && aligned16(a) && aligned16(b) && aligned16(base) && aligned16(out) && aligned16(v);
  const bool few = !drop.thr && lora_few_shape(M, N, K);
  if (path == TQ_PATH_AUTO) {
    path = tq_lora_path(M, L, N, K, rank, drop.thr != 0, al ? 1 : 0);
    if (path == TQ_PATH_PREFILL && !v && few && al) path = TQ_PATH_DECODE;
    if (path == TQ_PATH_PREFILL && !aligned16(v)) path = TQ_PATH_GENERIC;
  } else if (path == TQ_PATH_DECODE) {
    if (!few) return TQ_ERR_PATH;
    if (!al) return TQ_ERR_ALIGN;
  } else if (path == TQ_PATH_PREFILL && !aligned16(v)) {
    return TQ_ERR_ALIGN;
  }
  const bool bf16 = dtype == TQ_BF16;
  if (path == TQ_PATH_DECODE)
    return to_status(tq::launch_lora_few(
        bf16,
        tq::LoraFewArgs{x, a, b, base, out, v, scaling, offsets, order, M, N, K, static_cast<int>(L), rank},
        as_stream(stream)));
  if (!v) return TQ_ERR_NULL;
  tq::LoraArgs s = lora_sum(x, a, true, K, rank, M, L, v, scaling, offsets, order);
  s.drop = drop;
  const cudaError_t e = tq::launch_lora_reduce(bf16, path, s, as_stream(stream));
  if (e != cudaSuccess) return to_status(e);
  s = lora_sum(nullptr, b, false, N, rank, M, L, v, scaling, offsets, order);
  s.base = base;
  s.O = out;
  return to_status(tq::launch_lora_expand(bf16, path, s, as_stream(stream)));
}

size_t tq_lora_workspace_size(int64_t M, int64_t L, int rank) {
  if (M < 0 || M > kLoraMaxRows || L < 1 || L > TQ_LORA_MAX_ADAPTERS || rank < 1 || rank > TQ_LORA_MAX_RANK) return 0;
  return tq::lora_workspace(nullptr, M, L, rank).bytes;
}

int tq_lora_backward(const void* dy, const void* x, int dtype, const void* a, const void* b, const float* scaling,
                     const float* v, void* workspace, size_t workspace_bytes, const void* base_dx, void* dx, void* da,
                     void* db, const int32_t* offsets, const int32_t* order, double p, const int64_t* rng,
                     int64_t M, int64_t L,
                     int64_t N, int64_t K, int rank, int path, void* stream) {
  tq::DropArgs drop;
  const int st = check_lora(dtype, M, L, N, K, rank, path, p, rng, &drop);
  if (st != TQ_OK) return st;
  if (path == TQ_PATH_DECODE) return TQ_ERR_PATH;
  if (!dx && !da && !db) return TQ_OK;
  if (!offsets || (drop.thr && !rng)) return TQ_ERR_NULL;
  if (M > 0 && (!workspace || (N > 0 && (!dy || !b)) || !v || (da && !x) || (dx && !a))) return TQ_ERR_NULL;
  if (!aligned16(workspace)) return TQ_ERR_ALIGN;
  if (M > 0 && workspace_bytes < tq_lora_workspace_size(M, L, rank)) return TQ_ERR_SHAPE;
  if (path == TQ_PATH_AUTO) path = aligned16(v) ? TQ_PATH_PREFILL : TQ_PATH_GENERIC;
  if (path == TQ_PATH_PREFILL && !aligned16(v)) return TQ_ERR_ALIGN;
  const bool bf16 = dtype == TQ_BF16;
  cudaStream_t s = as_stream(stream);
  cudaError_t e = cudaSuccess;
  const tq::LoraWorkspace w = tq::lora_workspace(workspace, M, L, rank);
  const bool tc = path != TQ_PATH_GENERIC;
  const bool scaled = tc && !bf16;  // the powers of two of v and dv are found on the way
  const bool reduced = M > 0 && (dx || da || scaled);
  if (reduced) {
    tq::LoraArgs g = lora_sum(dy, b, false, N, rank, M, L, w.dv, scaling, offsets, order);
    if (scaled) {
      g.V2 = v;
      g.most2 = w.most[0];
      g.most = w.most[1];
    }
    e = tq::launch_lora_reduce(bf16, path, g, s);
    if (e == cudaSuccess && tc && (da || db))
      e = tq::launch_lora_split(bf16, da != nullptr, w, v, offsets, M, L, rank, tq::lora_reduce_split(g), s);
  } else if (M > 0 && tc && db) {
    e = tq::launch_lora_split(bf16, false, w, v, offsets, M, L, rank, 1, s);
  }
  if (e == cudaSuccess && dx && M > 0) {
    tq::LoraArgs g = lora_sum(nullptr, a, true, K, rank, M, L, w.dv, scaling, offsets, order);
    g.base = base_dx;
    g.O = dx;
    g.drop = drop;
    e = tq::launch_lora_expand(bf16, path, g, s);
  }
  tq::LoraArgs ga = lora_sum(x, nullptr, true, K, rank, M, L, w.dv, scaling, offsets, order);
  ga.O = da;
  ga.drop = drop;
  ga.Q = w.Q[1];
  ga.inv = w.inv[1];
  ga.behind = reduced;
  tq::LoraArgs gb = lora_sum(dy, nullptr, false, N, rank, M, L, const_cast<float*>(v), scaling, offsets, order);
  gb.O = db;
  gb.Q = w.Q[0];
  gb.inv = w.inv[0];
  gb.behind = reduced;
  const bool want_b = db && N > 0;
  // One launch for both saves a start and an end and evens out their tiles: dv, split and both for 3001 rows of 3
  // adapters, rank 16, 14336 -> 4096, 62 us apart and 49 together; 128 rows, rank 16, 4096 -> 4096, 15.5 and 12.7; 8192
  // rows, rank 128, 8192 -> 8192, 181 and 166; with 64 adapters in 2048 rows, 123 and 128.  With dropout, which only dA
  // has, its tiles take longer and set the pace of all: 8192 rows, rank 64, 4096 -> 4096, 91 apart, 100 together.
  if (da && want_b && !drop.thr) {
    if (e == cudaSuccess) e = tq::launch_lora_wgrad_both(bf16, path, ga, gb, s);
    return to_status(e);
  }
  if (e == cudaSuccess && da) e = tq::launch_lora_wgrad(bf16, path, ga, s);
  if (e == cudaSuccess && want_b) e = tq::launch_lora_wgrad(bf16, path, gb, s);
  return to_status(e);
}

int tq_dropout(const void* x, int dtype, void* out, double p, const int64_t* rng, int64_t M, int64_t K, void* stream) {
  if (!moe_dtype_ok(dtype)) return TQ_ERR_DTYPE;
  tq::DropArgs drop;
  if (M < 0 || M > kLoraMaxRows || K < 0 || K > (int64_t(1) << 28) || !drop_args(p, rng, &drop)) return TQ_ERR_SHAPE;
  if (M == 0 || K == 0) return TQ_OK;
  if (!x || !out || (drop.thr && !rng)) return TQ_ERR_NULL;
  return to_status(tq::launch_dropout(x, dtype, out, drop, M, K, as_stream(stream)));
}

}  // extern "C"

namespace {

int gemm_backward_impl(bool int4, const uint16_t* dy, const void* w, const uint16_t* sc, const uint8_t* zeros,
                       uint16_t* dx, uint16_t* rows, int64_t M, int64_t N, int64_t K, int path, void* stream) {
  if (M < 0 || N < 0 || K <= 0 || M > (int64_t(1) << 31) || N > (int64_t(1) << 31) || K > (int64_t(1) << 28))
    return TQ_ERR_SHAPE;
  if (int4 && K % 128 != 0) return TQ_ERR_SHAPE;
  if (path < TQ_PATH_AUTO || path > TQ_PATH_GENERIC || path == TQ_PATH_DECODE) return TQ_ERR_PATH;
  if (M == 0) return TQ_OK;
  if (!dx || (N > 0 && (!dy || !w || !sc))) return TQ_ERR_NULL;
  const bool copied = N % 8 != 0 || !aligned16(dy);  // rows of dy that TMA cannot address
  const bool al = aligned16(w) && aligned16(dx) && (!copied || aligned16(rows));
  const bool fits = tq::dx_supported(M, N, K) && (!copied || rows);
  if (path == TQ_PATH_AUTO) {
    path = al && fits ? TQ_PATH_PREFILL : TQ_PATH_GENERIC;
  } else if (path == TQ_PATH_PREFILL) {
    if (!tq::dx_supported(M, N, K)) return TQ_ERR_PATH;
    if (copied && !rows) return TQ_ERR_NULL;
    if (!al) return TQ_ERR_ALIGN;
  }
  tq::DxArgs a = {};
  a.dy = reinterpret_cast<const __half*>(dy);
  a.rows = copied ? reinterpret_cast<__half*>(rows) : nullptr;
  a.w = static_cast<const uint8_t*>(w);
  a.sc = reinterpret_cast<const __half*>(sc);
  a.zp = zeros;
  a.dx = reinterpret_cast<__half*>(dx);
  a.M = M;
  a.N = N;
  a.K = K;
  return to_status(tq::launch_dx(int4, path, a, as_stream(stream)));
}

}  // namespace

extern "C" {

int tq_gemm_backward(const uint16_t* dy, const uint8_t* packed, const uint16_t* scale, uint16_t* dx, uint16_t* rows,
                     int64_t M, int64_t N, int64_t K, int path, void* stream) {
  return gemm_backward_impl(false, dy, packed, scale, nullptr, dx, rows, M, N, K, path, stream);
}

int w4g_gemm_backward(const uint16_t* dy, const int32_t* qweight, const uint16_t* scales, const uint8_t* zeros,
                      uint16_t* dx, uint16_t* rows, int64_t M, int64_t N, int64_t K, int path, void* stream) {
  return gemm_backward_impl(true, dy, qweight, scales, zeros, dx, rows, M, N, K, path, stream);
}

}  // extern "C"
