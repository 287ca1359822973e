// tq_moe_api.cu -- the extern "C" boundary of the mixture-of-experts calls (include/tq_moe.h):
// argument validation and dispatch.
#include "../../include/tq_moe.h"
#include "tq_common.cuh"

namespace {

inline bool moe_dtype_ok(int d) { return d == TQ_F32 || d == TQ_F16 || d == TQ_BF16; }
inline int moe_elem(int d) { return d == TQ_F32 ? 4 : 2; }
constexpr int64_t kMoeMaxSlots = (int64_t(1) << 31) - 1;
constexpr int64_t kMoeMaxRows = (int64_t(1) << 31) - 1024;  // a tile past the last weight row stays an int

// T tokens of top_k choices
int check_slots(int64_t T, int top_k) {
  if (T < 0 || top_k < 1 || top_k > TQ_MOE_MAX_TOP_K || T > kMoeMaxSlots / top_k) return TQ_ERR_SHAPE;
  return TQ_OK;
}

int check_rows(int64_t T, int64_t H, int top_k, int dtype) {
  if (!moe_dtype_ok(dtype)) return TQ_ERR_DTYPE;
  if (H < 1 || H > (int64_t(1) << 24)) return TQ_ERR_SHAPE;
  return check_slots(T, top_k);
}

int check_route(int64_t T, int64_t E, int top_k, int dtype) {
  if (!moe_dtype_ok(dtype)) return TQ_ERR_DTYPE;
  if (E < 1 || E > TQ_MOE_MAX_EXPERTS || top_k > E) return TQ_ERR_SHAPE;
  return check_slots(T, top_k);
}

int gemm_experts_impl(bool int4, const uint16_t* x, const void* w, const uint16_t* sc, const uint8_t* zeros,
                      const uint16_t* bias, uint16_t* y, const int32_t* offsets, const int32_t* order, uint16_t* rows,
                      int64_t X, int64_t R, int64_t E, int64_t N, int64_t K, int top_k, int path, void* stream) {
  if (X < 0 || R < 0 || X > kMoeMaxSlots || R > kMoeMaxSlots) return TQ_ERR_SHAPE;
  if (E < 1 || E > TQ_MOE_MAX_EXPERTS || N < 0 || N > kMoeMaxRows / E) return TQ_ERR_SHAPE;
  if (K <= 0 || K > (int64_t(1) << 28) || top_k < 1) return TQ_ERR_SHAPE;
  if (int4 && K % 128 != 0) return TQ_ERR_SHAPE;
  if (path < TQ_PATH_AUTO || path > TQ_PATH_GENERIC) return TQ_ERR_PATH;
  if (R == 0 || N == 0) return TQ_OK;
  if (!w || !sc || !y || !offsets || (!x && X > 0)) return TQ_ERR_NULL;
  const bool al = aligned16(x) && aligned16(w) && aligned16(y);
  const int fmt = int4 ? TQ_FMT_W4G128 : TQ_FMT_TERNARY;
  if (path == TQ_PATH_AUTO) {
    path = tq_experts_path(fmt, R, E, N, K, al ? 1 : 0);
    if (path == TQ_PATH_PREFILL && order && (!rows || !aligned16(rows))) path = TQ_PATH_DECODE;
  } else if (path != TQ_PATH_GENERIC) {
    if (K % 64 != 0) return TQ_ERR_PATH;
    if (path == TQ_PATH_PREFILL && order && !rows) return TQ_ERR_NULL;
    if (!al || (path == TQ_PATH_PREFILL && order && !aligned16(rows))) return TQ_ERR_ALIGN;
  }
  tq::ExpertArgs a = {};
  a.x = reinterpret_cast<const __half*>(x);
  a.w = static_cast<const uint8_t*>(w);
  a.sc = reinterpret_cast<const __half*>(sc);
  a.zp = zeros;
  a.bias = reinterpret_cast<const __half*>(bias);
  a.y = reinterpret_cast<__half*>(y);
  a.offsets = offsets;
  a.order = order;
  a.rows = reinterpret_cast<__half*>(rows);
  a.X = X;
  a.R = R;
  a.N = N;
  a.K = K;
  a.E = static_cast<int>(E);
  a.top_k = top_k;
  return to_status(tq::launch_gemm_experts(int4, path, a, as_stream(stream)));
}

}  // namespace

extern "C" {

int tq_moe_route(const void* logits, int dtype, float* weights, int32_t* ids, int64_t T, int64_t E, int top_k,
                 int renormalize, void* stream) {
  const int st = check_route(T, E, top_k, dtype);
  if (st != TQ_OK || T == 0) return st;
  if (!logits || !weights || !ids) return TQ_ERR_NULL;
  return to_status(tq::launch_moe_route(logits, dtype, weights, ids, T, E, top_k, renormalize != 0, as_stream(stream)));
}

int tq_moe_route_backward(const float* dweights, const void* logits, int dtype, const float* weights,
                          const int32_t* ids, void* dlogits, int64_t T, int64_t E, int top_k, int renormalize,
                          void* stream) {
  const int st = check_route(T, E, top_k, dtype);
  if (st != TQ_OK || T == 0) return st;
  if (!dweights || !logits || !weights || !ids || !dlogits) return TQ_ERR_NULL;
  return to_status(tq::launch_moe_route_bwd(dweights, logits, dtype, weights, ids, dlogits, T, E, top_k,
                                            renormalize != 0, as_stream(stream)));
}

int tq_moe_sort(const int32_t* ids, int32_t* offsets, int32_t* order, int32_t* pos, int64_t R, int64_t E, void* stream) {
  if (R < 0 || R > kMoeMaxSlots || E < 1 || E > TQ_MOE_MAX_EXPERTS) return TQ_ERR_SHAPE;
  if (!offsets || (R > 0 && (!ids || !order || !pos))) return TQ_ERR_NULL;
  return to_status(tq::launch_moe_sort(ids, offsets, order, pos, R, E, as_stream(stream)));
}

int tq_moe_gather(const void* x, int dtype, const int32_t* order, const int32_t* offsets, void* rows, int64_t T,
                  int64_t H, int top_k, int64_t E, void* stream) {
  const int st = check_rows(T, H, top_k, dtype);
  if (st != TQ_OK) return st;
  if (E < 1 || E > TQ_MOE_MAX_EXPERTS) return TQ_ERR_SHAPE;
  if (T == 0) return TQ_OK;
  if (!x || !order || !offsets || !rows) return TQ_ERR_NULL;
  return to_status(tq::launch_moe_gather(x, moe_elem(dtype), order, offsets, rows, T, H, top_k, E, as_stream(stream)));
}

int tq_moe_combine(const void* y, int dtype, const int32_t* pos, const float* weights, void* out, int64_t T, int64_t R,
                   int64_t H, int top_k, void* stream) {
  const int st = check_rows(T, H, top_k, dtype);
  if (st != TQ_OK) return st;
  if (R < 0 || R > kMoeMaxSlots) return TQ_ERR_SHAPE;
  if (T == 0) return TQ_OK;
  if (!pos || !out || (!y && R > 0)) return TQ_ERR_NULL;
  return to_status(tq::launch_moe_combine(y, dtype, pos, weights, out, T, R, H, top_k, as_stream(stream)));
}

int tq_moe_combine_backward(const void* dout, const void* y, int dtype, const int32_t* pos, const float* weights,
                            void* dy, float* dweights, int64_t T, int64_t R, int64_t H, int top_k, void* stream) {
  const int st = check_rows(T, H, top_k, dtype);
  if (st != TQ_OK) return st;
  if (R < 0 || R > kMoeMaxSlots) return TQ_ERR_SHAPE;
  if (T == 0 || (!dy && !dweights)) return TQ_OK;
  if (!dout || !pos || (dweights && !y && R > 0) || (dy && !weights)) return TQ_ERR_NULL;
  return to_status(
      tq::launch_moe_combine_bwd(dout, y, dtype, pos, weights, dy, dweights, T, R, H, top_k, as_stream(stream)));
}

int tq_gemm_experts(const uint16_t* x, const uint8_t* packed, const uint16_t* scale, const uint16_t* bias, uint16_t* y,
                    const int32_t* offsets, const int32_t* order, uint16_t* rows, int64_t X, int64_t R, int64_t E,
                    int64_t N, int64_t K, int top_k, int path, void* stream) {
  return gemm_experts_impl(false, x, packed, scale, nullptr, bias, y, offsets, order, rows, X, R, E, N, K, top_k, path,
                           stream);
}

int w4g_gemm_experts(const uint16_t* x, const int32_t* qweight, const uint16_t* scales, const uint8_t* zeros,
                     const uint16_t* bias, uint16_t* y, const int32_t* offsets, const int32_t* order, uint16_t* rows,
                     int64_t X, int64_t R, int64_t E, int64_t N, int64_t K, int top_k, int path, void* stream) {
  return gemm_experts_impl(true, x, qweight, scales, zeros, bias, y, offsets, order, rows, X, R, E, N, K, top_k, path,
                           stream);
}

int tq_experts_path(int fmt, int64_t R, int64_t E, int64_t N, int64_t K, int aligned) {
  if (fmt != TQ_FMT_TERNARY && fmt != TQ_FMT_W4G128) return TQ_ERR_PATH;
  if (R < 0 || E < 1 || N < 0 || K <= 0) return TQ_ERR_SHAPE;
  if (fmt == TQ_FMT_W4G128 && K % 128 != 0) return TQ_ERR_SHAPE;
  if (R == 0 || N == 0 || !aligned || K % 64 != 0) return TQ_PATH_GENERIC;
  // The crossover by rows per expert on average, the only such number the host knows; one pass of the decode
  // kernel covers 8 rows.  us of the decode | tensor-core kernel, INT4 / ternary, rows spread at random:
  //   rows per expert        6                     8                        10
  //   8 of 4096 -> 14336     64 | 99 / 54 | 75     79 | 99 / 66 | 75        90 | 99 / 74 | 76
  //   64 of 2048 -> 2816     53 | 69 / 45 | 54     68 | 70 / 56 | 54        79 | 70 / 66 | 55
  //   32 of 4096 -> 2048     40 | 55 / 33 | 41     55.0 | 54.8 / 41 | 42    56 | 55 / 46 | 42
  //   128 of 2048 -> 768     32 | 45 / 27 | 35     41 | 45 / 34 | 35        44 | 45 / 37 | 35
  //   8 of 14336 -> 4096     64 | 104 / 51 | 89    90 | 104 / 72 | 89       119 | 104 / 95 | 89
  // With half of the rows on one expert it moves by two rows at most (8 of 4096 -> 14336 at 8: 87 | 99 / 72 | 76,
  // 128 of 2048 -> 768 at 10: 48 | 44 / 38 | 35).  R counts slots of no expert too: a caller who knows how many
  // there are asks with its own number of rows (8 of 64 experts, 4096 -> 14336, 34 of 256 slots: 63 | 103 / 52 | 78).
  return R <= 8 * E ? TQ_PATH_DECODE : TQ_PATH_PREFILL;
}

}  // extern "C"
