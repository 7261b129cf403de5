// Entry points of the operators without a context: checks of the arguments,
// then one launcher.  Nothing is enqueued when a check fails.
#include "ops.h"

using namespace moert;

namespace {

constexpr int64_t kInt32Bytes = (int64_t)1 << 31;
constexpr int64_t kMaxRows = kInt32Bytes - 4096;  // row counts, rounded up to tiles, stay int32
constexpr int64_t kMaxLd = (int64_t)1 << 40;
constexpr int32_t kMaxK = 1 << 30;  // the small kernel's 32-bit cursor runs up to 1,024 past K
constexpr int64_t kMaxPairs = (int64_t)1 << 24;  // each chunk of pairs sums the counts of all others

int64_t elem_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
bool is_act(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16; }
bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

moe_status bad(const char* where, const char* why) {
  return fail(nullptr, MOE_EINVAL, std::string(where) + ": " + why);
}

// a launch's status; HIP errors of calls without a context are not latched
moe_status done(const char* where, hipError_t e) {
  if (e == hipSuccess) return MOE_OK;
  (void)hipGetLastError();  // reported here, so not left for the thread's next caller
  if (e == hipErrorInvalidConfiguration)
    return bad(where, "too large: the call needs more workgroups than one launch may have");
  return hip_fail(nullptr, e, where);
}

// No exception crosses the C ABI: only the error texts allocate here.
template <typename F>
moe_status guarded(F f) {
  try {
    return f();
  } catch (...) {
    return MOE_ENOMEM;
  }
}

}  // namespace

extern "C" moe_status moe_mx_quantize(const void* x, moe_dtype x_dtype, int64_t rows, int32_t cols,
                                      int64_t ldx, uint8_t* codes, uint8_t* scales, moe_stream stream) {
  return guarded([&] {
    const char* me = "moe_mx_quantize";
    if (!is_act(x_dtype)) return fail(nullptr, MOE_EUNSUPPORTED, "moe_mx_quantize: x must be F32 or BF16");
    if (rows < 0 || cols < 32 || cols % 32) return bad(me, "rows must be >= 0 and cols a positive multiple of 32");
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return bad(me, "NULL argument");
    if (ldx < cols || ldx > kMaxLd || ldx * elem_bytes(x_dtype) % 16) return bad(me, "ldx must be >= cols and a multiple of 16 bytes");
    if (!aligned(x, 16) || !aligned(codes, 16)) return bad(me, "x and codes must be 16-byte aligned");
    return done(me, launch_mx_quantize(x, x_dtype == MOE_F32, rows, cols, ldx, codes, scales, (hipStream_t)stream));
  });
}

extern "C" moe_status moe_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                        int32_t cols, void* y, moe_dtype y_dtype, int64_t ldy,
                                        moe_stream stream) {
  return guarded([&] {
    const char* me = "moe_mx_dequantize";
    if (!is_act(y_dtype)) return fail(nullptr, MOE_EUNSUPPORTED, "moe_mx_dequantize: y must be F32 or BF16");
    if (rows < 0 || cols < 32 || cols % 32) return bad(me, "rows must be >= 0 and cols a positive multiple of 32");
    if (rows == 0) return MOE_OK;
    if (!codes || !scales || !y) return bad(me, "NULL argument");
    if (ldy < cols || ldy > kMaxLd) return bad(me, "ldy must be >= cols");
    if (!aligned(codes, 16) || !aligned(y, elem_bytes(y_dtype)))
      return bad(me, "codes must be 16-byte aligned and y aligned to its element");
    return done(me, launch_mx_dequantize(codes, scales, rows, cols, y, y_dtype == MOE_F32, ldy, (hipStream_t)stream));
  });
}

// Checks that the dense and the grouped product share.
static moe_status check_product(const char* me, const ProductArgs& a, int x_dtype, int w_dtype, int y_dtype,
                                int64_t ldx, int glu) {
  const bool xm = x_dtype == MOE_MXFP4, wm = w_dtype == MOE_MXFP4;
  if (!is_act(y_dtype) || !(x_dtype == MOE_BF16 || xm) || !(w_dtype == MOE_BF16 || wm) || (xm && !wm))
    return fail(nullptr, MOE_EUNSUPPORTED,
                std::string(me) + ": x and W must be (BF16, BF16), (BF16, MXFP4) or (MXFP4, MXFP4), y F32 or BF16");
  if (a.n_rows >= kMaxRows) return bad(me, "too many rows");
  if (a.n_rows < 0 || a.n_x < 0 || a.n_y < 0 || a.N < 1 || a.K < 1) return bad(me, "negative or empty size");
  if (a.K > kMaxK) return bad(me, "K must be at most 2^30");
  if (a.K % (wm ? 32 : 8)) return bad(me, "K must be a multiple of 32 with MXFP4 operands, else of 8");
  if ((glu != 0 && glu != 1) || (glu && a.N % 2)) return bad(me, "glu must be 0 or 1, and N even with it");
  if (a.n_rows == 0) return MOE_OK;
  if (!a.x || !a.w || !a.y || (xm && !a.xs) || (wm && !a.ws)) return bad(me, "NULL argument");
  if ((!xm && a.xs) || (!wm && a.ws)) return bad(me, "scales given for an operand that is not MXFP4");
  if (xm ? ldx != a.K : ldx < a.K || ldx > kMaxLd || ldx % 8) return bad(me, "ldx must be K for MXFP4 x, else >= K and a multiple of 8");
  if (a.ldy < (glu ? a.N / 2 : a.N) || a.ldy > kMaxLd) return bad(me, "ldy must be at least the columns of y");
  if (!aligned(a.x, 16) || !aligned(a.w, 16) || !aligned(a.y, elem_bytes(y_dtype)))
    return bad(me, "x and W must be 16-byte aligned and y aligned to its element");
  if ((int64_t)a.N * a.K / (wm ? 2 : 1) * (wm ? 1 : 2) >= kInt32Bytes) return bad(me, "a weight matrix must stay below 2^31 bytes");
  if (a.n_x < 1) return bad(me, "x needs a row");  // positions without one read the first, for nothing
  if ((!a.x_index && a.n_x < a.n_rows) || (!a.y_index && a.n_y < a.n_rows))
    return bad(me, "x and y need a row for every position unless an index is given");
  if (a.x_index && a.n_x > 0 && (int64_t)(a.n_x - 1) * a.x_ld + a.x_ld >= kInt32Bytes)
    return bad(me, "indexed rows of x must span less than 2^31 bytes");
  if (!aligned(a.x_index, 4) || !aligned(a.y_index, 4) || !aligned(a.offsets, 4))
    return bad(me, "offsets and indices must be 4-byte aligned");
  return MOE_OK;
}

extern "C" moe_status moe_mx_gemm(const void* x, moe_dtype x_dtype, const uint8_t* x_scales, int64_t ldx,
                                  const uint8_t* w_codes, const uint8_t* w_scales, void* y, moe_dtype y_dtype,
                                  int64_t ldy, int32_t M, int32_t N, int32_t K, moe_stream stream) {
  return guarded([&] {
    const char* me = "moe_mx_gemm";
    ProductArgs a{};
    a.x = (const uint8_t*)x;
    a.xs = x_scales;
    a.w = w_codes;
    a.ws = w_scales;
    a.x_ld = x_dtype == MOE_MXFP4 ? (int64_t)K / 2 : ldx * 2;
    a.y = y;
    a.ldy = ldy;
    a.n_experts = 1;
    a.n_rows = a.n_x = a.n_y = M;
    a.x_div = 1;
    a.N = N;
    a.K = K;
    a.y_f32 = y_dtype == MOE_F32;
    const moe_status st = check_product(me, a, x_dtype, MOE_MXFP4, y_dtype, ldx, 0);
    if (st != MOE_OK || M == 0) return st;
    return done(me, launch_product(a, x_dtype, MOE_MXFP4, false, (hipStream_t)stream));
  });
}

extern "C" moe_status moe_grouped_gemm(const moe_grouped_args* g, moe_stream stream) {
  return guarded([&] {
    const char* me = "moe_grouped_gemm";
    if (!g) return bad(me, "NULL argument");
    if (g->n_experts < 1 || g->n_experts > kMaxExperts) return bad(me, "n_experts must be in 1..1024");
    if (g->reserved) return bad(me, "reserved must be 0");
    if (g->x_index_div < 1) return bad(me, "x_index_div must be >= 1");
    ProductArgs a{};
    a.x = (const uint8_t*)g->x;
    a.xs = g->x_scales;
    a.w = (const uint8_t*)g->w;
    a.ws = g->w_scales;
    a.x_ld = g->x_dtype == MOE_MXFP4 ? (int64_t)g->K / 2 : g->ldx * 2;
    a.w_stride = g->w_stride;
    a.ws_stride = g->ws_stride;
    a.x_index = g->x_index;
    a.y_index = g->y_index;
    a.offsets = g->offsets;
    a.y = g->y;
    a.ldy = g->ldy;
    a.n_experts = g->n_experts;
    a.n_rows = g->n_rows;
    a.n_x = g->n_x;
    a.n_y = g->n_y;
    a.x_div = g->x_index_div;
    a.N = g->N;
    a.K = g->K;
    a.y_f32 = g->y_dtype == MOE_F32;
    const moe_status st = check_product(me, a, g->x_dtype, g->w_dtype, g->y_dtype, g->ldx, g->glu);
    if (st != MOE_OK || a.n_rows == 0) return st;
    if (!a.offsets) return bad(me, "NULL argument");
    if (a.w_stride % 16 || a.w_stride < 0 || a.ws_stride < 0)
      return bad(me, "expert strides must be >= 0, that of the weights a multiple of 16 bytes");
    return done(me, launch_product(a, g->x_dtype, g->w_dtype, g->glu != 0, (hipStream_t)stream));
  });
}

// T*k pairs when the sizes are in range, else -1
static int64_t pair_count(int32_t T, int32_t k, int32_t E) {
  if (T < 0 || k < 1 || E < 1 || E > kMaxExperts || (int64_t)T * k > kMaxPairs) return -1;
  return (int64_t)T * k;
}

extern "C" size_t moe_group_workspace(int32_t T, int32_t k, int32_t E) {
  const int64_t pairs = pair_count(T, k, E);
  return pairs < 0 ? 0 : group_workspace(pairs, E);
}

extern "C" moe_status moe_group_pairs(const int32_t* ids, int32_t T, int32_t k, int32_t E, int32_t* offsets,
                                      int32_t* perm, void* workspace, size_t workspace_bytes,
                                      moe_stream stream) {
  return guarded([&] {
    const char* me = "moe_group_pairs";
    const int64_t pairs = pair_count(T, k, E);
    if (pairs < 0) return bad(me, "T must be >= 0, k >= 1, E in 1..1024 and T*k at most 2^24");
    if (!offsets || (pairs && (!ids || !perm))) return bad(me, "NULL argument");
    const size_t need = group_workspace(pairs, E);
    if (need && (!workspace || workspace_bytes < need)) return bad(me, "workspace smaller than moe_group_workspace()");
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(perm, 4) || (need && !aligned(workspace, 4)))
      return bad(me, "ids, offsets, perm and workspace must be 4-byte aligned");
    return done(me, launch_group_pairs(ids, pairs, E, offsets, perm, (int32_t*)workspace, (hipStream_t)stream));
  });
}

extern "C" moe_status moe_combine_pairs(const void* p, moe_dtype p_dtype, int64_t ldp, const float* w,
                                        const int32_t* ids, int32_t E, int32_t T, int32_t k, int32_t H,
                                        void* y, moe_dtype y_dtype, int64_t ldy, moe_stream stream) {
  return guarded([&] {
    const char* me = "moe_combine_pairs";
    if (!is_act(p_dtype) || !is_act(y_dtype))
      return fail(nullptr, MOE_EUNSUPPORTED, "moe_combine_pairs: p and y must be F32 or BF16");
    if (T < 0 || k < 1 || k > 1 << 30 || H < 1 || H > 1 << 30) return bad(me, "T must be >= 0, k and H in 1..2^30");
    if (ids && E < 1) return bad(me, "E must be >= 1 with ids");
    if (T == 0) return MOE_OK;
    if (!p || !w || !y) return bad(me, "NULL argument");
    if (ldp < H || ldy < H || ldp > kMaxLd || ldy > kMaxLd) return bad(me, "ldp and ldy must be >= H");
    if (!aligned(p, elem_bytes(p_dtype)) || !aligned(y, elem_bytes(y_dtype)) || !aligned(w, 4) || !aligned(ids, 4))
      return bad(me, "every array must be aligned to its element");
    return done(me, launch_combine_pairs(p, p_dtype == MOE_F32, ldp, w, ids, E, T, k, H, y, y_dtype == MOE_F32, ldy,
                                         (hipStream_t)stream));
  });
}
