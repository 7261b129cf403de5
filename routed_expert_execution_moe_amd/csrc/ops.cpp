// Entry points of the operators without a context: checks of the arguments,
// then one launcher.  Nothing is enqueued when a check fails.
#include <cmath>

#include "ops.h"

using namespace moert;

namespace {

constexpr int64_t kInt32Bytes = (int64_t)1 << 31;
constexpr int64_t kMaxRows = kInt32Bytes - 4096;  // row counts, rounded up to tiles, stay int32
constexpr int64_t kMaxLd = (int64_t)1 << 40;
constexpr int32_t kMaxK = 1 << 30;  // the small kernel's 32-bit cursor runs up to 1,024 past K
constexpr int64_t kMaxPairs = (int64_t)1 << 24;  // each chunk of pairs sums the counts of all others

int64_t elem_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
int64_t row_bytes(int dtype) { return dtype == MOE_F8 ? 1 : elem_bytes(dtype); }  // of an element, F8 codes among them
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

// Rows of an array: their number, and bytes from one to the next and of one.
struct Rows {
  const void* at;
  int64_t n, pitch, width;
};

// Whether two arrays of rows share memory.  Rows may lie beside one another, as columns of
// one wider matrix or of every n-th of its rows; else all that lies between the first
// and the last byte counts.
bool overlap(const Rows& a, const Rows& b) {
  typedef __int128 wide;
  const wide a0 = (wide)(uintptr_t)a.at, a1 = a0 + (wide)(a.n - 1) * a.pitch + a.width;
  const wide b0 = (wide)(uintptr_t)b.at, b1 = b0 + (wide)(b.n - 1) * b.pitch + b.width;
  if (a1 <= b0 || b1 <= a0) return false;
  const int64_t pa = a.n > 1 ? a.pitch : b.pitch, pb = b.n > 1 ? b.pitch : pa;  // a single row has any pitch
  const int64_t pitch = std::min(pa, pb);
  if ((a.n == 1 && b.n == 1) || pa % pitch || pb % pitch) return true;
  const wide d = ((b0 - a0) % pitch + pitch) % pitch;  // b's place in the wider row
  return d < a.width || d + b.width > pitch;
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
  const bool xm = x_dtype == MOE_MXFP4, wm = w_dtype == MOE_MXFP4, f8 = x_dtype == MOE_F8;
  if (!is_act(y_dtype) || (f8 ? w_dtype != MOE_F8 : !(x_dtype == MOE_BF16 || xm) || !(w_dtype == MOE_BF16 || wm) || (xm && !wm)))
    return fail(nullptr, MOE_EUNSUPPORTED,
                std::string(me) + ": x and W must be (BF16, BF16), (BF16, MXFP4), (MXFP4, MXFP4) or (F8, F8), y F32 or BF16");
  if (a.n_rows >= kMaxRows) return bad(me, "too many rows");
  if (a.n_rows < 0 || a.n_x < 0 || a.n_y < 0 || a.N < 1 || a.K < 1) return bad(me, "negative or empty size");
  if (a.K > kMaxK) return bad(me, "K must be at most 2^30");
  if (a.K % (wm ? 32 : f8 ? 16 : 8)) return bad(me, "K must be a multiple of 32 with MXFP4 operands, of 16 with F8, else of 8");
  if ((glu != 0 && glu != 1) || (glu && a.N % 2)) return bad(me, "glu must be 0 or 1, and N even with it");
  if (a.n_rows == 0) return MOE_OK;
  if (!a.x || !a.w || !a.y || ((xm || f8) && !a.xs) || ((wm || f8) && !a.ws)) return bad(me, "NULL argument");
  if ((!xm && !f8 && a.xs) || (!wm && !f8 && a.ws)) return bad(me, "scales given for an operand that is not MXFP4 or F8");
  if (xm ? ldx != a.K : ldx < a.K || ldx > kMaxLd || ldx % (f8 ? 16 : 8))
    return bad(me, "ldx must be K for MXFP4 x, else >= K and a multiple of 16 bytes");
  if (a.ldy < (glu ? a.N / 2 : a.N) || a.ldy > kMaxLd) return bad(me, "ldy must be at least the columns of y");
  if (!aligned(a.x, 16) || !aligned(a.w, 16) || !aligned(a.y, elem_bytes(y_dtype)))
    return bad(me, "x and W must be 16-byte aligned and y aligned to its element");
  if (f8 && (!aligned(a.xs, 4) || !aligned(a.ws, 4) || a.ws_stride % 4)) return bad(me, "F8 scales must be 4-byte aligned");
  if ((int64_t)a.N * a.K / (wm ? 2 : 1) * (wm || f8 ? 1 : 2) >= kInt32Bytes) return bad(me, "a weight matrix must stay below 2^31 bytes");
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
    if (x_dtype == MOE_F8) return fail(nullptr, MOE_EUNSUPPORTED, "moe_mx_gemm: x must be BF16 or MXFP4");
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

// Checks that both F8 conversions share; v: the side in F32 or BF16.
static moe_status check_f8(const char* me, const void* v, int dtype, int32_t n_mats, int64_t rows, int32_t cols,
                           int64_t ld, int64_t stride, int32_t block_rows, const uint8_t* codes, const float* scales) {
  if (!is_act(dtype)) return fail(nullptr, MOE_EUNSUPPORTED, std::string(me) + ": the values must be F32 or BF16");
  if (block_rows != 1 && block_rows != 128) return bad(me, "block_rows must be 1 or 128");
  if (n_mats < 0 || rows < 0 || cols < 16 || cols % 16 || cols > kMaxK)
    return bad(me, "sizes must be >= 0 and cols a positive multiple of 16, at most 2^30");
  if (block_rows == 1 && n_mats > 1) return bad(me, "rows of their own scales are one matrix");
  if (n_mats == 0 || rows == 0) return MOE_OK;
  if (rows > kMaxLd / ((cols + 127) / 128)) return bad(me, "too many rows");
  if (!v || !codes || !scales) return bad(me, "NULL argument");
  if (ld < cols || ld > kMaxLd || stride < 0 || stride > kMaxLd) return bad(me, "rows must lie at least cols apart");
  if (!aligned(v, elem_bytes(dtype)) || !aligned(codes, 16) || !aligned(scales, 4))
    return bad(me, "codes must be 16-byte aligned, values and scales aligned to their elements");
  return MOE_OK;
}

extern "C" moe_status moe_f8_quantize(const void* x, moe_dtype x_dtype, int32_t n_mats, int64_t rows, int32_t cols,
                                      int64_t ldx, int64_t x_stride, int32_t block_rows, uint8_t* codes,
                                      float* scales, moe_stream stream) {
  return guarded([&] {
    const char* me = "moe_f8_quantize";
    const moe_status st = check_f8(me, x, x_dtype, n_mats, rows, cols, ldx, x_stride, block_rows, codes, scales);
    if (st != MOE_OK || n_mats == 0 || rows == 0) return st;
    return done(me, launch_f8_quantize(x, x_dtype == MOE_F32, n_mats, rows, cols, ldx, x_stride, block_rows > 1, codes, scales,
                                       (hipStream_t)stream));
  });
}

extern "C" moe_status moe_f8_dequantize(const uint8_t* codes, const float* scales, int32_t n_mats, int64_t rows,
                                        int32_t cols, int32_t block_rows, void* y, moe_dtype y_dtype, int64_t ldy,
                                        int64_t y_stride, moe_stream stream) {
  return guarded([&] {
    const char* me = "moe_f8_dequantize";
    const moe_status st = check_f8(me, y, y_dtype, n_mats, rows, cols, ldy, y_stride, block_rows, codes, scales);
    if (st != MOE_OK || n_mats == 0 || rows == 0) return st;
    // one behind another, or the rows of all of them in turn
    if (n_mats > 1) {
      typedef __int128 wide;
      const bool behind = y_stride >= (wide)(rows - 1) * ldy + cols, in_turn = y_stride >= cols && ldy >= (wide)(n_mats - 1) * y_stride + cols;
      if (!behind && !in_turn) return bad(me, "matrices of y must not overlap");
    }
    return done(me, launch_f8_dequantize(codes, scales, n_mats, rows, cols, block_rows > 1, y, y_dtype == MOE_F32, ldy, y_stride,
                                         (hipStream_t)stream));
  });
}

extern "C" moe_status moe_f8_gemm(const uint8_t* x, const float* x_scales, int64_t ldx, const uint8_t* w,
                                  const float* w_scales, void* y, moe_dtype y_dtype, int64_t ldy, int32_t M,
                                  int32_t N, int32_t K, moe_stream stream) {
  return guarded([&] {
    const char* me = "moe_f8_gemm";
    ProductArgs a{};
    a.x = x;
    a.xs = (const uint8_t*)x_scales;
    a.w = w;
    a.ws = (const uint8_t*)w_scales;
    a.x_ld = ldx;
    a.y = y;
    a.ldy = ldy;
    a.n_experts = 1;
    a.n_rows = a.n_x = a.n_y = M;
    a.x_div = 1;
    a.N = N;
    a.K = K;
    a.y_f32 = y_dtype == MOE_F32;
    const moe_status st = check_product(me, a, MOE_F8, MOE_F8, y_dtype, ldx, 0);
    if (st != MOE_OK || M == 0) return st;
    return done(me, launch_product(a, MOE_F8, MOE_F8, false, (hipStream_t)stream));
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
    a.x_ld = g->x_dtype == MOE_F8 ? g->ldx : g->x_dtype == MOE_MXFP4 ? (int64_t)g->K / 2 : g->ldx * 2;
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

// Checks of the rows that leave a norm, and of its weight; fills their part of n.
static moe_status check_norm(const char* me, NormArgs& n, const void* weight, int weight_dtype, int32_t H, void* y,
                             int y_dtype, float* y_scales, int64_t ldy) {
  const bool f8 = y_dtype == MOE_F8;
  if (!is_act(weight_dtype) || !(is_act(y_dtype) || f8))
    return fail(nullptr, MOE_EUNSUPPORTED, std::string(me) + ": weights must be F32 or BF16, y F32, BF16 or F8");
  if (!weight || !y || f8 != (y_scales != nullptr)) return bad(me, "weight and y are needed, y_scales with F8 y only");
  if (f8 && H % 16) return bad(me, "H must be a multiple of 16 for F8 y");
  if (ldy < H || ldy > kMaxLd || (f8 && ldy % 16)) return bad(me, "ldy must be >= H, for F8 a multiple of 16");
  if (!aligned(y, f8 ? 16 : elem_bytes(y_dtype)) || !aligned(weight, elem_bytes(weight_dtype)) || !aligned(y_scales, 4))
    return bad(me, "F8 y must be 16-byte aligned, other arrays aligned to their elements");
  n.weight = (const uint8_t*)weight;
  n.weight_f32 = weight_dtype == MOE_F32;
  n.y = (uint8_t*)y;
  n.ys = y_scales;
  n.y_dtype = y_dtype;
  n.ldy = ldy;
  return MOE_OK;
}

// its sizes and constants
static moe_status check_norm_sizes(const char* me, int64_t T, int32_t H, float eps) {
  if (T < 0 || T > kMaxLd || H < 1 || H > 32768) return bad(me, "T must be in 0..2^40, H in 1..32768");
  if (!(eps >= 0x1p-126f && eps < INFINITY)) return bad(me, "eps must be a positive normal number");
  return MOE_OK;
}

extern "C" moe_status moe_norm(const void* x, moe_dtype x_dtype, int64_t ldx, const void* weight,
                               moe_dtype weight_dtype, float eps, int64_t T, int32_t H, void* y, moe_dtype y_dtype,
                               float* y_scales, int64_t ldy, moe_stream stream) {
  return guarded([&] {
    const char* me = "moe_norm";
    if (!is_act(x_dtype)) return fail(nullptr, MOE_EUNSUPPORTED, "moe_norm: x must be F32 or BF16");
    moe_status st = check_norm_sizes(me, T, H, eps);
    if (st != MOE_OK || T == 0) return st;
    NormArgs n{};
    st = check_norm(me, n, weight, weight_dtype, H, y, y_dtype, y_scales, ldy);
    if (st != MOE_OK) return st;
    if (!x) return bad(me, "NULL argument");
    if (ldx < H || ldx > kMaxLd) return bad(me, "ldx must be >= H");
    if (!aligned(x, elem_bytes(x_dtype))) return bad(me, "x must be aligned to its element");
    if ((y != x || y_dtype != x_dtype || ldy != ldx) &&
        overlap({y, T, ldy * row_bytes(y_dtype), H * row_bytes(y_dtype)}, {x, T, ldx * elem_bytes(x_dtype), H * elem_bytes(x_dtype)}))
      return bad(me, "y must be x itself, with its type and ldx, or have memory of its own");
    n.p = (const uint8_t*)x;
    n.p_f32 = x_dtype == MOE_F32;
    n.ldp = ldx;
    n.T = T;
    n.H = H;
    n.eps = eps;
    return done(me, launch_norm(n, (hipStream_t)stream));
  });
}

extern "C" moe_status moe_combine_norm(const moe_combine_norm_args* g, moe_stream stream) {
  return guarded([&] {
    const char* me = "moe_combine_norm";
    if (!g) return bad(me, "NULL argument");
    if (g->reserved) return bad(me, "reserved must be 0");
    if (!is_act(g->p_dtype) || !is_act(g->residual_dtype) || !is_act(g->out_dtype) ||
        (g->post_weight && !is_act(g->post_dtype)) || (g->gate && !is_act(g->gate_dtype)))
      return fail(nullptr, MOE_EUNSUPPORTED, "moe_combine_norm: p, residual, out, post_weight and gate must be F32 or BF16");
    moe_status st = check_norm_sizes(me, g->T, g->H, g->eps);
    if (st != MOE_OK || g->T == 0) return st;
    if (g->k < 1 || g->k > 1 << 30 || g->T > kMaxLd / g->k) return bad(me, "k must be in 1..2^30 and T*k at most 2^40");
    if (!g->w && g->k != 1) return bad(me, "several rows a token need w");
    if (g->ids && g->n_experts < 1) return bad(me, "n_experts must be >= 1 with ids");
    if (!(g->scale > -INFINITY && g->scale < INFINITY)) return bad(me, "scale must be finite");
    if (g->gate ? g->gate_cols != 1 && g->gate_cols != g->H : g->gate_cols != 0) return bad(me, "gate_cols must be 1 or H, 0 without a gate");
    if (!g->p || !g->residual || !g->out) return bad(me, "NULL argument");
    if (g->ldp < g->H || g->ldres < g->H || g->ldout < g->H || std::max({g->ldp, g->ldres, g->ldout}) > kMaxLd)
      return bad(me, "ldp, ldres and ldout must be >= H");
    if (g->gate && (g->ldg < 0 || g->ldg > kMaxLd)) return bad(me, "ldg must be >= 0");
    if (!aligned(g->p, elem_bytes(g->p_dtype)) || !aligned(g->residual, elem_bytes(g->residual_dtype)) ||
        !aligned(g->out, elem_bytes(g->out_dtype)) || !aligned(g->w, 4) || !aligned(g->ids, 4) ||
        !aligned(g->post_weight, g->post_weight ? elem_bytes(g->post_dtype) : 1) ||
        !aligned(g->gate, g->gate ? elem_bytes(g->gate_dtype) : 1))
      return bad(me, "every array must be aligned to its element");
    NormArgs n{};
    if (g->weight) {
      st = check_norm(me, n, g->weight, g->weight_dtype, g->H, g->y, g->y_dtype, g->y_scales, g->ldy);
      if (st != MOE_OK) return st;
    } else if (g->y || g->y_scales) {
      return bad(me, "y needs weight");
    }
    // Rows that one workgroup writes while another still reads them.  A token's own
    // rows in the same places are read before they are written.
    auto rows = [&](const void* at, int64_t n, int64_t ld, int dtype) {
      return Rows{at, n, ld * row_bytes(dtype), g->H * row_bytes(dtype)};
    };
    const Rows out = rows(g->out, g->T, g->ldout, g->out_dtype), res = rows(g->residual, g->T, g->ldres, g->residual_dtype);
    const Rows p = rows(g->p, g->T * g->k, g->ldp, g->p_dtype);
    const bool at_res = g->out == g->residual && g->out_dtype == g->residual_dtype && g->ldout == g->ldres;
    const bool at_p = g->out == g->p && g->k == 1 && g->out_dtype == g->p_dtype && g->ldout == g->ldp;
    if ((!at_res && overlap(out, res)) || (!at_p && overlap(out, p)))
      return bad(me, "out must be residual or (k = 1) p itself, with its type and leading dimension, or have memory of its own");
    if (g->weight) {
      const Rows y = rows(g->y, g->T, g->ldy, g->y_dtype);
      if (overlap(y, out) || overlap(y, res) || overlap(y, p)) return bad(me, "y must have memory of its own");
    }
    n.p = (const uint8_t*)g->p;
    n.w = g->w;
    n.ids = g->ids;
    n.res = (const uint8_t*)g->residual;
    n.out = (uint8_t*)g->out;
    n.post = (const uint8_t*)g->post_weight;
    n.gate = (const uint8_t*)g->gate;
    n.ldp = g->ldp;
    n.ldres = g->ldres;
    n.ldout = g->ldout;
    n.ldg = g->ldg;
    n.T = g->T;
    n.k = g->k;
    n.H = g->H;
    n.E = g->n_experts;
    n.gate_cols = g->gate_cols;
    n.p_f32 = g->p_dtype == MOE_F32;
    n.res_f32 = g->residual_dtype == MOE_F32;
    n.out_f32 = g->out_dtype == MOE_F32;
    n.post_f32 = g->post_dtype == MOE_F32;
    n.gate_f32 = g->gate_dtype == MOE_F32;
    n.scale = g->scale;
    n.eps = g->eps;
    return done(me, launch_norm(n, (hipStream_t)stream));
  });
}
