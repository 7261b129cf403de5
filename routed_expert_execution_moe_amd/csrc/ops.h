// Shared by the operators that need no context: launcher declarations, the
// device-side arguments of the (grouped) products and their common device
// code.
#pragma once

#include <algorithm>
#include <tuple>

#include "internal.h"

namespace moert {

// ------------------------------------------------------------------ launchers
// hipLaunchKernel's own status: an error that an earlier caller left behind in
// the thread is neither taken for this launch's nor cleared
template <typename... P, typename... A>
inline hipError_t launch_op(void (*f)(P...), dim3 grid, dim3 block, hipStream_t s, A... a) {
  std::tuple<P...> p(a...);
  return std::apply(
      [&](auto&... v) {
        void* ptrs[] = {(void*)&v...};
        return hipLaunchKernel((const void*)f, grid, block, ptrs, 0, s);
      },
      p);
}

// Operands of y = x W^T, grouped by expert; a dense product is one group
// (offsets == nullptr) of n_rows rows.
struct ProductArgs {
  const uint8_t* x;         // rows of bf16 or of MXFP4 codes
  const uint8_t* xs;        // [n_x][K/32] scales of MXFP4 rows
  const uint8_t* w;         // expert e at w + e * w_stride, [N][K]
  const uint8_t* ws;        // [N][K/32] at ws + e * ws_stride
  int64_t x_ld;             // bytes from row to row of x
  int64_t w_stride, ws_stride;
  const int32_t* x_index;   // [n_rows] or nullptr
  const int32_t* y_index;   // [n_rows] or nullptr
  const int32_t* offsets;   // [E+1] or nullptr
  void* y;
  int64_t ldy;              // elements
  int n_experts, n_rows, n_x, n_y, x_div, N, K, y_f32;
};

hipError_t launch_mx_quantize(const void* x, bool f32, int64_t rows, int cols, int64_t ldx, uint8_t* codes,
                              uint8_t* scales, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols,
                                void* y, bool f32, int64_t ldy, hipStream_t s);
// x_dtype / w_dtype as in moe_grouped_gemm; hipErrorInvalidConfiguration when
// the product needs more workgroups than a launch may have
hipError_t launch_product(const ProductArgs& a, int x_dtype, int w_dtype, bool glu, hipStream_t s);
// Its variants: the streaming one of product.hip in blocks of 16, 32 and 64 rows, and
// the ones that stage tiles in LDS (product_tile.h), one source file per pair of types.
// A gate/up product has one 64-row tile: Shared with W4, else Deep.
enum class ProductVariant { kSmall16, kSmall32, kSmall64, kDeep, kShared, kHalf, kBig };
hipError_t launch_tile_bf16(const ProductArgs& a, bool glu, ProductVariant v, hipStream_t s);
hipError_t launch_tile_w4(const ProductArgs& a, bool glu, ProductVariant v, hipStream_t s);
hipError_t launch_tile_mx(const ProductArgs& a, bool glu, ProductVariant v, hipStream_t s);
size_t group_workspace(int64_t pairs, int E);
hipError_t launch_group_pairs(const int32_t* ids, int64_t pairs, int E, int32_t* offsets, int32_t* perm,
                              int32_t* ws, hipStream_t s);
// hipErrorInvalidConfiguration as above
hipError_t launch_combine_pairs(const void* p, bool p_f32, int64_t ldp, const float* w, const int32_t* ids,
                                int E, int T, int k, int H, void* y, bool y_f32, int64_t ldy, hipStream_t s);

// ------------------------------------------------------------------ device code
#if defined(__HIPCC__)
typedef __bf16 op_bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 op_bf16x8 __attribute__((ext_vector_type(8)));
typedef float op_f32x2 __attribute__((ext_vector_type(2)));
typedef float op_f32x4 __attribute__((ext_vector_type(4)));
typedef float op_f32x16 __attribute__((ext_vector_type(16)));
typedef int op_i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned int op_u32x4 __attribute__((ext_vector_type(4)));

// E8M0 byte to the float whose exponent the scaled converts use: byte 0 is
// 2^-127 (a subnormal), byte 255 an infinity, which the converts turn into NaN
__device__ inline float op_scale(uint32_t s) { return __uint_as_float(s ? s << 23 : 0x00400000u); }

// round to nearest even, NaN stays NaN
__device__ inline uint16_t op_bf16(float v) {
  const __bf16 b = (__bf16)v;
  return __builtin_bit_cast(uint16_t, b);
}

// two at once, one instruction: a in the low half
__device__ inline uint32_t op_bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(op_f32x2{a, b}, op_bf16x2));
}

// 8 MXFP4 codes times their block's scale to bf16 (exact)
__device__ inline op_bf16x8 op_fp4x8(uint32_t raw, float scale) {
  const op_bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw, scale, 0);
  const op_bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw, scale, 1);
  const op_bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw, scale, 2);
  const op_bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw, scale, 3);
  return op_bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// silu(g) * u.  With h = exp(-|g| / 2) the sigmoid is 1 / (1 + h^2), for g < 0
// times h^2: nothing overflows, and the reciprocal (1 ulp, a fraction of a correct
// division's instructions) is of 1..2, so it is no subnormal that the
// instruction would flush.  u comes between the two h: g * h * h alone leaves
// fp32's range below g = -92, where a large u's product is still within it.  Below
// -174 h is flushed to zero; the product is then under 1e-35 for any finite u.
// Nine instructions for the six of g / (1 + exp(-g)) * u, which gives 0 below g = -87
// and NaN for an infinite u there; the epilogue's paired roundings pay for them
// (W4A4 gate/up of 65,536 pairs, 4096 x 4096: 967 us either way).
__device__ inline float op_silu_mul(float g, float u) {
  const float h = __builtin_amdgcn_exp2f(-0.72134752f * fabsf(g));  // log2(e) / 2
  const float s = g * __builtin_amdgcn_rcpf(fmaf(h, h, 1.f));
  const float f = g < 0.f ? h : 1.f;
  return s * f * u * f;
}

struct OpTile {
  int e, pos0, rows;  // expert, first position, positions (1..BM)
};

// inclusive prefix sum over the 64 lanes, by DPP: shifts within rows of 16, then
// the last lane of a row (of two rows) onto the rows behind it
__device__ inline int op_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

// The BM-row tiles of all groups, expert by expert.  One wave on its own: lane
// l counts the tiles of its E/64 experts and a wave scan orders them; every
// lane then gets the total, and find() the t-th tile: the lane that holds it,
// then, its experts (at most 16) a lane each, the expert.  Offsets are clamped
// into 0..n_rows and the counts to what ascending ones can make (the launch
// keeps that below 2^24, so no sum overflows): bad offsets cost results but
// no access out of range.
struct OpTiles {
  int incl, mine, total;

  static __device__ inline int range(const ProductArgs& a, int e, int* lo) {
    *lo = min(max(a.offsets[e], 0), a.n_rows);
    return max(min(max(a.offsets[e + 1], 0), a.n_rows) - *lo, 0);
  }

  __device__ inline OpTiles(const ProductArgs& a, int BM) : incl(0), mine(0) {
    if (!a.offsets) {
      total = (a.n_rows + BM - 1) / BM;
      return;
    }
    const int lane = threadIdx.x & 63, per = (a.n_experts + 63) >> 6;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      int lo;
      if (e < a.n_experts) mine += (range(a, e, &lo) + BM - 1) / BM;
    }
    const int most = a.n_rows / BM + min(a.n_experts, a.n_rows);
    mine = min(mine, most);
    incl = op_scan(mine);
    total = min(__builtin_amdgcn_readlane(incl, 63), most);
  }

  __device__ inline bool find(const ProductArgs& a, int BM, int t, OpTile* out) const {
    if (!a.offsets) {
      out->e = 0;
      out->pos0 = t * BM;
      out->rows = min(BM, a.n_rows - out->pos0);
      return t < total;
    }
    const uint64_t past = __ballot(incl > t);
    if (!past) return false;
    const int owner = __builtin_ctzll(past), per = (a.n_experts + 63) >> 6;
    const int left = t - __builtin_amdgcn_readlane(incl - mine, owner);
    const int lane = threadIdx.x & 63, e = owner * per + lane;
    int lo = 0, n = 0;
    if (lane < per && e < a.n_experts) n = range(a, e, &lo);
    const int tiles = (n + BM - 1) / BM, upto = op_scan(tiles);
    const uint64_t hit = __ballot(upto > left);
    if (!hit) return false;  // offsets changed since they were counted
    const int at = __builtin_ctzll(hit);
    const int skip = (left - __builtin_amdgcn_readlane(upto - tiles, at)) * BM;
    out->e = owner * per + at;
    out->pos0 = __builtin_amdgcn_readlane(lo, at) + skip;
    out->rows = min(BM, __builtin_amdgcn_readlane(n, at) - skip);
    return true;
  }
};

// Tiles of bm rows that n_rows positions in E groups can make at most.  One group
// has no tile more: counted as the others, 4096 rows of bf16 came out as 17 tiles of
// 256, a second round of the chip's CUs (4096 x 4096 x 4096 139 us, 113 as 16).
inline int64_t op_max_tiles(const ProductArgs& a, int bm) {
  if (a.n_experts == 1) return (a.n_rows + bm - 1) / bm;
  return a.n_rows / bm + std::min(a.n_experts, a.n_rows);
}

// Row of x that position p reads, -1 for none (the product is a row of zeros).
__device__ inline int op_x_row(const ProductArgs& a, int p) {
  if (!a.x_index) return p;
  const int i = a.x_index[p];
  if (i < 0) return -1;
  const int r = a.x_div == 1 ? i : i / a.x_div;
  return r < a.n_x ? r : -1;
}

// Row of y that position p writes, -1 for none.
__device__ inline int op_y_row(const ProductArgs& a, int p) {
  if (!a.y_index) return p;
  const int i = a.y_index[p];
  return i < a.n_y ? i : -1;
}
#endif

}  // namespace moert
