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
  const uint8_t* x;         // rows of bf16 or of MXFP4 or F8 codes
  const uint8_t* xs;        // [n_x][K/32] scales of MXFP4 rows; F8: fp32 [n_x][ceil(K/128)]
  const uint8_t* w;         // expert e at w + e * w_stride, [N][K]
  const uint8_t* ws;        // [N][K/32] at ws + e * ws_stride; F8: fp32, one per 128 x 128 tile
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
// n_mats matrices of [rows][cols]; ldx and stride in elements
hipError_t launch_f8_quantize(const void* x, bool f32, int n_mats, int64_t rows, int cols, int64_t ldx,
                              int64_t stride, bool tiles, uint8_t* codes, float* scales, hipStream_t s);
hipError_t launch_f8_dequantize(const uint8_t* codes, const float* scales, int n_mats, int64_t rows, int cols,
                                bool tiles, void* y, bool f32, int64_t ldy, int64_t stride, hipStream_t s);

// The norm in front of a block (p = x, no residual) or the end of one; dimensions
// and strides in elements.
struct NormArgs {
  const uint8_t* p;
  const float* w;
  const int32_t* ids;
  const uint8_t* res;
  uint8_t* out;
  const uint8_t* post;
  const uint8_t* gate;
  const uint8_t* weight;
  uint8_t* y;
  float* ys;
  int64_t ldp, ldres, ldout, ldg, ldy, T;
  int k, H, E, gate_cols;
  int p_f32, res_f32, out_f32, post_f32, gate_f32, weight_f32;
  int y_dtype;
  int lg;  // log2 of the threads per row, or 10 and more for a whole workgroup
  float scale, eps;
};
hipError_t launch_norm(NormArgs a, hipStream_t s);

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
// F8 (product_f8.hip): Shared (64 x 128), Half (128 x 128), and with BF16 y Big (256 x 256)
hipError_t launch_tile_f8(const ProductArgs& a, bool glu, ProductVariant v, hipStream_t s);
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

// 8 e4m3 codes, first in the lowest byte, as bf16 (exact)
__device__ inline op_bf16x8 op_f8x8_values(uint32_t lo, uint32_t hi) {
  const op_bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
  const op_bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
  const op_bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
  const op_bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
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

// the largest of 16 lanes' values (a DPP row), in each of them
__device__ inline uint32_t op_max16(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));   // lane ^ 1
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));   // lane ^ 2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));  // mirrored in 8
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));  // mirrored in 16
  return v;
}

// F8 scale of a block and its reciprocal, from the bits of the largest magnitude
// (their order as integers is that of the magnitudes; infinities and NaN come out
// on top and make the block NaN, with codes of 0 from the reciprocal's flag)
struct OpF8Scale {
  float scale, inv;
  bool bad;
  __device__ inline explicit OpF8Scale(uint32_t top) {
    bad = top >= 0x7F800000u;
    const float s = fmaxf(__uint_as_float(bad ? 0 : top) / 448.f, 0x1p-126f);
    scale = bad ? __uint_as_float(0x7FC00000u) : s;
    inv = 1.f / s;
  }
};

// 8 e4m3 codes of v * inv, first in the lowest byte.  |v * inv| is below 448.0001, so
// nothing saturates.
__device__ inline uint2 op_f8x8(const float (&v)[8], const OpF8Scale& s) {
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * s.inv, v[1] * s.inv, lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * s.inv, v[3] * s.inv, lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * s.inv, v[5] * s.inv, hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * s.inv, v[7] * s.inv, hi, true);
  return s.bad ? make_uint2(0, 0) : make_uint2((uint32_t)lo, (uint32_t)hi);
}

// 16 and 8 bytes at an address of any alignment: global memory takes them in one access
typedef unsigned int op_u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int op_bytes16 __attribute__((ext_vector_type(4), aligned(1)));
typedef unsigned int op_bytes8 __attribute__((ext_vector_type(2), aligned(1)));

// 8 columns of a row in fp32 or bf16, as loaded
struct OpCols {
  op_u32x4 a, b;
};
__device__ inline OpCols op_cols_load(const uint8_t* row, bool f32, int64_t c) {
  OpCols v{};
  const uint8_t* p = row + c * (f32 ? 4 : 2);
  v.a = *(const op_bytes16*)p;
  if (f32) v.b = *(const op_bytes16*)(p + 16);
  return v;
}
// the first n of them (0 and fewer: none), the others zero
__device__ inline OpCols op_cols_load(const uint8_t* row, bool f32, int64_t c, int n) {
  if (n >= 8) return op_cols_load(row, f32, c);
  OpCols v{};
  if (f32) {
    const float* p = (const float*)row + c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < n) v.a[i] = __float_as_uint(p[i]);
      if (i + 4 < n) v.b[i] = __float_as_uint(p[i + 4]);
    }
  } else {
    const uint16_t* p = (const uint16_t*)row + c;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) v.a[i / 2] |= (uint32_t)p[i] << (i % 2 * 16);
  }
  return v;
}
__device__ inline void op_cols_get(const OpCols& c, bool f32, float (&v)[8]) {
  if (f32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(c.a[i]);
      v[4 + i] = __uint_as_float(c.b[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(c.a[i] << 16);
      v[2 * i + 1] = __uint_as_float(c.a[i] & 0xFFFF0000u);
    }
  }
}
// the first n columns of a row at c
__device__ inline void op_cols_store(uint8_t* row, bool f32, int64_t c, int n, const float (&v)[8]) {
  if (f32) {
    float* p = (float*)row + c;
    if (n >= 8) {
      *(op_bytes16*)p = op_u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
      *(op_bytes16*)(p + 4) = op_u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = v[i];
    }
  } else {
    uint16_t* p = (uint16_t*)row + c;
    if (n >= 8) {
      *(op_bytes16*)p = op_u32x4{op_bf16_pair(v[0], v[1]), op_bf16_pair(v[2], v[3]), op_bf16_pair(v[4], v[5]), op_bf16_pair(v[6], v[7])};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = op_bf16(v[i]);
    }
  }
}

// 8 columns at c but for the first lo (8 and more: none of them)
__device__ inline void op_cols_store_from(uint8_t* row, bool f32, int64_t c, int lo, const float (&v)[8]) {
  if (lo <= 0) {
    op_cols_store(row, f32, c, 8, v);
  } else {
#pragma unroll
    for (int i = 1; i < 8; ++i)
      if (i >= lo) {
        if (f32) ((float*)row)[c + i] = v[i];
        else ((uint16_t*)row)[c + i] = op_bf16(v[i]);
      }
  }
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
// then the expert.  Keep: up to 256 experts a lane's offsets are loaded at once and stay
// in registers (F8: clocks to the tile's expert 4,000 -> 3,400 with 128, down of 512
// tokens over 256 experts 103 -> 95 us); past that, and without Keep, they are read
// again, its experts (at most 16) a lane each.  The W4A4 256 x 256 tile does without: it
// fills its registers, and with GLU spills three of them with Keep, one without (65,536
// pairs, 4096 x 4096, 1,001 and 988 us).  Other W4A4 tiles keep them (up of 512 and 4,096 pairs
// 44.2 and 57.7 us, 45.2 and 58.5 without), bf16 too (down of 32,008 pairs 229.7, 230.4).  Offsets are clamped
// into 0..n_rows and the counts to what ascending ones can make (the launch
// keeps that below 2^24, so no sum overflows): bad offsets cost results but
// no access out of range.
template <bool Keep>
struct OpTiles {
  static constexpr int Few = 4;  // experts of a lane whose offsets stay in registers
  int incl, mine, total;
  int off[Few + 1];

  static __device__ inline int range(const ProductArgs& a, int e, int* lo) {
    *lo = min(max(a.offsets[e], 0), a.n_rows);
    return max(min(max(a.offsets[e + 1], 0), a.n_rows) - *lo, 0);
  }

  __device__ inline OpTiles(const ProductArgs& a, int BM) : incl(0), mine(0), off{} {
    if (!a.offsets) {
      total = (a.n_rows + BM - 1) / BM;
      return;
    }
    const int lane = threadIdx.x & 63, per = (a.n_experts + 63) >> 6;
    if (Keep && per <= Few) {
#pragma unroll
      for (int i = 0; i <= Few; ++i)
        off[i] = min(max(a.offsets[min(lane * per + min(i, per), a.n_experts)], 0), a.n_rows);
#pragma unroll
      for (int i = 0; i < Few; ++i) mine += (max(off[i + 1] - off[i], 0) + BM - 1) / BM;
    } else {
      for (int i = 0; i < per; ++i) {
        const int e = lane * per + i;
        int lo;
        if (e < a.n_experts) mine += (range(a, e, &lo) + BM - 1) / BM;
      }
    }
    const int most = a.n_rows / BM + min(a.n_experts, a.n_rows);
    mine = min(mine, most);
    incl = op_scan(mine);
    total = min(__builtin_amdgcn_readlane(incl, 63), most);
  }

  // The expert of the t-th tile: its number, first position, positions and first tile.
  __device__ inline bool expert(const ProductArgs& a, int BM, int t, int* e, int* lo_e, int* n_e, int* first) const {
    if (!a.offsets) {
      *e = *lo_e = *first = 0;
      *n_e = a.n_rows;
      return t < total;
    }
    const uint64_t past = __ballot(incl > t);
    if (!past) return false;
    const int owner = __builtin_ctzll(past), per = (a.n_experts + 63) >> 6;
    const int begin = __builtin_amdgcn_readlane(incl - mine, owner), left = t - begin;
    if (Keep && per <= Few) {
      int upto = 0;
      bool found = false;
#pragma unroll
      for (int i = 0; i < Few; ++i) {
        const int lo = __builtin_amdgcn_readlane(off[i], owner);
        const int n = max(__builtin_amdgcn_readlane(off[i + 1], owner) - lo, 0), tiles = (n + BM - 1) / BM;
        if (!found && upto + tiles > left) {
          *e = owner * per + i;
          *lo_e = lo;
          *n_e = n;
          *first = begin + upto;
          found = true;
        }
        upto += tiles;
      }
      return found;
    }
    const int lane = threadIdx.x & 63, i = owner * per + lane;
    int lo = 0, n = 0;
    if (lane < per && i < a.n_experts) n = range(a, i, &lo);
    const int tiles = (n + BM - 1) / BM, upto = op_scan(tiles);
    const uint64_t hit = __ballot(upto > left);
    if (!hit) return false;  // offsets changed since they were counted
    const int at = __builtin_ctzll(hit);
    *e = owner * per + at;
    *lo_e = __builtin_amdgcn_readlane(lo, at);
    *n_e = __builtin_amdgcn_readlane(n, at);
    *first = begin + __builtin_amdgcn_readlane(upto - tiles, at);
    return true;
  }

  __device__ inline bool find(const ProductArgs& a, int BM, int t, OpTile* out) const {
    int lo, n, first;
    if (!expert(a, BM, t, &out->e, &lo, &n, &first)) return false;
    const int skip = (t - first) * BM;
    out->pos0 = lo + skip;
    out->rows = min(BM, n - skip);
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

// blocks of K with a scale of their own, and the row of W's F8 scales that holds
// column n of part (0: all of W or the gate, 1: up)
__host__ __device__ inline int op_f8_blocks(int K) { return (K + 127) >> 7; }
__device__ inline int op_f8_w_block(const ProductArgs& a, bool glu, int n, int part) {
  return (n >> 7) + (glu && part ? (a.N / 2 + 127) >> 7 : 0);
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
