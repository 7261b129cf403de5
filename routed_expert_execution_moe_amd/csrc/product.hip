// Products y = x W^T with bf16 or MXFP4 operands, dense or ragged by expert:
// the variant for few rows, which streams weights.
//
// A workgroup of eight waves owns 16 rows of W (with GLU: 16 gate rows and the
// matching 16 up rows) against a tile of up to 16*MI rows of x.  The waves
// take K in turns of 128 elements, each lane loading its MFMA fragment straight
// from memory (16 bytes of one row of W: 64 contiguous bytes per row and
// load), so every weight byte is read once per tile and nothing waits at a
// barrier until the waves' sums meet in LDS, in a fixed order.
//
// W is the MFMA's first operand: a lane then holds four neighbouring columns of
// one row of y.  The order of K inside a turn is the same for both operands
// and chosen per format:
//   bf16 x bf16     slice c (0..3), lane group g: k = 32c + 8g + [0,8)
//   bf16 x MXFP4    slice s, lane group g: k = 32g + 8s + [0,8): a lane's codes
//                   are one 16-byte piece under one scale
//   MXFP4 x MXFP4   lane group g: k = 32g + [0,32), the scaled MFMA's own order
#include "ops.h"

namespace moert {

constexpr int kSmWaves = 8;
constexpr int kSmTurn = 128;  // elements of K per wave and turn

template <int AT, int WT, bool GLU, int MI>
__global__ __launch_bounds__(kSmWaves * 64) void product_small_kernel(ProductArgs a) {
  constexpr int NB = GLU ? 2 : 1;
  constexpr bool XM = AT == MOE_MXFP4, WM = WT == MOE_MXFP4;
  __shared__ op_f32x4 s_red[kSmWaves / 2][MI * NB][64];
  const int n_out = GLU ? a.N / 2 : a.N;
  const int n_blocks = (n_out + 15) >> 4;
  const int nb = blockIdx.x % n_blocks;
  OpTile t;
  if (!OpTiles(a, MI * 16).find(a, MI * 16, blockIdx.x / n_blocks, &t)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int K = a.K;

  const uint8_t* w[NB];
  const uint8_t* ws[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    // rows past the end repeat the last one; their columns are not written
    const int64_t n = min(nb * 16 + r, n_out - 1) + b * n_out;
    w[b] = a.w + (int64_t)t.e * a.w_stride + n * (WM ? K / 2 : K * 2);
    ws[b] = WM ? a.ws + (int64_t)t.e * a.ws_stride + n * (K / 32) : nullptr;
  }
  const uint8_t* x[MI];
  const uint8_t* xs[MI];
  bool live[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = i * 16 + r;
    const int row = m < t.rows ? op_x_row(a, t.pos0 + m) : -1;
    live[i] = row >= 0;
    x[i] = a.x + (int64_t)max(row, 0) * a.x_ld;
    xs[i] = XM ? a.xs + (int64_t)max(row, 0) * (K / 32) : nullptr;
  }

  op_f32x4 acc[MI][NB];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[i][b] = op_f32x4{};
  const op_u32x4 zero = {0, 0, 0, 0};

  for (int k0 = wave * kSmTurn; k0 < K; k0 += kSmWaves * kSmTurn) {
    if constexpr (!WM) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int k = k0 + 32 * c + 8 * g;
        op_u32x4 wf[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) wf[b] = k < K ? *(const op_u32x4*)(w[b] + (int64_t)k * 2) : zero;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const op_u32x4 xf = k < K && live[i] ? *(const op_u32x4*)(x[i] + (int64_t)k * 2) : zero;
#pragma unroll
          for (int b = 0; b < NB; ++b)
            acc[i][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(op_bf16x8, wf[b]),
                                                                __builtin_bit_cast(op_bf16x8, xf), acc[i][b], 0, 0, 0);
        }
      }
    } else {
      const int k = k0 + 32 * g;
      const bool in = k < K;
      op_u32x4 wf[NB];
      uint32_t wsc[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        wf[b] = in ? *(const op_u32x4*)(w[b] + k / 2) : zero;
        wsc[b] = in ? ws[b][k / 32] : 127;
      }
      if constexpr (XM) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const bool on = in && live[i];
          const op_u32x4 xf = on ? *(const op_u32x4*)(x[i] + k / 2) : zero;
          const uint32_t xsc = on ? xs[i][k / 32] : 127;
          const op_i32x8 xv = {(int)xf[0], (int)xf[1], (int)xf[2], (int)xf[3], 0, 0, 0, 0};
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const op_i32x8 wv = {(int)wf[b][0], (int)wf[b][1], (int)wf[b][2], (int)wf[b][3], 0, 0, 0, 0};
            acc[i][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, xv, acc[i][b], 4, 4, 0, (int)wsc[b], 0,
                                                                         (int)xsc);
          }
        }
      } else {
        op_bf16x8 wv[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int s = 0; s < 4; ++s) wv[b][s] = op_fp4x8(wf[b][s], op_scale(wsc[b]));
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const op_u32x4 xf = in && live[i] ? *(const op_u32x4*)(x[i] + (int64_t)(k + 8 * s) * 2) : zero;
#pragma unroll
            for (int b = 0; b < NB; ++b)
              acc[i][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[b][s], __builtin_bit_cast(op_bf16x8, xf),
                                                                  acc[i][b], 0, 0, 0);
          }
      }
    }
  }

  // the waves' sums, halved three times: always the same order
#pragma unroll
  for (int half = kSmWaves / 2; half; half >>= 1) {
    if (wave >= half && wave < 2 * half)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) s_red[wave - half][i * NB + b][lane] = acc[i][b];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int b = 0; b < NB; ++b) acc[i][b] += s_red[wave][i * NB + b][lane];
    __syncthreads();
  }
  if (wave) return;
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int m = i * 16 + r;
    const int row = m < t.rows ? op_y_row(a, t.pos0 + m) : -1;
    if (row < 0) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = nb * 16 + 4 * g + q;
      if (n >= n_out) continue;
      const float z = GLU ? op_silu_mul(acc[i][0][q], acc[i][NB - 1][q]) : acc[i][0][q];
      const float v = live[i] ? z : 0.f;
      const int64_t at = (int64_t)row * a.ldy + n;
      if (a.y_f32) ((float*)a.y)[at] = v;
      else ((uint16_t*)a.y)[at] = op_bf16(v);
    }
  }
}

template <int AT, int WT, bool GLU>
static hipError_t launch_small(const ProductArgs& a, hipStream_t s) {
  const int64_t n_blocks = ((GLU ? a.N / 2 : a.N) + 15) / 16;
  const bool few = a.n_rows <= 16 * (int64_t)a.n_experts;
  const int64_t wgs = op_max_tiles(a, few ? 16 : 64) * n_blocks;
  if (wgs * kSmWaves * 64 >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  return launch_op(few ? product_small_kernel<AT, WT, GLU, 1> : product_small_kernel<AT, WT, GLU, 4>,
                   dim3((unsigned)wgs), dim3(kSmWaves * 64), s, a);
}

template <int AT, int WT>
static hipError_t launch_typed(const ProductArgs& a, bool glu, hipStream_t s) {
  // The tile kernel addresses the rows of x of a tile with 32-bit offsets and
  // reads MXFP4 scales 8 at a time.
  const bool tile_ok = a.x_ld < (1 << 23) && (AT != MOE_MXFP4 || a.K >= 256);
  if (a.n_rows > 16 * (int64_t)a.n_experts && tile_ok) {
    if constexpr (AT == MOE_MXFP4) return launch_tile_mx(a, glu, s);
    else if constexpr (WT == MOE_MXFP4) return launch_tile_w4(a, glu, s);
    else return launch_tile_bf16(a, glu, s);
  }
  return glu ? launch_small<AT, WT, true>(a, s) : launch_small<AT, WT, false>(a, s);
}

hipError_t launch_product(const ProductArgs& a, int x_dtype, int w_dtype, bool glu, hipStream_t s) {
  if (x_dtype == MOE_MXFP4) return launch_typed<MOE_MXFP4, MOE_MXFP4>(a, glu, s);
  return w_dtype == MOE_MXFP4 ? launch_typed<MOE_BF16, MOE_MXFP4>(a, glu, s)
                              : launch_typed<MOE_BF16, MOE_BF16>(a, glu, s);
}

}  // namespace moert
