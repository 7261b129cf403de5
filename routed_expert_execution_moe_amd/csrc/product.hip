// Products y = x W^T with bf16, MXFP4 or F8 operands, dense or ragged by expert:
// the variant for few rows, and the choice between the variants.
//
// A workgroup of eight waves owns 16*NB rows of W (with GLU: as many gate rows
// and the matching up rows) against a tile of up to 16*MI rows of x, in 16x16
// MFMA blocks.  The waves take K in turns of 128 elements, each lane loading
// its fragments straight from memory (16 bytes of a row, four lanes 64
// neighbouring bytes), the next turn's before the current one is multiplied;
// nothing waits at a barrier until the waves' sums meet in LDS, in a fixed
// order.  So even a product of one token keeps every CU's loads in flight, and
// K costs a few memory latencies instead of one per step.
//
// W is the MFMA's first operand: a lane then holds four neighbouring columns of
// one row of y.  The order of K inside a turn is the same for both operands
// and chosen per format:
//   bf16 x bf16     slice c (0..3), lane group g: k = 32c + 8g + [0,8)
//   bf16 x MXFP4    slice s, lane group g: k = 32g + 8s + [0,8): a lane's codes
//                   are one 16-byte piece under one scale
//   MXFP4 x MXFP4   lane group g: k = 32g + [0,32), the scaled MFMA's own order
//   F8 x F8         piece c (0..1), lane group g: k = 64c + 16g + [0,16); a turn is
//                   one scale block, whose products are summed from zero and
//                   join the row's sum times both scales.  The codes are expanded
//                   to bf16, which is exact: the 8-bit matrix instructions keep
//                   13 bits of each product, and loads bound here
//
// One token against 4096 x 4096 in MXFP4 (8.9 MB) takes 5.6 us of kernel, in F8 (16.8 MB)
// 5.4, and a call for eight in MXFP4 6.8; 64 x 4096 x 4096 takes 13.7 us in 32 x 32 blocks, F8
// 12.0.  Of one token's 10,200 clocks in MXFP4 1,100 find the tile, 250 its rows, 6,800
// are a wave's four turns.  333 x 2040 x 2080 in 64 x 64 blocks takes 12.6 us, F8 11.2 (15.9
// and 14.4 when the sums were halved three times and one wave stored the whole
// block).  What bounds the turns past a few rows is their loads: fragments come
// through the vector cache once per wave, (MI + NB) of them per MI*NB products, and
// with W in 4 bits each of x is four times one of W.
#include <type_traits>

#include "ops.h"

namespace moert {

constexpr int kSmWaves = 8;
constexpr int kSmTurn = 128;  // elements of K per wave and turn

template <int AT, int WT, bool GLU, int MI, int NB>
__global__ __launch_bounds__(kSmWaves * 64, 2) void product_small_kernel(ProductArgs a) {
  constexpr int NW = GLU ? 2 * NB : NB;  // W blocks: gate blocks, then up blocks
  constexpr bool XM = AT == MOE_MXFP4, WM = WT == MOE_MXFP4, F8 = AT == MOE_F8;
  constexpr int CW = F8 ? 2 : WM ? 1 : 4, CX = F8 ? 2 : XM ? 1 : 4;  // 16-byte pieces per row and turn
  __shared__ op_f32x4 s_red[kSmWaves / 2][MI * NW][64];
  const int n_out = GLU ? a.N / 2 : a.N;
  const int n_blocks = (n_out + 16 * NB - 1) / (16 * NB);
  const int n0 = (blockIdx.x % n_blocks) * (16 * NB);
  OpTile t;
  if (!OpTiles<true>(a, MI * 16).find(a, MI * 16, blockIdx.x / n_blocks, &t)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int K = a.K;

  // rows of W past the end repeat the last one (their columns are not written),
  // rows of x past the tile's end or without a source the first (nor are these)
  const uint8_t* w[NW];
  const uint8_t* ws[NW];
#pragma unroll
  for (int b = 0; b < NW; ++b) {
    const int64_t n = min(n0 + (b % NB) * 16 + r, n_out - 1) + (b / NB) * n_out;
    w[b] = a.w + (int64_t)t.e * a.w_stride + n * (F8 ? K : WM ? K / 2 : K * 2);
    ws[b] = F8   ? a.ws + (int64_t)t.e * a.ws_stride + (int64_t)op_f8_w_block(a, GLU, min(n0 + (b % NB) * 16, n_out - 1), b / NB) * op_f8_blocks(K) * 4
            : WM ? a.ws + (int64_t)t.e * a.ws_stride + n * (K / 32)
                 : nullptr;
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
    xs[i] = F8 ? a.xs + (int64_t)max(row, 0) * op_f8_blocks(K) * 4 : XM ? a.xs + (int64_t)max(row, 0) * (K / 32) : nullptr;
  }

  op_f32x4 acc[MI][NW];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int b = 0; b < NW; ++b) acc[i][b] = op_f32x4{};

  struct Turn {
    op_u32x4 w[NW][CW], x[MI][CX];
    uint32_t ws[NW], xs[MI];
  };
  // a lane's element of piece c in the turn at k0
  auto at = [&](int k0, int c, bool codes) {
    if (F8) return k0 + 64 * c + 16 * g;
    return k0 + (codes ? 32 * g : WM ? 32 * g + 8 * c : 32 * c + 8 * g);
  };
  auto load = [&](int k0, auto whole_c) {
    constexpr bool whole = decltype(whole_c)::value;
    Turn f;
    const op_u32x4 zero = {0, 0, 0, 0};
    // pieces past the end of a row become zeros (and their scales 1)
    auto piece = [&](const uint8_t* row, int k, int bytes2) {
      const bool in = whole || k < K;
      const op_u32x4 v = *(const op_u32x4*)(row + (int64_t)(in ? k : 0) * bytes2 / 4);
      return in ? v : zero;
    };
    auto scale = [&](const uint8_t* row) {
      if (F8) return *(const uint32_t*)(row + (int64_t)(k0 / 128) * 4);
      const int b = k0 / 32 + g;
      const bool in = whole || b * 32 < K;
      const uint32_t v = row[in ? b : 0];
      return in ? v : 127u;
    };
#pragma unroll
    for (int b = 0; b < NW; ++b) {
#pragma unroll
      for (int c = 0; c < CW; ++c) f.w[b][c] = piece(w[b], at(k0, c, WM), F8 ? 4 : WM ? 2 : 8);
      if constexpr (WM || F8) f.ws[b] = scale(ws[b]);
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
      for (int c = 0; c < CX; ++c) f.x[i][c] = piece(x[i], at(k0, c, XM), F8 ? 4 : XM ? 2 : 8);
      if constexpr (XM || F8) f.xs[i] = scale(xs[i]);
    }
    return f;
  };
  auto multiply = [&](const Turn& f) {
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        op_bf16x8 xv[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) xv[c] = op_f8x8_values(f.x[i][c >> 1][c % 2 * 2], f.x[i][c >> 1][c % 2 * 2 + 1]);
#pragma unroll
        for (int b = 0; b < NW; ++b) {
          op_f32x4 part = {};
#pragma unroll
          for (int c = 0; c < 4; ++c)
            part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                op_f8x8_values(f.w[b][c >> 1][c % 2 * 2], f.w[b][c >> 1][c % 2 * 2 + 1]), xv[c], part, 0, 0, 0);
          const float s = __uint_as_float(f.xs[i]) * __uint_as_float(f.ws[b]);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][b][q] = fmaf(s, part[q], acc[i][b][q]);
        }
      }
    } else if constexpr (XM) {
#pragma unroll
      for (int b = 0; b < NW; ++b) {
        const op_i32x8 wv = {(int)f.w[b][0][0], (int)f.w[b][0][1], (int)f.w[b][0][2], (int)f.w[b][0][3], 0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const op_i32x8 xv = {(int)f.x[i][0][0], (int)f.x[i][0][1], (int)f.x[i][0][2], (int)f.x[i][0][3], 0, 0, 0, 0};
          acc[i][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, xv, acc[i][b], 4, 4, 0, (int)f.ws[b], 0,
                                                                       (int)f.xs[i]);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int b = 0; b < NW; ++b) {
          op_bf16x8 wv;
          if constexpr (WM) wv = op_fp4x8(f.w[b][0][c], op_scale(f.ws[b]));
          else wv = __builtin_bit_cast(op_bf16x8, f.w[b][c]);
#pragma unroll
          for (int i = 0; i < MI; ++i)
            acc[i][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(op_bf16x8, f.x[i][c]), acc[i][b],
                                                                0, 0, 0);
        }
    }
  };

  int k0 = wave * kSmTurn;
  constexpr int kNext = kSmWaves * kSmTurn;
  if (k0 + kSmTurn <= K) {
    Turn f = load(k0, std::true_type{});
    for (k0 += kNext; k0 + kSmTurn <= K; k0 += kNext) {
      const Turn n = load(k0, std::true_type{});
      multiply(f);
      f = n;
    }
    multiply(f);
  }
  if (k0 < K) multiply(load(k0, std::false_type{}));

  // The waves' sums meet in LDS, always in the same order: those of waves w and w + 4,
  // then (0 + 2) + (1 + 3), which every wave adds up for its own blocks and stores.
  if (wave >= kSmWaves / 2)
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int b = 0; b < NW; ++b) s_red[wave - kSmWaves / 2][i * NW + b][lane] = acc[i][b];
  __syncthreads();
  if (wave < kSmWaves / 2)
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int b = 0; b < NW; ++b) s_red[wave][i * NW + b][lane] = acc[i][b] + s_red[wave][i * NW + b][lane];
  __syncthreads();
  auto total = [&](int k) { return (s_red[0][k][lane] + s_red[2][k][lane]) + (s_red[1][k][lane] + s_red[3][k][lane]); };
#pragma unroll
  for (int u = 0; u < MI * NB; ++u) {
    if (wave != u % kSmWaves) continue;
    const int i = u / NB, b = u % NB, m = i * 16 + r;
    op_f32x4 v = total(i * NW + b);
    if constexpr (GLU) {
      const op_f32x4 up = total(i * NW + b + NB);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = op_silu_mul(v[q], up[q]);
    }
    if (!live[i]) v = op_f32x4{};
    const int row = m < t.rows ? op_y_row(a, t.pos0 + m) : -1;
    const int n = n0 + b * 16 + 4 * g;
    if (row < 0 || n >= n_out) continue;
    const int64_t o = (int64_t)row * a.ldy + n;
    if (n + 4 <= n_out) {
      if (a.y_f32) *(op_bytes16*)((float*)a.y + o) = __builtin_bit_cast(op_u32x4, v);
      else *(op_bytes8*)((uint16_t*)a.y + o) = op_u32x2{op_bf16_pair(v[0], v[1]), op_bf16_pair(v[2], v[3])};
    } else {
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        if (n + q >= n_out) continue;
        if (a.y_f32) ((float*)a.y)[o + q] = v[q];
        else ((uint16_t*)a.y)[o + q] = op_bf16(v[q]);
      }
    }
  }
}

template <int AT, int WT, bool GLU, int MI, int NB>
static hipError_t launch_small_as(const ProductArgs& a, hipStream_t s) {
  const int64_t n_blocks = ((GLU ? a.N / 2 : a.N) + 16 * NB - 1) / (16 * NB);
  const int64_t wgs = op_max_tiles(a, 16 * MI) * n_blocks;
  if (wgs * kSmWaves * 64 >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  return launch_op(product_small_kernel<AT, WT, GLU, MI, NB>, dim3((unsigned)wgs), dim3(kSmWaves * 64), s, a);
}

// Which variant of an F8 product (us on MI355X; "up" and "plain" as below, weights of
// several calls in rotation).  But for those of 8 rows or fewer the figures are from before
// all of the small variant's waves stored and short tiles had a third stage, which moved
// the border between few and more rows.  Small and Shared now, 2040 x 2080 at 256 and 512 rows
// 8.6, 11.5; 11.0, 11.7, both Shared by the rule; 24576 x 4096 at 9 and 16 29.6, 26.1; 32.4,
// 26.3, both small by it.
//   Big, BF16 rows only, by rounds of the chip: one of Big (256 workgroups) takes about 9/5 of one
//   of Half (512, two a CU).  Half and Big, N = K = 4096, 2,048, 3,000, 4,096 and 6,000
//   rows 44, 50; 65, 54; 79, 63; 114, 107 (a tie by the rule); 8192 x 512, 1,300 and
//   3,000 rows 17.3, 16.4; 27, 29.  Several experts: their last tiles are half
//   full on average.  8 experts of 256 rows, 4096 x 4096 87, 61; 16 of 256 rows,
//   GLU 2816 x 1024 31, 43.  Many tiles make no rounds, and Big's short tiles cost
//   only the rows they have: from 1,024 tiles and 128 mean rows always Big.  Up at 64, 128 and
//   256 rows 114, 128; 141, 134; 204, 171; plain at 128 and 256 93, 96; 147, 133.
//   Half, not Shared, from 257 tiles, and with several experts from 128 mean rows.
//   One expert 4096 x 4096, 1,024 and 2,048 rows 31, 26; 44, 48; FP32 rows 48, 45; 72, 83.
//   Up at 64 and 128 rows 114, 108; 141, 150; FP32 148, 148; 190, 213.
//   One expert's 8 rows or fewer stay with the small variant at any width, so that rows as
//   few keep all bits of the products.  Small and Half at 1, 4 and 8 rows: 36864 x 4096
//   35.7, 41.9; 40.0, 43.3; 41.2, 43.9; 152064 x 4096 124, 138; 137, 148; 146, 149; GLU
//   20480 x 4096 40, 44; 38, 43; 39, 43.  Half is ahead from 10 rows (152064 x 4096 154, 148;
//   FP32 rows from 12), at 8 of K = 8192 (128, 123) and with GLU of K = 1024 (65536 columns 30, 27).
//   FP32 rows 35.1, 45.7; 40.1, 50.0; 39.9, 48.8; 126, 143; 137, 152; 147, 153; 40, 50 thrice.
//   One expert's other few rows do up to 16 and up to a workgroup of 32 x 32 per CU:
//   small and Shared, 4096 x 4096 at 16, 64 and 128 rows 8.4, 15.9; 13.9, 16.6; 23, 16.5;
//   2040 x 2080 at 128 and 256 rows 7.8, 11.4; 10.7, 11.6; 8192 x 2048 at 32 and 64
//   9.2, 10.5; 14.0, 10.8.  FP32 rows, whose tiles expand both operands: up to two, and
//   up to one of 64 x 64: 4096 x 4096 at 128 and 256 rows 23.5, 27.0; 27.9, 27.8; 2040 x
//   2080 at 333 and 512 15.2, 18.2; 15.7, 18.7; 8192 x 2048 at 128 19.0, 17.4.
//   Several experts' up to 127 tiles (one token up 12.7, 14.0; two 16.5, 14.8), FP32 up to 256
//   (one token of 4096 x 2048 over 256 experts 19.0, 19.4; two 33, 27), FP32 with
//   GLU below 4 mean rows (up at 2, 4 and 8 rows 53, 59; 679, 645 for 4096 x 4096 over 256; 97, 86).
static ProductVariant choose_f8(const ProductArgs& a, bool glu) {
  const int64_t n_out = glu ? a.N / 2 : a.N, rows = a.n_rows / a.n_experts;
  const int groups = std::min(a.n_experts, a.n_rows), g = glu ? 2 : 1;
  const bool one = a.n_experts == 1;
  auto wide = [&](int n) { return (n_out + n - 1) / n; };
  auto tiles = [&](int m, int n) { return op_max_tiles(a, m) * wide(n); };
  auto rounds = [&](int m, int n, int at_once) {
    const int64_t t = one ? tiles(m, n) : (a.n_rows / m + groups / 2) * wide(n);
    return (t + at_once - 1) / at_once;
  };
  // the tile kernels address the rows of x of a tile with 32-bit offsets
  if (a.x_ld < (1 << 23) && !(one && a.n_rows <= 8)) {
    if (one || rows >= 128) {
      if (!a.y_f32 && ((!one && tiles(256, 256 / g) >= 1024) || 5 * rounds(128, 128 / g, 512) >= 9 * rounds(256, 256 / g, 256)))
        return ProductVariant::kBig;
      if (tiles(128, 128 / g) > 256) return ProductVariant::kHalf;
    }
    const bool few = one ? a.n_rows <= 16 || tiles(32, 32) <= (a.y_f32 ? 512 : 256) || (a.y_f32 && tiles(64, 64) <= 256)
                         : a.y_f32 && glu ? rows < 4 : tiles(64, 128 / g) < (a.y_f32 ? 257 : 128);
    if (!few) return ProductVariant::kShared;
  }
  const int avg = (a.n_rows + groups - 1) / groups;
  if (avg <= 16 || tiles(16, 16) <= 512) return ProductVariant::kSmall16;
  return avg <= 64 || tiles(32, 32) <= 512 ? ProductVariant::kSmall32 : ProductVariant::kSmall64;
}

// Which variant, by the tiles that a call can make at most and by the mean rows
// of an expert (us on MI355X, the small variant's before all of its waves stored;
// "up" is a GLU product of N = 1536, K = 2048 over 128 experts, "plain" one without
// GLU of N = 2048, K = 768, both with 8 experts a token):
//   Mid, not the small variant, from 64 tiles (W4, whose small variant is the
//   faster: 129).  W4A4 4096x4096 at 64 and 128 rows 11.8 small, 12.6 Mid and
//   16.8, 12.5; bf16 at 128 and 256 rows 29.5, 32.1 and 38.7, 31.9; W4 at 128, 512
//   rows 23.6, 28 and 57.8, 29; W4A4 up at 1 and 8 tokens 8.2, 10.0 and 17.3, 13.5.
//   One expert's 8 rows or fewer stay with the small variant, but for W4A4: at 1,
//   8 and 16 rows of 32768x2048 bf16 27, 32; 30, 32; 37, 32 and W4 15, 25; 20, 25;
//   26, 25 (W4A4 12.4, 11.0 at one).  Not so several experts, though with weights
//   from memory the small variant is often the faster there too, bf16's above all;
//   Mid and small, eight experts of one row each: bf16 4096x2048 37, 28; 8192x4096
//   124, 87; 8192x1024 27, 30; GLU 16384x4096 283, 171; W4 25, 18; 52, 52; 17, 22;
//   66, 84.
//   Mid is Shared beyond 256 tiles, one per CU.  W4A4 plain at 256 tokens 34
//   Shared, 55 Deep; 128x4096x4096 (64 tiles) 14.5 Shared, 12.5 Deep.
//   Half from 257 tiles of its own and 64 mean rows, W4 96.  Plain at 512 and 1,024
//   tokens (32, 64 rows), Half and Mid: bf16 86, 84 and 97, 99; W4A4 30, 30 and 36,
//   41; N = 4096, K = 2048 bf16 407, 408 and 441, 505, W4A4 140, 136 and 151, 170.
//   Uneven routing (expert e with (e + 1)^-0.6 of the tokens): bf16 98, 87 and 103,
//   100; W4 55, 50 at 64 rows and 76, 84 at 128.
//   Big, one expert, by rounds of 256 workgroups: one of Big takes as long as 8/3 of
//   Half, which share a CU (W4 10/3).  Half and Big, N = K = 4096, 2,048, 3,000 and
//   4,096 rows (2, 3 and 4 rounds of Half): bf16 71, 93; 108, 94; 138, 108; W4A4 27,
//   33; 40, 35; 49, 40; W4 66, 87; 98, 91; 134, 109; 3000^2, K = 2048 W4 46, 50;
//   1300x11000x4096 (4 rounds, 2 of Big) bf16 130, 174.
//   Big, several experts, from 256 tiles of its own (GLU 128) and these mean rows;
//   Half (GLU Mid) and Big, even | uneven:
//     bf16 192, K >= 2048 128.  Plain at 128 and 256 rows 126, 121 | 126, 136; 200,
//       191 | 213, 171; N = 4096, K = 2048 at 128 rows 609, 479 | 599, 542.  With
//       K = 256 Big loses: N = 2048 at 250 rows 85, 99.
//     W4A4 384, K >= 2048 192.  Plain at 256 and 384 rows 86, 100 | 86, 85; 154,
//       124; N = 4096, K = 2048 at 128 and 256 rows 215, 187 | 211, 219; 344, 300 |
//       363, 296.
//     W4 768.  N = 4096, K = 2048 at 512 and 1,024 rows 1155, 1172 | 1170, 1142;
//       2206, 2114 | 2216, 2110.
//     One expert, GLU, W4A4: from 65 tiles, where Mid's need a second round.  Mid and
//       Big at 64, 66, 96 and 128 tiles: 19.8, 31.2; 33.6, 31.6; 34.6, 31.8; 36.4, 32.1
//       (512x8192x4096, 512x8448x4096, 768x8192x4096, 1024x8192x4096); bf16 at 96 and
//       112 80, 92 and 81, 87.
//     GLU 128, W4 768.  Up at 64 and 128 rows, bf16 178, 166 | 176, 225; 235, 184 |
//       247, 233; W4A4 61, 49 | 60, 68; 86, 59 | 86, 82; W4 at 128, 512 and 1,024
//       rows 128, 121 | 130, 191; 429, 414 | 428, 416; 825, 761 | 826, 753.
template <int AT, int WT>
static ProductVariant choose(const ProductArgs& a, bool glu) {
  if constexpr (AT == MOE_F8) return choose_f8(a, glu);
  constexpr bool XM = AT == MOE_MXFP4, W4 = !XM && WT == MOE_MXFP4;
  const int64_t n_out = glu ? a.N / 2 : a.N, rows = a.n_rows / a.n_experts;
  auto tiles = [&](int m, int n) { return op_max_tiles(a, m) * ((n_out + n - 1) / n); };
  // the tile kernels address the rows of x of a tile with 32-bit offsets
  if (a.x_ld < (1 << 23)) {
    const int64_t big = glu ? tiles(256, 128) : tiles(256, 256), half = tiles(128, 128), mid = tiles(64, 128);
    auto rounds = [](int64_t n) { return (n + 255) / 256; };
    const bool use_big = a.n_experts == 1 && !glu
                             ? 3 * rounds(half) > (W4 ? 10 : 8) * rounds(big)
                             : big >= (!glu ? 256 : XM && a.n_experts == 1 ? 65 : 128) &&
                                   rows >= (W4 ? 768 : glu ? 128 : XM ? (a.K < 2048 ? 384 : 192) : a.K < 2048 ? 192 : 128);
    if (use_big) return ProductVariant::kBig;
    if (!glu && half > 256 && rows >= (W4 ? 96 : 64)) return ProductVariant::kHalf;
    const bool few = !XM && a.n_experts == 1 && a.n_rows <= 8;
    if (mid >= (W4 ? 129 : 64) && !few)
      return W4 || (!glu && mid > 256) ? ProductVariant::kShared : ProductVariant::kDeep;
  }
  // 16-row blocks while those of W still fill the chip's CUs once: 32 rows of
  // 2048x768 bf16 take 5.3 us in 16 x 16 blocks and 7.6 in 32 x 32, 128 rows of
  // 4096x4096 61 and 34 us (29.5 in 64 x 64).  For 16 rows either may be the faster:
  // W4 4096x4096 8.8 and 12.0, 8192x4096 14.1 and 12.3.
  const int groups = std::min(a.n_experts, a.n_rows);
  const int avg = (a.n_rows + groups - 1) / groups;
  if (avg <= 16 || tiles(16, 16) <= 512) return ProductVariant::kSmall16;
  if (avg <= 64 || tiles(32, 16) <= 512) return ProductVariant::kSmall32;
  return ProductVariant::kSmall64;
}

template <int AT, int WT, bool GLU>
static hipError_t launch_small(const ProductArgs& a, ProductVariant v, hipStream_t s) {
  if (v == ProductVariant::kSmall16) return launch_small_as<AT, WT, GLU, 1, 1>(a, s);
  if (v == ProductVariant::kSmall32) return launch_small_as<AT, WT, GLU, 2, 2>(a, s);
  return launch_small_as<AT, WT, GLU, 4, GLU ? 2 : 4>(a, s);
}

template <int AT, int WT>
static hipError_t launch_typed(const ProductArgs& a, bool glu, hipStream_t s) {
  const ProductVariant v = choose<AT, WT>(a, glu);
  if (v <= ProductVariant::kSmall64) return glu ? launch_small<AT, WT, true>(a, v, s) : launch_small<AT, WT, false>(a, v, s);
  if constexpr (AT == MOE_F8) return launch_tile_f8(a, glu, v, s);
  else if constexpr (AT == MOE_MXFP4) return launch_tile_mx(a, glu, v, s);
  else if constexpr (WT == MOE_MXFP4) return launch_tile_w4(a, glu, v, s);
  else return launch_tile_bf16(a, glu, v, s);
}

hipError_t launch_product(const ProductArgs& a, int x_dtype, int w_dtype, bool glu, hipStream_t s) {
  if (x_dtype == MOE_F8) return launch_typed<MOE_F8, MOE_F8>(a, glu, s);
  if (x_dtype == MOE_MXFP4) return launch_typed<MOE_MXFP4, MOE_MXFP4>(a, glu, s);
  return w_dtype == MOE_MXFP4 ? launch_typed<MOE_BF16, MOE_MXFP4>(a, glu, s)
                              : launch_typed<MOE_BF16, MOE_BF16>(a, glu, s);
}

static ProductVariant product_variant(const ProductArgs& a, int x_dtype, int w_dtype, bool glu) {
  if (x_dtype == MOE_MXFP4) return choose<MOE_MXFP4, MOE_MXFP4>(a, glu);
  return w_dtype == MOE_MXFP4 ? choose<MOE_BF16, MOE_MXFP4>(a, glu) : choose<MOE_BF16, MOE_BF16>(a, glu);
}

}  // namespace moert

// The rule's choice for a product of contiguous rows, as a number: the tests check
// that their sizes reach every variant.  Host arithmetic only; -1 for empty sizes.
extern "C" int moert_product_variant(int x_dtype, int w_dtype, int glu, int n_experts, int n_rows, int N, int K) {
  if (n_experts < 1 || n_rows < 1 || N < 1 || K < 1) return -1;
  moert::ProductArgs a{};
  a.x_ld = x_dtype == MOE_MXFP4 ? K / 2 : (int64_t)K * 2;
  a.n_experts = n_experts;
  a.n_rows = n_rows;
  a.N = N;
  a.K = K;
  return (int)moert::product_variant(a, x_dtype, w_dtype, glu != 0);
}

// The same for F8, whose choice goes by the type of y too.
extern "C" int moert_f8_variant(int y_f32, int glu, int n_experts, int n_rows, int N, int K) {
  if (n_experts < 1 || n_rows < 1 || N < 1 || K < 1) return -1;
  moert::ProductArgs a{};
  a.x_ld = K;
  a.n_experts = n_experts;
  a.n_rows = n_rows;
  a.N = N;
  a.K = K;
  a.y_f32 = y_f32;
  return (int)moert::choose_f8(a, glu != 0);
}
