// Products y = x W^T of F8 operands (e4m3 codes; scales per 128 columns of x and per
// 128 x 128 tile of W), dense or ragged by expert: the variants that stage tiles
// of both operands in LDS.
//
// Precision.  The 8-bit matrix instructions align the products of 8 neighbours of
// K, counted in each 16 bytes of a row, to the largest one's exponent and cut them below 2^-12 of it;
// such sums are then added in fp32 (seen with chosen products; all of the 8-bit shapes
// agree bit for bit).  A product of normal values is off by 1.3e-5 of its size: a 100th of a
// BF16 result's own rounding and less than a 1,000th of what rounding the operands to
// e4m3 moved, but 200 times an FP32 result's 6e-8.  Whole products cost twice the time.  So BF16 results take these instructions: over 8192 x 4096 x
// 4096 they are as far from fp64 as with whole products (1.659e-3 both), though one in 90 is the
// next BF16 value, and further where a sum cancels.  FP32 results expand the codes to bf16
// (exact) and take bf16 ones (Exact), at half the rate.
//
// A workgroup owns up to 16 MaxI WavesM rows of x against 16 NJ WavesN rows of W
// (with GLU half of them gate rows, half the matching up rows); a wave NI x NJ
// blocks of 16 x 16.  K goes in steps of 128, one scale block each: a block's products of
// a step are summed from zero and then join the block's fp32 sums times (x scale *
// W scale).  That costs four multiply-adds per matrix instruction of 32 cycles,
// which run beside the next ones.
//
// Steps pass through two or three LDS stages, by the tile's height, that direct-to-LDS
// loads fill; 16-byte pieces of a row are XOR-swizzled so that the fragment reads of 16
// rows spread over all banks.  The scales of both operands are copied to LDS as they are,
// four steps at a time; each lane reads those of its rows and W's at a step's start and
// keeps their products in registers.
//
// Measured, N = K = 4096: 8192 rows 118-130 us (2.1-2.3 PFLOP/s), 4096 rows 62; FP32 results
// 241 and 133 (1.1; 265 and 143 when a lane's pieces lay 64 bytes apart, which also made the
// stores of 32,008 rows of 2048 take 15 us longer).  Expanding takes its time: converting by
// way of fp32 303 for 263, two products ahead 257 for 259.  A step of the 256 x 256 tile takes 2,830 clocks, 2,048 of them
// products; 16,000 more begin and end the tile.  Power bounds long ones: 4096 x 4096 x
// 16384 takes 217 us, and 171 on constant operands.  Instructions of 32 x 32 x 64 were 7%
// slower, other paces of a step's copies up to 3%.
//
// W is the first MFMA operand: a lane holds four neighbouring columns of one
// row of x per block.  The rows of W lie in LDS in an order that makes what a lane
// stores at once 16 bytes of a row, and 64 bytes what a row's four lanes do: results
// leave in whole pieces without passing through LDS.
#include <type_traits>

#include "product_tile.h"

namespace moert {

// Area: bytes of LDS for the stages.  As many stages as fit, three at most: a short
// tile's products do not cover the latency of its copies, those of 256 rows do.
struct F8Big {
  static constexpr int WavesM = 2, WavesN = 4, MaxI = 8, NJ = 4, Area = 144 << 10, PerCu = 1;
};
struct F8Half {
  static constexpr int WavesM = 2, WavesN = 2, MaxI = 4, NJ = 4, Area = 72 << 10, PerCu = 2;
};
struct F8Mid {
  static constexpr int WavesM = 2, WavesN = 2, MaxI = 2, NJ = 4, Area = 72 << 10, PerCu = 2;
};

template <class C, bool GLU>
struct F8Shape {
  static constexpr int Waves = C::WavesM * C::WavesN, Threads = Waves * 64;
  static constexpr int M = 16 * C::MaxI * C::WavesM, N = 16 * C::NJ * C::WavesN;
  static constexpr int StageB = N * kTileRow;
  static constexpr int Parts = GLU ? 2 : N / 128;      // scale rows of W in a tile
  static constexpr int WaveParts = GLU ? 2 : 1;        // of those a wave's
  static constexpr int BLoads = StageB / (Waves * 1024);  // copies of a wave and step
  static constexpr int Chunk = 4;                      // steps whose scales come at once
};

template <bool GLU, class C, bool Exact>
__global__ __launch_bounds__(64 * C::WavesM * C::WavesN, C::PerCu) void product_f8_kernel(ProductArgs a) {
  using S = F8Shape<C, GLU>;
  using std::integral_constant;
  constexpr int NJ = C::NJ, NT = GLU ? S::N / 2 : S::N;
  __shared__ __attribute__((aligned(1024))) uint8_t s_st[C::Area];
  __shared__ __attribute__((aligned(16))) float s_xs[2][S::M][S::Chunk], s_ws[2][S::Parts][S::Chunk];
  __shared__ int32_t s_y[S::M];  // row of y per tile row, -1 = none
  __shared__ int32_t s_x[S::M];  // row of x (from x0), -1 = none: the product is a row of zeros

  const int n_out = GLU ? a.N / 2 : a.N;
  const int n_ntiles = (n_out + NT - 1) / NT;
  // XCD-aware order, as in product_tile.h: XCD i takes the i-th eighth of a list.
  // It goes by expert, then by groups of six of its M-tiles, then by N-tile: a
  // group that mixed experts would bring the W of those that it cuts twice.
  const OpTiles<true> tiles(a, S::M);
  const int per_xcd = (tiles.total * n_ntiles + 7) >> 3;  // the launch keeps this below 2^31
  const int local = blockIdx.x >> 3, f = (blockIdx.x & 7) * per_xcd + local;
  if (local >= per_xcd || f >= tiles.total * n_ntiles) return;
  OpTile t;
  int lo, n, first;
  if (!tiles.expert(a, S::M, f / n_ntiles, &t.e, &lo, &n, &first)) return;
  constexpr int MGroup = 6;  // 65,536 pairs over 256 experts, N = K = 4096: 2 1,505 us, 4 1,493, 6 and 8 1,485, about a setting's own spread
  const int in_expert = f - first * n_ntiles, grp = in_expert / (MGroup * n_ntiles);
  const int rem = in_expert - grp * MGroup * n_ntiles, in_grp = min(MGroup, (n + S::M - 1) / S::M - grp * MGroup);
  const int nt = rem / in_grp, skip = (grp * MGroup + rem - nt * in_grp) * S::M;
  t.pos0 = lo + skip;
  t.rows = min(S::M, n - skip);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WavesN, wn = wave % C::WavesN;
  const int r = lane & 15, g = lane >> 4;
  const int K = a.K, KB = op_f8_blocks(K);
  const int steps = KB, whole = K / kTileRow;
  const int n0 = nt * NT;

  const uint8_t* const x0 = a.x_index ? a.x : a.x + (int64_t)t.pos0 * a.x_ld;
  const float* const xs0 = (const float*)a.xs + (a.x_index ? 0 : (int64_t)t.pos0 * KB);
  const uint8_t* const w0 = a.w + (int64_t)t.e * a.w_stride;
  const float* const ws0 = (const float*)(a.ws + (int64_t)t.e * a.ws_stride);
  if (tid < S::M) {
    const bool in = tid < t.rows;
    s_y[tid] = in ? op_y_row(a, t.pos0 + tid) : -1;
    s_x[tid] = !in ? -1 : a.x_index ? op_x_row(a, t.pos0 + tid) : tid;
  }
  __syncthreads();
  auto x_row = [&](int m) { return max(s_x[m], 0); };
  // Row of W at place b of the stage.  Places are counted by wave, block j and the
  // block's row w; a lane holds rows 4g..4g+3 of each block.  U blocks share their
  // columns so that a lane's are 16 bytes of a row of y: row w of block j is column
  // (j / U) * 16 U + (w / 4) * 4 U + j % U * 4 + w % 4 of the wave (with GLU of the gate's
  // or the up's half of it).  Columns past the end repeat the last one.
  constexpr int Blocks = GLU ? NJ / 2 : NJ;  // of a wave's columns of y
  constexpr int U = Exact ? 1 : 2;           // Exact: y is FP32, else BF16
  auto w_row = [&](int b) {
    const int wv = b / (16 * NJ), j = b / 16 % NJ, w = b % 16, jb = j % Blocks;
    const int n = n0 + wv * 16 * Blocks + jb / U * 16 * U + w / 4 * 4 * U + jb % U * 4 + w % 4;
    return min(n, n_out - 1) + (j >= Blocks ? n_out : 0);
  };

  auto run = [&](auto ni_c) {
    constexpr int NI = decltype(ni_c)::value;
    constexpr int RowsA = 16 * NI * C::WavesM;
    constexpr int StageA = RowsA * kTileRow, Stage = StageA + S::StageB;
    constexpr int Stages = C::Area / Stage < 3 ? C::Area / Stage : 3;
    static_assert(Stages >= 2 && Stages <= S::Chunk + 1, "a chunk's copies are older than the newest Stages - 2 steps' at its first use");
    constexpr int ALoads = (RowsA + S::Waves * 8 - 1) / (S::Waves * 8);  // a wave copies 8 rows at once
    constexpr int Group = ALoads + S::BLoads;  // copies of a wave per step
    auto arow = [&](int i) { return (i * C::WavesM + wm) * 16; };  // first tile row of block i

    // Copies.  A lane's piece is the same in every row it copies: 8 Waves rows lie
    // between them, a multiple of the swizzle's period.
    const int cr = lane >> 3;
    const int piece = (lane & 7) ^ tile_key(wave * 8 + cr);
    uint32_t a_off[ALoads], b_off[S::BLoads];
#pragma unroll
    for (int q = 0; q < ALoads; ++q)
      a_off[q] = (uint32_t)x_row(min((q * S::Waves + wave) * 8 + cr, S::M - 1)) * (uint32_t)a.x_ld + piece * 16;
#pragma unroll
    for (int q = 0; q < S::BLoads; ++q)
      b_off[q] = (uint32_t)w_row((q * S::Waves + wave) * 8 + cr) * (uint32_t)K + piece * 16;
    auto st_a = [&](int buf) { return s_st + buf * Stage; };
    auto st_b = [&](int buf) { return s_st + buf * Stage + StageA; };
    auto copy = [&](int kt, int buf, int q) {
      if (q < ALoads) tile_copy16(x0 + (int64_t)kt * kTileRow, a_off[q], tile_lds(st_a(buf) + (q * S::Waves + wave) * 1024));
      else tile_copy16(w0 + (int64_t)kt * kTileRow, b_off[q - ALoads], tile_lds(st_b(buf) + ((q - ALoads) * S::Waves + wave) * 1024));
    };
    auto copy_some = [&](int kt, int buf, int from, int to) {
#pragma unroll
      for (int q = 0; q < Group; ++q)
        if (q >= from && q < to) copy(kt, buf, q);
    };
    // the last step, which ends inside: pieces past the row's end become zeros
    auto copy_end = [&](int kt, int buf) {
      if (kt * kTileRow + piece * 16 < K) {
        copy_some(kt, buf, 0, Group);
      } else {
        const op_u32x4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < ALoads; ++q) *(op_u32x4*)(st_a(buf) + (q * S::Waves + wave) * 1024 + lane * 16) = zero;
#pragma unroll
        for (int q = 0; q < S::BLoads; ++q) *(op_u32x4*)(st_b(buf) + (q * S::Waves + wave) * 1024 + lane * 16) = zero;
      }
    };
    // A whole step's copies begin in the last row of blocks of the step Stages before
    // it, when its stage is free, and go on through the first rows of the
    // next one.
    constexpr int Head = 4, PerRow = 2;

    // Scales, four steps' at once, copied as they are: a thread a row of x, and in the
    // next wave a thread a row of W's.  The last chunk begins early enough to end with
    // the row.  Rows of fewer than four come one by one, before the first step.
    auto sc_first = [&](int c) { return min(c * S::Chunk, KB - S::Chunk); };
    const uint32_t sc_off = tid < S::M ? (uint32_t)x_row(tid) * (uint32_t)KB * 4
                                       : (uint32_t)op_f8_w_block(a, GLU, GLU ? n0 : min(n0 + lane * 128, n_out - 1), min(lane, 1)) * (uint32_t)KB * 4;
    auto sc_copy = [&](int c) {
      const int at = sc_first(c);
      if (wave < (RowsA + 63) / 64) tile_copy16(xs0 + at, sc_off, tile_lds(&s_xs[c & 1][wave * 64][0]));
      else if (wave == S::M / 64 && lane < S::Parts) tile_copy16(ws0 + at, sc_off, tile_lds(&s_ws[c & 1][0][0]));
    };
    auto sc_few = [&] {
#pragma unroll
      for (int q = 0; q < S::Chunk; ++q) {
        if (tid < RowsA) s_xs[0][tid][q] = (xs0 + min(q, KB - 1))[sc_off / 4];
        if (wave == S::M / 64 && lane < S::Parts) s_ws[0][lane][q] = (ws0 + min(q, KB - 1))[sc_off / 4];
      }
    };
    const int my_part = GLU ? 0 : wn * 16 * NJ / 128;
    float sc[S::WaveParts][NI];
    auto sc_read = [&](int kt) {
      const int c = kt / S::Chunk, at = KB < S::Chunk ? kt : kt - sc_first(c);
#pragma unroll
      for (int i = 0; i < NI; ++i) sc[0][i] = s_xs[c & 1][arow(i) + r][at];
#pragma unroll
      for (int p = S::WaveParts - 1; p >= 0; --p) {
        const float w = s_ws[c & 1][my_part + p][at];
#pragma unroll
        for (int i = 0; i < NI; ++i) sc[p][i] = sc[0][i] * w;
      }
    };

    op_f32x4 acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = op_f32x4{};

    // fragments: pieces g and 4 + g of a row
    typedef op_u32x4 Frag[2];
    Frag xf[2], wf[NJ];
    // a lane's place in 16 rows, for each of its two pieces; whole blocks of 16 rows
    // leave the swizzle's key as it is
    const uint32_t at0 = tile_at(r, g), at1 = tile_at(r, 4 + g);
    const uint32_t xa = wm * 16 * kTileRow, wa = StageA + wn * NJ * 16 * kTileRow;
    auto read_x = [&](int buf, int i) {
      const uint8_t* p = s_st + buf * Stage + xa + (i % NI) * C::WavesM * 16 * kTileRow;
      xf[i & 1][0] = *(const op_u32x4*)(p + at0);
      xf[i & 1][1] = *(const op_u32x4*)(p + at1);
    };
    auto read_w = [&](int buf, int j) {
      const uint8_t* p = s_st + buf * Stage + wa + j * 16 * kTileRow;
      wf[j][0] = *(const op_u32x4*)(p + at0);
      wf[j][1] = *(const op_u32x4*)(p + at1);
    };
    // Exact: the fragments' codes as bf16, 8 of K each
    op_bf16x8 xb[Exact ? 4 : 1], wb[Exact ? NJ : 1][4];
    auto expand = [](const Frag& v, op_bf16x8 (&to)[4]) {
#pragma unroll
      for (int h = 0; h < 4; ++h) to[h] = op_f8x8_values(v[h / 2][h % 2 * 2], v[h / 2][h % 2 * 2 + 1]);
    };
    auto product = [&](int j, int i) -> op_f32x4 {
      if constexpr (Exact) {
        op_f32x4 v = {};
#pragma unroll
        for (int h = 0; h < 4; ++h) v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[j][h], xb[h], v, 0, 0, 0);
        return v;
      }
      const Frag &w = wf[j], &x = xf[i & 1];
      const op_i32x8 wv = {(int)w[0][0], (int)w[0][1], (int)w[0][2], (int)w[0][3], (int)w[1][0], (int)w[1][1], (int)w[1][2], (int)w[1][3]};
      const op_i32x8 xv = {(int)x[0][0], (int)x[0][1], (int)x[0][2], (int)x[0][3], (int)x[1][0], (int)x[1][1], (int)x[1][2], (int)x[1][3]};
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, xv, op_f32x4{}, 0, 0, 0, 0, 0, 0);
    };
    constexpr int Late = 3;  // products between one and its multiply-adds
    op_f32x4 part[Late + 1];
    auto add = [&](int n) {
      const int i = n / NJ, j = n % NJ;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        acc[i][j][q] = fmaf(sc[GLU ? j / (NJ / 2) : 0][i], part[n % (Late + 1)][q], acc[i][j][q]);
      // the sums have no side effects, and the compiler would move them all behind
      // the step's products, whose results then do not fit the registers
      asm volatile("" : "+v"(acc[i][j]));
    };

    // One step on stage buf, whose first fragments are in place.  steady: Stages more
    // whole steps follow, so exactly Stages - 2 steps' copies are newer than the next one's.
    auto step = [&](int kt, int buf, auto steady_c) {
      constexpr bool steady = decltype(steady_c)::value;
      const bool more = steady || kt + 1 < steps;
      const int next = buf + 1 == Stages ? 0 : buf + 1, before = buf == 0 ? Stages - 1 : buf - 1;
      sc_read(kt);
      if (kt % S::Chunk == 0 && kt + S::Chunk < steps) sc_copy(kt / S::Chunk + 1);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const bool last = i + 1 == NI;
        if (!last) {
          read_x(buf, i + 1);
        } else if (more) {
          // everyone has read this stage, and the next one is there
          if (steady) tile_sync<(Stages - 2) * Group>();
          else tile_sync<0>();
          read_x(next, NI);  // NI is even: fragment 0
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int n = i * NJ + j;
          if constexpr (Exact) {
            if (i == 0) expand(wf[j], wb[j]);
            if (j == 0) expand(xf[i & 1], xb);
          }
          part[n % (Late + 1)] = product(j, i);
          if (n >= Late) add(n - Late);
          if (last && more) read_w(next, j);  // over the fragment that was just used
          if (steady || kt + Stages - (last ? 0 : 1) < whole) {
            const int from = last ? 0 : Head + i * PerRow;
            const int most = last ? Head : i + 2 == NI ? Group : min(from + PerRow, Group);
            const int at = from + (most - from) * j / NJ, to = from + (most - from) * (j + 1) / NJ;
            copy_some(kt + Stages - (last ? 0 : 1), last ? buf : before, at, to);
          }
          __builtin_amdgcn_sched_barrier(0);  // the order as written
        }
      }
#pragma unroll
      for (int n = NI * NJ - Late; n < NI * NJ; ++n) add(n);
      if (!steady && kt + Stages == whole && whole < steps) copy_end(whole, buf);
    };

    if (KB < S::Chunk) sc_few();
    else sc_copy(0);
#pragma unroll
    for (int kt = 0; kt < Stages; ++kt) {
      if (kt < whole) copy_some(kt, kt, 0, kt + 1 < Stages ? Group : Head);
      else if (kt < steps) copy_end(kt, kt);
    }
    if (whole >= Stages) tile_sync<(Stages - 2) * Group + Head>();
    else tile_sync<0>();
    read_x(0, 0);
#pragma unroll
    for (int j = 0; j < NJ; ++j) read_w(0, j);
    int kt = 0, buf = 0;
#pragma unroll 1
    for (; kt + Stages < whole; ++kt) {
      step(kt, buf, std::true_type{});
      buf = buf + 1 == Stages ? 0 : buf + 1;
    }
#pragma unroll 1
    for (; kt < steps; ++kt) {
      step(kt, buf, std::false_type{});
      buf = buf + 1 == Stages ? 0 : buf + 1;
    }

    // Result: 16 bytes of a row per lane, 64 of its four lanes
    const int col = n0 + wn * 16 * Blocks + g * 4 * U;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int m = arow(i) + r;
      const int row = s_y[m];
      if (row < 0) continue;
      const bool live = s_x[m] >= 0;
      uint8_t* const y = (uint8_t*)a.y + (int64_t)row * a.ldy * (Exact ? 4 : 2);
#pragma unroll
      for (int h = 0; h < Blocks / U; ++h) {
        float v[4 * U];
#pragma unroll
        for (int q = 0; q < 4 * U; ++q) {
          const int j = h * U + q / 4;
          const float z = GLU ? op_silu_mul(acc[i][j][q % 4], acc[i][GLU ? j + Blocks : 0][q % 4]) : acc[i][j][q % 4];
          v[q] = live ? z : 0.f;
        }
        const int c = col + h * 16 * U, n = n_out - c;
        if constexpr (!Exact) {
          op_cols_store(y, false, c, n, v);
        } else if (n >= 4) {
          *(op_bytes16*)((float*)y + c) = op_u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        } else {
#pragma unroll
          for (int q = 0; q < 3; ++q)
            if (q < n) ((float*)y)[c + q] = v[q];
        }
      }
    }
  };
  const int ni = (t.rows + 32 * C::WavesM - 1) / (32 * C::WavesM);  // pairs of row blocks per wave
  if constexpr (C::MaxI == 2) {
    run(integral_constant<int, 2>{});
  } else if constexpr (C::MaxI == 4) {
    if (ni == 1) run(integral_constant<int, 2>{});
    else run(integral_constant<int, 4>{});
  } else {
    switch (ni) {
      case 1: run(integral_constant<int, 2>{}); break;
      case 2: run(integral_constant<int, 4>{}); break;
      case 3: run(integral_constant<int, 6>{}); break;
      default: run(integral_constant<int, 8>{}); break;
    }
  }
}

template <bool GLU, class C, bool Exact>
static hipError_t launch_f8_as(const ProductArgs& a, hipStream_t s) {
  using S = F8Shape<C, GLU>;
  const int n_out = GLU ? a.N / 2 : a.N, nt = GLU ? S::N / 2 : S::N;
  const int64_t n_ntiles = (n_out + nt - 1) / nt;
  const int64_t wgs = (op_max_tiles(a, S::M) * n_ntiles + 7) / 8 * 8;
  if (wgs * S::Threads >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  return launch_op(product_f8_kernel<GLU, C, Exact>, dim3((unsigned)wgs), dim3(S::Threads), s, a);
}

template <bool GLU>
static hipError_t launch_f8(const ProductArgs& a, ProductVariant v, hipStream_t s) {
  if (v == ProductVariant::kBig) return launch_f8_as<GLU, F8Big, false>(a, s);
  if (v == ProductVariant::kHalf) return a.y_f32 ? launch_f8_as<GLU, F8Half, true>(a, s) : launch_f8_as<GLU, F8Half, false>(a, s);
  return a.y_f32 ? launch_f8_as<GLU, F8Mid, true>(a, s) : launch_f8_as<GLU, F8Mid, false>(a, s);
}

hipError_t launch_tile_f8(const ProductArgs& a, bool glu, ProductVariant v, hipStream_t s) {
  return glu ? launch_f8<true>(a, v, s) : launch_f8<false>(a, v, s);
}

}  // namespace moert
