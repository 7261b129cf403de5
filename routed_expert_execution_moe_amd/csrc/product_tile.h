// Products y = x W^T, dense or ragged by expert: the variant for many rows.
//
// A workgroup of four waves owns a tile of up to 256 rows of x against 256
// rows of W (with GLU: 128 gate rows and the matching 128 up rows), in
// v_mfma 32x32 blocks with fp32 accumulation.  The waves stand side by side:
// each takes all of the tile's rows by 64 rows of W, NI x 2 blocks with NI =
// ceil(rows / 32), so a short last tile of an expert costs only the blocks it
// fills and loads every wave alike.  Per block pair a wave reads (NI + 2)
// fragments from LDS for 2 NI products, 0.63 at NI = 8.
//
// K goes in steps of 128 bytes of a row (64 bf16, 256 MXFP4) through two LDS
// stages.  Direct-to-LDS loads fill a stage one whole step before it is
// needed; 16-byte pieces of a row are XOR-swizzled so that the fragment reads
// of 32 rows spread over the banks.  Fragments are read one slice (a quarter
// of a step) ahead of the products that use them, also across the one barrier
// per step, which sits before a step's last slice: from there on every wave
// has read the stage, so the loads of the step after next may overwrite it.
//
// W is the first MFMA operand: a lane holds, of one row of y, four neighbouring
// columns at a time.  The result passes through LDS once more, so that rows
// leave in 16-byte pieces.
//
// Formats: bf16 x bf16 uses v_mfma_f32_32x32x16_bf16; MXFP4 x MXFP4 the scaled
// v_mfma 32x32x64 on the codes as they are, each lane passing the scale of its
// 32-element piece, held in registers (loaded one step ahead straight from
// memory: 8 bytes of a row per step); bf16 x MXFP4 keeps W as codes in LDS and
// expands a fragment with the scaled converts right before its products.
#pragma once

#include <type_traits>

#include "ops.h"

namespace moert {

constexpr int kTlM = 256, kTlN = 256, kTlRow = 128;
constexpr int kTlThreads = 256;
constexpr int kTlStageA = kTlM * kTlRow;

template <int AT, int WT>
struct TileShape {
  static constexpr bool XM = AT == MOE_MXFP4, WM = WT == MOE_MXFP4, W4 = WM && !XM;
  static constexpr int K = XM ? 256 : 64;        // elements of a step
  static constexpr int WRow = W4 ? 32 : kTlRow;  // bytes of a W row per step
  static constexpr int StageB = kTlN * WRow;
  static constexpr int BLoads = StageB / 4096;   // per wave and step
};

// 16 bytes per lane from base + voff to LDS at lds + 16 * lane
__device__ inline void tile_copy16(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               ::"v"(voff), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ inline uint32_t tile_lds(const void* p) { return (uint32_t)(uintptr_t)p; }

// place of 16-byte piece c of row r: two rows fill the 64 banks once, so the
// key changes every second row
__device__ inline int tile_at(int r, int c) { return r * kTlRow + ((c ^ ((r >> 1) & 7)) << 4); }

template <int AT, int WT, bool GLU>
__global__ __launch_bounds__(kTlThreads, 1) void product_tile_kernel(ProductArgs a) {
  using S = TileShape<AT, WT>;
  __shared__ __attribute__((aligned(1024))) uint8_t s_a[2][kTlStageA];
  __shared__ __attribute__((aligned(1024))) uint8_t s_b[2][S::StageB];
  __shared__ int32_t s_y[kTlM];     // row of y per tile row, -1 = none
  __shared__ uint8_t s_live[kTlM];  // 0: the product is a row of zeros

  const int n_out = GLU ? a.N / 2 : a.N;
  constexpr int NT = GLU ? kTlN / 2 : kTlN;
  const int n_ntiles = (n_out + NT - 1) / NT;

  // XCD-aware order: workgroups go round-robin over the 8 XCDs; XCD i takes the
  // i-th eighth of the M-tiles, in groups of four with the N-tiles outside,
  // so what runs together on an XCD shares rows of x and of W in its L2
  const OpTiles tiles(a, kTlM);
  const int xcd = blockIdx.x & 7, local = blockIdx.x >> 3;
  const int per_xcd = (tiles.total + 7) >> 3;
  const int grp = local / (4 * n_ntiles), rem = local - grp * 4 * n_ntiles;
  const int ml = grp * 4 + (rem & 3), nt = rem >> 2;
  OpTile t;
  if (ml >= per_xcd || !tiles.find(a, kTlM, xcd * per_xcd + ml, &t)) return;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 31, kg = lane >> 5;
  const int K = a.K, blocks = K / 32;
  const int x_bytes = S::XM ? K / 2 : K * 2;
  const int steps = (x_bytes + kTlRow - 1) / kTlRow;
  const int n0 = nt * NT;

  // every position's row of x once; a position without one, and the padding of
  // a short tile, read the tile's first valid row instead
  {
    const int p = t.pos0 + tid;
    const bool in = tid < t.rows;
    s_y[tid] = in ? op_y_row(a, p) : -1;
    s_live[tid] = in && op_x_row(a, p) >= 0;
  }
  // base of the tile's rows of x: the whole of x under an index (32-bit offsets),
  // else the tile's first row
  const uint8_t* x0 = a.x_index ? a.x : a.x + (int64_t)t.pos0 * a.x_ld;
  auto x_row = [&](int m) {
    if (!a.x_index) return m < t.rows ? m : 0;
    return max(m < t.rows ? op_x_row(a, t.pos0 + m) : -1, 0);
  };
  // row of W of tile row b, those past the end repeat the last one
  auto w_row = [&](int b) {
    if (GLU) return min(n0 + (b & (NT - 1)), n_out - 1) + (b >= NT ? n_out : 0);
    return min(n0 + b, n_out - 1);
  };

  auto run = [&](auto ni_c) {
    constexpr int NI = decltype(ni_c)::value;

    // Copies.  A lane's piece is the same in every row it copies: 32 rows lie
    // between them, a multiple of the swizzle's period.
    const int r8 = lane >> 3;
    const int piece = (lane & 7) ^ (((wave * 8 + r8) >> 1) & 7);
    uint32_t a_off[NI], b_off[S::BLoads];
#pragma unroll
    for (int q = 0; q < NI; ++q)
      a_off[q] = (uint32_t)x_row((q * 4 + wave) * 8 + r8) * (uint32_t)a.x_ld + piece * 16;
    const uint8_t* const w0 = a.w + (int64_t)t.e * a.w_stride;
    const int half = (lane & 1) ^ ((lane >> 4) & 1);  // W4: rows 8 apart share banks, their halves swap
#pragma unroll
    for (int q = 0; q < S::BLoads; ++q)
      b_off[q] = S::W4 ? (uint32_t)w_row((q * 4 + wave) * 32 + (lane >> 1)) * (uint32_t)(K / 2) + half * 16
                       : (uint32_t)w_row((q * 4 + wave) * 8 + r8) * (uint32_t)x_bytes + piece * 16;

    auto copy_a = [&](int kt, int buf) {
      const uint8_t* xb = x0 + (int64_t)kt * kTlRow;
#pragma unroll
      for (int q = 0; q < NI; ++q) tile_copy16(xb, a_off[q], tile_lds(s_a[buf] + wave * 1024 + q * 4096));
    };
    auto copy_b = [&](int kt, int buf) {
      const uint8_t* wb = w0 + (int64_t)kt * S::WRow;
#pragma unroll
      for (int q = 0; q < S::BLoads; ++q) tile_copy16(wb, b_off[q], tile_lds(s_b[buf] + wave * 1024 + q * 4096));
    };
    // a step that ends inside: pieces past the row's end become zeros
    auto issue_end = [&](int kt, int buf) {
      const op_u32x4 zero = {0, 0, 0, 0};
      const bool a_in = kt * kTlRow + piece * 16 < x_bytes;
      if (a_in) {
        copy_a(kt, buf);
      } else {
#pragma unroll
        for (int q = 0; q < NI; ++q) *(op_u32x4*)(s_a[buf] + wave * 1024 + q * 4096 + lane * 16) = zero;
      }
      if (S::W4 ? kt * 2 + half < blocks : a_in) {
        copy_b(kt, buf);
      } else {
#pragma unroll
        for (int q = 0; q < S::BLoads; ++q) *(op_u32x4*)(s_b[buf] + wave * 1024 + q * 4096 + lane * 16) = zero;
      }
    };

    // this wave's W rows within the tile: blocks j = 0, 1
    int brow[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) brow[j] = (GLU ? j * NT + wave * 32 : wave * 64 + j * 32) + lr;

    // scales: MXFP4 x MXFP4 8 bytes per row and step, shifted so that this
    // half's blocks 2 ks + kg are bytes 0 and 2 of the two words; W4 one byte
    uint2 sx[S::XM ? NI : 1], sw[2], sx_n[S::XM ? NI : 1], sw_n[2];
    uint32_t sx_off[S::XM ? NI : 1], sw_off[2];
    const uint8_t* const xs0 = S::XM ? (a.x_index ? a.xs : a.xs + (int64_t)t.pos0 * blocks) : nullptr;
    const uint8_t* const ws0 = S::WM ? a.ws + (int64_t)t.e * a.ws_stride : nullptr;
    if constexpr (S::XM)
#pragma unroll
      for (int i = 0; i < NI; ++i) sx_off[i] = (uint32_t)x_row(i * 32 + lr) * (uint32_t)blocks;
    if constexpr (S::WM)
#pragma unroll
      for (int j = 0; j < 2; ++j) sw_off[j] = (uint32_t)w_row(brow[j]) * (uint32_t)blocks;
    auto load_scales = [&](int kt) {
      if constexpr (S::XM) {
        // the last step may end inside its 8 blocks: it reads the row's last 8
        // and shifts them down below
        const int b = min(kt * 8, blocks - 8);
#pragma unroll
        for (int i = 0; i < NI; ++i) __builtin_memcpy(&sx_n[i], xs0 + b + sx_off[i], 8);
#pragma unroll
        for (int j = 0; j < 2; ++j) __builtin_memcpy(&sw_n[j], ws0 + b + sw_off[j], 8);
      } else if constexpr (S::W4) {
        const int b = kt * 2 + kg;
#pragma unroll
        for (int j = 0; j < 2; ++j) sw_n[j].x = b < blocks ? ws0[sw_off[j] + b] : 127;
      }
    };
    // claimed here, right after a wait for every load, so that the compiler's own
    // wait for these loads does not fall behind the next stage's copies
    auto take_scales = [&](int kt, bool whole_step) {
      auto take = [&](uint2 v) {
        asm volatile("" : "+v"(v.x), "+v"(v.y));
        const int past = kt * 8 + 8 - blocks;  // blocks past the row's end: scale 1
        if (!whole_step && past > 0) {         // (their codes are zeros, but zero times a NaN scale is not)
          uint64_t d = (uint64_t)v.y << 32 | v.x;
          d = d >> (8 * past) | 0x7F7F7F7F7F7F7F7Full << (64 - 8 * past);
          v = make_uint2((uint32_t)d, (uint32_t)(d >> 32));
        }
        return make_uint2(v.x >> (8 * kg), v.y >> (8 * kg));
      };
      if constexpr (S::XM) {
#pragma unroll
        for (int i = 0; i < NI; ++i) sx[i] = take(sx_n[i]);
#pragma unroll
        for (int j = 0; j < 2; ++j) sw[j] = take(sw_n[j]);
      } else if constexpr (S::W4) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          asm volatile("" : "+v"(sw_n[j].x));
          sw[j].x = sw_n[j].x;
        }
      }
    };

    op_f32x16 acc[NI][2];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = op_f32x16{};

    // fragments of slice ks: x piece 2 ks + kg of a row (W4: 4 kg + ks, so that
    // a lane's codes of a step are one piece under one scale)
    op_u32x4 fx[2][NI], fw[2][2];
    auto read = [&](int buf, int ks, int to) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        fx[to][i] = *(const op_u32x4*)(s_a[buf] + tile_at(i * 32 + lr, S::W4 ? 4 * kg + ks : 2 * ks + kg));
      if constexpr (!S::W4) {
#pragma unroll
        for (int j = 0; j < 2; ++j) fw[to][j] = *(const op_u32x4*)(s_b[buf] + tile_at(brow[j], 2 * ks + kg));
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          fw[to][j][0] = *(const uint32_t*)(s_b[buf] + brow[j] * 32 + ((kg ^ ((brow[j] >> 3) & 1)) << 4) + ks * 4);
      }
    };
    auto multiply = [&](auto ks_c, int from) {
      constexpr int ks = decltype(ks_c)::value;
      if constexpr (S::XM) {
        op_i32x8 wv[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          wv[j] = op_i32x8{(int)fw[from][j][0], (int)fw[from][j][1], (int)fw[from][j][2], (int)fw[from][j][3], 0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const op_i32x8 xv = {(int)fx[from][i][0], (int)fx[from][i][1], (int)fx[from][i][2], (int)fx[from][i][3], 0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                wv[j], xv, acc[i][j], 4, 4, (ks & 1) * 2, (int)(ks < 2 ? sw[j].x : sw[j].y), (ks & 1) * 2,
                (int)(ks < 2 ? sx[i].x : sx[i].y));
        }
      } else {
        op_bf16x8 wv[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if constexpr (S::W4) wv[j] = op_fp4x8(fw[from][j][0], op_scale(sw[j].x));
          else wv[j] = __builtin_bit_cast(op_bf16x8, fw[from][j]);
        }
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wv[j], __builtin_bit_cast(op_bf16x8, fx[from][i]),
                                                                acc[i][j], 0, 0, 0);
      }
    };
    // Products have no side effects, and the compiler sinks the scaled ones below
    // the step's barrier, past reads whose fragments then do not fit the
    // registers: an empty asm on every sum keeps a slice's products in place.
    auto hold = [&] {
      if constexpr (S::XM) {
#pragma unroll
        for (int i = 0; i < NI; ++i) asm volatile("" : "+a"(acc[i][0]), "+a"(acc[i][1]));
      }
    };
    using std::integral_constant;
    // one step on stage buf; slice 0 is in fragments 0.  steady: steps kt + 1 and
    // kt + 2 exist and are whole
    const int whole = x_bytes / kTlRow;
    auto step = [&](int kt, int buf, auto steady_c) {
      constexpr bool steady = decltype(steady_c)::value;
      const bool more = steady || kt + 1 < steps;
      if (more) load_scales(kt + 1);
      read(buf, 1, 1);
      multiply(integral_constant<int, 0>{}, 0);
      hold();
      read(buf, 2, 0);
      multiply(integral_constant<int, 1>{}, 1);
      hold();
      read(buf, 3, 1);
      multiply(integral_constant<int, 2>{}, 0);
      hold();
      if (more) {
        // this wave's copies into the other stage have landed and its reads of
        // this one are done
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (steady || kt + 2 < whole) {
          copy_a(kt + 2, buf);
          copy_b(kt + 2, buf);
        } else if (kt + 2 < steps) {
          issue_end(kt + 2, buf);
        }
        read(buf ^ 1, 0, 0);
      }
      multiply(integral_constant<int, 3>{}, 1);
      if (more) take_scales(kt + 1, steady);
    };

    load_scales(0);
    for (int kt = 0; kt < min(steps, 2); ++kt) {
      if (kt < whole) {
        copy_a(kt, kt);
        copy_b(kt, kt);
      } else {
        issue_end(kt, kt);
      }
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    take_scales(0, false);
    read(0, 0, 0);
    int kt = 0;
    for (; kt + 3 < whole; kt += 2) {
      step(kt, 0, std::true_type{});
      step(kt + 1, 1, std::true_type{});
    }
#pragma unroll 1
    for (; kt < steps; ++kt) step(kt, kt & 1, std::false_type{});

    // Result.  Element r of a lane's block: row lr of x, W row 8 (r/4) + 4 kg +
    // r%4.  32 rows at a time go through this wave's part of the first stage.
    constexpr int CW = GLU ? 32 : 64, CS = CW + 4;  // columns of a wave, padded stride
    constexpr int LPR = CW / 4, RPI = 64 / LPR;     // lanes per row, rows per pass
    static_assert(4 * 32 * CS * 4 <= 2 * kTlStageA, "the staging fits the x stages");
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // every wave is done with the stages
    float* const c = (float*)&s_a[0][0] + wave * (32 * CS);
    const int c4 = (lane % LPR) * 4, rs = lane / LPR;
    const int col = n0 + wave * CW + c4;
    const bool wide = a.y_f32 ? (((uintptr_t)a.y & 15) | (a.ldy & 3)) == 0 : (((uintptr_t)a.y & 7) | (a.ldy & 3)) == 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int j = 0; j < (GLU ? 1 : 2); ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          op_f32x4 v;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            v[u] = GLU ? op_silu_mul(acc[i][0][q * 4 + u], acc[i][1][q * 4 + u]) : acc[i][j][q * 4 + u];
          *(op_f32x4*)&c[lr * CS + j * 32 + q * 8 + kg * 4] = v;
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's rows are in LDS
#pragma unroll 2
      for (int q = 0; q < 32 / RPI; ++q) {
        const int rl = q * RPI + rs, m = i * 32 + rl;
        const int row = s_y[m];
        op_f32x4 v = *(const op_f32x4*)&c[rl * CS + c4];
        if (!s_live[m]) v = op_f32x4{0.f, 0.f, 0.f, 0.f};
        if (row < 0) continue;
        const int64_t at = (int64_t)row * a.ldy + col;
        if (wide && col + 4 <= n_out) {
          if (a.y_f32) *(op_f32x4*)((float*)a.y + at) = v;
          else
            *(uint2*)((uint16_t*)a.y + at) = make_uint2(op_bf16(v[0]) | (uint32_t)op_bf16(v[1]) << 16,
                                                        op_bf16(v[2]) | (uint32_t)op_bf16(v[3]) << 16);
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (col + u < n_out) {
              if (a.y_f32) ((float*)a.y)[at + u] = v[u];
              else ((uint16_t*)a.y)[at + u] = op_bf16(v[u]);
            }
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next 32 rows overwrite them
    }
  };
  switch ((t.rows + 31) >> 5) {
    case 1: run(std::integral_constant<int, 1>{}); break;
    case 2: run(std::integral_constant<int, 2>{}); break;
    case 3:
    case 4: run(std::integral_constant<int, 4>{}); break;
    case 5:
    case 6: run(std::integral_constant<int, 6>{}); break;
    default: run(std::integral_constant<int, 8>{}); break;
  }
}

template <int AT, int WT>
hipError_t launch_tile(const ProductArgs& a, bool glu, hipStream_t s) {
  const int n_out = glu ? a.N / 2 : a.N, nt = glu ? kTlN / 2 : kTlN;
  const int64_t n_ntiles = (n_out + nt - 1) / nt;
  const int64_t per_xcd = (op_max_tiles(a, kTlM) + 7) / 8;
  const int64_t wgs = 8 * ((per_xcd + 3) / 4 * 4) * n_ntiles;
  if (wgs * kTlThreads >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  return launch_op(glu ? product_tile_kernel<AT, WT, true> : product_tile_kernel<AT, WT, false>,
                   dim3((unsigned)wgs), dim3(kTlThreads), s, a);
}

}  // namespace moert
