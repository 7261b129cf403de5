// Products y = x W^T, dense or ragged by expert: the variants that stage tiles
// of both operands in LDS.
//
// A workgroup owns a tile of up to 32 MaxI WavesM rows of x against 128 J rows of
// W (with GLU, J = 2: 128 gate rows and the matching 128 up rows), in v_mfma 32x32
// blocks with fp32 accumulation.  Four waves stand side by side along W, 32 J rows
// each, against all row blocks of the tile, NI = ceil(rows / 32) of them; eight
// waves stand in two such rows, which take the row blocks in turn.  So a short
// last tile of an expert costs only the blocks it fills and loads every wave
// alike.
//
// K goes in steps of 128 bytes of a row (64 bf16 or 256 MXFP4) through a ring of
// LDS stages that direct-to-LDS loads fill Stages - 1 steps ahead; 16-byte pieces
// of a row are XOR-swizzled so that the fragment reads of 32 rows spread over the
// banks.  Fragments are read one slice (a quarter of a step) ahead of
// the products that use them, also across the one barrier per step, which sits
// before a step's last slice: from there on every wave has read the stage, so
// the next copies may overwrite it.
//
// W is the first MFMA operand: a lane holds, of one row of y, four neighbouring
// columns at a time.  The result passes through LDS once more, so that rows
// leave in 16-byte pieces.
//
// Formats: bf16 x bf16 uses v_mfma_f32_32x32x16_bf16; MXFP4 x MXFP4 the scaled
// v_mfma 32x32x64 on the codes as they are, each lane passing the scale of its
// 32-element piece; bf16 x MXFP4 keeps W as codes in LDS and expands a fragment
// with the scaled converts right before its products.
//
// Shapes.  Big, 256 x 256 with eight waves and two stages: a wave reads (NI + 2)
// fragments from LDS per 2 NI products, 0.75 at NI = 4, and two waves on a SIMD fill
// each other's waits (four waves with 128 x 2 blocks read 0.63 and leave one wave
// alone with its own: W4A4 8192 x 4096 x 4096 86.4 us, eight 80.0 then; bf16 222 and 215).
// Half, 128 x 128, and Mid, 64 x 128 (GLU 64 x 256), with four waves, for products
// whose larger tiles would leave CUs without one or spend their time before and
// after a short K.  They stay within 80 KB of LDS, so that one workgroup's first
// and last latencies are another's products; but Deep (Mid with more stages) has a
// CU to itself, where there are too few tiles to share one, and so has every GLU
// tile but W4's.
//
// 8192 x 4096 x 4096 takes 74-79 us with MXFP4 operands (3.5-3.7 PFLOP/s)
// and 208-217 us with bf16 (1.27-1.32).  A Big tile's time in clocks, 4096 x
// 4096 x 4096, W4A4: 1,300 to find it, 1,300 for its rows, 4,500 until the first stage
// is there; 33,000 of products within a loop of 48,200, whose rest waits for copies
// and fragments; 10,000 while all CUs write their tiles at once.  Steps of 64 bytes
// in four stages, tried with four waves, hide the waits of one tile alone better
// (1.04 against 1.11 us per 128 bytes of bf16), but asking for half cache lines costs
// more with all CUs at work (119 against 113 us).
#pragma once

#include <type_traits>

#include "ops.h"

namespace moert {

constexpr int kTileRow = 128;  // bytes of a row per step
typedef unsigned int tile_bytes16 __attribute__((ext_vector_type(4), aligned(1)));

template <int AT, int WT>
struct TileBig {
  static constexpr bool W4 = WT == MOE_MXFP4 && AT == MOE_BF16;
  static constexpr int Waves = 8, MaxI = 4, J = 2, Stages = W4 ? 3 : 2;
  static constexpr bool Unroll = !W4;
  // W4A4: 48 spills registers within the loop, 82.4 us for 80.0 (32: three, one with GLU, outside of it)
  static constexpr int ScaleBytes = WT != MOE_MXFP4 ? 0 : W4 ? 64 : 32;
};
template <int AT, int WT, bool GLU, bool Deep>
struct TileMid {
  static constexpr int Waves = 4, MaxI = 2, J = GLU ? 2 : 1;
  static constexpr bool Unroll = false;
  static constexpr int Stages = WT == MOE_MXFP4 && AT == MOE_BF16 ? 3 : !Deep ? 2 : GLU ? 3 : 4;
  static constexpr int ScaleBytes = WT != MOE_MXFP4 ? 0 : 64;
};

template <int AT, int WT>
struct TileHalf {
  static constexpr int Waves = 4, MaxI = 4, J = 1, Stages = 2;
  static constexpr bool Unroll = false;
  static constexpr int ScaleBytes = WT != MOE_MXFP4 ? 0 : 48;
};

template <int AT, int WT, class C>
struct TileShape {
  static constexpr bool XM = AT == MOE_MXFP4, WM = WT == MOE_MXFP4, W4 = WM && !XM;
  static constexpr int Waves = C::Waves, WavesM = Waves / 4, Threads = Waves * 64;
  static constexpr int M = 32 * C::MaxI * WavesM, N = 128 * C::J;
  static constexpr int Row = kTileRow, Parts = Row / 16;  // bytes, 16-byte pieces of a row per step
  static constexpr int WRow = W4 ? Row / 4 : Row;         // bytes of a W row per step
  static constexpr int StageA = M * Row, StageB = N * WRow, Stage = StageA + StageB;
  static constexpr int CopyRows = 1024 / Row;   // rows of one copy of a wave
  static constexpr int BLoads = StageB / (Waves * 1024);  // per wave and step
  static constexpr int ScalePitch = C::ScaleBytes + 8;  // 2 banks more than a multiple of 4
  static constexpr int ScaleRows = XM ? M + N : WM ? N : 0;
  static constexpr int ScaleTurns = (ScaleRows + Threads - 1) / Threads;
  static constexpr int StepBlocks = XM ? Row / 16 : 2;   // scales of a row per step
};

// 16 bytes per lane from base + voff to LDS at lds + 16 * lane
__device__ inline void tile_copy16(const void* base, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               ::"v"(voff), "s"(base), "s"(lds) : "memory", "m0");
}
// an LDS address that is the same in every lane, as a scalar
__device__ inline uint32_t tile_lds(const void* p) { return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)p); }

// swizzle key of row r and place of its 16-byte piece c: two rows fill the 64
// banks once, so the key changes from one pair to the next
__device__ inline int tile_key(int r) { return (r >> 1) & 7; }
__device__ inline int tile_at(int r, int c) { return r * kTileRow + ((c ^ tile_key(r)) << 4); }

// this wave's reads and all but its newest N copies are done, and every wave is here
template <int N>
__device__ inline void tile_sync() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(N) : "memory");
}

template <int AT, int WT, bool GLU, class C>
__global__ __launch_bounds__(C::Waves * 64, 1) void product_tile_kernel(ProductArgs a) {
  using S = TileShape<AT, WT, C>;
  using std::integral_constant;
  constexpr int J = C::J, Stages = C::Stages;
  static_assert(!GLU || J == 2, "a wave holds the gate and the up block of its columns");
  __shared__ __attribute__((aligned(1024))) uint8_t s_st[Stages * S::Stage];
  __shared__ __attribute__((aligned(16))) uint8_t s_sc[16 + S::ScaleRows * S::ScalePitch];
  __shared__ int32_t s_y[S::M];  // row of y per tile row, -1 = none
  __shared__ int32_t s_x[S::M];  // row of x (from x0), -1 = none: the product is a row of zeros

  const int n_out = GLU ? a.N / 2 : a.N;
  constexpr int NT = GLU ? S::N / 2 : S::N;
  const int n_ntiles = (n_out + NT - 1) / NT;

  // XCD-aware order: workgroups go round-robin over the 8 XCDs.  The tiles are
  // listed in groups of four M-tiles with the N-tiles outside, and XCD i takes the
  // i-th eighth of the list, so what runs together on an XCD shares rows of x and
  // of W in its L2.  Workgroups without a tile come last: between others they
  // would leave their turn of the shader engines empty (every fourth one with
  // work put all work on a quarter of the CUs).
  const OpTiles<!(S::XM && S::Waves == 8)> tiles(a, S::M);
  const int per_xcd = (tiles.total * n_ntiles + 7) >> 3;  // the launch keeps this below 2^31
  const int local = blockIdx.x >> 3, f = (blockIdx.x & 7) * per_xcd + local;
  if (local >= per_xcd || f >= tiles.total * n_ntiles) return;
  const int grp = f / (4 * n_ntiles), rem = f - grp * 4 * n_ntiles;
  const int in_grp = min(4, tiles.total - grp * 4);
  const int nt = rem / in_grp;
  OpTile t;
  if (!tiles.find(a, S::M, grp * 4 + rem - nt * in_grp, &t)) return;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;  // the wave's place along the rows of x and of W
  const int lr = lane & 31, kg = lane >> 5;
  const int K = a.K, blocks = K / 32;
  const int x_bytes = S::XM ? K / 2 : K * 2;
  const int steps = (x_bytes + S::Row - 1) / S::Row;
  const int whole = x_bytes / S::Row;  // steps that do not end inside
  const int n0 = nt * NT;

  // base of the tile's rows of x: the whole of x under an index (32-bit offsets),
  // else the tile's first row.  The padding of a short tile, and positions
  // without a row of x, read the first row.
  const uint8_t* const x0 = a.x_index ? a.x : a.x + (int64_t)t.pos0 * a.x_ld;
  const uint8_t* const w0 = a.w + (int64_t)t.e * a.w_stride;
  const uint8_t* const xs0 = S::XM ? (a.x_index ? a.xs : a.xs + (int64_t)t.pos0 * blocks) : nullptr;
  const uint8_t* const ws0 = S::WM ? a.ws + (int64_t)t.e * a.ws_stride : nullptr;
  if (tid < S::M) {
    const bool in = tid < t.rows;
    s_y[tid] = in ? op_y_row(a, t.pos0 + tid) : -1;
    s_x[tid] = !in ? -1 : a.x_index ? op_x_row(a, t.pos0 + tid) : tid;
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  auto x_row = [&](int m) { return max(s_x[m], 0); };
  // row of W of tile row b, those past the end repeat the last one
  auto w_row = [&](int b) {
    if (GLU) return min(n0 + (b & (NT - 1)), n_out - 1) + (b >= NT ? n_out : 0);
    return min(n0 + b, n_out - 1);
  };

  auto run = [&](auto ni_c) {
    constexpr int NI = decltype(ni_c)::value;
    constexpr int ALoads = (NI * S::WavesM * 32 + S::Waves * S::CopyRows - 1) / (S::Waves * S::CopyRows);
    constexpr int Group = ALoads + S::BLoads;  // copies of one wave per step

    // Copies.  A lane's piece is the same in every row it copies: Waves CopyRows rows
    // lie between them, a multiple of the swizzle's period.
    const int cr = lane / S::Parts;
    const int piece = (lane % S::Parts) ^ tile_key(wave * S::CopyRows + cr);
    uint32_t a_off[ALoads], b_off[S::BLoads];
#pragma unroll
    for (int q = 0; q < ALoads; ++q)
      a_off[q] = (uint32_t)x_row((q * S::Waves + wave) * S::CopyRows + cr) * (uint32_t)a.x_ld + piece * 16;
    const int half = (lane & 1) ^ ((lane >> 4) & 1);  // W4: rows 8 apart share banks, their halves swap
#pragma unroll
    for (int q = 0; q < S::BLoads; ++q)
      b_off[q] = S::W4 ? (uint32_t)w_row((q * S::Waves + wave) * 32 + (lane >> 1)) * (uint32_t)(K / 2) + half * 16
                       : (uint32_t)w_row((q * S::Waves + wave) * S::CopyRows + cr) * (uint32_t)x_bytes + piece * 16;
    auto st_a = [&](int buf) { return s_st + buf * S::Stage; };
    auto st_b = [&](int buf) { return s_st + buf * S::Stage + S::StageA; };
    // copy q of a wave's Group, x first
    auto copy = [&](const uint8_t* xb, const uint8_t* wb, int buf, int q) {
      if (q < ALoads) tile_copy16(xb, a_off[q], tile_lds(st_a(buf) + (q * S::Waves + wave) * 1024));
      else tile_copy16(wb, b_off[q - ALoads], tile_lds(st_b(buf) + ((q - ALoads) * S::Waves + wave) * 1024));
    };
    auto copy_some = [&](int kt, int buf, int from, int to) {
      const uint8_t* xb = x0 + (int64_t)kt * S::Row;
      const uint8_t* wb = w0 + (int64_t)kt * S::WRow;
#pragma unroll
      for (int q = 0; q < Group; ++q)
        if (q >= from && q < to) copy(xb, wb, buf, q);
    };
    auto issue = [&](int kt, int buf) { copy_some(kt, buf, 0, Group); };
    // a step that ends inside: pieces past the row's end become zeros
    auto issue_end = [&](int kt, int buf) {
      const op_u32x4 zero = {0, 0, 0, 0};
      const bool a_in = kt * S::Row + piece * 16 < x_bytes;
      if (a_in) {
        copy_some(kt, buf, 0, ALoads);
      } else {
#pragma unroll
        for (int q = 0; q < ALoads; ++q) *(op_u32x4*)(st_a(buf) + (q * S::Waves + wave) * 1024 + lane * 16) = zero;
      }
      if (S::W4 ? kt * 2 + half < blocks : a_in) {
        copy_some(kt, buf, ALoads, Group);
      } else {
#pragma unroll
        for (int q = 0; q < S::BLoads; ++q) *(op_u32x4*)(st_b(buf) + (q * S::Waves + wave) * 1024 + lane * 16) = zero;
      }
    };

    // this lane's W rows within the tile
    int brow[J];
#pragma unroll
    for (int j = 0; j < J; ++j) brow[j] = (GLU ? j * NT + wn * 32 : wn * 32 * J + j * 32) + lr;
    // its row blocks of x: every other one where two waves share them, so that a
    // short tile loads both
    auto arow = [&](int i) { return (i * S::WavesM + wm) * 32; };

    // Scales lie in LDS for ScaleBytes / StepBlocks steps at once: a row's scales of one step
    // are 2 to 8 bytes, too few for a load each.  A thread brings whole rows,
    // requested a step before they are needed, in pieces of 16.  Those of a row's
    // end overlap the ones before; a row with less than 16 left reads into the
    // past and writes that before its place, where nothing lies: the end of the
    // previous row's place, which is unused then, or the 16 bytes in front.  Rows
    // of less than 16 (K < 512) are one chunk, brought byte by byte: W4A4
    // 8192 x 4096 x 256 24 us, 95 when left to the small variant.
    constexpr int Pieces = C::ScaleBytes / 16;
    tile_bytes16 sc[S::WM ? S::ScaleTurns * Pieces : 1];
    uint32_t sc_off[S::WM ? S::ScaleTurns : 1];
    // whether a wave's 64 rows of turn u are rows of W
    auto sc_of_w = [&](int u) { return !S::XM || u * S::Threads + wave * 64 < S::N; };
    if constexpr (S::WM) {
#pragma unroll
      for (int u = 0; u < S::ScaleTurns; ++u) {
        const int r = min(u * S::Threads + tid, S::N + (S::XM ? NI * S::WavesM * 32 : 0) - 1);
        sc_off[u] = (uint32_t)(sc_of_w(u) ? w_row(r) : x_row(r - S::N)) * (uint32_t)blocks;
      }
    }
    auto load_scales = [&](int kt) {
      if constexpr (S::WM) {
        const int b0 = kt * S::StepBlocks, n = min(C::ScaleBytes, blocks - b0);
#pragma unroll
        for (int u = 0; u < S::ScaleTurns; ++u) {
          const uint8_t* const base = (sc_of_w(u) ? ws0 : xs0) + b0;
#pragma unroll
          for (int d = 0; d < Pieces; ++d)
            sc[u * Pieces + d] = *(const tile_bytes16*)(base + min(d * 16, n - 16) + sc_off[u]);
        }
      }
    };
    auto store_scales = [&](int kt) {
      if constexpr (S::WM) {
        const int n = min(C::ScaleBytes, blocks - kt * S::StepBlocks);
#pragma unroll
        for (int u = 0; u < S::ScaleTurns; ++u) {
          const int r = u * S::Threads + tid;
          if (r < S::N + (S::XM ? NI * S::WavesM * 32 : 0))
#pragma unroll
            for (int d = 0; d < Pieces; ++d)
              *(tile_bytes16*)(s_sc + 16 + r * S::ScalePitch + min(d * 16, n - 16)) = sc[u * Pieces + d];
        }
      }
    };
    auto few_scales = [&] {
      if constexpr (S::WM) {
#pragma unroll 1
        for (int u = 0; u < S::ScaleTurns; ++u) {
          const int r = u * S::Threads + tid;
          const uint8_t* const src = (sc_of_w(u) ? ws0 : xs0) + sc_off[u];
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = src[min(i, blocks - 1)];
          if (r < S::N + (S::XM ? NI * S::WavesM * 32 : 0))
#pragma unroll
            for (int i = 0; i < 4; ++i)
              ((uint32_t*)(s_sc + 16 + r * S::ScalePitch))[i] =
                  v[4 * i] | v[4 * i + 1] << 8 | v[4 * i + 2] << 16 | v[4 * i + 3] << 24;
        }
      }
    };
    // One step's: MXFP4 x MXFP4 the 8 of a row, shifted so that this half's
    // blocks 2 ks + kg are bytes 0 and 2 of each word, and those past the row's
    // end 1 (their codes are zeros, but zero times a NaN scale is not); W4 that of
    // block kg.
    uint2 sx[S::XM ? NI : 1], sw[J], sx_n[S::XM ? NI : 1], sw_n[J];
    auto read_scales = [&](int at) {  // at: offset of the step within the chunk
      if constexpr (S::XM) {
        auto get = [&](int r) {
          const uint8_t* p = s_sc + 16 + r * S::ScalePitch + at;
          return *(const uint2*)p;
        };
#pragma unroll
        for (int i = 0; i < NI; ++i) sx_n[i] = get(S::N + arow(i) + lr);
#pragma unroll
        for (int j = 0; j < J; ++j) sw_n[j] = get(brow[j]);
      } else if constexpr (S::WM) {
#pragma unroll
        for (int j = 0; j < J; ++j) sw_n[j].x = s_sc[16 + brow[j] * S::ScalePitch + at + kg];
      }
    };
    auto take_scales = [&](int kt, bool whole_step) {
      if constexpr (S::XM) {
        auto cut = [&](uint2 v) {
          const int past = (kt + 1) * S::StepBlocks - blocks;
          if (!whole_step && past > 0) {
            const int left = S::StepBlocks - past;  // 1 .. StepBlocks - 1
            const uint64_t keep = ~0ull >> (64 - 8 * left);
            const uint64_t d = (((uint64_t)v.y << 32 | v.x) & keep) | (0x7F7F7F7F7F7F7F7Full & ~keep);
            v = make_uint2((uint32_t)d, (uint32_t)(d >> 32));
          }
          return make_uint2(v.x >> (8 * kg), v.y >> (8 * kg));
        };
#pragma unroll
        for (int i = 0; i < NI; ++i) sx[i] = cut(sx_n[i]);
#pragma unroll
        for (int j = 0; j < J; ++j) sw[j] = cut(sw_n[j]);
      } else if constexpr (S::WM) {
#pragma unroll
        for (int j = 0; j < J; ++j) sw[j].x = whole_step || kt * 2 + kg < blocks ? sw_n[j].x : 127;
      }
    };

    op_f32x16 acc[NI][J];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) acc[i][j] = op_f32x16{};

    // fragments of slice ks: x piece 2 ks + kg of a row (W4: 4 kg + ks, so that
    // a lane's codes of a step are one piece under one scale)
    op_u32x4 fx[2][NI], fw[2][J];
    auto read = [&](int buf, int ks, int to) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        fx[to][i] = *(const op_u32x4*)(st_a(buf) + tile_at(arow(i) + lr, S::W4 ? 4 * kg + ks : 2 * ks + kg));
      if constexpr (!S::W4) {
#pragma unroll
        for (int j = 0; j < J; ++j) fw[to][j] = *(const op_u32x4*)(st_b(buf) + tile_at(brow[j], 2 * ks + kg));
      } else {
#pragma unroll
        for (int j = 0; j < J; ++j)
          fw[to][j][0] = *(const uint32_t*)(st_b(buf) + brow[j] * 32 + ((kg ^ ((brow[j] >> 3) & 1)) << 4) + ks * 4);
      }
    };
    // W fragments of a slice, ready for the MFMA
    op_i32x8 wq[J];
    op_bf16x8 wb[J];
    auto unpack = [&](int from) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const op_u32x4 f = fw[from][j];
        if constexpr (S::XM) wq[j] = op_i32x8{(int)f[0], (int)f[1], (int)f[2], (int)f[3], 0, 0, 0, 0};
        else if constexpr (S::W4) wb[j] = op_fp4x8(f[0], op_scale(sw[j].x));
        else wb[j] = __builtin_bit_cast(op_bf16x8, f);
      }
    };
    // the products of row block i.  They have no side effects, and the compiler
    // would sink them below the reads of later slices and the barrier, whose
    // fragments then do not fit the registers, or move the reads down to their
    // uses, each with its whole latency: the empty asm keeps a block's products
    // where they stand.
    auto block = [&](auto ks_c, int from, int i) {
      constexpr int ks = decltype(ks_c)::value;
      const op_u32x4 f = fx[from][i];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if constexpr (S::XM)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              wq[j], op_i32x8{(int)f[0], (int)f[1], (int)f[2], (int)f[3], 0, 0, 0, 0}, acc[i][j], 4, 4, (ks & 1) * 2,
              (int)(ks < 2 ? sw[j].x : sw[j].y), (ks & 1) * 2, (int)(ks < 2 ? sx[i].x : sx[i].y));
        else
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j], __builtin_bit_cast(op_bf16x8, f), acc[i][j], 0, 0, 0);
        asm volatile("" : "+a"(acc[i][j]));
      }
    };
    int sc_at = 0;  // offset of this step's scales within the chunk
    // a slice: the products of fragments `from` with the reads of the next slice
    // woven in, one per product
    auto slice = [&](auto ks_c, int buf, int from) {
      constexpr int ks = decltype(ks_c)::value;
      read(buf, ks + 1, from ^ 1);
      // the next step's scales; where they begin a chunk, read again below
      if constexpr (ks == 0 && S::WM) read_scales(sc_at + S::StepBlocks);
      constexpr int reads = NI + J + (ks == 0 && S::WM ? (S::XM ? NI + J : J) : 0);
      unpack(from);
#pragma unroll
      for (int i = 0; i < NI; ++i) block(ks_c, from, i);
#pragma unroll
      for (int n = 0; n < NI * J; ++n) {
        if constexpr (NI * J < reads) __builtin_amdgcn_sched_group_barrier(0x100, (reads + NI * J - 1) / (NI * J), 0);  // LDS reads
        else __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // One step on stage buf; slice 0 is in fragments 0.  steady: the next Stages
    // steps exist and are whole, so exactly Stages - 2 groups of copies are
    // newer than the next step's.
    auto step = [&](int kt, int buf, auto steady_c) {
      constexpr bool steady = decltype(steady_c)::value;
      const bool more = steady || kt + 1 < steps;
      const int next = buf + 1 == Stages ? 0 : buf + 1;
      // the next step's scales begin a chunk: requested now, in LDS after the barrier
      const bool chunk = S::WM && more && sc_at + S::StepBlocks == C::ScaleBytes;
      if (chunk) load_scales(kt + 1);
      slice(integral_constant<int, 0>{}, buf, 0);
      slice(integral_constant<int, 1>{}, buf, 1);
      slice(integral_constant<int, 2>{}, buf, 0);
      const integral_constant<int, 3> last{};
      if (more) {
        if (steady) tile_sync<(Stages - 2) * Group>();
        else tile_sync<0>();
        if constexpr (S::WM) {
          sc_at = chunk ? 0 : sc_at + S::StepBlocks;
          if (chunk) {
            store_scales(kt + 1);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            read_scales(0);
          }
        }
        read(next, 0, 0);
        __builtin_amdgcn_sched_barrier(0);  // requested before the products, not after
      }
      unpack(1);
      if (steady) {
        // the copies between the products
        const uint8_t* xb = x0 + (int64_t)(kt + Stages) * S::Row;
        const uint8_t* wb = w0 + (int64_t)(kt + Stages) * S::WRow;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          block(last, 1, i);
#pragma unroll
          for (int q = Group * i / NI; q < Group * (i + 1) / NI; ++q) copy(xb, wb, buf, q);
        }
        __builtin_amdgcn_sched_barrier(0);
      } else {
        if (kt + Stages < whole) issue(kt + Stages, buf);
        else if (kt + Stages < steps) issue_end(kt + Stages, buf);
#pragma unroll
        for (int i = 0; i < NI; ++i) block(last, 1, i);
      }
      if (more) take_scales(kt + 1, steady);
    };

    auto begin = [&](int kt) {
      if (kt < whole) issue(kt, kt);
      else if (kt < steps) issue_end(kt, kt);
    };
    begin(0);
    if (S::WM && blocks < 16) {
      few_scales();
    } else {
      load_scales(0);
      store_scales(0);
    }
#pragma unroll
    for (int kt = 1; kt < Stages; ++kt) begin(kt);
    if (whole >= Stages) tile_sync<(Stages - 1) * Group>();
    else tile_sync<0>();
    read_scales(0);
    take_scales(0, false);
    read(0, 0, 0);
    int kt = 0, buf = 0;
    if constexpr (C::Unroll) {  // stages at fixed addresses
      for (; kt + 2 * Stages - 1 < whole; kt += Stages)
#pragma unroll
        for (int u = 0; u < Stages; ++u) step(kt + u, u, std::true_type{});
    } else {
#pragma unroll 1
      for (; kt + Stages < whole; ++kt) {
        step(kt, buf, std::true_type{});
        buf = buf + 1 == Stages ? 0 : buf + 1;
      }
    }
#pragma unroll 1
    for (; kt < steps; ++kt) {
      step(kt, buf, std::false_type{});
      buf = buf + 1 == Stages ? 0 : buf + 1;
    }

    // Result.  Element r of a lane's block: row lr of x, W row 8 (r/4) + 4 kg +
    // r%4.  32 rows at a time go through this wave's part of the stages; what is
    // done to them on the way out is a rolled loop, since code that runs once per
    // tile costs its instruction fetches.
    constexpr int CW = GLU ? 32 : 32 * J, CS = 32 * J + 4;  // columns of y of a wave; padded stride
    constexpr int LPR = CW / 8, RPI = 64 / LPR;             // lanes per row (8 columns each), rows per pass
    static_assert(S::Waves * 32 * CS * 4 <= Stages * S::Stage, "the staging fits the stages");
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // every wave is done with the stages
    const int c8 = (lane % LPR) * 8, rs = lane / LPR;
    const int col = n0 + wn * CW + c8;
    const bool wide = (((uintptr_t)a.y & 15) | (a.ldy & (a.y_f32 ? 3 : 7))) == 0 && col + 8 <= n_out;
    auto out = [&](int i, const float* c) {
      op_f32x4 v[32 / RPI][2];
      int row[32 / RPI];
      bool live[32 / RPI];
#pragma unroll
      for (int q = 0; q < 32 / RPI; ++q) {
        const int rl = q * RPI + rs, m = arow(i) + rl;
        row[q] = s_y[m];
        live[q] = s_x[m] >= 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          op_f32x4 z = *(const op_f32x4*)&c[rl * CS + c8 + h * 4];
          if constexpr (GLU) {
            const op_f32x4 u = *(const op_f32x4*)&c[rl * CS + 32 + c8 + h * 4];
#pragma unroll
            for (int w = 0; w < 4; ++w) z[w] = op_silu_mul(z[w], u[w]);
          }
          v[q][h] = z;
        }
      }
#pragma unroll
      for (int q = 0; q < 32 / RPI; ++q) {
        if (row[q] < 0) continue;
        const int64_t at = (int64_t)row[q] * a.ldy + col;
        if (wide) {
          if (a.y_f32) {
            const op_f32x4 zero = {0.f, 0.f, 0.f, 0.f};
            *(op_f32x4*)((float*)a.y + at) = live[q] ? v[q][0] : zero;
            *(op_f32x4*)((float*)a.y + at + 4) = live[q] ? v[q][1] : zero;
          } else {
            op_u32x4 p;
#pragma unroll
            for (int w = 0; w < 4; ++w) p[w] = op_bf16_pair(v[q][w >> 1][(w & 1) * 2], v[q][w >> 1][(w & 1) * 2 + 1]);
            *(op_u32x4*)((uint16_t*)a.y + at) = live[q] ? p : op_u32x4{0, 0, 0, 0};
          }
        } else {
#pragma unroll
          for (int u = 0; u < 8; ++u)
            if (col + u < n_out) {
              const float z = live[q] ? v[q][u >> 2][u & 3] : 0.f;
              if (a.y_f32) ((float*)a.y)[at + u] = z;
              else ((uint16_t*)a.y)[at + u] = op_bf16(z);
            }
        }
      }
    };
    auto put = [&](const op_f32x16 (&z)[J], float* c) {
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(op_f32x4*)&c[lr * CS + j * 32 + q * 8 + kg * 4] =
              op_f32x4{z[j][q * 4], z[j][q * 4 + 1], z[j][q * 4 + 2], z[j][q * 4 + 3]};
    };
    // as many row blocks at once as the stages hold, up to two: one round of
    // latencies for both
    constexpr int Batch = NI % 2 == 0 && S::Waves * 2 * 32 * CS * 4 <= Stages * S::Stage ? 2 : 1;
    float* const c = (float*)s_st + wave * (Batch * 32 * CS);
#pragma unroll 1
    for (int i = 0; i < NI; i += Batch) {
      // the sums lie in registers, which have no index: one of the copies is taken
#pragma unroll
      for (int u = 0; u < NI; u += Batch)
        if (i == u)
#pragma unroll
          for (int h = 0; h < Batch; ++h) put(acc[u + h], c + h * 32 * CS);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's rows are in LDS
#pragma unroll
      for (int h = 0; h < Batch; ++h) out(i + h, c + h * 32 * CS);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next rows overwrite them
    }
  };
  const int ni = (t.rows + 32 * S::WavesM - 1) / (32 * S::WavesM);
  if constexpr (C::MaxI == 2) {
    if (ni == 1) run(integral_constant<int, 1>{});
    else run(integral_constant<int, 2>{});
  } else {
    switch (ni) {
      case 1: run(integral_constant<int, 1>{}); break;
      case 2: run(integral_constant<int, 2>{}); break;
      case 3: run(integral_constant<int, 3>{}); break;
      default: run(integral_constant<int, 4>{}); break;
    }
  }
}

template <int AT, int WT, bool GLU, class C>
hipError_t launch_tile_as(const ProductArgs& a, hipStream_t s) {
  using S = TileShape<AT, WT, C>;
  const int n_out = GLU ? a.N / 2 : a.N, nt = GLU ? S::N / 2 : S::N;
  const int64_t n_ntiles = (n_out + nt - 1) / nt;
  const int64_t wgs = (op_max_tiles(a, S::M) * n_ntiles + 7) / 8 * 8;
  if (wgs * S::Threads >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  return launch_op(product_tile_kernel<AT, WT, GLU, C>, dim3((unsigned)wgs), dim3(S::Threads), s, a);
}

template <int AT, int WT>
hipError_t launch_tile(const ProductArgs& a, bool glu, ProductVariant v, hipStream_t s) {
  constexpr bool W4 = AT == MOE_BF16 && WT == MOE_MXFP4;
  if (v == ProductVariant::kBig)
    return glu ? launch_tile_as<AT, WT, true, TileBig<AT, WT>>(a, s) : launch_tile_as<AT, WT, false, TileBig<AT, WT>>(a, s);
  // W4's stages are small enough for both at once; the other formats' GLU
  // tiles are too large to share a CU
  if (glu) return launch_tile_as<AT, WT, true, TileMid<AT, WT, true, !W4>>(a, s);
  if (v == ProductVariant::kHalf) return launch_tile_as<AT, WT, false, TileHalf<AT, WT>>(a, s);
  if constexpr (!W4)
    if (v == ProductVariant::kDeep) return launch_tile_as<AT, WT, false, TileMid<AT, WT, false, true>>(a, s);
  return launch_tile_as<AT, WT, false, TileMid<AT, WT, false, false>>(a, s);
}

}  // namespace moert
