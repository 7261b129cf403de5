// The norm in front of a block, and the end of a routed or plain block: sum of a
// token's expert rows, norm after the block, gate, scaled residual, norm in front
// of the next block.
//
// A row stays in registers from its first read to its last write: 8 neighbouring
// columns per thread and piece, up to four pieces (with four, past 8,192 columns, the end of
// a block spills 22-24 registers and a norm of fp32 rows 8: every instance keeps within the
// 128 that 1,024 threads leave, which only H > 16,384 needs).  Sums of squares are fp32: over a
// thread's columns, then over 16 lanes by DPP, the wave, and the waves through LDS,
// always in the same order.  Rows of up to 512 columns share a workgroup, 16, 32 or
// 64 threads each; a longer one has its own.  F8 rows are converted from the same
// registers: 16 neighbouring lanes hold a block of 128 columns.
//
// HBM bounds both up to 8,192 columns: 8192 tokens of 8 fp32 rows of 4,096, normed, gated, added
// and normed again, 237 us, 5.3 TB/s (a plain copy reaches 5.2); wider rows come one at a
// time, 2048 tokens of 8 rows of 12,288 in 227 us, 4.2 TB/s, bf16 171, 3.2.  Norm of 32768 x 4096 bf16 to F8 80 us,
// 5.0 TB/s, of 8192 x 4096 23.5, 4.3 TB/s with the start and end of a short launch.
#include "ops.h"

namespace moert {

constexpr int kNormShared = 256;  // threads of a workgroup that several rows share
constexpr int kNormMost = 1024;

template <int Ctrl>
__device__ inline float norm_move(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), Ctrl, 0xF, 0xF, false));
}

// Sum over the threads of a row, in each of them.  lg: as NormArgs; red: a place
// per wave.  Calls take two such arrays in turn: who writes one again has passed
// the other's barrier, and with it everyone's reads.
__device__ inline float norm_sum(float v, int lg, float* red) {
  v += norm_move<0xB1>(v);   // lane ^ 1
  v += norm_move<0x4E>(v);   // lane ^ 2
  v += norm_move<0x141>(v);  // mirrored in 8
  v += norm_move<0x140>(v);  // mirrored in 16
  if (lg >= 5) v += __shfl_xor(v, 16);
  if (lg >= 6) v += __shfl_xor(v, 32);
  if (lg >= 7) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
    const int waves = blockDim.x >> 6;
    for (int w = 0; w < waves; ++w) v += red[w];
  }
  return v;
}

// UNI: a wave's lanes belong to one row, whose index is a scalar then.  WIDE: H is 8
// at least.  A piece that would pass the row's end is the row's last 8 columns
// then, of which the first lo are other lanes': so every load is one access, and
// lanes without a column of their own go along.
template <bool CLOSE, bool PF32, int NV, bool UNI, bool WIDE>
__global__ __launch_bounds__(kNormMost) void norm_kernel(NormArgs a) {
  constexpr int PB = PF32 ? 4 : 2;
  constexpr bool Early = !CLOSE || NV == 1;  // weights and gate are requested with the row: one latency
  __shared__ float s_red[2][kNormMost / 64];
  const bool own = UNI && a.lg >= 7;  // the workgroup's one row
  const int G = own ? (int)blockDim.x : 1 << a.lg;
  const int t = own ? threadIdx.x : threadIdx.x & (G - 1);
  const int sub = own ? 0 : UNI ? __builtin_amdgcn_readfirstlane(threadIdx.x >> a.lg) : threadIdx.x >> a.lg;
  const int per = own ? 1 : blockDim.x >> a.lg;
  const int H = a.H;
  int col[NV], lo[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + t) * 8;
    col[i] = WIDE ? min(c, H - 8) : c;
    lo[i] = min(c - col[i], 8);
  }
  // columns of piece i that are this thread's
  auto mine = [&](int i, int c) { return WIDE ? c >= lo[i] : col[i] + c < H; };

  int slot = 0;
  auto mean_square = [&](const float (&v)[NV][8]) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (mine(i, c)) sum = fmaf(v[i][c], v[i][c], sum);
    slot ^= 1;
    return norm_sum(sum, a.lg, s_red[slot]) / (float)H;
  };
  // 1 / sqrt(mean(v^2) + eps).  Where that leaves fp32, v is taken 2^72 times smaller
  // from here on: the largest values' sum stays within it then.
  auto inverse_root = [&](float (&v)[NV][8]) {
    float ms = mean_square(v) + a.eps;
    if (ms == INFINITY) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) v[i][c] *= 0x1p-72f;
      ms = fmaf(a.eps * 0x1p-72f, 0x1p-72f, mean_square(v));
    }
    return 1.f / sqrtf(ms);
  };
  auto load = [&](const uint8_t* row, bool f32, int i) {
    return WIDE ? op_cols_load(row, f32, col[i]) : op_cols_load(row, f32, col[i], H - col[i]);
  };
  auto store = [&](uint8_t* row, bool f32, int i, const float (&v)[8]) {
    if (WIDE) op_cols_store_from(row, f32, col[i], lo[i], v);
    else op_cols_store(row, f32, col[i], H - col[i], v);
  };

  OpCols weight[NV], x[NV];  // x: the row to come, requested while its predecessor is at work
  if (Early && a.weight)
#pragma unroll
    for (int i = 0; i < NV; ++i) weight[i] = load(a.weight, a.weight_f32, i);
  auto request = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = load(a.p + (row < a.T ? row : 0) * a.ldp * PB, PF32, i);
  };
  const int64_t first = (int64_t)blockIdx.x * per, step = (int64_t)gridDim.x * per;
  if (!CLOSE) request(first + sub);
  for (int64_t row0 = first; row0 < a.T; row0 += step) {
    const int64_t row = row0 + sub;
    const bool live = row < a.T;  // lanes without a row go along, for the barriers
    const int64_t at = live ? row : 0;
    float r[NV][8];
    if constexpr (!CLOSE) {
#pragma unroll
      for (int i = 0; i < NV; ++i) op_cols_get(x[i], PF32, r[i]);
      if (row0 + step < a.T) request(row + step);
    } else {
      const uint8_t* const gate = a.gate ? a.gate + at * a.ldg * (a.gate_f32 ? 4 : 2) : nullptr;
      OpCols res[NV], post[NV], gates[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        res[i] = load(a.res + at * a.ldres * (a.res_f32 ? 4 : 2), a.res_f32, i);
        if (Early && a.post) post[i] = load(a.post, a.post_f32, i);
        if (Early && a.gate_cols > 1) gates[i] = load(gate, a.gate_f32, i);
      }
      float g0 = 1.f;
      if (a.gate_cols == 1) g0 = a.gate_f32 ? *(const float*)gate : __uint_as_float((uint32_t)*(const uint16_t*)gate << 16);
      float b[NV][8] = {};
      bool any = !a.ids;  // a row without experts keeps its residual, also where its gate is no number
      // Expert rows requested before the first is added.  Eight columns of four fp32 rows
      // are 32 registers, of eight 64, which with the rest pass the 128 that every
      // instance keeps within: 8192 x 8 x 4096 238 us, 316 with eight rows.
      constexpr int J = !WIDE ? 1 : 4 / NV;
      for (int j0 = 0; live && j0 < a.k; j0 += J) {
        OpCols v[J][NV];
        float w[J];
        bool ok[J];
#pragma unroll
        for (int q = 0; q < J; ++q) {
          const int64_t p = row * a.k + min(j0 + q, a.k - 1);
          ok[q] = j0 + q < a.k;
          if (a.ids) {
            const int e = a.ids[p];
            ok[q] = ok[q] && e >= 0 && e < a.E;
            any = any || ok[q];
          }
          w[q] = a.w ? a.w[p] : 1.f;
        }
#pragma unroll
        for (int q = 0; q < J; ++q)
          if (ok[q])
#pragma unroll
            for (int i = 0; i < NV; ++i) v[q][i] = load(a.p + (row * a.k + j0 + q) * a.ldp * PB, PF32, i);
#pragma unroll
        for (int q = 0; q < J; ++q)
          if (ok[q])
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              float f[8];
              op_cols_get(v[q][i], PF32, f);
#pragma unroll
              for (int c = 0; c < 8; ++c) b[i][c] = fmaf(w[q], f[c], b[i][c]);
            }
      }
      if (a.post) {
        const float inv = inverse_root(b);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float f[8];
          op_cols_get(Early ? post[i] : load(a.post, a.post_f32, i), a.post_f32, f);
#pragma unroll
          for (int c = 0; c < 8; ++c) b[i][c] = b[i][c] * inv * f[c];
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (a.gate_cols > 1) {
          float f[8];
          op_cols_get(Early ? gates[i] : load(gate, a.gate_f32, i), a.gate_f32, f);
#pragma unroll
          for (int c = 0; c < 8; ++c) b[i][c] *= f[c];
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) b[i][c] *= g0;
        }
        float f[8];
        op_cols_get(res[i], a.res_f32, f);
#pragma unroll
        for (int c = 0; c < 8; ++c) r[i][c] = any ? fmaf(a.scale, b[i][c], f[c]) : f[c];
        if (live) store(a.out + row * a.ldout * (a.out_f32 ? 4 : 2), a.out_f32, i, r[i]);
      }
      if (!a.weight) continue;
    }

    float inv = inverse_root(r);
    // A row far from 1 takes its power of two first, or its product with the weight may leave
    // fp32 where the result does not.  (Asked for every product, that costs norms to F8 5-8%.)
    if (inv > 0x1p10f || inv < 0x1p-10f) {
      const float power = __uint_as_float(__float_as_uint(inv) & 0x7F800000u);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) r[i][c] *= power;
      inv = __uint_as_float((__float_as_uint(inv) & 0x007FFFFFu) | 0x3F800000u);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[8];
      op_cols_get(Early ? weight[i] : load(a.weight, a.weight_f32, i), a.weight_f32, f);
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        r[i][c] = r[i][c] * f[c] * inv;  // bf16 x and weight: the first product is exact
        top = max(top, __float_as_uint(r[i][c]) & 0x7FFFFFFFu);
      }
      if (a.y_dtype != MOE_F8) {
        if (live) store(a.y + row * a.ldy * (a.y_dtype == MOE_F32 ? 4 : 2), a.y_dtype == MOE_F32, i, r[i]);
      } else {
        // H is a multiple of 16: pieces are whole or nobody's
        const OpF8Scale s(op_max16(lo[i] == 0 ? top : 0));
        const uint2 q = op_f8x8(r[i], s);
        if (live && lo[i] == 0) {
          *(uint2*)(a.y + row * a.ldy + col[i]) = q;
          if ((threadIdx.x & 15) == 0) a.ys[row * ((H + 127) >> 7) + (col[i] >> 7)] = s.scale;
        }
      }
    }
  }
}

template <bool CLOSE, bool PF32>
static hipError_t norm_typed(NormArgs& a, hipStream_t s) {
  // Two pieces a thread from 1,024 columns on, four past 8,192: fewer waves wait at a
  // row's barriers.  One, two and four pieces: norm 8192 x 4096 bf16 to F8 27.5, 23.4,
  // 26.2 us, 4096 x 16384 two and four 50.4, 47.9; end of a block 8192 x 2 x 2048 bf16
  // one and two 54, 44.  Its fp32 rows, which bring twice the bytes a column, one
  // piece up to 4,096 columns: 8192 x 8 x 4096 238 and 248.
  const int pieces = (a.H + 7) / 8;
  int threads = kNormShared, nv = 1;
  if (pieces <= 64) {
    a.lg = pieces <= 16 ? 4 : pieces <= 32 ? 5 : 6;
  } else {
    nv = pieces <= (CLOSE && PF32 ? 512 : 128) ? 1 : pieces <= 1024 ? 2 : 4;
    threads = (pieces + nv * 64 - 1) / (nv * 64) * 64;
    a.lg = 10;
  }
  const int64_t per = a.lg < 7 ? threads >> a.lg : 1;
  // Norms of several rows a workgroup, the next one's loads and the weights in hand:
  // twice the threads that the chip holds.  As many, twice as many and one row each:
  // 32768 x 4096 bf16 to F8 88, 80, 88 us, 65536 x 512 27.0, 24.0, 27.0 (each row's
  // weights anew, nothing ahead: 102 and 25).
  const int64_t most = CLOSE ? 1 << 20 : 2 * 256 * 2048 / threads;
  const dim3 grid((unsigned)std::min<int64_t>((a.T + per - 1) / per, most));
  auto k = a.H < 8    ? norm_kernel<CLOSE, PF32, 1, false, false>
           : a.lg < 6 ? norm_kernel<CLOSE, PF32, 1, false, true>
           : nv == 1  ? norm_kernel<CLOSE, PF32, 1, true, true>
           : nv == 2  ? norm_kernel<CLOSE, PF32, 2, true, true>
                      : norm_kernel<CLOSE, PF32, 4, true, true>;
  return launch_op(k, grid, dim3(threads), s, a);
}

hipError_t launch_norm(NormArgs a, hipStream_t s) {
  if (a.res) return a.p_f32 ? norm_typed<true, true>(a, s) : norm_typed<true, false>(a, s);
  return a.p_f32 ? norm_typed<false, true>(a, s) : norm_typed<false, false>(a, s);
}

}  // namespace moert
