// The norm in front of a block, and the end of a routed or plain block: sum of a
// token's expert rows, norm after the block, gate, scaled residual, norm in front
// of the next block.
//
// A row stays in registers from its first read to its last write: 8 neighbouring
// columns per thread and piece, up to four pieces.  Sums of squares are fp32: over a
// thread's columns, then over 16 lanes by DPP, the wave, and the waves through LDS,
// always in the same order.  Rows of up to 512 columns share a workgroup, 16, 32 or
// 64 threads each; a longer one has its own.  F8 rows are converted from the same
// registers: 16 neighbouring lanes hold a block of 128 columns.
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

template <bool CLOSE, bool PF32, int NV>
__global__ __launch_bounds__(kNormMost) void norm_kernel(NormArgs a) {
  constexpr int PB = PF32 ? 4 : 2;
  __shared__ float s_red[2][kNormMost / 64];
  const bool own = a.lg >= 7;  // the workgroup's one row
  const int G = own ? (int)blockDim.x : 1 << a.lg;
  const int t = own ? threadIdx.x : threadIdx.x & (G - 1);
  const int sub = own ? 0 : threadIdx.x >> a.lg, per = own ? 1 : blockDim.x >> a.lg;
  const int H = a.H;
  int n[NV];  // columns of each piece, 0 and fewer past the row's end
#pragma unroll
  for (int i = 0; i < NV; ++i) n[i] = H - (i * G + t) * 8;
  auto col = [&](int i) { return (int64_t)(i * G + t) * 8; };

  int slot = 0;
  auto mean_square = [&](const float (&v)[NV][8]) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < n[i]) sum = fmaf(v[i][c], v[i][c], sum);
    slot ^= 1;
    return norm_sum(sum, a.lg, s_red[slot]) / (float)H;
  };
  // 1 / sqrt(mean(v^2) + eps).  Where the squares leave fp32, v is taken 2^72 times
  // smaller from here on: the largest values' sum stays within it then, and eps
  // is nothing beside it.
  auto inverse_root = [&](float (&v)[NV][8]) {
    float ms = mean_square(v) + a.eps;
    if (ms == INFINITY) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) v[i][c] *= 0x1p-72f;
      ms = mean_square(v);
    }
    return 1.f / sqrtf(ms);
  };

  for (int64_t row0 = (int64_t)blockIdx.x * per; row0 < a.T; row0 += (int64_t)gridDim.x * per) {
    const int64_t row = row0 + sub;
    const bool live = row < a.T;  // lanes without a row go along, for the barriers
    float r[NV][8];
    if constexpr (!CLOSE) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        op_cols_get(op_cols_load(a.p + (live ? row : 0) * a.ldp * PB, PF32, col(i), live ? n[i] : 0), PF32, r[i]);
    } else {
      OpCols res[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i)
        res[i] = op_cols_load(a.res + (live ? row : 0) * a.ldres * (a.res_f32 ? 4 : 2), a.res_f32, col(i), live ? n[i] : 0);
      float b[NV][8] = {};
      constexpr int J = NV == 1 ? 8 : NV == 2 ? 4 : 2;  // expert rows requested before the first is added
      for (int j0 = 0; live && j0 < a.k; j0 += J) {
        OpCols v[J][NV];
        float w[J];
        bool ok[J];
#pragma unroll
        for (int q = 0; q < J; ++q) {
          const int64_t p = row * a.k + j0 + q;
          ok[q] = j0 + q < a.k;
          if (ok[q] && a.ids) {
            const int e = a.ids[p];
            ok[q] = e >= 0 && e < a.E;
          }
          w[q] = 1.f;
          if (ok[q]) {
            if (a.w) w[q] = a.w[p];
#pragma unroll
            for (int i = 0; i < NV; ++i) v[q][i] = op_cols_load(a.p + p * a.ldp * PB, PF32, col(i), n[i]);
          }
        }
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
          op_cols_get(op_cols_load(a.post, a.post_f32, col(i), n[i]), a.post_f32, f);
#pragma unroll
          for (int c = 0; c < 8; ++c) b[i][c] = b[i][c] * inv * f[c];
        }
      }
      const uint8_t* const gate = a.gate ? a.gate + (live ? row : 0) * a.ldg * (a.gate_f32 ? 4 : 2) : nullptr;
      float g0 = 1.f;
      if (a.gate_cols == 1) g0 = a.gate_f32 ? *(const float*)gate : __uint_as_float((uint32_t)*(const uint16_t*)gate << 16);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (a.gate_cols > 1) {
          float f[8];
          op_cols_get(op_cols_load(gate, a.gate_f32, col(i), n[i]), a.gate_f32, f);
#pragma unroll
          for (int c = 0; c < 8; ++c) b[i][c] *= f[c];
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) b[i][c] *= g0;
        }
        float f[8];
        op_cols_get(res[i], a.res_f32, f);
#pragma unroll
        for (int c = 0; c < 8; ++c) r[i][c] = fmaf(a.scale, b[i][c], f[c]);
        if (live) op_cols_store(a.out + row * a.ldout * (a.out_f32 ? 4 : 2), a.out_f32, col(i), n[i], r[i]);
      }
      if (!a.weight) continue;
    }

    const float inv = inverse_root(r);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[8];
      op_cols_get(op_cols_load(a.weight, a.weight_f32, col(i), n[i]), a.weight_f32, f);
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        r[i][c] = r[i][c] * inv * f[c];
        top = max(top, __float_as_uint(r[i][c]) & 0x7FFFFFFFu);
      }
      if (a.y_dtype != MOE_F8) {
        if (live) op_cols_store(a.y + row * a.ldy * (a.y_dtype == MOE_F32 ? 4 : 2), a.y_dtype == MOE_F32, col(i), n[i], r[i]);
      } else {
        const OpF8Scale s(op_max16(n[i] > 0 ? top : 0));
        const uint2 q = op_f8x8(r[i], s);
        if (live && n[i] > 0) {
          *(uint2*)(a.y + row * a.ldy + col(i)) = q;
          if ((threadIdx.x & 15) == 0) a.ys[row * ((H + 127) >> 7) + (col(i) >> 7)] = s.scale;
        }
      }
    }
  }
}

template <bool CLOSE, bool PF32>
static hipError_t norm_typed(NormArgs& a, hipStream_t s) {
  const int pieces = (a.H + 7) / 8;
  int threads = kNormShared, nv = 1;
  if (pieces <= 64) {
    a.lg = pieces <= 16 ? 4 : pieces <= 32 ? 5 : 6;
  } else {
    nv = pieces <= kNormMost ? 1 : pieces <= 2 * kNormMost ? 2 : 4;
    threads = (pieces + nv * 64 - 1) / (nv * 64) * 64;
    a.lg = 10;
  }
  const int64_t per = a.lg < 7 ? threads >> a.lg : 1;
  const dim3 grid((unsigned)std::min<int64_t>((a.T + per - 1) / per, 1 << 20));
  auto k = nv == 1 ? norm_kernel<CLOSE, PF32, 1> : nv == 2 ? norm_kernel<CLOSE, PF32, 2> : norm_kernel<CLOSE, PF32, 4>;
  return launch_op(k, grid, dim3(threads), s, a);
}

hipError_t launch_norm(NormArgs a, hipStream_t s) {
  if (a.res) return a.p_f32 ? norm_typed<true, true>(a, s) : norm_typed<true, false>(a, s);
  return a.p_f32 ? norm_typed<false, true>(a, s) : norm_typed<false, false>(a, s);
}

}  // namespace moert
