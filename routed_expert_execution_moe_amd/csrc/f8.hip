// F8 conversion: e4m3 codes with one fp32 scale per 128 columns of a row or per
// 128 x 128 tile, and back.
//
// Sixteen lanes hold 128 neighbouring columns of a row, 8 each.  A block's largest
// magnitude is an integer maximum of the magnitudes' bits, over the 8 and, by DPP,
// over the 16 lanes; scale and reciprocal are two correctly rounded divisions per
// lane and block, the codes products rounded by the hardware's convert.
//
// HBM bounds both ways: 32768 x 4096 fp32 to F8, in rows or tiles, 115 us (5.8 TB/s; a
// plain copy reaches 5.2), back 114; 8192 x 4096 bf16 rows 21 us, 4.8 TB/s.  A workgroup walks
// over (row, block) pairs, so narrow rows fill it too: 65536 x 768 fp32 44 us, 5.7 TB/s.
#include "ops.h"

namespace moert {

constexpr int kF8Threads = 256;
constexpr int kF8Groups = kF8Threads / 16;  // blocks of 128 columns a workgroup takes at once

// A walk over (row, block of 128 columns), `step` pairs at a time.
struct F8Walk {
  int64_t r;
  int b;
  __device__ inline F8Walk(int64_t u, int64_t units, int nb) {
    r = units >> 32 ? u / nb : (int64_t)((uint32_t)u / (uint32_t)nb);
    b = (int)(u - r * nb);
  }
  __device__ inline void next(int64_t dr, int db, int nb) {
    r += dr;
    b += db;
    if (b >= nb) {
      b -= nb;
      ++r;
    }
  }
};

// 8 columns of a row; Stream: past the caches
template <bool F32, bool Stream>
__device__ inline OpCols f8_load(const uint8_t* row, int c) {
  if constexpr (!Stream) return op_cols_load(row, F32, c);
  OpCols v{};
  const op_bytes16* p = (const op_bytes16*)(row + (int64_t)c * (F32 ? 4 : 2));
  v.a = __builtin_nontemporal_load(p);
  if constexpr (F32) v.b = __builtin_nontemporal_load(p + 1);
  return v;
}

__device__ inline uint32_t f8_top(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

template <bool F32, bool Stream>
__global__ __launch_bounds__(kF8Threads) void f8_quantize_rows_kernel(const uint8_t* __restrict__ x, int64_t rows,
                                                                    int cols, int64_t ld_bytes, int64_t dr, int db,
                                                                    uint8_t* __restrict__ codes,
                                                                    float* __restrict__ scales) {
  const int nb = (cols + 127) >> 7, l = threadIdx.x & 15;
  F8Walk at((int64_t)blockIdx.x * kF8Groups + (threadIdx.x >> 4), rows * nb, nb);
  for (; at.r < rows; at.next(dr, db, nb)) {
    const int c = at.b * 128 + l * 8;
    const bool in = c < cols;  // pieces of 8 are whole: cols is a multiple of 16
    float v[8];
    op_cols_get(f8_load<F32, Stream>(x + at.r * ld_bytes, in ? c : 0), F32, v);
    if (!in)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    const OpF8Scale s(op_max16(f8_top(v)));
    const uint2 q = op_f8x8(v, s);
    if (in) *(uint2*)(codes + at.r * cols + c) = q;
    if (l == 0) scales[at.r * nb + at.b] = s.scale;
  }
}

// One 128 x 128 tile per step: 16 rows at a time, eight times, all of it in
// registers, so x is read once.
template <bool F32, bool Stream>
__global__ __launch_bounds__(kF8Threads) void f8_quantize_tiles_kernel(const uint8_t* __restrict__ x, int n_mats,
                                                                     int64_t rows, int cols, int64_t ld_bytes,
                                                                     int64_t stride_bytes,
                                                                     uint8_t* __restrict__ codes,
                                                                     float* __restrict__ scales) {
  __shared__ uint32_t s_top[2][kF8Threads / 64];
  const int nb = (cols + 127) >> 7, l = threadIdx.x & 15, sub = threadIdx.x >> 4;
  const int64_t rb = (rows + 127) >> 7;
  int slot = 0;
  for (int64_t m = blockIdx.y; m < n_mats; m += gridDim.y)
    for (int64_t t = blockIdx.x; t < rb * nb; t += gridDim.x) {
      const int64_t tr = (rb * nb) >> 32 ? t / nb : (int64_t)((uint32_t)t / (uint32_t)nb);
      const int c = (int)(t - tr * nb) * 128 + l * 8;
      const uint8_t* const xm = x + m * stride_bytes;
      OpCols raw[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t r = tr * 128 + i * 16 + sub;
        raw[i] = OpCols{};
        if (r < rows && c < cols) raw[i] = f8_load<F32, Stream>(xm + r * ld_bytes, c);
      }
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v[8];
        op_cols_get(raw[i], F32, v);
        top = max(top, f8_top(v));
      }
      top = op_max16(top);
      top = max(top, (uint32_t)__shfl_xor((int)top, 16));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32));
      // two slots in turn: who writes one again has passed the other's barrier, and
      // with it everyone's reads
      if ((threadIdx.x & 63) == 0) s_top[slot][threadIdx.x >> 6] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kF8Threads / 64; ++w) top = max(top, s_top[slot][w]);
      slot ^= 1;
      const OpF8Scale s(top);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t r = tr * 128 + i * 16 + sub;
        float v[8];
        op_cols_get(raw[i], F32, v);
        if (r < rows && c < cols) *(uint2*)(codes + (m * rows + r) * cols + c) = op_f8x8(v, s);
      }
      if (threadIdx.x == 0) scales[m * rb * nb + t] = s.scale;
    }
}

template <bool F32>
__global__ __launch_bounds__(kF8Threads) void f8_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                 const float* __restrict__ scales, int n_mats,
                                                                 int64_t rows, int cols, int tile_shift, int64_t dr,
                                                                 int db, uint8_t* __restrict__ y, int64_t ld_bytes,
                                                                 int64_t stride_bytes) {
  const int nb = (cols + 127) >> 7, l = threadIdx.x & 15;
  const int64_t sr = (rows + (1 << tile_shift) - 1) >> tile_shift;  // rows of scales
  for (int64_t m = blockIdx.y; m < n_mats; m += gridDim.y) {
    F8Walk at((int64_t)blockIdx.x * kF8Groups + (threadIdx.x >> 4), rows * nb, nb);
    for (; at.r < rows; at.next(dr, db, nb)) {
      const int c = at.b * 128 + l * 8;
      if (c >= cols) continue;
      const uint2 q = *(const uint2*)(codes + (m * rows + at.r) * cols + c);
      const float s = scales[(m * sr + (at.r >> tile_shift)) * nb + at.b];
      const op_f32x2 v0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, false), v1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, true);
      const op_f32x2 v2 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, false), v3 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, true);
      const float v[8] = {v0[0] * s, v0[1] * s, v1[0] * s, v1[1] * s, v2[0] * s, v2[1] * s, v3[0] * s, v3[1] * s};
      op_cols_store(y + m * stride_bytes + at.r * ld_bytes, F32, c, 8, v);
    }
  }
}

// workgroups for `units` blocks of 128 columns, and the walk's step as rows and blocks
static unsigned f8_walk(int64_t units, int nb, int64_t* dr, int* db) {
  const int64_t wgs = std::min<int64_t>((units + kF8Groups - 1) / kF8Groups, 1 << 16);
  *dr = wgs * kF8Groups / nb;
  *db = (int)(wgs * kF8Groups % nb);
  return (unsigned)wgs;
}

hipError_t launch_f8_quantize(const void* x, bool f32, int n_mats, int64_t rows, int cols, int64_t ldx,
                              int64_t stride, bool tiles, uint8_t* codes, float* scales, hipStream_t s) {
  const int nb = (cols + 127) / 128;
  const int64_t b = f32 ? 4 : 2;
  // An x that the memory-side cache cannot hold next to the codes is read past the
  // caches, which then keep the codes for their reader: 32768 x 4096 fp32 in tiles and
  // back 253 -> 229 us (the quantiser alone 116, 118), bf16 157 -> 142.  Smaller ones may
  // still lie there from their writer.
  const bool stream = (double)rows * cols * n_mats * b >= (double)(128 << 20);
  if (tiles) {
    const int64_t n = (rows + 127) / 128 * nb;
    const dim3 grid((unsigned)std::min<int64_t>(n, 1 << 16), (unsigned)std::min(n_mats, 1024));
    auto k = f32 ? (stream ? f8_quantize_tiles_kernel<true, true> : f8_quantize_tiles_kernel<true, false>)
                 : (stream ? f8_quantize_tiles_kernel<false, true> : f8_quantize_tiles_kernel<false, false>);
    return launch_op(k, grid, dim3(kF8Threads), s,
                     (const uint8_t*)x, n_mats, rows, cols, ldx * b, stride * b, codes, scales);
  }
  int64_t dr;
  int db;
  const unsigned wgs = f8_walk(rows * nb, nb, &dr, &db);
  auto k = f32 ? (stream ? f8_quantize_rows_kernel<true, true> : f8_quantize_rows_kernel<true, false>)
               : (stream ? f8_quantize_rows_kernel<false, true> : f8_quantize_rows_kernel<false, false>);
  return launch_op(k, dim3(wgs), dim3(kF8Threads), s,
                   (const uint8_t*)x, rows, cols, ldx * b, dr, db, codes, scales);
}

hipError_t launch_f8_dequantize(const uint8_t* codes, const float* scales, int n_mats, int64_t rows, int cols,
                                bool tiles, void* y, bool f32, int64_t ldy, int64_t stride, hipStream_t s) {
  const int nb = (cols + 127) / 128;
  const int64_t b = f32 ? 4 : 2;
  int64_t dr;
  int db;
  const unsigned wgs = f8_walk(rows * nb, nb, &dr, &db);
  return launch_op(f32 ? f8_dequantize_kernel<true> : f8_dequantize_kernel<false>, dim3(wgs, (unsigned)std::min(n_mats, 1024)),
                   dim3(kF8Threads), s, codes, scales, n_mats, rows, cols, tiles ? 7 : 0, dr, db, (uint8_t*)y, ldy * b,
                   stride * b);
}

}  // namespace moert
