// MXFP4 conversion: rows to e2m1 codes with one e8m0 scale per 32 elements,
// and back.
//
// A thread holds 8 neighbouring elements, four threads a block: the block's
// largest magnitude is an integer maximum of the magnitudes' bits (the order of
// non-negative floats; infinities and NaN come out on top) over the 8 and over
// the four lanes, and its exponent field gives floor(log2 max) without any
// rounding (a subnormal maximum lies below 2^-126, where the exponent clamps
// to -127 anyway).  The division by the block's power of two, the rounding to
// the e2m1 grid with ties to even and the saturation at 6 are the gfx950
// scaled convert; the sign of what rounded to zero is taken off afterwards.
//
// HBM bounds both ways: 32768 x 4096 fp32 to MXFP4 110 us (5.5 TB/s), back 105-117
// us (5.2-5.8 TB/s; a plain copy reaches 5.1).  Four rows a thread at once were
// slower (130 us), and so were stores past the caches (back: 211 us).  A workgroup
// takes one row at a time, 2048 columns of it, so narrow rows leave lanes without
// work: 32008 x 768 bf16 16.8 us for 12.2 at the copy rate, 65536 x 64 fp32 30.7
// for 3.7.
#include "ops.h"

namespace moert {

constexpr int kMxThreads = 256;

template <bool Stream, typename V>
__device__ inline V mx_load(const uint8_t* p) {
  if constexpr (Stream) return __builtin_nontemporal_load((const V*)p);
  else return *(const V*)p;
}

// 8 elements of the row piece at x, as fp32
template <bool F32, bool Stream>
__device__ inline void mx_load8(const uint8_t* x, float (&v)[8]) {
  if constexpr (F32) {
    const op_f32x4 a = mx_load<Stream, op_f32x4>(x), b = mx_load<Stream, op_f32x4>(x + 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    const op_u32x4 a = mx_load<Stream, op_u32x4>(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}

// the block's scale byte and this lane's 8 codes; four neighbouring lanes
// hold one block
__device__ inline uint32_t mx_encode8(const float (&v)[8], uint32_t* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2));
  const uint32_t field = m >> 23;  // biased exponent of the maximum
  uint32_t s = field > 2 ? field - 2 : 0;
  s = m == 0 ? 127 : s;
  const float f = op_scale(s);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], f, 3);
  const uint32_t nonzero = (c | c >> 1 | c >> 2) & 0x11111111u;
  c &= 0x77777777u | nonzero << 3;
  const bool bad = field == 255;  // an infinity or a NaN
  *scale = bad ? 255 : s;
  return bad ? 0 : c;
}

// One row per blockIdx.y step, 8 elements per thread.
template <bool F32, bool Stream>
__global__ __launch_bounds__(kMxThreads) void mx_quantize_kernel(const uint8_t* __restrict__ x, int64_t rows,
                                                                int cols, int64_t ld_bytes,
                                                                uint8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
  const int c = blockIdx.x * kMxThreads + threadIdx.x;  // piece of 8 within the row
  const int n = cols >> 3;
  if (c >= n) return;  // whole blocks of four lanes leave together: n is a multiple of 4
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    float v[8];
    mx_load8<F32, Stream>(x + r * ld_bytes + (int64_t)c * (F32 ? 32 : 16), v);
    uint32_t s;
    const uint32_t q = mx_encode8(v, &s);
    *(uint32_t*)(codes + r * (cols >> 1) + (int64_t)c * 4) = q;
    if ((c & 3) == 0) scales[r * (cols >> 5) + (c >> 2)] = (uint8_t)s;
  }
}

template <bool F32>
__global__ __launch_bounds__(kMxThreads) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  int64_t rows, int cols,
                                                                  uint8_t* __restrict__ y, int64_t ldy,
                                                                  int vec) {
  const int c = blockIdx.x * kMxThreads + threadIdx.x;
  if (c >= cols >> 3) return;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const uint32_t q = *(const uint32_t*)(codes + r * (cols >> 1) + (int64_t)c * 4);
    const float f = op_scale(scales[r * (cols >> 5) + (c >> 2)]);
    if constexpr (F32) {
      op_f32x2 v[4];
      v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, f, 0);
      v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, f, 1);
      v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, f, 2);
      v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, f, 3);
      float* o = (float*)y + r * ldy + (int64_t)c * 8;
      if (vec) {
        *(op_f32x4*)o = op_f32x4{v[0][0], v[0][1], v[1][0], v[1][1]};
        *(op_f32x4*)(o + 4) = op_f32x4{v[2][0], v[2][1], v[3][0], v[3][1]};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = v[i >> 1][i & 1];
      }
    } else {
      const op_bf16x8 v = op_fp4x8(q, f);
      __bf16* o = (__bf16*)y + r * ldy + (int64_t)c * 8;
      if (vec) {
        *(op_bf16x8*)o = v;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = v[i];
      }
    }
  }
}

static dim3 mx_grid(int64_t rows, int cols) {
  const int gx = (cols / 8 + kMxThreads - 1) / kMxThreads;
  return dim3(gx, (unsigned)std::min<int64_t>(rows, 65535));
}

hipError_t launch_mx_quantize(const void* x, bool f32, int64_t rows, int cols, int64_t ldx, uint8_t* codes,
                              uint8_t* scales, hipStream_t s) {
  // An x that the memory-side cache cannot hold next to the codes is read past
  // the caches, which then keep the codes for their reader: 32768 x 4096 fp32 and
  // back 249 -> 215 us (the quantiser alone 104 -> 109).  Smaller ones may still lie
  // there from their writer: 8192 x 4096 bf16 16 us, 18 past the caches.
  const bool stream = rows * cols * (f32 ? 4 : 2) >= (int64_t)128 << 20;
  auto k = f32 ? (stream ? mx_quantize_kernel<true, true> : mx_quantize_kernel<true, false>)
               : (stream ? mx_quantize_kernel<false, true> : mx_quantize_kernel<false, false>);
  return launch_op(k, mx_grid(rows, cols), dim3(kMxThreads), s, (const uint8_t*)x, rows, cols,
                   ldx * (f32 ? 4 : 2), codes, scales);
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols,
                                void* y, bool f32, int64_t ldy, hipStream_t s) {
  const int64_t b = f32 ? 4 : 2;
  const int vec = ((uintptr_t)y & 15) == 0 && ldy * b % 16 == 0;
  return launch_op(f32 ? mx_dequantize_kernel<true> : mx_dequantize_kernel<false>, mx_grid(rows, cols),
                   dim3(kMxThreads), s, codes, scales, rows, cols, (uint8_t*)y, ldy, vec);
}

}  // namespace moert
