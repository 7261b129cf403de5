// The routed pairs of a call grouped by expert, and the weighted sum of a
// token's expert rows.
//
// Grouping is a stable counting sort by expert, with the pairs of no expert as
// one more bucket E.  A workgroup takes a chunk of consecutive pairs and each
// of its waves a run of it, 64 pairs at a time; a pair's rank among its
// wave's equal ids comes from matching the lanes' ids bit by bit with ballots,
// so ranks follow the pair order and no atomic decides anything.  Up to
// kGroupOne pairs are one workgroup's work.  Beyond that a first launch writes
// each chunk's histogram to the workspace and the second sums, per expert, the
// histograms before its own chunk and all of them, sixteen loads in flight (one
// after the other they took 15 of 22 us at 65,536 pairs and 256 experts).
// Latency bounds it: 3.4 us for 64 pairs, 7 for 4,096, 3.3 + 7.1 for 65,536.  Past
// that the second launch's sums grow with the square of the chunks: with 256 (1,024)
// experts 14.8 (25) us at 2^18 pairs, 38 (70) at 2^20, 3.6 (9.6) ms at the 2^24 that
// a call may have.
#include "ops.h"

namespace moert {

constexpr int kGroupWave = 256;     // pairs of one wave
constexpr int kGroupOne = 4096;     // one workgroup of 16 waves
constexpr int kGroupFew = 1024;     // one workgroup of 4 waves
constexpr int kGroupMany = 2048;    // chunk of a workgroup of 8 waves
constexpr int kBuckets = kMaxExperts + 1;

__device__ inline int group_bucket(const int32_t* ids, int64_t i, int64_t pairs, int E) {
  if (i >= pairs) return -1;
  const int e = ids[i];
  return e >= 0 && e < E ? e : E;
}

__global__ __launch_bounds__(256) void pairs_hist_kernel(const int32_t* __restrict__ ids, int64_t pairs, int E,
                                                         int32_t* __restrict__ hist) {
  __shared__ int32_t h[kMaxExperts];
  for (int e = threadIdx.x; e < E; e += 256) h[e] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kGroupMany + threadIdx.x;
#pragma unroll
  for (int q = 0; q < kGroupMany / 256; ++q) {
    const int b = group_bucket(ids, base + q * 256, pairs, E);
    if (b >= 0 && b < E) atomicAdd(&h[b], 1);  // integer counts: the order does not matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256) hist[(int64_t)blockIdx.x * E + e] = h[e];
}

// WAVES waves; hist == nullptr: this workgroup's chunk is the whole call.
template <int WAVES>
__global__ __launch_bounds__(WAVES * 64) void pairs_rank_kernel(const int32_t* __restrict__ ids, int64_t pairs,
                                                              int E, const int32_t* __restrict__ hist,
                                                              int n_chunks, int32_t* __restrict__ offsets,
                                                              int32_t* __restrict__ perm) {
  constexpr int T = WAVES * 64, G = kGroupWave / 64;
  __shared__ int32_t s_next[WAVES][kBuckets];  // counts, then next position per wave and bucket
  __shared__ int32_t s_scan[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t first = ((int64_t)blockIdx.x * WAVES + wave) * kGroupWave;
  int b[G];
#pragma unroll
  for (int g = 0; g < G; ++g) b[g] = group_bucket(ids, first + g * 64 + lane, pairs, E);
  for (int e = lane; e <= E; e += 64) s_next[wave][e] = 0;  // each wave its own
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int g = 0; g < G; ++g)
    if (b[g] >= 0) atomicAdd(&s_next[wave][b[g]], 1);
  __syncthreads();
  // Buckets in order, T at a time: the total of each (all chunks), their
  // exclusive scan, then the first position of each wave of this chunk.
  int carry = 0;
  for (int e0 = 0; e0 <= E; e0 += T) {
    const int e = e0 + tid;
    int total = 0, before = 0;
    if (e < E) {
      if (hist) {
        // sixteen chunks' counts requested before the first is added
        for (int c0 = 0; c0 < n_chunks; c0 += 16) {
          int n[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) n[i] = c0 + i < n_chunks ? hist[(int64_t)(c0 + i) * E + e] : 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            total += n[i];
            before += c0 + i < (int)blockIdx.x ? n[i] : 0;
          }
        }
      } else {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) total += s_next[w][e];
      }
    }
    int incl = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 63) s_scan[wave] = incl;
    __syncthreads();
    int start = carry + incl - total;
    int sum = 0;
    for (int w = 0; w < WAVES; ++w) {
      if (w < wave) start += s_scan[w];
      sum += s_scan[w];
    }
    if (e <= E) {
      if (blockIdx.x == 0) offsets[e] = start;
      int at = start + before;
      if (e < E)
        for (int w = 0; w < WAVES; ++w) {
          const int n = s_next[w][e];
          s_next[w][e] = at;
          at += n;
        }
    }
    carry += sum;
    __syncthreads();
  }
  // bucket E: positions from offsets[E] = carry on; which of them a pair takes
  // does not matter, they all receive -1, so the tail is simply filled
  for (int64_t i = carry + (int64_t)blockIdx.x * T + tid; i < pairs; i += (int64_t)gridDim.x * T) perm[i] = -1;
  // ranks: runs of 64 pairs in order, equal ids matched bit by bit
  int bits = 0;
  while ((1 << bits) < E) ++bits;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const bool in = b[g] >= 0 && b[g] < E;
    uint64_t same = __ballot(in);
    for (int i = 0; i < bits; ++i) {
      const uint64_t set = __ballot((b[g] >> i) & 1);
      same &= ((b[g] >> i) & 1) ? set : ~set;
    }
    if (in) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      const int at = s_next[wave][b[g]];
      perm[at + rank] = (int32_t)(first + g * 64 + lane);
      // the last of the equal lanes moves the wave's cursor on; a wave's LDS
      // accesses are in order, so the read above came first
      if ((same >> lane) == 1) s_next[wave][b[g]] = at + rank + 1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

size_t group_workspace(int64_t pairs, int E) {
  return pairs <= kGroupOne ? 0 : (size_t)((pairs + kGroupMany - 1) / kGroupMany) * E * 4;
}

hipError_t launch_group_pairs(const int32_t* ids, int64_t pairs, int E, int32_t* offsets, int32_t* perm,
                              int32_t* ws, hipStream_t s) {
  if (pairs <= kGroupFew)
    return launch_op(pairs_rank_kernel<4>, dim3(1), dim3(256), s, ids, pairs, E, (const int32_t*)nullptr, 1,
                     offsets, perm);
  if (pairs <= kGroupOne)
    return launch_op(pairs_rank_kernel<16>, dim3(1), dim3(1024), s, ids, pairs, E, (const int32_t*)nullptr, 1,
                     offsets, perm);
  const int chunks = (int)((pairs + kGroupMany - 1) / kGroupMany);
  hipError_t e = launch_op(pairs_hist_kernel, dim3(chunks), dim3(256), s, ids, pairs, E, ws);
  if (e != hipSuccess) return e;
  return launch_op(pairs_rank_kernel<8>, dim3(chunks), dim3(512), s, ids, pairs, E, (const int32_t*)ws, chunks,
                   offsets, perm);
}

// ------------------------------------------------------------------ combine
// y[t][h] = sum over ascending j of w[t][j] * p[t*k + j][h].  A thread holds V
// columns of one token; eight rows are requested before the first product, so
// their latencies overlap.  HBM bounds it: 65,536 fp32 rows of 4,096 into 8,192
// bf16 rows take 197 us, 5.8 TB/s (a plain copy reaches 5.1); eight tokens 3.5 us.
template <bool PF32, bool YF32, int V>
__global__ __launch_bounds__(256) void combine_kernel(const uint8_t* __restrict__ p, int64_t ldp,
                                                      const float* __restrict__ w,
                                                      const int32_t* __restrict__ ids, int E, int T, int k,
                                                      int H, uint8_t* __restrict__ y, int64_t ldy) {
  const int h = (blockIdx.x * 64 + (threadIdx.x & 63)) * V;
  if (h >= H) return;
  constexpr int PB = PF32 ? 4 : 2, YB = YF32 ? 4 : 2;
  for (int64_t t = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6); t < T; t += (int64_t)gridDim.y * 4) {
    float acc[V] = {};
    for (int j0 = 0; j0 < k; j0 += 8) {
      float v[8][V], wv[8];
      bool ok[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int64_t i = t * k + j0 + q;
        ok[q] = j0 + q < k;
        if (ok[q] && ids) {
          const int e = ids[i];
          ok[q] = e >= 0 && e < E;
        }
        wv[q] = 0.f;
#pragma unroll
        for (int c = 0; c < V; ++c) v[q][c] = 0.f;
        if (ok[q]) {
          wv[q] = w[i];
          const uint8_t* src = p + (i * ldp + h) * PB;
          if constexpr (PF32 && V == 4) {
            const op_f32x4 a = *(const op_f32x4*)src;
#pragma unroll
            for (int c = 0; c < 4; ++c) v[q][c] = a[c];
          } else if constexpr (!PF32 && V == 4) {
            const uint2 a = *(const uint2*)src;
            v[q][0] = __uint_as_float(a.x << 16);
            v[q][1] = __uint_as_float(a.x & 0xFFFF0000u);
            v[q][2] = __uint_as_float(a.y << 16);
            v[q][3] = __uint_as_float(a.y & 0xFFFF0000u);
          } else if constexpr (PF32) {
            v[q][0] = *(const float*)src;
          } else {
            v[q][0] = __uint_as_float((uint32_t)*(const uint16_t*)src << 16);
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (ok[q])
#pragma unroll
          for (int c = 0; c < V; ++c) acc[c] = fmaf(wv[q], v[q][c], acc[c]);
    }
    uint8_t* o = y + (t * ldy + h) * YB;
    if constexpr (YF32 && V == 4) {
      *(op_f32x4*)o = op_f32x4{acc[0], acc[1], acc[2], acc[3]};
    } else if constexpr (V == 4) {
      *(uint2*)o = make_uint2(op_bf16(acc[0]) | (uint32_t)op_bf16(acc[1]) << 16,
                              op_bf16(acc[2]) | (uint32_t)op_bf16(acc[3]) << 16);
    } else if constexpr (YF32) {
      *(float*)o = acc[0];
    } else {
      *(uint16_t*)o = op_bf16(acc[0]);
    }
  }
}

template <bool PF32, bool YF32>
static hipError_t combine_typed(const uint8_t* p, int64_t ldp, const float* w, const int32_t* ids, int E,
                                int T, int k, int H, uint8_t* y, int64_t ldy, hipStream_t s) {
  constexpr int64_t PB = PF32 ? 16 : 8, YB = YF32 ? 16 : 8;  // bytes of four columns
  const bool vec = H % 4 == 0 && (uintptr_t)p % PB == 0 && ldp % 4 == 0 && (uintptr_t)y % YB == 0 && ldy % 4 == 0;
  const int V = vec ? 4 : 1;
  const dim3 g((H + 64 * V - 1) / (64 * V), std::min((T - 1) / 4 + 1, 65535));
  if ((int64_t)g.x * 256 >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  return launch_op(vec ? combine_kernel<PF32, YF32, 4> : combine_kernel<PF32, YF32, 1>, g, dim3(256), s, p,
                   ldp, w, ids, E, T, k, H, y, ldy);
}

hipError_t launch_combine_pairs(const void* p, bool p_f32, int64_t ldp, const float* w, const int32_t* ids,
                                int E, int T, int k, int H, void* y, bool y_f32, int64_t ldy, hipStream_t s) {
  auto f = p_f32 ? (y_f32 ? combine_typed<true, true> : combine_typed<true, false>)
                 : (y_f32 ? combine_typed<false, true> : combine_typed<false, false>);
  return f((const uint8_t*)p, ldp, w, ids, E, T, k, H, (uint8_t*)y, ldy, s);
}

}  // namespace moert
