// What the norms' kernels share: sums over the lanes that hold a row, and a
// row's mean and standard deviation.
#pragma once

#include "common.h"
#include "vec8.h"

namespace moe {

// Below this mean of squares (eps included) squares may have lost bits that
// count to f32's least number; such rows, and rows whose sums leave f32's
// range, are summed in f64.
constexpr float kLeastSquares = 0x1p-80f;

// The lanes that hold one row: L = 16, 32 or 64 lanes of a wave (rows of one
// block then need no barrier), or the whole block (L = 0). Every lane gets the
// sum; its order does not depend on scheduling. `part` is one array for each
// of a row's sums in turn, 16 entries each, so that one barrier a sum is
// enough: where a block goes from row to row, an array is written again only
// behind the barrier of another one.
template <int L>
__device__ __forceinline__ float lanes_sum(float v, float* part) {
  if constexpr (L == 64) {
    return wave_sum(v);
  } else if constexpr (L != 0) {
    return group_sum<L>(v);
  } else {
    v = wave_sum(v);
    if (lane_id() == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    float total = 0.f;
    for (int w = 0; w < (int)(blockDim.x / kWave); ++w) total += part[w];
    return total;
  }
}

template <int L>
__device__ __forceinline__ double lanes_sum_f64(double v, double* part) {
#pragma unroll
  for (int o = (L == 0 ? kWave : L) / 2; o > 0; o /= 2) v += __shfl_xor(v, o, kWave);
  if constexpr (L == 0) {
    if (lane_id() == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < (int)(blockDim.x / kWave); ++w) v += part[w];
    __syncthreads();  // rows like this are rare: the array may be used again at once
  }
  return v;
}

// A row's deviation from its mean (CENTRED) or the row itself, over its
// standard deviation (eps included), in place; returns 1 / that deviation.
//
// The mean m of an f32 sum is off by some 2^-24 of the row's largest values,
// which is much where the mean is far above the deviation. So the deviations
// from m are summed once more, beside their squares: their mean d corrects
// both, mean = m + d and variance = mean((h - m)^2) - d^2, for no further
// pass over the row. Where d^2 is not small beside the rest (a row of nearly
// equal values, with an eps below their squares' last bits), f64 as well.
template <bool CENTRED, int VPT, int L>
__device__ __forceinline__ double normalize_row(float (&h)[VPT][8], int first, int stride, int nvec,
                                                int H, float eps, float (*part)[16]) {
  const float width = (float)H;
  float m = 0.f, d = 0.f;
  if constexpr (CENTRED) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (first + j * stride < nvec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s += h[j][i];
      }
    m = lanes_sum<L>(s, part[0]) / width;
  }
  float ss = 0.f, sd = 0.f;
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    if (first + j * stride < nvec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = CENTRED ? h[j][i] - m : h[j][i];
        ss = fmaf(c, c, ss);
        if constexpr (CENTRED) sd += c;
      }
    }
  ss = lanes_sum<L>(ss, part[1]);
  if constexpr (CENTRED) d = lanes_sum<L>(sd, part[2]) / width;
  const float var = (CENTRED ? fmaxf(ss / width - d * d, 0.f) : ss / width) + eps;
  // the same for all of the row's lanes; false for a NaN too
  if (var >= kLeastSquares && var >= 16.f * (d * d) && ss < INFINITY) {
    const float r = 1.0f / sqrtf(var);
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = CENTRED ? ((h[j][i] - m) - d) * r : h[j][i] * r;
    return r;
  }
  __shared__ double wide[16];
  double mean = 0.0;
  if constexpr (CENTRED) {
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (first + j * stride < nvec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s += (double)h[j][i];
      }
    mean = lanes_sum_f64<L>(s, wide) / H;
  }
  double sq = 0.0;
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    if (first + j * stride < nvec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double c = (double)h[j][i] - mean;
        sq = fma(c, c, sq);
      }
    }
  const double r = 1.0 / sqrt(lanes_sum_f64<L>(sq, wide) / H + (double)eps);
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) h[j][i] = (float)(((double)h[j][i] - mean) * r);
  return r;
}

// Lanes of a row of nvec vectors of 8 values: part of a wave up to 64 vectors.
constexpr int norm_lanes(int nvec) { return nvec <= 16 ? 16 : nvec <= 32 ? 32 : nvec <= 64 ? 64 : 0; }
constexpr int kNormGroupThreads = 256;  // of a block whose rows are parts of waves

}  // namespace moe
