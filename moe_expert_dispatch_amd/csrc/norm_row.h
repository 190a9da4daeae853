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

// The sum of a value a wave (up to 16), of which this lane has read that of wave
// lane % 16: one LDS read and four steps, where a loop over the waves waits for
// LDS as often as there are waves.
__device__ __forceinline__ float over_waves(float v) {
  return group_sum<16>((lane_id() & 15) < (int)(blockDim.x / kWave) ? v : 0.f);
}

// The lanes that hold one row: L = 16, 32 or 64 lanes of a wave (rows of one
// block then need no barrier), or the whole block (L = 0). Every lane gets the
// sum; its order does not depend on scheduling. `part` is one array for each
// of a row's sums in turn (RowParts), so that one barrier a sum is enough: where
// a block goes from row to row, an array is written again only behind the
// barrier of another one.
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
    return over_waves(part[lane_id() & 15]);
  }
}

// Two sums with one barrier.
template <int L>
__device__ __forceinline__ float2 lanes_sum2(float a, float b, float2* part) {
  if constexpr (L == 64) {
    return make_float2(wave_sum(a), wave_sum(b));
  } else if constexpr (L != 0) {
    return make_float2(group_sum<L>(a), group_sum<L>(b));
  } else {
    a = wave_sum(a);
    b = wave_sum(b);
    if (lane_id() == 0) part[threadIdx.x / kWave] = make_float2(a, b);
    __syncthreads();
    const float2 v = part[lane_id() & 15];
    return make_float2(over_waves(v.x), over_waves(v.y));
  }
}

struct RowParts {
  float mean[16];
  float2 spread[16], again[16], grad[16];  // of the deviations; of a gradient's sums
};

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

// v in f64, behind what `s` holds so far: values that rarely pass are taken one
// by one, so that their f64 forms do not take the registers of the common path
// (104 to 82 of the layer norm's gradient).
__device__ __forceinline__ double in_turn(float v, double& s) {
  asm volatile("" : "+v"(v), "+v"(s));
  return (double)v;
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
//
// Where the whole block holds a row, one vector a thread, that is a barrier for
// m and a second one. There `guess`, the mean of the row's first 8 values, takes
// the place of m first: d then is some third of the deviation, and the same two
// sums do if d^2 is no more than the variance; only the other rows go on with
// m = guess + d (gradient of 16384 rows of 4096: 121 us with two barriers, 108).
template <bool CENTRED, int VPT, int L>
__device__ __forceinline__ float normalize_row(float (&h)[VPT][8], int first, int stride, int nvec,
                                                int H, float eps, RowParts& part,
                                                float guess = 0.f) {
  const float width = (float)H;
  float m = guess, d = 0.f, ss = 0.f, var = 0.f;
  auto spread = [&](float2* into) {
    float sd = 0.f;
    ss = 0.f;
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
    const float2 sums = lanes_sum2<L>(ss, sd, into);
    ss = sums.x;
    if constexpr (CENTRED) d = sums.y / width;
    var = (CENTRED ? fmaxf(ss / width - d * d, 0.f) : ss / width) + eps;
  };
  if constexpr (CENTRED && !(L == 0 && VPT == 1)) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (first + j * stride < nvec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s += h[j][i];
      }
    m = lanes_sum<L>(s, part.mean) / width;
    spread(part.spread);
  } else {
    spread(part.spread);
    if constexpr (CENTRED) {
      // the same for all of the row's lanes; true for a NaN too
      if (!(var - eps >= d * d)) {
        m += d;
        spread(part.again);
      }
    }
  }
  const float least = CENTRED && L == 0 && VPT == 1 ? 1.f : 16.f;
  // the same for all of the row's lanes; false for a NaN too
  if (var >= kLeastSquares && var >= least * (d * d) && ss < INFINITY) {
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
        for (int i = 0; i < 8; ++i) s += in_turn(h[j][i], s);
      }
    mean = lanes_sum_f64<L>(s, wide) / H;
  }
  double sq = 0.0;
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    if (first + j * stride < nvec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double c = in_turn(h[j][i], sq) - mean;
        sq = fma(c, c, sq);
      }
    }
  double r = 1.0 / sqrt(lanes_sum_f64<L>(sq, wide) / H + (double)eps);
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) h[j][i] = (float)((in_turn(h[j][i], r) - mean) * r);
  return (float)r;
}

// The guess for rows of one vector a thread that the block holds.
__device__ __forceinline__ float mean8(const float* v) {
  return (((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]))) * 0.125f;
}

// Lanes of a row of nvec vectors of 8 values: part of a wave up to 64 vectors.
constexpr int norm_lanes(int nvec) { return nvec <= 16 ? 16 : nvec <= 32 ? 32 : nvec <= 64 ? 64 : 0; }
constexpr int kNormGroupThreads = 256;  // of a block whose rows are parts of waves

}  // namespace moe
