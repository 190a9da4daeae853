// Expert weights in 4 bits: quantisation to E2M1 codes with one E8M0 scale
// for 32 weights, its inverse, and the grouped products that read them.
//
// Format: code s ee m, value (-1)^s {0, 0.5, 1, 1.5, 2, 3, 4, 6}; two codes
// a byte, the even index in the low four bits; scale byte b = 2^(b - 127),
// 255 = NaN. A code times its scale is a bfloat16 number (two significant
// bits), so the products run on the bf16 matrix cores without any rounding
// of the weights: gfx950 converts two codes and applies the scale in one
// instruction (v_cvt_scalef32_pk_bf16_fp4).
//
// The SwiGLU rows between the two products are rounded to bf16, since the
// matrix cores' operand is bf16 (in f32 they would be two bf16 parts: twice the
// matrix instructions and bytes). All sums and the experts' outputs are f32. The
// bf16 layer is within 0.0023-0.0024 (relative to the output's norm) of 64
// bits so, and within 0.0017 with f32 rows, which is the output's own rounding.
#include "route_token.h"
#include "vec8.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));

// The scale byte as the f32 whose exponent field it is. The conversions use
// only that field: 0 stands for 2^-127, 255 gives NaN.
__device__ __forceinline__ float e8m0(uint32_t b) { return __uint_as_float(b << 23); }

template <int SEL>
__device__ __forceinline__ uint32_t cvt_pair(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t,
                            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, SEL));
}

// Eight codes (one word) to eight bf16 values.
__device__ __forceinline__ uint4 cvt8(uint32_t codes, float scale) {
  return make_uint4(cvt_pair<0>(codes, scale), cvt_pair<1>(codes, scale),
                    cvt_pair<2>(codes, scale), cvt_pair<3>(codes, scale));
}


// Four lanes a group, 8 values each, one pass. 131072 x 4096 bf16: 240 us (5.7
// TB/s), the inverse to bf16 228 us (6.0 TB/s): bound by the bytes, the
// rounding is one instruction for two values. b = floor(log2 amax) - 2 + 127 puts the
// largest magnitude into [4, 8): above 6 it saturates. The exponent is read
// from amax's bits (a subnormal amax gives b = 0). A group with a non-finite
// value gets the NaN scale.
template <typename XT>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(const XT* __restrict__ w, int64_t n8,
                                                             uint32_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scale) {
  const int64_t i = (int64_t)folded_block() * blockDim.x + threadIdx.x;
  if (i >= n8) return;  // n8 is a multiple of 4: whole quads leave
  float v[8];
  load8(w + i * 8, v);
  uint32_t top = 0;  // largest magnitude's bits: non-finite values are the largest
#pragma unroll
  for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
  top = max(top, dpp_u32<kDppQuad1032>(top));
  top = max(top, dpp_u32<kDppQuad2301>(top));
  const int e = (int)(top >> 23);
  const uint32_t b = e == 255 ? 255u : (uint32_t)max(e - 2, 0);
  const float s = e8m0(b);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  codes[i] = c;
  if ((threadIdx.x & 3) == 0) scale[i >> 2] = (uint8_t)b;
}

template <typename OT>
__global__ __launch_bounds__(256) void dequantize_mxfp4_kernel(const uint32_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scale,
                                                               int64_t n8, OT* __restrict__ w) {
  const int64_t i = (int64_t)folded_block() * blockDim.x + threadIdx.x;
  if (i >= n8) return;
  const uint4 p = cvt8(codes[i], e8m0(scale[i >> 2]));
  if constexpr (sizeof(OT) == 2) {
    *reinterpret_cast<uint4*>(w + i * 8) = p;
  } else {
    const uint32_t u[4] = {p.x, p.y, p.z, p.w};
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = bf16_to_f32(u[k] & 0xffffu);
      v[2 * k + 1] = bf16_to_f32(u[k] >> 16);
    }
    store8(w + i * 8, v);
  }
}

// ---------------------------------------------------------------- products, few rows
// Bound by the stream of the codes. One block per (16 WN output columns,
// slot): eight waves, WN column tiles times WK waves that split the
// contraction. v_mfma_f32_16x16x32_bf16 with the weights as the first
// operand: lane l supplies weight row l mod 16 and token row l mod 16, the
// k's 32 (l / 16) .. + 31 of a 128 in four steps of 8, so a lane's codes are
// 16 consecutive bytes under one scale. Register r of lane l then holds
// column 4 (l / 16) + r of token row l mod 16. A wave walks its k's 128 RUN
// at a time with the next codes in flight, and meets no barrier on the way:
// the token rows, RB at a time, wait in LDS (all their k's, or a window of
// them where they are too long), fetched once for the block's columns. The
// WK partial sums are added in LDS in wave order.
//
// 64 slots, N = 1024 gate/up columns of Kd = 4096 (285 MB of codes and scales):
// 59 us at 1 to 4 rows a slot, 67 at 8 and 10 (4.8 and 4.2 TB/s; reading the
// same bytes and nothing else 52 us). Every wave loading its own 16-row
// fragments of the tokens from the caches instead: 84 us at 2 rows, 101 at 8.

// The codes and scales of one lane for a step: of its weight row the 16 bytes
// at k0 + 128 i + 32 g, and in byte g of s[i] their scale.
template <int M, int RUN>
struct StepWeights {
  uint4 q[M][RUN];
  uint32_t s[M][RUN];
};

// The codes' loads stand in no branch, so that they can be waited for one by
// one: at and behind kend (a wave's last k, Kd at most) they fetch the row's
// last 32 k's before it again, and the token rows in LDS hold zeros there (a
// weight among them that is no number is one of the same row, whose outputs
// are none already).
// The scales of a whole step come in one load, of whatever alignment the row
// has (a load for each 128 costs a quarter of the time at Kd = 4096).
template <int M, int RUN>
__device__ __forceinline__ void load_step(StepWeights<M, RUN>& v, const uint8_t* __restrict__ w,
                                          const uint8_t* __restrict__ w_scale,
                                          const uint32_t (&row)[M], int Kd, int k0, int kend,
                                          int g) {
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const uint32_t cb = row[i] * (uint32_t)(Kd / 2);
    const uint32_t sb = row[i] * (uint32_t)(Kd / 32);
#pragma unroll
    for (int j = 0; j < RUN; ++j)
      v.q[i][j] = *reinterpret_cast<const uint4*>(
          w + (cb + (uint32_t)min(k0 + 128 * j + 32 * g, kend - 32) / 2));
    if (k0 + 128 * RUN <= kend) {
      __builtin_memcpy(v.s[i], w_scale + (sb + (uint32_t)k0 / 32), 4 * RUN);
    } else {
#pragma unroll
      for (int j = 0; j < RUN; ++j)
        v.s[i][j] =
            (uint32_t)w_scale[sb + (uint32_t)min(k0 + 128 * j + 32 * g, kend - 32) / 32] << (8 * g);
    }
  }
}

// The scale of a lane's codes of one run.
__device__ __forceinline__ float step_scale(uint32_t s, int g) { return e8m0((s >> (8 * g)) & 255u); }

// The slot of blockIdx.y: itself, or with `find` the blockIdx.y-th slot that
// has rows (fewer rows than slots: the grid then has one line a row). Every
// wave computes it for itself. False where there is none.
__device__ __forceinline__ bool block_slot(const int32_t* __restrict__ offsets, int S,
                                           int max_rows, bool find, int* slot, int* r0, int* r1) {
  if (!find) {
    *slot = blockIdx.y;
    *r0 = min(offsets[blockIdx.y], max_rows);
    *r1 = min(offsets[blockIdx.y + 1], max_rows);
    return *r0 < *r1;
  }
  const int lane = lane_id();
  int want = blockIdx.y;
  for (int s0 = 0; s0 < S; s0 += kWave) {
    const int s = s0 + lane;
    int a = 0, b = 0;
    if (s < S) {
      a = min(offsets[s], max_rows);
      b = min(offsets[s + 1], max_rows);
    }
    uint64_t some = __ballot(b > a);
    const int n = __popcll(some);
    if (want < n) {
      for (; want > 0; --want) some &= some - 1;
      const int l = __ffsll((unsigned long long)some) - 1;
      *slot = s0 + l;
      *r0 = __builtin_amdgcn_readlane(a, l);
      *r1 = __builtin_amdgcn_readlane(b, l);
      return true;
    }
    want -= n;
  }
  return false;
}

constexpr int kStreamWaves = 8;
constexpr int kStreamLds = 64 * 1024;  // of the token rows in a block: two blocks a CU

// k's of a window: all, or equal parts that fit, in whole steps of WK waves.
__host__ __device__ inline int stream_window(int Kd, int RB, int WK) {
  const int fit = kStreamLds / (2 * RB);
  const int parts = ceil_div(Kd, fit);
  return ceil_div(ceil_div(Kd, parts), WK * 128) * WK * 128;
}
// 16-byte vectors of a row in LDS: one more, so that rows start in other banks
__host__ __device__ inline int stream_row_vecs(int window) { return window / 8 + 1; }

template <int OP, bool GATHER, typename CT, int WK, int RB, int RUN, bool PIPE,
          bool PAIRS = false>
__global__ __launch_bounds__(64 * kStreamWaves) void mxfp4_stream_kernel(
    const uint16_t* __restrict__ a, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ sorted_pairs, int topk, int S, int max_rows, int find,
    const uint8_t* __restrict__ w, const uint8_t* __restrict__ w_scale, int N, int Kd,
    CT* __restrict__ c, PairRouting routing) {
  constexpr int M = OP == MOE_GEMM_GATE_UP_SWIGLU ? 2 : 1;  // matrices (gate and up, or down)
  constexpr int WN = kStreamWaves / WK;
  extern __shared__ uint4 lds[];
  int s, r0, r1;
  if constexpr (PAIRS) {  // a pair a line, row = pair
    r0 = blockIdx.y;
    r1 = r0 + 1;
    if (routing.lanes > 0) {
      // Every block routes its pair's token; the first of a pair writes the map
      // for the down product. One token of 60 experts: 4.4 + 7.5 us as a launch
      // of its own, 11.0 in here, and the call 22.0 -> 17.9 us.
      __shared__ int routed;
      if (threadIdx.x < kWave) {
        const bool write = blockIdx.x == 0;
        const int got = routing.lanes == 8    ? route_pair<8>(routing, r0, topk, write)
                        : routing.lanes == 16 ? route_pair<16>(routing, r0, topk, write)
                                              : route_pair<32>(routing, r0, topk, write);
        if (threadIdx.x == 0) routed = got;
      }
      __syncthreads();
      s = __builtin_amdgcn_readfirstlane(routed);
      if (s < 0) return;
    } else {
      s = routing.map.slot[r0];
      if (routing.map.mask[r0] == 0 || s < 0 || s >= S) return;
    }
  } else {
    if (!block_slot(offsets, S, max_rows, find != 0, &s, &r0, &r1)) return;
  }
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wk = wave % WK, wn = wave / WK;
  const int m = lane & 15, g = lane >> 4;
  const int n0 = (blockIdx.x * WN + wn) * 16;
  const bool tile = n0 < N;  // N is a multiple of 16
  uint32_t wrow[M];
#pragma unroll
  for (int i = 0; i < M; ++i) wrow[i] = (uint32_t)(i * N + (tile ? n0 : 0) + m);
  const size_t rows_s = (size_t)s * M * N;
  const uint8_t* ws = w + rows_s * (size_t)(Kd / 2);
  const uint8_t* ss = w_scale + rows_s * (size_t)(Kd / 32);
  const int window = stream_window(Kd, RB, WK);
  const int per = window / WK;  // k's of a wave in a window, whole 128s
  const int rvecs = stream_row_vecs(window);
  const int pieces = ceil_div(window, 8 * kWave);

  for (int rt = r0; rt < r1; rt += RB) {
    const int nr = min(r1 - rt, RB);
    // keeps the first loads, and with them the conversions, from being moved
    // out of the loop, where the converted codes would fill 128 registers
    asm volatile("" ::: "memory");
    floatx4 acc[M];
#pragma unroll
    for (int i = 0; i < M; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
    StepWeights<M, RUN> cur, next;
    load_step<M, RUN>(cur, ws, ss, wrow, Kd, wk * per, min((wk + 1) * per, Kd), g);
    for (int base = 0; base < Kd; base += window) {
      if (base != 0) __syncthreads();  // the last window is read
      // a wave fetches 512 k's of a row at a time
      for (int u = wave; u < nr * pieces; u += kStreamWaves) {
        const int r = u / pieces;
        const int v = (u - r * pieces) * kWave + lane;
        int row = rt + r;
        if constexpr (PAIRS)
          row = row / topk;
        else if constexpr (GATHER)
          row = sorted_pairs[row] / topk;
        if (v < window / 8)
          lds[r * rvecs + v] =
              base + 8 * v < Kd
                  ? *reinterpret_cast<const uint4*>(a + (size_t)row * Kd + base + 8 * v)
                  : make_uint4(0, 0, 0, 0);
      }
      __syncthreads();
      for (int at = 0; at < per; at += 128 * RUN) {
        if constexpr (PIPE) {
          // the next step's codes: in this window, or the first of the next
          const bool last = at + 128 * RUN >= per;
          const int nbase = base + (last ? window : 0) + wk * per;
          load_step<M, RUN>(next, ws, ss, wrow, Kd, nbase + (last ? 0 : at + 128 * RUN),
                                     min(nbase + per, Kd), g);
        }
        const uint4* x = lds + (m < nr ? m : 0) * rvecs + (wk * per + at) / 8 + 4 * g;
#pragma unroll
        for (int j = 0; j < RUN; ++j) {
          if (at + 128 * j >= per) break;  // the same for the whole block
          uint4 b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) b[e] = m < nr ? x[16 * j + e] : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < M; ++i) {
            const float sc = step_scale(cur.s[i][j], g);
            const uint32_t qq[4] = {cur.q[i][j].x, cur.q[i][j].y, cur.q[i][j].z, cur.q[i][j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8_t, cvt8(qq[e], sc)),
                  __builtin_bit_cast(bf16x8_t, b[e]), acc[i], 0, 0, 0);
          }
        }
        if constexpr (PIPE) cur = next;
      }
    }
    if constexpr (WK > 1) {
      __syncthreads();  // the rows are read: the partial sums take their place
      floatx4* red = reinterpret_cast<floatx4*>(lds) + wn * WK * M * kWave;
#pragma unroll
      for (int i = 0; i < M; ++i) red[(wk * M + i) * kWave + lane] = acc[i];
      __syncthreads();
      if (wk == 0) {
#pragma unroll
        for (int i = 0; i < M; ++i)
          for (int u = 1; u < WK; ++u) acc[i] += red[(u * M + i) * kWave + lane];
      }
    }
    if (wk == 0 && tile && m < nr) {
      float o[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        o[r] = acc[0][r];
        if constexpr (M == 2) o[r] = o[r] / (1.0f + expf(-o[r])) * acc[1][r];
      }
      CT* p = c + (size_t)(rt + m) * N + n0 + 4 * g;
      if constexpr (sizeof(CT) == 2)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
      else
        *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
    }
    if (rt + RB < r1) __syncthreads();  // rows and partial sums are read
  }
}

// The same for contractions of at most 512 WK k's and very few rows: a wave's
// part is one step, and it keeps its own k's of the rows, RB = 4 of them, in
// its own LDS, so waves meet only to add up. Many short blocks leave no tail:
// with 66 of 80 slots in use (N = 1024, Kd = 4096) the kernel above has 528
// blocks for 256 places, a third round for 16 of them: 77 us, this one 66.
// Past RB rows a slot it reads the codes again: 69 against 60 us at 4 rows a
// slot everywhere.
template <int OP, bool GATHER, typename CT, int WK>
__global__ __launch_bounds__(64 * kStreamWaves) void mxfp4_quick_kernel(
    const uint16_t* __restrict__ a, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ sorted_pairs, int topk, int S, int max_rows, int find,
    const uint8_t* __restrict__ w, const uint8_t* __restrict__ w_scale, int N, int Kd,
    CT* __restrict__ c) {
  constexpr int M = OP == MOE_GEMM_GATE_UP_SWIGLU ? 2 : 1;
  constexpr int WN = kStreamWaves / WK;
  constexpr int RUN = 4;
  constexpr int RB = 4;
  constexpr int kRowVecs = 128 * RUN / 8 + 1;
  __shared__ uint4 lds[kStreamWaves][RB * kRowVecs];
  __shared__ floatx4 red[WK > 1 ? kStreamWaves : 1][M][kWave];
  int s, r0, r1;
  if (!block_slot(offsets, S, max_rows, find != 0, &s, &r0, &r1)) return;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int wk = wave % WK, wn = wave / WK;
  const int m = lane & 15, g = lane >> 4;
  const int n0 = (blockIdx.x * WN + wn) * 16;
  const bool tile = n0 < N;
  uint32_t wrow[M];
#pragma unroll
  for (int i = 0; i < M; ++i) wrow[i] = (uint32_t)(i * N + (tile ? n0 : 0) + m);
  const size_t rows_s = (size_t)s * M * N;
  const uint8_t* ws = w + rows_s * (size_t)(Kd / 2);
  const uint8_t* ss = w_scale + rows_s * (size_t)(Kd / 32);
  const int per = ceil_div(ceil_div(Kd, 128), WK) * 128;  // at most 128 * RUN
  const int k0 = wk * per;
  const int kend = min(k0 + per, Kd);
  for (int rt = r0; rt < r1; rt += RB) {
    // keeps the loads, and with them the conversions, from being moved out of the loop, where
    // the converted codes would fill 128 registers
    asm volatile("" ::: "memory");
    const int nr = min(r1 - rt, RB);
    StepWeights<M, RUN> v;
    load_step<M, RUN>(v, ws, ss, wrow, Kd, k0, kend, g);
    for (int r = 0; r < nr; ++r) {
      int row = rt + r;
      if constexpr (GATHER) row = sorted_pairs[row] / topk;
      lds[wave][r * kRowVecs + lane] =
          k0 + 8 * lane < kend
              ? *reinterpret_cast<const uint4*>(a + (size_t)row * Kd + k0 + 8 * lane)
              : make_uint4(0, 0, 0, 0);
    }
    wave_lds_fence();
    floatx4 acc[M];
#pragma unroll
    for (int i = 0; i < M; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
    const uint4* x = &lds[wave][(m < nr ? m : 0) * kRowVecs + 4 * g];
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      uint4 b[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = m < nr ? x[16 * j + e] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const float sc = step_scale(v.s[i][j], g);
        const uint32_t qq[4] = {v.q[i][j].x, v.q[i][j].y, v.q[i][j].z, v.q[i][j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_t, cvt8(qq[e], sc)), __builtin_bit_cast(bf16x8_t, b[e]),
              acc[i], 0, 0, 0);
      }
    }
    if constexpr (WK > 1) {
#pragma unroll
      for (int i = 0; i < M; ++i) red[wave][i][lane] = acc[i];
      __syncthreads();
      if (wk == 0) {
#pragma unroll
        for (int i = 0; i < M; ++i)
          for (int u = 1; u < WK; ++u) acc[i] += red[wave + u][i][lane];
      }
    }
    if (wk == 0 && tile && m < nr) {
      float o[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        o[r] = acc[0][r];
        if constexpr (M == 2) o[r] = o[r] / (1.0f + expf(-o[r])) * acc[1][r];
      }
      CT* p = c + (size_t)(rt + m) * N + n0 + 4 * g;
      if constexpr (sizeof(CT) == 2)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
      else
        *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
    }
    if (WK > 1 && rt + RB < r1) __syncthreads();
  }
}

// ---------------------------------------------------------------- products, many rows
// One block per (up to 160 token rows of a slot, 256 weight rows): the same
// 128 gate and up rows, or 256 rows of down. Four waves, each with 64 weight rows
// (gate and up of 32 columns, or 64 columns) against all the tokens, so a
// weight is converted once in a block and never passes through LDS; the
// tokens' rows, which all waves need, do: stages of 64 k's, two of them,
// fetched into registers while the other feeds the matrix cores
// (v_mfma_f32_32x32x16_bf16, weights first). Lane l holds weight row
// l mod 32 and the k's 32 (l / 32) .. + 31 of a stage: 16 bytes of codes
// under one scale. LDS rows are 128 bytes, their 16-byte chunks XOR-swizzled
// by (row / 2 mod 8): 16 lanes then read from all 64 banks.
//
// 64 slots of N = 1024 gate/up columns, Kd = 4096: 165 us at 128 rows a slot
// (835 TFLOP/s), 188 at 160 (910), 319 at 320 (1080; a library product of
// 8192^3 reaches 1240). Tiles up to 128 rows need a third one, of 4 rows, at
// 260 rows a slot, at half the cost of a whole one: 393 us, with these 315.
// Their sums fill 160 registers of 256, so the codes of a tile over 128 rows
// are fetched one unit ahead instead of two. LDS reads run two ahead of their
// matrix instructions (left to the compiler's order and with loads in
// branches: 171 us at 128 rows, 328 at 320; three or four ahead: no
// difference). Stages of 128 k's (half the barriers, twice the distance of the
// fetches) were no faster, nor were 8 waves that share the tile by rows and
// convert every weight twice (533 TFLOP/s at 128 rows).
constexpr int kTileRows = 160;
constexpr int kTileWeights = 256;
constexpr int kStage = 64;

typedef float floatx16 __attribute__((ext_vector_type(16)));

// Finds row tile `tile` of the slots, in slot order: the slot, its rows
// [r0, r1) in the tile; false behind the last. A slot has as few tiles of at
// most TR rows as hold its rows, of one size in whole 32s (the last one less).
// Every wave computes it for itself (a scan over 64 slots at a time).
template <int TR>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ offsets, int S,
                                          int max_rows, int tile, int* slot, int* r0, int* r1) {
  const int lane = lane_id();
  for (int s0 = 0; s0 < S; s0 += kWave) {
    const int s = s0 + lane;
    int a = 0, b = 0;
    if (s < S) {
      a = min(offsets[s], max_rows);
      b = min(offsets[s + 1], max_rows);
    }
    const int n = ceil_div(b - a, TR);
    int incl = n;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int v = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += v;
    }
    const uint64_t hit = __ballot(incl > tile);
    if (hit != 0) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int count = __builtin_amdgcn_readlane(n, l);
      const int at = tile - (__builtin_amdgcn_readlane(incl, l) - count);
      const int first = __builtin_amdgcn_readlane(a, l);
      const int end = __builtin_amdgcn_readlane(b, l);
      const int step = ceil_div(ceil_div(end - first, count), 32) * 32;
      *slot = s0 + l;
      *r0 = first + at * step;
      *r1 = min(*r0 + step, end);
      return true;
    }
    tile -= __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  return false;
}

// NT: 32-token blocks of the tile that hold rows.
template <int OP, typename CT, int NT>
__device__ __forceinline__ void tile_product(uint4 (*stage)[kTileRows * 8],
                                             const uint16_t* const (&src)[5], int r0, int rows,
                                             const uint8_t* __restrict__ w,
                                             const uint8_t* __restrict__ w_scale, int n0, int N,
                                             int Kd, CT* __restrict__ c) {
  constexpr bool GU = OP == MOE_GEMM_GATE_UP_SWIGLU;
  const int tid = threadIdx.x;
  const int lane = lane_id();
  const int wave = tid / kWave;
  const int m = lane & 31, h = lane >> 5;
  // first columns of the wave's two blocks of 32 weight rows (whole blocks:
  // N is a multiple of 32); a block past the end computes on another's rows
  const int col0 = GU ? n0 + 32 * wave : n0 + 64 * wave;
  const int col1 = GU ? col0 : col0 + 32;
  const int row0 = min(col0, N - 32) + m;
  const int row1 = GU ? N + row0 : min(col1, N - 32) + m;
  // 32-bit offsets into the slot's panel (below 2^31 bytes: weight_panel_ok);
  // a sixteenth of a code's offset is that of its scale
  const uint32_t wp[2] = {(uint32_t)row0 * (uint32_t)(Kd / 2), (uint32_t)row1 * (uint32_t)(Kd / 2)};

  constexpr int AHEAD = 2;  // LDS reads in flight before the first product
  floatx16 acc[2][NT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = floatx16{};

  // Thread tid fetches chunk tid % 8 of rows tid / 8 + 32 i. Loads stand in no
  // branch (see load_step): past Kd they fetch what was before it again, and
  // zeros are put for the tokens.
  const int chunk = tid & 7;
  uint4 fa[NT];
  auto fetch = [&](int k0) {
    const int at = min(k0 + 8 * chunk, Kd - 8);
#pragma unroll
    for (int i = 0; i < NT; ++i) fa[i] = *reinterpret_cast<const uint4*>(src[i] + at);
  };
  auto put = [&](int b, int k0) {
    const int r = tid >> 3;
    if (k0 + kStage > Kd && k0 + 8 * chunk >= Kd)
#pragma unroll
      for (int i = 0; i < NT; ++i) fa[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NT; ++i) stage[b][(r + 32 * i) * 8 + (chunk ^ ((r >> 1) & 7))] = fa[i];
  };
  // Codes and scales of U units of 64 k's, fetched as many ahead: two, or one
  // where the sums of 160 rows leave no registers.
  constexpr int U = NT <= 4 ? 2 : 1;
  uint4 q[2][U], qn[2][U];
  uint32_t sc[2][U], scn[2][U];
  auto load_codes = [&](int k0, uint4 (&qq)[2][U], uint32_t (&ss)[2][U]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t at = wp[i] + (uint32_t)min(k0 + kStage * u + 32 * h, Kd - 32) / 2;
        qq[i][u] = *reinterpret_cast<const uint4*>(w + at);
        ss[i][u] = w_scale[at / 16];
      }
  };
  auto compute = [&](int b, int u) {
    __builtin_amdgcn_sched_barrier(0);  // the next stage's loads are on their way
    const float s0 = e8m0(sc[0][u]), s1 = e8m0(sc[1][u]);
    const uint32_t q0[4] = {q[0][u].x, q[0][u].y, q[0][u].z, q[0][u].w};
    const uint32_t q1[4] = {q[1][u].x, q[1][u].y, q[1][u].z, q[1][u].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8_t a0 = __builtin_bit_cast(bf16x8_t, cvt8(q0[j], s0));
      const bf16x8_t a1 = __builtin_bit_cast(bf16x8_t, cvt8(q1[j], s1));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const bf16x8_t x = __builtin_bit_cast(
            bf16x8_t, stage[b][(32 * t + m) * 8 + ((4 * h + j) ^ ((m >> 1) & 7))]);
        acc[0][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a0, x, acc[0][t], 0, 0, 0);
        acc[1][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a1, x, acc[1][t], 0, 0, 0);
      }
    }
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
    for (int i = 0; i < 4 * NT - AHEAD; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, 2 * AHEAD, 0);
  };

  fetch(0);
  load_codes(0, q, sc);
  put(0, 0);
  __syncthreads();
  for (int k0 = 0; k0 < Kd; k0 += 2 * kStage) {
#pragma unroll
    for (int v = 0; v < 2; ++v) {  // the stage in buffer v, the next into the other
      fetch(k0 + (v + 1) * kStage);
      if (U == 1 || v == 0) load_codes(k0 + (U == 1 ? v + 1 : 2) * kStage, qn, scn);
      compute(v, U == 1 ? 0 : v);
      put(v ^ 1, k0 + (v + 1) * kStage);
      __syncthreads();
      if (U == 1 || v == 1) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            q[i][u] = qn[i][u];
            sc[i][u] = scn[i][u];
          }
      }
    }
  }

#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int tok = 32 * t + m;
    if (tok >= rows) continue;
    CT* crow = c + (size_t)(r0 + tok) * N;
#pragma unroll
    for (int i = 0; i < (GU ? 1 : 2); ++i) {
      const int cb = i == 0 ? col0 : col1;
      if (cb >= N) continue;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[e] = acc[i][t][4 * v + e];
          if constexpr (GU) o[e] = o[e] / (1.0f + expf(-o[e])) * acc[1][t][4 * v + e];
        }
        CT* p = crow + cb + 8 * v + 4 * h;
        if constexpr (sizeof(CT) == 2)
          *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
        else
          *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// Blocks b, b + 8, ... run on one XCD (workgroups are dealt round-robin, and the
// lines of a folded grid are whole eights):
// it takes whole groups of two row tiles and all their columns, so the two
// tiles of a slot share its weights in that XCD's L2.
template <int OP, bool GATHER, typename CT>
__global__ __launch_bounds__(256, 2) void mxfp4_tile_kernel(
    const uint16_t* __restrict__ a, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ sorted_pairs, int topk, int S, int max_rows,
    const uint8_t* __restrict__ w, const uint8_t* __restrict__ w_scale, int N, int Kd,
    CT* __restrict__ c) {
  constexpr int M = OP == MOE_GEMM_GATE_UP_SWIGLU ? 2 : 1;
  __shared__ uint4 stage[2][kTileRows * 8];
  const int ncol = ceil_div(N, kTileWeights / M);
  const int group = 2 * ncol;
  const int in = (int)(folded_block() >> 3);
  const int tile = ((in / group) * 8 + (int)(folded_block() & 7)) * 2 + (in % group) % 2;
  const int n0 = (in % group) / 2 * (kTileWeights / M);
  int s = 0, r0 = 0, r1 = 0;
  if (!find_tile<kTileRows>(offsets, S, max_rows, tile, &s, &r0, &r1)) return;
  const int rows = r1 - r0;
  const uint16_t* src[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    int row = r0 + min((int)(threadIdx.x >> 3) + 32 * i, rows - 1);
    if constexpr (GATHER) row = sorted_pairs[row] / topk;
    src[i] = a + (size_t)row * Kd;
  }
  const size_t wrow = (size_t)s * M * N;
  const uint8_t* ws = w + wrow * (Kd / 2);
  const uint8_t* ss = w_scale + wrow * (Kd / 32);
  if (rows <= 32)
    tile_product<OP, CT, 1>(stage, src, r0, rows, ws, ss, n0, N, Kd, c);
  else if (rows <= 64)
    tile_product<OP, CT, 2>(stage, src, r0, rows, ws, ss, n0, N, Kd, c);
  else if (rows <= 96)
    tile_product<OP, CT, 3>(stage, src, r0, rows, ws, ss, n0, N, Kd, c);
  else if (rows <= 128)
    tile_product<OP, CT, 4>(stage, src, r0, rows, ws, ss, n0, N, Kd, c);
  else
    tile_product<OP, CT, 5>(stage, src, r0, rows, ws, ss, n0, N, Kd, c);
}

// ---------------------------------------------------------------- products, some rows
// Between the two: tiles of 32 NT token rows against 256 weight rows, still
// bound by the stream of the codes. Eight waves: four of 64 weight rows, as
// above, twice, the two halves taking every other run of 64 U k's, so a block
// has twice the loads in flight and half the steps; the second half's sums
// are added in LDS at the end. A step's codes and the tokens' rows are fetched
// a step ahead. NT = 1 with steps of 128 k's (U = 2: two blocks a compute unit)
// 64 slots of N = 1024 gate/up columns, Kd = 4096: 88 us from 4 to 32 rows a
// slot, where the tiles above take 120 to 130; NT = 2, U = 4: 113 us at
// 64 rows against 137. For the down product (Kd = 1024) NT = 1 takes 43 to 47
// us against 51 to 57, NT = 2 no less than the tiles above (68 to 88 against
// 57 to 65), so it is not there.
template <int OP, bool GATHER, typename CT, int NT, int U>
__global__ __launch_bounds__(512, U == 2 ? 2 : 1) void mxfp4_split_kernel(
    const uint16_t* __restrict__ a, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ sorted_pairs, int topk, int S, int max_rows,
    const uint8_t* __restrict__ w, const uint8_t* __restrict__ w_scale, int N, int Kd,
    CT* __restrict__ c) {
  constexpr bool GU = OP == MOE_GEMM_GATE_UP_SWIGLU;
  constexpr int M = GU ? 2 : 1;
  constexpr int TR = 32 * NT;
  constexpr int kRun64 = 64 * U;              // k's of a half's step
  constexpr int kVecs = TR * 8 * U;           // 16-byte vectors of a half's stage
  constexpr int kFetch = kVecs / 256;         // of them a thread's
  __shared__ uint4 stage[2][2][kVecs];        // [half][buffer][unit, row, swizzled chunk]
  static_assert(sizeof(stage) >= 2u * NT * 16 * 4 * 256, "the second half's sums fit");
  const int ncol = ceil_div(N, kTileWeights / M);
  const int group = 2 * ncol;
  const int bi = (int)(folded_block() >> 3);
  const int tile = ((bi / group) * 8 + (int)(folded_block() & 7)) * 2 + (bi % group) % 2;
  const int n0 = (bi % group) / 2 * (kTileWeights / M);
  int s = 0, r0 = 0, r1 = 0;
  if (!find_tile<TR>(offsets, S, max_rows, tile, &s, &r0, &r1)) return;
  const int rows = r1 - r0;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int half = wave >> 2, wn = wave & 3;
  const int tid = threadIdx.x & 255;  // in the half
  const int m = lane & 31, h = lane >> 5;
  const int col0 = GU ? n0 + 32 * wn : n0 + 64 * wn;
  const int col1 = GU ? col0 : col0 + 32;
  const uint32_t row[2] = {(uint32_t)(min(col0, N - 32) + m),
                           (uint32_t)(GU ? N + min(col0, N - 32) + m : min(col1, N - 32) + m)};
  const size_t wrow = (size_t)s * M * N;
  const uint8_t* ws = w + wrow * (Kd / 2);
  const uint8_t* ss = w_scale + wrow * (Kd / 32);

  struct Codes {
    uint4 q[2][U];
    uint32_t s[2][(U + 1) / 2];  // byte 2 u + h: the scale of unit u
  };
  auto load_codes = [&](Codes& v, int kb) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t cb = row[i] * (uint32_t)(Kd / 2);
      const uint32_t sb = row[i] * (uint32_t)(Kd / 32);
#pragma unroll
      for (int u = 0; u < U; ++u)
        v.q[i][u] = *reinterpret_cast<const uint4*>(
            ws + (cb + (uint32_t)min(kb + 64 * u + 32 * h, Kd - 32) / 2));
      if (kb + kRun64 <= Kd) {
        __builtin_memcpy(v.s[i], ss + (sb + (uint32_t)kb / 32), 2 * U);
      } else {
#pragma unroll
        for (int x = 0; x < U / 2; ++x) v.s[i][x] = 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
          v.s[i][u / 2] |= (uint32_t)ss[sb + (uint32_t)min(kb + 64 * u + 32 * h, Kd - 32) / 32]
                           << (16 * (u & 1) + 8 * h);
      }
    }
  };
  // vector v = tid + 256 i of a stage: unit v / (8 TR), row (v / 8) mod TR, chunk v mod 8
  const uint16_t* src[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    int r = r0 + min((tid >> 3) + 32 * i, rows - 1);
    if constexpr (GATHER) r = sorted_pairs[r] / topk;
    src[i] = a + (size_t)r * Kd;
  }
  uint4 fa[kFetch];
  const int chunk = tid & 7;
  auto fetch = [&](int kb) {
#pragma unroll
    for (int i = 0; i < kFetch; ++i)
      fa[i] = *reinterpret_cast<const uint4*>(src[i % NT] +
                                              min(kb + 64 * (i / NT) + 8 * chunk, Kd - 8));
  };
  auto put = [&](int b, int kb) {
    if (kb + kRun64 > Kd) {
#pragma unroll
      for (int i = 0; i < kFetch; ++i)
        if (kb + 64 * (i / NT) + 8 * chunk >= Kd) fa[i] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kFetch; ++i) {
      const int r = (tid >> 3) + 32 * (i % NT);
      stage[half][b][(i / NT) * TR * 8 + r * 8 + (chunk ^ ((r >> 1) & 7))] = fa[i];
    }
  };

  floatx16 acc[2][NT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = floatx16{};
  const int steps = ceil_div(Kd, 2 * kRun64);
  const int kb0 = half * kRun64;
  Codes cur, next;
  load_codes(cur, kb0);
  fetch(kb0);
  put(0, kb0);
  __syncthreads();
  for (int st = 0; st < steps; ++st) {
    const int kn = kb0 + (st + 1) * 2 * kRun64;
    if (st + 1 < steps) {
      load_codes(next, kn);
      fetch(kn);
    }
    __builtin_amdgcn_sched_barrier(0);
    const int b = st & 1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float s0 = e8m0((cur.s[0][u / 2] >> (16 * (u & 1) + 8 * h)) & 255u);
      const float s1 = e8m0((cur.s[1][u / 2] >> (16 * (u & 1) + 8 * h)) & 255u);
      const uint32_t q0[4] = {cur.q[0][u].x, cur.q[0][u].y, cur.q[0][u].z, cur.q[0][u].w};
      const uint32_t q1[4] = {cur.q[1][u].x, cur.q[1][u].y, cur.q[1][u].z, cur.q[1][u].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8_t a0 = __builtin_bit_cast(bf16x8_t, cvt8(q0[j], s0));
        const bf16x8_t a1 = __builtin_bit_cast(bf16x8_t, cvt8(q1[j], s1));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const bf16x8_t x = __builtin_bit_cast(
              bf16x8_t,
              stage[half][b][u * TR * 8 + (32 * t + m) * 8 + ((4 * h + j) ^ ((m >> 1) & 7))]);
          acc[0][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a0, x, acc[0][t], 0, 0, 0);
          acc[1][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a1, x, acc[1][t], 0, 0, 0);
        }
      }
    }
    if (st + 1 < steps) {
      put(b ^ 1, kn);
      cur = next;
    }
    __syncthreads();
  }

  floatx4* red = reinterpret_cast<floatx4*>(&stage[0][0][0]);
  if (half == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          red[((i * NT + t) * 4 + v) * 256 + tid] =
              floatx4{acc[i][t][4 * v], acc[i][t][4 * v + 1], acc[i][t][4 * v + 2],
                      acc[i][t][4 * v + 3]};
  }
  __syncthreads();
  if (half == 1) return;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int tok = 32 * t + m;
    if (tok >= rows) continue;
    CT* crow = c + (size_t)(r0 + tok) * N;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const floatx4 e0 = red[(t * 4 + v) * 256 + tid];
      const floatx4 e1 = red[((NT + t) * 4 + v) * 256 + tid];
      float o[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[0][e] = acc[0][t][4 * v + e] + e0[e];
        o[1][e] = acc[1][t][4 * v + e] + e1[e];
        if constexpr (GU) o[0][e] = o[0][e] / (1.0f + expf(-o[0][e])) * o[1][e];
      }
#pragma unroll
      for (int i = 0; i < (GU ? 1 : 2); ++i) {
        const int cb = i == 0 ? col0 : col1;
        if (cb >= N) continue;
        CT* p = crow + cb + 8 * v + 4 * h;
        if constexpr (sizeof(CT) == 2)
          *reinterpret_cast<uint2*>(p) =
              make_uint2(pack_bf16x2(o[i][0], o[i][1]), pack_bf16x2(o[i][2], o[i][3]));
        else
          *reinterpret_cast<float4*>(p) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
      }
    }
  }
}

// ---------------------------------------------------------------- a few tokens
// The down product of a token's pairs and their weighted sum in one: block
// (16 output columns, token). The waves share the token's (pair, run of 512
// k's) units; each adds weight * partial product to its sums, and the sums
// are added in LDS in wave order. Of the 16 token columns of the matrix
// instruction one is used: the codes' stream, not the product, is the bound.
template <typename OT>
__global__ __launch_bounds__(512) void mxfp4_pair_down_kernel(
    const uint16_t* __restrict__ act, const int32_t* __restrict__ slot,
    const uint8_t* __restrict__ mask, const float* __restrict__ weight, int topk, int S,
    const uint8_t* __restrict__ w, const uint8_t* __restrict__ w_scale, int N, int Kd,
    OT* __restrict__ out, int accumulate, const uint16_t* __restrict__ shared) {
  constexpr int RUN = 4;
  __shared__ floatx4 red[kStreamWaves][4];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int m = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * 16;
  const int t = blockIdx.y;
  const uint32_t row[1] = {(uint32_t)(n0 + m)};
  const int runs = ceil_div(Kd, 128 * RUN);
  floatx4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int u = wave; u < topk * runs; u += kStreamWaves) {
    const int p = t * topk + u / runs;
    const int k0 = (u % runs) * 128 * RUN;
    const int s = slot[p];
    if (mask[p] == 0 || s < 0 || s >= S) continue;  // the same for the whole wave
    const float wt = weight[p];
    StepWeights<1, RUN> v;
    load_step<1, RUN>(v, w + (size_t)s * N * (size_t)(Kd / 2),
                               w_scale + (size_t)s * N * (size_t)(Kd / 32), row, Kd, k0,
                               min(k0 + 128 * RUN, Kd), g);
    const uint16_t* x = act + (size_t)p * Kd + k0 + 32 * g;
    uint4 b[RUN][4];
#pragma unroll
    for (int j = 0; j < RUN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        b[j][e] = m == 0 && k0 + 128 * j + 32 * g < Kd
                      ? *reinterpret_cast<const uint4*>(x + 128 * j + 8 * e)
                      : make_uint4(0, 0, 0, 0);
    floatx4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      const float sc = step_scale(v.s[0][j], g);
      const uint32_t qq[4] = {v.q[0][j].x, v.q[0][j].y, v.q[0][j].z, v.q[0][j].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            __builtin_bit_cast(bf16x8_t, cvt8(qq[e], sc)), __builtin_bit_cast(bf16x8_t, b[j][e]),
            acc, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) sum[r] = fmaf(wt, acc[r], sum[r]);
  }
  if (m == 0) red[wave][g] = sum;
  __syncthreads();
  if (threadIdx.x < 4) {
    floatx4 o = red[0][threadIdx.x];
    for (int v = 1; v < kStreamWaves; ++v) o += red[v][threadIdx.x];
    const size_t at = (size_t)t * N + n0 + 4 * threadIdx.x;
    if (shared != nullptr) {
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] += bf16_to_f32(shared[at + r]);
    }
    OT* p = out + at;
    if constexpr (sizeof(OT) == 2) {
      if (accumulate) {
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = bf16_to_f32(p[r]) + o[r];
      }
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    } else {
      if (accumulate) {
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = p[r] + o[r];
      }
      *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
    }
  }
}

// Which kernel, by the rows a slot has on the average of all (rows / S: the
// rows to expect, those of one share of the tokens' pairs; the host knows no
// more, and max_rows bounds them all: a caller's capacity far over the rows
// there are takes the kernel of the capacity). Slots far over the average are
// right in every kernel, but in the streaming ones a block reads its codes
// again for every RB rows. Measured with rows drawn evenly. Both sides in us at
// 64 slots, Kd = 4096 / N = 1024 gate/up and Kd = 1024 / N = 4096 down: 16 rows a
// slot 71 and 42 streamed
// (16 rows at a time), 88 and 45 split, but a slot past 16 streams its codes
// twice (12 rows a slot on the average already have one in six past it); at 31
// 88 and 46 split, but past 32 twice; at 64 113 split by 64 rows, 137 in tiles.
// 64 rows pay where the contraction is long: at 48 rows a slot Kd = 4096 99
// and 118 us, 2560 67 and 69, 1280 41 and 33, 640 32 and 20.
// A few large slots leave the chip empty with tiles of 160 rows, so there the
// smaller ones are taken while all of them run at once: 8 slots of 100 rows,
// Kd = 4096 / N = 1024: 38 us by 32 rows, 41 by 64, 71 in tiles; of 160 rows 59, 43
// and 70; of 500 115, 83 and 76. Down, Kd = 1024 / N = 4096, 32 rows and tiles:
// 20 and 25 us at 100 rows, 35 and 27 at 250.
constexpr int kStreamRows = 10;
constexpr int kSplitRows1 = 24;
constexpr int kSplitRows2 = 56;

template <int OP, bool GATHER, typename CT>
void launch_product(const void* a, const int32_t* offsets, const int32_t* sorted_pairs, int topk,
                    int S, int max_rows, int rows, const uint8_t* w, const uint8_t* w_scale,
                    int N, int Kd, void* c, hipStream_t stream) {
  using std::integral_constant;
  constexpr int M = OP == MOE_GEMM_GATE_UP_SWIGLU ? 2 : 1;
  // Blocks for all tiles of `tr` rows, of which there are at most this many
  // whatever the slots' counts: groups of two row tiles, eight XCDs.
  auto tile_grid = [&](int tr, int threads) {
    const int64_t tiles = (int64_t)max_rows / tr + S;
    return folded((tiles + 15) / 16 * 8 * 2 * ceil_div(N, kTileWeights / M), threads, 8);
  };
  const uint16_t* a16 = static_cast<const uint16_t*>(a);
  CT* ct = static_cast<CT*>(c);
  const long long want = device_cu_count();
  if (rows > kStreamRows * S) {
    // tiles of `tr` rows to expect, the slots' last ones half full
    auto tiles = [&](int tr) {
      return ((long long)rows / tr + (S + 1) / 2) * ceil_div(N, kTileWeights / M);
    };
    auto split = [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      mxfp4_split_kernel<OP, GATHER, CT, NT, NT == 1 ? 2 : 4>
          <<<tile_grid(32 * NT, 512), 512, 0, stream>>>(a16, offsets, sorted_pairs, topk, S,
                                                     max_rows, w, w_scale, N, Kd, ct);
    };
    if (rows <= kSplitRows1 * S || tiles(32) <= (M == 2 ? want : 2 * want)) {
      split(integral_constant<int, 1>{});
      return;
    }
    if constexpr (M == 2) {
      if ((rows <= kSplitRows2 * S && Kd > 2560) || tiles(64) <= want) {
        split(integral_constant<int, 2>{});
        return;
      }
    }
    mxfp4_tile_kernel<OP, GATHER, CT><<<tile_grid(kTileRows, 256), 256, 0, stream>>>(
        a16, offsets, sorted_pairs, topk, S, max_rows, w, w_scale, N, Kd, ct);
    return;
  }
  const int lines = max_rows < S ? max_rows : S;  // slots that can have rows
  auto go = [&](auto wk, auto rb, auto run, auto pipe) {
    constexpr int WK = decltype(wk)::value, RB = decltype(rb)::value;
    const size_t rows_lds = (size_t)RB * stream_row_vecs(stream_window(Kd, RB, WK)) * 16;
    const size_t red_lds = WK > 1 ? (size_t)kStreamWaves * M * kWave * 16 : 0;
    mxfp4_stream_kernel<OP, GATHER, CT, WK, RB, decltype(run)::value, decltype(pipe)::value>
        <<<dim3(ceil_div(N, 16 * kStreamWaves / WK), lines), 64 * kStreamWaves,
           rows_lds > red_lds ? rows_lds : red_lds, stream>>>(
            a16, offsets, sorted_pairs, topk, S, max_rows, max_rows < S, w, w_scale, N, Kd, ct,
            PairRouting{});
  };
  // The contraction is split among waves where the columns alone leave the
  // chip without a block for every compute unit, and where it is short: up to 1024
  // a wave's part is one step, and many light blocks beat few that walk two
  // steps (S = 64, N = 4096, Kd = 1024: 32 against 36 us).
  int split = Kd <= 512 || Kd > 1024 ? 1 : 2;
  while (split < kStreamWaves && split * 512 < Kd &&
         (long long)ceil_div(N, 16 * kStreamWaves / split) * lines < want)
    split *= 2;
  using i1 = integral_constant<int, 1>;
  using i2 = integral_constant<int, 2>;
  using i4 = integral_constant<int, 4>;
  using i8 = integral_constant<int, 8>;
  // Short blocks (mxfp4_quick_kernel), us against the streaming kernel's at
  // rows drawn evenly over the slots. Gate/up: up to two rows a slot (past that
  // the codes come twice: 81 at 4), where three quarters of the steps hold k's
  // (Kd = 4096 66 : 77, 2048 36 : 46; but 2560 49 : 40, 1536 25 : 19) and the
  // other's blocks are more than one round (64 x 4 blocks, Kd = 2048: 19 : 15).
  // Down, one step or two: up to 1.5 rows (Kd = 1024 26 : 27 and 512 8.0 : 9.2 at one
  // row, 35 : 34 and 10.5 : 10.4 at two; Kd = 1536 152 : 123).
  const long long blocks = (long long)ceil_div(N, 16 * kStreamWaves) * lines;
  const bool one_round = split == 1 && blocks <= want;
  const int steps = Kd <= 2048 ? 2048 : 4096;  // k's of the gate/up form's 4 or 8 steps
  if (lines >= 16 &&
      (M == 2 ? Kd <= 4096 && 4 * Kd > 3 * steps && rows <= 2 * S && !one_round
              : Kd <= 1024 && 2 * rows <= 3 * S)) {
    auto quick = [&](auto wk) {
      constexpr int WK = decltype(wk)::value;
      mxfp4_quick_kernel<OP, GATHER, CT, WK>
          <<<dim3(ceil_div(N, 16 * kStreamWaves / WK), lines), 64 * kStreamWaves, 0, stream>>>(
              a16, offsets, sorted_pairs, topk, S, max_rows, max_rows < S, w, w_scale, N, Kd, ct);
    };
    if constexpr (M == 2) {
      if (Kd <= 2048)
        quick(i4{});
      else
        quick(i8{});
    } else {
      if (Kd <= 512)
        quick(i1{});
      else
        quick(i2{});
    }
    return;
  }
  auto pick = [&](auto rb) {
    // one window, and of it one step of 512 a wave
    const int window = stream_window(Kd, decltype(rb)::value, split);
    const bool one = window >= Kd && window <= 512 * split;
    if constexpr (decltype(rb)::value == 8) {  // 4096 k's or more
      if (one)
        go(i8{}, rb, i4{}, std::false_type{});
      else if (split > 1)
        go(i8{}, rb, i2{}, std::true_type{});
      else  // 512 a step: one block a compute unit (164 registers), 60 against 66 us
        go(i1{}, rb, i4{}, std::true_type{});
    } else if (one) {
      if (split == 1)
        go(i1{}, rb, i4{}, std::false_type{});
      else if (split == 2)
        go(i2{}, rb, i4{}, std::false_type{});
      else  // 4: eight waves split more than 2048 k's, of which 16 rows are two windows
        go(i4{}, rb, i4{}, std::false_type{});
    } else if (split > 1) {
      go(i8{}, rb, i2{}, std::true_type{});
    } else if constexpr (M == 1) {
      go(i1{}, rb, i4{}, std::true_type{});
    } else {  // 256 a step, two blocks of gate/up: 15.5 against 16.6 us (N = 512, Kd = 2048)
      go(i1{}, rb, i2{}, std::true_type{});
    }
  };
  // Rows at a time: 16, so that few slots read their codes twice (at 4 rows a
  // slot on the average 16 us against 26, S = 64, N = 512, Kd = 2048), but 8 where
  // they fill the rows' LDS by themselves (Kd = 4096: 80 against 99 us at 3, 94
  // and 94 at 6).
  if constexpr (M == 2) {
    if (Kd >= 4096 && rows <= 4 * S) {
      pick(i8{});
      return;
    }
  }
  pick(integral_constant<int, 16>{});
}

}  // namespace

moe_status_t launch_quantize_mxfp4(const void* w, bool bf16, int64_t n, uint8_t* codes,
                                   uint8_t* scale, hipStream_t stream) {
  if (n == 0) return MOE_OK;
  const int64_t n8 = n / 8;
  const dim3 blocks = folded((n8 + 255) / 256, 256);
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  if (bf16)
    quantize_mxfp4_kernel<uint16_t>
        <<<blocks, 256, 0, stream>>>(static_cast<const uint16_t*>(w), n8, c, scale);
  else
    quantize_mxfp4_kernel<float>
        <<<blocks, 256, 0, stream>>>(static_cast<const float*>(w), n8, c, scale);
  return launch_status();
}

moe_status_t launch_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scale, int64_t n,
                                     void* w, bool bf16, hipStream_t stream) {
  if (n == 0) return MOE_OK;
  const int64_t n8 = n / 8;
  const dim3 blocks = folded((n8 + 255) / 256, 256);
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  if (bf16)
    dequantize_mxfp4_kernel<uint16_t>
        <<<blocks, 256, 0, stream>>>(c, scale, n8, static_cast<uint16_t*>(w));
  else
    dequantize_mxfp4_kernel<float>
        <<<blocks, 256, 0, stream>>>(c, scale, n8, static_cast<float*>(w));
  return launch_status();
}

moe_status_t launch_gemm_mxfp4(moe_gemm_op_t op, const void* a, const int32_t* sorted_pairs,
                               int topk, const int32_t* offsets, int S, int max_rows, int rows,
                               const uint8_t* w, const uint8_t* w_scale, int H, int I, void* c,
                               bool c_f32, hipStream_t stream) {
  if (max_rows == 0) return MOE_OK;
  if (op == MOE_GEMM_GATE_UP_SWIGLU) {
    if (sorted_pairs != nullptr)
      launch_product<MOE_GEMM_GATE_UP_SWIGLU, true, uint16_t>(
          a, offsets, sorted_pairs, topk, S, max_rows, rows, w, w_scale, I, H, c, stream);
    else
      launch_product<MOE_GEMM_GATE_UP_SWIGLU, false, uint16_t>(
          a, offsets, nullptr, 1, S, max_rows, rows, w, w_scale, I, H, c, stream);
  } else if (c_f32) {
    launch_product<MOE_GEMM_DOWN, false, float>(a, offsets, nullptr, 1, S, max_rows, rows, w,
                                                w_scale, H, I, c, stream);
  } else {
    launch_product<MOE_GEMM_DOWN, false, uint16_t>(a, offsets, nullptr, 1, S, max_rows, rows, w,
                                                   w_scale, H, I, c, stream);
  }
  return launch_status();
}

moe_status_t launch_mxfp4_pairs_gate_up(const void* x, const PairRouting& routing, int T,
                                        int topk, const uint8_t* w_gate_up,
                                        const uint8_t* gate_up_scale, int H, int I, void* act,
                                        hipStream_t stream) {
  using std::integral_constant;
  const int P = T * topk;
  const int S = routing.map.S;
  uint16_t* act16 = static_cast<uint16_t*>(act);
  auto gate_up = [&](auto wk, auto pipe) {
    constexpr int WK = decltype(wk)::value, RB = 8;
    static_assert(mxfp4_pair_columns(WK == 8 ? 4096 : 2048) == 16 * kStreamWaves / WK,
                  "columns of a block");
    constexpr int RUN = decltype(pipe)::value ? 2 : 4;
    const size_t rows_lds = (size_t)stream_row_vecs(stream_window(H, RB, WK)) * 16;  // one row
    const size_t red_lds = WK > 1 ? (size_t)kStreamWaves * 2 * kWave * 16 : 0;
    mxfp4_stream_kernel<MOE_GEMM_GATE_UP_SWIGLU, true, uint16_t, WK, RB, RUN,
                        decltype(pipe)::value, true>
        <<<dim3(ceil_div(I, mxfp4_pair_columns(H)), P), 64 * kStreamWaves,
           rows_lds > red_lds ? rows_lds : red_lds, stream>>>(
            static_cast<const uint16_t*>(x), nullptr, nullptr, topk, S, P, 0, w_gate_up,
            gate_up_scale, I, H, act16, routing);
  };
  if (H > 4096)
    gate_up(integral_constant<int, 8>{}, std::true_type{});
  else if (H > 2048)
    gate_up(integral_constant<int, 8>{}, std::false_type{});
  else
    gate_up(integral_constant<int, 4>{}, std::false_type{});
  return launch_status();
}

moe_status_t launch_mxfp4_pairs_down(const void* act, const MapOut& map, int T, int topk,
                                     const uint8_t* w_down, const uint8_t* down_scale, int H,
                                     int I, void* out, bool out_bf16, int accumulate,
                                     const void* shared, hipStream_t stream) {
  auto down = [&](auto o) {
    using OT = decltype(o);
    mxfp4_pair_down_kernel<OT><<<dim3(H / 16, T), 512, 0, stream>>>(
        static_cast<const uint16_t*>(act), map.slot, map.mask, map.w_masked, topk, map.S, w_down,
        down_scale, H, I, static_cast<OT*>(out), accumulate,
        static_cast<const uint16_t*>(shared));
  };
  if (out_bf16)
    down(uint16_t{});
  else
    down(float{});
  return launch_status();
}

}  // namespace moe
