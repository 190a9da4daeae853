// Expert weights in 4 bits: quantisation to E2M1 codes with one E8M0 scale
// for 32 weights, its inverse, and the grouped products that read them.
//
// Format: code s ee m, value (-1)^s {0, 0.5, 1, 1.5, 2, 3, 4, 6}; two codes
// a byte, the even index in the low four bits; scale byte b = 2^(b - 127),
// 255 = NaN. A code times its scale is a bfloat16 number (two significant
// bits), so the products run on the bf16 matrix cores without any rounding
// of the weights: gfx950 converts two codes and applies the scale in one
// instruction (v_cvt_scalef32_pk_bf16_fp4).
#include "common.h"
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


// Four lanes a group, 8 values each. b = floor(log2 amax) - 2 + 127 puts the
// largest magnitude into [4, 8): above 6 it saturates. The exponent is read
// from amax's bits (a subnormal amax gives b = 0). A group with a non-finite
// value gets the NaN scale.
template <typename XT>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(const XT* __restrict__ w, int64_t n8,
                                                             uint32_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scale) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
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
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
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

// ---------------------------------------------------------------- products
// One block per (16 output columns, slot): its four waves split the
// contraction into chunks of 128 (wave w takes chunks w, w + 4, ...), hold
// 16 x 16 sums for 16 weight rows and 16 token rows, and add up in LDS in
// wave order. v_mfma_f32_16x16x32_bf16 with the weights as the first operand:
// lane l supplies weight row l mod 16 and token row l mod 16, the k's
// 32 (l / 16) .. + 31 of the chunk in four steps of 8, so a lane's codes are
// 16 consecutive bytes under one scale. Register r of lane l then holds
// column 4 (l / 16) + r of token row l mod 16.
constexpr int kProdWaves = 4;

template <int OP, bool GATHER, typename CT>
__global__ __launch_bounds__(256) void mxfp4_product_kernel(
    const uint16_t* __restrict__ a, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ sorted_pairs, int topk, int max_rows,
    const uint8_t* __restrict__ w, const uint8_t* __restrict__ w_scale, int N, int Kd,
    CT* __restrict__ c) {
  constexpr int M = OP == MOE_GEMM_GATE_UP_SWIGLU ? 2 : 1;  // matrices (gate and up, or down)
  __shared__ floatx4 red[kProdWaves][M][kWave];
  const int s = blockIdx.y;
  const int r0 = offsets[s];
  const int r1 = min(offsets[s + 1], max_rows);
  if (r0 >= r1) return;
  const int n0 = blockIdx.x * 16;
  const int lane = lane_id();
  const int wave = threadIdx.x / kWave;
  const int m = lane & 15, g = lane >> 4;
  const int n = min(n0 + m, N - 1);
  const size_t rows_s = (size_t)s * M * N;
  for (int rt = r0; rt < r1; rt += 16) {
    int row = min(rt + m, r1 - 1);
    if constexpr (GATHER) row = sorted_pairs[row] / topk;
    const uint16_t* arow = a + (size_t)row * Kd;
    floatx4 acc[M];
#pragma unroll
    for (int i = 0; i < M; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int k0 = wave * 128; k0 < Kd; k0 += kProdWaves * 128) {
      const int k = k0 + 32 * g;
      const bool in = k < Kd;  // Kd is a multiple of 32
      uint4 b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[j] = in ? *reinterpret_cast<const uint4*>(arow + k + 8 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < M; ++i) {
        const size_t wr = rows_s + (size_t)i * N + n;
        uint4 q = make_uint4(0, 0, 0, 0);
        float sc = 1.0f;
        if (in) {
          q = *reinterpret_cast<const uint4*>(w + (wr * Kd + k) / 2);
          sc = e8m0(w_scale[(wr * Kd + k) / 32]);
        }
        const uint32_t qq[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8_t, cvt8(qq[j], sc)), __builtin_bit_cast(bf16x8_t, b[j]),
              acc[i], 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < M; ++i) red[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int i = 0; i < M; ++i)
        for (int v = 1; v < kProdWaves; ++v) acc[i] += red[v][i][lane];
      if (rt + m < r1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int col = n0 + 4 * g + r;
          if (col >= N) continue;
          float v = acc[0][r];
          if constexpr (M == 2) v = v / (1.0f + expf(-v)) * acc[1][r];
          CT* o = c + (size_t)(rt + m) * N + col;
          if constexpr (sizeof(CT) == 2)
            *o = (CT)(pack_bf16x2(v, 0.f) & 0xffffu);
          else
            *o = v;
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- products, many rows
// One block per (128 token rows of a slot, 256 weight rows): the same 128
// gate and up rows, or 256 rows of down. Four waves, each with 64 weight rows
// (gate and up of 32 columns, or 64 columns) against all 128 tokens, so a
// weight is converted once in a block and never passes through LDS; the
// tokens' rows, which all waves need, do: stages of 64 k's, two of them,
// fetched into registers while the other feeds the matrix cores
// (v_mfma_f32_32x32x16_bf16, weights first). Lane l holds weight row
// l mod 32 and the k's 32 (l / 32) .. + 31 of a stage: 16 bytes of codes
// under one scale. LDS rows are 128 bytes, their 16-byte chunks XOR-swizzled
// by (row mod 8).
constexpr int kTileRows = 128;
constexpr int kTileWeights = 256;
constexpr int kStage = 64;

typedef float floatx16 __attribute__((ext_vector_type(16)));

// Finds row tile `tile` of the slots' tiles of kTileRows rows, in slot order:
// the slot, its rows [r0, r1) in the tile; false behind the last. Every wave
// computes it for itself (a scan over 64 slots at a time).
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
    const int n = ceil_div(b - a, kTileRows);
    int incl = n;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int v = __shfl_up(incl, o, kWave);
      if (lane >= o) incl += v;
    }
    const uint64_t hit = __ballot(incl > tile);
    if (hit != 0) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int first = tile - (__builtin_amdgcn_readlane(incl, l) -
                                __builtin_amdgcn_readlane(n, l));
      *slot = s0 + l;
      *r0 = __builtin_amdgcn_readlane(a, l) + first * kTileRows;
      *r1 = min(*r0 + kTileRows, __builtin_amdgcn_readlane(b, l));
      return true;
    }
    tile -= __builtin_amdgcn_readlane(incl, kWave - 1);
  }
  return false;
}

// NT: 32-token blocks of the tile that hold rows.
template <int OP, typename CT, int NT>
__device__ __forceinline__ void tile_product(uint4 (*stage)[kTileRows * 8],
                                             const uint16_t* const (&src)[4], int r0, int rows,
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
  // 32-bit offsets into the slot's panel (below 2^31 bytes: weight_panel_ok)
  const uint32_t wp[2] = {(uint32_t)row0 * (uint32_t)(Kd / 2) + 16 * h,
                          (uint32_t)row1 * (uint32_t)(Kd / 2) + 16 * h};
  const uint32_t sp[2] = {(uint32_t)row0 * (uint32_t)(Kd / 32) + h,
                          (uint32_t)row1 * (uint32_t)(Kd / 32) + h};

  floatx16 acc[2][NT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = floatx16{};

  // thread tid fetches chunk tid % 8 of rows tid / 8 + 32 i
  const int chunk = tid & 7;
  uint4 fa[NT];
  auto fetch = [&](int k0) {
    const bool in = k0 + 8 * chunk < Kd;
#pragma unroll
    for (int i = 0; i < NT; ++i)
      fa[i] = in ? *reinterpret_cast<const uint4*>(src[i] + k0) : make_uint4(0, 0, 0, 0);
  };
  auto put = [&](int b) {
    const int r = tid >> 3;
#pragma unroll
    for (int i = 0; i < NT; ++i) stage[b][(r + 32 * i) * 8 + (chunk ^ (r & 7))] = fa[i];
  };
  uint4 q[2][2], qn[2][2];
  uint32_t sc[2][2], scn[2][2];
  auto load_codes = [&](int k0, uint4 (&qq)[2][2], uint32_t (&ss)[2][2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool in = k0 + kStage * u + 32 * h < Kd;
        qq[i][u] = make_uint4(0, 0, 0, 0);
        ss[i][u] = 127;
        if (in) {
          qq[i][u] = *reinterpret_cast<const uint4*>(w + (wp[i] + (uint32_t)(k0 + kStage * u) / 2));
          ss[i][u] = w_scale[sp[i] + (uint32_t)(k0 + kStage * u) / 32];
        }
      }
  };
  auto compute = [&](int b, int u) {
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
            bf16x8_t, stage[b][(32 * t + m) * 8 + ((4 * h + j) ^ (m & 7))]);
        acc[0][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a0, x, acc[0][t], 0, 0, 0);
        acc[1][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a1, x, acc[1][t], 0, 0, 0);
      }
    }
  };

  fetch(0);
  load_codes(0, q, sc);
  put(0);
  __syncthreads();
  for (int k0 = 0; k0 < Kd; k0 += 2 * kStage) {
    fetch(k0 + kStage);
    load_codes(k0 + 2 * kStage, qn, scn);
    compute(0, 0);
    put(1);
    __syncthreads();
    fetch(k0 + 2 * kStage);
    compute(1, 1);
    put(0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        q[i][u] = qn[i][u];
        sc[i][u] = scn[i][u];
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

// Blocks b, b + 8, ... run on one XCD (workgroups are dealt round-robin):
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
  const int in = (int)(blockIdx.x >> 3);
  const int tile = ((in / group) * 8 + (int)(blockIdx.x & 7)) * 2 + (in % group) % 2;
  const int n0 = (in % group) / 2 * (kTileWeights / M);
  int s = 0, r0 = 0, r1 = 0;
  if (!find_tile(offsets, S, max_rows, tile, &s, &r0, &r1)) return;
  const int rows = r1 - r0;
  const uint16_t* src[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int row = r0 + min((int)(threadIdx.x >> 3) + 32 * i, rows - 1);
    if constexpr (GATHER) row = sorted_pairs[row] / topk;
    src[i] = a + (size_t)row * Kd + 8 * (threadIdx.x & 7);
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
  else
    tile_product<OP, CT, 4>(stage, src, r0, rows, ws, ss, n0, N, Kd, c);
}

template <int OP, bool GATHER, typename CT>
void launch_product(const void* a, const int32_t* offsets, const int32_t* sorted_pairs, int topk,
                    int S, int max_rows, const uint8_t* w, const uint8_t* w_scale, int N, int Kd,
                    void* c, hipStream_t stream) {
  if (max_rows >= 32 * S) {
    constexpr int M = OP == MOE_GEMM_GATE_UP_SWIGLU ? 2 : 1;
    // at most this many row tiles, whatever the slots' counts
    const int64_t tiles = (int64_t)max_rows / kTileRows + S;
    const int64_t group = 2 * ceil_div(N, kTileWeights / M);
    const int64_t groups = (tiles + 15) / 16 * 8;  // groups of two row tiles, eight XCDs
    mxfp4_tile_kernel<OP, GATHER, CT><<<(unsigned)(groups * group), 256, 0, stream>>>(
        static_cast<const uint16_t*>(a), offsets, sorted_pairs, topk, S, max_rows, w, w_scale, N,
        Kd, static_cast<CT*>(c));
    return;
  }
  mxfp4_product_kernel<OP, GATHER, CT><<<dim3(ceil_div(N, 16), S), 256, 0, stream>>>(
      static_cast<const uint16_t*>(a), offsets, sorted_pairs, topk, max_rows, w, w_scale, N, Kd,
      static_cast<CT*>(c));
}

}  // namespace

moe_status_t launch_quantize_mxfp4(const void* w, bool bf16, int64_t n, uint8_t* codes,
                                   uint8_t* scale, hipStream_t stream) {
  if (n == 0) return MOE_OK;
  const int64_t n8 = n / 8;
  const unsigned blocks = (unsigned)((n8 + 255) / 256);
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
  const unsigned blocks = (unsigned)((n8 + 255) / 256);
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
                               int topk, const int32_t* offsets, int S, int max_rows,
                               const uint8_t* w, const uint8_t* w_scale, int H, int I, void* c,
                               bool c_f32, hipStream_t stream) {
  if (max_rows == 0) return MOE_OK;
  if (op == MOE_GEMM_GATE_UP_SWIGLU) {
    if (sorted_pairs != nullptr)
      launch_product<MOE_GEMM_GATE_UP_SWIGLU, true, uint16_t>(
          a, offsets, sorted_pairs, topk, S, max_rows, w, w_scale, I, H, c, stream);
    else
      launch_product<MOE_GEMM_GATE_UP_SWIGLU, false, uint16_t>(
          a, offsets, nullptr, 1, S, max_rows, w, w_scale, I, H, c, stream);
  } else if (c_f32) {
    launch_product<MOE_GEMM_DOWN, false, float>(a, offsets, nullptr, 1, S, max_rows, w, w_scale,
                                                H, I, c, stream);
  } else {
    launch_product<MOE_GEMM_DOWN, false, uint16_t>(a, offsets, nullptr, 1, S, max_rows, w,
                                                   w_scale, H, I, c, stream);
  }
  return launch_status();
}

}  // namespace moe
