// Gradients of the grouped products in bf16 on the matrix cores.
//
//   rows:     da[r, :]  = dc[r, :] W_s            (W_s [Kd, N] as stored)
//             with h = [g, u] (the SwiGLU's input, [rows, 2N]):
//             dh = [da u s(g) (1 + g (1 - s(g))), da g s(g)],  s = sigmoid
//   weights:  dW_s[m, n] = sum over the slot's rows r of dc[r, m] a[r, n]
//
// Both contract an operand along the dimension in which it is not contiguous:
// the rows' gradient the weights, the weights' gradient both. The tiles of
// such operands lie in LDS as they do in memory, 64 rows of the contraction by
// 256 columns, and reach the matrix cores through transposing LDS reads
// (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 columns, each lane gets the
// 4 rows of its column).
#include "grouped_tiles.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef int int32x4_t __attribute__((ext_vector_type(4)));
typedef int int32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kTile = kGradTileBf16;  // rows and columns of an output tile
constexpr int kSlice = 64;        // of the contraction at a time
constexpr int kThreads = 512;     // 8 waves, 2 x 4 of 128 x 64
constexpr int kPartVec = kTile * kSlice / 8;  // 16-byte vectors of one operand's slice (32 KB)
constexpr uint32_t kOOB = 0x80000000u;        // past every resource here
constexpr int kXcdItems = 32, kGroupCols = 4;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           0x00020000);
}

// LDS place, in vectors, of 16-byte chunk ch of row r: of a tile whose rows are
// 64 contracted values (128 bytes), and of one whose rows are 256 columns (512
// bytes). Both spread the reads of a half wave over all banks.
__device__ __forceinline__ int swz_k(int r, int ch) { return r * 8 + (ch ^ ((r >> 1) & 7)); }
__device__ __forceinline__ int swz_t(int r, int ch) { return r * 32 + (ch ^ ((r & 3) << 2)); }

// 8 contracted values of this lane's column from a tile of the second kind;
// `at` is the byte offset of the first four, the others lie 4 rows below.
__device__ __forceinline__ bf16x8_t read_tr(const uint4* part, int at) {
  typedef short s16x8_t __attribute__((ext_vector_type(8)));
  typedef __attribute__((address_space(3))) s16x4_t* lds_s16x4_t;
  typedef __attribute__((address_space(3))) char* lds_char_t;
  const lds_char_t p = (lds_char_t)(lds_ptr_t)const_cast<uint4*>(part) + at;
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)p);
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)(p + 4 * 512));
  return __builtin_bit_cast(bf16x8_t,
                            (s16x8_t)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ bf16x8_t read_k(const uint4* part, int at) {
  return *reinterpret_cast<const bf16x8_t*>(reinterpret_cast<const char*>(part) + at);
}

// Two runs of 4 consecutive columns a lane (accumulator groups g and g + 1 of
// the lane halves) become 8 consecutive columns: group g for lanes 0..31,
// g + 1 for the others.
__device__ __forceinline__ void join8(const float* lo, const float* hi, float* o) {
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(lo[v]), __float_as_uint(hi[v]),
                                                    false, false);
    o[v] = __uint_as_float(s[0]);
    o[4 + v] = __uint_as_float(s[1]);
  }
}

__device__ __forceinline__ int32x4_t pack8(const float* o) {
  return int32x4_t{(int)pack_bf16x2(o[0], o[1]), (int)pack_bf16x2(o[2], o[3]),
                   (int)pack_bf16x2(o[4], o[5]), (int)pack_bf16x2(o[6], o[7])};
}

__device__ __forceinline__ void unpack8(int32x4_t q, float* o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = bf16_to_f32((uint32_t)q[i] & 0xffffu);
    o[2 * i + 1] = bf16_to_f32((uint32_t)q[i] >> 16);
  }
}

enum Kind {
  kRows = 0,        // da [rows, N]
  kRowsSwiglu = 1,  // dh [rows, 2N] from h
  kWeights = 2,     // dW [S, M, N] bf16
  kWeightsF32 = 3,  // dW [S, M, N] f32
};

struct Args {
  const uint16_t* m_side;  // dc [rows, Kd], or dc [rows, M]
  const uint16_t* n_side;  // w [S, Kd, N], or a [rows, N]
  const int32_t* offsets;
  int S, max_rows, M, N, Kd;  // Kd: rows' gradient; M: weights'
  const uint16_t* h;
  void* out;
  int accumulate, splits;  // weights'; splits > 1: out is [splits, S, M, N]
};

// A persistent block takes items (output tiles) in turn. LDS holds two slices
// of both operands, each in an array of its own, so that the compiler sees
// that the reads of one do not wait for the copies into the other.
template <int KIND>
__global__ __launch_bounds__(kThreads, 1) void grouped_grad_kernel(Args p) {
  constexpr bool WEIGHTS = KIND >= kWeights;
  __shared__ uint4 stage0[2 * kPartVec], stage1[2 * kPartVec];
  __shared__ int32_t tp[WEIGHTS ? 1 : MOE_MAX_SLOTS + 1];
  __shared__ int32_t scratch[WEIGHTS ? 1 : kThreads];
  const int lane = lane_id();
  const int wave = uniform_i32(threadIdx.x / kWave);
  const int wm = wave >> 2, wn = wave & 3;

  const int NT = ceil_div(p.N, kTile);
  const int MT = WEIGHTS ? ceil_div(p.M, kTile) : 0;
  int RT = 0;
  if constexpr (!WEIGHTS) {
    tile_prefix<kThreads, kTile>(p.offsets, p.S, p.max_rows, tp, scratch);
    RT = uniform_i32(tp[p.S]);
  }
  const int GN = NT < kGroupCols ? NT : kGroupCols;
  const int GM = kXcdItems / GN;
  const int total = WEIGHTS ? p.S * p.splits * MT * NT : RT * NT;  // the host keeps it in 31 bits

  // Byte offsets of this lane's fragments in a stage.
  int m_at[4], n_at[2];  // M side: 32 rows i; N side: 32 columns j
  const int tr_row = (lane >> 5) * 8 + ((lane & 15) >> 2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (WEIGHTS) {
      const int ch = wm * 16 + i * 4 + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
      m_at[i] = swz_t(tr_row, ch) * 16 + (lane & 1) * 8;
    } else {  // i: the chunk of contracted block kb; rows 32 further lie 4 KB further
      m_at[i] = swz_k(wm * 128 + (lane & 31), 2 * i + (lane >> 5)) * 16;
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int ch = wn * 8 + j * 4 + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
    n_at[j] = swz_t(tr_row, ch) * 16 + (lane & 1) * 8;
  }

  for (int item = first_item(blockIdx.x, gridDim.x); item < total; item += gridDim.x) {
    // the tile: its slot, output rows and columns, and what is contracted
    int s, m0, n0, rows, row0, nd, split = 0;
    if constexpr (WEIGHTS) {
      const int z = item / (MT * NT);
      int mt, nt;
      item_tile(item - z * MT * NT, MT, NT, GM, GN, &mt, &nt);
      s = z / p.splits;
      split = z - s * p.splits;
      int lo, hi;
      slot_rows(p.offsets, s, p.max_rows, &lo, &hi);
      const int whole = ceil_div(hi - lo, kSlice);
      const int each = ceil_div(whole, p.splits) * kSlice;  // rows of a split
      row0 = uniform_i32(min(lo + split * each, hi));
      rows = uniform_i32(min(hi - row0, each));
      nd = ceil_div(rows, kSlice);
      m0 = mt * kTile;
      n0 = nt * kTile;
    } else {
      int rt, nt;
      item_tile(item, RT, NT, GM, GN, &rt, &nt);
      s = uniform_i32(tile_slot(tp, p.S, rt));
      int lo, hi;
      slot_rows(p.offsets, s, p.max_rows, &lo, &hi);
      row0 = uniform_i32(lo + (rt - tp[s]) * kTile);
      rows = uniform_i32(min(kTile, hi - row0));
      nd = ceil_div(p.Kd, kSlice);
      m0 = 0;
      n0 = nt * kTile;
    }
    const uint32_t m_row = (uint32_t)(WEIGHTS ? p.M : p.Kd) * 2u, n_row = (uint32_t)p.N * 2u;

    // offsets of the lane's chunks in a slice
    uint32_t m_off[4], n_off[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = wave * 4 + i;  // KB of the part
      const int r = q * 2 + (lane >> 5);
      const int c = (lane & 31) ^ ((r & 3) << 2);
      n_off[i] = n0 + c * 8 < p.N ? (uint32_t)r * n_row + (uint32_t)(n0 + c * 8) * 2u : kOOB;
      if constexpr (WEIGHTS) {
        m_off[i] = m0 + c * 8 < p.M ? (uint32_t)r * m_row + (uint32_t)(m0 + c * 8) * 2u : kOOB;
      } else {
        const int rr = q * 8 + (lane >> 3);
        const int ch = (lane & 7) ^ ((rr >> 1) & 7);
        m_off[i] = (uint32_t)rr * m_row + (uint32_t)ch * 16u;
      }
    }

    auto fetch = [&](uint4* stage, int d) {
      if constexpr (WEIGHTS) {
        const int left = rows - d * kSlice < kSlice ? rows - d * kSlice : kSlice;
        const size_t r = (size_t)row0 + (size_t)d * kSlice;
        const __amdgpu_buffer_rsrc_t rm = make_rsrc(p.m_side + r * p.M, (uint32_t)left * m_row);
        const __amdgpu_buffer_rsrc_t rn = make_rsrc(p.n_side + r * p.N, (uint32_t)left * n_row);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(rm, (lds_ptr_t)(stage + (wave * 4 + i) * 64), 16,
                                                   m_off[i], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              rn, (lds_ptr_t)(stage + kPartVec + (wave * 4 + i) * 64), 16, n_off[i], 0, 0, 0);
      } else {
        const __amdgpu_buffer_rsrc_t rm =
            make_rsrc(p.m_side + (size_t)row0 * p.Kd, (uint32_t)rows * m_row);
        const __amdgpu_buffer_rsrc_t rn =
            make_rsrc(p.n_side + (size_t)s * p.Kd * p.N, (uint32_t)p.Kd * n_row);
        const bool tail = (d + 1) * kSlice > p.Kd;  // the chunks past Kd belong to the next row
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = (wave * 4 + i) * 8 + (lane >> 3);
          const int ch = (lane & 7) ^ ((rr >> 1) & 7);
          const uint32_t o = m_off[i] + (uint32_t)d * (kSlice * 2);
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              rm, (lds_ptr_t)(stage + (wave * 4 + i) * 64), 16,
              tail && d * kSlice + ch * 8 >= p.Kd ? kOOB : o, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(
              rn, (lds_ptr_t)(stage + kPartVec + (wave * 4 + i) * 64), 16,
              n_off[i] == kOOB ? kOOB : n_off[i] + (uint32_t)d * kSlice * n_row, 0, 0, 0);
      }
    };

    floatx16 acc[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = floatx16{};

    // a wave whose part of the tile is empty only copies
    const bool live = WEIGHTS ? m0 + wm * 128 < p.M && n0 + wn * 64 < p.N
                              : wm * 128 < rows && n0 + wn * 64 < p.N;
    auto compute = [&](const uint4* stage) {
      if (!live) return;
#pragma unroll
      for (int kb = 0; kb < kSlice / 16; ++kb) {
        bf16x8_t fm[4], fn[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (WEIGHTS) fm[i] = read_tr(stage, m_at[i] + kb * (16 * 512));
          else fm[i] = read_k(stage, m_at[kb] + i * 4096);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) fn[j] = read_tr(stage + kPartVec, n_at[j] + kb * (16 * 512));
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fn[j], fm[i], acc[j][i], 0, 0, 0);
      }
    };
    // this wave's copies are done; with the barrier everyone's are, and nobody
    // reads the other stage
    auto arrive = [&]() {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
    };

    __syncthreads();  // the previous item's reads are done
    if (nd > 0) fetch(stage0, 0);
    for (int d = 0; d < nd; d += 2) {
      arrive();
      if (d + 1 < nd) fetch(stage1, d + 1);
      compute(stage0);
      if (d + 1 >= nd) break;
      arrive();
      if (d + 2 < nd) fetch(stage0, d + 2);
      compute(stage1);
    }
    if (!live) continue;

    // register v of acc[j][i]: column 8 (v / 4) + 4 (lane / 32) + v % 4 of the 32
    // of j, row lane % 32 of the 32 of i
    const int ch8 = 8 * (lane >> 5);
    if constexpr (KIND == kRows || KIND == kRowsSwiglu) {
      const uint32_t cols = KIND == kRowsSwiglu ? 2u * (uint32_t)p.N : (uint32_t)p.N;
      const uint32_t bytes = (uint32_t)rows * cols * 2u;
      const __amdgpu_buffer_rsrc_t rc =
          make_rsrc(static_cast<uint16_t*>(p.out) + (size_t)row0 * cols, bytes);
      const __amdgpu_buffer_rsrc_t rh =
          make_rsrc(KIND == kRowsSwiglu ? p.h + (size_t)row0 * cols : nullptr,
                    KIND == kRowsSwiglu ? bytes : 0u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t r = (uint32_t)(wm * 128 + i * 32 + (lane & 31));
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int g = 0; g < 4; g += 2) {
            const int col = n0 + wn * 64 + j * 32 + 8 * g + ch8;
            float lo[4], hi[4], o[8];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              lo[v] = acc[j][i][4 * g + v];
              hi[v] = acc[j][i][4 * g + 4 + v];
            }
            join8(lo, hi, o);
            const uint32_t at = col < p.N ? (r * cols + (uint32_t)col) * 2u : kOOB;
            if constexpr (KIND == kRows) {
              __builtin_amdgcn_raw_buffer_store_b128(pack8(o), rc, at, 0, 0);
            } else {
              const uint32_t up = col < p.N ? at + (uint32_t)p.N * 2u : kOOB;
              float gt[8], u[8];
              unpack8(__builtin_amdgcn_raw_buffer_load_b128(rh, at, 0, 0), gt);
              unpack8(__builtin_amdgcn_raw_buffer_load_b128(rh, up, 0, 0), u);
#pragma unroll
              for (int v = 0; v < 8; ++v) {
                const float sg = 1.0f / (1.0f + __expf(-gt[v]));
                const float silu = gt[v] * sg;
                gt[v] = o[v] * u[v] * (sg + silu * (1.0f - sg));
                u[v] = o[v] * silu;
              }
              __builtin_amdgcn_raw_buffer_store_b128(pack8(gt), rc, at, 0, 0);
              __builtin_amdgcn_raw_buffer_store_b128(pack8(u), rc, up, 0, 0);
            }
          }
      }
    } else {
      constexpr uint32_t OB = KIND == kWeightsF32 ? 4u : 2u;
      const size_t first = (((size_t)split * p.S + s) * p.M + m0) * p.N;
      const int high = p.M - m0 < kTile ? p.M - m0 : kTile;
      const __amdgpu_buffer_rsrc_t rc = make_rsrc(static_cast<char*>(p.out) + first * OB,
                                                  (uint32_t)high * (uint32_t)p.N * OB);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t r = (uint32_t)(wm * 128 + i * 32 + (lane & 31));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if constexpr (KIND == kWeightsF32) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const int col = n0 + wn * 64 + j * 32 + 8 * g + 4 * (lane >> 5);
              const uint32_t at = col < p.N ? (r * (uint32_t)p.N + (uint32_t)col) * 4u : kOOB;
              int32x4_t o;
              if (p.accumulate) {
                const int32x4_t prev = __builtin_amdgcn_raw_buffer_load_b128(rc, at, 0, 0);
#pragma unroll
                for (int v = 0; v < 4; ++v)
                  o[v] = __float_as_int(__int_as_float(prev[v]) + acc[j][i][4 * g + v]);
              } else {
#pragma unroll
                for (int v = 0; v < 4; ++v) o[v] = __float_as_int(acc[j][i][4 * g + v]);
              }
              __builtin_amdgcn_raw_buffer_store_b128(o, rc, at, 0, 0);
            }
          } else {
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
              const int col = n0 + wn * 64 + j * 32 + 8 * g + ch8;
              const uint32_t at = col < p.N ? (r * (uint32_t)p.N + (uint32_t)col) * 2u : kOOB;
              float lo[4], hi[4], o[8];
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                lo[v] = acc[j][i][4 * g + v];
                hi[v] = acc[j][i][4 * g + 4 + v];
              }
              join8(lo, hi, o);
              if (p.accumulate) {
                float prev[8];
                unpack8(__builtin_amdgcn_raw_buffer_load_b128(rc, at, 0, 0), prev);
#pragma unroll
                for (int v = 0; v < 8; ++v) o[v] = prev[v] + o[v];
              }
              __builtin_amdgcn_raw_buffer_store_b128(pack8(o), rc, at, 0, 0);
            }
          }
        }
      }
    }
  }
}

}  // namespace

int grad_splits(int S, int max_rows, int M, int N, int tile) {
  const int64_t tiles = (int64_t)S * ceil_div(M, tile) * ceil_div(N, tile);
  const int64_t want = (2 * kSplitBlocks + tiles - 1) / tiles;  // two rounds of the chip
  const int64_t most = max_rows / ((int64_t)S * 512);          // 512 rows each
  const int64_t n = want < most ? want : most;
  return tiles >= kSplitBlocks || n < 2 ? 1 : n > kMaxSplits ? kMaxSplits : (int)n;
}

moe_status_t launch_gemm_backward_bf16(const void* dc, const int32_t* offsets, int S, int max_rows,
                                       const void* w, int Kd, int N, const void* h, void* out,
                                       hipStream_t stream) {
  Args p{};
  p.m_side = static_cast<const uint16_t*>(dc);
  p.n_side = static_cast<const uint16_t*>(w);
  p.offsets = offsets;
  p.S = S; p.max_rows = max_rows; p.N = N; p.Kd = Kd; p.splits = 1;
  p.h = static_cast<const uint16_t*>(h);
  p.out = out;
  const int64_t items = (int64_t)(max_rows / kTile + 1 + (S < max_rows ? S : max_rows)) * ceil_div(N, kTile);
  const int cus = device_cu_count();
  const int G = items < cus ? (int)items : cus;
  if (h != nullptr)
    grouped_grad_kernel<kRowsSwiglu><<<G, kThreads, 0, stream>>>(p);
  else
    grouped_grad_kernel<kRows><<<G, kThreads, 0, stream>>>(p);
  return launch_status();
}

moe_status_t launch_gemm_weight_grad_bf16(const void* dc, const void* a, const int32_t* offsets,
                                          int S, int max_rows, int M, int N, void* dw, bool dw_f32,
                                          int accumulate, void* ws, hipStream_t stream) {
  Args p{};
  p.m_side = static_cast<const uint16_t*>(dc);
  p.n_side = static_cast<const uint16_t*>(a);
  p.offsets = offsets;
  p.S = S; p.max_rows = max_rows; p.M = M; p.N = N;
  p.splits = grad_splits(S, max_rows, M, N, kTile);
  p.out = p.splits > 1 ? ws : dw;
  p.accumulate = p.splits > 1 ? 0 : accumulate;
  const int64_t items = (int64_t)S * p.splits * ceil_div(M, kTile) * ceil_div(N, kTile);
  const int cus = device_cu_count();
  const int G = items < cus ? (int)items : cus;
  if (dw_f32 || p.splits > 1)
    grouped_grad_kernel<kWeightsF32><<<G, kThreads, 0, stream>>>(p);
  else
    grouped_grad_kernel<kWeights><<<G, kThreads, 0, stream>>>(p);
  if (p.splits > 1)
    return launch_fold_splits(static_cast<const float*>(ws), p.splits, (size_t)S * M * N, dw, dw_f32,
                              accumulate, stream);
  return launch_status();
}

}  // namespace moe
