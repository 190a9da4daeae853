// Gradients of the grouped products in bf16 on the matrix cores.
//
//   rows:     da[r, :]  = dc[r, :] W_s            (W_s [Kd, N] as stored)
//             with h = [g, u] (the SwiGLU's input, [rows, 2N]):
//             dh = [da u s(g) (1 + g (1 - s(g))), da g s(g)],  s = sigmoid
//   weights:  dW_s[m, n] = sum over the slot's rows r of dc[r, m] a[r, n]
//
// Both contract an operand along the dimension in which it is not contiguous:
// the rows' gradient the weights, the weights' gradient both. The tiles of
// such operands lie in LDS as they do in memory, 64 or 32 rows of the contraction
// by the tile's 256, 128 or 32 columns, and reach the matrix cores through transposing LDS reads
// (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 columns, each lane gets the
// 4 rows of its column).
#include <algorithm>

#include "grouped_tiles.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef int int32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr uint32_t kOOB = 0x80000000u;  // past every resource here
constexpr int kXcdItems = 32, kGroupCols = 4;

// An output tile: WM x WN waves of NI x NJ fragments of 32 rows by 32 columns.
// A wave's columns are consecutive. Its fragments of rows lie WM fragments
// apart, so that the rows that a slot's last tile has are shared out among the
// waves, 32 at a time. SLICE values of the contraction at a time.
template <int WM_, int NI_, int WN_, int NJ_, int SLICE>
struct Shape {
  static constexpr int kSlice = SLICE;
  static constexpr int WM = WM_, NI = NI_, WN = WN_, NJ = NJ_;
  static constexpr int kRowsM = WM * NI * 32, kColsN = WN * NJ * 32;
  static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
  static constexpr int kVecM = kRowsM * kSlice / 8, kVecN = kColsN * kSlice / 8;  // of a slice
  static constexpr int kCopiesM = kVecM / kThreads, kCopiesN = kVecN / kThreads;  // a wave, 1 KB each
  static_assert(kVecM % kThreads == 0 && kVecN % kThreads == 0, "whole copies");
};
typedef Shape<2, 4, 4, 2, 64> Large;  // 256 x 256: 64 KB a slice, one block a compute unit
typedef Shape<1, 1, 4, 2, 64> Small;  // rows' gradient, 32 x 256: 36 KB a slice, two blocks a compute unit
typedef Shape<1, 4, 4, 2, 32> Half;   // weights' gradient, 128 x 256: 24 KB a slice, two blocks a compute unit
static_assert(Large::kRowsM == kGradTileBf16 && Large::kColsN == kGradTileBf16, "the host's tile");

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           0x00020000);
}

// The same of values that every lane holds alike: said with readfirstlane, without
// which the compiler may keep them in vector registers and loop over the lanes at
// each copy (the weights' gradient of 131072 rows of 2048 x 4096 took 2.66 ms so).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = (uint32_t)uniform_i32((int)(uint32_t)a);
  const uint32_t hi = (uint32_t)uniform_i32((int)(uint32_t)(a >> 32));
  return make_rsrc(reinterpret_cast<const void*>(((uint64_t)hi << 32) | lo),
                   (uint32_t)uniform_i32((int)bytes));
}

// 16 bytes a lane from byte offset `off` to LDS, 1 KB in a row from `to`; out of
// range, zeros. (A function of its own, not a template: the host's pass drops a
// kernel's stub without a word where it looks at this size inside one.)
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t from, uint4* to, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_ptr_t)to, 16, off, 0, 0, 0);
}

// LDS place, in vectors, of 16-byte chunk ch of row r: of a tile whose rows are
// 64 contracted values (128 bytes), and of one whose rows are COLS columns.
// Both spread the reads of a half wave over all banks.
__device__ __forceinline__ int swz_k(int r, int ch) { return r * 8 + (ch ^ ((r >> 1) & 7)); }
template <int COLS>
__device__ __forceinline__ int swz_t(int r, int ch) {
  return r * (COLS / 8) + (ch ^ ((r & 3) << 2));
}

// 8 contracted values of this lane's column from a tile of the second kind;
// `at` is the byte offset of the first four, the others lie 4 rows below.
template <int COLS>
__device__ __forceinline__ bf16x8_t read_tr(const uint4* part, int at) {
  typedef short s16x8_t __attribute__((ext_vector_type(8)));
  typedef __attribute__((address_space(3))) s16x4_t* lds_s16x4_t;
  typedef __attribute__((address_space(3))) char* lds_char_t;
  const lds_char_t p = (lds_char_t)(lds_ptr_t)const_cast<uint4*>(part) + at;
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)p);
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t)(p + 4 * COLS * 2));
  return __builtin_bit_cast(bf16x8_t,
                            (s16x8_t)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ bf16x8_t read_k(const uint4* part, int at) {
  return *reinterpret_cast<const bf16x8_t*>(reinterpret_cast<const char*>(part) + at);
}

// Two runs of 4 consecutive columns a lane (accumulator groups g and g + 1 of the
// lane halves) packed to 8 consecutive columns: group g for lanes 0..31, g + 1 for
// the others.
__device__ __forceinline__ uint4 join_packed(const float* lo, const float* hi) {
  const auto a = __builtin_amdgcn_permlane32_swap(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(hi[0], hi[1]),
                                                  false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[2], hi[3]),
                                                  false, false);
  return make_uint4(a[0], b[0], a[1], b[1]);
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
  int splits;  // weights'; splits > 1: out is [splits, S, M, N]
};

// A tile: its slot, output rows and columns, and what is contracted.
template <typename SH>
struct Item {
  int s, split, m0, n0, row0, rows, nd;
  const uint16_t *m_next, *n_next;  // weights' gradient: of the next slice to ask for
  int left;                         // and the rows from there on
  uint32_t m_off[SH::kCopiesM], n_off[SH::kCopiesN];  // of the lane's chunks in a slice
};

// Waits until at most N vector memory operations of the wave are outstanding.
template <int N>
__device__ __forceinline__ void vm_wait() {
  static_assert(N < 64, "six bits of the count, in two fields");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | ((N >> 4) << 14));
}

// LDS beside the stages: the rows' gradient finds a tile's slot in a prefix; the
// weights' gradient has 4 KB a wave that its results pass through.
template <bool WEIGHTS, typename SH>
struct Beside {
  int32_t tp[MOE_MAX_SLOTS + 1];
  int32_t scratch[SH::kThreads];
};
template <typename SH>
struct Beside<true, SH> {
  uint4 out[SH::kWaves][256];
};

// A persistent block takes items (output tiles) in turn. LDS holds two slices
// of both operands, each in an array of its own, so that the compiler sees
// that the reads of one need not wait for the copies into the other. The copy
// of slice d + 1 runs while slice d is multiplied.
//
// The next item's first slices are asked for before an item's results are
// stored, and waited for by the number of younger operations outstanding (the
// completion of a wave's vector memory operations, stores among them, is reported
// in the order of their execution). The rows' gradient passes its results through its part of
// stage 1 and asks for the first slice alone, and for the second behind the
// stores; as compiled that first slice is waited for before the first result is
// written to LDS, so it does not overlap the stores, and through the SwiGLU each 8
// rows' gates and ups are read, waited for and stored in turn. The weights' gradient
// has room for its results elsewhere and asks for two slices: the first is multiplied
// while the stores drain (bf16, 64 slots of 2048 x 4096 with 512 rows each 754 -> 735
// us), before the second the compiler waits for half of them (a wait of its own, for
// tiles of fewer rows, whose paths meet there).
//
// What bounds it, at 131072 rows of 2048 x 4096 in 64 slots, f32 results (2.2
// TFLOP, 2.21 to 2.29 ms, 960 to 995 TFLOP/s): the products alone, without copies and
// stores, take 1.70 ms, the copies alone 1.57 ms (11 TB/s into LDS), both 1.93, and the
// stores add the rest: their 2.1 GB at the rate of plain writes are 0.5 ms. Rows'
// gradient of 32768 rows in 64 slots: gate/up (2048 x 4096) 575 us (956 TFLOP/s), down
// through the SwiGLU (4096 x 1024) 391 (703). Measured and not
// kept: slices of 32 values in four stages (3.2 ms), the last block's products over
// the next slice's reads and copies (2.32 to 2.40), blocks out of step with each
// other (2.36), non-temporal stores (2.43), tiles of several forms by columns too.
template <int KIND, typename SH, bool ADD = false>
__global__ __launch_bounds__(SH::kThreads, 2) void grouped_grad_kernel(Args p) {
  constexpr bool WEIGHTS = KIND >= kWeights;
  constexpr int BM = SH::kRowsM, BN = SH::kColsN, NI = SH::NI, NJ = SH::NJ;
  __shared__ uint4 stage0[SH::kVecM + SH::kVecN], stage1[SH::kVecM + SH::kVecN];
  __shared__ Beside<WEIGHTS, SH> beside;
  constexpr int kCopies = SH::kCopiesM + SH::kCopiesN;
  const int lane = lane_id();
  const int wave = uniform_i32(threadIdx.x / kWave);
  const int wm = wave / SH::WN, wn = wave % SH::WN;

  const int NT = ceil_div(p.N, BN);
  const int MT = WEIGHTS ? ceil_div(p.M, BM) : 0;
  int RT = 0;
  if constexpr (!WEIGHTS) {
    tile_prefix<SH::kThreads, BM>(p.offsets, p.S, p.max_rows, beside.tp, beside.scratch);
    RT = uniform_i32(beside.tp[p.S]);
  }
  const int GN = NT < kGroupCols ? NT : kGroupCols;
  const int GM = kXcdItems / GN;
  const int total = WEIGHTS ? p.S * p.splits * MT * NT : RT * NT;  // the host keeps it in 31 bits

  // Byte offsets of this lane's fragments in a stage.
  int m_at[4], n_at[NJ];
  const int tr_row = (lane >> 5) * 8 + ((lane & 15) >> 2);
  const int tr_ch = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (WEIGHTS)
      m_at[i] = swz_t<BM>(tr_row, (i * SH::WM + wm) * 4 + tr_ch) * 16 + (lane & 1) * 8;
    else  // i: the chunk of contracted block i of the slice; fragments of rows lie 4 KB apart
      m_at[i] = swz_k(wm * 32 + (lane & 31), 2 * i + (lane >> 5)) * 16;
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    n_at[j] = swz_t<BN>(tr_row, (wn * NJ + j) * 4 + tr_ch) * 16 + (lane & 1) * 8;

  Item<SH> it;
  const uint32_t m_row = (uint32_t)(WEIGHTS ? p.M : p.Kd) * 2u, n_row = (uint32_t)p.N * 2u;

  auto setup = [&](int item) {
    int lo, hi;
    if constexpr (WEIGHTS) {
      const int z = item / (MT * NT);
      int mt, nt;
      item_tile(item - z * MT * NT, MT, NT, GM, GN, &mt, &nt);
      it.s = z / p.splits;
      it.split = z - it.s * p.splits;
      slot_rows(p.offsets, it.s, p.max_rows, &lo, &hi);
      split_rows(lo, hi, SH::kSlice, p.splits, it.split, &it.row0, &it.rows);
      it.row0 = uniform_i32(it.row0);
      it.rows = uniform_i32(it.rows);
      it.nd = ceil_div(it.rows, SH::kSlice);
      it.m0 = mt * BM;
      it.n0 = nt * BN;
      it.m_next = p.m_side + (size_t)it.row0 * p.M;
      it.n_next = p.n_side + (size_t)it.row0 * p.N;
      it.left = it.rows;
    } else {
      int rt, nt;
      item_tile(item, RT, NT, GM, GN, &rt, &nt);
      it.s = uniform_i32(tile_slot(beside.tp, p.S, rt));
      slot_rows(p.offsets, it.s, p.max_rows, &lo, &hi);
      it.row0 = uniform_i32(lo + (rt - beside.tp[it.s]) * BM);
      it.rows = uniform_i32(min(BM, hi - it.row0));
      it.nd = ceil_div(p.Kd, SH::kSlice);
      it.m0 = 0;
      it.n0 = nt * BN;
    }
#pragma unroll
    for (int i = 0; i < SH::kCopiesM; ++i) {
      const int v = (wave * SH::kCopiesM + i) * kWave + lane;  // vector of the slice
      if constexpr (WEIGHTS) {
        const int r = v / (BM / 8), c = it.m0 + ((v % (BM / 8)) ^ ((r & 3) << 2)) * 8;
        it.m_off[i] = c < p.M ? (uint32_t)r * m_row + (uint32_t)c * 2u : kOOB;
      } else {
        const int r = v / 8, ch = (v % 8) ^ ((r >> 1) & 7);
        it.m_off[i] = (uint32_t)r * m_row + (uint32_t)ch * 16u;
      }
    }
#pragma unroll
    for (int i = 0; i < SH::kCopiesN; ++i) {
      const int v = (wave * SH::kCopiesN + i) * kWave + lane;
      const int r = v / (BN / 8), c = it.n0 + ((v % (BN / 8)) ^ ((r & 3) << 2)) * 8;
      it.n_off[i] = c < p.N ? (uint32_t)r * n_row + (uint32_t)c * 2u : kOOB;
    }
  };

  // Asks for slice d, each in turn (past the last one: for nothing, LDS gets
  // zeros). What lies outside of the tile's rows, columns and contraction
  // arrives as zeros.
  auto fetch = [&](uint4* stage, int d) {
    uint4* to_m = stage + wave * SH::kCopiesM * kWave;
    uint4* to_n = stage + SH::kVecM + wave * SH::kCopiesN * kWave;
    if constexpr (WEIGHTS) {
      const uint32_t have = (uint32_t)max(0, min(it.left, SH::kSlice));
      const __amdgpu_buffer_rsrc_t rm = uniform_rsrc(it.m_next, have * m_row);
      const __amdgpu_buffer_rsrc_t rn = uniform_rsrc(it.n_next, have * n_row);
      it.m_next += (size_t)SH::kSlice * p.M;
      it.n_next += (size_t)SH::kSlice * p.N;
      it.left -= SH::kSlice;
#pragma unroll
      for (int i = 0; i < SH::kCopiesM; ++i)
        copy16(rm, to_m + i * kWave, it.m_off[i]);
#pragma unroll
      for (int i = 0; i < SH::kCopiesN; ++i)
        copy16(rn, to_n + i * kWave, it.n_off[i]);
    } else {
      const bool live = d < it.nd;
      const __amdgpu_buffer_rsrc_t rm =
          uniform_rsrc(p.m_side + (size_t)it.row0 * p.Kd, live ? (uint32_t)it.rows * m_row : 0u);
      const __amdgpu_buffer_rsrc_t rn =
          uniform_rsrc(p.n_side + (size_t)it.s * p.Kd * p.N, live ? (uint32_t)p.Kd * n_row : 0u);
      const bool tail = (d + 1) * SH::kSlice > p.Kd;  // chunks past Kd belong to the next row
#pragma unroll
      for (int i = 0; i < SH::kCopiesM; ++i) {
        const int v = (wave * SH::kCopiesM + i) * kWave + lane;
        const int ch = (v % 8) ^ ((v / 8 >> 1) & 7);
        copy16(rm, to_m + i * kWave,
               tail && d * SH::kSlice + ch * 8 >= p.Kd ? kOOB : it.m_off[i] + (uint32_t)d * (SH::kSlice * 2));
      }
#pragma unroll
      for (int i = 0; i < SH::kCopiesN; ++i)
        copy16(rn, to_n + i * kWave,
               it.n_off[i] == kOOB ? kOOB : it.n_off[i] + (uint32_t)d * SH::kSlice * n_row);
    }
  };

  // Multiplies a slice: the wave's first ni fragments of rows.
  auto multiply = [&](const uint4* stage, auto& acc) {
    constexpr int ni = sizeof(acc[0]) / sizeof(floatx16);
#pragma unroll
    for (int kb = 0; kb < SH::kSlice / 16; ++kb) {
      bf16x8_t fm[ni], fn[NJ];
#pragma unroll
      for (int i = 0; i < ni; ++i) {
        if constexpr (WEIGHTS) fm[i] = read_tr<BM>(stage, m_at[i] + kb * (16 * BM * 2));
        else fm[i] = read_k(stage, m_at[kb] + i * (SH::WM * 4096));
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        fn[j] = read_tr<BN>(stage + SH::kVecM, n_at[j] + kb * (16 * BN * 2));
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < ni; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fn[j], fm[i], acc[j][i], 0, 0, 0);
    }
  };
  // All slices of the item, the first of which has arrived for this wave; `use`
  // multiplies the one in a stage. `behind`: stores issued since slice 1 was asked
  // for (none or those of a full tile).
  constexpr int kStores = (KIND == kWeightsF32 || KIND == kRowsSwiglu ? 8 : 4) * NI;  // of a full tile, a wave
  int behind = 0;
  auto contract = [&](auto use) {
    __syncthreads();
    use(stage0);
    for (int d = 1; d < it.nd; d += 2) {
      if (WEIGHTS && behind != 0) vm_wait<WEIGHTS ? kStores : 0>();
      else vm_wait<0>();
      behind = 0;
      __syncthreads();
      if (d + 1 < it.nd) fetch(stage0, d + 1);
      use(stage1);
      if (d + 1 >= it.nd) break;
      vm_wait<0>();
      __syncthreads();
      if (d + 2 < it.nd) fetch(stage1, d + 2);
      use(stage0);
    }
    __syncthreads();  // both stages have been read
  };

  // Stores the wave's first ni fragments of rows of tile t through LDS, so that
  // whole lines are written. Register v of acc[j][i] is column 8 (v / 4) +
  // 4 (lane / 32) + v % 4 of the 32 of j, row lane % 32 of the 32 of i.
  auto store = [&](const Item<SH>& t, auto& acc) {
    constexpr int ni = sizeof(acc[0]) / sizeof(floatx16);
    constexpr uint32_t OB = KIND == kWeightsF32 ? 4u : 2u;
    const uint32_t cols = KIND == kRowsSwiglu ? 2u * (uint32_t)p.N : (uint32_t)p.N;
    const size_t first = WEIGHTS ? (((size_t)t.split * p.S + t.s) * p.M + t.m0) * p.N
                                 : (size_t)t.row0 * cols;
    const uint32_t bytes = (uint32_t)(WEIGHTS ? min(p.M - t.m0, BM) : t.rows) * cols * OB;
    const __amdgpu_buffer_rsrc_t rc = uniform_rsrc(static_cast<char*>(p.out) + first * OB, bytes);
    if constexpr (WEIGHTS) {
      // 32 rows of 128 bytes at a time: 32 columns of f32, or 64 of bf16. What they are
      // added to is read in the same lines, two such steps ahead (bf16, 60 slots of 2816
      // x 2048 with 32 rows each: 271 us, read where it is added 454).
      uint4* out = beside.out[wave];
      auto place = [&](int r, int ch) { return out + r * 8 + (ch ^ ((r >> 1) & 7)); };
      const int r8 = lane >> 3, c8 = lane & 7;  // row and chunk of a line of 128 bytes
      constexpr int kParts = KIND == kWeights ? 1 : NJ, kCols = 128 / (int)OB;
      auto at = [&](int i, int part, int l) {
        const int col = t.n0 + wn * NJ * 32 + part * 32 + c8 * (kCols / 8);
        const uint32_t row = (uint32_t)((i * SH::WM + wm) * 32 + l + r8);
        return col < p.N ? (row * cols + (uint32_t)col) * OB : kOOB;
      };
      constexpr int kSteps = ni * kParts, kAhead = ADD ? 2 : 1;
      int32x4_t prev[kAhead][4];
      auto ask = [&](int q) {
#pragma unroll
        for (int l = 0; l < 4; ++l)
          prev[q % kAhead][l] =
              __builtin_amdgcn_raw_buffer_load_b128(rc, at(q / kParts, q % kParts, l * 8), 0, 0);
      };
      if constexpr (ADD) {
#pragma unroll
        for (int q = 0; q < kAhead && q < kSteps; ++q) ask(q);
      }
#pragma unroll
      for (int q = 0; q < kSteps; ++q) {
        const int i = q / kParts, part = q % kParts;
        if constexpr (KIND == kWeights) {
          if constexpr (ADD) {  // to the accumulators' lanes
#pragma unroll
            for (int l = 0; l < 4; ++l)
              *place(l * 8 + r8, c8) = __builtin_bit_cast(uint4, prev[q % kAhead][l]);
            wave_lds_fence();
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const uint2 v = reinterpret_cast<const uint2*>(place(lane & 31, j * 4 + g))[lane >> 5];
                acc[j][i][4 * g] = bf16_to_f32(v.x & 0xffffu) + acc[j][i][4 * g];
                acc[j][i][4 * g + 1] = bf16_to_f32(v.x >> 16) + acc[j][i][4 * g + 1];
                acc[j][i][4 * g + 2] = bf16_to_f32(v.y & 0xffffu) + acc[j][i][4 * g + 2];
                acc[j][i][4 * g + 3] = bf16_to_f32(v.y >> 16) + acc[j][i][4 * g + 3];
              }
            wave_lds_fence();
          }
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
              float lo[4], hi[4];
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                lo[v] = acc[j][i][4 * g + v];
                hi[v] = acc[j][i][4 * g + 4 + v];
              }
              *place(lane & 31, j * 4 + g + (lane >> 5)) = join_packed(lo, hi);
            }
        } else {
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *place(lane & 31, 2 * g + (lane >> 5)) = make_uint4(
                __float_as_uint(acc[part][i][4 * g]), __float_as_uint(acc[part][i][4 * g + 1]),
                __float_as_uint(acc[part][i][4 * g + 2]), __float_as_uint(acc[part][i][4 * g + 3]));
        }
        wave_lds_fence();
#pragma unroll
        for (int l = 0; l < 4; ++l) {
          int32x4_t o = __builtin_bit_cast(int32x4_t, *place(l * 8 + r8, c8));
          if constexpr (ADD && KIND == kWeightsF32) {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              o[v] = __float_as_int(__int_as_float(prev[q % kAhead][l][v]) + __int_as_float(o[v]));
          }
          __builtin_amdgcn_raw_buffer_store_b128(o, rc, at(i, part, l * 8), 0, 0);
        }
        wave_lds_fence();
        if constexpr (ADD) {
          if (q + kAhead < kSteps) ask(q + kAhead);
        }
      }
    } else {
      // 32 rows of 64 columns of f32 at a time through the wave's own parts of stage 1:
      // nobody else copies or reads there
      constexpr int kLanes = 8, kLines = 8;  // 8 columns a lane, rows a step
      auto place = [&](int r, int ch) {
        static_assert(NJ == 2 && SH::kCopiesN * kWave * (NI == 1 ? 1 : 2) == 512,
                      "32 rows of 256 bytes");
        const int half = NI == 1 || r >= 16 ? SH::kVecM : 0;  // which of the wave's parts
        return stage1 + half + wave * SH::kCopiesN * kWave + (NI == 1 ? r : r & 15) * 16 +
               (ch ^ (r & 15));
      };
      const __amdgpu_buffer_rsrc_t rh = uniform_rsrc(
          KIND == kRowsSwiglu ? p.h + first : nullptr, KIND == kRowsSwiglu ? bytes : 0u);
      const int col = t.n0 + wn * NJ * 32 + (lane % kLanes) * 8;
#pragma unroll
      for (int i = 0; i < ni; ++i) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *place(lane & 31, j * 8 + 2 * g + (lane >> 5)) = make_uint4(
                __float_as_uint(acc[j][i][4 * g]), __float_as_uint(acc[j][i][4 * g + 1]),
                __float_as_uint(acc[j][i][4 * g + 2]), __float_as_uint(acc[j][i][4 * g + 3]));
        wave_lds_fence();
#pragma unroll
        for (int l = 0; l < 32; l += kLines) {
          const int r = l + lane / kLanes;
          float o[8];
#pragma unroll
          for (int c = 0; c < 8; c += 4) {
            const uint4 q = *place(r, ((lane % kLanes) * 8 + c) / 4);
            o[c] = __uint_as_float(q.x);
            o[c + 1] = __uint_as_float(q.y);
            o[c + 2] = __uint_as_float(q.z);
            o[c + 3] = __uint_as_float(q.w);
          }
          const uint32_t row = (uint32_t)((i * SH::WM + wm) * 32 + r);
          const uint32_t at = col < p.N ? (row * cols + (uint32_t)col) * 2u : kOOB;
          if constexpr (KIND == kRowsSwiglu) {
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
          } else {
            __builtin_amdgcn_raw_buffer_store_b128(pack8(o), rc, at, 0, 0);
          }
        }
        wave_lds_fence();
      }
    }
  };

  int item = first_item(blockIdx.x, gridDim.x);
  if (item >= total) return;
  setup(item);
  fetch(stage0, 0);
  fetch(stage1, 1);
  vm_wait<kCopies>();
  bool more = true;
  while (more) {
    const int next = item + gridDim.x;
    more = next < total;
    // Slice 1 of an item of one slice is nothing, but has to have been there before
    // its place is used for results.
    if (!WEIGHTS && it.nd < 2) vm_wait<0>();
    auto go_on = [&]() {
      if (more) {
        setup(next);
        fetch(stage0, 0);
        if constexpr (WEIGHTS) fetch(stage1, 1);
      }
    };
    // A wave with ni fragments of rows: the accumulators live here alone, so that
    // the forms' registers do not add up.
    auto work = [&](auto nic) {
      constexpr int ni = decltype(nic)::value;
      floatx16 acc[NJ][ni];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < ni; ++i) acc[j][i] = floatx16{};
      contract([&](const uint4* stage) { multiply(stage, acc); });
      const Item<SH> done = it;
      go_on();
      __builtin_amdgcn_sched_barrier(0);  // the counts below go by this order
      store(done, acc);
      __builtin_amdgcn_sched_barrier(0);
      if (!WEIGHTS && more) fetch(stage1, 1);
      // the next item's slice 0, with slice 1 and the stores behind it
      vm_wait<kCopies + kStores / NI * ni>();
      behind = WEIGHTS && ni == NI ? 1 : 0;
    };
    const int high = WEIGHTS ? min(p.M - it.m0, BM) : it.rows;
    const int ni = max(0, (ceil_div(high, 32) - wm + SH::WM - 1) / SH::WM);
    if (ni == 0 || it.n0 + wn * NJ * 32 >= p.N) {  // copies alone
      contract([](const uint4*) {});
      go_on();
      if (!WEIGHTS && more) fetch(stage1, 1);
      vm_wait<kCopies>();
      behind = 0;
    } else if (ni == 1 || NI == 1) {
      work(std::integral_constant<int, 1>{});
    } else if constexpr (NI == 4) {
      if (ni == 2) work(std::integral_constant<int, 2>{});
      else if (ni == 3) work(std::integral_constant<int, 3>{});
      else work(std::integral_constant<int, 4>{});
    }
    item = next;
  }
  vm_wait<0>();  // no copy into LDS outlives the block
}

}  // namespace

int grad_splits(int S, int max_rows, int M, int N, int tile) {
  const int64_t tiles = (int64_t)S * ceil_div(M, tile) * ceil_div(N, tile);
  const int64_t want = (2 * kSplitBlocks + tiles - 1) / tiles;  // two rounds of the chip
  const int64_t most = max_rows / ((int64_t)S * 512);          // 512 rows each
  const int64_t n = want < most ? want : most;
  return tiles >= kSplitBlocks || n < 2 ? 1 : n > kMaxSplits ? kMaxSplits : (int)n;
}

namespace {

// Small tiles where the large ones would leave the chip half empty, or, with up to
// 24 rows a slot (a tile each, bound by reading the weights), the last round of
// them. Measured with large and small tiles: 16 slots of 1024 x 512 (32 and 64
// large tiles) at 12 rows 21 and 18 us, at 192 rows 37 and 19; 60 slots of 2048 x
// 1408 (360 and 480) at 4 rows 101 and 70, 137 and 124, at 24 rows 104 and 80, 135
// and 128, at 32 rows 106 and 110, 136 and 165 (slots of two small tiles); 64
// slots of 4096 x 1024 (256: a full round) at 12 rows 104 and 121.
constexpr int kFewRows = 24;

bool take_small(int S, int max_rows, int N, int cus) {
  const bool few = max_rows <= (int64_t)S * kFewRows;
  const int64_t slots = S < max_rows ? S : max_rows;
  const int64_t tiles = (few ? slots : (int64_t)max_rows / Large::kRowsM + slots) *
                        ceil_div(N, Large::kColsN);
  const int64_t rounds = (tiles + cus - 1) / cus;
  return 2 * tiles <= cus || (few && 20 * tiles < 19 * rounds * cus);
}

// Half tiles of the weights' gradient, whose two blocks a compute unit copy, multiply
// and store independently of each other: where large tiles would leave the chip half
// empty, or would be at most one round of short contractions, and for bf16 results of
// few rows a slot, whose stores are what takes the time. Measured with large and half
// tiles: 1 slot of 2048 x 1408 (48 large tiles), 1000 rows 25.2 and 19.2 us; 16 of
// 1024 x 512 (128) at 32 rows 9.6 and 8.9, 1000 27.0 and 23.6; 20 of 1408 x 512 (240)
// at 96 rows 11.8 and 10.4, f32 15.8 and 13.9, at 510 19.5 and 19.8, 1000 30.2 and
// 32.4; 60 of 2816 x 2048 at 32 rows 145 and 135, 96 213 and 189, 192 262 and 257, f32
// results at 32 rows 263 and 274, added to bf16 271 and 279; 64 of 2048 x 4096 at 32
// rows 220 and 218, 96 326 and 317, 128 357 and 362, 510 669 and 722.
constexpr int kHalfRows = 96, kHalfRoundRows = 256;

bool take_half(int S, int splits, int max_rows, int M, int N, bool f32, bool add, int cus) {
  const int64_t tiles = (int64_t)S * splits * ceil_div(M, Large::kRowsM) * ceil_div(N, Large::kColsN);
  return 2 * tiles <= cus || (tiles <= cus && max_rows <= (int64_t)S * kHalfRoundRows) ||
         (!f32 && !add && max_rows <= (int64_t)S * kHalfRows);
}

}  // namespace

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
  auto go = [&](auto kind, auto shape) {
    typedef decltype(shape) SH;
    const int64_t items = (int64_t)(max_rows / SH::kRowsM + 1 + (S < max_rows ? S : max_rows)) *
                          ceil_div(N, SH::kColsN);
    const int64_t blocks = (int64_t)device_cu_count() * (SH::kWaves == 8 ? 1 : 2);
    grouped_grad_kernel<decltype(kind)::value, SH>
        <<<(int)std::min(items, blocks), SH::kThreads, 0, stream>>>(p);
  };
  auto by_kind = [&](auto shape) {
    if (h != nullptr) go(std::integral_constant<int, kRowsSwiglu>{}, shape);
    else go(std::integral_constant<int, kRows>{}, shape);
  };
  if (take_small(S, max_rows, N, device_cu_count())) by_kind(Small{});
  else by_kind(Large{});
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
  p.splits = grad_splits(S, max_rows, M, N, kGradTileBf16);
  p.out = p.splits > 1 ? ws : dw;
  const bool f32 = dw_f32 || p.splits > 1, add = accumulate && p.splits == 1;
  auto go = [&](auto kind, auto shape, auto adds) {
    typedef decltype(shape) SH;
    const int64_t items = (int64_t)S * p.splits * ceil_div(M, SH::kRowsM) * ceil_div(N, SH::kColsN);
    const int64_t blocks = (int64_t)device_cu_count() * (SH::kWaves == 8 ? 1 : 2);
    grouped_grad_kernel<decltype(kind)::value, SH, decltype(adds)::value>
        <<<(int)std::min(items, blocks), SH::kThreads, 0, stream>>>(p);
  };
  auto by_add = [&](auto kind, auto shape) {
    if (add) go(kind, shape, std::true_type{});
    else go(kind, shape, std::false_type{});
  };
  auto by_kind = [&](auto shape) {
    if (f32) by_add(std::integral_constant<int, kWeightsF32>{}, shape);
    else by_add(std::integral_constant<int, kWeights>{}, shape);
  };
  if (take_half(S, p.splits, max_rows, M, N, f32, add, device_cu_count())) by_kind(Half{});
  else by_kind(Large{});
  if (p.splits > 1)
    return launch_fold_splits(static_cast<const float*>(ws), p.splits, (size_t)S * M * N, dw, dw_f32,
                              accumulate, stream);
  return launch_status();
}

}  // namespace moe
