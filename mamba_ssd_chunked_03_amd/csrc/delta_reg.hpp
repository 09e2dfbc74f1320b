// Tiles of the bf16 kernels of the gated delta rule that stay in registers.
//
// A product's accumulator tile D (16 x 16) leaves lane (q, r) with rows 4q..4q+3 of
// column r, and an MFMA operand of depth 32 wants 8 consecutive depths 8q..8q+7 in lane
// group q.  Rows of a 32-row block are therefore dealt to its two tiles (t = 0, 1) so
// that row 4q + e of tile t is row 8q + 4t + e of the block: the two tiles' registers,
// side by side, are then an operand of the next product (the contraction running over
// those rows) with nothing moved between lanes.  Operand rows are read in the same
// order (row32 below); a transposing LDS read takes its four groups of four columns
// eight apart (cols32).
#pragma once

#include "delta.hpp"

namespace ssd {

// row of a 32-row block that operand row r (0..15) of tile t stands for
__device__ __forceinline__ int row32(int r, int t) { return 8 * (r >> 2) + 4 * t + (r & 3); }

// Lower triangular 64 x 64 matrices (R, P) in operand order: row tile (B, t), column
// block S <= B; transposed ones: row tile (S, t), column block B >= S.
__host__ __device__ __forceinline__ int low_block(int B, int t, int S) { return B == 0 ? t : 2 + 2 * t + S; }
__host__ __device__ __forceinline__ int up_block(int S, int t, int B) { return S == 1 ? 4 + t : 2 * t + B; }

// LDS tile of 64 token rows of NP bf16 (NP = 32, 64, 128): rows 16 dwords apart modulo the
// 64 banks, and shifted by four dwords every eight rows.  The 16 rows of an operand read
// (row32) then fill the banks once, and the transposing reads take twice their minimum.
template <int NP>
struct TokTile {
  static constexpr int LD = NP == 128 ? 160 : NP == 64 ? 96 : 32, SIZE = kDeltaChunk * LD + 64;
  static __device__ __forceinline__ int at(int row, int col) { return row * LD + 8 * (row >> 3) + col; }
};

// Operand of depth 32 from such a tile: rows row0 + row32(r, t), depths col0 + 8q..8q+7.
template <int NP>
__device__ __forceinline__ bf16x8 tok_rows(const uint16_t* p, int row0, int t, int col0, int lane) {
  return as_bf16x8(*(const u32x4*)(p + TokTile<NP>::at(row0 + row32(lane & 15, t), col0 + 8 * (lane >> 4))));
}
// ... the contraction along the rows: depths row0 + 8q..8q+7, operand row 4g + e <-> column
// col0 + 8g + 4t + e, by transposing reads.
template <int NP>
__device__ __forceinline__ bf16x8 tok_cols(const uint16_t* tile, int row0, int t, int col0, int lane) {
  const int j = lane & 15;
  const uint16_t* p = tile + TokTile<NP>::at(row0 + 8 * (lane >> 4), col0 + 8 * (j & 3) + 4 * t) + (j >> 2) * TokTile<NP>::LD;
  v4i16 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)p);
  v4i16 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(p + 4 * TokTile<NP>::LD));
  v8i16 c = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8, c);
}

// two tiles (rows 8q + 0..3, 8q + 4..7 of a 32-row block) -> operand planes
template <int NP>
__device__ __forceinline__ Planes<NP> tile_planes(f32x4 a, f32x4 b) {
  u32x4 o[NP];
  split8<NP>(a, b, o);
  Planes<NP> f;
#pragma unroll
  for (int i = 0; i < NP; ++i) f.p[i] = as_bf16x8(o[i]);
  return f;
}

// Scheduling pattern of the region before it: M matrix instructions, V vector ones after each.
template <int M, int V>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < M; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
  }
}

// Chain waves a tile of 16 columns of headdim: the 128 columns of the state are dealt to two.
template <int N>
constexpr int kSplit = N == 128 ? 2 : 1;

constexpr int kNumCu = 256;
// Tiles a workgroup of a chain: two where one each would not fit the CUs at once.
inline bool two_tiles(int64_t heads, int ptiles) { return ptiles >= 2 && heads * ptiles > kNumCu; }

// (sequence, workgroup of the sequence) of a chain's workgroup: each XCD takes the same part
// of every sequence's `per` workgroups (heads of one group share K and Q in its L2), so that
// a long sequence among short ones is spread over all of them.
__device__ __forceinline__ void chain_order(int per, int& s, int& i) {
  const int wg = blockIdx.x;
  if (per % kNumXcd == 0) {
    const int part = per / kNumXcd, slot = wg / kNumXcd;
    s = slot / part;
    i = wg % kNumXcd * part + slot % part;
  } else {
    const int l = xcd_order(wg, gridDim.x);
    s = l / per;
    i = l % per;
  }
}

}  // namespace ssd
