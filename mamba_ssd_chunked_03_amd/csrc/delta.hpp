// Shared pieces of the gated delta rule's kernels (k_delta_*.hip) and the host
// side's description of one problem.
//
// Per sequence and head, with the state S (P x N), a_t = exp(g_t):
//   S_t = a_t S_{t-1} + b_t (v_t - a_t S_{t-1} k_t) k_t^T,   o_t = scale S_t q_t.
// In chunks of C = 64 tokens, with G the running sum of g inside the chunk,
// D_ij = exp(G_i - G_j) and S the state entering the chunk (rows are tokens):
//   M = strict lower part of (K K^T . D),  R = M (I + diag(b) M)^-1  (strictly lower),
//   X = V - exp(G) K S^T,   Z = X - R (b X),   U = b Z,
//   O = scale (exp(G) Q S^T + (Q K^T . D) U),   S' = exp(G_C) S + (exp(G_C - G) U)^T K.
// (I + b M)^-1 = I - b R and (I + M b)^-1 = I - R b, so that R alone serves the
// forward, the backward and the gradient of b, also where b is zero.
//
// Precision.  The states and the gates' gradients are fp32 results, and an error of
// the state is carried through every later chunk.  Matrix products run on the bf16
// MFMA with fp32 accumulation, each fp32 operand split into bf16 planes
// (x = x0 + x1 [+ x2], each the rounding of what the ones before leave): two planes
// where the inputs are bf16 (those are one exact plane), the products x0 y0 + x0 y1
// + x1 y0 leaving about 2^-17 of a product; three planes and six products where the
// inputs are fp32.  Two planes cost 2-3 matrix instructions a product and stay 2-3
// times above the fp32 matrix cores' rate.
#pragma once

#include "internal.hpp"

namespace ssd {

constexpr int kDeltaChunk = 64;

// Natural-log gates below this are taken as this: exp of it is zero in fp32, and
// running sums of it stay finite (a gate of -inf resets the state).
constexpr float kDeltaMinGate = -256.f;
// (a NaN stays one)
__device__ __forceinline__ float min_gate(float g) { return g < kDeltaMinGate ? kDeltaMinGate : g; }

// Whether sequence b of a call on slots runs (asked by a whole workgroup of 256): its slot lies in
// [0, nslots) and no earlier sequence names it.  mine = slots[min(threadIdx.x, b)], loaded by
// the caller beside its data.
__device__ __forceinline__ bool slot_runs(const int32_t* slots, int b, int slot, int nslots, int32_t mine) {
  int dup = (int)threadIdx.x < b && mine == slot;
  for (int i = threadIdx.x + 256; i < b; i += 256) dup |= slots[i] == slot;
  return !__syncthreads_or(dup) && slot >= 0 && slot < nslots;
}

struct DeltaProb {
  int32_t B, L, H, P, N, G;
  int32_t nst;   // state slots: batch rows, or packed sequences
  int32_t io;    // 0 fp32, 1 bf16
  int32_t packed;
  int32_t flags;
  float scale;
  int64_t nck;   // chunk slots of 64 tokens
  ChunkMap map;
};

// Regions of the workspace (byte offsets, 256-byte aligned).
struct DeltaLayout {
  size_t tab, seq_off, gates, R, Pm, fwd_end;  // the forward's
  size_t Rt, Pt, S, Z, dS, F, parts, end;      // kept for the backward, and the backward's
};

// Per-problem pointers of the chunked kernels.
struct DeltaArgs {
  ChunkMap map;
  int32_t H, G, P, N, L;
  float scale;
  const void *q, *k, *v;
  const float *g, *beta, *init;
  void* out;
  float* final_states;
  float* gates;                // (nck, H, kDeltaGates): see below
  uint16_t *R, *Pm, *Rt, *Pt;  // plane-split chunk matrices in operand order (null: not kept)
  float *S, *Z;                // kept for the backward: states entering each chunk, Z (see below)
  // backward
  const void* dout;
  const float* d_final;
  float *dS, *F;               // adjoints of the states leaving each chunk, F (see below)
  float* d_init;
  void *dq, *dk, *dv;
  float *dg, *dbeta;
  float* parts;                // (nck, H, 2, 64, dstate): each head's dq and dk, or null: summed in one workgroup
};

// Per (chunk, head), 64 tokens each: running log2 decay G (high part, low part), beta; and
// where io is bf16 exp(G), beta exp(G_C - G), exp(G_C - G), beta exp(G).  Past the chunk's
// end G stays and beta is zero.
constexpr int kDeltaGates = 7 * kDeltaChunk;

// States and their adjoints per (chunk, head), and Z and F, are kept in fp32 in the order of the
// chains' accumulator tiles, 16 columns of headdim after the other, so that a wave stores
// 1 KB runs: states (P / 16, NP / 32, 2, 64 lanes, 4), NP = dstate or 32, lane 16 q + r of
// tile (k, t) holding row r, columns 32k + 8q + 4t + 0..3; Z, F (P / 16, 4, 64 lanes, 4),
// lane 16 q + r of tile i column r of tokens 32 (i / 2) + 8q + 4 (i % 2) + 0..3.  (As the two planes
// that the products take, <S, dS> would lose three digits: 4e-5 of dg over a few tokens.)
__host__ __device__ __forceinline__ int state_cols(int N) { return N < 32 ? 32 : N; }
// float offset of columns n..n+3 (n a multiple of 4) of headdim row p
__device__ __forceinline__ int state_at(int p, int n, int NP) {
  return ((((p >> 4) * (NP >> 5) + (n >> 5)) * 2 + ((n >> 2) & 1)) * 64 + ((n & 31) >> 3) * 16 + (p & 15)) * 4;
}
__device__ __forceinline__ int row_at(int p, int t) {
  return (((p >> 4) * 4 + (t >> 5) * 2 + ((t >> 2) & 1)) * 64 + ((t & 31) >> 3) * 16 + (p & 15)) * 4 + (t & 3);
}

hipError_t launch_delta_f32_fwd(const DeltaProb& p, const DeltaArgs& a, hipStream_t st);
hipError_t launch_delta_f32_bwd(const DeltaProb& p, const DeltaArgs& a, hipStream_t st);
hipError_t launch_delta_prep(const DeltaProb& p, const DeltaArgs& a, hipStream_t st);
hipError_t launch_delta_fwd(const DeltaProb& p, const DeltaArgs& a, hipStream_t st);
hipError_t launch_delta_bwd_chain(const DeltaProb& p, const DeltaArgs& a, hipStream_t st);
hipError_t launch_delta_bwd_grads(const DeltaProb& p, const DeltaArgs& a, hipStream_t st);
hipError_t launch_delta_step(const DeltaProb& p, const void* q, const void* k, const void* v, const float* g,
                             const float* beta, const int32_t* slots, int nslots, float* states, void* out,
                             hipStream_t st);
hipError_t launch_state_cache(bool write, int n, int nslots, int H, int P, int N, int format, float* states,
                              const int32_t* slots, void* codes, float* scales, hipStream_t st);

// ------------------------------------------------------------- io types ----
// PI: bf16 planes that hold an input exactly; PM: planes of a computed operand.
struct IoBf16 {
  using T = uint16_t;
  static constexpr int PI = 1, PM = 2;
};
struct IoF32 {
  using T = float;
  static constexpr int PI = 3, PM = 3;
};

template <int NP>
struct Planes {
  bf16x8 p[NP];
};

// x - h for each half h of the bf16 pair w and its own x, exactly: one v_dot2c_f32_bf16 with
// (-1, 0) or (0, -1) instead of a shift or mask and a subtraction.  (The masks come from
// registers the compiler cannot see into: as an inline constant it prints -1.0, which the
// instruction takes as fp32, that is for the other half.  Exact over 4 million pairs of
// random bits, subnormals included; an infinity makes its neighbour's rest a NaN.)
__device__ __forceinline__ void sub_bf2(uint32_t w, float& x0, float& x1) {
  uint32_t c0 = 0x0000bf80u, c1 = 0xbf800000u;
  asm("" : "+s"(c0));
  asm("" : "+s"(c1));
  const bf16x2v h = __builtin_bit_cast(bf16x2v, w);
  x0 = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2v, c0), x0, false);
  x1 = __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf16x2v, c1), x1, false);
}

// planes of 4 floats, 8 bytes each (consecutive elements)
template <int NP>
__device__ __forceinline__ void split4(f32x4 x, uint2 (&o)[NP]) {
  float f[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    o[i] = make_uint2(pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]));
    if (i + 1 < NP) {
      sub_bf2(o[i].x, f[0], f[1]);
      sub_bf2(o[i].y, f[2], f[3]);
    }
  }
}
// planes of 8 floats
template <int NP>
__device__ __forceinline__ void split8(f32x4 a, f32x4 b, u32x4 (&o)[NP]) {
  uint2 x[NP], y[NP];
  split4<NP>(a, x);
  split4<NP>(b, y);
#pragma unroll
  for (int i = 0; i < NP; ++i) o[i] = u32x4{x[i].x, x[i].y, y[i].x, y[i].y};
}

// c += sum of the products of planes i of a and j of b with i + j < PM, smallest first.
template <int PM, int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Planes<NA>& a, const Planes<NB>& b, f32x4 c) {
#pragma unroll
  for (int s = PM - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) c = mfma_bf16(a.p[i], b.p[s - i], c);
  return c;
}

// MFMA operand from LDS planes stored [row][k] (k contiguous, row stride ld elements):
// lane (q, r) reads elements 8q..8q+7 of row r.  `t` points at [row0][k0] of plane 0.
template <int NP>
__device__ __forceinline__ Planes<NP> lds_rows(const uint16_t* t, int ld, int plane, int lane) {
  Planes<NP> f;
#pragma unroll
  for (int i = 0; i < NP; ++i)
    f.p[i] = as_bf16x8(*(const u32x4*)(t + i * plane + (lane & 15) * ld + 8 * (lane >> 4)));
  return f;
}
// ... stored [k][row] (the contraction along the LDS rows), by transposing reads.
template <int NP>
__device__ __forceinline__ Planes<NP> lds_cols(const uint16_t* t, int ld, int plane, int lane) {
  Planes<NP> f;
#pragma unroll
  for (int i = 0; i < NP; ++i) f.p[i] = frag_kmajor(t + i * plane, ld, lane);
  return f;
}

// 16-byte load at a vector and a scalar offset
__device__ __forceinline__ u32x4 buf_load16(brsrc r, uint32_t off, int soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, 0));
}

// An io row's 8 elements as raw 16-byte pieces (one for bf16, two for fp32), loaded
// through a range-checked resource, and their planes.
template <class IO>
struct Raw8;
template <>
struct Raw8<IoBf16> {
  u32x4 v;
  __device__ __forceinline__ void load(brsrc r, uint32_t off) { v = buf_load16(r, off); }
  __device__ __forceinline__ void planes(u32x4 (&o)[1]) const { o[0] = v; }
};
template <>
struct Raw8<IoF32> {
  f32x4 a, b;
  __device__ __forceinline__ void load(brsrc r, uint32_t off) {
    a = __builtin_bit_cast(f32x4, buf_load16(r, off));
    b = __builtin_bit_cast(f32x4, buf_load16(r, off + 16));
  }
  __device__ __forceinline__ void planes(u32x4 (&o)[3]) const { split8<3>(a, b, o); }
};
template <class IO>
__device__ __forceinline__ Planes<IO::PI> raw_planes(const Raw8<IO>& x) {
  u32x4 o[IO::PI];
  x.planes(o);
  Planes<IO::PI> f;
#pragma unroll
  for (int i = 0; i < IO::PI; ++i) f.p[i] = as_bf16x8(o[i]);
  return f;
}

// 4 consecutive io elements: raw, as fp32, and stored.  (Raw where a load is used later:
// widening a loaded value waits for it.)
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
template <class IO>
struct Raw4;
template <>
struct Raw4<IoBf16> {
  u32x2v v;
  __device__ __forceinline__ void load(brsrc r, uint32_t off) {
    v = __builtin_bit_cast(u32x2v, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
  }
  __device__ __forceinline__ f32x4 get() const { return f32x4{bf_lo(v[0]), bf_hi(v[0]), bf_lo(v[1]), bf_hi(v[1])}; }
};
template <>
struct Raw4<IoF32> {
  u32x4 v;
  __device__ __forceinline__ void load(brsrc r, uint32_t off) { v = buf_load16(r, off); }
  __device__ __forceinline__ f32x4 get() const { return __builtin_bit_cast(f32x4, v); }
};
__device__ __forceinline__ void store4io(brsrc r, uint32_t off, f32x4 v, IoBf16) {
  const u32x2v w = {pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3])};
  __builtin_amdgcn_raw_buffer_store_b64(w, r, off, 0, 0);
}
__device__ __forceinline__ void store4io(brsrc r, uint32_t off, f32x4 v, IoF32) {
  buf_store16(r, off, __builtin_bit_cast(u32x4, v));
}

// 2^(h + l) of a high and a small low part (their sum in fp32 would drop the low one)
__device__ __forceinline__ float exp2_hl(float h, float l) {
  const float e = exp2_fast(h);
  return fmaf(e, l * 0.6931471805599453f, e);
}

// The chunk slots [c0, c1) and tokens [start, end) of sequence s, as scalars (uniform over
// the workgroup: what is derived from them stays in scalar registers).
struct SeqSpan {
  int c0, c1, start, end;
};
__device__ __forceinline__ SeqSpan seq_span(const ChunkMap& m, int s) {
  SeqSpan x;
  if (!m.packed) {
    x.c0 = s * m.ncs;
    x.c1 = x.c0 + m.ncs;
    x.start = s * m.seqlen;
    x.end = x.start + m.seqlen;
  } else {
    x.c0 = min(m.seq_off[s], m.nck);
    x.c1 = min(m.seq_off[s + 1], m.nck);
    x.start = x.end = 0;
    if (x.c1 > x.c0) {
      const int4 a = m.tab[x.c0], b = m.tab[x.c1 - 1];
      x.start = a.x;
      x.end = b.x + b.y;
    }
  }
  x.c0 = __builtin_amdgcn_readfirstlane(x.c0);
  x.c1 = __builtin_amdgcn_readfirstlane(x.c1);
  x.start = __builtin_amdgcn_readfirstlane(x.start);
  x.end = __builtin_amdgcn_readfirstlane(x.end);
  return x;
}

// A buffer offset that no resource covers (loads zero, stores nothing).
constexpr uint32_t kNoOffset = 0x80000000u;

// ------------------------------------------------- chunk matrices, stored ----
// R and P (64 x 64, lower triangular) and their transposes (upper triangular) are kept
// as the six 16 x 32 blocks that are not all zero, 1 KB a block and plane in the order
// of an MFMA operand load (lane (q, r): columns 8q..8q+7 of row r).  Row block R of a
// lower matrix needs column block 0, and 1 from R = 2 on; of a transposed one column
// block 1, and 0 up to R = 1.
constexpr int kTriBlocks = 6, kTriPlane = kTriBlocks * 512;  // elements of one plane
__host__ __device__ __forceinline__ int tri_block(int R, int S) { return R < 2 ? R : 2 * (R - 1) + S; }
__host__ __device__ __forceinline__ int trit_block(int R, int S) { return R < 2 ? 2 * R + S : R + 2; }

}  // namespace ssd
