// Gated delta rule, per chunk of 64 tokens and head: the running decay, and the chunk
// matrices R = M (I + diag(b) M)^-1 with M = strict lower (K K^T . D), and
// P = scale Q K^T . D (lower), plane-split and in the order MFMA operand loads read.
//
// A workgroup takes one chunk and up to four heads of one group: its four waves form
// K K^T and Q K^T once (MFMA, into LDS), then each wave solves one head's triangle by
// forward substitution in fp32, row i of R from the rows above it,
//   R_i = M_i - sum_{j<i} M_ij b_j R_j,
// with a lane per column: it is backward stable whatever the keys (equal keys and
// b = 1 leave entries that a product of powers of M would cancel to nothing).
// The running sums of g are taken in fp64 and kept as a high and a low fp32 part:
// exponents are differences of them.
#include "delta.hpp"

namespace ssd {

constexpr int kMatLd = 68;  // row stride of the 64 x 64 fp32 matrices in LDS

// rows R, columns 8q..8q+7 of column block S of an fp32 LDS matrix (transposed: of its
// transpose) as planes, stored where block `blk` of each plane lies.
template <int NP, bool TR>
__device__ __forceinline__ void store_block(const float* m, uint16_t* dst, int blk, int R, int S, int lane) {
  const int r = 16 * R + (lane & 15), c = 32 * S + 8 * (lane >> 4);
  f32x4 a, b;
  if constexpr (TR) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = m[(c + e) * kMatLd + r];
      b[e] = m[(c + 4 + e) * kMatLd + r];
    }
  } else {
    a = *(const f32x4*)(m + r * kMatLd + c);
    b = *(const f32x4*)(m + r * kMatLd + c + 4);
  }
  u32x4 o[NP];
  split8<NP>(a, b, o);
#pragma unroll
  for (int i = 0; i < NP; ++i) *(u32x4*)(dst + i * kTriPlane + blk * 512 + lane * 8) = o[i];
}

template <int N, class IO>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a, int hsplit) {
  constexpr int PI = IO::PI, PM = IO::PM, KS = (N + 31) / 32, ES = sizeof(typename IO::T);
  __shared__ __align__(16) float mats[6][kDeltaChunk * kMatLd];
  float* KK = mats[4];
  float* QK = mats[5];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  const int wg = xcd_order(blockIdx.x, gridDim.x);
  const int hs = wg % hsplit, grp = (wg / hsplit) % a.G, ck = wg / hsplit / a.G;
  ChunkInfo ci = chunk_info(a.map, ck);
  ci.start = __builtin_amdgcn_readfirstlane(ci.start);
  ci.len = __builtin_amdgcn_readfirstlane(ci.len);
  if (ci.len <= 0) return;  // an unused slot
  const int per = a.H / a.G, h = grp * per + hs * 4 + w;
  const bool mine = hs * 4 + w < per;

  // K K^T and Q K^T, lower block triangle: wave w rows 16w..16w+15
  {
    const uint32_t row = (uint32_t)a.G * N * ES;
    const int64_t base = ((int64_t)ci.start * a.G + grp) * N * ES;
    const uint32_t span = (uint32_t)(ci.len - 1) * row + N * ES;
    const brsrc rk = make_rsrc((const char*)a.k + base, span), rq = make_rsrc((const char*)a.q + base, span);
    auto frag = [&](brsrc rs, int R, int ks) {
      Raw8<IO> x;
      x.load(rs, 32 * ks + 8 * q < N ? (16 * R + r) * row + (32 * ks + 8 * q) * ES : kNoOffset);
      return raw_planes<IO>(x);
    };
    Planes<PI> kf[KS], qf[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      kf[ks] = frag(rk, w, ks);
      qf[ks] = frag(rq, w, ks);
    }
    for (int J = 0; J <= w; ++J) {
      f32x4 kk = {0.f, 0.f, 0.f, 0.f}, qk = kk;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const Planes<PI> jf = frag(rk, J, ks);
        kk = mma<PM>(kf[ks], jf, kk);
        qk = mma<PM>(qf[ks], jf, qk);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        KK[(16 * w + 4 * q + e) * kMatLd + 16 * J + r] = kk[e];
        QK[(16 * w + 4 * q + e) * kMatLd + 16 * J + r] = qk[e];
      }
    }
  }
  __syncthreads();
  if (!mine) return;

  // gates: lane = token; past the chunk's end the decay stays and beta is zero
  const int64_t tok = (int64_t)ci.start + lane;
  const float gv = lane < ci.len ? fmaxf(a.g[tok * a.H + h], kDeltaMinGate) : 0.f;
  const float bv = lane < ci.len ? a.beta[tok * a.H + h] : 0.f;
  double G = (double)gv * 1.4426950408889634073599;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double up = __shfl_up(G, d);
    if (lane >= d) G += up;
  }
  const float Gh = (float)G, Gl = (float)(G - (double)Gh);
  const int64_t kh = (int64_t)ck * a.H + h;
  float* gt = a.gates + kh * (3 * kDeltaChunk);
  gt[lane] = Gh;
  gt[kDeltaChunk + lane] = Gl;
  gt[2 * kDeltaChunk + lane] = bv;

  float* M = mats[w];
  // M (strict lower), lane = column
#pragma unroll 8
  for (int i = 0; i < kDeltaChunk; ++i) {
    const float d = (__shfl(Gh, i) - Gh) + (__shfl(Gl, i) - Gl);
    M[i * kMatLd + lane] = lane < i ? KK[i * kMatLd + lane] * exp2_fast(d) : 0.f;
  }
  __builtin_amdgcn_wave_barrier();
  // forward substitution, row by row in place: br[j] = b_j R_j (this lane's column)
  float br[kDeltaChunk];
#pragma unroll
  for (int i = 0; i < kDeltaChunk; ++i) {
    float s[4] = {M[i * kMatLd + lane], 0.f, 0.f, 0.f};
#pragma unroll
    for (int j4 = 0; j4 < (i + 3) / 4; ++j4) {
      const f32x4 m = *(const f32x4*)(M + i * kMatLd + 4 * j4);  // one address: a broadcast
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (4 * j4 + e < i) s[e] -= m[e] * br[4 * j4 + e];
    }
    const float x = (s[0] + s[1]) + (s[2] + s[3]);
    __builtin_amdgcn_wave_barrier();
    M[i * kMatLd + lane] = x;
    br[i] = x * __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bv), i));
  }
  __builtin_amdgcn_wave_barrier();
  {
    uint16_t* dst = a.R + kh * (PM * kTriPlane);
#pragma unroll
    for (int R = 0; R < 4; ++R)
#pragma unroll
      for (int S = 0; S <= (R >= 2); ++S) store_block<PM, false>(M, dst, tri_block(R, S), R, S, lane);
    if (a.Rt) {
      dst = a.Rt + kh * (PM * kTriPlane);
#pragma unroll
      for (int R = 0; R < 4; ++R)
#pragma unroll
        for (int S = R >= 2; S < 2; ++S) store_block<PM, true>(M, dst, trit_block(R, S), R, S, lane);
    }
  }
  __builtin_amdgcn_wave_barrier();
  // P over the same buffer (inclusive lower triangle)
#pragma unroll 8
  for (int i = 0; i < kDeltaChunk; ++i) {
    const float d = (__shfl(Gh, i) - Gh) + (__shfl(Gl, i) - Gl);
    M[i * kMatLd + lane] = lane <= i ? a.scale * (QK[i * kMatLd + lane] * exp2_fast(d)) : 0.f;
  }
  __builtin_amdgcn_wave_barrier();
  {
    constexpr int PF = PI;  // planes of P that the output takes (bf16 outputs: one)
    uint16_t* dst = a.Pm + kh * (PF * kTriPlane);
#pragma unroll
    for (int R = 0; R < 4; ++R)
#pragma unroll
      for (int S = 0; S <= (R >= 2); ++S) store_block<PF, false>(M, dst, tri_block(R, S), R, S, lane);
    if (a.Pt) {
      dst = a.Pt + kh * (PM * kTriPlane);
#pragma unroll
      for (int R = 0; R < 4; ++R)
#pragma unroll
        for (int S = R >= 2; S < 2; ++S) store_block<PM, true>(M, dst, trit_block(R, S), R, S, lane);
    }
  }
}

hipError_t launch_delta_prep(const DeltaProb& p, const DeltaArgs& a, hipStream_t st) {
  if (p.nck == 0) return hipSuccess;
  const int hsplit = (p.H / p.G + 3) / 4;
  const dim3 grid((unsigned)(p.nck * p.G * hsplit)), block(256);
  auto go = [&](auto io) {
    using IO = decltype(io);
    switch (p.N) {
      case 16: hipLaunchKernelGGL((delta_prep_kernel<16, IO>), grid, block, 0, st, a, hsplit); break;
      case 32: hipLaunchKernelGGL((delta_prep_kernel<32, IO>), grid, block, 0, st, a, hsplit); break;
      case 64: hipLaunchKernelGGL((delta_prep_kernel<64, IO>), grid, block, 0, st, a, hsplit); break;
      default: hipLaunchKernelGGL((delta_prep_kernel<128, IO>), grid, block, 0, st, a, hsplit); break;
    }
  };
  if (p.io)
    go(IoBf16{});
  else
    go(IoF32{});
  return hipGetLastError();
}

}  // namespace ssd
