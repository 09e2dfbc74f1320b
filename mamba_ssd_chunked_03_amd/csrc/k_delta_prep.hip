// Gated delta rule, per chunk of 64 tokens and head: the running decay, and the
// chunk matrices R = M (I + diag(b) M)^-1 with M = strict lower (K K^T . D), and
// P = scale Q K^T . D (lower), as bf16 planes in the order the chains' operands take; for
// bf16 io R as R diag(b) for the forward and (diag(b) R)^T for the backward, which saves the
// chains a product with b on their way (the split is of the product, so nothing is rounded
// twice).
//
// One wave per (chunk, up to HPW heads of one group), or, where there are few, one for R and
// one for P; waves do not interact.  K K^T and Q K^T are computed transposed, so that a lane
// holds four (P: eight) consecutive entries of a row: M is then an fp32 MFMA operand, and P a
// stored one, as it comes out.
//
// R by blocks of 16: the diagonal blocks by forward substitution in fp32, all four at
// once (lane = block and column),  R_i = M_i - sum_{j<i} M_ij b_j R_j,  then
//   Y_IJ = M_IJ - sum_{K=J}^{I-1} M_IK b_K R_KJ,   R_IJ = Y_IJ - R_II (b_I Y_IJ)
// on the fp32 matrix cores, an accumulator tile being the next product's operand without
// a move (row 4q + e of a tile is depth 4q + e of step e).  Substitution inside the
// blocks keeps it backward stable whatever the keys: equal keys and b = 1 leave entries
// that a product of powers of M would cancel to nothing.
//
// The running sums of g are taken in fp64 and kept as a high and a low fp32 part:
// exponents are differences of them.
#include <algorithm>

#include "delta_reg.hpp"

namespace ssd {

constexpr int kPrepLd = 68;               // row stride of the 64 x 64 fp32 matrix

template <int N, class IO, bool SAVE>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a, int hpw, int roles, int64_t items) {
  constexpr int KS = (N + 31) / 32, C = kDeltaChunk, PI = IO::PI, PM = IO::PM, ES = sizeof(typename IO::T);
  constexpr bool BF16 = PI == 1;
  __shared__ __align__(16) float lds[4][C * kPrepLd + 3 * C];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, q = lane >> 4, r = lane & 15;
  float *Rm = lds[w], *gh = Rm + C * kPrepLd, *gl = gh + C, *bb = gl + C;
  const int per = a.H / a.G, parts = (per + hpw - 1) / hpw;
  const int64_t slot = (int64_t)xcd_order(blockIdx.x, gridDim.x) * 4 + w, item = roles == 2 ? slot >> 1 : slot;
  if (item >= items) return;
  const bool solves = roles == 1 || (slot & 1) == 0, forms_p = roles == 1 || (slot & 1) == 1;
  const int part = (int)(item % parts), grp = (int)(item / parts % a.G), ck = (int)(item / parts / a.G);
  ChunkInfo ci = chunk_info(a.map, ck);
  const int start = __builtin_amdgcn_readfirstlane(ci.start), len = __builtin_amdgcn_readfirstlane(ci.len);
  if (len <= 0) return;  // an unused slot
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  const uint32_t row = (uint32_t)a.G * N * ES;
  const int64_t base = ((int64_t)start * a.G + grp) * N * ES;
  const uint32_t span = (uint32_t)(len - 1) * row + N * ES;
  const brsrc rk = make_rsrc((const char*)a.k + base, span), rq = make_rsrc((const char*)a.q + base, span);
  // an operand's row of tile t of a block of 32 rows, in the order of the io's chains
  auto rowof = [&](int t) { return BF16 ? row32(r, t) : 16 * t + r; };
  // K K^T, 16 x 16 blocks J <= I: lane (q, r) row 16I + r, columns 16J + 4q + e.  Q K^T in the
  // operands' row order.  qk[B][t][2S + u]: row 32B + rowof(t), columns 32S + 8q + 4u + e;
  // qt[S][u][2B + t] (for P^T): row 32S + rowof(u), columns 32B + 8q + 4t + e
  f32x4 kk[4][4], qk[2][2][4], qt[2][2][4];
  if constexpr (BF16) {
    auto frag = [&](brsrc rs, int t, int ks) {
      return as_bf16x8(buf_load16(rs, 32 * ks + 8 * q < N ? t * row + (32 * ks + 8 * q) * 2 : kNoOffset));
    };
    if (solves) {
      bf16x8 kf[4][KS];
#pragma unroll
      for (int I = 0; I < 4; ++I)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) kf[I][ks] = frag(rk, 16 * I + r, ks);
#pragma unroll
      for (int I = 0; I < 4; ++I)
#pragma unroll
        for (int J = 0; J <= I; ++J) {
          kk[I][J] = zero;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) kk[I][J] = mfma_bf16(kf[J][ks], kf[I][ks], kk[I][J]);
        }
    }
    if (forms_p) {
      bf16x8 kf[2][2][KS], qf[2][2][KS];
#pragma unroll
      for (int B = 0; B < 2; ++B)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            kf[B][t][ks] = frag(rk, 32 * B + row32(r, t), ks);
            qf[B][t][ks] = frag(rq, 32 * B + row32(r, t), ks);
          }
#pragma unroll
      for (int B = 0; B < 2; ++B)
#pragma unroll
        for (int S = 0; S <= B; ++S)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              qk[B][t][2 * S + u] = zero;
#pragma unroll
              for (int ks = 0; ks < KS; ++ks)
                qk[B][t][2 * S + u] = mfma_bf16(kf[S][u][ks], qf[B][t][ks], qk[B][t][2 * S + u]);
              if constexpr (SAVE) {
                qt[S][u][2 * B + t] = zero;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                  qt[S][u][2 * B + t] = mfma_bf16(qf[B][t][ks], kf[S][u][ks], qt[S][u][2 * B + t]);
              }
            }
    }
  } else {
    // three planes an operand: 32 columns at a time
#pragma unroll
    for (int I = 0; I < 4; ++I)
#pragma unroll
      for (int J = 0; J < 4; ++J) kk[I][J] = qk[I >> 1][I & 1][J] = qt[I >> 1][I & 1][J] = zero;
#pragma unroll 1
    for (int ks = 0; ks < KS; ++ks) {
      auto frag = [&](brsrc rs, int t) {
        Raw8<IO> x;
        x.load(rs, 32 * ks + 8 * q < N ? t * row + (32 * ks + 8 * q) * ES : kNoOffset);
        return raw_planes<IO>(x);
      };
      Planes<PI> kn[4];  // K, tiles 2B + t with rows 32B + rowof(t)
#pragma unroll
      for (int I = 0; I < 4; ++I) kn[I] = frag(rk, 16 * I + r);
      if (solves)
#pragma unroll
        for (int I = 0; I < 4; ++I)
#pragma unroll
          for (int J = 0; J <= I; ++J) kk[I][J] = mma<PM>(kn[J], kn[I], kk[I][J]);
      if (forms_p) {
        Planes<PI> kc[4], qx[4];  // K in row32's order, Q in rowof's and then in row32's
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          kc[i] = frag(rk, 32 * (i >> 1) + row32(r, i & 1));
          qx[i] = frag(rq, 32 * (i >> 1) + rowof(i & 1));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if ((j >> 1) <= (i >> 1)) qk[i >> 1][i & 1][j] = mma<PM>(kc[j], qx[i], qk[i >> 1][i & 1][j]);
        if constexpr (SAVE) {
#pragma unroll
          for (int i = 0; i < 4; ++i) qx[i] = frag(rq, 32 * (i >> 1) + row32(r, i & 1));
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if ((i >> 1) <= (j >> 1)) qt[i >> 1][i & 1][j] = mma<PM>(qx[j], kn[i], qt[i >> 1][i & 1][j]);
        }
      }
    }
  }

  for (int hh = part * hpw; hh < min(per, (part + 1) * hpw); ++hh) {
    const int h = grp * per + hh;
    const int64_t kh = (int64_t)ck * a.H + h;
    // gates: lane = token; past the chunk's end the decay stays and beta is zero
    const int64_t tok = (int64_t)start + lane;
    const float gv = lane < len ? min_gate(a.g[tok * a.H + h]) : 0.f;
    const float bv = lane < len ? a.beta[tok * a.H + h] : 0.f;
    double G = (double)gv * 1.4426950408889634073599;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double up = __shfl_up(G, d);
      if (lane >= d) G += up;
    }
    const float Gh = (float)G, Gl = (float)(G - (double)Gh);
    const float Ch = wave_last(Gh), Cl = wave_last(Gl);
    float* gt = a.gates + kh * kDeltaGates;
    if (solves) {
      gt[lane] = Gh;
      gt[C + lane] = Gl;
      gt[2 * C + lane] = bv;
      if constexpr (BF16) {
        const float eG = exp2_hl(Gh, Gl), eR = exp2_fast((Ch - Gh) + (Cl - Gl));
        gt[3 * C + lane] = eG;
        gt[4 * C + lane] = bv * eR;
        gt[5 * C + lane] = eR;
        gt[6 * C + lane] = bv * eG;
      }
    }
    __builtin_amdgcn_wave_barrier();
    gh[lane] = Gh;
    gl[lane] = Gl;
    bb[lane] = bv;
    __builtin_amdgcn_wave_barrier();

    if (solves) {
      // M, and its diagonal blocks in LDS where R's will be
      f32x4 m[4][4];
#pragma unroll
      for (int I = 0; I < 4; ++I) {
        const float hi = gh[16 * I + r], li = gl[16 * I + r];
#pragma unroll
        for (int J = 0; J <= I; ++J) {
          const f32x4 hj = *(const f32x4*)(gh + 16 * J + 4 * q), lj = *(const f32x4*)(gl + 16 * J + 4 * q);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float d = exp2_fast((hi - hj[e]) + (li - lj[e]));
            m[I][J][e] = J < I || 4 * q + e < r ? kk[I][J][e] * d : 0.f;
          }
        }
        *(f32x4*)(Rm + (16 * I + r) * kPrepLd + 16 * I + 4 * q) = m[I][I];
      }
      __builtin_amdgcn_wave_barrier();
      // diagonal blocks: lane (q, r) column r of block q; row i of R takes the place of row i
      // of M, which no later row reads
      {
        float* mb = Rm + 16 * q * kPrepLd + 16 * q;
        float br[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float s[2] = {mb[i * kPrepLd + r], 0.f};
#pragma unroll
          for (int j4 = 0; j4 < (i + 3) / 4; ++j4) {
            const f32x4 x = *(const f32x4*)(mb + i * kPrepLd + 4 * j4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (4 * j4 + e < i) s[e & 1] -= x[e] * br[4 * j4 + e];
          }
          const float x = s[0] + s[1];
          __builtin_amdgcn_wave_barrier();
          mb[i * kPrepLd + r] = x;
          br[i] = bb[16 * q + i] * x;
        }
        // the blocks right of the first and third diagonal ones are read with them
#pragma unroll
        for (int B = 0; B < 2; ++B)
          *(f32x4*)(Rm + (32 * B + r) * kPrepLd + 32 * B + 16 + 4 * q) = zero;
      }
      __builtin_amdgcn_wave_barrier();
      // the blocks below, column by column: br[K] = b_K R_KJ (K = J: minus the identity)
#pragma unroll
      for (int J = 0; J < 3; ++J) {
        f32x4 br[4];
        {
          const f32x4 b = *(const f32x4*)(bb + 16 * J + 4 * q);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            br[J][e] = b[e] * Rm[(16 * J + 4 * q + e) * kPrepLd + 16 * J + r] - (4 * q + e == r ? 1.f : 0.f);
        }
#pragma unroll
        for (int I = J + 1; I < 4; ++I) {
          f32x4 y = zero;
#pragma unroll
          for (int K = J; K < I; ++K)
#pragma unroll
            for (int e = 0; e < 4; ++e) y = mfma_f32(m[I][K][e], br[K][e], y);
          y = -y;
          const f32x4 b = *(const f32x4*)(bb + 16 * I + 4 * q);
          const f32x4 rd = *(const f32x4*)(Rm + (16 * I + r) * kPrepLd + 16 * I + 4 * q);
          const f32x4 by = b * y;
          f32x4 x = zero;
#pragma unroll
          for (int e = 0; e < 4; ++e) x = mfma_f32(rd[e], by[e], x);
          x = y - x;
          br[I] = b * x;
#pragma unroll
          for (int e = 0; e < 4; ++e) Rm[(16 * I + 4 * q + e) * kPrepLd + 16 * J + r] = x[e];
        }
      }
      __builtin_amdgcn_wave_barrier();
      {
        uint16_t* dst = a.R + kh * (PM * kTriPlane) + lane * 8;
        uint16_t* dt = SAVE ? a.Rt + kh * (PM * kTriPlane) + lane * 8 : nullptr;
#pragma unroll
        for (int B = 0; B < 2; ++B)
#pragma unroll
          for (int S = 0; S <= B; ++S)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              // bf16 io: forward R diag(b), backward (diag(b) R)^T
              const float* src = Rm + (32 * B + rowof(t)) * kPrepLd + 32 * S + 8 * q;
              const float* bc = bb + 32 * S + 8 * q;
              f32x4 x = *(const f32x4*)src, y = *(const f32x4*)(src + 4);
              if constexpr (BF16) {
                x *= *(const f32x4*)bc;
                y *= *(const f32x4*)(bc + 4);
              }
              u32x4 o[PM];
              split8<PM>(x, y, o);
#pragma unroll
              for (int i = 0; i < PM; ++i) *(u32x4*)(dst + i * kTriPlane + low_block(B, t, S) * 512) = o[i];
              if constexpr (SAVE) {
                src = Rm + (32 * B + 8 * q) * kPrepLd + 32 * S + rowof(t);
                bc = bb + 32 * B + 8 * q;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  x[e] = (BF16 ? bc[e] : 1.f) * src[e * kPrepLd];
                  y[e] = (BF16 ? bc[e + 4] : 1.f) * src[(e + 4) * kPrepLd];
                }
                split8<PM>(x, y, o);
#pragma unroll
                for (int i = 0; i < PM; ++i) *(u32x4*)(dt + i * kTriPlane + up_block(S, t, B) * 512) = o[i];
              }
            }
      }
    }
    // P and its transpose
    if (forms_p) {
      uint16_t* dst = a.Pm + kh * (PI * kTriPlane) + lane * 8;
      uint16_t* dt = SAVE ? a.Pt + kh * (PM * kTriPlane) + lane * 8 : nullptr;
#pragma unroll
      for (int B = 0; B < 2; ++B)
#pragma unroll
        for (int S = 0; S <= B; ++S)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int ro = rowof(t);
            f32x4 v[2];
            {
              const float hi = gh[32 * B + ro], li = gl[32 * B + ro];
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int c = 8 * q + 4 * u;
                const f32x4 hj = *(const f32x4*)(gh + 32 * S + c), lj = *(const f32x4*)(gl + 32 * S + c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float d = exp2_fast((hi - hj[e]) + (li - lj[e]));
                  v[u][e] = S < B || c + e <= ro ? a.scale * (qk[B][t][2 * S + u][e] * d) : 0.f;
                }
              }
              u32x4 o[PI];  // (bf16 io: one plane, the output is rounded to bf16)
              split8<PI>(v[0], v[1], o);
#pragma unroll
              for (int i = 0; i < PI; ++i) *(u32x4*)(dst + i * kTriPlane + low_block(B, t, S) * 512) = o[i];
            }
            if constexpr (SAVE) {
              const float hj = gh[32 * S + ro], lj = gl[32 * S + ro];
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int c = 8 * q + 4 * u;
                const f32x4 hi = *(const f32x4*)(gh + 32 * B + c), li = *(const f32x4*)(gl + 32 * B + c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float d = exp2_fast((hi[e] - hj) + (li[e] - lj));
                  v[u][e] = S < B || c + e >= ro ? a.scale * (qt[S][t][2 * B + u][e] * d) : 0.f;
                }
              }
              u32x4 o[PM];
              split8<PM>(v[0], v[1], o);
#pragma unroll
              for (int i = 0; i < PM; ++i) *(u32x4*)(dt + i * kTriPlane + up_block(S, t, B) * 512) = o[i];
            }
          }
    }
  }
}

hipError_t launch_delta_prep(const DeltaProb& p, const DeltaArgs& a, hipStream_t st) {
  if (p.nck == 0) return hipSuccess;
  // Heads a wave, which share K K^T and Q K^T, while the waves still fill the chip (2048 at once:
  // 256 registers each).  Us with one | two | four heads: 64 chunks and heads 16 | 22 | 33, 1088
  // with P and its transpose 29 | 29 | 44, 16384 so 254 | 188 | 161, 65536 706 | 492 | 417.
  // R and P by two waves where all are there at once: 64 chunks and heads 12 us instead of 16,
  // 512 of fp32 io 16 instead of 22, 16384 209 instead of 188.
  const int64_t all = p.nck * p.H;
  const int per = p.H / p.G, hpw = std::min(per, all >= 16384 ? 4 : all >= 1024 ? 2 : 1);
  const int64_t items = p.nck * p.G * ((per + hpw - 1) / hpw);
  const int roles = items <= 2048 ? 2 : 1;
  const dim3 grid((unsigned)((items * roles + 3) / 4)), block(256);
  auto go = [&](auto n, auto io) {
    constexpr int N = decltype(n)::value;
    using IO = decltype(io);
    if (a.Rt)
      hipLaunchKernelGGL((delta_prep_kernel<N, IO, true>), grid, block, 0, st, a, hpw, roles, items);
    else
      hipLaunchKernelGGL((delta_prep_kernel<N, IO, false>), grid, block, 0, st, a, hpw, roles, items);
  };
  auto pick = [&](auto io) {
    switch (p.N) {
      case 16: go(std::integral_constant<int, 16>{}, io); break;
      case 32: go(std::integral_constant<int, 32>{}, io); break;
      case 64: go(std::integral_constant<int, 64>{}, io); break;
      default: go(std::integral_constant<int, 128>{}, io); break;
    }
  };
  p.io ? pick(IoBf16{}) : pick(IoF32{});
  return hipGetLastError();
}

}  // namespace ssd
