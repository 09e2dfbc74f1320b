// Gated delta rule, bf16 io, backward chain: the reverse walk over one sequence's chunks
// for 16 columns of headdim of one head a wave, with the adjoint dS of the state leaving
// the chunk in registers, from what the forward kept (R and P transposed, the gates).
// With U = b Z and O = scale exp(G) Q S^T + P U, per chunk:
//   E = P^T dO + exp(G_C - G) K dS^T          (adjoint of U)
//   F = E - R^T (b E),   dX = b F = dV         (adjoints of U in full, and of X)
//   dS <- exp(G_C) dS + (scale exp(G) dO)^T Q - (exp(G) dX)^T K
// F and the dS of every chunk are stored for k_delta_grads.hip, which forms the other
// gradients chunk by chunk.  Registers, staging and the split over waves are those of
// k_delta_fwd.hip; two planes throughout.
#include "delta_reg.hpp"

namespace ssd {

template <int N, int NS>
__global__ __launch_bounds__(256, 1) void delta_bwd_kernel(DeltaArgs a, int ptiles) {
  constexpr int C = kDeltaChunk, NP = N < 32 ? 32 : N, KS = NP / 32, KW = (KS + NS - 1) / NS, NPT = 4 / NS;
  constexpr int LK = NP + 8, LV = 16 * NPT + 8;
  constexpr int EK = C * LK, ER = 2 * kTriPlane, EV = C * LV;
  struct Buf {
    uint16_t K[EK], Q[EK], R[ER], P[ER], O[EV];
    float g[3 * C];  // beta, exp(G), exp(G_C - G)
  };
  __shared__ __align__(16) Buf buf[2];
  constexpr int XCH = NS > 1 ? NPT * NS * 4 * 64 : 1;
  __shared__ __align__(16) f32x4 xk[XCH];

  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, q = lane >> 4, r = lane & 15;
  const int pt = w / NS, ns = w % NS;
  const int np = (ptiles + NPT - 1) / NPT;
  const int wg = xcd_order(blockIdx.x, gridDim.x);
  const int pg = wg % np, h = (wg / np) % a.H, s = wg / np / a.H;
  const int p0 = pg * 16 * NPT;
  const int pw = 16 * min(NPT, ptiles - pg * NPT);
  const bool live = 16 * pt < pw;
  const int pc = p0 + 16 * pt + r;
  const int grp = h / (a.H / a.G);
  const SeqSpan sp = seq_span(a.map, s);
  const int c0 = sp.c0, c1 = sp.c1;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  f32x4 S[KW][2];
  const int64_t srow = (((int64_t)s * a.H + h) * a.P + pc) * N;
  auto scol = [&](int k, int t) { return 32 * (ns * KW + k) + 8 * q + 4 * t; };
#pragma unroll
  for (int k = 0; k < KW; ++k)
#pragma unroll
    for (int t = 0; t < 2; ++t)
      S[k][t] = a.d_final && live && scol(k, t) < N ? *(const f32x4*)(a.d_final + srow + scol(k, t)) : zero;

  if constexpr (N < 32) {
    for (int e = tid; e < 2 * C; e += 256)
      for (int c = N; c < 32; c += 4) {
        *(uint2*)(buf[e / C].K + (e % C) * LK + c) = make_uint2(0u, 0u);
        *(uint2*)(buf[e / C].Q + (e % C) * LK + c) = make_uint2(0u, 0u);
      }
  }

  constexpr int KC = (C * N / 8 + 255) / 256, RC = ER / 8 / 256, VP = 2 * NPT, VC = (C * VP + 255) / 256;
  struct Loads {
    u32x4 k[KC], q[KC], R[RC], P[RC], o[VC];
    float g;
  };
  auto load = [&](Loads& x, int c) {
    const int start = sp.start + (c - c0) * C, len = min(C, sp.end - start);
    const uint32_t row = (uint32_t)a.G * N * 2, span = (uint32_t)(len - 1) * row + N * 2;
    const int64_t base = ((int64_t)start * a.G + grp) * N * 2;
    const brsrc rk = make_rsrc((const char*)a.k + base, span), rq = make_rsrc((const char*)a.q + base, span);
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int e = tid + i * 256;
      const uint32_t off = e < C * N / 8 ? (e / (N / 8)) * row + (e % (N / 8)) * 16 : kNoOffset;
      x.k[i] = buf_load16(rk, off);
      x.q[i] = buf_load16(rq, off);
    }
    const int64_t kh = (int64_t)c * a.H + h;
    const brsrc rr = make_rsrc(a.Rt + kh * ER, ER * 2), rp = make_rsrc(a.Pt + kh * ER, ER * 2);
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      x.R[i] = buf_load16(rr, (tid + i * 256) * 16);
      x.P[i] = buf_load16(rp, (tid + i * 256) * 16);
    }
    const uint32_t vrow = (uint32_t)a.H * a.P * 2;
    const brsrc ro = make_rsrc((const char*)a.dout + (((int64_t)start * a.H + h) * a.P + p0) * 2,
                               (uint32_t)(len - 1) * vrow + pw * 2);
#pragma unroll
    for (int i = 0; i < VC; ++i) {
      const int e = tid + i * 256;
      x.o[i] = buf_load16(ro, e < C * VP && 8 * (e % VP) < pw ? (e / VP) * vrow + (e % VP) * 16 : kNoOffset);
    }
    x.g = tid < 3 * C ? a.gates[kh * kDeltaGates + 2 * C + tid] : 0.f;
  };
  auto put = [&](const Loads& x, Buf& b) {
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int e = tid + i * 256;
      if (e < C * N / 8) {
        *(u32x4*)(b.K + (e / (N / 8)) * LK + (e % (N / 8)) * 8) = x.k[i];
        *(u32x4*)(b.Q + (e / (N / 8)) * LK + (e % (N / 8)) * 8) = x.q[i];
      }
    }
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      *(u32x4*)(b.R + (tid + i * 256) * 8) = x.R[i];
      *(u32x4*)(b.P + (tid + i * 256) * 8) = x.P[i];
    }
#pragma unroll
    for (int i = 0; i < VC; ++i) {
      const int e = tid + i * 256;
      if (e < C * VP) *(u32x4*)(b.O + (e / VP) * LV + (e % VP) * 8) = x.o[i];
    }
    if (tid < 3 * C) b.g[tid] = x.g;
  };

  Loads x;
  if (c0 < c1) {
    load(x, c1 - 1);
    put(x, buf[0]);
    if (c1 - 2 >= c0) load(x, c1 - 2);
  }
  __syncthreads();
  for (int c = c1 - 1; c >= c0; --c) {
    const Buf& b = buf[(c1 - 1 - c) & 1];
    const int64_t kh = (int64_t)c * a.H + h;
    f32x4 ks[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) ks[i >> 1][i & 1] = zero;
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const int kk = ns * KW + k;
      if (KS % NS == 0 || kk < KS) {
        const Planes<2> sf = tile_planes<2>(S[k][0], S[k][1]);
        if (live)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (scol(k, t) < N) *(f32x4*)(a.dS + (kh * a.P + pc) * N + scol(k, t)) = S[k][t];
#pragma unroll
        for (int B = 0; B < 2; ++B)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            ks[B][t] = mma1<2>(as_bf16x8(*(const u32x4*)(b.K + (32 * B + row32(r, t)) * LK + 32 * kk + 8 * q)), sf, ks[B][t]);
      }
    }
    if constexpr (NS > 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) xk[((pt * NS + ns) * 4 + i) * 64 + lane] = ks[i >> 1][i & 1];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 y = xk[(pt * NS * 4 + i) * 64 + lane];
#pragma unroll
        for (int j = 1; j < NS; ++j) y += xk[((pt * NS + j) * 4 + i) * 64 + lane];
        ks[i >> 1][i & 1] = y;
      }
    }
    auto tri = [&](const uint16_t* m, int S2, int t, int B) {
      Planes<2> f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        f.p[i] = as_bf16x8(*(const u32x4*)(m + i * kTriPlane + up_block(S2, t, B) * 512 + lane * 8));
      return f;
    };
    // E: tile (B, t) has tokens 32B + 8q + 4t + e
    f32x4 E[2][2], bt[2][2], eg[2][2];
    Planes<2> ef[2], of2[2];
    bf16x8 of[2];
#pragma unroll
    for (int B = 0; B < 2; ++B) of[B] = frag_kmajor(b.O + 32 * B * LV + 16 * pt, LV, lane);
#pragma unroll
    for (int B = 0; B < 2; ++B) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int tk = 32 * B + 8 * q + 4 * t;
        bt[B][t] = *(const f32x4*)(b.g + tk);
        eg[B][t] = *(const f32x4*)(b.g + C + tk);
        f32x4 e = *(const f32x4*)(b.g + 2 * C + tk) * ks[B][t];
#pragma unroll
        for (int B2 = 1; B2 >= B; --B2) e = mma1t<2>(tri(b.P, B, t, B2), of[B2], e);
        E[B][t] = e;
      }
      ef[B] = tile_planes<2>(bt[B][0] * E[B][0], bt[B][1] * E[B][1]);
      const u32x4 ow = __builtin_bit_cast(u32x4, of[B]);
      f32x4 o[2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
        o[t] = (a.scale * eg[B][t]) *
               f32x4{bf_lo(ow[2 * t]), bf_hi(ow[2 * t]), bf_lo(ow[2 * t + 1]), bf_hi(ow[2 * t + 1])};
      of2[B] = tile_planes<2>(o[0], o[1]);
    }
    const int start = sp.start + (c - c0) * C, len = min(C, sp.end - start);
    uint16_t* dv = (uint16_t*)a.dv + ((int64_t)start * a.H + h) * a.P + pc;
    Planes<2> wf[2];
#pragma unroll
    for (int B = 0; B < 2; ++B) {
      f32x4 wv[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 f = zero;
#pragma unroll
        for (int B2 = 1; B2 >= B; --B2) f = mma<2>(tri(b.R, B, t, B2), ef[B2], f);
        f = E[B][t] - f;
        const f32x4 dx = bt[B][t] * f;
        wv[t] = -eg[B][t] * dx;
        if (live && (NS == 1 || (2 * B + t) % NS == ns)) {
          const int tk = 32 * B + 8 * q + 4 * t;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a.F[(kh * C + tk + e) * a.P + pc] = f[e];
            if (tk + e < len) dv[(int64_t)(tk + e) * a.H * a.P] = f2bf(dx[e]);
          }
        }
      }
      wf[B] = tile_planes<2>(wv[0], wv[1]);
    }
    const float eC = b.g[C + C - 1];
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const int kk = ns * KW + k;
      if (KS % NS == 0 || kk < KS) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          f32x4 y = eC * S[k][t];
#pragma unroll
          for (int B = 0; B < 2; ++B) {
            y = mma1<2>(cols32(b.Q + 32 * B * LK + 32 * kk, LK, t, lane), of2[B], y);
            y = mma1<2>(cols32(b.K + 32 * B * LK + 32 * kk, LK, t, lane), wf[B], y);
          }
          S[k][t] = y;
        }
      }
    }
    if (c > c0) {
      put(x, buf[(c1 - c) & 1]);
      if (c - 2 >= c0) load(x, c - 2);
    }
    __syncthreads();
  }
  if (a.d_init && live) {
#pragma unroll
    for (int k = 0; k < KW; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (scol(k, t) < N) *(f32x4*)(a.d_init + srow + scol(k, t)) = S[k][t];
  }
}

hipError_t launch_delta_bwd_chain(const DeltaProb& p, const DeltaArgs& a, hipStream_t st) {
  if (!p.io) return launch_delta_f32_bwd(p, a, st);
  if (p.nst == 0) return hipSuccess;
  const int ptiles = p.P / 16;
  const int64_t heads = (int64_t)p.nst * p.H;
  auto go = [&](auto n, auto ns) {
    constexpr int NS = decltype(ns)::value, NPT = 4 / NS;
    hipLaunchKernelGGL((delta_bwd_kernel<decltype(n)::value, NS>),
                       dim3((unsigned)(heads * ((ptiles + NPT - 1) / NPT))), dim3(256), 0, st, a, ptiles);
  };
  auto pick = [&](auto n) {
    const int64_t tiles = heads * ptiles;
    if (tiles >= 512 && ptiles >= 4)
      go(n, std::integral_constant<int, 1>{});
    else if (tiles >= 256 && ptiles >= 2)
      go(n, std::integral_constant<int, 2>{});
    else
      go(n, std::integral_constant<int, 4>{});
  };
  switch (p.N) {
    case 16: pick(std::integral_constant<int, 16>{}); break;
    case 32: pick(std::integral_constant<int, 32>{}); break;
    case 64: pick(std::integral_constant<int, 64>{}); break;
    default: pick(std::integral_constant<int, 128>{}); break;
  }
  return hipGetLastError();
}

}  // namespace ssd
