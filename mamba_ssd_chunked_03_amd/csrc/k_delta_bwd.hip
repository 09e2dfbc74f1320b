// Gated delta rule, bf16 io, backward chain: the reverse walk over one sequence's chunks
// for 16 columns of headdim of one head, with the adjoint dS of the state leaving the
// chunk, from what the forward kept (R and P transposed, the gates).  With U = b Z and
// O = scale exp(G) Q S^T + P U, per chunk:
//   E = P^T dO + exp(G_C - G) K dS^T          (adjoint of U)
//   F = E - (b R)^T E,   dX = b F = dV         (adjoints of U in full, and of X)
//   dS <- exp(G_C) dS + (scale exp(G) dO)^T Q - (exp(G) dX)^T K
// F and the dS of every chunk are stored for k_delta_grads.hip, which forms the gradients
// chunk by chunk.  Registers, waves and tiles as in k_delta_fwd.hip.  The helper waves form
// what does not wait for dS a chunk ahead: E0 = P^T dO and T = (scale exp(G) dO)^T Q.
//   interval A(c)  chain: K dS^T, E                 helpers: T(c), Q, P, dO(c - 1) to LDS
//   interval B(c)  chain: (b R)^T E, F, the new dS   helpers: K, R(c - 1) to LDS, E0, T of c - 1
// Two planes throughout (the error of dS is not a result: 3e-6 of the gradients).
// 2 x 8192 tokens of 64 heads of 64 x 128: 380 us (one wave a tile, four tiles: 440), of
// which dS and F written (805 MB) are 160 at the rate of a large copy.
#include "delta_reg.hpp"

namespace ssd {

template <int N, int NPT>
__global__ __launch_bounds__(64 * NPT * kSplit<N> + 256, 1) void delta_bwd_kernel(DeltaArgs a, int ptiles) {
  constexpr int C = kDeltaChunk, NP = N < 32 ? 32 : N, KS = NP / 32, SPLIT = kSplit<N>, CW = NPT * SPLIT;
  constexpr int KH = KS / SPLIT;  // blocks of 32 columns of the state a chain wave holds
  using Tile = TokTile<NP>;
  constexpr int LV = 16 * NPT + 8, EV = C * LV, ER = 2 * kTriPlane;
  __shared__ __align__(16) uint16_t Kl[2][Tile::SIZE], Ql[Tile::SIZE], Rl[2][ER], Pl[ER], Ol[EV];
  __shared__ __align__(16) float gl[2][3 * C];  // exp(G), exp(G_C - G), beta exp(G)
  __shared__ __align__(16) f32x4 Ex[NPT][4][64], Tx[NPT][KS][2][64];  // E0 and T, tile order
  __shared__ __align__(16) f32x4 Kx[SPLIT == 2 ? NPT : 1][SPLIT][4][64];  // parts of K dS^T

  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, q = lane >> 4, r = lane & 15;
  const int np = ptiles / NPT;
  int s, wg;
  chain_order(a.H * np, s, wg);
  const int pg = wg % np, h = wg / np;
  const int p0 = pg * 16 * NPT;
  const int grp = h / (a.H / a.G);
  const SeqSpan sp = seq_span(a.map, s);
  const int c0 = sp.c0, c1 = sp.c1;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  if (w < CW) {
    // ------------------------------------------------------------ chain wave ----
    const int tw = w / SPLIT, half = w % SPLIT, kb = half * KH;
    const int pc = p0 + 16 * tw + r;
    f32x4 S[KH][2];  // columns 32(kb + k) + 8q + 4t + e of row pc
    const int64_t srow = (((int64_t)s * a.H + h) * a.P + pc) * N;
    auto scol = [&](int k, int t) { return 32 * (kb + k) + 8 * q + 4 * t; };
#pragma unroll
    for (int k = 0; k < KH; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        S[k][t] = a.d_final && scol(k, t) < N ? *(const f32x4*)(a.d_final + srow + scol(k, t)) : zero;
    f32x4* kS = (f32x4*)a.dS + (int64_t)(pc >> 4) * (KS * 2) * 64 + lane;  // of chunk slot 0
    f32x4* kF = (f32x4*)a.F + (int64_t)(pc >> 4) * 4 * 64 + lane;
    __syncthreads();
    __syncthreads();
    if constexpr (SPLIT == 2) {
      for (int c = c1 - 1; c >= c0; --c) {
        const uint16_t* K = Kl[(c1 - 1 - c) & 1];
        const float* g = gl[(c1 - 1 - c) & 1];
        const int64_t kh = (int64_t)c * a.H + h;
        // interval A: this half's part of K dS^T
        f32x4 ks[4], E[4], er[4], wg4[4];
        Planes<2> ef[2], Rf[6], sf[KH];
        bf16x8 kt[KH][2][2], kf[KH][4];
        const float eC = g[C - 1];
#pragma unroll
        for (int k = 0; k < KH; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) kf[k][i] = tok_rows<NP>(K, 32 * (i >> 1), i & 1, 32 * (kb + k), lane);
        sf[0] = tile_planes<2>(S[0][0], S[0][1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ks[i] = zero;
          E[i] = Ex[tw][i][lane];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < KH; ++k) {
#pragma unroll
          for (int m = 1; m >= 0; --m)
#pragma unroll
            for (int i = 0; i < 4; ++i) ks[i] = mfma_bf16(kf[k][i], sf[k].p[m], ks[i]);
          if (k + 1 < KH) sf[k + 1] = tile_planes<2>(S[k + 1][0], S[k + 1][1]);
#pragma unroll
          for (int t = 0; t < 2; ++t) kS[(kh * (a.P / 16) * (KS * 2) + (kb + k) * 2 + t) * 64] = S[k][t];
          if (k + 1 == KH) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              er[i] = *(const f32x4*)(g + C + 32 * (i >> 1) + 8 * q + 4 * (i & 1));
              wg4[i] = *(const f32x4*)(g + 2 * C + 32 * (i >> 1) + 8 * q + 4 * (i & 1));
            }
#pragma unroll
            for (int i = 0; i < 6; ++i)
#pragma unroll
              for (int m = 0; m < 2; ++m)
                Rf[i].p[m] = as_bf16x8(*(const u32x4*)(Rl[(c1 - 1 - c) & 1] + m * kTriPlane + i * 512 + lane * 8));
          }
          interleave<8, 3>();
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) Kx[tw][half][i][lane] = ks[i];
#pragma unroll
        for (int k = 0; k < KH; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int B = 0; B < 2; ++B) kt[k][t][B] = tok_cols<NP>(K, 32 * B, t, 32 * (kb + k), lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) E[i] += er[i] * ks[i];
        __syncthreads();
        // interval B: E from both parts and F (each wave forms all of them, to the order of one
        // sum), and this half of the new dS
        f32x4 F[4], kx[4];
#pragma unroll
        for (int i = 3; i >= 0; --i) kx[i] = Kx[tw][1 - half][i][lane];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) F[i] = zero;
#pragma unroll
        for (int i = 2; i < 4; ++i) E[i] += er[i] * kx[i];
        ef[1] = tile_planes<2>(E[2], E[3]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < 3; ++m) {
#pragma unroll
          for (int t = 0; t < 2; ++t) F[2 + t] = mfma_bf16(Rf[up_block(1, t, 1)].p[m == 0], ef[1].p[m == 1], F[2 + t]);
#pragma unroll
          for (int t = 0; t < 2; ++t) F[t] = mfma_bf16(Rf[up_block(0, t, 1)].p[m == 0], ef[1].p[m == 1], F[t]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) E[i] += er[i] * kx[i];
        ef[0] = tile_planes<2>(E[0], E[1]);
        interleave<12, 3>();
        __builtin_amdgcn_sched_barrier(0);
        Planes<2> wf[2];
        auto form_w = [&](int B) {
          f32x4 wv[2];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int i = 2 * B + t;
            F[i] = E[i] - F[i];
            if (B == half) kF[(kh * (a.P / 16) * 4 + i) * 64] = F[i];
            wv[t] = -(wg4[i] * F[i]);
          }
          wf[B] = tile_planes<2>(wv[0], wv[1]);
        };
#pragma unroll
        for (int m = 0; m < 3; ++m)
#pragma unroll
          for (int t = 0; t < 2; ++t) F[t] = mfma_bf16(Rf[up_block(0, t, 0)].p[m == 0], ef[0].p[m == 1], F[t]);
#pragma unroll
        for (int k = 0; k < KH; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) S[k][t] = eC * S[k][t] + Tx[tw][kb + k][t][lane];
        form_w(1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int B = 1; B >= 0; --B) {
#pragma unroll
          for (int m = 1; m >= 0; --m)
#pragma unroll
            for (int k = 0; k < KH; ++k)
#pragma unroll
              for (int t = 0; t < 2; ++t) S[k][t] = mfma_bf16(kt[k][t][B], wf[B].p[m], S[k][t]);
          if (B == 1) form_w(0);
          interleave<4 * KH, 4>();
          __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
      }
    } else {
      for (int c = c1 - 1; c >= c0; --c) {
        const uint16_t* K = Kl[(c1 - 1 - c) & 1];
        const float* g = gl[(c1 - 1 - c) & 1];
        const int64_t kh = (int64_t)c * a.H + h;
        // interval A: E, tile i = 2B + t with tokens 32B + 8q + 4t + e; block 1 of the tokens with
        // dS's planes on the way, block 0 with E of block 1
        f32x4 ks[4], E[4], er[4], wg4[4];
        Planes<2> ef[2], Rf[6];
        bf16x8 kt[KS][2][2];  // K^T, by block of tokens
        const float eC = g[C - 1];
        bf16x8 kf[KS][2], kg[KS][2];
        Planes<2> sf[KS];
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) kf[k][t] = tok_rows<NP>(K, 32, t, 32 * k, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ks[i] = zero;
          E[i] = Ex[w][i][lane];
          er[i] = *(const f32x4*)(g + C + 32 * (i >> 1) + 8 * q + 4 * (i & 1));
          wg4[i] = *(const f32x4*)(g + 2 * C + 32 * (i >> 1) + 8 * q + 4 * (i & 1));
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) kg[k][t] = tok_rows<NP>(K, 0, t, 32 * k, lane);
        sf[0] = tile_planes<2>(S[0][0], S[0][1]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
#pragma unroll
          for (int m = 1; m >= 0; --m)
#pragma unroll
            for (int t = 0; t < 2; ++t) ks[2 + t] = mfma_bf16(kf[k][t], sf[k].p[m], ks[2 + t]);
          if (k + 1 < KS) sf[k + 1] = tile_planes<2>(S[k + 1][0], S[k + 1][1]);
#pragma unroll
          for (int t = 0; t < 2; ++t) kS[(kh * (a.P / 16) * (KS * 2) + k * 2 + t) * 64] = S[k][t];
          interleave<4, 4>();
          __builtin_amdgcn_sched_barrier(0);
        }
        auto form_e = [&](int B) {
#pragma unroll
          for (int i = 2 * B; i < 2 * B + 2; ++i) E[i] += er[i] * ks[i];
          ef[B] = tile_planes<2>(E[2 * B], E[2 * B + 1]);
        };
        // (and what the next interval starts with)
#pragma unroll
        for (int i = 0; i < 6; ++i)
#pragma unroll
          for (int m = 0; m < 2; ++m)
            Rf[i].p[m] = as_bf16x8(*(const u32x4*)(Rl[(c1 - 1 - c) & 1] + m * kTriPlane + i * 512 + lane * 8));
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) kt[k][t][1] = tok_cols<NP>(K, 32, t, 32 * k, lane);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int m = 1; m >= 0; --m)
#pragma unroll
            for (int t = 0; t < 2; ++t) ks[t] = mfma_bf16(kg[k][t], sf[k].p[m], ks[t]);
        form_e(1);
        interleave<4 * KS, 3>();
        __builtin_amdgcn_sched_barrier(0);
        form_e(0);
        __syncthreads();
        // interval B: F = E - (b R)^T E, by planes, with dS's decay on the way
        f32x4 F[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) F[i] = zero;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) kt[k][t][0] = tok_cols<NP>(K, 0, t, 32 * k, lane);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < 3; ++m)
#pragma unroll
          for (int t = 0; t < 2; ++t) F[2 + t] = mfma_bf16(Rf[up_block(1, t, 1)].p[m == 0], ef[1].p[m == 1], F[2 + t]);
#pragma unroll
        for (int B2 = 1; B2 >= 0; --B2)
#pragma unroll
          for (int m = 0; m < 3; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t) F[t] = mfma_bf16(Rf[up_block(0, t, B2)].p[m == 0], ef[B2].p[m == 1], F[t]);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) S[k][t] = eC * S[k][t] + Tx[w][k][t][lane];
        interleave<18, 2>();
        __builtin_amdgcn_sched_barrier(0);
        Planes<2> wf[2];
        auto form_w = [&](int B) {
          f32x4 wv[2];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int i = 2 * B + t;
            F[i] = E[i] - F[i];
            kF[(kh * (a.P / 16) * 4 + i) * 64] = F[i];
            wv[t] = -(wg4[i] * F[i]);
          }
          wf[B] = tile_planes<2>(wv[0], wv[1]);
        };
        form_w(1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int B = 1; B >= 0; --B) {
#pragma unroll
          for (int m = 1; m >= 0; --m)
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int t = 0; t < 2; ++t) S[k][t] = mfma_bf16(kt[k][t][B], wf[B].p[m], S[k][t]);
          if (B == 1) form_w(0);
          interleave<4 * KS, 2>();
          __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
      }
    }
    if (a.d_init) {
#pragma unroll
      for (int k = 0; k < KH; ++k)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (scol(k, t) < N) *(f32x4*)(a.d_init + srow + scol(k, t)) = S[k][t];
    }
    return;
  }

  // --------------------------------------------------------------- helper wave ----
  // (of a tile: HT blocks of 16 tokens of E0 and TK blocks of 32 columns of T a wave)
  constexpr int HT = NPT, TK = KS * NPT < 4 ? 1 : KS * NPT / 4;
  const int ht = tid - 64 * CW, tile = (w - CW) % NPT, i0 = (w - CW) / NPT * HT, k0 = (w - CW) / NPT * TK;
  const bool sums = k0 < KS;
  if constexpr (N < 32) {
    for (int e = ht; e < C; e += 256)
      for (int c = N; c < 32; c += 4) {
        *(uint2*)(Kl[0] + Tile::at(e, c)) = make_uint2(0u, 0u);
        *(uint2*)(Kl[1] + Tile::at(e, c)) = make_uint2(0u, 0u);
        *(uint2*)(Ql + Tile::at(e, c)) = make_uint2(0u, 0u);
      }
  }
  constexpr int KC = (C * N / 8 + 255) / 256, RC = ER / 8 / 256, VP = 2 * NPT, VC = (C * VP + 255) / 256;
  constexpr bool KX = C * N / 8 % 256 == 0, VX = C * VP % 256 == 0;
  u32x4 xk[KC], xq[KC], xr[RC], xp[RC], xo[VC];
  float xg;
  auto krsrc = [&](const void* p, int c, uint32_t& row) {
    const int start = sp.start + (c - c0) * C, len = min(C, sp.end - start);
    row = (uint32_t)a.G * N * 2;
    return make_rsrc((const char*)p + ((int64_t)start * a.G + grp) * N * 2, (uint32_t)(len - 1) * row + N * 2);
  };
  auto load_k = [&](int c) {
    uint32_t row;
    const brsrc rk = krsrc(a.k, c, row);
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int e = ht + i * 256;
      xk[i] = buf_load16(rk, KX || e < C * N / 8 ? (e / (N / 8)) * row + (e % (N / 8)) * 16 : kNoOffset);
    }
  };
  auto load_r = [&](int c) {
    const brsrc rr = make_rsrc(a.Rt + ((int64_t)c * a.H + h) * ER, ER * 2);
#pragma unroll
    for (int i = 0; i < RC; ++i) xr[i] = buf_load16(rr, (ht + i * 256) * 16);
  };
  auto load_ahead = [&](int c) {
    uint32_t row;
    const brsrc rq = krsrc(a.q, c, row);
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int e = ht + i * 256;
      xq[i] = buf_load16(rq, KX || e < C * N / 8 ? (e / (N / 8)) * row + (e % (N / 8)) * 16 : kNoOffset);
    }
    const int start = sp.start + (c - c0) * C, len = min(C, sp.end - start);
    const uint32_t vrow = (uint32_t)a.H * a.P * 2;
    const brsrc ro = make_rsrc((const char*)a.dout + (((int64_t)start * a.H + h) * a.P + p0) * 2,
                               (uint32_t)(len - 1) * vrow + 32 * NPT);
#pragma unroll
    for (int i = 0; i < VC; ++i) {
      const int e = ht + i * 256;
      xo[i] = buf_load16(ro, VX || e < C * VP ? (e / VP) * vrow + (e % VP) * 16 : kNoOffset);
    }
    const int64_t kh = (int64_t)c * a.H + h;
    const brsrc rp = make_rsrc(a.Pt + kh * ER, ER * 2);
#pragma unroll
    for (int i = 0; i < RC; ++i) xp[i] = buf_load16(rp, (ht + i * 256) * 16);
    const int gi = ht < C ? 3 * C + ht : 4 * C + ht;  // exp(G); exp(G_C - G), beta exp(G)
    xg = buf_load_f32(make_rsrc(a.gates + kh * kDeltaGates, kDeltaGates * 4), gi * 4);
  };
  auto put_k = [&](int buf) {
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int e = ht + i * 256;
      if (KX || e < C * N / 8) *(u32x4*)(Kl[buf] + Tile::at(e / (N / 8), (e % (N / 8)) * 8)) = xk[i];
    }
  };
  auto put_r = [&](int buf) {
#pragma unroll
    for (int i = 0; i < RC; ++i) *(u32x4*)(Rl[buf] + (ht + i * 256) * 8) = xr[i];
  };
  auto put_ahead = [&](int buf) {  // what the helpers read, and the gates
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int e = ht + i * 256;
      if (KX || e < C * N / 8) *(u32x4*)(Ql + Tile::at(e / (N / 8), (e % (N / 8)) * 8)) = xq[i];
    }
#pragma unroll
    for (int i = 0; i < RC; ++i) *(u32x4*)(Pl + (ht + i * 256) * 8) = xp[i];
#pragma unroll
    for (int i = 0; i < VC; ++i) {
      const int e = ht + i * 256;
      if (VX || e < C * VP) *(u32x4*)(Ol + (e / VP) * LV + (e % VP) * 8) = xo[i];
    }
    if (ht < 3 * C) gl[buf][ht] = xg;
  };
  f32x4 T[TK][2];
  // E0 (to LDS) and T (kept) of the chunk in Pl, Ol, Ql
  auto ahead = [&](int buf) {
    const float* g = gl[buf];
    Planes<2> Pf[HT][2], df[2];
    bf16x8 of[2];
#pragma unroll
    for (int B = 0; B < 2; ++B) of[B] = frag_kmajor(Ol + 32 * B * LV + 16 * tile, LV, lane);
#pragma unroll
    for (int ii = 0; ii < HT; ++ii)
#pragma unroll
      for (int B2 = 0; B2 < 2; ++B2) {
        const int i = i0 + ii;
        if (B2 || i < 2)
#pragma unroll
          for (int m = 0; m < 2; ++m)
            Pf[ii][B2].p[m] =
                as_bf16x8(*(const u32x4*)(Pl + m * kTriPlane + up_block(i >> 1, i & 1, B2) * 512 + lane * 8));
      }
    f32x4 e0[HT];
#pragma unroll
    for (int ii = 0; ii < HT; ++ii) e0[ii] = zero;
#pragma unroll
    for (int m = 1; m >= 0; --m)
#pragma unroll
      for (int B2 = 1; B2 >= 0; --B2)
#pragma unroll
        for (int ii = 0; ii < HT; ++ii)
          if (B2 || i0 + ii < 2) e0[ii] = mfma_bf16(Pf[ii][B2].p[m], of[B2], e0[ii]);
#pragma unroll
    for (int ii = 0; ii < HT; ++ii) Ex[tile][i0 + ii][lane] = e0[ii];
    if (!sums) return;
#pragma unroll
    for (int B = 0; B < 2; ++B) {
      const u32x4 ow = __builtin_bit_cast(u32x4, of[B]);
      f32x4 d[2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
        d[t] = (a.scale * *(const f32x4*)(g + 32 * B + 8 * q + 4 * t)) *
               f32x4{bf_lo(ow[2 * t]), bf_hi(ow[2 * t]), bf_lo(ow[2 * t + 1]), bf_hi(ow[2 * t + 1])};
      df[B] = tile_planes<2>(d[0], d[1]);
    }
#pragma unroll
    for (int k = 0; k < TK; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t) T[k][t] = zero;
#pragma unroll
    for (int B = 0; B < 2; ++B) {
      bf16x8 qf[TK][2];
#pragma unroll
      for (int k = 0; k < TK; ++k)
#pragma unroll
        for (int t = 0; t < 2; ++t) qf[k][t] = tok_cols<NP>(Ql, 32 * B, t, 32 * (k0 + k), lane);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 1; m >= 0; --m)
#pragma unroll
        for (int k = 0; k < TK; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) T[k][t] = mfma_bf16(qf[k][t], df[B].p[m], T[k][t]);
    }
  };
  // (The loads run on to the first chunk again instead of stopping under a branch, at whose
  // join they would be waited for.)
  if (c0 < c1) {
    load_ahead(c1 - 1);
    load_k(c1 - 1);
    load_r(c1 - 1);
    put_ahead(0);
    put_k(0);
    put_r(0);
    load_ahead(max(c1 - 2, c0));
    load_k(max(c1 - 2, c0));
    load_r(max(c1 - 2, c0));
  }
  __syncthreads();
  if (c0 < c1) ahead(0);
  __syncthreads();
  for (int c = c1 - 1; c >= c0; --c) {
    const int nb = (c1 - c) & 1;  // the next chunk's buffer
    // interval A
    if (sums) {
#pragma unroll
      for (int k = 0; k < TK; ++k)
#pragma unroll
        for (int t = 0; t < 2; ++t) Tx[tile][k0 + k][t][lane] = T[k][t];
    }
    put_ahead(nb);
    load_ahead(max(c - 2, c0));
    __syncthreads();
    // interval B
    put_k(nb);
    put_r(nb);
    load_k(max(c - 2, c0));
    load_r(max(c - 2, c0));
    ahead(nb);
    __syncthreads();
  }
}

hipError_t launch_delta_bwd_chain(const DeltaProb& p, const DeltaArgs& a, hipStream_t st) {
  if (!p.io) return launch_delta_f32_bwd(p, a, st);
  if (p.nst == 0) return hipSuccess;
  const int ptiles = p.P / 16;
  const int64_t heads = (int64_t)p.nst * p.H;
  auto go = [&](auto n, auto npt) {
    constexpr int N = decltype(n)::value, NPT = decltype(npt)::value;
    hipLaunchKernelGGL((delta_bwd_kernel<N, NPT>), dim3((unsigned)(heads * (ptiles / NPT))),
                       dim3(64 * NPT * kSplit<N> + 256), 0, st, a, ptiles);
  };
  auto pick = [&](auto n) {
    two_tiles(heads, ptiles) ? go(n, std::integral_constant<int, 2>{}) : go(n, std::integral_constant<int, 1>{});
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
