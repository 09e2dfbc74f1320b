// Gated delta rule, bf16 io, forward chain.  Per sequence and head, chunk by chunk (64
// tokens), for 16 columns of headdim (they do not interact):
//   X = V - exp(G) K S^T,   Z = X - R (b X),   U = b Z,
//   S <- exp(G_C) S + (exp(G_C - G) U)^T K,    O = scale exp(G) Q S^T + P U.
//
// A workgroup has chain waves, one or two (kSplit) for each of its NPT tiles of 16 columns,
// and four helper waves.
// * A chain wave walks the recurrence.  S, X, Z and U never leave its registers: each
//   product's accumulator tiles are the next product's operand (delta_reg.hpp); K, R, V
//   come through LDS.  The issue of its one wave bounds a chunk (560 instructions, 3650
//   cycles at dstate 128), so there two waves share a tile: each holds half of the state's
//   columns, forms its part of K S^T and the new state, and both form X and Z, from their
//   own part and the other's (through LDS).  With dstate 64 it is worth nothing (156 and
//   162 us for 2 x 4096 tokens of 64 heads).
// * The helpers keep memory away from the chain: they load the chunks ahead into
//   registers and copy them to LDS, and form the output half a chunk behind the chain, from
//   the planes of S and from Z, which it leaves in LDS.
// Two barriers a chunk:
//   interval A(c)  chain: S's planes, K S^T       helpers: Q(c) to LDS, O of c - 1
//   interval B(c)  chain: (R b) X, Z, the new S    helpers: K, R, V(c + 1), P(c) to LDS, Q S^T of c
// (X is formed in A by a wave that has all of S.)  A matrix instruction occupies the matrix
// core for 16 cycles and the issue of its wave for four: the chain's vector work (planes,
// scalings) is placed between the products that do not wait for it.
//
// Two tiles a workgroup (two_tiles) where one each would not fit the CUs at once: a compute
// unit takes in 50 KB a chunk with one or two, 1000 cycles of its load path at the least and
// 2000 when they come from HBM.  2 x 8192 tokens of 64 heads of 64 x 128, states and Z kept:
// one tile 592 us, two 400, four (one wave each) 515.  A packed batch of 8191 tokens: 231,
// 170, 190.  131072 tokens of 32 heads, 128 workgroups: one 2980 us, two 3990; 3340 with one
// wave a tile.  The loads a second chunk ahead, or eight helpers (loads and outputs apart),
// gain nothing.
//
// Planes (delta.hpp): S, X and U two.  The state's update takes three of its operand,
// since what it rounds away stays in the state: the final states come out at fp32's own
// error (3e-7 against 2e-6 with two, for sixteen more instructions of a chunk's 142).
#include "delta_reg.hpp"

namespace ssd {

template <int N, int NPT, bool SAVE>
__global__ __launch_bounds__(64 * NPT * kSplit<N> + 256, 1) void delta_fwd_kernel(DeltaArgs a, int ptiles) {
  constexpr int C = kDeltaChunk, NP = N < 32 ? 32 : N, KS = NP / 32, SPLIT = kSplit<N>, CW = NPT * SPLIT;
  constexpr int KH = KS / SPLIT;  // blocks of 32 columns of the state a chain wave holds
  using Tile = TokTile<NP>;
  constexpr int LV = 16 * NPT + 8, EV = C * LV, ER = 2 * kTriPlane, EP = kTriPlane;
  __shared__ __align__(16) uint16_t Kl[2][Tile::SIZE], Ql[Tile::SIZE], Rl[2][ER], Pl[EP], Vl[EV];
  __shared__ __align__(16) float gl[2][3 * C];  // beta, exp(G), beta exp(G_C - G)
  __shared__ __align__(16) u32x4 Sx[NPT][KS][2][64];  // planes of S, operand order
  __shared__ __align__(16) f32x4 Zx[NPT][4][64];      // Z, tile order
  __shared__ __align__(16) f32x4 Kx[SPLIT == 2 ? NPT : 1][SPLIT][4][64];  // parts of K S^T

  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, q = lane >> 4, r = lane & 15;
  const int np = ptiles / NPT;
  int s, wg;
  chain_order(a.H * np, s, wg);
  const int pg = wg % np, h = wg / np;
  const int p0 = pg * 16 * NPT;                      // the workgroup's columns
  const int grp = h / (a.H / a.G);
  const SeqSpan sp = seq_span(a.map, s);
  const int c0 = sp.c0, c1 = sp.c1;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  if (w < CW) {
    // ------------------------------------------------------------ chain wave ----
    const int tw = w / SPLIT, half = w % SPLIT, kb = half * KH;
    const int pc = p0 + 16 * tw + r;  // this lane's column of headdim
    // the state: S[k][t] holds columns 32(kb + k) + 8q + 4t + e of row pc
    f32x4 S[KH][2];
    const int64_t srow = (((int64_t)s * a.H + h) * a.P + pc) * N;
    auto scol = [&](int k, int t) { return 32 * (kb + k) + 8 * q + 4 * t; };
#pragma unroll
    for (int k = 0; k < KH; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        S[k][t] = a.init && scol(k, t) < N ? *(const f32x4*)(a.init + srow + scol(k, t)) : zero;
    f32x4* kS = (f32x4*)a.S + (int64_t)(pc >> 4) * (KS * 2) * 64 + lane;  // of chunk slot 0 (SAVE)
    f32x4* kZ = (f32x4*)a.Z + (int64_t)(pc >> 4) * 4 * 64 + lane;
    __syncthreads();
    if constexpr (SPLIT == 2) {
      for (int c = c0; c < c1; ++c) {
        const uint16_t* K = Kl[(c - c0) & 1];
        const float* g = gl[(c - c0) & 1];
        const int64_t kh = (int64_t)c * a.H + h;
        // interval A: this half's part of K S^T
        f32x4 ks[4], X[4], eg[4], wg4[4];
        u32x4 vw[2];
        Planes<2> xf[2], Rf[6], sf[KH];
        bf16x8 kt[KH][2][2], kf[KH][4];
        const float eC = g[C + C - 1];
#pragma unroll
        for (int k = 0; k < KH; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) kf[k][i] = tok_rows<NP>(K, 32 * (i >> 1), i & 1, 32 * (kb + k), lane);
        sf[0] = tile_planes<2>(S[0][0], S[0][1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) ks[i] = zero;
#pragma unroll
        for (int B = 0; B < 2; ++B) vw[B] = __builtin_bit_cast(u32x4, frag_kmajor(Vl + 32 * B * LV + 16 * tw, LV, lane));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < KH; ++k) {
#pragma unroll
          for (int m = 1; m >= 0; --m)
#pragma unroll
            for (int i = 0; i < 4; ++i) ks[i] = mfma_bf16(kf[k][i], sf[k].p[m], ks[i]);
          if (k + 1 < KH) sf[k + 1] = tile_planes<2>(S[k + 1][0], S[k + 1][1]);
#pragma unroll
          for (int m = 0; m < 2; ++m) Sx[tw][kb + k][m][lane] = __builtin_bit_cast(u32x4, sf[k].p[m]);
          if constexpr (SAVE)
#pragma unroll
            for (int t = 0; t < 2; ++t) kS[(kh * (a.P / 16) * (KS * 2) + (kb + k) * 2 + t) * 64] = S[k][t];
          if (k + 1 == KH) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              eg[i] = *(const f32x4*)(g + C + 32 * (i >> 1) + 8 * q + 4 * (i & 1));
              wg4[i] = *(const f32x4*)(g + 2 * C + 32 * (i >> 1) + 8 * q + 4 * (i & 1));
            }
#pragma unroll
            for (int i = 0; i < 6; ++i)
#pragma unroll
              for (int m = 0; m < 2; ++m)
                Rf[i].p[m] = as_bf16x8(*(const u32x4*)(Rl[(c - c0) & 1] + m * kTriPlane + i * 512 + lane * 8));
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
        for (int i = 0; i < 4; ++i)
          X[i] = f32x4{bf_lo(vw[i >> 1][2 * (i & 1)]), bf_hi(vw[i >> 1][2 * (i & 1)]), bf_lo(vw[i >> 1][2 * (i & 1) + 1]),
                       bf_hi(vw[i >> 1][2 * (i & 1) + 1])} -
                 eg[i] * ks[i];
        __syncthreads();
        // interval B: X from both parts and Z (each wave forms all of them, to the order of one
        // sum), and this half of the new state
        f32x4 Z[4], kx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) kx[i] = Kx[tw][1 - half][i][lane];
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) Z[i] = zero;
#pragma unroll
        for (int i = 0; i < 2; ++i) X[i] = X[i] - eg[i] * kx[i];
        xf[0] = tile_planes<2>(X[0], X[1]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < 3; ++m) {
#pragma unroll
          for (int t = 0; t < 2; ++t) Z[t] = mfma_bf16(Rf[low_block(0, t, 0)].p[m == 0], xf[0].p[m == 1], Z[t]);
#pragma unroll
          for (int t = 0; t < 2; ++t) Z[2 + t] = mfma_bf16(Rf[low_block(1, t, 0)].p[m == 0], xf[0].p[m == 1], Z[2 + t]);
        }
#pragma unroll
        for (int i = 2; i < 4; ++i) X[i] = X[i] - eg[i] * kx[i];
        xf[1] = tile_planes<2>(X[2], X[3]);
        interleave<12, 3>();
        __builtin_amdgcn_sched_barrier(0);
        Planes<3> wf[2];
        auto form_w = [&](int B) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int i = 2 * B + t;
            Z[i] = X[i] - Z[i];
            if (B == half) {
              Zx[tw][i][lane] = Z[i];
              if constexpr (SAVE)
                kZ[(kh * (a.P / 16) * 4 + i) * 64] = Z[i];
            }
          }
          wf[B] = tile_planes<3>(wg4[2 * B] * Z[2 * B], wg4[2 * B + 1] * Z[2 * B + 1]);
        };
#pragma unroll
        for (int m = 0; m < 3; ++m)
#pragma unroll
          for (int t = 0; t < 2; ++t) Z[2 + t] = mfma_bf16(Rf[low_block(1, t, 1)].p[m == 0], xf[1].p[m == 1], Z[2 + t]);
#pragma unroll
        for (int k = 0; k < KH; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) S[k][t] = eC * S[k][t];
        form_w(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int B = 0; B < 2; ++B) {
#pragma unroll
          for (int m = 2; m >= 0; --m)
#pragma unroll
            for (int k = 0; k < KH; ++k)
#pragma unroll
              for (int t = 0; t < 2; ++t) S[k][t] = mfma_bf16(kt[k][t][B], wf[B].p[m], S[k][t]);
          if (B == 0) form_w(1);
          interleave<6 * KH, 4>();
          __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
      }
    } else {
      for (int c = c0; c < c1; ++c) {
        const uint16_t* K = Kl[(c - c0) & 1];
        const float* g = gl[(c - c0) & 1];
        const int64_t kh = (int64_t)c * a.H + h;
        // interval A: K S^T, tile i = 2B + t with tokens 32B + 8q + 4t + e; block 0 of the tokens
        // with S's planes on the way, block 1 with X of block 0
        f32x4 ks[4], X[4], eg[4], wg4[4];
        u32x4 vw[2];
        Planes<2> xf[2], Rf[6];
        bf16x8 kt[KS][2][2];  // K^T, by block of tokens
        const float eC = g[C + C - 1];
        bf16x8 kf[KS][2], kg[KS][2];
        Planes<2> sf[KS];
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) kf[k][t] = tok_rows<NP>(K, 0, t, 32 * k, lane);
#pragma unroll
        for (int B = 0; B < 2; ++B) vw[B] = __builtin_bit_cast(u32x4, frag_kmajor(Vl + 32 * B * LV + 16 * w, LV, lane));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ks[i] = zero;
          eg[i] = *(const f32x4*)(g + C + 32 * (i >> 1) + 8 * q + 4 * (i & 1));
          wg4[i] = *(const f32x4*)(g + 2 * C + 32 * (i >> 1) + 8 * q + 4 * (i & 1));
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) kg[k][t] = tok_rows<NP>(K, 32, t, 32 * k, lane);
        sf[0] = tile_planes<2>(S[0][0], S[0][1]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
#pragma unroll
          for (int m = 1; m >= 0; --m)
#pragma unroll
            for (int t = 0; t < 2; ++t) ks[t] = mfma_bf16(kf[k][t], sf[k].p[m], ks[t]);
          if (k + 1 < KS) sf[k + 1] = tile_planes<2>(S[k + 1][0], S[k + 1][1]);
#pragma unroll
          for (int m = 0; m < 2; ++m) Sx[w][k][m][lane] = __builtin_bit_cast(u32x4, sf[k].p[m]);
          if constexpr (SAVE)
#pragma unroll
            for (int t = 0; t < 2; ++t) kS[(kh * (a.P / 16) * (KS * 2) + k * 2 + t) * 64] = S[k][t];
          interleave<4, 4>();
          __builtin_amdgcn_sched_barrier(0);
        }
        auto form_x = [&](int B) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const f32x4 v = {bf_lo(vw[B][2 * t]), bf_hi(vw[B][2 * t]), bf_lo(vw[B][2 * t + 1]), bf_hi(vw[B][2 * t + 1])};
            X[2 * B + t] = v - eg[2 * B + t] * ks[2 * B + t];
          }
          xf[B] = tile_planes<2>(X[2 * B], X[2 * B + 1]);
        };
        // (and what the next interval starts with)
#pragma unroll
        for (int i = 0; i < 6; ++i)
#pragma unroll
          for (int m = 0; m < 2; ++m)
            Rf[i].p[m] = as_bf16x8(*(const u32x4*)(Rl[(c - c0) & 1] + m * kTriPlane + i * 512 + lane * 8));
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) kt[k][t][0] = tok_cols<NP>(K, 0, t, 32 * k, lane);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int m = 1; m >= 0; --m)
#pragma unroll
            for (int t = 0; t < 2; ++t) ks[2 + t] = mfma_bf16(kg[k][t], sf[k].p[m], ks[2 + t]);
        form_x(0);
        interleave<4 * KS, 3>();
        __builtin_amdgcn_sched_barrier(0);
        form_x(1);
        __syncthreads();
        // interval B: Z = X - (R b) X, by planes (low x high, high x low, high x high), with the
        // state's decay on the way
        f32x4 Z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) Z[i] = zero;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) kt[k][t][1] = tok_cols<NP>(K, 32, t, 32 * k, lane);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < 3; ++m)
#pragma unroll
          for (int t = 0; t < 2; ++t) Z[t] = mfma_bf16(Rf[low_block(0, t, 0)].p[m == 0], xf[0].p[m == 1], Z[t]);
#pragma unroll
        for (int S2 = 0; S2 < 2; ++S2)
#pragma unroll
          for (int m = 0; m < 3; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t) Z[2 + t] = mfma_bf16(Rf[low_block(1, t, S2)].p[m == 0], xf[S2].p[m == 1], Z[2 + t]);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int t = 0; t < 2; ++t) S[k][t] = eC * S[k][t];
        interleave<18, 2>();
        __builtin_amdgcn_sched_barrier(0);
        Planes<3> wf[2];
        auto form_w = [&](int B) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int i = 2 * B + t;
            Z[i] = X[i] - Z[i];
            Zx[w][i][lane] = Z[i];
            if constexpr (SAVE)
              kZ[(kh * (a.P / 16) * 4 + i) * 64] = Z[i];
          }
          wf[B] = tile_planes<3>(wg4[2 * B] * Z[2 * B], wg4[2 * B + 1] * Z[2 * B + 1]);
        };
        form_w(0);
        __builtin_amdgcn_sched_barrier(0);
        // the state; U of the second block of tokens during the first one's products
#pragma unroll
        for (int B = 0; B < 2; ++B) {
#pragma unroll
          for (int m = 2; m >= 0; --m)
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int t = 0; t < 2; ++t) S[k][t] = mfma_bf16(kt[k][t][B], wf[B].p[m], S[k][t]);
          if (B == 0) form_w(1);
          interleave<6 * KS, 2>();
          __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
      }
    }
    __syncthreads();
    if (a.final_states) {
#pragma unroll
      for (int k = 0; k < KH; ++k)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (scol(k, t) < N) *(f32x4*)(a.final_states + srow + scol(k, t)) = S[k][t];
    }
    return;
  }

  // --------------------------------------------------------------- helper wave ----
  // (the outputs of a tile: HT blocks of 16 tokens a wave)
  constexpr int HT = NPT;
  const int ht = tid - 64 * CW, tile = (w - CW) % NPT, i0 = (w - CW) / NPT * HT;
  const bool outs = a.out;  // (no output where a backward recomputes)
  if constexpr (N < 32) {  // the products' depth is 32: columns past N are zero
    for (int e = ht; e < C; e += 256)
      for (int c = N; c < 32; c += 4) {
        *(uint2*)(Kl[0] + Tile::at(e, c)) = make_uint2(0u, 0u);
        *(uint2*)(Kl[1] + Tile::at(e, c)) = make_uint2(0u, 0u);
        *(uint2*)(Ql + Tile::at(e, c)) = make_uint2(0u, 0u);
      }
  }
  // 16-byte pieces of a chunk a thread: K, Q, R, P, V
  constexpr int KC = (C * N / 8 + 255) / 256, RC = ER / 8 / 256, VP = 2 * NPT, VC = (C * VP + 255) / 256;
  constexpr bool KX = C * N / 8 % 256 == 0, VX = C * VP % 256 == 0;  // every thread has a piece
  u32x4 xk[KC], xq[KC], xr[RC], xp[2], xv[VC];
  float xg;
  auto krsrc = [&](const void* p, int c, uint32_t& row) {
    const int start = sp.start + (c - c0) * C, len = min(C, sp.end - start);
    row = (uint32_t)a.G * N * 2;
    return make_rsrc((const char*)p + ((int64_t)start * a.G + grp) * N * 2, (uint32_t)(len - 1) * row + N * 2);
  };
  auto load_q = [&](int c) {
    uint32_t row;
    const brsrc rq = krsrc(a.q, c, row);
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int e = ht + i * 256;
      xq[i] = buf_load16(rq, KX || e < C * N / 8 ? (e / (N / 8)) * row + (e % (N / 8)) * 16 : kNoOffset);
    }
  };
  auto load = [&](int c) {
    uint32_t row;
    const brsrc rk = krsrc(a.k, c, row);
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int e = ht + i * 256;
      xk[i] = buf_load16(rk, KX || e < C * N / 8 ? (e / (N / 8)) * row + (e % (N / 8)) * 16 : kNoOffset);
    }
    const int start = sp.start + (c - c0) * C, len = min(C, sp.end - start);
    const uint32_t vrow = (uint32_t)a.H * a.P * 2;
    const brsrc rv = make_rsrc((const char*)a.v + (((int64_t)start * a.H + h) * a.P + p0) * 2,
                               (uint32_t)(len - 1) * vrow + 32 * NPT);
#pragma unroll
    for (int i = 0; i < VC; ++i) {
      const int e = ht + i * 256;
      xv[i] = buf_load16(rv, VX || e < C * VP ? (e / VP) * vrow + (e % VP) * 16 : kNoOffset);
    }
    const int64_t kh = (int64_t)c * a.H + h;
    const brsrc rr = make_rsrc(a.R + kh * ER, ER * 2);
#pragma unroll
    for (int i = 0; i < RC; ++i) xr[i] = buf_load16(rr, (ht + i * 256) * 16);
    xg = buf_load_f32(make_rsrc(a.gates + kh * kDeltaGates + 2 * C, 3 * C * 4), ht * 4);
  };
  auto load_p = [&](int c) {
    const brsrc rp = make_rsrc(a.Pm + ((int64_t)c * a.H + h) * EP, EP * 2);
#pragma unroll
    for (int i = 0; i < 2; ++i) xp[i] = buf_load16(rp, (ht + i * 256) * 16);  // (the last half is past the end)
  };
  auto put_q = [&]() {
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int e = ht + i * 256;
      if (KX || e < C * N / 8) *(u32x4*)(Ql + Tile::at(e / (N / 8), (e % (N / 8)) * 8)) = xq[i];
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int e = ht + i * 256;
      if (KX || e < C * N / 8) *(u32x4*)(Kl[buf] + Tile::at(e / (N / 8), (e % (N / 8)) * 8)) = xk[i];
    }
#pragma unroll
    for (int i = 0; i < VC; ++i) {
      const int e = ht + i * 256;
      if (VX || e < C * VP) *(u32x4*)(Vl + (e / VP) * LV + (e % VP) * 8) = xv[i];
    }
#pragma unroll
    for (int i = 0; i < RC; ++i) *(u32x4*)(Rl[buf] + (ht + i * 256) * 8) = xr[i];
    if (ht < 3 * C) gl[buf][ht] = xg;
  };
  auto put_p = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if ((ht + i * 256) * 8 < EP) *(u32x4*)(Pl + (ht + i * 256) * 8) = xp[i];
  };

  f32x4 qs[HT];
  // O of chunk c = scale exp(G) Q S^T (in qs) + P U, stored with rows headdim: four elements
  // of a token a lane
  auto finish = [&](int c) {
    const float* g = gl[(c - c0) & 1];
    bf16x8 pf[HT][2];
    f32x4 z[4];
    Planes<2> uf[2];
    const bool second = i0 + HT > 2;  // (of the two blocks of 32 tokens)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < 2 || second) z[i] = *(const f32x4*)(g + 32 * (i >> 1) + 8 * q + 4 * (i & 1)) * Zx[tile][i][lane];
#pragma unroll
    for (int ii = 0; ii < HT; ++ii)
#pragma unroll
      for (int S2 = 0; S2 < 2; ++S2) {
        const int i = i0 + ii;
        if (2 * S2 <= i) pf[ii][S2] = as_bf16x8(*(const u32x4*)(Pl + low_block(i >> 1, i & 1, S2) * 512 + lane * 8));
      }
#pragma unroll
    for (int B = 0; B < 2; ++B)
      if (B == 0 || second) uf[B] = tile_planes<2>(z[2 * B], z[2 * B + 1]);
#pragma unroll
    for (int m = 1; m >= 0; --m)
#pragma unroll
      for (int S2 = 0; S2 < 2; ++S2)
#pragma unroll
        for (int ii = 0; ii < HT; ++ii)
          if (2 * S2 <= i0 + ii) qs[ii] = mfma_bf16(uf[S2].p[m], pf[ii][S2], qs[ii]);
    const int start = sp.start + (c - c0) * C, len = min(C, sp.end - start);
    const uint32_t vrow = (uint32_t)a.H * a.P * 2;
    const brsrc ro = make_rsrc((char*)a.out + (((int64_t)start * a.H + h) * a.P + p0) * 2,
                               (uint32_t)(len - 1) * vrow + 32 * NPT);
#pragma unroll
    for (int ii = 0; ii < HT; ++ii)
      store4io(ro, (32 * ((i0 + ii) >> 1) + row32(r, (i0 + ii) & 1)) * vrow + (16 * tile + 4 * q) * 2, qs[ii], IoBf16{});
  };

  // (The loads run on to the last chunk again instead of stopping under a branch, at whose
  // join they would be waited for.)
  if (c0 < c1) {
    load(c0);
    put(0);
    load_q(c0);
    load_p(c0);
    load(min(c0 + 1, c1 - 1));
  }
  __syncthreads();
  for (int c = c0; c < c1; ++c) {
    // interval A
    put_q();
    load_q(min(c + 1, c1 - 1));
    if (outs && c > c0) finish(c - 1);
    __syncthreads();
    // interval B
    put((c + 1 - c0) & 1);
    put_p();
    load(min(c + 2, c1 - 1));
    load_p(min(c + 1, c1 - 1));
    if (outs) {
      const float* g = gl[(c - c0) & 1];
#pragma unroll
      for (int i = 0; i < HT; ++i) qs[i] = zero;
      bf16x8 qf[2][HT];
      Planes<2> sf[2];
      auto fetch = [&](int k) {
#pragma unroll
        for (int m = 0; m < 2; ++m) sf[k & 1].p[m] = as_bf16x8(Sx[tile][k][m][lane]);
#pragma unroll
        for (int i = 0; i < HT; ++i) qf[k & 1][i] = tok_rows<NP>(Ql, 32 * ((i0 + i) >> 1), (i0 + i) & 1, 32 * k, lane);
      };
      fetch(0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        if (k + 1 < KS) fetch(k + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 1; m >= 0; --m)
#pragma unroll
          for (int i = 0; i < HT; ++i) qs[i] = mfma_bf16(sf[k & 1].p[m], qf[k & 1][i], qs[i]);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int i = 0; i < HT; ++i) qs[i] = (a.scale * g[C + 32 * ((i0 + i) >> 1) + row32(r, (i0 + i) & 1)]) * qs[i];
    }
    __syncthreads();
  }
  // (the chain's last barrier: the last chunk's Z and P are there since the one before)
  __syncthreads();
  if (outs && c0 < c1) finish(c1 - 1);
}

hipError_t launch_delta_fwd(const DeltaProb& p, const DeltaArgs& a, hipStream_t st) {
  if (!p.io) return launch_delta_f32_fwd(p, a, st);
  if (p.nst == 0) return hipSuccess;
  const int ptiles = p.P / 16;
  const int64_t heads = (int64_t)p.nst * p.H;
  auto go = [&](auto n, auto npt, auto save) {
    constexpr int N = decltype(n)::value, NPT = decltype(npt)::value;
    hipLaunchKernelGGL((delta_fwd_kernel<N, NPT, decltype(save)::value>),
                       dim3((unsigned)(heads * (ptiles / NPT))), dim3(64 * NPT * kSplit<N> + 256), 0, st, a,
                       ptiles);
  };
  auto pick_npt = [&](auto n, auto save) {
    two_tiles(heads, ptiles) ? go(n, std::integral_constant<int, 2>{}, save)
                             : go(n, std::integral_constant<int, 1>{}, save);
  };
  auto pick = [&](auto save) {
    switch (p.N) {
      case 16: pick_npt(std::integral_constant<int, 16>{}, save); break;
      case 32: pick_npt(std::integral_constant<int, 32>{}, save); break;
      case 64: pick_npt(std::integral_constant<int, 64>{}, save); break;
      default: pick_npt(std::integral_constant<int, 128>{}, save); break;
    }
  };
  a.S ? pick(std::true_type{}) : pick(std::false_type{});
  return hipGetLastError();
}

}  // namespace ssd
