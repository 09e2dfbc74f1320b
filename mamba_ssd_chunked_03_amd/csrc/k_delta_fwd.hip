// Gated delta rule, bf16 io, forward chain: a wave walks one sequence's chunks for 16
// columns of headdim of one head (those do not interact).  Per chunk of 64 tokens:
//   X = V - exp(G) K S^T,   Z = X - R (b X),   U = b Z,
//   S <- exp(G_C) S + (exp(G_C - G) U)^T K,    O = scale exp(G) Q S^T + P U.
// S, X, Z and U never leave the wave's registers: each product's accumulator tiles are
// the next product's operand (delta_reg.hpp).  Only K, Q, R, P, V come through LDS, shared
// by the workgroup's four waves, double buffered, the chunk after the next in flight.
//
// The four waves are 4 / NS tiles of 16 columns, each split over NS waves along dstate
// (NS > 1 where heads and sequences are too few to give every compute unit four tiles):
// the NS partial sums of K S^T and Q S^T meet in LDS, R X is computed by each.
//
// Planes (delta.hpp): S, X and U two.  The state's update takes three of its operand,
// since what it rounds away stays in the state: the final states come out at fp32's own
// error (3e-7 against 2e-6 with two, for two more instructions in eight of a chunk's
// hundred and forty).
#include "delta_reg.hpp"

namespace ssd {

template <int N, int NS, bool SAVE>
__global__ __launch_bounds__(256, 1) void delta_fwd_kernel(DeltaArgs a, int ptiles) {
  constexpr int C = kDeltaChunk, NP = N < 32 ? 32 : N, KS = NP / 32, KW = (KS + NS - 1) / NS, NPT = 4 / NS;
  constexpr int LK = NP + 8, LV = 16 * NPT + 8;
  constexpr int EK = C * LK, ER = 2 * kTriPlane, EP = kTriPlane, EV = C * LV;
  struct Buf {
    uint16_t K[EK], Q[EK], R[ER], P[EP], V[EV];
    float g[3 * C];  // beta, exp(G), exp(G_C - G)
  };
  __shared__ __align__(16) Buf buf[2];
  constexpr int XCH = NS > 1 ? NPT * NS * 4 * 64 : 1;
  __shared__ __align__(16) f32x4 xk[XCH], xq[XCH];

  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, q = lane >> 4, r = lane & 15;
  const int pt = w / NS, ns = w % NS;  // tile of the workgroup, part of dstate
  const int np = (ptiles + NPT - 1) / NPT;
  const int wg = xcd_order(blockIdx.x, gridDim.x);
  const int pg = wg % np, h = (wg / np) % a.H, s = wg / np / a.H;
  const int p0 = pg * 16 * NPT;           // the workgroup's columns
  const int pw = 16 * min(NPT, ptiles - pg * NPT);
  const bool live = 16 * pt < pw;         // (a workgroup's last waves may have no tile)
  const int pc = p0 + 16 * pt + r;        // this lane's column of headdim
  const int grp = h / (a.H / a.G);
  const SeqSpan sp = seq_span(a.map, s);
  const int c0 = sp.c0, c1 = sp.c1;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  // the state: S[k][t] holds columns 32 (ns KW + k) + 8q + 4t + e of row pc
  f32x4 S[KW][2];
  const int64_t srow = (((int64_t)s * a.H + h) * a.P + pc) * N;
  auto scol = [&](int k, int t) { return 32 * (ns * KW + k) + 8 * q + 4 * t; };
#pragma unroll
  for (int k = 0; k < KW; ++k)
#pragma unroll
    for (int t = 0; t < 2; ++t)
      S[k][t] = a.init && live && scol(k, t) < N ? *(const f32x4*)(a.init + srow + scol(k, t)) : zero;

  if constexpr (N < 32) {  // the products' depth is 32: columns past N are zero
    for (int e = tid; e < 2 * C; e += 256)
      for (int c = N; c < 32; c += 4) {
        *(uint2*)(buf[e / C].K + (e % C) * LK + c) = make_uint2(0u, 0u);
        *(uint2*)(buf[e / C].Q + (e % C) * LK + c) = make_uint2(0u, 0u);
      }
  }

  // staging: 16-byte pieces, loaded to registers a chunk ahead of their LDS copy
  constexpr int KC = (C * N / 8 + 255) / 256, RC = ER / 8 / 256, VP = 2 * NPT, VC = (C * VP + 255) / 256;
  struct Loads {
    u32x4 k[KC], q[KC], R[RC], P[2], v[VC];
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
    const brsrc rr = make_rsrc(a.R + kh * ER, ER * 2), rp = make_rsrc(a.Pm + kh * EP, EP * 2);
#pragma unroll
    for (int i = 0; i < RC; ++i) x.R[i] = buf_load16(rr, (tid + i * 256) * 16);
#pragma unroll
    for (int i = 0; i < 2; ++i) x.P[i] = buf_load16(rp, (tid + i * 256) * 16);  // (the last half is past the end)
    const uint32_t vrow = (uint32_t)a.H * a.P * 2;
    const brsrc rv = make_rsrc((const char*)a.v + (((int64_t)start * a.H + h) * a.P + p0) * 2,
                               (uint32_t)(len - 1) * vrow + pw * 2);
#pragma unroll
    for (int i = 0; i < VC; ++i) {
      const int e = tid + i * 256;
      x.v[i] = buf_load16(rv, e < C * VP && 8 * (e % VP) < pw ? (e / VP) * vrow + (e % VP) * 16 : kNoOffset);
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
    for (int i = 0; i < RC; ++i) *(u32x4*)(b.R + (tid + i * 256) * 8) = x.R[i];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if ((tid + i * 256) * 8 < EP) *(u32x4*)(b.P + (tid + i * 256) * 8) = x.P[i];
#pragma unroll
    for (int i = 0; i < VC; ++i) {
      const int e = tid + i * 256;
      if (e < C * VP) *(u32x4*)(b.V + (e / VP) * LV + (e % VP) * 8) = x.v[i];
    }
    if (tid < 3 * C) b.g[tid] = x.g;
  };

  Loads x;
  if (c0 < c1) {
    load(x, c0);
    put(x, buf[0]);
    if (c0 + 1 < c1) load(x, c0 + 1);
  }
  __syncthreads();
  for (int c = c0; c < c1; ++c) {
    const Buf& b = buf[(c - c0) & 1];
    const int64_t kh = (int64_t)c * a.H + h;
    // K S^T (rows tokens) and (Q S^T)^T (rows headdim) over this wave's part of dstate
    f32x4 ks[2][2], qs[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) ks[i >> 1][i & 1] = qs[i >> 1][i & 1] = zero;
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const int kk = ns * KW + k;
      if (KS % NS == 0 || kk < KS) {
        const Planes<2> sf = tile_planes<2>(S[k][0], S[k][1]);
        if constexpr (SAVE)
          if (live)
#pragma unroll
            for (int t = 0; t < 2; ++t)
              if (scol(k, t) < N) *(f32x4*)(a.S + (kh * a.P + pc) * N + scol(k, t)) = S[k][t];
#pragma unroll
        for (int B = 0; B < 2; ++B)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int o = (32 * B + row32(r, t)) * LK + 32 * kk + 8 * q;
            ks[B][t] = mma1<2>(as_bf16x8(*(const u32x4*)(b.K + o)), sf, ks[B][t]);
            qs[B][t] = mma1t<2>(sf, as_bf16x8(*(const u32x4*)(b.Q + o)), qs[B][t]);
          }
      }
    }
    if constexpr (NS > 1) {  // the parts' sums, in order of the parts
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xk[((pt * NS + ns) * 4 + i) * 64 + lane] = ks[i >> 1][i & 1];
        xq[((pt * NS + ns) * 4 + i) * 64 + lane] = qs[i >> 1][i & 1];
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 y = xk[(pt * NS * 4 + i) * 64 + lane];
#pragma unroll
        for (int j = 1; j < NS; ++j) y += xk[((pt * NS + j) * 4 + i) * 64 + lane];
        ks[i >> 1][i & 1] = y;
        if (i % NS == ns) {  // the output's tiles are shared out
          f32x4 z = xq[(pt * NS * 4 + i) * 64 + lane];
#pragma unroll
          for (int j = 1; j < NS; ++j) z += xq[((pt * NS + j) * 4 + i) * 64 + lane];
          qs[i >> 1][i & 1] = z;
        }
      }
    }
    // X, Z, U: tile (B, t) has tokens 32B + 8q + 4t + e
    f32x4 X[2][2], bt[2][2];
    Planes<2> xf[2], uf[2];
    Planes<3> wf[2];
#pragma unroll
    for (int B = 0; B < 2; ++B) {
      const bf16x8 vf = frag_kmajor(b.V + 32 * B * LV + 16 * pt, LV, lane);
      const u32x4 vw = __builtin_bit_cast(u32x4, vf);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int tk = 32 * B + 8 * q + 4 * t;
        const f32x4 v = {bf_lo(vw[2 * t]), bf_hi(vw[2 * t]), bf_lo(vw[2 * t + 1]), bf_hi(vw[2 * t + 1])};
        bt[B][t] = *(const f32x4*)(b.g + tk);
        X[B][t] = v - *(const f32x4*)(b.g + C + tk) * ks[B][t];
      }
      xf[B] = tile_planes<2>(bt[B][0] * X[B][0], bt[B][1] * X[B][1]);
    }
    auto rfrag = [&](int B, int t, int S2) {
      Planes<2> f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        f.p[i] = as_bf16x8(*(const u32x4*)(b.R + i * kTriPlane + low_block(B, t, S2) * 512 + lane * 8));
      return f;
    };
#pragma unroll
    for (int B = 0; B < 2; ++B) {
      f32x4 u[2], wv[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        f32x4 z = zero;
#pragma unroll
        for (int S2 = 0; S2 <= B; ++S2) z = mma<2>(rfrag(B, t, S2), xf[S2], z);
        z = X[B][t] - z;
        const int tk = 32 * B + 8 * q + 4 * t;
        if constexpr (SAVE)
          if (live && (NS == 1 || (2 * B + t) % NS == ns))
#pragma unroll
            for (int e = 0; e < 4; ++e) a.Z[(kh * C + tk + e) * a.P + pc] = z[e];
        u[t] = bt[B][t] * z;
        wv[t] = *(const f32x4*)(b.g + 2 * C + tk) * u[t];
      }
      uf[B] = tile_planes<2>(u[0], u[1]);
      wf[B] = tile_planes<3>(wv[0], wv[1]);
    }
    // the state
    const float eC = b.g[C + C - 1];
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const int kk = ns * KW + k;
      if (KS % NS == 0 || kk < KS) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          f32x4 y = eC * S[k][t];
#pragma unroll
          for (int B = 0; B < 2; ++B) y = mma1<3>(cols32(b.K + 32 * B * LK + 32 * kk, LK, t, lane), wf[B], y);
          S[k][t] = y;
        }
      }
    }
    // the output, rows headdim: four consecutive elements of a token a lane (none where the
    // backward recomputes what a forward keeps)
    if (a.out && live) {
      const int start = sp.start + (c - c0) * C, len = min(C, sp.end - start);
      const uint32_t vrow = (uint32_t)a.H * a.P * 2;
      const brsrc ro = make_rsrc((char*)a.out + (((int64_t)start * a.H + h) * a.P + p0) * 2,
                                 (uint32_t)(len - 1) * vrow + pw * 2);
#pragma unroll
      for (int B = 0; B < 2; ++B)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (NS == 1 || (2 * B + t) % NS == ns) {
            const int tk = 32 * B + row32(r, t);
            f32x4 y = (a.scale * b.g[C + tk]) * qs[B][t];
#pragma unroll
            for (int S2 = 0; S2 <= B; ++S2)
              y = mma1t<2>(uf[S2], as_bf16x8(*(const u32x4*)(b.P + low_block(B, t, S2) * 512 + lane * 8)), y);
            store4io(ro, tk * vrow + (16 * pt + 4 * q) * 2, y, IoBf16{});
          }
    }
    if (c + 1 < c1) {
      put(x, buf[(c + 1 - c0) & 1]);
      if (c + 2 < c1) load(x, c + 2);
    }
    __syncthreads();
  }
  if (a.final_states && live) {
#pragma unroll
    for (int k = 0; k < KW; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (scol(k, t) < N) *(f32x4*)(a.final_states + srow + scol(k, t)) = S[k][t];
  }
}

hipError_t launch_delta_fwd(const DeltaProb& p, const DeltaArgs& a, hipStream_t st) {
  if (!p.io) return launch_delta_f32_fwd(p, a, st);
  if (p.nst == 0) return hipSuccess;
  const int ptiles = p.P / 16;
  const int64_t heads = (int64_t)p.nst * p.H;
  auto go = [&](auto n, auto ns, auto save) {
    constexpr int NS = decltype(ns)::value, NPT = 4 / NS;
    hipLaunchKernelGGL((delta_fwd_kernel<decltype(n)::value, NS, decltype(save)::value>),
                       dim3((unsigned)(heads * ((ptiles + NPT - 1) / NPT))), dim3(256), 0, st, a, ptiles);
  };
  auto pick_ns = [&](auto n, auto save) {
    const int64_t tiles = heads * ptiles;
    if (tiles >= 512 && ptiles >= 4)
      go(n, std::integral_constant<int, 1>{}, save);
    else if (tiles >= 256 && ptiles >= 2)
      go(n, std::integral_constant<int, 2>{}, save);
    else
      go(n, std::integral_constant<int, 4>{}, save);
  };
  auto pick = [&](auto save) {
    switch (p.N) {
      case 16: pick_ns(std::integral_constant<int, 16>{}, save); break;
      case 32: pick_ns(std::integral_constant<int, 32>{}, save); break;
      case 64: pick_ns(std::integral_constant<int, 64>{}, save); break;
      default: pick_ns(std::integral_constant<int, 128>{}, save); break;
    }
  };
  a.S ? pick(std::true_type{}) : pick(std::false_type{});
  return hipGetLastError();
}

}  // namespace ssd
