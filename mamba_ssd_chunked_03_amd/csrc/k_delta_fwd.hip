// Gated delta rule, forward chain: a workgroup of four waves walks one sequence's
// chunks for PT columns of headdim of one head (those do not interact), the PT x N
// state in registers in fp32.  Per chunk of 64 tokens:
//   1. K S^T and Q S^T (tokens x PT; wave w: tokens 16w..16w+15), X = V - exp(G) K S^T;
//   2. Z = X - R (b X), U = b Z;
//   3. S <- exp(G_C) S + (exp(G_C - G) U)^T K  (wave w: a quarter of the N columns);
//   4. O = scale exp(G) Q S^T + P U.
// Operands that change owners between the steps go through LDS as bf16 planes, three
// barriers a chunk.  All tiles are computed transposed (rows headdim or dstate, columns
// tokens or headdim), so that a lane holds four consecutive elements of a row of V, O,
// the state and the planes.
//
// The output is formed here rather than in a kernel of its own: that would store and
// read back a state (P N fp32) and Z for every chunk and head.
#include "delta.hpp"

namespace ssd {

template <int N, int PT, class IO, bool SAVE>
__global__ __launch_bounds__(256) void delta_fwd_kernel(DeltaArgs a) {
  using T = typename IO::T;
  constexpr int PI = IO::PI, PM = IO::PM, PF = IO::PI, ES = sizeof(T);
  constexpr int NP = N < 32 ? 32 : N, KS = NP / 32, NT = PT / 16;
  constexpr int TN = N / 16, TW = (TN + 3) / 4;   // column tiles of the state, of a wave
  constexpr int LK = NP + 8, LX = PT;             // LDS row strides (elements)
  constexpr int C = kDeltaChunk, KPLANE = C * LK, SPLANE = PT * LK, XPLANE = C * LX;
  __shared__ __align__(16) uint16_t Kl[2][PI * KPLANE];
  __shared__ __align__(16) uint16_t Sl[PM * SPLANE];
  __shared__ __align__(16) uint16_t Xl[PM * XPLANE], Ul[PM * XPLANE], Wl[PM * XPLANE];

  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, q = lane >> 4, r = lane & 15;
  const int np = a.P / PT;
  const int wg = xcd_order(blockIdx.x, gridDim.x);
  const int p0 = (wg % np) * PT, h = (wg / np) % a.H, s = wg / np / a.H;
  const int grp = h / (a.H / a.G);
  const SeqSpan sp = seq_span(a.map, s);
  const int c0 = sp.c0, c1 = sp.c1;

  // the state: tile (i, t) of wave w holds columns 16 (w TW + i) + 4q + e, row p0 + 16t + r
  f32x4 S[TW][NT];
  const int64_t sbase = ((int64_t)s * a.H + h) * a.P * N;
#pragma unroll
  for (int i = 0; i < TW; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int nt = w * TW + i;
      S[i][t] = a.init && nt < TN ? *(const f32x4*)(a.init + sbase + (int64_t)(p0 + 16 * t + r) * N + 16 * nt + 4 * q)
                                  : f32x4{0.f, 0.f, 0.f, 0.f};
    }
  auto put_state = [&]() {
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int nt = w * TW + i;
        if (nt < TN) {
          uint2 o[PM];
          split4<PM>(S[i][t], o);
#pragma unroll
          for (int e = 0; e < PM; ++e)
            *(uint2*)(Sl + e * SPLANE + (16 * t + r) * LK + 16 * nt + 4 * q) = o[e];
        }
      }
  };
  if constexpr (N < 32) {  // the products' depth is 32: columns past N are zero
    for (int e = tid; e < 2 * PI * C; e += 256)
      for (int c = N; c < 32; c += 4) *(uint2*)(&Kl[0][0] + e * LK + c) = make_uint2(0u, 0u);
    for (int e = tid; e < PM * PT; e += 256)
      for (int c = N; c < 32; c += 4) *(uint2*)(Sl + e * LK + c) = make_uint2(0u, 0u);
  }
  put_state();

  // what a chunk reads from memory, loaded a chunk ahead
  constexpr int PC = N / 8, KC = (C * PC + 255) / 256;  // 8-element pieces of a K row, of a thread
  struct Loads {
    Raw8<IO> k[KC], q[KS];
    u32x4 R[2][PM], P[2][PF];
    Raw4<IO> v[NT];
    float Gh, Gl, b, Ch, Cl;
  };
  auto load = [&](Loads& x, int c) {
    const int start = sp.start + (c - c0) * C, len = min(C, sp.end - start);
    const uint32_t row = (uint32_t)a.G * N * ES, span = (uint32_t)(len - 1) * row + N * ES;
    const int64_t base = ((int64_t)start * a.G + grp) * N * ES;
    const brsrc rk = make_rsrc((const char*)a.k + base, span), rq = make_rsrc((const char*)a.q + base, span);
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int e = tid + i * 256;
      x.k[i].load(rk, e < C * PC ? (e / PC) * row + (e % PC) * 8 * ES : kNoOffset);
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      x.q[ks].load(rq, 32 * ks + 8 * q < N ? (16 * w + r) * row + (32 * ks + 8 * q) * ES : kNoOffset);
    const int64_t kh = (int64_t)c * a.H + h;
    const uint16_t* R = a.R + kh * (PM * kTriPlane) + lane * 8;
    const uint16_t* P = a.Pm + kh * (PF * kTriPlane) + lane * 8;
#pragma unroll
    for (int S2 = 0; S2 < 2; ++S2) {
      const int blk = tri_block(w, w >= 2 ? S2 : 0) * 512;  // (waves 0, 1: block 1 is not used)
#pragma unroll
      for (int e = 0; e < PM; ++e) x.R[S2][e] = *(const u32x4*)(R + e * kTriPlane + blk);
#pragma unroll
      for (int e = 0; e < PF; ++e) x.P[S2][e] = *(const u32x4*)(P + e * kTriPlane + blk);
    }
    const uint32_t vrow = (uint32_t)a.H * a.P * ES;
    const brsrc rv = make_rsrc((const char*)a.v + (((int64_t)start * a.H + h) * a.P + p0) * ES,
                               (uint32_t)(len - 1) * vrow + PT * ES);
#pragma unroll
    for (int t = 0; t < NT; ++t) x.v[t].load(rv, (16 * w + r) * vrow + (16 * t + 4 * q) * ES);
    const float* gt = a.gates + kh * (3 * C);
    x.Gh = gt[16 * w + r];
    x.Gl = gt[C + 16 * w + r];
    x.b = gt[2 * C + 16 * w + r];
    x.Ch = gt[C - 1];
    x.Cl = gt[2 * C - 1];
  };
  auto put_k = [&](const Loads& x, int buf) {
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      const int e = tid + i * 256;
      u32x4 o[PI];
      x.k[i].planes(o);
      if (e < C * PC)
#pragma unroll
        for (int m = 0; m < PI; ++m) *(u32x4*)(&Kl[buf][0] + m * KPLANE + (e / PC) * LK + (e % PC) * 8) = o[m];
    }
  };

  Loads x;
  if (c0 < c1) {
    load(x, c0);
    put_k(x, 0);
  }
  __syncthreads();
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  for (int c = c0; c < c1; ++c) {
    const uint16_t* Kc = Kl[(c - c0) & 1];
    const int64_t kh = (int64_t)c * a.H + h;
    const float eG = exp2_hl(x.Gh, x.Gl), eC = exp2_hl(x.Ch, x.Cl);
    const float eR = exp2_fast((x.Ch - x.Gh) + (x.Cl - x.Gl)), b = x.b;
    f32x4 ks_[NT], qs[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) ks_[t] = qs[t] = zero;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const Planes<PI> kf = lds_rows<PI>(Kc + 16 * w * LK + 32 * ks, LK, KPLANE, lane), qf = raw_planes<IO>(x.q[ks]);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const Planes<PM> sf = lds_rows<PM>(Sl + 16 * t * LK + 32 * ks, LK, SPLANE, lane);
        ks_[t] = mma<PM>(sf, kf, ks_[t]);
        qs[t] = mma<PM>(sf, qf, qs[t]);
      }
    }
    const int xo = (16 * w + r) * LX + 4 * q;
    f32x4 X[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      X[t] = x.v[t].get() - eG * ks_[t];
      uint2 o[PM];
      split4<PM>(b * X[t], o);
#pragma unroll
      for (int e = 0; e < PM; ++e) *(uint2*)(Xl + e * XPLANE + xo + 16 * t) = o[e];
    }
    // the next chunk's loads are in flight from here on
    Planes<PM> Rf[2];
    Planes<PF> Pf[2];
#pragma unroll
    for (int S2 = 0; S2 < 2; ++S2) {
#pragma unroll
      for (int e = 0; e < PM; ++e) Rf[S2].p[e] = as_bf16x8(x.R[S2][e]);
#pragma unroll
      for (int e = 0; e < PF; ++e) Pf[S2].p[e] = as_bf16x8(x.P[S2][e]);
    }
    if (c + 1 < c1) load(x, c + 1);
    __syncthreads();
    // 2. Z = X - R (b X)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      f32x4 z = zero;
      z = mma<PM>(lds_cols<PM>(Xl + 16 * t, LX, XPLANE, lane), Rf[0], z);
      if (w >= 2) z = mma<PM>(lds_cols<PM>(Xl + 32 * LX + 16 * t, LX, XPLANE, lane), Rf[1], z);
      z = X[t] - z;
      if constexpr (SAVE) *(f32x4*)(a.Z + (kh * C + 16 * w + r) * a.P + p0 + 16 * t + 4 * q) = z;
      uint2 o[PM];
      split4<PM>(b * z, o);
#pragma unroll
      for (int e = 0; e < PM; ++e) *(uint2*)(Ul + e * XPLANE + xo + 16 * t) = o[e];
      split4<PM>((eR * b) * z, o);
#pragma unroll
      for (int e = 0; e < PM; ++e) *(uint2*)(Wl + e * XPLANE + xo + 16 * t) = o[e];
    }
    __syncthreads();
    // 3. the state
#pragma unroll
    for (int i = 0; i < TW; ++i) {
      const int nt = w * TW + i;
      if (nt < TN) {
        Planes<PI> kf[2];
#pragma unroll
        for (int S2 = 0; S2 < 2; ++S2) kf[S2] = lds_cols<PI>(Kc + 32 * S2 * LK + 16 * nt, LK, KPLANE, lane);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if constexpr (SAVE)
            *(f32x4*)(a.S + (kh * a.P + p0 + 16 * t + r) * N + 16 * nt + 4 * q) = S[i][t];
          f32x4 acc = eC * S[i][t];
#pragma unroll
          for (int S2 = 0; S2 < 2; ++S2)
            acc = mma<PM>(kf[S2], lds_cols<PM>(Wl + 32 * S2 * LX + 16 * t, LX, XPLANE, lane), acc);
          S[i][t] = acc;
        }
      }
    }
    put_state();
    // 4. the output (none where the backward recomputes what a forward keeps)
    if (a.out) {
      const int start = sp.start + (c - c0) * C, len = min(C, sp.end - start);
      const uint32_t vrow = (uint32_t)a.H * a.P * ES;
      const brsrc ro = make_rsrc((char*)a.out + (((int64_t)start * a.H + h) * a.P + p0) * ES,
                                 (uint32_t)(len - 1) * vrow + PT * ES);
      const float se = a.scale * eG;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        f32x4 o = se * qs[t];
        o = mma<PM>(lds_cols<PM>(Ul + 16 * t, LX, XPLANE, lane), Pf[0], o);
        if (w >= 2) o = mma<PM>(lds_cols<PM>(Ul + 32 * LX + 16 * t, LX, XPLANE, lane), Pf[1], o);
        store4io(ro, (16 * w + r) * vrow + (16 * t + 4 * q) * ES, o, IO{});
      }
    }
    if (c + 1 < c1) put_k(x, (c + 1 - c0) & 1);
    __syncthreads();
  }
  if (a.final_states) {
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int nt = w * TW + i;
        if (nt < TN) *(f32x4*)(a.final_states + sbase + (int64_t)(p0 + 16 * t + r) * N + 16 * nt + 4 * q) = S[i][t];
      }
  }
}

hipError_t launch_delta_fwd(const DeltaProb& p, const DeltaArgs& a, hipStream_t st) {
  if (p.nst == 0) return hipSuccess;
  auto go = [&](auto n, auto io, auto save) {
    constexpr int N = decltype(n)::value;
    using IO = decltype(io);
    constexpr int PT = 16;
    hipLaunchKernelGGL((delta_fwd_kernel<N, PT, IO, decltype(save)::value>),
                       dim3((unsigned)((int64_t)p.nst * p.H * (p.P / PT))), dim3(256), 0, st, a);
  };
  auto pick = [&](auto io, auto save) {
    switch (p.N) {
      case 16: go(std::integral_constant<int, 16>{}, io, save); break;
      case 32: go(std::integral_constant<int, 32>{}, io, save); break;
      case 64: go(std::integral_constant<int, 64>{}, io, save); break;
      default: go(std::integral_constant<int, 128>{}, io, save); break;
    }
  };
  if (p.io)
    a.S ? pick(IoBf16{}, std::true_type{}) : pick(IoBf16{}, std::false_type{});
  else
    a.S ? pick(IoF32{}, std::true_type{}) : pick(IoF32{}, std::false_type{});
  return hipGetLastError();
}

}  // namespace ssd
