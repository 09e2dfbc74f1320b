// Gated delta rule, gradients of q, k, g and beta, one workgroup per chunk and group of
// heads, from what the chains kept: per head the state S entering the chunk, the adjoint
// dS of the one leaving it, Z and F (U = b Z, dX = b F).  With
//   dP = scale (dO U^T) . D (lower),  dM = -(dX U^T) . D (strictly lower):
//   dq       = scale exp(G) dO S + dP K
//   dk_read  = -exp(G) dX S + dM K            (k erasing)
//   dk_write = exp(G_C - G) U dS + dP^T Q + dM^T K   (k written into the state)
//   dbeta_i  = F_i . Z_i
// The gates act through the running sum G only, and each row of Q, K enters with its
// exp(+-G), so dL/dG_i = q_i . dq_i + k_i . dk_read_i - k_i . dk_write_i, plus
// <S', dS> at the chunk's end for the whole decay (S' the state leaving it).  S' holds
// the writes w_j = k_j . (exp(G_C - G) U dS)_j that dk_write takes out again: kept apart,
// w_j enters dg_i as the sum over j < i and exp(G_C) <S, dS> alone is carried, instead of
// two large sums that cancel.  dg is the suffix sum of dL/dG within the chunk.
//
// dq and dk are summed over the group's heads in registers, in order.  Eight waves: wave
// w has tokens 16 (w % 4).. and one half of the N columns (w / 4); dP, dM are formed by
// the two halves.
#include "delta.hpp"

namespace ssd {

template <int N, int P, class IO>
__global__ __launch_bounds__(512) void delta_grads_kernel(DeltaArgs a) {
  using T = typename IO::T;
  constexpr int PI = IO::PI, PM = IO::PM, ES = sizeof(T), C = kDeltaChunk, NTH = 512;
  constexpr int NP = N < 32 ? 32 : N;
  // columns of headdim staged at a time (the products' depth is 32; past P they are zero)
  constexpr int PB = P < 32 ? 32 : (P > (PM == 2 ? 64 : 32) ? (PM == 2 ? 64 : 32) : P), NB = (P + PB - 1) / PB;
  constexpr int LN = N + 8, LP = PB + 8, LC = C + 8;  // rows: dstate; headdim; tokens
  constexpr int TN = N / 16, TH = (TN + 1) / 2;  // column tiles, of one half
  constexpr int SPL = PB * LN, UPL = PB * LC, OPL = C * LP, KPL = C * LN, CPL = C * LC;
  // bf16 io: K and Q stay in LDS over the heads; fp32 io: they share the states' place
  constexpr bool KEEP = PI == 1;
  constexpr int PH1 = 2 * PM * SPL + 2 * PM * UPL + PI * OPL, PH2 = 2 * PM * CPL + (KEEP ? 0 : 2 * PI * KPL);
  __shared__ __align__(16) uint16_t lds[(PH1 > PH2 ? PH1 : PH2) + (KEEP ? 2 * PI * KPL : 0)];
  uint16_t *Sl = lds, *Dl = Sl + PM * SPL, *Ul = Dl + PM * SPL, *Xl = Ul + PM * UPL, *Ol = Xl + PM * UPL;
  uint16_t *Pl = lds, *Ml = Pl + PM * CPL;
  uint16_t *Kl = KEEP ? lds + (PH1 > PH2 ? PH1 : PH2) : Ml + PM * CPL, *Ql = Kl + PI * KPL;
  __shared__ __align__(16) float gl[3 * C];
  __shared__ float red[2][2][C], sd[NTH / 64], bsum[2][C];

  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, q = lane >> 4, r = lane & 15;
  const int tb = w & 3, nh = w >> 2, tok = 16 * tb + r;
  const int wg = xcd_order(blockIdx.x, gridDim.x);
  const int ck = wg / a.G, grp = wg % a.G, per = a.H / a.G;
  ChunkInfo ci = chunk_info(a.map, ck);
  const int start = __builtin_amdgcn_readfirstlane(ci.start), len = __builtin_amdgcn_readfirstlane(ci.len);
  if (len <= 0) return;
  const uint32_t krow = (uint32_t)a.G * N * ES, kspan = (uint32_t)(len - 1) * krow + N * ES;
  const int64_t kbase = ((int64_t)start * a.G + grp) * N * ES;
  const brsrc rk = make_rsrc((const char*)a.k + kbase, kspan), rq = make_rsrc((const char*)a.q + kbase, kspan);
  const uint32_t vrow = (uint32_t)a.H * P * ES;
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  auto put_kq = [&]() {
    for (int e = tid; e < C * N / 8; e += NTH) {
      const int t = e / (N / 8), col = (e % (N / 8)) * 8;
      Raw8<IO> k8, q8;
      k8.load(rk, t * krow + col * ES);
      q8.load(rq, t * krow + col * ES);
      u32x4 o[PI];
      k8.planes(o);
#pragma unroll
      for (int m = 0; m < PI; ++m) *(u32x4*)(Kl + m * KPL + t * LN + col) = o[m];
      q8.planes(o);
#pragma unroll
      for (int m = 0; m < PI; ++m) *(u32x4*)(Ql + m * KPL + t * LN + col) = o[m];
    }
  };
  if constexpr (KEEP) put_kq();

  // What a head (and block of headdim) needs from memory: the states (PB x N), Z and F
  // (PB x 64) in tile order, dO (64 x PB), beta of this thread's tokens, the gates.  Loaded
  // into registers while the one before is worked on, all through range-checked resources
  // (past headdim they are zero).
  constexpr int SE = PB * NP / 4, RE = PB * C / 4, OE = C * PB / 8;
  constexpr int SC = (SE + NTH - 1) / NTH, RC = (RE + NTH - 1) / NTH;
  static_assert(OE <= NTH && 3 * C <= NTH, "one piece a thread");
  const int tk4 = 32 * ((w & 3) >> 1) + 8 * q + 4 * (w & 1);  // (a thread's tokens are the same in every tile)
  const int ot = tid / (PB / 8), oc = (tid % (PB / 8)) * 8;
  u32x4 xs[SC], xd[SC], xz[RC], xf_[RC], xb;
  Raw8<IO> xo;
  float xg;
  auto scol = [&](int e) { return 32 * (((e >> 6) % (NP / 16)) >> 1) + 8 * q + 4 * ((e >> 6) & 1); };
  auto load = [&](int hh, int pb) {
    const int h = grp * per + hh;
    const int64_t kh = (int64_t)ck * a.H + h;
    const brsrc rs = make_rsrc(a.S + kh * P * NP, P * NP * 4), rd = make_rsrc(a.dS + kh * P * NP, P * NP * 4);
#pragma unroll
    for (int i = 0; i < SC; ++i) {
      const int e = tid + i * NTH;
      const uint32_t off = (SE % NTH == 0 || e < SE) && (N == NP || scol(e) < N) ? (pb * SE + e) * 16 : kNoOffset;
      xs[i] = buf_load16(rs, off);
      xd[i] = buf_load16(rd, off);
    }
    const brsrc rz = make_rsrc(a.Z + kh * C * P, C * P * 4), rf = make_rsrc(a.F + kh * C * P, C * P * 4);
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      const int e = tid + i * NTH;
      xz[i] = buf_load16(rz, (pb * RE + e) * 16);
      xf_[i] = buf_load16(rf, (pb * RE + e) * 16);
    }
    const brsrc ro = make_rsrc((const char*)a.dout + ((int64_t)start * a.H + h) * P * ES,
                               (uint32_t)(len - 1) * vrow + P * ES);
    xo.load(ro, tid < OE && pb * PB + oc < P ? ot * vrow + (pb * PB + oc) * ES : kNoOffset);
    const brsrc rg = make_rsrc(a.gates + kh * kDeltaGates, 3 * C * 4);
    xb = buf_load16(rg, (2 * C + tk4) * 4);
    xg = buf_load_f32(rg, tid * 4);
  };

  f32x4 dqs[TH], dks[TH];
#pragma unroll
  for (int i = 0; i < TH; ++i) dqs[i] = dks[i] = zero;

  load(0, 0);
#pragma unroll 1
  for (int hh = 0; hh < per; ++hh) {
    const int h = grp * per + hh;
    const brsrc rdv = make_rsrc((char*)a.dv + ((int64_t)start * a.H + h) * P * ES, (uint32_t)(len - 1) * vrow + P * ES);
    f32x4 dq[TH], dr[TH], dw[TH], cc[4];
#pragma unroll
    for (int i = 0; i < TH; ++i) dq[i] = dr[i] = dw[i] = zero;
#pragma unroll
    for (int i = 0; i < 4; ++i) cc[i] = zero;
    float sdot = 0.f;
    f32x4 bdot = zero;  // F . Z of four tokens, this thread's rows
#pragma unroll 1
    for (int pb = 0; pb < NB; ++pb) {
#pragma unroll
      for (int i = 0; i < SC; ++i) {
        const int e = tid + i * NTH, row = (e >> 6) / (NP / 16) * 16 + r, col = scol(e);
        const f32x4 x = __builtin_bit_cast(f32x4, xs[i]), y = __builtin_bit_cast(f32x4, xd[i]);
        sdot += x[0] * y[0] + x[1] * y[1] + x[2] * y[2] + x[3] * y[3];
        if ((SE % NTH == 0 || e < SE) && (N == NP || col < N)) {
          uint2 o[PM];
          split4<PM>(x, o);
#pragma unroll
          for (int m = 0; m < PM; ++m) *(uint2*)(Sl + m * SPL + row * LN + col) = o[m];
          split4<PM>(y, o);
#pragma unroll
          for (int m = 0; m < PM; ++m) *(uint2*)(Dl + m * SPL + row * LN + col) = o[m];
        }
      }
      const f32x4 b = __builtin_bit_cast(f32x4, xb);
#pragma unroll
      for (int i = 0; i < RC; ++i) {
        const int e = tid + i * NTH, row = (e >> 8) * 16 + r;
        const f32x4 z = __builtin_bit_cast(f32x4, xz[i]), f = __builtin_bit_cast(f32x4, xf_[i]);
        bdot += z * f;
        uint2 o[PM];
        split4<PM>(b * z, o);
#pragma unroll
        for (int m = 0; m < PM; ++m) *(uint2*)(Ul + m * UPL + row * LC + tk4) = o[m];
        split4<PM>(b * f, o);
#pragma unroll
        for (int m = 0; m < PM; ++m) *(uint2*)(Xl + m * UPL + row * LC + tk4) = o[m];
      }
      if (OE == NTH || tid < OE) {
        u32x4 o[PI];
        xo.planes(o);
#pragma unroll
        for (int m = 0; m < PI; ++m) *(u32x4*)(Ol + m * OPL + ot * LP + oc) = o[m];
      }
      if (tid < 3 * C) gl[tid] = xg;
      if constexpr (NB > 1) {
        const int it = min(hh * NB + pb + 1, per * NB - 1);
        load(it / NB, it % NB);
      }
      __syncthreads();
      // (the lane, as the compiler cannot see it to be the same: operand addresses are formed
      // anew in each phase rather than kept in registers over the heads)
      int ln = lane;
      asm("" : "+v"(ln));
#pragma unroll 1
      for (int ks = 0; ks < PB / 32; ++ks) {
        const Planes<PI> of = lds_rows<PI>(Ol + 16 * tb * LP + 32 * ks, LP, OPL, ln);
        const Planes<PM> xf = lds_cols<PM>(Xl + 32 * ks * LC + 16 * tb, LC, UPL, ln);
        const Planes<PM> uf = lds_cols<PM>(Ul + 32 * ks * LC + 16 * tb, LC, UPL, ln);
#pragma unroll
        for (int i = 0; i < TH; ++i) {
          const int nt = nh * TH + i;
          if (nt < TN) {
            const Planes<PM> sf = lds_cols<PM>(Sl + 32 * ks * LN + 16 * nt, LN, SPL, ln);
            dq[i] = mma<PM>(sf, of, dq[i]);
            dr[i] = mma<PM>(sf, xf, dr[i]);
            dw[i] = mma<PM>(lds_cols<PM>(Dl + 32 * ks * LN + 16 * nt, LN, SPL, ln), uf, dw[i]);
          }
        }
        // dX rounded to bf16 is its first plane: dV (the fp32 chain stores its own)
        if constexpr (PI == 1)
          if (nh == 0 && pb * PB + 32 * ks + 8 * (ln >> 4) < P)
            buf_store16(rdv, (16 * tb + (ln & 15)) * vrow + (pb * PB + 32 * ks + 8 * (ln >> 4)) * ES, __builtin_bit_cast(u32x4, xf.p[0]));
        // rows j (block J), columns i: the first half dO U^T, the second dX U^T
#pragma unroll
        for (int J = 0; J < 4; ++J)
          if (J <= tb) {
            const Planes<PM> jf = lds_cols<PM>(Ul + 32 * ks * LC + 16 * J, LC, UPL, ln);
            cc[J] = nh == 0 ? mma<PM>(jf, of, cc[J]) : mma<PM>(jf, xf, cc[J]);
          }
      }
      __syncthreads();
    }
    const float Gh = gl[tok], Gl = gl[C + tok];
    const float eG = exp2_hl(Gh, Gl), eR = exp2_fast((gl[C - 1] - Gh) + (gl[2 * C - 1] - Gl));
#pragma unroll
    for (int i = 0; i < TH; ++i) {
      dq[i] = (a.scale * eG) * dq[i];
      dr[i] = -eG * dr[i];
      dw[i] = eR * dw[i];
    }
    // dP (first half) or dM (second), [i][j]; the block right of an even diagonal one is read
    // in the same step of 32 and written as zero
    {
      uint16_t* dst = nh == 0 ? Pl : Ml;
      const float f = nh == 0 ? a.scale : -1.f;
#pragma unroll
      for (int J = 0; J < 4; ++J) {
        if (J > tb && !(J == tb + 1 && (tb & 1) == 0)) continue;
        f32x4 v = zero;
        if (J <= tb) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = 16 * J + 4 * q + e;
            const float d = exp2_fast((Gh - gl[j]) + (Gl - gl[C + j]));
            v[e] = (nh == 0 ? j <= tok : j < tok) ? f * (cc[J][e] * d) : 0.f;
          }
        }
        uint2 o[PM];
        split4<PM>(v, o);
#pragma unroll
        for (int m = 0; m < PM; ++m) *(uint2*)(dst + m * CPL + tok * LC + 16 * J + 4 * q) = o[m];
      }
    }
    if constexpr (!KEEP) put_kq();
    __syncthreads();
    // (one block of headdim: the next head's loads, where the registers of the first part are free)
    if constexpr (NB == 1) load(min(hh + 1, per - 1), 0);
    int l2 = lane;
    asm("" : "+v"(l2));
    const int q2 = l2 >> 4, t2 = 16 * tb + (l2 & 15);
    float da = 0.f, dwr = 0.f;  // this lane's part of dL/dG and of w
#pragma unroll
    for (int i = 0; i < TH; ++i) {
      const int nt = nh * TH + i;
      if (nt < TN) {
        const f32x4 w0 = dw[i];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          const Planes<PI> kf = lds_cols<PI>(Kl + 32 * ks * LN + 16 * nt, LN, KPL, l2);
          if (ks == 0 || tb >= 2) {  // i in this block, j up to it
            dq[i] = mma<PM>(kf, lds_rows<PM>(Pl + 16 * tb * LC + 32 * ks, LC, CPL, l2), dq[i]);
            dr[i] = mma<PM>(kf, lds_rows<PM>(Ml + 16 * tb * LC + 32 * ks, LC, CPL, l2), dr[i]);
          }
          if (ks == 1 || tb < 2) {  // j in this block, i from it on
            const Planes<PI> qf = lds_cols<PI>(Ql + 32 * ks * LN + 16 * nt, LN, KPL, l2);
            dw[i] = mma<PM>(qf, lds_cols<PM>(Pl + 32 * ks * LC + 16 * tb, LC, CPL, l2), dw[i]);
            dw[i] = mma<PM>(kf, lds_cols<PM>(Ml + 32 * ks * LC + 16 * tb, LC, CPL, l2), dw[i]);
          }
        }
        f32x4 kv = zero, qv = zero;  // (planes add up to the input exactly)
#pragma unroll
        for (int m = PI - 1; m >= 0; --m) {
          const uint2 kw = *(const uint2*)(Kl + m * KPL + t2 * LN + 16 * nt + 4 * q2);
          const uint2 qw = *(const uint2*)(Ql + m * KPL + t2 * LN + 16 * nt + 4 * q2);
          kv += f32x4{bf_lo(kw.x), bf_hi(kw.x), bf_lo(kw.y), bf_hi(kw.y)};
          qv += f32x4{bf_lo(qw.x), bf_hi(qw.x), bf_lo(qw.y), bf_hi(qw.y)};
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          da += qv[e] * dq[i][e] + kv[e] * (dr[i][e] - (dw[i][e] - w0[e]));
          dwr += kv[e] * w0[e];
        }
        dqs[i] += dq[i];
        dks[i] += dr[i] + dw[i];
      }
    }
    da += __shfl_xor(da, 16);
    da += __shfl_xor(da, 32);
    dwr += __shfl_xor(dwr, 16);
    dwr += __shfl_xor(dwr, 32);
    if (q == 0) {
      red[0][nh][tok] = da;
      red[1][nh][tok] = dwr;
    }
    sdot = wave_sum(sdot);
    if (lane == 0) sd[w] = sdot;
    // F . Z over the rows: 16 lanes, then two waves in order
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = row_sum16(bdot[e]);
      if (r == 0) bsum[w >> 2][tk4 + e] = v;
    }
    __syncthreads();
    if (w == 0) {
      double x = (double)red[0][0][lane] + (double)red[0][1][lane];
      double y = (double)red[1][0][lane] + (double)red[1][1][lane];
      const double wj = y;
      if (lane == C - 1) {
        float t = 0.f;
        for (int i = 0; i < NTH / 64; ++i) t += sd[i];
        x += (double)(exp2_hl(gl[C - 1], gl[2 * C - 1]) * t);
      }
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double u = __shfl_down(x, d), v = __shfl_up(y, d);
        if (lane + d < 64) x += u;
        if (lane >= d) y += v;
      }
      if (lane < len) {
        const int64_t at = ((int64_t)start + lane) * a.H + h;
        a.dg[at] = (float)(x + (y - wj));
        a.dbeta[at] = bsum[0][lane] + bsum[1][lane];
      }
    }
    __syncthreads();  // (the next head's data goes where P, M and the gates are)
  }
  const brsrc wq = make_rsrc((char*)a.dq + kbase, kspan), wk = make_rsrc((char*)a.dk + kbase, kspan);
#pragma unroll
  for (int i = 0; i < TH; ++i) {
    const int nt = nh * TH + i;
    if (nt < TN) {
      store4io(wq, tok * krow + (16 * nt + 4 * q) * ES, dqs[i], IO{});
      store4io(wk, tok * krow + (16 * nt + 4 * q) * ES, dks[i], IO{});
    }
  }
}

hipError_t launch_delta_bwd_grads(const DeltaProb& p, const DeltaArgs& a, hipStream_t st) {
  if (p.nck == 0) return hipSuccess;
  const dim3 grid((unsigned)(p.nck * p.G)), block(512);
  auto pick_p = [&](auto n, auto io) {
    constexpr int N = decltype(n)::value;
    using IO = decltype(io);
    switch (p.P) {
      case 16: hipLaunchKernelGGL((delta_grads_kernel<N, 16, IO>), grid, block, 0, st, a); break;
      case 32: hipLaunchKernelGGL((delta_grads_kernel<N, 32, IO>), grid, block, 0, st, a); break;
      case 64: hipLaunchKernelGGL((delta_grads_kernel<N, 64, IO>), grid, block, 0, st, a); break;
      default: hipLaunchKernelGGL((delta_grads_kernel<N, 128, IO>), grid, block, 0, st, a); break;
    }
  };
  auto pick = [&](auto io) {
    switch (p.N) {
      case 16: pick_p(std::integral_constant<int, 16>{}, io); break;
      case 32: pick_p(std::integral_constant<int, 32>{}, io); break;
      case 64: pick_p(std::integral_constant<int, 64>{}, io); break;
      default: pick_p(std::integral_constant<int, 128>{}, io); break;
    }
  };
  p.io ? pick(IoBf16{}) : pick(IoF32{});
  return hipGetLastError();
}

}  // namespace ssd
