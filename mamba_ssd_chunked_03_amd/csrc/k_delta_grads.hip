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
// dq and dk are summed over the group's heads in registers, in order (of few chunks and groups, a
// workgroup takes one head, and delta_head_sum_kernel adds them up).  Eight waves: wave w
// has tokens 32 (w % 2)..+31 and a quarter (w / 2) of the N columns, which reads each
// operand from LDS two to four times (16 tokens and half the columns a wave: 1.3 times as
// much; sixteen waves, 1.5 times as much, 925 us below), and three of the 24 blocks of dP and
// dM that are formed (16 rows a wave: 5% more).  The running sums of a head's gates are formed
// by one wave while the others begin the next head.
// 2 x 8192 tokens, 64 heads in 8 groups, 64 x 128: 737 us, 11 a head, of which a workgroup's
// matrix instructions take 1.7, vector ones 3.5, and LDS 5 with its conflicts: phases between
// barriers, two waves a SIMD, with the next head's loads in flight (2.6 TB/s).  (LDS rows
// exchanged by an exclusive or instead of padded: a third of the conflicts, 12% more vector
// instructions, the same time.)
#include "delta.hpp"

namespace ssd {

template <int N, int P, class IO>
__global__ __launch_bounds__(512) void delta_grads_kernel(DeltaArgs a) {
  using T = typename IO::T;
  constexpr int PI = IO::PI, PM = IO::PM, ES = sizeof(T), C = kDeltaChunk, NW = 8, NTH = 64 * NW;
  constexpr int NP = N < 32 ? 32 : N;
  // columns of headdim staged at a time (the products' depth is 32; past P they are zero)
  constexpr int PB = P < 32 ? 32 : (P > (PM == 2 ? 64 : 32) ? (PM == 2 ? 64 : 32) : P), NB = (P + PB - 1) / PB;
  constexpr int LN = N + 8, LP = PB + 8, LC = C + 8;  // rows: dstate; headdim; tokens
  // a wave's part of the products: TB blocks of 16 tokens, one NQ-th of the column tiles
  constexpr int TN = N / 16, TB = 2, NT = 4 / TB, NQ = NW / NT, TQ = (TN + NQ - 1) / NQ;
  constexpr bool FULL = TN % NQ == 0;
  constexpr int SPL = PB * LN, UPL = PB * LC, OPL = C * LP, KPL = C * LN, CPL = C * LC;
  // bf16 io: K and Q stay in LDS over the heads; fp32 io: they share the states' place
  constexpr bool KEEP = PI == 1;
  constexpr int PH1 = 2 * PM * SPL + 2 * PM * UPL + PI * OPL, PH2 = 2 * PM * CPL + (KEEP ? 0 : 2 * PI * KPL);
  __shared__ __align__(16) uint16_t lds[(PH1 > PH2 ? PH1 : PH2) + (KEEP ? 2 * PI * KPL : 0)];
  uint16_t *Sl = lds, *Dl = Sl + PM * SPL, *Ul = Dl + PM * SPL, *Xl = Ul + PM * UPL, *Ol = Xl + PM * UPL;
  uint16_t *Pl = lds, *Ml = Pl + PM * CPL;
  uint16_t *Kl = KEEP ? lds + (PH1 > PH2 ? PH1 : PH2) : Ml + PM * CPL, *Ql = Kl + PI * KPL;
  // gates; row dots (of G and of w) of the NQ parts; parts of <S, dS> and exp(G_C); parts of dbeta
  __shared__ __align__(16) float gl[3 * C];
  __shared__ float red[2][NQ][C], sd[NW + 1], bsum[NW / 4][C];

  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, q = lane >> 4, r = lane & 15;
  const int tp = w % NT, nq = w / NT;
  // dP (first half of the waves) or dM, 16 x 16: ten blocks at or below the diagonal and, since a
  // product takes 32 columns at once, zeros right of two of them; block i of a wave's
  constexpr int CB = (12 + NW / 2 - 1) / (NW / 2);
  const int md = w / (NW / 2);
  auto low = [&](int i, int& t, int& j) {
    const int b = w % (NW / 2) + i * (NW / 2);
    t = (0x8ffa94 >> (2 * b)) & 3;
    j = (0xde4910 >> (2 * b)) & 3;
    return b < 12;
  };
  const int wg = xcd_order(blockIdx.x, gridDim.x);
  // heads h0..h1-1 of group grp: all of them, or one (their sums then follow in a kernel of its own)
  const int per = a.H / a.G, nh = a.parts ? a.H : a.G, ck = wg / nh, grp = a.parts ? wg % nh / per : wg % nh;
  const int h0 = a.parts ? wg % nh : grp * per, h1 = a.parts ? h0 + 1 : h0 + per;
  ChunkInfo ci = chunk_info(a.map, ck);
  const int start = __builtin_amdgcn_readfirstlane(ci.start), len = __builtin_amdgcn_readfirstlane(ci.len);
  if (len <= 0) return;
  const bool bare = ci.first && !a.init;
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
  constexpr int SC = (SE + NTH - 1) / NTH, RC = (RE + NTH - 1) / NTH, TPR = NP / 16;
  static_assert(OE <= NTH && 3 * C <= NTH && RE % NTH == 0 && NW % TPR == 0, "pieces of a thread");
  // wave w's tile i of the states: rows 16 (i NW / TPR + w / TPR).., column tile w % TPR; of Z
  // and F: rows 16 (i NW / 4 + w / 4).., token tile w % 4
  const int tk4 = 32 * ((w & 3) >> 1) + 8 * q + 4 * (w & 1);  // (the same tokens in each)
  const int scol = 32 * ((w % TPR) >> 1) + 8 * q + 4 * (w & 1);
  u32x4 xs[SC], xd[SC], xz[RC], xf_[RC], xb;
  Raw8<IO> xo;
  float xg;
  auto load_s = [&](int hh, int pb) {
    const int64_t kh = (int64_t)ck * a.H + hh;
    int td = tid;
    asm("" : "+v"(td));
    const brsrc rs = make_rsrc(a.S + kh * P * NP, P * NP * 4), rd = make_rsrc(a.dS + kh * P * NP, P * NP * 4);
#pragma unroll
    for (int i = 0; i < SC; ++i) {
      const uint32_t off = (SE % NTH == 0 || td + i * NTH < SE) && (N == NP || scol < N) ? td * 16 : kNoOffset;
      xs[i] = buf_load16(rs, off, (pb * SE + i * NTH) * 16);
      xd[i] = buf_load16(rd, off, (pb * SE + i * NTH) * 16);
    }
  };
  auto load = [&](int hh, int pb) {
    const int h = hh;
    const int64_t kh = (int64_t)ck * a.H + h;
    int td = tid;  // (not seen to be the same: the offsets are formed anew)
    asm("" : "+v"(td));
    const brsrc rz = make_rsrc(a.Z + kh * C * P, C * P * 4), rf = make_rsrc(a.F + kh * C * P, C * P * 4);
#pragma unroll
    for (int i = 0; i < RC; ++i) {
      xz[i] = buf_load16(rz, td * 16, (pb * RE + i * NTH) * 16);
      xf_[i] = buf_load16(rf, td * 16, (pb * RE + i * NTH) * 16);
    }
    const brsrc ro = make_rsrc((const char*)a.dout + ((int64_t)start * a.H + h) * P * ES,
                               (uint32_t)(len - 1) * vrow + P * ES);
    const int ot = td / (PB / 8), oc = pb * PB + (td % (PB / 8)) * 8;
    xo.load(ro, td < OE && oc < P ? ot * vrow + oc * ES : kNoOffset);
    const brsrc rg = make_rsrc(a.gates + kh * kDeltaGates, 3 * C * 4);
    xb = buf_load16(rg, (2 * C + tk4) * 4);
    xg = buf_load_f32(rg, td * 4);
  };

  f32x4 dqs[TB][TQ], dks[TB][TQ];
#pragma unroll
  for (int b = 0; b < TB; ++b)
#pragma unroll
    for (int i = 0; i < TQ; ++i) dqs[b][i] = dks[b][i] = zero;
  // dg and dbeta of a head from its parts in LDS (one wave)
  auto gates = [&](int hh) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) t += sd[i];
    // suffix sums with the tokens in reverse over the lanes, prefix sums in order
    int lane = tid & 63;
    asm("" : "+v"(lane));
    const int rl = C - 1 - lane;
    float x = 0.f, wj = 0.f, db = 0.f;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      x += red[0][i][rl];
      wj += red[1][i][lane];
    }
#pragma unroll
    for (int i = 0; i < NW / 4; ++i) db += bsum[i][lane];
    if (lane == 0) x += sd[NW] * t;
    x = wave_inclusive_sum(x);
    const float y = wave_inclusive_sum(wj) - wj;
    x = __shfl(x, rl);
    if (lane < len) {
      const int64_t at = ((int64_t)start + lane) * a.H + hh;
      // (a gate with no state to decay: what is left of the sums there is their rounding)
      a.dg[at] = bare && lane == 0 ? 0.f * (x + y) : x + y;
      a.dbeta[at] = db;
    }
  };

  load_s(h0, 0);
  load(h0, 0);
#pragma unroll 1
  for (int hh = h0; hh < h1; ++hh) {
    const int h = hh;
    const brsrc rdv = make_rsrc((char*)a.dv + ((int64_t)start * a.H + h) * P * ES, (uint32_t)(len - 1) * vrow + P * ES);
    f32x4 dq[TB][TQ], dr[TB][TQ], dw[TB][TQ], cc[CB];
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int i = 0; i < TQ; ++i) dq[b][i] = dr[b][i] = dw[b][i] = zero;
#pragma unroll
    for (int i = 0; i < CB; ++i) cc[i] = zero;
    float sdot = 0.f;
    f32x4 bdot = zero;  // F . Z of four tokens, this thread's rows
#pragma unroll 1
    for (int pb = 0; pb < NB; ++pb) {
      int td = tid;
      asm("" : "+v"(td));
      const int lr = td & 15;
#pragma unroll
      for (int i = 0; i < SC; ++i) {
        const int at = (16 * (i * (NW / TPR) + w / TPR) + lr) * LN + scol;
        const f32x4 x = __builtin_bit_cast(f32x4, xs[i]), y = __builtin_bit_cast(f32x4, xd[i]);
        sdot += x[0] * y[0] + x[1] * y[1] + x[2] * y[2] + x[3] * y[3];
        if ((SE % NTH == 0 || td + i * NTH < SE) && (N == NP || scol < N)) {
          uint2 o[PM];
          split4<PM>(x, o);
#pragma unroll
          for (int m = 0; m < PM; ++m) *(uint2*)(Sl + m * SPL + at) = o[m];
          split4<PM>(y, o);
#pragma unroll
          for (int m = 0; m < PM; ++m) *(uint2*)(Dl + m * SPL + at) = o[m];
        }
      }
      const f32x4 b = __builtin_bit_cast(f32x4, xb);
#pragma unroll
      for (int i = 0; i < RC; ++i) {
        const int at = (16 * (NW / 4 * i + (w >> 2)) + lr) * LC + tk4;
        const f32x4 z = __builtin_bit_cast(f32x4, xz[i]), f = __builtin_bit_cast(f32x4, xf_[i]);
        bdot += z * f;
        uint2 o[PM];
        split4<PM>(b * z, o);
#pragma unroll
        for (int m = 0; m < PM; ++m) *(uint2*)(Ul + m * UPL + at) = o[m];
        split4<PM>(b * f, o);
#pragma unroll
        for (int m = 0; m < PM; ++m) *(uint2*)(Xl + m * UPL + at) = o[m];
      }
      if (OE == NTH || td < OE) {
        u32x4 o[PI];
        xo.planes(o);
#pragma unroll
        for (int m = 0; m < PI; ++m) *(u32x4*)(Ol + m * OPL + td / (PB / 8) * LP + (td % (PB / 8)) * 8) = o[m];
      }
      if (tid < 3 * C) gl[tid] = xg;
      if (pb == 0 && hh > h0 && w == hh % NW) gates(hh - 1);
      if constexpr (NB > 1) {
        const int it = min(hh * NB + pb + 1, h1 * NB - 1);
        load(it / NB, it % NB);
      }
      __syncthreads();
      // (the lane, as the compiler cannot see it to be the same: operand addresses are formed
      // anew in each phase rather than kept in registers over the heads)
      int ln = lane;
      asm("" : "+v"(ln));
#pragma unroll 1
      for (int ks = 0; ks < PB / 32; ++ks) {
        Planes<PI> of[TB];
        Planes<PM> xf[TB], uf[TB];
#pragma unroll
        for (int b = 0; b < TB; ++b) {
          of[b] = lds_rows<PI>(Ol + 16 * (TB * tp + b) * LP + 32 * ks, LP, OPL, ln);
          xf[b] = lds_cols<PM>(Xl + 32 * ks * LC + 16 * (TB * tp + b), LC, UPL, ln);
          uf[b] = lds_cols<PM>(Ul + 32 * ks * LC + 16 * (TB * tp + b), LC, UPL, ln);
        }
#pragma unroll
        for (int i = 0; i < TQ; ++i) {
          const int nt = nq * TQ + i;
          if (FULL || nt < TN) {
            const Planes<PM> sf = lds_cols<PM>(Sl + 32 * ks * LN + 16 * nt, LN, SPL, ln);
            const Planes<PM> df = lds_cols<PM>(Dl + 32 * ks * LN + 16 * nt, LN, SPL, ln);
#pragma unroll
            for (int b = 0; b < TB; ++b) {
              dq[b][i] = mma<PM>(sf, of[b], dq[b][i]);
              dr[b][i] = mma<PM>(sf, xf[b], dr[b][i]);
              dw[b][i] = mma<PM>(df, uf[b], dw[b][i]);
            }
          }
        }
        // dX rounded to bf16 is its first plane: dV (the fp32 chain stores its own)
        if constexpr (PI == 1) {
          const int p = pb * PB + 32 * ks + 8 * (ln >> 4);
          if (nq == 0 && p < P)
#pragma unroll
            for (int b = 0; b < TB; ++b)
              buf_store16(rdv, (16 * (TB * tp + b) + (ln & 15)) * vrow + p * ES, __builtin_bit_cast(u32x4, xf[b].p[0]));
        }
        // rows j (block J) of dO U^T or dX U^T, columns i (block I)
#pragma unroll
        for (int i = 0; i < CB; ++i) {
          int I, J;
          if (low(i, I, J) && J <= I) {
            const Planes<PM> jf = lds_cols<PM>(Ul + 32 * ks * LC + 16 * J, LC, UPL, ln);
            if (md == 0)
              cc[i] = mma<PM>(jf, lds_rows<PI>(Ol + 16 * I * LP + 32 * ks, LP, OPL, ln), cc[i]);
            else
              cc[i] = mma<PM>(jf, lds_cols<PM>(Xl + 32 * ks * LC + 16 * I, LC, UPL, ln), cc[i]);
          }
        }
      }
      if constexpr (NB > 1) {
        const int it = min(hh * NB + pb + 1, h1 * NB - 1);
        load_s(it / NB, it % NB);
      }
      __syncthreads();
    }
#pragma unroll
    for (int b = 0; b < TB; ++b) {
      const int tok = 16 * (TB * tp + b) + r;
      const float Gh = gl[tok], Gl = gl[C + tok];
      const float eG = exp2_hl(Gh, Gl), eR = exp2_fast((gl[C - 1] - Gh) + (gl[2 * C - 1] - Gl));
#pragma unroll
      for (int i = 0; i < TQ; ++i) {
        dq[b][i] = (a.scale * eG) * dq[b][i];
        dr[b][i] = -eG * dr[b][i];
        dw[b][i] = eR * dw[b][i];
      }
    }
    // dP or dM, [i][j]
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      int I, J;
      if (!low(i, I, J)) continue;
      uint16_t* dst = md == 0 ? Pl : Ml;
      const float f = md == 0 ? a.scale : -1.f;
      const int tok = 16 * I + r;
      f32x4 v = zero;
      if (J <= I) {
        const float Gh = gl[tok], Gl = gl[C + tok];
        const f32x4 jh = *(const f32x4*)(gl + 16 * J + 4 * q), jl = *(const f32x4*)(gl + C + 16 * J + 4 * q);
        const int last = tok - md - (16 * J + 4 * q);  // (dP with its diagonal, dM without)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = f * (cc[i][e] * exp2_fast((Gh - jh[e]) + (Gl - jl[e])));
          asm("" : "+v"(x));  // (formed in any case: no branch an element)
          v[e] = e <= last ? x : 0.f;
        }
      }
      uint2 o[PM];
      split4<PM>(v, o);
#pragma unroll
      for (int m = 0; m < PM; ++m) *(uint2*)(dst + m * CPL + tok * LC + 16 * J + 4 * q) = o[m];
    }
    if constexpr (!KEEP) put_kq();
    __syncthreads();
    // (one block of headdim: the next head's loads, where the registers of the first part are free)
    if constexpr (NB == 1) load(min(hh + 1, h1 - 1), 0);
    int l2 = lane;
    asm("" : "+v"(l2));
    const int q2 = l2 >> 4, r2 = l2 & 15;
    // k and q of a tile's token and columns (planes add up to the input exactly)
    auto value = [&](const uint16_t* X, int tok, int nt) {
      auto plane = [&](int m) {
        const uint2 x = *(const uint2*)(X + m * KPL + tok * LN + 16 * nt + 4 * q2);
        return f32x4{bf_lo(x.x), bf_hi(x.x), bf_lo(x.y), bf_hi(x.y)};
      };
      f32x4 v = plane(PI - 1);
#pragma unroll
      for (int m = PI - 2; m >= 0; --m) v += plane(m);
      return v;
    };
    float dwr[TB];  // this lane's part of w
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < TB; ++b) dwr[b] = 0.f;
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int i = 0; i < TQ; ++i)
        if (FULL || nq * TQ + i < TN) {
          const f32x4 kv = value(Kl, 16 * (TB * tp + b) + r2, nq * TQ + i);
#pragma unroll
          for (int e = 0; e < 4; ++e) dwr[b] += kv[e] * dw[b][i][e];
        }
    // (one block of tokens at a time, in parts that the scheduler keeps apart: registers)
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int b = 0; b < TB; ++b) {
        const int t0 = 16 * (TB * tp + b);
        if (ks == 0 || TB * tp >= 2) {  // j in this block, up to i
          const Planes<PM> pr = lds_rows<PM>(Pl + t0 * LC + 32 * ks, LC, CPL, l2);
          const Planes<PM> mr = lds_rows<PM>(Ml + t0 * LC + 32 * ks, LC, CPL, l2);
#pragma unroll
          for (int i = 0; i < TQ; ++i)
            if (FULL || nq * TQ + i < TN) {
              const Planes<PI> kf = lds_cols<PI>(Kl + 32 * ks * LN + 16 * (nq * TQ + i), LN, KPL, l2);
              dq[b][i] = mma<PM>(kf, pr, dq[b][i]);
              dr[b][i] = mma<PM>(kf, mr, dr[b][i]);
            }
        }
        if (ks == 1 || TB * tp < 2) {  // i in this block, from j on
          const Planes<PM> pc = lds_cols<PM>(Pl + 32 * ks * LC + t0, LC, CPL, l2);
          const Planes<PM> mc = lds_cols<PM>(Ml + 32 * ks * LC + t0, LC, CPL, l2);
#pragma unroll
          for (int i = 0; i < TQ; ++i)
            if (FULL || nq * TQ + i < TN) {
              const Planes<PI> kf = lds_cols<PI>(Kl + 32 * ks * LN + 16 * (nq * TQ + i), LN, KPL, l2);
              const Planes<PI> qf = lds_cols<PI>(Ql + 32 * ks * LN + 16 * (nq * TQ + i), LN, KPL, l2);
              dw[b][i] = mma<PM>(qf, pc, dw[b][i]);
              dw[b][i] = mma<PM>(kf, mc, dw[b][i]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    if constexpr (NB == 1) load_s(min(hh + 1, h1 - 1), 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < TB; ++b) {
      const int tok = 16 * (TB * tp + b) + r2;
      float da = dwr[b];  // this lane's part of dL/dG
#pragma unroll
      for (int i = 0; i < TQ; ++i)
        if (FULL || nq * TQ + i < TN) {
          const f32x4 kv = value(Kl, tok, nq * TQ + i), qv = value(Ql, tok, nq * TQ + i);
#pragma unroll
          for (int e = 0; e < 4; ++e) da += qv[e] * dq[b][i][e] + kv[e] * (dr[b][i][e] - dw[b][i][e]);
          dqs[b][i] += dq[b][i];
          dks[b][i] += dr[b][i] + dw[b][i];
        }
      da += __shfl_xor(da, 16);
      da += __shfl_xor(da, 32);
      dwr[b] += __shfl_xor(dwr[b], 16);
      dwr[b] += __shfl_xor(dwr[b], 32);
      if (q == 0) {
        red[0][nq][tok] = da;
        red[1][nq][tok] = dwr[b];
      }
    }
    sdot = wave_sum(sdot);
    if (lane == 0) sd[w] = sdot;
    if (tid == 0) sd[NW] = exp2_hl(gl[C - 1], gl[2 * C - 1]);
    // F . Z over the rows: 16 lanes, then two waves in order
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = row_sum16(bdot[e]);
      if (r == 0) bsum[w >> 2][tk4 + e] = v;
    }
    __syncthreads();  // (the next head's data goes where P and M are)
  }
  if (w == 0) gates(h1 - 1);
  if (a.parts) {
    float* part = a.parts + ((int64_t)ck * a.H + h0) * 2 * C * N;
#pragma unroll
    for (int b = 0; b < TB; ++b)
#pragma unroll
      for (int i = 0; i < TQ; ++i) {
        const int nt = nq * TQ + i, at = (16 * (TB * tp + b) + r) * N + 16 * nt + 4 * q;
        if (FULL || nt < TN) {
          *(f32x4*)(part + at) = dqs[b][i];
          *(f32x4*)(part + C * N + at) = dks[b][i];
        }
      }
    return;
  }
  const brsrc wq = make_rsrc((char*)a.dq + kbase, kspan), wk = make_rsrc((char*)a.dk + kbase, kspan);
#pragma unroll
  for (int b = 0; b < TB; ++b)
#pragma unroll
    for (int i = 0; i < TQ; ++i) {
      const int nt = nq * TQ + i;
      if (FULL || nt < TN) {
        const uint32_t off = (16 * (TB * tp + b) + r) * krow + (16 * nt + 4 * q) * ES;
        store4io(wq, off, dqs[b][i], IO{});
        store4io(wk, off, dks[b][i], IO{});
      }
    }
}

// dq and dk of a chunk and group from its heads' parts, added in the order of the heads (the sums
// are those of a workgroup that takes all of them).
template <int N, class IO>
__global__ __launch_bounds__(256) void delta_head_sum_kernel(DeltaArgs a) {
  constexpr int C = kDeltaChunk, ES = sizeof(typename IO::T), ROWS = 1024 / N;
  const int blk = blockIdx.x % (C / ROWS), wg = blockIdx.x / (C / ROWS);
  const int ck = wg / a.G, grp = wg % a.G, per = a.H / a.G;
  const ChunkInfo ci = chunk_info(a.map, ck);
  const int tok = blk * ROWS + threadIdx.x / (N / 4), col = threadIdx.x % (N / 4) * 4;
  if (tok >= ci.len) return;
  const float* p = a.parts + (((int64_t)ck * a.H + grp * per) * 2 * C + tok) * N + col;
  f32x4 dq = {0.f, 0.f, 0.f, 0.f}, dk = dq;
  for (int h = 0; h < per; ++h, p += 2 * C * N) {
    dq += *(const f32x4*)p;
    dk += *(const f32x4*)(p + C * N);
  }
  const int start = __builtin_amdgcn_readfirstlane(ci.start), len = __builtin_amdgcn_readfirstlane(ci.len);
  const uint32_t row = (uint32_t)a.G * N * ES;
  const int64_t at = ((int64_t)start * a.G + grp) * N * ES;
  const uint32_t span = (uint32_t)(len - 1) * row + N * ES;
  store4io(make_rsrc((char*)a.dq + at, span), tok * row + col * ES, dq, IO{});
  store4io(make_rsrc((char*)a.dk + at, span), tok * row + col * ES, dk, IO{});
}

hipError_t launch_delta_bwd_grads(const DeltaProb& p, const DeltaArgs& a, hipStream_t st) {
  if (p.nck == 0) return hipSuccess;
  const dim3 grid((unsigned)(p.nck * (a.parts ? p.H : p.G)));
  auto go = [&](auto n, auto pp, auto io) {
    constexpr int N = decltype(n)::value, P = decltype(pp)::value;
    using IO = decltype(io);
    hipLaunchKernelGGL((delta_grads_kernel<N, P, IO>), grid, dim3(512), 0, st, a);
  };
  auto pick_p = [&](auto n, auto io) {
    switch (p.P) {
      case 16: go(n, std::integral_constant<int, 16>{}, io); break;
      case 32: go(n, std::integral_constant<int, 32>{}, io); break;
      case 64: go(n, std::integral_constant<int, 64>{}, io); break;
      default: go(n, std::integral_constant<int, 128>{}, io); break;
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
  if (!a.parts) return hipGetLastError();
  auto sum = [&](auto n, auto io) {
    constexpr int N = decltype(n)::value;
    hipLaunchKernelGGL((delta_head_sum_kernel<N, decltype(io)>), dim3((unsigned)(p.nck * p.G * (kDeltaChunk * N / 1024))),
                       dim3(256), 0, st, a);
  };
  auto pick_sum = [&](auto io) {
    switch (p.N) {
      case 16: sum(std::integral_constant<int, 16>{}, io); break;
      case 32: sum(std::integral_constant<int, 32>{}, io); break;
      case 64: sum(std::integral_constant<int, 64>{}, io); break;
      default: sum(std::integral_constant<int, 128>{}, io); break;
    }
  };
  p.io ? pick_sum(IoBf16{}) : pick_sum(IoF32{});
  return hipGetLastError();
}

}  // namespace ssd
