// Gated delta rule, recurrent form: T >= 1 tokens of each sequence of a decode batch,
// on states that stay in place in a slotted cache (fp32).
//
//   a = exp(g), r = v - a (S k), u = b r, S <- a S + u k^T, o = scale S q,
// with o evaluated as scale (a (S q) + u (k . q)), so that S k and S q are reduced
// together, before the update.  State rows (headdim) do not interact: a workgroup
// takes some rows of one (sequence, head), N / 4 lanes a row with 4 elements each, and
// holds them in registers over the T tokens.
//
// Bound: the states' bytes, read once and written once (8 bytes an element), past the caches
// (250 sequences of 64 heads of 64 x 128, 1.05 GB: 176 us, 5.95 TB/s; 183 us with plain loads and
// stores; 5.95 TB/s is also what a copy in place reaches).  One sequence: 3.8 us, latency.
//
// A sequence whose slot is out of range is padding: nothing of it is read or written.
// Of several sequences that name one slot the first runs and the others are treated
// as padding: running them together would race on the state.
#include "delta.hpp"

namespace ssd {

// Sum over the LPR = N / 4 lanes of a row, 4 | 8 | 16 | 32 consecutive lanes.
template <int LPR>
__device__ __forceinline__ float row_total(float v) {
  if constexpr (LPR >= 16) {
    v = row_sum16(v);
    if constexpr (LPR == 32) {
      const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
      v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    }
  } else {
    v += dpp_f<kQuadXor1>(0.f, v);
    v += dpp_f<kQuadXor2>(0.f, v);
    if constexpr (LPR == 8) v += dpp_f<kRowHalfMirror>(0.f, v);
  }
  return v;
}

__device__ __forceinline__ f32x4 io4(const uint16_t* p) {
  const uint2 w = *(const uint2*)p;
  return f32x4{bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y)};
}
__device__ __forceinline__ f32x4 io4(const float* p) { return *(const f32x4*)p; }
__device__ __forceinline__ float io1(const uint16_t* p) { return bf2f(*p); }
__device__ __forceinline__ float io1(const float* p) { return *p; }
__device__ __forceinline__ void put1(uint16_t* p, float v) { *p = f2bf(v); }
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) {
  return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
}

// RPT rows a thread, E groups of four columns of each (N / 4E lanes a row)
template <int N, class IO, int RPT, int E>
__global__ __launch_bounds__(256) void delta_step_kernel(int T, int H, int G, int P, float scale,
                                                         const typename IO::T* __restrict__ Q,
                                                         const typename IO::T* __restrict__ K,
                                                         const typename IO::T* __restrict__ V,
                                                         const float* __restrict__ g, const float* __restrict__ beta,
                                                         const int32_t* __restrict__ slots, int nslots,
                                                         float* __restrict__ states, typename IO::T* __restrict__ out) {
  constexpr int LPR = N / (4 * E), RP = 256 / LPR, NC = N / E;  // lanes a row, rows a pass
  const int blocks = (P + RP * RPT - 1) / (RP * RPT);
  const int rb = blockIdx.x % blocks, h = (int)((blockIdx.x / blocks) % H), b = (int)(blockIdx.x / blocks / H);
  const int lr = threadIdx.x / LPR, n0 = (threadIdx.x % LPR) * 4;
  const int slot = slots ? slots[b] : b;
  // a token's inputs, loaded while the one before is worked on (the first: beside the slots; the
  // state after them: before the slots' check it costs 10%, its reads then run ahead of the writes)
  const int grp = h / (H / G);
  f32x4 k[E], q[E];
  float gt, bt, v[RPT];
  int p[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) p[i] = rb * RP * RPT + i * RP + lr;
  auto load = [&](int t) {
    const int64_t tok = (int64_t)b * T + t;
#pragma unroll
    for (int c = 0; c < E; ++c) {
      k[c] = io4(K + (tok * G + grp) * N + c * NC + n0);
      q[c] = io4(Q + (tok * G + grp) * N + c * NC + n0);
    }
    gt = g[tok * H + h];
    bt = beta[tok * H + h];
#pragma unroll
    for (int i = 0; i < RPT; ++i) v[i] = io1(V + (tok * H + h) * P + min(p[i], P - 1));
  };
  const int32_t mine = slots ? slots[min((int)threadIdx.x, b)] : 0;
  load(0);
  if (slots && !slot_runs(slots, b, slot, nslots, mine)) return;  // (the same for the whole workgroup)
  float* S = states + ((int64_t)slot * H + h) * P * N;
  f32x4 s[RPT][E];
#pragma unroll
  for (int i = 0; i < RPT; ++i)
#pragma unroll
    for (int c = 0; c < E; ++c)
      s[i][c] = p[i] < P ? __builtin_nontemporal_load((const f32x4*)(S + (int64_t)p[i] * N + c * NC + n0))
                         : f32x4{0.f, 0.f, 0.f, 0.f};
  auto dot = [](const f32x4 (&x)[E], const f32x4 (&y)[E]) {
    float d = dot4(x[0], y[0]);
#pragma unroll
    for (int c = 1; c < E; ++c) d += dot4(x[c], y[c]);
    return row_total<LPR>(d);
  };
  for (int t = 0; t < T; ++t) {
    const int64_t tok = (int64_t)b * T + t;
    f32x4 kt[E], qt[E];
    float vt[RPT];
#pragma unroll
    for (int c = 0; c < E; ++c) {
      kt[c] = k[c];
      qt[c] = q[c];
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) vt[i] = v[i];
    const float a = expf(min_gate(gt)), b1 = bt;
    if (t + 1 < T) load(t + 1);
    const float kq = dot(kt, qt);
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float sk = dot(s[i], kt), sq = dot(s[i], qt);
      const float u = b1 * (vt[i] - a * sk);
#pragma unroll
      for (int c = 0; c < E; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][c][e] = a * s[i][c][e] + u * kt[c][e];
      if (n0 == 0 && p[i] < P) put1(out + (tok * H + h) * P + p[i], scale * (a * sq + u * kq));
    }
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i)
#pragma unroll
    for (int c = 0; c < E; ++c)
      if (p[i] < P) __builtin_nontemporal_store(s[i][c], (f32x4*)(S + (int64_t)p[i] * N + c * NC + n0));
}

template <int N, class IO>
static void step_go(const DeltaProb& p, const void* q, const void* k, const void* v, const float* g,
                    const float* beta, const int32_t* slots, int nslots, float* states, void* out, hipStream_t st) {
  using T = typename IO::T;
  constexpr int E = N >= 64 ? 2 : 1;
  auto go = [&](auto rpt, auto e, int64_t wgs) {
    hipLaunchKernelGGL((delta_step_kernel<N, IO, decltype(rpt)::value, decltype(e)::value>), dim3((unsigned)wgs),
                       dim3(256), 0, st, p.L, p.H, p.G, p.P, p.scale, (const T*)q, (const T*)k, (const T*)v, g, beta,
                       slots, nslots, states, (T*)out);
  };
  auto count = [&](int rows) { return (int64_t)p.B * p.H * ((p.P + rows - 1) / rows); };
  // rows a workgroup: two, four or eight groups of four columns a thread
  constexpr int R1 = 2 * 1024 / N, R2 = 4 * 1024 / N, R3 = 8 * 1024 / N;
  // Several tokens: more groups a thread, which share a token's loads, k . q and gate, dealt to few
  // rows, whose sums then take fewer lanes, while they fill the CUs.  5 tokens, 24 sequences of 32
  // heads of 128 x 128, us by rows a thread x groups: 1 x 2 36, 2 x 1 36, 4 x 1 32, 2 x 2 29, 1 x 4
  // 34, 4 x 2 26, 2 x 4 25.  One token: two rows (250 sequences of 64 heads of 64 x 128: one 289 us,
  // two 188, four 202, eight 199; one sequence: 3.7, 3.9, 5.3, 5.6).
  if constexpr (N >= 64)
    if (p.L > 1 && p.P % R3 == 0 && count(R3) >= 1024) {
      go(std::integral_constant<int, 2>{}, std::integral_constant<int, 4>{}, count(R3));
      return;
    }
  if (p.L > 1 && count(R2) >= 1024)
    go(std::integral_constant<int, 4 / E>{}, std::integral_constant<int, E>{}, count(R2));
  else
    go(std::integral_constant<int, 2>{}, std::integral_constant<int, 1>{}, count(R1));
}

hipError_t launch_delta_step(const DeltaProb& p, const void* q, const void* k, const void* v, const float* g,
                             const float* beta, const int32_t* slots, int nslots, float* states, void* out,
                             hipStream_t st) {
  if (p.B == 0 || p.L == 0) return hipSuccess;
  auto go = [&](auto io) {
    using IO = decltype(io);
    switch (p.N) {
      case 16: step_go<16, IO>(p, q, k, v, g, beta, slots, nslots, states, out, st); break;
      case 32: step_go<32, IO>(p, q, k, v, g, beta, slots, nslots, states, out, st); break;
      case 64: step_go<64, IO>(p, q, k, v, g, beta, slots, nslots, states, out, st); break;
      default: step_go<128, IO>(p, q, k, v, g, beta, slots, nslots, states, out, st); break;
    }
  };
  if (p.io)
    go(IoBf16{});
  else
    go(IoF32{});
  return hipGetLastError();
}

}  // namespace ssd
