// C ABI of the gated delta rule and the state cache: argument validation, workspace
// layout and launch order (conventions as in api.cpp: every check the host can make
// comes before the first launch; nothing is allocated, no state is kept).
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <memory>
#include <new>

#include "delta.hpp"
#include "ssd.h"

using namespace ssd;

namespace {

bool aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if ((uintptr_t)p & 15u) return false;
  return true;
}
bool okdim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

ssd_status make_delta(const ssd_delta_problem* pr, int packed, DeltaProb& p) {
  if (!pr) return SSD_ERR_NULL;
  if (pr->batch < 0 || pr->seqlen < 0 || pr->nheads <= 0 || pr->headdim <= 0 || pr->dstate <= 0 || pr->ngroups <= 0)
    return SSD_ERR_SHAPE;
  if (pr->nheads % pr->ngroups) return SSD_ERR_SHAPE;
  if (packed && (pr->batch != 1 || pr->nseq < 0)) return SSD_ERR_SHAPE;
  if (pr->flags & ~(SSD_FLAG_SAVE_FOR_BWD | SSD_FLAG_FROM_SAVED)) return SSD_ERR_UNSUPPORTED;
  if (pr->io_dtype != SSD_F32 && pr->io_dtype != SSD_BF16) return SSD_ERR_UNSUPPORTED;
  if (!okdim(pr->headdim) || !okdim(pr->dstate)) return SSD_ERR_UNSUPPORTED;
  if (!std::isfinite(pr->scale)) return SSD_ERR_UNSUPPORTED;
  const int64_t tokens = (int64_t)pr->batch * pr->seqlen;
  if (tokens > INT32_MAX / 2 || pr->nheads > 65535) return SSD_ERR_UNSUPPORTED;
  // (so that 32-bit byte offsets reach the token rows of a chunk: 64 x 65535 x 128 x 4 < 2^31)
  std::memset(&p, 0, sizeof(p));
  p.B = pr->batch;
  p.L = pr->seqlen;
  p.H = pr->nheads;
  p.P = pr->headdim;
  p.N = pr->dstate;
  p.G = pr->ngroups;
  p.io = pr->io_dtype;
  p.packed = packed;
  p.flags = pr->flags;
  p.scale = pr->scale;
  p.nst = packed ? pr->nseq : pr->batch;
  if (packed && p.nst > 65535) return SSD_ERR_UNSUPPORTED;
  const int Q = kDeltaChunk;
  p.nck = packed ? ((int64_t)p.L + (int64_t)p.nst * (Q - 1)) / Q : (int64_t)p.B * ((p.L + Q - 1) / Q);
  // 1-D grids over (chunk, head) and (state, head, 16 rows) of up to 512 threads stay below
  // the 2^32 threads of a launch
  if (p.nck * (int64_t)p.H >= 1 << 23 || (int64_t)p.nst * p.H * (p.P / 16) >= 1 << 23) return SSD_ERR_UNSUPPORTED;
  p.map.Q = Q;
  p.map.nck = (int32_t)p.nck;
  p.map.packed = packed;
  p.map.seqlen = p.L;
  p.map.ncs = (p.L + Q - 1) / Q;
  return SSD_OK;
}

// Whether the gradients take a workgroup a head, and the heads' dq and dk are added up after (in
// the same order: the bits do not change).  Backward calls from a saved forward, dstate 128, us
// with a group's heads in one workgroup | apart: 16 chunks and groups of 8 heads 79 | 39, 64 of 8
// 91 | 68, 128 of 4 64 | 68, 128 of 8 114 | 125, 512 of 4 184 | 266.
bool split_heads(const DeltaProb& p) { return p.G < p.H && p.nck * p.G <= 64; }

DeltaLayout delta_layout(const DeltaProb& p) {
  DeltaLayout l;
  std::memset(&l, 0, sizeof(l));
  if (p.nck == 0 && !p.packed) return l;
  const size_t ch = (size_t)p.nck * p.H, state = (size_t)p.P * state_cols(p.N) * 4, rows = (size_t)kDeltaChunk * p.P * 4;
  const size_t PM = p.io ? IoBf16::PM : IoF32::PM, PF = p.io ? IoBf16::PI : IoF32::PI;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += lay_up(bytes);
    return at;
  };
  l.tab = take(p.packed ? (size_t)p.nck * 16 : 0);
  l.seq_off = take(p.packed ? ((size_t)p.nst + 1) * 4 : 0);
  l.gates = take(ch * kDeltaGates * 4);
  l.R = take(ch * PM * kTriPlane * 2);
  l.Pm = take(ch * PF * kTriPlane * 2);
  l.fwd_end = o;
  l.Rt = take(ch * PM * kTriPlane * 2);
  l.Pt = take(ch * PM * kTriPlane * 2);
  l.S = take(ch * state);
  l.Z = take(ch * rows);
  l.dS = take(ch * state);
  l.F = take(ch * rows);
  l.parts = take(split_heads(p) ? ch * 2 * kDeltaChunk * p.N * 4 : 0);
  l.end = o;
  return l;
}

// Point the chunk map at the table in the workspace and, unless a forward kept it there,
// queue its build (SSD_DEBUG=1: after checking cu_seqlens on the host).
ssd_status setup_map(DeltaProb& p, const DeltaLayout& l, const int32_t* cu, char* ws, hipStream_t st) {
  if (!p.packed) return SSD_OK;
  p.map.tab = (const int4*)(ws + l.tab);
  p.map.seq_off = (const int32_t*)(ws + l.seq_off);
  const char* dbg = std::getenv("SSD_DEBUG");
  if (dbg && dbg[0] == '1') {
    const size_t n = (size_t)p.nst + 1;
    std::unique_ptr<int32_t[]> hcu(new (std::nothrow) int32_t[n]);
    if (!hcu || hipMemcpyAsync(hcu.get(), cu, n * 4, hipMemcpyDeviceToHost, st) != hipSuccess ||
        hipStreamSynchronize(st) != hipSuccess)
      return SSD_ERR_HIP;
    if (hcu[0] != 0 || hcu[p.nst] != p.L) return SSD_ERR_VARLEN;
    for (int s = 0; s < p.nst; ++s)
      if (hcu[s + 1] < hcu[s]) return SSD_ERR_VARLEN;
  }
  if (p.flags & SSD_FLAG_FROM_SAVED) return SSD_OK;
  Prob t;
  std::memset(&t, 0, sizeof(t));
  t.nseq = p.nst;
  t.L = p.L;
  t.Q = kDeltaChunk;
  t.nck = p.nck;
  return launch_build_table(t, cu, (int4*)(ws + l.tab), (int32_t*)(ws + l.seq_off), st) == hipSuccess ? SSD_OK
                                                                                                     : SSD_ERR_HIP;
}

DeltaArgs make_args(const DeltaProb& p, const DeltaLayout& l, char* ws, const void* q, const void* k, const void* v,
                    const float* g, const float* beta, const float* init, bool keep) {
  DeltaArgs a;
  std::memset(&a, 0, sizeof(a));
  a.map = p.map;
  a.H = p.H; a.G = p.G; a.P = p.P; a.N = p.N; a.L = p.L;
  a.scale = p.scale;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.init = init;
  a.gates = (float*)(ws + l.gates);
  a.R = (uint16_t*)(ws + l.R);
  a.Pm = (uint16_t*)(ws + l.Pm);
  if (keep) {
    a.Rt = (uint16_t*)(ws + l.Rt);
    a.Pt = (uint16_t*)(ws + l.Pt);
    a.S = (float*)(ws + l.S);
    a.Z = (float*)(ws + l.Z);
  }
  return a;
}

#define DELTA_TRY(expr)                           \
  do {                                            \
    if ((expr) != hipSuccess) return SSD_ERR_HIP; \
  } while (0)

ssd_status cache_check(const ssd_cache_problem* pr) {
  if (!pr) return SSD_ERR_NULL;
  if (pr->n < 0 || pr->nslots < 0 || pr->nheads <= 0 || pr->headdim <= 0 || pr->dstate <= 0) return SSD_ERR_SHAPE;
  if (!okdim(pr->dstate) || (pr->format != SSD_CACHE_INT8 && pr->format != SSD_CACHE_E4M3)) return SSD_ERR_UNSUPPORTED;
  if (pr->n > 65535 || (int64_t)pr->nheads * pr->headdim >= (int64_t)1 << 24) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

ssd_status cache_run(bool write, const ssd_cache_problem* pr, const float* states, const int32_t* slots, void* codes,
                     const float* scales, void* stream) {
  const ssd_status s = cache_check(pr);
  if (s != SSD_OK) return s;
  if (pr->n > 0 && (pr->nslots == 0 || (!slots && pr->nslots < pr->n))) return SSD_ERR_SHAPE;
  if (pr->n > 0 && (!states || !codes || !scales)) return SSD_ERR_NULL;
  if (!aligned({states, slots, codes, scales})) return SSD_ERR_ALIGN;
  if (pr->n == 0) return SSD_OK;
  DELTA_TRY(launch_state_cache(write, pr->n, pr->nslots, pr->nheads, pr->headdim, pr->dstate, pr->format,
                               const_cast<float*>(states), slots, codes, const_cast<float*>(scales),
                               (hipStream_t)stream));
  return SSD_OK;
}

}  // namespace

extern "C" {

size_t ssd_delta_fwd_workspace_bytes(const ssd_delta_problem* pr, int32_t packed) {
  DeltaProb p;
  if (make_delta(pr, packed != 0, p) != SSD_OK) return 0;
  return delta_layout(p).fwd_end;
}

size_t ssd_delta_bwd_workspace_bytes(const ssd_delta_problem* pr, int32_t packed) {
  DeltaProb p;
  if (make_delta(pr, packed != 0, p) != SSD_OK) return 0;
  return delta_layout(p).end;
}

ssd_status ssd_delta_fwd(const ssd_delta_problem* pr, const void* q, const void* k, const void* v, const float* g,
                         const float* beta, const float* init_states, const int32_t* cu_seqlens, void* out,
                         float* final_states, void* workspace, size_t workspace_bytes, void* stream) {
  DeltaProb p;
  ssd_status s = make_delta(pr, cu_seqlens != nullptr, p);
  if (s != SSD_OK) return s;
  if (p.flags & SSD_FLAG_FROM_SAVED) return SSD_ERR_UNSUPPORTED;
  if ((int64_t)p.B * p.L > 0 && (!q || !k || !v || !g || !beta || !out)) return SSD_ERR_NULL;
  if (!aligned({q, k, v, g, beta, init_states, cu_seqlens, out, final_states, workspace})) return SSD_ERR_ALIGN;
  const DeltaLayout l = delta_layout(p);
  const bool save = (p.flags & SSD_FLAG_SAVE_FOR_BWD) != 0;
  const size_t need = save ? l.end : l.fwd_end;
  if (need > 0 && (!workspace || workspace_bytes < need)) return SSD_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  char* ws = (char*)workspace;
  s = setup_map(p, l, cu_seqlens, ws, st);
  if (s != SSD_OK) return s;
  DeltaArgs a = make_args(p, l, ws, q, k, v, g, beta, init_states, save);
  a.out = out;
  a.final_states = final_states;
  DELTA_TRY(launch_delta_prep(p, a, st));
  DELTA_TRY(launch_delta_fwd(p, a, st));
  return SSD_OK;
}

ssd_status ssd_delta_bwd(const ssd_delta_problem* pr, const void* q, const void* k, const void* v, const float* g,
                         const float* beta, const float* init_states, const int32_t* cu_seqlens, const void* dout,
                         const float* d_final_states, void* dq, void* dk, void* dv, float* dg, float* dbeta,
                         float* d_init_states, void* workspace, size_t workspace_bytes, void* stream) {
  DeltaProb p;
  ssd_status s = make_delta(pr, cu_seqlens != nullptr, p);
  if (s != SSD_OK) return s;
  if (p.flags & SSD_FLAG_SAVE_FOR_BWD) return SSD_ERR_UNSUPPORTED;
  if ((int64_t)p.B * p.L > 0 && (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta))
    return SSD_ERR_NULL;
  if (!aligned({q, k, v, g, beta, init_states, cu_seqlens, dout, d_final_states, dq, dk, dv, dg, dbeta, d_init_states,
                workspace}))
    return SSD_ERR_ALIGN;
  const DeltaLayout l = delta_layout(p);
  if (l.end > 0 && (!workspace || workspace_bytes < l.end)) return SSD_ERR_WORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  char* ws = (char*)workspace;
  s = setup_map(p, l, cu_seqlens, ws, st);
  if (s != SSD_OK) return s;
  DeltaArgs a = make_args(p, l, ws, q, k, v, g, beta, init_states, true);
  if (!(p.flags & SSD_FLAG_FROM_SAVED)) {
    DELTA_TRY(launch_delta_prep(p, a, st));
    DELTA_TRY(launch_delta_fwd(p, a, st));  // (no output: what the backward reads alone)
  }
  a.dout = dout;
  a.d_final = d_final_states;
  a.dS = (float*)(ws + l.dS);
  a.F = (float*)(ws + l.F);
  a.d_init = d_init_states;
  a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta;
  a.parts = split_heads(p) ? (float*)(ws + l.parts) : nullptr;
  DELTA_TRY(launch_delta_bwd_chain(p, a, st));
  DELTA_TRY(launch_delta_bwd_grads(p, a, st));
  return SSD_OK;
}

ssd_status ssd_delta_step(const ssd_delta_problem* pr, const void* q, const void* k, const void* v, const float* g,
                          const float* beta, const int32_t* slots, int32_t nslots, float* states, void* out,
                          void* stream) {
  DeltaProb p;
  ssd_status s = make_delta(pr, 0, p);
  if (s != SSD_OK) return s;
  if (p.flags || pr->nseq) return SSD_ERR_UNSUPPORTED;
  if (nslots < 0 || (p.B > 0 && (nslots == 0 || (!slots && nslots < p.B)))) return SSD_ERR_SHAPE;
  if ((int64_t)p.B * p.L > 0 && (!q || !k || !v || !g || !beta || !out || !states)) return SSD_ERR_NULL;
  if (!aligned({q, k, v, g, beta, slots, states, out})) return SSD_ERR_ALIGN;
  DELTA_TRY(launch_delta_step(p, q, k, v, g, beta, slots, nslots, states, out, (hipStream_t)stream));
  return SSD_OK;
}

ssd_status ssd_state_cache_write(const ssd_cache_problem* pr, const float* states, const int32_t* slots, void* codes,
                                 float* scales, void* stream) {
  return cache_run(true, pr, states, slots, codes, scales, stream);
}

ssd_status ssd_state_cache_read(const ssd_cache_problem* pr, const void* codes, const float* scales,
                                const int32_t* slots, float* states, void* stream) {
  return cache_run(false, pr, states, slots, const_cast<void*>(codes), scales, stream);
}

}  // extern "C"
