// The state cache: fp32 states (n, H, P, N) parked in 8 bits in the slots of a cache
// (codes (nslots, H, P, N), one fp32 scale a state row of N values) and read back.
//
//   int8: scale = max|x| / 127 (rounded to fp32), code = x / scale rounded to nearest
//         (ties to even), exactly: a code next to a border is decided by the residual
//         x - code scale, which a fused multiply-add forms without rounding;
//   e4m3: scale = the smallest power of two with max|x| / scale <= 448, code = x / scale
//         rounded to nearest by the hardware conversion (the division is exact).
// A row of zeros has scale 0.  A row that holds an infinity or a NaN has scale NaN and
// reads back as NaN: a state gone bad stays visible.
//
// A value is off by at most scale / 2 (int8: max|x| / 254) or, as e4m3, by 2^-4 of
// itself or 2^-10 scale, whichever is more.  One scale a row: rows differ in size (each
// is one value channel's memory), and the scales add 4 bytes to N codes.
//
// Bound: bytes, 5 an element plus the scales.  N / 4 lanes hold a row, 4 elements each;
// a workgroup's rows belong to one sequence, so its slot is looked up once.  96 states of 32
// heads of 128 x 128 (252 MB): written in 43 us (5.9 TB/s), read back in 35 us (7.2 TB/s, the
// codes out of the last cache).
#include "delta.hpp"

namespace ssd {

// Rows a thread (96 states of 32 heads of 128 x 128, written: one row 56 us, two 56, four 60, eight
// 64), the states past the caches (43 us).
constexpr int kCacheRows = 2;

// Largest over the LPR = 4 | 8 | 16 | 32 consecutive lanes of a row (compared as integers).
template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  auto other = [&](auto ctrl) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, decltype(ctrl)::value, 15, 15, true); };
  v = max(v, other(std::integral_constant<int, kQuadXor1>{}));
  v = max(v, other(std::integral_constant<int, kQuadXor2>{}));
  if constexpr (LPR >= 8) v = max(v, other(std::integral_constant<int, kRowHalfMirror>{}));
  if constexpr (LPR >= 16) v = max(v, other(std::integral_constant<int, kRowRor8>{}));
  if constexpr (LPR == 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(a[0], a[1]);
  }
  return v;
}

__device__ __forceinline__ int int8_code(float x, float s, float inv) {
  float c = rintf(x * inv);
  const float r2 = 2.f * fmaf(-c, s, x);  // exact: x - c s is a multiple of ulp(s) / 2 or x itself
  const bool odd = ((int)c & 1) != 0;
  if (r2 > s || (r2 == s && odd)) c += 1.f;
  if (r2 < -s || (r2 == -s && odd)) c -= 1.f;
  return (int)fminf(fmaxf(c, -127.f), 127.f);
}

template <int N, bool E4M3>
__global__ __launch_bounds__(256) void state_cache_write_kernel(int nslots, int rows, const float* __restrict__ states,
                                                                const int32_t* __restrict__ slots,
                                                                uint32_t* __restrict__ codes,
                                                                float* __restrict__ scales) {
  constexpr int LPR = N / 4, RP = 256 / LPR;
  const int s = blockIdx.y;
  const int row0 = blockIdx.x * RP * kCacheRows + threadIdx.x / LPR, c4 = threadIdx.x % LPR;
  const int slot = slots ? slots[s] : s;
  const int32_t mine = slots ? slots[min((int)threadIdx.x, s)] : 0;
  f32x4 x[kCacheRows];
#pragma unroll
  for (int i = 0; i < kCacheRows; ++i) {
    const int row = row0 + i * RP;
    x[i] = row < rows ? __builtin_nontemporal_load((const f32x4*)(states + ((int64_t)s * rows + row) * N + c4 * 4)) : f32x4{0.f, 0.f, 0.f, 0.f};
  }
  if (slots && !slot_runs(slots, s, slot, nslots, mine)) return;
#pragma unroll
  for (int i = 0; i < kCacheRows; ++i) {
    const int row = row0 + i * RP;
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(x[i][e]) & 0x7fffffffu);
    top = row_max<LPR>(top);  // (as integers: a NaN or an infinity is above every finite value)
    float scale;
    uint32_t code = 0;
    if (top >= 0x7f800000u) {
      scale = __uint_as_float(0x7fc00000u);
    } else if constexpr (E4M3) {
      // max = m 2^e with m in [1, 2): the power is e - 8, one more where m > 1.75
      const int e = max((int)(top >> 23) - 127, -118) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
      scale = top ? __uint_as_float((uint32_t)(e + 127) << 23) : 0.f;
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[i][0] * inv, x[i][1] * inv, 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(x[i][2] * inv, x[i][3] * inv, w, true);
      code = (uint32_t)w;
    } else {
      scale = __uint_as_float(top) / 127.f;
      if (scale > 0.f) {
        // (a scale whose reciprocal overflows: divide instead)
        const bool tiny = scale < 0x1p-126f;
        const float inv = 1.f / scale;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = tiny ? int8_code(x[i][e] / scale, 1.f, 1.f) : int8_code(x[i][e], scale, inv);
          code |= (uint32_t)(c & 255) << (8 * e);
        }
      }
    }
    if (row < rows) {
      const int64_t at = (int64_t)slot * rows + row;
      codes[at * LPR + c4] = code;
      if (c4 == 0) scales[at] = scale;
    }
  }
}

template <int N, bool E4M3>
__global__ __launch_bounds__(256) void state_cache_read_kernel(int nslots, int rows, float* __restrict__ states,
                                                               const int32_t* __restrict__ slots,
                                                               const uint32_t* __restrict__ codes,
                                                               const float* __restrict__ scales) {
  constexpr int LPR = N / 4, RP = 256 / LPR;
  const int s = blockIdx.y;
  const int row0 = blockIdx.x * RP * kCacheRows + threadIdx.x / LPR, c4 = threadIdx.x % LPR;
  const int slot = slots ? slots[s] : s;
  const bool in = slot >= 0 && slot < nslots;  // out of range: a state of zeros
  uint32_t w[kCacheRows];
  float sc[kCacheRows];
#pragma unroll
  for (int i = 0; i < kCacheRows; ++i) {
    const int64_t at = (int64_t)(in ? slot : 0) * rows + min(row0 + i * RP, rows - 1);
    w[i] = codes[at * LPR + c4];
    sc[i] = scales[at];
  }
#pragma unroll
  for (int i = 0; i < kCacheRows; ++i) {
    const int row = row0 + i * RP;
    f32x4 x;
    if constexpr (E4M3) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
      x = f32x4{lo[0], lo[1], hi[0], hi[1]};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = (float)(int8_t)(w[i] >> (8 * e));
    }
    x = in ? x * sc[i] : f32x4{0.f, 0.f, 0.f, 0.f};
    if (row < rows) __builtin_nontemporal_store(x, (f32x4*)(states + ((int64_t)s * rows + row) * N + c4 * 4));
  }
}

hipError_t launch_state_cache(bool write, int n, int nslots, int H, int P, int N, int format, float* states,
                              const int32_t* slots, void* codes, float* scales, hipStream_t st) {
  if (n == 0) return hipSuccess;
  const int rows = H * P, per = 256 / (N / 4) * kCacheRows;
  const dim3 grid((unsigned)((rows + per - 1) / per), (unsigned)n), block(256);
  auto go = [&](auto nc, auto fc) {
    constexpr int NN = decltype(nc)::value;
    constexpr bool F = decltype(fc)::value;
    if (write)
      hipLaunchKernelGGL((state_cache_write_kernel<NN, F>), grid, block, 0, st, nslots, rows, states, slots,
                         (uint32_t*)codes, scales);
    else
      hipLaunchKernelGGL((state_cache_read_kernel<NN, F>), grid, block, 0, st, nslots, rows, states, slots,
                         (const uint32_t*)codes, scales);
  };
  auto pick = [&](auto fc) {
    switch (N) {
      case 16: go(std::integral_constant<int, 16>{}, fc); break;
      case 32: go(std::integral_constant<int, 32>{}, fc); break;
      case 64: go(std::integral_constant<int, 64>{}, fc); break;
      default: go(std::integral_constant<int, 128>{}, fc); break;
    }
  };
  if (format)
    pick(std::true_type{});
  else
    pick(std::false_type{});
  return hipGetLastError();
}

}  // namespace ssd
