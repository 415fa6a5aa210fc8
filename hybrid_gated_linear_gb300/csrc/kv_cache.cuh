// kv_cache.cuh -- what the kernels of the 8-bit paged cache share: the view of the cache
// and of the rotary table, the storage order, code <-> value conversion and the checks of
// device-side page numbers and positions.
#pragma once

#include <cuda_fp16.h>
#include <math.h>

#include "lizard_dev.cuh"
#include "lizard_internal.h"

namespace lz {

// Place of the 16-byte chunk c of row r inside its row of D bytes.
template <int D>
__device__ __forceinline__ int chunk_place(int r, int c) {
  return D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
}

// The four e4m3 codes of a word as two half2 (exact; the two NaN codes, which only bytes never
// written can hold, come out as NaN).  One conversion per pair at the rate of the integer
// pipe; moving the fields with shifts and masks takes four operations per pair.
__device__ __forceinline__ void e4m3x4_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// The four signed bytes of a word as two half2: 1024 + 128 + x is exact in binary16 with x's
// offset form in the low byte.
__device__ __forceinline__ void i8x4_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
  lo = *reinterpret_cast<const uint32_t*>(&x);
  hi = *reinterpret_cast<const uint32_t*>(&y);
}

// Codes as halves: F = 0 e4m3, 1 signed bytes.
template <int F>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (F == 0) e4m3x4_to_half(w, lo, hi);
  else i8x4_to_half(w, lo, hi);
}
// Four codes as floats, in units of the scale.
template <int F>
__device__ __forceinline__ float4 codes_to_float(uint32_t w) {
  uint32_t lo, hi;
  codes_to_half<F>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

// Four values (already divided by the scale) to codes, ties to even, saturating.
template <int F>
__device__ __forceinline__ uint32_t float_to_codes(float a, float b, float c, float d) {
  if (F == 0) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
  auto q = [](float x) { return (uint32_t)(__float2int_rn(fminf(fmaxf(x, -127.f), 127.f)) & 0xff); };
  return q(a) | (q(b) << 8) | (q(c) << 16) | (q(d) << 24);
}

// The exponent e of the smallest power of two with amax <= max code * 2^e, -126 at least:
// amax = m 2^k exceeds max code = 1.75 * 2^8 (e4m3) or 127/64 * 2^6 (bytes) at the same
// exponent where its mantissa bits do.
template <int F>
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int k = (int)(u >> 23) - 127;
  const uint32_t top = F == 0 ? 0x600000u : 0x7e0000u;
  const int e = k - (F == 0 ? 8 : 6) + ((u & 0x7fffffu) > top ? 1 : 0);
  return e < -126 ? -126 : e;
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Four consecutive elements as loaded, and as floats: loads in one loop, conversions (the
// first uses, which wait) in the next.
template <typename T> struct Raw4;
template <> struct alignas(16) Raw4<float> {
  float4 v;
  __device__ __forceinline__ float4 value() const { return v; }
};
template <> struct alignas(8) Raw4<bf16> {
  uint2 v;
  __device__ __forceinline__ float4 value() const {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
  }
};
template <typename T>
__device__ __forceinline__ Raw4<T> raw4(const T* p) { return *reinterpret_cast<const Raw4<T>*>(p); }

// cos and sin of position p of a pair (times the factor): p * turns wraps to the exact
// fraction of a turn; its upper 32 bits, as a signed count of half turns / 2^31, are rounded
// once to fp32 (an angle error of pi 2^-25 at most).
__device__ __forceinline__ void rope_angle(uint64_t turns, int64_t p, float f, float& co, float& si) {
  const int32_t t = (int32_t)((uint64_t)(p * (int64_t)turns) >> 32);
  sincospif((float)t * 0x1p-31f, &si, &co);
  co *= f;
  si *= f;
}

// A position that counts and windows can be added to and taken from.
__device__ __forceinline__ bool position_ok(int64_t p) { return p >= 0 && p < (1ll << 62); }

// The last of cnt positions from p on; beyond the end of int64 it wraps below p.
__device__ __forceinline__ int64_t last_of(int64_t p, int cnt) { return (int64_t)((uint64_t)p + (uint64_t)(cnt - 1)); }

// The pages that tokens lo..hi (lo <= hi) of a sequence touch fit its table, positions are
// not negative and logical pages fit 31 bits.
__device__ __forceinline__ bool span_ok(const CacheArgs& c, int64_t lo, int64_t hi) {
  return lo >= 0 && hi >= lo && (hi >> c.log_p) < 0x7fffffffll &&
         (hi >> c.log_p) - (lo >> c.log_p) < c.max_pages;
}

// Pool page of logical page j of sequence n, or -1.
__device__ __forceinline__ int pool_page(const CacheArgs& c, int n, uint32_t j) {
  const int id = c.table[(size_t)n * c.max_pages + j % (uint32_t)c.max_pages];
  return (unsigned)id < (unsigned)c.pages ? id : -1;
}

}  // namespace lz
