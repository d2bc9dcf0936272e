// What the attention kernels of the 8-bit KV cache share: visibility, exponentials and query scaling.
#pragma once

#include <math.h>

#include "kv8.h"

namespace ssd {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kPShift = 14.f;  // partial sums and outputs count softmax weights times 2^14

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What rounding (a, b) to hi left over.
__device__ __forceinline__ uint32_t pack_rest2(float a, float b, uint32_t hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return pack_half2(a - f.x, b - f.y);
}

// Tiles of 2^SHIFT slots: those of the prefix, then those that hold new slots past them.
template <int SHIFT>
struct Tiles {
  int n_prefix, first_new, n;
  __host__ __device__ __forceinline__ Tiles(int prefix, int base, int rows) {
    constexpr int up = (1 << SHIFT) - 1;
    n_prefix = (prefix + up) >> SHIFT;
    first_new = base >> SHIFT;
    if (first_new < n_prefix) first_new = n_prefix;
    const int end = (base + rows + up) >> SHIFT;
    n = n_prefix + (end > first_new ? end - first_new : 0);
  }
  __device__ __forceinline__ int slot(int t) const { return (t < n_prefix ? t : first_new + t - n_prefix) << SHIFT; }
};

__device__ __forceinline__ bool visible(int slot, int prefix, int base, unsigned long long mask) {
  const unsigned e = (unsigned)(slot - base);
  return slot < prefix || (e < 64u && ((mask >> e) & 1ull));
}

// Whether any row sees one of the sixteen slots from `slot` on.
__device__ __forceinline__ bool visible_any(int slot, const Kv8AttnArgs& a) {
  if (slot < a.prefix) return true;
  const int e = slot - a.base;
  if (e <= -16 || e >= 64) return false;
  return ((e >= 0 ? a.any >> e : a.any << -e) & 0xffffull) != 0;
}

// The capped score in the log2 domain, inv = 1 / cap.  For 16-bit queries tanh y = 1 - 2 / (1 + e^2y), whose error of a few 2^-24 is
// absolute, so that a score is off by that many parts of the cap.  EXACT (fp32 queries): below 0.7 Lambert's fraction
// y / (1 + y^2 / (3 + y^2 / (5 + y^2 / (7 + y^2 / 9)))), off by less than y^10 / 9.8e6 of the value, and (e^2y - 1) /
// (e^2y + 1) above, each a few 2^-24 of the value.
template <bool EXACT>
__device__ __forceinline__ float capped(float x, float cap, float inv) {
  if (!EXACT) {
    const float e = exp2_approx(x * (2.f * kLog2e * inv));
    return cap * kLog2e * (1.f - __fdividef(2.f, 1.f + e));
  }
  const float y = x * inv, z = y * y;
  const float e = exp2_approx((y > 10.f ? 10.f : y) * (2.f * kLog2e));
  const float n0 = y * fmaf(z, z + 105.f, 945.f), d0 = fmaf(z, fmaf(z, 15.f, 420.f), 945.f);
  const float n1 = e - 1.f, d1 = e + 1.f;
  const bool small = fabsf(y) < 0.7f;
  return cap * kLog2e * __fdividef(small ? n0 : n1, small ? d0 : d1);
}

// The power of two that brings a query's largest magnitude into [128, 256), and its inverse.
__device__ __forceinline__ void query_factor(float amax, float& f, float& inv) {
  int ex = (int)(__float_as_uint(amax) >> 23);
  f = inv = 1.f;
  if (amax > 0.f && ex < 255) {
    ex = max(ex, 16);
    f = __uint_as_float((uint32_t)(261 - ex) << 23);
    inv = __uint_as_float((uint32_t)(ex - 7) << 23);
  }
}

// A pair of neighbouring query elements as fp32.
__device__ __forceinline__ float2 load2(const float* p) { return __ldg(reinterpret_cast<const float2*>(p)); }
__device__ __forceinline__ float2 load2(const __half* p) { return __half22float2(__ldg(reinterpret_cast<const __half2*>(p))); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
  return __bfloat1622float2(__ldg(reinterpret_cast<const __nv_bfloat162*>(p)));
}

// Four neighbouring values of an output row.
template <typename T>
__device__ __forceinline__ void store4(T* p, const float4& y) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = y;
  } else {
    __align__(8) T t[4] = {Io<T>::from_f(y.x), Io<T>::from_f(y.y), Io<T>::from_f(y.z), Io<T>::from_f(y.w)};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(t);
  }
}

__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m - kPShift + log2f(l)) * kLn2; }

}  // namespace ssd
