// Device-side definitions shared by the kernels of the 8-bit KV cache: where a
// page, a row and a scale lie, and how codes become 16-bit numbers.
//
// A cache keeps, for each layer, codes [pool_pages][n_kv][64][hd] of one byte
// (int8 in [-127, 127], or e4m3) and scales [pool_pages][n_kv][64 / T] in
// fp32, one for each block of T tokens and KV head; a slot's value is
// code * scale.  Every code is exact in fp16, so fp16 MMAs multiply the codes
// as they are, and a block's scale is applied to the fp32 products (K) or to
// the softmax weights (V).
#pragma once

#include "common.cuh"

namespace ssd {

enum Kv8Code { KV8_INT8 = 0, KV8_E4M3 = 1 };

// One layer of a cache, as the kernels see it.
struct Kv8View {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  const int* btab;  // [n_pages] logical page -> physical page
  int pool;         // physical pages; an entry of btab outside [0, pool) holds no tokens
  int n_kv, hd;
  int tshift;       // log2 T
  int code;         // Kv8Code

  // first byte of (physical page, head)'s 64 rows
  __device__ __forceinline__ size_t page_row(int page, int h) const { return ((size_t)page * n_kv + h) * kPage * hd; }
  // scale of (physical page, head, slot of the page)
  __device__ __forceinline__ size_t scale_at(int page, int h, int in_page) const {
    return (((size_t)page * n_kv + h) << (6 - tshift)) + (in_page >> tshift);
  }
  __device__ __forceinline__ bool page_ok(int page) const { return (unsigned)page < (unsigned)pool; }
};

// D += A B, A 16x16 fp16 (row), B 16x8 fp16 (col), D 16x8 fp32.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same with nothing in D before.
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Transpose of an 8x8 matrix of 16-bit values held one row pair per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two) {
  uint32_t r;
  const uint16_t s = (uint16_t)two;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(s));
  return r;
}

__device__ __forceinline__ uint32_t hsub2_u32(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Four codes of a word as fp16: (byte 0, byte 1) and (byte 2, byte 3).
// int8: byte ^ 0x80 = code + 128 under the high byte 0x64 is the fp16 number 1024 + code + 128.
template <int CODE>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& h01, uint32_t& h23) {
  if (CODE == KV8_INT8) {
    w ^= 0x80808080u;
    h01 = hsub2_u32(__byte_perm(w, 0x64646464u, 0x4140), 0x64806480u);
    h23 = hsub2_u32(__byte_perm(w, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    h01 = e4m3x2_to_half2(w);
    h23 = e4m3x2_to_half2(w >> 16);
  }
}

// Byte i of words a and b side by side as fp16, for i = 0..3.
template <int CODE>
__device__ __forceinline__ void pair_to_half(uint32_t a, uint32_t b, uint32_t (&h)[4]) {
  const uint32_t z01 = __byte_perm(a, b, 0x5140), z23 = __byte_perm(a, b, 0x7362);
  codes_to_half<CODE>(z01, h[0], h[1]);
  codes_to_half<CODE>(z23, h[2], h[3]);
}

// Values of the four codes of a word under scale s (fp32 products of numbers that are exact in fp16).
template <int CODE>
__device__ __forceinline__ void decode4(uint32_t w, float s, float* x) {
  uint32_t h01, h23;
  codes_to_half<CODE>(w, h01, h23);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h01));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h23));
  x[0] = __fmul_rn(a.x, s), x[1] = __fmul_rn(a.y, s), x[2] = __fmul_rn(b.x, s), x[3] = __fmul_rn(b.y, s);
}

// Four codes, packed, of x under the inverse scale m: the fp32 products rounded to the nearest codes (ties to even),
// clamped to the largest one.  NaN becomes 0; the product of an infinity and m > 0 clamps.  ODD: whether x may hold a
// NaN or an infinity; without one |x m| rounds to qmax at most, since the scale is no smaller than the block's
// largest magnitude over qmax.
template <int CODE, bool ODD>
__device__ __forceinline__ uint32_t encode4(const float* x, float m) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = __fmul_rn(x[i], m);
    if (ODD) {
      constexpr float lim = CODE == KV8_INT8 ? 127.f : 448.f;
      y[i] = m > 0.f && x[i] == x[i] ? fminf(lim, fmaxf(-lim, y[i])) : 0.f;
    }
  }
  if (CODE == KV8_INT8) {
    // 1.5 2^23 + y: the sum's low byte is y rounded to the nearest integer, ties to even, in two's complement
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(__fadd_rn(y[i], 12582912.f));
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
  uint16_t lo, hi;  // (cvt's first source is the upper half)
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1]), "f"(y[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3]), "f"(y[2]));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Scale of a block whose largest finite magnitude is amax (0 where that is below the smallest normal
// number, so that its inverse is finite), and the inverse that its codes are taken with.
template <int CODE>
__device__ __forceinline__ float block_scale(float amax) {
  const float s = __fdiv_rn(amax, CODE == KV8_INT8 ? 127.f : 448.f);
  return s < 1.17549435e-38f ? 0.f : s;
}
__device__ __forceinline__ float inverse_scale(float s) { return s > 0.f ? __frcp_rn(s) : 0.f; }

}  // namespace ssd
