// Attention over the 8-bit KV cache, and the weight that each slot drew.
//
// Row r sees slots [0, prefix) and base + e for every bit e of mask[r], the
// framework's visibility rule.  With codes c and block scales a,
//   s_rj = scale * a^K_j * (q_r . c^K_j)          (optionally cap * tanh(s / cap))
//   out_r = sum_j p_rj a^V_j c^V_j / sum_j p_rj,  p_rj = exp(s_rj - max_j s_rj).
//
// k_kv8_attention computes S^T = K Q^T and O^T = V^T P^T with 16x8x16 fp16
// MMAs: sixteen keys (or sixteen head dims) are the M dimension and eight
// queries of one KV head the N dimension, so the group of a decoded token
// fills the tile.  Codes are exact in fp16; a query row is scaled by a power
// of two and, when it is fp32, split into hi + lo (22 bits), and so are its
// softmax weights.  Every warp takes sixteen-key tiles of its own, straight
// from global memory into registers (a lane's sixteen bytes of a row are the
// MMA's k indices in an order that Q is laid out to match), and keeps a
// running maximum, sum and O^T in registers; warps and CTAs merge at the end
// in a fixed order.  A tile lies inside one scale block, so its scales are
// one number each.
//
// k_kv8_weights recomputes the scores and adds exp(s - lse) over the chosen
// rows and the KV head's queries to an accumulator: each sixteen-slot tile is
// one warp's, so nothing is shared and the sums have one order.
#include <math.h>

#include "kv8.h"

namespace ssd {

namespace {

constexpr int kAttnWarps = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kPShift = 14.f;  // softmax weights are held times 2^14, within fp16's normal range

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_rest2(float a, float b, uint32_t hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return pack_half2(a - f.x, b - f.y);
}

// Tiles of sixteen slots: those of the prefix, then those that hold new slots past them.
struct Tiles {
  int n_prefix, first_new, n;
  __device__ __forceinline__ Tiles(int prefix, int base, int rows) {
    n_prefix = (prefix + 15) >> 4;
    first_new = max(n_prefix, base >> 4);
    n = n_prefix + max(0, ((base + rows + 15) >> 4) - first_new);
  }
  __device__ __forceinline__ int slot(int t) const { return (t < n_prefix ? t : first_new + t - n_prefix) << 4; }
};

__device__ __forceinline__ bool visible(int slot, int prefix, int base, unsigned long long mask) {
  const unsigned e = (unsigned)(slot - base);
  return slot < prefix || (e < 64u && ((mask >> e) & 1ull));
}

__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// Query element e (0..hd) of row q of the query block, as fp32.
template <typename T>
__device__ __forceinline__ float q_elem(const T* p, int e) {
  if constexpr (sizeof(T) == 4)
    return p[e];
  else
    return Io<T>::to_f(p[e]);
}

// Lay out eight queries as the MMA's B operand in shared memory: word (step, half, lane) holds the fp16 pair
// that lane (column g = lane / 4, c = lane % 4) multiplies in k step `step`.  Lane c's k indices of step
// 4 j + i are bytes 4 i .. 4 i + 3 of the row's sixteen-byte chunk c + 4 j.  One warp for each query;
// returns its inverse scale.
template <typename T, int HD, bool SPLIT>
__device__ __forceinline__ float stage_query(const T* q, uint32_t* hi, uint32_t* lo, int col, int lane) {
  constexpr int EPL = HD / 32;  // elements per lane: pairs (2 lane + 64 i)
  float x[EPL];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < EPL / 2; ++i) {
    x[2 * i] = q ? q_elem(q, 64 * i + 2 * lane) : 0.f;
    x[2 * i + 1] = q ? q_elem(q, 64 * i + 2 * lane + 1) : 0.f;
    amax = fmaxf(amax, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
  }
  amax = warp_max(amax);
  // a power of two that brings the largest magnitude into [128, 256)
  int ex = (int)(__float_as_uint(amax) >> 23);
  float f = 1.f, inv = 1.f;
  if (amax > 0.f && ex < 255) {
    ex = max(ex, 16);
    f = __uint_as_float((uint32_t)(261 - ex) << 23);
    inv = __uint_as_float((uint32_t)(ex - 7) << 23);
  }
#pragma unroll
  for (int i = 0; i < EPL / 2; ++i) {
    const int e = 64 * i + 2 * lane;  // even element of the pair
    const int chunk = e >> 4, word = (e >> 2) & 3, half = (e >> 1) & 1;
    const int step = (chunk >> 2) * 4 + word;
    const int at = (step * 2 + half) * 32 + col * 4 + (chunk & 3);
    const float a = x[2 * i] * f, b = x[2 * i + 1] * f;
    const uint32_t h = pack_half2(a, b);
    hi[at] = h;
    if (SPLIT) lo[at] = pack_rest2(a, b, h);
  }
  return inv;
}

__device__ __forceinline__ uint32_t word_of(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

// S^T += K Q^T for a tile of sixteen keys (klo: rows g, khi: rows g + 8) and QT query columns of eight.
template <int HD, int CODE, bool SPLIT, int QT>
__device__ __forceinline__ void scores(float (&s)[QT][4], const uint4 (&klo)[HD / 64], const uint4 (&khi)[HD / 64],
                                       const uint32_t* qhi, const uint32_t* qlo, int lane) {
  constexpr int QW = HD / 16 * 64;  // words of one eight-query operand
#pragma unroll
  for (int j = 0; j < HD / 64; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a[4];
      codes_to_half<CODE>(word_of(klo[j], i), a[0], a[2]);
      codes_to_half<CODE>(word_of(khi[j], i), a[1], a[3]);
      const int at = (4 * j + i) * 64 + lane;
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        mma16816(s[t], a, qhi[t * QW + at], qhi[t * QW + at + 32]);
        if (SPLIT) mma16816(s[t], a, qlo[t * QW + at], qlo[t * QW + at + 32]);
      }
    }
  }
}

// Score in the log2 domain of product x with coefficient c (scale * inverse scales [* log2 e without a cap]).
__device__ __forceinline__ float capped(float x, float c, float cap) { return cap * tanhf(x * c / cap) * kLog2e; }

// Grid (splits, KV heads, query blocks of 8 QT).
template <typename T, int HD, int CODE, int QT>
__global__ void __launch_bounds__(kAttnWarps * 32, 2) k_kv8_attention(const __grid_constant__ Kv8AttnArgs a) {
  constexpr bool SPLIT = sizeof(T) == 4;
  constexpr int NJ = HD / 64;        // sixteen-byte chunks of a row per lane
  constexpr int QB = 8 * QT;
  constexpr int QW = HD / 16 * 64;   // words of one eight-query operand
  constexpr int DT = HD / 16;        // head-dim tiles of O^T
  constexpr int OS = QB + 1;         // row stride of the merge buffer
  extern __shared__ uint32_t smem[];
  uint32_t* s_hi = smem;                       // [QT][QW]
  uint32_t* s_lo = smem + QT * QW;             // [QT][QW] when SPLIT
  float* s_o = reinterpret_cast<float*>(smem); // after the loop: [warps][HD][OS]
  __shared__ float s_inv[QB];
  __shared__ float s_m[kAttnWarps][QB], s_l[kAttnWarps][QB];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int split = blockIdx.x, h = blockIdx.y, q0 = blockIdx.z * QB;
  const int nq = a.rows * a.group;
  griddep_launch();
  for (int q = warp; q < QB; q += kAttnWarps) {
    const int qi = q0 + q;
    const T* p = nullptr;
    if (qi < nq) {
      const int r = qi / a.group;
      p = reinterpret_cast<const T*>(a.q) + (size_t)r * a.ld_q + (size_t)(h * a.group + qi - r * a.group) * HD;
    }
    const float inv = stage_query<T, HD, SPLIT>(p, s_hi + (q >> 3) * QW, s_lo + (q >> 3) * QW, q & 7, lane);
    if (lane == 0) s_inv[q] = inv;
  }
  __syncthreads();

  const Tiles tiles(a.prefix, a.base, a.rows);
  const int t_first = (int)((long long)tiles.n * split / a.n_split);
  const int t_last = (int)((long long)tiles.n * (split + 1) / a.n_split);
  const bool cap = a.cap > 0.f;

  float coef[QT][2];
  unsigned long long mask[QT][2];
  float m[QT][2], l[QT][2], o[QT][DT][4];
  float vref = 0.f;  // O^T is held in units of this scale of V
#pragma unroll
  for (int t = 0; t < QT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int q = t * 8 + 2 * c + e;
      coef[t][e] = a.scale * s_inv[q] * (cap ? 1.f : kLog2e);
      mask[t][e] = q0 + q < nq ? a.mask[(q0 + q) / a.group] : 0ull;
      m[t][e] = -INFINITY;
      l[t][e] = 0.f;
    }
#pragma unroll
  for (int t = 0; t < QT; ++t)
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][d][e] = 0.f;

  for (int ti = t_first + warp; ti < t_last; ti += kAttnWarps) {
    const int slot0 = tiles.slot(ti);
    const int page = a.c.btab[slot0 / kPage];
    if (!a.c.page_ok(page)) continue;
    const size_t row0 = a.c.page_row(page, h) + (size_t)(slot0 % kPage) * HD;
    uint4 klo[NJ], khi[NJ], v[4][HD / 128 ? 1 : 1];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      klo[j] = ld16(a.c.k + row0 + (size_t)g * HD + (c + 4 * j) * 16);
      khi[j] = ld16(a.c.k + row0 + (size_t)(g + 8) * HD + (c + 4 * j) * 16);
    }
    // V: keys 2c, 2c + 1, 2c + 8, 2c + 9; head dims g * HD / 8 ..
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint8_t* p = a.c.v + row0 + (size_t)(2 * c + (e & 1) + (e >> 1) * 8) * HD + g * (HD / 8);
      if (HD == 128) {
        v[e][0] = ld16(p);
      } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
        v[e][0] = make_uint4(u.x, u.y, 0u, 0u);
      }
    }
    const size_t sc = a.c.scale_at(page, h, slot0 % kPage);
    const float ks = __ldg(a.c.ks + sc);
    float vs = __ldg(a.c.vs + sc);

    float s[QT][4];
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
    scores<HD, CODE, SPLIT, QT>(s, klo, khi, s_hi, s_lo, lane);

    const bool full = slot0 + 16 <= a.prefix;
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float cf = coef[t][e & 1] * ks;
        s[t][e] = cap ? capped(s[t][e], cf, a.cap) : s[t][e] * cf;
        if (!full && !visible(slot0 + g + (e >> 1) * 8, a.prefix, a.base, mask[t][e & 1])) s[t][e] = -INFINITY;
      }
    if (!full) {  // rows that hold no token may hold any bits
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!visible(slot0 + 2 * c + (e & 1) + (e >> 1) * 8, a.prefix, a.base, a.any)) v[e][0] = make_uint4(0u, 0u, 0u, 0u);
    }

    // running maximum of each query column
    float alpha[QT][2];
    bool grow = vs > vref;
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(s[t][e], s[t][e + 2]);
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        const float mn = fmaxf(m[t][e], x);
        alpha[t][e] = mn > m[t][e] ? exp2_approx(m[t][e] - mn) : 1.f;  // (m = -inf: 0)
        grow |= mn > m[t][e];
        m[t][e] = mn;
        l[t][e] *= alpha[t][e];
      }
    if (__any_sync(0xffffffffu, grow)) {
      float av = 1.f;
      if (vs > vref) {
        av = vref / vs;
        vref = vs;
      }
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][d][e] *= alpha[t][e & 1] * av;
    }
    const float rv = vref > 0.f ? vs / vref : 0.f;  // at most 1

    uint32_t ph[QT][2], pl[QT][2];
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // keys g (e = 0) and g + 8
        float p[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float mm = m[t][u] == -INFINITY ? 0.f : m[t][u];
          const float x = exp2_approx(s[t][2 * e + u] - mm + kPShift);
          l[t][u] += x;
          p[u] = x * rv;
        }
        const uint32_t hi = pack_half2(p[0], p[1]);
        ph[t][e] = transpose8x8(hi);
        if (SPLIT) pl[t][e] = transpose8x8(pack_rest2(p[0], p[1], hi));
      }
    // O^T += V^T P^T: head-dim tile d holds dims 2d and 2d + 1 of every lane's run
#pragma unroll
    for (int w = 0; w < DT / 2; ++w) {
      uint32_t x0[4], x1[4];
      pair_to_half<CODE>(word_of(v[0][0], w), word_of(v[1][0], w), x0);
      pair_to_half<CODE>(word_of(v[2][0], w), word_of(v[3][0], w), x1);
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const uint32_t fa[4] = {x0[2 * d], x0[2 * d + 1], x1[2 * d], x1[2 * d + 1]};
#pragma unroll
        for (int t = 0; t < QT; ++t) {
          mma16816(o[t][2 * w + d], fa, ph[t][0], ph[t][1]);
          if (SPLIT) mma16816(o[t][2 * w + d], fa, pl[t][0], pl[t][1]);
        }
      }
    }
  }

  // Merge the warps: sums over the lanes of a column, then over the warps in order.
#pragma unroll
  for (int t = 0; t < QT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[t][e];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      if (g == 0) {
        s_m[warp][t * 8 + 2 * c + e] = m[t][e];
        s_l[warp][t * 8 + 2 * c + e] = x;
      }
    }
  __syncthreads();  // the staged queries are not read any more
#pragma unroll
  for (int t = 0; t < QT; ++t)
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dim = g * (HD / 8) + 2 * d + (e >> 1);
        s_o[(warp * HD + dim) * OS + t * 8 + 2 * c + (e & 1)] = o[t][d][e] * vref;
      }
  __syncthreads();
  for (int i = threadIdx.x; i < QB * HD; i += kAttnWarps * 32) {
    const int q = i / HD, d = i - q * HD, qi = q0 + q;
    if (qi >= nq) break;
    float M = s_m[0][q];
#pragma unroll
    for (int w = 1; w < kAttnWarps; ++w) M = fmaxf(M, s_m[w][q]);
    const float ref = M == -INFINITY ? 0.f : M;
    float x = 0.f, L = 0.f;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      const float f = exp2_approx(s_m[w][q] - ref);
      x += s_o[(w * HD + d) * OS + q] * f;
      L += s_l[w][q] * f;
    }
    if (a.n_split > 1) {
      const size_t at = ((size_t)h * nq + qi) * a.n_split + split;
      a.part_o[at * HD + d] = x;
      if (d == 0) a.part_ml[at] = make_float2(M, L);
    } else {
      const int r = qi / a.group, head = h * a.group + qi - r * a.group;
      const float y = L == 0.f ? 0.f : x / L;
      T* out = reinterpret_cast<T*>(a.out) + (size_t)r * a.ld_out + (size_t)head * HD + d;
      if constexpr (SPLIT)
        *out = y;
      else
        *out = Io<T>::from_f(y);
      if (d == 0 && a.lse) a.lse[(size_t)r * a.n_q + head] = L == 0.f ? -INFINITY : (M - kPShift + log2f(L)) * kLn2;
    }
  }
}

// Grid (queries / 4): one warp for each query adds its splits in order.
template <typename T, int HD>
__global__ void __launch_bounds__(128) k_kv8_merge(const __grid_constant__ Kv8AttnArgs a) {
  constexpr int DPL = HD / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nq = a.rows * a.group;
  const int i = blockIdx.x * 4 + warp;
  griddep_wait();
  if (i >= a.c.n_kv * nq) return;
  const int h = i / nq, qi = i - h * nq, r = qi / a.group, head = h * a.group + qi - r * a.group;
  const float2* ml = a.part_ml + (size_t)i * a.n_split;
  float M = -INFINITY;
  for (int s = lane; s < a.n_split; s += 32) M = fmaxf(M, ml[s].x);
  M = warp_max(M);
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f, x[DPL];
#pragma unroll
  for (int d = 0; d < DPL; ++d) x[d] = 0.f;
  const float* po = a.part_o + (size_t)i * a.n_split * HD + lane * DPL;
#pragma unroll 8
  for (int s = 0; s < a.n_split; ++s) {
    const float2 t = ml[s];
    const float f = exp2_approx(t.x - ref);
    L += t.y * f;
#pragma unroll
    for (int d = 0; d < DPL; ++d) x[d] += po[(size_t)s * HD + d] * f;
  }
  T* out = reinterpret_cast<T*>(a.out) + (size_t)r * a.ld_out + (size_t)head * HD + lane * DPL;
#pragma unroll
  for (int d = 0; d < DPL; ++d) {
    const float y = L == 0.f ? 0.f : x[d] / L;
    if constexpr (sizeof(T) == 4)
      out[d] = y;
    else
      out[d] = Io<T>::from_f(y);
  }
  if (lane == 0 && a.lse) a.lse[(size_t)r * a.n_q + head] = L == 0.f ? -INFINITY : (M - kPShift + log2f(L)) * kLn2;
}

// ---------------------------------------------------------------- accumulated weights

constexpr int kWWarps = 8;
constexpr int kWQ = 8;  // queries staged at once are kWQ eights

// Grid (groups of kWWarps tiles, KV heads): each warp owns one sixteen-slot tile, the CTA walks over the
// chosen queries.
template <typename T, int HD, int CODE>
__global__ void __launch_bounds__(kWWarps * 32) k_kv8_weights(const __grid_constant__ Kv8AttnArgs a, int n_slots) {
  constexpr bool SPLIT = sizeof(T) == 4;
  constexpr int NJ = HD / 64;
  constexpr int QW = HD / 16 * 64;
  extern __shared__ uint32_t smem[];
  uint32_t* s_hi = smem;
  uint32_t* s_lo = smem + kWQ * QW;
  __shared__ float s_coef[kWQ * 8], s_lse[kWQ * 8];
  __shared__ unsigned long long s_mask[kWQ * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int h = blockIdx.y;
  const int slot0 = (blockIdx.x * kWWarps + warp) * 16;
  const bool cap = a.cap > 0.f;
  const bool full = slot0 + 16 <= a.prefix;
  const bool some = slot0 < a.prefix || (slot0 < a.base + a.rows && slot0 + 16 > a.base);
  const int page = slot0 < n_slots && some ? a.c.btab[slot0 / kPage] : -1;
  const bool live = a.c.page_ok(page);
  uint4 klo[NJ], khi[NJ];
  float ks = 0.f;
#pragma unroll
  for (int j = 0; j < NJ; ++j) klo[j] = khi[j] = make_uint4(0u, 0u, 0u, 0u);
  if (live) {
    const size_t row0 = a.c.page_row(page, h) + (size_t)(slot0 % kPage) * HD;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      klo[j] = ld16(a.c.k + row0 + (size_t)g * HD + (c + 4 * j) * 16);
      khi[j] = ld16(a.c.k + row0 + (size_t)(g + 8) * HD + (c + 4 * j) * 16);
    }
    ks = __ldg(a.c.ks + a.c.scale_at(page, h, slot0 % kPage));
  }
  float sum[2] = {0.f, 0.f};  // slots g and g + 8
  const int nq = a.n_take * a.group;
  for (int q0 = 0; q0 < nq; q0 += kWQ * 8) {
    const int eights = min(kWQ, (nq - q0 + 7) / 8);
    __syncthreads();
    for (int q = warp; q < eights * 8; q += kWWarps) {
      const int qi = q0 + q;
      const T* p = nullptr;
      float lse = 0.f;
      unsigned long long mask = 0ull;
      if (qi < nq) {
        const int ti = qi / a.group, r = a.take[ti], head = h * a.group + qi - ti * a.group;
        p = reinterpret_cast<const T*>(a.q) + (size_t)r * a.ld_q + (size_t)head * HD;
        lse = a.lse[(size_t)r * a.n_q + head];
        mask = a.mask[r];
      }
      const float inv = stage_query<T, HD, SPLIT>(p, s_hi + (q >> 3) * QW, s_lo + (q >> 3) * QW, q & 7, lane);
      if (lane == 0) {
        s_coef[q] = qi < nq ? a.scale * inv * (cap ? 1.f : kLog2e) : 0.f;
        // a padding query, and a row that saw nothing (lse -inf), adds exp2(-inf) = 0
        s_lse[q] = qi < nq && lse != -INFINITY ? lse * kLog2e : INFINITY;
        s_mask[q] = mask;
      }
    }
    __syncthreads();
    if (!live) continue;
    for (int t = 0; t < eights; ++t) {
      float s[1][4] = {{0.f, 0.f, 0.f, 0.f}};
      scores<HD, CODE, SPLIT, 1>(s, klo, khi, s_hi + t * QW, s_lo + t * QW, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int q = t * 8 + 2 * c + (e & 1);
        const float cf = s_coef[q] * ks;
        const float x = cap ? capped(s[0][e], cf, a.cap) - s_lse[q] : fmaf(s[0][e], cf, -s_lse[q]);
        const bool see = full || visible(slot0 + g + (e >> 1) * 8, a.prefix, a.base, s_mask[q]);
        sum[e >> 1] += see ? exp2_approx(x) : 0.f;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
    sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
  }
  if (c < 2) {
    const int slot = slot0 + g + c * 8;
    if (slot < n_slots) {
      const size_t at = (size_t)h * a.ld_w + slot;
      a.w_out[at] = (a.w_in ? a.w_in[at] : 0.f) + sum[c];
    }
  }
}

template <typename T, int HD, int CODE, int QT>
bool run_attention(const Kv8AttnArgs& a, cudaStream_t st) {
  constexpr int QB = 8 * QT;
  constexpr size_t stage = (size_t)QT * (HD / 16 * 64) * 4 * (sizeof(T) == 4 ? 2 : 1);
  constexpr size_t merge = (size_t)kAttnWarps * HD * (QB + 1) * 4;
  constexpr size_t smem = stage > merge ? stage : merge;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(k_kv8_attention<T, HD, CODE, QT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess)
    return false;
  const int nq = a.rows * a.group;
  k_kv8_attention<T, HD, CODE, QT><<<dim3(a.n_split, a.c.n_kv, (nq + QB - 1) / QB), kAttnWarps * 32, smem, st>>>(a);
  if (a.n_split > 1) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((a.c.n_kv * nq + 3) / 4);
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, k_kv8_merge<T, HD>, a) != cudaSuccess) return false;
  }
  return cudaGetLastError() == cudaSuccess;
}

template <typename T, int HD, int CODE>
bool run_attention_q(const Kv8AttnArgs& a, cudaStream_t st) {
  return a.rows * a.group <= 8 ? run_attention<T, HD, CODE, 1>(a, st) : run_attention<T, HD, CODE, 2>(a, st);
}

template <typename T, int HD, int CODE>
bool run_weights(const Kv8AttnArgs& a, cudaStream_t st) {
  constexpr size_t smem = (size_t)kWQ * (HD / 16 * 64) * 4 * (sizeof(T) == 4 ? 2 : 1);
  const int n_slots = a.prefix > a.base + a.rows ? a.prefix : a.base + a.rows;
  const int tiles = (n_slots + 15) / 16;
  k_kv8_weights<T, HD, CODE>
      <<<dim3((tiles + kWWarps - 1) / kWWarps, a.c.n_kv), kWWarps * 32, smem, st>>>(a, n_slots);
  return cudaGetLastError() == cudaSuccess;
}

template <typename T>
bool attention_of(const Kv8AttnArgs& a, cudaStream_t st) {
  const bool i8 = a.c.code == KV8_INT8;
  if (a.c.hd == 128)
    return i8 ? run_attention_q<T, 128, KV8_INT8>(a, st) : run_attention_q<T, 128, KV8_E4M3>(a, st);
  return i8 ? run_attention_q<T, 64, KV8_INT8>(a, st) : run_attention_q<T, 64, KV8_E4M3>(a, st);
}

template <typename T>
bool weights_of(const Kv8AttnArgs& a, cudaStream_t st) {
  const bool i8 = a.c.code == KV8_INT8;
  if (a.c.hd == 128) return i8 ? run_weights<T, 128, KV8_INT8>(a, st) : run_weights<T, 128, KV8_E4M3>(a, st);
  return i8 ? run_weights<T, 64, KV8_INT8>(a, st) : run_weights<T, 64, KV8_E4M3>(a, st);
}

}  // namespace

int kv8_attention_splits(int rows, int group, int n_kv, int slots) {
  const int nq = rows * group;
  const int blocks = n_kv * (nq <= 8 ? 1 : (nq + 15) / 16);
  const int tiles = (slots + 15) / 16;
  const int fit = 304 / blocks;                          // two CTAs on each of 152 SMs
  const int most = (tiles + kAttnWarps - 1) / kAttnWarps;  // a tile for every warp
  const int n = fit < most ? fit : most;
  return n < 1 ? 1 : n;
}

bool launch_kv8_attention(const Kv8AttnArgs& a, int io, cudaStream_t st) {
  return io == 0 ? attention_of<__nv_bfloat16>(a, st) : io == 1 ? attention_of<__half>(a, st) : attention_of<float>(a, st);
}

bool launch_kv8_weights(const Kv8AttnArgs& a, int io, cudaStream_t st) {
  return io == 0 ? weights_of<__nv_bfloat16>(a, st) : io == 1 ? weights_of<__half>(a, st) : weights_of<float>(a, st);
}

}  // namespace ssd
