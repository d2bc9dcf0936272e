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
// softmax weights (16-bit queries keep 11 bits of a weight, less than their
// output's own rounding).  Every warp takes 32-slot tiles of its own: codes by
// cp.async into its ring in shared memory, from there into registers (a lane's
// sixteen bytes of a row are the MMA's k indices in an order that Q is laid
// out to match), and keeps a running maximum, sum and O^T in registers; warps
// and CTAs merge at the end in a fixed order.  A tile's halves of sixteen
// slots lie inside one scale block each, so a half's scales are one number.
//
// What bounds it (one GB300, times of a captured call):
//   one bf16 token, 64 heads on 8, 65532 e4m3 slots (134 MB): 26.8 us, 5.0 TB/s
//     of a copy's 6.8; 23 us of it are the stream, at 63 % of the DRAM's cycles
//     with a third of the ALU's for the conversions, the rest the merge kernel;
//   7 fp32 rows, 32 heads on 8, 4100 int8 slots: 14.2 us, a tile for every
//     warp: latency (staging, one tile, two merges); MMAs are 17 % of it;
//   one fp32 token, 32 heads on 8, 641 slots: 7.2 us, latency.
// Chunks of many queries run on the fifth-generation tensor cores instead
// (launch_kv8_attention_tc).
//
// k_kv8_weights recomputes the scores and adds exp(s - lse) over the chosen
// rows and the KV head's queries to an accumulator: each sixteen-slot tile is
// one warp's, so nothing is shared and the sums have one order.  5 rows of 64
// heads on 8 over 32776 e4m3 slots: 16.0 us, 36 MB (2.2 TB/s); bound by the
// MMAs and exponentials of 40 queries a slot, 28 and 24 % of their pipes, and
// the latency between them (three CTAs an SM: 18.9 us; K two tiles ahead:
// 18.0).
#include <cooperative_groups.h>

#include "kv8_attn.cuh"

namespace ssd {

namespace {

constexpr int kTileSlots = 32;   // slots that a warp takes at a time, all in one page
constexpr int kMaxCluster = 8;   // key splits that merge in distributed shared memory
constexpr int kMaxSplits = 152;  // key splits that merge through global memory
__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

// Lay out a query as column `col` of the MMA's B operand in shared memory.  Lane (g, c) of the MMA multiplies column
// g; its k indices of step 4 j + i are bytes 4 i .. 4 i + 3 of the row's sixteen-byte chunk c + 4 j.  The words (fp16
// pairs) of two steps lie side by side, so that a lane reads them sixteen bytes at a time: word
// ((step / 2) 32 + lane) 4 + (step % 2) 2 + half.  One warp for each query; returns its inverse scale.
template <typename T, int HD, bool SPLIT>
__device__ __forceinline__ float stage_query(const T* q, uint32_t* hi, uint32_t* lo, int col, int lane) {
  constexpr int EPL = HD / 32;  // elements per lane: pairs (2 lane + 64 i)
  float x[EPL];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < EPL / 2; ++i) {
    const float2 v = q ? load2(q + 64 * i + 2 * lane) : make_float2(0.f, 0.f);
    x[2 * i] = v.x;
    x[2 * i + 1] = v.y;
    amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
  }
  float f, inv;
  query_factor(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax))), f, inv);  // (amax >= 0)
#pragma unroll
  for (int i = 0; i < EPL / 2; ++i) {
    const int e = 64 * i + 2 * lane;  // even element of the pair
    const int chunk = e >> 4, word = (e >> 2) & 3, half = (e >> 1) & 1;
    const int step = (chunk >> 2) * 4 + word;
    const int at = ((step >> 1) * 32 + col * 4 + (chunk & 3)) * 4 + (step & 1) * 2 + half;
    const float a = x[2 * i] * f, b = x[2 * i + 1] * f;
    const uint32_t h = pack_half2(a, b);
    hi[at] = h;
    if (SPLIT) lo[at] = pack_rest2(a, b, h);
  }
  return inv;
}

__device__ __forceinline__ uint32_t word_of(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

// S^T = K Q^T for two halves of sixteen keys (klo: rows g, khi: rows g + 8) and QT columns of eight queries.
template <int HD, int CODE, bool SPLIT, int QT>
__device__ __forceinline__ void scores(float (&s)[2][QT][4], const uint4 (&klo)[2][HD / 64], const uint4 (&khi)[2][HD / 64],
                                       const uint32_t* qhi, const uint32_t* qlo, int lane) {
  constexpr int QW = HD / 16 * 64;  // words of one eight-query operand
#pragma unroll
  for (int p = 0; p < HD / 32; ++p) {  // pairs of k steps
    uint32_t a[2][2][4];               // [step of the pair][half]
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        codes_to_half<CODE>(word_of(klo[b][p >> 1], (p & 1) * 2 + i), a[i][b][0], a[i][b][2]);
        codes_to_half<CODE>(word_of(khi[b][p >> 1], (p & 1) * 2 + i), a[i][b][1], a[i][b][3]);
      }
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const uint4 h = *reinterpret_cast<const uint4*>(qhi + t * QW + (p * 32 + lane) * 4);
      if (SPLIT) {
        // The tensor cores cut off what does not fit an accumulator, so a pair of steps starts from nothing, with its
        // small part first, and the pairs are added rounded (one chain of all steps was about twice as far off).
        const uint4 l = *reinterpret_cast<const uint4*>(qlo + t * QW + (p * 32 + lane) * 4);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float d[4];
          mma16816_first(d, a[0][b], l.x, l.y);
          mma16816(d, a[1][b], l.z, l.w);
          mma16816(d, a[0][b], h.x, h.y);
          mma16816(d, a[1][b], h.z, h.w);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[b][t][e] = p == 0 ? d[e] : s[b][t][e] + d[e];
        }
      } else {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (p == 0)
            mma16816_first(s[b][t], a[0][b], h.x, h.y);
          else
            mma16816(s[b][t], a[0][b], h.x, h.y);
          mma16816(s[b][t], a[1][b], h.z, h.w);
        }
      }
    }
  }
}

// A warp's ring of 32-slot tiles in shared memory: the K rows, then the V rows.  Sixteen-byte chunks are swizzled
// inside 128-byte lines, so that neither a lane's chunks of its own K row nor its run of four V rows meet in a bank.
template <int HD, int STAGES>
struct Ring {
  static constexpr int kStages = STAGES;
  static constexpr int kTensor = kTileSlots * HD;  // bytes of K (or V) of one tile
  static constexpr int kStage = 2 * kTensor;
  static constexpr int kWarp = kStages * kStage;
  static __device__ __forceinline__ int at(int row, int byte) {
    if (HD == 128) return row * 128 + (byte ^ ((row & 7) << 4));
    return (row >> 1) * 128 + ((((row & 1) << 6) | byte) ^ (((row >> 1) & 3) << 5));
  }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr bool cluster_fits(int queries, bool fp32) { return queries < 32 || !fp32; }

// Warps of a CTA and stages of a warp's ring.  Eight queries leave registers for twelve warps, which hide the
// latency of the conversions, with two stages each (8 KB under way a warp, 96 KB an SM); the larger blocks run
// eight warps with three.
template <int HD, int QT>
struct AttnShape {
  static constexpr int W = QT == 1 ? 12 : 8;
  using R = Ring<HD, QT == 1 ? 2 : 3>;
};

template <typename T, int HD, int QT>
struct AttnSmem {
  using R = typename AttnShape<HD, QT>::R;
  static constexpr int W = AttnShape<HD, QT>::W;
  static constexpr int QB = 8 * QT;
  static constexpr int QW = HD / 16 * 64;                                   // words of one eight-query operand
  static constexpr int kQ = QT * QW * 4 * (sizeof(T) == 4 ? 2 : 1);         // staged queries
  static constexpr int kRing = W * R::kWarp;
  static constexpr int OS = HD + 4;                                         // row stride of the merge buffers
  static constexpr int kMerge = W * QB * OS * 4;                            // over the ring, after the loop
  static constexpr int kHead = W * R::kStages * 32;                         // tile headers (TileHead)
  // partial results that the other CTAs of a cluster send (32 fp32 queries leave no room, and use scratch)
  static constexpr int kPart = cluster_fits(QB, sizeof(T) == 4) ? (QB * HD / 4 + kMaxCluster) * 16 : 0;
  static constexpr int kLoop = kQ + (kRing > kMerge ? kRing : kMerge);
  static constexpr int kBytes = kLoop + kHead + kPart;
};

struct __align__(16) TileHead {
  float ks[2], vs[2];  // scales of the tile's halves
  int used, pad[3];    // whether the tile's page is one
};

// Grid (splits, KV heads, query blocks of 8 QT).  With part_o the splits' results go to scratch; else, when there
// is more than one, the splits of a query block are one cluster.
template <typename T, int HD, int CODE, int QT>
__global__ void __launch_bounds__(AttnShape<HD, QT>::W * 32, 1) k_kv8_attention(const __grid_constant__ Kv8AttnArgs a) {
  namespace cg = cooperative_groups;
  using L = AttnSmem<T, HD, QT>;
  using R = typename L::R;
  constexpr int W = L::W;
  constexpr bool SPLIT = sizeof(T) == 4;
  constexpr int NJ = HD / 64;        // sixteen-byte chunks of a K row per lane
  constexpr int QB = L::QB, QW = L::QW, OS = L::OS;
  constexpr int DT = HD / 16;        // head-dim tiles of O^T
  extern __shared__ __align__(128) unsigned char s_dyn[];
  uint32_t* s_hi = reinterpret_cast<uint32_t*>(s_dyn);   // [QT][QW]
  uint32_t* s_lo = s_hi + QT * QW;                       // [QT][QW] when SPLIT
  float* s_o = reinterpret_cast<float*>(s_dyn + L::kQ);  // after the loop: [warps][QB][OS]
  __shared__ float s_inv[QB];
  __shared__ float s_m[W][QB], s_l[W][QB];
  __shared__ float2 s_ml[QB];        // this CTA's maximum and sum
  __shared__ float2 s_f[kMaxCluster][QB];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int split = blockIdx.x, h = blockIdx.y, q0 = blockIdx.z * QB;
  const int nq = a.rows * a.group;
  const bool clustered = !a.part_o && a.n_split > 1;
  if (clustered) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // waited for before the merge
  griddep_launch();
  griddep_wait();

  const Tiles<5> tiles(a.prefix, a.base, a.rows);
  const int t_first = split * a.split_tiles, t_last = min(tiles.n, t_first + a.split_tiles);
  const unsigned char* ring = s_dyn + L::kQ + warp * R::kWarp;
  TileHead* heads = reinterpret_cast<TileHead*>(s_dyn + L::kLoop) + warp * R::kStages;

  // Tile ti (physical page `page`) into ring stage st; one group of copies whether or not there is a tile.
  auto fill = [&](int st, int ti, int page) {
    const bool ok = ti < t_last && a.c.page_ok(page);
    if (ok) {
      const int in_page = tiles.slot(ti) % kPage;
      const size_t row0 = a.c.page_row(page, h) + (size_t)in_page * HD + lane * 16;
      const uint32_t dst = smem_u32(ring + st * R::kStage);
#pragma unroll
      for (int i = 0; i < HD / 16; ++i) {
        const int x = (i * 32 + lane) * 16, to = R::at(x / HD, x % HD);
        cp_async16(dst + to, a.c.k + row0 + i * 512);
        cp_async16(dst + R::kTensor + to, a.c.v + row0 + i * 512);
      }
      if (lane < 4)
        cp_async4(smem_u32(&heads[st]) + lane * 4,
                  (lane & 2 ? a.c.vs : a.c.ks) + a.c.scale_at(page, h, in_page + (lane & 1) * 16));
    }
    if (lane == 4) heads[st].used = ok;
    cp_async_commit();
  };
  auto page_of = [&](int ti) { return ti < t_last ? __ldg(a.c.btab + tiles.slot(ti) / kPage) : -1; };

  int pages[R::kStages];
#pragma unroll
  for (int i = 0; i < R::kStages; ++i) pages[i] = page_of(t_first + warp + i * W);
#pragma unroll
  for (int i = 0; i < R::kStages - 1; ++i) fill(i, t_first + warp + i * W, pages[i]);
  int page_next = pages[R::kStages - 1];

#pragma unroll 4
  for (int q = warp; q < QB; q += W) {
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

  const bool cap = a.cap > 0.f;
  const float inv_cap = cap ? 1.f / a.cap : 0.f;
  float coef[QT][2];
  float m[QT][2], l[QT][2], o[QT][DT][4];
  float vref = 0.f, vinv = 0.f;  // O^T is held in units of vref, a scale of V
#pragma unroll
  for (int t = 0; t < QT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      coef[t][e] = a.scale * s_inv[t * 8 + 2 * c + e] * (cap ? 1.f : kLog2e);
      m[t][e] = -INFINITY;
      l[t][e] = 0.f;
    }
#pragma unroll
  for (int t = 0; t < QT; ++t)
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][d][e] = 0.f;

  int st = 0;
  for (int ti = t_first + warp; ti < t_last; ti += W) {
    cp_async_wait<R::kStages - 2>();
    __syncwarp();  // every lane's copies of this stage have landed; the stage before it is free
    {
      const int ahead = ti + (R::kStages - 1) * W;
      fill(st == 0 ? R::kStages - 1 : st - 1, ahead, page_next);
      page_next = page_of(ahead + W);
    }
    const unsigned char* kbuf = ring + st * R::kStage;
    const unsigned char* vbuf = kbuf + R::kTensor;
    const TileHead head = heads[st];
    st = st + 1 == R::kStages ? 0 : st + 1;
    if (!head.used) continue;
    const int slot0 = tiles.slot(ti);

    uint4 klo[2][NJ], khi[2][NJ];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        klo[b][j] = *reinterpret_cast<const uint4*>(kbuf + R::at(b * 16 + g, (c + 4 * j) * 16));
        khi[b][j] = *reinterpret_cast<const uint4*>(kbuf + R::at(b * 16 + g + 8, (c + 4 * j) * 16));
      }
    float s[2][QT][4];  // halves of sixteen keys
    scores<HD, CODE, SPLIT, QT>(s, klo, khi, s_hi, s_lo, lane);

    const bool full = slot0 + kTileSlots <= a.prefix;
    float vmax = fmaxf(head.vs[0], head.vs[1]);
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int r = 0; r < 2; ++r) s[b][t][2 * r + u] *= coef[t][u] * head.ks[b];
    if (cap) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[b][t][e] = capped<SPLIT>(s[b][t][e], a.cap, inv_cap);
    }
    if (!full) {
      vmax = fmaxf(visible_any(slot0, a) ? head.vs[0] : 0.f, visible_any(slot0 + 16, a) ? head.vs[1] : 0.f);
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int qi = q0 + t * 8 + 2 * c + u;
          const unsigned long long mask = qi < nq ? a.mask[qi / a.group] : 0ull;
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (!visible(slot0 + b * 16 + r * 8 + g, a.prefix, a.base, mask)) s[b][t][2 * r + u] = -INFINITY;
        }
    }

    // running maximum of each query column
    bool grow = vmax > vref;
    float top[QT][2];
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float x = fmaxf(fmaxf(s[0][t][u], s[0][t][u + 2]), fmaxf(s[1][t][u], s[1][t][u + 2]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        top[t][u] = x;
        grow |= x > m[t][u];
      }
    if (__any_sync(0xffffffffu, grow)) {
      float av = 1.f;
      if (vmax > vref) {
        av = vref / vmax;
        vref = vmax;
        vinv = 1.f / vmax;
      }
#pragma unroll
      for (int t = 0; t < QT; ++t) {
        float alpha[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float mn = fmaxf(m[t][u], top[t][u]);
          alpha[u] = mn > m[t][u] ? exp2_approx(m[t][u] - mn) : 1.f;  // (m = -inf: 0)
          m[t][u] = mn;
          l[t][u] *= alpha[u];
          alpha[u] *= av;
        }
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][d][e] *= alpha[e & 1];
      }
    }
    float shift[QT][2];  // what is left of a score before the exponential
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) shift[t][u] = kPShift - (m[t][u] == -INFINITY ? 0.f : m[t][u]);

#pragma unroll
    for (int b = 0; b < 2; ++b) {
      // at most 1 where the half has a visible slot (elsewhere the scale may be anything, and no weight is used)
      const float rv = head.vs[b] <= vref ? head.vs[b] * vinv : 0.f;
      uint32_t ph[QT][2], pl[QT][2];
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {  // keys g and g + 8
          float p[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float x = exp2_approx(s[b][t][2 * r + u] + shift[t][u]);
            l[t][u] += x;
            p[u] = x * rv;
          }
          const uint32_t hi = pack_half2(p[0], p[1]);
          ph[t][r] = transpose8x8(hi);
          if (SPLIT) pl[t][r] = transpose8x8(pack_rest2(p[0], p[1], hi));
        }
      // V: keys 2c, 2c + 1, 2c + 8, 2c + 9 of the half; head dims g * HD / 8 ..
      uint4 v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = b * 16 + 2 * c + (e & 1) + (e >> 1) * 8;
        if (HD == 128) {
          v[e] = *reinterpret_cast<const uint4*>(vbuf + R::at(row, g * 16));
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(vbuf + R::at(row, g * 8));
          v[e] = make_uint4(w.x, w.y, 0u, 0u);
        }
      }
      if (!full) {  // rows that hold no token may hold any bits
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!visible(slot0 + b * 16 + 2 * c + (e & 1) + (e >> 1) * 8, a.prefix, a.base, a.any))
            v[e] = make_uint4(0u, 0u, 0u, 0u);
      }
      // O^T += V^T P^T: head-dim tile d holds dims 2d and 2d + 1 of every lane's run
#pragma unroll
      for (int w = 0; w < DT / 2; ++w) {
        uint32_t x0[4], x1[4];
        pair_to_half<CODE>(word_of(v[0], w), word_of(v[1], w), x0);
        pair_to_half<CODE>(word_of(v[2], w), word_of(v[3], w), x1);
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
  }
  cp_async_wait<0>();

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
  __syncthreads();  // no warp reads its ring any more
#pragma unroll
  for (int t = 0; t < QT; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int d = 0; d < DT; d += 2)
        *reinterpret_cast<float4*>(s_o + (size_t)(warp * QB + t * 8 + 2 * c + e) * OS + g * (HD / 8) + 2 * d) =
            make_float4(o[t][d][e] * vref, o[t][d][e + 2] * vref, o[t][d + 1][e] * vref, o[t][d + 1][e + 2] * vref);
  __syncthreads();
  constexpr int ITEMS = QB * HD / 4;  // four dims of a query
  constexpr int PER = (ITEMS + W * 32 - 1) / (W * 32);
  float4 mine[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = threadIdx.x + j * W * 32;
    if (i >= ITEMS) break;
    const int q = i / (HD / 4), d = (i % (HD / 4)) * 4;
    float M = s_m[0][q];
#pragma unroll
    for (int w = 1; w < W; ++w) M = fmaxf(M, s_m[w][q]);
    const float ref = M == -INFINITY ? 0.f : M;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = exp2_approx(s_m[w][q] - ref);
      const float4 y = *reinterpret_cast<const float4*>(s_o + (size_t)(w * QB + q) * OS + d);
      x.x += y.x * f, x.y += y.y * f, x.z += y.z * f, x.w += y.w * f;
      sum += s_l[w][q] * f;
    }
    mine[j] = x;
    if (d == 0) s_ml[q] = make_float2(M, sum);
  }

  auto output = [&](int q, int d, const float4& x, float M, float sum) {
    const int qi = q0 + q;
    if (qi >= nq) return;
    const int r = qi / a.group, head = h * a.group + qi - r * a.group;
    const float f = sum == 0.f ? 0.f : 1.f / sum;
    store4(reinterpret_cast<T*>(a.out) + (size_t)r * a.ld_out + (size_t)head * HD + d,
           make_float4(x.x * f, x.y * f, x.z * f, x.w * f));
    if (d == 0 && a.lse) a.lse[a.lse_at(r, head)] = lse_of(M, sum);
  };

  __syncthreads();
  if (a.part_o) {  // partial results, merged by k_kv8_merge
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = threadIdx.x + j * W * 32;
      if (i >= ITEMS) break;
      const int q = i / (HD / 4), d = (i % (HD / 4)) * 4, qi = q0 + q;
      if (qi >= nq) break;
      const size_t at = ((size_t)h * nq + qi) * a.n_split + split;
      *reinterpret_cast<float4*>(a.part_o + at * HD + d) = mine[j];
      if (d == 0) a.part_ml[at] = s_ml[q];
    }
  } else if (a.n_split == 1) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = threadIdx.x + j * W * 32;
      if (i >= ITEMS) break;
      const int q = i / (HD / 4), d = (i % (HD / 4)) * 4;
      output(q, d, mine[j], s_ml[q].x, s_ml[q].y);
    }
  } else if constexpr (L::kPart > 0) {
    // The cluster's partial results: rank r adds every n_split-th item, which the others put into its shared memory
    // (a buffer of its own, since r may still be working on its tiles).
    cg::cluster_group cl = cg::this_cluster();
    float4* s_part = reinterpret_cast<float4*>(s_dyn + L::kLoop + L::kHead);  // [ranks][items of this rank]
    const int n = a.n_split, per = (ITEMS + n - 1) / n;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA of the cluster has started
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = threadIdx.x + j * W * 32;
      if (i < ITEMS) cl.map_shared_rank(s_part, i % n)[split * per + i / n] = mine[j];
    }
    for (int i = threadIdx.x; i < QB * n; i += W * 32) cl.map_shared_rank(&s_f[split][i % QB], i / QB)[0] = s_ml[i % QB];
    cl.sync();
    for (int k = threadIdx.x; k * n + split < ITEMS; k += W * 32) {
      const int i = k * n + split, q = i / (HD / 4), d = (i % (HD / 4)) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < n) M = fmaxf(M, s_f[r][q].x);
      const float ref = M == -INFINITY ? 0.f : M;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      float sum = 0.f;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < n) {
          const float2 ml = s_f[r][q];
          const float f = exp2_approx(ml.x - ref);
          const float4 y = s_part[r * per + k];
          x.x += y.x * f, x.y += y.y * f, x.z += y.z * f, x.w += y.w * f;
          sum += ml.y * f;
        }
      output(q, d, x, M, sum);
    }
  }
}

// Grid (queries of all heads): thread t adds dim t of its query over the splits, in order.  About 3 us behind the kernel
// before it, most of that one launch and two round trips to L2.  (A warp for each query: 1.0 to 1.8 us longer for one
// token to 28 queries a head, 0.9 shorter for 512.)
template <typename T, int HD>
__global__ void __launch_bounds__(HD) k_kv8_merge(const __grid_constant__ Kv8AttnArgs a) {
  __shared__ float2 s_f[kMaxSplits];
  __shared__ float red[HD / 32];
  const int nq = a.rows * a.group;
  const int i = blockIdx.x;
  const int h = i / nq, qi = i - h * nq, r = qi / a.group, head = h * a.group + qi - r * a.group;
  griddep_launch();
  griddep_wait();
  const float2* ml = a.part_ml + (size_t)i * a.n_split;
  const float* po = a.part_o + (size_t)i * a.n_split * HD + threadIdx.x;
  float first[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) first[s] = s < a.n_split ? po[(size_t)s * HD] : 0.f;
  float M = -INFINITY;
  for (int s = threadIdx.x; s < a.n_split; s += HD) {
    const float2 t = ml[s];
    s_f[s] = t;
    M = fmaxf(M, t.x);
  }
  M = warp_max(M);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < HD / 32; ++w) M = fmaxf(M, red[w]);
  const float ref = M == -INFINITY ? 0.f : M;
  float sum = 0.f, x = 0.f;
#pragma unroll
  for (int s = 0; s < 8; ++s)
    if (s < a.n_split) {
      const float2 t = s_f[s];
      const float f = exp2_approx(t.x - ref);
      sum += t.y * f;
      x += first[s] * f;
    }
#pragma unroll 8
  for (int s = 8; s < a.n_split; ++s) {
    const float2 t = s_f[s];
    const float f = exp2_approx(t.x - ref);
    sum += t.y * f;
    x += po[(size_t)s * HD] * f;
  }
  const float y = sum == 0.f ? 0.f : x / sum;
  T* out = reinterpret_cast<T*>(a.out) + (size_t)r * a.ld_out + (size_t)head * HD + threadIdx.x;
  if constexpr (sizeof(T) == 4)
    *out = y;
  else
    *out = Io<T>::from_f(y);
  if (threadIdx.x == 0 && a.lse) a.lse[a.lse_at(r, head)] = lse_of(M, sum);
}

// ---------------------------------------------------------------- accumulated weights

constexpr int kWWarps = 8;
constexpr int kWEights = 8;  // eights of queries staged at once

// Grid (CTAs, KV heads).  The CTA stages up to 64 chosen queries, then its warps walk over their sixteen-slot tiles:
// a tile's K is converted once, in registers, while the next tile's is on its way, and multiplied by every eight.
// More queries go round again (their K comes from L2); a slot's sum stays with one lane pair throughout.
template <typename T, int HD, int CODE, bool CAP>
__global__ void __launch_bounds__(kWWarps * 32, 2) k_kv8_weights(const __grid_constant__ Kv8AttnArgs a, int n_slots) {
  constexpr bool SPLIT = sizeof(T) == 4;
  constexpr int NJ = HD / 64, STEPS = HD / 16;
  constexpr int QW = HD / 16 * 64;
  extern __shared__ __align__(16) uint32_t smem[];
  uint32_t* s_hi = smem;
  uint32_t* s_lo = smem + kWEights * QW;
  __shared__ __align__(8) float s_coef[kWEights * 8], s_lse[kWEights * 8];
  __shared__ unsigned long long s_mask[kWEights * 8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int h = blockIdx.y;
  const int n_tiles = (n_slots + 15) >> 4, stride = gridDim.x * kWWarps;
  const int first = blockIdx.x * kWWarps + warp;
  const int nq = a.n_take * a.group;
  const float inv_cap = CAP ? 1.f / a.cap : 0.f;
  griddep_launch();
  griddep_wait();

  // Page of tile ti as the table has it (checked where it is used, a tile later), or -1 where no row sees the tile.
  auto page_of = [&](int ti) { return ti < n_tiles && visible_any(ti * 16, a) ? __ldg(a.c.btab + ti * 16 / kPage) : -1; };
  struct Tile {
    uint4 lo[NJ], hi[NJ];  // codes of rows g and g + 8
    float ks;
    bool live;
  };
  auto load = [&](Tile& t, int ti, int page) {
    t.live = a.c.page_ok(page);
    if (!t.live) return;
    const int in_page = ti * 16 % kPage;
    const size_t row0 = a.c.page_row(page, h) + (size_t)(in_page + g) * HD + c * 16;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      t.lo[j] = ld16(a.c.k + row0 + j * 64);
      t.hi[j] = ld16(a.c.k + row0 + 8 * HD + j * 64);
    }
    t.ks = __ldg(a.c.ks + a.c.scale_at(page, h, in_page));
  };

  for (int q0 = 0; q0 == 0 || q0 < nq; q0 += kWEights * 8) {
    const int eights = nq ? min(kWEights, (nq - q0 + 7) / 8) : 0;
    Tile cur;
    load(cur, first, page_of(first));
    int page = page_of(first + stride);
    if (q0) __syncthreads();
#pragma unroll 8
    for (int q = warp; q < eights * 8; q += kWWarps) {
      const int qi = q0 + q;
      const T* p = nullptr;
      float lse = 0.f;
      unsigned long long mask = 0ull;
      if (qi < nq) {
        const int ti = qi / a.group, r = a.take[ti], head = h * a.group + qi - ti * a.group;
        p = reinterpret_cast<const T*>(a.q) + (size_t)r * a.ld_q + (size_t)head * HD;
        lse = __ldg(a.lse + a.lse_at(r, head));
        mask = a.mask[r];
      }
      const float inv = stage_query<T, HD, SPLIT>(p, s_hi + (q >> 3) * QW, s_lo + (q >> 3) * QW, q & 7, lane);
      if (lane == 0) {
        s_coef[q] = qi < nq ? a.scale * inv * (CAP ? 1.f : kLog2e) : 0.f;
        // a padding query, and a row that saw nothing (lse -inf), adds exp2(-inf) = 0
        s_lse[q] = qi < nq && lse != -INFINITY ? lse * kLog2e : INFINITY;
        s_mask[q] = mask;
      }
    }
    __syncthreads();

    for (int ti = first; ti < n_tiles; ti += stride) {
      const int slot0 = ti * 16;
      float sum[2] = {0.f, 0.f};  // slots g and g + 8
      const bool live = cur.live;
      const float ks = cur.ks;
      uint32_t k[STEPS][4];
      if (live) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          codes_to_half<CODE>(word_of(cur.lo[i >> 2], i & 3), k[i][0], k[i][2]);
          codes_to_half<CODE>(word_of(cur.hi[i >> 2], i & 3), k[i][1], k[i][3]);
        }
      }
      load(cur, ti + stride, page);
      page = page_of(ti + 2 * stride);
      const int slot = slot0 + g + c * 8;  // of lanes c = 0 and 1
      const size_t at = (size_t)h * a.ld_w + slot;
      const bool mine = c < 2 && slot < n_slots;
      const float before = !mine ? 0.f : q0 ? a.w_out[at] : a.w_in ? a.w_in[at] : 0.f;
      // Scores of the tile and eight t, in the log2 domain and less the rows' log-sum-exp.
      auto weigh = [&](int t, float (&x)[4]) {
        float s0[4], s1[4];
#pragma unroll
        for (int p = 0; p < STEPS / 2; ++p) {
          const uint4 hi = *reinterpret_cast<const uint4*>(s_hi + t * QW + (p * 32 + lane) * 4);
          if (p == 0) {
            mma16816_first(s0, k[0], hi.x, hi.y);
            mma16816_first(s1, k[1], hi.z, hi.w);
          } else {
            mma16816(s0, k[2 * p], hi.x, hi.y);
            mma16816(s1, k[2 * p + 1], hi.z, hi.w);
          }
          if (SPLIT) {
            const uint4 lo = *reinterpret_cast<const uint4*>(s_lo + t * QW + (p * 32 + lane) * 4);
            mma16816(s0, k[2 * p], lo.x, lo.y);
            mma16816(s1, k[2 * p + 1], lo.z, lo.w);
          }
        }
        const float2 cf = *reinterpret_cast<const float2*>(s_coef + t * 8 + 2 * c);
        const float2 lse = *reinterpret_cast<const float2*>(s_lse + t * 8 + 2 * c);
        const float c0 = cf.x * ks, c1 = cf.y * ks;
        if (CAP) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = capped<SPLIT>((s0[e] + s1[e]) * (e & 1 ? c1 : c0), a.cap, inv_cap) - (e & 1 ? lse.y : lse.x);
        } else {
          x[0] = fmaf(s0[0] + s1[0], c0, -lse.x), x[1] = fmaf(s0[1] + s1[1], c1, -lse.y);
          x[2] = fmaf(s0[2] + s1[2], c0, -lse.x), x[3] = fmaf(s0[3] + s1[3], c1, -lse.y);
        }
      };
      if (live && slot0 + 16 <= a.prefix) {
#pragma unroll 4
        for (int t = 0; t < eights; ++t) {
          float x[4];
          weigh(t, x);
          sum[0] += exp2_approx(x[0]) + exp2_approx(x[1]);
          sum[1] += exp2_approx(x[2]) + exp2_approx(x[3]);
        }
      } else if (live) {
        for (int t = 0; t < eights; ++t) {
          float x[4];
          weigh(t, x);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (visible(slot0 + g + (e >> 1) * 8, a.prefix, a.base, s_mask[t * 8 + 2 * c + (e & 1)]))
              sum[e >> 1] += exp2_approx(x[e]);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
      }
      if (mine) a.w_out[at] = before + (c ? sum[1] : sum[0]);
    }
  }
}

template <typename T, int HD, int CODE, int QT>
bool run_attention(Kv8AttnArgs a, cudaStream_t st) {
  const Tiles<5> tiles(a.prefix, a.base, a.rows);
  a.split_tiles = (tiles.n + a.n_split - 1) / a.n_split;
  using L = AttnSmem<T, HD, QT>;
  const auto kern = k_kv8_attention<T, HD, CODE, QT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) != cudaSuccess) return false;
  const int nq = a.rows * a.group;
  return launch_kv8(kern, dim3(a.n_split, a.c.n_kv, (nq + L::QB - 1) / L::QB), L::W * 32, L::kBytes, st,
                    a.part_o ? 1 : a.n_split, a);
}

// Query eights of a CTA: all of a KV head's queries up to four eights.
int query_eights(int nq) { return nq <= 8 ? 1 : nq <= 16 ? 2 : nq <= 24 ? 3 : 4; }

template <typename T, int HD, int CODE>
bool run_attention_q(const Kv8AttnArgs& a, cudaStream_t st) {
  switch (query_eights(a.rows * a.group)) {
    case 1: return run_attention<T, HD, CODE, 1>(a, st);
    case 2: return run_attention<T, HD, CODE, 2>(a, st);
    case 3: return run_attention<T, HD, CODE, 3>(a, st);
  }
  return run_attention<T, HD, CODE, 4>(a, st);
}

template <typename T, int HD, int CODE>
bool run_weights(const Kv8AttnArgs& a, cudaStream_t st) {
  constexpr size_t smem = (size_t)kWEights * (HD / 16 * 64) * 4 * (sizeof(T) == 4 ? 2 : 1);
  const int n_slots = a.prefix > a.base + a.rows ? a.prefix : a.base + a.rows;
  const int groups = ((n_slots + 15) / 16 + kWWarps - 1) / kWWarps;  // CTAs with a tile for every warp
  int fit = 2 * 152 / a.c.n_kv;                                       // two CTAs on each of 152 SMs
  if (fit < 1) fit = 1;
  const dim3 grid(groups < fit ? groups : fit, a.c.n_kv);
  return launch_kv8(a.cap > 0.f ? k_kv8_weights<T, HD, CODE, true> : k_kv8_weights<T, HD, CODE, false>, grid, kWWarps * 32,
                    smem, st, 1, a, n_slots);
}

// Add up the splits of scratch.
template <typename T>
bool run_merge(const Kv8AttnArgs& a, cudaStream_t st) {
  return launch_kv8(a.c.hd == 128 ? k_kv8_merge<T, 128> : k_kv8_merge<T, 64>, a.c.n_kv * a.rows * a.group, a.c.hd, 0, st, 1,
                    a);
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

// The tcgen05 kernel runs where a KV head has more than 64 queries and the 32-query blocks times the slots of all heads
// reach kTcWork (us, this kernel and the other, on heads 64 over 8: 64 bf16 rows over 1564 slots, 200192 of these units,
// 27.5 and 26.2; 24 rows over 4024, 193152, 23.8 and 24.8; 64 rows over 16064 59.9 and 159; fp32 24 rows over 4024 36.8
// and 31.8, 64 over 4064 51.0 and 67.9).  Of 33 to 64 queries, which fill half a block at most, only 16-bit ones, and
// from kTcWorkHalf on (5 bf16 rows over 16005 slots, 256080 units, 30.8 and 28.9, and 0.95 and 1.1 us for every thousand
// slots more; fp32 48.3 and 37.0, 1.4 and 1.6).
constexpr long long kTcWork = 200000, kTcWorkHalf = 500000;

Kv8Splits kv8_attention_splits(int rows, int group, int n_kv, int slots, int io) {
  const int nq = rows * group;
  const long long work = (long long)n_kv * ((nq + 31) / 32) * slots;
  const bool tc = nq > 64 ? work >= kTcWork : nq > 32 && io != 2 && work >= kTcWorkHalf;
  const int qb = tc ? (io == 2 ? 128 : 256) : 8 * query_eights(nq);
  const int blocks = n_kv * ((nq + qb - 1) / qb);
  const int slots_a_tile = tc ? 128 : kTileSlots;
  const int tiles = (slots + slots_a_tile - 1) / slots_a_tile;
  const int fit = kMaxSplits / blocks;                     // one CTA on each of 152 SMs
  const int warps = tc ? 1 : qb == 8 ? 12 : 8;
  const int most = (tiles + warps - 1) / warps;            // a tile for every warp (for the CTA)
  int n = fit < most ? fit : most;
  if (n <= 1) return {1, false, tc};
  const int per = (tiles + n - 1) / n;
  n = (tiles + per - 1) / per;                             // no split without a tile
  // A GPC's sixteen to twenty SMs hold few whole clusters: past these counts the launch runs in two waves (72 queries a
  // head over 4000 slots: 34.2 us as 144 CTAs in clusters of six, 18.7 merged through scratch; 192 queries: 49.3 us as 144
  // CTAs in clusters of three).
  const bool cluster = !tc && cluster_fits(qb, io == 2) && n <= kMaxCluster && n * blocks <= (n <= 4 ? 128 : 76);
  return {n, !cluster, tc};
}

bool launch_kv8_attention(const Kv8AttnArgs& a, int io, bool tc, cudaStream_t st) {
  if (tc) {
    if (!launch_kv8_attention_tc(a, io, st)) return false;
  } else if (!(io == 0 ? attention_of<__nv_bfloat16>(a, st) : io == 1 ? attention_of<__half>(a, st) : attention_of<float>(a, st))) {
    return false;
  }
  if (!a.part_o) return true;
  return io == 0 ? run_merge<__nv_bfloat16>(a, st) : io == 1 ? run_merge<__half>(a, st) : run_merge<float>(a, st);
}

bool launch_kv8_weights(const Kv8AttnArgs& a, int io, cudaStream_t st) {
  return io == 0 ? weights_of<__nv_bfloat16>(a, st) : io == 1 ? weights_of<__half>(a, st) : weights_of<float>(a, st);
}

}  // namespace ssd
