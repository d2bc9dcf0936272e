// Writing, reading and thinning out the 8-bit KV cache.
//
// k_kv8_append  quantises new K/V rows: one CTA for each block of T tokens
//               and KV head, which holds the block's values of both tensors
//               in registers between the search for the largest magnitude
//               and the encoding, so the rows are read once and the codes
//               written once.
// k_kv8_read    the values of consecutive slots.
// k_kv8_select  the slots of one KV head that stay: a radix select over the
//               accumulated weights, by one cluster of CTAs for each head.
// k_kv8_gather  the kept slots, requantised into the blocks of other pages.
#include <cooperative_groups.h>

#include "kv8.h"

namespace ssd {

namespace {

constexpr int kQuantThreads = 512;

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = reinterpret_cast<const float4*>(p)[i];
      x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = f.z, x[4 * i + 3] = f.w;
    }
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    Io<T>::unpack8(a, x);
    Io<T>::unpack8(b, x + 8);
  }
}

template <int CODE>
__device__ __forceinline__ void decode16(const uint4& u, float s, float (&x)[16]) {
  decode4<CODE>(u.x, s, x);
  decode4<CODE>(u.y, s, x + 4);
  decode4<CODE>(u.z, s, x + 8);
  decode4<CODE>(u.w, s, x + 12);
}

template <int CODE, bool ODD>
__device__ __forceinline__ uint4 encode16(const float (&x)[16], float m) {
  return make_uint4(encode4<CODE, ODD>(x, m), encode4<CODE, ODD>(x + 4, m), encode4<CODE, ODD>(x + 8, m),
                    encode4<CODE, ODD>(x + 12, m));
}
// Values that may hold a NaN or an infinity: out of line, so that the usual path is not computed beside it.
template <int CODE>
__device__ __noinline__ uint4 encode16_odd(float x0, float x1, float x2, float x3, float x4, float x5, float x6, float x7,
                                           float x8, float x9, float x10, float x11, float x12, float x13, float x14, float x15,
                                           float m) {
  const float x[16] = {x0, x1, x2, x3, x4, x5, x6, x7, x8, x9, x10, x11, x12, x13, x14, x15};
  return encode16<CODE, true>(x, m);
}
template <int CODE>
__device__ __forceinline__ void store_codes(uint8_t* to, const float (&x)[16], float m, bool odd) {
  if (odd)
    *reinterpret_cast<uint4*>(to) = encode16_odd<CODE>(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], x[8], x[9], x[10],
                                                       x[11], x[12], x[13], x[14], x[15], m);
  else
    *reinterpret_cast<uint4*>(to) = encode16<CODE, false>(x, m);
}

// The larger of a and the magnitudes of x (NaN compares as absent), and a number that is NaN if x holds a NaN or an
// infinity.
__device__ __forceinline__ void amax16(const float (&x)[16], float& a, float& odd) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a = fmaxf(a, fabsf(x[i]));
    odd = fmaf(x[i], 0.f, odd);
  }
}
// The same over finite magnitudes only.
__device__ __forceinline__ float finite_amax16(const float (&x)[16], float a) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float v = fabsf(x[i]);
    if (v > a && v < INFINITY) a = v;
  }
  return a;
}

// The largest of two non-negative magnitudes over the CTA; true if odd is NaN in any thread.
__device__ __forceinline__ bool block_max2(float& a, float& b, float odd, uint32_t (&red)[3][32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  // (magnitudes order like their bits)
  const uint32_t x = __reduce_max_sync(0xffffffffu, __float_as_uint(a));
  const uint32_t y = __reduce_max_sync(0xffffffffu, __float_as_uint(b));
  const bool o = __any_sync(0xffffffffu, odd != odd);
  if (lane == 0) red[0][warp] = x, red[1][warp] = y, red[2][warp] = o;
  __syncthreads();
  a = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < warps ? red[0][lane] : 0u));
  b = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < warps ? red[1][lane] : 0u));
  return __any_sync(0xffffffffu, lane < warps && red[2][lane]);
}

// Grid (blocks of T tokens, KV heads).  A block holds T * hd / 16 chunks of sixteen values (64..512) of K and of V, one
// of each for every thread.  scale = amax / qmax over the block's finite values, code = rne(x / scale) by one product
// with the rounded inverse.  Bound by HBM: 16384 bf16 rows of 8 heads of 128 into int8, 100 MB, take 19.1 us (5.3 TB/s
// of a copy's 6.8); one row takes 3.4 us, a launch and two round trips to memory.  K and V share a CTA, which halves
// its barriers.
template <typename T, int CODE>
__global__ void __launch_bounds__(kQuantThreads, 2) k_kv8_append(Kv8View c, Kv8RowsArgs a) {
  __shared__ uint32_t red[3][32];
  const int h = blockIdx.y;
  const int rshift = c.hd == 128 ? 3 : 2;  // 2^rshift chunks a row
  griddep_launch();
  griddep_wait();
  const int slot0 = ((a.first >> c.tshift) + blockIdx.x) << c.tshift;
  const int page = c.btab[slot0 / kPage];
  const int t = threadIdx.x >> rshift, row = slot0 + t - a.first;
  const bool fresh = row >= 0 && row < a.rows;
  float x[2][16];
  float amax[2] = {0.f, 0.f}, odd = 0.f;  // of the new rows
  if (fresh) {
    const size_t at = (size_t)h * c.hd + (threadIdx.x - (t << rshift)) * 16;
    load16(reinterpret_cast<const T*>(a.k) + (size_t)row * a.ld_k + at, x[0]);
    load16(reinterpret_cast<const T*>(a.v) + (size_t)row * a.ld_v + at, x[1]);
    amax16(x[0], amax[0], odd);
    amax16(x[1], amax[1], odd);
  }
  if (!c.page_ok(page)) return;
  const size_t at = c.page_row(page, h) + (size_t)(slot0 % kPage) * c.hd + threadIdx.x * 16;
  const size_t sc = c.scale_at(page, h, slot0 % kPage);
  float least[2] = {0.f, 0.f};
  if (slot0 < a.first) {  // slots before the new rows stay, under a scale no smaller than theirs
    least[0] = c.ks[sc];
    least[1] = c.vs[sc];
#pragma unroll
    for (int w = 0; w < 2; ++w)
      if (!(least[w] < INFINITY)) least[w] = 0.f;  // what stands in a block that was never written
    if (row < 0) {
      float unused = 0.f;
      decode16<CODE>(*reinterpret_cast<const uint4*>(c.k + at), least[0], x[0]);
      decode16<CODE>(*reinterpret_cast<const uint4*>(c.v + at), least[1], x[1]);
      amax16(x[0], unused, odd);
      amax16(x[1], unused, odd);
    }
  }
  // (the barrier also orders every read of kept codes and scales before the writes)
  const bool any_odd = block_max2(amax[0], amax[1], odd, red);
  if (any_odd) {
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 2; ++w) amax[w] = fresh ? finite_amax16(x[w], 0.f) : 0.f;
    block_max2(amax[0], amax[1], 0.f, red);
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const float s = fmaxf(block_scale<CODE>(amax[w]), least[w]);
    if (row < a.rows) store_codes<CODE>((w ? c.v : c.k) + at, x[w], inverse_scale(s), any_odd);
    if (threadIdx.x == 0) (w ? c.vs : c.ks)[sc] = s;
  }
}

// Grid (runs of `run` slots, a divisor of sixteen, so that they share a scale; K / V; parts of a row).  A thread makes
// sixteen bytes of output (4 fp32 or 8 16-bit values) at a time, for the same columns of every row of its run, so that
// the scale and the address are found once.  Bound by HBM, four fifths of it writes: 16384 slots of 8 heads of 128 take
// 19.8 us in bf16 (100 MB, 5.1 TB/s) and 29.3 in fp32 (168 MB, 5.7 TB/s).  Eight rows under way a thread were slower
// (34.8 us in fp32).
template <typename T, int CODE>
__global__ void __launch_bounds__(256) k_kv8_read(Kv8View c, Kv8RowsArgs a, int run) {
  constexpr int N = 16 / sizeof(T);
  const int per_row = c.hd / N, per_slot = per_row * c.n_kv;
  const int which = blockIdx.y;
  const int slot0 = (a.first / run + blockIdx.x) * run;
  griddep_launch();
  griddep_wait();
  const int page = c.btab[slot0 / kPage];
  const bool ok = c.page_ok(page);
  const int r0 = max(0, a.first - slot0), r1 = min(run, a.first + a.rows - slot0);
  const uint8_t* from = (which ? c.v : c.k) + (ok ? c.page_row(page, 0) : 0) + (size_t)(slot0 % kPage) * c.hd;
  const float* scales = (which ? c.vs : c.ks) + (ok ? c.scale_at(page, 0, slot0 % kPage) : 0);
  T* to = reinterpret_cast<T*>(which ? a.v : a.k) + ((ptrdiff_t)slot0 - a.first) * (ptrdiff_t)(which ? a.ld_v : a.ld_k);
  const size_t ld = which ? a.ld_v : a.ld_k;
  const int i = blockIdx.z * blockDim.x + threadIdx.x;
  if (i < per_slot) {
    const int h = i / per_row, d = (i - h * per_row) * N;
    const uint8_t* p = from + (size_t)h * kPage * c.hd + d;
    const float s = ok ? scales[(size_t)h << (6 - c.tshift)] : 0.f;
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
      float x[N];
#pragma unroll
      for (int e = 0; e < N; e += 4)
        decode4<CODE>(ok ? __ldg(reinterpret_cast<const uint32_t*>(p + r * c.hd + e)) : 0u, s, x + e);
      T* o = to + (size_t)r * ld + (size_t)i * N;
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(o) = make_float4(x[0], x[1], x[2], x[3]);
      } else {
        __align__(16) T t[N];
#pragma unroll
        for (int e = 0; e < N; ++e) t[e] = Io<T>::from_f(x[e]);
        *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(t);
      }
    }
  }
}

// ---------------------------------------------------------------- eviction

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelCluster = 8;
constexpr int kSelKeys = 8;      // keys that a thread holds in registers
constexpr int kDigitBits = 11;   // 32 bits in rounds of 11, 11 and 10
constexpr int kBins = 1 << kDigitBits;
constexpr int kCoarse = kBins / kSelWarps;  // 64

// A key that orders weights as unsigned integers: larger weight, larger key; -0 and +0 alike; NaN below all.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b >> 31) ? ~b : b | 0x80000000u;
}

// Sum of v over the lanes up to this one.
__device__ __forceinline__ int warp_prefix(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if ((int)(threadIdx.x & 31) >= o) v += t;
  }
  return v;
}

// Each warp's sum v (the same in its lanes): the sum over the warps before this one, and over all.
__device__ __forceinline__ int warps_before(int v, int* sums, int& total) {
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) sums[warp] = v;
  __syncthreads();
  const int s = warp_prefix(sums[threadIdx.x & 31]);  // (32 warps)
  total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, (warp + 31) & 31);
  __syncthreads();
  return warp ? before : 0;
}

// Grid (cluster CTAs, heads).  The keep - recent heaviest of slots [0, n - recent), the lowest slots among equal ones,
// in slot order, then the recent ones.  A radix select: three rounds of a shared-memory histogram of the next digit
// over the keys that still agree with the threshold, added up over the cluster.  Of the other CTAs' histograms only the
// sums of 64 bins each and then the 64 bins of one sum are read (all of them: 64 KB a CTA and round, 2.5 us).  A thread
// holds its keys in registers (RELOAD: more than fit are read again each round).  Bound by latency: 2.1 MB of weights
// (65531 slots of 8 heads) take 12 us, four cluster barriers and a dozen of the CTA's; clusters of sixteen were no
// faster.
template <bool RELOAD>
__global__ void __launch_bounds__(kSelThreads) k_kv8_select(Kv8SelectArgs a) {
  namespace cg = cooperative_groups;
  __shared__ int hist[2][kBins];
  __shared__ int coarse[2][kSelWarps];          // sums of kCoarse bins
  __shared__ int sums[kSelWarps];
  __shared__ int s_bin, s_above, s_part, s_part_above;
  __shared__ int2 s_count[kSelCluster];         // each rank's candidates above / equal to the threshold
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), nr = cl.num_blocks();
  const int h = blockIdx.y, tid = threadIdx.x;
  griddep_launch();
  griddep_wait();
  const float* w = a.weight + (size_t)h * a.ld_weight;
  const int cand = a.n - a.recent, want = a.keep - a.recent;
  int* index = a.index + (size_t)h * a.keep;
  float* kept = a.kept_weight ? a.kept_weight + (size_t)h * a.keep : nullptr;
  for (int i = rank * kSelThreads + tid; i < a.recent; i += nr * kSelThreads) {
    index[want + i] = cand + i;
    if (kept) kept[want + i] = w[cand + i];
  }
  if (want == 0) return;  // the same in every CTA of the cluster
  // CTA r holds candidates [r span, (r + 1) span), in runs; a warp has 32 kSelKeys consecutive ones of a run, a lane
  // every 32nd of them
  constexpr int RUN = kSelThreads * kSelKeys;
  const int span = (cand + nr - 1) / nr;
  const int i0 = min(cand, rank * span), i1 = min(cand, i0 + span);
  const int mine = i0 + (tid >> 5) * 32 * kSelKeys + (tid & 31);
  uint32_t key[kSelKeys];  // made once, since the rounds' arithmetic over eight keys a thread is what bounds the kernel
  uint32_t valid = 0;      // bit e: key e is a candidate's
  auto load = [&](int run) {
    float x[kSelKeys];
    valid = 0;
#pragma unroll
    for (int e = 0; e < kSelKeys; ++e) {
      const bool v = mine + run + e * 32 < i1;
      x[e] = v ? __ldg(w + mine + run + e * 32) : 0.f;
      valid |= (uint32_t)v << e;
    }
#pragma unroll
    for (int e = 0; e < kSelKeys; ++e) key[e] = weight_key(x[e]);
  };
  const int n_run = RELOAD ? (i1 - i0 + RUN - 1) / RUN * RUN : RUN;
  if (!RELOAD) load(0);
  uint32_t prefix = 0;  // the threshold's leading bits found so far
  int need = want;      // candidates still to take among those that share them
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int bits = round == 2 ? 10 : kDigitBits, shift = round == 0 ? 21 : round == 1 ? 10 : 0;
    int* hs = hist[round & 1];
    for (int b = tid; b < kBins; b += kSelThreads) hs[b] = 0;
    __syncthreads();
    for (int run = 0; run < n_run; run += RUN) {
      if (RELOAD) load(run);
      const uint32_t digit = (1u << bits) - 1;
#pragma unroll
      for (int e = 0; e < kSelKeys; ++e)
        if ((valid >> e & 1u) && (round == 0 || (key[e] >> (shift + bits)) == prefix)) atomicAdd(&hs[(key[e] >> shift) & digit], 1);
    }
    __syncthreads();
    {
      const int2 t = *reinterpret_cast<const int2*>(hs + 2 * tid);  // warp w's lanes hold coarse bin w
      const int c = __reduce_add_sync(0xffffffffu, t.x + t.y);
      if ((tid & 31) == 0) coarse[round & 1][tid >> 5] = c;
    }
    cl.sync();
    if (tid < 32) {  // the coarse bin, from the top one down, where the count reaches need
      int v = 0;
#pragma unroll
      for (int r = 0; r < kSelCluster; ++r)
        if (r < nr) v += cl.map_shared_rank(coarse[round & 1], r)[31 - tid];
      const int above = warp_prefix(v) - v;
      if (above < need && above + v >= need) {
        s_part = 31 - tid;
        s_part_above = above;
      }
      __syncwarp();
      // and the bin among its 64, two a lane
      const int top = s_part * kCoarse + kCoarse - 2 - 2 * tid;
      int2 u = make_int2(0, 0);
#pragma unroll
      for (int r = 0; r < kSelCluster; ++r)
        if (r < nr) {
          const int2 t = *reinterpret_cast<const int2*>(cl.map_shared_rank(hs, r) + top);
          u.x += t.x;
          u.y += t.y;
        }
      int at = s_part_above + warp_prefix(u.x + u.y) - u.x - u.y;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = e ? u.x : u.y;
        if (at < need && at + n >= need) {
          s_bin = top + 1 - e;
          s_above = at;
        }
        at += n;
      }
    }
    __syncthreads();
    prefix = (prefix << bits) | (uint32_t)s_bin;
    need -= s_above;
    // (hist[round & 1] is cleared again two rounds on: after every CTA has passed the next round's cluster barrier)
  }
  // prefix is the threshold's key; candidates above it are taken, and the first `need` equal ones.
  int gt = 0, eq = 0;  // of this warp
  auto count = [&]() {
    gt = eq = 0;
#pragma unroll
    for (int e = 0; e < kSelKeys; ++e) {
      gt += __popc(__ballot_sync(0xffffffffu, (valid >> e & 1u) && key[e] > prefix));
      eq += __popc(__ballot_sync(0xffffffffu, (valid >> e & 1u) && key[e] == prefix));
    }
  };
  int cta_gt = 0, cta_eq = 0;
  for (int run = 0; run < n_run; run += RUN) {
    if (RELOAD) load(run);
    count();
    int tg, te;
    warps_before(gt, sums, tg);
    warps_before(eq, sums, te);
    cta_gt += tg;
    cta_eq += te;
  }
  if (tid < nr) cl.map_shared_rank(s_count, tid)[rank] = make_int2(cta_gt, cta_eq);
  cl.sync();  // (no CTA's shared memory is read by another after this)
  int base_gt = 0, base_eq = 0;  // in the CTAs before this one
#pragma unroll
  for (int r = 0; r < kSelCluster; ++r)
    if (r < rank) {
      base_gt += s_count[r].x;
      base_eq += s_count[r].y;
    }
  for (int run = 0; run < n_run; run += RUN) {
    if (RELOAD) {
      load(run);
      count();
    }
    int tg, te;
    int ng = base_gt + warps_before(gt, sums, tg), ne = base_eq + warps_before(eq, sums, te);
    const unsigned below = (1u << (tid & 31)) - 1;
#pragma unroll
    for (int e = 0; e < kSelKeys; ++e) {
      const bool g = (valid >> e & 1u) && key[e] > prefix, q = (valid >> e & 1u) && key[e] == prefix;
      const unsigned bg = __ballot_sync(0xffffffffu, g), bq = __ballot_sync(0xffffffffu, q);
      const int eq_before = ne + __popc(bq & below);
      if (g || (q && eq_before < need)) {
        const int pos = ng + __popc(bg & below) + min(eq_before, need);
        index[pos] = mine + run + e * 32;
        if (kept) kept[pos] = __ldg(w + mine + run + e * 32);  // (as it stands there, NaN and -0 among them)
      }
      ng += __popc(bg);
      ne += __popc(bq);
    }
    base_gt += tg;
    base_eq += te;
  }
}

// The largest magnitude of sixteen codes under scale s, which is one product, since rounding keeps the codes' order.
// NaN or infinite where a value is.
template <int CODE>
__device__ __forceinline__ float codes_amax(const uint4& u, float s) {
  uint32_t h[8];
  codes_to_half<CODE>(u.x, h[0], h[1]);
  codes_to_half<CODE>(u.y, h[2], h[3]);
  codes_to_half<CODE>(u.z, h[4], h[5]);
  codes_to_half<CODE>(u.w, h[6], h[7]);
  __half2 m = __habs2(*reinterpret_cast<const __half2*>(&h[0]));
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __half2*>(&h[i])));
  return __fmul_rn(__half2float(__hmax_nan(__low2half(m), __high2half(m))), fabsf(s));
}

// Grid (CTAs, heads): a CTA takes every gridDim.x-th block of the kept slots.  A row's index, page and codes are three
// round trips to memory, so they are asked for three, two and one blocks ahead; a thread keeps its two chunks as codes
// over the reduction.  Bound by instructions (fourteen a value at 0.75 a clock and scheduler), not by HBM: 16381 slots of
// 8 heads of 128, 67 MB, take 19.6 us (3.4 TB/s; 22.6 with one block a CTA and no prefetch).
template <int FROM, int TO>
__global__ void __launch_bounds__(kQuantThreads, 2) k_kv8_gather(Kv8View src, Kv8View dst, const int* index, int keep) {
  __shared__ uint32_t red[2][3][32];
  const int h = blockIdx.y;
  const int rshift = dst.hd == 128 ? 3 : 2;
  const int t = threadIdx.x >> rshift, step = gridDim.x << dst.tshift;
  const int chunk = (threadIdx.x - (t << rshift)) * 16;
  struct Codes {
    uint4 u[2];
    float s[2];
  };
  griddep_launch();
  griddep_wait();
  index += (size_t)h * keep;
  auto index_of = [&](int slot0) { return slot0 + t < keep ? __ldg(index + slot0 + t) : -1; };
  auto page_of = [&](int slot) { return slot >= 0 ? __ldg(src.btab + slot / kPage) : -1; };
  auto codes_of = [&](int slot, int page) {
    Codes c = {{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)}, {0.f, 0.f}};
    if (src.page_ok(page)) {  // (a slot that is not one has page -1)
      const size_t at = src.page_row(page, h) + (size_t)(slot % kPage) * src.hd + chunk;
      const size_t sc = src.scale_at(page, h, slot % kPage);
      c.u[0] = __ldg(reinterpret_cast<const uint4*>(src.k + at));
      c.u[1] = __ldg(reinterpret_cast<const uint4*>(src.v + at));
      c.s[0] = __ldg(src.ks + sc);
      c.s[1] = __ldg(src.vs + sc);
    }
    return c;
  };
  auto target = [&](int slot0) { return slot0 < keep ? dst.btab[slot0 / kPage] : -1; };
  const int first = blockIdx.x << dst.tshift;
  const int slot = index_of(first);
  int to = target(first);
  Codes now = codes_of(slot, page_of(slot));
  int s2 = index_of(first + step), s3 = index_of(first + 2 * step), p2 = page_of(s2);
  int round = 0;
  for (int slot0 = first; slot0 < keep; slot0 += step, round ^= 1) {
    const Codes next = codes_of(s2, p2);
    s2 = s3;
    p2 = page_of(s2);
    s3 = index_of(slot0 + 3 * step);
    const int page = to;
    to = target(slot0 + step);
    const bool used = slot0 + t < keep;
    float amax[2], odd = 0.f;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      amax[w] = codes_amax<FROM>(now.u[w], now.s[w]);
      if (!(amax[w] < INFINITY)) amax[w] = 0.f, odd = NAN;
    }
    const bool any_odd = block_max2(amax[0], amax[1], odd, red[round]);
    if (any_odd) {
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float x[16];
        decode16<FROM>(now.u[w], now.s[w], x);
        amax[w] = used ? finite_amax16(x, 0.f) : 0.f;
      }
      block_max2(amax[0], amax[1], 0.f, red[round]);
    }
    if (dst.page_ok(page)) {
      const size_t at = dst.page_row(page, h) + (size_t)(slot0 % kPage) * dst.hd + threadIdx.x * 16;
      const size_t sc = dst.scale_at(page, h, slot0 % kPage);
      // (the even lanes find K's scale, the odd ones V's)
      const float mine = block_scale<TO>(threadIdx.x & 1 ? amax[1] : amax[0]), inv = inverse_scale(mine);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const float m = __shfl_sync(0xffffffffu, inv, w);
        if (used) {
          float x[16];
          decode16<FROM>(now.u[w], now.s[w], x);
          store_codes<TO>((w ? dst.v : dst.k) + at, x, m, any_odd);
        }
      }
      if (threadIdx.x < 2) (threadIdx.x ? dst.vs : dst.ks)[sc] = mine;
    }
    now = next;
  }
}

}  // namespace

bool launch_kv8_append(const Kv8View& c, const Kv8RowsArgs& a, int io, cudaStream_t st) {
  const int t0 = a.first >> c.tshift, t1 = (a.first + a.rows - 1) >> c.tshift;
  const dim3 grid(t1 - t0 + 1, c.n_kv);
  const int threads = (c.hd / 16) << c.tshift;
  const auto kern = c.code == KV8_INT8 ? (io == 0   ? k_kv8_append<__nv_bfloat16, KV8_INT8>
                                          : io == 1 ? k_kv8_append<__half, KV8_INT8>
                                                    : k_kv8_append<float, KV8_INT8>)
                                       : (io == 0   ? k_kv8_append<__nv_bfloat16, KV8_E4M3>
                                          : io == 1 ? k_kv8_append<__half, KV8_E4M3>
                                                    : k_kv8_append<float, KV8_E4M3>);
  return launch_kv8(kern, grid, threads, 0, st, 1, c, a);
}

bool launch_kv8_read(const Kv8View& c, const Kv8RowsArgs& a, int io, cudaStream_t st) {
  const int per_slot = c.n_kv * c.hd / (io == 2 ? 4 : 8);
  const int threads = per_slot < 256 ? (per_slot + 31) / 32 * 32 : 256;
  const int parts = (per_slot + threads - 1) / threads;
  int run = 16;  // shorter runs where sixteen would leave an SM without eight CTAs
  while (run > 1 && (long long)a.rows / run * 2 * parts < 8 * 152) run /= 2;
  const dim3 grid((a.first + a.rows - 1) / run - a.first / run + 1, 2, parts);
  const auto kern = c.code == KV8_INT8 ? (io == 0   ? k_kv8_read<__nv_bfloat16, KV8_INT8>
                                          : io == 1 ? k_kv8_read<__half, KV8_INT8>
                                                    : k_kv8_read<float, KV8_INT8>)
                                       : (io == 0   ? k_kv8_read<__nv_bfloat16, KV8_E4M3>
                                          : io == 1 ? k_kv8_read<__half, KV8_E4M3>
                                                    : k_kv8_read<float, KV8_E4M3>);
  return launch_kv8(kern, grid, threads, 0, st, 1, c, a, run);
}

bool launch_kv8_evict(const Kv8View& src, const Kv8View& dst, const Kv8SelectArgs& a, cudaStream_t st) {
  const int cand = a.n - a.recent;
  int nr = 1;  // CTAs of a head: enough that a thread has few keys, eight at most
  while (nr < kSelCluster && cand > nr * kSelThreads * 4) nr *= 2;
  const bool reload = cand > nr * kSelThreads * kSelKeys;
  if (!launch_kv8(reload ? k_kv8_select<true> : k_kv8_select<false>, dim3(nr, src.n_kv), kSelThreads, 0, st, nr, a))
    return false;
  const auto gather = src.code == KV8_INT8
                          ? (dst.code == KV8_INT8 ? k_kv8_gather<KV8_INT8, KV8_INT8> : k_kv8_gather<KV8_INT8, KV8_E4M3>)
                          : (dst.code == KV8_INT8 ? k_kv8_gather<KV8_E4M3, KV8_INT8> : k_kv8_gather<KV8_E4M3, KV8_E4M3>);
  const int threads = (dst.hd / 16) << dst.tshift, blocks = ((a.keep - 1) >> dst.tshift) + 1;
  const int fit = (152 * 2 * kQuantThreads / threads + src.n_kv - 1) / src.n_kv;  // CTAs of a head that run at once
  const int per = (blocks + fit - 1) / fit;
  return launch_kv8(gather, dim3((blocks + per - 1) / per, src.n_kv), threads, 0, st, 1, src, dst, (const int*)a.index, a.keep);
}

}  // namespace ssd
