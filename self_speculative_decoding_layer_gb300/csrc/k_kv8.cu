// Writing, reading and thinning out the 8-bit KV cache.
//
// k_kv8_append  quantises new K/V rows: one CTA for each block of T tokens,
//               KV head and tensor, which holds the block's values in
//               registers between the search for the largest magnitude and
//               the encoding, so the rows are read once and the codes written
//               once.
// k_kv8_read    the values of consecutive slots.
// k_kv8_select  the slots of one KV head that stay: a radix select over the
//               accumulated weights, eight bits a round, by one cluster of
//               CTAs for each head.
// k_kv8_gather  the kept slots, requantised into the blocks of other pages.
#include <cooperative_groups.h>

#include "kv8.h"

namespace ssd {

namespace {

constexpr int kQuantThreads = 256;

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

template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&x)[16]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
    __align__(16) T t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = Io<T>::from_f(x[i]);
    reinterpret_cast<uint4*>(p)[0] = reinterpret_cast<const uint4*>(t)[0];
    reinterpret_cast<uint4*>(p)[1] = reinterpret_cast<const uint4*>(t)[1];
  }
}

__device__ __forceinline__ void decode16(const uint4& u, float s, int code, float (&x)[16]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(code_value((uint8_t)(w[i >> 2] >> ((i & 3) * 8)), code), s);
}

__device__ __forceinline__ uint4 encode16(const float (&x)[16], float m, int code) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[j] |= (uint32_t)encode(x[4 * j + i], m, code) << (8 * i);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest finite magnitude (NaN compares false, infinities are left out).
__device__ __forceinline__ float amax16(const float (&x)[16], float a) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float v = fabsf(x[i]);
    if (v > a && v < INFINITY) a = v;
  }
  return a;
}

__device__ __forceinline__ float block_max(float a, float* red) {
  a = warp_max(a);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  a = red[0];
  for (int w = 1; w < (int)(blockDim.x >> 5); ++w) a = fmaxf(a, red[w]);
  return a;
}

// A block holds T * hd / 16 sixteen-value chunks (64..512); a thread takes chunk threadIdx.x and, in the
// largest block, chunk threadIdx.x + 256.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads) k_kv8_append(Kv8View c, Kv8RowsArgs a) {
  __shared__ float red[kQuantThreads / 32];
  const int h = blockIdx.y, which = blockIdx.z;
  const int tokens = 1 << c.tshift, per_row = c.hd / 16;
  const int block = (a.first >> c.tshift) + blockIdx.x;
  const int slot0 = block << c.tshift;
  const int page = c.btab[slot0 / kPage];
  if (!c.page_ok(page)) return;
  uint8_t* codes = (which ? c.v : c.k) + c.page_row(page, h) + (size_t)(slot0 % kPage) * c.hd;
  float* scale = (which ? c.vs : c.ks) + c.scale_at(page, h, slot0 % kPage);
  const T* src = reinterpret_cast<const T*>(which ? a.v : a.k) + (size_t)h * c.hd;
  const size_t ld = which ? a.ld_v : a.ld_k;
  const bool keeps = slot0 < a.first;  // slots before the new rows stay, under a scale no smaller than theirs
  const float s_old = keeps ? *scale : 0.f;
  float x[2][16];
  bool mine[2];
  float amax = 0.f;  // of the new rows
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = threadIdx.x + j * kQuantThreads;
    const int t = i / per_row, d = (i - t * per_row) * 16;
    const int row = slot0 + t - a.first;
    mine[j] = t < tokens && row < a.rows;
    if (!mine[j]) continue;
    if (row >= 0) {
      load16(src + (size_t)row * ld + d, x[j]);
      amax = amax16(x[j], amax);
    } else {
      decode16(*reinterpret_cast<const uint4*>(codes + (size_t)t * c.hd + d), s_old, c.code, x[j]);
    }
  }
  amax = block_max(amax, red);  // (also orders every read of the kept codes and scale before the writes)
  const float s = fmaxf(block_scale(amax, c.code), s_old);
  const float m = inverse_scale(s);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (!mine[j]) continue;
    const int i = threadIdx.x + j * kQuantThreads;
    const int t = i / per_row, d = (i - t * per_row) * 16;
    *reinterpret_cast<uint4*>(codes + (size_t)t * c.hd + d) = encode16(x[j], m, c.code);
  }
  if (threadIdx.x == 0) *scale = s;
}

template <typename T>
__global__ void __launch_bounds__(256) k_kv8_read(Kv8View c, Kv8RowsArgs a) {
  const int per_row = c.hd / 16, per_slot = per_row * c.n_kv;
  const int which = blockIdx.y;
  const long long n = (long long)a.rows * per_slot;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    const int row = (int)(i / per_slot), rest = (int)(i - (long long)row * per_slot);
    const int h = rest / per_row, d = (rest - h * per_row) * 16;
    const int slot = a.first + row, page = c.btab[slot / kPage];
    float x[16];
    if (c.page_ok(page)) {
      const uint8_t* codes = (which ? c.v : c.k) + c.page_row(page, h) + (size_t)(slot % kPage) * c.hd + d;
      const float s = (which ? c.vs : c.ks)[c.scale_at(page, h, slot % kPage)];
      decode16(__ldg(reinterpret_cast<const uint4*>(codes)), s, c.code, x);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.f;
    }
    store16(reinterpret_cast<T*>(which ? a.v : a.k) + (size_t)row * (which ? a.ld_v : a.ld_k) + h * c.hd + d, x);
  }
}

// ---------------------------------------------------------------- eviction

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;

// A key that orders weights as unsigned integers: larger weight, larger key; -0 and +0 alike; NaN below all.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b >> 31) ? ~b : b | 0x80000000u;
}

// Grid (cluster CTAs, heads).  The keep - recent heaviest of slots [0, n - recent), the lowest slots among
// equal ones, in slot order, then the recent ones.
__global__ void __launch_bounds__(kSelThreads) k_kv8_select(Kv8SelectArgs a) {
  namespace cg = cooperative_groups;
  __shared__ int hist[2][256];
  __shared__ int total[256];
  __shared__ int s_bin, s_above;
  __shared__ int s_count[2];           // this CTA's candidates above / equal to the threshold
  __shared__ int w_gt[kSelWarps], w_eq[kSelWarps];
  cg::cluster_group cl = cg::this_cluster();
  const int rank = cl.block_rank(), nr = cl.num_blocks();
  const int h = blockIdx.y;
  griddep_launch();
  const float* w = a.weight + (size_t)h * a.ld_weight;
  const int cand = a.n - a.recent, want = a.keep - a.recent;
  const int per = (cand + nr - 1) / nr;
  const int i0 = min(cand, rank * per), i1 = min(cand, i0 + per);
  int* index = a.index + (size_t)h * a.keep;
  float* kept = a.kept_weight ? a.kept_weight + (size_t)h * a.keep : nullptr;
  for (int i = rank * kSelThreads + threadIdx.x; i < a.recent; i += nr * kSelThreads) {
    index[want + i] = cand + i;
    if (kept) kept[want + i] = w[cand + i];
  }
  if (want == 0) return;  // the same in every CTA of the cluster
  uint32_t prefix = 0;    // the threshold's leading bits found so far
  int need = want;        // candidates still to take among those that share them
  for (int round = 0; round < 4; ++round) {
    const int shift = 24 - 8 * round;
    int* hs = hist[round & 1];
    for (int b = threadIdx.x; b < 256; b += kSelThreads) hs[b] = 0;
    __syncthreads();
    for (int i = i0 + threadIdx.x; i < i1; i += kSelThreads) {
      const uint32_t k = weight_key(w[i]);
      if (round == 0 || (k >> (shift + 8)) == prefix) atomicAdd(&hs[(k >> shift) & 255], 1);
    }
    cl.sync();
    if (threadIdx.x < 256) {
      int t = 0;
      for (int r = 0; r < nr; ++r) t += cl.map_shared_rank(hs, r)[threadIdx.x];
      total[threadIdx.x] = t;
    }
    __syncthreads();
    // the bin where the count from the top reaches need
    if (threadIdx.x < 32) {
      int v[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = total[255 - (threadIdx.x * 8 + e)];
        sum += v[e];
      }
      int inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, inc, o);
        if ((int)threadIdx.x >= o) inc += t;
      }
      int above = inc - sum;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (above < need && above + v[e] >= need) {
          s_bin = 255 - (threadIdx.x * 8 + e);
          s_above = above;
        }
        above += v[e];
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | (uint32_t)s_bin;
    need -= s_above;
    // hist[round & 1] is cleared again two rounds on: after every CTA has passed the next round's cluster barrier
  }
  // prefix is the threshold's key; candidates above it are taken, and the first `need` equal ones.
  int gt = 0, eq = 0;
  for (int i = i0 + threadIdx.x; i < i1; i += kSelThreads) {
    const uint32_t k = weight_key(w[i]);
    gt += k > prefix;
    eq += k == prefix;
  }
  if (threadIdx.x < 2) s_count[threadIdx.x] = 0;
  __syncthreads();
  atomicAdd(&s_count[0], gt);
  atomicAdd(&s_count[1], eq);
  cl.sync();
  int base_gt = 0, base_eq = 0;  // in the CTAs before this one
  for (int r = 0; r < rank; ++r) {
    const int* c = cl.map_shared_rank(s_count, r);
    base_gt += c[0];
    base_eq += c[1];
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int j0 = i0; j0 < i1; j0 += kSelThreads) {
    const int i = j0 + threadIdx.x;
    const float x = i < i1 ? w[i] : 0.f;
    const uint32_t k = weight_key(x);
    const bool g = i < i1 && k > prefix, e = i < i1 && k == prefix;
    const unsigned bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, e);
    if (lane == 0) {
      w_gt[warp] = __popc(bg);
      w_eq[warp] = __popc(be);
    }
    __syncthreads();
    int ng = base_gt, ne = base_eq, tg = 0, te = 0;
    for (int q = 0; q < kSelWarps; ++q) {
      if (q < warp) {
        ng += w_gt[q];
        ne += w_eq[q];
      }
      tg += w_gt[q];
      te += w_eq[q];
    }
    ng += __popc(bg & ((1u << lane) - 1));
    ne += __popc(be & ((1u << lane) - 1));
    if (g || (e && ne < need)) {
      const int pos = ng + min(ne, need);
      index[pos] = i;
      if (kept) kept[pos] = x;
    }
    base_gt += tg;
    base_eq += te;
    __syncthreads();
  }
  cl.sync();  // no CTA leaves while another may read its counters
}

// Grid (blocks of the kept slots, heads, K / V).
__global__ void __launch_bounds__(kQuantThreads) k_kv8_gather(Kv8View src, Kv8View dst, const int* index, int keep) {
  __shared__ float red[kQuantThreads / 32];
  const int h = blockIdx.y, which = blockIdx.z;
  const int tokens = 1 << dst.tshift, per_row = dst.hd / 16;
  const int slot0 = blockIdx.x << dst.tshift;
  griddep_wait();
  const int page = dst.btab[slot0 / kPage];
  if (!dst.page_ok(page)) return;
  const uint8_t* from = which ? src.v : src.k;
  const float* from_scale = which ? src.vs : src.ks;
  float x[2][16];
  bool mine[2];
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int i = threadIdx.x + j * kQuantThreads;
    const int t = i / per_row, d = (i - t * per_row) * 16;
    mine[j] = t < tokens && slot0 + t < keep;
    if (!mine[j]) continue;
    const int s = index[(size_t)h * keep + slot0 + t];
    const int p = src.btab[s / kPage];
    if (src.page_ok(p)) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(from + src.page_row(p, h) + (size_t)(s % kPage) * src.hd + d));
      decode16(u, from_scale[src.scale_at(p, h, s % kPage)], src.code, x[j]);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[j][e] = 0.f;
    }
    amax = amax16(x[j], amax);
  }
  amax = block_max(amax, red);
  const float s = block_scale(amax, dst.code), m = inverse_scale(s);
  uint8_t* to = (which ? dst.v : dst.k) + dst.page_row(page, h) + (size_t)(slot0 % kPage) * dst.hd;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (!mine[j]) continue;
    const int i = threadIdx.x + j * kQuantThreads;
    const int t = i / per_row, d = (i - t * per_row) * 16;
    *reinterpret_cast<uint4*>(to + (size_t)t * dst.hd + d) = encode16(x[j], m, dst.code);
  }
  if (threadIdx.x == 0) (which ? dst.vs : dst.ks)[dst.scale_at(page, h, slot0 % kPage)] = s;
}

}  // namespace

bool launch_kv8_append(const Kv8View& c, const Kv8RowsArgs& a, int io, cudaStream_t st) {
  const int t0 = a.first >> c.tshift, t1 = (a.first + a.rows - 1) >> c.tshift;
  const dim3 grid(t1 - t0 + 1, c.n_kv, 2);
  const int chunks = (c.hd / 16) << c.tshift;
  const int threads = chunks < kQuantThreads ? chunks : kQuantThreads;
  if (io == 0)
    k_kv8_append<__nv_bfloat16><<<grid, threads, 0, st>>>(c, a);
  else if (io == 1)
    k_kv8_append<__half><<<grid, threads, 0, st>>>(c, a);
  else
    k_kv8_append<float><<<grid, threads, 0, st>>>(c, a);
  return cudaGetLastError() == cudaSuccess;
}

bool launch_kv8_read(const Kv8View& c, const Kv8RowsArgs& a, int io, cudaStream_t st) {
  const long long n = (long long)a.rows * c.n_kv * (c.hd / 16);
  const long long blocks = (n + 255) / 256;
  const dim3 grid((unsigned)(blocks < 152 * 8 ? blocks : 152 * 8), 2);
  if (io == 0)
    k_kv8_read<__nv_bfloat16><<<grid, 256, 0, st>>>(c, a);
  else if (io == 1)
    k_kv8_read<__half><<<grid, 256, 0, st>>>(c, a);
  else
    k_kv8_read<float><<<grid, 256, 0, st>>>(c, a);
  return cudaGetLastError() == cudaSuccess;
}

bool launch_kv8_evict(const Kv8View& src, const Kv8View& dst, const Kv8SelectArgs& a, cudaStream_t st) {
  int nr = 1;
  while (nr < 8 && (a.n - a.recent) > nr * 2 * kSelThreads) nr *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nr;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(nr, src.n_kv);
  cfg.blockDim = dim3(kSelThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, k_kv8_select, a) != cudaSuccess) return false;
  const int chunks = (dst.hd / 16) << dst.tshift;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(((a.keep - 1) >> dst.tshift) + 1, src.n_kv, 2);
  cfg.blockDim = dim3(chunks < kQuantThreads ? chunks : kQuantThreads);
  return cudaLaunchKernelEx(&cfg, k_kv8_gather, src, dst, (const int*)a.index, a.keep) == cudaSuccess;
}

}  // namespace ssd
