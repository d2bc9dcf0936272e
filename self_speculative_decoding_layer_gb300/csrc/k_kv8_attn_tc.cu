// Attention over the 8-bit KV cache for many queries of a KV head (long verify trees, prefill chunks), on the
// fifth-generation tensor cores.
//
// A CTA holds 128 or 256 queries of one KV head and walks over its split's
// 128-slot tiles.  S = Q K^T and O += P V run as 128-wide fp16 tcgen05.mma
// with fp32 accumulators in TMEM: Q, K and V come from shared memory (128-byte
// swizzle; V as stored, key by key, is the transposed operand), P from TMEM,
// where the softmax writes it over S.  Every code becomes fp16 once for all of
// the CTA's queries (eight converter warps, which also prefetch the next
// tile's codes in registers), and every score is read twice from TMEM by its
// row's thread (once for the maximum, once for the exponential).
//
// 64 bf16 rows of 64 heads on 8 over 16448 int8 slots, 34.4 GFLOP: 57 us with
// the merge, 0.6 PFLOP/s, the tensor pipe busy for 27 % and the ALU for 26.
// What bounds it is latency: of about 4800 clocks a tile each block spends
// 1900 to 2700 in its softmax (1000 of them the exponentials of two warps a
// scheduler) and the rest between its weights and its next scores, where the
// MMAs take 75 to 150 clocks instead of 64 beside the other block's softmax.
// Measured worse: one pass over the scores with the maximum checked chunk by
// chunk (it spilled, 70 to 77 us), one issuer for both blocks (60.4), stages
// of K and V released apart (59.2), softmaxes that take turns (70).
//
// fp32 queries are split into hi + lo, and so are their softmax weights; they
// run one block of 128 queries, 16-bit ones two, whose softmax and MMAs
// alternate.  Scales: K's multiplies the scores, V's goes into the exponent
// (2^(x + log2 r), r = the block's scale over the split's largest, divided out
// of the sum again), so it costs nothing per element; a weight times r below
// 2^-34 is lost to fp16, which is that part of the split's largest V value.
// The running maximum may
// lag by 2^kSlack before O is rescaled, which after the first tiles hardly
// ever happens.
#include "kv8_attn.cuh"

namespace ssd {

namespace {

constexpr int kTcTile = 128;      // slots of a tile
constexpr int kConvWarps = 8;
constexpr int kMmaWarp = 8 + kConvWarps;
constexpr int kTcThreads = (kMmaWarp + 2) * 32;  // warps 0-3 and 4-7: softmax of query blocks 0 and 1; converters; the
                                                 // blocks' MMA issuers (one for both waits for the block whose turn it is)
constexpr int kTcStages = 2;
constexpr float kTcShift = 9.f;   // softmax weights are held times 2^9, and grow to 2^(9 + kSlack) < 2^16
constexpr float kSlack = 6.f;

struct TcHead {                   // of a stage's tile, for each sixteen slots
  float ks[8], lrv[8], irv[8];    // K's scale; log2 r and 1 / r of V's
  int full, ok;                   // every slot is visible; bit p: page p of the tile is one
};

template <typename T, int HD>
struct TcSmem {
  static constexpr bool SPLIT = sizeof(T) == 4;
  static constexpr int NQT = SPLIT ? 1 : 2;
  static constexpr int kMat = 128 * HD * 2;  // one 128-row fp16 operand
  static constexpr int kQ = NQT * (SPLIT ? 2 : 1) * kMat;
  static constexpr int kStage = 2 * kMat;    // K, V
  static constexpr int kTail = kTcStages * (int)sizeof(TcHead) + NQT * 128 * 4 + 256;
  static constexpr int kBytes = 1024 + kQ + kTcStages * kStage + kTail;
};

// Shared-memory descriptors, 128-byte swizzle (8-row atoms of 1024 bytes, tile base 1024-byte aligned).  K-major:
// rows of 64 K elements.  MN-major: the same bytes read as the transposed operand, rows of 64 M or N elements, `lead`
// bytes to the next 64.
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lead) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// kind::f16, A and B fp16, fp32 accumulator, M = 128, N = n; trans_b: B is MN-major.
__device__ __forceinline__ constexpr uint32_t idesc_h(int n, bool trans_b) {
  return (1u << 4) | (trans_b ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// Issued by the lane that `issue` names; the whole warp executes the code around, so that descriptors stay in uniform
// registers.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accum, uint32_t issue) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accum), "r"(issue)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accum, uint32_t issue) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accum), "r"(issue)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t issue) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar)),
      "r"(issue)
      : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Ask for 32 columns of this warp's 32 TMEM lanes; r holds them after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32_async(uint32_t t, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}
// Wait for every load that this thread has asked for; the operands keep r's uses behind the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
               :
               : "memory");
  asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t t, float (&f)[32]) {
  uint32_t r[32];
  tmem_ld32_async(t, r);
  tmem_wait_ld(r);
#pragma unroll
  for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(r[i]);
}
// The largest of sixteen.
__device__ __forceinline__ float max16(const uint32_t* r) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = fmaxf(__uint_as_float(r[i]), __uint_as_float(r[i + 8]));
#pragma unroll
  for (int n = 4; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) y[i] = fmaxf(y[i], y[i + n]);
  return y[0];
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(t)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Grid (splits, KV heads, blocks of 128 NQT queries).
template <typename T, int HD, int CODE>
__global__ void __launch_bounds__(kTcThreads, 1) k_kv8_attention_tc(const __grid_constant__ Kv8AttnArgs a) {
  using L = TcSmem<T, HD>;
  constexpr bool SPLIT = L::SPLIT;
  constexpr int NQT = L::NQT, HB = HD / 64;   // 64-wide blocks of the head dim
  constexpr int BLK = 128 * 128;              // bytes of 128 rows of one block
  extern __shared__ unsigned char s_raw[];
  unsigned char* smem = s_raw + ((1024 - (smem_u32(s_raw) & 1023)) & 1023);
  unsigned char* s_q = smem;                  // [NQT][hi, lo][HB][128][128 bytes]
  unsigned char* s_kv = smem + L::kQ;         // [stages][K, V][HB][128][128 bytes]
  TcHead* s_head = reinterpret_cast<TcHead*>(s_kv + kTcStages * L::kStage);
  float* s_inv = reinterpret_cast<float*>(s_head + kTcStages);  // [NQT][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_inv + NQT * 128);
  uint64_t* kv_full = bars;                   // [stages] converters -> MMA, softmax
  uint64_t* kv_empty = bars + kTcStages;      // [stages] MMA -> converters
  uint64_t* s_full = kv_empty + kTcStages;    // [NQT] MMA -> softmax
  uint64_t* p_full = s_full + NQT;            // [NQT] softmax -> MMA
  uint64_t* pv_done = p_full + NQT;           // [NQT] MMA -> softmax, after the last tile
  uint64_t* turn = pv_done + NQT;             // issuer of block 0 -> of block 1
  __shared__ uint32_t s_tmem;
  __shared__ float s_red[kConvWarps], s_vref;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, h = blockIdx.y, q0 = blockIdx.z * 128 * NQT;
  const int nq = a.rows * a.group;
  const int n_act = min(NQT, (nq - q0 + 127) / 128);  // query blocks in use, one at least
  griddep_launch();
  const Tiles<7> tiles(a.prefix, a.base, a.rows);
  const int t_first = min(tiles.n, split * a.split_tiles), t_last = min(tiles.n, t_first + a.split_tiles);
  const int n_tile = t_last - t_first;

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    if (lane == 0) {
      for (int i = 0; i < kTcStages; ++i) {
        mbar_init(&kv_full[i], kConvWarps * 32);
        mbar_init(&kv_empty[i], n_act);
      }
      for (int i = 0; i < NQT; ++i) {
        mbar_init(&s_full[i], 1);
        mbar_init(&p_full[i], 128);
        mbar_init(&pv_done[i], 1);
      }
      mbar_init(turn, 1);
      fence_barrier_init();
    }
  }
  griddep_wait();
  // Converters: thread ct takes sixteen-byte chunk ct % CH of rows ct / CH + RS i of every tile.  What they need
  // first is asked for before the queries are staged.
  constexpr int CH = HD / 16, RS = kConvWarps * 32 / CH, NI = 128 / RS;
  const int ct = threadIdx.x - 256, ch = ct & (CH - 1), r0 = (ct & (kConvWarps * 32 - 1)) / CH;
  // Page `half` of tile j as the table has it (checked where it is used, a tile later), or -1 where no row sees a slot
  // of it.
  auto page_of = [&](int j, int half) {
    if (j >= n_tile) return -1;
    const int slot = tiles.slot(t_first + j) + half * kPage;
    if (!visible_any(slot, a) && !visible_any(slot + 16, a) && !visible_any(slot + 32, a) && !visible_any(slot + 48, a))
      return -1;
    return __ldg(a.c.btab + slot / kPage);
  };
  auto checked = [&](int page) { return a.c.page_ok(page) ? page : -1; };
  uint4 k[NI], v[NI];
  // Byte offset of this thread's first chunk in a page's rows of this head.
  auto page_at = [&](int page) { return page < 0 ? (size_t)0 : a.c.page_row(page, h) + (size_t)r0 * HD + ch * 16; };
  auto load = [&](int i, int j, int page, size_t at, bool whole) {  // chunk i of tile j: row r0 + RS i
    // (rows that hold no token may hold any bits)
    if (page >= 0 && (whole || visible(tiles.slot(t_first + j) + r0 + RS * i, a.prefix, a.base, a.any))) {
      const size_t o = at + (RS * i % kPage) * HD;
      k[i] = __ldg(reinterpret_cast<const uint4*>(a.c.k + o));
      v[i] = __ldg(reinterpret_cast<const uint4*>(a.c.v + o));
    } else {
      k[i] = v[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  };
  auto whole_of = [&](int j) { return tiles.slot(t_first + j) + kTcTile <= a.prefix; };
  const bool converter = warp >= 8 && warp < kMmaWarp;
  int p0 = -1, p1 = -1;
  if (converter && n_tile > 0) {
    p0 = checked(page_of(0, 0));
    p1 = checked(page_of(0, 1));
    const size_t a0 = page_at(p0), a1 = page_at(p1);
#pragma unroll
    for (int i = 0; i < NI; ++i) load(i, 0, RS * i < kPage ? p0 : p1, RS * i < kPage ? a0 : a1, whole_of(0));
  }
  float vref = 1.f;
  if (converter) {  // (while the other warps stage the queries)
    float vmax = 0.f;  // V's largest scale in the split
    for (int i = ct; i < n_tile * 8; i += kConvWarps * 32) {
      const int slot = tiles.slot(t_first + (i >> 3)) + (i & 7) * 16;
      if (!visible_any(slot, a)) continue;
      const int page = __ldg(a.c.btab + slot / kPage);
      if (a.c.page_ok(page)) vmax = fmaxf(vmax, __ldg(a.c.vs + a.c.scale_at(page, h, slot % kPage)));
    }
    vmax = warp_max(vmax);
    if (lane == 0) s_red[warp - 8] = vmax;
    asm volatile("bar.sync 1, %0;" ::"n"(kConvWarps * 32) : "memory");
    vmax = warp_max(s_red[lane % kConvWarps]);
    vref = vmax > 0.f ? vmax : 1.f;
    if (ct == 0) s_vref = vref;
  }
  // Queries: a warp takes eight at a time (all of their loads first), as fp16 rows times their power of two.
  constexpr int QG = 8;
  for (int g0 = (warp < 8 ? warp : warp - kConvWarps) * QG; !converter && g0 < n_act * 128; g0 += 10 * QG) {
    float2 x[QG][HB];
    int r = (q0 + g0) / a.group, e = q0 + g0 - r * a.group;
#pragma unroll
    for (int u = 0; u < QG; ++u) {
      const T* p = reinterpret_cast<const T*>(a.q) + (size_t)r * a.ld_q + (size_t)(h * a.group + e) * HD;
#pragma unroll
      for (int b = 0; b < HB; ++b) x[u][b] = r < a.rows ? load2(p + b * 64 + 2 * lane) : make_float2(0.f, 0.f);
      if (++e == a.group) e = 0, ++r;
    }
#pragma unroll
    for (int u = 0; u < QG; ++u) {
      const int q = g0 + u, row = q & 127;
      float amax = 0.f;
#pragma unroll
      for (int b = 0; b < HB; ++b) amax = fmaxf(amax, fmaxf(fabsf(x[u][b].x), fabsf(x[u][b].y)));
      float f, inv;
      query_factor(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax))), f, inv);  // (amax >= 0)
      unsigned char* to = s_q + (q >> 7) * (SPLIT ? 2 : 1) * L::kMat + row * 128 +
                          ((((lane >> 2) ^ (row & 7)) << 4) | ((lane & 3) << 2));
#pragma unroll
      for (int b = 0; b < HB; ++b) {
        const float x0 = x[u][b].x * f, x1 = x[u][b].y * f;
        const uint32_t hi = pack_half2(x0, x1);
        *reinterpret_cast<uint32_t*>(to + b * BLK) = hi;
        if (SPLIT) *reinterpret_cast<uint32_t*>(to + L::kMat + b * BLK) = pack_rest2(x0, x1, hi);
      }
      if (lane == 0) s_inv[q] = inv;
    }
  }
  fence_proxy_async();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;
  // TMEM columns: S of block qt (P hi over its first half); P lo (SPLIT, one block); O of block qt
  const uint32_t c_lo = 128, c_o = 256;

  if (converter) {
    // ---- converters
    int t0 = page_of(1, 0), t1 = page_of(1, 1);
    for (int j = 0; j < n_tile; ++j) {
      const int st = j & 1, n0 = checked(t0), n1 = checked(t1);
      t0 = page_of(j + 2, 0);
      t1 = page_of(j + 2, 1);
      float ks = 0.f, vs = 0.f;  // of sixteen slots, for eight of the threads
      const int slot0 = tiles.slot(t_first + j);
      if (ct < 8) {
        const int page = ct < 4 ? p0 : p1;
        if (page >= 0 && visible_any(slot0 + ct * 16, a)) {  // (elsewhere the scales may be anything)
          const size_t sc = a.c.scale_at(page, h, (ct & 3) * 16);
          ks = __ldg(a.c.ks + sc);
          vs = __ldg(a.c.vs + sc);
        }
      }
      if (j >= kTcStages && !mbar_wait_bounded(&kv_empty[st], (uint32_t)((j >> 1) - 1) & 1u)) break;
      unsigned char* dst = s_kv + st * L::kStage + (ch >> 2) * BLK + r0 * 128;
      const size_t a0 = page_at(n0), a1 = page_at(n1);
      const bool more = j + 1 < n_tile, whole = more && whole_of(j + 1);
      // Chunk i becomes two sixteen-byte chunks of fp16 for K and for V, stored in an order that alternates with the
      // 64-wide block, so that a row's lanes meet in no bank.  (r0 + RS i and r0 have the same three low bits.)
      const int flip = ch >> 2, c0 = (ch & 3) * 2;
      const uint32_t o0 = (uint32_t)((c0 + flip) ^ (r0 & 7)) << 4, o1 = (uint32_t)((c0 + 1 - flip) ^ (r0 & 7)) << 4;
      auto convert = [&](const uint4& u, unsigned char* to) {
        uint4 w0, w1;
        codes_to_half<CODE>(flip ? u.z : u.x, w0.x, w0.y);
        codes_to_half<CODE>(flip ? u.w : u.y, w0.z, w0.w);
        codes_to_half<CODE>(flip ? u.x : u.z, w1.x, w1.y);
        codes_to_half<CODE>(flip ? u.y : u.w, w1.z, w1.w);
        *reinterpret_cast<uint4*>(to + o0) = w0;
        *reinterpret_cast<uint4*>(to + o1) = w1;
      };
      if (whole && n0 >= 0 && n1 >= 0) {
        const uint8_t *k0 = a.c.k + a0, *k1 = a.c.k + a1, *v0 = a.c.v + a0, *v1 = a.c.v + a1;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          convert(k[i], dst + i * RS * 128);
          convert(v[i], dst + i * RS * 128 + L::kMat);
          k[i] = __ldg(reinterpret_cast<const uint4*>((RS * i < kPage ? k0 : k1) + (RS * i % kPage) * HD));
          v[i] = __ldg(reinterpret_cast<const uint4*>((RS * i < kPage ? v0 : v1) + (RS * i % kPage) * HD));
        }
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          convert(k[i], dst + i * RS * 128);
          convert(v[i], dst + i * RS * 128 + L::kMat);
          if (more) load(i, j + 1, RS * i < kPage ? n0 : n1, RS * i < kPage ? a0 : a1, whole);
        }
      }
      if (ct < 8) {
        const float r = vs / vref;
        s_head[st].ks[ct] = ks;
        s_head[st].lrv[ct] = vs > 0.f ? fmaxf(log2f(r), -60.f) : 0.f;  // (all codes 0: any scale does)
        s_head[st].irv[ct] = vs > 0.f ? exp2f(-fmaxf(log2f(r), -60.f)) : 1.f;
        if (ct == 0) {
          s_head[st].full = slot0 + kTcTile <= a.prefix && p0 >= 0 && p1 >= 0;
          s_head[st].ok = (p0 >= 0 ? 1 : 0) | (p1 >= 0 ? 2 : 0);
        }
      }
      fence_proxy_async();
      arrive(&kv_full[st]);
      p0 = n0;
      p1 = n1;
    }
  } else if (warp >= kMmaWarp) {
    const int qt = warp - kMmaWarp;
    if (n_tile > 0 && qt < n_act) {
      // ---- MMA issuer
      const uint32_t issue = lane == 0;
      constexpr uint32_t id_s = idesc_h(kTcTile, false), id_o = idesc_h(HD, true);
      const uint64_t dq = desc_k(smem_u32(s_q)), dk = desc_k(smem_u32(s_kv));
      const uint64_t dv = desc_mn(smem_u32(s_kv) + L::kMat, BLK);
      // (descriptors count addresses in sixteen bytes; all of shared memory fits their field)
      auto qk = [&](int st) {
        const uint64_t q = dq + (uint32_t)(qt * (SPLIT ? 2 : 1) * L::kMat >> 4), k = dk + (uint32_t)(st * L::kStage >> 4);
#pragma unroll
        for (int part = SPLIT ? 1 : 0; part >= 0; --part)  // (lo first: an accumulator cuts off what does not fit it)
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t off = (kk >> 2) * BLK + (kk & 3) * 32;
            mma_ss(tmem + qt * 128, q + ((part * L::kMat + off) >> 4), k + (off >> 4), id_s, part < (SPLIT ? 1 : 0) || kk > 0,
                   issue);
          }
        commit(&s_full[qt], issue);
      };
      auto pv = [&](int st, bool first) {
        const uint64_t v = dv + (uint32_t)(st * L::kStage >> 4);
#pragma unroll
        for (int part = 0; part < (SPLIT ? 2 : 1); ++part)
#pragma unroll
          for (int kk = 0; kk < kTcTile / 16; ++kk)
            mma_ts(tmem + c_o + qt * 128, tmem + (part ? c_lo : qt * 128) + kk * 8, v + kk * (2048 >> 4), id_o,
                   !(first && part == 0 && kk == 0), issue);
      };
      bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(&kv_full[0], 0u));
      // (block 1 starts when block 0 has its first weights, so that their softmaxes do not begin side by side)
      if (NQT == 2 && qt == 1 && ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(turn, 0u));
      fence_after();
      if (ok) qk(0);
      for (int j = 0; ok && j < n_tile; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&p_full[qt], (uint32_t)j & 1u));
        if (!ok) break;
        if (NQT == 2 && qt == 0 && j == 0 && lane == 0) arrive(turn);
        fence_after();
        pv(j & 1, j == 0);
        commit(&kv_empty[j & 1], issue);
        if (j + 1 < n_tile) {
          ok = __all_sync(0xffffffffu, mbar_wait_bounded(&kv_full[(j + 1) & 1], (uint32_t)((j + 1) >> 1) & 1u));
          if (!ok) break;
          fence_after();
          qk((j + 1) & 1);
        } else {
          commit(&pv_done[qt], issue);
        }
      }
    }
  } else if (warp < 8 && (warp >> 2) < n_act) {
    // ---- softmax: one thread for each query row
    const int qt = warp >> 2, row = threadIdx.x & 127, qi = q0 + qt * 128 + row;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + qt * 128, tl = tmem + lanes + c_lo, to = tmem + lanes + c_o + qt * 128;
    const bool cap = a.cap > 0.f;
    const float inv_cap = cap ? 1.f / a.cap : 0.f;
    const float coef = a.scale * s_inv[qt * 128 + row] * (cap ? 1.f : kLog2e);
    const unsigned long long mask = qi < nq ? a.mask[qi / a.group] : 0ull;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    // Which of the 32 slots from `slot` on this row sees.
    auto bits_of = [&](int slot, int page_ok) -> uint32_t {
      if (!page_ok) return 0u;
      const int n = a.prefix - slot, e = slot - a.base;
      uint32_t b = n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1u : 0u;
      if (e > -32 && e < 64) b |= (uint32_t)(e >= 0 ? mask >> e : mask << -e);
      return b;
    };
    for (int j = 0; j < n_tile; ++j) {
      const int st = j & 1;
      ok = mbar_wait_bounded(&kv_full[st], (uint32_t)(j >> 1) & 1u) && mbar_wait_bounded(&s_full[qt], (uint32_t)j & 1u);
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_after();
      const TcHead& hd = s_head[st];
      const bool full = hd.full;
      const int slot0 = tiles.slot(t_first + j);
      // scores of 32 columns in the log2 domain, where the tile is not plain
      auto slow = [&](float (&x)[32], int c) {
        const uint32_t b = bits_of(slot0 + c * 32, (hd.ok >> (c >> 1)) & 1);
        const float f[2] = {coef * hd.ks[2 * c], coef * hd.ks[2 * c + 1]};
        if (cap) {  // (apart from the masks, so that the elements' chains overlap)
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = capped<SPLIT>(x[i] * f[i >> 4], a.cap, inv_cap);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] *= f[i >> 4];
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = (b >> i) & 1u ? x[i] : -INFINITY;
      };
      // A plain tile's columns are asked for a chunk ahead; the others' loops stay rolled, so that the code fits the
      // instruction cache.
      float top = -INFINITY;
      if (full) {
        uint32_t x[2][32];
        tmem_ld32_async(ts, x[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_wait_ld(x[c & 1]);
          if (c < 3) tmem_ld32_async(ts + (c + 1) * 32, x[(c + 1) & 1]);
          top = fmaxf(top, fmaxf(max16(x[c & 1]) * (coef * hd.ks[2 * c]), max16(x[c & 1] + 16) * (coef * hd.ks[2 * c + 1])));
        }
        if (cap) top = capped<SPLIT>(top, a.cap, inv_cap);  // (the cap keeps the order, to its rounding)
      } else {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float x[32];
          tmem_ld32(ts + c * 32, x);
          slow(x, c);
#pragma unroll
          for (int i = 0; i < 32; ++i) top = fmaxf(top, x[i]);
        }
      }
      const bool lags = top > m + kSlack || (m == -INFINITY && top > m);
      if (__any_sync(0xffffffffu, lags)) {
        const float f = lags ? exp2_approx(m - top) : 1.f;  // (m = -inf: 0)
        if (lags) m = top;
        l *= f;
        if (j > 0) {  // (the products of the tiles before are in O: they were committed before these scores)
#pragma unroll 1
          for (int c = 0; c < HD / 32; ++c) {
            float x[32];
            tmem_ld32(to + c * 32, x);
            uint32_t y[2][16];
#pragma unroll
            for (int i = 0; i < 32; ++i) y[i >> 4][i & 15] = __float_as_uint(x[i] * f);
            tmem_st16(to + c * 32, y[0]);
            tmem_st16(to + c * 32 + 16, y[1]);
          }
        }
      }
      const float ref = kTcShift - (m == -INFINITY ? 0.f : m);
      // Weights of 32 columns whose scores (times cf0 / cf1) are x: into P, over columns that have been read already.
      auto weigh = [&](const uint32_t (&x)[32], int c, float cf0, float cf1) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float cf = b ? cf1 : cf0, add = ref + hd.lrv[2 * c + b];
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float p0 = exp2_approx(fmaf(__uint_as_float(x[b * 16 + i]), cf, add));
            const float p1 = exp2_approx(fmaf(__uint_as_float(x[b * 16 + i + 1]), cf, add));
            sum[(i & 2)] += p0;
            sum[(i & 2) + 1] += p1;
            hi[b * 8 + i / 2] = pack_half2(p0, p1);
            if (SPLIT) lo[b * 8 + i / 2] = pack_rest2(p0, p1, hi[b * 8 + i / 2]);
          }
          l = fmaf((sum[0] + sum[1]) + (sum[2] + sum[3]), hd.irv[2 * c + b], l);
        }
        tmem_st16(ts + c * 16, hi);
        if (SPLIT) tmem_st16(tl + c * 16, lo);
      };
      if (full && !cap) {
        uint32_t x[2][32];
        tmem_ld32_async(ts, x[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_wait_ld(x[c & 1]);
          if (c < 3) tmem_ld32_async(ts + (c + 1) * 32, x[(c + 1) & 1]);
          weigh(x[c & 1], c, coef * hd.ks[2 * c], coef * hd.ks[2 * c + 1]);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float x[32];
          uint32_t y[32];
          tmem_ld32(ts + c * 32, x);
          slow(x, c);
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = __float_as_uint(x[i]);
          weigh(y, c, 1.f, 1.f);
        }
      }
      tmem_wait_st();
      fence_before();
      arrive(&p_full[qt]);
    }
    // ---- output
    if (n_tile > 0 && __all_sync(0xffffffffu, ok)) ok = mbar_wait_bounded(&pv_done[qt], 0u);
    if (__all_sync(0xffffffffu, ok)) {
      fence_after();
      const float vref = n_tile > 0 ? *(volatile float*)&s_vref : 0.f;
      const int r = qi / a.group, head = h * a.group + qi - r * a.group;
      const size_t at = ((size_t)h * nq + qi) * a.n_split + split;
      const float f = a.part_o ? vref : l == 0.f ? 0.f : vref / l;
      const float top = m + (kPShift - kTcShift);
      float4* s_rows = reinterpret_cast<float4*>(s_q + qt * (SPLIT ? 2 : 1) * L::kMat + (warp & 3) * 4096);
#pragma unroll
      for (int c = 0; c < HD / 32; ++c) {
        float x[32];
        if (n_tile > 0) {
          tmem_ld32(to + c * 32, x);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0.f;
        }
        // Rows to coalesced lines, through the block's queries, which no MMA reads any more: 32 rows of 32 columns a
        // warp, chunks swizzled by the row.  (A row for each thread, as TMEM has them: 8 us for 512 queries a head.)
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          s_rows[lane * 8 + (i ^ (lane & 7))] = make_float4(x[4 * i] * f, x[4 * i + 1] * f, x[4 * i + 2] * f, x[4 * i + 3] * f);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = i * 4 + (lane >> 3), to_q = qi - lane + row;
          const float4 y = s_rows[row * 8 + ((lane & 7) ^ (row & 7))];
          if (to_q >= nq) continue;
          const int col = c * 32 + (lane & 7) * 4;
          if (a.part_o) {
            *reinterpret_cast<float4*>(a.part_o + (((size_t)h * nq + to_q) * a.n_split + split) * HD + col) = y;
          } else {
            const int to_r = to_q / a.group;
            store4(reinterpret_cast<T*>(a.out) + (size_t)to_r * a.ld_out + (size_t)(h * a.group + to_q - to_r * a.group) * HD + col,
                   y);
          }
        }
      }
      if (qi < nq) {
        if (a.part_o)
          a.part_ml[at] = make_float2(top, l);
        else if (a.lse)
          a.lse[a.lse_at(r, head)] = lse_of(top, l);
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

template <typename T, int HD, int CODE>
bool run_tc(Kv8AttnArgs a, cudaStream_t st) {
  using L = TcSmem<T, HD>;
  const auto kern = k_kv8_attention_tc<T, HD, CODE>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) != cudaSuccess) return false;
  const Tiles<7> tiles(a.prefix, a.base, a.rows);
  a.split_tiles = (tiles.n + a.n_split - 1) / a.n_split;
  const int qb = 128 * L::NQT, nq = a.rows * a.group;
  return launch_kv8(kern, dim3(a.n_split, a.c.n_kv, (nq + qb - 1) / qb), kTcThreads, L::kBytes, st, 1, a);
}

template <typename T>
bool tc_of(const Kv8AttnArgs& a, cudaStream_t st) {
  const bool i8 = a.c.code == KV8_INT8;
  if (a.c.hd == 128) return i8 ? run_tc<T, 128, KV8_INT8>(a, st) : run_tc<T, 128, KV8_E4M3>(a, st);
  return i8 ? run_tc<T, 64, KV8_INT8>(a, st) : run_tc<T, 64, KV8_E4M3>(a, st);
}

}  // namespace

bool launch_kv8_attention_tc(const Kv8AttnArgs& a, int io, cudaStream_t st) {
  return io == 0 ? tc_of<__nv_bfloat16>(a, st) : io == 1 ? tc_of<__half>(a, st) : tc_of<float>(a, st);
}

}  // namespace ssd
