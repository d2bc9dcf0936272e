// The 8-bit KV cache's entry points: argument checks, then the kernels of
// k_kv8.cu, k_kv8_attn.cu and k_kv8_attn_tc.cu on the caller's stream.
#include <math.h>

#include "../../include/ssd.h"
#include "kv8.h"

using namespace ssd;

namespace {

constexpr int kMaxPages = 1 << 24;  // of a block table: slot numbers and the tiles past them stay far inside an int
constexpr int kMaxHeads = 4096;     // KV heads, and query heads of one: grids stay inside their limits

constexpr int64_t kMaxStride = (int64_t)1 << 40;

size_t io_size(int dtype) { return dtype == SSD_F32 ? 4 : 2; }
bool io_ok(int dtype) { return dtype == SSD_BF16 || dtype == SSD_FP16 || dtype == SSD_F32; }
bool aligned(const void* p, size_t a) { return p && ((uintptr_t)p & (a - 1)) == 0; }

// One layer of a cache; false if the descriptor is not valid.
bool view_of(const ssd_kv8_cache* c, Kv8View* v) {
  if (!c || !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->block_table, 4))
    return false;
  if (c->n_pages < 1 || c->n_pages > kMaxPages || c->pool_pages < 1 || c->layer < 0) return false;
  if (c->n_kv_heads < 1 || c->n_kv_heads > kMaxHeads || (c->head_dim != 64 && c->head_dim != 128)) return false;
  if (c->dtype != SSD_I8 && c->dtype != SSD_E4M3) return false;
  if (c->block_tokens != 16 && c->block_tokens != 32 && c->block_tokens != 64) return false;
  const size_t heads = (size_t)c->layer * c->pool_pages * c->n_kv_heads;  // (page, head) units before this layer
  v->tshift = c->block_tokens == 16 ? 4 : c->block_tokens == 32 ? 5 : 6;
  v->k = (uint8_t*)c->k + heads * kPage * c->head_dim;
  v->v = (uint8_t*)c->v + heads * kPage * c->head_dim;
  v->ks = c->k_scale + (heads << (6 - v->tshift));
  v->vs = c->v_scale + (heads << (6 - v->tshift));
  v->btab = c->block_table;
  v->pool = c->pool_pages;
  v->n_kv = c->n_kv_heads;
  v->hd = c->head_dim;
  v->code = c->dtype == SSD_I8 ? KV8_INT8 : KV8_E4M3;
  return true;
}

// A matrix of `rows` rows of `width` elements, `ld` apart, that 16-byte accesses can read.
bool rows_ok(const void* p, int64_t ld, int64_t width, int dtype) {
  return aligned(p, 16) && ld >= width && ld <= kMaxStride && (ld * (int64_t)io_size(dtype)) % 16 == 0;
}

bool rows_args(const ssd_kv8_cache* c, const ssd_kv8_rows* r, Kv8View* v, Kv8RowsArgs* a) {
  if (!view_of(c, v) || !r || !io_ok(r->dtype)) return false;
  const int64_t width = (int64_t)c->n_kv_heads * c->head_dim;
  if (!rows_ok(r->k, r->ld_k, width, r->dtype) || !rows_ok(r->v, r->ld_v, width, r->dtype)) return false;
  if (r->rows < 1 || r->first < 0 || (int64_t)r->first + r->rows > (int64_t)c->n_pages * kPage) return false;
  a->k = r->k;
  a->v = r->v;
  a->ld_k = (size_t)r->ld_k;
  a->ld_v = (size_t)r->ld_v;
  a->first = r->first;
  a->rows = r->rows;
  return true;
}

// Everything the attention and weights calls share; out is checked by the attention.
bool attn_args(const ssd_kv8_cache* c, const ssd_kv8_attention_args* p, Kv8AttnArgs* a) {
  if (!view_of(c, &a->c) || !p || !io_ok(p->dtype)) return false;
  if (p->rows < 1 || p->rows > kMaxRows || p->prefix < 0 || p->base < 0) return false;
  if (p->n_q_heads < 1 || p->n_q_heads % c->n_kv_heads || p->n_q_heads / c->n_kv_heads > kMaxHeads) return false;
  const int64_t slots = (int64_t)c->n_pages * kPage;
  if (p->prefix > slots || (int64_t)p->base + p->rows > slots) return false;
  if (!rows_ok(p->q, p->ld_q, (int64_t)p->n_q_heads * c->head_dim, p->dtype)) return false;
  if (p->lse && !aligned(p->lse, 4)) return false;
  if (!(p->scale > 0.f) || !isfinite(p->scale) || !(p->softcap >= 0.f) || !isfinite(p->softcap)) return false;
  if (p->softcap > 0.f && !(p->softcap >= 1e-30f && p->softcap <= 1e30f)) return false;  // (its inverse has to be a number)
  a->q = p->q;
  a->ld_q = (size_t)p->ld_q;
  a->lse = p->lse;
  if (p->ld_lse < 0 || p->step_lse < 0 || p->ld_lse > kMaxStride || p->step_lse > kMaxStride) return false;
  const bool plain = p->ld_lse == 0 && p->step_lse == 0;
  a->ld_lse = plain ? (size_t)p->n_q_heads : (size_t)p->ld_lse;
  a->step_lse = plain ? 1 : (size_t)p->step_lse;
  a->n_q = p->n_q_heads;
  a->group = p->n_q_heads / c->n_kv_heads;
  a->rows = p->rows;
  a->prefix = p->prefix;
  a->base = p->base;
  a->scale = p->scale;
  a->cap = p->softcap;
  const unsigned long long all = p->rows == 64 ? ~0ull : (1ull << p->rows) - 1;
  a->any = 0;
  for (int r = 0; r < p->rows; ++r) {
    a->mask[r] = p->mask[r] & all;
    a->any |= a->mask[r];
  }
  return true;
}

int slots_of(const Kv8AttnArgs& a) { return a.prefix > a.base + a.rows ? a.prefix : a.base + a.rows; }

// Sets a's key splits; bytes of scratch that they need.
size_t split(Kv8AttnArgs* a, int io, bool* tc) {
  const Kv8Splits s = kv8_attention_splits(a->rows, a->group, a->c.n_kv, slots_of(*a), io);
  a->n_split = s.n;
  *tc = s.tc;
  return s.scratch ? (size_t)a->c.n_kv * a->rows * a->group * s.n * (a->c.hd + 2) * 4 : 0;
}

}  // namespace

ssd_status ssd_kv8_append(const ssd_kv8_cache* cache, const ssd_kv8_rows* rows, void* stream) {
  Kv8View v;
  Kv8RowsArgs a;
  if (!rows_args(cache, rows, &v, &a)) return SSD_ERR_INVALID_ARG;
  return launch_kv8_append(v, a, rows->dtype, (cudaStream_t)stream) ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_kv8_read(const ssd_kv8_cache* cache, const ssd_kv8_rows* rows, void* stream) {
  Kv8View v;
  Kv8RowsArgs a;
  if (!rows_args(cache, rows, &v, &a)) return SSD_ERR_INVALID_ARG;
  return launch_kv8_read(v, a, rows->dtype, (cudaStream_t)stream) ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_kv8_attention_scratch_bytes(const ssd_kv8_cache* cache, const ssd_kv8_attention_args* args) {
  Kv8AttnArgs a{};
  if (!attn_args(cache, args, &a)) return 0;
  bool tc;
  const size_t b = split(&a, args->dtype, &tc);
  return b < 256 ? 256 : (b + 255) / 256 * 256;
}

ssd_status ssd_kv8_attention(const ssd_kv8_cache* cache, const ssd_kv8_attention_args* args, void* scratch,
                             size_t scratch_bytes, void* stream) {
  Kv8AttnArgs a{};
  if (!attn_args(cache, args, &a)) return SSD_ERR_INVALID_ARG;
  if (!rows_ok(args->out, args->ld_out, (int64_t)a.n_q * a.c.hd, args->dtype)) return SSD_ERR_INVALID_ARG;
  a.out = args->out;
  a.ld_out = (size_t)args->ld_out;
  bool tc;
  const size_t need = split(&a, args->dtype, &tc);
  if (need) {
    if (!scratch || ((uintptr_t)scratch & 255)) return SSD_ERR_INVALID_ARG;
    if (scratch_bytes < need) return SSD_ERR_CAPACITY;
    a.part_o = (float*)scratch;
    a.part_ml = (float2*)(a.part_o + (size_t)a.c.n_kv * a.rows * a.group * a.n_split * a.c.hd);
  }
  return launch_kv8_attention(a, args->dtype, tc, (cudaStream_t)stream) ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_kv8_weights(const ssd_kv8_cache* cache, const ssd_kv8_attention_args* args, uint64_t row_set,
                           const float* weight_in, float* weight_out, int64_t ld_weight, void* stream) {
  Kv8AttnArgs a{};
  if (!attn_args(cache, args, &a) || !a.lse) return SSD_ERR_INVALID_ARG;
  if (!aligned(weight_out, 4) || (weight_in && !aligned(weight_in, 4)) || ld_weight < slots_of(a))
    return SSD_ERR_INVALID_ARG;
  for (int r = 0; r < a.rows; ++r)
    if ((row_set >> r) & 1) a.take[a.n_take++] = (unsigned char)r;
  a.w_in = weight_in;
  a.w_out = weight_out;
  a.ld_w = (size_t)ld_weight;
  return launch_kv8_weights(a, args->dtype, (cudaStream_t)stream) ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status ssd_kv8_evict(const ssd_kv8_cache* from, const ssd_kv8_cache* to, const ssd_kv8_evict_args* p,
                         void* stream) {
  Kv8View src, dst;
  if (!view_of(from, &src) || !view_of(to, &dst) || !p) return SSD_ERR_INVALID_ARG;
  if (src.n_kv != dst.n_kv || src.hd != dst.hd) return SSD_ERR_INVALID_ARG;
  if (!aligned(p->weight, 4) || !aligned(p->index, 4) || (p->kept_weight && !aligned(p->kept_weight, 4)))
    return SSD_ERR_INVALID_ARG;
  if (p->n < 1 || (int64_t)p->n > (int64_t)from->n_pages * kPage || p->keep < 1 || p->keep > p->n || p->recent < 0 ||
      p->recent > p->keep || p->ld_weight < p->n)
    return SSD_ERR_INVALID_ARG;
  if (src.k == dst.k && src.btab == dst.btab) return SSD_ERR_INVALID_ARG;  // onto itself
  if ((int64_t)p->keep > (int64_t)to->n_pages * kPage) return SSD_ERR_CAPACITY;
  Kv8SelectArgs a{};
  a.weight = p->weight;
  a.ld_weight = (size_t)p->ld_weight;
  a.n = p->n;
  a.keep = p->keep;
  a.recent = p->recent;
  a.index = p->index;
  a.kept_weight = p->kept_weight;
  return launch_kv8_evict(src, dst, a, (cudaStream_t)stream) ? SSD_OK : SSD_ERR_CUDA;
}
