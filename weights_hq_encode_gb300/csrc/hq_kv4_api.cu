// hq_kv4_api.cu -- host entry points of the 4-bit window cache's C ABI
// (include/hq_kv4.h): argument checks and workspace layout.
#include <cmath>
#include <cstring>

#include <cuda_runtime.h>

#include "hq_kv4.h"

namespace {

using namespace hq;

constexpr int64_t kMaxCapacity = (int64_t)1 << 30;
// so that 1 / cap and cap log2(e) are normal numbers, and scale log2(e) is finite
constexpr float kMinCap = 0x1p-20f, kMaxCap = 0x1p120f, kMaxScale = 0x1p120f;

bool aligned(const void *ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }
size_t round256(size_t v) { return (v + 255) / 256 * 256; }
bool kind_ok(int k) { return k == HQ_T_BF16 || k == HQ_T_F32 || k == HQ_T_F16; }
size_t size_of(int k) { return k == HQ_T_F32 ? 4 : 2; }

// The sizes of a cache; its pointers are looked at only by cache_ok.
bool sizes_ok(const hq_kv4_cache *c) {
  return c && c->n_pages > 0 && c->n_pages <= INT32_MAX && c->page_tokens > 0 &&
         c->page_tokens % HQ_KV4_UNIT == 0 && c->n_kv_heads > 0 && c->n_kv_heads <= 65535 &&
         c->n_seqs >= 0 && c->n_seqs <= 65535 && c->table_width >= 0 &&
         (int64_t)c->table_width * c->page_tokens <= kMaxCapacity &&
         // 16 x a unit's number in the pool fits 32 bits
         c->n_pages < (1 << 28) / c->n_kv_heads / (c->page_tokens / HQ_KV4_UNIT);
}

bool cache_ok(const hq_kv4_cache *c) {
  return sizes_ok(c) && c->d_pages && aligned(c->d_pages, 16) &&
         ((int64_t)c->n_seqs * c->table_width == 0 || c->d_table) && aligned(c->d_table, 4) &&
         c->d_signs && aligned(c->d_signs, 4);
}

Kv4View view_of(const hq_kv4_cache *c) {
  Kv4View v;
  v.pages = static_cast<unsigned char *>(c->d_pages);
  v.n_pages = c->n_pages;
  v.page_tokens = c->page_tokens;
  v.page_units = c->page_tokens / HQ_KV4_UNIT;
  v.page_shift = pow2_shift(c->page_tokens);
  v.n_kv = c->n_kv_heads;
  v.kv_shift = pow2_shift(c->n_kv_heads);
  v.table = c->d_table;
  v.n_seqs = c->n_seqs;
  v.width = c->table_width;
  v.signs = c->d_signs;
  return v;
}

// Whether a row's 16-byte pieces may be moved whole: base and strides on
// 16-byte boundaries.
bool whole(const void *p, size_t size, int64_t s0, int64_t s1) {
  return aligned(p, 16) && (s0 * (int64_t)size) % 16 == 0 && (s1 * (int64_t)size) % 16 == 0;
}

int rows_call(const hq_kv4_cache *c, const void *k, const void *v, int kind, int64_t k_token,
              int64_t k_head, int64_t v_token, int64_t v_head, const int32_t *d_seq,
              const int32_t *d_pos, int64_t n_tokens, uint32_t *d_status, hq_stream_t stream,
              int (*launch)(const Kv4RowArgs &, cudaStream_t)) {
  if (!cache_ok(c) || !kind_ok(kind) || n_tokens < 0 || !d_status) return HQ_ERR_INVALID;
  if (n_tokens == 0) return HQ_OK;
  if (!k || !v || !d_seq || !d_pos || !aligned(k, size_of(kind)) || !aligned(v, size_of(kind)))
    return HQ_ERR_INVALID;
  if (n_tokens > ((int64_t)1 << 34) / c->n_kv_heads) return HQ_ERR_INVALID;   // grid of 2^29 blocks
  Kv4RowArgs a;
  a.c = view_of(c);
  a.rows = Kv4Rows{k, v, k_token, k_head, v_token, v_head, kind, 0};
  a.rows.vec = whole(k, size_of(kind), k_token, k_head) && whole(v, size_of(kind), v_token, v_head);
  a.seq = d_seq;
  a.pos = d_pos;
  a.n_tokens = n_tokens;
  a.status = d_status;
  return launch(a, reinterpret_cast<cudaStream_t>(stream)) == 0 ? HQ_OK : HQ_ERR_CUDA;
}

struct AttnSizes {
  size_t part = 0, stat = 0, joins = 0, z = 0, row_stat = 0;
  size_t total() const { return part + stat + joins + z + row_stat; }
};

bool attn_sizes(const hq_kv4_cache *c, int q_len, int Hq, int want_mass, AttnSizes *s) {
  if (!sizes_ok(c) || q_len <= 0 || q_len > 65535 || Hq <= 0 || Hq % c->n_kv_heads != 0) return false;
  const int64_t rows = (int64_t)c->n_seqs * q_len * Hq;
  if ((int64_t)q_len * (Hq / c->n_kv_heads) > (1 << 24) || rows > ((int64_t)1 << 31)) return false;
  s->part = round256(kv4_part_bytes(q_len * (Hq / c->n_kv_heads)));
  s->stat = round256(kv4_stat_bytes(q_len * (Hq / c->n_kv_heads)));
  s->joins = round256(kv4_join_bytes());
  if (want_mass) {
    const size_t cap = (size_t)c->table_width * c->page_tokens;
    if (cap != 0 && (size_t)rows > ((size_t)1 << 44) / cap) return false;
    s->z = round256((size_t)rows * cap * sizeof(float));
    s->row_stat = round256((size_t)rows * sizeof(float2));
  }
  return true;
}

}  // namespace

extern "C" {

size_t hq_kv4_page_bytes(int n_kv_heads, int page_tokens) {
  if (n_kv_heads <= 0 || page_tokens <= 0 || page_tokens % HQ_KV4_UNIT != 0) return 0;
  return (size_t)n_kv_heads * (page_tokens / HQ_KV4_UNIT) * HQ_KV4_UNIT_BYTES;
}

int hq_kv4_append(const hq_kv4_cache *c, const void *d_k, const void *d_v, int kind,
                  int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                  int64_t v_head_stride, const int32_t *d_seq, const int32_t *d_pos,
                  int64_t n_tokens, uint32_t *d_status, hq_stream_t stream) {
  return rows_call(c, d_k, d_v, kind, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                   d_seq, d_pos, n_tokens, d_status, stream, hq::launch_kv4_append);
}

int hq_kv4_read(const hq_kv4_cache *c, const int32_t *d_seq, const int32_t *d_pos,
                int64_t n_tokens, void *d_k, void *d_v, int kind, int64_t k_token_stride,
                int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                uint32_t *d_status, hq_stream_t stream) {
  return rows_call(c, d_k, d_v, kind, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                   d_seq, d_pos, n_tokens, d_status, stream, hq::launch_kv4_read);
}

size_t hq_kv4_attention_workspace_bytes(const hq_kv4_cache *c, int q_len, int Hq, int want_mass) {
  AttnSizes s;
  return attn_sizes(c, q_len, Hq, want_mass, &s) ? s.total() : 0;
}

int hq_kv4_attention(const hq_kv4_cache *c, const int32_t *d_lengths, const void *d_q, int q_kind,
                     int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride,
                     int q_len, int Hq, float scale, float cap, void *d_out, int out_kind,
                     float *d_lse, const float *d_mass_in, float *d_mass_out, void *d_ws,
                     size_t ws_bytes, uint32_t *d_status, hq_stream_t stream) {
  AttnSizes s;
  if (!cache_ok(c) || !kind_ok(q_kind) || !kind_ok(out_kind) || !d_status || !(std::fabs(scale) <= kMaxScale) ||
      !(cap == 0.0f || (cap >= kMinCap && cap <= kMaxCap)) || (d_mass_in && !d_mass_out) ||
      !attn_sizes(c, q_len, Hq, d_mass_out != nullptr, &s))
    return HQ_ERR_INVALID;
  if (c->n_seqs == 0) return HQ_OK;
  if (!d_lengths || !d_q || !d_out || !d_ws || ws_bytes < s.total() || !aligned(d_ws, 256) ||
      !aligned(d_out, 16) || !aligned(d_q, size_of(q_kind)) || !aligned(d_lse, 4) ||
      !aligned(d_mass_in, 4) || !aligned(d_mass_out, 4))
    return HQ_ERR_INVALID;
  Kv4AttnArgs a;
  a.c = view_of(c);
  a.lengths = d_lengths;
  a.q = d_q;
  a.q_seq = q_seq_stride;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.kind = q_kind;
  a.out_kind = out_kind;
  a.q_vec = whole(d_q, size_of(q_kind), q_token_stride, q_head_stride) &&
            (q_seq_stride * (int64_t)size_of(q_kind)) % 16 == 0;
  a.q_len = q_len;
  a.Hq = Hq;
  a.G = Hq / c->n_kv_heads;
  a.R = q_len * a.G;
  a.scale = scale;
  a.cap = cap;
  a.cap_l2 = cap * 1.4426950408889634f;
  a.by_cap = cap > 0.0f ? 1.0f / cap : 0.0f;
  a.out = d_out;
  a.lse = d_lse;
  a.mass_in = d_mass_in;
  a.mass_out = d_mass_out;
  char *ws = static_cast<char *>(d_ws);
  a.row_tiles = kv4_row_tiles(a.R);
  a.part = reinterpret_cast<float *>(ws);
  ws += s.part;
  a.stat = reinterpret_cast<float *>(ws);
  ws += s.stat;
  a.joins = reinterpret_cast<int *>(ws);
  ws += s.joins;
  a.z = reinterpret_cast<float *>(ws);
  a.row_stat = reinterpret_cast<float2 *>(ws + s.z);
  a.status = d_status;
  return hq::launch_kv4_attention(a, reinterpret_cast<cudaStream_t>(stream)) == 0 ? HQ_OK : HQ_ERR_CUDA;
}

int hq_kv4_evict(const hq_kv4_cache *src, const int32_t *d_lengths, const float *d_mass,
                 const hq_kv4_cache *dst, int budget, int recent, int32_t *d_kept,
                 int32_t *d_new_lengths, float *d_new_mass, uint32_t *d_status,
                 hq_stream_t stream) {
  if (!cache_ok(src) || !cache_ok(dst) || !d_status || budget < 1 ||
      budget > kMaxCapacity || recent < 0 || recent > budget ||
      src->n_seqs != dst->n_seqs || src->n_kv_heads != dst->n_kv_heads)
    return HQ_ERR_INVALID;
  if (src->n_seqs == 0) return HQ_OK;
  const int64_t cap = (int64_t)src->table_width * src->page_tokens;
  const int64_t dcap = (int64_t)dst->table_width * dst->page_tokens;
  if (dcap < (budget < cap ? budget : cap) || !d_lengths || !d_kept || !d_new_lengths ||
      (cap > 0 && (!d_mass || !d_new_mass || src->d_table == dst->d_table || d_new_mass == d_mass)) ||
      d_new_lengths == d_lengths)
    return HQ_ERR_INVALID;
  if (!aligned(d_mass, 4) || !aligned(d_new_mass, 4) || !aligned(d_kept, 4) ||
      !aligned(d_lengths, 4) || !aligned(d_new_lengths, 4))
    return HQ_ERR_INVALID;
  Kv4EvictArgs a;
  a.src = view_of(src);
  a.dst = view_of(dst);
  a.lengths = d_lengths;
  a.mass = d_mass;
  a.budget = budget;
  a.recent = recent;
  a.kept = d_kept;
  a.new_lengths = d_new_lengths;
  a.new_mass = d_new_mass;
  a.status = d_status;
  return hq::launch_kv4_evict(a, reinterpret_cast<cudaStream_t>(stream)) == 0 ? HQ_OK : HQ_ERR_CUDA;
}

}  // extern "C"
