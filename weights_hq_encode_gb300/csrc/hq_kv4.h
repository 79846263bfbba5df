// hq_kv4.h -- arguments of the 4-bit window cache's kernels, shared by their
// launchers and the C ABI, and the cache's addressing.
#pragma once
#include "../../include/hq_kv4.h"
#include "hq_internal.h"

namespace hq {

constexpr int kUnit = HQ_KV4_UNIT;               // tokens of a unit
constexpr int kUnitBytes = HQ_KV4_UNIT_BYTES;
// Byte offsets inside a unit: K codes [16 tokens][64], V codes [8 token
// pairs][8 chunks of 16 dimensions][2 tokens][8], K scales [16] bf16, V
// scales [16] bf16.  Dimension d of a row is the low (even d) or high nibble
// of its byte d / 2.
constexpr int kUnitV = 1024, kUnitKs = 2048, kUnitVs = 2080;

struct Kv4View {
  unsigned char *pages;
  int64_t n_pages;
  int page_tokens, page_units;
  int page_shift;           // log2(page_tokens) when a power of two, else -1
  int n_kv;
  int kv_shift;             // log2(n_kv) likewise
  const int32_t *table;     // [n_seqs][width] page numbers
  int n_seqs, width;
  const uint32_t *signs;    // 128-bit sign mask
  __host__ __device__ int64_t capacity() const { return (int64_t)width * page_tokens; }
};

// Rows of K and V entering or leaving the cache: element strides between
// tokens and between heads, the 128 values of a row contiguous.
struct Kv4Rows {
  const void *k, *v;
  int64_t k_token, k_head, v_token, v_head;
  int kind;                 // HQ_T_*
  int vec;                  // every row starts on a 16-byte boundary
};

struct Kv4RowArgs {
  Kv4View c;
  Kv4Rows rows;
  const int32_t *seq, *pos; // [n_tokens]
  int64_t n_tokens;
  uint32_t *status;
};

struct Kv4AttnArgs {
  Kv4View c;
  const int32_t *lengths;   // [n_seqs]
  const void *q;
  int64_t q_seq, q_token, q_head;
  int kind, out_kind;
  int q_vec;
  int q_len, Hq, G, R;      // G query heads a KV head, R = q_len * G rows a KV head
  float scale;              // softmax scale
  float cap, cap_l2, by_cap;   // cap of the scores (0: none), times log2(e), and 1 / cap
  void *out;                // [n_seqs][q_len][Hq][128]
  float *lse;               // [n_seqs][q_len][Hq] or nullptr
  const float *mass_in;     // [n_seqs][n_kv][capacity] or nullptr
  float *mass_out;          // the same, or nullptr: no mass
  int whole;                // set by the launch: a block a (sequence, head, row tile), no joins
  int by_pair;              // likewise: joins are kept a (sequence, head, row tile), not a block
  int row_tiles;            // tiles of rows a KV head has
  float *part;              // workspace: sums that several blocks share
  float *stat;              // workspace: their references and sums of weights
  int *joins;               // workspace: what is left to be joined
  float *z;                 // workspace [n_seqs][n_kv][R][capacity] when mass is wanted
  float2 *row_stat;         // workspace [n_seqs][n_kv][R]: a row's reference and log2 of its sum beside it
  uint32_t *status;
};

struct Kv4EvictArgs {
  Kv4View src, dst;
  const int32_t *lengths;
  const float *mass;        // [n_seqs][n_kv][src capacity]
  int budget, recent;
  int32_t *kept;            // [n_seqs][n_kv][budget]
  int32_t *new_lengths;     // [n_seqs]
  float *new_mass;          // [n_seqs][n_kv][dst capacity]
  uint32_t *status;
};

constexpr int kKv4MaxBlocks = 1024;              // most blocks of one attention launch
int kv4_row_tiles(int R);
size_t kv4_part_bytes(int R);
size_t kv4_stat_bytes(int R);
size_t kv4_join_bytes();

int launch_kv4_append(const Kv4RowArgs &a, cudaStream_t st);
int launch_kv4_read(const Kv4RowArgs &a, cudaStream_t st);
int launch_kv4_attention(const Kv4AttnArgs &a, cudaStream_t st);
int launch_kv4_evict(const Kv4EvictArgs &a, cudaStream_t st);

#ifdef __CUDACC__
// x / y of nonnegative x and positive y, by a 32-bit division where it fits or a shift (>= 0).
__device__ __forceinline__ int64_t kv4_divide(int64_t x, int64_t y, int shift = -1) {
  if (shift >= 0) return x >> shift;
  return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}
// The place of (sequence, position, head): 16 x its unit's number in the pool +
// its token in the unit, or kNoPlace where there is no such position or the
// table names none of the pool's pages.
constexpr uint32_t kNoPlace = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t kv4_place(const Kv4View &c, int seq, int pos, int h) {
  if (seq >= c.n_seqs || pos < 0 || pos >= c.capacity()) return kNoPlace;
  const int j = (int)kv4_divide(pos, c.page_tokens, c.page_shift), in_page = pos - j * c.page_tokens;
  const int page = c.table[(int64_t)seq * c.width + j];
  if (page < 0 || page >= c.n_pages) return kNoPlace;
  return (uint32_t)((page * c.n_kv + h) * c.page_units + in_page / kUnit) * kUnit + (uint32_t)(in_page % kUnit);
}
__device__ __forceinline__ unsigned char *kv4_unit(const Kv4View &c, uint32_t place) {
  return c.pages + (int64_t)(place / kUnit) * kUnitBytes;
}
// A sequence's length, held to [0, capacity]; *bad when it was outside.
__device__ __forceinline__ int kv4_length(const Kv4View &c, const int32_t *lengths, int seq, bool *bad) {
  const int n = lengths[seq], cap = c.width * c.page_tokens;
  *bad = n < 0 || n > cap;
  return n < 0 ? 0 : n > cap ? cap : n;
}
__device__ __forceinline__ float bf16_to_f32(uint32_t bits) { return __uint_as_float(bits << 16); }
#endif

}  // namespace hq
