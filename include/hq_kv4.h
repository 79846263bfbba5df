/*
 * hq_kv4.h -- C ABI of the paged 4-bit window cache of the GB300 (sm_103a)
 * HyperQuant library: the part of a KV cache that a serving loop still
 * appends to, attends to token by token and drops tokens from, beside the
 * entropy-coded streams of hq.h, which are written once and hold what no
 * longer changes.
 *
 * Format.  A token of one KV head is one 128-wide tile of the codec (Method 1:
 * the randomized Hadamard transform), at a fixed rate:
 *   y = H D x / sqrt(128)           D the diagonal of the sign mask
 *   s = bf16(max |y| / 7.5)         one scale a tile, round to nearest even
 *   c = min(max(floor(y / s + 8), 0), 15),   value (c - 7.5) s
 * The transform spreads a row's outliers over its 128 coordinates, so that
 * one scale and 16 uniform levels serve the whole tile.  A tile with a
 * non-finite value, or whose H D x overflows fp32, is stored as zeros
 * (HQ_ERR_RANGE); one whose s would be below 2^-126 is stored as zeros too.
 *
 * Layout.  16 tokens of one KV head form a unit of 2112 contiguous bytes:
 *   0     K codes, [16 tokens][64 bytes]
 *   1024  V codes, [8 token pairs][8 chunks of 16 dimensions][2 tokens][8 bytes]
 *   2048  K scales, [16] bf16;  2080  V scales, [16] bf16
 * Dimension d of a row is the low (even d) or high (odd d) nibble of byte
 * d / 2.  A page is [n_kv_heads][page_tokens / 16] units, the pool is
 * [n_pages] pages.  Position t of sequence b is token t % page_tokens of page
 * d_table[b][t / page_tokens].  Sequences may share pages that none of them
 * writes.
 *
 * Conventions are those of hq.h: the caller owns every buffer, nothing is
 * allocated or kept between calls, every call is asynchronous on `stream`
 * and can be captured into a graph, and the return value reports argument
 * errors (HQ_ERR_INVALID, nothing launched) and failed launches
 * (HQ_ERR_CUDA).  Every tensor lies on the current device.
 */
#ifndef HQ_KV4_H_
#define HQ_KV4_H_

#include "hq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* OR-ed into *d_status beside the bits of hq.h: a sequence number, position,
 * length or page number outside its range.  What it names is left out: a row
 * is not written (append, evict) or reads as zeros (read), a page's tokens
 * get no weight (attention), a length counts as the nearest valid one. */
enum { HQ_ERR_PAGE = 64 };

/* Element types of the rows that enter and leave the cache. */
enum { HQ_T_BF16 = 0, HQ_T_F32 = 1, HQ_T_F16 = 2 };

#define HQ_KV4_UNIT 16
#define HQ_KV4_UNIT_BYTES 2112
#define HQ_KV4_MAX_DRAFTS 256      /* drafted tokens of a sequence in one tree */
#define HQ_KV4_MAX_RESIZE 16384    /* sequences of one hq_kv4_resize call */

/* A pool of pages and the block table through which a call sees it.
 *   d_pages       [n_pages][n_kv_heads][page_tokens / 16][2112] bytes, 16-byte
 *                 aligned; n_pages >= 1
 *   page_tokens   a positive multiple of 16
 *   d_table       [n_seqs][table_width] int32 page numbers; entries past a
 *                 sequence's length are not read
 *   d_signs       [4] uint32: the sign mask of every tile (hq_make_layer_signs)
 * table_width * page_tokens, a sequence's capacity, is at most 2^30, and the
 * pool holds fewer than 2^28 units (567 GB). */
typedef struct hq_kv4_cache {
  void *d_pages;
  int64_t n_pages;
  int32_t page_tokens;
  int32_t n_kv_heads;
  const int32_t *d_table;
  int32_t n_seqs;
  int32_t table_width;
  const uint32_t *d_signs;
} hq_kv4_cache;

/* Bytes of one page, 0 for invalid sizes. */
size_t hq_kv4_page_bytes(int n_kv_heads, int page_tokens);

/* Writes K and V rows of new tokens into the cache (prompt rows as well as
 * one token a sequence).
 *   d_k, d_v    row (i, h) starts at element i * token_stride + h * head_stride
 *               of its tensor, its 128 values contiguous; kind: HQ_T_*
 *   d_seq       [n_tokens] int32: the token's sequence; negative: a padding
 *               token, skipped
 *   d_pos       [n_tokens] int32: its position in the sequence
 * Two tokens of a call may not name the same place.  d_status is OR-ed with
 * HQ_ERR_RANGE and HQ_ERR_PAGE. */
int hq_kv4_append(const hq_kv4_cache *c, const void *d_k, const void *d_v, int kind,
                  int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                  int64_t v_head_stride, const int32_t *d_seq, const int32_t *d_pos,
                  int64_t n_tokens, uint32_t *d_status, hq_stream_t stream);

/* Gives rows of the cache back as the values they stand for,
 * D H (c - 7.5) s / sqrt(128) rounded to `kind`.  Arguments as for
 * hq_kv4_append, d_k and d_v being written (no two rows overlap; a token may be
 * read more than once); padding tokens' rows are left as
 * they were, rows that HQ_ERR_PAGE names become zeros.  With the head stride
 * of [n_kv_heads][tokens][128] the rows are a slab for hq_encode. */
int hq_kv4_read(const hq_kv4_cache *c, const int32_t *d_seq, const int32_t *d_pos,
                int64_t n_tokens, void *d_k, void *d_v, int kind, int64_t k_token_stride,
                int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                uint32_t *d_status, hq_stream_t stream);

/* Bytes of device workspace hq_kv4_attention needs (0 for invalid sizes): at
 * most 18 MB without mass.  With it, 4 bytes more for every query row and position
 * that the table has room for, n_seqs * q_len * Hq * table_width * page_tokens,
 * whatever the lengths. */
size_t hq_kv4_attention_workspace_bytes(const hq_kv4_cache *c, int q_len, int Hq, int want_mass);

/* Attention of the last q_len tokens of every sequence over its cache, read
 * straight from the codes: with h = hq / (Hq / n_kv_heads) and L the
 * sequence's length, query token j sees the tokens t <= L - q_len + j:
 *   z = scale * q . Khat[t]       capped to cap * tanh(z / cap) when cap > 0
 *   p = softmax of z over the tokens seen,   out = sum p Vhat[t]
 *   lse = log sum exp z
 *   mass_out[b][h][t] = mass_in[b][h][t] + the sum of p over h's query rows
 * A row that sees no token gets zeros and lse -inf.  Scores, weights and sums
 * are held in fp32; the contractions run on fp16 tensor-core operands, each
 * query value and each weight split into two fp16 parts (|x - hi - lo| <=
 * 2^-22 |x| + 2^-25 of the row's power-of-two scale), the codes being exact
 * in fp16: an fp32-level result.  The order of all sums is fixed.  Scores may
 * be of any size: a row stays a weighted mean of V's rows, with weights that
 * add up to 1, while |q|, |scale| |q| and |scale| |q| |Khat| (norms) are below
 * 2^110; beyond, and for a query that is not finite, that row may come out
 * non-finite.  The cache is streamed once for every 16 query rows of a KV
 * head, q_len * Hq / n_kv_heads: made for one to some tens of new tokens.
 *   d_lengths   [n_seqs] int32, the new tokens included
 *   d_q         row (b, j, hq) starts at element b * q_seq_stride +
 *               j * q_token_stride + hq * q_head_stride; kind q_kind
 *   scale       at most 2^120 in magnitude; cap 0 (none) or 2^-20 .. 2^120
 *   d_out       [n_seqs][q_len][Hq][128] of out_kind, 16-byte aligned
 *   d_lse       [n_seqs][q_len][Hq] fp32, or NULL
 *   d_mass_in   [n_seqs][n_kv_heads][table_width * page_tokens] fp32, or NULL: zeros
 *   d_mass_out  the same, NULL: no mass; may be d_mass_in.  Entries from a
 *               sequence's length on are left as they were.
 *   d_ws        >= hq_kv4_attention_workspace_bytes(), 256-byte aligned; calls
 *               that may overlap need workspaces of their own
 * d_status is OR-ed with HQ_ERR_PAGE. */
int hq_kv4_attention(const hq_kv4_cache *c, const int32_t *d_lengths, const void *d_q, int q_kind,
                     int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride,
                     int q_len, int Hq, float scale, float cap, void *d_out, int out_kind,
                     float *d_lse, const float *d_mass_in, float *d_mass_out, void *d_ws,
                     size_t ws_bytes, uint32_t *d_status, hq_stream_t stream);

/* Eviction by accumulated attention weight: of a sequence longer than
 * `budget`, each KV head keeps its last `recent` tokens and the
 * budget - recent others of the largest mass (equal masses: the lower
 * position; a NaN counts as the least value, -0 as 0), in order; a shorter
 * sequence is kept whole.  The rows are written, codes unchanged, to the
 * pages of `dst`, which must not be pages of src's sequences; src stays as it
 * was.
 *   d_mass         [n_seqs][n_kv_heads][src capacity] fp32
 *   dst            n_seqs, n_kv_heads and signs of src; capacity >= min(budget,
 *                  src capacity)
 *   budget         1 .. 2^30; recent: 0 .. budget
 *   d_kept         [n_seqs][n_kv_heads][budget] int32: the positions kept,
 *                  then -1
 *   d_new_lengths  [n_seqs] int32: min(length, budget)
 *   d_new_mass     [n_seqs][n_kv_heads][dst capacity] fp32: the kept tokens'
 *                  mass; entries from the new length on are left as they were
 * d_kept, d_new_lengths and d_new_mass overlap no input (new lengths or masses
 * in the place of the old ones are refused).  d_status is OR-ed
 * with HQ_ERR_PAGE; what d_kept, d_new_lengths and d_new_mass count then
 * includes rows that were left out of dst, so dst is not to be used. */
int hq_kv4_evict(const hq_kv4_cache *src, const int32_t *d_lengths, const float *d_mass,
                 const hq_kv4_cache *dst, int budget, int recent, int32_t *d_kept,
                 int32_t *d_new_lengths, float *d_new_mass, uint32_t *d_status,
                 hq_stream_t stream);

/* Gives sequences the pages that new lengths need, takes back those that
 * they leave, and lists the new tokens: a step's block table and slot map.
 * Sequence b has ceil(lengths[b] / page_tokens) pages and is to have
 * ceil(wanted[b] / page_tokens).
 *   - Pages given back go behind the free list's end, the first of them (by
 *     sequence, then place) last; their entries in the table stay as they were.
 *   - Pages taken come from the list's end then, in the order of sequence and
 *     place, and are written to c's table, which this call alone changes.  So a
 *     call that only grows sequences and the one that takes it back leave the
 *     list as it was.
 *   - A sequence that needs pages keeps its length when it and all before it
 *     that need some want more than there are, those given back included
 *     (HQ_ERR_CAPACITY).
 *   d_lengths, d_wanted  [n_seqs] int32; a length outside 0 .. capacity counts
 *                  as the nearest valid one (HQ_ERR_PAGE)
 *   d_free, d_n_free  [n_pages] int32 page numbers and their count, changed in
 *                  place; pages in sequences that shrink may not be shared
 *   d_new_lengths  [n_seqs] int32: wanted[b], or lengths[b] where it was refused;
 *                  neither of the two inputs
 *   d_starts       [n_seqs + 1] int32, or NULL: where each sequence's new tokens
 *                  begin in the lists, and their number (at most 2^31 - 1)
 *   d_seq, d_pos   [max_tokens] int32, or both NULL with max_tokens 0: sequence and
 *                  position of the new tokens, sequence by sequence, as
 *                  hq_kv4_append takes them; then -1 and 0.  More than max_tokens:
 *                  HQ_ERR_CAPACITY, the rest is not listed
 * n_seqs is at most HQ_KV4_MAX_RESIZE.  A page number outside the pool in the list or
 * in a place given back sets HQ_ERR_PAGE and is passed on as it is.  d_pages is not
 * looked into. */
int hq_kv4_resize(const hq_kv4_cache *c, const int32_t *d_lengths, const int32_t *d_wanted,
                  int32_t *d_free, int32_t *d_n_free, int32_t *d_new_lengths, int32_t *d_starts,
                  int32_t *d_seq, int32_t *d_pos, int64_t max_tokens, uint32_t *d_status,
                  hq_stream_t stream);

/* Bytes of device workspace hq_kv4_tree_attention needs (0 for invalid sizes). */
size_t hq_kv4_tree_attention_workspace_bytes(const hq_kv4_cache *c, int q_len, int Hq);

/* Attention of a tree of drafted tokens behind each sequence's committed ones:
 * draft j of sequence b is token lengths[b] + j of its cache (appended before
 * this call) and sees the lengths[b] committed tokens, its ancestors in the
 * tree, and itself.  Formulas and types are those of hq_kv4_attention, lse and
 * out likewise, and so is the precision, but for outputs of 16 bits with more than
 * 32 rows a KV head, q_len * Hq / n_kv_heads, over tables with room for many tokens:
 * their weights are rounded once to fp16, by at most 2^-11 of them and 2^-31 of the
 * row's largest weight times the largest of V's scales.
 *   d_lengths   [n_seqs] int32: committed tokens, without the drafts
 *   d_parents   [n_seqs][q_len] int32: the draft that j follows, below j; -1: the
 *               last committed token; -2: j is padding.  Padding gets zeros and lse
 *               -inf, its place in the cache is not looked at.  Other values
 *               count as -2 and set HQ_ERR_PAGE, as do drafts behind padding and
 *               drafts past the capacity (which get and give no weight)
 *   q_len       1 .. HQ_KV4_MAX_DRAFTS drafts a sequence, padding included
 *   d_ws        >= hq_kv4_tree_attention_workspace_bytes(), 256-byte aligned; calls
 *               that may overlap need workspaces of their own
 * The other arguments are those of hq_kv4_attention. */
int hq_kv4_tree_attention(const hq_kv4_cache *c, const int32_t *d_lengths, const int32_t *d_parents,
                          const void *d_q, int q_kind, int64_t q_seq_stride,
                          int64_t q_token_stride, int64_t q_head_stride, int q_len, int Hq,
                          float scale, float cap, void *d_out, int out_kind, float *d_lse,
                          void *d_ws, size_t ws_bytes, uint32_t *d_status, hq_stream_t stream);

/* Keeps the accepted path of each sequence's tree: the row of draft path[b][i],
 * at position lengths[b] + path[b][i], moves to position lengths[b] + i, codes
 * and scales unchanged; other rows stay as they were.
 *   d_path         [n_seqs][max_path] int32: drafts in ascending order, then -1.  A
 *                  path ends at its first negative entry; one that does not ascend
 *                  or leads past the capacity ends there too, with HQ_ERR_PAGE
 *   d_new_lengths  [n_seqs] int32: lengths[b] + the path's length; not d_lengths
 * A row whose old or new place has no valid page is not moved (HQ_ERR_PAGE).  The
 * pages of the drafts are not shared between sequences. */
int hq_kv4_accept(const hq_kv4_cache *c, const int32_t *d_lengths, const int32_t *d_path,
                  int max_path, int32_t *d_new_lengths, uint32_t *d_status, hq_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif  /* HQ_KV4_H_ */
