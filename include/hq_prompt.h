/*
 * hq_prompt.h -- C ABI of the attention over whole prompts of the GB300
 * (sm_103a) HyperQuant library: what a serving loop computes from a prompt's
 * K and V rows before it appends them to the 4-bit window cache (hq_kv4.h) or
 * encodes them (hq.h).
 *
 * Conventions are those of hq.h: the caller owns every buffer, nothing is
 * allocated or kept between calls, every call is asynchronous on `stream`
 * and can be captured into a graph, and the return value reports argument
 * errors (HQ_ERR_INVALID, nothing launched) and failed launches
 * (HQ_ERR_CUDA).  Every tensor lies on the current device.
 */
#ifndef HQ_PROMPT_H_
#define HQ_PROMPT_H_

#include "hq_kv4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of device workspace hq_prompt_attention needs (0 for invalid sizes): 48 for
 * every 128 query rows and pair of heads, and, for calls of few rows, whose keys
 * may be split, 43 MB. */
size_t hq_prompt_attention_workspace_bytes(int n_seqs, int64_t n_tokens, int Hq, int n_kv_heads);

/* Causal attention of packed sequences, heads grouped.  Sequence b has the
 * query rows starts[b] .. starts[b + 1] - 1 and the K and V rows k_starts[b] ..
 * k_starts[b + 1] - 1, of which its query rows' own are the last: with n query
 * and m + n K rows, query row i sees the K rows 0 .. m + i of its sequence
 * (m > 0: earlier tokens, read back from a cache; m < 0: the first -m rows see
 * nothing).  For h = hq / (Hq / n_kv_heads):
 *   z = scale * q . K[t]          capped to cap * tanh(z / cap) when cap > 0
 *   p = softmax of z over the rows seen,   out = sum p V[t],   lse = log sum exp z
 * A row that sees nothing gets zeros and lse -inf.  Scores, weights and sums
 * are held in fp32; the products run on the tensor cores with fp32 sums, for
 * which each weight is rounded once to the inputs' type, as the tensor cores take
 * it: by at most half a step (bf16 2^-8, fp16 2^-11 of it), and in fp16 by up
 * to 2^-35 of the row's largest weight (2^-25 where scores pass 10^7).  The order of
 * all sums is fixed.  Rows before starts[0] and behind the last
 * sequence are left as they were.  K and V of a sequence are to be finite:
 * a value that is not reaches rows of the same sequence up to 127 before its
 * own, but no other sequence.  In bf16 the magnitudes of V that a row sees are to come to
 * less than 2^96 in every dimension (beyond, that row may come out non-finite), and parts of
 * an output below 2^-96 may be lost.
 *   d_starts     [n_seqs + 1] int32, ascending, at most n_tokens
 *   d_k_starts   the same for K and V, at most n_k_tokens; NULL: d_starts, and
 *                n_k_tokens must be n_tokens
 *   d_q          row (i, hq) starts at element i * q_token_stride + hq *
 *                q_head_stride, its 128 values contiguous; n_tokens rows
 *   d_k, d_v     likewise, n_k_tokens rows; all three 16-byte aligned, their
 *                strides positive multiples of 8 (not looked at for a single
 *                token or head)
 *   kind         HQ_T_BF16 or HQ_T_F16: of q, k, v and out
 *   scale        at most 2^120 in magnitude; cap 0 (none) or 2^-20 .. 2^120
 *   d_out        [n_tokens][Hq][128], 16-byte aligned
 *   d_lse        [n_tokens][Hq] fp32, or NULL
 *   d_ws         >= hq_prompt_attention_workspace_bytes(), 256-byte aligned;
 *                calls that may overlap need workspaces of their own
 * q . K[t] and scale * q . K[t] are to be finite in fp32.  n_seqs, n_kv_heads and
 * Hq are at most 65535, n_tokens and n_k_tokens below 2^31 - 1024, and so are the
 * 128-row tiles of all heads.  *d_status is OR-ed with HQ_ERR_PAGE for starts
 * outside their range or not ascending: they count as the nearest valid ones, and what
 * the rows of such sequences get is not defined; nor is any row's where the sequences
 * come to more 128-row tiles than n_tokens rows can have. */
int hq_prompt_attention(const int32_t *d_starts, const int32_t *d_k_starts, int n_seqs,
                        const void *d_q, int64_t q_token_stride, int64_t q_head_stride,
                        int64_t n_tokens, int Hq, const void *d_k, int64_t k_token_stride,
                        int64_t k_head_stride, const void *d_v, int64_t v_token_stride,
                        int64_t v_head_stride, int64_t n_k_tokens, int n_kv_heads, int kind,
                        float scale, float cap, void *d_out, float *d_lse, void *d_ws,
                        size_t ws_bytes, uint32_t *d_status, hq_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif  /* HQ_PROMPT_H_ */
