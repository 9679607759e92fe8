/*
 * moe_decode.h -- the operators around the MoE layer in a decode or verify step: the residual addition with
 * its root-mean-square norm, the paged key-value cache (its writer and the attention that reads it), and the
 * whole MoE layer for a few tokens in one kernel.
 *
 * A decoder block of one step, T = n_seqs * L rows (L new tokens of every request; L = 8 in the verify batch of
 * 64 requests x 8 rows that moe.h describes):
 *   moe_add_rms_norm -> (q, k, v projections) -> moe_kv_append -> moe_paged_attention -> (output projection)
 *   -> moe_add_rms_norm -> moe_forward, or moe_forward_few for up to MOE_FEW_MAX_T rows.
 *
 * The conventions of moe.h hold: device pointers, asynchronous on `stream`, no allocation inside a call, the
 * returned status covers host-side checks and launch errors.  Strides are counted in elements.  Every call is
 * capturable into a CUDA graph.
 */
#ifndef MOE_DECODE_H_
#define MOE_DECODE_H_

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Residual addition and root-mean-square norm of T rows of d columns:
 *   t   = x + residual                       (fp32; t = x where residual is NULL)
 *   sum = bf16(t)                            the new residual stream
 *   y   = bf16(t * w / sqrt(mean(t^2) + eps))
 *   y_q, y_s = the MXFP8 form of the bf16 rows y: E4M3 codes and one E8M0 byte per 32 columns, exactly what
 *         moe_permute writes for y (rows contiguous: [T, d] and [T, d / 32]); a valid input of moe_expert_ffn.
 * The mean and the norm use the unrounded fp32 t; every bf16 output is rounded once.  The squares are summed in fp32: a
 * row's root of the sum of squares is to lie below 1.8e19, and values below 1e-22 count as 0 in it.
 *   x, residual, sum, y   bf16, 16-byte aligned, row strides a multiple of 8 and at least d (0 = d).
 *   weight                [d], bf16 or fp32 (weight_f32 != 0), 16-byte aligned.
 *   d                     a multiple of 8 up to 65536, of 32 where y_q is asked for; T >= 0; eps >= 0.
 * sum, y and the pair y_q / y_s may each be NULL (not written; at least one of them is given).  sum may be x
 * or residual itself and y may be x, with the same stride; other overlaps are not allowed.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED (d, GPU), MOE_ERR_CUDA.
 */
typedef struct {
  const void* x;
  const void* residual;
  const void* weight;
  void* sum;
  void* y;
  uint8_t* y_q;
  uint8_t* y_s;
  int64_t x_stride, residual_stride, sum_stride, y_stride;
  int32_t T, d;
  int32_t weight_f32;
  float eps;
} moe_norm_t;

MOE_API moe_status_t moe_add_rms_norm(const moe_norm_t* args, moe_stream_t stream);

/*
 * A paged key-value cache of one layer, described by value: the caller owns every buffer.
 *   k, v         pages [n_pages][page_size][n_kv_heads][head_dim]; element (page, row, head, i) at
 *                page * page_stride + row * row_stride + head * head_stride + i, the same for k and v, so any
 *                order of page rows and heads can be described.  16-byte aligned.
 *   format       MOE_KV_BF16: bf16 elements.  MOE_KV_MXFP8: E4M3 codes with one E8M0 byte per 32 elements of a
 *                row in k_s / v_s, at the same strides divided by 32 (bytes 0..254).
 *   strides      multiples of 8 (bf16) or 32 (MXFP8).
 *   block_table  int32 [n_seqs][max_pages]: page of the request's tokens [j * page_size, (j + 1) * page_size).
 *                Entries past a request's length are never read.
 *   seq_lens     int32 [n_seqs]: tokens of every request, the step's L new ones included; may be 0.
 *   status       device int32 or NULL: sticky error bits (MOE_KV_BAD_LENGTH: a length below 0 or above
 *                max_pages * page_size, used as 0 or as that bound; MOE_KV_BAD_PAGE: a page outside
 *                [0, n_pages), which is not accessed: its request's result is not meaningful).
 *   head_dim     64 or 128; page_size >= 1; n_kv_heads >= 1.
 * Pages may be shared by requests as long as no call writes to them.
 */
enum { MOE_KV_BF16 = 0, MOE_KV_MXFP8 = 1 };
enum { MOE_KV_BAD_LENGTH = 1, MOE_KV_BAD_PAGE = 2 };
typedef struct {
  void* k;
  void* v;
  uint8_t* k_s;
  uint8_t* v_s;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int32_t* status;
  int64_t page_stride, row_stride, head_stride;
  int32_t format;
  int32_t n_pages, page_size, n_kv_heads, head_dim;
  int32_t n_seqs, max_pages;
} moe_kv_cache_t;

/*
 * Write the L new tokens of every request into the cache: token l of request b goes to position
 * seq_lens[b] - L + l (a negative position is skipped).  k_new, v_new: bf16 rows (b * L + l) of n_kv_heads *
 * head_dim elements at k_stride / v_stride (multiples of 8; 0 = contiguous), 16-byte aligned: views of a fused
 * projection's output serve.  MXFP8 caches receive the codes and scales of moe.h's MXFP8 rule, exact.
 * L >= 0: one token, a verify step's rows or a whole prompt.
 */
MOE_API moe_status_t moe_kv_append(const moe_kv_cache_t* cache, const void* k_new, int64_t k_stride,
                                   const void* v_new, int64_t v_stride, int32_t L, moe_stream_t stream);

/*
 * Attention of the L newest tokens of every request over the request's cache.  Row (b, l) sees positions
 * t < seq_lens[b] - L + 1 + l (causal among the new tokens); with h' = h / (n_q_heads / n_kv_heads):
 *   s_t = scale * q[b, l, h] . k[t, h'];  out = sum_t softmax(s)_t v[t, h'];  lse = log sum_t exp(s_t).
 * A row that sees nothing gets out = 0 and lse = -inf; a NaN in q or among the keys that a row sees makes both NaN,
 * one among the values their column of out.  Positions that a row does not see never change its result, whatever they
 * hold (NaN and infinities included).
 *   q, out   bf16 rows (b * L + l) of n_q_heads * head_dim elements at q_stride / out_stride (multiples of 8;
 *            0 = contiguous), 16-byte aligned.
 *   lse      fp32 [n_seqs, L, n_q_heads] or NULL.
 *   n_q_heads a multiple of n_kv_heads; L >= 0; scale finite; k and v span less than 64 GB each; the keys of an MXFP8
 *            cache lie below 2^100 (their block sums are held in fp32 before q's own scale).
 *   workspace  at least moe_paged_attention_workspace(cache, n_q_heads, L) bytes, 256-byte aligned.  Its first
 *            MOE_ATTENTION_COUNTER_BYTES bytes must be ZERO before its first use; every call leaves them zero, and what
 *            else it holds does not matter.  So one buffer serves any calls, of any caches and shapes, that run one
 *            after another; calls that may overlap need one each.
 * The result does not depend on timing: the work is split over the length by a rule on the lengths alone and
 * joined in a fixed order.
 */
#define MOE_ATTENTION_COUNTER_BYTES 4096
typedef struct {
  const void* q;
  void* out;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
  int64_t q_stride, out_stride;
  int32_t n_q_heads;
  int32_t L;
  float scale;
} moe_attention_t;

MOE_API size_t moe_paged_attention_workspace(const moe_kv_cache_t* cache, int32_t n_q_heads, int32_t L);
MOE_API moe_status_t moe_paged_attention(const moe_kv_cache_t* cache, const moe_attention_t* args,
                                         moe_stream_t stream);

/*
 * moe_forward for a batch of at most MOE_FEW_MAX_T rows, in one kernel: the same routing, MXFP8 activations,
 * experts and combine (see moe.h), with the weighted expert rows summed in fp32 as they are; a token's row has the
 * same bits alone and in any company.  The faster call for one or two rows; above four moe_forward is.  The codes of a row
 * of x or h are held in fp16 with the block scales relative to the row's largest: exact where a block's scale is at most
 * 2^22 below that, with fewer bits further down, and possibly 0 where it is more than 2^31 below.  The experts' scales lie below 2^96.
 * Arguments and errors are moe_forward's, and three limits more, each MOE_ERR_UNSUPPORTED: the expert sets must use
 * MOE_ACT_MXFP8; n_experts <= 512 for the learned router; and the rows must leave room in shared memory for the weights:
 *   rows          1      2      3      4      5      6      7     8
 *   d_model  <= any  39680  26112  19200  15104  12544  10496  8960
 * topk_ids int32 [T, top_k] and topk_w fp32 [T, top_k] receive the routing (each may be NULL).  Uses the
 * workspace of `experts`.  The kernel's blocks wait on one another: it is launched cooperatively, one block per
 * SM, and every wait is bounded by the handle's wait budget (moe_check reports MOE_ERR_TIMEOUT).
 */
#define MOE_FEW_MAX_T 8
MOE_API moe_status_t moe_forward_few(const moe_input_t* x, const float* router_w, const float* router_bias,
                                     moe_experts_t experts, moe_experts_t shared, void* out_bf16, int32_t* topk_ids,
                                     float* topk_w, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DECODE_H_ */
