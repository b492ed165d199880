/*
 * dmtp_ops.h - operators of one decode step over a paged K/V cache (GB300, sm_103a).
 *
 * The round of dmtp.h keeps one contiguous cache per sequence inside its workspace. An
 * engine that serves many requests keeps their K/V in pages of one pool instead; these
 * calls are the pieces of its decode step next to the round's own:
 *   dmtp_paged_write       rotary positions on new q and k rows; k and v into the pages
 *   dmtp_paged_read        rows of the pages back as dense rows
 *   dmtp_paged_attention   attention of a sequence's newest rows (one token, or the rows
 *                          of a verify) over its pages
 *   dmtp_add_rmsnorm_e4m3  residual addition, RMS norm, E4M3 rows (the draft heads' 8-bit
 *                          row format)
 *   dmtp_sample_rows       temperature, top-k, top-p and min-p from given random numbers
 * They are for inference: none has a backward pass.
 *
 * Memory. The caller owns every buffer; nothing is allocated. Pointers are device
 * pointers on the current device, and work is enqueued on `stream` (NULL: the default
 * stream), so every call can be captured into a CUDA graph. A workspace belongs to one
 * call at a time: calls (or replays of captured calls) that may overlap on the GPU each
 * need their own. A workspace needs no initialisation. The first call of an operator on a
 * device sets its kernels up and should come before any stream capture.
 *
 * Errors. DMTP_EINVAL is detected on the host before any launch. DMTP_ECUDA: a CUDA call
 * or launch failed, or a CUDA error was already pending on the calling thread (nothing is
 * launched then and it is not cleared). What only the device can see - a page or sequence
 * index out of range - is skipped by the kernel and OR-ed into *err (device uint32, may be
 * NULL), as DMTP_OPS_ERR_* bits; no access leaves the buffers described by the arguments.
 *
 * Types. dtype 0: fp32, 1: bf16 (as in dmtp_config). An E4M3 row is the framework's: scale
 * s = 2^e with e the smallest integer >= -126 such that max|row| <= 448 s (over the row's
 * finite values; 1 for a row without a non-zero one), and values rounded to nearest even
 * of value / s; a NaN or an infinity is stored as the E4M3 NaN.
 */
#ifndef DMTP_OPS_H
#define DMTP_OPS_H

#include "dmtp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bits of the operators' error word */
#define DMTP_OPS_ERR_POS 2u   /* a position or length outside the block table's reach */
#define DMTP_OPS_ERR_PAGE 16u /* a block table entry outside [0, n_pages)             */
#define DMTP_OPS_ERR_SEQ 32u  /* a sequence index >= n_seqs                           */

#define DMTP_OPS_MAX_HEAD_DIM 256
#define DMTP_OPS_MAX_ROWS 8          /* query rows of one sequence in one attention call */
#define DMTP_OPS_MAX_NORM_D 16384
#define DMTP_OPS_MAX_SAMPLE_VOCAB 262144

/* A paged K/V cache of one layer. Page p holds, for every kv head, page_size rows of
 * head_dim values: k + p * page_stride is [n_kv_heads][page_size][head_dim] (elements),
 * likewise v. e4m3 = 0: values of `dtype`, k_scale and v_scale unused. e4m3 = 1: E4M3
 * values, and k_scale + p * scale_stride is [n_kv_heads][page_size] fp32 scales of the
 * rows (positive normal numbers below 2^127; dmtp_paged_write makes powers of two), likewise
 * v_scale.
 * Position j of sequence s lies in page table[s * table_stride + j / page_size], row
 * j % page_size; 0 <= j < max_blocks * page_size. Entries past a sequence's length are not
 * read, nor are those whose positions all lie before the window of every row. Several entries may name one page (a shared prefix).
 * Limits: head_dim a multiple of 16 up to DMTP_OPS_MAX_HEAD_DIM; 1 <= page_size <= 65536;
 * max_blocks * page_size < 2^31 - 65536; k and v 16-byte aligned, page_stride
 * >= n_kv_heads page_size head_dim and a multiple of 16 bytes; scale_stride
 * >= n_kv_heads page_size; table_stride >= max_blocks. */
typedef struct {
  void *k, *v;
  float *k_scale, *v_scale;
  const int32_t* table;
  int64_t page_stride, scale_stride, table_stride;
  int n_pages, page_size, n_kv_heads, head_dim;
  int n_seqs, max_blocks;
  int dtype, e4m3;
} dmtp_paged_kv;

/* New rows: row r of k and v (both [n_rows][n_kv_heads][head_dim], with the given strides
 * in elements; head_dim dense) belongs at position pos[r] of sequence seq[r] (device
 * int32). A row with seq[r] < 0 is skipped (padding); its q_out row is left as it was. A
 * position that two rows of one call name gets the values of one of them, or a mixture (in an
 * E4M3 cache bytes of one may meet the other's scale): a call's positions should differ.
 * rope_theta > 0: k (and q) are rotated first, pairs (i, i + head_dim / 2) by the angle
 * pos * rope_theta^(-2 i / head_dim), formed to pos 2^-53 turns (2^-30 at position 2^23, 2^-22
 * at the last); 0: stored as they are. q (optional, NULL): [n_rows][n_heads][head_dim], rotated into
 * q_out [n_rows][n_heads][head_dim] (both may be the same memory with the same strides).
 * All are of the cache's dtype. Row pointers and strides are multiples of four elements
 * (bf16: 8 bytes, fp32: 16 bytes). The rotation is computed in fp32 from fp32 sines. */
typedef struct {
  const void *q, *k, *v;
  void* q_out;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, qo_row, qo_head;
  const int32_t *seq, *pos;
  int n_rows, n_heads;
  float rope_theta;
} dmtp_paged_rows;

int dmtp_paged_write(const dmtp_paged_kv* c, const dmtp_paged_rows* r, uint32_t* err,
                     void* stream);

/* Row i of k_out and v_out ([n_rows][n_kv_heads][head_dim], dense, of the cache's dtype,
 * 16-byte aligned) becomes position pos[i] of sequence seq[i] (an E4M3 value times its
 * scale, rounded once to dtype). Rows with seq[i] < 0 are left as they were; so are rows
 * that set an error bit. */
int dmtp_paged_read(const dmtp_paged_kv* c, const int32_t* seq, const int32_t* pos, int n_rows,
                    void* k_out, void* v_out, uint32_t* err, void* stream);

/* The newest `rows` (1..DMTP_OPS_MAX_ROWS) rows of each of the n_seqs sequences attend
 * over its cache, which already holds them: with L = kv_len[s] (device int32; L <= 0: the
 * sequence is idle), row i is at position p = L - rows + i and
 *   out[s][i][h] = sum_j softmax_j(scale q[s][i][h] . k_j) v_j
 * over the positions 0 <= j <= p, and, for window > 0, j > p - window. kv head h / (n_heads
 * / n_kv_heads) serves query head h. A row that sees no position (idle sequences, p < 0)
 * gets zeros. q and out: the cache's dtype, strides in elements, head_dim dense; row
 * pointers 16-byte aligned, strides multiples of 16 bytes. Lengths past the block table's
 * reach are cut there and set DMTP_OPS_ERR_POS; a bad page sets DMTP_OPS_ERR_PAGE and its
 * positions are left out. A NaN or an infinity reaches the rows that see its position (a value
 * whose weight rounds to 0 may not) and no other. |scale| <= 1e30.
 * Scores, softmax statistics and sums are fp32; products of bf16 rows run on the tensor
 * cores with the weights as bf16 pairs (16 bits), of E4M3 rows with fp16 queries (scaled; exact but
 * for elements below 2^-29 of a query's largest) and fp16 weights (11 bits): a
 * weight times its v_scale is rounded against the largest such product of the query so far, in
 * which value rows of zeros with a v_scale of at least 1 (dmtp_paged_write gives them 1) do not
 * count (v_scale up to 2^40; values of rows scaled by less than 2^-60 count to 2^-76). The sum of
 * weights times values is fp32 before it is divided by the sum of weights: it must stay below
 * 2^120 or so. Results do not depend on timing: the same call gives the same bits. */
typedef struct {
  const void* q;
  void* out;
  int64_t q_seq, q_row, q_head, o_seq, o_row, o_head;
  const int32_t* kv_len;
  int rows, n_heads, window;
  float scale;
} dmtp_paged_query;

/* Bytes of workspace for dmtp_paged_attention (256-byte aligned; 0: none, and workspace may be
 * NULL). Of `a` only rows and n_heads matter. */
int dmtp_paged_attention_workspace(const dmtp_paged_kv* c, const dmtp_paged_query* a,
                                   size_t* bytes);
int dmtp_paged_attention(const dmtp_paged_kv* c, const dmtp_paged_query* a, void* workspace,
                         size_t ws_bytes, uint32_t* err, void* stream);

/* x_out = x + y (rounded to x's type), and the unrounded sum's norm as E4M3 rows:
 * h = (x + y) / sqrt(mean((x + y)^2) + eps) * gain, q [rows][d] E4M3 values with row pitch
 * q_row, scale [rows] fp32. x, x_out: x_dtype; y: y_dtype; gain [d]: gain_dtype; row
 * pitches in elements. The sum of squares is fp32: |x + y| up to about 1e17 (and, with an
 * eps below about 1e-30, the row's largest from 1e-17 on; of zeros with eps 0 it is 0 / 0). An infinite
 * x + y makes the row's finite values 0, a NaN all of them NaN. x_out may be x; y may be NULL (no
 * addition; x_out may then be NULL too). Limits: d a multiple of 8 up to DMTP_OPS_MAX_NORM_D; row
 * starts 16-byte aligned (q: 8-byte), pitches >= d and multiples of 8; eps >= 0 and finite. */
typedef struct {
  const void *x, *y, *gain;
  void *x_out, *q;
  float* scale;
  int64_t x_row, y_row, xo_row, q_row;
  int rows, d, x_dtype, y_dtype, gain_dtype;
  float eps;
} dmtp_norm_args;
int dmtp_add_rmsnorm_e4m3(const dmtp_norm_args* a, void* stream);

/* One token per row of logits [rows][vocab] (dtype 0 or 1, row pitch `ld` elements).
 * Weights w_v = exp((l_v - max) / temperature); the tokens that are kept are those that
 * pass every filter:
 *   top_k > 0   the top_k largest logits;
 *   top_p < 1   the shortest run of those, from the largest down, whose weight reaches
 *               top_p times the weight of the top_k (the first one always);
 *   min_p > 0   w_v >= min_p (of the largest weight; at most 1).
 * Equal logits rank by id, the lowest first. ids[r] is the first kept id, in order of id,
 * at which the running weight exceeds u[r] times the kept weight, u in [0, 1) (values
 * outside, and NaN, are taken as the nearest end, NaN as 0). temperature <= 0 or NaN: the
 * largest logit's id. A logit of -infinity or NaN is never kept; +infinity counts as
 * the largest finite number; a temperature counts as the nearest in [1e-30, 1e30]. A row that
 * keeps nothing gets id -1. kept[r] (optional) is the number of kept tokens. temperature, top_k, top_p, min_p: device arrays [rows], each
 * optional (NULL: 1, off, off, off). u: device fp32 [rows]. Weights and their sums are
 * integers (steps of 2^-44 of the largest, computed to about 2^-39), so a row's result depends
 * on nothing but its inputs. Limits: 1 <= vocab <= DMTP_OPS_MAX_SAMPLE_VOCAB, ld >= vocab. */
typedef struct {
  const void* logits;
  int64_t ld;
  int rows, vocab, dtype;
  const float *u, *temperature;
  const int32_t* top_k;
  const float *top_p, *min_p;
  int32_t *ids, *kept;
} dmtp_sample_args;
int dmtp_sample_rows(const dmtp_sample_args* a, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DMTP_OPS_H */
