/*
 * fc_paged.h -- a paged K/V cache of many sequences of different lengths, and
 * single-token decode attention over it.
 *
 * The compressed archive of fc.h holds one (B, H, T, D) batch whose rows have
 * one common length. The calls here hold sequences that start, grow, fork and
 * end on their own, uncompressed (bf16 or fp32) or as int8 rows (one fp32
 * scale per (token, kv head), the quantiser of fc.h applied to a token's row):
 * the form for short or recent sequences, which fc_paged_read hands over to
 * the codec as the dense rows fc_compress_blocks takes.
 *
 * Token t of a sequence lies in row t mod P of page table[slot][t / P], P the
 * page size. Pages are shared by the layers (the same page number in every
 * layer's pool) and may be shared by sequences (fork); a shared page is
 * copied before it is written.
 *
 * Attention, per sequence of length n and query head:
 *   seen(t) = t < n and (window == 0 or t >= n - window or t < sinks)
 *   s_t = sigma q.k_t,  m = max s_t,  l = sum e^(s_t - m),
 *   out = sum e^(s_t - m) v_t / l,  lse = m + ln l   over the seen t.
 * An infinity or a NaN in a query or in a seen row acts as the formula has it in
 * fp32 (a score of -infinity is a token without weight, an infinite element of V
 * an infinite output of its channel) and stays in its row and kv head. int8 rows
 * with one read as NaN, and an int8 head whose query has one is NaN.
 * The tokens of all sequences are split evenly over the GPU; the parts of one
 * sequence are joined in a fixed order, so equal inputs give equal bits.
 *
 * Conventions are those of fc.h (caller-owned memory, element strides,
 * asynchronous on `stream`, host validation before any launch, an fc_status
 * return, no exception, no fallback), and:
 *   - The map of sequences to pages is kept twice: in the caller's host arrays
 *     (h_table, h_lens, h_refs), which the bookkeeping calls fc_pages_* read
 *     and change, and in device arrays the kernels read. Each bookkeeping call
 *     queues the device's copy of its changes on `stream`; on an error neither
 *     copy has changed. They are host decisions: a call on a stream that is
 *     being captured is FC_ERR_INVALID.
 *   - The batch of the current step (fc_pages_begin) is device data too, so a
 *     captured graph of fc_paged_append / _attention / _step launches may be
 *     replayed after each fc_pages_begin with at most as many rows (the rows
 *     past them are then empty), with at most as many new tokens as a captured
 *     append was offered (B * M), and with at most one in each row where a step
 *     was captured (a row with none attends only). A replay cannot refuse:
 *     tokens beyond these count as present, and nothing has written them. A
 *     captured fc_paged_read has the slot's length of its call. A replay without
 *     a new batch repeats the last one: it must not follow a fork, free or crop
 *     of its slots, or a restore.
 *   - Queue all calls of one cache on one stream, or order the streams.
 *
 * Supported sizes: D in {32, 64, 128, 256}; Hq a multiple of H with G = Hq / H
 * in {1, 2, 4, 8, 16}; P a power of two, 8 <= P <= 1024.
 */
#ifndef FC_PAGED_H_
#define FC_PAGED_H_

#include "fc.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Storage and map of one paged cache.
 *
 *   k, v        device, (n_layers, n_pages, H, P, D) of dtype, 16-byte
 *               aligned; within one (layer, page, head) the (P, D) rows are
 *               contiguous; strides in elements, multiples of 16 bytes.
 *   k_scales, v_scales  device, (n_layers, n_pages, H, P) fp32, contiguous
 *               along P, 16-byte aligned, strides multiples of 4; required
 *               when dtype == FC_DTYPE_I8, must be NULL otherwise.
 *   dtype       FC_DTYPE_BF16, FC_DTYPE_F32 or FC_DTYPE_I8.
 *   table       device, (n_slots, max_pages) int32, contiguous; lens device,
 *               (n_slots); batch device, (n_slots, 4) int32, 16-byte aligned:
 *               per row of the open batch {slot, length, first new token,
 *               new tokens}, slot -1 for a padding row.
 *   h_table, h_lens  host arrays of the same shapes; h_refs host, (n_pages):
 *               how many table entries name each page (0: free).
 *   first_free, n_free   no page below first_free is free; free pages.
 *   n_rows, n_tokens, one_each   the open batch (host): its rows, its new
 *               tokens, whether every row has exactly one; n_rows == 0: none.
 *   device_rows   rows of `batch` that may not be empty on the device.
 * fc_pages_reset, the first call on a new cache, sets the map and the host
 * fields; they are the library's from then on.
 */
typedef struct fc_pages {
  void* k;
  void* v;
  float* k_scales;
  float* v_scales;
  int32_t dtype;
  int32_t page_size;
  int64_t n_layers, n_pages, H, D;
  int64_t stride_layer, stride_page, stride_head;
  int64_t scale_stride_layer, scale_stride_page, scale_stride_head;
  int64_t n_slots, max_pages;
  int32_t* table;
  int32_t* lens;
  int32_t* batch;
  int32_t* h_table;
  int32_t* h_lens;
  int32_t* h_refs;
  int64_t first_free, n_free;
  int64_t n_rows, n_tokens;
  int32_t one_each;
  int32_t device_rows;
} fc_pages;

/* fc_pages_reset -- empty every slot: all pages free, tables -1, no batch. */
int fc_pages_reset(fc_pages* p, fc_stream stream);

/*
 * fc_pages_restore -- take over a map: slot s holds lens[s] tokens in pages
 * table[s][0 .. ceil(lens[s] / P)) (HOST arrays of h_table's and h_lens'
 * shapes; a page may be named by several slots, not twice by one). Entries
 * past a slot's last page are ignored and become -1. FC_ERR_INVALID for a
 * page or length out of range.
 */
int fc_pages_restore(fc_pages* p, const int32_t* table, const int32_t* lens,
                     fc_stream stream);

/*
 * fc_pages_begin -- open the batch of a step: row i is slot slots[i], which
 * grows by counts[i] >= 0 new tokens (counts NULL: one each). Missing pages
 * are taken, the lowest free ones first, in row order; a partly filled last
 * page that other slots share is copied to a new page in every layer before
 * it will be written. Rows n .. n_rows - 1 are padding (empty sequences).
 *
 *   slots, counts   HOST arrays of n; slots distinct, 0 <= slot < n_slots.
 *   1 <= n <= n_rows <= n_slots.
 * FC_ERR_CAPACITY (nothing changed) when the pages or a table row do not
 * suffice. The new tokens count as present from here on; fc_paged_append or
 * fc_paged_step writes them, once per layer.
 */
int fc_pages_begin(fc_pages* p, const int32_t* slots, const int32_t* counts,
                   int64_t n, int64_t n_rows, fc_stream stream);

/*
 * fc_pages_fork -- slot dst[i] (empty) becomes a copy of slot src[i]: its
 * pages are shared, its length taken over; no data moves until one of them
 * writes to the shared last page. HOST arrays; the dst are distinct and none
 * is a src. Closes the open batch.
 */
int fc_pages_fork(fc_pages* p, const int32_t* src, const int32_t* dst,
                  int64_t n, fc_stream stream);

/*
 * fc_pages_free -- empty the slots (HOST array, distinct); pages no other slot
 * names become free. Closes the open batch.
 */
int fc_pages_free(fc_pages* p, const int32_t* slots, int64_t n,
                  fc_stream stream);

/*
 * fc_pages_crop -- remove the last -tokens_to_remove tokens of a slot (a
 * negative count as in fc_crop; all of them when it exceeds the length; 0
 * does nothing); pages past the new end become free unless shared. Closes the
 * open batch unless nothing is removed.
 */
int fc_pages_crop(fc_pages* p, int32_t slot, int64_t tokens_to_remove,
                  fc_stream stream);

/*
 * fc_pages_compact -- pack the live pages into [0, *n_live): the i-th live
 * page at or above n_live moves to the i-th free page below it (both
 * ascending), in every layer, and the tables follow. The open batch stays.
 * n_live may be NULL.
 */
int fc_pages_compact(fc_pages* p, int64_t* n_live, fc_stream stream);

/*
 * fc_paged_append -- write the new tokens of the open batch to their pages in
 * one layer.
 *   k, v      device, (B, H, M, D) of dtype with element strides [4],
 *             innermost 1: new token j of the batch (rows in order, each
 *             row's tokens in order) is element (j / M, :, j mod M, :).
 *             B * M >= the batch's new tokens; further elements are ignored
 *             (a captured launch writes as many of later batches as they have,
 *             up to B * M).
 *   dtype     the pages' dtype; FC_DTYPE_BF16 or FC_DTYPE_F32 for int8 pages.
 * int8 pages: scale = max_d |x| / 127 in fp32, code = x / (max_d |x| / 127)
 * rounded to nearest, ties to even, decided exactly; an all-zero row stores
 * scale 0 and codes 0, a row with a NaN or an infinity scale NaN and codes 0.
 */
int fc_paged_append(const fc_pages* p, int64_t layer, const void* k,
                    const void* v, int32_t dtype, const int64_t* k_strides,
                    const int64_t* v_strides, int64_t B, int64_t M,
                    fc_stream stream);

/*
 * fc_paged_workspace_bytes -- workspace fc_paged_attention and fc_paged_step
 * need on the current device; 0 for unsupported sizes.
 */
size_t fc_paged_workspace_bytes(int64_t Hq, int64_t H, int64_t D);

/*
 * fc_paged_capture_id -- a number that no other capture of the process has, of
 * the capture that `stream` takes part in; 0 when it takes part in none. The
 * launches that one capture records on one stream run in their order, so they
 * may share a workspace; those of two captures may not.
 */
uint64_t fc_paged_capture_id(fc_stream stream);

/*
 * fc_paged_attention -- attention of one token per row of the open batch over
 * that row's sequence in one layer.
 *   q, out    device, (n_rows, Hq, 1, D); q FC_DTYPE_BF16 or FC_DTYPE_F32, out
 *             FC_DTYPE_F32 or FC_DTYPE_BF16; element strides [4], innermost 1.
 *   softmax_scale   sigma; <= 0 selects D^-0.5.
 *   window    0: every token; > 0: the last `window` tokens (the newest one
 *             included) and the first `sinks` ones.
 *   lse       device, (n_rows, Hq) fp32 contiguous, or NULL.
 *   workspace >= fc_paged_workspace_bytes, 256-byte aligned, all zero before
 *             its first use; every call leaves it fit for the next. Calls
 *             that share one must not overlap on the GPU.
 * A row that sees no token (padding, an empty sequence), or only tokens whose
 * scores are -infinity, gives out = 0 and lse = -infinity. Masked tokens are not read. One kernel launch.
 */
int fc_paged_attention(const fc_pages* p, int64_t layer, const void* q,
                       int32_t q_dtype, const int64_t* q_strides, int64_t Hq,
                       float softmax_scale, int64_t window, int64_t sinks,
                       void* workspace, size_t workspace_bytes, void* out,
                       int32_t out_dtype, const int64_t* out_strides,
                       float* lse, fc_stream stream);

/*
 * fc_paged_step -- fc_paged_append of one new token per row (k_new, v_new:
 * (n_rows, H, 1, D), element strides [4]; padding rows are not read), then
 * fc_paged_attention, in one launch and with the results of the two calls.
 * FC_ERR_INVALID unless the open batch has one new token in every row.
 */
int fc_paged_step(const fc_pages* p, int64_t layer, const void* q,
                  int32_t q_dtype, const int64_t* q_strides, int64_t Hq,
                  const void* k_new, const void* v_new, int32_t new_dtype,
                  const int64_t* k_strides, const int64_t* v_strides,
                  float softmax_scale, int64_t window, int64_t sinks,
                  void* workspace, size_t workspace_bytes, void* out,
                  int32_t out_dtype, const int64_t* out_strides, float* lse,
                  fc_stream stream);

/*
 * fc_paged_read -- the tokens of one slot in one layer as dense rows: k_out
 * and v_out device, (1, H, T, D) of out_dtype (FC_DTYPE_BF16 or FC_DTYPE_F32),
 * T >= the slot's length, 16-byte aligned, element strides [4]: innermost 1,
 * the others multiples of 16 bytes. Rows past the length are not written.
 * int8 rows are code * scale in fp32, rounded once to out_dtype.
 */
int fc_paged_read(const fc_pages* p, int64_t layer, int64_t slot, void* k_out,
                  void* v_out, int32_t out_dtype, const int64_t* k_strides,
                  const int64_t* v_strides, int64_t T, fc_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* FC_PAGED_H_ */
