/*
 * cac_kv8.h — a paged 8-bit K/V cache shared by many sequences, and attention
 * over it (C ABI).  Same conventions as cac.h: status codes, device pointers
 * owned by the caller, asynchronous on `stream`, row-major layouts.
 *
 * Sequences of any length in one byte per value, in pages that forked sequences
 * share, read under a chunked-causal mask with optional first tokens that stay
 * visible.  The mask is the one of the streaming encoder ("True streaming
 * encode", §Why this is provably correct: left context and chunk on absolute
 * positions); the scores are not: here they are scale * q . k, where the
 * encoder's attention has a term for relative positions, and its beam's
 * hypotheses are LSTM states without K and V.  So the encoder and the decoders
 * of this library go on with their own states and call nothing of this; it is
 * for models beside them whose attention has the plain form.
 *
 * Layout.  Token t of sequence s lies in page table[s][t / page_tokens], row
 * t % page_tokens.  A page holds, for each layer and K/V head, page_tokens rows
 * of head_dim codes for K and for V, and one fp32 scale for each block of 16
 * tokens and head: value = scale * code.
 *   CAC_KV8_INT8  signed 8-bit integers in [-127, 127]
 *   CAC_KV8_E4M3  8-bit floating point (4 exponent, 3 mantissa bits, |x| <= 448)
 *
 * Quantisation (top = 127 or 448).  A block's scale is max(amax * (1 / top),
 * 2^-100) in fp32 over the block's finite values; the code is the one nearest
 * x * (1 / scale), ties to even.  When tokens are added to a block that holds
 * older ones, its scale is the larger of the old one and what the new tokens
 * need; where that grows, the older codes are rounded again from code *
 * (old scale / new scale).  An infinite input takes the block's largest code, a
 * NaN takes code 0, and either latches CAC_E_NONFINITE in *status.  A scale of 0
 * marks a block that an extend began and no write has filled.
 *
 * Nothing here reads device state on the host: lengths, tables and free pages
 * live on the device, so every call can be captured into a CUDA graph and
 * replayed.  What only the device can see wrong (an id outside the cache, the
 * same id twice in a call that changes it, no free page left) is latched in
 * *status (first error wins, read by cac_kv8_check), and that call, or that
 * sequence of it, changes nothing.
 *
 * Calls that change a cache must be ordered with every other call on it (one
 * stream, or events between).  cac_kv8_read and cac_kv8_attend change nothing
 * and may run at the same time on several streams, each with its own outputs
 * and workspace.  Which free page a call takes is not specified; no value
 * depends on it.
 */
#ifndef CAC_KV8_H_
#define CAC_KV8_H_

#include <stddef.h>
#include <stdint.h>

#include "cac.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CAC_KV8_INT8  0
#define CAC_KV8_E4M3  1
#define CAC_KV8_BLOCK 16   /* tokens that share a scale */

typedef struct cac_kv8 {
    int32_t n_layers;      /* >= 1 */
    int32_t kv_heads;      /* 1 .. 65535 */
    int32_t head_dim;      /* multiple of 16, 16 .. 256 */
    int32_t page_tokens;   /* multiple of 16, 16 .. 1024 */
    int32_t n_pages;       /* pages of the pool, shared by all sequences */
    int32_t max_seqs;      /* sequence ids 0 .. max_seqs-1 */
    int32_t max_pages;     /* pages of one sequence; max_pages * page_tokens < 2^30 */
    int32_t code;          /* CAC_KV8_INT8 / CAC_KV8_E4M3 */
    int32_t device;        /* CUDA device of every pointer below */
    int32_t reserved;
    void* k;               /* [n_layers][n_pages][kv_heads][page_tokens][head_dim] bytes, 16-byte aligned */
    void* v;
    float* k_scale;        /* [n_layers][n_pages][kv_heads][page_tokens / 16] */
    float* v_scale;
    int32_t* table;        /* [max_seqs][max_pages]; -1: no page */
    int32_t* lens;         /* [max_seqs] tokens of each sequence */
    int32_t* refs;         /* [n_pages] tables that name the page */
    int32_t* free_list;    /* [n_pages]; the first *n_free entries are the free pages */
    int32_t* n_free;       /* [1] */
    int32_t* pending;      /* [max_seqs][2], 8-byte aligned: what the last extend made room for, and its place
                              in that call */
    int32_t* work;         /* cac_kv8_work_ints ints, zero before the first call */
    int32_t* status;       /* [1] */
} cac_kv8;

/* Ints of `work` for this shape; 0 for an invalid one.  Reads no pointer. */
size_t cac_kv8_work_ints(const cac_kv8* c);

/* Empties the cache: every sequence has length 0, every page is free.  The
 * arrays may hold anything before.  Codes and scales are left as they are. */
int cac_kv8_init(const cac_kv8* c, void* stream);

/* The sequences of a call: ids device int32 [n], distinct where the call
 * changes them (read and attend take an id twice).  Their rows in k, v, q and
 * out lie one after another: sequence i has rows starts[i] .. starts[i+1]-1
 * (starts: device int32 [n+1], starts[0] >= 0, never falling), or, where starts is
 * NULL, the same number of rows each. */

/* Make room for new tokens of each sequence (`each`, or starts[i+1] -
 * starts[i]): free pages enter its table, a last page that is not full and that other
 * sequences name too is copied, and the length grows.  All sequences of the call
 * get their pages, or none does: CAC_E_NOMEM (not enough free pages),
 * CAC_E_LIMIT (longer than max_pages), CAC_E_BOUNDS (id out of range or negative
 * count), CAC_E_INVAL (an id twice), CAC_E_STATE (the last page was released by
 * trim before a truncate into it) are latched.  Tokens that no write fills have
 * unspecified values in that layer; tokens added after them do not suffer.  A
 * refused call ends the right to write of the sequences that it names, so that a
 * write behind it does not go to the tokens before. */
int cac_kv8_extend(const cac_kv8* c, int n, const int32_t* ids, const int32_t* starts, int each, void* stream);

/* Quantise one layer's K and V of the tokens that the last extend made room
 * for; same ids in the same order and same counts (a sequence for which that does
 * not hold latches CAC_E_STATE and is skipped).
 *   k, v  device [rows][kv_heads][head_dim], dtype CAC_DTYPE_F32 or CAC_DTYPE_BF16,
 *         a row every k_stride / v_stride elements (>= kv_heads * head_dim);
 *         pointers and row strides multiples of 16 bytes (CAC_E_ALIGN)
 * With starts, a sequence whose rows pass `rows` latches CAC_E_BOUNDS and is skipped. */
int cac_kv8_write(const cac_kv8* c, int layer, int n, const int32_t* ids, const int32_t* starts, int rows,
                  const void* k, const void* v, long long k_stride, long long v_stride, int dtype, void* stream);

/* The values of tokens first[i] .. first[i] + count - 1 of each sequence (first:
 * device int32 [n]) as k, v [n][count][kv_heads][head_dim] of dtype; either may be
 * NULL.  Tokens before 0, past the end or in a released page read as zero; so do
 * those of an id out of range, which latches CAC_E_BOUNDS. */
int cac_kv8_read(const cac_kv8* c, int layer, int n, const int32_t* ids, const int32_t* first, int count, void* k,
                 void* v, int dtype, void* stream);

/* Attention of each sequence's last tokens over its cache.  A sequence with m
 * rows here has its queries at positions len - m .. len - 1 (append first, then
 * attend).  The query at position p, with b = floor(p / att_chunk) * att_chunk,
 * sees token j when j < min(b + att_chunk, len), its page is there, and
 * b - att_left <= j or j < sinks; att_left < 0 means no left limit.
 *   q     device [rows][heads][head_dim], heads a multiple of kv_heads: query head h
 *         reads K/V head h / (heads / kv_heads); a row every q_stride elements
 *   out   as q; a row that sees no token (an empty sequence, a position before 0)
 *         is zero.  out may not overlap q.
 *   lse   device fp32 [rows][heads], log of the sum of exp(scores) over the tokens
 *         seen (-inf where there is none), or NULL
 *   score = scale * q . k; pointers and row strides multiples of 16 bytes
 *   max_new: no sequence has more rows than this (one that has latches
 *         CAC_E_BOUNDS, and its rows are zero); used where starts is given.  A
 *         sequence whose rows pass `rows` latches CAC_E_BOUNDS too, and its rows are
 *         left as they were, as do starts that fall
 *   workspace: cac_kv8_attend_workspace bytes, 16-byte aligned, this call's own
 *         until it has run (NULL where that is 0)
 * Rows of out and lse that belong to no sequence are left as they were.  Rows of
 * a sequence that has tokens that an extend made room for and no write has filled
 * have unspecified values where a query of the call sees one of the same block.
 * V blocks may differ in size by any amount up to largest values of 2^80; beside
 * larger ones, tokens of blocks 2^115 times smaller may be lost from the norm.
 * A bounded wait inside the kernels that gives up latches CAC_E_TIMEOUT.
 * CAC_E_LIMIT: more than 2^26 tiles of 16 query rows (rows * heads / 16). */
int cac_kv8_attend(const cac_kv8* c, int layer, int n, const int32_t* ids, const int32_t* starts, int rows,
                   int max_new, int heads, float scale, int att_left, int att_chunk, int sinks, const void* q,
                   long long q_stride, void* out, long long out_stride, float* lse, int dtype, void* workspace,
                   size_t workspace_bytes, void* stream);
/* Enough for a call with these arguments, with starts or (then for rows / n
 * queries of each sequence, whatever max_new is) without. */
size_t cac_kv8_attend_workspace(const cac_kv8* c, int n, int rows, int max_new, int heads, int att_left,
                                int att_chunk, int sinks);

/* Make sequence dst[i] a copy of src[i] (device int32 [n]) that shares its
 * pages; what dst[i] held is released.  A source may be forked several times.
 * An entry whose dst is out of range (CAC_E_BOUNDS), listed twice or also
 * a source of the call (CAC_E_INVAL) is skipped.  Tokens that an extend made room
 * for and no write has filled yet can no longer be written. */
int cac_kv8_fork(const cac_kv8* c, int n, const int32_t* src, const int32_t* dst, void* stream);

/* Shorten each sequence to new_len[i] tokens (device int32 [n]; NULL: `each`
 * tokens, 0 frees it) and release the pages past it.  Never lengthens. */
int cac_kv8_truncate(const cac_kv8* c, int n, const int32_t* ids, const int32_t* new_len, int each, void* stream);

/* Release the pages of each sequence that no query at its next position or
 * later sees under this window: those wholly before floor(len / att_chunk) *
 * att_chunk - att_left and wholly past the first `sinks` tokens.  Positions and the
 * length stay. */
int cac_kv8_trim(const cac_kv8* c, int n, const int32_t* ids, int att_left, int att_chunk, int sinks, void* stream);

/* Move the pages in use to the front of the pool, so that pages 0 .. used-1
 * hold everything and the rest of the pool is one free piece.  Values and
 * lengths stay. */
int cac_kv8_compact(const cac_kv8* c, void* stream);

/* Synchronise the device and return the latched status, clearing it. */
int cac_kv8_check(const cac_kv8* c);

#ifdef __cplusplus
}
#endif
#endif /* CAC_KV8_H_ */
