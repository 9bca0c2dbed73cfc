/*
 * cac_ops.h — op-level entry points of the GB300 cache-aware Conformer
 * library, for kernel-level parity tests and microbenchmarks.  Same
 * conventions as cac.h (status codes, device pointers owned by the caller,
 * asynchronous on `stream`).
 */
#ifndef CAC_OPS_H_
#define CAC_OPS_H_

#include <stdint.h>

#include "cac.h"

#ifdef __cplusplus
extern "C" {
#endif

/* C[M][N] = A[M][K] * B[N][K]^T (+ bias[N]) on the tcgen05/TMEM tensor-core
 * GEMM that every projection of the encoder step uses (feed-forward, Q/K/V,
 * out-projection, pointwise convolutions, joint projection: "True streaming
 * encode", §Per-chunk flow step 3).  A and B bf16, row-major (K contiguous);
 * C fp32 row-major; bias fp32 or NULL.  K % 64 == 0, N % 64 == 0, M >= 1;
 * 16-byte aligned pointers.  splits: 1..4 K-splits per output tile (reduced
 * in a thread-block cluster), 0 = the library's choice.
 * a_split != 0: A is a split operand [M][2K] — row r holds hi[r][0..K) then
 * lo[r][0..K), two bf16 terms of one higher-precision activation — and the
 * product is (hi + lo) * B^T (the form in which the encoder's LayerNorm
 * outputs enter their projections). */
int cac_op_gemm_bf16(int M, int N, int K, const void* A, const void* B, const float* bias, float* C, int splits,
                     int a_split, void* stream);

/* C = A W^T (+ bias) with palette weights ("Fast Accuracy-Preserving RNNT Beam
 * Search on Apple Silicon", §1.3: 64-entry lookup tables, 6-bit palettes) on
 * the tensor cores (bf16 x bf16, fp32 accumulation).
 *   A       device bf16 [M][K], row-major, 16-byte aligned
 *   packed  device bytes [N][3K/4]: row n's indices as a little-endian bit
 *           stream, index k in bits [6k, 6k + 6); 16-byte aligned
 *   table   device bf16 [64]: W[n][k] = table[index]
 *   bias    device fp32 [N] or NULL;  C  device fp32 [M][N], 16-byte aligned
 *   status  device int or NULL: a bounded wait that gave up latches
 *           CAC_E_TIMEOUT there (first error wins)
 * N and K multiples of 64.  Asynchronous on `stream`.  CAC_E_INVAL for bad
 * sizes or NULL operands, CAC_E_ALIGN for misaligned pointers. */
int cac_op_gemm_palette(int M, int N, int K, const void* A, const void* packed, const void* table,
                        const float* bias, float* C, int* status, void* stream);

/* Bounds of cac_op_gemm_w4. */
#define CAC_W4_MAX_K 131072
#define CAC_W4_MAX_M 65535

/* Weights at 4 bits with a scale for each group of consecutive k:
 *   W[n][k] = scale[n][k / group] * (code[n][k] - zero[n][k / group])
 * Code k of row n is the low half of byte k / 2 where k is even, the high half
 * where it is odd. */
typedef struct cac_w4 {
    int32_t n, k;          /* rows >= 1; depth, a multiple of group */
    int32_t group;         /* 32, 64 or 128 */
    int32_t device;        /* CUDA device of every pointer of the call */
    const void* packed;    /* device bytes [n][k / 2], 16-byte aligned */
    const void* scale;     /* device bf16 [n][k / group], 4-byte aligned; below 2^100 in size */
    const uint8_t* zero;   /* device [n][k / group], 0 .. 15, 4-byte aligned; NULL: 8 everywhere */
} cac_w4;

/* C[M][n] = A[M][k] W^T (+ bias[n]), for the few rows of a decoding step (the
 * weights are read once for each 32 rows or fewer).
 *   A, C  device, both CAC_DTYPE_BF16 or both CAC_DTYPE_F32; a row every a_stride /
 *         c_stride elements (>= k / n); A 16-byte aligned with a_stride a multiple
 *         of 16 bytes, C aligned to its elements.  C may not overlap A.
 *   bias  device fp32 [n] or NULL
 * A group's products are summed with the codes less their zero points as they
 * are and scaled in fp32; sums are fp32, C is rounded once.  An element of A is
 * exact (bf16) or held to 22 bits (fp32), but for elements 2^29 and 2^17 times
 * smaller than the largest among k of the same 256: those are off by up to 2^-39
 * of it.  The result does not depend on timing.  A row of A with an infinity or
 * NaN gives infinities or NaNs in its row of C and touches no other row.
 * Nothing is allocated; the call can be captured into a CUDA graph.
 * CAC_E_INVAL / CAC_E_ALIGN for arguments outside the above, CAC_E_LIMIT for k or M
 * past their bounds. */
int cac_op_gemm_w4(const cac_w4* w, int M, const void* A, long long a_stride, const float* bias, void* C,
                   long long c_stride, int dtype, void* stream);

/* Rotation of queries and keys by their position, with an optional norm for each
 * head before it.  For each row and head, x of head_dim elements:
 *   u = x / sqrt(mean(x^2) + eps) * gain            (u = x where gain is NULL)
 *   the pairs (a, b) of u's first rot_dim elements, at position p, i < rot_dim / 2:
 *     a' = amplitude * (a cos(p f_i) - b sin(p f_i))
 *     b' = amplitude * (a sin(p f_i) + b cos(p f_i))
 *   CAC_ROTARY_HALF:  a, b = elements i and i + rot_dim / 2
 *   CAC_ROTARY_PAIRS: a, b = elements 2 i and 2 i + 1
 * Elements from rot_dim on are u's.  With a gain, a NaN makes its head NaN; an
 * infinity becomes NaN itself (in its pair), and the finite elements beside it 0.
 * Arithmetic is fp32, rounded once; the angle p f_i is a whole product of p and
 * steps[i], exact to 2^-33 of a turn at any position. */
#define CAC_ROTARY_HALF  0
#define CAC_ROTARY_PAIRS 1

typedef struct cac_rotary {
    int32_t head_dim;      /* multiple of 16, 16 .. 256 */
    int32_t rot_dim;       /* even, 0 .. head_dim */
    int32_t layout;        /* CAC_ROTARY_HALF / CAC_ROTARY_PAIRS */
    int32_t dtype;         /* of q, k and the results: CAC_DTYPE_BF16 / CAC_DTYPE_F32 */
    int32_t device;        /* CUDA device of every pointer of the call */
    float amplitude;       /* finite */
    float eps;             /* >= 1e-20 */
    int32_t reserved;
    const uint64_t* steps; /* device [rot_dim / 2]: f_i in 2^-64 of a turn (cac_op_rotary_steps); NULL where rot_dim is 0 */
    const float* q_gain;   /* device [head_dim] or NULL: no norm of the queries */
    const float* k_gain;   /* the same for the keys */
} cac_rotary;

/* What becomes of the frequencies base^(-2 i / rot_dim) for contexts longer than
 * those they were made for. */
#define CAC_ROTARY_NONE   0
#define CAC_ROTARY_LINEAR 1 /* all divided by factor */
#define CAC_ROTARY_BASE   2 /* base times factor^(rot_dim / (rot_dim - 2)) (rot_dim > 2) */
#define CAC_ROTARY_RAMP   3 /* f * (r + (1 - r) / factor), r from 0 to 1 as f's turns over `original` tokens go from low to high */

/* Writes rot_dim / 2 steps to host memory.  base > 1, factor >= 1; original > 0
 * and high > low >= -1e300 for CAC_ROTARY_RAMP.  No GPU is needed. */
int cac_op_rotary_steps(int rot_dim, double base, int scaling, double factor, double original, double low, double high,
                        uint64_t* steps);

/* Row t of q and k is at positions[t] (device int32, any value).
 *   q, k          device [rows][heads][head_dim] and [rows][kv_heads][head_dim], a row
 *                 every q_stride / k_stride elements; either may be NULL with 0 heads
 *   q_out, k_out  the same shapes, with strides of their own; an output may be its
 *                 input (same pointer and stride) and may not overlap it otherwise
 * Pointers and row strides are multiples of 16 bytes; heads, kv_heads <= 65535
 * (CAC_E_INVAL beyond), rows < 2^30 (CAC_E_LIMIT). */
int cac_op_rotate(const cac_rotary* r, int rows, const int32_t* positions, int heads, const void* q, long long q_stride,
                  void* q_out, long long q_out_stride, int kv_heads, const void* k, long long k_stride, void* k_out,
                  long long k_out_stride, void* stream);

/* Failure-path self-test of the library's bounded device waits: runs the
 * wait the library uses with nothing that can satisfy it and returns the
 * status the device latched — CAC_E_TIMEOUT when the wait gave up as designed.
 *   which 0: an mbarrier wait (the TMA / tensor-core pipelines' wait) on a
 *            barrier no thread arrives at; gives up after about 2 s;
 *   which 1: the decoder's grid-wide barrier in a cooperative launch whose
 *            first block never arrives; the others give up after about 1 s,
 *            raise the abort word and return.
 * Synchronous; the kernels exit normally, so the context stays usable.
 * CAC_E_INVAL for another `which`, CAC_E_CUDA if a launch failed. */
int cac_op_wait_selftest(int which, void* stream);

/* Self-test of the checked build (cac_build_checked() == 1): a kernel whose
 * threads index past a 32-float buffer runs with the library's index check,
 * which keeps every access in bounds; returns the status it latched —
 * CAC_E_BOUNDS as designed.  Synchronous.  CAC_E_UNSUPPORTED in the default
 * build (nothing is launched). */
int cac_op_bounds_selftest(void* stream);

#ifdef __cplusplus
}
#endif
#endif /* CAC_OPS_H_ */
