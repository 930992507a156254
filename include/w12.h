/*
 * w12.h -- C ABI of libw12.so: the W12 lossless 12-bit weight format and the skinny GEMMs
 * that read it on AMD Instinct MI355X (gfx950).
 *
 * The format (SpecPilot, arXiv 2611.02501, figure-captions page, Fig. 5(a)): every bfloat16
 * weight of W [n, k] (PyTorch Linear layout, n = output channels) is split into three 4-bit
 * planes -- A (sign and mantissa bits 6..4), E (exponent offset inside a 16-binade window
 * chosen per output channel) and B (mantissa bits 3..0).  Weights outside their row's window
 * go to an exact escape list.  A and E together are the 8-bit view that a low-precision
 * "Q pass" reads without touching B (same page, Fig. 5(a) and Fig. 7).
 *
 * Logical content of a record (the pages fix only the plane contents; this layout is ours):
 *   base[n]      u8   lowest biased exponent of row n's window, 1..239 (window = base..base+15)
 *   AE[n][k]     u8   s<<7 | E<<3 | m[6:4],  E = e - base       (the 8-bit view)
 *   B[n][k/2]    u8   B plane.  For weights k = 8g+i (i = 0..7) the nibble m[3:0] is in byte
 *                     4g + (i % 4) of the row: low nibble for i < 4, high nibble for i >= 4
 *   esc_ptr[n+1] u32  row CSR offsets into the escape arrays, esc_ptr[0] = 0
 *   esc_col[]    u32  column k of each escape, strictly ascending within a row
 *   esc_val[]    u16  exact bfloat16 bits of each escape
 * Storage order of the AE and B planes on the device (`ae`, `lo` below): tiles of 16 rows x 128
 * columns in row-tile-major order, rows padded with zero bytes to npad = 16 * ceil(n / 16).
 * Inside a tile (2048 bytes of AE, 1024 bytes of B), the AE byte of (row r, column c) sits at
 * 1024*((c % 32) / 16) + 16*(r + 16*(c / 32)) + c % 16, and the 16 B-plane bytes of row r for
 * columns 32g..32g+31 (row bytes 16g..16g+15 of the tile's 64) sit at 16*(r + 16*g).  Every
 * wave-wide 128-bit load of a kernel then reads 1 KiB of contiguous memory, already in the lane
 * order of the 16x16x32 matrix-core operand.
 * Window rule: the window holds as many of the row's weights as possible; ties go to the
 * smallest base; a row with no normal weight gets base 1.  Zeros, subnormals, Inf and NaN
 * (exponent field 0 or 255) are never inside a window, so they are always escapes.  An
 * escaped slot holds AE = 0 and a zero nibble.  Decoding reproduces every input bit (NaN
 * payloads and -0 included).
 *
 * Conventions for every call:
 *   - Pointers named as device memory must be device memory of the current HIP device,
 *     16-byte aligned; the caller owns every buffer and keeps it alive until the stream work
 *     is finished.  The only device memory the library allocates is the GEMM workspace below;
 *     it keeps no other per-call state.
 *   - Calls may come from several threads.  Those that share a stream's GEMM workspace or the same scratch
 *     must not be made at the same time: a call may launch several kernels, and another's would fall
 *     between them.
 *   - GEMM workspace: a GEMM call whose shape has too few 16-row tiles to occupy the device
 *     (for example W [1024, 5120], or [5120, 17408] at up to 32 rows of x) splits each row into
 *     k ranges whose partial sums go to a 64 MiB device buffer, then adds them in range order;
 *     a W12 or Q8 call with more than 64 rows of x puts a transposed copy of each pass's (up to
 *     128) rows there (k x 256 bytes; with k > 262144 the passes stay at 64 rows and need none).
 *     The buffer belongs to the (device, stream) pair, is allocated with hipMalloc on the first
 *     such call on that stream (also while the stream is being captured into a graph: the
 *     allocation is made under the relaxed capture mode) and is kept until the process ends
 *     or w12_release_workspace(stream).
 *     Calls on one stream are ordered by the stream; a captured graph uses the buffer of the
 *     stream it was captured on, so replaying it concurrently with other GEMM calls on that
 *     stream races.  Whether a shape splits depends only on the shape and the device, so
 *     repeated calls give bit-identical results.
 *   - `stream` is a hipStream_t (NULL = the null stream).  Calls enqueue work and return
 *     without synchronising, except w12_encode (see there).
 *   - Arguments are checked on the host before anything is launched; on a non-zero status
 *     nothing has been enqueued unless stated, and w12_last_error() returns a message
 *     (thread-local, valid until the next call on the same thread).  Faults inside kernels
 *     surface at the caller's next synchronisation, as usual in HIP.
 *   - k must be a multiple of 128 (W12_ERR_SHAPE otherwise) and at most 2^24, n below 2^31
 *     (W12_ERR_RANGE otherwise).
 */
#ifndef W12_H
#define W12_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define W12_ABI_VERSION 1

/* status codes */
#define W12_OK            0
#define W12_ERR_ARG      (-1)  /* null pointer, n, k or m <= 0, unknown flag */
#define W12_ERR_SHAPE    (-2)  /* k % 128 != 0 */
#define W12_ERR_ALIGN    (-3)  /* a device pointer is not 16-byte aligned */
#define W12_ERR_CAPACITY (-4)  /* esc_cap smaller than the escape total (w12_encode) */
#define W12_ERR_RANGE    (-5)  /* escape total >= 2^32 - 1, k > 2^24, n or m >= 2^31 */
#define W12_ERR_HIP      (-6)  /* HIP runtime or launch error; message from hipGetErrorString */

/* flags for the GEMM calls: which kernel family runs */
#define W12_PATH_AUTO 0u  /* the family measured fastest for the shape: the streaming kernel for
                           * 3 <= m <= 16 on shapes of at least 1.5 16-row tiles per compute unit
                           * and k <= 8192, for 17 <= m <= 32 on at least 2 tiles per unit
                           * (the 8-bit passes: 2 to 24; the dense baseline: 2 to 6), for
                           * 33 <= m <= 64 on 1.5 to 3 tiles per unit (the dense baseline:
                           * every shape), and above 64 rows on 1.5 to 2.5 (the dense baseline:
                           * at most 3); otherwise the GEMV
                           * with wave reductions for m <= 2, and for m <= 5 on shapes of at most
                           * 1024 tiles and k <= 8192; bf16 MFMA otherwise (w12_mx4_gemm: its own
                           * choice, stated there) */
#define W12_PATH_GEMV 1u  /* force the GEMV (m > 8 runs as several passes of <= 8 rows) */
#define W12_PATH_MFMA 2u  /* force the MFMA kernel (any m; columns padded to 16; passes of 32
                           * rows above 32 on shapes of fewer than 1.5 tiles per unit) */
#define W12_PATH_STREAM 3u /* force the streaming kernel (one workgroup per CU owning whole 16-row
                            * tiles, every wave of it an equal share of their 128-column blocks;
                            * passes of <= 64 rows of x; a wave finalises up to three tiles at
                            * 3..16 rows and two at 17..64 rows, and shapes with more tiles than
                            * that in equal row groups, all in one launch; W12_ERR_SHAPE when k is
                            * 2^26 or more or no phase length fits the LDS) */
/* w12_q8_gemm only, or-ed with a path: read the dropped B nibble as 8 (the midpoint of the 16
 * values the 8-bit view stands for) instead of 0; escapes stay exact */
#define W12_Q8_MIDPOINT 0x10u
/* flag for w12_gemm, w12_q8_gemm and w12_bf16_gemm: y is written as bfloat16 bits instead of
 * float -- each output is the float result of the same call without the flag, rounded to nearest
 * (ties to even; NaN stays NaN).  y then points to uint16_t [m][n] (2-byte aligned), passed as the
 * float* argument.  The rounding happens where the output is stored (the GEMM's epilogue, or the
 * ordered sum of a split-k launch), so no float copy of y is written; a GEMV whose x rows do not
 * fit LDS in one piece (several k slices) adds them in float in the GEMM workspace first.  The
 * error bound becomes 1e-3 * sum_k |x[m][k] * W[n][k]| plus half a bfloat16 unit in the last
 * place of the output. */
#define W12_OUT_BF16 0x20u

/* A W12 tensor: a non-owning view.  Every pointer is device memory owned by the caller. */
typedef struct w12_weight {
    int64_t   n;        /* output channels (rows of W)  */
    int64_t   k;        /* input features (columns of W) */
    uint8_t  *base;     /* [n]                           */
    uint8_t  *ae;       /* [npad * k]      tiled storage */
    uint8_t  *lo;       /* [npad * k / 2]  tiled storage */
    uint32_t *esc_ptr;  /* [n + 1]                       */
    uint32_t *esc_col;  /* [esc_cap]                     */
    uint16_t *esc_val;  /* [esc_cap]                     */
    uint64_t  esc_cap;  /* entries available in esc_col / esc_val */
} w12_weight;

/*
 * w12_encode -- bfloat16 W [n, k] (device, row-major) -> W12 record `out`.
 * Implements the plane split, window choice and escape list of Fig. 5(a) (figure-captions
 * page) under the rules above.  The result is byte-identical to a canonical CPU encoder.
 * Steps: per-row exponent histogram and window choice (writes base and per-row escape
 * counts), an in-place scan into esc_ptr, one synchronisation of `stream` to read the
 * escape total into *n_esc (host pointer), then the pack kernel writes ae, lo and the
 * escapes.  If out->esc_cap < *n_esc the call returns W12_ERR_CAPACITY after the sync:
 * base, esc_ptr and *n_esc are valid, ae/lo/escapes are not written; allocate and call
 * again.  out->n, out->k must be set by the caller.  n_esc may not be NULL.
 */
int w12_encode(const uint16_t *w, w12_weight *out, uint64_t *n_esc, void *stream);

/*
 * w12_decode -- W12 record -> bfloat16 bits W [n, k] (device, row-major).  Bit-exact inverse of
 * w12_encode (the format is lossless: figure-captions page, Fig. 5(a) "exact escape list";
 * summary page, "Key Contributions" 3).  Reads 1.5 bytes per weight plus metadata, writes 2.
 */
int w12_decode(const w12_weight *wt, uint16_t *w_out, void *stream);

/*
 * w12_gemm -- the exact pass: y[m][n] = sum_k x[m][k] * W[n][k], fp32 accumulate, fp32 y.
 * x is bfloat16 [m, k] (device, row-major), y is float [m, n] (device, row-major, fully
 * overwritten).  W is read only through its record: the planes are decoded to bfloat16 in
 * registers (figure-captions page, Fig. 5(b)) and each escape is patched exactly.
 * Error bound: |y - y_exact| <= 1e-3 * sum_k |x[m][k] * W[n][k]| per element.
 */
int w12_gemm(const uint16_t *x, int64_t m, const w12_weight *wt, float *y, uint32_t flags,
             void *stream);

/*
 * w12_gemm_noalloc -- w12_gemm for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc).  Same arguments, flags,
 * kernels and results as w12_gemm (bit-identical for every shape whose split-k partial sums and
 * 128-row passes fit the fixed scratch below, which covers every 27B-class projection).  The
 * scratch a call needs (split-k partial sums, the transposed x of passes of more than 64 rows)
 * comes from a fixed 16 MiB array of device memory in the library (W12_NOALLOC_SCRATCH_BYTES),
 * one per GPU, held from the library's first use on that GPU until the process ends; the call
 * itself allocates nothing (no hipMalloc, no allocating library routine).  Split-k ranges and
 * 128-row passes adapt to that size; a call that cannot fit -- bfloat16 outputs on the GEMV path
 * whose x rows need several k slices, with more than 16 MiB of float partial outputs
 * (min(m, 8) x n x 4 bytes) -- returns W12_ERR_RANGE before anything is enqueued.  Every call on
 * one GPU shares that GPU's array: calls that overlap in time on one GPU (on different streams, or
 * graphs replayed concurrently) race on it and must be ordered by the caller.  Nothing in the
 * array needs to start at zero; it keeps the last call's contents.
 */
#define W12_NOALLOC_SCRATCH_BYTES (16u << 20)
int w12_gemm_noalloc(const uint16_t *x, int64_t m, const w12_weight *wt, float *y, uint32_t flags,
                     void *stream);

/*
 * w12_q8_gemm -- the Q pass of two-level verification (figure-captions page, Fig. 7):
 * the same product with every in-window weight taken from the 8-bit view alone (A + E, the
 * B nibble read as 0, i.e. the bfloat16 bits & 0xFFF0) and escapes exact.  Reads base, ae
 * and the escape arrays only; wt->lo may be NULL.  Same shapes and error bound as
 * w12_gemm, against that truncated weight.  With W12_Q8_MIDPOINT in flags the in-window weight
 * is bits & 0xFFF0 | 0x8 instead (same bytes read, half the worst-case weight error).
 */
int w12_q8_gemm(const uint16_t *x, int64_t m, const w12_weight *wt, float *y, uint32_t flags,
                void *stream);

/*
 * w12_q8_top1 / w12_gemm_top1 -- the top-1 output of each row of x, for the Q pass (8-bit view,
 * as w12_q8_gemm) or the exact pass (as w12_gemm), without writing the [m, n] outputs: the
 * two-level verification compares only the argmax chain of the cheap pass with the exact one
 * (figure-captions page, Fig. 7; summary page, Main Findings: 98.7% top-1 agreement).
 * idx[j] (int32, device) = the n at which y[j][n] is largest, ties to the smallest n; val[j]
 * (float, device) = that y[j][n] (a NaN output counts as the largest).  Where the automatic path
 * of w12_q8_gemm / w12_gemm takes the streaming kernel for all m <= 32 rows, y is exactly that
 * path's output; otherwise y is computed exactly as the matrix-core path computes it for a shape
 * too large to split, in passes of up to 32 rows of x (each pass reads the weights once).  Either
 * kernel reduces its outputs to per-workgroup keys in the workspace instead of writing them, and
 * one small kernel per pass picks the winners.  Uses the GEMM workspace (see the conventions
 * above).
 * Same record checks as w12_q8_gemm / w12_gemm; idx and val 4-byte aligned.  flags: 0, or for
 * w12_q8_top1 W12_Q8_MIDPOINT (the midpoint view, as in w12_q8_gemm); anything else is
 * W12_ERR_ARG.
 */
int w12_q8_top1(const uint16_t *x, int64_t m, const w12_weight *wt, int32_t *idx, float *val,
                uint32_t flags, void *stream);
int w12_gemm_top1(const uint16_t *x, int64_t m, const w12_weight *wt, int32_t *idx, float *val,
                  uint32_t flags, void *stream);

/*
 * w12_interleave_rows -- the record of the gate and up projections of an MLP stacked with their
 * rows interleaved in groups of 8: output rows 16 t .. 16 t + 7 are gate rows 8 t .. 8 t + 7 and
 * rows 16 t + 8 .. 16 t + 15 are up rows 8 t .. 8 t + 7, so the two inputs of one
 * SiLU(gate) * up output sit in one 16-row tile (summary page, Main Findings: W12 also speeds up
 * plain decoding, where gate and up feed SiLU(gate) * up).  Built on the device from the two
 * records without decoding (windows and escape lists are per row); byte-identical to w12_encode
 * of the interleaved matrix.  gate and up: same [I, k], I % 8 == 0.  out: a record of
 * [2 I, k] sized for it.  Synchronises `stream` once to read the parts' escape totals into
 * *n_esc (host); if out->esc_cap is smaller, returns W12_ERR_CAPACITY before writing anything.
 */
int w12_interleave_rows(const w12_weight *gate, const w12_weight *up, w12_weight *out, uint64_t *n_esc,
                        void *stream);

/*
 * w12_gemm_silu_mul -- the exact pass on row-interleaved gate+up weights (w12_interleave_rows)
 * with the MLP activation applied where the outputs are stored: h[j][i] = silu(g) * u, where
 * g = y[j][16 (i / 8) + i % 8] and u = y[j][16 (i / 8) + i % 8 + 8] are the gate and up outputs of
 * w12_gemm on the same record and silu(z) = z / (1 + exp(-z)) in float.  x bfloat16 [m, k]; h is
 * float [m, n / 2] (or bfloat16 bits with W12_OUT_BF16: each h rounded to nearest even), fully
 * overwritten; wt->n % 16 == 0 (W12_ERR_SHAPE otherwise).  flags: W12_PATH_*, W12_OUT_BF16.
 * The y values are never written to memory except as split-k partial sums in the GEMM workspace.
 * Error bound per output, with B = 1e-3 * sum_k |x[j][k] W[row][k]| of each input row:
 * 1.1 B_g (|u| + B_u) + |silu(g)| B_u + 2^-20 |h| (1.1 bounds the slope of silu), plus half a
 * bfloat16 unit in the last place with W12_OUT_BF16.
 */
int w12_gemm_silu_mul(const uint16_t *x, int64_t m, const w12_weight *wt, float *h, uint32_t flags,
                      void *stream);

/*
 * The separate 8-bit copy for the Q pass (summary page, Main Findings: the RTX PRO 6000 port reads
 * an INT6/INT8 copy of the weights in the Q pass instead of the zero-copy 8-bit view).  It sits
 * beside a W12 record and shares that record's exact escape list.  The pages give no quantiser;
 * this one is linear per output row: M_n = the largest magnitude among the row's in-window
 * weights (2^(base - 127), the window's smallest magnitude, for a row with none), scale
 * s_n = M_n / 127 in float32, and every in-window weight becomes q = round-half-even(w / s_n)
 * (float32 division), clamped to +-127; escaped slots hold q = 0.  The Q pass then sees s_n * q
 * for in-window weights and the exact value for escapes.  1 byte per weight plus 4 per row, the
 * same bytes per pass as the 8-bit view, and 1 extra byte per weight of memory.
 */
typedef struct w12_i8 {
    int64_t  n;        /* rows of W (must equal the record's)    */
    int64_t  k;        /* columns of W (must equal the record's) */
    int8_t  *q;        /* [npad * k] codes, in the storage order of the record's AE plane (device, 16-byte aligned) */
    float   *scale;    /* [n] per-row scale (device, 4-byte aligned) */
} w12_i8;

/*
 * w12_i8_build -- the 8-bit copy of record `wt` into the caller's out->q and out->scale (out->n,
 * out->k set by the caller to the record's).  Reads the whole record (planes and escape list);
 * padding rows of the storage get code 0.  Enqueued on `stream`, no synchronisation.
 */
int w12_i8_build(const w12_weight *wt, w12_i8 *out, void *stream);

/*
 * w12_i8_gemm -- the Q pass on the 8-bit copy: y[m][n] = s_n * sum_k x[m][k] q[n][k] + the exact
 * escapes' products, fp32 accumulate.  Reads cp->q, cp->scale and wt's escape arrays (wt->base,
 * wt->ae and wt->lo are not read and may be NULL).  Same x, y, flags (W12_PATH_*, W12_OUT_BF16),
 * kernel families and error bound as w12_q8_gemm, against the weights s_n * q; more than 64 rows
 * of x run as passes of at most 64.  W12_Q8_MIDPOINT is W12_ERR_ARG.
 */
int w12_i8_gemm(const uint16_t *x, int64_t m, const w12_i8 *cp, const w12_weight *wt, float *y,
                uint32_t flags, void *stream);

/*
 * w12_i8_top1 -- top-1 of the Q pass on the 8-bit copy per row of x, as w12_q8_top1 (idx int32,
 * val float; ties to the smallest n); flags must be 0.
 */
int w12_i8_top1(const uint16_t *x, int64_t m, const w12_i8 *cp, const w12_weight *wt, int32_t *idx,
                float *val, uint32_t flags, void *stream);

/*
 * The microscaled 4-bit copy for the Q pass: block floating point with the element and block sizes
 * of the OCP microscaling formats (E2M1 elements, blocks of 32 columns, power-of-two scales),
 * beside a W12 record whose window bottoms and exact escape list it shares; 17/32 byte per weight.
 * Per block, e = the largest exponent field among its in-window weights (the window bottom for a
 * block with none), scale 2^(e - 129); an in-window weight becomes the code of the value nearest to
 * weight / scale among +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, ties to the even code, larger magnitudes
 * than 6 to 6; escaped slots hold code 0.  The Q pass then sees scale * value for in-window weights
 * and the exact value for escapes.
 * Storage: a record of 1088 bytes per tile of 16 rows x 128 columns, row-tile-major, rows padded
 * with zero bytes: for row r and column group g (columns 32 g .. +31) of the tile the 32 codes are the
 * 16 bytes at 16 (r + 16 g), column 2 i in the low and 2 i + 1 in the high nibble of byte i (sign in
 * bit 3), and the scale is the byte e - 2 - base + 112 (110..125) at 1024 + r + 16 g.
 */
typedef struct w12_mx4 {
    int64_t  n;        /* rows of W (must equal the record's)    */
    int64_t  k;        /* columns of W (must equal the record's) */
    uint8_t *q;        /* [npad * k * 17 / 32] tile records (device, 16-byte aligned) */
    /* the record's escapes that are not zero (a zero's slot holds code 0, so the product needs no
     * correction there), in the record's order: row i's are entries nz_ptr[i] .. nz_end[i] - 1; the
     * rows of a 16-row tile follow each other, tiles may have gaps between them */
    uint32_t *nz_ptr;  /* [n + 1], nz_ptr[n] = nz_end[n - 1]     */
    uint32_t *nz_end;  /* [n]                                    */
    uint32_t *nz_col;  /* [nz_cap]                               */
    uint16_t *nz_val;  /* [nz_cap]                               */
    uint64_t  nz_cap;  /* entries available, at least the record's esc_cap */
} w12_mx4;

/*
 * w12_mx4_build -- the 4-bit copy of record `wt` into the caller's arrays of `out` (out->n, out->k and
 * out->nz_cap set by the caller; W12_ERR_CAPACITY if nz_cap < wt->esc_cap).  Reads the planes and
 * the escape list.  Enqueued on `stream`, no synchronisation.
 */
int w12_mx4_build(const w12_weight *wt, w12_mx4 *out, void *stream);

/*
 * w12_mx4_decode -- the bfloat16 matrix [n, k] (device, row-major) the Q pass on the copy multiplies:
 * scale * value at in-window slots (exact in bfloat16), the record's own bits at escaped ones.  Reads
 * cp->q and wt's base and escape arrays (wt->ae and wt->lo may be NULL).
 */
int w12_mx4_decode(const w12_mx4 *cp, const w12_weight *wt, uint16_t *w_out, void *stream);

/*
 * w12_mx4_gemm / w12_mx4_top1 -- the Q pass on the 4-bit copy and its top-1 per row of x, as
 * w12_i8_gemm and w12_i8_top1 (same x, outputs, flags, workspace and error bound, against the weights
 * w12_mx4_decode gives).  Read the copy and wt->base (wt's other arrays may be NULL).  W12_PATH_AUTO
 * here: the GEMV at one row of x, and at two for k <= 8192 and at most 6 tiles per compute unit;
 * the matrix cores otherwise, in passes of up to 64 rows.  The top-1 takes y from the kernel of 32
 * rows a pass, so where w12_mx4_gemm runs another one their values differ in the last bits.  A row of
 * x with an infinity or a NaN gives infinities or NaN (an escaped slot's code 0 meets it too).
 */
int w12_mx4_gemm(const uint16_t *x, int64_t m, const w12_mx4 *cp, const w12_weight *wt, float *y,
                 uint32_t flags, void *stream);
int w12_mx4_top1(const uint16_t *x, int64_t m, const w12_mx4 *cp, const w12_weight *wt, int32_t *idx,
                 float *val, uint32_t flags, void *stream);

/*
 * w12_concat_rows -- the record of W = [W_0; W_1; ...; W_{count-1}] (the parts' rows stacked in
 * order) built on the device from the parts' records, without decoding or re-encoding.  Windows
 * and escape lists are per output row (figure-captions page, Fig. 5(a)), so the stacked record is
 * the parts' window bottoms, planes and escapes side by side, with the escape offsets rebased; it
 * is byte-identical to w12_encode of the stacked matrix.  Used to run projections that read the
 * same activations (q, k and v; gate and up) as one GEMM.
 * parts: host array of `count` (1..64) records; every part has the same k, and every part but
 * the last has n % 16 == 0 (whole 16-row tiles of the storage order).  out: a record whose n is
 * the sum of the parts' n and whose arrays are sized for it (ae npad*k, lo npad*k/2, base n,
 * esc_ptr n+1, esc_col/esc_val esc_cap entries).  Synchronises `stream` once to read the parts'
 * escape totals into *n_esc (host); if out->esc_cap is smaller, returns W12_ERR_CAPACITY before
 * writing anything.  The parts must not overlap `out`.
 */
int w12_concat_rows(const w12_weight *parts, int count, w12_weight *out, uint64_t *n_esc,
                    void *stream);

/*
 * w12_embed -- embedding lookup: out[j][c] = scale * W[ids[j]][c], with W read from its W12 record, so
 * a model whose embedding table is its LM head keeps one record for both ends of a step.  ids:
 * `count` int32, or int64 with W12_IDS_I64 (device, naturally aligned); an id outside 0 .. n-1
 * (padding) reads nothing and gives a row of zeros at any scale (-0 at a negative finite one).
 * out: [count][k] float (device, 16-byte aligned, fully overwritten): the weight times scale in
 * float; with W12_OUT_BF16 bfloat16 bits, that product rounded to nearest even, or for scale = 1 the
 * weight's own bits (NaN payloads and -0 included).  flags: W12_OUT_BF16, W12_IDS_I64.  Uses no
 * workspace.
 */
#define W12_IDS_I64 0x40u
int w12_embed(const void *ids, int64_t count, const w12_weight *wt, float scale, void *out,
              uint32_t flags, void *stream);

/*
 * w12_logprobs -- log probabilities of given tokens, entropy and the top alternatives of m rows of
 * logits (the outputs of a GEMM call over an LM head), in one pass over them: what a verification
 * step, a draft tree (the sum of log probabilities along a path orders its nodes: summary page,
 * best-first tree) or the scoring of a given text reads off the logits.
 * y: rows of n logits, row j at y + j * ldy elements (ldy >= n): float, 4-byte aligned, or
 * bfloat16 bits (W12_LOGITS_BF16), 2-byte aligned.  tokens: [m][n_tok] int32, or int64 with
 * W12_IDS_I64 (n_tok = 0: none, tokens and logp may be NULL).  Outputs (device, 4-byte aligned):
 *   logp[j][t]      = y[j][token] - log(sum_c e^y[j][c]); -Inf for a token outside 0 .. n-1
 *   entropy[j]      = -sum_c p log p (natural logarithm; p = 0 contributes 0)
 *   top_idx[j][i], top_logp[j][i], i < top: the columns of the `top` largest logits in descending
 *                     order and their log probabilities; equal logits (-0 equals +0) by the lower
 *                     column, a NaN logit above every number.  0 <= top <= 64 and top <= n
 *                     (W12_ERR_RANGE otherwise); with top = 0 both may be NULL.
 * -Inf logits (masked tokens) have probability 0.  A row of -Inf alone has no distribution: its
 * log probabilities are -Inf, its entropy 0, its alternatives columns 0 .. top-1.  A row with a NaN
 * or +Inf logit gives NaN log probabilities (a token outside 0 .. n-1 still -Inf) and entropy.
 * All sums are held in float; finite logits may have any magnitude; a logit whose e^(y - max) is below
 * 2^-126 may count as 0.  scratch: w12_logprobs_scratch bytes of device memory of the caller's
 * (16-byte aligned; NULL when that is 0; W12_ERR_CAPACITY if scratch_bytes is smaller), in use until
 * the call's work on `stream` is finished.  Its first bytes are counters that must be zero when
 * the work starts and are zero again when it ends: clear it once, then reuse it for calls of any
 * sizes that follow each other on one stream.  Calls with different scratch never touch each
 * other's, on any streams or in any graphs.
 */
#define W12_LOGITS_BF16 0x80u
int w12_logprobs_scratch(int64_t m, int64_t n, int top, uint32_t flags, uint64_t *bytes);
int w12_logprobs(const void *y, int64_t m, int64_t n, int64_t ldy, const void *tokens, int64_t n_tok,
                 int top, float *logp, float *entropy, int32_t *top_idx, float *top_logp,
                 void *scratch, uint64_t scratch_bytes, uint32_t flags, void *stream);

/*
 * The paged key/value cache of a decoding step, and the new tokens of a batch of sequences.
 *
 * A cache is pages of `page` token places for each of `heads` key/value heads of `dim` values:
 * element (p, h, r, c) of page p, head h, place r, column c lies at k (or v) + p * page_stride +
 * h * head_stride + r * token_stride + c elements, so a head's places may lie side by side
 * ([pages, heads, page, dim]) or a place's heads ([pages, page, heads, dim]).  Values are bfloat16, or with
 * W12_KV_E4M3 8-bit floats (OCP e4m3fn) that stand for value * k_scale[h] (v_scale[h]).
 */
#define W12_KV_E4M3 0x1u
typedef struct w12_kv {
    int64_t pages;        /* 1 .. 2^31 - 1                                      */
    int64_t heads;        /* key/value heads, at most 2^16                      */
    int64_t page;         /* token places of a page: a multiple of 16, at most 1024 */
    int64_t dim;          /* 64, 128 or 256                                     */
    void   *k, *v;        /* device, 16-byte aligned                            */
    int64_t page_stride;  /* in elements, multiples of 16 (8 in bfloat16), not negative; */
    int64_t head_stride;  /* the same for k and v                               */
    int64_t token_stride; /* at most 2^24                                       */
    const float *k_scale; /* [heads], W12_KV_E4M3 only (both NULL: 1)           */
    const float *v_scale;
    uint32_t flags;       /* W12_KV_E4M3 or 0                                   */
} w12_kv;

/*
 * The new tokens of a step: sequence s has lens[s] places in the cache, the last T_s of them its new
 * tokens; new token j is row q_start[s] + j of the step's rows, T_s = q_start[s + 1] - q_start[s]
 * (without q_start: row s, T_s = 1).  Its place is c = lens[s] - T_s + j, on page table[s][c / page].
 * Rows from q_start[seqs] on (padding) belong to no sequence: nothing is read or written for them.
 * All arrays are device memory, read when the work runs, so a captured graph takes new lengths and
 * tables on each replay.  A place outside the table, or on a page outside 0 .. pages - 1, does not exist:
 * nothing is appended there and nobody sees it.  A q_start may pass m: the rows below m exist, with the places
 * that they have among all T_s, the others are nothing.  q_start must not fall; with other values the result is
 * undefined (where sequences' rows below m add up to more than m, w12_attention writes nothing), but nothing
 * outside the arrays is accessed.
 */
typedef struct w12_kv_batch {
    int64_t seqs;             /* below 2^20                                        */
    const int32_t *table;     /* [seqs][table_cols], rows table_stride apart       */
    int64_t table_cols;       /* 1 .. 2^30 / page                                  */
    int64_t table_stride;
    const int32_t *lens;      /* [seqs]                                            */
    const int32_t *q_start;   /* [seqs + 1], or NULL                               */
    const int32_t *positions; /* [rows] position of the rotation, or NULL: the place */
    const uint64_t *tree;     /* [rows] masks, or NULL (w12_attention)             */
} w12_kv_batch;

/*
 * w12_kv_append -- rotates the new tokens' q and k by position and puts k and v into the cache.
 * q, k, v: rows of hq, kv->heads and kv->heads heads of kv->dim values, row i at q + i * ldq (k + i *
 * ldk, v + i * ldv) elements (16-byte aligned, strides multiples of 8, or of 4 in float): bfloat16 bits,
 * or float with W12_IN_F32 -- the rows of a GEMM over stacked q, k and v records, for instance.
 * rope: [rope_rows][rot] float, row p the cosines of position p's rot / 2 angles and then their sines
 * (16-byte aligned; rot a multiple of 16 up to dim; rot = 0: no rotation, rope NULL).  The pair (x_a, x_b)
 * becomes (x_a cos - x_b sin, x_b cos + x_a sin) in float, a = i, b = i + rot / 2, or with
 * W12_ROPE_PAIRS a = 2 i, b = 2 i + 1; columns from rot on stay.  Results are rounded once, to nearest
 * even: q to q_out [m][hq * dim] bfloat16, k and v to the cache's type (e4m3: divided by the scale and
 * clamped to +-448 first; NaN stays NaN).  q and q_out may be NULL (hq = 0).  A token without a place
 * in the cache, or with a position outside 0 .. rope_rows - 1, is not appended; the latter's row of
 * q_out is zero.  Two tokens with one place (a page shared by tables) leave either's values.
 * q_out may be q itself (bfloat16, ldq = hq * dim), and else must not overlap q, k or v.  Uses no workspace.
 */
#define W12_IN_F32     0x100u
#define W12_ROPE_PAIRS 0x200u
int w12_kv_append(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                  int64_t m, int64_t hq, const float *rope, int64_t rope_rows, int64_t rot,
                  const w12_kv *kv, const w12_kv_batch *batch, uint16_t *q_out, uint32_t flags, void *stream);

/*
 * w12_attention -- attention of the new tokens over the cache: y[i][h] = sum_t p_t v_t with p the
 * softmax over the places t that row i sees of scale * q[i][h] . k_t, keys and values of head h /
 * (hq / kv->heads); hq a multiple of kv->heads.  Row i, new token j of its sequence, sees the places
 * before the new tokens (t < lens - T) and of the new ones those up to its own -- or with batch->tree
 * those t = lens - T + b, b < min(T, 64), whose bit b its mask tree[i] has (the nodes of a draft tree on its path:
 * figure-captions page, Fig. 6).  A row that sees nothing, or only scores of -Inf, gives zeros.
 * Values of places that a row does not see never reach it, NaN and infinities included; a NaN or an
 * infinity it sees gives NaN or an infinity.  q: bfloat16, row i at q + i * ldq elements (16-byte aligned, ldq a multiple of 8); y:
 * [m][hq * dim] bfloat16 (16-byte aligned), rounded once to nearest even.  Scores, softmax and sums
 * are held in float, the probabilities that meet v in 16 significant bits (over an e4m3 cache in 22, but
 * in 11 where a key head has more than 32 rows of q a sequence on average, 16 at 256 columns).  Their products
 * add up before they are divided by the probabilities' sum: v times the places seen times 2^8 (e4m3: 2^15)
 * must stay below float's largest.  y may be q itself (ldq = hq * dim), and else must not overlap it.
 * scratch: w12_attention_scratch bytes of the caller's device memory (16-byte aligned), in use until
 * the call's work on `stream` is finished; what it holds before does not matter.  Calls with different
 * scratch never touch each other's.  Which places are summed together depends on the lengths of the
 * whole batch and the device; equal calls give equal bits.
 */
int w12_attention_scratch(int64_t m, int64_t hq, const w12_kv *kv, const w12_kv_batch *batch, uint64_t *bytes);
int w12_attention(const uint16_t *q, int64_t ldq, int64_t m, int64_t hq, const w12_kv *kv,
                  const w12_kv_batch *batch, float scale, uint16_t *y, void *scratch, uint64_t scratch_bytes,
                  uint32_t flags, void *stream);

/*
 * w12_sample -- a token for each of m rows of logits, drawn with the caller's random numbers.
 * y, n (at most 2^20), ldy and W12_LOGITS_BF16 as in w12_logprobs.  Per row (each array [m] on the device, or NULL
 * for the value that switches it off): temperature (NULL: 1), top_k (0 or less: off), top_p (1 or more,
 * or NaN: off), min_p (0 or less, or NaN: off), and u, the random number in [0, 1).
 * With x the row, M its largest logit and w_c = e^((x_c - M) / temperature), tokens are ordered by
 * descending logit, equal ones (-0 equals +0) by the lower column, and kept as follows:
 *   the first top_k of them, but none of -Inf;
 *   of those each one that the ones before it do not yet give the mass top_p * (mass of those);
 *   of those the ones with w >= min_p; the first token of the order always.
 * token[j] is the first kept column, in column order, at which the mass of the kept columns up to and with
 * it exceeds u * (mass of all kept) (u below 0 or NaN: as 0; 1 or more: the last kept column of any mass; w
 * below 2^-1000 is no mass),
 * logp[j] = ln(w / mass of all kept) its log probability among the kept ones, kept[j] their number
 * (token or logp or kept may be NULL).  A temperature of 0 or less takes the first token of the order.
 * A row of -Inf alone gives token -1, logp -Inf and kept 0, one with a NaN or +Inf logit, or a
 * temperature of NaN, token -1, logp NaN and kept 0.
 * Weights and sums that decide are held in double or, where thousands are kept, in integers of 2^-61 of what may
 * be kept (in the sum of a whole row, weights below 2^-24 of those around them to float's 24 bits), in a fixed
 * order: equal calls give equal results.  flags: W12_LOGITS_BF16.
 * scratch: w12_sample_scratch bytes of the caller's device memory (16-byte aligned), in use until the
 * call's work on `stream` is finished; its contents on entry do not matter.
 */
int w12_sample_scratch(int64_t m, int64_t n, uint32_t flags, uint64_t *bytes);
int w12_sample(const void *y, int64_t m, int64_t n, int64_t ldy, const float *temperature, const int32_t *top_k,
               const float *top_p, const float *min_p, const float *u, int32_t *token, float *logp,
               int32_t *kept, void *scratch, uint64_t scratch_bytes, uint32_t flags, void *stream);

/*
 * w12_bf16_gemm -- same-build dense baseline: y = x * W^T with W bfloat16 in the same tiled
 * storage order as the W12 planes (npad * k values, from w12_bf16_to_tiles), same kernel
 * structure and flags as w12_gemm, 2 bytes per weight.
 */
int w12_bf16_gemm(const uint16_t *x, int64_t m, const uint16_t *w_tiles, int64_t n, int64_t k,
                  float *y, uint32_t flags, void *stream);

/*
 * w12_bf16_to_tiles -- dense bfloat16 W [n, k] (device, row-major) -> the tiled storage order of
 * the baseline (out: npad * k values; padding rows zero).  Inside a tile (16 rows x 128 columns,
 * 4096 bytes) the 8 values of row r at columns 32g + 8q .. +7 sit at byte 1024*q + 16*(r + 16g).
 */
int w12_bf16_to_tiles(const uint16_t *w, int64_t n, int64_t k, uint16_t *out, void *stream);

/*
 * w12_read_probe -- bandwidth probe: streams `bytes` bytes of `buf` (device, 16-byte
 * aligned, bytes % 16 == 0) with 128-bit loads and writes one word per workgroup of a
 * checksum to `sink` (device, at least 4096 u32).  Measures the achievable HBM read rate.
 */
int w12_read_probe(const void *buf, uint64_t bytes, uint32_t *sink, void *stream);

/*
 * w12_release_workspace -- frees the GEMM workspace of (current device, `stream`), if the
 * library allocated one (see the conventions above), for callers that create and destroy
 * streams (per request or per thread): without it a destroyed stream's 64 MiB stay allocated
 * until the process ends.  Waits for the stream's work first (hipStreamSynchronize), then frees
 * the buffer; a later GEMM call on the stream allocates a new one.  Graphs captured on the
 * stream still point at the freed buffer: do not replay them after this call.  Returns W12_OK
 * whether or not there was a buffer; not for use while `stream` is being captured.
 */
int w12_release_workspace(void *stream);

/* Message for the last non-zero status returned on this thread ("" if none). */
const char *w12_last_error(void);

/* W12_ABI_VERSION of the loaded library. */
int w12_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* W12_H */
