/*
 * zpq.h -- C ABI of libzpq: block-quantized communication kernels of ZeRO++
 * (qwZ and qgZ) for AMD Instinct MI355X (gfx950).
 *
 * Sources (web pages about "ZeRO++: Extremely Efficient Collective
 * Communication for Giant Model Training", arXiv 2306.10209):
 *   [SUM] atlas.scime.ai summary page ("ZeRO++: ... for Large Model Training")
 *   [ABS] mlsanity.com index page, section "Abstract (arXiv)"
 *   [LIT] anthology-of-the-sota record LIT-102, section "Key takeaways"
 *
 * Quantizer (the pages say only "block-wise"; it is fixed here as follows):
 *   a block is `block` consecutive elements; its scale is
 *   s = fl32(max|x| / qmax) with qmax = 127 (INT8) or 7 (INT4); each code is
 *   q = clamp(round_half_even(fl32(x / s)), -qmax, qmax) using IEEE fp32
 *   division; a block whose scale is 0 has all codes 0.  Dequantization is
 *   d = fl32(q * s), rounded to nearest even into the output type.  INT4
 *   codes are two's-complement nibbles, two per byte, element 2k in the low
 *   nibble of byte k.  Results are bit-identical to that definition for all
 *   finite inputs, with two qualifications: where the definition itself
 *   produces a NaN (a reduced sum that meets +inf and -inf), the result is a
 *   NaN of unspecified sign and payload; and a block whose reduced sums are
 *   not all finite has unspecified INT4 codes and scale (the quantizer is
 *   defined on finite values only).  Non-finite inputs give unspecified (but
 *   in-bounds) results.
 *
 * Conventions shared by every entry point:
 *   - All buffer arguments are DEVICE pointers owned by the caller; the
 *     library allocates nothing, keeps no state between calls and never
 *     synchronizes.  Work is enqueued on `stream` (a hipStream_t; NULL is the
 *     null stream) and the call returns before it completes.
 *   - Arguments are checked on the host before anything is launched; on any
 *     error nothing is launched and nothing is written.  Checked: pointers
 *     non-NULL (may be NULL only when there are no elements), 16-byte aligned,
 *     and input and output ranges disjoint; sizes non-negative and whole
 *     blocks (callers pad, as ZeRO pads partitions); block in
 *     {32, 64, 128, 256, 512}; element types valid.
 *   - Element counts are 64-bit, at most 2^40 (else ZPQ_ERR_SIZE); buffers
 *     above 2^31 bytes are supported.
 *   - ZPQ_ERR_LAUNCH reports a launch failure from the HIP runtime (for
 *     example a device other than gfx950), read with hipGetLastError after
 *     the launches: an error left pending by an earlier HIP call on the same
 *     host thread is reported (and cleared) the same way.
 *   - Calls that write the same output concurrently race; calls on one
 *     stream are ordered.
 */
#ifndef ZPQ_H
#define ZPQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ZPQ_ABI_VERSION 1

typedef enum {
    ZPQ_OK = 0,
    ZPQ_ERR_NULL = 1,    /* a required pointer is NULL */
    ZPQ_ERR_SIZE = 2,    /* negative size, or not a whole number of blocks / slices */
    ZPQ_ERR_BLOCK = 3,   /* block not in {32, 64, 128, 256, 512} */
    ZPQ_ERR_ALIGN = 4,   /* a pointer is not 16-byte aligned */
    ZPQ_ERR_DTYPE = 5,   /* element type not supported by this entry point */
    ZPQ_ERR_MODE = 6,    /* not exactly one output mode selected */
    ZPQ_ERR_LAUNCH = 7,  /* the HIP runtime refused the launch */
    ZPQ_ERR_ARG = 8,     /* other invalid argument (L, N, n_src, divisor) */
    ZPQ_ERR_ALIAS = 9    /* an output range overlaps an input range */
} zpq_status;

/* Element types of float tensors (passed as int32_t). */
typedef enum { ZPQ_F32 = 0, ZPQ_F16 = 1, ZPQ_BF16 = 2 } zpq_dtype;

typedef void* zpq_stream; /* hipStream_t */

/*
 * qwZ quantize: INT8 block quantization of a weight shard before the forward
 * all-gather ([SUM] "Approach": block-wise INT8 quantization of weights for
 * the forward all-gather; [ABS]: block-quantization based all-gather).
 *
 *   x      [n] elements of type x_dtype (ZPQ_F32, ZPQ_F16 or ZPQ_BF16)
 *   codes  [n] int8 codes in [-127, 127], same order as x        (written)
 *   scales [n / block] fp32 scales, one per block, in order       (written)
 */
zpq_status zpq_quant_i8(const void* x, int32_t x_dtype, int64_t n, int32_t block,
                        int8_t* codes, float* scales, zpq_stream stream);

/*
 * qwZ dequantize: the gathered INT8 buffer back to a float type after the
 * all-gather ([SUM] "Approach"; [ABS]).  A gathered buffer of W shards is the
 * concatenation of their codes and of their scales, so this is one call.
 *
 *   codes  [n] int8, scales [n / block] fp32
 *   y      [n] elements of type y_dtype: RNE(fl32(q * s))          (written)
 */
zpq_status zpq_dequant_i8(const int8_t* codes, const float* scales, int64_t n,
                          int32_t block, void* y, int32_t y_dtype, zpq_stream stream);

/*
 * Non-blocked (per-tensor) INT8 quantization: one scale for the whole tensor.
 * The ablation baseline of qwZ ([SUM] Measured effects table: basic
 * non-blocked instead of block-based quantization, which hurt convergence;
 * Surprising findings: naive non-blocked INT8 weights diverged).
 *
 *   x      [n] elements of type x_dtype; n % 16 == 0 (callers pad with zeros)
 *   codes  [n] int8 codes in [-127, 127]                          (written)
 *   scale  [1] fp32: fl32(max|x| / 127)                            (written)
 * The codes buffer also holds intermediate per-workgroup maxima during the
 * call (three kernels on `stream`); nothing else is touched.
 */
zpq_status zpq_quant_i8_tensor(const void* x, int32_t x_dtype, int64_t n, int8_t* codes,
                               float* scale, zpq_stream stream);

/*
 * qgZ, before the intra-node all-to-all: tensor-slice reordering fused with
 * INT4 block quantization ([SUM] "Approach": slice reordering for correct
 * placement ahead of a 2-hop all-to-all of INT4 gradients; [ABS]: all-to-all
 * based quantized gradient averaging in place of reduce-scatter).
 *
 * The W = L*N ranks are numbered r = node*L + local; rank r owns flat slice r
 * of S = n / W elements.  Send position p = j*N + m (j < L, m < N) carries
 * slice m*L + j, so that after hop 1 (chunk j -> local rank j) and hop 2
 * (position m of a chunk -> node m) every slice sits at its owner.
 *
 *   grad   [n] elements of type g_dtype; n % (L*N*block) == 0
 *   codes  [n / 2] bytes: packed INT4 codes of the reordered tensor;
 *          bytes [j*n/(2L), (j+1)*n/(2L)) are the hop-1 chunk for local rank j
 *   scales [n / block] fp32 scales of the reordered tensor (chunk j is
 *          [j*n/(L*block), (j+1)*n/(L*block)))
 */
zpq_status zpq_qgz_reorder_quant_i4(const void* grad, int32_t g_dtype, int64_t n,
                                    int32_t local_ranks, int32_t nodes, int32_t block,
                                    uint8_t* codes, float* scales, zpq_stream stream);

/*
 * qgZ, after each all-to-all hop: dequantize the n_src received INT4 chunks,
 * reduce them in fp32 in source order 0..n_src-1 starting from +0 (one
 * rounding per addition, no fused multiply-add), then either
 *   mode I4 (hop 1): requantize the sum to INT4 with the same block size;
 *            the result is the hop-2 send buffer (position m = slice for
 *            node m)   -- out_codes [chunk/2], out_scales [chunk/block];
 *   mode FLOAT (hop 2): y = RNE_out(fl32(sum / divisor)) -- the averaged
 *            gradient slice; divisor is the world size W  -- out_vals [chunk]
 *            of type out_dtype (ZPQ_F32, ZPQ_F16 or ZPQ_BF16).
 * Exactly one mode: (out_codes, out_scales non-NULL and out_vals NULL) or
 * the reverse, else ZPQ_ERR_MODE.  FLOAT mode needs 0 < divisor < inf.
 * ([SUM] "Approach" and "Surprising findings": dequantize before reduction,
 * two hops, intra-node then inter-node; [LIT] second bullet: reduction done
 * locally in higher precision.)
 *
 *   in_codes  [n_src][chunk/2] bytes, source-major (as received)
 *   in_scales [n_src][chunk/block] fp32
 * Scales must be finite.
 */
zpq_status zpq_qgz_dequant_reduce_requant_i4(const uint8_t* in_codes, const float* in_scales,
                                             int32_t n_src, int64_t chunk_elems, int32_t block,
                                             uint8_t* out_codes, float* out_scales,
                                             void* out_vals, int32_t out_dtype, float divisor,
                                             zpq_stream stream);

/* ------------------------------------------------------------------------
 * The ends of the step around qwZ and qgZ: the averaged gradient slice of hop
 * 2 goes into zpq_adamw_step, whose 16-bit copy of the weights is what qwZ
 * quantizes for the next all-gather; the gathered INT8 table is read by
 * zpq_embedding_i8 as it is; zpq_embedding_grad makes the table's gradient,
 * which qgZ sends.  (The pages name the optimizer step only as what follows
 * the gradient average; these operators are defined here.)
 *
 * They follow the conventions above, except that sizes need not be whole
 * blocks and that pointers need the alignment of their element only: 16-byte
 * alignment is faster, not required.
 */

/* Bytes of device memory that a table of `count` tensors takes, for
 * zpq_list_make and for zpq_adamw_plan_make (16-byte aligned). */
#define ZPQ_LIST_BYTES(count) ((int64_t)(count) * 32 + 20736)
#define ZPQ_PLAN_BYTES(count) ((int64_t)(count) * 128 + 64)

/* A list of tensors of one type: a table in the caller's device memory, and
 * what the host has to know of it.  Filled by zpq_list_make; the table's
 * contents (addresses among them) stand until it is made again.  The table also
 * holds the partial sums of the zpq_grad_sumsq call that runs on it, so calls on
 * one list must be ordered (one stream, or events). */
typedef struct {
    void* table;
    int64_t elems;     /* of all tensors */
    int64_t chunks;    /* workgroup shares */
    int32_t count;
    int32_t dtype;
} zpq_list;

/*
 * Describe `count` tensors: ptrs[i] holds sizes[i] elements of type `dtype`
 * (NULL only where sizes[i] is 0).  The table is written by small kernels on
 * `stream`, so later work on that stream sees it; ptrs and sizes are host
 * arrays and may go when the call returns.
 */
zpq_status zpq_list_make(const void* const* ptrs, const int64_t* sizes, int32_t count,
                         int32_t dtype, void* table, int64_t table_bytes, zpq_list* list,
                         zpq_stream stream);

/*
 * Sum of squares over a list (the squared norm that clipping needs; ranks add
 * theirs): out[0] = sum of g^2, or out[0] += with accumulate, in binary64
 * throughout, in an order that depends on the sizes and the number of compute
 * units only.  One launch.
 */
zpq_status zpq_grad_sumsq(const zpq_list* list, double* out, int32_t accumulate, zpq_stream stream);

/* One tensor of an optimizer step; all device pointers.  The tensors of one
 * plan must not overlap one another, nor a tensor's own parts. */
typedef struct {
    void* p;             /* [n] weights                                    (updated) */
    const void* g;       /* [n] gradient */
    void* m;             /* [n] first moment: fp32, or 8-bit codes         (updated) */
    void* v;             /* [n] second moment: fp32 >= 0, or 8-bit codes   (updated) */
    uint8_t* m_exp;      /* [ceil(n/256)] exponent bytes of 8-bit states, else NULL */
    uint8_t* v_exp;      /* [ceil(n/256)] likewise                         (updated) */
    void* copy;          /* [n] the new weights in copy_dtype, or NULL     (written) */
    int64_t n;
    double weight_decay;
} zpq_adamw_tensor;

typedef struct {
    void* table;
    int64_t elems, chunks;
    int32_t count, p_dtype, g_dtype, copy_dtype, state_bits;
} zpq_adamw_plan;

/*
 * Lay out `count` tensors for zpq_adamw_step.  p_dtype and g_dtype: any element
 * type.  copy_dtype: ZPQ_F16 or ZPQ_BF16 with p_dtype ZPQ_F32 and every copy
 * set, or -1 and every copy NULL (ZPQ_ERR_MODE otherwise).  state_bits: 32
 * or 8.  table, table_bytes, stream: as in zpq_list_make.
 */
zpq_status zpq_adamw_plan_make(const zpq_adamw_tensor* tensors, int32_t count, int32_t p_dtype,
                               int32_t g_dtype, int32_t copy_dtype, int32_t state_bits,
                               void* table, int64_t table_bytes, zpq_adamw_plan* plan,
                               zpq_stream stream);

typedef struct {
    double lr, beta1, beta2, eps;  /* lr >= 0, 0 <= beta < 1, eps >= 1e-30 */
    double grad_scale;             /* > 0: gradients are multiplied by it (loss scale, averaging) */
    double max_norm;               /* > 0: largest norm of the scaled gradients; infinity: none */
    int64_t step;                  /* >= 1: which step this is, for the bias corrections */
    uint64_t seed;                 /* of the random numbers that round 8-bit states */
} zpq_adamw_hyper;

/*
 * One AdamW step over all tensors of a plan, element by element:
 *   c  = fl32(grad_scale * min(1, max_norm / (grad_scale * sqrt(sumsq) + 1e-6)))
 *   g' = g * c
 *   m' = beta1 * m + (1 - beta1) * g'
 *   v' = beta2 * v + ((1 - beta2) * g') * g'
 *   p' = p * (1 - lr * weight_decay)
 *        - lr / (1 - beta1^step) * (m' / (sqrt(v') / sqrt(1 - beta2^step) + eps))
 * in binary32, one rounding an operation (the root within 1 ulp, the quotient
 * as a product with a reciprocal within 1 ulp), the constants rounded once from
 * binary64; p' is rounded to nearest even into p_dtype and copy_dtype.  (A v'
 * that rounds to 0 in binary32, below 2^-150, leaves eps alone in the quotient.)
 *
 * sumsq: device pointer to the squared norm of the unscaled gradients (all
 * ranks'), or NULL: c = fl32(grad_scale), and max_norm must be infinite
 * (ZPQ_ERR_ARG).  A sumsq that is not finite leaves every output as it was.
 *
 * 8-bit states: blocks of 256 consecutive elements of a tensor (the last one
 * may be short) have one exponent byte e >= 1, the binary32 exponent field of
 * the block's largest magnitude after rounding it up to 3 fraction bits.  m
 * is a sign, a 4-bit exponent field f and 3 fraction bits q, v a 5-bit field
 * and 3 fraction bits: with T = 15 or 31 the value is
 * (1 + q/8) * 2^(f - T + e - 127), or q/8 * 2^(1 - T + e - 127) for f = 0.
 * New states are rounded up or down at random, up with the probability of the
 * distance, 16 random bits a value: an average that a step moves by 1 part in
 * a thousand would stand still under rounding to nearest.  A v' above 0 never
 * becomes 0.  A block with a value that is not finite, or over 1.875 * 2^127,
 * becomes infinite as a whole.  The random bits are a hash of (seed, step,
 * element): element i of tensor t counts as b_t + i, b_t the sum of the sizes
 * before t, each rounded up to 256.
 */
zpq_status zpq_adamw_step(const zpq_adamw_plan* plan, const zpq_adamw_hyper* hyper,
                          const double* sumsq, zpq_stream stream);

/*
 * The same with the hyperparameters in device memory, read when the step runs: a
 * captured graph replays zpq_adamw_step with the step number that it was captured
 * with, and this one with whatever *hyper holds by then (an earlier node may count
 * hyper->step up).  Values out of range leave every output as it was; max_norm is
 * not looked at where sumsq is NULL.  Two launches; the first writes into the plan's
 * table, so calls on one plan must be ordered.
 */
zpq_status zpq_adamw_step_at(const zpq_adamw_plan* plan, const zpq_adamw_hyper* hyper,
                             const double* sumsq, zpq_stream stream);

/* 8-bit states to and from float tensors (checkpoints); moment: 1 (m) or 2
 * (v).  Packing rounds to nearest even, magnitudes of v (its sign is lost);
 * blocks as above, of one tensor of n elements. */
zpq_status zpq_state8_unpack(const uint8_t* codes, const uint8_t* exps, int64_t n, int32_t moment,
                             void* y, int32_t y_dtype, zpq_stream stream);
zpq_status zpq_state8_pack(const void* x, int32_t x_dtype, int64_t n, int32_t moment,
                           uint8_t* codes, uint8_t* exps, zpq_stream stream);

/*
 * Embedding lookup: out row t = RNE(scale * table row (ids[t] - first)), the
 * product in binary32; a row of zeros where ids[t] - first is not in [0, rows)
 * (padding, or a row of another shard of the vocabulary).
 *   table [rows] rows of dim elements of type t_dtype, ld_table elements apart
 *   ids   [tokens] of 4 or 8 bytes (id_bytes)
 *   out   [tokens] rows of dim elements of type out_dtype, ld_out apart
 * zpq_embedding_i8 reads the table as qwZ gathers it: INT8 codes [rows * dim]
 * and one fp32 scale for each `block` of them (rows need not be whole blocks;
 * scales [ceil(rows * dim / block)]); its row element is fl32(code * scale).
 * dim >= 1, ld >= dim; tokens, rows < 2^31.
 */
zpq_status zpq_embedding(const void* table, int32_t t_dtype, int64_t rows, int64_t dim,
                         int64_t ld_table, const void* ids, int32_t id_bytes, int64_t tokens,
                         int64_t first, float scale, void* out, int32_t out_dtype, int64_t ld_out,
                         zpq_stream stream);
zpq_status zpq_embedding_i8(const int8_t* codes, const float* scales, int64_t rows, int64_t dim,
                            int32_t block, const void* ids, int32_t id_bytes, int64_t tokens,
                            int64_t first, float scale, void* out, int32_t out_dtype,
                            int64_t ld_out, zpq_stream stream);

/*
 * Gradient of the lookup, dense: for each row r
 *   grad[r] = RNE([grad[r] +] fl32(scale * sum of dy[t] over t with ids[t] - first = r))
 * (with accumulate the fp32 sum of both is rounded once, and rows without a
 * token are not touched; without, they become zeros).  The sum is in binary32,
 * in an order that depends on the ids and the sizes only: the tokens are sorted by
 * row, equal rows in token order, and long rows are summed in parts; no
 * floating-point atomics.  Ids outside [first, first + rows) and ids
 * equal to `padding` count for nothing (give padding = -1, or any id outside,
 * for none).
 *   dy    [tokens] rows of dim elements of type dy_dtype, ld_dy apart
 *   grad  [rows] rows of dim elements of type grad_dtype, ld_grad apart
 *   workspace: zpq_embedding_grad_bytes bytes of device memory, 16-byte
 *   aligned, contents irrelevant
 * tokens <= 2^28, rows <= 2^27, dim <= 2^28.
 */
zpq_status zpq_embedding_grad_bytes(int64_t tokens, int64_t rows, int64_t dim, int64_t* bytes);
zpq_status zpq_embedding_grad(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* ids,
                              int32_t id_bytes, int64_t tokens, int64_t first, int64_t padding,
                              int64_t rows, int64_t dim, float scale, void* grad,
                              int32_t grad_dtype, int64_t ld_grad, int32_t accumulate,
                              void* workspace, int64_t workspace_bytes, zpq_stream stream);

/* ------------------------------------------------------------------------
 * Matrix products of the step, from 8-bit floating-point blocks.  A rank quantizes
 * its rows of a weight in tiles (zpq_quant_f8); whole tiles gather by
 * concatenation as qwZ's codes do, and the products take the gathered buffer as it
 * is.  (Defined here, as the operators above; the same conventions.)
 *
 * A matrix [rows, cols] in 8-bit floating point, quantized along its rows:
 *   codes   [rows][128 * kb] bytes, kb = ceil(cols / 128): OCP E4M3 or E5M2; codes
 *           past the last column are 0 (0 or NaN in a block with a value that is not finite)
 *   scales  [rows][kb4] exponent bytes, kb4 = kb rounded up to a multiple of 4; those
 *           past kb are 0.  One for each 128 elements of a row, or in tiles, [ceil(rows / 128)][kb4]:
 *           one for each 128 x 128.
 * An element is code * 2^(byte - 127).  With a the block's largest magnitude, byte is
 * the smallest for which a <= 1.75 * 2^t * 2^(byte - 127), t = 8 for E4M3 and 15 for E5M2
 * (the format's largest value), at least 0; code = RNE(x * 2^(127 - byte)).  A
 * block with a value that is not finite has byte 255 and NaNs for codes.
 * Pointers to codes and scales are 16-byte aligned.  128 * kb at most 2^23.
 */
typedef enum { ZPQ_E4M3 = 0, ZPQ_E5M2 = 1 } zpq_f8_kind;

/*
 * Quantize x, `rows` rows of cols elements of x_dtype, ld apart: along its rows into codes
 * and scales, along its columns into codes_t [cols][128 * ceil(rows / 128)] and scales_t
 * (the transposed matrix along its rows), or both at once; each pair may be NULL, not
 * both (ZPQ_ERR_MODE).  With tile, blocks are 128 x 128, and both pairs hold the same values.
 * x needs its element's alignment; rows * kb below 2^28, and of tiles and column
 * blocks below 2^24 squares of 128 x 128.
 */
zpq_status zpq_quant_f8(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ld,
                        int32_t kind, int32_t tile, uint8_t* codes, uint8_t* scales,
                        uint8_t* codes_t, uint8_t* scales_t, zpq_stream stream);

/* Values back, rounded to nearest even into y_dtype: y [rows] rows of cols elements, ld apart. */
zpq_status zpq_dequant_f8(const uint8_t* codes, int32_t kind, const uint8_t* scales, int64_t rows,
                          int64_t cols, int32_t tile, void* y, int32_t y_dtype, int64_t ld,
                          zpq_stream stream);

/* The transposed matrix of one in tiles, the same values: [cols][128 * ceil(rows / 128)]. */
zpq_status zpq_transpose_f8(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                            uint8_t* codes_t, uint8_t* scales_t, zpq_stream stream);

typedef struct {
    const uint8_t* codes;
    const uint8_t* scales;
    int32_t kind;        /* zpq_f8_kind */
    int32_t tile;        /* scales of 128 x 128 */
} zpq_f8_operand;

/*
 * out = [out +] A * B^T for A [m, k] and B [n, k]:
 *   out[i][j] = RNE([out[i][j] +] sum over k of a[i][k] * b[j][k])
 * with exact products and sums in binary32, in an order that depends on the sizes and on
 * whether results are bf16 only.
 *   ZPQ_F32 and ZPQ_F16 results: elements are multiplied as 16-bit floats of binary32's range,
 *   which holds them exactly, at half the rate; a binary16 result is the binary32 one rounded.  An
 *   element over the largest binary32 is infinite there, and one below 2^-126 may count as 0.
 *   ZPQ_BF16 results: the 8-bit matrix instructions add the products of 8 consecutive elements
 *   (0 to 7, 8 to 15, ...) in units of 2^-13 of the largest's power of two, cutting off what lies
 *   below, also where the large ones cancel: at most 7 * 2^-13 of the largest product of each 8
 *   (quantizing changes an element by up to 2^-4 of it, E5M2 2^-3).  As a root mean square that is
 *   1e-5 of a sum of like values, 5e-5 (9e-5) with one element in a hundred 30 (1000) times as
 *   large; the result's rounding is 1.7e-3.
 * With x, dy the input and output gradient [tokens, .] and w [outputs, inputs]: y = x w^T;
 * dx = dy w takes w's transposed tiles for B; dw = dy^T x takes both along their columns.
 *   out [m] rows of n elements of out_dtype, ld apart; read with accumulate only
 *   workspace: zpq_matmul_f8_bytes bytes of device memory (0 for most sizes),
 *   16-byte aligned, contents irrelevant
 * m < 2^31, n <= 2^26, ceil(m / 64) * ceil(n / 64) < 2^23; k = 0 is a sum of nothing.  Whole
 * blocks are summed: codes past k count, and are 0 as quantized.
 */
zpq_status zpq_matmul_f8_bytes(int64_t m, int64_t n, int64_t k, int64_t* bytes);
zpq_status zpq_matmul_f8(const zpq_f8_operand* a, const zpq_f8_operand* b, int64_t m, int64_t n,
                         int64_t k, void* out, int32_t out_dtype, int64_t ld, int32_t accumulate,
                         void* workspace, int64_t workspace_bytes, zpq_stream stream);

/* ------------------------------------------------------------------------
 * Orthogonalising updates, and the Muon step of a layer's matrices beside AdamW's of the
 * rest.  Conventions as above.
 *
 * The Newton-Schulz iteration on a matrix U [rows, cols]:
 *   X = U / |U|_F (0 where the norm is 0), transposed while rows > cols
 *   for each of `steps` triples (a, b, c) in coeffs [steps][3], a host array:
 *       A = X X^T;  X = a X + (b A + c A A) X
 * which drives the singular values that are not 0 to about 1: with (3.4445, -4.7750, 2.0315)
 * five times, to between 0.7 and 1.2.  Products take 16-bit operands (11 bits), with
 * sums and X itself in binary32.  As a root mean square the result is within 2.5e-3 of the exact
 * iteration's (less for large matrices and low ranks), 3.5e-3 where only a few rows or columns
 * differ or are not 0, so that roundings add up; so it comes in 16 bits.  A side up to 32 goes in
 * 64 bits, to the result's own rounding.  A matrix with a value that is not finite comes out as NaN.
 * 1 <= steps <= 32, coefficients at most 64 in size, such that the entries of A and of
 * b A + c A A stay under 60 (binary16 at the operands' scale; over it results are not finite).
 * rows, cols <= 2^22, rows * cols <= 2^34.
 */
/*
 * out_i = iteration(x_i) for `count` matrices of one shape, at most 2^20.
 *   x     [rows] rows of cols elements of x_dtype, ld_x apart, matrices stride_x apart
 *   out   likewise; out_dtype ZPQ_F16 or ZPQ_BF16
 *   workspace: zpq_orthogonalize_bytes bytes of device memory, 256-byte aligned,
 *   contents irrelevant: ZPQ_MUON_BYTES(count), and room for the matrices that are worked on at a
 *   time, consecutive ones up to 2^26 elements and 2^30 bytes, one at least, with up to 2^29 bytes
 *   for parts of long sums.  A matrix takes about 14 bytes an element; one with a side up to
 *   32 takes 4, and 32 for each element of the other side, 13 KB at least.
 */
zpq_status zpq_orthogonalize_bytes(int64_t count, int64_t rows, int64_t cols, int64_t* bytes);
zpq_status zpq_orthogonalize(const void* x, int32_t x_dtype, int64_t count, int64_t rows,
                             int64_t cols, int64_t ld_x, int64_t stride_x, const double* coeffs,
                             int32_t steps, void* out, int32_t out_dtype, int64_t ld_out,
                             int64_t stride_out, void* workspace, int64_t workspace_bytes,
                             zpq_stream stream);

/* One matrix of a Muon step, rows * cols consecutive elements each; device
 * pointers.  The matrices of a plan must not overlap, nor a matrix's own parts. */
typedef struct {
    void* p;             /* weights                                        (updated) */
    const void* g;       /* gradient */
    void* m;             /* momentum, fp32                                 (updated) */
    void* copy;          /* the new weights in copy_dtype, or NULL         (written) */
    int64_t rows, cols;
    double weight_decay; /* >= 0 */
    double scale;        /* >= 0: of the orthogonal update; 0.2 * sqrt(max(rows, cols)) gives it
                            about the size of an AdamW update */
} zpq_muon_matrix;

typedef struct {
    void* memory;
    const zpq_muon_matrix* matrices;   /* the host array, which has to stay as it is */
    int32_t count, p_dtype, g_dtype, copy_dtype;
} zpq_muon_plan;

/* Device memory of a plan's table alone; zpq_muon_plan_bytes: with the workspace, which
 * is bounded as zpq_orthogonalize's. */
#define ZPQ_MUON_BYTES(count) ((int64_t)(count) * 248 + 64)

/*
 * Lay out `count` matrices for zpq_muon_step, at most 2^20.  Types as in zpq_adamw_plan_make.  The
 * table in memory (256-byte aligned) is written by small kernels on `stream`; the rest of the
 * memory is the step's workspace, so steps of one plan must be ordered.
 */
zpq_status zpq_muon_plan_bytes(const zpq_muon_matrix* matrices, int32_t count, int64_t* bytes);
zpq_status zpq_muon_plan_make(const zpq_muon_matrix* matrices, int32_t count, int32_t p_dtype,
                              int32_t g_dtype, int32_t copy_dtype, void* memory,
                              int64_t memory_bytes, zpq_muon_plan* plan, zpq_stream stream);

typedef struct {
    double lr, momentum;           /* lr >= 0, 0 <= momentum < 1 */
    double grad_scale, max_norm;   /* as in zpq_adamw_hyper */
    const double* coeffs;          /* host, [steps][3] */
    int32_t steps, nesterov;
} zpq_muon_hyper;

/*
 * One Muon step of all matrices of a plan:
 *   g' = g * c, with c from grad_scale, max_norm and sumsq as in zpq_adamw_step
 *   m' = momentum * m + g'
 *   u  = nesterov ? g' + momentum * m' : m'
 *   p' = p * (1 - lr * weight_decay) - lr * scale * iteration(u)
 * elementwise operations in binary32, one rounding each, the iteration as above; p' is
 * rounded to nearest even into p_dtype and copy_dtype.  A sumsq that is not finite
 * leaves every output as it was.
 */
zpq_status zpq_muon_step(const zpq_muon_plan* plan, const zpq_muon_hyper* hyper,
                         const double* sumsq, zpq_stream stream);

/* Human-readable name of a status code (static string, never NULL). */
const char* zpq_status_str(zpq_status s);

/* ZPQ_ABI_VERSION of the loaded library. */
int32_t zpq_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ZPQ_H */
