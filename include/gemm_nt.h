/*
 * gemm_nt.h -- C ABI of the GB300 (sm_103a) fp16 -> fp32 matrix product
 *
 *     Out = A @ B.T
 *
 * with A (M,K) and B (N,K) row-major IEEE binary16, Out (M,N) row-major float32,
 * float32 accumulation.  This is the product computed by the two worked examples
 * of the Apache TVM TIRx programming guides: "Warp Matrix Instructions" (opening
 * paragraph and "From Shared Memory to a Matrix Product": A (16,16), B (8,16),
 * ldmatrix + mma.sync m16n8k16, fp32 accumulators) and "Blackwell Tensor Cores"
 * ("The Accumulator's Lifetime": A (128,64), B (64,64), tcgen05.mma kind::f16
 * with the fp32 accumulator in Tensor Memory).  Both examples start a fresh
 * accumulator (C = 0, accum=False), so Out is overwritten: there is no alpha,
 * beta or C input.
 *
 * The pages run each kernel as compiled(a, b, out) on torch CUDA tensors (the
 * listings that compile the kernel and compare it with torch, in "Warp Matrix
 * Instructions" and "Blackwell Tensor Cores") and define no C interface.  The
 * entry points here take that call's three operands as device pointers, in the
 * same order (A, B, Out), followed by the sizes, the leading dimensions, the
 * batch strides and batch count where there are any, and the stream.  Status
 * codes 0-6 are those of the plain and batched products; 7 and 8 belong to the
 * entry points that choose a kernel or allocate nothing.
 *
 * Conventions shared by every entry point
 *   - Pointers A, B, Out are DEVICE pointers owned by the caller.  A and B hold
 *     fp16 bit patterns (__half / uint16_t).  The library keeps no reference to
 *     them after the call's work has run.
 *   - Sizes and leading dimensions are in ELEMENTS; rows are contiguous:
 *       A[i,k] = A[i*lda + k],  B[j,k] = B[j*ldb + k],  Out[i,j] = Out[i*ldo + j].
 *     Batched forms add b*strideA, b*strideB, b*strideO elements for batch b.
 *   - Calls are asynchronous and ordered on `stream` (a cudaStream_t / CUstream;
 *     NULL = the legacy default stream).  Argument errors are detected on the
 *     host, return immediately and launch nothing.
 *   - Empty cases: M == 0, N == 0 or batch == 0 -> GEMM_OK, nothing launched.
 *     K == 0 -> Out is filled with zeros (the empty sum).
 *   - Any alignment is accepted.  The tensor-core kernels need 16-byte aligned
 *     A/B bases and lda, ldb (and strideA, strideB) multiples of 8 elements;
 *     other inputs run on the warp-MMA kernel, which accepts any layout.
 *   - Device-side failures (a bounded wait inside a kernel that ran out) are
 *     recorded in a per-device status word and reported by gemm_nt_check().
 *   - Thread safety: all entry points may be called concurrently from several
 *     host threads.  Calls whose Out ranges overlap must not run concurrently.
 *   - Only devices of compute capability 10.3 (GB300, sm_103a) are supported.
 *   - Per-device set-up (kernel attributes, the status word's address) is done
 *     once, by the first call on a device that passes the argument checks (a
 *     set-up that failed is tried again by the next call), and kept for the
 *     life of the process: after cudaDeviceReset() on a device, make no further
 *     call on that device.
 */
#ifndef GEMM_NT_H
#define GEMM_NT_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t and CUstream. */
struct CUstream_st;
typedef struct CUstream_st *gemm_stream_t;

typedef enum gemm_status {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_VALUE = 1,      /* null pointer, negative size, ld < row length, ... */
    GEMM_ERR_MISALIGNED = 2,         /* reserved, never returned: layouts the tensor-core kernels
                                        cannot read run on the warp-MMA kernel instead */
    GEMM_ERR_OVERLAP = 3,            /* Out overlaps A or B, or batches of Out overlap */
    GEMM_ERR_LAUNCH = 4,             /* a CUDA runtime/driver call failed (launch, tensor map,
                                        synchronisation, per-device set-up) */
    GEMM_ERR_DEVICE_TIMEOUT = 5,     /* a kernel's bounded wait ran out; Out is undefined */
    GEMM_ERR_UNSUPPORTED_DEVICE = 6, /* current device is not compute capability 10.3 */
    /* Codes 7 and 8 belong to entry points beyond the plain and batched products: */
    GEMM_ERR_NOT_SUPPORTED = 7,      /* the requested kernel cannot take these arguments */
    GEMM_ERR_SCRATCH_TOO_SMALL = 8   /* gemm_nt_f16_f32_batched_no_alloc: the call needs more
                                        scratch than the library's fixed array holds;
                                        gemm_nt_moe: than the workspace given */
} gemm_status_t;

/* Element types of gemm_nt_batched_ex. */
typedef enum gemm_dtype {
    GEMM_DTYPE_F16 = 0,  /* IEEE binary16 */
    GEMM_DTYPE_BF16 = 1, /* bfloat16: the upper half of an IEEE binary32 */
    GEMM_DTYPE_F32 = 2,  /* IEEE binary32 (Out only) */
    GEMM_DTYPE_E4M3 = 3, /* 8-bit float, 4 exponent bits (bias 7), 3 fraction bits, no infinities,
                            largest value 448 (A and B only) */
    GEMM_DTYPE_E5M2 = 4, /* 8-bit float, 5 exponent bits (bias 15), 2 fraction bits: the upper byte
                            of an IEEE binary16 (A and B only) */
    /* 6- and 4-bit floats (A and B only), no infinities or NaN, packed along K with
       little-endian bit order: element k of a row occupies bits [b*k, b*k + b) of the
       row's bit string (b = 6 or 4; byte i holds bits [8i, 8i + 8)), so fp4 holds
       element 2t in the low nibble of byte t and element 2t+1 in its high nibble: */
    GEMM_DTYPE_E2M3 = 5, /* sign bit 5, 2 exponent bits (bias 1), 3 fraction bits; largest 7.5 */
    GEMM_DTYPE_E3M2 = 6, /* sign bit 5, 3 exponent bits (bias 3), 2 fraction bits; largest 28 */
    GEMM_DTYPE_E2M1 = 7  /* sign bit 3, 2 exponent bits (bias 1), 1 fraction bit; largest 6 */
} gemm_dtype_t;

/* Kernel choice.  GEMM_PATH_AUTO lets the library pick (see gemm_nt_select_path). */
typedef enum gemm_path {
    GEMM_PATH_AUTO = 0,
    GEMM_PATH_TC05 = 1,     /* persistent tcgen05 kernel, TMEM accumulator, one CTA per tile */
    GEMM_PATH_SKINNY = 2,   /* tcgen05 with swapped operands and split K, for small M */
    GEMM_PATH_MMASYNC = 3,  /* ldmatrix + mma.sync m16n8k16 warp kernel, any layout */
    GEMM_PATH_TC05_PAIR = 4, /* tcgen05 on a CTA pair (cta_group::2), 256-row tiles */
    GEMM_PATH_TC05_M64 = 5,  /* one CTA per 64-row tile, plain M = 64 tcgen05.mma (few rows of A) */
    GEMM_PATH_TC05_WS = 6    /* one CTA per 32- or 64-row tile, weight-stationary tcgen05.mma.ws
                                (M = 32 when M <= 32, else 64) */
} gemm_path_t;

/*
 * Out = A @ B.T for one problem.
 *   A   : M x K, leading dimension lda >= K
 *   B   : N x K, leading dimension ldb >= K
 *   Out : M x N float32, leading dimension ldo >= N; must not overlap A or B.
 * Returns GEMM_OK once the work is enqueued on `stream`.
 */
gemm_status_t gemm_nt_f16_f32(const void *A, const void *B, float *Out,
                              int64_t M, int64_t N, int64_t K,
                              int64_t lda, int64_t ldb, int64_t ldo,
                              gemm_stream_t stream);

/*
 * Strided batch of independent products: for b < batch,
 *   Out_b = A_b @ B_b.T,  A_b = A + b*strideA,  B_b = B + b*strideB,  Out_b = Out + b*strideO.
 * strideA or strideB may be 0 (the operand is shared by every batch); strideO
 * must separate the batches of Out (strideO >= (M-1)*ldo + N when batch > 1).
 */
gemm_status_t gemm_nt_f16_f32_batched(const void *A, const void *B, float *Out,
                                      int64_t M, int64_t N, int64_t K,
                                      int64_t lda, int64_t ldb, int64_t ldo,
                                      int64_t strideA, int64_t strideB, int64_t strideO,
                                      int64_t batch, gemm_stream_t stream);

/*
 * As gemm_nt_f16_f32_batched, on an explicitly chosen kernel.  Returns
 * GEMM_ERR_NOT_SUPPORTED (and launches nothing) if that kernel cannot take the
 * arguments, e.g. a tensor-core path with unaligned A.  GEMM_PATH_TC05_M64 and
 * GEMM_PATH_TC05_WS ("Blackwell Tensor Cores" names the M = 64 and the
 * weight-stationary tcgen05.mma forms beside its 128-row example) put 64 rows
 * of A (32 on the weight-stationary form when M <= 32) on each tile's MMA
 * side; they take the same inputs as GEMM_PATH_TC05 except block scales and
 * an MN-major A (GEMM_ERR_NOT_SUPPORTED).  GEMM_PATH_AUTO never picks them.
 * A path value outside gemm_path_t: GEMM_ERR_INVALID_VALUE.
 */
gemm_status_t gemm_nt_f16_f32_batched_path(const void *A, const void *B, float *Out,
                                           int64_t M, int64_t N, int64_t K,
                                           int64_t lda, int64_t ldb, int64_t ldo,
                                           int64_t strideA, int64_t strideB, int64_t strideO,
                                           int64_t batch, gemm_path_t path,
                                           gemm_stream_t stream);

/*
 * The strided batched product with other element types: A and B both fp16 or
 * both bf16 ("Warp Matrix Instructions", "Other Fragment Shapes and
 * Transfers", names the float16 and bfloat16 forms of the warp MMA; the
 * tcgen05 kind::f16 MMA of "Blackwell Tensor Cores" takes either), products
 * accumulated in fp32 as always, and Out stored as fp32, or rounded to nearest
 * even into fp16 or bf16 (Out's element size is then 2 bytes; ldo and strideO
 * still count elements).  Same conventions, layouts and error behaviour as
 * gemm_nt_f16_f32_batched_path; gemm_nt_f16_f32_batched_path(...) equals
 * gemm_nt_batched_ex(..., GEMM_DTYPE_F16, GEMM_DTYPE_F32, ...).  An fp16 Out
 * overflows to infinity beyond 65504.  Products that would split K across CTAs
 * (few output tiles, long K) run on whole tiles when Out is not fp32, since
 * the partial sums are kept in fp32 only.
 *
 * A and B may also both be 8-bit floats (E4M3 or E5M2; lda, ldb and the batch
 * strides then count bytes), or both one of the 6- and 4-bit floats E2M3,
 * E3M2, E2M1, packed along K (lda, ldb and the batch strides count elements
 * and must start every row on a byte: multiples of 2 for E2M1, of 4 for the
 * 6-bit types; K-major only, else GEMM_ERR_INVALID_VALUE).  The packed types run
 * on the tcgen05 kernels only (kind::f8f6f4, whose tensor maps spread every 16
 * packed elements to a 16-byte chunk of shared memory), which need K a
 * multiple of 128, A and B 32-byte aligned, and pitches and batch strides of
 * whole multiples of 32 bytes; other layouts, and the warp kernel path, give
 * GEMM_ERR_NOT_SUPPORTED.  "Blackwell Tensor Cores" names the block-scaled
 * low-precision forms of the tcgen05 MMA beside kind::f16; these run on its
 * kind::f8f6f4 form without scale factors (products exact, fp32 accumulation),
 * at twice the fp16 rate.  The tensor-core kernels want 16-byte aligned bases
 * and pitches that are multiples of 16; other layouts, and MN-major 8-bit
 * operands (gemm_nt_batched_major), run on the warp kernel, which widens the
 * 8-bit values to fp16 (exact).  Any other dtype value: GEMM_ERR_INVALID_VALUE.
 */
gemm_status_t gemm_nt_batched_ex(const void *A, const void *B, void *Out,
                                 gemm_dtype_t ab_type, gemm_dtype_t out_type,
                                 int64_t M, int64_t N, int64_t K,
                                 int64_t lda, int64_t ldb, int64_t ldo,
                                 int64_t strideA, int64_t strideB, int64_t strideO,
                                 int64_t batch, gemm_path_t path, gemm_stream_t stream);

/* Storage order of one operand of gemm_nt_batched_major.  The operand is the
 * logical (rows, K) matrix of the product (A: rows = M; B: rows = N).
 *   GEMM_MAJOR_K : element (r, k) at base[r*ld + k], ld >= K  -- row-major (rows, K),
 *                  the layout of every other entry point;
 *   GEMM_MAJOR_MN: element (r, k) at base[k*ld + r], ld >= rows -- row-major (K, rows),
 *                  i.e. the operand's transpose stored row-major. */
typedef enum gemm_major {
    GEMM_MAJOR_K = 0,
    GEMM_MAJOR_MN = 1
} gemm_major_t;

/*
 * The product Out[b] = A[b] @ B[b].T with each operand stored K-major or
 * MN-major: with B MN-major, B is given as a row-major (K, N) matrix and the
 * call computes the plain row-major product A @ B ("NN"); with A MN-major too,
 * A is given as (K, M) and the call computes A.T @ B ("TN").  "Warp Matrix
 * Instructions" ("Other Fragment Shapes and Transfers") names ldmatrix's
 * .trans form, and "copy -> ldstmatrix" ("Algorithm" step 3) selects it for a
 * column-major shared tile whose column stride is a multiple of 8 elements:
 * the warp kernel stages an MN-major operand that way.  The tcgen05 kernels
 * (the pages show them K-major only) read it through the instruction
 * descriptor's transpose bit and an MN-major 128-byte-swizzled shared-memory
 * descriptor, as the PTX ISA defines them.
 *
 * Arguments as gemm_nt_batched_ex, plus a_major and b_major; lda and ldb are
 * the row pitches of the stored matrices (ld >= K for K-major, ld >= M or N
 * for MN-major) and strideA / strideB the batch strides, all in elements.
 * gemm_nt_batched_ex(...) equals this call with both operands GEMM_MAJOR_K.
 * The tensor-core kernels need 16-byte aligned A/B bases and ld, strides that
 * are multiples of 8 elements (else the warp kernel runs, as for K-major).
 * An MN-major operand on the CTA-pair kernel always uses 256-wide tiles, and
 * the skinny kernel's row split (an even share of rows per CTA) is K-major
 * only.  Any other major value: GEMM_ERR_INVALID_VALUE.
 */
gemm_status_t gemm_nt_batched_major(const void *A, gemm_major_t a_major, const void *B,
                                    gemm_major_t b_major, void *Out,
                                    gemm_dtype_t ab_type, gemm_dtype_t out_type,
                                    int64_t M, int64_t N, int64_t K,
                                    int64_t lda, int64_t ldb, int64_t ldo,
                                    int64_t strideA, int64_t strideB, int64_t strideO,
                                    int64_t batch, gemm_path_t path, gemm_stream_t stream);

/*
 * Block-scaled 8-bit product ("Blackwell Tensor Cores", on the other TMEM
 * operations: tcgen05.cp brings the scale factors of a block-scaled MMA into
 * Tensor Memory; the MMA reference it points to lists block scaling).  A and B
 * are E4M3, E5M2, E2M3, E3M2 or E2M1 (both the same), K-major, as in
 * gemm_nt_batched_ex; every
 * run of 32 consecutive K elements of a row of A (of B) shares one scale, an
 * E8M0 byte e standing for 2^(e-127) (255 is NaN), and
 *   Out[b,i,j] = sum_k (A[b,i,k] * 2^(sa[b,i,k/32]-127)) * (B[b,j,k] * 2^(sb[b,j,k/32]-127))
 * accumulated in fp32 on the tcgen05 kind::mxf8f6f4 MMA, Out fp32, fp16 or
 * bf16.
 *
 * SA and SB hold the scales in the packed atom layout (device memory, 16-byte
 * aligned): for each 128 rows and each 128 elements of K one 512-byte atom
 * whose byte 16*r + 4*q + s is the scale of row 32*q + r of the row block, K
 * block s of the K block group; atoms stored row block-major, so atom
 * (rb, kg) is at byte (rb * ceil(K/128) + kg) * 512; rows and K blocks past
 * the matrix are ignored (any value but 255).  One matrix of scales takes
 * gemm_nt_mx_scale_bytes(rows, K) bytes; the matrices of a batch follow one
 * another, except that an operand with batch stride 0 (shared by every batch)
 * has one matrix of scales.  gemm_nt_mx_pack_scales makes this layout from
 * the plain one.
 *
 * path: GEMM_PATH_AUTO, GEMM_PATH_TC05 (128 x 64 or 128 x 128 tiles),
 * GEMM_PATH_SKINNY (M <= 64) or GEMM_PATH_TC05_PAIR (256 x 256 tiles on CTA
 * pairs when Out rows are 32-byte aligned and K is not split, else 256 x 192);
 * AUTO takes SKINNY for M <= 64 and N >= 1024, the pairs for M and N
 * above 128, else TC05.  The warp kernel takes no scales
 * (GEMM_ERR_NOT_SUPPORTED), nor does any kernel a layout the tensor-core
 * kernels cannot read (unaligned bases, pitches not multiples of 16 bytes).  Null SA / SB with K > 0, a 16-bit ab_type, or
 * unaligned SA / SB: GEMM_ERR_INVALID_VALUE; Out overlapping A, B, SA or SB:
 * GEMM_ERR_OVERLAP.  Other arguments and errors as gemm_nt_batched_ex.
 */
gemm_status_t gemm_nt_mx(const void *A, const void *SA, const void *B, const void *SB, void *Out,
                         gemm_dtype_t ab_type, gemm_dtype_t out_type,
                         int64_t M, int64_t N, int64_t K,
                         int64_t lda, int64_t ldb, int64_t ldo,
                         int64_t strideA, int64_t strideB, int64_t strideO,
                         int64_t batch, gemm_path_t path, gemm_stream_t stream);

/* Bytes of one packed scale matrix for `rows` rows and K elements of K:
 * ceil(rows/128) * ceil(K/128) * 512; -1 for negative arguments. */
int64_t gemm_nt_mx_scale_bytes(int64_t rows, int64_t K);

/*
 * Packs block scales on the device: `plain` holds, for each of `batch`
 * matrices (batch stride `stride` bytes, 0 = one shared matrix), `rows` rows of
 * ceil(K/32) E8M0 bytes with row pitch `ld` bytes (ld >= ceil(K/32));
 * `packed` receives batch * gemm_nt_mx_scale_bytes(rows, K) bytes in the
 * layout gemm_nt_mx reads (padding atoms filled with 127).  Stream-ordered;
 * GEMM_ERR_INVALID_VALUE for null pointers or pitches too small.
 */
gemm_status_t gemm_nt_mx_pack_scales(const void *plain, int64_t ld, int64_t stride, void *packed,
                                     int64_t rows, int64_t K, int64_t batch, gemm_stream_t stream);

/*
 * Products with one fp32 scale for each block of 128 elements of K.
 *
 * A gemm_scale128_t describes the scales of one operand, a logical
 * (rows_of_operand / rows, ceil(K/128)) fp32 matrix in device memory (4-byte
 * aligned) with any strides, in elements: the scale of row r and K block c
 * (elements [128c, 128c+128)) of batch b is
 *   data[b*batch_stride + (r / rows)*row_stride + c*kb_stride].
 * rows is 1 (a scale for each row: activations, gradients) or 128 (a scale for
 * each 128 x 128 block: weights).  gemm_nt_block128_quantize leaves scales with
 * rows == 1 K block by K block (row_stride 1), the order the kernels read
 * without gathering.
 */
typedef struct gemm_scale128 {
    const float *data;
    int32_t rows;          /* 1 or 128 */
    int64_t row_stride;    /* >= 0 */
    int64_t kb_stride;     /* >= 0 */
    int64_t batch_stride;  /* >= 0; 0: shared by every batch */
} gemm_scale128_t;

/*
 * The 8-bit product with those scales:
 *   Out[b,i,j] = sum_c sa[b,i,c] * sb[b,j,c] * sum_{k in block c} A[b,i,k] * B[b,j,k]
 * A and B both E4M3 or both E5M2, K-major, the last K block as long as K leaves
 * it.  The inner sums are exact products accumulated in fp32 by the tensor
 * cores; they are scaled and summed over c in fp32 registers.  Out is fp32, or
 * that sum rounded once to nearest even into fp16 or bf16.  sa and sb may hold
 * any fp32 values: a block's term is right wherever it lies in fp32's normal range,
 * whatever sa * sb, or the inner sum times one of them, would be on the way (scales
 * below 2^-94, E4M3 2^-109, or above 2^80 cost time).  Infinities and NaN follow IEEE
 * arithmetic.
 *
 * path: GEMM_PATH_AUTO, GEMM_PATH_TC05_PAIR (256 x 256 tiles on CTA pairs),
 * GEMM_PATH_SKINNY (128 rows of B by up to 128 rows of A per CTA, K split over
 * a cluster when there are few tiles) or GEMM_PATH_MMASYNC (warp MMA, any
 * layout).  The first two need 16-byte aligned A and B with lda, ldb and batch
 * strides that are multiples of 16, else GEMM_ERR_NOT_SUPPORTED; AUTO takes the
 * warp kernel then.  Other paths: GEMM_ERR_NOT_SUPPORTED.  Null scales with
 * K > 0, rows other than 1 or 128, negative scale strides or other types:
 * GEMM_ERR_INVALID_VALUE; Out overlapping an operand or its scales:
 * GEMM_ERR_OVERLAP.  Other arguments and errors as gemm_nt_batched_ex; the
 * result does not depend on the run (no atomics).
 */
gemm_status_t gemm_nt_block128(const void *A, const gemm_scale128_t *SA, const void *B, const gemm_scale128_t *SB,
                               void *Out, gemm_dtype_t ab_type, gemm_dtype_t out_type,
                               int64_t M, int64_t N, int64_t K,
                               int64_t lda, int64_t ldb, int64_t ldo,
                               int64_t strideA, int64_t strideB, int64_t strideO,
                               int64_t batch, gemm_path_t path, gemm_stream_t stream);

/*
 * Quantises X (rows x cols, fp32, fp16 or bf16, row pitch ldx) into the
 * operands gemm_nt_block128 reads.  For each block of 1 x 128 (SQ->rows == 1)
 * or 128 x 128 (SQ->rows == 128) elements, with F the type's largest value (448
 * for E4M3, 57344 for E5M2),
 *   a = max(max |x|, 2^-100),  scale = a * (1/F),  q = round_to_nearest_even(x * (F * (1/a)))
 * with every step rounded to fp32; a NaN in a block makes its scale NaN, an infinity makes
 * the scale infinite and the infinite elements NaN.
 *
 * Q (rows x cols, pitch ldq bytes) and its scales SQ, or QT (cols x rows, pitch
 * ldqt) and its scales ST, or both are written, in one pass over X: QT is X
 * transposed, quantised in blocks of its own rows (128 rows of X each) -- the
 * operand of the product that sums over X's rows, a weight gradient.  Null Q
 * (then SQ is ignored) or null QT leaves that form out.  With both, SQ->rows
 * and ST->rows agree; with 128 both hold the same values and scales.  The
 * scales' data are written here although the struct's pointer is const.
 * Scale matrices must not overlap themselves (row_stride and kb_stride that
 * separate the elements).  Empty X: GEMM_OK, nothing launched.  Errors:
 * GEMM_ERR_INVALID_VALUE as elsewhere; GEMM_ERR_OVERLAP when an output overlaps
 * X or another output (the byte spans, counting pitches).
 */
gemm_status_t gemm_nt_block128_quantize(const void *X, gemm_dtype_t x_type, int64_t rows, int64_t cols, int64_t ldx,
                                        void *Q, int64_t ldq, const gemm_scale128_t *SQ,
                                        void *QT, int64_t ldqt, const gemm_scale128_t *ST,
                                        gemm_dtype_t q_type, gemm_stream_t stream);

/*
 * A mixture-of-experts layer for a few tokens, in two kernels.  For token t
 * with router logits l (fp32, `experts` of them, row pitch ldl):
 *   e_0, e_1, ... = the `topk` largest logits, best first, ties to the lower
 *                   index; an expert whose logit is -inf is never taken
 *   p_j = exp(l[e_j] - l[e_0]) / sum, the sum over the chosen experts
 *         (renormalize != 0) or over all of them (softmax first)
 *   h_j = silu(Wg x) * (Wu x),  silu(v) = v / (1 + exp(-v)),
 *         Wg = W13[e_j] rows [0, inner), Wu = W13[e_j] rows [inner, 2*inner)
 *   Out[t] = sum_j p_j * W2[e_j] h_j
 * A token whose logits are all -inf gets zeros.  A NaN among a token's logits
 * makes its row NaN, as softmax does.
 *
 * X (tokens x hidden) and Out (tokens x hidden) have x_type fp16 or bf16; W13
 * (experts x 2*inner x hidden) and W2 (experts x hidden x inner), row pitches
 * ldw13 and ldw2, expert strides strideW13 and strideW2, are of x_type, or
 * E4M3 with scales S13 and S2 (rows 1 or 128, batch_stride the expert stride;
 * null for 16-bit weights).  Only the weights of experts that a token chose are
 * read.  x and the weights are multiplied exactly (8-bit weights widened to 16
 * bits) and accumulated in fp32, by the tensor cores over 64 elements of K at a time and
 * to nearest over those; h is computed in fp32 and multiplied in two parts
 * that hold at least 16 significant bits of it; Out is rounded once to x_type.
 * Sums over experts follow the expert index, so results do not depend on the run.
 *
 * topk below 1 or above experts: GEMM_ERR_INVALID_VALUE.  tokens <= 128, experts <=
 * 1024, topk <= 32, hidden and inner <= 2^20: more is GEMM_ERR_NOT_SUPPORTED.
 * `workspace` (device memory, 16-byte aligned, the
 * caller's, at least gemm_nt_moe_workspace_bytes(tokens, topk, inner) bytes) is
 * overwritten; less is GEMM_ERR_SCRATCH_TOO_SMALL.  Out or the workspace overlapping
 * an operand, its scales or each other: GEMM_ERR_OVERLAP.  Any pitch and alignment is
 * accepted; rows that start on 16-byte boundaries are read fastest.  tokens or
 * hidden 0: nothing to do.  inner 0: Out is zero whatever the logits, weights and
 * workspace are not looked at and any number of tokens will do.
 */
gemm_status_t gemm_nt_moe(const void *X, int64_t ldx, const float *logits, int64_t ldl,
                          const void *W13, int64_t ldw13, int64_t strideW13, const gemm_scale128_t *S13,
                          const void *W2, int64_t ldw2, int64_t strideW2, const gemm_scale128_t *S2,
                          void *Out, int64_t ldo, gemm_dtype_t x_type, gemm_dtype_t w_type,
                          int64_t tokens, int64_t experts, int64_t topk, int64_t hidden, int64_t inner,
                          int renormalize, void *workspace, int64_t workspace_bytes, gemm_stream_t stream);

/* Bytes of workspace gemm_nt_moe needs (-1 for negative arguments, and where the number
 * would not fit). */
int64_t gemm_nt_moe_workspace_bytes(int64_t tokens, int64_t topk, int64_t inner);

/* Activations of the gated product. */
typedef enum gemm_act {
    GEMM_ACT_SILU = 0,      /* g / (1 + exp(-g)) */
    GEMM_ACT_GELU = 1,      /* g (1 + erf(g / sqrt 2)) / 2 */
    GEMM_ACT_GELU_TANH = 2  /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */
} gemm_act_t;

/*
 * The first half of a gated feed-forward block, in one kernel:
 *   g = X Wg^T,  u = X Wu^T,  H = act(g) * u
 * with Wg = W13 rows [0, inner) and Wu = W13 rows [inner, 2*inner).  X (tokens x
 * hidden, row pitch ldx), W13 (2*inner x hidden, row pitch ldw) and H (tokens x
 * inner, row pitch ldh) are all fp16 or all bf16 (`type`).  g and u are accumulated and
 * multiplied in fp32; H is rounded once.  GU (tokens x 2*inner, row pitch ldgu; null to
 * leave it out) receives g and u, each rounded to `type`, for gemm_nt_gated_grad.
 *
 * path: GEMM_PATH_AUTO, or one of
 *   GEMM_PATH_SKINNY     a stream of the weights on the warp MMA: up to 16 tokens, and
 *                        tokens * hidden (rounded up to 64) <= 65536
 *   GEMM_PATH_TC05       tcgen05 with the weights as rows: up to 64 tokens
 *   GEMM_PATH_TC05_PAIR  tcgen05 on CTA pairs, 256 tokens x 128 columns of H
 *   GEMM_PATH_MMASYNC    warp MMA, any layout
 * SKINNY needs W13 on 16-byte boundaries (base and ldw), TC05 and TC05_PAIR X (base and
 * ldx) too, a matrix of a single row its base alone; a path that cannot take the
 * arguments, and the other paths, are GEMM_ERR_NOT_SUPPORTED.  AUTO takes one that can, by
 * the tokens and the weights' bytes; paths differ in the order of their sums.
 *
 * tokens or inner 0: nothing to do; hidden 0: zeros; hidden above 2^30 or inner above
 * 2^30 - 1: GEMM_ERR_INVALID_VALUE.  Any pitch and alignment is
 * accepted; rows that start on 16-byte boundaries are read fastest.  Outputs that
 * overlap an operand or each other (the byte spans, counting pitches):
 * GEMM_ERR_OVERLAP.  Infinities and NaN follow IEEE arithmetic.  Nothing is allocated,
 * no two calls share memory of the library's, and the result does not depend on the run.
 */
gemm_status_t gemm_nt_gated(const void *X, int64_t ldx, const void *W13, int64_t ldw, void *H, int64_t ldh,
                            void *GU, int64_t ldgu, gemm_dtype_t type, gemm_act_t act,
                            int64_t tokens, int64_t hidden, int64_t inner, gemm_path_t path,
                            gemm_stream_t stream);

/*
 * The gradient at the two projections of gemm_nt_gated, from dH (tokens x inner) and the
 * GU it kept:
 *   dGU = [dH * u * act'(g),  dH * act(g)]     (tokens x 2*inner)
 * computed in fp32 and rounded once to `type` (dH's, GU's and dGU's).  The gradients of X
 * and W13 are two products of gemm_nt_batched_major with the operands as they lie:
 *   dX   = dGU @ W13    A = dGU K-major, B = W13 MN-major  (tokens, hidden, 2*inner)
 *   dW13 = dGU^T @ X    A = dGU MN-major, B = X MN-major   (2*inner, hidden, tokens)
 * Arguments, empty calls and errors as gemm_nt_gated.
 */
gemm_status_t gemm_nt_gated_grad(const void *dH, int64_t ldd, const void *GU, int64_t ldgu, void *dGU, int64_t ldo,
                                 gemm_dtype_t type, gemm_act_t act, int64_t tokens, int64_t inner,
                                 gemm_stream_t stream);

/*
 * Copies a matrix of `rows` rows of `bytes` bytes, row pitch lds, to dst, whose base and
 * row pitch ldd lie on 16-byte boundaries (pitches in bytes): the layout that the
 * tensor-core kernels read.  Worth its time before gemm_nt_gated, its backward products and
 * gemm_nt_w4 whenever an operand's rows lie off that grid, as those of an odd number of
 * elements do.  Bytes between dst's rows are left alone.  dst off the grid, pitches below
 * `bytes`, null: GEMM_ERR_INVALID_VALUE; dst overlapping src: GEMM_ERR_OVERLAP.
 */
gemm_status_t gemm_nt_copy_rows(const void *src, int64_t lds, void *dst, int64_t ldd, int64_t rows, int64_t bytes,
                                gemm_stream_t stream);

/*
 * 4-bit weights (rows x K): element k of row r stands for
 *   (code - zero) * scale,   code = the low (k even) or high (k odd) half of byte
 *   codes[r*ldc + k/2],      scale = scales[r*lds + k/group],  zero = zeros[r*ldz + k/group]
 * codes 0 to 15, scales in 16 bits (the type of the product's X), zeros 0 to 15 or null: 8.
 * group: 32, 64 or 128; the last group of a row as long as K leaves it.  Pitches in
 * elements of each array.  The high half of an odd row's last byte and bytes between
 * rows are not looked at.
 */
typedef struct gemm_w4 {
    const uint8_t *codes;
    int64_t ldc;
    const void *scales;
    int64_t lds;
    const uint8_t *zeros;
    int64_t ldz;
    int32_t group;
} gemm_w4_t;

/*
 * Quantises W (rows x cols, fp32, fp16 or bf16, row pitch ldw) into Q, whose arrays are
 * written although its pointers are const.  For each group of a row, in fp32 with every
 * step rounded,
 *   Q->zeros null:  a = max |w|, s = a * (1/7) rounded to s_type (fp16 or bf16),
 *                   code = clamp(rint(w * (1/s)), -8, 7) + 8
 *   else            lo = min(w, 0), hi = max(w, 0), s = (hi - lo) * (1/15) rounded to s_type,
 *                   z = clamp(rint(-lo * (1/s)), 0, 15), code = clamp(rint(w * (1/s)) + z, 0, 15)
 * A group whose s is below 2^-126 is zero (s = 0); an infinity or NaN makes its group's
 * scale NaN.  The high half of an odd row's last byte is written as 0, bytes between rows are
 * left alone.  Empty W: GEMM_OK, nothing launched.  W or an output overlapping an output:
 * GEMM_ERR_OVERLAP.
 */
gemm_status_t gemm_nt_w4_quantize(const void *W, gemm_dtype_t w_type, int64_t rows, int64_t cols, int64_t ldw,
                                  const gemm_w4_t *Q, gemm_dtype_t s_type, gemm_stream_t stream);

/*
 * Out = X @ W^T with 4-bit weights: X (M x K) and Out (M x N) both fp16 or both bf16
 * (`type`, also that of W's scales).  Sums in fp32, Out rounded once.
 *
 * path: as gemm_nt_gated, without TC05_PAIR.  SKINNY (up to 16 rows of X, and M * K
 * (rounded up to 256) <= 65536) and MMASYNC multiply whole numbers code - zero, exactly, and scale
 * each group's sum in fp32.  TC05 takes any M; it multiplies (code - zero) * scale rounded
 * to nearest in `type`, so that one sum runs over all groups: each weight is off by at most
 * half a step (bf16 2^-8 of it, fp16 2^-11), and one beyond fp16's largest value is
 * infinite.  AUTO takes SKINNY for few rows and small weights, else TC05, and MMASYNC where
 * alignment leaves nothing else: SKINNY needs the codes on 16-byte boundaries (base and
 * ldc), TC05 X as well.  A group whose scale is infinite or NaN makes its row's sums NaN or
 * infinite, however it is reached.
 * M or N 0: nothing to do; K 0: zeros; K above 2^30: GEMM_ERR_INVALID_VALUE.  The rest as
 * gemm_nt_gated.
 */
gemm_status_t gemm_nt_w4(const void *X, int64_t ldx, const gemm_w4_t *W, void *Out, int64_t ldo, gemm_dtype_t type,
                         int64_t M, int64_t N, int64_t K, gemm_path_t path, gemm_stream_t stream);

/* gemm_nt_gated with 4-bit weights W13 (2*inner rows), its paths those of gemm_nt_w4. */
gemm_status_t gemm_nt_w4_gated(const void *X, int64_t ldx, const gemm_w4_t *W13, void *H, int64_t ldh,
                               gemm_dtype_t type, gemm_act_t act, int64_t tokens, int64_t hidden, int64_t inner,
                               gemm_path_t path, gemm_stream_t stream);

/*
 * Host-side pipeline for callers whose data lives in host memory: copies A and
 * B (packed: lda = ldb = K, strideA = M*K, strideB = N*K) from host to the
 * caller's device buffers dA, dB, runs the batched product into dOut (packed,
 * ldo = N, strideO = M*N) and copies dOut back to host Out.  The work is cut
 * into up to sixteen chunks (row blocks of A and Out when batch == 1, groups of
 * batches otherwise) so that copies in both directions overlap the products:
 * inputs travel on a library-owned copy stream, each chunk's product runs on
 * `stream` once its inputs have arrived, and its Out travels back on a second
 * library-owned stream; `stream` finally waits for the last copy, so
 * synchronising `stream` is enough before reading Out.  For the copies to be
 * asynchronous the host buffers must be pinned.  No device memory is
 * allocated; the two copy streams and ten events are created once per device,
 * on the first call (make that first call outside any stream capture).  Calls
 * on one device are enqueued one at a time (an internal lock).
 */
gemm_status_t gemm_nt_f16_f32_from_host(const void *A_host, const void *B_host, float *Out_host,
                                        void *dA, void *dB, float *dOut,
                                        int64_t M, int64_t N, int64_t K, int64_t batch,
                                        gemm_stream_t stream);

/*
 * Same product as gemm_nt_f16_f32_batched, for callers that must not allocate
 * device memory.  (The source pages have no counterpart to this entry point;
 * it exists for users of this library.)  Code running inside CUDA stream
 * capture may not call cudaMalloc, applications whose device memory is owned by
 * their own pool allocator may forbid any other allocation, and latency-
 * critical code cannot afford an allocation on its first call - yet the
 * automatic path allocates a workspace (about 38 MB per stream, once) when it
 * splits a problem with few output tiles and a long K across the GPU.
 *
 * This entry point always runs the CTA-pair tensor-core kernel (so A and B
 * must meet the tensor-core alignment rule, else GEMM_ERR_NOT_SUPPORTED) and
 * plans the split exactly as the automatic path does, but takes its scratch
 * from one fixed array inside the library: 8 MiB for the partial results of
 * up to 16 CTA pairs plus 4 KiB of counters for up to 64 split tiles.  Every
 * GPU that loads the library holds that array until the process exits.  A call
 * whose split would need more (a problem of 5 to about 37 tiles of 256 x 256
 * with K >= 6144 on a 152-SM GB300) returns GEMM_ERR_SCRATCH_TOO_SMALL and
 * launches nothing; problems that are not split use no scratch at all.
 *
 * It calls no cudaMalloc, cudaFree or other allocating routine.  Argument
 * errors are returned before any CUDA call, as for every entry point.  The
 * first call on a device whose arguments pass the checks (and are not empty)
 * looks up the array's device address (cudaGetSymbolAddress) with that device
 * current; make that first call before any stream capture.  A lookup that
 * failed is tried again on the next call.  The address is kept for the life of
 * the process, so after cudaDeviceReset() on a device make no further call on
 * it.  Before each split launch the counters are cleared on `stream`
 * (cudaMemsetAsync, which allocates nothing).  All calls share the one array:
 * calls that may overlap on the GPU (different streams, or several host threads
 * without ordering) race on it and give wrong results, so order them on one
 * stream.
 */
gemm_status_t gemm_nt_f16_f32_batched_no_alloc(const void *A, const void *B, float *Out,
                                               int64_t M, int64_t N, int64_t K,
                                               int64_t lda, int64_t ldb, int64_t ldo,
                                               int64_t strideA, int64_t strideB, int64_t strideO,
                                               int64_t batch, gemm_stream_t stream);

/*
 * The kernel GEMM_PATH_AUTO would choose for these arguments (host-only: reads
 * no device state and makes no CUDA call).  Pointers are used only for their
 * alignment.
 */
gemm_path_t gemm_nt_select_path(const void *A, const void *B, const float *Out,
                                int64_t M, int64_t N, int64_t K,
                                int64_t lda, int64_t ldb, int64_t ldo,
                                int64_t strideA, int64_t strideB, int64_t strideO,
                                int64_t batch);

/*
 * Synchronises `stream`, then returns and clears the current device's status
 * word: GEMM_ERR_DEVICE_TIMEOUT if any kernel launched since the last check hit
 * its bounded-wait limit, GEMM_ERR_LAUNCH if the synchronisation failed, else GEMM_OK.
 */
gemm_status_t gemm_nt_check(gemm_stream_t stream);

/* Static, human-readable text for a status code ("unknown status" for a value
 * outside gemm_status_t).  Never NULL. */
const char *gemm_nt_error_string(gemm_status_t status);

/*
 * Diagnostic: one warp executes the warp example of "Warp Matrix Instructions"
 * ("From Shared Memory to a Matrix Product") on device inputs A (16x16, row-
 * major fp16) and B (8x16): stage to shared memory, ldmatrix.x4 / .x2, one
 * mma.sync m16n8k16 with C = 0.  It writes the raw per-lane registers to device
 * buffers ar (32x4 uint32), br (32x2 uint32), dr (32x4 float), lane-major, so
 * the fragment maps can be checked.
 */
gemm_status_t gemm_nt_probe_m16n8k16(const void *A, const void *B, uint32_t *ar, uint32_t *br,
                                     float *dr, gemm_stream_t stream);

/*
 * Test hooks for the bounded waits (not for production use).  Sets, for the
 * calling process, the wait limit in SM clock cycles of the tcgen05 kernels
 * (0 restores the default of about two seconds) and a fault to inject into the
 * next launches on CTA 0: 0 none, 1 the producer drops its first stage, 2 the
 * MMA thread skips its first stage release.  With a fault injected the kernel
 * gives up after the limit and gemm_nt_check() returns GEMM_ERR_DEVICE_TIMEOUT.
 */
void gemm_nt_debug_set_wait_limit(uint64_t cycles);
void gemm_nt_debug_set_fault(int fault);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_NT_H */
