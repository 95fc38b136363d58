// block128_api.cu -- C ABI of the products with one fp32 scale per 128 elements
// of K, their quantiser, and the few-token expert layer (include/gemm_nt.h):
// argument checks and kernel selection.
#include <algorithm>

#include "gemm_nt.h"
#include "block128.h"

namespace gnt {

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t kblocks(int64_t K) { return (K + 127) / 128; }

// Bytes [lo, hi) that an array of strided dimensions touches (at least one element each).
struct Span {
    uintptr_t lo, hi;
};
Span span_of(const void* base, int64_t esize, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2 = 1,
             int64_t s2 = 0)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(base);
    return {lo, lo + static_cast<uintptr_t>(((n0 - 1) * s0 + (n1 - 1) * s1 + (n2 - 1) * s2 + 1) * esize)};
}
bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// Whether n0 x n1 x n2 elements with these strides end within 2^62 bytes (sizes are below 2^31).
bool in_range(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2 = 1, int64_t s2 = 0)
{
    const double e = static_cast<double>(n0) * static_cast<double>(s0) + static_cast<double>(n1) * static_cast<double>(s1) +
                     static_cast<double>(n2) * static_cast<double>(s2);
    return e * 4.0 < 4.0e18;
}

bool sizes_ok(std::initializer_list<int64_t> v)
{
    for (int64_t x : v)
        if (x < 0 || x > INT32_MAX)
            return false;
    return true;
}

bool scale_ok(const gemm_scale128_t* s, int64_t rows, int64_t K, int64_t batch)
{
    return s && s->data && aligned(s->data, 4) && (s->rows == 1 || s->rows == 128) && s->row_stride >= 0 &&
           s->kb_stride >= 0 && s->batch_stride >= 0 &&
           in_range(rows, s->row_stride, kblocks(K), s->kb_stride, batch, s->batch_stride);
}

ScaleView view(const gemm_scale128_t& s)
{
    return {s.data, s.rows == 128 ? 7 : 0, s.row_stride, s.kb_stride, s.batch_stride};
}

Span scale_span(const gemm_scale128_t& s, int64_t rows, int64_t K, int64_t batch)
{
    return span_of(s.data, 4, (rows + s.rows - 1) / s.rows, s.row_stride, kblocks(K), s.kb_stride, batch, s.batch_stride);
}

int kernel_out(gemm_dtype_t t) { return t == GEMM_DTYPE_F16 ? kOutF16 : (t == GEMM_DTYPE_BF16 ? kOutBF16 : kOutF32); }

bool f8(gemm_dtype_t t) { return t == GEMM_DTYPE_E4M3 || t == GEMM_DTYPE_E5M2; }

// Whether tensor maps can describe A and B: 16-byte aligned bases, pitches and
// batch strides of whole 16 bytes below 2^40, batches that step over matrices.
bool maps_ok(const BlkParams& p)
{
    const auto ok = [&](const void* base, int64_t rows, int64_t ld, int64_t stride) {
        return aligned(base, 16) && ld % 16 == 0 && ld < (int64_t(1) << 40) &&
               (p.batch == 1 || stride == 0 ||
                (stride % 16 == 0 && stride >= rows * ld && stride < (int64_t(1) << 40)));
    };
    return ok(p.A, p.M, p.lda, p.stride_a) && ok(p.B, p.N, p.ldb, p.stride_b);
}

gemm_path_t select(const BlkParams& p, const DeviceInfo& d, int64_t pair_tiles)
{
    if (p.K == 0 || !maps_ok(p) || 16 * pair_tiles > INT32_MAX)
        return GEMM_PATH_MMASYNC;
    // Pairs once their tiles occupy a third of them, half where B has a scale for
    // every row (the pairs' arithmetic is then twice as long).  Measured, pairs
    // against single CTAs: 512 x 4096 x 4096 (32 tiles) 18.9 and 20.7 us, by row 25.9
    // and 20.3; 1024 x 4096 x 4096 (64 tiles) 20.0 and 37.4, by row 26.7 and 36.6.
    const int part = p.sb.shift ? 3 : 2;
    return p.M > 128 && d.block_pairs > 0 && part * pair_tiles >= d.block_pairs ? GEMM_PATH_TC05_PAIR : GEMM_PATH_SKINNY;
}

gemm_status_t status_of(cudaError_t e) { return e == cudaSuccess ? GEMM_OK : GEMM_ERR_LAUNCH; }

}  // namespace
}  // namespace gnt

using namespace gnt;

extern "C" {

gemm_status_t gemm_nt_block128(const void* A, const gemm_scale128_t* SA, const void* B, const gemm_scale128_t* SB,
                               void* Out, gemm_dtype_t ab_type, gemm_dtype_t out_type, int64_t M, int64_t N, int64_t K,
                               int64_t lda, int64_t ldb, int64_t ldo, int64_t strideA, int64_t strideB, int64_t strideO,
                               int64_t batch, gemm_path_t path, gemm_stream_t stream)
{
    if (!sizes_ok({M, N, K, batch}))
        return GEMM_ERR_INVALID_VALUE;
    if (M == 0 || N == 0 || batch == 0)
        return GEMM_OK;
    if (!f8(ab_type) || (out_type != GEMM_DTYPE_F32 && out_type != GEMM_DTYPE_F16 && out_type != GEMM_DTYPE_BF16))
        return GEMM_ERR_INVALID_VALUE;
    const int64_t osize = out_type == GEMM_DTYPE_F32 ? 4 : 2;
    if (!Out || !aligned(Out, static_cast<uintptr_t>(osize)) || ldo < N || strideO < 0 ||
        !in_range(M, ldo, N, 1, batch, strideO))
        return GEMM_ERR_INVALID_VALUE;
    if (K > 0 && (!A || !B || lda < K || ldb < K || strideA < 0 || strideB < 0 || !in_range(M, lda, K, 1, batch, strideA) ||
                  !in_range(N, ldb, K, 1, batch, strideB) || !scale_ok(SA, M, K, batch) || !scale_ok(SB, N, K, batch)))
        return GEMM_ERR_INVALID_VALUE;
    if (path < GEMM_PATH_AUTO || path > GEMM_PATH_TC05_WS)
        return GEMM_ERR_INVALID_VALUE;
    if (batch > 1 && strideO < (M - 1) * ldo + N)
        return GEMM_ERR_OVERLAP;
    const Span out = span_of(Out, osize, M, ldo, N, 1, batch, strideO);
    if (K > 0 && (overlap(out, span_of(A, 1, M, lda, K, 1, batch, strideA)) ||
                  overlap(out, span_of(B, 1, N, ldb, K, 1, batch, strideB)) ||
                  overlap(out, scale_span(*SA, M, K, batch)) || overlap(out, scale_span(*SB, N, K, batch))))
        return GEMM_ERR_OVERLAP;
    DeviceInfo d;
    gemm_status_t st = static_cast<gemm_status_t>(device_info(&d));
    if (st != GEMM_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    BlkParams p{};
    p.A = A;
    p.B = B;
    p.out = Out;
    p.out_type = kernel_out(out_type);
    p.e5m2 = ab_type == GEMM_DTYPE_E5M2;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.batch = static_cast<int>(batch);
    p.num_kb = static_cast<int>(kblocks(K));
    p.lda = M == 1 ? (K + 15) / 16 * 16 : lda;  // a single row's pitch is never stepped by
    p.ldb = N == 1 ? (K + 15) / 16 * 16 : ldb;
    p.ldo = ldo;
    p.stride_a = strideA;
    p.stride_b = strideB;
    p.stride_o = strideO;
    if (K > 0) {
        p.sa = view(*SA);
        p.sb = view(*SB);
    }
    p.status = d.status;
    p.wait_limit = d.wait_limit;
    p.fault = d.fault;
    const int64_t pair_tiles = ((M + 255) / 256) * ((N + 255) / 256) * batch;
    if (path == GEMM_PATH_AUTO)
        path = select(p, d, pair_tiles);
    if (path == GEMM_PATH_MMASYNC)
        return status_of(block128_any_launch(p, s));
    if ((path != GEMM_PATH_TC05_PAIR && path != GEMM_PATH_SKINNY) || (K > 0 && !maps_ok(p)) ||
        (path == GEMM_PATH_TC05_PAIR && d.block_pairs < 1) || 16 * pair_tiles > INT32_MAX)
        return GEMM_ERR_NOT_SUPPORTED;
    if (K == 0)  // nothing to multiply: zeros, which the warp kernel stores in any layout
        return status_of(block128_any_launch(p, s));
    // what Out's rows allow: stores of 8 or 4 elements, or of single ones
    const auto rows_on = [&](int64_t n) {
        return aligned(Out, static_cast<uintptr_t>(n * osize)) && ldo % n == 0 && (batch == 1 || strideO % n == 0);
    };
    p.vec = rows_on(8) ? 8 : (rows_on(4) ? 4 : 1);
    p.idesc_bits = p.e5m2 ? (1u << 7) | (1u << 10) : 0;
    if (path == GEMM_PATH_TC05_PAIR)
        return status_of(block128_pair_launch(p, d.block_pairs, s));
    return status_of(block128_swap_launch(p, d.num_sms, s));
}

gemm_status_t gemm_nt_block128_quantize(const void* X, gemm_dtype_t x_type, int64_t rows, int64_t cols, int64_t ldx,
                                        void* Q, int64_t ldq, const gemm_scale128_t* SQ, void* QT, int64_t ldqt,
                                        const gemm_scale128_t* ST, gemm_dtype_t q_type, gemm_stream_t stream)
{
    if (!sizes_ok({rows, cols}))
        return GEMM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0)
        return GEMM_OK;
    if (!f8(q_type) || (x_type != GEMM_DTYPE_F32 && x_type != GEMM_DTYPE_F16 && x_type != GEMM_DTYPE_BF16))
        return GEMM_ERR_INVALID_VALUE;
    const int64_t xsize = x_type == GEMM_DTYPE_F32 ? 4 : 2;
    if (!X || !aligned(X, static_cast<uintptr_t>(xsize)) || ldx < cols || !in_range(rows, ldx, cols, 1) || (!Q && !QT))
        return GEMM_ERR_INVALID_VALUE;
    if (Q && (ldq < cols || !in_range(rows, ldq, cols, 1) || !scale_ok(SQ, rows, cols, 1)))
        return GEMM_ERR_INVALID_VALUE;
    if (QT && (ldqt < rows || !in_range(cols, ldqt, rows, 1) || !scale_ok(ST, cols, rows, 1)))
        return GEMM_ERR_INVALID_VALUE;
    if (Q && QT && SQ->rows != ST->rows)
        return GEMM_ERR_INVALID_VALUE;
    // the scales of one matrix must not share elements: one stride steps over
    // the other dimension whole
    const auto separate = [](const gemm_scale128_t& s, int64_t r, int64_t K) {
        const int64_t n = (r + s.rows - 1) / s.rows, c = kblocks(K);
        const bool ok_r = n == 1 || s.row_stride > 0, ok_c = c == 1 || s.kb_stride > 0;
        return ok_r && ok_c && (n == 1 || c == 1 || s.row_stride > (c - 1) * s.kb_stride || s.kb_stride > (n - 1) * s.row_stride);
    };
    if ((Q && !separate(*SQ, rows, cols)) || (QT && !separate(*ST, cols, rows)))
        return GEMM_ERR_OVERLAP;
    Span spans[5] = {span_of(X, xsize, rows, ldx, cols, 1)};
    int n = 1;
    if (Q) {
        spans[n++] = span_of(Q, 1, rows, ldq, cols, 1);
        spans[n++] = scale_span(*SQ, rows, cols, 1);
    }
    if (QT) {
        spans[n++] = span_of(QT, 1, cols, ldqt, rows, 1);
        spans[n++] = scale_span(*ST, cols, rows, 1);
    }
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if (overlap(spans[i], spans[j]))
                return GEMM_ERR_OVERLAP;
    DeviceInfo d;
    gemm_status_t st = static_cast<gemm_status_t>(device_info(&d));
    if (st != GEMM_OK)
        return st;
    QuantParams p{};
    p.x = X;
    p.x_type = x_type;
    p.rows = rows;
    p.cols = cols;
    p.ldx = ldx;
    p.e5m2 = q_type == GEMM_DTYPE_E5M2;
    p.num_sms = d.num_sms;
    p.vec_x = aligned(X, 16) && ldx * xsize % 16 == 0;
    if (Q) {
        p.q = static_cast<uint8_t*>(Q);
        p.ldq = ldq;
        p.sq = const_cast<float*>(SQ->data);
        p.sq_rs = SQ->row_stride;
        p.sq_ks = SQ->kb_stride;
        p.vec_q = aligned(Q, 8) && ldq % 8 == 0;
    }
    if (QT) {
        p.qt = static_cast<uint8_t*>(QT);
        p.ldqt = ldqt;
        p.st = const_cast<float*>(ST->data);
        p.st_rs = ST->row_stride;
        p.st_ks = ST->kb_stride;
        p.vec_qt = aligned(QT, 16) && ldqt % 16 == 0;
    }
    return status_of(block128_quantize_launch(p, (Q ? SQ : ST)->rows == 128, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t gemm_nt_moe_workspace_bytes(int64_t tokens, int64_t topk, int64_t inner)
{
    int64_t bytes;
    if (tokens < 0 || topk < 0 || inner < 0 || inner > INT64_MAX - 15 || __builtin_mul_overflow(tokens, topk, &bytes) ||
        __builtin_mul_overflow(bytes, moe_ldh(inner), &bytes) || __builtin_mul_overflow(bytes, int64_t(4), &bytes))
        return -1;
    return bytes;
}

gemm_status_t gemm_nt_moe(const void* X, int64_t ldx, const float* logits, int64_t ldl, const void* W13, int64_t ldw13,
                          int64_t strideW13, const gemm_scale128_t* S13, const void* W2, int64_t ldw2,
                          int64_t strideW2, const gemm_scale128_t* S2, void* Out, int64_t ldo, gemm_dtype_t x_type,
                          gemm_dtype_t w_type, int64_t tokens, int64_t experts, int64_t topk, int64_t hidden,
                          int64_t inner, int renormalize, void* workspace, int64_t workspace_bytes,
                          gemm_stream_t stream)
{
    if (!sizes_ok({tokens, experts, topk, hidden, inner}))
        return GEMM_ERR_INVALID_VALUE;
    if (tokens == 0 || hidden == 0)
        return GEMM_OK;
    if ((x_type != GEMM_DTYPE_F16 && x_type != GEMM_DTYPE_BF16) || (w_type != x_type && w_type != GEMM_DTYPE_E4M3))
        return GEMM_ERR_INVALID_VALUE;
    const bool w8 = w_type == GEMM_DTYPE_E4M3;
    const int64_t wsize = w8 ? 1 : 2;
    if (topk < 1 || topk > experts)
        return GEMM_ERR_INVALID_VALUE;
    if (!X || !logits || !Out || !aligned(X, 2) || !aligned(Out, 2) || !aligned(logits, 4) || ldx < hidden || ldo < hidden ||
        ldl < experts || !in_range(tokens, std::max({ldx, ldo, ldl}), hidden, 1))
        return GEMM_ERR_INVALID_VALUE;
    const Span out = span_of(Out, 2, tokens, ldo, hidden, 1);
    if (overlap(out, span_of(X, 2, tokens, ldx, hidden, 1)) || overlap(out, span_of(logits, 4, tokens, ldl, experts, 1)))
        return GEMM_ERR_OVERLAP;
    if (inner > 0) {
        if (!W13 || !W2 || !aligned(W13, static_cast<uintptr_t>(wsize)) || !aligned(W2, static_cast<uintptr_t>(wsize)) ||
            ldw13 < hidden || ldw2 < inner || strideW13 < 0 || strideW2 < 0 ||
            !in_range(2 * inner, ldw13, hidden, 1, experts, strideW13) || !in_range(hidden, ldw2, inner, 1, experts, strideW2))
            return GEMM_ERR_INVALID_VALUE;
        if (w8 ? !scale_ok(S13, 2 * inner, hidden, experts) || !scale_ok(S2, hidden, inner, experts) : S13 || S2)
            return GEMM_ERR_INVALID_VALUE;
        const Span w13 = span_of(W13, wsize, 2 * inner, ldw13, hidden, 1, experts, strideW13);
        const Span w2 = span_of(W2, wsize, hidden, ldw2, inner, 1, experts, strideW2);
        if (overlap(out, w13) || overlap(out, w2) ||
            (w8 && (overlap(out, scale_span(*S13, 2 * inner, hidden, experts)) ||
                    overlap(out, scale_span(*S2, hidden, inner, experts)))))
            return GEMM_ERR_OVERLAP;
        if (tokens > kMoeMaxTokens || experts > kMoeMaxExperts || topk > kMoeMaxTopk || hidden > (1 << 20) ||
            inner > (1 << 20))
            return GEMM_ERR_NOT_SUPPORTED;
        if (!workspace || !aligned(workspace, 16))
            return GEMM_ERR_INVALID_VALUE;
        if (workspace_bytes < gemm_nt_moe_workspace_bytes(tokens, topk, inner))
            return GEMM_ERR_SCRATCH_TOO_SMALL;
        const Span ws = span_of(workspace, 1, 1, 0, workspace_bytes, 1);
        if (overlap(ws, out) || overlap(ws, span_of(X, 2, tokens, ldx, hidden, 1)) || overlap(ws, w13) || overlap(ws, w2) ||
            overlap(ws, span_of(logits, 4, tokens, ldl, experts, 1)) ||
            (w8 && (overlap(ws, scale_span(*S13, 2 * inner, hidden, experts)) ||
                    overlap(ws, scale_span(*S2, hidden, inner, experts)))))
            return GEMM_ERR_OVERLAP;
    }
    DeviceInfo d;
    gemm_status_t st = static_cast<gemm_status_t>(device_info(&d));
    if (st != GEMM_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (inner == 0)
        return status_of(cudaMemset2DAsync(Out, ldo * 2, 0, hidden * 2, tokens, s));
    MoeParams p{};
    p.x = X;
    p.ldx = ldx;
    p.logits = logits;
    p.ldl = ldl;
    p.w13 = W13;
    p.ldw13 = ldw13;
    p.stride_w13 = strideW13;
    p.w2 = W2;
    p.ldw2 = ldw2;
    p.stride_w2 = strideW2;
    if (w8) {
        p.s13 = view(*S13);
        p.s2 = view(*S2);
    }
    p.out = Out;
    p.ldo = ldo;
    p.h = static_cast<float*>(workspace);
    p.ldh = moe_ldh(inner);
    p.tokens = static_cast<int>(tokens);
    p.experts = static_cast<int>(experts);
    p.topk = static_cast<int>(topk);
    p.hidden = static_cast<int>(hidden);
    p.inner = static_cast<int>(inner);
    p.renorm = renormalize != 0;
    p.bf16 = x_type == GEMM_DTYPE_BF16;
    p.w8 = w8;
    p.vec_x = aligned(X, 16) && ldx % 8 == 0;
    p.vec_13 = aligned(W13, 16) && ldw13 * wsize % 16 == 0 && strideW13 * wsize % 16 == 0;
    p.vec_2 = aligned(W2, 16) && ldw2 * wsize % 16 == 0 && strideW2 * wsize % 16 == 0;
    p.status = d.status;
    p.wait_limit = d.wait_limit;
    return status_of(moe_launch(p, d.num_sms, s));
}

}  // extern "C"
