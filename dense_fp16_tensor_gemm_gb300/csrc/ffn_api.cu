// ffn_api.cu -- C ABI of the gated feed-forward product, its gradient and the
// products with 4-bit weights (include/gemm_nt.h): argument checks and kernel
// selection.
#include <algorithm>

#include "gemm_nt.h"
#include "api_checks.h"
#include "block128.h"
#include "ffn.h"

namespace gnt {

namespace {

// The longest sum: the kernels step along K in 32 bits.
constexpr int64_t kMaxK = int64_t(1) << 30;

bool real16(gemm_dtype_t t) { return t == GEMM_DTYPE_F16 || t == GEMM_DTYPE_BF16; }
bool act_ok(gemm_act_t a) { return a == GEMM_ACT_SILU || a == GEMM_ACT_GELU || a == GEMM_ACT_GELU_TANH; }

// A matrix of `esize`-byte elements: rows x cols, row pitch ld.
bool matrix_ok(const void* p, int64_t esize, int64_t rows, int64_t cols, int64_t ld)
{
    return p && aligned(p, static_cast<uintptr_t>(esize)) && ld >= cols && in_range(rows, ld, cols, 1);
}
Span matrix_span(const void* p, int64_t esize, int64_t rows, int64_t cols, int64_t ld)
{
    return span_of(p, esize, rows, ld, cols, 1);
}

int64_t groups(const gemm_w4_t& w, int64_t K) { return (K + w.group - 1) / w.group; }

bool w4_ok(const gemm_w4_t* w, int64_t rows, int64_t K)
{
    return w && (w->group == 32 || w->group == 64 || w->group == 128) &&
           matrix_ok(w->codes, 1, rows, (K + 1) / 2, w->ldc) && matrix_ok(w->scales, 2, rows, groups(*w, K), w->lds) &&
           (!w->zeros || matrix_ok(w->zeros, 1, rows, groups(*w, K), w->ldz));
}

// The spans of the codes, the scales and (if any) the zeros; returns how many.
int w4_spans(const gemm_w4_t& w, int64_t rows, int64_t K, Span* out)
{
    out[0] = matrix_span(w.codes, 1, rows, (K + 1) / 2, w.ldc);
    out[1] = matrix_span(w.scales, 2, rows, groups(w, K), w.lds);
    if (!w.zeros)
        return 2;
    out[2] = matrix_span(w.zeros, 1, rows, groups(w, K), w.ldz);
    return 3;
}

bool overlaps_any(const Span& a, const Span* b, int n)
{
    for (int i = 0; i < n; ++i)
        if (overlap(a, b[i]))
            return true;
    return false;
}

int shift_of(int32_t group) { return group == 32 ? 5 : (group == 64 ? 6 : 7); }

// Whether tensor maps can describe X and the weights (as two matrices where gated, of
// the gate and of the up rows): 16-byte aligned bases, pitches of whole 16 bytes below
// 2^40.
bool maps_ok(const FfnParams& p)
{
    const int64_t lim = int64_t(1) << 39;
    return p.k > 0 && aligned(p.x, 16) && aligned(p.w, 16) && p.ldx % 8 == 0 && p.ldw % (p.scales ? 16 : 8) == 0 &&
           p.ldx < lim && p.ldw < lim / p.n;
}

bool pair_ok(const FfnParams& p)
{
    const int64_t tiles = ((int64_t(p.tokens) + 255) / 256) * ((int64_t(p.n) + 127) / 128);
    return p.gated && !p.scales && maps_ok(p) && tiles <= INT32_MAX / 2;
}

// The warp MMA's kernel, which streams the weights for up to 16 tokens.
bool few_ok(const FfnParams& p)
{
    return p.k > 0 && few_tokens_fit(p.tokens, p.k, p.scales != nullptr) && aligned(p.w, 16) &&
           p.ldw * (p.scales ? 1 : 2) % 16 == 0;
}

// tcgen05 with the weights as rows, on single CTAs.
bool swap_ok(const FfnParams& p)
{
    const int64_t tiles = ((int64_t(p.tokens) + 31) / 32) * ((int64_t(p.n) + 63) / 64);
    return (p.scales || (p.gated && p.tokens <= kSwapTokens)) && maps_ok(p) && tiles <= INT32_MAX / 2;
}

// Whether the stream of the warp MMA is the faster of the two.  It starts sooner, but its time
// grows with the tokens while the tensor cores' does not, so it has one token, and of more the
// smaller weights.  Measured (us, stream and tcgen05), tokens x hidden x inner, gated 16-bit: 1 x
// 4096 x 8192 (134 MB) 23.8 and 24.9, x 32768 (537 MB) 78.9 and 87.3; 2 x 4096 x 4096 (67 MB) 16.1
// and 17.3; 8 x 2048 x 4096 (34 MB) 11.1 and 11.4, x 4096 x 4096 16.9 and 16.7, x 8192 26.5 and
// 24.9; 16 x 1024 x 2048 (8 MB) 5.9 and 7.2, x 2048 x 4096 (34 MB) 12.2 and 11.1.  4-bit, tokens x
// K x N: 1 x 16384 x 8192 (67 MB) 27.2 and 29.8; 2 x 16384 x 4096 (34 MB) 18.9 and 19.1, x 8192
// 30.9 and 29.9; 4 x 8192 x 4096 (17 MB) 12.8 and 13.2, x 16384 x 4096 23.0 and 18.9; 8 x 4096 x
// 4096 (8 MB) 8.8 and 10.2, x 8192 x 4096 16.9 and 13.1; 16 x 2048 x 4096 (4 MB) 8.2 and 8.5, x
// 4096 x 4096 13.7 and 9.9.
bool few_first(const FfnParams& p)
{
    const int64_t rows = p.gated ? 2 * int64_t(p.n) : p.n;
    const int64_t mb = rows * p.k * (p.scales ? 1 : 4) / 2 >> 20;
    if (p.tokens == 1)
        return true;
    if (p.scales)
        return mb < (p.tokens == 2 ? 64 : p.tokens <= 4 ? 32 : p.tokens <= 8 ? 16 : 5);
    return mb < (p.tokens <= 8 ? 80 : 16);
}

// Selects the kernel and launches the product.
gemm_status_t run(FfnParams& p, gemm_path_t path, cudaStream_t stream)
{
    DeviceInfo d;
    gemm_status_t st = static_cast<gemm_status_t>(device_info(&d));
    if (st != GEMM_OK)
        return st;
    p.status = d.status;
    p.wait_limit = d.wait_limit;
    p.fault = d.fault;
    if (p.tokens == 1)
        p.ldx = (int64_t(p.k) + 7) / 8 * 8;  // a single row's pitch is never stepped by
    if (p.n == 1 && !p.gated)
        p.ldw = ((int64_t(p.k) + 1) / 2 + 15) / 16 * 16;  // (plain: codes)
    const bool few = few_ok(p), swap = swap_ok(p), any = path == GEMM_PATH_AUTO;
    if (any && few && (!swap || few_first(p)))
        path = GEMM_PATH_SKINNY;
    else if (any)
        path = swap ? GEMM_PATH_TC05 : GEMM_PATH_TC05_PAIR;
    if (path == GEMM_PATH_SKINNY && few)
        return status_of(ffn_few_launch(p, d.device, d.num_sms, stream));
    if (path == GEMM_PATH_TC05 && swap)
        return status_of(ffn_swap_launch(p, d.device, d.num_sms, stream));
    if (path == GEMM_PATH_TC05_PAIR) {
        int pairs = 0;
        if (pair_ok(p) && gated_pairs(p.act, d.device, &pairs) != cudaSuccess)
            return GEMM_ERR_LAUNCH;
        if (pairs > 0)
            return status_of(gated_pair_launch(p, pairs, stream));
        if (any)
            path = GEMM_PATH_MMASYNC;
    }
    if (path == GEMM_PATH_MMASYNC)
        return status_of(ffn_any_launch(p, d.num_sms, stream));
    return GEMM_ERR_NOT_SUPPORTED;
}

// The plain (inner == n) or gated product with 4-bit weights.
gemm_status_t w4_product(const void* X, int64_t ldx, const gemm_w4_t* W, void* Out, int64_t ldo, gemm_dtype_t type,
                         int gated, int act, int64_t tokens, int64_t n, int64_t K, gemm_path_t path,
                         gemm_stream_t stream)
{
    if (K > kMaxK || path < GEMM_PATH_AUTO || path > GEMM_PATH_TC05_WS)
        return GEMM_ERR_INVALID_VALUE;
    if (tokens == 0 || n == 0)
        return GEMM_OK;
    const int64_t rows = gated ? 2 * n : n;
    if (!real16(type) || !matrix_ok(Out, 2, tokens, n, ldo))
        return GEMM_ERR_INVALID_VALUE;
    if (K > 0 && (!matrix_ok(X, 2, tokens, K, ldx) || !w4_ok(W, rows, K)))
        return GEMM_ERR_INVALID_VALUE;
    FfnParams p{};
    if (K > 0) {
        Span in[4] = {matrix_span(X, 2, tokens, K, ldx)};
        if (overlaps_any(matrix_span(Out, 2, tokens, n, ldo), in, 1 + w4_spans(*W, rows, K, in + 1)))
            return GEMM_ERR_OVERLAP;
        p.x = X;
        p.ldx = ldx;
        p.w = W->codes;
        p.ldw = W->ldc;
        p.scales = W->scales;
        p.lds = W->lds;
        p.zeros = W->zeros;
        p.ldz = W->ldz;
        p.group_shift = shift_of(W->group);
    }
    p.out = Out;
    p.ldo = ldo;
    p.tokens = static_cast<int>(tokens);
    p.n = static_cast<int>(n);
    p.k = static_cast<int>(K);
    p.gated = gated;
    p.act = act;
    p.bf16 = type == GEMM_DTYPE_BF16;
    return run(p, path, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace gnt

using namespace gnt;

extern "C" {

gemm_status_t gemm_nt_gated(const void* X, int64_t ldx, const void* W13, int64_t ldw, void* H, int64_t ldh, void* GU,
                            int64_t ldgu, gemm_dtype_t type, gemm_act_t act, int64_t tokens, int64_t hidden,
                            int64_t inner, gemm_path_t path, gemm_stream_t stream)
{
    if (!sizes_ok({tokens, hidden, inner}) || inner > INT32_MAX / 2 || hidden > kMaxK || path < GEMM_PATH_AUTO ||
        path > GEMM_PATH_TC05_WS)
        return GEMM_ERR_INVALID_VALUE;
    if (tokens == 0 || inner == 0)
        return GEMM_OK;
    if (!real16(type) || !act_ok(act) || !matrix_ok(H, 2, tokens, inner, ldh) ||
        (GU && !matrix_ok(GU, 2, tokens, 2 * inner, ldgu)))
        return GEMM_ERR_INVALID_VALUE;
    if (hidden > 0 && (!matrix_ok(X, 2, tokens, hidden, ldx) || !matrix_ok(W13, 2, 2 * inner, hidden, ldw)))
        return GEMM_ERR_INVALID_VALUE;
    const Span h = matrix_span(H, 2, tokens, inner, ldh);
    const Span gu = GU ? matrix_span(GU, 2, tokens, 2 * inner, ldgu) : Span{0, 0};
    if (GU && overlap(h, gu))
        return GEMM_ERR_OVERLAP;
    if (hidden > 0) {
        const Span in[2] = {matrix_span(X, 2, tokens, hidden, ldx), matrix_span(W13, 2, 2 * inner, hidden, ldw)};
        if (overlaps_any(h, in, 2) || (GU && overlaps_any(gu, in, 2)))
            return GEMM_ERR_OVERLAP;
    }
    FfnParams p{};
    p.x = X;
    p.ldx = ldx;
    p.w = W13;
    p.ldw = ldw;
    p.out = H;
    p.ldo = ldh;
    p.gu = GU;
    p.ldgu = ldgu;
    p.tokens = static_cast<int>(tokens);
    p.n = static_cast<int>(inner);
    p.k = static_cast<int>(hidden);
    p.gated = 1;
    p.act = act;
    p.bf16 = type == GEMM_DTYPE_BF16;
    return run(p, path, reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_nt_gated_grad(const void* dH, int64_t ldd, const void* GU, int64_t ldgu, void* dGU, int64_t ldo,
                                 gemm_dtype_t type, gemm_act_t act, int64_t tokens, int64_t inner,
                                 gemm_stream_t stream)
{
    if (!sizes_ok({tokens, inner}) || inner > INT32_MAX / 2)
        return GEMM_ERR_INVALID_VALUE;
    if (tokens == 0 || inner == 0)
        return GEMM_OK;
    if (!real16(type) || !act_ok(act) || !matrix_ok(dH, 2, tokens, inner, ldd) ||
        !matrix_ok(GU, 2, tokens, 2 * inner, ldgu) || !matrix_ok(dGU, 2, tokens, 2 * inner, ldo))
        return GEMM_ERR_INVALID_VALUE;
    const Span in[2] = {matrix_span(dH, 2, tokens, inner, ldd), matrix_span(GU, 2, tokens, 2 * inner, ldgu)};
    if (overlaps_any(matrix_span(dGU, 2, tokens, 2 * inner, ldo), in, 2))
        return GEMM_ERR_OVERLAP;
    DeviceInfo d;
    gemm_status_t st = static_cast<gemm_status_t>(device_info(&d));
    if (st != GEMM_OK)
        return st;
    GradParams p{};
    p.dh = dH;
    p.ldd = ldd;
    p.gu = GU;
    p.ldgu = ldgu;
    p.out = dGU;
    p.ldo = ldo;
    p.tokens = tokens;
    p.n = inner;
    p.act = act;
    p.bf16 = type == GEMM_DTYPE_BF16;
    return status_of(gated_grad_launch(p, d.num_sms, reinterpret_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_nt_copy_rows(const void* src, int64_t lds, void* dst, int64_t ldd, int64_t rows, int64_t bytes,
                                gemm_stream_t stream)
{
    if (!sizes_ok({rows}) || bytes < 0 || bytes > (int64_t(1) << 40))
        return GEMM_ERR_INVALID_VALUE;
    if (rows == 0 || bytes == 0)
        return GEMM_OK;
    if (!matrix_ok(src, 1, rows, bytes, lds) || !matrix_ok(dst, 1, rows, bytes, ldd) || !aligned(dst, 16) ||
        (rows > 1 && ldd % 16 != 0))
        return GEMM_ERR_INVALID_VALUE;
    if (overlap(matrix_span(dst, 1, rows, bytes, ldd), matrix_span(src, 1, rows, bytes, lds)))
        return GEMM_ERR_OVERLAP;
    DeviceInfo d;
    gemm_status_t st = static_cast<gemm_status_t>(device_info(&d));
    if (st != GEMM_OK)
        return st;
    return status_of(copy_rows_launch(src, lds, dst, ldd, rows, bytes, reinterpret_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_nt_w4_quantize(const void* W, gemm_dtype_t w_type, int64_t rows, int64_t cols, int64_t ldw,
                                  const gemm_w4_t* Q, gemm_dtype_t s_type, gemm_stream_t stream)
{
    if (!sizes_ok({rows, cols}))
        return GEMM_ERR_INVALID_VALUE;
    if (rows == 0 || cols == 0)
        return GEMM_OK;
    if ((w_type != GEMM_DTYPE_F32 && !real16(w_type)) || !real16(s_type) ||
        !matrix_ok(W, w_type == GEMM_DTYPE_F32 ? 4 : 2, rows, cols, ldw) || !w4_ok(Q, rows, cols))
        return GEMM_ERR_INVALID_VALUE;
    Span spans[4] = {matrix_span(W, w_type == GEMM_DTYPE_F32 ? 4 : 2, rows, cols, ldw)};
    const int n = 1 + w4_spans(*Q, rows, cols, spans + 1);
    for (int i = 0; i < n; ++i)
        if (overlaps_any(spans[i], spans + i + 1, n - i - 1))
            return GEMM_ERR_OVERLAP;
    DeviceInfo d;
    gemm_status_t st = static_cast<gemm_status_t>(device_info(&d));
    if (st != GEMM_OK)
        return st;
    Quant4Params p{};
    p.w = W;
    p.w_type = w_type;
    p.rows = rows;
    p.cols = cols;
    p.ldw = ldw;
    p.codes = const_cast<uint8_t*>(static_cast<const uint8_t*>(Q->codes));
    p.ldc = Q->ldc;
    p.scales = const_cast<void*>(Q->scales);
    p.lds = Q->lds;
    p.zeros = const_cast<uint8_t*>(Q->zeros);
    p.ldz = Q->ldz;
    p.group_shift = shift_of(Q->group);
    p.s_bf16 = s_type == GEMM_DTYPE_BF16;
    return status_of(w4_quantize_launch(p, d.num_sms, reinterpret_cast<cudaStream_t>(stream)));
}

gemm_status_t gemm_nt_w4(const void* X, int64_t ldx, const gemm_w4_t* W, void* Out, int64_t ldo, gemm_dtype_t type,
                         int64_t M, int64_t N, int64_t K, gemm_path_t path, gemm_stream_t stream)
{
    if (!sizes_ok({M, N, K}))
        return GEMM_ERR_INVALID_VALUE;
    return w4_product(X, ldx, W, Out, ldo, type, 0, 0, M, N, K, path, stream);
}

gemm_status_t gemm_nt_w4_gated(const void* X, int64_t ldx, const gemm_w4_t* W13, void* H, int64_t ldh,
                               gemm_dtype_t type, gemm_act_t act, int64_t tokens, int64_t hidden, int64_t inner,
                               gemm_path_t path, gemm_stream_t stream)
{
    if (!sizes_ok({tokens, hidden, inner}) || inner > INT32_MAX / 2 || !act_ok(act))
        return GEMM_ERR_INVALID_VALUE;
    return w4_product(X, ldx, W13, H, ldh, type, 1, act, tokens, inner, hidden, path, stream);
}

}  // extern "C"
