// ffn_swap.cu -- the products of ffn_swap.cuh: launch, and the gated forms for bf16
// and for 16-bit weights (the others are compiled apart, beside these).
#include "ffn_swap.cuh"

namespace gnt {

using namespace swp;

cudaError_t ffn_swap_f16(int shift, int nt, const CUtensorMap* maps, const SwapParams& p, const Launch& l);
cudaError_t ffn_swap_plain(int shift, int nt, const CUtensorMap* maps, const SwapParams& p, const Launch& l);
cudaError_t ffn_swap_plain_f16(int shift, int nt, const CUtensorMap* maps, const SwapParams& p, const Launch& l);

namespace {

// shift 0: 16-bit weights (whose types differ in the instruction descriptor alone).
cudaError_t by_kind(bool gated, int shift, bool bf16, int nt, const CUtensorMap* maps, const SwapParams& p, const Launch& l)
{
    if (shift == 0)
        return by_tokens<false, true, true, 0>(nt, maps, p, l);
    if (!gated)
        return bf16 ? ffn_swap_plain(shift, nt, maps, p, l) : ffn_swap_plain_f16(shift, nt, maps, p, l);
    return bf16 ? by_group<true, true>(shift, nt, maps, p, l) : ffn_swap_f16(shift, nt, maps, p, l);
}

}  // namespace

cudaError_t ffn_swap_launch(const FfnParams& f, int device, int num_sms, cudaStream_t stream)
{
    const bool w4 = f.scales != nullptr;
    const int dtype = f.bf16 ? GEMM_DTYPE_BF16 : GEMM_DTYPE_F16;
    const int nt = f.tokens <= 32 ? 32 : (f.tokens <= 64 ? 64 : (f.tokens <= 128 ? 128 : 256));
    SwapParams p{};
    p.f = f;
    p.tiles_w = static_cast<int>((int64_t(f.n) + (f.gated ? 63 : 127)) / (f.gated ? 64 : 128));
    p.tiles_t = static_cast<int>((int64_t(f.tokens) + nt - 1) / nt);
    p.num_tiles = p.tiles_w * p.tiles_t;  // (the caller's bound)
    p.num_kb = static_cast<int>((int64_t(f.k) + BK - 1) / BK);
    p.idesc = idesc_f16_f32(128, nt) | (f.bf16 ? (1u << 7) | (1u << 10) : 0u);
    const auto on = [](const void* q, uintptr_t a, int64_t bytes) { return reinterpret_cast<uintptr_t>(q) % a == 0 && bytes % a == 0; };
    p.vec_s = on(f.scales, 16, 2 * f.lds);
    p.vec_z = on(f.zeros, 8, f.ldz);
    // Few tiles: clusters share out K, down to two stages of codes (512 of K) each.
    p.splits = 1;
    const int groups = (p.num_kb + kRawKb - 1) / kRawKb;
    while (p.splits < 8 && p.num_tiles * p.splits * 2 <= num_sms && groups >= 4 * p.splits)
        p.splits *= 2;
    // the weights (the gate's and the up rows apart), the same in turns of 16 rows, the tokens
    CUtensorMap maps[3];
    const int64_t width = w4 ? (int64_t(f.k) + 1) / 2 : f.k;
    const int wtype = w4 ? GEMM_DTYPE_E4M3 : dtype;  // (codes: bytes)
    if (!call_map(&maps[0], f.w, f.n, width, f.ldw, f.gated ? 2 : 1, int64_t(f.n) * f.ldw, f.gated ? 16 : 128, wtype) ||
        !call_map(&maps[2], f.x, f.tokens, f.k, f.ldx, 1, 0, nt, dtype))
        return cudaErrorInvalidValue;
    maps[1] = maps[0];
    if (f.gated && f.n >= 64) {
        if (!interleaved_map(&maps[1], f.w, f.n, width, f.ldw, wtype))
            return cudaErrorInvalidValue;
        p.whole = f.n % 16 == 0 ? (f.n + 63) / 64 * 64 : f.n;
    }
    const int grid = p.splits > 1 ? p.num_tiles * p.splits : std::min(p.num_tiles, num_sms);
    return by_kind(f.gated, f.group_shift, f.bf16, nt, maps, p, Launch{device, grid, stream});
}

}  // namespace gnt
