// ffn_swap_f16.cu -- the gated products of ffn_swap.cuh with 4-bit weights for fp16 tokens.
#include "ffn_swap.cuh"

namespace gnt {

cudaError_t ffn_swap_f16(int shift, int nt, const CUtensorMap* maps, const swp::SwapParams& p, const swp::Launch& l)
{
    return swp::by_group<false, true>(shift, nt, maps, p, l);
}

}  // namespace gnt
