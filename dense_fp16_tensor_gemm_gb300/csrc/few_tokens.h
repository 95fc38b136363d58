// few_tokens.h -- which tokens the stream of the weights (ffn_few.cu) takes: their number,
// and what of shared memory holds them, rows in whole steps of 128 bytes of the weights.
#pragma once
#include <cstdint>

namespace gnt {

constexpr int kFewTokens = 16;
constexpr int64_t kFewBytes = 128 * 1024;

// Bytes of the tokens in shared memory; codes: 4-bit weights.
inline int64_t few_token_bytes(int64_t tokens, int64_t k, bool codes)
{
    const int64_t step = codes ? 256 : 64;
    return (k + step - 1) / step * step * 2 * tokens;
}
inline bool few_tokens_fit(int64_t tokens, int64_t k, bool codes)
{
    return tokens <= kFewTokens && few_token_bytes(tokens, k, codes) <= kFewBytes;
}

}  // namespace gnt
