// The two kernels of attention of one new token (not part of the ABI).
#pragma once

#include <algorithm>

#include "attn_plan.hpp"

namespace mx {

// Groups of a call with so many tiles at most, `most` of which run at once.
inline uint32_t decode_groups(int64_t tiles, int64_t most) {
  const int64_t n = std::min(std::max<int64_t>(most, 1), tiles);
  return static_cast<uint32_t>(n <= 8 ? n : (n + 7) / 8 * 8);
}

// Whether the query heads of a key head go through the second kernel, as rows of attn_decode_rows.hip.
bool decode_by_rows(int32_t G, int32_t D, bool latent, bool fp8);
// Bytes of its parts (0 if no call of these sizes takes it).
size_t decode_rows_part_bytes(int64_t B, int32_t H, int32_t Hkv, int32_t D, int64_t max_tokens);
void launch_decode_rows(DecodeArgs a, int32_t D, bool fp8, int64_t max_tokens, hipStream_t stream);

}  // namespace mx
