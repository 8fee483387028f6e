// The paged key-value cache as the kernels see it (not part of the ABI).
#pragma once

#include "common.hpp"

namespace mx {

struct KvCache {
  const uint8_t* k;          // codes, or BF16
  const uint8_t* v;          // equal to k in a latent cache
  const uint8_t* ks;         // E8M0 bytes (MXFP8 only)
  const uint8_t* vs;
  const int32_t* table;      // [B, max_pages]
  uint32_t max_pages;
  uint32_t pages;
  uint32_t page_shift;
  uint32_t Hkv;
};

// Two e4m3 codes (low or high 16 bits of `codes`) times 2^e as packed BF16; `sbits` holds e + 127 in the FP32 exponent
// field.  Codes of a block whose scale byte is 0xFF have to be NaN already (nan_codes).
template <bool HI_WORD>
__device__ __forceinline__ uint32_t dequant_pair(uint32_t codes, float sbits) {
  typedef __bf16 v2bf_t __attribute__((ext_vector_type(2)));
  const v2bf_t r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(static_cast<int>(codes), sbits, HI_WORD);
  return __builtin_bit_cast(uint32_t, r);
}

// What to OR into four codes under scale byte s: NaN codes for the NaN scale.
__device__ __forceinline__ uint32_t nan_codes(uint32_t s) { return s == 0xFFu ? 0x7F7F7F7Fu : 0u; }

}  // namespace mx
