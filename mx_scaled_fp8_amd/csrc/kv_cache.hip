// Writing the tokens' keys and values into the paged cache, and reading sequences back (gfx950).
//
// Both are one pass over the data and bound by HBM: the write reads 2 and writes 1 + 1/32 bytes an element (2 for a BF16
// cache), the read the other way round.  (8192 tokens of 8 heads of 128, keys and values, to MXFP8: 10.9 us, 4.7 TB/s; 91,807
// cached tokens of them read back as BF16: 119 us for 570 MB, 4.8 TB/s; 64 new tokens 3 us, a launch.  A copy
// reaches 5.1 TB/s.)
#include <algorithm>

#include "kv_cache.hpp"

namespace mx {

namespace {

constexpr int kThreads = 256;

struct WriteArgs {
  const uint16_t* src[2];    // k, v
  int64_t stride[2];         // elements between tokens
  uint8_t* cache[2];
  uint8_t* scale[2];
  const int64_t* slots;
  uint32_t units;            // T * C
  uint32_t C;                // 8-element chunks of a token's row
  uint32_t CD;               // of a head
  DivU32 c_div, cd_div;
  uint32_t Hkv;
  uint32_t page_shift;
  int64_t rows;              // pages * page_size
};

__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0xB1, 0xF, 0xF, false)));
  return max(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x4E, 0xF, 0xF, false)));
}

// A thread takes 8 consecutive elements of one token (one 16-byte load), four threads a block of 32, whose maximum they
// share by DPP.  blockIdx.y: keys, values.
template <bool FP8>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(WriteArgs a) {
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= a.units) return;                       // units is a multiple of 4: a block of 32 is in or out
  const int which = blockIdx.y;
  const uint32_t t = div_u32(u, a.c_div), c = u - t * a.C;
  const uint4 v = *reinterpret_cast<const uint4*>(a.src[which] + static_cast<int64_t>(t) * a.stride[which] + c * 8);
  const int64_t slot = a.slots[t];
  if (slot < 0 || slot >= a.rows) return;         // the same for the four threads of a block
  const uint32_t h = div_u32(c, a.cd_div), cd = c - h * a.CD;
  const int64_t page = slot >> a.page_shift;
  const int64_t row = ((page * a.Hkv + h) << a.page_shift) + (slot - (page << a.page_shift));
  if constexpr (!FP8) {
    *reinterpret_cast<uint4*>(a.cache[which] + (row * a.CD + cd) * 16) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
  m = quad_max(m);
  const bool finite = m < 0x7F80u;
  const int e = e8m0_exponent<8>(finite ? m : 0);
  const float sbits = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  typedef short v2s __attribute__((ext_vector_type(2)));
  v2s lo = {0, 0}, hi = {0, 0};
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(v2bf, w[0]), sbits, false);
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(v2bf, w[1]), sbits, true);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(v2bf, w[2]), sbits, false);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(v2bf, w[3]), sbits, true);
  const uint2 codes = finite ? make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi))
                             : make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  *reinterpret_cast<uint2*>(a.cache[which] + (row * a.CD + cd) * 8) = codes;
  if ((cd & 3) == 0)
    a.scale[which][row * (a.CD >> 2) + (cd >> 2)] = finite ? static_cast<uint8_t>(e + 127) : uint8_t(0xFF);
}

struct ReadArgs {
  KvCache c;
  const int32_t* offsets;
  uint16_t* out[2];
  uint32_t B, rows;
  uint32_t C, CD;            // 8-element chunks of a row, of a head
  DivU32 c_div, cd_div;
};

constexpr uint32_t kReadRows = 16;     // rows of a block

// A block takes kReadRows rows of the output.  Its first threads find each row's place in the cache (the sequence by
// bisection in the offsets, the page from the table); then all threads copy, 8 elements a thread and step, keys and
// values together so that two loads are under way.
template <bool FP8>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(ReadArgs a) {
  __shared__ int64_t place[kReadRows];            // the row of head 0, -1: NaN, -2: left as it is
  const uint32_t r0 = blockIdx.x * kReadRows;
  if (threadIdx.x < kReadRows) {
    const uint32_t r = r0 + threadIdx.x;
    int64_t at = -2;
    if (r < a.rows && static_cast<int64_t>(r) >= a.offsets[0] && static_cast<int64_t>(r) < a.offsets[a.B]) {
      uint32_t lo = 0, hi = a.B;                  // offsets[lo] <= r < offsets[hi]
      while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (a.offsets[mid] <= static_cast<int32_t>(r)) lo = mid; else hi = mid;
      }
      const uint32_t i = r - static_cast<uint32_t>(a.offsets[lo]), p = i >> a.c.page_shift;
      at = -1;
      if (p < a.c.max_pages) {
        const uint32_t page = static_cast<uint32_t>(a.c.table[static_cast<int64_t>(lo) * a.c.max_pages + p]);
        if (page < a.c.pages)
          at = ((static_cast<int64_t>(page) * a.c.Hkv) << a.c.page_shift) + (i & ((1u << a.c.page_shift) - 1));
      }
    }
    place[threadIdx.x] = at;
  }
  __syncthreads();
  const uint32_t units = kReadRows * a.C;
  const bool both = a.out[1] != nullptr;
  for (uint32_t u = threadIdx.x; u < units; u += kThreads) {
    const uint32_t t = div_u32(u, a.c_div), c = u - t * a.C;
    const int64_t at = place[t];
    if (at == -2) continue;
    const uint32_t h = div_u32(c, a.cd_div), cd = c - h * a.CD;
    const int64_t row = at + (static_cast<int64_t>(h) << a.c.page_shift);
    const size_t to = (static_cast<size_t>(r0 + t) * a.C + c) * 8;
    const uint32_t nan = 0x7FC07FC0u;
    uint4 o[2] = {make_uint4(nan, nan, nan, nan), make_uint4(nan, nan, nan, nan)};
    if (at >= 0) {
      if constexpr (FP8) {
        uint2 q[2];
        uint32_t s[2];
        q[0] = *reinterpret_cast<const uint2*>(a.c.k + (row * a.CD + cd) * 8);
        s[0] = a.c.ks[row * (a.CD >> 2) + (cd >> 2)];
        if (both) {
          q[1] = *reinterpret_cast<const uint2*>(a.c.v + (row * a.CD + cd) * 8);
          s[1] = a.c.vs[row * (a.CD >> 2) + (cd >> 2)];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i == 1 && !both) break;
          const float sb = __uint_as_float(s[i] << 23);
          const uint32_t x = q[i].x | nan_codes(s[i]), y = q[i].y | nan_codes(s[i]);
          o[i] = make_uint4(dequant_pair<false>(x, sb), dequant_pair<true>(x, sb), dequant_pair<false>(y, sb),
                            dequant_pair<true>(y, sb));
        }
      } else {
        o[0] = *reinterpret_cast<const uint4*>(a.c.k + (row * a.CD + cd) * 16);
        if (both) o[1] = *reinterpret_cast<const uint4*>(a.c.v + (row * a.CD + cd) * 16);
      }
    }
    *reinterpret_cast<uint4*>(a.out[0] + to) = o[0];
    if (both) *reinterpret_cast<uint4*>(a.out[1] + to) = o[1];
  }
}

}  // namespace

mx_status launch_kv_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t T, int32_t Hkv,
                          int32_t D, const int64_t* slots, bool fp8, void* k_cache, uint8_t* k_scale, void* v_cache,
                          uint8_t* v_scale, int64_t pages, uint32_t page_shift, hipStream_t stream) {
  WriteArgs a;
  a.src[0] = static_cast<const uint16_t*>(k);
  a.src[1] = static_cast<const uint16_t*>(v);
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.cache[0] = static_cast<uint8_t*>(k_cache);
  a.cache[1] = static_cast<uint8_t*>(v_cache);
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.slots = slots;
  a.CD = static_cast<uint32_t>(D) / 8;
  a.C = a.CD * static_cast<uint32_t>(Hkv);
  a.units = static_cast<uint32_t>(T) * a.C;
  a.c_div = make_div(a.C);
  a.cd_div = make_div(a.CD);
  a.Hkv = static_cast<uint32_t>(Hkv);
  a.page_shift = page_shift;
  a.rows = pages << page_shift;
  const dim3 grid((a.units + kThreads - 1) / kThreads, v ? 2 : 1);
  if (fp8) hipLaunchKernelGGL(kv_write_kernel<true>, grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL(kv_write_kernel<false>, grid, dim3(kThreads), 0, stream, a);
  return launch_status("mx_kv_cache_write");
}

mx_status launch_kv_read(const KvCache& c, bool fp8, int32_t D, int64_t B, const int32_t* offsets, int64_t rows,
                         void* k, void* v, hipStream_t stream) {
  ReadArgs a;
  a.c = c;
  a.offsets = offsets;
  a.out[0] = static_cast<uint16_t*>(k);
  a.out[1] = static_cast<uint16_t*>(v);
  a.B = static_cast<uint32_t>(B);
  a.rows = static_cast<uint32_t>(rows);
  a.CD = static_cast<uint32_t>(D) / 8;
  a.C = a.CD * c.Hkv;
  a.c_div = make_div(a.C);
  a.cd_div = make_div(a.CD);
  const dim3 grid(static_cast<uint32_t>((rows + kReadRows - 1) / kReadRows));
  if (fp8) hipLaunchKernelGGL(kv_read_kernel<true>, grid, dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL(kv_read_kernel<false>, grid, dim3(kThreads), 0, stream, a);
  return launch_status("mx_kv_cache_read");
}

}  // namespace mx
