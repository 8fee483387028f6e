// Attention of 32 query rows a wave over tiles of keys and values in LDS (gfx950; not part of the ABI).
//
//   S^T[t,q] = K[t,:] . Q[q,:],  P = exp2(c S - m_q),  O^T[:,q] += V^T[:,t] P^T[t,q],  c = scale * log2(e),
// with the running maximum m and sum l of the softmax.  Both products run on 32x32x16 BF16 MFMAs with the query rows as
// columns.  S^T leaves a lane with 16 keys of one query row, the two lanes of a row with all 32; that is P^T as the second
// product's B operand wants it, if V^T's tokens are numbered the same way: P stays in registers, and m, l and the
// rescaling of O^T are a lane's own but for one exchange between the two lanes of a row.
//
// LDS holds rows of K and V as they come, in 16-byte chunks permuted by chunk ^ swizzle(row): its readers of K take one
// chunk of 32 rows, those of V (ds_read_b64_tr_b16, which transposes 4 rows x 16 columns) 64 bytes of each of 8 rows, and
// swizzle(row) = 4 (row % 4) + row / 4 % 4 spreads both over the banks.  So one tile serves as both in a latent cache.
#pragma once

#include "common.hpp"

namespace mx {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) v4s lds_v4s_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8_t;

// Weights of up to 2^kSlack are let stand before O and l are rescaled to a new maximum.
constexpr float kSlack = 8.0f;

// 16 bytes a lane from the buffer to LDS, 1024 bytes in lane order.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t from, uint8_t* to, uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void_t*)to, 16, offset, 0, 0, 0);
}

// The same from an address of each lane.
__device__ __forceinline__ void dma16_at(const uint8_t* from, uint8_t* to) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from, (lds_void_t*)to, 16, 0, 0);
}

__device__ __forceinline__ v2u read_transposed(const uint8_t* at) {
  return __builtin_bit_cast(v2u, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)at));
}

// The place of 16-byte chunk c of a row of D elements in LDS.  Rows of 64 elements are 128 bytes, two of them the 256
// bytes of all banks: they have 8 chunks to spread, by row / 2.
template <int D>
__device__ __forceinline__ uint32_t swizzled(uint32_t c, uint32_t row) {
  if constexpr (D >= 128) return c ^ (((row & 3) << 2) | ((row >> 2) & 3));
  else return c ^ ((((row >> 1) & 1) << 2) | ((row >> 2) & 3));
}

// The value of the other half of the wave beside the lane's own: {lanes 0..31's, lanes 32..63's}, in every lane.
__device__ __forceinline__ float2 halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The schedule of MFMAS matrix instructions with PER LDS reads each: the reads of one come AHEAD instructions before it,
// so that their latency passes under the others.  (Left alone, the compiler puts them right before their use.)
template <int PER, int MFMAS, int AHEAD>
__device__ __forceinline__ void read_ahead() {
  __builtin_amdgcn_sched_group_barrier(0x100, PER * AHEAD, 0);
#pragma unroll
  for (int i = 0; i < MFMAS - AHEAD; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, AHEAD, 0);
}

// HALVES 2: two waves share 32 rows, each with half of D: O's and, in the first product, Q's and K's, whose partial scores
// they exchange (a row of 512 is too much for one wave's registers).
template <int D, int KT, int HALVES>
struct AttnTile {
  static constexpr int SUB = KT / 32;
  static constexpr int DH = D / HALVES;
  static constexpr int KS = DH / 16;
  static constexpr int DT = DH / 32;
  static constexpr int KA = KS < 8 ? KS : 8;            // chunks of K, groups of V within 256 bytes
  static constexpr int VA = DT < 4 ? DT : 4;
  v8bf qf[KS];
  v16f acc[DT];
  float m, l;
  uint32_t kbase, vbase[2];
  int hf;

  __device__ __forceinline__ void begin(int half) {
    const uint32_t lane = threadIdx.x & 63, col = lane & 31;
    hf = lane >> 5;
    // K: row col of 32, chunk 2 j + hf, whose place differs from chunk hf's by the exclusive or of 2 j
    kbase = col * (D * 2) + half * (DH * 2) + (swizzled<D>(hf, col) << 4);
    // V: row 8 n + 4 hf + (lane % 16) / 4, columns 16 ((lane / 16) % 2) + 4 (lane % 4) of 32; n odd and even apart, since
    // the swizzle has row / 4 % 4
    const uint32_t r = hf * 4 + ((lane & 15) >> 2), c = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
#pragma unroll
    for (int n = 0; n < 2; ++n)
      vbase[n] = (n * 8 + r) * (D * 2) + half * (DH * 2) + (swizzled<D>(c, n * 8 + r) << 4) + (lane & 1) * 8;
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
  }

  // The lane's query row, in global memory (its half, if shared).
  __device__ __forceinline__ void load_q(const uint16_t* row) {
#pragma unroll
    for (int j = 0; j < KS; ++j) qf[j] = *reinterpret_cast<const v8bf*>(row + j * 16 + hf * 8);
  }

  // Element i of s[u] is key 32 u + key_of(i) of the tile.
  __device__ __forceinline__ int key_of(int i) const { return (i >> 2) * 8 + hf * 4 + (i & 3); }

  __device__ __forceinline__ void scores(const uint8_t* kt, v16f (&s)[SUB]) const {
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const v8bf kf = *reinterpret_cast<const v8bf*>(kt + (kbase ^ (j % KA << 5)) + u * 32 * D * 2 + (j / KA) * 256);
        s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[j], s[u], 0, 0, 0);
      }
    read_ahead<1, KS * SUB, 4>();
  }

  // Partial scores summed with those of the wave that has the other half of D: `mine` and `other` are places of
  // SUB * 4096 bytes.  All waves of the workgroup come here.
  __device__ __forceinline__ static void exchange(v16f (&s)[SUB], uint8_t* mine, const uint8_t* other, bool active) {
    const uint32_t lane = threadIdx.x & 63;
    if (active) {
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<float4*>(mine + (u * 4 + c) * 1024 + lane * 16) =
              make_float4(s[u][4 * c], s[u][4 * c + 1], s[u][4 * c + 2], s[u][4 * c + 3]);
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (active) {
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float4 x = *reinterpret_cast<const float4*>(other + (u * 4 + c) * 1024 + lane * 16);
          s[u][4 * c] += x.x;
          s[u][4 * c + 1] += x.y;
          s[u][4 * c + 2] += x.z;
          s[u][4 * c + 3] += x.w;
        }
    }
  }

  // The bases as the compiler cannot see through, so that it forms the addresses where they are used and does not hold
  // them all in registers that a wide row needs.
  __device__ __forceinline__ void hide_bases() {
    if constexpr (D >= 256) asm volatile("" : "+v"(kbase), "+v"(vbase[0]), "+v"(vbase[1]));
  }

  // Scores to weights: the new maximum, O and l rescaled if it is much larger, P in BF16.
  __device__ __forceinline__ void weights(const v16f (&s)[SUB], float scale, v8bf (&pf)[SUB][2]) {
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int i = 0; i < 16; i += 2) top = fmaxf(fmaxf(top, s[u][i]), s[u][i + 1]);
    const float2 both = halves(top);
    top = fmaxf(both.x, both.y) * scale;
    if (__any(top > m + kSlack)) {
      const float to = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - (to == -INFINITY ? 0.0f : to));
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] *= f;
      m = to;
    }
    const float base = m == -INFINITY ? 0.0f : m;       // nothing but -inf so far: all weights are 0
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      float w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][i], scale, -base));
#pragma unroll
      for (int i = 0; i < 16; i += 4) l += (w[i] + w[i + 1]) + (w[i + 2] + w[i + 3]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v4u x = {pack_bf16x2(w[8 * h], w[8 * h + 1]), pack_bf16x2(w[8 * h + 2], w[8 * h + 3]),
                       pack_bf16x2(w[8 * h + 4], w[8 * h + 5]), pack_bf16x2(w[8 * h + 6], w[8 * h + 7])};
        pf[u][h] = __builtin_bit_cast(v8bf, x);
      }
    }
  }

  // V^T's operand: tokens 16 n .. + 15 of the tile in the order of P, columns 32 d .. + 31.
  __device__ __forceinline__ v4u v_operand(const uint8_t* vt, int d, int n) const {
    const uint32_t at = n * 16 * D * 2 + (d / VA) * 256;
    const v2u x = read_transposed(vt + (vbase[0] ^ (d % VA << 6)) + at), y = read_transposed(vt + (vbase[1] ^ (d % VA << 6)) + at);
    return v4u{x[0], x[1], y[0], y[1]};
  }

  __device__ __forceinline__ void values(const uint8_t* vt, const v8bf (&pf)[SUB][2]) {
#pragma unroll
    for (int n = 0; n < 2 * SUB; ++n)
#pragma unroll
      for (int d = 0; d < DT; ++d)
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, v_operand(vt, d, n)), pf[n / 2][n % 2],
                                                         acc[d], 0, 0, 0);
    read_ahead<2, 2 * SUB * DT, 3>();
  }

  // As values(), where the lane's row sees only the first `seen` keys of the tile.  A hidden key's weight is 0, but
  // 0 * Inf is not: values that are not finite go into the product as 0, and the rows that see one get it back by a
  // product of its own, of what is seen (0 or 1) with 1 for +Inf, 2^8 for -Inf and 2^16 for NaN, whose sums over at most 64
  // keys tell the three apart.
  __device__ __forceinline__ void values_masked(const uint8_t* vt, const v8bf (&pf)[SUB][2], int seen) {
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      uint32_t odd = 0;
#pragma unroll
      for (int n = 0; n < 2 * SUB; ++n) {
        v4u x = v_operand(vt, d, n);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // all ones in the halves of x that are not finite: adding 2^7 to the exponent field's place carries out of it
          const uint32_t c = ((x[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
          const uint32_t bad = (c >> 15) * 0xFFFFu;
          x[k] &= ~bad;
          odd |= c;
        }
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, x), pf[n / 2][n % 2], acc[d], 0, 0, 0);
      }
      if (__any(odd != 0)) restore(vt, d, seen);
    }
  }

  __device__ __forceinline__ void restore(const uint8_t* vt, int d, int seen) {
    v16f found;
#pragma unroll
    for (int i = 0; i < 16; ++i) found[i] = 0.0f;
#pragma unroll 1
    for (int n = 0; n < 2 * SUB; ++n) {
      const v4u x = v_operand(vt, d, n);
      v4u what, see;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t kind[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t y = (x[k] >> (16 * e)) & 0xFFFFu, g = y & 0x7FFFu;
          kind[e] = g < 0x7F80u ? 0u : g > 0x7F80u ? 0x4780u : y == g ? 0x3F80u : 0x4380u;
        }
        const int t = n * 16 + key_of(2 * k);
        what[k] = kind[0] | (kind[1] << 16);
        see[k] = (t < seen ? 0x3F80u : 0u) | (t + 1 < seen ? 0x3F800000u : 0u);
      }
      found = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, what), __builtin_bit_cast(v8bf, see), found, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t c = static_cast<uint32_t>(found[i]);
      acc[d][i] += (c & 0xFFu) ? INFINITY : 0.0f;
      acc[d][i] -= (c & 0xFF00u) ? INFINITY : 0.0f;
      acc[d][i] = (c >> 16) ? __builtin_nanf("") : acc[d][i];
    }
  }
};

}  // namespace mx
