// Attention of a wave's query rows over tiles of keys and values in LDS (gfx950; not part of the ABI).
//
//   S^T[t,q] = K[t,:] . Q[q,:],  P = exp2(c S - m_q),  O^T[:,q] += V^T[:,t] P^T[t,q],  c = scale * log2(e),
// with the running maximum m and sum l of the softmax.  Both products run on BF16 MFMAs with the query rows as columns.
// S^T leaves a lane with several keys of one query row; that is P^T as the second product's B operand wants it, if V^T's
// tokens are numbered the same way: P stays in registers, and m, l and the rescaling of O^T are a lane's own but for an
// exchange between the lanes of a row.
//
// Two shapes: 32 rows a wave on 32x32x16 MFMAs (AttnTile), which take half the LDS reads for the same work, and, for
// rows of 512, whose O and Q would not fit a wave's registers, 16 rows on 16x16x32 (AttnTile16).
//
// LDS holds rows of K and V as they come, in 16-byte chunks permuted by chunk ^ swizzle(row): the readers of K take one
// chunk of many rows, those of V (ds_read_b64_tr_b16, which transposes 4 rows x 16 columns) a few chunks of several rows,
// and the swizzle spreads both over the banks.  So one tile serves as both in a latent cache.
#pragma once

#include "common.hpp"

namespace mx {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
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

// The place of 16-byte chunk c of a row of D elements in LDS.  A row is a multiple of the 256 bytes of all banks; of
// 64 elements, two rows are, and they have 8 chunks to spread, by row / 2.
template <int D>
__device__ __forceinline__ uint32_t swizzled(uint32_t c, uint32_t row) {
  // V: 2 chunks of 8 rows at a time.  K: a chunk of 16 rows, but the banks serve rows 0..3, 12..15 of one chunk together
  // with rows 4..11 of the next, so that row / 4 % 2, not row / 8, tells rows 8 apart.
  if constexpr (D >= 512) return c ^ (((row & 7) << 1) | ((row >> 2) & 1));
  else if constexpr (D >= 128) return c ^ (((row & 3) << 2) | ((row >> 2) & 3));   // 4 chunks of 4 rows
  else return c ^ ((((row >> 1) & 1) << 2) | ((row >> 2) & 3));
}

// The value of the other half of the wave beside the lane's own: {lanes 0..31's, lanes 32..63's}, in every lane.
__device__ __forceinline__ float2 halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// f over the four lanes whose numbers are the same modulo 16, in all of them.
template <class F>
__device__ __forceinline__ float quarters(F f, float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  const float2 both = halves(f(__uint_as_float(r[0]), __uint_as_float(r[1])));
  return f(both.x, both.y);
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

// In the halves of x that are not finite BF16: all ones.  (Adding 2^7 to the exponent field carries out of it there.)
__device__ __forceinline__ uint32_t not_finite(uint32_t x) {
  return ((((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u) >> 15) * 0xFFFFu;
}

// 1 for +Inf, 2^8 for -Inf, 2^16 for NaN and 0 for the rest, of each half, in BF16.
__device__ __forceinline__ uint32_t kind_of(uint32_t x) {
  uint32_t kind[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint32_t y = (x >> (16 * e)) & 0xFFFFu, g = y & 0x7FFFu;
    kind[e] = g < 0x7F80u ? 0u : g > 0x7F80u ? 0x4780u : y == g ? 0x3F80u : 0x4380u;
  }
  return kind[0] | (kind[1] << 16);
}

// O's element after `found`, the sum of kinds over the at most 64 keys of a tile that its row sees.
__device__ __forceinline__ float restored(float o, float found) {
  const uint32_t c = static_cast<uint32_t>(found);
  o += (c & 0xFFu) ? INFINITY : 0.0f;
  o -= (c & 0xFF00u) ? INFINITY : 0.0f;
  return (c >> 16) ? __builtin_nanf("") : o;
}

// Both shapes have:
//   ROWS                    query rows of a wave; the lane's is row()
//   load_q(row)             the lane's row from global memory
//   scores(kt, s)           of the tile at kt
//   mask(s, seen)           keys from `seen` on hidden from the lane's row
//   weights(s, scale, p)    the new maximum, O and l rescaled if it is much larger, P in BF16
//   values(vt, p)           O += P V
//   values_masked(vt, p, seen)   the same, where a row does not see all of the tile.  A hidden key's weight is 0, but 0 * Inf
//                           is not: values that are not finite go into the product as 0, and the rows that see one get it
//                           back by a product of its own, of what is seen (0 or 1) with kind_of().
//   sum()                   the row's l
//   QUADS, quad(i, d)       O in fours: elements d .. d + 3 of the lane's row

template <int D, int KT>
struct AttnTile {
  static constexpr int ROWS = 32, SUB = KT / 32, KS = D / 16, DT = D / 32;
  static constexpr int KA = KS < 8 ? KS : 8;            // chunks of K, groups of V within 256 bytes
  static constexpr int VA = DT < 4 ? DT : 4;
  static constexpr int QUADS = DT * 4;
  struct Scores { v16f s[SUB]; };
  struct Weights { v8bf p[2 * SUB]; };
  v8bf qf[KS];
  v16f acc[DT];
  float m, l;
  uint32_t kbase, vbase[2];
  int hf;

  __device__ __forceinline__ static int row() { return threadIdx.x & 31; }
  __device__ __forceinline__ static bool first_lane() { return (threadIdx.x & 32) == 0; }   // of the row's

  __device__ __forceinline__ void begin() {
    const uint32_t lane = threadIdx.x & 63, col = lane & 31;
    hf = lane >> 5;
    // K: row col of 32, chunk 2 j + hf, whose place differs from chunk hf's by the exclusive or of 2 j
    kbase = col * (D * 2) + (swizzled<D>(hf, col) << 4);
    // V: row 8 n + 4 hf + (lane % 16) / 4, columns 16 ((lane / 16) % 2) + 4 (lane % 4) of 32; n odd and even apart, since
    // the swizzle has row / 4 % 4
    const uint32_t r = hf * 4 + ((lane & 15) >> 2), c = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
#pragma unroll
    for (int n = 0; n < 2; ++n) vbase[n] = (n * 8 + r) * (D * 2) + (swizzled<D>(c, n * 8 + r) << 4) + (lane & 1) * 8;
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
  }

  __device__ __forceinline__ void load_q(const uint16_t* row) {
#pragma unroll
    for (int j = 0; j < KS; ++j) qf[j] = *reinterpret_cast<const v8bf*>(row + j * 16 + hf * 8);
  }

  // The bases as the compiler cannot see through, so that it forms the addresses where they are used and does not hold
  // them all in registers that a wide row needs.
  __device__ __forceinline__ void hide_bases() {
    if constexpr (D >= 256) asm volatile("" : "+v"(kbase), "+v"(vbase[0]), "+v"(vbase[1]));
  }

  // Element i of s[u] is key 32 u + key_of(i) of the tile.
  __device__ __forceinline__ int key_of(int i) const { return (i >> 2) * 8 + hf * 4 + (i & 3); }

  __device__ __forceinline__ void scores(const uint8_t* kt, Scores& x) {
    hide_bases();
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) x.s[u][i] = 0.0f;
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const v8bf kf = *reinterpret_cast<const v8bf*>(kt + (kbase ^ (j % KA << 5)) + u * 32 * D * 2 + (j / KA) * 256);
        x.s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[j], x.s[u], 0, 0, 0);
      }
    read_ahead<1, KS * SUB, 4>();
  }

  __device__ __forceinline__ void mask(Scores& x, int seen) const {
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) x.s[u][i] = u * 32 + key_of(i) < seen ? x.s[u][i] : -INFINITY;
  }

  __device__ __forceinline__ void weights(const Scores& x, float scale, Weights& y) {
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int i = 0; i < 16; i += 2) top = fmaxf(fmaxf(top, x.s[u][i]), x.s[u][i + 1]);
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
      for (int i = 0; i < 16; ++i) w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x.s[u][i], scale, -base));
#pragma unroll
      for (int i = 0; i < 16; i += 4) l += (w[i] + w[i + 1]) + (w[i + 2] + w[i + 3]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        y.p[2 * u + h] = __builtin_bit_cast(v8bf, (v4u{pack_bf16x2(w[8 * h], w[8 * h + 1]), pack_bf16x2(w[8 * h + 2], w[8 * h + 3]),
                                                        pack_bf16x2(w[8 * h + 4], w[8 * h + 5]), pack_bf16x2(w[8 * h + 6], w[8 * h + 7])}));
    }
  }

  // V^T's operand: tokens 16 n .. + 15 of the tile in the order of P, columns 32 d .. + 31.
  __device__ __forceinline__ v4u v_operand(const uint8_t* vt, int d, int n) const {
    const uint32_t at = n * 16 * D * 2 + (d / VA) * 256;
    const v2u x = read_transposed(vt + (vbase[0] ^ (d % VA << 6)) + at), y = read_transposed(vt + (vbase[1] ^ (d % VA << 6)) + at);
    return v4u{x[0], x[1], y[0], y[1]};
  }

  __device__ __forceinline__ void values(const uint8_t* vt, const Weights& y) {
#pragma unroll
    for (int n = 0; n < 2 * SUB; ++n)
#pragma unroll
      for (int d = 0; d < DT; ++d)
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, v_operand(vt, d, n)), y.p[n], acc[d], 0, 0, 0);
    read_ahead<2, 2 * SUB * DT, 3>();
  }

  __device__ __forceinline__ void values_masked(const uint8_t* vt, const Weights& y, int seen) {
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      uint32_t odd = 0;
#pragma unroll
      for (int n = 0; n < 2 * SUB; ++n) {
        v4u x = v_operand(vt, d, n);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t bad = not_finite(x[k]);
          x[k] &= ~bad;
          odd |= bad;
        }
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, x), y.p[n], acc[d], 0, 0, 0);
      }
      if (!__any(odd != 0)) continue;
      v16f found;
#pragma unroll
      for (int i = 0; i < 16; ++i) found[i] = 0.0f;
#pragma unroll 1
      for (int n = 0; n < 2 * SUB; ++n) {
        const v4u x = v_operand(vt, d, n);
        v4u what, see;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = n * 16 + key_of(2 * k);
          what[k] = kind_of(x[k]);
          see[k] = (t < seen ? 0x3F80u : 0u) | (t + 1 < seen ? 0x3F800000u : 0u);
        }
        found = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, what), __builtin_bit_cast(v8bf, see), found, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[d][i] = restored(acc[d][i], found[i]);
    }
  }

  __device__ __forceinline__ float sum() const {
    const float2 both = halves(l);
    return both.x + both.y;
  }

  __device__ __forceinline__ float4 quad(int i, int& d) const {
    d = (i >> 2) * 32 + (i & 3) * 8 + hf * 4;
    const v16f& a = acc[i >> 2];
    const int r = (i & 3) * 4;
    return make_float4(a[r], a[r + 1], a[r + 2], a[r + 3]);
  }
};

// AHEAD: see read_ahead(); what a kernel has registers for.
template <int D, int KT, int AHEAD>
struct AttnTile16 {
  static_assert(D % 256 == 0 && KT == 32, "rows of whole 256 bytes, one operand of weights");
  static constexpr int ROWS = 16, KS = D / 32, DT = D / 16, QUADS = DT;
  struct Scores { v4f s[2]; };
  struct Weights { v8bf p; };
  v8bf qf[KS];
  v4f acc[DT];
  float m, l;
  uint32_t kbase, vbase;
  int g;

  __device__ __forceinline__ static int row() { return threadIdx.x & 15; }
  __device__ __forceinline__ static bool first_lane() { return (threadIdx.x & 48) == 0; }

  __device__ __forceinline__ void begin(uint32_t lane = threadIdx.x & 63) {
    const uint32_t col = lane & 15;
    g = lane >> 4;
    // K: row col of 16, chunk 4 j + g.  V: row 4 g + (lane % 16) / 4 of 16, columns 4 (lane % 4) of 16.
    kbase = col * (D * 2) + (swizzled<D>(g, col) << 4);
    const uint32_t r = g * 4 + (col >> 2);
    vbase = r * (D * 2) + (swizzled<D>((lane & 3) >> 1, r) << 4) + (lane & 1) * 8;
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d) acc[d] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  }

  __device__ __forceinline__ void load_q(const uint16_t* row) {
#pragma unroll
    for (int j = 0; j < KS; ++j) qf[j] = *reinterpret_cast<const v8bf*>(row + j * 32 + g * 8);
  }

  // Element i of s[u] is key 16 u + 4 g + i of the tile.
  __device__ __forceinline__ void scores(const uint8_t* kt, Scores& x) {
    asm volatile("" : "+v"(kbase), "+v"(vbase));        // addresses are formed where they are used
    x.s[0] = x.s[1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const v8bf kf = *reinterpret_cast<const v8bf*>(kt + (kbase ^ (j % 4 << 6)) + u * 16 * D * 2 + (j / 4) * 256);
        x.s[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[j], x.s[u], 0, 0, 0);
      }
    read_ahead<1, KS * 2, AHEAD>();
  }

  __device__ __forceinline__ void mask(Scores& x, int seen) const {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) x.s[u][i] = u * 16 + g * 4 + i < seen ? x.s[u][i] : -INFINITY;
  }

  __device__ __forceinline__ void weights(const Scores& x, float scale, Weights& y) {
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < 2; ++u) top = fmaxf(fmaxf(fmaxf(top, x.s[u][0]), x.s[u][1]), fmaxf(x.s[u][2], x.s[u][3]));
    top = quarters([](float a, float b) { return fmaxf(a, b); }, top) * scale;
    if (__any(top > m + kSlack)) {
      const float to = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - (to == -INFINITY ? 0.0f : to));
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d) acc[d] *= f;
      m = to;
    }
    const float base = m == -INFINITY ? 0.0f : m;       // nothing but -inf so far: all weights are 0
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x.s[i >> 2][i & 3], scale, -base));
    l += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
    y.p = __builtin_bit_cast(v8bf, (v4u{pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]), pack_bf16x2(w[4], w[5]),
                                        pack_bf16x2(w[6], w[7])}));
  }

  // V^T's operand: the 32 tokens in the order of P, columns 16 d .. + 15.
  __device__ __forceinline__ v4u v_operand(const uint8_t* vt, int d) const {
    const uint8_t* at = vt + (vbase ^ (d % 8 << 5)) + (d / 8) * 256;
    const v2u x = read_transposed(at), y = read_transposed(at + 16 * D * 2);
    return v4u{x[0], x[1], y[0], y[1]};
  }

  __device__ __forceinline__ void values(const uint8_t* vt, const Weights& y) {
#pragma unroll
    for (int d = 0; d < DT; ++d)
      acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, v_operand(vt, d)), y.p, acc[d], 0, 0, 0);
    read_ahead<2, DT, AHEAD>();
  }

  __device__ __forceinline__ void values_masked(const uint8_t* vt, const Weights& y, int seen) {
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const v4u raw = v_operand(vt, d);
      v4u x = raw;
      uint32_t odd = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t bad = not_finite(x[k]);
        x[k] &= ~bad;
        odd |= bad;
      }
      acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x), y.p, acc[d], 0, 0, 0);
      if (!__any(odd != 0)) continue;
      v4u what, see;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = (k >> 1) * 16 + g * 4 + (k & 1) * 2;
        what[k] = kind_of(raw[k]);
        see[k] = (t < seen ? 0x3F80u : 0u) | (t + 1 < seen ? 0x3F800000u : 0u);
      }
      const v4f found = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, what), __builtin_bit_cast(v8bf, see),
                                                               (v4f{0.0f, 0.0f, 0.0f, 0.0f}), 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[d][i] = restored(acc[d][i], found[i]);
    }
  }

  __device__ __forceinline__ float sum() const {
    return quarters([](float a, float b) { return a + b; }, l);
  }

  __device__ __forceinline__ float4 quad(int i, int& d) const {
    d = i * 16 + g * 4;
    return make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  }
};

// The tile of rows of D, and its keys.
template <int D, int AHEAD = 6>
struct TileOf { using type = AttnTile<D, D <= 128 ? 64 : 32>; };
template <int AHEAD>
struct TileOf<512, AHEAD> { using type = AttnTile16<512, 32, AHEAD>; };
template <int D>
constexpr int key_tile() { return D <= 128 ? 64 : 32; }

}  // namespace mx
