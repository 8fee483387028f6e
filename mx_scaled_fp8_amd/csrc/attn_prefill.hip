// Causal attention over packed prompts (gfx950).
//
// A workgroup takes 128 query rows of one prompt and head, 32 for each of its four waves, and runs over the keys in
// tiles of KT with the running maximum m and sum l of the softmax:
//   S^T[t,q] = K[t,:] . Q[q,:],  P = exp2(c S - m_q),  O^T[:,q] += V^T[:,t] P^T[t,q],  c = scale * log2(e).
// Both products run on 32x32x16 BF16 MFMAs with the query rows as columns.  S^T leaves a lane with 16 keys of one query row,
// the two lanes of a row with all 32; that is P^T as the second product's B operand wants it, if V^T's tokens are numbered
// the same way, so P stays in registers and m, l and the rescaling of O^T are a lane's own, but for one exchange between
// the two lanes of a row.
// K and V tiles go from global memory to LDS by buffer-load DMA (two buffers: the next tile is under way while this one
// is used; rows past the end are zeros by the buffer's bound), rows in 16-byte chunks that are permuted on the way in:
// chunk ^ row % 16 for K (its readers take one chunk of 32 rows), 64-byte groups ^ row % 4 for V (its readers are
// ds_read_b64_tr_b16, which take 4 rows x 16 columns and transpose them).
#include <algorithm>

#include "common.hpp"

namespace mx {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) v4s lds_v4s_t;
typedef __attribute__((address_space(3))) uint8_t lds_u8_t;

constexpr int kThreads = 256;
constexpr int kRows = 128;             // query rows of a workgroup

struct PrefillArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* q_offsets;
  const int32_t* k_offsets;
  uint16_t* out;
  float scale;               // times log2(e)
  uint32_t B, Tq, Tk, H, Hkv, G;
  uint32_t tiles;            // bound on the row tiles of all prompts
};

// 16 bytes a lane from the buffer to LDS, 1024 bytes in lane order.
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t from, uint8_t* to, uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (lds_void_t*)to, 16, offset, 0, 0, 0);
}

// Offset b cut to [0, T].
__device__ __forceinline__ uint32_t cut(const int32_t* offsets, uint32_t b, uint32_t T) {
  return min(static_cast<uint32_t>(max(offsets[b], 0)), T);
}

template <int D>
__global__ __launch_bounds__(kThreads, D >= 256 ? 1 : 2) void attn_prefill_kernel(PrefillArgs a) {
  constexpr int KT = D <= 128 ? 64 : 32;                // keys of a tile
  constexpr int CH = D / 8;                             // 16-byte chunks of a row
  constexpr int TB = KT * D * 2;                        // bytes of a tile
  constexpr int ND = TB / 1024 / 4;                     // a wave's DMA instructions for one tile
  constexpr int SUB = KT / 32;
  constexpr int KS = D / 16;
  constexpr int DT = D / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[4 * TB];   // K, V, K, V
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 31, hf = lane >> 5;

  // (row tile, head): heads of one key head side by side, key heads fastest, so that with workgroups dealt to the XCDs in
  // turn an XCD's L2 serves few key heads; last row tiles first, which have the most keys.
  uint32_t id = blockIdx.x;
  const uint32_t kvh = id % a.Hkv;
  id /= a.Hkv;
  const uint32_t head = kvh * a.G + id % a.G;
  const uint32_t rt = a.tiles - 1 - id / a.G;
  // prompt b's row tiles are numbered from offsets[b] / kRows + b, which leaves room for every ragged end
  uint32_t lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (cut(a.q_offsets, mid, a.Tq) / kRows + mid <= rt) lo = mid; else hi = mid;
  }
  const uint32_t q0 = cut(a.q_offsets, lo, a.Tq), q1 = cut(a.q_offsets, lo + 1, a.Tq);
  const uint32_t k0 = cut(a.k_offsets, lo, a.Tk), k1 = cut(a.k_offsets, lo + 1, a.Tk);
  const uint32_t first = (rt - (q0 / kRows + lo)) * kRows;         // of the prompt's rows
  if (q1 <= q0 || first >= q1 - q0) return;
  const int32_t Lq = static_cast<int32_t>(q1 - q0), Lk = k1 > k0 ? static_cast<int32_t>(k1 - k0) : 0;
  const int32_t i0 = static_cast<int32_t>(first) + wave * 32;      // the wave's first row
  const int32_t i = i0 + col;                                      // the lane's row
  const int32_t seen = Lk - Lq + i;                                // its last key, below 0 if none
  // keys that the workgroup's, the wave's rows see
  const int32_t wg_keys = min(Lk, Lk - Lq + min(static_cast<int32_t>(first) + kRows, Lq));
  const int32_t w_keys = i0 < Lq ? min(Lk, Lk - Lq + min(i0 + 32, Lq)) : 0;
  const int32_t full = Lk - Lq + i0 + 1;                           // keys that each of the wave's rows sees
  const int32_t n_tiles = wg_keys > 0 ? (wg_keys + KT - 1) / KT : 0;

  v8bf qf[KS];
  {
    const uint16_t* row = a.q + static_cast<int64_t>(q0 + min(i, Lq - 1)) * a.q_stride + head * D + hf * 8;
#pragma unroll
    for (int j = 0; j < KS; ++j) qf[j] = *reinterpret_cast<const v8bf*>(row + j * 16);
  }

  // DMA: an instruction fills 1024 bytes of LDS in lane order; instruction x of a tile holds rows from x * 1024 / (2 D)
  const uint16_t* kbase = a.k + static_cast<int64_t>(k0) * a.k_stride + kvh * D;
  const uint16_t* vbase = a.v + static_cast<int64_t>(k0) * a.v_stride + kvh * D;
  uint32_t koff[ND], voff[ND];
#pragma unroll
  for (int x = 0; x < ND; ++x) {
    const uint32_t at = (wave * ND + x) * 64 + lane, r = at / CH, c = at % CH;
    uint32_t ck, cv;
    if constexpr (D >= 128) {
      ck = c ^ (r & 15);
      cv = c ^ ((r & 3) << 2);
    } else {                                            // two rows in the 256 bytes of all banks
      ck = c ^ ((r >> 1) & 7);
      cv = c ^ (((r >> 1) & 1) << 2);
    }
    koff[x] = r * static_cast<uint32_t>(a.k_stride) * 2 + ck * 16;
    voff[x] = r * static_cast<uint32_t>(a.v_stride) * 2 + cv * 16;
  }
  auto dma = [&](int32_t tile, int buf) {
    const int32_t r0 = tile * KT, rows = min(KT, Lk - r0);
    const __amdgpu_buffer_rsrc_t kr = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(kbase + r0 * a.k_stride), 0,
        (rows - 1) * static_cast<int>(a.k_stride) * 2 + D * 2, kBufferFlags);
    const __amdgpu_buffer_rsrc_t vr = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(vbase + r0 * a.v_stride), 0,
        (rows - 1) * static_cast<int>(a.v_stride) * 2 + D * 2, kBufferFlags);
    uint8_t* to = lds + buf * 2 * TB;
#pragma unroll
    for (int x = 0; x < ND; ++x) dma16(kr, to + (wave * ND + x) * 1024, koff[x]);
#pragma unroll
    for (int x = 0; x < ND; ++x) dma16(vr, to + TB + (wave * ND + x) * 1024, voff[x]);
  };

  // where a lane reads: K row col of a group of 32, chunk 2 kk + hf; V rows 4 hf + (lane % 16) / 4 of a group of 8,
  // columns 16 ((lane / 16) % 2) + 4 (lane % 4) of 32
  const uint32_t kswz = D >= 128 ? col & 15 : (col >> 1) & 7;
  const uint32_t krow = col * (D * 2);
  const uint32_t vr4 = (lane & 15) >> 2, vswz = D >= 128 ? vr4 : vr4 >> 1;
  const uint32_t vrow = (hf * 4 + vr4) * (D * 2) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;

  float m = -INFINITY, l = 0.0f;
  v16f acc[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[d][r] = 0.0f;

  if (n_tiles > 0) dma(0, 0);
  for (int32_t tile = 0; tile < n_tiles; ++tile) {
    // this wave's part of the tile is in LDS, and after the barrier everyone's; everyone has read the other buffer
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (tile + 1 < n_tiles) dma(tile + 1, (tile + 1) & 1);
    const int32_t t0 = tile * KT;
    if (t0 >= w_keys) continue;
    const uint8_t* kt = lds + (tile & 1) * 2 * TB;
    const uint8_t* vt = kt + TB;
    v16f s[SUB];
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[u][r] = 0.0f;
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const v8bf kf = *reinterpret_cast<const v8bf*>(kt + u * 32 * D * 2 + krow + (((2 * j + hf) ^ kswz) << 4));
        s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[j], s[u], 0, 0, 0);
      }
    const bool masked = t0 + KT > full;                 // some row of the wave does not see all of the tile
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if (masked && t0 + u * 32 + (r >> 2) * 8 + hf * 4 + (r & 3) > seen) s[u][r] = -INFINITY;
        top = fmaxf(top, s[u][r]);
      }
    top = fmaxf(top, __shfl_xor(top, 32)) * a.scale;
    top = fmaxf(m, top);
    const float base = top == -INFINITY ? 0.0f : top;   // nothing but -inf so far: all weights are 0
    if (__any(top > m)) {
      const float f = __builtin_amdgcn_exp2f(m - base);
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[d][r] *= f;
      m = top;
    }
    v8bf pf[SUB][2];
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      float w[16];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        w[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][r], a.scale, -base));
        l += w[r];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v4u x = {pack_bf16x2(w[8 * h], w[8 * h + 1]), pack_bf16x2(w[8 * h + 2], w[8 * h + 3]),
                       pack_bf16x2(w[8 * h + 4], w[8 * h + 5]), pack_bf16x2(w[8 * h + 6], w[8 * h + 7])};
        pf[u][h] = __builtin_bit_cast(v8bf, x);
      }
    }
    auto v_frag = [&](int d, int u, int h) {            // tokens 16 (2 u + h) + .. of the tile, columns 32 d + ..
      const uint8_t* at = vt + (u * 32 + h * 16) * D * 2 + vrow + ((d ^ vswz) << 6);
      const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)at);
      const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s_t*)(at + 8 * D * 2));
      const v2u xu = __builtin_bit_cast(v2u, x), yu = __builtin_bit_cast(v2u, y);
      return v4u{xu[0], xu[1], yu[0], yu[1]};
    };
    if (!masked) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, v_frag(d, u, h)), pf[u][h], acc[d], 0, 0, 0);
    } else {
      // A hidden key's weight is 0, but 0 * Inf is not: values that are not finite go into the product as 0, and the
      // rows that see one get it back by a product of its own, of what is seen (0 or 1) with 1 for +Inf, 2^8 for -Inf and
      // 2^16 for NaN, whose sums over at most 64 keys tell the three apart.
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        uint32_t odd = 0;
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v4u x = v_frag(d, u, h);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const bool b0 = (x[k] & 0x7F80u) == 0x7F80u, b1 = (x[k] & 0x7F800000u) == 0x7F800000u;
              x[k] &= (b0 ? 0xFFFF0000u : ~0u) & (b1 ? 0xFFFFu : ~0u);
              odd |= static_cast<uint32_t>(b0 | b1);
            }
            acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, x), pf[u][h], acc[d], 0, 0, 0);
          }
        if (__any(odd != 0)) {
          v16f found;
#pragma unroll
          for (int r = 0; r < 16; ++r) found[r] = 0.0f;
#pragma unroll
          for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const v4u x = v_frag(d, u, h);
              v4u what, see;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                what[k] = see[k] = 0;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t y = (x[k] >> (16 * e)) & 0xFFFFu;
                  const uint32_t kind = y == 0x7F80u ? 0x3F80u : y == 0xFF80u ? 0x4380u : (y & 0x7F80u) == 0x7F80u ? 0x4780u : 0u;
                  const int j = k * 2 + e;              // key of element j: 4 hf + j, then 8 + 4 hf + (j - 4)
                  const int32_t t = t0 + u * 32 + h * 16 + (j >> 2) * 8 + hf * 4 + (j & 3);
                  what[k] |= kind << (16 * e);
                  see[k] |= (t <= seen ? 0x3F80u : 0u) << (16 * e);
                }
              }
              found = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, what), __builtin_bit_cast(v8bf, see),
                                                             found, 0, 0, 0);
            }
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const uint32_t n = static_cast<uint32_t>(found[r]);
            if (n & 0xFFu) acc[d][r] += INFINITY;
            if (n & 0xFF00u) acc[d][r] -= INFINITY;
            if (n >> 16) acc[d][r] = __builtin_nanf("");
          }
        }
      }
    }
  }

  if (i >= Lq) return;
  l += __shfl_xor(l, 32);
  const float inv = seen >= 0 && Lk > 0 ? 1.0f / l : 0.0f;
  uint16_t* row = a.out + (static_cast<int64_t>(q0 + i) * a.H + head) * D + hf * 4;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      *reinterpret_cast<uint2*>(row + d * 32 + r * 8) =
          make_uint2(pack_bf16x2(acc[d][4 * r] * inv, acc[d][4 * r + 1] * inv),
                     pack_bf16x2(acc[d][4 * r + 2] * inv, acc[d][4 * r + 3] * inv));
}

template <int D>
void launch(const PrefillArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(attn_prefill_kernel<D>, dim3(a.tiles * a.H), dim3(kThreads), 0, stream, a);
}

}  // namespace

size_t prefill_workspace_bytes(int64_t, int64_t, int64_t, int32_t, int32_t, int32_t) { return 0; }

mx_status launch_attn_prefill(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, const int32_t* q_offsets, const int32_t* k_offsets, int64_t B,
                              int64_t Tq, int64_t Tk, int32_t H, int32_t Hkv, int32_t D, float scale, void* out,
                              void* workspace, hipStream_t stream) {
  (void)workspace;
  PrefillArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_offsets = q_offsets;
  a.k_offsets = k_offsets;
  a.out = static_cast<uint16_t*>(out);
  a.scale = scale * 1.44269504088896340736f;
  a.B = static_cast<uint32_t>(B);
  a.Tq = static_cast<uint32_t>(Tq);
  a.Tk = static_cast<uint32_t>(Tk);
  a.H = static_cast<uint32_t>(H);
  a.Hkv = static_cast<uint32_t>(Hkv);
  a.G = a.H / a.Hkv;
  a.tiles = static_cast<uint32_t>(Tq / kRows + B);
  switch (D) {
    case 64: launch<64>(a, stream); break;
    case 128: launch<128>(a, stream); break;
    case 256: launch<256>(a, stream); break;
    default: launch<512>(a, stream); break;
  }
  return launch_status("mx_attn_prefill");
}

}  // namespace mx
