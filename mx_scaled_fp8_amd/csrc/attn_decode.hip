// Attention of one new token for each sequence over the paged cache (gfx950).
//
// For a sequence of n cached tokens and up to 16 query heads that share a key head,
//   S[t,h] = K[t,:] . Q[h,:],  P = exp2(c S - m_h),  O[h,:] = sum_t P[t,h] V[t,:] / sum_t P[t,h],  c = scale * log2(e),
// in one pass with the running maximum m and sum of the softmax.  What bounds it is the cache, which is read once from HBM:
// 2 D (1 + 1/32) bytes a token and head in MXFP8.
//
// The products run on 16x16x32 BF16 MFMAs with the tokens as rows: S^T = K Q^T leaves each lane with four tokens of one
// head (its column), which is what the second product O^T = V^T P^T wants of P^T, its B operand, if V^T's tokens are
// numbered the same way.  So P never leaves its lane, statistics are per column, and the rescaling of O^T too.
// A wave takes 32 tokens at a time, straight from global memory into registers:
//  - K: lane (c, g) = (lane % 16, lane / 16) holds 16-byte pieces of token c, the pieces of the four g side by side;
//    the order of D inside the product follows that, for Q too.
//  - V: lane (c, g) holds tokens 4g..4g+3 and 16 + 4g..+3 (the tokens of its P), elements c * DPL .. + DPL - 1 of each:
//    row c of MFMA i is element c * DPL + i, so that an operand is formed by v_perm of two tokens' BF16 pairs, with
//    no transposition through LDS.
// Codes become BF16 (exact) by v_cvt_scalef32_pk_bf16_fp8 with their block's scale.
//
// P is rounded to BF16 for the second product, which has no wider operand at this rate: up to 2^-8 of each weight, against 2^-8 of
// the result that BF16 outputs have anyway; m, the sum (of the unrounded P), S and O are FP32, the parts of a stream too.
//
// Work is shared as attn_plan.hpp says, in tiles of 128 tokens, 32 for each of the four waves.
//
// (MI355X.  64 sequences of up to 8192 tokens, 8 key heads of 128, 4 heads each, MXFP8: 116 us and 4 for the join, 4.8 TB/s of
// cache; 3 of up to 50,021 tokens, 4 key heads, BF16: 31 and 4.6 us, 6 TB/s, part of it from the caches behind L2.  One
// sequence of 1000 tokens: 6 and 3 us, a chain of latencies: lengths, table, K, V, parts.)
#include "attn_decode.hpp"

namespace mx {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

constexpr int kTile = 128;             // tokens of a tile of a share: 32 for each of four waves
constexpr int kHeads = 16;             // query heads of a stream: one (sequence, key head, group of up to 16 query heads)

__device__ __forceinline__ float across_groups_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16));
  return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float across_groups_sum(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

// Shapes of a wave's 32 tokens in registers.
template <int D, bool FP8>
struct Shape {
  static constexpr int EB = FP8 ? 1 : 2;                // bytes of an element
  static constexpr int KP = D * EB / 64;                // 16-byte pieces of a K row in a lane
  static constexpr int KS = D / 32;                     // MFMA steps of the first product
  static constexpr int PANEL = FP8 ? (D < 256 ? D : 256) : (D < 128 ? D : 128);
  static constexpr int NP = D / PANEL;
  static constexpr int DPL = PANEL / 16;                // elements of V in a lane, panel and token
  static constexpr int VW = DPL * EB / 4;               // their words
  static constexpr int SB = D / 32;                     // scale bytes of a row
  static constexpr int SW = (SB + 3) / 4;               // their words
  static constexpr bool WIDE = SB <= 4;                 // V's scales of 4 tokens by one load of all their bytes
  // As many registers as one wave's loads of a tile take; two tiles are held where two waves a SIMD still have room.
  static constexpr int REGS = 2 * 4 * KP + 8 * NP * VW + (FP8 ? 2 * SW + (WIDE ? 2 * SB : 8 * NP) : 0);
  static constexpr bool AHEAD = 2 * REGS + D / 4 + D / 8 <= 170;
  // Rows of 512 fill the registers with O and Q: the second 16 rows of K are loaded when the first are used up, V after
  // that.  (All of a tile at once spilled registers.)
  static constexpr bool LATE = D >= 512;
};

// What a wave reads of 32 tokens.
template <int D, bool FP8>
struct Tokens {
  using S = Shape<D, FP8>;
  v4u k[2][S::KP];
  uint32_t ks[2][FP8 ? S::SW : 1];
  uint32_t v[8][S::NP][S::VW];
  uint32_t vs[FP8 ? (S::WIDE ? 2 * S::SB : 8 * S::NP) : 1];
  int64_t rows[2];           // the cache row of token 16 u
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t* to, const uint8_t* from) {
  if constexpr (N == 4) *reinterpret_cast<v4u*>(to) = *reinterpret_cast<const v4u*>(from);
  else if constexpr (N == 2) *reinterpret_cast<v2u*>(to) = *reinterpret_cast<const v2u*>(from);
  else if constexpr (N == 1) *to = *reinterpret_cast<const uint32_t*>(from);
  else {
    load_words<4>(to, from);
    load_words<N - 4>(to + 4, from + 16);
  }
}

template <int D, bool FP8>
__device__ __forceinline__ void load_k(const KvCache& c, int u, Tokens<D, FP8>& x) {
  using S = Shape<D, FP8>;
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const uint8_t* kp = c.k + (x.rows[u] + col) * (D * S::EB) + g * 16;
#pragma unroll
  for (int j = 0; j < S::KP; ++j) x.k[u][j] = *reinterpret_cast<const v4u*>(kp + j * 64);
  if constexpr (FP8) {
    const uint8_t* sp = c.ks + (x.rows[u] + col) * S::SB;
    if constexpr (S::SB == 2) x.ks[u][0] = *reinterpret_cast<const uint16_t*>(sp);
    else load_words<S::SW>(x.ks[u], sp);
  }
}

template <int D, bool FP8>
__device__ __forceinline__ void load_v(const KvCache& c, int p, Tokens<D, FP8>& x) {
  using S = Shape<D, FP8>;
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t row = x.rows[u] + g * 4;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      load_words<S::VW>(x.v[u * 4 + j][p], c.v + ((row + j) * D + p * S::PANEL + col * S::DPL) * S::EB);
    if constexpr (FP8) {
      if constexpr (S::WIDE) {
        load_words<S::SB>(&x.vs[u * S::SB], c.vs + row * S::SB);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x.vs[(u * 4 + j) * S::NP + p] = c.vs[(row + j) * S::SB + (p * S::PANEL + col * S::DPL) / 32];
      }
    }
  }
}

// WHOLE: every workgroup takes one stream from end to end, nothing is left to join.
template <int D, bool WHOLE>
constexpr int waves_of() { return WHOLE && D <= 256 ? 8 : 4; }

template <int D, bool FP8, bool WHOLE>
__global__ __launch_bounds__((64 * waves_of<D, WHOLE>()), D <= 128 ? 2 : 1) void attn_decode_kernel(DecodeArgs a) {
  using S = Shape<D, FP8>;
  constexpr int WAVES = waves_of<D, WHOLE>(), TILE = 32 * WAVES;
  constexpr int DPL = S::DPL, NP = S::NP, PANEL = S::PANEL;
  __shared__ float sml[WAVES][kHeads][2];
  __shared__ __attribute__((aligned(16))) float sacc[WAVES][kHeads][D + 4];   // + 4: the columns' rows in different banks
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, g = lane >> 4;

  Share sh;
  if constexpr (WHOLE) {                                // tiles numbered from this sequence's first
    const uint32_t x = blockIdx.x / a.head_blocks;
    sh.block = blockIdx.x - x * a.head_blocks;
    sh.b = x / a.c.Hkv;
    const uint32_t of = (tokens_of(a, sh.b) + TILE - 1) / TILE, kvh = x - sh.b * a.c.Hkv;
    sh.group = sh.first = 0;
    sh.t = kvh * of;
    sh.end = sh.t + of;
    if (of == 0) {
      const uint32_t h0 = kvh * a.G + sh.block * kHeads;
      const uint32_t heads = min(static_cast<uint32_t>(kHeads), (kvh + 1) * a.G - h0);
      for (uint32_t e = threadIdx.x * 4; e < heads * D; e += 64 * WAVES * 4)
        *reinterpret_cast<uint2*>(a.out + (static_cast<size_t>(sh.b) * a.H + h0) * D + e) = make_uint2(0, 0);
    }
  } else {
    sh = find_share<TILE, 1>(a);
  }
  while (sh.t < sh.end) {
    const Piece pc = piece_of<TILE, kHeads>(a, sh);
    const uint32_t b = sh.b, kvh = pc.kvh, h0 = pc.h0, heads = pc.heads, tile0 = pc.tile0, n = pc.tiles;
    const bool whole = WHOLE || n == pc.of;
    const uint32_t len = tokens_of(a, b);
    bool bad = a.lens[b] > static_cast<int32_t>(len);   // longer than its table

    // Q, the B operand: column `col` is query head h0 + col (the last one again past it), D in the order of K's pieces
    v8bf qf[S::KS];
    {
      const uint16_t* qrow = a.q + static_cast<int64_t>(b) * a.q_stride + (h0 + min(static_cast<uint32_t>(col), heads - 1)) * D;
#pragma unroll
      for (int j = 0; j < S::KS; ++j) {
        const int d = FP8 ? (j >> 1) * 64 + g * 16 + (j & 1) * 8 : j * 32 + g * 8;
        qf[j] = *reinterpret_cast<const v8bf*>(qrow + d);
      }
    }
    float m = -INFINITY, l = 0.0f;
    v4f acc[NP][DPL];
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int i = 0; i < DPL; ++i) acc[p][i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    const int32_t* table = a.c.table + static_cast<int64_t>(b) * a.c.max_pages;
    // The wave's tokens of tile i of the piece, if there are any, and the rows of its two groups of 16, each inside one
    // page; a group past the end reads the first one again.
    auto token = [&](uint32_t i) { return (tile0 + i) * TILE + static_cast<uint32_t>(wave) * 32; };
    auto some = [&](uint32_t i) { return i < n && token(i) < len; };
    uint32_t page[2] = {0, 0};
    auto find_pages = [&](uint32_t i) {
      if (!some(i)) return;
      const uint32_t t0 = token(i), t1 = t0 + 16 < len ? t0 + 16 : t0;
      page[0] = static_cast<uint32_t>(table[t0 >> a.c.page_shift]);
      page[1] = static_cast<uint32_t>(table[t1 >> a.c.page_shift]);
    };
    auto load = [&](uint32_t i, Tokens<D, FP8>& x) {
      if (!some(i)) return;
      const uint32_t t0 = token(i), t1 = t0 + 16 < len ? t0 + 16 : t0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (page[u] >= a.c.pages) {
          bad = true;
          page[u] = 0;
        }
        x.rows[u] = ((static_cast<int64_t>(page[u]) * a.c.Hkv + kvh) << a.c.page_shift) + ((u ? t1 : t0) & ((1u << a.c.page_shift) - 1));
      }
      load_k<D, FP8>(a.c, 0, x);
      if constexpr (!S::LATE) {
        load_k<D, FP8>(a.c, 1, x);
        load_v<D, FP8>(a.c, 0, x);
      }
    };
    auto compute = [&](uint32_t i, Tokens<D, FP8>& x) {
      const uint32_t tok0 = token(i);
      v4f s2[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < S::KP; ++j) {
          if constexpr (FP8) {
            const uint32_t byte = 2 * j + (g >> 1), sc = (x.ks[u][j / 2] >> (8 * (byte & 3))) & 0xFFu;
            const float sb = __uint_as_float(sc << 23);
            const uint32_t nan = nan_codes(sc);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t w0 = x.k[u][j][half * 2] | nan, w1 = x.k[u][j][half * 2 + 1] | nan;
              const v4u op = {dequant_pair<false>(w0, sb), dequant_pair<true>(w0, sb), dequant_pair<false>(w1, sb),
                              dequant_pair<true>(w1, sb)};
              y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, op), qf[j * 2 + half], y, 0, 0, 0);
            }
          } else {
            y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x.k[u][j]), qf[j], y, 0, 0, 0);
          }
        }
        s2[u] = y;
        if constexpr (S::LATE) {
          asm volatile("" ::: "memory");               // not before the products
          if (u == 0) load_k<D, FP8>(a.c, 1, x);
          else load_v<D, FP8>(a.c, 0, x);
        }
      }
      const bool tail = tok0 + 32 > len;
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float y = s2[u][r] * a.scale;
          if (tail && tok0 + u * 16 + g * 4 + r >= len) y = -INFINITY;
          s2[u][r] = y;
          top = fmaxf(top, y);
        }
      top = fmaxf(m, across_groups_max(top));
      const float base = top == -INFINITY ? 0.0f : top;   // nothing but -inf so far: all weights are 0
      if (__any(top > m)) {
        const float f = __builtin_amdgcn_exp2f(m - base);
        l *= f;
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
          for (int k = 0; k < DPL; ++k) acc[p][k] *= f;
        m = top;
      }
      uint32_t pw[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          w[r] = __builtin_amdgcn_exp2f(s2[u][r] - base);
          l += w[r];
        }
        pw[u * 2] = pack_bf16x2(w[0], w[1]);
        pw[u * 2 + 1] = pack_bf16x2(w[2], w[3]);
      }
      const v8bf pf = __builtin_bit_cast(v8bf, (v4u{pw[0], pw[1], pw[2], pw[3]}));
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        if (p + 1 < NP) load_v<D, FP8>(a.c, p + 1, x);
        uint32_t pair[8][DPL / 2];                        // BF16 pairs of the lane's 8 tokens
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool out = tail && tok0 + (j >> 2) * 16 + g * 4 + (j & 3) >= len;   // whatever lies there, it counts as 0
          if constexpr (FP8) {
            uint32_t sc;
            if constexpr (S::WIDE) {                      // byte `at` of row j % 4
              const uint32_t at = col * DPL / 32;
              if constexpr (S::SB == 4) sc = (x.vs[j] >> (8 * at)) & 0xFFu;
              else sc = (x.vs[j >> 1] >> (8 * ((j & 1) * 2 + at))) & 0xFFu;
            } else {
              sc = x.vs[j * NP + p];
            }
            if (out) sc = 127;
            const float sb = __uint_as_float(sc << 23);
            const uint32_t nan = nan_codes(sc);
#pragma unroll
            for (int k = 0; k < S::VW; ++k) {
              const uint32_t w = out ? 0u : x.v[j][p][k] | nan;
              pair[j][k * 2] = dequant_pair<false>(w, sb);
              pair[j][k * 2 + 1] = dequant_pair<true>(w, sb);
            }
          } else {
#pragma unroll
            for (int k = 0; k < S::VW; ++k) pair[j][k] = out ? 0u : x.v[j][p][k];
          }
        }
#pragma unroll
        for (int k = 0; k < DPL / 2; ++k) {
          v4u even, odd;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            even[j] = __builtin_amdgcn_perm(pair[2 * j + 1][k], pair[2 * j][k], 0x05040100u);
            odd[j] = __builtin_amdgcn_perm(pair[2 * j + 1][k], pair[2 * j][k], 0x07060302u);
          }
          acc[p][2 * k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, even), pf, acc[p][2 * k], 0, 0, 0);
          acc[p][2 * k + 1] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, odd), pf, acc[p][2 * k + 1], 0, 0, 0);
        }
      }
    };

    find_pages(0);
    if constexpr (S::AHEAD) {
      Tokens<D, FP8> x, y;
      load(0, x);
      find_pages(1);
      for (uint32_t i = 0; some(i); i += 2) {
        load(i + 1, y);
        find_pages(i + 2);
        compute(i, x);
        load(i + 2, x);
        find_pages(i + 3);
        if (some(i + 1)) compute(i + 1, y);
      }
    } else {
      Tokens<D, FP8> x;
      for (uint32_t i = 0; some(i); ++i) {
        load(i, x);
        find_pages(i + 1);
        compute(i, x);
      }
    }

    // the waves' parts into one
    l = across_groups_sum(l);
    if (bad) l = __builtin_nanf("");
    __syncthreads();                                      // the last stream's parts have been read
    if (g == 0) {
      sml[wave][col][0] = m;
      sml[wave][col][1] = l;
    }
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < DPL; i += 4)
          *reinterpret_cast<v4f*>(&sacc[wave][col][p * PANEL + (g * 4 + r) * DPL + i]) =
              v4f{acc[p][i][r], acc[p][i + 1][r], acc[p][i + 2][r], acc[p][i + 3][r]};
    __syncthreads();
    float* part = part_of(a, sh.group, sh.block, tile0 == 0, kHeads * (D + 2));
    for (uint32_t e = threadIdx.x * 4; e < heads * D; e += 64 * WAVES * 4) {
      const uint32_t h = e / D, d = e % D;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = fmaxf(top, sml[w][h][0]);
      const float base = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f;
      v4f o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float f = __builtin_amdgcn_exp2f(sml[w][h][0] - base);
        sum += sml[w][h][1] * f;
        o += *reinterpret_cast<const v4f*>(&sacc[w][h][d]) * f;
      }
      if (whole) {
        const float inv = 1.0f / sum;
        *reinterpret_cast<uint2*>(a.out + (static_cast<size_t>(b) * a.H + h0 + h) * D + d) =
            make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
      } else {
        *reinterpret_cast<v4f*>(part + h * D + d) = o;
        if (d == 0) {
          part[kHeads * D + h] = top;
          part[kHeads * D + kHeads + h] = sum;
        }
      }
    }
    if constexpr (WHOLE) return;
    advance(a, sh, pc);
  }
}

// Groups of a call: as many as run at once, and no more than there can be tiles.  Heads of 64 and 128 leave registers for two
// workgroups on a compute unit, heads of 256 and 512 for one.  (256 groups and 512, heads of 256: 3 sequences up to 50,021 tokens, 2 x
// 7 heads, MXFP8 31.2 us and 38.9, BF16 45.5 and 52.6; 8 up to 2000, 4 x 4 heads, BF16 15.0 and 18.7; 64 up to 8192, MXFP8 131.2 and
// 129.7.)
uint32_t groups_of(int64_t B, int32_t Hkv, uint32_t head_blocks, int32_t D, int64_t max_tokens) {
  return decode_groups(B * Hkv * ((max_tokens + kTile - 1) / kTile), (D >= 256 ? 256 : 512) / head_blocks);
}

uint32_t head_blocks_of(int32_t G) { return static_cast<uint32_t>((G + kHeads - 1) / kHeads); }

// Whether streams are short enough for one workgroup each, which saves the second kernel.  (8 key heads of 128, MXFP8, in a
// graph: one sequence of 300 tokens 6.8 us whole and 8.3 in shares, of 1000 tokens 12.5 and 8.9; 64 sequences up to 1000
// tokens 25.4 and 28.0, up to 2000 39.2 and 37.8.)
bool short_streams(int64_t streams, int64_t max_tokens) { return max_tokens <= (streams >= 512 ? 1024 : 512); }

template <int D, bool FP8>
void launch(DecodeArgs a, int64_t max_tokens, hipStream_t stream) {
  if (short_streams(static_cast<int64_t>(a.B) * a.c.Hkv * a.head_blocks, max_tokens)) {
    hipLaunchKernelGGL((attn_decode_kernel<D, FP8, true>), dim3(a.B * a.c.Hkv * a.head_blocks), dim3(64 * waves_of<D, true>()), 0, stream, a);
    return;
  }
  a.groups = groups_of(a.B, static_cast<int32_t>(a.c.Hkv), a.head_blocks, D, max_tokens);
  hipLaunchKernelGGL((attn_decode_kernel<D, FP8, false>), dim3(a.groups * a.head_blocks), dim3(64 * waves_of<D, false>()), 0, stream, a);
  hipLaunchKernelGGL((attn_join_kernel<D, kTile, kHeads>), dim3(a.B * a.H), dim3(kJoinThreads), 0, stream, a);
}

size_t plan_bytes(int64_t B) { return (static_cast<size_t>(B) + 1 + 3) / 4 * 16; }

}  // namespace

size_t decode_workspace_bytes(int64_t B, int32_t H, int32_t Hkv, int32_t D, int64_t max_tokens) {
  const uint32_t blocks = head_blocks_of(H / Hkv);
  const size_t few = static_cast<size_t>(groups_of(B, Hkv, blocks, D, max_tokens)) * blocks * 2 * kHeads * (D + 2) * 4;
  return plan_bytes(B) + std::max(few, decode_rows_part_bytes(B, H, Hkv, D, max_tokens));
}

mx_status launch_attn_decode(const void* q, int64_t q_stride, int64_t B, int32_t H, int32_t D, bool fp8,
                             const KvCache& c, const int32_t* lens, float scale, void* out, void* workspace,
                             hipStream_t stream) {
  DecodeArgs a;
  a.c = c;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.lens = lens;
  a.out = static_cast<uint16_t*>(out);
  a.plan = static_cast<uint32_t*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan_bytes(B));
  a.scale = scale * kLog2E;
  a.B = static_cast<uint32_t>(B);
  a.H = static_cast<uint32_t>(H);
  a.G = a.H / c.Hkv;
  const int64_t max_tokens = static_cast<int64_t>(c.max_pages) << c.page_shift;
  if (decode_by_rows(static_cast<int32_t>(a.G), D, c.k == c.v && c.ks == c.vs, fp8)) {
    launch_decode_rows(a, D, fp8, max_tokens, stream);
  } else {
    a.head_blocks = head_blocks_of(static_cast<int32_t>(a.G));
    a.part_heads = kHeads;
    switch (D) {
      case 64: fp8 ? launch<64, true>(a, max_tokens, stream) : launch<64, false>(a, max_tokens, stream); break;
      case 128: fp8 ? launch<128, true>(a, max_tokens, stream) : launch<128, false>(a, max_tokens, stream); break;
      case 256: fp8 ? launch<256, true>(a, max_tokens, stream) : launch<256, false>(a, max_tokens, stream); break;
      default: fp8 ? launch<512, true>(a, max_tokens, stream) : launch<512, false>(a, max_tokens, stream); break;
    }
  }
  return launch_status("mx_attn_decode");
}

}  // namespace mx
