// Attention of one new token where many query heads share a key head (gfx950): a latent cache above all.
//
// With 128 heads over a key of 512 elements a token costs 2^18 operations for 528 bytes: the matrix cores bound it, not the
// cache.  So the heads are the rows of attn_tile.hpp's products, 128 to a workgroup, and a tile of keys is brought to LDS
// once for all of them, as BF16: MXFP8 codes are loaded into registers a turn ahead (their pages' numbers two), become
// BF16 (exact) and are written to the buffer that the last turn read, under this turn's products.
// Work is shared as attn_plan.hpp says.
#include "attn_decode.hpp"
#include "attn_tile.hpp"

namespace mx {

namespace {

constexpr int kRows = 128;             // query heads of a stream
constexpr int kMinTokens = 256;        // of a share: its part is up to 128 rows of FP32, as much as 500 cached tokens

template <int D>
constexpr int key_tile() { return D <= 128 ? 64 : 32; }
template <int D>
constexpr int halves_of() { return D >= 512 ? 2 : 1; }
template <int D>
constexpr int threads_of() { return 256 * halves_of<D>(); }

template <int D, bool FP8, bool SAME>
__global__ __launch_bounds__(threads_of<D>(), 2) void attn_decode_rows_kernel(DecodeArgs a) {
  constexpr int HALVES = halves_of<D>(), THREADS = threads_of<D>(), KT = key_tile<D>();
  constexpr int TB = KT * D * 2;                        // bytes of a tile in LDS
  constexpr int EB = FP8 ? 1 : 2;
  constexpr int CE = 16 / EB;                           // elements of a 16-byte chunk in the cache
  constexpr int CPR = D / CE;                           // chunks of a row
  constexpr int NC = KT * CPR / THREADS;                // a thread's chunks of a tile
  constexpr int RS = THREADS / CPR;                     // tokens between two of them
  constexpr int KV = SAME ? 1 : 2;
  using Tile = AttnTile<D, KT, HALVES>;
  constexpr int SUB = Tile::SUB;
  static_assert(NC >= 1 && KT % RS == 0, "every thread has its share of a tile");
  __shared__ __attribute__((aligned(1024))) uint8_t buf[2][KV][TB];
  __shared__ __attribute__((aligned(16))) uint8_t partial[HALVES == 1 ? 16 : 8 * SUB * 4096];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 31;
  const int group = wave & 3, half = wave >> 2;
  const uint32_t tok = threadIdx.x / CPR, chunk = threadIdx.x % CPR;   // of the thread's first chunk

  Share sh = find_share<KT, kMinTokens / KT>(a);
  while (sh.t < sh.end) {
    const Piece pc = piece_of<KT, kRows>(a, sh);
    const uint32_t len = tokens_of(a, sh.b);
    bool bad = a.lens[sh.b] > static_cast<int32_t>(len);
    const int32_t* table = a.c.table + static_cast<int64_t>(sh.b) * a.c.max_pages;
    const bool active = static_cast<uint32_t>(group * 32) < pc.heads;   // the wave has heads

    Tile w;
    w.begin(half);
    w.load_q(a.q + static_cast<int64_t>(sh.b) * a.q_stride + (pc.h0 + min(static_cast<uint32_t>(group * 32 + col), pc.heads - 1)) * D +
             half * Tile::DH);

    uint32_t page[NC];
    v4u code[KV][NC];
    uint32_t scale[KV][NC];
    const uint32_t last = pc.tile0 + pc.tiles;
    auto pages = [&](uint32_t tile) {                   // the pages' numbers of a tile's tokens
#pragma unroll
      for (int x = 0; x < NC; ++x) {
        const uint32_t at = tile * KT + tok + x * RS;
        page[x] = tile < last && at < len ? static_cast<uint32_t>(table[at >> a.c.page_shift]) : 0u;
      }
    };
    auto load = [&](uint32_t tile) {
      if (tile >= last) return;
#pragma unroll
      for (int x = 0; x < NC; ++x) {
        const uint32_t at = tile * KT + tok + x * RS;
        if (page[x] >= a.c.pages) {
          bad = true;
          page[x] = 0;
        }
        const int64_t row = ((static_cast<int64_t>(page[x]) * a.c.Hkv + pc.kvh) << a.c.page_shift) + (at & ((1u << a.c.page_shift) - 1));
#pragma unroll
        for (int i = 0; i < KV; ++i) {
          code[i][x] = *reinterpret_cast<const v4u*>((i == 0 ? a.c.k : a.c.v) + row * (D * EB) + chunk * 16);
          if constexpr (FP8) scale[i][x] = (i == 0 ? a.c.ks : a.c.vs)[row * (D / 32) + chunk / 2];
        }
      }
    };
    auto store = [&](uint32_t tile, uint8_t (&to)[KV][TB]) {   // rows past the end as zeros
      if (tile >= last) return;
#pragma unroll
      for (int x = 0; x < NC; ++x) {
        const uint32_t r = tok + x * RS;
        const bool out = tile * KT + r >= len;
#pragma unroll
        for (int i = 0; i < KV; ++i) {
          v4u v = code[i][x];
          if constexpr (FP8) {
            const float sb = __uint_as_float(scale[i][x] << 23);
            const uint32_t nan = nan_codes(scale[i][x]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w0 = v[2 * h] | nan, w1 = v[2 * h + 1] | nan;
              v4u o = {dequant_pair<false>(w0, sb), dequant_pair<true>(w0, sb), dequant_pair<false>(w1, sb), dequant_pair<true>(w1, sb)};
              if (out) o = v4u{0, 0, 0, 0};
              *reinterpret_cast<v4u*>(&to[i][r * D * 2 + (swizzled<D>(chunk * 2 + h, r) << 4)]) = o;
            }
          } else {
            if (out) v = v4u{0, 0, 0, 0};
            *reinterpret_cast<v4u*>(&to[i][r * D * 2 + (swizzled<D>(chunk, r) << 4)]) = v;
          }
        }
      }
    };
    auto step = [&](uint32_t tile, uint8_t (&now)[KV][TB], uint8_t (&next)[KV][TB]) {
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // the tile is whole; everyone has read `next`
      store(tile + 1, next);
      load(tile + 2);
      pages(tile + 3);
      v16f s[SUB];
      w.hide_bases();
      if (active) w.scores(now[0], s);
      if constexpr (HALVES == 2) Tile::exchange(s, partial + wave * SUB * 4096, partial + (wave ^ 4) * SUB * 4096, active);
      if (!active) return;
      const int32_t seen = static_cast<int32_t>(len - tile * KT);
      if (seen < KT) {
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int x = 0; x < 16; ++x) s[u][x] = u * 32 + w.key_of(x) < seen ? s[u][x] : -INFINITY;
      }
      v8bf pf[SUB][2];
      w.weights(s, a.scale, pf);
      w.values(now[KV - 1], pf);
    };

    uint32_t tile = pc.tile0;
    pages(tile);
    load(tile);
    pages(tile + 1);
    __syncthreads();                                    // the last piece's tiles have been read
    store(tile, buf[0]);
    load(tile + 1);
    pages(tile + 2);
    for (; tile < last; tile += 2) {
      step(tile, buf[0], buf[1]);
      if (tile + 1 < last) step(tile + 1, buf[1], buf[0]);
    }

    const float2 sums = halves(w.l);
    w.l = sums.x + sums.y;
    // a bad page is some thread's: all rows are NaN
    if (__syncthreads_or(bad)) w.l = __builtin_nanf("");
    const uint32_t r = group * 32 + col;
    if (active && r < pc.heads) {
      if (pc.tiles == pc.of) {
        const float inv = 1.0f / w.l;
        uint16_t* row = a.out + (static_cast<size_t>(sh.b) * a.H + pc.h0 + r) * D + half * Tile::DH + w.hf * 4;
#pragma unroll
        for (int d = 0; d < Tile::DT; ++d)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint2*>(row + d * 32 + x * 8) =
                make_uint2(pack_bf16x2(w.acc[d][4 * x] * inv, w.acc[d][4 * x + 1] * inv),
                           pack_bf16x2(w.acc[d][4 * x + 2] * inv, w.acc[d][4 * x + 3] * inv));
      } else {
        float* part = part_of(a, blockIdx.x, pc.tile0 == 0, kRows * (D + 2));
        float* row = part + r * D + half * Tile::DH + w.hf * 4;
#pragma unroll
        for (int d = 0; d < Tile::DT; ++d)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<float4*>(row + d * 32 + x * 8) =
                make_float4(w.acc[d][4 * x], w.acc[d][4 * x + 1], w.acc[d][4 * x + 2], w.acc[d][4 * x + 3]);
        if (w.hf == 0 && half == 0) {
          part[kRows * D + r] = w.m;
          part[kRows * D + kRows + r] = w.l;
        }
      }
    }
    advance(a, sh, pc);
  }
}

uint32_t head_blocks_of(int32_t G) { return static_cast<uint32_t>((G + kRows - 1) / kRows); }

// Workgroups: as many as run at once, and no more than there can be tiles.
uint32_t groups_of(int64_t B, uint32_t streams, int32_t D, int64_t max_tokens) {
  const int64_t kt = D <= 128 ? 64 : 32, tiles = B * streams * ((max_tokens + kt - 1) / kt);
  return static_cast<uint32_t>(std::min<int64_t>(D >= 512 ? 256 : 512, tiles));
}

template <int D, bool FP8>
void launch(const DecodeArgs& a, uint32_t groups, hipStream_t stream) {
  const dim3 block(threads_of<D>());
  if (D >= 512 || (a.c.k == a.c.v && a.c.ks == a.c.vs)) {
    hipLaunchKernelGGL((attn_decode_rows_kernel<D, FP8, true>), dim3(groups), block, 0, stream, a);
  } else if constexpr (D < 512) {
    hipLaunchKernelGGL((attn_decode_rows_kernel<D, FP8, false>), dim3(groups), block, 0, stream, a);
  }
  hipLaunchKernelGGL((attn_join_kernel<D, key_tile<D>(), kRows>), dim3(a.B * a.H), dim3(kJoinThreads), 0, stream, a);
}

}  // namespace

// From 32 heads on the rows fill at least one wave's products, and the cache is read once, not once for each 16 heads.
// Rows of 512 have no room in LDS for values of their own.
bool decode_by_rows(int32_t G, int32_t D, bool latent) { return G >= 32 && (D < 512 || latent); }

size_t decode_rows_part_bytes(int64_t B, int32_t H, int32_t Hkv, int32_t D, int64_t max_tokens) {
  const int32_t G = H / Hkv;
  if (!decode_by_rows(G, D, true)) return 0;
  return static_cast<size_t>(groups_of(B, Hkv * head_blocks_of(G), D, max_tokens)) * 2 * kRows * (D + 2) * 4;
}

void launch_decode_rows(DecodeArgs a, int32_t D, bool fp8, int64_t max_tokens, hipStream_t stream) {
  a.head_blocks = head_blocks_of(static_cast<int32_t>(a.G));
  a.streams = a.c.Hkv * a.head_blocks;
  const uint32_t groups = groups_of(a.B, a.streams, D, max_tokens);
  switch (D) {
    case 64: fp8 ? launch<64, true>(a, groups, stream) : launch<64, false>(a, groups, stream); break;
    case 128: fp8 ? launch<128, true>(a, groups, stream) : launch<128, false>(a, groups, stream); break;
    case 256: fp8 ? launch<256, true>(a, groups, stream) : launch<256, false>(a, groups, stream); break;
    default: fp8 ? launch<512, true>(a, groups, stream) : launch<512, false>(a, groups, stream); break;
  }
}

}  // namespace mx
