// Attention of one new token where many query heads share a key head (gfx950): a latent cache above all.
//
// With 128 heads over a key of 512 elements a token costs 2^18 operations for 528 bytes: the matrix cores bound it, not the
// cache.  So the heads are the rows of attn_tile.hpp's products, 128 to a workgroup, and a tile of keys is brought to LDS
// once for all of them.  BF16 rows come by DMA as in the prompt attention.  MXFP8 codes come by DMA into a place of their own
// a turn ahead, where the wave that asked for them makes BF16 of them (exact) under the other waves' products and writes
// it to the buffer that the last turn read; registers hold O and Q and have no room for codes under way.
// Work is shared as attn_plan.hpp says.
#include <type_traits>

#include "attn_decode.hpp"
#include "attn_tile.hpp"

namespace mx {

namespace {

constexpr int kMinTokens = 256;        // of a share: its part is up to 128 rows of FP32, as much as 500 cached tokens

// Query heads of a workgroup: 32 or 16 for each of four waves, half of what a compute unit runs, so that two workgroups,
// which know nothing of each other's barriers, fill it.
constexpr int rows_of(int) { return 128; }
constexpr int threads_of(int D) { return D >= 512 ? 512 : 256; }

template <int D, bool FP8, bool SAME>
__global__ __launch_bounds__(threads_of(D), 2) void attn_decode_rows_kernel(DecodeArgs a) {
  using Tile = typename TileOf<D, 4>::type;              // (6 ahead: no registers, and the compiler reads none ahead)
  constexpr int ROWS = rows_of(D), WAVES = ROWS / Tile::ROWS, KT = key_tile<D>();
  constexpr int TB = KT * D * 2;                        // bytes of a tile in LDS
  constexpr int EB = FP8 ? 1 : 2;
  constexpr int RW = KT / WAVES;                        // rows that a wave brings: of one page
  constexpr int RPI = 1024 / (D * EB);                  // of one DMA instruction
  constexpr int CPR = D * EB / 16;                      // 16-byte chunks of a row in the cache
  constexpr int NI = RW / RPI;                          // instructions
  constexpr int SB = D / 32;                            // scale bytes of a row
  constexpr int KV = SAME ? 1 : 2;
  constexpr int RAW = FP8 ? KT * D : 16;
  static_assert(NI >= 1 && 16 % RW == 0 && RW * SB <= 256, "a wave's rows are of one page, their scales a word a lane");
  __shared__ __attribute__((aligned(1024))) uint8_t buf0[KV][TB], buf1[KV][TB], raw[KV][RAW];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t r = wave * Tile::ROWS + Tile::row();   // the lane's row

  Share sh = find_share<KT, kMinTokens / KT>(a);
  while (sh.t < sh.end) {
    const Piece pc = piece_of<KT, ROWS>(a, sh);
    const uint32_t len = tokens_of(a, sh.b);
    const bool bad = a.lens[sh.b] > static_cast<int32_t>(len);   // longer than its table
    const int32_t* table = a.c.table + static_cast<int64_t>(sh.b) * a.c.max_pages;
    const bool active = static_cast<uint32_t>(wave * Tile::ROWS) < pc.heads;   // the wave has heads

    Tile w;
    w.begin();
    w.load_q(a.q + static_cast<int64_t>(sh.b) * a.q_stride + (pc.h0 + min(r, pc.heads - 1)) * D);

    // A wave brings rows wave * RW .. of a tile.  Rows of a page outside the cache are read from page 0 and made NaN
    // (`lost`); rows past the end are zeros.
    const uint32_t last = pc.tile0 + pc.tiles;
    uint32_t page = 0, scale[KV];                         // scale: the rows' scale bytes, four a lane
    bool lost = false, lost_next = false;
    auto first_token = [&](uint32_t tile) { return tile * KT + static_cast<uint32_t>(wave) * RW; };
    // The page's number by a scalar load (nothing writes the table meanwhile), which holds no vector register and does not
    // wait behind the DMA; past the end, the last token's page again.
    const auto* numbers = (const __attribute__((address_space(4))) int32_t*)table;
    auto find_page = [&](uint32_t tile) {
      page = static_cast<uint32_t>(numbers[__builtin_amdgcn_readfirstlane(min(first_token(tile), len - 1) >> a.c.page_shift)]);
    };
    // The lane's number as the compiler cannot see through: addresses are formed where they are used, and not held in
    // registers that a wide row needs.
    auto hidden = [&]() {
      uint32_t x = lane;
      if constexpr (D >= 256) asm volatile("" : "+v"(x));
      return x;
    };
    auto load = [&](uint32_t tile, uint8_t (&to)[KV][TB]) {
      if (tile >= last) return;
      const uint32_t lane = hidden();
      lost_next = page >= a.c.pages;
      const uint32_t at = lost_next ? 0u : page;
      const int64_t row = ((static_cast<int64_t>(at) * a.c.Hkv + pc.kvh) << a.c.page_shift) +
                          (min(first_token(tile), len - 1) & ((1u << a.c.page_shift) - 1) & ~(RW - 1));
#pragma unroll
      for (int i = 0; i < KV; ++i) {
        const uint8_t* from = (i == 0 ? a.c.k : a.c.v) + row * (D * EB);
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const uint32_t r0 = wave * RW + x * RPI;
          if constexpr (FP8) dma16_at(from + x * 1024 + lane * 16, &raw[i][r0 * D]);
          else dma16_at(from + x * 1024 + lane / CPR * (D * 2) + (swizzled<D>(lane % CPR, r0 + lane / CPR) << 4), &to[i][r0 * D * 2]);
        }
        if constexpr (FP8)
          scale[i] = *reinterpret_cast<const uint32_t*>((i == 0 ? a.c.ks : a.c.vs) + row * SB + lane * 4 % (RW * SB));
      }
    };
    // The wave's codes, which are there, to BF16.
    auto convert_rows = [&](auto EDGE, uint32_t tile, uint8_t (&to)[KV][TB]) {
      const uint32_t lane = hidden(), c = lane % CPR;
#pragma unroll
      for (int i = 0; i < KV; ++i) {
        v4u v[NI];
        uint32_t sc[NI];
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const uint32_t byte = (x * RPI + lane / CPR) * SB + c / 2;
          v[x] = *reinterpret_cast<const v4u*>(&raw[i][(wave * RW + x * RPI) * D + lane * 16]);
          sc[x] = __shfl(scale[i], byte / 4) >> (8 * (byte & 3)) & 0xFFu;
        }
        asm volatile("" ::: "memory");                  // all reads under way before the first is used
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          const uint32_t r = wave * RW + x * RPI + lane / CPR;   // row of the tile
          const float sb = __uint_as_float(sc[x] << 23);
          const uint32_t nan = nan_codes(sc[x]);
          // half of the lanes write their second eight elements first, so that 16 lanes meet all banks
          const uint32_t turned = (c >> 3) & 1;
          if (turned) v[x] = v4u{v[x][2], v[x][3], v[x][0], v[x][1]};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w0 = v[x][2 * h] | nan, w1 = v[x][2 * h + 1] | nan;
            v4u o = {dequant_pair<false>(w0, sb), dequant_pair<true>(w0, sb), dequant_pair<false>(w1, sb), dequant_pair<true>(w1, sb)};
            if constexpr (EDGE) {
              const uint32_t fill = lost ? 0x7FC07FC0u : 0u;
              if (lost || tile * KT + r >= len) o = v4u{fill, fill, fill, fill};
            }
            *reinterpret_cast<v4u*>(&to[i][r * D * 2 + (swizzled<D>(c * 2 + (h ^ turned), r) << 4)]) = o;
          }
        }
      }
    };
    auto convert = [&](uint32_t tile, uint8_t (&to)[KV][TB]) {
      if (tile >= last) return;
      if (lost || (tile + 1) * KT > len) convert_rows(std::true_type{}, tile, to);
      else convert_rows(std::false_type{}, tile, to);
    };
    // The wave's BF16 rows, which are there: those past the end to zeros, those of a lost page to NaN.
    auto mend = [&](uint32_t tile, uint8_t (&at)[KV][TB]) {
      if (!lost && (tile + 1) * KT <= len) return;
      const uint32_t lane = hidden();
#pragma unroll
      for (int x = 0; x < NI; ++x) {
        const uint32_t r0 = wave * RW + x * RPI;
        const uint32_t fill = lost ? 0x7FC07FC0u : 0u;
#pragma unroll
        for (int i = 0; i < KV; ++i)
          if (lost || tile * KT + r0 + lane / CPR >= len) *reinterpret_cast<v4u*>(&at[i][r0 * D * 2 + lane * 16]) = v4u{fill, fill, fill, fill};
      }
    };
    // What this wave asked for is there.
    auto landed = [&]() {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(wait_vm(0));
      asm volatile("" ::: "memory");
    };
    auto step = [&](auto RAGGED, uint32_t tile, uint8_t (&now)[KV][TB], uint8_t (&next)[KV][TB]) {
      landed();
      lost = lost_next;
      find_page(tile + (FP8 ? 2 : 1));
      if constexpr (!FP8) mend(tile, now);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(kWaitLgkmOnly);
      asm volatile("s_barrier" ::: "memory");           // the tile is whole; everyone has read `next`
      if constexpr (FP8) {
        convert(tile + 1, next);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(kWaitLgkmOnly);      // the codes are read, their place is free
      }
      load(tile + (FP8 ? 2 : 1), next);
      if (!active) return;
      typename Tile::Scores s;
      typename Tile::Weights p;
      w.scores(now[0], s);
      if constexpr (RAGGED) w.mask(s, static_cast<int32_t>(len - tile * KT));
      w.weights(s, a.scale, p);
      w.values(now[KV - 1], p);
    };

    uint32_t tile = pc.tile0;
    __syncthreads();                                    // the last piece's tiles have been read
    find_page(tile);
    load(tile, buf0);
    if constexpr (FP8) {
      find_page(tile + 1);
      landed();
      lost = lost_next;
      convert(tile, buf0);
      __builtin_amdgcn_s_waitcnt(kWaitLgkmOnly);
      load(tile + 1, buf1);
    }
    // Whole tiles two to a turn of the loop, so that each buffer is an object of its own; then what is left, an odd one and
    // the one with the end.
    const uint32_t pairs = pc.tile0 + ((last - (last * KT > len ? 1 : 0) - pc.tile0) & ~1u);
    for (; tile < pairs; tile += 2) {
      step(std::false_type{}, tile, buf0, buf1);
      step(std::false_type{}, tile + 1, buf1, buf0);
    }
#pragma unroll 1
    for (; tile < last; ++tile) {
      const bool second = ((tile - pc.tile0) & 1) != 0;
      step(std::true_type{}, tile, second ? buf1 : buf0, second ? buf0 : buf1);
    }

    float l = w.sum();
    if (bad) l = __builtin_nanf("");
    if (active && r < pc.heads) {
      if (pc.tiles == pc.of) {
        const float inv = 1.0f / l;
        uint16_t* row = a.out + (static_cast<size_t>(sh.b) * a.H + pc.h0 + r) * D;
#pragma unroll
        for (int x = 0; x < Tile::QUADS; ++x) {
          int d;
          const float4 o = w.quad(x, d);
          *reinterpret_cast<uint2*>(row + d) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        }
      } else {
        float* part = part_of(a, sh.group, sh.block, pc.tile0 == 0, ROWS * (D + 2));
#pragma unroll
        for (int x = 0; x < Tile::QUADS; ++x) {
          int d;
          const float4 o = w.quad(x, d);
          *reinterpret_cast<float4*>(part + r * D + d) = o;
        }
        if (Tile::first_lane()) {
          part[ROWS * D + r] = w.m;
          part[ROWS * D + ROWS + r] = l;
        }
      }
    }
    advance(a, sh, pc);
  }
}

uint32_t head_blocks_of(int32_t G, int32_t D) { return static_cast<uint32_t>((G + rows_of(D) - 1) / rows_of(D)); }

// Groups: as many as run at once, and no more than there can be tiles.
uint32_t groups_of(int64_t B, int32_t Hkv, uint32_t head_blocks, int32_t D, int64_t max_tokens) {
  const int64_t kt = D <= 128 ? 64 : 32;
  return decode_groups(B * Hkv * ((max_tokens + kt - 1) / kt), (D >= 512 ? 256 : 512) / head_blocks);
}

template <int D, bool FP8>
void launch(const DecodeArgs& a, hipStream_t stream) {
  const dim3 grid(a.groups * a.head_blocks), block(threads_of(D));
  if (D >= 512 || (a.c.k == a.c.v && a.c.ks == a.c.vs)) {
    hipLaunchKernelGGL((attn_decode_rows_kernel<D, FP8, true>), grid, block, 0, stream, a);
  } else if constexpr (D < 512) {
    hipLaunchKernelGGL((attn_decode_rows_kernel<D, FP8, false>), grid, block, 0, stream, a);
  }
  hipLaunchKernelGGL((attn_join_kernel<D, key_tile<D>(), rows_of(D)>), dim3(a.B * a.H), dim3(kJoinThreads), 0, stream, a);
}

}  // namespace

// From 32 heads on the rows fill at least one wave's products, and the cache is read once, not once for each 16 heads.
// Rows of 512 have no room in LDS for values of their own.
bool decode_by_rows(int32_t G, int32_t D, bool latent) { return G >= 32 && (D < 512 || latent); }

size_t decode_rows_part_bytes(int64_t B, int32_t H, int32_t Hkv, int32_t D, int64_t max_tokens) {
  const int32_t G = H / Hkv;
  if (!decode_by_rows(G, D, true)) return 0;
  const uint32_t blocks = head_blocks_of(G, D);
  return static_cast<size_t>(groups_of(B, Hkv, blocks, D, max_tokens)) * blocks * 2 * rows_of(D) * (D + 2) * 4;
}

void launch_decode_rows(DecodeArgs a, int32_t D, bool fp8, int64_t max_tokens, hipStream_t stream) {
  a.head_blocks = head_blocks_of(static_cast<int32_t>(a.G), D);
  a.groups = groups_of(a.B, static_cast<int32_t>(a.c.Hkv), a.head_blocks, D, max_tokens);
  switch (D) {
    case 64: fp8 ? launch<64, true>(a, stream) : launch<64, false>(a, stream); break;
    case 128: fp8 ? launch<128, true>(a, stream) : launch<128, false>(a, stream); break;
    case 256: fp8 ? launch<256, true>(a, stream) : launch<256, false>(a, stream); break;
    default: fp8 ? launch<512, true>(a, stream) : launch<512, false>(a, stream); break;
  }
}

}  // namespace mx
