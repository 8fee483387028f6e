// Attention of one new token where many query heads share a key head (gfx950): a latent cache above all.
//
// With 128 heads over a key of 512 elements a token costs 2^18 operations for 528 bytes: the matrix cores bound it, not the
// cache.  So the heads are the rows of attn_tile.hpp's products, 128 to a workgroup, and a tile of keys is brought to LDS
// once for all of them.  BF16 rows come by DMA as in the prompt attention.  MXFP8 codes come by DMA into a place of their own
// a turn ahead, where the wave that asked for them makes BF16 of them (exact) under the other waves' products and writes
// it to the buffer that the last turn read; registers hold O and Q and have no room for codes under way.  Latent rows of 512,
// the widest, multiply with the codes themselves where they are keys (CodesTile).
// Work is shared as attn_plan.hpp says.
//
// (MI355X, 128 heads, 64 sequences of up to 32,768 tokens, 512 wide, MXFP8: 320 us and 17 for the join, 0.84 PFLOP/s; up to 8192
// tokens in BF16 125 to 136 us.  A turn of 32 tokens is 4700 cycles, of them 2050 of the matrix cores; timing copies: without the
// products with V 95 us less, without S 80, the conversion 30 to 37, DMA 27 to 40, softmax 8 to 22.  The rest is waiting:
// registers for two waves a SIMD only, and operands that are read no further ahead than registers reach.)
#include <type_traits>
#include <utility>

#include "attn_decode.hpp"
#include "attn_tile.hpp"

namespace mx {

namespace {

// Of a share: its part is up to 128 rows of FP32, as much as 500 cached tokens.  (Us of 64, 128 and 256: one sequence of 1000
// tokens, 128 heads of 512 27, 28 and 35, of 6566 42, 38 and 40; 4 of 2000, 64 heads of 256 21, 23 and 29; 2 of 30,000, 32 heads of
// 128 22.5, 22.7 and 21.)
constexpr int kMinTokens = 128;

// Query heads of a workgroup: 32 for each of four waves, half of what a compute unit runs, so that two workgroups, which know
// nothing of each other's barriers, fill it; in rows of 512, 16 for each of eight, so that codes are converted once for all 128
// (405 us with 64 to a workgroup, 376 with 128).
constexpr int rows_of(int) { return 128; }
constexpr int threads_of(int D) { return D >= 512 ? 512 : 256; }

typedef int v8i __attribute__((ext_vector_type(8)));

// Rows of 512 over MXFP8 codes: S comes from the codes themselves, by v_mfma_scale_f32_16x16x128_f8f6f4 with their block
// scales, and from Q as the sum of two MXFP8 numbers.  A BF16 number has 8 significant bits, an e4m3 code 4: with e the
// scale of the block, hi = e4m3(q 2^-e) leaves at most 8 steps of q's last bit, which lo = e4m3((q - hi 2^e) 2^(4-e)) holds.
// So Q is exact but for elements below 2^-14 of their block's largest, which are off by up to 2^-21 of that: what a sum of
// FP32 products over the block loses too.  The two products take the time of one in BF16, but K is half as many bytes to read
// from LDS, and its reads need not wait for the conversion, which only V's do.  (64 sequences up to 32,768 tokens, 128 heads: 376
// us by the BF16 copy, 338 so.)
struct CodesTile : AttnTile16<512, 32, 3> {
  static constexpr int D = 512, J = D / 128;
  // Operands of K and V under way (us: 1 and 4 365, 2 and 4 363, 2 and 5 348, 2 and 6, which spills in the loop, 354).
  static constexpr int KN = 2, VN = 5;
  v8i hi[J], lo[J];
  uint32_t qs, cbase, sbase;                            // qs: byte j is the scale byte of block 4 j + g of the lane's row

  // The operand layout: lane row + 16 g holds bytes 16 g .. + 15 and 64 + 16 g .. + 15 of 128, and the scale of block g of
  // 32 (the layout that linear_mx32.hip found).  In LDS, chunk c of row r of the codes is at c ^ r % 16.
  __device__ __forceinline__ void begin() {
    uint32_t lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));                      // found again for each piece: no registers for what never changes
    AttnTile16::begin(lane);
    const uint32_t r = lane & 15;
    cbase = r * D + ((static_cast<uint32_t>(g) ^ r) << 4);
    sbase = r * (D / 32) + g * 4;
  }

  // Of the two BF16 numbers in w: what hi is made of.  Above 240 2^120 the nearest code is 2^128, which has no remainder in FP32; 240
  // leaves up to 15 2^120, which lo holds.
  __device__ __forceinline__ static uint32_t below_top(uint32_t w) {
    typedef uint16_t v2u16 __attribute__((ext_vector_type(2)));
    const v2u16 size = __builtin_elementwise_min(__builtin_bit_cast(v2u16, w & 0x7FFF7FFFu), (v2u16{0x7F70, 0x7F70}));
    return __builtin_bit_cast(uint32_t, size) | (w & 0x80008000u);
  }

  __device__ __forceinline__ void load_q(const uint16_t* q) {
    uint32_t lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const uint32_t g = lane >> 4;
    qs = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      uint32_t bytes = 0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint4* at = reinterpret_cast<const uint4*>(q + j * 128 + half * 64 + g * 16);
        const uint4 a = at[0], b = at[1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));   // the block's other half
        const bool finite = top < 0x7F80u;
        const int e = max(e8m0_exponent<8>(finite ? top : 0), -123);
        const float se = __uint_as_float(static_cast<uint32_t>(e + 127) << 23), sl = __uint_as_float(static_cast<uint32_t>(e + 123) << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          typedef short v2s __attribute__((ext_vector_type(2)));
          typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
          v2s h = {0, 0}, l = {0, 0};
          uint32_t back[2], rest[2];
          h = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(h, __builtin_bit_cast(v2bf, below_top(w[2 * i])), se, false);
          h = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(h, __builtin_bit_cast(v2bf, below_top(w[2 * i + 1])), se, true);
          back[0] = dequant_pair<false>(__builtin_bit_cast(uint32_t, h), se);
          back[1] = dequant_pair<true>(__builtin_bit_cast(uint32_t, h), se);
#pragma unroll
          for (int k = 0; k < 2; ++k)                   // exact, in FP32 and in BF16
            rest[k] = pack_bf16x2(__uint_as_float(w[2 * i + k] << 16) - __uint_as_float(back[k] << 16),
                                  __uint_as_float(w[2 * i + k] & 0xFFFF0000u) - __uint_as_float(back[k] & 0xFFFF0000u));
          l = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(l, __builtin_bit_cast(v2bf, rest[0]), sl, false);
          l = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(l, __builtin_bit_cast(v2bf, rest[1]), sl, true);
          hi[j][half * 4 + i] = __builtin_bit_cast(int, h);
          lo[j][half * 4 + i] = __builtin_bit_cast(int, l);
        }
        bytes |= (finite ? static_cast<uint32_t>(e + 127) : 0xFFu) << (8 * half);
      }
      // blocks 0, 1 are the first halves of lanes g 0 and 2, blocks 2, 3 their second
      bytes = static_cast<uint32_t>(__shfl(static_cast<int>(bytes), (lane & 15) + 32 * (g & 1)));
      qs |= (bytes >> (8 * (g >> 1)) & 0xFFu) << (8 * j);
    }
  }

  __device__ __forceinline__ v8i codes_of(const uint8_t* codes, int j, int u) const {
    const uint8_t* row = codes + u * 16 * D + (j / 2) * 256;
    const v4u a = *reinterpret_cast<const v4u*>(row + (cbase ^ ((j % 2 * 8) << 4)));
    const v4u b = *reinterpret_cast<const v4u*>(row + (cbase ^ ((j % 2 * 8 + 4) << 4)));
    return v8i{static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]), static_cast<int>(a[3]),
               static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]), static_cast<int>(b[3])};
  }

  template <int N>
  __device__ __forceinline__ void products(const v8i& k, uint32_t ks, uint32_t qlo, Scores& x) {
    x.s[N % 2] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, hi[N / 2], x.s[N % 2], 0, 0, N / 2, ks, N / 2, qs);
    x.s[N % 2] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, lo[N / 2], x.s[N % 2], 0, 0, N / 2, ks, N / 2, qlo);
  }

  // Of the codes of a tile and their scale bytes, [row][g][j].  Eight times two products; the codes are read KN times
  // ahead, and between() is other work to do under the n-th products.
  template <class F>
  __device__ __forceinline__ void scores(const uint8_t* codes, const uint8_t* scales, Scores& x, F between) {
    asm volatile("" : "+v"(cbase), "+v"(sbase), "+v"(kbase), "+v"(vbase));
    x.s[0] = x.s[1] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t qlo = qs - 0x04040404u;              // no byte is below 4; of a NaN block, one NaN is enough
    const uint32_t ks[2] = {*reinterpret_cast<const uint32_t*>(scales + sbase),
                            *reinterpret_cast<const uint32_t*>(scales + sbase + 16 * (D / 32))};
    v8i k[KN + 1];
#pragma unroll
    for (int n = 0; n < KN; ++n) k[n] = codes_of(codes, n / 2, n % 2);
    each(std::make_integer_sequence<int, 8>{}, [&](auto N) {
      constexpr int n = N;
      if constexpr (n + KN < 8) k[(n + KN) % (KN + 1)] = codes_of(codes, (n + KN) / 2, (n + KN) % 2);
      between(N);
      products<n>(k[n % (KN + 1)], ks[n % 2], qlo, x);
      __builtin_amdgcn_sched_barrier(0);
    });
  }

  // O += P V, V's operands read VN products ahead; between() as above.
  template <class F>
  __device__ __forceinline__ void values(const uint8_t* vt, const Weights& y, F between) {
    v4u f[VN];
#pragma unroll
    for (int d = 0; d < VN; ++d) f[d] = v_operand(vt, d);
    __builtin_amdgcn_sched_barrier(0);
    each(std::make_integer_sequence<int, DT>{}, [&](auto N) {
      constexpr int d = N;
      acc[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, f[d % VN]), y.p, acc[d], 0, 0, 0);
      if constexpr (d + VN < DT) f[d % VN] = v_operand(vt, d + VN);
      between(N);
      __builtin_amdgcn_sched_barrier(0);
    });
  }

  template <int... N, class F>
  __device__ __forceinline__ static void each(std::integer_sequence<int, N...>, F f) {
    (f(std::integral_constant<int, N>{}), ...);
  }
};

template <int D, bool FP8, bool SAME>
__global__ __launch_bounds__(threads_of(D), 2) void attn_decode_rows_kernel(DecodeArgs a) {
  constexpr bool CODES = FP8 && D == 512;               // S by the codes themselves
  using Tile = std::conditional_t<CODES, CodesTile, typename TileOf<D, 4>::type>;   // (6 ahead: no registers, and the
                                                                                    // compiler reads none ahead)
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
  // Codes that S reads stay until all waves have read them, those of the next tile are converted meanwhile, and those of the
  // one after it are on their way: three places in turn.
  constexpr int MORE = CODES ? TB : 16, SCALES = CODES ? KT * SB : 16;
  __shared__ __attribute__((aligned(1024))) uint8_t buf0[KV][TB], buf1[KV][TB], buf2[KV][MORE], raw0[KV][RAW], raw1[CODES ? KV : 1][RAW],
      raw2[CODES ? KV : 1][RAW], scales0[SCALES], scales1[SCALES], scales2[SCALES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  auto lane_row = [&]() {                               // of the workgroup's rows; found where it is used
    uint32_t x = Tile::row();
    if constexpr (D >= 512) asm volatile("" : "+v"(x));
    return wave * Tile::ROWS + x;
  };

  Share sh = find_share<KT, kMinTokens / KT>(a);
  while (sh.t < sh.end) {
    const Piece pc = piece_of<KT, ROWS>(a, sh);
    const uint32_t len = tokens_of(a, sh.b);
    const bool bad = a.lens[sh.b] > static_cast<int32_t>(len);   // longer than its table
    const int32_t* table = a.c.table + static_cast<int64_t>(sh.b) * a.c.max_pages;
    const bool active = static_cast<uint32_t>(wave * Tile::ROWS) < pc.heads;   // the wave has heads

    Tile w;
    w.begin();

    // A wave brings rows wave * RW .. of a tile.  Rows of a page outside the cache are read from page 0 and made NaN
    // (`lost`); rows past the end are zeros.
    const uint32_t last = pc.tile0 + pc.tiles;
    uint32_t page = 0, scale[KV];                         // scale: the rows' scale bytes, four a lane
    bool lost = false, lost_next = false;
    auto first_token = [&](uint32_t tile) { return tile * KT + static_cast<uint32_t>(wave) * RW; };
    // The page's number by a scalar load (nothing writes the table meanwhile), which holds no vector register and does not
    // wait behind the DMA; past the end, the last token's page again.
    const auto* numbers = (const __attribute__((address_space(4))) int32_t*)table;
    // The lane's number as the compiler cannot see through: addresses are formed where they are used, and not held in
    // registers that a wide row needs.
    auto hidden = [&]() {
      uint32_t x = lane;
      if constexpr (D >= 256) asm volatile("" : "+v"(x));
      return x;
    };
    // The codes of CODES: a lane's place in the cache among the wave's first two rows, and its place in the tile, where its
    // first eight elements go, or its second, as write_half() has it.  For the next two rows both differ by what is added below.
    const uint32_t lane0 = hidden(), row0 = wave * RW + lane0 / 32, chunk0 = lane0 % 32 ^ (row0 & 15);
    uint32_t chunk = lane0 / 32 * 512 + chunk0 * 16;
    uint32_t put = row0 * D * 2 + (swizzled<D>(chunk0 * 2 + (chunk0 >> 3 & 1), row0) << 4);
    auto hide_places = [&]() {                          // as hidden() does
      if constexpr (CODES) asm volatile("" : "+v"(chunk), "+v"(put));
    };
    auto find_page = [&](uint32_t tile) {
      page = static_cast<uint32_t>(numbers[__builtin_amdgcn_readfirstlane(min(first_token(tile), len - 1) >> a.c.page_shift)]);
    };
    auto load_rows = [&](uint32_t tile, uint8_t (&to)[KV][TB], uint8_t (*raw)[RAW]) {
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
          if constexpr (CODES) {
            const uint32_t at = (chunk ^ (x << 5)) + x * 1024;          // row + 2 x: two bits of the row's number
            dma16_at(from + at, &raw[i][r0 * D]);
          } else if constexpr (FP8) dma16_at(from + x * 1024 + lane * 16, &raw[i][r0 * D]);
          else dma16_at(from + x * 1024 + lane / CPR * (D * 2) + (swizzled<D>(lane % CPR, r0 + lane / CPR) << 4), &to[i][r0 * D * 2]);
        }
        if constexpr (FP8)
          scale[i] = *reinterpret_cast<const uint32_t*>((i == 0 ? a.c.ks : a.c.vs) + row * SB + lane * 4 % (RW * SB));
      }
    };
    auto load = [&](uint32_t tile, uint8_t (&to)[KV][TB], uint8_t (*raw)[RAW]) {
      if (tile < last) load_rows(tile, to, raw);
    };
    // The wave's codes, which are there, to BF16.  One DMA instruction's codes of cache i, and their scales:
    auto read_codes = [&](uint32_t lane, int i, int x, const uint8_t (*raw)[RAW], uint32_t scale, v4u& v, uint32_t& sc) {
      if constexpr (CODES) {
        v = *reinterpret_cast<const v4u*>(&raw[i][(wave * RW + x * RPI) * D + lane * 16]);
        // the scale byte is number chunk / 32 of the first two rows', or its neighbour of the next two
        const uint32_t byte = chunk / 32, word = __builtin_amdgcn_ds_bpermute((byte & ~3u) + x * 2 * SB, scale);
        sc = word >> ((byte & 3) * 8 ^ x << 3) & 0xFFu;
      } else {
        const uint32_t byte = (x * RPI + lane / CPR) * SB + lane % CPR / 2;
        v = *reinterpret_cast<const v4u*>(&raw[i][(wave * RW + x * RPI) * D + lane * 16]);
        sc = __shfl(scale, byte / 4) >> (8 * (byte & 3)) & 0xFFu;
      }
    };
    // Half h of them to the tile.  Half of the lanes write their second eight elements first, so that 16 lanes meet all banks.
    auto write_half = [&](auto EDGE, uint32_t lane, uint32_t tile, int x, int h, const v4u& v, uint32_t sc, uint8_t* to) {
      const uint32_t c = lane % CPR, r = wave * RW + x * RPI + lane / CPR;   // row of the tile
      const uint32_t turned = (CODES ? chunk >> 7 : c >> 3) & 1;
      const float sb = __uint_as_float(sc << 23);
      const uint32_t a0 = v[0], a1 = v[1], b0 = v[2], b1 = v[3], nan = nan_codes(sc);
      const bool second = (turned ^ h) != 0;
      const uint32_t w0 = (second ? b0 : a0) | nan, w1 = (second ? b1 : a1) | nan;
      v4u o = {dequant_pair<false>(w0, sb), dequant_pair<true>(w0, sb), dequant_pair<false>(w1, sb), dequant_pair<true>(w1, sb)};
      if constexpr (EDGE) {
        if (tile * KT + r >= len) o = v4u{0, 0, 0, 0};
      }
      const uint32_t at = CODES ? (put ^ (h << 4)) + x * 2 * D * 2 : r * D * 2 + (swizzled<D>(c * 2 + (h ^ turned), r) << 4);
      *reinterpret_cast<v4u*>(&to[at]) = o;
    };
    auto convert_rows = [&](auto EDGE, uint32_t tile, uint8_t (&to)[KV][TB], const uint8_t (*raw)[RAW], const uint32_t (&scale)[KV]) {
#pragma unroll
      for (int i = 0; i < KV; ++i) {
        const uint32_t lane = hidden();
        v4u v[NI];
        uint32_t sc[NI];
#pragma unroll
        for (int x = 0; x < NI; ++x) read_codes(lane, i, x, raw, scale[i], v[x], sc[x]);
        asm volatile("" ::: "memory");                  // all reads under way before the first is used
#pragma unroll
        for (int x = 0; x < NI; ++x) {
          write_half(EDGE, lane, tile, x, 0, v[x], sc[x], to[i]);
          write_half(EDGE, lane, tile, x, 1, v[x], sc[x], to[i]);
        }
      }
    };
    // Their scale bytes to LDS, [row][g][j]: of the four that a lane has, of blocks 4 j + g.
    auto keep_scales = [&](uint8_t* to, uint32_t bytes) {
      if constexpr (CODES) {
        const uint32_t lane = hidden() % (RW * SB / 4); // (the others have the same)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          to[wave * RW * SB + lane / (SB / 4) * SB + g * (SB / 4) + lane % (SB / 4)] = static_cast<uint8_t>(bytes >> (8 * g));
      }
    };
    auto convert = [&](uint32_t tile, uint8_t (&to)[KV][TB], const uint8_t (*raw)[RAW], const uint32_t (&scale)[KV]) {
      if ((tile + 1) * KT > len) convert_rows(std::true_type{}, tile, to, raw, scale);
      else convert_rows(std::false_type{}, tile, to, raw, scale);
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
    // The next codes are there: those of a lost page are NaN by their scales.
    auto scales_landed = [&]() {
#pragma unroll
      for (int i = 0; i < KV; ++i) scale[i] = lost_next ? 0xFFFFFFFFu : scale[i];
    };
    auto all_here = [&]() {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(kWaitLgkmOnly);
      asm volatile("s_barrier" ::: "memory");           // the tile is whole; everyone has read what comes next's place
    };
    auto step = [&](auto RAGGED, uint32_t tile, uint8_t (&now)[KV][TB], uint8_t (&next)[KV][TB]) {
      landed();
      if constexpr (FP8) scales_landed();
      else lost = lost_next;
      find_page(tile + (FP8 ? 2 : 1));
      if constexpr (!FP8) mend(tile, now);
      all_here();
      if constexpr (FP8) {
        if (tile + 1 < last) convert(tile + 1, next, raw0, scale);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(kWaitLgkmOnly);      // the codes are read, their place is free
      }
      load(tile + (FP8 ? 2 : 1), next, raw0);
      if (!active) return;
      typename Tile::Scores s;
      typename Tile::Weights p;
      if constexpr (!CODES) w.scores(now[0], s);
      if constexpr (RAGGED) w.mask(s, static_cast<int32_t>(len - tile * KT));
      w.weights(s, a.scale, p);
      if constexpr (!CODES) w.values(now[KV - 1], p);
    };
    // In turns.  The codes of the next tile are converted under the products with V.
    auto turn = [&](auto RAGGED, uint32_t tile, uint8_t (&now)[KV][TB], uint8_t (&next)[KV][TB],
                    const uint8_t (*codes)[RAW], const uint8_t (*codes_next)[RAW], uint8_t (*codes_after)[RAW],
                    const uint8_t* scales, uint8_t* scales_next) {
      landed();
      scales_landed();
      const uint32_t sc[KV] = {scale[0]};
      hide_places();
      all_here();
      auto load_after = [&]() {
        load(tile + 2, next, codes_after);
        find_page(tile + 3);                            // a turn ahead: a scalar load is long
      };
      auto convert_next = [&]() {
        if (tile + 1 >= last) return;
        keep_scales(scales_next, sc[0]);
        convert(tile + 1, next, codes_next, sc);
      };
      if (!active) {
        load_after();
        convert_next();
        return;
      }
      typename Tile::Scores s;
      typename Tile::Weights p;
      if constexpr (!CODES) return;
      else if constexpr (RAGGED) {
        load_after();
        convert_next();
        w.scores(codes[0], scales, s, [](auto) {});
        w.mask(s, static_cast<int32_t>(len - tile * KT));
        w.weights(s, a.scale, p);
        w.values(now[0], p, [](auto) {});
      } else {
        w.scores(codes[0], scales, s, [&](auto N) {
          if constexpr (N == 1) {                       // also past the last tile: no harm, and no branch among the products
            load_rows(tile + 2, next, codes_after);
            find_page(tile + 3);
          }
        });
        w.weights(s, a.scale, p);
        v4u v;
        uint32_t vs;
        w.values(now[0], p, [&](auto N) {               // the next tile's conversion, in pieces
          constexpr int n = N;
          static_assert(NI == 2 || !CODES, "two to each");
          if constexpr (n == 0) keep_scales(scales_next, sc[0]);
          if constexpr (n == 1 || n == 13) read_codes(hidden(), 0, n / 13, codes_next, sc[0], v, vs);
          if constexpr (n == 8 || n == 11 || n == 20 || n == 23) write_half(std::false_type{}, 0, tile + 1, n / 13, n % 12 / 11, v, vs, next[0]);
        });
      }
    };

    uint32_t tile = pc.tile0;
    landed();                                           // what the last piece asked for past its end
    __syncthreads();                                    // its tiles have been read
    find_page(tile);
    load(tile, buf0, raw0);
    w.load_q(a.q + static_cast<int64_t>(sh.b) * a.q_stride + (pc.h0 + min(lane_row(), pc.heads - 1)) * D);
    if constexpr (FP8) {
      find_page(tile + 1);
      landed();
      scales_landed();
      if constexpr (CODES) keep_scales(scales0, scale[0]);
      convert(tile, buf0, raw0, scale);
      __builtin_amdgcn_s_waitcnt(kWaitLgkmOnly);
      if constexpr (CODES) load(tile + 1, buf1, raw1);
      else load(tile + 1, buf1, raw0);
      if constexpr (CODES) find_page(tile + 2);
    }
    // Tiles that are whole (and the next one too, with CODES), as many to a turn of the loop as there are places, so that each
    // is an object of its own; then what is left.
    const uint32_t rest = (last * KT > len ? 1 : 0) + (CODES ? 1 : 0);
    const uint32_t whole = pc.tile0 + (pc.tiles > rest ? pc.tiles - rest : 0);
    if constexpr (CODES) {
      while (tile < whole) {
        turn(std::false_type{}, tile, buf0, buf1, raw0, raw1, raw2, scales0, scales1);
        if (++tile == whole) break;
        turn(std::false_type{}, tile, buf1, buf2, raw1, raw2, raw0, scales1, scales2);
        if (++tile == whole) break;
        turn(std::false_type{}, tile, buf2, buf0, raw2, raw0, raw1, scales2, scales0);
        ++tile;
      }
#pragma unroll 1
      for (; tile < last; ++tile) {
        const uint32_t n = (tile - pc.tile0) % 3;
        turn(std::true_type{}, tile, n == 0 ? buf0 : n == 1 ? buf1 : buf2,
             n == 0 ? buf1 : n == 1 ? buf2 : buf0, n == 0 ? raw0 : n == 1 ? raw1 : raw2, n == 0 ? raw1 : n == 1 ? raw2 : raw0,
             n == 0 ? raw2 : n == 1 ? raw0 : raw1, n == 0 ? scales0 : n == 1 ? scales1 : scales2,
             n == 0 ? scales1 : n == 1 ? scales2 : scales0);
      }
    } else {
      for (; tile + 2 <= whole; tile += 2) {
        step(std::false_type{}, tile, buf0, buf1);
        step(std::false_type{}, tile + 1, buf1, buf0);
      }
#pragma unroll 1
      for (; tile < last; ++tile) {
        const bool odd = ((tile - pc.tile0) & 1) != 0;
        step(std::true_type{}, tile, odd ? buf1 : buf0, odd ? buf0 : buf1);
      }
    }

    const uint32_t r = lane_row();
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
        float* part = part_of(a, sh.group, sh.block, pc.tile0 == 0, a.part_heads * (D + 2));
#pragma unroll
        for (int x = 0; x < Tile::QUADS; ++x) {
          int d;
          const float4 o = w.quad(x, d);
          *reinterpret_cast<float4*>(part + r * D + d) = o;
        }
        if (Tile::first_lane()) {
          part[a.part_heads * D + r] = w.m;
          part[a.part_heads * D + a.part_heads + r] = l;
        }
      }
    }
    advance(a, sh, pc);
  }
}

uint32_t head_blocks_of(int32_t G, int32_t D) { return static_cast<uint32_t>((G + rows_of(D) - 1) / rows_of(D)); }

// Heads of a part: a multiple of 4, so that every part is 16-byte aligned.
int32_t part_heads_of(int32_t G, int32_t D) { return std::min((G + 3) / 4 * 4, rows_of(D)); }

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
// Rows of 512 have no room in LDS for values of their own.  A latent BF16 row of 512, read twice by the other kernel, which has no
// registers to read ahead, goes here for any number of heads (64 sequences up to 8192 tokens: one head 55 us here, 64 there, 16 heads
// 62 and 76; 2 up to 2000, 4 heads 15.9 and 15.4, the half microsecond that short calls lose); in MXFP8 one head is 68 and 50, 20
// heads 75 and 96 but over 2 times 2000 tokens 26 and 16.
bool decode_by_rows(int32_t G, int32_t D, bool latent, bool fp8) {
  return D == 512 ? latent && (G >= 32 || !fp8) : G >= 32;
}

size_t decode_rows_part_bytes(int64_t B, int32_t H, int32_t Hkv, int32_t D, int64_t max_tokens) {
  const int32_t G = H / Hkv;
  if (!decode_by_rows(G, D, true, false)) return 0;
  const uint32_t blocks = head_blocks_of(G, D);
  return static_cast<size_t>(groups_of(B, Hkv, blocks, D, max_tokens)) * blocks * 2 * part_heads_of(G, D) * (D + 2) * 4;
}

void launch_decode_rows(DecodeArgs a, int32_t D, bool fp8, int64_t max_tokens, hipStream_t stream) {
  a.head_blocks = head_blocks_of(static_cast<int32_t>(a.G), D);
  a.part_heads = static_cast<uint32_t>(part_heads_of(static_cast<int32_t>(a.G), D));
  a.groups = groups_of(a.B, static_cast<int32_t>(a.c.Hkv), a.head_blocks, D, max_tokens);
  switch (D) {
    case 64: fp8 ? launch<64, true>(a, stream) : launch<64, false>(a, stream); break;
    case 128: fp8 ? launch<128, true>(a, stream) : launch<128, false>(a, stream); break;
    case 256: fp8 ? launch<256, true>(a, stream) : launch<256, false>(a, stream); break;
    default: fp8 ? launch<512, true>(a, stream) : launch<512, false>(a, stream); break;
  }
}

}  // namespace mx
