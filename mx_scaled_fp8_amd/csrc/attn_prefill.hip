// Causal attention over packed prompts (gfx950).
//
// The query rows of a prompt and head are its tokens; in prompts of few tokens, the tokens' `pack` heads that share a key
// head: row f is head f % pack of token f / pack, so that they read the keys once and fill a row tile.  A workgroup
// takes 128 rows (64 in rows of 512 that are keys and values), 32 or 16 for each wave (attn_tile.hpp), and runs over the
// keys in tiles of KT.  K and V tiles go from global memory to LDS by buffer-load DMA, the next one while this one is
// used; rows past the end are zeros by the buffer's bound.  Tiles that every row sees whole run first, two to a turn of
// the loop, so that each of the two buffers is an object of its own and the compiler waits for no DMA but what a read
// needs; the last few, which hold the diagonal and the ragged end, go through a loop with masks.
//
// Few row tiles with many keys are split along the keys over `splits` workgroups, whose parts (O, m, l) a second
// kernel joins.
//
// What bounds it is the matrix cores and, beside them, the issue of what the softmax needs: of 8192 tokens, 32 heads of 128, the
// products alone take 357 us at the clock that the power allows, the kernel 505 to 540 (1.02 to 1.09 PFLOP/s; a library product
// of 8192^3 reaches 1.2 to 1.45).  P is rounded to BF16 for the second product; m, the sum of the unrounded P, S and O
// are FP32, parts too.
#include <algorithm>

#include "attn_tile.hpp"

namespace mx {

namespace {

// Fewest keys of a split, of an average prompt and of any row tile: its parts, O in FP32, are written and read again.  (Us of 256,
// 512 and 1024: 64 rows over 8000 tokens, 16 heads of 512 on one 119, 78 and 73; 4 prompts of 17 rows over 3972, 6 heads of 128 on
// each of 4 31, 26 and 36; 200 rows over 3000, 4 heads of 128 on each of 2 28, 26 and 31.  Of a row tile alone, 256 and 512: 8192 rows,
// 2 heads of 512 on one 252 and 231; 2 prompts of 2000, 4 heads of 256 on each of 2 68 and 62; 4096 rows, 8 heads of 256 on one 115
// and 120.)
constexpr int kMinKeys = 512;

struct PrefillArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* q_offsets;
  const int32_t* k_offsets;
  uint16_t* out;
  float* parts;              // [row tile, pack of heads, split][O: rows x D, m, l: a row each], FP32
  float scale;               // times log2(e)
  uint32_t B, Tq, Tk, H, Hkv;
  uint32_t pack, packs;      // heads of a row tile; packs of a key head
  uint32_t tiles;            // bound on the row tiles of all prompts
  uint32_t splits;
};

// Offset b cut to [0, T].
__device__ __forceinline__ uint32_t cut(const int32_t* offsets, uint32_t b, uint32_t T) {
  return min(static_cast<uint32_t>(max(offsets[b], 0)), T);
}

// A row tile: its prompt's rows and keys, and which of them it has.
struct RowTile {
  uint32_t q0, k0;           // where the prompt's rows and keys begin
  int32_t Lq, Lk;            // tokens, keys
  int32_t rows;              // Lq * pack
  int32_t first;             // row of the prompt
  int32_t keys;              // keys that some row of the tile sees
  bool any;                  // the tile has rows
};

// Keys that row f of the prompt, or its last row, sees.
__device__ __forceinline__ int32_t keys_of(const PrefillArgs& a, const RowTile& t, int32_t f) {
  return max(t.Lk - t.Lq + min(static_cast<int32_t>(static_cast<uint32_t>(f) / a.pack), t.Lq - 1) + 1, 0);
}

template <int ROWS>
__device__ __forceinline__ RowTile row_tile(const PrefillArgs& a, uint32_t rt) {
  // prompt b's row tiles are numbered from offsets[b] * pack / ROWS + b, which leaves room for every ragged end
  uint32_t lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (cut(a.q_offsets, mid, a.Tq) * a.pack / ROWS + mid <= rt) lo = mid; else hi = mid;
  }
  RowTile t;
  t.q0 = cut(a.q_offsets, lo, a.Tq);
  t.k0 = cut(a.k_offsets, lo, a.Tk);
  const uint32_t q1 = cut(a.q_offsets, lo + 1, a.Tq), k1 = cut(a.k_offsets, lo + 1, a.Tk);
  t.Lq = q1 > t.q0 ? static_cast<int32_t>(q1 - t.q0) : 0;
  t.Lk = k1 > t.k0 ? static_cast<int32_t>(k1 - t.k0) : 0;
  const uint32_t first = (rt - (t.q0 * a.pack / ROWS + lo)) * ROWS;
  t.rows = t.Lq * static_cast<int32_t>(a.pack);
  t.any = first < static_cast<uint32_t>(t.rows);
  t.first = static_cast<int32_t>(first);
  t.keys = t.any ? keys_of(a, t, t.first + ROWS - 1) : 0;
  return t;
}

// Splits that a row tile with so many keys is really cut into, and the tiles of each.
template <int D>
__device__ __forceinline__ uint32_t split_tiles(int32_t keys, uint32_t splits, uint32_t& used) {
  const uint32_t n = (static_cast<uint32_t>(keys) + key_tile<D>() - 1) / key_tile<D>();
  const uint32_t per = max((n + splits - 1) / splits, static_cast<uint32_t>(kMinKeys / key_tile<D>()));
  used = max((n + per - 1) / per, 1u);
  return per;
}

// Query rows of a workgroup.  Four waves are half of what a compute unit runs: two workgroups, which know nothing of each
// other's barriers, fill it.  (Rows of 512 whose K and V both need LDS: one of eight waves.)
template <int D, bool SAME>
constexpr int rows_of() { return D >= 512 && SAME ? 64 : 128; }
template <int D, bool SAME>
constexpr int threads_of() { return rows_of<D, SAME>() / TileOf<D>::type::ROWS * 64; }

template <int D, bool SAME>
__global__ __launch_bounds__((threads_of<D, SAME>()), 2) void attn_prefill_kernel(PrefillArgs a) {
  using Tile = typename TileOf<D>::type;
  constexpr int ROWS = rows_of<D, SAME>(), WAVES = ROWS / Tile::ROWS, KT = key_tile<D>();
  constexpr int CH = D / 8;                             // 16-byte chunks of a row
  constexpr int TB = KT * D * 2;                        // bytes of a tile
  constexpr int ND = TB / 1024 / WAVES;                 // a wave's DMA instructions for one tile
  __shared__ __attribute__((aligned(1024))) uint8_t kbuf0[TB], kbuf1[TB], vbuf0[SAME ? 16 : TB], vbuf1[SAME ? 16 : TB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // (row tile, split, pack, key head): key heads fastest, so that with workgroups dealt to the XCDs in turn an XCD's L2
  // serves few key heads; last row tiles first, which have the most keys.
  uint32_t id = blockIdx.x;
  const uint32_t kvh = id % a.Hkv;
  id /= a.Hkv;
  const uint32_t head0 = (kvh * a.packs + id % a.packs) * a.pack;   // the first of the pack
  id /= a.packs;
  const uint32_t split = id % a.splits, rt = a.tiles - 1 - id / a.splits;
  const RowTile t = row_tile<ROWS>(a, rt);
  uint32_t used;
  const uint32_t per = split_tiles<D>(t.keys, a.splits, used);
  if (!t.any || split >= used) return;
  // the wave's first row, and the lane's: its number, token, head and the keys that it sees
  const int32_t f0 = t.first + wave * Tile::ROWS;
  struct Row { int32_t f, token; uint32_t head; int32_t sees; };
  auto lane_row = [&](int32_t in_wave) {
    Row r;
    r.f = f0 + in_wave;
    const int32_t at = min(r.f, t.rows - 1);
    r.token = static_cast<int32_t>(static_cast<uint32_t>(at) / a.pack);
    r.head = head0 + (at - r.token * static_cast<int32_t>(a.pack));
    r.sees = keys_of(a, t, at);
    return r;
  };
  const int32_t w_keys = f0 < t.rows ? keys_of(a, t, f0 + Tile::ROWS - 1) : 0;   // that some row of the wave sees
  const int32_t n_tiles = min((t.keys + KT - 1) / KT, static_cast<int32_t>((split + 1) * per));
  const int32_t begin = split * per;
  // whole tiles: those that the workgroup's first row sees whole; an even number of them
  const int32_t whole = max(min(n_tiles, keys_of(a, t, t.first) / KT) - begin, 0) & ~1;

  Tile w;
  w.begin();
  {
    const Row r = lane_row(Tile::row());
    w.load_q(a.q + static_cast<int64_t>(t.q0 + r.token) * a.q_stride + r.head * D);
  }

  // DMA: an instruction fills 1024 bytes of LDS, RPI rows, in lane order.  The swizzle repeats after 16 rows, so that a
  // wave's PAT instructions of one PERIOD of rows serve all of them.
  constexpr int RPI = 512 / D, PERIOD = RPI * WAVES > 16 ? RPI * WAVES : 16, PAT = PERIOD / RPI / WAVES;
  const uint16_t* kbase = a.k + static_cast<int64_t>(t.k0) * a.k_stride + kvh * D;
  const uint16_t* vbase = a.v + static_cast<int64_t>(t.k0) * a.v_stride + kvh * D;
  const uint32_t ks2 = static_cast<uint32_t>(a.k_stride) * 2, vs2 = static_cast<uint32_t>(a.v_stride) * 2;
  uint32_t koff[PAT], voff[PAT];
#pragma unroll
  for (int x = 0; x < PAT; ++x) {
    const uint32_t r = (wave * PAT + x) * RPI + lane / CH, c = swizzled<D>(lane % CH, r);
    koff[x] = r * ks2 + c * 16;
    voff[x] = r * vs2 + c * 16;
  }
  auto dma_rows = [&](int32_t tile, const uint16_t* base, int64_t stride, uint32_t s2, const uint32_t (&off)[PAT], uint8_t* to) {
#pragma unroll
    for (int x = 0; x < ND; ++x) {
      const int32_t r0 = tile * KT + (x / PAT) * PERIOD, rows = min(PERIOD, t.Lk - r0);   // of this period
      const __amdgpu_buffer_rsrc_t from = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint16_t*>(base + r0 * stride), 0, rows > 0 ? (rows - 1) * static_cast<int>(s2) + D * 2 : 0,
          kBufferFlags);
      dma16(from, to + ((x / PAT) * PERIOD + (wave * PAT + x % PAT) * RPI) * D * 2, off[x % PAT]);
    }
  };
  auto dma = [&](int32_t tile, uint8_t* kto, uint8_t* vto) {
    dma_rows(tile, kbase, a.k_stride, ks2, koff, kto);
    if constexpr (!SAME) dma_rows(tile, vbase, a.v_stride, vs2, voff, vto);
  };
  // this wave's part of the tile is in LDS, and after the barrier everyone's; everyone has read the other buffer
  auto turn = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
    asm volatile("s_barrier" ::: "memory");
  };
  auto step = [&](int32_t tile, const uint8_t* kt, const uint8_t* vt, uint8_t* knext, uint8_t* vnext) {
    turn();
    if (tile + 1 < n_tiles) dma(tile + 1, knext, vnext);
    typename Tile::Scores s;
    typename Tile::Weights p;
    w.scores(kt, s);
    w.weights(s, a.scale, p);
    w.values(SAME ? kt : vt, p);
  };

  int32_t tile = begin;
  if (tile < n_tiles) dma(tile, kbuf0, vbuf0);
  for (; tile < begin + whole; tile += 2) {
    step(tile, kbuf0, vbuf0, kbuf1, vbuf1);
    step(tile + 1, kbuf1, vbuf1, kbuf0, vbuf0);
  }
  // (found again rather than held in registers, of which rows of 512 leave none)
  int32_t in_wave = Tile::row();
  asm volatile("" : "+v"(in_wave));
  const Row row = lane_row(in_wave);
#pragma unroll 1
  for (; tile < n_tiles; ++tile) {
    const bool second = ((tile - begin) & 1) != 0;
    turn();
    if (tile + 1 < n_tiles) dma(tile + 1, second ? kbuf0 : kbuf1, second ? vbuf0 : vbuf1);
    const int32_t t0 = tile * KT;
    if (t0 >= w_keys) continue;
    const uint8_t* kt = second ? kbuf1 : kbuf0;
    const uint8_t* vt = SAME ? kt : second ? vbuf1 : vbuf0;
    const int32_t seen = row.sees - t0;                     // of the tile
    typename Tile::Scores s;
    typename Tile::Weights p;
    w.scores(kt, s);
    w.mask(s, seen);
    w.weights(s, a.scale, p);
    w.values_masked(vt, p, seen);
  }

  const float l = w.sum();
  if (used > 1) {
    const size_t unit = static_cast<size_t>(rt) * (a.H / a.pack) + head0 / a.pack;
    float* part = a.parts + (unit * a.splits + split) * ROWS * (D + 2);
    const int r = wave * Tile::ROWS + in_wave;
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
    return;
  }
  if (row.f >= t.rows) return;
  const float inv = row.sees > 0 ? 1.0f / l : 0.0f;
  uint16_t* to = a.out + (static_cast<int64_t>(t.q0 + row.token) * a.H + row.head) * D;
#pragma unroll
  for (int x = 0; x < Tile::QUADS; ++x) {
    int d;
    const float4 o = w.quad(x, d);
    *reinterpret_cast<uint2*>(to + d) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
}

// A workgroup takes kJoinRows rows of a row tile and pack: the splits' parts joined in their order.
constexpr int kJoinRows = 16, kJoinThreads = 256;
template <int D, int ROWS>
__global__ __launch_bounds__(kJoinThreads) void attn_prefill_join_kernel(PrefillArgs a) {
  uint32_t id = blockIdx.x;
  const uint32_t r0 = id % (ROWS / kJoinRows) * kJoinRows;
  id /= ROWS / kJoinRows;
  const uint32_t heads = a.H / a.pack, pack = id % heads, rt = id / heads;
  const RowTile t = row_tile<ROWS>(a, rt);
  uint32_t used;
  split_tiles<D>(t.keys, a.splits, used);
  if (!t.any || used == 1) return;
  const float* parts = a.parts + (static_cast<size_t>(rt) * heads + pack) * a.splits * ROWS * (D + 2);
  for (uint32_t e = threadIdx.x * 4; e < kJoinRows * D; e += kJoinThreads * 4) {
    const uint32_t r = r0 + e / D, d = e % D;
    const int32_t f = t.first + static_cast<int32_t>(r);
    if (f >= t.rows) break;
    const uint32_t i = static_cast<uint32_t>(f) / a.pack, head = pack * a.pack + (f - i * a.pack);
    float m = -INFINITY, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (uint32_t s = 0; s < used; ++s) {
      const float* p = parts + static_cast<size_t>(s) * ROWS * (D + 2);
      const float x = p[ROWS * D + r], top = fmaxf(m, x), base = top == -INFINITY ? 0.0f : top;
      const float f = __builtin_amdgcn_exp2f(m - base), g = __builtin_amdgcn_exp2f(x - base);
      const float4 v = *reinterpret_cast<const float4*>(p + r * D + d);
      l = l * f + p[ROWS * D + ROWS + r] * g;
      o = make_float4(o.x * f + v.x * g, o.y * f + v.y * g, o.z * f + v.z * g, o.w * f + v.w * g);
      m = top;
    }
    const float inv = keys_of(a, t, f) > 0 ? 1.0f / l : 0.0f;
    *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(t.q0 + i) * a.H + head) * D + d) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
}

bool same(const void* k, int64_t k_stride, const void* v, int64_t v_stride) { return k == v && k_stride == v_stride; }

// Query rows of a workgroup (rows_of, of a call).
int rows_of_call(int32_t D, bool latent) { return D >= 512 && latent ? 64 : 128; }

// Heads of a row tile: those that share a key head where an average prompt has fewer tokens than a row tile has rows.  (7
// rows of 4 prompts over 30000 tokens, 4 heads a key head: 142 us with, 268 without.  With full row tiles of their own the
// heads are as fast unpacked: 8192 rows 534 us packed, 529 not.)
int32_t pack_of(int64_t B, int64_t Tq, int32_t H, int32_t Hkv, int rows) { return Tq / B < rows ? H / Hkv : 1; }

// Bound on the row tiles of all prompts.
int64_t row_tiles(int64_t B, int64_t Tq, int32_t pack, int rows) { return Tq * pack / rows + B; }

// How many workgroups share the keys of one row tile and pack.  512 run at once; up to twice as many, as long as every part
// has some keys, keep them busy and let those that run together read the same keys.  `units` goes by the bound of row tiles, which
// for one prompt of whole row tiles is one more than there are: 4096 rows are 33, and 8 heads of them 3 splits, not 4.  (3 and 4
// splits: 4096 rows over 30011 earlier tokens, 8 heads of 128 520 us and 512, 2048 over 98,000 830 and 780; prompts from their
// beginning, whose first rows have few keys to split, 8192 rows, 4 heads of 128 90 and 93, 4096 rows, 8 heads of 256 115 and 130,
// 2048 rows, 16 heads of 512 89 and 118.)
uint32_t split_count(int64_t B, int64_t Tk, int64_t units) {
  return static_cast<uint32_t>(std::max<int64_t>(1, std::min(1024 / units, (Tk / B + 63) / kMinKeys)));   // (tiles of 64)
}

// (row tile, pack) pairs.
int64_t units_of(int64_t B, int64_t Tq, int32_t H, int32_t Hkv, int rows) {
  const int32_t pack = pack_of(B, Tq, H, Hkv, rows);
  return row_tiles(B, Tq, pack, rows) * (H / pack);
}

size_t part_bytes(int64_t B, int64_t Tq, int64_t Tk, int32_t H, int32_t Hkv, int32_t D, int rows) {
  const size_t units = units_of(B, Tq, H, Hkv, rows), splits = split_count(B, Tk, units);
  return splits == 1 ? 0 : splits * units * rows * (D + 2) * 4;
}

template <int D, bool SAME>
void launch(const PrefillArgs& a, hipStream_t stream) {
  constexpr int ROWS = rows_of<D, SAME>();
  const uint32_t units = a.tiles * (a.H / a.pack);
  hipLaunchKernelGGL((attn_prefill_kernel<D, SAME>), dim3(units * a.splits), dim3(threads_of<D, SAME>()), 0, stream, a);
  if (a.splits > 1)
    hipLaunchKernelGGL((attn_prefill_join_kernel<D, ROWS>), dim3(units * (ROWS / kJoinRows)), dim3(kJoinThreads), 0, stream, a);
}

template <int D>
void launch(const PrefillArgs& a, bool latent, hipStream_t stream) {
  if (latent) launch<D, true>(a, stream);
  else launch<D, false>(a, stream);
}

}  // namespace

// Of either kind of call: the sizes do not say whether v is k.
size_t prefill_workspace_bytes(int64_t B, int64_t Tq, int64_t Tk, int32_t H, int32_t Hkv, int32_t D) {
  return std::max(part_bytes(B, Tq, Tk, H, Hkv, D, rows_of_call(D, false)),
                  part_bytes(B, Tq, Tk, H, Hkv, D, rows_of_call(D, true)));
}

mx_status launch_attn_prefill(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, const int32_t* q_offsets, const int32_t* k_offsets, int64_t B,
                              int64_t Tq, int64_t Tk, int32_t H, int32_t Hkv, int32_t D, float scale, void* out,
                              void* workspace, hipStream_t stream) {
  const bool latent = same(k, k_stride, v, v_stride);
  const int rows = rows_of_call(D, latent);
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
  a.parts = static_cast<float*>(workspace);
  a.scale = scale * kLog2E;
  a.B = static_cast<uint32_t>(B);
  a.Tq = static_cast<uint32_t>(Tq);
  a.Tk = static_cast<uint32_t>(Tk);
  a.H = static_cast<uint32_t>(H);
  a.Hkv = static_cast<uint32_t>(Hkv);
  a.pack = static_cast<uint32_t>(pack_of(B, Tq, H, Hkv, rows));
  a.packs = a.H / a.Hkv / a.pack;
  a.tiles = static_cast<uint32_t>(row_tiles(B, Tq, static_cast<int32_t>(a.pack), rows));
  a.splits = split_count(B, Tk, units_of(B, Tq, H, Hkv, rows));
  switch (D) {
    case 64: launch<64>(a, latent, stream); break;
    case 128: launch<128>(a, latent, stream); break;
    case 256: launch<256>(a, latent, stream); break;
    default: launch<512>(a, latent, stream); break;
  }
  return launch_status("mx_attn_prefill");
}

}  // namespace mx
