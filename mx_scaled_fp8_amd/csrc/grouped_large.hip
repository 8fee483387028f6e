// The grouped MXFP8 product's kernel for large groups (gfx950): 256 rows x 256 columns per tile, one resident workgroup
// per compute unit.
//
//   out[r, n] = bf16( sum_k  x[src(r), k] 2^(sx-127) * W[e(r), n, k] 2^(sw-127) ),  E8M0 scales per 32 consecutive K
//
// Four waves of 128 x 128 on v_mfma_scale_f32_32x32x64_f8f6f4, accumulators in AGPRs.  K moves 128 bytes per stage
// through two 64 KiB LDS buffers filled by LDS-DMA; a stage runs in two halves of 64 K,
//   front: MFMAs of half 0 beside the fragment reads of half 1; wait, barrier;
//   back:  MFMAs of half 1 beside the DMA of the stage after next into the buffer just read out (one instruction per
//          MFMA: a burst stalls the wave on the address unit) and the fragment reads of the next stage's half 0,
// and the pipeline runs on through the tile boundaries: the next tile's first two stages and scales are fetched during
// the current tile's last two, and a tile's epilogue is folded into the first half-stage of the next.
//
// What differs from the dense batched GEMM of bmm.hip, whose pipeline this is:
//  * The tiles come from a list in device memory (the groups' sizes are known there alone), walked by expert, then
//    column tile, then row tile: the row tiles that share a weight tile run together on one XCD's L2.
//  * The activation rows of a tile lie anywhere in x: each lane keeps the byte offsets of the 8 rows it fetches.
//    Rows behind the group's last have an offset behind the buffer resource, which fetches nothing.
//  * Any number of stages from kLargeMinStages on.  An odd number gets one more, which fetches nothing (zeros), so that
//    every tile begins in the same buffer.
//  * Four scales per row and stage.  An MFMA half h takes, in lane group q, the byte of block 2 h + q; a 4-byte word
//    holds a block's bytes of the wave's four 32-row tiles, picked by the instruction's byte select.  The words are
//    built four stages (a window) at a time, 8 bytes per row and thread, transposed with v_perm, one window ahead.
//  * K need not be a multiple of 128: the weight's chunks behind K re-read the row's last one, whose products with the
//    activation's zero codes vanish, and scale bytes behind K are cleared.
//
// The 512 registers of a lane do not hold it all: 23 (80 bytes of scratch a lane) are spilled, the row and column limits
// of the epilogue and the addresses of the next tile's fetches among them.  A tile's first and last stages and a change
// of the scale window reload some.  The fold reloads two, right behind the next stage's DMA and after the first stores,
// and each reload waits for that DMA.
//
// Measured (one MI355X, whole calls): 65536 rows of 32 groups of about 2048, N = 4608, K = 5120: 1460 to 1500 us, 2.1 PFLOP/s;
// with groups of exactly 2048 rows 1330 (a group's last, ragged tile takes a whole tile's time).  What bounds it is the
// way of the operands to LDS as much as the MFMAs: a 256 x 256 tile takes 64 KiB per 128 K, and a kernel of such tiles
// took 1285 us for the DMA alone (580 when every tile reads the same lines) and 1130 without any.  Half of the L2's
// requests miss.  Where tiles begin in K decides what they share there: turned by the row tile, so that the tiles that
// read the same activation rows are at the same K, 1460; by row and column tile 1490, by the column tile 1505, not at
// all 1490.
#include <type_traits>

#include "grouped.hpp"

namespace mx {

namespace {

constexpr int kT = 256;                    // rows and columns of a tile
constexpr int kOp = kT * kStageK;          // 32 KiB per operand and stage
constexpr int kFoldStores = 32;            // stores a wave issues in a whole tile's epilogue
constexpr uint32_t kNoRow = 0xFFFFFF80u;   // a row offset behind every resource, chunk bits clear

// calls f(integral_constant<int, k>) for k = B .. E-1, in order
template <int B, int E, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    static_for<B + 1, E>(f);
  }
}
// the order of the 16 MFMAs of a half-stage (W tile I, x tile J): each fragment is first used as late as the reading
// order (w0 x0 x1 w1 x2 w2 x3 w3) allows
constexpr int kOrdI[16] = {0, 0, 1, 1, 0, 1, 2, 2, 2, 0, 1, 2, 3, 3, 3, 3};
constexpr int kOrdJ[16] = {0, 1, 0, 1, 2, 2, 0, 1, 2, 3, 3, 3, 0, 1, 2, 3};

template <int I, int J, bool FIRST>
__device__ __forceinline__ void mfma_ij(v16f (&acc)[4][4], const v8i (&w)[4], const v8i (&x)[4], uint32_t sw,
                                        uint32_t sx) {
  const v16f zero = {};
  acc[I][J] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[I], x[J], FIRST ? zero : acc[I][J], 0, 0, I,
                                                             static_cast<int>(sw), J, static_cast<int>(sx));
}

typedef const __attribute__((address_space(4))) int32_t* const_i32;

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

struct Tile {
  int e, row0, rows, n0, cols;
  int turn;                                // the pair of stages it starts at
};

__device__ __forceinline__ void grouped_large(const GemmArgs& p) {
  __shared__ __attribute__((aligned(1024))) uint8_t st0[2 * kOp];
  __shared__ __attribute__((aligned(1024))) uint8_t st1[2 * kOp];
  // scale words of two windows of four stages: [stage][block][W | x][half of the tile][row % 32], a byte per 32-row
  // tile
  __shared__ __attribute__((aligned(16))) uint32_t sc[2][4][4][2][2][32];
  // 4 KiB per wave: the epilogue's staging; between epilogues the next tile's row offsets in xq (256 words) and in xs
  __shared__ __attribute__((aligned(16))) uint32_t stage_lds[4096];
  constexpr int kScBlk = 2 * 2 * 32, kScStep = 4 * kScBlk;   // words

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wt = wave >> 1;
  const int r32 = lane & 31, q2 = lane >> 5;
  const int KB = p.KB, KE = (KB + 1) & ~1;             // stages, made even
  const int K32 = p.K / 32, windows = (KE + 3) >> 2;
  const uint32_t slab = static_cast<uint32_t>(p.rows) * kStageK;   // bytes of a K block of the activation
  const int pairs = KE / 2;

  // ---- tiles of this workgroup: every XCD takes a contiguous range of the list, its workgroups one tile of each round
  // of wg_per_xcd tiles, rotated by 8 from round to round so that no compute unit leads in all of them
  const const_i32 list = (const_i32)(uintptr_t)p.tiles;
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  const int total = list[2] * p.n_tiles;               // tiles[0].count
  const int per_xcd = (total + 7) >> 3;
  auto tile_at = [&](int r, Tile& t) {
    const int li = (slot + r * 8) % p.wg_per_xcd + r * p.wg_per_xcd;
    const int work = xcd * per_xcd + li;
    if (li >= per_xcd || work >= total) return false;
    const const_i32 d = list + 8 * (1 + work / p.n_tiles);
    const int local = work - d[1] * p.n_tiles, count = d[2];
    t.e = uniform(d[0]);
    t.row0 = uniform(d[3] + local % count * kT);
    t.rows = uniform(min(kT, d[4] - t.row0));
    t.n0 = uniform(local / count * kT);
    t.cols = uniform(min(kT, p.N - t.n0));
    t.turn = uniform(local % count % pairs);
    return true;
  };
  // rows of round r only: where a workgroup's rounds have a gap there are no later tiles either (li grows with r)

  // what tile row r reads: its slot where the rows are gathered
  auto row_source = [&](const Tile& t, int r) {
    const int rr = t.row0 + min(r, t.rows - 1);
    return p.row_slot ? p.row_slot[rr] : rr;
  };
  // and that source's byte offsets in xq and xs; a source outside x reads row 0 and gets NaN scales
  auto row_offsets = [&](const Tile& t, int r, int source, uint32_t& xq_off, uint32_t& xs_off) {
    const int row = p.row_slot && source >= 0 ? static_cast<int>(div_u32(static_cast<uint32_t>(source), p.k_div)) : source;
    const bool bad = row < 0 || row >= p.rows;
    const uint32_t at = bad ? 0u : static_cast<uint32_t>(row);
    xq_off = r < t.rows ? at * kStageK : kNoRow;
    xs_off = bad ? 0xFFFFFFFFu : at * static_cast<uint32_t>((KB + 3) & ~3) * 4;
  };

  // ---- DMA: wave `wave` fills rows it*32 + wave*8 + lane/8 of each operand, lane i -> physical chunk i % 8
  const int dma_row = wave * 8 + (lane >> 3);
  const uint32_t chunk = static_cast<uint32_t>((lane & 7) ^ swz8(dma_row)) * 16;   // swz8(r) = swz8(r % 16)
  const __amdgpu_buffer_rsrc_t xres = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.xq), 0, static_cast<int>(static_cast<uint32_t>(KB) * slab), kBufferFlags);
  const uint8_t* wptr;         // the tile's weight rows, and their bytes
  int wbytes;
  const uint32_t baseW = static_cast<uint32_t>(dma_row) * static_cast<uint32_t>(p.K);
  uint32_t capW;               // offset of the tile's last weight row
  uint32_t offX[8];
  int pk = 0;                  // the stage to fetch next, of the tile set by dma_tile (which turns it, see Tile)
  uint32_t behind = 0;         // or-ed into the offsets where there is nothing to fetch: behind K, or no further tile
  auto dma_tile = [&](const Tile& t) {
    wptr = p.w + (static_cast<size_t>(uniform(t.e)) * p.N + uniform(t.n0)) * p.K;
    wbytes = uniform(t.cols * p.K);
    pk = 2 * t.turn;
    capW = static_cast<uint32_t>(t.cols - 1) * static_cast<uint32_t>(p.K);
  };
  auto dma_w = [&](auto IT, uint8_t* buf, uint32_t k, uint32_t none) {
    constexpr int it = decltype(IT)::value;
    uint32_t b = baseW;
    asm volatile("" : "+v"(b));                        // formed here, not held for every `it`
    const uint32_t off = min(b + static_cast<uint32_t>(it * 32) * static_cast<uint32_t>(p.K), capW) + k;
    const __amdgpu_buffer_rsrc_t wres =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(wptr), 0, wbytes, kBufferFlags);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(wres, (lds_void_t*)(buf + (it * 32 + wave * 8) * kStageK), 16, off | none, 0,
                                             0, 0);
  };
  auto dma_x = [&](auto IT, uint8_t* buf, uint32_t k, uint32_t none) {
    constexpr int it = decltype(IT)::value;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(xres, (lds_void_t*)(buf + kOp + (it * 32 + wave * 8) * kStageK), 16,
                                             offX[it] | none, static_cast<int>(k), 0, 0);
  };
  auto chunk_k = [&]() { return min(static_cast<uint32_t>(pk * kStageK) + chunk, static_cast<uint32_t>(p.K - 16)); };
  auto next_stage = [&]() { pk = pk + 1 < KE ? pk + 1 : 0; };
  auto issue = [&](uint8_t* buf) {                     // the whole stage at once, in the prologue
    const uint32_t k = chunk_k(), none = pk < KB ? 0u : kNoRow;
    static_for<0, 8>([&](auto it) { dma_w(it, buf, k, none); });
    static_for<0, 8>([&](auto it) { dma_x(it, buf, min(pk, KB - 1) * slab, none); });
    next_stage();
  };

  // ---- scales: thread (operand, half, two of the four stages, r32) builds the words of rows r32 + 32 i of its half
  const int s_op = tid >> 7, s_half = (tid >> 6) & 1, s_pair = (tid >> 5) & 1, s_r = tid & 31;
  const uint8_t* s_base;       // W: the tile's first scale row; x: xs
  uint32_t s_off[4];
  uint32_t s_room = 0;         // W: the last offset from s_base at which 8 bytes of the tensor begin
  uint64_t s_own[4];
  int lwin = 0;                // window to load next, counted from the tile's turn
  int s_turn = 0;
  auto scale_tile = [&](const Tile& t, auto offset_of) {
    s_turn = t.turn;
    if (s_op == 0) {
      const size_t first = static_cast<size_t>(t.e) * p.N + t.n0;
      s_base = static_cast<const uint8_t*>(p.ws) + first * K32;
      const size_t left = (static_cast<size_t>(p.E) * p.N - first) * K32 - 8;
      s_room = static_cast<uint32_t>(min(left, static_cast<size_t>(1) << 31));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s_off[i] = static_cast<uint32_t>(min(s_half * 128 + 32 * i + s_r, t.cols - 1)) * static_cast<uint32_t>(K32);
    } else {
      s_base = reinterpret_cast<const uint8_t*>(p.xs);
      s_room = 0xFFFFFFFFu;
#pragma unroll
      for (int i = 0; i < 4; ++i) s_off[i] = offset_of(s_half * 128 + 32 * i + s_r);
    }
  };
  // this thread's pair of stages in window lwin (one behind the last pair is never used)
  auto scale_pair = [&]() {
    const int at = 2 * lwin + s_pair + s_turn;
    return at < pairs ? at : min(at - pairs, pairs - 1);
  };
  auto scale_at = [&](int i, int pair, uint32_t& back) {   // where row i's 8 bytes of it are read
    const uint32_t row = s_op == 1 && s_off[i] == 0xFFFFFFFFu ? 0u : s_off[i];
    const uint32_t off = row + static_cast<uint32_t>(8 * pair);
    back = off > s_room ? off - s_room : 0u;
    return s_base + (off - back);
  };
  uint32_t s_back[4];
  int s_left;                  // 32-K blocks of the row from the loaded pair on
  uint32_t s_bad;              // bit i: row i has no source
  auto load_scales = [&]() {
    s_bad = 0;
    const int pair = scale_pair();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t back;
      __builtin_memcpy(&s_own[i], scale_at(i, pair, back), 8);
      s_back[i] = back;
      s_bad |= (s_op == 1 && s_off[i] == 0xFFFFFFFFu ? 1u : 0u) << i;
    }
    s_left = K32 - 8 * pair;
    ++lwin;
  };
  auto store_scales = [&](int buf) {
    uint32_t* const dst = &sc[buf][2 * s_pair][0][s_op][s_half][s_r];
    const uint64_t keep = s_left >= 8 ? ~uint64_t(0) : s_left <= 0 ? 0 : (uint64_t(1) << (8 * s_left)) - 1;
    uint64_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (s_own[i] >> (8 * s_back[i]) & keep) | (s_bad >> i & 1 ? ~uint64_t(0) : 0);
#pragma unroll
    for (int st = 0; st < 2; ++st) {
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = static_cast<uint32_t>(v[i] >> (32 * st));
      // 4 x 4 byte transpose: word b = byte b of rows 0, 1, 2, 3
      const uint32_t t0 = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u), t1 = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u);
      const uint32_t t2 = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u), t3 = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
      dst[st * kScStep] = __builtin_amdgcn_perm(t1, t0, 0x05040100u);
      dst[st * kScStep + kScBlk] = __builtin_amdgcn_perm(t1, t0, 0x07060302u);
      dst[st * kScStep + 2 * kScBlk] = __builtin_amdgcn_perm(t3, t2, 0x05040100u);
      dst[st * kScStep + 3 * kScBlk] = __builtin_amdgcn_perm(t3, t2, 0x07060302u);
    }
  };
  uint32_t sw[2], sx[2];       // this stage's words, by half
  auto read_scales = [&](int buf, int st, uint32_t (&w)[2], uint32_t (&x)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = sc[buf][st][2 * h + q2][0][wn][r32];
      x[h] = sc[buf][st][2 * h + q2][1][wt][r32];
    }
  };

  // ---- fragments: row wn*128 + 32 i + lane%32 (W), wt*128 + 32 j + lane%32 (x); for half h, lane group q takes the
  // logical chunks 4 h + q and 4 h + q + 2
  const int rdW = (wn * 128 + r32) * kStageK;
  const int rdX = kOp + (wt * 128 + r32) * kStageK;
  const int sz = swz8(r32);
  const int ch00 = (q2 ^ sz) << 4, ch01 = ((q2 + 2) ^ sz) << 4;
  const int ch10 = ((4 + q2) ^ sz) << 4, ch11 = ((6 + q2) ^ sz) << 4;
  v8i fw[2][4], fx[2][4];
  auto read_frag = [&](const uint8_t* q, int c0, int c1) {
    const uint4 lo = *reinterpret_cast<const uint4*>(q + c0), hi = *reinterpret_cast<const uint4*>(q + c1);
    v8i v;
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    return v;
  };
  auto read_k = [&](auto KK, const uint8_t* buf, int c0, int c1, v8i (&w)[4], v8i (&x)[4]) {
    constexpr int k = decltype(KK)::value;             // w0 x0 x1 w1 x2 w2 x3 w3
    constexpr bool isW = k == 0 || k == 3 || k == 5 || k == 7;
    constexpr int idx = k == 0 ? 0 : k == 1 ? 0 : k == 2 ? 1 : k == 3 ? 1 : k == 4 ? 2 : k == 5 ? 2 : 3;
    if constexpr (isW)
      w[idx] = read_frag(buf + rdW + idx * 32 * kStageK, c0, c1);
    else
      x[idx] = read_frag(buf + rdX + idx * 32 * kStageK, c0, c1);
  };
  v16f acc[4][4];
  // the MFMAs are pure: without a use the compiler would sink them below the waits and the barrier
  auto pin_acc = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) asm volatile("" ::"a"(acc[i][j]));
  };

  // ---- state of the tile being multiplied
  Tile cur, nxt;
  bool more;
  int source = 0;              // of row `tid` of the next tile, on its way to LDS

  // front of the stage in `buf`, up to its barrier
  auto front = [&](const uint8_t* buf, auto first) {
    __builtin_amdgcn_sched_barrier(0);
    static_for<0, 16>([&](auto KK) {
      constexpr int k = decltype(KK)::value;
      mfma_ij<kOrdI[k], kOrdJ[k], decltype(first)::value>(acc, fw[0], fx[0], sw[0], sx[0]);
      if constexpr (k < 8) read_k(KK, buf, ch10, ch11, fw[1], fx[1]);
      __builtin_amdgcn_sched_barrier(0);
    });
    pin_acc();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
  };
  // back of stage s in `cur_buf`, the next stage in `nxt_buf`: fetches stage pk, reads the words of stage st of scale
  // buffer wb
  auto back = [&](uint8_t* cur_buf, const uint8_t* nxt_buf, int wb, int st) {
    uint32_t sw1[2], sx1[2];
    read_scales(wb, st, sw1, sx1);                     // before the DMA, which the compiler would make them wait for
    const uint32_t none = pk < KB ? behind : kNoRow;
    const uint32_t k = chunk_k();
    const uint32_t kx = min(pk, KB - 1) * slab;
    next_stage();
    __builtin_amdgcn_sched_barrier(0);
    static_for<0, 16>([&](auto KK) {
      constexpr int kk = decltype(KK)::value;
      mfma_ij<kOrdI[kk], kOrdJ[kk], false>(acc, fw[1], fx[1], sw[1], sx[1]);
      if constexpr (kk < 8)
        dma_w(KK, cur_buf, k, none);
      else
        dma_x(std::integral_constant<int, kk - 8>{}, cur_buf, kx, none);
      if constexpr (kk < 8) read_k(KK, nxt_buf, ch00, ch01, fw[0], fx[0]);
      __builtin_amdgcn_sched_barrier(0);
    });
    pin_acc();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sw[h] = sw1[h];
      sx[h] = sx1[h];
    }
  };

  // The epilogue of `cur` folded into the first half-stage of the next tile (fragments fw[0], fx[0], buffer `buf`): the
  // wave's 128 x 128 results leave in 8 chunks of 32 rows x 64 columns, through LDS so that a store writes 8 rows of
  // 128 bytes.  As soon as a chunk is in LDS the two MFMAs that start the next tile's sums in its blocks are issued.
  // LDS and MFMAs here are inline asm, with their own waits: as plain accesses the compiler waits for the DMA before
  // each, and as builtins the new sums get registers of their own.
  uint8_t* const stg = reinterpret_cast<uint8_t*>(stage_lds) + wave * 4096;
  const int er = lane >> 3, ec = lane & 7;
  typedef unsigned int v4u_t __attribute__((ext_vector_type(4)));
  auto front_fold = [&](const uint8_t* buf) {
    const uint32_t wa = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(stg));   // the low 32 bits address LDS
    const int trow = wt * 128 + er, ncol = wn * 128 + ec * 8;
    uint16_t* const obase = p.out + static_cast<size_t>(cur.row0 + trow) * p.N + cur.n0 + ncol;
    const size_t rs8 = static_cast<size_t>(8) * p.N;
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(kWaitLgkmOnly);         // the fragments of this half have landed
    static_for<0, 8>([&](auto C) {
      constexpr int c8 = decltype(C)::value, j = c8 >> 1, ip = c8 & 1;
#pragma unroll
      for (int ii = 0; ii < 2; ++ii) {
        const v16f& v = acc[2 * ip + ii][j];
#pragma unroll
        for (int pp = 0; pp < 2; ++pp) {
          const uint32_t x0 = pack_bf16x2(v[8 * pp + 0], v[8 * pp + 1]), x1 = pack_bf16x2(v[8 * pp + 2], v[8 * pp + 3]);
          const uint32_t y0 = pack_bf16x2(v[8 * pp + 4], v[8 * pp + 5]), y1 = pack_bf16x2(v[8 * pp + 6], v[8 * pp + 7]);
          const auto s0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
          const auto s1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
          const int c = ii * 4 + pp * 2 + q2;
          const uint32_t a = wa + r32 * 128 + ((c ^ (r32 & 7)) << 4);
          const v4u_t dv = {s0[0], s1[0], s0[1], s1[1]};
          asm volatile("ds_write_b128 %0, %1" ::"v"(a), "v"(dv) : "memory");
        }
      }
      asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, 0, %3, %4 op_sel:[%5,%6,0] op_sel_hi:[%7,%8,0]"
                   : "+a"(acc[2 * ip][j])
                   : "v"(fw[0][2 * ip]), "v"(fx[0][j]), "v"(sw[0]), "v"(sx[0]), "n"((2 * ip) & 1), "n"(j & 1),
                     "n"((2 * ip) >> 1), "n"(j >> 1));
      asm volatile("v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, 0, %3, %4 op_sel:[%5,%6,0] op_sel_hi:[%7,%8,0]"
                   : "+a"(acc[2 * ip + 1][j])
                   : "v"(fw[0][2 * ip + 1]), "v"(fx[0][j]), "v"(sw[0]), "v"(sx[0]), "n"((2 * ip + 1) & 1), "n"(j & 1),
                     "n"((2 * ip + 1) >> 1), "n"(j >> 1));
      v4u_t d0, d1, d2, d3;
      asm volatile(
          "s_waitcnt lgkmcnt(0)\n"
          "ds_read_b128 %0, %4\n"
          "ds_read_b128 %1, %4 offset:1024\n"
          "ds_read_b128 %2, %4 offset:2048\n"
          "ds_read_b128 %3, %4 offset:0xc00\n"
          "s_waitcnt lgkmcnt(0)"
          : "=&v"(d0), "=&v"(d1), "=&v"(d2), "=&v"(d3)
          : "v"(wa + er * 128 + ((ec ^ er) << 4))
          : "memory");
      const v4u_t d[4] = {d0, d1, d2, d3};
#pragma unroll
      for (int sg = 0; sg < 4; ++sg) {
        if (trow + j * 32 + sg * 8 < cur.rows && ncol + ip * 64 < cur.cols)
          *reinterpret_cast<uint4*>(obase + (j * 4 + sg) * rs8 + ip * 64) =
              make_uint4(d[sg][0], d[sg][1], d[sg][2], d[sg][3]);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    static_for<0, 8>([&](auto KK) { read_k(KK, buf, ch10, ch11, fw[1], fx[1]); });
    pin_acc();
    __builtin_amdgcn_sched_barrier(0);
    // A whole tile issued kFoldStores stores behind the DMA that this waits for (and reloads of spilled registers, which
    // have waited for that DMA already, so that as built the wait finds it done); they may stay in flight.
    if (cur.rows == kT && cur.cols == kT)
      __builtin_amdgcn_s_waitcnt(wait_vm(kFoldStores));
    else
      __builtin_amdgcn_s_waitcnt(wait_vm(0));
  };

  // ---- the first tile
  if (!tile_at(0, cur)) return;
  more = tile_at(1, nxt);
  {
    uint32_t a, b;
    row_offsets(cur, tid, row_source(cur, tid), a, b);
    stage_lds[tid] = a;
    stage_lds[256 + tid] = b;
    __syncthreads();
    dma_tile(cur);
#pragma unroll
    for (int it = 0; it < 8; ++it) offX[it] = stage_lds[it * 32 + dma_row] | chunk;
    scale_tile(cur, [&](int r) { return stage_lds[256 + r]; });
    __syncthreads();
  }
  issue(st0);
  load_scales();
  issue(st1);
  store_scales(0);
  load_scales();
  if (more) source = row_source(nxt, tid);
  __builtin_amdgcn_s_waitcnt(wait_vm(0));
  __syncthreads();
  read_scales(0, 0, sw, sx);
  static_for<0, 8>([&](auto KK) { read_k(KK, st0, ch00, ch01, fw[0], fx[0]); });
  front(st0, std::true_type{});
  __builtin_amdgcn_s_barrier();

  const std::false_type no{};
  // the next window's scales into buffer b, at the end of the window's last stage; then the one after is asked for
  auto next_window = [&]() {
    if (lwin == windows) {                             // on to the next tile's windows
      lwin = 0;
      if (more) scale_tile(nxt, [&](int r) { return stage_lds[256 + r]; });
    }
    load_scales();
  };
  int wbuf = 0;                                        // scale buffer of stage s
  for (int round = 0;;) {
    // On entry stage 0's half 0 is done and its half 1 in registers; stage 1 is on its way or landed.
    for (int s = 0; s + 2 < KE; s += 2) {
      back(st0, st1, wbuf, (s + 1) & 3);
      front(st1, no);
      const bool end = (s & 3) == 2;                   // stage s + 1 is a window's last
      if (end) store_scales(wbuf ^ 1);
      if (s == 0) {
        uint32_t a = 0, b = 0;
        if (more) row_offsets(nxt, tid, source, a, b);
        stage_lds[tid] = a;
        stage_lds[256 + tid] = b;
      }
      __builtin_amdgcn_s_waitcnt(kWaitLgkmOnly);
      __builtin_amdgcn_s_barrier();
      if (end) next_window();
      wbuf ^= end ? 1 : 0;
      back(st1, st0, wbuf, (s + 2) & 3);
      front(st0, no);
      __builtin_amdgcn_s_barrier();
    }
    // the last two stages, while the next tile's first two are fetched
    if (more) {
      dma_tile(nxt);
#pragma unroll
      for (int it = 0; it < 8; ++it) offX[it] = stage_lds[it * 32 + dma_row] | chunk;
    } else {
      behind = kNoRow;
    }
    back(st0, st1, wbuf, (KE - 1) & 3);
    front(st1, no);
    store_scales(wbuf ^ 1);
    __builtin_amdgcn_s_waitcnt(kWaitLgkmOnly);
    __builtin_amdgcn_s_barrier();
    next_window();
    wbuf ^= 1;
    back(st1, st0, wbuf, 0);
    front_fold(st0);
    __builtin_amdgcn_s_barrier();
    if (!more) break;
    cur = nxt;
    more = tile_at(++round + 1, nxt);
    if (more) source = row_source(nxt, tid);
  }
  __builtin_amdgcn_s_waitcnt(wait_vm(0));              // no DMA outlives the workgroup
}

__global__ __launch_bounds__(256, 1) void grouped_large_kernel(GemmArgs p) {
  grouped_large(p);
}

}  // namespace

void launch_grouped_large(const GemmArgs& a, hipStream_t stream) {
  grouped_large_kernel<<<8 * a.wg_per_xcd, 256, 0, stream>>>(a);
}

}  // namespace mx
