// The grouped and block-128 products' kernel for small groups (gfx950): 32 rows per tile, bound by the stream of the
// weights.
//
//   out[r, n] = bf16( sum_k  x[src(r), k] sx * W[e(r), n, k] sw ),  scales as in grouped.hip
//
// What costs here is everything that lets the stream pause: tiles that end at different times, a pipeline that fills
// and drains for each of them, and scales that arrive by loads of their own.  So
//  * one resident workgroup per compute unit takes an equal share of the whole product: the (expert, 16 or 32 columns)
//    units are numbered through and cut into as many ranges as there are workgroups.  A range is walked in tiles of up
//    to 64 columns (an expert's row tiles one after the other on the same columns: the weight comes from HBM once).
//  * the pipeline runs on through the tile boundaries: a ring of S super-stages of WGK x 128 K in LDS, filled by
//    LDS-DMA S - 1 super-stages ahead of the MFMAs, whatever tile those belong to.
//  * the scale words (and the row indices of the next tile) come by LDS-DMA too, so one count of vector-memory
//    instructions orders everything, and nothing else waits for memory.  LDS is read and written in inline asm with its
//    own waits: the compiler, which cannot tell the slots of a ring apart, would drain the DMA before each access.
//  * rows behind the group's last and columns behind the tile's last are not fetched: their offsets lie behind the
//    buffer resource.
// Eight waves: two share a tile's 64 columns, and four such pairs each take every fourth 128 K; their sums meet in the
// slot that was multiplied last.  A step is short, so its instructions count: DMA offsets are registers fixed per tile,
// the place in K a scalar offset, and what is not to be fetched has a resource of no bytes (and a scalar offset of 0:
// the bounds are checked against the bytes less that offset).
//
// Measured (one MI355X): one token of 8 experts, N = 4608, K = 5120 (195 MB): 39 us, 5.0 TB/s (whole
// call 44; with a workgroup per tile 55).  512 bytes of a row at a time is what HBM wants: the pattern alone reads 5.7
// TB/s, with 128 bytes 4.2 by way of LDS.  For 64 or 128 rows the same ring lost against plain tiles (48 rows a group:
// 117 against 99 us): the scale words and the steps' control are not hidden there.
#include "grouped.hpp"

namespace mx {

namespace {

typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(4))) int32_t* const_i32;

// Columns of a unit of work.  With FP32 scales the 32 columns of an MFMA tile share one, so they may not straddle a
// block of 128.
constexpr int unit_columns(bool f32) { return f32 ? 32 : 16; }
constexpr uint32_t kNone = 0xFFFFFF80u;    // an offset behind every resource
constexpr int kSlotBufs = 8;               // tiles whose row indices are held in LDS
constexpr int kSlotWords = 64;             // of a tile: its rows' indices, in the one word a lane that a DMA writes

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));   // the low 32 bits of a generic address
}
__device__ __forceinline__ uint32_t lds_read(uint32_t at) {
  uint32_t v;
  asm volatile("ds_read_b32 %0, %1\ns_waitcnt lgkmcnt(0)" : "=&v"(v) : "v"(at) : "memory");
  return v;
}
__device__ __forceinline__ v8i join(const v4u lo, const v4u hi) {
  v8i v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = static_cast<int>(lo[i]);
    v[4 + i] = static_cast<int>(hi[i]);
  }
  return v;
}

// The fragments of a wave's W row and x row for 64 K: chunks at w0, w1 and x0, x1.  One block of asm, with its wait.
__device__ __forceinline__ void read_fragments(uint32_t w0, uint32_t w1, uint32_t x0, uint32_t x1, v8i& fw, v8i& fx) {
  v4u a0, a1, c0, c1;
  asm volatile("ds_read_b128 %0, %4\nds_read_b128 %1, %5\nds_read_b128 %2, %6\nds_read_b128 %3, %7\n"
               "s_waitcnt lgkmcnt(0)"
               : "=&v"(a0), "=&v"(a1), "=&v"(c0), "=&v"(c1)
               : "v"(w0), "v"(w1), "v"(x0), "v"(x1)
               : "memory");
  fw = join(a0, a1);
  fx = join(c0, c1);
}

struct Tile {
  int e, row0, rows, n0, cols, turn;
};

// ODD: K is no multiple of 128 (the last stage is short), or the MXFP8 weight's scale words are not 4-byte aligned (a
// row's four of a super-stage then lie in the five aligned words around them: 46 rows of 8 groups, N = 3584, K = 4448:
// 38.5 us against 56.5 with two words for each of the four; K = 4480: 36).
template <bool F32, bool ODD>
__device__ __forceinline__ void grouped_stream(const GemmArgs& p) {
  constexpr int BM = 32, BN = 64, WGN = 2, WGK = 4, S = 3;
  constexpr int kWaves = WGN * WGK;
  constexpr int kSub = (BN + BM) * kStageK;            // one 128-K stage: W rows, then x rows
  constexpr int kSlot = kSub * WGK;
  constexpr bool kTail = ODD && !F32;
  constexpr int kScW = WGK + (kTail ? 1 : 0);          // words of a W row's scales; unaligned, they lie in one more
  constexpr int kScX = WGK * BM;                       // words of the x rows' scales
  constexpr int kScWords = kScX + kScW * BN;
  constexpr int kScIns = kScWords / 64;                // DMA instructions of a super-stage's scales
  constexpr int kXIns = WGK * BM / 8, kWIns = WGK * BN / 8;
  constexpr int XPW = (kXIns + kWaves - 1) / kWaves, WPW = kWIns / kWaves, SPW = (kScIns + kWaves - 1) / kWaves;
  constexpr int kDma = XPW + WPW + SPW;                // per wave and super-stage; where there are fewer, some repeat
  constexpr int kUnit = unit_columns(F32), kPer = BN / kUnit;   // columns of a unit, units of a tile
  static_assert(kWIns % kWaves == 0 && (S - 2) * kDma <= 63, "instruction counts");
  static_assert((WGK - 1) * WGN * 4096 <= kSlot, "the partial sums fit a slot");
  static_assert(BM <= kSlotWords, "the row indices fit a buffer");
  __shared__ __attribute__((aligned(1024))) uint8_t ring[S * kSlot];
  __shared__ __attribute__((aligned(256))) uint32_t scales[S * kScWords];
  __shared__ __attribute__((aligned(256))) int32_t slots[kSlotBufs * kSlotWords];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int wn = wave % WGN, wk = wave / WGN;
  const int r32 = lane & 31, q2 = lane >> 5;
  const int KB = p.KB, KS = (KB + WGK - 1) / WGK, K32 = p.K / 32;
  const int NU = (p.N + kUnit - 1) / kUnit, NB = (p.N + 127) / 128;
  const uint32_t slab = static_cast<uint32_t>(p.rows) * kStageK;

  // ---- this workgroup's range of units: a unit is 16 or 32 columns of one row tile, numbered by expert, BN columns,
  // row tile, unit.  Workgroup i runs on XCD i % 8: an XCD's workgroups take neighbouring ranges.
  const const_i32 list = (const_i32)(uintptr_t)p.tiles;
  const int total_mt = p.tiles ? list[2] : (p.S + BM - 1) / BM;   // tiles[0].count
  const int units = total_mt * NU;                     // below 2^31, see the host's checks
  const int wgs = gridDim.x, wg = (blockIdx.x & 7) * (wgs >> 3) + (blockIdx.x >> 3);
  const int share = units / wgs, extra = units - share * wgs;
  const int u0 = share * wg + min(wg, extra), u1 = u0 + share + (wg < extra ? 1 : 0);
  if (u0 >= u1) return;
  // The tile that begins with unit u; moves u behind it.  Tiles start at different places of K and go round, so that
  // they do not all read the same few channels' lines: `turn` is the last tile's start.
  auto tile_at = [&](int& u, int turn) {
    Tile t;
    int first = 0, count = total_mt, lo = 0, hi = p.S;
    t.e = 0;
    if (p.tiles) {
      const const_i32 d = list + 8 * (1 + static_cast<int>(div_u32(static_cast<uint32_t>(u), p.nu_div)));
      t.e = d[0];
      first = d[1];
      count = d[2];
      lo = d[3];
      hi = d[4];
    }
    const int local = u - first * NU;
    int b = local / kPer, m = 0, c = local % kPer;     // BN-column block, row tile, unit in the block
    if (count > 1) {
      b = local / (kPer * count);
      const int rem = local - b * kPer * count, width = min(kPer, NU - b * kPer);
      m = rem / width;
      c = rem - m * width;
    }
    const int n = min(min(kPer, NU - b * kPer) - c, u1 - u);
    t.e = uniform(t.e);
    t.row0 = uniform(lo + m * BM);
    t.rows = uniform(min(BM, hi - t.row0));
    t.n0 = uniform((b * kPer + c) * kUnit);
    t.cols = uniform(min(n * kUnit, p.N - t.n0));
    t.turn = uniform(turn + 1 < KS ? turn + 1 : 0);
    u += n;
    return t;
  };

  // ---- producer: the DMA of tile `pt` (the pidx-th of this workgroup), super-stage pks next
  Tile pt;
  int pu = u0;             // the unit behind pt
  int pks = 0, pidx = 0, pslot = 0;
  bool more = true;            // there is something to fetch
  const uint32_t xbytes = static_cast<uint32_t>(KB) * slab;
  const uint32_t ring0 = lds_address(ring), scales0 = lds_address(scales), slots0 = lds_address(slots);
  uint32_t offX[XPW], offW[WPW], offT[WPW], offS[SPW];   // offT: in a short last stage
  const uint8_t* wptr;
  int wbytes;
  const uint8_t* sptr[SPW];
  uint32_t sbytes[SPW];
  auto resource = [](const void* at, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(at), 0, static_cast<int>(bytes), kBufferFlags);
  };

  // x row of tile row r, -1 outside x
  auto x_row = [&](const Tile& t, int idx, int r) {
    int s = t.row0 + r;
    if (p.row_slot) {
      const int id = static_cast<int>(lds_read(slots0 + static_cast<uint32_t>((idx % kSlotBufs) * kSlotWords + r) * 4));
      s = id < 0 ? -1 : static_cast<int>(div_u32(static_cast<uint32_t>(id), p.k_div));
    }
    return s >= p.rows ? -1 : s;
  };
  auto fetch_slots = [&](const Tile& t, int idx) {     // row indices of a tile (every wave issues one instruction)
    if (!p.row_slot) return;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(resource(p.row_slot + t.row0, static_cast<uint32_t>(t.rows) * 4),
                                             (lds_void_t*)(slots + (idx % kSlotBufs) * kSlotWords), 4, lane * 4, 0, 0, 0);
  };
  auto set_producer = [&](const Tile& t, int idx) {
    pks = 0;
    wptr = p.w + (static_cast<size_t>(t.e) * p.N + t.n0) * p.K;
    wbytes = t.cols * p.K;
    const int dr = lane >> 3;
#pragma unroll
    for (int u = 0; u < XPW; ++u) {
      const int r = (wave + u * kWaves) % kXIns % (BM / 8) * 8 + dr;
      const int row = max(x_row(t, idx, min(r, t.rows - 1)), 0);
      offX[u] = r < t.rows ? static_cast<uint32_t>(row) * kStageK + ((lane & 7) ^ swz8(r)) * 16 : kNone;
    }
#pragma unroll
    for (int u = 0; u < WPW; ++u) {
      const int r = (wave + u * kWaves) % (BN / 8) * 8 + dr;
      const uint32_t chunk = ((lane & 7) ^ swz8(r)) * 16, at = static_cast<uint32_t>(r) * static_cast<uint32_t>(p.K);
      offW[u] = r < t.cols ? at + chunk : kNone;
      // chunks behind K re-read the row's last one: the activation's codes there are zero
      offT[u] = r < t.cols ? at + min(chunk, static_cast<uint32_t>(p.K - 16 - (KB - 1) * kStageK)) : kNone;
    }
    const uint32_t row_bytes = static_cast<uint32_t>((KB + 3) & ~3) * 4;
#pragma unroll
    for (int u = 0; u < SPW; ++u) {
      const int i = (wave + u * kWaves) % kScIns;
      if (i < kScX / 64) {
        const int word = (i * 64 + lane) % (WGK * BM), r = word % BM;
        offS[u] = static_cast<uint32_t>(max(x_row(t, idx, min(r, t.rows - 1)), 0)) * row_bytes + word / BM * 4;
        sptr[u] = reinterpret_cast<const uint8_t*>(p.xs);
        sbytes[u] = static_cast<uint32_t>(p.rows) * row_bytes;
      } else {
        const int j = i - kScX / 64, r = j % (BN / 64) * 64 + lane, sub = j / (BN / 64);
        if constexpr (F32) {
          // every column brings its 128-block's scale (one for the whole tile, which lies inside a block)
          const float* const at = static_cast<const float*>(p.ws) + static_cast<size_t>(t.e) * NB * KB;
          sptr[u] = reinterpret_cast<const uint8_t*>(at);
          sbytes[u] = static_cast<uint32_t>(NB) * static_cast<uint32_t>(KB) * 4;
          offS[u] = static_cast<uint32_t>(min((t.n0 + r) / 128, NB - 1)) * static_cast<uint32_t>(KB) * 4 + sub * 4;
        } else {
          const uint8_t* const end = static_cast<const uint8_t*>(p.ws) + static_cast<size_t>(p.E) * p.N * K32;
          const uint8_t* const at =
              static_cast<const uint8_t*>(p.ws) + (static_cast<size_t>(t.e) * p.N + t.n0) * K32;
          const uint32_t mis = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at) & 3);
          sptr[u] = at - mis;
          // up to the aligned word that holds the tensor's last byte
          const size_t left = static_cast<size_t>(end - sptr[u]) + 3;
          sbytes[u] = static_cast<uint32_t>(min(left, static_cast<size_t>(1) << 30)) & ~3u;
          offS[u] = ((mis + static_cast<uint32_t>(min(r, t.cols - 1)) * static_cast<uint32_t>(K32)) & ~3u) + 4 * sub;
        }
      }
    }
  };
  // one super-stage into the next slot; the number of instructions is the same for every call
  auto issue_next = [&]() {
    if (pks == KS) {
      if (pu < u1) {
        pt = tile_at(pu, pt.turn);
        ++pidx;
        if (p.row_slot && KS < S - 1) {                // else the waits of the last KS steps cover the row indices
          __builtin_amdgcn_s_waitcnt(wait_vm(0));
          __builtin_amdgcn_s_barrier();
        }
        set_producer(pt, pidx);
        int nu = pu;
        if (nu < u1) fetch_slots(tile_at(nu, 0), pidx + 1);
      } else {
        more = false;
        pks = 0;
      }
    }
    const int ks = pks + pt.turn < KS ? pks + pt.turn : pks + pt.turn - KS;
    ++pks;
    uint8_t* const slot = ring + pslot * kSlot;
    uint32_t* const sc = scales + pslot * kScWords;
    pslot = pslot + 1 < S ? pslot + 1 : 0;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < WPW; ++u) {
      const int i = wave + u * kWaves, sub = i / (BN / 8), kb = ks * WGK + sub;
      const bool in = more && kb < KB;
      const uint32_t off = ODD && kb == KB - 1 ? offT[u] : offW[u];
      __builtin_amdgcn_raw_ptr_buffer_load_lds(resource(wptr, in ? static_cast<uint32_t>(wbytes) : 0u),
                                               (lds_void_t*)(slot + sub * kSub + i % (BN / 8) * 8 * kStageK), 16, off,
                                               in ? kb * kStageK : 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < XPW; ++u) {
      const int i = (wave + u * kWaves) % kXIns, sub = i / (BM / 8), rg = i % (BM / 8), kb = ks * WGK + sub;
      const bool in = more && kb < KB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(resource(p.xq, in ? xbytes : 0u),
                                               (lds_void_t*)(slot + sub * kSub + (BN + rg * 8) * kStageK), 16, offX[u],
                                               in ? static_cast<int>(static_cast<uint32_t>(kb) * slab) : 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < SPW; ++u) {
      const int i = (wave + u * kWaves) % kScIns;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(resource(sptr[u], more ? sbytes[u] : 0u), (lds_void_t*)(sc + i * 64), 4,
                                               offS[u], more ? 4 * WGK * ks : 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // ---- consumer
  const int sz = swz8(r32);
  uint32_t rdW[4], rdX[4];     // chunks 4 h + q and 4 h + q + 2 of the wave's first rows, h = 0, 1
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t chunk = static_cast<uint32_t>(((q2 + 2 * c) ^ sz) << 4);
    rdW[c] = ring0 + wk * kSub + (wn * 32 + r32) * kStageK + chunk;
    rdX[c] = ring0 + wk * kSub + (BN + r32) * kStageK + chunk;
  }
  const uint32_t rdSx = scales0 + (wk * BM + r32) * 4;
  const uint32_t rdSw = scales0 + (kScX + wk * BN + wn * 32 + r32) * 4;
  v16f acc = {};
  int cslot = 0;
  auto compute = [&](int kb, uint32_t misalign) {
    const uint32_t so = static_cast<uint32_t>(cslot) * kSlot, co = static_cast<uint32_t>(cslot) * kScWords * 4;
    const uint32_t sx = lds_read(rdSx + co);
    uint32_t sw = lds_read(rdSw + co);
    if constexpr (kTail) {
      sw = __builtin_amdgcn_alignbyte(lds_read(rdSw + co + BN * 4), sw, misalign);
      // blocks behind K: 2^-127, not what follows the row (which may be a NaN scale); their codes are zero
      if (kb == KB - 1 && (K32 & 3) != 0) sw &= (1u << (8 * (K32 & 3))) - 1;
    }
    v8i fw[2], fx[2];
    read_fragments(rdW[0] + so, rdW[1] + so, rdX[0] + so, rdX[1] + so, fw[0], fx[0]);
    read_fragments(rdW[2] + so, rdW[3] + so, rdX[2] + so, rdX[3] + so, fw[1], fx[1]);
    if constexpr (F32) {
      const float s = __uint_as_float(sx) * __uint_as_float(sw);
      v16f part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[0], fx[0], v16f{}, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
      part = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[1], fx[1], part, 0, 0, 0, 0x7F7F7F7F, 0, 0x7F7F7F7F);
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[r] = __builtin_fmaf(part[r], s, acc[r]);
    } else {
      // lane group q passes block 2 h + q: byte 2 h of the word moved down by q bytes
      const int swq = static_cast<int>(sw >> (8 * q2)), sxq = static_cast<int>(sx >> (8 * q2));
      acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[0], fx[0], acc, 0, 0, 0, swq, 0, sxq);
      acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[1], fx[1], acc, 0, 0, 2, swq, 2, sxq);
    }
  };

  // ---- the first tile; its row indices and the next tile's
  pt = tile_at(pu, wg % KS);
  fetch_slots(pt, 0);
  {
    int nu = pu;
    if (nu < u1) fetch_slots(tile_at(nu, 0), 1);
  }
  __builtin_amdgcn_s_waitcnt(wait_vm(0));
  __builtin_amdgcn_s_barrier();
  set_producer(pt, 0);
  Tile ct = pt;
  int cu = pu;
  int cidx = 0;
  for (int i = 0; i < S - 1; ++i) issue_next();
  for (;;) {
    const bool active = wn * 32 < ct.cols;
    const uint32_t misalign = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>(p.ws) +
        (static_cast<size_t>(ct.e) * p.N + ct.n0 + min(wn * 32 + r32, ct.cols - 1)) * K32) & 3;
    for (int i = 0; i < KS; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(wait_vm_only((S - 2) * kDma));
      __builtin_amdgcn_s_barrier();                    // this super-stage is in its slot; the slot before is free
      issue_next();
      const int ks = i + ct.turn < KS ? i + ct.turn : i + ct.turn - KS;
      if (active && ks * WGK + wk < KB) compute(ks * WGK + wk, misalign);
      __builtin_amdgcn_sched_barrier(0);
      if (i + 1 < KS) cslot = cslot + 1 < S ? cslot + 1 : 0;
    }

    // ---- the sums of the WGK sets, in the slot multiplied last, added in order by the first set
    constexpr int kSet = WGN * 4096;
    const uint32_t at = ring0 + static_cast<uint32_t>(cslot) * kSlot + wn * 4096 + lane * 16;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    if (wk > 0 && active) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const v4u v = {__float_as_uint(acc[4 * q]), __float_as_uint(acc[4 * q + 1]), __float_as_uint(acc[4 * q + 2]),
                       __float_as_uint(acc[4 * q + 3])};
        asm volatile("ds_write_b128 %0, %1" ::"v"(at + (wk - 1) * kSet + q * 1024), "v"(v) : "memory");
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    if (wk == 0 && active) {
#pragma unroll
      for (int s = 0; s < WGK - 1; ++s) {
        v4u v0, v1, v2, v3;
        asm volatile(
            "ds_read_b128 %0, %4\nds_read_b128 %1, %4 offset:1024\nds_read_b128 %2, %4 offset:2048\n"
            "ds_read_b128 %3, %4 offset:0xc00\ns_waitcnt lgkmcnt(0)"
            : "=&v"(v0), "=&v"(v1), "=&v"(v2), "=&v"(v3)
            : "v"(at + s * kSet)
            : "memory");
        const v4u v[4] = {v0, v1, v2, v3};
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[r] += __uint_as_float(v[r >> 2][r & 3]);
      }
      const bool bad = x_row(ct, cidx, min(r32, ct.rows - 1)) < 0;
      uint16_t* const orow = p.out + static_cast<size_t>(ct.row0 + r32) * p.N + ct.n0;
#pragma unroll
      for (int pp = 0; pp < 2; ++pp) {
        const uint32_t x0 = pack_bf16x2(acc[8 * pp + 0], acc[8 * pp + 1]), x1 = pack_bf16x2(acc[8 * pp + 2], acc[8 * pp + 3]);
        const uint32_t y0 = pack_bf16x2(acc[8 * pp + 4], acc[8 * pp + 5]), y1 = pack_bf16x2(acc[8 * pp + 6], acc[8 * pp + 7]);
        const auto s0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
        const int n = wn * 32 + 16 * pp + 8 * q2;
        uint4 o = make_uint4(s0[0], s1[0], s0[1], s1[1]);
        if (bad) o = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
        if (r32 < ct.rows && n < ct.cols) *reinterpret_cast<uint4*>(orow + n) = o;
      }
    }
    if (cu >= u1) break;
    ct = tile_at(cu, ct.turn);
    ++cidx;
    acc = v16f{};
    cslot = cslot + 1 < S ? cslot + 1 : 0;
  }
  __builtin_amdgcn_s_waitcnt(wait_vm(0));              // no DMA outlives the workgroup
}

template <bool F32, bool ODD>
__global__ __launch_bounds__(512, 1) void grouped_stream_kernel(GemmArgs p) {
  grouped_stream<F32, ODD>(p);
}

}  // namespace

void launch_grouped_stream(bool f32, const GemmArgs& a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(8 * a.wg_per_xcd);
  const int unit = unit_columns(f32);
  GemmArgs g = a;
  g.nu_div = make_div(static_cast<uint32_t>((a.N + unit - 1) / unit));
  const bool odd = a.K % 128 != 0 || (!f32 && !aligned(a.ws, 4));
  if (f32 && odd)
    grouped_stream_kernel<true, true><<<grid, 512, 0, stream>>>(g);
  else if (f32)
    grouped_stream_kernel<true, false><<<grid, 512, 0, stream>>>(g);
  else if (odd)
    grouped_stream_kernel<false, true><<<grid, 512, 0, stream>>>(g);
  else
    grouped_stream_kernel<false, false><<<grid, 512, 0, stream>>>(g);
}

}  // namespace mx
