// Products of BF16 rows with FP8 weights, grouped by expert or dense, on block-scaled FP8 MFMA (gfx950):
// mx_grouped_linear (MXFP8 or FP32 block-128 weights) and mx_linear_block128.
//
//   out[r, n] = bf16( sum_k  Q(x[src(r), k]) * W[e(r), n, k] )
//
// The rows r are sorted by expert: expert e owns rows [offsets[e], offsets[e+1]), known on the device alone.  Q rounds
// the activation to e4m3 with one scale per row and K block, the weight's own block length along K:
//   MXFP8   block 32, E8M0 on both sides: the scaled MFMA applies both scales.
//   FP32    block 128 on the activation, 128 x 128 on the weight.  Such scales are no powers of two, so the MFMA cannot
//           apply them: each 128-K block's partial sum P (two chained 32x32x64 MFMAs from zero) joins the running sum
//           as acc += P * (sa * sw), one fma per element and 128 K on the vector unit beside the matrix unit.
//
// Two launches:
//  * quant_rows_kernel: every activation row once (not once per expert that reads it): codes [KB, rows, 128] and one
//    4-byte scale word per 128 K [rows, KB4] (four E8M0 bytes, or one FP32) into the workspace, KB = K / 128 rounded
//    up, KB4 = KB rounded up to 4, with zero codes behind K.  The codes lie by K block first: row by row, the rows of a
//    tile, a multiple of 512 bytes apart as a rule, would meet in a few of the memory channels at every stage.  With
//    act = SwiGLU it reads [gate | up] and rounds silu(gate) * up to BF16 first.  One more workgroup turns the offsets
//    into a list of row tiles.  Bound by memory: 8192 x 4096 (100 MB) 20 us, 5 TB/s.
//  * a product over tiles of 32, 64, 128 or 256 rows (pick_shape): grouped_stream.hip for 32, grouped_large.hip for
//    many tiles of 256 with MXFP8 scales and 1024 K or more, and here grouped_gemm_kernel, one workgroup per BM x BN
//    tile.  Rows of the activation are gathered by their index as the LDS-DMA reads them, so no copy per expert is
//    written.
//
// What bounds grouped_gemm_kernel (one MI355X, kernel times):
//   128 x 128, 1544 rows of 32 groups, N = 5120, K = 2304, MXFP8: 95 us for 377 MB of weights, 4.0 TB/s.  The same
//     without MFMAs takes as long, with every tile on the same weight rows 52, without the x rows 88, without stores
//     86: the weights' stream, and the tiles' other traffic in its gaps.
//   256 x 256, 8192 rows, N = 5120, K = 4096, FP32 scales: 180 to 205 us, 1.7 to 1.9 PFLOP/s.  Without the fma's 6 %
//     less, with no DMA 20 % less, with operands of zeros 12 % less (the clock follows the power that the operands'
//     bits draw).
#include <type_traits>

#include "grouped.hpp"

namespace mx {

namespace {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef short v2s __attribute__((ext_vector_type(2)));
typedef const __attribute__((address_space(4))) uint32_t* const_u32;   // read through the scalar cache
// ------------------------------------------------------------------ quantiser

struct QuantRowsArgs {
  const uint16_t* x;          // BF16 [rows, K], or [rows, 2K] = gate | up
  uint8_t* xq;                // [KB, rows, 128] e4m3 codes
  uint32_t* xs;               // [rows, KB4] scale words, KB4 = KB rounded up to 4
  uint32_t rows, K, KB;
  uint32_t units;             // rows * KB
  DivU32 kb_div;
  // row tiles (workgroup 0 when offsets is set)
  const int32_t* offsets;     // [E + 1] or null
  RowTile* tiles;             // tiles[0].count = number of tiles, the tiles from 1 on
  int32_t E, S, BM, max_tiles;
};

// Expert e owns rows [offsets[e], offsets[e+1]) cut to [0, S); an interval that runs backwards is empty.  The list is
// cut at max_tiles, so offsets that overlap cannot make it longer than its space.
__device__ void build_row_tiles(const QuantRowsArgs& a) {
  __shared__ int32_t part[256];
  const int tid = threadIdx.x;
  const int per = (a.E + 255) / 256;
  const int e0 = min(tid * per, a.E), e1 = min(e0 + per, a.E);
  auto bounds = [&](int e, int& lo, int& hi) {
    lo = min(max(a.offsets[e], 0), a.S);
    hi = min(max(a.offsets[e + 1], lo), a.S);
  };
  int n = 0;
  for (int e = e0; e < e1; ++e) {
    int lo, hi;
    bounds(e, lo, hi);
    n += (hi - lo + a.BM - 1) / a.BM;
    n = min(n, a.max_tiles);
  }
  part[tid] = n;
  __syncthreads();
  for (int d = 1; d < 256; d *= 2) {
    const int v = tid >= d ? part[tid - d] : 0;
    __syncthreads();
    part[tid] = min(part[tid] + v, a.max_tiles);
    __syncthreads();
  }
  int first = tid > 0 ? part[tid - 1] : 0;
  for (int e = e0; e < e1; ++e) {
    int lo, hi;
    bounds(e, lo, hi);
    const int count = min((hi - lo + a.BM - 1) / a.BM, a.max_tiles - first);
    for (int i = 0; i < count; ++i) a.tiles[1 + first + i] = RowTile{e, first, count, lo, hi, {0, 0, 0}};
    first += count;
  }
  if (tid == 255) a.tiles[0].count = part[255];
}

__device__ __forceinline__ float silu_mul(float g, float u) {
  // g / (1 + 2^(-g log2 e)) * u.  Rounding g log2 e moves the exponential by |g| 2^-24 relative, the rest by a few 2^-24:
  // below 2^-16 in all for |g| <= 128 (beyond, the result is 0 or g u), under the BF16 rounding's 2^-8 that follows.
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Sixteen lanes (a DPP row) quantise one 128-K block of one row, 8 consecutive elements each.
template <bool F32, bool ACT>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantRowsArgs a) {
  uint32_t block = blockIdx.x;
  if (a.offsets != nullptr) {
    if (block == 0) {
      build_row_tiles(a);
      return;
    }
    --block;
  }
  const uint32_t raw = block * 16 + (threadIdx.x >> 4);
  const uint32_t unit = min(raw, a.units - 1);   // every lane takes part in the reductions
  const uint32_t row = div_u32(unit, a.kb_div), kb = unit - row * a.KB;
  const uint32_t l = threadIdx.x & 15, k = kb * kStageK + l * 8;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (k < a.K) {                                 // K is a multiple of 16: a chunk is inside or outside
    const uint16_t* src = a.x + static_cast<size_t>(row) * a.K * (ACT ? 2 : 1) + k;
    v = *reinterpret_cast<const uint4*>(src);
    if constexpr (ACT) {
      const uint4 u = *reinterpret_cast<const uint4*>(src + a.K);
      const uint32_t gw[4] = {v.x, v.y, v.z, v.w}, uw[4] = {u.x, u.y, u.z, u.w};
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[i] = pack_bf16x2(silu_mul(bf16_lo(gw[i]), bf16_lo(uw[i])), silu_mul(bf16_hi(gw[i]), bf16_hi(uw[i])));
      v = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
  // over the 4 lanes of a 32-K block, or all 16
  auto dpp = [](uint32_t x, auto ctrl) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(x), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  m = max(m, dpp(m, std::integral_constant<int, 0xB1>{}));   // quad_perm [1,0,3,2]
  m = max(m, dpp(m, std::integral_constant<int, 0x4E>{}));   // quad_perm [2,3,0,1]
  if constexpr (F32) {
    m = max(m, dpp(m, std::integral_constant<int, 0x128>{}));   // row_ror:8
    m = max(m, dpp(m, std::integral_constant<int, 0x124>{}));   // row_ror:4
  }
  const bool finite = m < 0x7F80u;
  uint2 codes;
  uint32_t word;
  if constexpr (F32) {
    // scale amax / 448; codes of the quotients x * 448 / amax.  They are formed from x and amax scaled by 2^-E (E the
    // exponent of amax, so nothing overflows), and corrected by one residual step: v = x r is off by up to two
    // roundings, which would break ties (BF16 inputs have many) either way; x * 448 - v * amax is exact in an fma.
    const float amax = fmaxf(__uint_as_float((finite ? m : 0) << 16), 0x1p-96f);
    const int E = min(static_cast<int>(__float_as_uint(amax) >> 23) - 127, 126);
    const float p2 = __uint_as_float(static_cast<uint32_t>(127 - E) << 23);
    const float am = amax * p2, rinv = 1.0f / am, r = 448.0f * rinv;
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float xl = bf16_lo(w[i]) * p2, xh = bf16_hi(w[i]) * p2;
      const float vl = xl * r, vh = xh * r;
      const float ql = __builtin_fmaf(__builtin_fmaf(-vl, am, xl * 448.0f), rinv, vl);
      const float qh = __builtin_fmaf(__builtin_fmaf(-vh, am, xh * 448.0f), rinv, vh);
      q[2 * i] = __builtin_amdgcn_fmed3f(ql, -448.0f, 448.0f);
      q[2 * i + 1] = __builtin_amdgcn_fmed3f(qh, -448.0f, 448.0f);
    }
    int lo = 0, hi = 0;
    lo = cvt_fp8x2<false>(q[0], q[1], lo);
    lo = cvt_fp8x2<true>(q[2], q[3], lo);
    hi = cvt_fp8x2<false>(q[4], q[5], hi);
    hi = cvt_fp8x2<true>(q[6], q[7], hi);
    codes = make_uint2(static_cast<uint32_t>(lo), static_cast<uint32_t>(hi));
    word = finite ? __float_as_uint(amax / 448.0f) : 0x7FC00000u;
  } else {
    const int e = e8m0_exponent<8>(finite ? m : 0);
    const float sbits = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    v2s lo = {0, 0}, hi = {0, 0};
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(v2bf, w[0]), sbits, false);
    lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(lo, __builtin_bit_cast(v2bf, w[1]), sbits, true);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(v2bf, w[2]), sbits, false);
    hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(hi, __builtin_bit_cast(v2bf, w[3]), sbits, true);
    codes = make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
    // the four quads' bytes into one word, in every lane
    word = (finite ? static_cast<uint32_t>(e + 127) : 0xFFu) << (8 * (l >> 2));
    word |= dpp(word, std::integral_constant<int, 0x128>{});
    word |= dpp(word, std::integral_constant<int, 0x124>{});
  }
  if (!finite) codes = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  if (raw >= a.units) return;
  *reinterpret_cast<uint2*>(a.xq + (static_cast<size_t>(kb) * a.rows + row) * kStageK + l * 8) = codes;
  if (l == 0) a.xs[row * ((a.KB + 3) & ~3u) + kb] = word;
}

// ----------------------------------------------------------------------- GEMM

constexpr uint32_t kNone = 0xFFFFFFF0u;    // an offset behind every resource

template <int HALF>
__device__ __forceinline__ v16f mfma_mx(const v8i& w, const v8i& x, const v16f& c, uint32_t sw, uint32_t sx) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, c, 0, 0, 2 * HALF, static_cast<int>(sw), 2 * HALF,
                                                         static_cast<int>(sx));
}

// Tiles of 256 rows take fewer MFMAs where they have fewer rows.
template <int BM>
constexpr bool kParts = BM == 256;

// WGM x WGN waves share a BM (rows) x BN (columns) tile; with WGK > 1 that many sets of them each take every WGK-th
// stage and their sums meet in LDS at the end.  Two super-stages of WGK x 128 K in LDS.
//
// v_mfma_scale_f32_32x32x64_f8f6f4, weight first: lane l holds row l % 32 of each operand, K [16q, 16q+16) and
// [32+16q, 32+16q+16) of the 64 with q = l / 32, and passes the scale of 32-K block q; its 16 results are the columns
// 8 (r / 4) + 4 q + r % 4 of activation row l % 32.
template <bool F32, int BM, int BN, int WGM, int WGN, int WGK>
__device__ __forceinline__ void grouped_gemm(const GemmArgs& p) {
  constexpr int NW = WGM * WGN * WGK;
  constexpr int WTM = BM / WGM, WTN = BN / WGN;        // a wave's sub-tile
  constexpr int JT = WTM / 32, IT = WTN / 32;          // its MFMA tiles
  constexpr int kSub = (BM + BN) * kStageK;            // bytes of one 128-K stage: W rows, then x rows
  constexpr int kStage = kSub * WGK;
  constexpr int A_INS = WGK * BM / 8, W_INS = WGK * BN / 8;   // DMA instructions of a super-stage (8 rows each)
  constexpr int APW = (A_INS + NW - 1) / NW, WPW = (W_INS + NW - 1) / NW;
  static_assert(IT * JT * 16 * 256 * (WGK - 1) * WGM * WGN <= kStage, "the partial sums fit a stage buffer");
  __shared__ __attribute__((aligned(1024))) uint8_t st0[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t st1[kStage];
  // scale words of two windows of four stages.  MXFP8: W rows, then x rows, four E8M0 bytes each.  FP32: the products
  // of an x row's scale with the column block's, for each of the tile's column blocks.
  constexpr int kCB = (BN + 127) / 128;
  constexpr int kScRows = F32 ? BM * kCB : BN + BM;
  __shared__ __attribute__((aligned(16))) uint32_t sc[2][4][kScRows];
  __shared__ int32_t src_row[BM];                      // x row of each tile row; -1: outside x

  // ---- the tile.  Workgroup i runs on XCD i % 8; every XCD takes a contiguous range of the tiles, ordered by expert,
  // band of row tiles, column tile, row tile, so that the tiles that share operands run together on one XCD's L2.
  const int total_mt = p.tiles ? p.tiles[0].count : (p.S + BM - 1) / BM;
  const int total = total_mt * p.n_tiles;
  const int per_xcd = (total + 7) >> 3;
  const int first_work = (blockIdx.x & 7) * per_xcd, mine = min(per_xcd, total - first_work);
  int slot = blockIdx.x >> 3;
  // Tiles of 256 rows come one to a compute unit, in rounds.  Where the last round would leave half of the compute
  // units idle, or three quarters, its tiles are cut into two or four parts of fewer rows, with fewer MFMAs for every
  // wave (640 tiles on 256 compute units, K = 4096: 223 -> 213 us; 576 tiles: 223 -> 217.  Halves that leave every
  // second wave without rows gained nothing).
  int part = 0, parts = 1;
  if constexpr (kParts<BM>) {
    const int rem = mine > 0 ? mine % p.wg_per_xcd : 0, cut = mine - rem;
    if (4 * rem <= p.wg_per_xcd)
      parts = 4;
    else if (2 * rem <= p.wg_per_xcd)
      parts = 2;
    if (slot >= cut) {
      part = (slot - cut) & (parts - 1);
      slot = cut + (slot - cut) / parts;
    } else {
      parts = 1;
    }
  }
  if (slot >= mine) return;
  const int work = first_work + slot;
  int e = 0, row_lo = 0, row_hi = p.S, first = 0, count = total_mt;
  if (p.tiles) {
    const RowTile t = p.tiles[1 + work / p.n_tiles];
    e = __builtin_amdgcn_readfirstlane(t.expert);
    first = __builtin_amdgcn_readfirstlane(t.first);
    count = __builtin_amdgcn_readfirstlane(t.count);
    row_lo = __builtin_amdgcn_readfirstlane(t.row_lo);
    row_hi = __builtin_amdgcn_readfirstlane(t.row_hi);
  }
  // Within a group, bands of 6 row tiles: the 32 tiles that an XCD holds at once then share 12 operand tiles, not 33
  // (8192 rows, N = 5120, K = 4096, FP32 scales: 205 -> 196 us; bands of 4 or 8: 198).
  constexpr int kBand = 6;
  const int local = work - first * p.n_tiles, band = local / (kBand * p.n_tiles);
  const int in_band = local - band * kBand * p.n_tiles, height = min(kBand, count - band * kBand);
  int mt = band * kBand + in_band % height, nt = in_band / height;
  mt = __builtin_amdgcn_readfirstlane(mt);
  nt = __builtin_amdgcn_readfirstlane(nt);
  const int bm = BM / __builtin_amdgcn_readfirstlane(parts);           // rows of the tile, or of its part
  const int row0 = row_lo + mt * BM + __builtin_amdgcn_readfirstlane(part) * bm, n0 = nt * BN;
  const int rows = min(bm, row_hi - row0), cols = min(BN, p.N - n0);
  if (rows <= 0) return;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave % WGN, wm = (wave / WGN) % WGM, wk = wave / (WGN * WGM);
  const int r32 = lane & 31, q2 = lane >> 5;
  const int KB = p.KB, KS = (KB + WGK - 1) / WGK;
  const int jt = kParts<BM> ? (rows + 32 * WGM - 1) / (32 * WGM) : JT, wtm = 32 * jt;   // a wave's MFMA tiles, its rows

  for (int r = tid; r < BM; r += 64 * NW) {
    const int rr = row0 + min(r, rows - 1);            // rows behind the tile's last re-read it
    int s = rr;
    if (p.row_slot) {
      const int slot_id = p.row_slot[rr];
      s = slot_id < 0 ? -1 : static_cast<int>(div_u32(static_cast<uint32_t>(slot_id), p.k_div));
    }
    src_row[r] = s >= p.rows ? -1 : s;
  }
  __syncthreads();

  // ---- DMA sources.  Instruction i of an operand moves 8 rows x 128 bytes: stage i / (rows / 8) of the super-stage,
  // rows 8 (i % (rows / 8)).. of the tile.  Where there are fewer instructions than waves some repeat another's.
  const uint32_t slab = static_cast<uint32_t>(p.rows) * kStageK;   // bytes of a K block of the activation
  const __amdgpu_buffer_rsrc_t ares = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.xq), 0, static_cast<int>(static_cast<uint32_t>(KB) * slab), kBufferFlags);
  const __amdgpu_buffer_rsrc_t wres = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(p.w + (static_cast<size_t>(e) * p.N + n0) * p.K), 0, cols * p.K, kBufferFlags);
  // The rows of an instruction are a scalar offset in the weight (a tile's rows begin at a multiple of 16, so a lane's
  // chunk is the same for all of them), and gathered ones in the activation.
  uint32_t offA[APW], noneW[WPW];
  int ldsA[APW], ldsW[WPW], subA[APW], subW[WPW], rowW[WPW];
#pragma unroll
  for (int u = 0; u < APW; ++u) {
    const int i = (wave + u * NW) % A_INS, sub = i / (BM / 8), rg = i % (BM / 8);
    const int r = rg * 8 + (lane >> 3);
    // rows behind the tile's last are not fetched (an offset behind the resource): an MFMA's rows are independent
    offA[u] = r < rows ? static_cast<uint32_t>(max(src_row[r], 0)) * kStageK + ((lane & 7) ^ swz8(r)) * 16 : kNone;
    subA[u] = sub;
    ldsA[u] = sub * kSub + BN * kStageK + rg * 8 * kStageK;
  }
  static_assert(NW % 2 == 0 && BN % 16 == 0, "every instruction of a wave begins at the same row of 16");
  const uint32_t dmaW = static_cast<uint32_t>(lane >> 3) * static_cast<uint32_t>(p.K);
  const uint32_t chW = ((lane & 7) ^ swz8((wave & 1) * 8 + (lane >> 3))) * 16;
#pragma unroll
  for (int u = 0; u < WPW; ++u) {
    const int i = (wave + u * NW) % W_INS, sub = i / (BN / 8), rg = i % (BN / 8);
    // so are columns behind the tile's last (the bounds are checked against the bytes less the scalar offset, which
    // must not exceed them)
    rowW[u] = rg * 8 < cols ? rg * 8 * p.K : 0;
    noneW[u] = rg * 8 < cols ? 0u : kNone;
    subW[u] = sub;
    ldsW[u] = sub * kSub + rg * 8 * kStageK;
  }
  constexpr int kWindow = 4 / WGK;                     // super-stages whose scales are brought together
  const int windows = (KS + kWindow - 1) / kWindow;
  // Chunks of the weight at or behind K re-read the row's last one: the activation's codes there are zero.  A
  // super-stage behind the last is asked for all the same, at offsets behind the resources: nothing is fetched.
  auto issue = [&](uint8_t* buf, int ks) {
    uint32_t behind = ks < KS ? 0u : kNone;
    asm("" : "+s"(behind));                           // or-ed in: as a choice of offsets it became branches
#pragma unroll
    for (int u = 0; u < WPW; ++u) {
      const uint32_t k = min(static_cast<uint32_t>((ks * WGK + subW[u]) * kStageK) + chW, static_cast<uint32_t>(p.K - 16));
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wres, (lds_void_t*)(buf + ldsW[u]), 16, (dmaW + k) | noneW[u] | behind,
                                               rowW[u], 0, 0);
    }
#pragma unroll
    for (int u = 0; u < APW; ++u) {
      const int kb = min(ks * WGK + subA[u], KB - 1);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ares, (lds_void_t*)(buf + ldsA[u]), 16, offA[u] | behind,
                                               static_cast<int>(static_cast<uint32_t>(kb) * slab), 0, 0);
    }
  };

  // ---- scales: thread t owns rows t, t + threads, .. of the tile's operands (W rows, then x rows; FP32: x rows alone)
  // and brings four stages' words at a time, one window ahead.  (One word per row, lane and stage, gathered by every
  // wave for itself, took the address unit longer than the operands: 1945 against 1607 us for 65536 rows, N = 4608,
  // K = 5120 without any scale loads.)
  constexpr int kScOwn = F32 ? BM : BN + BM;
  constexpr int SPT = (kScOwn + 64 * NW - 1) / (64 * NW);
  const int K32 = p.K / 32, NB = (p.N + 127) / 128;
  struct Words { uint32_t v[4]; };
  Words own[SPT], colw[F32 ? kCB : 1];
  // A thread's row of scale words, 4 bytes a stage for either operand.  A window is one 16-byte load, unconditional, so
  // that nothing waits for it before it is stored a window later.  An x row is whole windows; a W row's load may reach
  // behind the row, and is moved back to end with the tensor (undone when it is stored).
  const size_t wrow = static_cast<size_t>(e) * p.N + n0;               // the tile's first W row
  const uint8_t* const wsp = static_cast<const uint8_t*>(p.ws) + wrow * K32;
  const uint32_t room = F32 ? 0 : static_cast<uint32_t>(min((static_cast<size_t>(p.E) * p.N - wrow) * K32,
                                                            static_cast<size_t>(1) << 31)) - 16;   // last place of a load
  uint32_t soff[SPT];                                                  // the row's offset from wsp, or from xs
#pragma unroll
  for (int u = 0; u < SPT; ++u) {
    const int t = min(tid + u * 64 * NW, kScOwn - 1);
    if (!F32 && t < BN)
      soff[u] = static_cast<uint32_t>(min(t, cols - 1)) * static_cast<uint32_t>(K32);
    else
      soff[u] = static_cast<uint32_t>(max(src_row[F32 ? t : t - BN], 0)) * static_cast<uint32_t>((KB + 3) & ~3) * 4;
  }
  auto load_scales = [&](int win) {
    const int kb = 4 * win;
    const uint8_t* const xsp = reinterpret_cast<const uint8_t*>(p.xs);
#pragma unroll
    for (int u = 0; u < SPT; ++u) {
      const uint32_t at = soff[u] + static_cast<uint32_t>(16 * win);
      const bool is_w = !F32 && tid + u * 64 * NW < BN;
      __builtin_memcpy(&own[u], is_w ? wsp + min(at, room) : xsp + at, 16);
    }
    if constexpr (F32) {
#pragma unroll
      for (int c = 0; c < kCB; ++c) {
        const const_u32 src = (const_u32)(uintptr_t)(static_cast<const uint32_t*>(p.ws) +
                                                     (static_cast<size_t>(e) * NB + min(n0 / 128 + c, NB - 1)) * KB + kb);
#pragma unroll
        for (int q = 0; q < 4; ++q) colw[c].v[q] = src[min(q, KB - 1 - kb)];
      }
    }
  };
  auto store_scales = [&](int win, int buf) {
    const int left = K32 - 16 * win;                   // 32-K blocks of the row from this window on
#pragma unroll
    for (int u = 0; u < SPT; ++u) {
      const int t = tid + u * 64 * NW;
      if constexpr (!F32) {
        const int back = static_cast<int>(soff[u] + static_cast<uint32_t>(16 * win) - room);
        if (t < BN && back > 0) {                      // the tensor's last rows
          uint64_t v[2];
          __builtin_memcpy(v, &own[u], 16);
          const int sh = 8 * back;
          v[0] = sh < 64 ? v[0] >> sh | v[1] << (64 - sh) : v[1] >> (sh - 64);
          v[1] = sh < 64 ? v[1] >> sh : 0;
          __builtin_memcpy(&own[u], v, 16);
        }
        // blocks behind K: 2^-127, not the next row's scale (which may be NaN); their codes are zero
        if (left < 16) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int b = left - 4 * q;
            own[u].v[q] &= b >= 4 ? 0xFFFFFFFFu : b <= 0 ? 0u : (1u << (8 * b)) - 1;
          }
        }
      }
      if (t >= kScOwn) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (F32) {
#pragma unroll
          for (int c = 0; c < kCB; ++c)
            sc[buf][q][c * BM + t] = __float_as_uint(__uint_as_float(own[u].v[q]) * __uint_as_float(colw[c].v[q]));
        } else {
          sc[buf][q][t] = own[u].v[q];
        }
      }
    }
  };
  // scale words of this wave's MFMA tiles for stage q of the window in a buffer
  auto read_scales = [&](int buf, int q, uint32_t (&sw)[IT], uint32_t (&sx)[JT]) {
    const uint32_t* const row = sc[buf][q];
#pragma unroll
    for (int j = 0; j < JT; ++j)
      sx[j] = row[(F32 ? wn * WTN / 128 * BM : BN) + wm * wtm + 32 * j + r32];
    if constexpr (!F32) {
#pragma unroll
      for (int i = 0; i < IT; ++i) sw[i] = row[wn * WTN + 32 * i + r32];
    }
  };

  v16f acc[IT][JT];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int j = 0; j < JT; ++j) acc[i][j] = v16f{};

  // A lane's 16-byte chunks of a row, 4 half + q and 4 half + q + 2, at chunk ^ sz: their places differ in bits 5 and 6
  // alone.
  const int sz = swz8(r32);
  const int rd0 = wk * kSub + r32 * kStageK + ((q2 ^ sz) << 4);
  const int rdW = wn * WTN * kStageK, rdA = (BN + wm * wtm) * kStageK;
  auto frag = [&](const uint8_t* base, int half) {
    const uint4 lo = *reinterpret_cast<const uint4*>(base + (rd0 ^ (64 * half)));
    const uint4 hi = *reinterpret_cast<const uint4*>(base + (rd0 ^ (64 * half + 32)));
    v8i v;
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    return v;
  };
  const bool has_rows = wm * wtm < rows && wn * WTN < cols;   // a wave without output of its own only moves data
  // over the wave's first J row tiles
  auto compute = [&](auto J, const uint8_t* buf, int ks, const uint32_t (&sw)[IT], const uint32_t (&sx)[JT]) {
    if (!has_rows || ks * WGK + wk >= KB) return;
    constexpr int n = decltype(J)::value;
    if constexpr (F32) {
      // A tile's fma's are issued under the next one's MFMAs, and the reads of the next x rows between two MFMAs (one
      // after the other: 245 us against 228 at 16384 rows, N = 2304, K = 4096).
      v8i fw[IT][2], fx[2][2];
      v16f part[2];
      auto read_w = [&](int i) {
        fw[i][0] = frag(buf + rdW + 32 * i * kStageK, 0);
        fw[i][1] = frag(buf + rdW + 32 * i * kStageK, 1);
      };
      auto read_x = [&](int j) {
        fx[j & 1][0] = frag(buf + rdA + 32 * j * kStageK, 0);
        fx[j & 1][1] = frag(buf + rdA + 32 * j * kStageK, 1);
      };
      auto add = [&](int t) {
        const float s = __uint_as_float(sx[t / IT]);
#pragma unroll
        for (int r = 0; r < 16; ++r)
          acc[t % IT][t / IT][r] = __builtin_fmaf(part[t & 1][r], s, acc[t % IT][t / IT][r]);
      };
      read_w(0);
      read_x(0);
#pragma unroll
      for (int t = 0; t < IT * n; ++t) {
        const int i = t % IT, j = t / IT;
        __builtin_amdgcn_sched_barrier(0);
        part[t & 1] = mfma_mx<0>(fw[i][0], fx[j & 1][0], v16f{}, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        if (j == 0 && i + 1 < IT) read_w(i + 1);
        if (i == IT - 1 && j + 1 < n) read_x(j + 1);
        __builtin_amdgcn_sched_barrier(0);
        part[t & 1] = mfma_mx<0>(fw[i][1], fx[j & 1][1], part[t & 1], 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        __builtin_amdgcn_sched_barrier(0);
        if (t > 0) add(t - 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      add(IT * n - 1);
    } else {
      // lane group q passes block 2 half + q of the stage: byte 0 (half 0) or 2 (half 1) of the word moved down by q
      uint32_t swq[IT], sxq[JT];
#pragma unroll
      for (int i = 0; i < IT; ++i) swq[i] = sw[i] >> (8 * q2);
#pragma unroll
      for (int j = 0; j < JT; ++j) sxq[j] = sx[j] >> (8 * q2);
      auto half = [&](auto H) {
        constexpr int h = decltype(H)::value;
        v8i fw[IT], fx[n];
#pragma unroll
        for (int i = 0; i < IT; ++i) fw[i] = frag(buf + rdW + 32 * i * kStageK, h);
#pragma unroll
        for (int j = 0; j < n; ++j) fx[j] = frag(buf + rdA + 32 * j * kStageK, h);
#pragma unroll
        for (int j = 0; j < n; ++j)
#pragma unroll
          for (int i = 0; i < IT; ++i) acc[i][j] = mfma_mx<h>(fw[i], fx[j], acc[i][j], swq[i], sxq[j]);
      };
      half(std::integral_constant<int, 0>{});
      half(std::integral_constant<int, 1>{});
    }
  };

  // ---- ring.  At the top of step ks its DMA is in flight.
  issue(st0, 0);
  load_scales(0);
  auto ring = [&](auto J) {
    auto step = [&](const uint8_t* buf, uint8_t* refill, int ks) {
      const int win = ks / kWindow, wbuf = win & 1;
      const bool window = ks % kWindow == 0;
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(wait_vm_only(0));
      if (window) store_scales(win, wbuf);
      __builtin_amdgcn_s_waitcnt(kWaitLgkmOnly);         // the scales are written; reads of the buffer before are done
      __builtin_amdgcn_s_barrier();                      // super-stage ks is in LDS; the buffer before it is free
      __builtin_amdgcn_sched_barrier(0);
      uint32_t sw[IT], sx[JT];
      read_scales(wbuf, (ks * WGK + wk) & 3, sw, sx);
      if (window) load_scales(min(win + 1, windows - 1));
      __builtin_amdgcn_sched_barrier(0);                 // the loads go out before the DMA, and are waited for before it
      issue(refill, ks + 1);
      __builtin_amdgcn_sched_barrier(0);
      compute(J, buf, ks, sw, sx);
      __builtin_amdgcn_sched_barrier(0);
    };
    for (int ks = 0; ks < KS; ks += 2) {
      step(st0, st1, ks);
      if (ks + 1 < KS) step(st1, st0, ks + 1);
    }
  };
  if constexpr (kParts<BM>) {
    static_assert(JT == 4, "the cases");
    if (jt == 1)
      ring(std::integral_constant<int, 1>{});
    else if (jt == 2)
      ring(std::integral_constant<int, 2>{});
    else if (jt == 3)
      ring(std::integral_constant<int, 3>{});
    else
      ring(std::integral_constant<int, 4>{});
  } else {
    ring(std::integral_constant<int, JT>{});
  }

  __builtin_amdgcn_s_waitcnt(wait_vm_only(0));         // no DMA outlives the tile or meets the sums below

  // ---- the WGK partial sums, added in order by the first set of waves
  if constexpr (WGK > 1) {
    __syncthreads();
    float* const red = reinterpret_cast<float*>(st0);
    const int set = wave % (WGM * WGN);
    if (wk > 0) {
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int j = 0; j < JT; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            red[((((wk - 1) * WGM * WGN + set) * IT + i) * JT + j) * 1024 + r * 64 + lane] = acc[i][j][r];
    }
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
      for (int j = 0; j < JT; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          for (int s = 0; s < WGK - 1; ++s)
            acc[i][j][r] += red[((((s * WGM * WGN) + set) * IT + i) * JT + j) * 1024 + r * 64 + lane];
  }

  // ---- out.  The lanes l and l + 32 hold alternating groups of four columns of one row: a swap of every second
  // register pair leaves lane l columns 16 p .. 16 p + 7 and lane l + 32 columns 16 p + 8 .. 16 p + 15.
#pragma unroll
  for (int j = 0; j < JT; ++j) {
    if (kParts<BM> && j >= jt) break;
    const int m = wm * wtm + 32 * j + r32;
    const bool bad = src_row[m] < 0;
    uint16_t* const orow = p.out + static_cast<size_t>(row0 + m) * p.N;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const v16f& v = acc[i][j];
#pragma unroll
      for (int pp = 0; pp < 2; ++pp) {
        const uint32_t x0 = pack_bf16x2(v[8 * pp + 0], v[8 * pp + 1]), x1 = pack_bf16x2(v[8 * pp + 2], v[8 * pp + 3]);
        const uint32_t y0 = pack_bf16x2(v[8 * pp + 4], v[8 * pp + 5]), y1 = pack_bf16x2(v[8 * pp + 6], v[8 * pp + 7]);
        const auto s0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
        const auto s1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
        const int n = wn * WTN + 32 * i + 16 * pp + 8 * q2;
        uint4 o = make_uint4(s0[0], s1[0], s0[1], s1[1]);
        if (bad) o = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
        if (m < rows && n < cols) *reinterpret_cast<uint4*>(orow + n0 + n) = o;
      }
    }
  }
}

template <bool F32, int BM, int BN, int WGM, int WGN, int WGK>
__global__ __launch_bounds__(64 * WGM * WGN * WGK, 1) void grouped_gemm_kernel(GemmArgs p) {
  grouped_gemm<F32, BM, BN, WGM, WGN, WGK>(p);
}

// ------------------------------------------------------------------- dispatch

struct Shape {
  int BM, BN;
  bool split = false;          // the waves split over K
  bool large = false;          // 256 x 256: grouped_large.hip where it can
};

// The tile for S rows of E groups, by the rows of an average group (the groups' sizes are known on the device alone)
// and the tiles that makes for 256 compute units.  Measured on one MI355X, whole calls, us:
//   <= 32 rows: grouped_stream.hip (32 groups of a row, N = 4608, K = 2304, MXFP8: 69 against 79 with 128 x 128; 16
//     groups of 8 rows, N = K = 2048: 18.0 against 18.9), but not for short rows where a workgroup's share is more than
//     one of its tiles, whose few stages hide nothing: there 128 x 128 as below (8 groups, N = 3584, K = 1152: 16.3
//     against 13.7, K = 576: 14.4, 10.1; N = 2048: 10.2, 12.7 and 9.0, 9.5).
//   256 x 256 where it pads the average group by no more than a quarter over 128 x 128 and takes nine sixteenths of the
//     compute units, or 128 x 128 would not fit them in one round of two (8 groups of 192 rows, N = 5120, K = 4096,
//     MXFP8: 54 against 62; 640 rows: 130 against 162.  Else, 320 rows: 95 against 75; 128 tiles, 16 groups of 192
//     rows, N = K = 2048: 29.5 against 27.6).  With MXFP8 scales and groups of 1024 rows or more: grouped_large.hip (32
//     groups, N = 4608, K = 5120, groups of 2048 rows, more or less 25: 1608 against 1696; 1024 rows: 862 against 872;
//     512 rows: 499 against 490, its ragged tiles cost it more).
//   While the tiles are no more than the compute units: 64 x 64, 64 x 128 or 128 x 128 (the first that are), with the
//     waves split over K, four, two and two ways (FP32 scales, N = 5120, K = 4096, 256 rows: 27.6, 21.7, 26.3; 512
//     rows: 39.7, 39.2, 29.1; 128 x 128 with one set of waves 35.5; 8 groups of 100 rows, N = K = 2048, MXFP8: 20.5,
//     16.3, 17.9).
//   Else 128 x 128, two workgroups per compute unit, whose pauses cover each other (800 rows: 44 against 52 split; 48
//     rows a group, 32 groups, N = 5120, K = 2304: 98; 64 x 128 with three workgroups 106, 128 x 256 with one 109).
Shape pick_shape(int64_t S, int64_t E, int64_t N, int64_t K) {
  const int64_t groups = S < E ? S : E, per = (S + E - 1) / E;
  auto ceil_to = [](int64_t v, int64_t m) { return (v + m - 1) / m * m; };
  auto tiles = [&](int64_t bm, int64_t bn) { return groups * (ceil_to(per, bm) / bm) * (ceil_to(N, bn) / bn); };
  if (per <= 32) return K <= 1152 && tiles(128, 128) > 128 ? Shape{128, 128} : Shape{32, 64};
  if (4 * ceil_to(per, 256) <= 5 * ceil_to(per, 128) && (tiles(256, 256) >= 144 || tiles(128, 128) > 512))
    return {256, 256, false, per >= 1024};
  if (tiles(64, 64) <= 256) return {64, 64, true};
  if (tiles(64, 128) <= 256) return {64, 128, true};
  return {128, 128, tiles(128, 128) <= 256};
}

int64_t max_row_tiles(int64_t S, int64_t E, int BM) { return S / BM + (S < E ? S : E); }

size_t align_up(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

template <bool F32>
void launch_gemm(const Shape s, const GemmArgs& a, int64_t tiles, hipStream_t stream) {
  const unsigned per_xcd = static_cast<unsigned>((tiles + 7) / 8);
  if (s.BM == 64 && s.BN == 64)
    grouped_gemm_kernel<F32, 64, 64, 1, 2, 4><<<8 * per_xcd, 512, 0, stream>>>(a);
  else if (s.BM == 64)
    grouped_gemm_kernel<F32, 64, 128, 2, 2, 2><<<8 * per_xcd, 512, 0, stream>>>(a);
  else if (s.BM == 128 && s.split)
    grouped_gemm_kernel<F32, 128, 128, 2, 2, 2><<<8 * per_xcd, 512, 0, stream>>>(a);
  else if (s.BM == 128)
    grouped_gemm_kernel<F32, 128, 128, 2, 2, 1><<<8 * per_xcd, 256, 0, stream>>>(a);
  else                                                 // and up to one more round of parts
    grouped_gemm_kernel<F32, 256, 256, 2, 4, 1><<<8 * (per_xcd + a.wg_per_xcd), 512, 0, stream>>>(a);
}

}  // namespace

size_t grouped_workspace_bytes(int64_t rows, int64_t S, int64_t E, int64_t N, int64_t K) {
  if (rows <= 0 || S <= 0 || E <= 0) return 0;
  const int64_t KB = (K + kStageK - 1) / kStageK;
  const Shape s = pick_shape(S, E, N, K);
  return align_up(sizeof(RowTile) * (1 + max_row_tiles(S, E, s.BM))) + align_up(rows * KB * kStageK) +
         align_up(rows * ((KB + 3) / 4 * 4) * 4);
}

mx_status launch_grouped(const void* x, int64_t rows, const uint8_t* w, const void* ws, bool f32, bool act,
                         const int32_t* offsets, const int32_t* row_slot, int32_t k, int64_t S, int64_t E, int64_t N,
                         int64_t K, void* out, void* workspace, hipStream_t stream, const char* what) {
  const int64_t KB = (K + kStageK - 1) / kStageK;
  const Shape s = pick_shape(S, E, N, K);
  const int64_t mt = max_row_tiles(S, E, s.BM);
  uint8_t* at = static_cast<uint8_t*>(workspace);
  RowTile* const tiles = reinterpret_cast<RowTile*>(at);
  at += align_up(sizeof(RowTile) * (1 + mt));
  uint8_t* const xq = at;
  at += align_up(rows * KB * kStageK);
  uint32_t* const xs = reinterpret_cast<uint32_t*>(at);

  QuantRowsArgs q{};
  q.x = static_cast<const uint16_t*>(x);
  q.xq = xq;
  q.xs = xs;
  q.rows = static_cast<uint32_t>(rows);
  q.K = static_cast<uint32_t>(K);
  q.KB = static_cast<uint32_t>(KB);
  q.units = static_cast<uint32_t>(rows * KB);
  q.kb_div = make_div(static_cast<uint32_t>(KB));
  q.offsets = offsets;
  q.tiles = tiles;
  q.E = static_cast<int32_t>(E);
  q.S = static_cast<int32_t>(S);
  q.BM = s.BM;
  q.max_tiles = static_cast<int32_t>(mt);
  const unsigned qgrid = (q.units + 15) / 16 + (offsets ? 1 : 0);
  if (f32 && act)
    quant_rows_kernel<true, true><<<qgrid, 256, 0, stream>>>(q);
  else if (f32)
    quant_rows_kernel<true, false><<<qgrid, 256, 0, stream>>>(q);
  else if (act)
    quant_rows_kernel<false, true><<<qgrid, 256, 0, stream>>>(q);
  else
    quant_rows_kernel<false, false><<<qgrid, 256, 0, stream>>>(q);
  mx_status st = launch_status(what);
  if (st != MX_OK) return st;

  GemmArgs g{};
  g.xq = xq;
  g.xs = xs;
  g.w = w;
  g.ws = ws;
  g.out = static_cast<uint16_t*>(out);
  g.tiles = offsets ? tiles : nullptr;
  g.row_slot = row_slot;
  g.k_div = make_div(static_cast<uint32_t>(k));
  g.rows = static_cast<int32_t>(rows);
  g.S = static_cast<int32_t>(S);
  g.E = static_cast<int32_t>(E);
  g.N = static_cast<int32_t>(N);
  g.K = static_cast<int32_t>(K);
  g.KB = static_cast<int32_t>(KB);
  g.wg_per_xcd = device_cu_count() >= 8 ? device_cu_count() / 8 : 1;
  g.n_tiles = static_cast<int32_t>((N + s.BN - 1) / s.BN);
  const int64_t total = (offsets ? mt : (S + s.BM - 1) / s.BM) * g.n_tiles;
  if (s.BM == 32)
    launch_grouped_stream(f32, g, stream);
  else if (s.large && !f32 && KB >= kLargeMinStages)
    launch_grouped_large(g, stream);
  else if (f32)
    launch_gemm<true>(s, g, total, stream);
  else
    launch_gemm<false>(s, g, total, stream);
  return launch_status(what);
}

}  // namespace mx
