// How the attention of one new token for each sequence is shared among workgroups (gfx950; not part of the ABI).
//
// A stream is one (sequence, key head).  Its keys are cut into tiles, the tiles of all streams are numbered, sequence by
// sequence, and every group takes an equal share of consecutive ones: a long sequence is spread over many groups, many
// short ones share one.  A group is as many workgroups as a key head has blocks of query heads; they read the same keys,
// and are dealt to the same XCD, whose L2 then has them for all.  A stream that a group does not cover whole leaves its part
// (O, m, l) in the workspace, at most two of them for a group: in place 0 where the share begins inside the stream, in
// place 1 where it ends inside one that it holds from its first tile.  A second kernel joins the parts.
#pragma once

#include "kv_cache.hpp"

namespace mx {

struct DecodeArgs {
  KvCache c;
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* lens;
  uint16_t* out;
  float* parts;              // [group][head block][2][O: part_heads x D, then m and l]
  uint32_t* plan;            // [0] share, [1 + b] first tile of sequence b
  float scale;               // times log2(e)
  uint32_t B, H, G;          // G query heads a key head
  uint32_t groups;           // up to 8 or a multiple of 8
  uint32_t head_blocks;
  uint32_t part_heads;       // up to a block's heads
};

// Tokens of sequence b, cut to what its table holds.
__device__ __forceinline__ uint32_t tokens_of(const DecodeArgs& a, uint32_t b) {
  return min(static_cast<uint32_t>(max(a.lens[b], 0)), a.c.max_pages << a.c.page_shift);
}

// A workgroup's share: tiles t .. end - 1, the first of them of sequence b, whose tiles begin at `first`, for one block of
// heads.
struct Share {
  uint32_t t, end, b, first, group, block;
};

// One stream's stretch of a share.
struct Piece {
  uint32_t kvh, h0, heads;   // key head, first query head, how many
  uint32_t tile0, tiles, of; // of the stream's `of`
};

// Every wave finds its workgroup's share by itself, 64 sequences at a time, without a barrier; t == end: nothing to do.
// A share is at least MIN tiles.  Workgroup 0 leaves the plan for the second kernel.
template <int TILE, int MIN>
__device__ __forceinline__ Share find_share(const DecodeArgs& a) {
  const uint32_t lane = threadIdx.x & 63;
  auto tiles = [&](uint32_t b) { return b < a.B ? (tokens_of(a, b) + TILE - 1) / TILE : 0u; };
  auto scan = [&](uint32_t x) {                        // sums up to and with each lane
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t y = __shfl_up(x, d);
      if (lane >= static_cast<uint32_t>(d)) x += y;
    }
    return x;
  };
  uint32_t total = 0, n = 0, upto = 0;
  for (uint32_t b0 = 0; b0 < a.B; b0 += 64) {
    n = tiles(b0 + lane);
    upto = scan(n);
    if (blockIdx.x == 0 && threadIdx.x < 64 && b0 + lane < a.B) a.plan[1 + b0 + lane] = (total + upto - n) * a.c.Hkv;
    total += __builtin_amdgcn_readlane(upto, 63);
  }
  const uint32_t all = total * a.c.Hkv;
  const uint32_t share = max((all + a.groups - 1) / a.groups, static_cast<uint32_t>(MIN));
  if (blockIdx.x == 0 && threadIdx.x == 0) a.plan[0] = share;
  // consecutive workgroups go to the XCDs in turn: the blocks of one group are 8 apart
  const uint32_t side = min(a.groups, 8u), x = blockIdx.x / side;
  Share s;
  s.block = x % a.head_blocks;
  s.group = x / a.head_blocks * side + blockIdx.x % side;
  s.t = s.group * share;
  s.end = min(s.t + share, all);
  s.b = s.first = 0;
  if (s.t >= all) {
    s.end = s.t;
    return s;
  }
  uint32_t done = 0;
  for (uint32_t b0 = 0;; b0 += 64) {                   // ends: s.t is below the sum of all
    if (a.B > 64) {                                    // of up to 64 sequences n and upto are still there
      n = tiles(b0 + lane);
      upto = scan(n);
    }
    const uint64_t behind = __ballot(s.t < (done + upto) * a.c.Hkv);
    if (behind != 0) {
      const int at = __builtin_ctzll(behind);
      s.b = b0 + at;
      s.first = (done + __builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(n, at)) * a.c.Hkv;
      return s;
    }
    done += __builtin_amdgcn_readlane(upto, 63);
  }
}

// The piece at s.t, with HEADS query heads a block.
template <int TILE, int HEADS>
__device__ __forceinline__ Piece piece_of(const DecodeArgs& a, const Share& s) {
  Piece p;
  p.of = (tokens_of(a, s.b) + TILE - 1) / TILE;
  const uint32_t x = (s.t - s.first) / p.of;
  p.tile0 = (s.t - s.first) - x * p.of;
  p.tiles = min(p.of - p.tile0, s.end - s.t);
  p.kvh = x;
  p.h0 = x * a.G + s.block * HEADS;
  p.heads = min(static_cast<uint32_t>(HEADS), (p.kvh + 1) * a.G - p.h0);
  return p;
}

// Past the piece, to the next sequence that has tokens if this one's streams are done and the share is not.
__device__ __forceinline__ void advance(const DecodeArgs& a, Share& s, const Piece& p) {
  s.t += p.tiles;
  if (s.t == s.first + p.of * a.c.Hkv && s.t < s.end) {
    s.first = s.t;
    do ++s.b; while (tokens_of(a, s.b) == 0);            // a tile is left, so a sequence that has one
  }
}

// Where the part of a piece that is not its stream's whole goes.
__device__ __forceinline__ float* part_of(const DecodeArgs& a, uint32_t group, uint32_t block, bool begins, uint32_t size) {
  return a.parts + ((static_cast<size_t>(group) * a.head_blocks + block) * 2 + (begins ? 1 : 0)) * size;
}

constexpr int kJoinThreads = 256;

// A workgroup joins the parts of one query head (blockIdx.x: sequence and head) that the workgroups left of its stream,
// zeros for a sequence of no tokens.  A stream that one workgroup covered is done already.  D / 4 threads take a part at a
// time, four of them under way, the others every so many-th of the others; their sums meet in LDS, in a fixed order.
template <int D, int TILE, int HEADS>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(DecodeArgs a) {
  constexpr uint32_t DT = D / 4, LANES = kJoinThreads / DT;
  __shared__ __attribute__((aligned(16))) float sum[LANES][D];
  __shared__ float tops[LANES], weights[LANES];
  const uint32_t b = blockIdx.x / a.H, h = blockIdx.x - b * a.H;
  const uint32_t kvh = h / a.G, block = (h - kvh * a.G) / HEADS, r = (h - kvh * a.G) - block * HEADS;
  const uint32_t heads = a.part_heads, share = a.plan[0], begin = a.plan[1 + b];
  const uint32_t nt = (tokens_of(a, b) + TILE - 1) / TILE;
  const uint32_t lane = threadIdx.x / DT, d = threadIdx.x % DT * 4;
  uint2* out = reinterpret_cast<uint2*>(a.out + (static_cast<size_t>(b) * a.H + h) * D + d);
  if (nt == 0) {
    if (lane == 0) *out = make_uint2(0, 0);
    return;
  }
  const uint32_t t0 = begin + kvh * nt;
  const uint32_t w0 = t0 / share, w1 = (t0 + nt - 1) / share;
  if (w0 == w1) return;
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (uint32_t w = w0 + lane; w <= w1; w += 4 * LANES) {
    float4 x[4];
    float pm[4], pl[4], top = m;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool some = w + k * LANES <= w1;
      const float* p = part_of(a, some ? w + k * LANES : w, block, w + k * LANES == w0 || (!some && w == w0), heads * (D + 2));
      x[k] = *reinterpret_cast<const float4*>(p + r * D + d);
      pm[k] = some ? p[heads * D + r] : -INFINITY;
      pl[k] = p[heads * D + heads + r];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) top = fmaxf(top, pm[k]);
    const float base = top == -INFINITY ? 0.0f : top, f = __builtin_amdgcn_exp2f(m - base);
    l *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (w + k * LANES <= w1) {
        const float g = __builtin_amdgcn_exp2f(pm[k] - base);
        l += pl[k] * g;
        o = make_float4(o.x + x[k].x * g, o.y + x[k].y * g, o.z + x[k].z * g, o.w + x[k].w * g);
      }
    m = top;
  }
  *reinterpret_cast<float4*>(&sum[lane][d]) = o;
  if (d == 0) {
    tops[lane] = m;
    weights[lane] = l;
  }
  __syncthreads();
  if (lane != 0) return;
  float top = -INFINITY;
#pragma unroll
  for (uint32_t k = 0; k < LANES; ++k) top = fmaxf(top, tops[k]);
  const float base = top == -INFINITY ? 0.0f : top;
  l = 0.0f;
  o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (uint32_t k = 0; k < LANES; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(&sum[k][d]);
    const float f = __builtin_amdgcn_exp2f(tops[k] - base);
    l += weights[k] * f;
    o = make_float4(o.x + x.x * f, o.y + x.y * f, o.z + x.z * f, o.w + x.w * f);
  }
  const float inv = 1.0f / l;
  *out = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
}

}  // namespace mx
