// How the attention of one new token for each sequence is shared among workgroups (gfx950; not part of the ABI).
//
// A stream is one (sequence, key head, block of its query heads).  Its keys are cut into tiles, the tiles of all streams
// are numbered, sequence by sequence, and every workgroup takes an equal share of consecutive ones: a long sequence is
// spread over many workgroups, many short ones share one.  A stream that a workgroup does not cover whole leaves its
// part (O, m, l) in the workspace, at most two of them for a workgroup: in place 0 where the share begins inside the stream,
// in place 1 where it ends inside one that it holds from its first tile.  A second kernel joins the parts.
#pragma once

#include "kv_cache.hpp"

namespace mx {

struct DecodeArgs {
  KvCache c;
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* lens;
  uint16_t* out;
  float* parts;              // [groups][2][O: heads x D, then m and l]
  uint32_t* plan;            // [0] share, [1 + b] first tile of sequence b
  float scale;               // times log2(e)
  uint32_t B, H, G;          // G query heads a key head
  uint32_t streams;          // a sequence's: Hkv * head_blocks
  uint32_t head_blocks;
};

// Tokens of sequence b, cut to what its table holds.
__device__ __forceinline__ uint32_t tokens_of(const DecodeArgs& a, uint32_t b) {
  return min(static_cast<uint32_t>(max(a.lens[b], 0)), a.c.max_pages << a.c.page_shift);
}

// Sum over the workgroup of the threads' v, and the sum of those before this thread.
template <int THREADS>
__device__ __forceinline__ uint32_t scan(uint32_t v, uint32_t* buf, uint32_t& before) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) buf[wave] = x;
  __syncthreads();
  uint32_t sum = 0, base = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    if (w < wave) base += buf[w];
    sum += buf[w];
  }
  before = base + x - v;
  return sum;
}

// A workgroup's share: tiles t .. end - 1, the first of them of sequence b, whose tiles begin at `first`.
struct Share {
  uint32_t t, end, b, first;
};

// One stream's stretch of a share.
struct Piece {
  uint32_t kvh, h0, heads;   // key head, first query head, how many
  uint32_t tile0, tiles, of; // of the stream's `of`
};

// All threads of the workgroup; t == end: nothing to do.
template <int TILE, int THREADS>
__device__ __forceinline__ Share find_share(const DecodeArgs& a) {
  __shared__ uint32_t buf[THREADS / 64], found[2];
  auto tiles = [&](uint32_t b) { return b < a.B ? (tokens_of(a, b) + TILE - 1) / TILE : 0u; };
  uint32_t total = 0;
  for (uint32_t b0 = 0; b0 < a.B; b0 += THREADS) {
    const uint32_t b = b0 + threadIdx.x;
    uint32_t before;
    const uint32_t sum = scan<THREADS>(tiles(b), buf, before);
    if (blockIdx.x == 0 && b < a.B) a.plan[1 + b] = (total + before) * a.streams;
    total += sum;
  }
  total *= a.streams;
  const uint32_t share = max((total + gridDim.x - 1) / gridDim.x, 1u);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.plan[0] = share;
  Share s;
  s.t = blockIdx.x * share;
  s.end = min(s.t + share, total);
  if (s.t >= total) {
    s.end = s.t;
    return s;
  }
  uint32_t done = 0;
  for (uint32_t b0 = 0; b0 < a.B; b0 += THREADS) {
    const uint32_t b = b0 + threadIdx.x;
    uint32_t before;
    const uint32_t n = tiles(b);
    const uint32_t sum = scan<THREADS>(n, buf, before);
    const uint32_t first = (done + before) * a.streams;
    if (s.t >= first && s.t < first + n * a.streams) {
      found[0] = b;
      found[1] = first;
    }
    done += sum;
    if (s.t < done * a.streams) break;
  }
  __syncthreads();
  s.b = __builtin_amdgcn_readfirstlane(found[0]);
  s.first = __builtin_amdgcn_readfirstlane(found[1]);
  return s;
}

// The piece at s.t, with HEADS query heads a block.
template <int TILE, int HEADS>
__device__ __forceinline__ Piece piece_of(const DecodeArgs& a, const Share& s) {
  Piece p;
  p.of = (tokens_of(a, s.b) + TILE - 1) / TILE;
  const uint32_t x = (s.t - s.first) / p.of;
  p.tile0 = (s.t - s.first) - x * p.of;
  p.tiles = min(p.of - p.tile0, s.end - s.t);
  p.kvh = x / a.head_blocks;
  p.h0 = p.kvh * a.G + (x - p.kvh * a.head_blocks) * HEADS;
  p.heads = min(static_cast<uint32_t>(HEADS), (p.kvh + 1) * a.G - p.h0);
  return p;
}

// Past the piece, to the next sequence that has tokens if this one's streams are done and the share is not.
__device__ __forceinline__ void advance(const DecodeArgs& a, Share& s, const Piece& p) {
  s.t += p.tiles;
  if (s.t == s.first + p.of * a.streams && s.t < s.end) {
    s.first = s.t;
    do ++s.b; while (tokens_of(a, s.b) == 0);            // a tile is left, so a sequence that has one
  }
}

// Where the part of a piece that is not its stream's whole goes.
__device__ __forceinline__ float* part_of(const DecodeArgs& a, uint32_t group, bool begins, uint32_t size) {
  return a.parts + (static_cast<size_t>(group) * 2 + (begins ? 1 : 0)) * size;
}

}  // namespace mx
