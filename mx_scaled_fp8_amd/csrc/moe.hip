// The router of a mixture of experts and the join of its experts' rows (gfx950): mx_moe_route, mx_moe_combine.
//
// Router.  Per token, the k experts of largest key, their weights, and then all T * k slots grouped by expert:
//
//   l' = l, NaN taken as -inf, +inf as the largest finite FP32 (-inf masks an expert out)
//   p  = softmax(l') or 1 / (1 + exp(-l'));   key = l' without a bias, p + bias with one, -inf for masked experts
//   w_j = p_j / sum_j p_j * scale             (0 when the sum is 0: every expert masked)
//
// Without a bias both scores grow with l', so the logits themselves are compared and no rounding decides.  With one,
// keys are formed in FP64, which leaves near-ties of different scores to the exact order.  Equal keys: lowest index.
//
// Two launches, bound by latency (a few kilobytes to a few megabytes):
//  * route_topk_kernel: a wave per token, each lane holding E / 64 consecutive experts, k rounds of a wave-wide
//    maximum over order-preserving integer keys; the workgroup's tokens form a chunk whose experts it counts in LDS.
//  * route_scatter_kernel: a workgroup per chunk.  Thread e sums the counts of expert e over all chunks (its start)
//    and over the chunks before (its place), then walks the chunk's slots in order, so the order within an expert is
//    the slots' own without any atomics on positions.
// With one chunk the first kernel does the second's work in LDS, in the same launch.
//
// Join.  out[t] = shared[t] + sum_j w[t, j] * y[slot_row[t, j]] in FP32, rounded once; bound by HBM.
#include "common.hpp"

namespace mx {

namespace {

constexpr int kRouteThreads = 1024;      // 16 waves, a token each at a time
constexpr int kChunkTokens = 64;         // tokens of a chunk, doubled until kMaxChunks suffice
constexpr int kMaxChunks = 256;
constexpr int kScanSlots = 2048;         // slots held in LDS at a time by the grouping
constexpr int kMaxExperts = 1024;

struct RouteArgs {
  const void* logits;       // [T, E] FP32 or BF16
  const float* bias;        // [E] or null
  int32_t* ids;             // [T, k]
  float* weights;           // [T, k]
  int32_t* offsets;         // [E + 1]
  int32_t* row_slot;        // [T * k]
  int32_t* slot_row;        // [T * k]
  int32_t* counts;          // [chunks, E]
  int32_t T, E, k;
  int32_t chunk_tokens, chunks;
  int32_t score, renormalize;
  float scale;
};

// order-preserving integers of floating-point values (-inf is above 0, which marks an expert already taken)
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
  return b >> 63 ? ~b : b | (uint64_t(1) << 63);
}
__device__ __forceinline__ float no_zero_sign(float v) { return v + 0.0f; }   // -0 and 0 are one key
__device__ __forceinline__ double no_zero_sign(double v) { return v + 0.0; }

template <typename V>
__device__ __forceinline__ V wave_max(V v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const V o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// One token by one wave.  V: the type of scores and keys (double with a bias), U its ordered integer, EI: experts per
// lane.  Lane j < k leaves with the token's j-th id.
template <typename V, typename U, int EI>
__device__ __forceinline__ int route_token(const RouteArgs& a, bool f32, int64_t t, int lane) {
  V l[EI], p[EI];
  U key[EI];
  const int e0 = lane * EI;
  const V ninf = -__builtin_inf();
  V top = ninf;
#pragma unroll
  for (int i = 0; i < EI; ++i) {
    const int e = e0 + i;
    float v = -__builtin_inff();
    if (e < a.E)
      v = f32 ? static_cast<const float*>(a.logits)[t * a.E + e]
              : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.logits)[t * a.E + e]) << 16);
    v = v != v ? -__builtin_inff() : fminf(v, __FLT_MAX__);
    l[i] = static_cast<V>(v);
    top = l[i] > top ? l[i] : top;
  }
  V total = 1;
  if (a.score == MX_ROUTE_SOFTMAX) {
    top = wave_max(top);
    total = 0;
#pragma unroll
    for (int i = 0; i < EI; ++i) {
      p[i] = l[i] == ninf ? V(0) : exp_of(l[i] - top);
      total += p[i];
    }
    total = wave_sum(total);
  } else {
#pragma unroll
    for (int i = 0; i < EI; ++i) p[i] = V(1) / (V(1) + exp_of(-l[i]));
  }
  const V inv = total > V(0) ? V(1) / total : V(0);
#pragma unroll
  for (int i = 0; i < EI; ++i) {
    p[i] *= inv;
    V v = l[i];
    if (a.bias != nullptr && v != ninf) {
      v = p[i] + static_cast<V>(a.bias[e0 + i]);
      if (v != v) v = ninf;
    }
    key[i] = e0 + i < a.E ? ordered(no_zero_sign(v)) : U(0);
  }

  int my_id = 0;
  V my_p = 0, sum = 0;
  for (int j = 0; j < a.k; ++j) {
    U best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < EI; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const U most = wave_max(best);
    const int owner = __ffsll(static_cast<unsigned long long>(__ballot(best == most))) - 1;   // lowest index of equals
    V pv = 0;
#pragma unroll
    for (int i = 0; i < EI; ++i)
      if (i == at) pv = p[i];
    const int id = __shfl(e0 + at, owner);
    pv = __shfl(pv, owner);
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < EI; ++i)
        if (i == at) key[i] = U(0);
    }
    sum += pv;
    if (lane == j) {
      my_id = id;
      my_p = pv;
    }
  }
  if (lane < a.k) {
    V w = my_p;
    if (a.renormalize) w = sum > V(0) ? w / sum : V(0);
    a.ids[t * a.k + lane] = my_id;
    a.weights[t * a.k + lane] = static_cast<float>(w * static_cast<V>(a.scale));
  }
  return my_id;
}

// Grouping of one chunk by a workgroup of kRouteThreads: thread e owns expert e.  `place` is where the chunk's first
// row of expert e goes.  The slots' experts are read from `ids` kScanSlots at a time.
__device__ __forceinline__ void scatter_chunk(const RouteArgs& a, int chunk, int place, uint16_t* lds_ids) {
  const int tid = threadIdx.x;
  const int64_t s0 = static_cast<int64_t>(chunk) * a.chunk_tokens * a.k;
  const int64_t all = static_cast<int64_t>(a.T) * a.k;
  const int64_t s1 = min(s0 + static_cast<int64_t>(a.chunk_tokens) * a.k, all);
  for (int64_t b = s0; b < s1; b += kScanSlots) {
    const int n = static_cast<int>(min(static_cast<int64_t>(kScanSlots), s1 - b));
    __syncthreads();
    for (int i = tid; i < kScanSlots; i += kRouteThreads)
      lds_ids[i] = i < n ? static_cast<uint16_t>(a.ids[b + i]) : static_cast<uint16_t>(0xFFFF);
    __syncthreads();
    if (tid < a.E) {
      for (int i = 0; i < n; i += 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(lds_ids + i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t id = q & 1 ? w[q >> 1] >> 16 : w[q >> 1] & 0xFFFFu;
          if (id == static_cast<uint32_t>(tid)) {
            const int32_t s = static_cast<int32_t>(b + i + q);
            a.row_slot[place] = s;
            a.slot_row[s] = place;
            ++place;
          }
        }
      }
    }
  }
}

// exclusive prefix sum over the workgroup
__device__ __forceinline__ int block_exclusive(int v, int* part) {
  const int tid = threadIdx.x;
  part[tid] = v;
  __syncthreads();
  for (int d = 1; d < kRouteThreads; d *= 2) {
    const int o = tid >= d ? part[tid - d] : 0;
    __syncthreads();
    part[tid] += o;
    __syncthreads();
  }
  return part[tid] - v;
}

template <int EI>
__global__ __launch_bounds__(kRouteThreads) void route_topk_kernel(RouteArgs a, int f32) {
  __shared__ int32_t hist[kMaxExperts];
  __shared__ int32_t part[kRouteThreads];
  __shared__ __attribute__((aligned(16))) uint16_t lds_ids[kScanSlots];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < kMaxExperts; e += kRouteThreads) hist[e] = 0;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.chunk_tokens;
  const int64_t t1 = min(t0 + a.chunk_tokens, static_cast<int64_t>(a.T));
  for (int64_t t = t0 + wave; t < t1; t += kRouteThreads / 64) {
    const int id = a.bias != nullptr ? route_token<double, uint64_t, EI>(a, f32 != 0, t, lane)
                                     : route_token<float, uint32_t, EI>(a, f32 != 0, t, lane);
    if (lane < a.k) atomicAdd(&hist[id], 1);
  }
  __syncthreads();                               // also orders the ids written above before scatter_chunk reads them
  if (a.chunks > 1) {
    for (int e = tid; e < a.E; e += kRouteThreads) a.counts[static_cast<int64_t>(blockIdx.x) * a.E + e] = hist[e];
    return;
  }
  const int n = tid < a.E ? hist[tid] : 0;
  const int first = block_exclusive(n, part);
  if (tid < a.E) a.offsets[tid] = first;
  if (tid == a.E - 1) a.offsets[a.E] = first + n;
  scatter_chunk(a, 0, first, lds_ids);
}

__global__ __launch_bounds__(kRouteThreads) void route_scatter_kernel(RouteArgs a) {
  __shared__ int32_t part[kRouteThreads];
  __shared__ __attribute__((aligned(16))) uint16_t lds_ids[kScanSlots];
  const int tid = threadIdx.x;
  int before = 0, n = 0;
  if (tid < a.E) {
    for (int c = 0; c < a.chunks; ++c) {
      const int v = a.counts[static_cast<int64_t>(c) * a.E + tid];
      before += c < static_cast<int>(blockIdx.x) ? v : 0;
      n += v;
    }
  }
  const int first = block_exclusive(n, part);
  if (blockIdx.x == 0) {
    if (tid < a.E) a.offsets[tid] = first;
    if (tid == a.E - 1) a.offsets[a.E] = first + n;
  }
  scatter_chunk(a, blockIdx.x, first + before, lds_ids);
}

// ----------------------------------------------------------------------- join

struct CombineArgs {
  const uint16_t* y;          // [rows, N] BF16
  const int32_t* slot_row;    // [T, k]
  const float* weights;       // [T, k]
  const uint16_t* shared;     // [T, N] or null
  uint16_t* out;              // [T, N]
  int32_t rows, k;
  uint32_t N8;                // N / 8
  uint64_t total;             // T * N8
};

// A thread owns 8 consecutive columns of one token.
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.total) return;
  const uint64_t t = i / a.N8;
  const uint32_t c = static_cast<uint32_t>(i - t * a.N8);
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (a.shared != nullptr) {
    const uint4 v = reinterpret_cast<const uint4*>(a.shared)[i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      s[2 * q] = bf16_lo(w[q]);
      s[2 * q + 1] = bf16_hi(w[q]);
    }
  }
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < a.k; ++j) {
    const int r = a.slot_row[t * a.k + j];
    const float wt = a.weights[t * a.k + j];
    if (r < 0 || r >= a.rows || wt == 0.f) continue;   // a dropped slot
    const uint4 v = reinterpret_cast<const uint4*>(a.y)[static_cast<uint64_t>(r) * a.N8 + c];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      sum[2 * q] = __builtin_fmaf(wt, bf16_lo(w[q]), sum[2 * q]);
      sum[2 * q + 1] = __builtin_fmaf(wt, bf16_hi(w[q]), sum[2 * q + 1]);
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(sum[2 * q] + s[2 * q], sum[2 * q + 1] + s[2 * q + 1]);
  reinterpret_cast<uint4*>(a.out)[i] = make_uint4(o[0], o[1], o[2], o[3]);
}

int route_chunk_tokens(int64_t T) {
  int64_t c = kChunkTokens;
  while ((T + c - 1) / c > kMaxChunks) c *= 2;
  return static_cast<int>(c);
}

}  // namespace

size_t route_workspace_bytes(int64_t T, int32_t E) {
  const int64_t c = route_chunk_tokens(T), chunks = (T + c - 1) / c;
  return chunks > 1 ? static_cast<size_t>(chunks) * E * 4 : 0;
}

mx_status launch_moe_route(const void* logits, int32_t f32, const float* bias, int64_t T, int32_t E, int32_t k,
                           int32_t score, int32_t renormalize, float scale, int32_t* ids, float* weights,
                           int32_t* offsets, int32_t* row_slot, int32_t* slot_row, void* workspace,
                           hipStream_t stream) {
  RouteArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.offsets = offsets;
  a.row_slot = row_slot;
  a.slot_row = slot_row;
  a.counts = static_cast<int32_t*>(workspace);
  a.T = static_cast<int32_t>(T);
  a.E = E;
  a.k = k;
  a.chunk_tokens = route_chunk_tokens(T);
  a.chunks = T > 0 ? static_cast<int32_t>((T + a.chunk_tokens - 1) / a.chunk_tokens) : 1;
  a.score = score;
  a.renormalize = renormalize;
  a.scale = scale;
  if (E <= 64)
    route_topk_kernel<1><<<a.chunks, kRouteThreads, 0, stream>>>(a, f32);
  else if (E <= 128)
    route_topk_kernel<2><<<a.chunks, kRouteThreads, 0, stream>>>(a, f32);
  else if (E <= 256)
    route_topk_kernel<4><<<a.chunks, kRouteThreads, 0, stream>>>(a, f32);
  else if (E <= 512)
    route_topk_kernel<8><<<a.chunks, kRouteThreads, 0, stream>>>(a, f32);
  else
    route_topk_kernel<16><<<a.chunks, kRouteThreads, 0, stream>>>(a, f32);
  mx_status st = launch_status("mx_moe_route");
  if (st != MX_OK || a.chunks == 1) return st;
  route_scatter_kernel<<<a.chunks, kRouteThreads, 0, stream>>>(a);
  return launch_status("mx_moe_route (grouping)");
}

mx_status launch_moe_combine(const void* y, int64_t rows, int64_t N, const int32_t* slot_row, const float* weights,
                             int64_t T, int32_t k, const void* shared, void* out, hipStream_t stream) {
  CombineArgs a{};
  a.y = static_cast<const uint16_t*>(y);
  a.slot_row = slot_row;
  a.weights = weights;
  a.shared = static_cast<const uint16_t*>(shared);
  a.out = static_cast<uint16_t*>(out);
  a.rows = static_cast<int32_t>(rows);
  a.k = k;
  a.N8 = static_cast<uint32_t>(N / 8);
  a.total = static_cast<uint64_t>(T) * a.N8;
  combine_kernel<<<static_cast<unsigned>((a.total + 255) / 256), 256, 0, stream>>>(a);
  return launch_status("mx_moe_combine");
}

}  // namespace mx
