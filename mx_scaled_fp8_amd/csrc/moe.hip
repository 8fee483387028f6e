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
//  * route_topk_kernel: 16 or 64 lanes a token, each holding every 16th or 64th expert; k rounds of a maximum across
//    the lanes.  A workgroup takes a block of up to 64 tokens and notes in LDS, per expert, which
//    of them picked it: a 64-bit mask.
//  * route_scatter_kernel: the row of slot (t, j) is the number of slots of lower experts, plus those of its expert in
//    the blocks before (sums of the masks' bit counts), plus the bits below t in its own block's mask.  So the rows of
//    an expert are in slot order, and nothing is placed by the order of atomics.
// A single block does the second's work in the first launch.
// Measured (one MI355X, kernel times): 4 tokens, 64 experts, k = 6, BF16 logits: 4 us.  8192 tokens, 256 experts, k =
// 8, sigmoid with a bias: 10 and 6 us; the logits alone would take 2.  The rest is the scores (FP64 only for experts
// that an FP32 bound leaves in question: 83 us for all of them), k rounds of maxima, and the masks' way through memory.
//
// Join.  out[t] = shared[t] + sum_j w[t, j] * y[slot_row[t, j]] in FP32, rounded once; bound by HBM: 8192 tokens, k =
// 8, N = 5120 (839 MB) 140 us, 6.0 TB/s, with the loads of eight rows in flight and past the caches (one row at a time
// 186).
#include "common.hpp"

namespace mx {

namespace {

constexpr int kTopkThreads = 512;         // 32 tokens of 16 lanes at a time
constexpr int kScatterThreads = 1024;
constexpr int kBlockTokens = 64;         // most tokens of a block: the bits of its masks
constexpr int kMaxSpans = 256;           // workgroups of the second launch, each a run of blocks
constexpr int kMaxExperts = MX_ROUTE_MAX_EXPERTS;
static_assert(kMaxExperts == kScatterThreads && kMaxExperts == 2 * kTopkThreads, "experts per thread");

struct RouteArgs {
  const void* logits;       // [T, E] FP32 or BF16
  const float* bias;        // [E] or null
  int32_t* ids;             // [T, k]
  float* weights;           // [T, k]
  int32_t* offsets;         // [E + 1]
  int32_t* row_slot;        // [T * k]
  int32_t* slot_row;        // [T * k]
  uint64_t* masks;          // [blocks, E]
  uint32_t* counts;         // [blocks, E4 / 4], four experts' counts a word
  int32_t T, E, k;
  int32_t E4;               // E rounded up to 4
  int32_t block_tokens;     // tokens of a block, at most kBlockTokens
  int32_t blocks;
  int32_t span;             // blocks per workgroup of the second launch
  DivU32 k_div;
  int32_t score, renormalize;
  float scale;
};

// Keys.  Without a bias: the logit as an order-preserving integer (-inf, a masked expert, above 0, an expert already
// taken).  With one: the FP64 key itself, -inf (masked) kept as the lowest finite value above -inf (taken).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);   // -0 and 0 are one key
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
__device__ __forceinline__ double key_of(double v) { return fmax(v, -__DBL_MAX__); }   // NaN too
template <typename K>
__device__ __forceinline__ K taken_key() {
  if constexpr (sizeof(K) == 4) return 0u;
  else return -__builtin_inf();
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp32(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL, typename V>
__device__ __forceinline__ V dpp(V v) {
  if constexpr (sizeof(V) == 4) {
    return __builtin_bit_cast(V, dpp32<CTRL>(__builtin_bit_cast(uint32_t, v)));
  } else {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(V, static_cast<uint64_t>(dpp32<CTRL>(static_cast<uint32_t>(b >> 32))) << 32 |
                                     dpp32<CTRL>(static_cast<uint32_t>(b)));
  }
}
// f over the LANES lanes of a token, in every one of them: rotations of a DPP row by 8, 4, 2, 1, then across rows
template <int LANES, typename V, typename F>
__device__ __forceinline__ V across(V v, F f) {
  v = f(v, dpp<0x128>(v));
  v = f(v, dpp<0x124>(v));
  v = f(v, dpp<0x122>(v));
  v = f(v, dpp<0x121>(v));
  if constexpr (LANES == 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}
struct Max {
  template <typename V>
  __device__ V operator()(V a, V b) const { return a > b ? a : b; }
};
struct Min {
  template <typename V>
  __device__ V operator()(V a, V b) const { return a < b ? a : b; }
};
struct Sum {
  template <typename V>
  __device__ V operator()(V a, V b) const { return a + b; }
};

// The logits of the experts sub, sub + LANES, .. of token t (-inf behind E), cleaned: NaN to -inf, +inf to the largest
// finite value.
template <int LANES, int EI>
__device__ __forceinline__ void load_logits(const RouteArgs& a, bool f32, int64_t t, int sub, float (&l)[EI]) {
  // every load before any use
  if (f32) {
    const float* const row = static_cast<const float*>(a.logits) + t * a.E;
#pragma unroll
    for (int i = 0; i < EI; ++i) l[i] = row[min(i * LANES + sub, a.E - 1)];
  } else {
    const uint16_t* const row = static_cast<const uint16_t*>(a.logits) + t * a.E;
    uint16_t h[EI];
#pragma unroll
    for (int i = 0; i < EI; ++i) h[i] = row[min(i * LANES + sub, a.E - 1)];
#pragma unroll
    for (int i = 0; i < EI; ++i) l[i] = __uint_as_float(static_cast<uint32_t>(h[i]) << 16);
  }
#pragma unroll
  for (int i = 0; i < EI; ++i) {
    if (i * LANES + sub >= a.E || l[i] != l[i]) l[i] = -__builtin_inff();
    l[i] = fminf(l[i], __FLT_MAX__);
  }
}

// One round of the choice: the largest key over a token's lanes and its expert (the lowest index of equal keys), known
// to every lane; the key is marked as taken.
template <typename K, int LANES, int EI>
__device__ __forceinline__ int take_largest(K (&key)[EI], int sub, K& most) {
  K best = key[0];
  int at = 0;
#pragma unroll
  for (int i = 1; i < EI; ++i) {
    const bool more = key[i] > best;
    best = more ? key[i] : best;
    at = more ? i : at;
  }
  most = across<LANES>(best, Max());
  const uint32_t mine = static_cast<uint32_t>(at * LANES + sub);
  const uint32_t id = across<LANES>(best == most ? mine : 0xFFFFFFFFu, Min());
  const int gone = id == mine ? at : -1;
#pragma unroll
  for (int i = 0; i < EI; ++i) key[i] = i == gone ? taken_key<K>() : key[i];
  return static_cast<int>(id);
}

// Token t by LANES lanes, of which this is number `sub`, without a bias: the logits are the keys, and only the chosen
// ones' scores are needed (all of a softmax's sum unless the weights are renormalised).  Sets `bit` in the masks of the
// token's experts.  A sigmoid far below 0 is 0 in FP32 (exp(-l) overflows at l = -88.7) while the weights, ratios of
// such scores, are not: tokens with a chosen logit below kFarLogit, where exp(-l) and the score are far inside FP32's
// normal range, take their k scores in FP64, as those with a bias do.
constexpr float kFarLogit = -64.0f;
template <int LANES, int EI>
__device__ __forceinline__ void route_token_plain(const RouteArgs& a, bool f32, int64_t t, int sub, uint32_t* mask,
                                                  uint32_t bit) {
  float l[EI];
  uint32_t key[EI];
  load_logits<LANES>(a, f32, t, sub, l);
#pragma unroll
  for (int i = 0; i < EI; ++i) key[i] = i * LANES + sub < a.E ? key_of(l[i]) : taken_key<uint32_t>();
  int my_id = 0;
  uint32_t my_key = 0, top_key = 0, low_key = 0;
  for (int j = 0; j < a.k; ++j) {
    const int id = take_largest<uint32_t, LANES>(key, sub, low_key);
    top_key = j == 0 ? low_key : top_key;
    my_id = sub == j ? id : my_id;
    my_key = sub == j ? low_key : my_key;
  }
  const float ninf = -__builtin_inff();
  const float x = value_of(my_key), top = value_of(top_key);
  const bool chosen = sub < a.k && x != ninf;
  float w;
  if (a.score == MX_ROUTE_SIGMOID && value_of(low_key) < kFarLogit) {
    double p = chosen ? 1 / (1 + exp(-static_cast<double>(x))) : 0;
    if (a.renormalize) {
      const double sum = across<LANES>(p, Sum());
      p = sum > 0 ? p / sum : 0;
    }
    w = static_cast<float>(p * static_cast<double>(a.scale));
  } else {
    float p = 0.f;
    if (chosen) p = a.score == MX_ROUTE_SOFTMAX ? expf(x - top) : 1.0f / (1.0f + expf(-x));
    if (a.renormalize) {
      const float sum = across<LANES>(p, Sum());
      p = sum > 0.f ? p / sum : 0.f;
    } else if (a.score == MX_ROUTE_SOFTMAX) {
      float total = 0.f;
#pragma unroll
      for (int i = 0; i < EI; ++i) total += l[i] == ninf ? 0.f : __expf(l[i] - top);
      total = across<LANES>(total, Sum());
      p = total > 0.f ? p / total : 0.f;
    }
    w = p * a.scale;
  }
  if (sub < a.k) {
    a.ids[t * a.k + sub] = my_id;
    a.weights[t * a.k + sub] = w;
    atomicOr(&mask[my_id], bit);
  }
}

// The same with a bias, scores and keys in FP64.
template <int LANES, int EI>
__device__ __forceinline__ void route_token_biased(const RouteArgs& a, bool f32, int64_t t, int sub, uint32_t* mask,
                                                   uint32_t bit) {
  float l[EI], bias[EI];
#pragma unroll
  for (int i = 0; i < EI; ++i) bias[i] = a.bias[min(i * LANES + sub, a.E - 1)];
  load_logits<LANES>(a, f32, t, sub, l);
  double p[EI], key[EI];
  const float ninf = -__builtin_inff();
  // p[i] = f(l[i]) in a loop that is not unrolled, the arrays rotating through their registers: unrolled, FP64
  // exponentials are kilobytes of code that a wave runs once, at the pace of the instruction fetch
  auto each = [&](auto f) {
#pragma unroll 1
    for (int n = 0; n < EI; ++n) {
      const float x = l[0];
      const double v = f(static_cast<double>(x));
#pragma unroll
      for (int i = 0; i + 1 < EI; ++i) {
        l[i] = l[i + 1];
        p[i] = p[i + 1];
      }
      l[EI - 1] = x;
      p[EI - 1] = v;
    }
  };
  double inv = 1;
  if (a.score == MX_ROUTE_SOFTMAX) {
    float top = ninf;
#pragma unroll
    for (int i = 0; i < EI; ++i) top = fmaxf(top, l[i]);
    top = across<LANES>(top, Max());
    double total = 0;
    each([&](double x) {
      const double v = x == static_cast<double>(ninf) ? 0.0 : exp(x - static_cast<double>(top));
      total += v;
      return v;
    });
    total = across<LANES>(total, Sum());
    inv = total > 0 ? 1 / total : 0;
  } else {
    each([&](double x) { return 1 / (1 + exp(-x)); });
  }
#pragma unroll
  for (int i = 0; i < EI; ++i) {
    p[i] *= inv;
    const double v = l[i] != ninf ? p[i] + static_cast<double>(bias[i]) : static_cast<double>(ninf);
    key[i] = i * LANES + sub < a.E ? key_of(v) : taken_key<double>();
  }
  int my_id = 0;
  double my_p = 0;
  for (int j = 0; j < a.k; ++j) {
    double most, pv = p[0];
    const int id = take_largest<double, LANES>(key, sub, most);
    const int at = id / LANES;
#pragma unroll
    for (int i = 1; i < EI; ++i) pv = i == at ? p[i] : pv;
    pv = __shfl(pv, static_cast<int>(threadIdx.x & 63) - sub + id % LANES);
    my_id = sub == j ? id : my_id;
    my_p = sub == j ? pv : my_p;
  }
  if (a.renormalize) {
    const double sum = across<LANES>(my_p, Sum());
    my_p = sum > 0 ? my_p / sum : 0;
  }
  if (sub < a.k) {
    a.ids[t * a.k + sub] = my_id;
    a.weights[t * a.k + sub] = static_cast<float>(my_p * static_cast<double>(a.scale));
    atomicOr(&mask[my_id], bit);
  }
}

// Scores with a bias, without FP64 keys for every expert (a softmax's sum takes their FP64 exponentials all the same).
// FP32 keys find the k-th largest of different ones, which is at most the k-th largest; an FP32 key is within 2^-20 (1
// + |key|) of its FP64 one (an exponential, a reciprocal or a product of values up to 1, the bias's addition: a few
// 2^-24 each), so the k largest are among the experts whose FP32 key is at least that one's less 2^-18 (1 + |key|).
// Those, k and rarely more, get FP64 keys and are ordered by counting, for each, the ones before it.  Returns false,
// nothing written, if they do not fit (many equal keys, or fewer than k different ones left) or the bound is not finite.
template <int LANES>
struct Candidates {
  static constexpr int kMost = LANES == 16 ? 32 : 64;
  double key[kMost], p[kMost], sorted[LANES == 16 ? 16 : MX_ROUTE_MAX_K];
  int32_t id[kMost];
  int32_t count;
};

template <int LANES, int EI, bool SOFT>
__device__ __forceinline__ bool route_token_preselected(const RouteArgs& a, bool f32, int64_t t, int sub,
                                                        uint32_t* mask, uint32_t bit, Candidates<LANES>& c) {
  float l[EI], bias[EI], key[EI];
  uint32_t left[EI];
#pragma unroll
  for (int i = 0; i < EI; ++i) bias[i] = a.bias[min(i * LANES + sub, a.E - 1)];
  load_logits<LANES, EI>(a, f32, t, sub, l);
  if (sub == 0) c.count = 0;
  float top = 0;
  double inv = 1;
  if constexpr (SOFT) {
    top = l[0];
#pragma unroll
    for (int i = 1; i < EI; ++i) top = fmaxf(top, l[i]);
    top = across<LANES>(top, Max());
    double sum = 0;
#pragma unroll 1
    for (int n = 0; n < EI; ++n) {               // the logits rotate: see route_token_biased
      const float x = l[0];
      sum += exp(static_cast<double>(x) - static_cast<double>(top));
#pragma unroll
      for (int i = 0; i + 1 < EI; ++i) l[i] = l[i + 1];
      l[EI - 1] = x;
    }
    inv = 1.0 / across<LANES>(sum, Sum());       // NaN if every expert is masked, and so are the keys
  }
  const float finv = static_cast<float>(inv);
#pragma unroll
  for (int i = 0; i < EI; ++i) {
    const float v = (SOFT ? __expf(l[i] - top) * finv : __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]))) + bias[i];
    key[i] = l[i] == -__builtin_inff() || v != v ? -__builtin_inff() : v;
    left[i] = i * LANES + sub < a.E ? key_of(key[i]) : 0u;
  }
  // the next smaller key is `most` plus the largest difference modulo 2^32: of the smaller ones those are the largest
  uint32_t most = 0;
  bool below = true;
  for (int j = 0; j < a.k; ++j) {
    uint32_t d = left[0] - most;
#pragma unroll
    for (int i = 1; i < EI; ++i) d = max(d, left[i] - most);
    d = across<LANES>(d, Max()) + most;
    below = below && (j == 0 || d < most);
    most = d;
  }
  const float kth = value_of(most);
  // NaN or -inf where kth is infinite, and -inf for a kth next to the lowest value (a bias that masks), where masked
  // experts, whose FP32 key is -inf too, would be among the candidates
  const float least = kth - 0x1p-18f * (1.0f + fabsf(kth));
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < EI; ++i) mine |= (i * LANES + sub < a.E && key[i] >= least ? 1u : 0u) << i;
  const int total = across<LANES>(static_cast<int>(__popc(mine)), Sum());
  if (!below || !(least >= -__FLT_MAX__) || total > c.kMost) return false;

  while (mine != 0) {
    const int i = __ffs(mine) - 1;
    mine &= mine - 1;
    float x = l[0], b = bias[0];
#pragma unroll
    for (int q = 1; q < EI; ++q) {
      x = q == i ? l[q] : x;
      b = q == i ? bias[q] : b;
    }
    const double e = exp(SOFT ? static_cast<double>(x) - static_cast<double>(top) : -static_cast<double>(x));
    const double p = SOFT ? e * inv : 1.0 / (1.0 + e);
    const int at = atomicAdd(&c.count, 1);       // any order: the ranks below do not depend on it
    c.key[at] = p + static_cast<double>(b);
    c.p[at] = p;
    c.id[at] = i * LANES + sub;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  for (int n = sub; n < total; n += LANES) {
    const double mykey = c.key[n];
    const int id = c.id[n];
    int rank = 0;
    for (int o = 0; o < total; ++o) {
      const double ok = c.key[o];
      rank += ok > mykey || (ok == mykey && c.id[o] < id) ? 1 : 0;
    }
    if (rank < a.k) {
      c.sorted[rank] = c.p[n];
      a.ids[t * a.k + rank] = id;
      atomicOr(&mask[id], bit);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (sub < a.k) {
    double sum = 0;
    for (int j = 0; j < a.k; ++j) sum += c.sorted[j];
    double w = c.sorted[sub];
    if (a.renormalize) w = sum > 0 ? w / sum : 0;
    a.weights[t * a.k + sub] = static_cast<float>(w * static_cast<double>(a.scale));
  }
  return true;
}

// Exclusive prefix sum over the workgroup's threads.
template <int THREADS>
__device__ __forceinline__ int block_exclusive(int v) {
  __shared__ int32_t wave_sum[THREADS / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(s, d);
    s += lane >= d ? o : 0;
  }
  if (lane == 63) wave_sum[wave] = s;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) before += w < wave ? wave_sum[w] : 0;
  return before + s - v;
}

__device__ __forceinline__ int bits_below(uint32_t lo, uint32_t hi, int t) {
  return t < 32 ? __popc(lo & ((1u << t) - 1)) : __popc(lo) + __popc(hi & ((1u << (t - 32)) - 1));
}

template <bool BIAS, int LANES, int EI>
__global__ __launch_bounds__(kTopkThreads) void route_topk_kernel(RouteArgs a, int f32) {
  __shared__ uint32_t mask[2][kMaxExperts];      // tokens 0..31 and 32..63 of the block
  __shared__ int32_t start[kMaxExperts];
  __shared__ Candidates<LANES> cand[BIAS ? kTopkThreads / LANES : 1];
  const int tid = threadIdx.x;
  const int sub = tid & (LANES - 1), group = tid / LANES;
  constexpr int threads = kTopkThreads, groups = threads / LANES;
  for (int e = tid; e < kMaxExperts; e += threads) mask[0][e] = mask[1][e] = 0;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.block_tokens;
#pragma unroll 1
  for (int q = group; q < a.block_tokens && t0 + q < a.T; q += groups) {
    uint32_t* const m = mask[q >> 5];
    const uint32_t bit = 1u << (q & 31);
    if constexpr (BIAS) {
      const bool done = a.score == MX_ROUTE_SOFTMAX
                            ? route_token_preselected<LANES, EI, true>(a, f32 != 0, t0 + q, sub, m, bit, cand[group])
                            : route_token_preselected<LANES, EI, false>(a, f32 != 0, t0 + q, sub, m, bit, cand[group]);
      if (!done)
        route_token_biased<LANES, EI>(a, f32 != 0, t0 + q, sub, m, bit);
    } else {
      route_token_plain<LANES, EI>(a, f32 != 0, t0 + q, sub, m, bit);
    }
  }
  __syncthreads();
  if (a.blocks > 1) {
    for (int e = tid; e < a.E; e += threads)
      a.masks[static_cast<int64_t>(blockIdx.x) * a.E + e] = static_cast<uint64_t>(mask[1][e]) << 32 | mask[0][e];
    if (4 * tid < a.E4) {
      uint32_t c = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b) c |= static_cast<uint32_t>(__popc(mask[0][4 * tid + b]) + __popc(mask[1][4 * tid + b])) << (8 * b);
      a.counts[static_cast<int64_t>(blockIdx.x) * (a.E4 / 4) + tid] = c;
    }
    return;
  }
  int n[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * tid + i;
    n[i] = e < a.E ? __popc(mask[0][e]) + __popc(mask[1][e]) : 0;
  }
  const int first = block_exclusive<threads>(n[0] + n[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * tid + i, at = first + (i ? n[0] : 0);
    if (e < a.E) start[e] = a.offsets[e] = at;
    if (e == a.E - 1) a.offsets[a.E] = at + n[i];
  }
  __syncthreads();
  for (int s = tid; s < a.T * a.k; s += threads) {
    const int id = a.ids[s], q = static_cast<int>(div_u32(static_cast<uint32_t>(s), a.k_div));
    const int row = start[id] + bits_below(mask[0][id], mask[1][id], q);
    a.row_slot[row] = s;
    a.slot_row[s] = row;
  }
}

__global__ __launch_bounds__(kScatterThreads) void route_scatter_kernel(RouteArgs a) {
  __shared__ int32_t total[kMaxExperts], place[kMaxExperts];
  const int tid = threadIdx.x;
  const int b0 = static_cast<int>(blockIdx.x) * a.span, b1 = min(b0 + a.span, a.blocks);
  const int64_t s0 = static_cast<int64_t>(b0) * a.block_tokens * a.k, all_slots = static_cast<int64_t>(a.T) * a.k;
  // a thread's first slot and its block's mask, asked for before the sums: they need no place
  const bool has = tid < a.block_tokens * a.k && s0 + tid < all_slots;
  const int id0 = has ? a.ids[s0 + tid] : 0;
  const uint64_t m0 = a.masks[static_cast<int64_t>(b0) * a.E + id0];
  for (int e = tid; e < kMaxExperts; e += kScatterThreads) total[e] = place[e] = 0;
  __syncthreads();

  // slots of every expert in all blocks, and in the blocks before this span: a thread sums every `parts`-th block of
  // four experts (integer sums, in any order the same)
  const int quads = a.E4 / 4, parts = kScatterThreads / quads, part = tid / quads, q = tid - part * quads;
  if (part < parts) {
    int all[4] = {0, 0, 0, 0}, before[4] = {0, 0, 0, 0};
#pragma unroll 8
    for (int b = part; b < a.blocks; b += parts) {
      const uint32_t c = a.counts[static_cast<int64_t>(b) * quads + q];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = (c >> (8 * i)) & 0xFF;
        all[i] += v;
        before[i] += b < b0 ? v : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      atomicAdd(&total[4 * q + i], all[i]);
      atomicAdd(&place[4 * q + i], before[i]);
    }
  }
  __syncthreads();
  const int n = tid < a.E ? total[tid] : 0;
  const int first = block_exclusive<kScatterThreads>(n);
  if (tid < a.E) {
    place[tid] += first;
    if (blockIdx.x == 0) {
      a.offsets[tid] = first;
      if (tid == a.E - 1) a.offsets[a.E] = first + n;
    }
  }
  __syncthreads();
  for (int b = b0; b < b1; ++b) {
    const uint64_t* const masks = a.masks + static_cast<int64_t>(b) * a.E;
    const int64_t t0 = static_cast<int64_t>(b) * a.block_tokens;
    const int slots = static_cast<int>(min(static_cast<int64_t>(a.block_tokens), a.T - t0)) * a.k;
    for (int i = tid; i < slots; i += kScatterThreads) {
      const int32_t s = static_cast<int32_t>(t0 * a.k) + i;
      const bool first_slot = b == b0 && i == tid;
      const int id = first_slot ? id0 : a.ids[s];
      const uint64_t m = first_slot ? m0 : masks[id];
      const int row = place[id] + bits_below(static_cast<uint32_t>(m), static_cast<uint32_t>(m >> 32),
                                             static_cast<int>(div_u32(static_cast<uint32_t>(i), a.k_div)));
      a.row_slot[row] = s;
      a.slot_row[s] = row;
    }
    if (b + 1 < b1) {
      __syncthreads();
      if (tid < a.E) place[tid] += __popcll(masks[tid]);
      __syncthreads();
    }
  }
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
  DivU32 n8_div;
  uint64_t total;             // T * N8
};

// A thread owns 8 consecutive columns of one token.  J slots' rows are in flight at a time, at most 8, so that the last
// turn is full too (k = 4, 6868 x 5080: 84 us with 8, 64); a dropped slot reads row 0 and is left out of the sum (a
// select, so that what the row holds does not matter).
template <int J>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a) {
  typedef unsigned v4u __attribute__((ext_vector_type(4)));
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= a.total) return;
  const uint64_t t = a.total <= 0xFFFFFFFFu ? div_u32(static_cast<uint32_t>(i), a.n8_div) : i / a.N8;
  const uint32_t c = static_cast<uint32_t>(i - t * a.N8);
  v4u sh = {0, 0, 0, 0};
  if (a.shared != nullptr) sh = reinterpret_cast<const v4u*>(a.shared)[i];
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (a.rows > 0) {
    for (int j0 = 0; j0 < a.k; j0 += J) {
      int r[J];
      float w[J];
      v4u v[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint64_t s = t * a.k + min(j0 + j, a.k - 1);
        r[j] = a.slot_row[s];
        w[j] = a.weights[s];
        if (j0 + j >= a.k || r[j] < 0 || r[j] >= a.rows) {
          r[j] = 0;
          w[j] = 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < J; ++j)
        v[j] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(a.y) + (static_cast<uint64_t>(r[j]) * a.N8 + c));
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const bool in = w[j] != 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float lo = __builtin_fmaf(w[j], bf16_lo(v[j][q]), sum[2 * q]);
          const float hi = __builtin_fmaf(w[j], bf16_hi(v[j][q]), sum[2 * q + 1]);
          sum[2 * q] = in ? lo : sum[2 * q];
          sum[2 * q + 1] = in ? hi : sum[2 * q + 1];
        }
      }
    }
  }
  v4u o;
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(sum[2 * q] + bf16_lo(sh[q]), sum[2 * q + 1] + bf16_hi(sh[q]));
  reinterpret_cast<v4u*>(a.out)[i] = o;
}

// 16 lanes a token while its experts' scores and keys fit the registers and k the lanes, and 64 lanes else, or where
// there are several experts a lane and few tokens, so that latency counts (256 experts, k = 8, kernels of a call, us:
// 64 tokens, softmax with a bias 11.6 against 30.1, without 8.9 against 12.0; 2048 tokens 14.2 against 21.9 and 11.3
// against 12.2; 64 experts, 500 tokens 8.6 against 7.6).
bool route_wide(int64_t T, int32_t E, int32_t k) { return k > 16 || E > 256 || (E > 128 && T > 32 && T <= 8 * 256); }
// Tokens of a block.  One block takes up to 64, in one launch.  More are cut into blocks of 32, the tokens that a
// workgroup works on at once with 16 lanes each (8192 tokens, 256 experts, sigmoid with a bias: 30 against 35 us with
// 64 when this was measured), until longer blocks fill the chip too and halve the masks that the second launch reads.
// With 64 lanes a token a workgroup works on 8 at once: blocks of 8 then, while they are no more than the compute units
// (450 experts, 79 tokens: 11 to 16 us by the score, 23 to 41 with blocks of 32).
int route_block_tokens(int64_t T, int32_t E) {
  if (T > 32 * 1024) return kBlockTokens;
  if (T <= (E > 256 ? 16 : E > 128 ? 32 : kBlockTokens)) return kBlockTokens;
  if (E > 128 && T <= 8 * 256) return 8;
  return E > 256 && T <= 16 * 256 ? 16 : 32;
}
int route_blocks(int64_t T, int32_t E) {
  const int b = route_block_tokens(T, E);
  return T > 0 ? static_cast<int>((T + b - 1) / b) : 1;
}

template <bool BIAS>
void launch_topk(const RouteArgs& a, int32_t f32, hipStream_t stream) {
#define MX_TOPK(LANES, EI) route_topk_kernel<BIAS, LANES, EI><<<a.blocks, kTopkThreads, 0, stream>>>(a, f32)
  if (route_wide(a.T, a.E, a.k)) {
    if (a.E <= 64) MX_TOPK(64, 1);
    else if (a.E <= 128) MX_TOPK(64, 2);
    else if (a.E <= 256) MX_TOPK(64, 4);
    else if (a.E <= 512) MX_TOPK(64, 8);
    else MX_TOPK(64, 16);
  } else if (a.E <= 16) MX_TOPK(16, 1);
  else if (a.E <= 32) MX_TOPK(16, 2);
  else if (a.E <= 64) MX_TOPK(16, 4);
  else if (a.E <= 128) MX_TOPK(16, 8);
  else MX_TOPK(16, 16);
#undef MX_TOPK
}

}  // namespace

size_t route_workspace_bytes(int64_t T, int32_t E) {
  const int64_t blocks = route_blocks(T, E);
  return blocks > 1 ? static_cast<size_t>(blocks) * (8 * static_cast<size_t>(E) + (E + 3) / 4 * 4) : 0;
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
  a.T = static_cast<int32_t>(T);
  a.E = E;
  a.k = k;
  a.E4 = (E + 3) / 4 * 4;
  a.block_tokens = route_block_tokens(T, E);
  a.blocks = route_blocks(T, E);
  a.masks = static_cast<uint64_t*>(workspace);
  a.counts = reinterpret_cast<uint32_t*>(a.masks + static_cast<int64_t>(a.blocks) * E);
  a.span = (a.blocks + kMaxSpans - 1) / kMaxSpans;
  a.k_div = make_div(static_cast<uint32_t>(k));
  a.score = score;
  a.renormalize = renormalize;
  a.scale = scale;
  if (bias)
    launch_topk<true>(a, f32, stream);
  else
    launch_topk<false>(a, f32, stream);
  mx_status st = launch_status("mx_moe_route");
  if (st != MX_OK || a.blocks == 1) return st;
  route_scatter_kernel<<<(a.blocks + a.span - 1) / a.span, kScatterThreads, 0, stream>>>(a);
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
  a.n8_div = make_div(a.N8);
  a.total = static_cast<uint64_t>(T) * a.N8;
  const unsigned grid = static_cast<unsigned>((a.total + 255) / 256);
  const int turns = (k + 7) / 8;
  switch ((k + turns - 1) / turns) {
    case 1: combine_kernel<1><<<grid, 256, 0, stream>>>(a); break;
    case 2: combine_kernel<2><<<grid, 256, 0, stream>>>(a); break;
    case 3: combine_kernel<3><<<grid, 256, 0, stream>>>(a); break;
    case 4: combine_kernel<4><<<grid, 256, 0, stream>>>(a); break;
    case 5: combine_kernel<5><<<grid, 256, 0, stream>>>(a); break;
    case 6: combine_kernel<6><<<grid, 256, 0, stream>>>(a); break;
    case 7: combine_kernel<7><<<grid, 256, 0, stream>>>(a); break;
    default: combine_kernel<8><<<grid, 256, 0, stream>>>(a); break;
  }
  return launch_status("mx_moe_combine");
}

}  // namespace mx
