// Routing of tokens to experts: the top_k largest of each token's logits, their
// weights, the rows sorted by expert, and the balance loss with its gradient.
//
//     p = softmax(l) over the experts
//     weight of a chosen expert: p, or exp(l) / sum of exp(l) over the chosen
//     balance = E sum_e f_e P_e,  f_e = rows of e / all rows,  P_e = mean p_e
//
// Tokens are taken 64 at a time (a chunk).  16 lanes hold a token's logits, so
// that every reduction is four DPP rotations and serves four tokens; a key of
// the logit's first bits over the expert's index (26 over 6 for up to 64 experts,
// 22 over 10 for more than 512) makes an extraction one subtraction and half a
// maximum a logit (a maximum with a separate search for its index takes three
// times that).  bf16 logits fit such a key; fp32 logits that agree in a key's bits
// next to the chosen ones are chosen again with all 32.
//
// The sorted order is a counting sort without a sort: a token chooses an
// expert at most once, so an expert's tokens of a chunk are 64 bits, a pair's
// place in the chunk is a population count, and the chunks' counts need one
// prefix sum an expert.  One chunk runs as one launch, more as three.
//
// One token of 256 experts 5.4 us; 16384 tokens 16.1 (choice, a chunk a compute
// unit: vector instructions fill 36 % of the SIMDs' cycles, and a wavefront waits
// for data or at a barrier 58 % of its time) + 4.4 + 4.8 us, where the 19 MB alone would
// take 4.
#include <algorithm>
#include <type_traits>

#include "stq_launch.hpp"
#include "stq_rows.hpp"

namespace stq {
namespace {

constexpr int kChunk = 64;
constexpr int kLanes = 16;        // lanes of a token
constexpr int kMaxExperts = kRouteMaxExperts;
static_assert(kRouteMaxTop <= 2 * kLanes, "a lane holds two of a token's pairs");
// bits of a key that hold the column, for kN logits a lane
constexpr int index_bits(int n) { return n == 4 ? 6 : n == 8 ? 7 : n == 16 ? 8 : n == 32 ? 9 : 10; }

// exp(x) within three halves of a step of fp32 or so for x from -87 to 0, 0 below:
// exp2 of the rounded product x log2(e), times one plus what the rounding left (the
// exponent's own rounding would cost 40 steps at x = -60).  -inf counts as -200, a
// NaN stays one.  (256 experts 21.5 -> 22.1 us for 16384 tokens, 1024 57.8 -> 61.5.)
__device__ __forceinline__ float exp_of(float x) {
  constexpr double kLog2e = 1.44269504088896340736;
  constexpr float kHigh = static_cast<float>(kLog2e), kLow = static_cast<float>(kLog2e - kHigh), kLn2 = 0.69314718055994530942f;
  x = x < -200.0f ? -200.0f : x;
  const float t = x * kHigh;
  const float left = fmaf(x, kLow, fmaf(x, kHigh, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, left * kLn2, e);
}

// Column of a lane's j-th logit: four neighbours a lane, 64 a step
__device__ __forceinline__ int column(int lane16, int j) { return (j >> 2) * 64 + lane16 * 4 + (j & 3); }

// Bits that order like the value; -0 and +0 alike.  -inf gives 0x007FFFFF, so
// 0 stands for "none".
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ uint32_t max16(uint32_t v) {
  return reduce16(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ uint32_t min16(uint32_t v) {
  return reduce16(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}
__device__ __forceinline__ float fmax16(float v) {
  return reduce16(v, [](float a, float b) { return fmaxf(a, b); });
}

// A token's logits, kN a lane; columns from `experts` on read as -inf
template <typename T, int kN>
__device__ __forceinline__ void load_logits(const T* row, int lane16, int experts, bool valid, float (&v)[kN]) {
#pragma unroll
  for (int q = 0; q < kN / 4; ++q) {
    const int c = column(lane16, 4 * q);
    if (valid && c + 4 <= experts) {
      if constexpr (sizeof(T) == 4) {
        const u32x4_t w = load16b(row + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * q + e] = __builtin_bit_cast(float, static_cast<uint32_t>(w[e]));
      } else {
        const u32x2_t w = reinterpret_cast<const Words8*>(row + c)->v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[4 * q + e] = __builtin_bit_cast(float, (e & 1) ? (w[e >> 1] & 0xFFFF0000u) : (w[e >> 1] << 16));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * q + e] = valid && c + e < experts ? widen(row[c + e]) : -INFINITY;
    }
  }
}

// exp(l - max) of a token's logits into v's place; returns their sum: NaN for
// a token with a NaN or +inf, 0 for one that is masked throughout.
template <int kN>
__device__ __forceinline__ float exponents(float (&v)[kN], float& top) {
  float m = v[0];
#pragma unroll
  for (int j = 1; j < kN; ++j) m = fmaxf(m, v[j]);
  m = fmax16(m);
  top = m;
  // masked logits count for nothing, under a masked maximum too; a NaN stays one
  const float base = m == -INFINITY ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    v[j] = exp_of(v[j] - base);
    s += v[j];
  }
  return sum16(s);
}

struct RouteKernelArgs {
  RouteArgs a;
  int chunks;
  int32_t* hist;    // [experts][chunks]
  float* prob;      // [experts][chunks]
  float* prob_total;
};

// Inclusive prefix sum over a wavefront: shifts inside 16 lanes, then the last
// lanes of the rows below.
__device__ __forceinline__ int scan64(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// The experts' counts turned into their first rows (`first`, LDS, n + 1
// entries), and the balance loss, by one wavefront: a lane has kPer
// neighbouring experts.  count(e) and prob(e) are their counts and summed
// probabilities.
template <int kPer, typename C, typename P>
__device__ __forceinline__ float scan_experts(int n, int top_k, int* first, C count, P prob) {
  const int lane = threadIdx.x & 63;
  int c[kPer], own = 0;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * kPer + i;
    c[i] = e < n ? count(e) : 0;
    if (e < n) s = fmaf(static_cast<float>(c[i]), prob(e), s);
    own += c[i];
  }
  const int sum = scan64(own);
  int at = sum - own;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane * kPer + i;
    if (e < n) first[e] = at;
    at += c[i];
  }
  const int total = __builtin_amdgcn_readlane(sum, 63);
  if (lane == 0) first[n] = total;
  s = sum64(s);
  const float rows = static_cast<float>(max(total, 1));
  return s * (static_cast<float>(n) / rows) * (static_cast<float>(top_k) / rows);
}

// Tokens of the chunk before token tl among those in an expert's 64 bits
__device__ __forceinline__ int before(const uint32_t (&m)[2], int tl) {
  const uint32_t lo = tl < 32 ? m[0] & ((1u << tl) - 1u) : m[0];
  const uint32_t hi = tl < 32 ? 0u : m[1] & ((1u << (tl - 32)) - 1u);
  return __popc(lo) + __popc(hi);
}

// One chunk: choice, weights, counts and summed probabilities; with kOne (the
// only chunk) the sorted rows too.
template <typename T, int kN, int kThreads, bool kOne>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteKernelArgs g) {
  constexpr int kAtOnce = kThreads / kLanes, kCols = kLanes * kN;
  constexpr uint32_t kIndex = (1u << index_bits(kN)) - 1u;
  constexpr int kGroups = kThreads > kCols ? kThreads / kCols : 1;   // threads a column
  constexpr int kPerThread = kCols > kThreads ? kCols / kThreads : 1;  // columns a thread
  constexpr int kPairs = kOne ? kChunk * kRouteMaxTop : 1;
  const RouteArgs& a = g.a;
  const int E = a.experts, k = a.top_k;
  __shared__ __align__(16) float prob[kAtOnce][kCols];
  __shared__ uint32_t mask[kCols][2];   // an expert's tokens of the chunk
  __shared__ int first[kOne ? kCols + 1 : 1], pair_e[kPairs];
  __shared__ float pair_w[kPairs];
  const int lane16 = threadIdx.x & (kLanes - 1);
  for (int i = threadIdx.x; i < kCols; i += kThreads) mask[i][0] = mask[i][1] = 0u;
  __syncthreads();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kChunk;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(kChunk), a.tokens - t0));
  float acc[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) acc[i] = 0.0f;
  for (int tp = 0; tp < tokens; tp += kAtOnce) {
    const int tl = tp + static_cast<int>(threadIdx.x) / kLanes;
    const bool valid = tl < tokens;
    if (__any(valid)) {
      const int64_t t = t0 + tl;
      const T* row = static_cast<const T*>(a.logits) + (valid ? t : 0) * a.stride;
      float v[kN];
      load_logits<T, kN>(row, lane16, E, valid, v);
      uint32_t key[kN];
#pragma unroll
      for (int j = 0; j < kN; ++j)   // (columns past the experts: below a masked expert's, so never among E)
        key[j] = (order_bits(v[j]) & ~kIndex) | (kIndex - column(lane16, j));
      float top;
      const float sum = exponents<kN>(v, top);
      // nothing for a token that is masked throughout, NaN for one without a distribution
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int q = 0; q < kN / 4; ++q)
        *reinterpret_cast<f32x4_t*>(&prob[tl - tp][column(lane16, 4 * q)]) =
            f32x4_t{v[4 * q] * inv, v[4 * q + 1] * inv, v[4 * q + 2] * inv, v[4 * q + 3] * inv};
      // extraction: after step i, lane i % 16 holds the i-th key.  Less the last
      // one, in 32 bits that wrap, keys taken already are small and those that
      // are left are large, so nothing has to be taken out.
      uint32_t mine[2] = {0u, 0u}, last = 0u;
      bool unsure = false;
      const int steps = sizeof(T) == 4 ? min(k + 1, E) : k;
      for (int i = 0; i < steps; ++i) {
        uint32_t m = key[0] - last;
#pragma unroll
        for (int j = 1; j < kN; ++j) m = max(m, key[j] - last);
        m = max16(m) + last;
        unsure |= i > 0 && ((m ^ last) & ~kIndex) == 0u;
        last = m;
        if (lane16 == (i & 15) && i < k) mine[i >> 4] = m;
      }
      int pick[2] = {static_cast<int>(kIndex - (mine[0] & kIndex)), static_cast<int>(kIndex - (mine[1] & kIndex))};
      if (sizeof(T) == 4 && __any(unsure && valid)) {
        // some keys agree: once more with whole values, the lowest index first
        load_logits<T, kN>(row, lane16, E, valid, v);
#pragma unroll
        for (int j = 0; j < kN; ++j) key[j] = column(lane16, j) < E ? order_bits(v[j]) : 0u;
        for (int i = 0; i < k; ++i) {
          uint32_t m = key[0];
#pragma unroll
          for (int j = 1; j < kN; ++j) m = max(m, key[j]);
          m = max16(m);
          uint32_t c = ~0u;
#pragma unroll
          for (int j = kN - 1; j >= 0; --j) c = key[j] == m ? static_cast<uint32_t>(column(lane16, j)) : c;
          c = min16(c);
#pragma unroll
          for (int j = 0; j < kN; ++j) key[j] = static_cast<uint32_t>(column(lane16, j)) == c ? 0u : key[j];
          if (lane16 == (i & 15)) pick[i >> 4] = static_cast<int>(c);
        }
      }
      // weights; a token without a distribution goes nowhere
      const bool routed = valid && top != -INFINITY && sum == sum;
      __builtin_amdgcn_wave_barrier();   // the token's probabilities are its own wavefront's
      float w[2] = {0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (routed && lane16 + 16 * h < k) w[h] = prob[tl - tp][pick[h]];
      const float norm = a.renorm ? 1.0f / sum16(w[0] + w[1]) : 1.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = lane16 + 16 * h;
        if (!valid || i >= k) continue;
        const int64_t p = t * k + i;
        const int e = routed ? pick[h] : -1;
        const float weight = routed ? w[h] * norm : top == -INFINITY && sum == sum ? 0.0f : NAN;
        a.pair_expert[p] = e;
        a.pair_weight[p] = weight;
        if constexpr (kOne) {
          pair_e[p] = e;
          pair_w[p] = weight;
        }
        if (routed) atomicOr(&mask[e][tl >> 5], 1u << (tl & 31));
      }
    }
    __syncthreads();
    const int rows = min(kAtOnce, tokens - tp);
    if constexpr (kPerThread == 1) {
      for (int r = static_cast<int>(threadIdx.x) / kCols; r < rows; r += kGroups) acc[0] += prob[r][threadIdx.x % kCols];
    } else {
#pragma unroll
      for (int i = 0; i < kPerThread; ++i)
        for (int r = 0; r < rows; ++r) acc[i] += prob[r][threadIdx.x + i * kThreads];
    }
    __syncthreads();
  }
  // the threads of a column joined, in the place of the first tokens' probabilities
  float* const part = &prob[0][0];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) part[threadIdx.x + i * kThreads] = acc[i];
  __syncthreads();
  auto expert_prob = [&](int e) {
    float s = part[e];
#pragma unroll
    for (int i = 1; i < kGroups; ++i) s += part[i * kCols + e];
    return s;
  };
  auto expert_count = [&](int e) { return __popc(mask[e][0]) + __popc(mask[e][1]); };
  if constexpr (!kOne) {
    for (int e = threadIdx.x; e < E; e += kThreads) {
      g.prob[static_cast<int64_t>(e) * g.chunks + blockIdx.x] = expert_prob(e);
      g.hist[static_cast<int64_t>(e) * g.chunks + blockIdx.x] = expert_count(e);
    }
  } else {
    if (threadIdx.x < 64) {
      const float b = scan_experts<kCols / 64>(E, k, first, expert_count, expert_prob);
      if (threadIdx.x == 0) *a.balance = b;
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kThreads) {
      a.offsets[e] = first[e];
      if (e < E) a.counts[e] = expert_count(e);
    }
    const int pairs = tokens * k, total = first[E];
    for (int p = threadIdx.x; p < pairs; p += kThreads) {
      const int tl = p / k, e = pair_e[p];
      int at = -1;
      if (e >= 0) {
        at = first[e] + before(mask[e], tl);
        a.row_token[at] = tl;
        a.row_weight[at] = pair_w[p];
      }
      a.pair_row[p] = at;
      if (p >= total) {
        a.row_token[p] = 0;
        a.row_weight[p] = 0.0f;
      }
    }
  }
}

// An expert's counts over the chunks turned into the rows before each chunk,
// and its probabilities added up; a wavefront an expert, 256 chunks at a time.
__global__ __launch_bounds__(256) void route_scan_kernel(RouteKernelArgs g) {
  constexpr int kAt = 4;
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (e >= g.a.experts) return;
  int32_t* hist = g.hist + static_cast<int64_t>(e) * g.chunks;
  const float* prob = g.prob + static_cast<int64_t>(e) * g.chunks;
  int before = 0;
  float p = 0.0f;
  for (int c0 = 0; c0 < g.chunks; c0 += 64 * kAt) {
    int own[kAt];
    float more[kAt];
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      const int c = c0 + 64 * i + lane;
      own[i] = c < g.chunks ? hist[c] : 0;
      more[i] = c < g.chunks ? prob[c] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kAt; ++i) {
      const int c = c0 + 64 * i + lane;
      const int sum = scan64(own[i]);
      if (c < g.chunks) hist[c] = before + sum - own[i];
      before += __builtin_amdgcn_readlane(sum, 63);
      p += more[i];
    }
  }
  p = sum64(p);
  if (lane == 0) {
    g.a.counts[e] = before;
    g.prob_total[e] = p;
  }
}

// A chunk's pairs to their rows.  Everything it reads is on its way before the
// first barrier.
__global__ __launch_bounds__(512) void route_scatter_kernel(RouteKernelArgs g) {
  constexpr int kAt = 4;   // pairs a thread: 64 tokens of 32
  __shared__ uint32_t mask[kMaxExperts][2];
  __shared__ int count[kMaxExperts], base[kMaxExperts], first[kMaxExperts + 1];
  const RouteArgs& a = g.a;
  const int E = a.experts, k = a.top_k;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kChunk;
  const int pairs = static_cast<int>(min(static_cast<int64_t>(kChunk), a.tokens - t0)) * k;
  const int64_t p0 = t0 * k;
  int e[kAt];
  float w[kAt];
#pragma unroll
  for (int i = 0; i < kAt; ++i) {
    const int p = threadIdx.x + 512 * i;
    e[i] = p < pairs ? a.pair_expert[p0 + p] : -1;
    w[i] = p < pairs ? a.pair_weight[p0 + p] : 0.0f;
  }
  for (int x = threadIdx.x; x < E; x += 512) {
    mask[x][0] = mask[x][1] = 0u;
    count[x] = a.counts[x];
    base[x] = g.hist[static_cast<int64_t>(x) * g.chunks + blockIdx.x];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAt; ++i) {
    const int tl = (threadIdx.x + 512 * i) / k;
    if (e[i] >= 0) atomicOr(&mask[e[i]][tl >> 5], 1u << (tl & 31));
  }
  if (threadIdx.x < 64) {
    const bool lead = blockIdx.x == 0;
    auto prob = [&](int x) { return lead ? g.prob_total[x] : 0.0f; };
    auto counted = [&](int x) { return count[x]; };
    const float b = E <= 256 ? scan_experts<4>(E, k, first, counted, prob) : scan_experts<16>(E, k, first, counted, prob);
    if (lead && threadIdx.x == 0) *a.balance = b;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int x = threadIdx.x; x <= E; x += 512) a.offsets[x] = first[x];
  const int64_t total = first[E];
#pragma unroll
  for (int i = 0; i < kAt; ++i) {
    const int p = threadIdx.x + 512 * i, tl = p / k;
    if (p >= pairs) break;
    int at = -1;
    if (e[i] >= 0) {
      at = first[e[i]] + base[e[i]] + before(mask[e[i]], tl);
      a.row_token[at] = static_cast<int32_t>(t0) + tl;
      a.row_weight[at] = w[i];
    }
    a.pair_row[p0 + p] = at;
    if (p0 + p >= total) {
      a.row_token[p0 + p] = 0;
      a.row_weight[p0 + p] = 0.0f;
    }
  }
}

// Gradient: 16 lanes a token again.  The chosen experts' share goes through a
// row of LDS, from the lanes that hold the pairs to those that hold the
// logits.
template <typename T, int kN, int kThreads>
__global__ __launch_bounds__(kThreads) void route_bwd_kernel(RouteBwdArgs a) {
  constexpr int kTok = kThreads / kLanes, kCols = kLanes * kN;
  __shared__ float coef[kCols];          // d balance / d p_e of one token, times grad_balance
  __shared__ float chosen[kTok][kCols];
  __shared__ float wsum[kThreads / 64];
  const int E = a.experts, k = a.top_k;
  const int lane16 = threadIdx.x & (kLanes - 1), tl = threadIdx.x / kLanes;
  float total = 0.0f;
  if (a.g_balance) {
    int n = 0;
    for (int e = threadIdx.x; e < E; e += kThreads) n += a.counts[e];
    // whole numbers below 2^31: exact in two halves
    const float hi = sum64(static_cast<float>(n >> 12)), lo = sum64(static_cast<float>(n & 4095));
    if ((threadIdx.x & 63) == 0) wsum[threadIdx.x >> 6] = hi * 4096.0f + lo;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) total += wsum[i];
  }
  const float rows = fmaxf(total, 1.0f);
  const float scale = a.g_balance ? *a.g_balance * (static_cast<float>(E) / rows) * (static_cast<float>(k) / rows) : 0.0f;
  for (int e = threadIdx.x; e < kCols; e += kThreads)
    coef[e] = a.g_balance && e < E ? scale * static_cast<float>(a.counts[e]) : 0.0f;
  const int64_t steps = (a.tokens + kTok - 1) / kTok;
  for (int64_t st = blockIdx.x; st < steps; st += gridDim.x) {
    const int64_t t = st * kTok + tl;
    const bool valid = t < a.tokens;
    const T* row = static_cast<const T*>(a.logits) + (valid ? t : 0) * a.stride;
    float v[kN];
    load_logits<T, kN>(row, lane16, E, valid, v);
    float top;
    const float sum = exponents<kN>(v, top);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int q = 0; q < kN / 4; ++q) *reinterpret_cast<f32x4_t*>(&chosen[tl][column(lane16, 4 * q)]) = f32x4_t{0, 0, 0, 0};
    __syncthreads();
    float w[2] = {0.0f, 0.0f}, gw[2] = {0.0f, 0.0f};
    int e[2] = {-1, -1};
    if (a.g_weight && valid) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = lane16 + 16 * h;
        if (i >= k) continue;
        const int64_t p = t * k + i;
        const int ex = a.pair_expert[p];
        int64_t at = p;
        if (a.pair_row) at = a.pair_row[p];
        if (ex < 0 || ex >= E || at < 0 || at >= a.tokens * k) continue;
        e[h] = ex;
        gw[h] = a.g_weight[at];
        const float l = widen(row[ex]);
        w[h] = l == -INFINITY ? 0.0f : exp_of(l - top);
      }
    }
    if (a.renorm) {
      const float ws = sum16(w[0] + w[1]);
      const float winv = ws == 0.0f ? 0.0f : 1.0f / ws;
      const float mean = sum16(fmaf(w[0], gw[0], w[1] * gw[1])) * winv;
#pragma unroll
      for (int h = 0; h < 2; ++h) gw[h] = w[h] * winv * (gw[h] - mean);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (e[h] >= 0) atomicAdd(&chosen[tl][e[h]], gw[h]);
    __syncthreads();
    // renorm: d = p (c - sum c p) + the chosen's own; else their gradient joins c
    float cv[kN], dot = 0.0f;
#pragma unroll
    for (int q = 0; q < kN / 4; ++q) {
      const int c = column(lane16, 4 * q);
      const f32x4_t co = *reinterpret_cast<const f32x4_t*>(&coef[c]), ch = *reinterpret_cast<const f32x4_t*>(&chosen[tl][c]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = 4 * q + i;
        v[j] *= inv;
        cv[j] = a.renorm ? co[i] : co[i] + ch[i];
        dot = fmaf(cv[j], v[j], dot);
      }
    }
    dot = sum16(dot);
    T* out = static_cast<T*>(a.d_logits) + t * a.d_stride;
#pragma unroll
    for (int q = 0; q < kN / 4; ++q) {
      const int c = column(lane16, 4 * q);
      if (!valid || c >= E) continue;
      const f32x4_t ch = *reinterpret_cast<const f32x4_t*>(&chosen[tl][c]);
      float d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float base = v[4 * q + i] * (cv[4 * q + i] - dot);
        d[i] = a.renorm ? base + ch[i] : base;
      }
      if (c + 4 <= E) {
        if constexpr (sizeof(T) == 4) store16b(out + c, __builtin_bit_cast(u32x4_t, f32x4_t{d[0], d[1], d[2], d[3]}));
        else reinterpret_cast<Words8*>(out + c)->v = u32x2_t{bf16_round(d[0]) | bf16_round(d[1]) << 16, bf16_round(d[2]) | bf16_round(d[3]) << 16};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c + i < E) out[c + i] = narrow<T>(d[i]);
      }
    }
    // (lanes of tokens past the end come here too: a wavefront may hold both)
    __syncthreads();
  }
}

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

}  // namespace

RouteLayout route_layout(int64_t tokens, int64_t experts) {
  const int64_t chunks = (tokens + kChunk - 1) / kChunk;
  if (chunks <= 1) return RouteLayout{chunks, 0, 0, 0};
  const int64_t part = round256(chunks * experts * 4);
  return RouteLayout{chunks, part, 2 * part, 2 * part + round256(experts * 4)};
}

hipError_t launch_route(const RouteArgs& a, void* ws, hipStream_t s) {
  const RouteLayout l = route_layout(a.tokens, a.experts);
  char* base = static_cast<char*>(ws);
  const bool one = l.chunks <= 1;
  const RouteKernelArgs g{a, static_cast<int>(l.chunks),
                          one ? nullptr : reinterpret_cast<int32_t*>(base), one ? nullptr : reinterpret_cast<float*>(base + l.prob),
                          one ? nullptr : reinterpret_cast<float*>(base + l.prob_total)};
  const dim3 grid(static_cast<unsigned>(one ? 1 : l.chunks));
  auto go = [&](auto t, auto n, auto threads) {
    using T = decltype(t);
    constexpr int kN = decltype(n)::value, kThreads = decltype(threads)::value;
    if (one) hipLaunchKernelGGL((route_kernel<T, kN, kThreads, true>), grid, dim3(kThreads), 0, s, g);
    else hipLaunchKernelGGL((route_kernel<T, kN, kThreads, false>), grid, dim3(kThreads), 0, s, g);
  };
  // logits a lane, and as many threads as their registers leave room for
  auto with_n = [&](auto t) {
    if (a.experts <= 64) go(t, std::integral_constant<int, 4>{}, std::integral_constant<int, 1024>{});
    else if (a.experts <= 128) go(t, std::integral_constant<int, 8>{}, std::integral_constant<int, 1024>{});
    else if (a.experts <= 256) go(t, std::integral_constant<int, 16>{}, std::integral_constant<int, 1024>{});
    else if (a.experts <= 512) go(t, std::integral_constant<int, 32>{}, std::integral_constant<int, 512>{});
    else go(t, std::integral_constant<int, 64>{}, std::integral_constant<int, 256>{});
  };
  a.bf16 ? with_n(bf16_t{}) : with_n(0.0f);
  if (!one) {
    hipLaunchKernelGGL(route_scan_kernel, dim3((a.experts + 3) / 4), dim3(256), 0, s, g);
    hipLaunchKernelGGL(route_scatter_kernel, grid, dim3(512), 0, s, g);
  }
  return hipGetLastError();
}

hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t s) {
  auto go = [&](auto t, auto n) {
    constexpr int kN = decltype(n)::value, kThreads = 256;
    const int64_t steps = (a.tokens + kThreads / kLanes - 1) / (kThreads / kLanes);
    hipLaunchKernelGGL((route_bwd_kernel<decltype(t), kN, kThreads>), dim3(static_cast<unsigned>(std::min<int64_t>(steps, 8192))),
                       dim3(kThreads), 0, s, a);
  };
  auto with_n = [&](auto t) {
    if (a.experts <= 64) go(t, std::integral_constant<int, 4>{});
    else if (a.experts <= 128) go(t, std::integral_constant<int, 8>{});
    else if (a.experts <= 256) go(t, std::integral_constant<int, 16>{});
    else if (a.experts <= 512) go(t, std::integral_constant<int, 32>{});
    else go(t, std::integral_constant<int, 64>{});
  };
  a.bf16 ? with_n(bf16_t{}) : with_n(0.0f);
  return hipGetLastError();
}

}  // namespace stq
