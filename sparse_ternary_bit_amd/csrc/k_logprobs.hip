// Log probabilities of given tokens, log-sum-exp, entropy and the most likely
// alternatives of every row of logits, and their gradient.
//
// With m = max l, e_i = exp(l_i - m), s = sum e_i and t = sum e_i (l_i - m):
//     lse = m + log s      log p_i = (l_i - m) - log s      H = log s - t / s
// so one pass over a row with a running (m, s, t) gives everything but the
// alternatives.  Logits of -inf (a masked vocabulary) have e = 0 and count
// for nothing; the products e (l - m) use l - m held above -200 / log2(e), so
// that 0 times infinity never appears.
//
// Alternatives.  A thread also keeps the largest value it met and the first
// 16-byte chunk that held it.  The largest of each lane over the workgroup's
// wavefronts are 64 keys (value, chunk) of disjoint parts of the row; the
// n-th largest of them bounds the row's n-th largest element from below, and
// only threads whose own key reaches that bound can hold one of the n.  On
// random rows that is little more than n of the 512 threads, so the second
// look at the row touches a few percent of it, from the L2 cache.  The
// elements at or above the bound are collected and ranked by counting.  Ties
// go to the lowest id, exactly, because a key carries its position.
#include <float.h>

#include "stq_device.hpp"
#include "stq_launch.hpp"

namespace stq {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kCap = 1024;           // candidates ranked at once
constexpr int kMaxTop = 32;
constexpr int kMaxSplits = 64;       // one lane each where they are joined
static_assert(kMaxTop * kMaxTop <= kCap, "the join's candidates fit");
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kFloor = -200.0f;    // exp2 of anything at or below this is 0 in fp32

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// (value, position) as one integer that orders by value, then lowest
// position; -0 and +0 are the same value.  0 stands for "none".
__device__ __forceinline__ uint64_t make_key(float v, uint32_t pos) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);
  const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return (static_cast<uint64_t>(o) << 32) | (0xFFFFFFFFu - pos);
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __builtin_bit_cast(float, (o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ uint32_t key_pos(uint64_t k) { return 0xFFFFFFFFu - static_cast<uint32_t>(k); }

// Running maximum m, sum of 2^x and first moment of x, x = l log2(e) - m2.
struct Stat {
  float m, s, t;
};

// Maxima so large that m2's rounding is no longer small, or overflows (the
// type's lowest value as a mask on a whole row, say): x is (l - m) log2(e).
__device__ __forceinline__ bool wide(float m) { return fabsf(m) > 1024.0f; }
__device__ __forceinline__ float m2_of(float m) { return m * kLog2e; }
// What x holds beyond (l - m) log2(e): m log2(e) - m2, exactly
__device__ __forceinline__ float excess(float m) { return wide(m) ? 0.0f : fmaf(m, kLog2e, -m2_of(m)); }

__device__ __forceinline__ void rescale(Stat& a, float m) {
  if (a.m == -INFINITY) {        // nothing but masked logits (or NaN, which s keeps) so far
    a.m = m;
    return;
  }
  float dlt;
  {
#pragma clang fp contract(off)
    dlt = wide(a.m) || wide(m) ? (a.m - m) * kLog2e - excess(a.m) + excess(m) : m2_of(a.m) - m2_of(m);
  }
  dlt = fmaxf(dlt, kFloor);
  const float f = __builtin_amdgcn_exp2f(dlt);
  a.t = f * fmaf(a.s, dlt, a.t);
  a.s *= f;
  a.m = m;
}

__device__ __forceinline__ Stat merge(Stat a, Stat b) {
  const float m = fmaxf(a.m, b.m);
  if (a.m < m) rescale(a, m);
  if (b.m < m) rescale(b, m);
  return Stat{m, a.s + b.s, a.t + b.t};
}

// Reductions over a wavefront: row shifts inside 16 lanes, then the row
// broadcasts; every lane gets the result.
template <int kCtrl>
__device__ __forceinline__ float dpp(float old, float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v),
                                                               kCtrl, 0xF, 0xF, false));
}
__device__ __forceinline__ float last_lane(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<0x111>(v, v));
  v = fmaxf(v, dpp<0x112>(v, v));
  v = fmaxf(v, dpp<0x114>(v, v));
  v = fmaxf(v, dpp<0x118>(v, v));
  v = fmaxf(v, dpp<0x142>(v, v));
  v = fmaxf(v, dpp<0x143>(v, v));
  return last_lane(v);
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x111>(0.0f, v);
  v += dpp<0x112>(0.0f, v);
  v += dpp<0x114>(0.0f, v);
  v += dpp<0x118>(0.0f, v);
  // lane 15 (then 31) of the rows below into the rows above only
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x142, 0xA, 0xF, false));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x143, 0xC, 0xF, false));
  return last_lane(v);
}
__device__ __forceinline__ Stat merge_wave(Stat st) {
  const float m = wave_max(st.m);
  if (st.m < m) rescale(st, m);
  return Stat{m, wave_sum(st.s), wave_sum(st.t)};
}

// Lane j's value, j the same for every lane
__device__ __forceinline__ uint64_t lane64(uint64_t v, int j) {
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(v), j);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(v >> 32), j);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}

template <typename T>
struct Row;  // one row of logits cut into 16-byte chunks on 16-byte boundaries

template <>
struct Row<float> {
  static constexpr int kE = 4;
  static __device__ __forceinline__ void unpack(const u32x4_t& r, float (&v)[kE]) {
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const uint32_t w = r[i];
      v[i] = __builtin_bit_cast(float, w);
    }
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};

template <>
struct Row<uint16_t> {
  static constexpr int kE = 8;
  static __device__ __forceinline__ void unpack(const u32x4_t& r, float (&v)[kE]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __builtin_bit_cast(float, r[i] << 16);
      v[2 * i + 1] = __builtin_bit_cast(float, r[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ float one(const uint16_t* p) {
    return __builtin_bit_cast(float, static_cast<uint32_t>(*p) << 16);
  }
};

// Chunk c of a row holds elements c * kE - skew ...; a chunk that reaches
// past either end of the row is read element by element and filled with -inf.
template <typename T>
struct RowView {
  const T* p;
  int vocab;
  int skew;
  int chunks;
  __device__ __forceinline__ RowView(const T* row, int64_t n) : p(row), vocab(static_cast<int>(n)) {
    skew = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    chunks = (vocab + skew + Row<T>::kE - 1) / Row<T>::kE;
  }
  __device__ __forceinline__ int first(int c) const { return c * Row<T>::kE - skew; }
  __device__ __forceinline__ bool whole(int c) const {
    const int i = first(c);
    return i >= 0 && i + Row<T>::kE <= vocab;
  }
  __device__ __forceinline__ u32x4_t raw(int c) const {  // a whole chunk
    return *reinterpret_cast<const u32x4_t*>(p + first(c));
  }
  __device__ __forceinline__ void load(int c, float (&v)[Row<T>::kE]) const {
    const int i0 = first(c);
    if (whole(c)) {
      Row<T>::unpack(raw(c), v);
    } else {
#pragma unroll
      for (int i = 0; i < Row<T>::kE; ++i)
        v[i] = (i0 + i >= 0 && i0 + i < vocab) ? Row<T>::one(p + i0 + i) : -INFINITY;
    }
  }
};

struct LArgs {
  const void* logits;
  int64_t stride;       // elements
  int64_t rows;
  int64_t vocab;
  const int32_t* targets;
  float* logprob;
  float* lse;
  float* entropy;
  int32_t* top_ids;
  float* top_lp;
  int top_n;
  int splits;
  int64_t per;          // chunks per split
  float* stats;         // [rows, splits, 4]: m, s, t (splits > 1)
  uint64_t* keys;       // [rows, splits, top_n]
};

struct SelectSmem {
  uint64_t lane_key[kWaves][64];
  uint64_t bound;
  int count;
  int n_thr;
  uint64_t best;
  uint16_t thr[kThreads];
  uint64_t cand[kCap];
};

// Rank of each of `count` distinct keys by counting the larger ones; the n
// largest go to out(rank, key), ranks past `count` get key 0.
template <typename F>
__device__ __forceinline__ void rank_out(const uint64_t* cand, int count, int n, F out) {
  for (int i = threadIdx.x; i < count; i += kThreads) {
    const uint64_t k = cand[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += cand[j] > k;
    if (rank < n) out(rank, k);
  }
  for (int i = count + threadIdx.x; i < n; i += kThreads) out(i, uint64_t{0});
}

// n-th largest of the 64 keys held one per lane by a wavefront (0 if fewer
// than n are nonzero), n <= 64.
__device__ __forceinline__ uint64_t nth_of_wave(uint64_t k, int n) {
  if (k == 0) k = threadIdx.x & 63;  // below every key, and all keys differ
  int rank = 0;
#pragma unroll
  for (int j = 0; j < 64; ++j) rank += lane64(k, j) > k;
  const uint64_t b = lane64(k, __builtin_ctzll(__ballot(rank == n - 1)));
  return b < 64 ? 0 : b;
}

// The n largest elements of the workgroup's chunks [c0, c1): out(rank, key).
// best / best_chunk: this thread's largest value and the first of its chunks
// that holds it (best_chunk < 0: no chunk).
template <typename T, typename F>
__device__ __forceinline__ void select_top(const RowView<T>& row, int c0, int c1, int n, float best,
                                           int best_chunk, SelectSmem& sh, F out) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint64_t mine = best_chunk < 0 ? 0 : make_key(best, static_cast<uint32_t>(best_chunk));
  sh.lane_key[wave][lane] = mine;
  if (tid == 0) {
    sh.count = 0;
    sh.n_thr = 0;
  }
  __syncthreads();
  if (wave == 0) {
    uint64_t k = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) k = max(k, sh.lane_key[w][lane]);
    const uint64_t b = nth_of_wave(k, n);
    if (lane == 0) sh.bound = b;
  }
  __syncthreads();
  const uint64_t bound = sh.bound;
  if (mine != 0 && mine >= bound) sh.thr[atomicAdd(&sh.n_thr, 1)] = static_cast<uint16_t>(tid);
  __syncthreads();
  // every chunk of those threads, dealt over the workgroup
  const int n_thr = sh.n_thr;
  const int per = (c1 - c0 + kThreads - 1) / kThreads;
  auto scan = [&](auto visit) {
    for (int64_t w = tid; w < static_cast<int64_t>(n_thr) * per; w += kThreads) {
      const int j = static_cast<int>(w / per);
      const int c = c0 + sh.thr[j] + static_cast<int>(w - static_cast<int64_t>(j) * per) * kThreads;
      if (c >= c1) continue;
      float v[Row<T>::kE];
      row.load(c, v);
      const int i0 = row.first(c);
#pragma unroll
      for (int i = 0; i < Row<T>::kE; ++i) {
        if (i0 + i < 0 || i0 + i >= row.vocab) continue;
        // against the bound by chunk position, as the bound was made
        if (make_key(v[i], static_cast<uint32_t>(c)) >= bound) visit(make_key(v[i], static_cast<uint32_t>(i0 + i)));
      }
    }
  };
  scan([&](uint64_t k) {
    const int at = atomicAdd(&sh.count, 1);
    if (at < kCap) sh.cand[at] = k;
  });
  __syncthreads();
  const int count = sh.count;
  if (count <= kCap) {
    rank_out(sh.cand, count, n, out);
    return;
  }
  // more candidates than fit (a few threads hold most of the row's largest):
  // take them one by one, each the largest below the last
  uint64_t last = ~uint64_t{0};
  for (int i = 0; i < n; ++i) {
    if (tid == 0) sh.best = 0;
    __syncthreads();
    uint64_t k = 0;
    scan([&](uint64_t c) {
      if (c < last && c > k) k = c;
    });
    if (k) atomicMax(reinterpret_cast<unsigned long long*>(&sh.best), static_cast<unsigned long long>(k));
    __syncthreads();
    last = sh.best;
    if (tid == 0) out(i, last);
    __syncthreads();
  }
}

// What a row's statistics say: no distribution when the sum is not a positive
// finite number (all masked, or a NaN or +inf among the logits).
struct Result {
  Stat a;
  bool ok;
  float log_s;   // log of the sum as it is (the library's logf: the hardware's log2 loses digits where a likely
                 // token leaves s near 1)
  float log_sm;  // relative to m itself: m2's rounding taken out
  __device__ __forceinline__ explicit Result(const Stat& st) : a(st) {
    ok = st.s > 0.0f && st.s < INFINITY;
    log_s = ok ? logf(st.s) : 0.0f;
    log_sm = fmaf(-kLn2, excess(st.m), log_s);
  }
  __device__ __forceinline__ float lse() const {
    if (!ok) return a.s == 0.0f ? -INFINITY : NAN;
    return a.m + log_sm;
  }
  __device__ __forceinline__ float logprob(float l) const {
    if (!ok) return NAN;
    return (l - a.m) - log_sm;
  }
  __device__ __forceinline__ float entropy() const { return ok ? log_s - kLn2 * (a.t / a.s) : NAN; }
};

template <typename T>
__device__ __forceinline__ void write_row(const LArgs& a, int64_t r, const Result& res) {
  const int32_t t = a.targets[r];
  float lp = NAN;
  if (t >= 0 && t < a.vocab) lp = res.logprob(Row<T>::one(static_cast<const T*>(a.logits) + r * a.stride + t));
  a.logprob[r] = lp;
  if (a.lse) a.lse[r] = res.lse();
  if (a.entropy) a.entropy[r] = res.entropy();
}

__device__ __forceinline__ void write_top(const LArgs& a, int64_t r, const Result& res, int rank, uint64_t k) {
  const bool ok = res.ok && k != 0;
  a.top_ids[r * a.top_n + rank] = ok ? static_cast<int32_t>(key_pos(k)) : -1;
  a.top_lp[r * a.top_n + rank] = ok ? res.logprob(key_value(k)) : NAN;
}

// Workgroup (split, row): thread i takes chunks c0 + i, c0 + i + 512, ..., four
// loads in flight.
template <typename T>
__global__ __launch_bounds__(kThreads, 8) void logprobs_kernel(LArgs a) {
  __shared__ SelectSmem sh;
  __shared__ Stat wst[kWaves];
  constexpr int kE = Row<T>::kE;
  constexpr int kFlight = 4;
  const int tid = threadIdx.x;
  const int split = blockIdx.x % a.splits;
  const int64_t r = blockIdx.x / a.splits;
  const RowView<T> row(static_cast<const T*>(a.logits) + r * a.stride, a.vocab);
  const int c0 = static_cast<int>(min(static_cast<int64_t>(row.chunks), split * a.per));
  const int c1 = static_cast<int>(min(static_cast<int64_t>(row.chunks), c0 + a.per));

  Stat st{-INFINITY, 0.0f, 0.0f};
  float best = -INFINITY;
  int best_chunk = -1;
  auto add = [&](const float (&v)[kE]) {
    const float m = st.m == -INFINITY ? 0.0f : st.m;
    if (!wide(m)) {
      const float m2 = m2_of(m);
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        const float x = fmaf(v[i], kLog2e, -m2);
        const float e = __builtin_amdgcn_exp2f(x);
        st.s += e;
        st.t = fmaf(e, fmaxf(x, kFloor), st.t);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        const float x = (v[i] - m) * kLog2e;
        const float e = __builtin_amdgcn_exp2f(x);
        st.s += e;
        st.t = fmaf(e, fmaxf(x, kFloor), st.t);
      }
    }
  };
  auto top = [&](const float (&v)[kE], int c) {
    float cm = v[0];
#pragma unroll
    for (int i = 1; i < kE; ++i) cm = fmaxf(cm, v[i]);
    if (cm > best || best_chunk < 0) {
      best = cm;
      best_chunk = c;
    }
  };
  auto one = [&](int c) {
    float v[kE];
    row.load(c, v);
    top(v, c);
    if (best > st.m) rescale(st, best);
    add(v);
  };
  int c = c0 + tid;
  if (c < c1 && !row.whole(c)) {  // the row's first chunk, if it starts inside one (or its only one)
    one(c);
    c += kThreads;
  }
  const int cw = c1 - (c1 > c0 && !row.whole(c1 - 1) ? 1 : 0);  // whole chunks end here
  for (; c + (kFlight - 1) * kThreads < cw; c += kFlight * kThreads) {
    u32x4_t w[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) w[f] = row.raw(c + f * kThreads);
    // the running maximum moves at most once per four chunks
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      float v[kE];
      Row<T>::unpack(w[f], v);
      top(v, c + f * kThreads);
    }
    if (best > st.m) rescale(st, best);
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      float v[kE];
      Row<T>::unpack(w[f], v);
      add(v);
    }
  }
  for (; c < c1; c += kThreads) one(c);
  st = merge_wave(st);
  if ((tid & 63) == 0) wst[tid >> 6] = st;
  __syncthreads();
  st = wst[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) st = merge(st, wst[w]);

  if (a.splits == 1) {
    const Result res(st);
    if (tid == 0) write_row<T>(a, r, res);
    if (a.top_n)
      select_top(row, c0, c1, a.top_n, best, best_chunk, sh,
                 [&](int rank, uint64_t k) { write_top(a, r, res, rank, k); });
  } else {
    const int64_t at = r * a.splits + split;
    if (tid == 0) *reinterpret_cast<float4*>(a.stats + at * 4) = make_float4(st.m, st.s, st.t, 0.0f);
    if (a.top_n)
      select_top(row, c0, c1, a.top_n, best, best_chunk, sh,
                 [&](int rank, uint64_t k) { a.keys[at * a.top_n + rank] = k; });
  }
}

// Joins the splits of a row: one workgroup a row.  Every split's list is
// sorted, so the n-th largest of the lists' heads bounds the n-th largest key,
// as in select_top.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprobs_join_kernel(LArgs a) {
  __shared__ uint64_t cand[kCap];
  __shared__ uint64_t bound;
  __shared__ int count;
  __shared__ Stat total;
  constexpr int kKeys = kMaxSplits * kMaxTop / kThreads;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.x;
  const uint64_t* keys = a.keys + r * a.splits * a.top_n;
  const int n_keys = a.splits * a.top_n;
  uint64_t mine[kKeys];
#pragma unroll
  for (int i = 0; i < kKeys; ++i) mine[i] = tid + i * kThreads < n_keys ? keys[tid + i * kThreads] : 0;
  if (tid == 0) count = 0;
  if (tid < 64) {
    Stat st{-INFINITY, 0.0f, 0.0f};
    uint64_t head = 0;
    if (tid < a.splits) {
      const float4 v = *reinterpret_cast<const float4*>(a.stats + (r * a.splits + tid) * 4);
      st = Stat{v.x, v.y, v.z};
      if (a.top_n) head = keys[tid * a.top_n];
    }
    st = merge_wave(st);
    if (a.top_n) {
      const uint64_t b = nth_of_wave(head, a.top_n);
      if (tid == 0) bound = b;
    }
    if (tid == 0) total = st;
  }
  __syncthreads();
  const Result res(total);
  if (tid == 0) write_row<T>(a, r, res);
  if (!a.top_n) return;
  // only the lists whose head reaches the bound hold such keys: top_n^2 at most
#pragma unroll
  for (int i = 0; i < kKeys; ++i)
    if (mine[i] != 0 && mine[i] >= bound) cand[atomicAdd(&count, 1)] = mine[i];
  __syncthreads();
  rank_out(cand, count, a.top_n, [&](int rank, uint64_t k) { write_top(a, r, res, rank, k); });
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------

struct BArgs {
  const void* logits;
  int64_t stride;
  int64_t rows;
  int64_t vocab;
  const int32_t* targets;
  const float* lse;
  const float* entropy;
  const float* g_lp;
  const float* g_ent;
  void* out;
  int64_t out_stride;
};

// bf16 of fp32, round to nearest even
__device__ __forceinline__ uint32_t bf16_bits(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

template <typename T>
__device__ __forceinline__ u32x4_t pack(const float (&v)[Row<T>::kE]) {
  u32x4_t o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) o[i] = __builtin_bit_cast(uint32_t, v[i]);
    else o[i] = bf16_bits(v[2 * i]) | (bf16_bits(v[2 * i + 1]) << 16);
  }
  return o;
}

constexpr int kBwdThreads = 256;
constexpr int kBwdChunks = 8;       // chunks per thread
constexpr int kBwdChunksSmall = 2;  // where that would leave CUs idle

// d l_i = g_lp (1[i = target] - p_i) - g_ent p_i (log p_i + H), element by
// element: workgroup (part, row).  Reads a row once and writes it once; the
// same thread reads and writes an element, so `out` may be the logits.
template <typename T, int kChunks>
__global__ __launch_bounds__(kBwdThreads) void logprobs_bwd_kernel(BArgs a, int parts) {
  constexpr int kE = Row<T>::kE;
  const int64_t r = blockIdx.x / parts;
  const int part = blockIdx.x % parts;
  const RowView<T> row(static_cast<const T*>(a.logits) + r * a.stride, a.vocab);
  T* out = static_cast<T*>(a.out) + r * a.out_stride;
  // both rows on the same 16-byte phase: whole chunks move 16 bytes at a time
  const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row.p)) & 15) == 0;
  const float lse = a.lse[r];
  const int32_t tgt = a.targets[r];
  const bool has = tgt >= 0 && tgt < a.vocab;
  const float g = a.g_lp && has ? a.g_lp[r] : 0.0f;
  const float ge = a.g_ent ? a.g_ent[r] : 0.0f;
  const float ent = a.g_ent ? a.entropy[r] : 0.0f;
  const bool empty = lse == -INFINITY;
  auto grad = [&](float (&v)[kE], int i0) {
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      const float lp = v[i] - lse;
      const float p = __builtin_amdgcn_exp2f(lp * kLog2e);
      v[i] = empty ? 0.0f : -p * fmaf(ge, fmaxf(lp, kFloor) + ent, g);
    }
    const int at = tgt - i0;
    if (at >= 0 && at < kE && !empty) {
#pragma unroll
      for (int i = 0; i < kE; ++i)
        if (i == at) v[i] += g;
    }
  };
  // whole chunks first, all loads in flight together; then the ends of the row
  // (and everything, where the two rows' phases differ) element by element
  const int first = part * kChunks * kBwdThreads + threadIdx.x;
  u32x4_t w[kChunks];
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int c = first + j * kBwdThreads;
    if (same && row.whole(c)) w[j] = row.raw(c);
  }
#pragma unroll
  for (int j = 0; j < kChunks; ++j) {
    const int c = first + j * kBwdThreads;
    if (same && row.whole(c)) {
      float v[kE];
      Row<T>::unpack(w[j], v);
      grad(v, row.first(c));
      __builtin_nontemporal_store(pack<T>(v), reinterpret_cast<u32x4_t*>(out + row.first(c)));
    }
  }
  for (int j = 0; j < kChunks; ++j) {
    const int c = first + j * kBwdThreads;
    if (c >= row.chunks || (same && row.whole(c))) continue;
    float v[kE];
    row.load(c, v);
    const int i0 = row.first(c);
    grad(v, i0);
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      if (i0 + i < 0 || i0 + i >= row.vocab) continue;
      if constexpr (sizeof(T) == 4) out[i0 + i] = v[i];
      else out[i0 + i] = static_cast<T>(bf16_bits(v[i]));
    }
  }
}

}  // namespace

// Few rows leave most of the chip idle, so a row is cut into splits until
// about two workgroups a CU are busy, down to one chunk a thread (below that
// a split would cost its launch and join more than it saves).
LogprobsPlan plan_logprobs(int64_t rows, int64_t vocab, int elem_bytes, int top_n, int cus) {
  LogprobsPlan p{};
  const int64_t chunks = (vocab * elem_bytes + 15) / 16 + 1;  // one more where a row starts inside a chunk
  int64_t splits = rows > 0 ? (2 * cus) / rows : 1;
  splits = splits < chunks / kThreads ? splits : chunks / kThreads;
  if (splits > kMaxSplits) splits = kMaxSplits;
  if (splits < 1) splits = 1;
  p.per = (chunks + splits - 1) / splits;
  p.splits = static_cast<int>((chunks + p.per - 1) / p.per);
  if (p.splits > 1) {
    p.stats_bytes = (rows * p.splits * 16 + 255) / 256 * 256;
    p.bytes = p.stats_bytes + rows * p.splits * top_n * 8;
  }
  return p;
}

hipError_t launch_logprobs(const LogprobsArgs& g, const LogprobsPlan& plan, void* ws, hipStream_t s) {
  LArgs a{g.logits, g.stride, g.rows, g.vocab, g.targets, g.logprob, g.lse, g.entropy, g.top_ids, g.top_lp,
          g.top_n, plan.splits, plan.per, nullptr, nullptr};
  if (plan.splits > 1) {
    a.stats = static_cast<float*>(ws);
    a.keys = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + plan.stats_bytes);
  }
  const dim3 grid(static_cast<unsigned>(g.rows * plan.splits));
  if (g.bf16) hipLaunchKernelGGL(logprobs_kernel<uint16_t>, grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL(logprobs_kernel<float>, grid, dim3(kThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.splits == 1) return e;
  const dim3 jg(static_cast<unsigned>(g.rows));
  if (g.bf16) hipLaunchKernelGGL(logprobs_join_kernel<uint16_t>, jg, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL(logprobs_join_kernel<float>, jg, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

namespace {
int64_t bwd_parts(const LogprobsBwdArgs& g, int chunks_per_thread) {
  const int64_t esz = g.bf16 ? 2 : 4, per = 16 / esz;
  const bool alike = g.rows == 1 || g.stride * esz % 16 == 0;  // every row starts in its chunk where the first does
  const int64_t skew = alike ? (reinterpret_cast<uintptr_t>(g.logits) & 15) / esz : per - 1;
  const int64_t chunks = (g.vocab + skew + per - 1) / per;
  return (chunks + kBwdThreads * chunks_per_thread - 1) / (kBwdThreads * chunks_per_thread);
}
}  // namespace

int64_t logprobs_bwd_parts(const LogprobsBwdArgs& g) { return bwd_parts(g, kBwdChunks); }

hipError_t launch_logprobs_bwd(const LogprobsBwdArgs& g, hipStream_t s) {
  const BArgs a{g.logits, g.stride, g.rows, g.vocab, g.targets, g.lse, g.entropy, g.g_lp, g.g_ent, g.out, g.out_stride};
  const bool small = g.rows * bwd_parts(g, kBwdChunks) < 2 * cus_of_stream(s);
  const int64_t parts = bwd_parts(g, small ? kBwdChunksSmall : kBwdChunks);
  const dim3 grid(static_cast<unsigned>(g.rows * parts));
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(kBwdThreads), 0, s, a, static_cast<int>(parts)); };
  if (g.bf16) small ? go(logprobs_bwd_kernel<uint16_t, kBwdChunksSmall>) : go(logprobs_bwd_kernel<uint16_t, kBwdChunks>);
  else small ? go(logprobs_bwd_kernel<float, kBwdChunksSmall>) : go(logprobs_bwd_kernel<float, kBwdChunks>);
  return hipGetLastError();
}

}  // namespace stq
