// Softmax cross entropy of an output head, and its gradients, without keeping
// the logits.
//
//     l = x W^T (times the scales of 8-bit rows)
//     loss = log sum exp(l) - l_target
//     dl = g (softmax(l) - 1[target])       dx = dl W        dW = dl^T x
//
// Everything that costs is a product of rows with rows (the sum along both
// operands' memory), so one kernel does all of it, with what belongs to each
// product behind its sums: the running maximum and sum of exponentials of a
// tile of logits (forward), dl in bf16 (the logits once more, a piece of the
// vocabulary at a time), or sums stored or added up (dx, dW).  dl is stored both
// ways from the tile in LDS, and x transposed once, so that dW is such a product
// too; dx takes W as it lies, a row for every term of its sum, with transposing
// reads.  A piece has at most 2^26 logits (256 words under more than 2^18 rows), so
// that its dl, 134 MB, and its transpose stay near the 256 MB of the last-level cache.
//
// Sums are in fp32 (8-bit operands': exact, in int32), statistics in fp32.  dl
// is rounded to bf16 once, half a step of 2^-8 relative to each of its values,
// because the matrix cores take dx's and dW's factors in it.  The many small
// terms' roundings average out in dx; the target's is as large as all the others
// together, so what its rounding leaves is kept in fp32 and enters dx at the end.
// dW of few rows, where a target's term makes up its word's row, takes that rest
// as rows of its own; those of many rows average out there as well.
//
// 4096 rows under 131072 x 7168 in bf16: 5.2 to 5.3 ms, 1.46 PFLOP/s (a large
// library product 1.56); matrix cores 75 % busy at 1.8 of 2.4 GHz, so the card's
// power is the bound.  The same vocabulary's gradients: 2048 rows under the head
// in 8 bits 4.4 to 4.5 ms (8-bit logits 2.5 POP/s, dx 1.3 to 1.4 PFLOP/s), 4099
// rows under a bf16 head with dW 6.8 to 6.9 ms, 1.30 PFLOP/s.
#include <algorithm>
#include <type_traits>

#include "stq_launch.hpp"
#include "stq_rows.hpp"
#include "stq_device.hpp"

namespace stq {
namespace {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kXcds = 8;
constexpr int kStep = 64;         // bytes along the sum in one matrix-core step
constexpr int kBK = 2 * kStep;    // bytes along the sum in a stage

enum Epilogue { kStats, kGrad, kSum };

struct NtArgs {
  const char* a;          // "tokens": m rows, lda bytes apart
  int64_t lda;
  const char* w;          // "channels": n rows, ldw bytes apart
  int64_t ldw;
  int64_t m, n;
  int64_t kbytes;         // bytes of a row that count
  int64_t words;          // channels that lie along the other way: rows of w
  int tm, tn;             // tiles
  // logits
  const float* as;        // 8-bit rows: scales of tokens and channels
  const float* ws;
  const int32_t* targets;
  int64_t v0;             // vocabulary index of channel 0
  // kStats
  float2* stats;          // [parts][m]: maximum, sum of exp(l - maximum), a part for each wavefront along the channels
  float* hit;             // [m]: the target's logit
  // kGrad
  const float* lse;
  const float* g;
  int64_t vocab;          // the whole vocabulary
  uint16_t* dl;           // [m][ld_dl], zeros in channels n .. n_pad - 1
  int64_t ld_dl;
  float* rest;            // [m]: what the rounding of the target's dl leaves
  uint16_t* dlt;          // [n][ld_dlt], zeros in tokens m .. m_pad - 1; may be NULL
  int64_t ld_dlt;
  int64_t rest_at;        // few rows: the targets' rest in dlt's columns from here on, beside zeros; 0: not there
  int64_t n_pad, m_pad;
  const char* head;       // (dx) the whole head, for the targets' rows
  // kSum
  uint16_t* out;          // bf16 [m][ld_out]
  int64_t ld_out;
  // sums of channels that lie across
  float* acc;             // [splits][m][ld_acc], ld_acc a multiple of 8: where the sums go if out is NULL
  int64_t ld_acc;
  int add;                // begin with what acc holds
  int splits;             // parts of the sum
};

// Output channels of a pair of 16-row MFMA tiles: row r of tile h stands for
// channel 8 (r >> 2) + 4 h + (r & 3) of the pair's 32, so that a lane, which
// holds rows 4q .. 4q+3 of both tiles, ends with eight neighbouring channels.
__device__ __forceinline__ int pair_channel(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

__device__ __forceinline__ void lds_load16(Rsrc rs, void* lds, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      rs, reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(lds)), 16,
      static_cast<int>(voff), 0, 0, 0);
}

__device__ __forceinline__ uint32_t byte_mask(int bytes) {
  return bytes >= 4 ? 0xFFFFFFFFu : (1u << (8 * max(0, bytes))) - 1u;
}

// LDS slot of a row's 16-byte chunk (eight a row): the 16 rows that one
// operand read takes fall on 16 different 16-byte bank groups.
__device__ __forceinline__ int token_swizzle(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int channel_swizzle(int row) { return ((row >> 1) & 1) | ((row >> 2) & 6); }
// The same for the finished tile [token][channel], which is read along either
__device__ __forceinline__ int tile_swizzle(int t) { return 2 * ((t & 3) | ((t >> 1) & 4)); }

// Transposing LDS reads of 8 bytes a lane: 16 lanes give 4 rows of 16 16-bit
// elements, or 8 rows of 16 bytes, and lane r takes back column r.
__device__ __forceinline__ u32x2_t turned16(const char* at) {
  typedef int16_t i16x4_t __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)at));
}
__device__ __forceinline__ u32x2_t turned8(const char* at) {
  typedef int32_t i32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2_t*)at));
}

template <bool kI8>
struct Mfma;
template <>
struct Mfma<true> {
  typedef i32x4_t acc_t;
  static __device__ __forceinline__ acc_t run(u32x4_t w, u32x4_t a, acc_t c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, w), __builtin_bit_cast(i32x4_t, a), c, 0, 0, 0);
  }
};
template <>
struct Mfma<false> {
  typedef f32x4_t acc_t;
  static __device__ __forceinline__ acc_t run(u32x4_t w, u32x4_t a, acc_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w), __builtin_bit_cast(bf16x8_t, a), c, 0, 0, 0);
  }
};

// A row without a gradient: left out, its target past the vocabulary, or every logit -inf
__device__ __forceinline__ bool no_gradient(int64_t target, int64_t vocab, float lse) {
  return target < 0 || target >= vocab || lse == -INFINITY;
}

// What the rounding of d to bf16 leaves (nothing, if that is infinite or no number)
__device__ __forceinline__ float rounding_rest(float d) {
  const float f = __builtin_bit_cast(float, bf16_round(d) << 16);
  return fabsf(f) < INFINITY ? d - f : 0.0f;
}

// exp(x) with the error of exp2's rounded argument, |x| 2^-24 of it: a logit |x| below
// the largest is as far off in its own last digits, and its term then counts e^-|x|
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// Rows of bf16 that a wavefront holds as products, on their way to memory: 32
// tokens x kC channels of LDS of its own, 16-byte chunks XORed by the token so
// that whole rows and the transposing reads both fall on different banks.
template <int kC>
struct Slab {
  static constexpr int kChunks = kC / 8;
  char* mem;
  int lane;
  __device__ __forceinline__ char* at(int t, int chunk) const { return mem + t * kC * 2 + ((chunk ^ (tile_swizzle(t) & (kChunks - 1))) << 4); }
  // this wavefront's stores before, its loads after (LDS serves a wavefront in order)
  static __device__ __forceinline__ void fence() { asm volatile("" ::: "memory"); }
  // rows t < rows, chunks below `width` channels, to out
  __device__ __forceinline__ void store_rows(uint16_t* out, int64_t ld, int rows, int width) const {
#pragma unroll
    for (int i = 0; i < 32 * kChunks / 64; ++i) {
      const int t = (i * 64 + lane) / kChunks, c = (i * 64 + lane) % kChunks;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(at(t, c));
      if (t < rows && c * 8 < width) store16b(out + t * ld + c * 8, v);
    }
  }
  // the same transposed: out[channel][token], channels below `width`, tokens below `rows` (a multiple of 8).
  // 16 lanes give four tokens' 16 channels to the transposing read and each takes back four tokens of one.
  __device__ __forceinline__ void store_columns(uint16_t* out, int64_t ld, int rows, int width) const {
    const int q = lane >> 4, r = lane & 15;
    const int t = 8 * q + (r >> 2);
#pragma unroll
    for (int i = 0; i < kC / 16; ++i) {
      const uint32_t from = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at(t, 2 * i + ((r & 3) >> 1)))) + (r & 1) * 8;
      u32x2_t lo, hi;
      asm volatile("ds_read_b64_tr_b16 %0, %2\n\tds_read_b64_tr_b16 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
                   : "=&v"(lo), "=&v"(hi)
                   : "v"(from), "n"(4 * kC * 2)
                   : "memory");
      if (8 * q < rows && 16 * i + r < width)
        *reinterpret_cast<u32x4_t*>(out + (16 * i + r) * ld + 8 * q) = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
    }
  }
};

// What becomes of a wavefront's sums: FM x 16 tokens from m0, FN x 16 channels
// from n0, nv of them inside the product (less than 1: none).  A lane holds
// token 16 j + r, channels 32 p + 8 q + 0..7.  `part`: this wavefront's row of
// the statistics; `slab`: 32 x FN x 16 x 2 bytes of LDS of its own.
// kAcc: the sums are in accumulation registers, and leave them 16 tokens at a
// time.
template <bool kI8, int kEpi, int FM, int FN, bool kAcc>
__device__ __forceinline__ void finish(const NtArgs& a, typename Mfma<kI8>::acc_t (&acc)[FN][FM], int64_t m0, int64_t n0, int nv, int part,
                                       char* slab) {
  constexpr int kC = FN * 16, kP = FN / 2;
  // an opaque copy: what depends on the lane here is worked out here, not
  // before the products and kept (spilled) beside them
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  const int q = lane >> 4, r = lane & 15;
  // (dl's transpose has zeros for tokens up to a whole stage)
  if (m0 >= (kEpi == kGrad ? a.m_pad : a.m)) return;
  auto value = [&](int j, int p, int e) -> float { return static_cast<float>(acc[2 * p + (e >> 2)][j][e & 3]); };
  auto take = [&](int j) {
    if constexpr (kAcc) {
      static_assert(FN == 8, "the operands of this statement");
      asm volatile("" : "+a"(acc[0][j]), "+a"(acc[1][j]), "+a"(acc[2][j]), "+a"(acc[3][j]), "+a"(acc[4][j]), "+a"(acc[5][j]),
                   "+a"(acc[6][j]), "+a"(acc[7][j]));
    }
  };
  if constexpr (kEpi == kSum) {
    const Slab<kC> sl{slab, lane};
#pragma unroll
    for (int j = 0; j < FM; ++j) {   // whole rows, through LDS
      take(j);
      const int64_t tok = m0 + 16 * j + r;
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        const int c = 32 * p + 8 * q;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = value(j, p, e);
        const Raw8<bf16_t> o = pack8<bf16_t>(v);
        *reinterpret_cast<u32x4_t*>(sl.at(16 * (j & 1) + r, c / 8)) = o.w[0];
        // the last channels of an odd width belong to no whole chunk
        if (c + 8 > nv && c < nv && tok < a.m) store8<bf16_t>(reinterpret_cast<bf16_t*>(a.out) + tok * a.ld_out, n0 + c, a.n, o);
      }
      if ((j & 1) || j + 1 == FM) {
        sl.fence();
        const int64_t t0 = m0 + 16 * (j & ~1);
        sl.store_rows(a.out + t0 * a.ld_out + n0, a.ld_out, static_cast<int>(min(static_cast<int64_t>(16 + 16 * (j & 1)), a.m - t0)), nv & ~7);
        sl.fence();
      }
    }
    return;
  }
  float wsc[kP][8];
  if constexpr (kI8) {
#pragma unroll
    for (int p = 0; p < kP; ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e) wsc[p][e] = 32 * p + 8 * q + e < nv ? a.ws[n0 + 32 * p + 8 * q + e] : 0.0f;
  }
  int64_t target[FM];
  float ts[FM];
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int64_t tok = m0 + 16 * j + r;
    target[j] = tok < a.m ? a.targets[tok] : -1;
    ts[j] = kI8 && tok < a.m ? a.as[tok] : 1.0f;
  }
  auto logit = [&](int j, int p, int e) { return kI8 ? value(j, p, e) * ts[j] * wsc[p][e] : value(j, p, e); };
  if constexpr (kEpi == kStats) {
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      take(j);
      const int64_t tok = m0 + 16 * j + r;
      float l[kP][8];
#pragma unroll
      for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) l[p][e] = logit(j, p, e);
      const int64_t want = target[j] - a.v0 - n0 - 8 * q;   // (a target of -1 is below 0 here too)
      if (__any(target[j] >= 0 && want >= 0 && want < kC)) {
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (target[j] >= 0 && want == 32 * p + e && want + 8 * q < nv) a.hit[tok] = l[p][e];
      }
      if (nv < kC) {
#pragma unroll
        for (int p = 0; p < kP; ++p)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (32 * p + 8 * q + e >= nv) l[p][e] = -INFINITY;
      }
      float m = l[0][0];
#pragma unroll
      for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, l[p][e]);
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float base = m == -INFINITY ? 0.0f : m;
      float s[kP];
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        s[p] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s[p] += exp_of(l[p][e] - base);
      }
#pragma unroll
      for (int p = 1; p < kP; ++p) s[0] += s[p];
      s[0] += __shfl_xor(s[0], 16);
      s[0] += __shfl_xor(s[0], 32);
      if (q == 0 && tok < a.m) a.stats[part * a.m + tok] = float2{m, s[0]};
    }
  }
  if constexpr (kEpi == kGrad) {
    float lse[FM], g[FM];
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int64_t tok = m0 + 16 * j + r;
      lse[j] = tok < a.m ? a.lse[tok] : 0.0f;
      g[j] = tok < a.m ? a.g[tok] : 0.0f;
    }
    const Slab<kC> sl{slab, lane};
    constexpr bool kRestRows = !kI8 && FM <= 4;   // (the tiles of few rows)
    float rest[2];
    int hot_at[2];   // this lane's target: channels from 8 q on
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      take(j);
      if constexpr (kRestRows) rest[j & 1] = 0.0f, hot_at[j & 1] = -1;
      const bool dead = no_gradient(target[j], a.vocab, lse[j]);
      const float gj = dead ? 0.0f : g[j];
      const int64_t want = target[j] - a.v0 - n0 - 8 * q;
      const bool hot = __any(want >= 0 && want < kC);
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = exp_of(logit(j, p, e) - lse[j]);
        if (hot) {
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] -= want == 32 * p + e ? 1.0f : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[e] *= gj;
          if (kI8) d[e] *= wsc[p][e];
          if (dead) d[e] = 0.0f;
        }
        if (nv < kC) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (32 * p + 8 * q + e >= nv) d[e] = 0.0f;
        }
        *reinterpret_cast<u32x4_t*>(sl.at(16 * (j & 1) + r, 4 * p + q)) = pack8<bf16_t>(d).w[0];
        if (hot) {
          const int64_t at = want - 32 * p;
          if (!dead && at >= 0 && at < 8 && want + 8 * q < nv) {
            float t = d[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) t = at == e ? d[e] : t;
            t = rounding_rest(t);
            a.rest[m0 + 16 * j + r] = t;
            if constexpr (kRestRows) rest[j & 1] = t, hot_at[j & 1] = static_cast<int>(want);
          }
        }
      }
      if ((j & 1) || j + 1 == FM) {
        sl.fence();
        const int64_t t0 = m0 + 16 * (j & ~1);
        const int tokens = 16 + 16 * (j & 1);
        sl.store_rows(a.dl + t0 * a.ld_dl + n0, a.ld_dl, static_cast<int>(min(static_cast<int64_t>(tokens), a.m - t0)),
                      static_cast<int>(min(static_cast<int64_t>(kC), a.n_pad - n0)));
        if (a.dlt)
          sl.store_columns(a.dlt + n0 * a.ld_dlt + t0, a.ld_dlt, static_cast<int>(min(static_cast<int64_t>(tokens), a.m_pad - t0)), nv);
        if constexpr (kRestRows) {
          if (a.dlt && a.rest_at) {
            sl.fence();
#pragma unroll
            for (int h = 0; h <= (j & 1); ++h) {
#pragma unroll
              for (int p = 0; p < kP; ++p) *reinterpret_cast<u32x4_t*>(sl.at(16 * h + r, 4 * p + q)) = u32x4_t{0, 0, 0, 0};
              if (hot_at[h] >= 0)
                reinterpret_cast<uint16_t*>(sl.at(16 * h + r, 4 * (hot_at[h] >> 5) + q))[hot_at[h] & 7] = static_cast<uint16_t>(bf16_round(rest[h]));
            }
            sl.fence();
            sl.store_columns(a.dlt + n0 * a.ld_dlt + a.rest_at + t0, a.ld_dlt, static_cast<int>(min(static_cast<int64_t>(tokens), a.m_pad - t0)), nv);
          }
        }
        sl.fence();
      }
    }
  }
}

// Workgroup of WM x WN wavefronts, TM tokens x TN channels.  Both
// operands stream into LDS 128 bytes of the sum at a time (direct 16-byte
// loads) through kBuf buffers.  While the matrix cores work on one 64-byte
// step, the operands of the next are read from LDS: a token operand into the
// registers that its last use has just freed, the channel operands into a
// second set.  Halfway through a stage a barrier says that the next stage has
// landed and that every wavefront has the rest of this one in registers; the
// loads of stage s + kBuf then start into its buffer.
template <bool kI8, int kEpi, int TM, int TN, int WM, int WN, int kBuf, int kWavesPerSimd>
__global__ __launch_bounds__(WM * WN * 64, kWavesPerSimd) void nt_kernel(NtArgs a) {
  constexpr int kNW = WM * WN;
  constexpr int FM = TM / WM / 16, FN = TN / WN / 16;
  constexpr int NA = TM / 8 / kNW, NW = TN / 8 / kNW;  // load instructions a stage and wavefront, 8 rows each
  static_assert(FN % 2 == 0, "channel tiles come in pairs");
  static_assert(NA * 8 * kNW == TM && NW * 8 * kNW == TN, "every wavefront issues the same loads");
  static_assert(kBuf * (TM + TN) * kBK >= kNW * 32 * FN * 16 * 2, "the slabs fit where the stages were");
  typedef typename Mfma<kI8>::acc_t acc_t;
  __shared__ __align__(16) char smem[kBuf * (TM + TN) * kBK];
  char(*const sa)[TM * kBK] = reinterpret_cast<char(*)[TM * kBK]>(smem);
  char(*const sw)[TN * kBK] = reinterpret_cast<char(*)[TN * kBK]>(smem + kBuf * TM * kBK);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;
  // Workgroups are dealt to the XCDs in turn: each XCD takes one run of tiles,
  // in bands of 8 token tiles, so that its L2 serves a compact block of both
  // operands.
  const int tiles = a.tm * a.tn;
  const int per = (tiles + kXcds - 1) / kXcds;
  const int id = (blockIdx.x % kXcds) * per + blockIdx.x / kXcds;
  if (id >= tiles) return;
  const int band = id / (8 * a.tn), rows = min(8, a.tm - band * 8), in = id - band * 8 * a.tn;
  const int tile_n = in / rows;
  const int64_t m0 = static_cast<int64_t>(band * 8 + in % rows) * TM, n0 = static_cast<int64_t>(tile_n) * TN;
  const int mv = static_cast<int>(min(static_cast<int64_t>(TM), a.m - m0));
  const int nv = static_cast<int>(min(static_cast<int64_t>(TN), a.n - n0));
  const uint32_t kpad = static_cast<uint32_t>((a.kbytes + 15) & ~15);
  const Rsrc ra = make_rsrc(a.a + m0 * a.lda, static_cast<uint32_t>((mv - 1) * a.lda) + kpad);
  const Rsrc rw = make_rsrc(a.w + n0 * a.ldw, static_cast<uint32_t>((nv - 1) * a.ldw) + kpad);
  uint32_t va[NA], vw[NW];
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int row = (wave + i * kNW) * 8 + (lane >> 3);
    va[i] = row * static_cast<uint32_t>(a.lda) + (((lane & 7) ^ token_swizzle(row)) << 4);
  }
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const int row = (wave + i * kNW) * 8 + (lane >> 3);
    vw[i] = row * static_cast<uint32_t>(a.ldw) + (((lane & 7) ^ channel_swizzle(row)) << 4);
  }
  const int ns = static_cast<int>((a.kbytes + kBK - 1) / kBK);
  auto stage = [&](int s, int buf) {
#pragma unroll
    for (int i = 0; i < NA; ++i) lds_load16(ra, sa[buf] + (wave + i * kNW) * 1024, va[i] + s * kBK);
#pragma unroll
    for (int i = 0; i < NW; ++i) lds_load16(rw, sw[buf] + (wave + i * kNW) * 1024, vw[i] + s * kBK);
  };
  acc_t acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = acc_t{0, 0, 0, 0};
  const int wm = wave / WN, wn = wave % WN;
  const int tok_row = wm * FM * 16 + r;
  const int ch_row = wn * FN * 16 + pair_channel(r, 0);
  int oa[2], ow[2];  // this lane's chunk of either step
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    oa[h] = tok_row * kBK + (((4 * h + q) ^ token_swizzle(tok_row)) << 4);
    ow[h] = ch_row * kBK + (((4 * h + q) ^ channel_swizzle(ch_row)) << 4);
  }
  u32x4_t fa[FM], fw[2][FN];
  auto read_w = [&](int buf, int h, int i) {
    return *reinterpret_cast<const u32x4_t*>(sw[buf] + ow[h] + ((i >> 1) * 32 + (i & 1) * 4) * kBK);
  };
  auto read_a = [&](int buf, int h, int j) { return *reinterpret_cast<const u32x4_t*>(sa[buf] + oa[h] + j * 16 * kBK); };
  // Product group j of a step (token operand j with every channel operand),
  // then the reads that its registers were waiting for: token operand j of
  // the next step, and with group j0 the channel operands and the token
  // operands of the groups before it.
  auto group = [&](int h, int j) {
#pragma unroll
    for (int i = 0; i < FN; ++i) acc[i][j] = Mfma<kI8>::run(fw[h][i], fa[j], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto reads = [&](int h, int j, int j0, int next_buf) {
    if (j == j0) {
#pragma unroll
      for (int i = 0; i < FN; ++i) fw[h ^ 1][i] = read_w(next_buf, h ^ 1, i);
#pragma unroll
      for (int e = 0; e < j0; ++e) fa[e] = read_a(next_buf, h ^ 1, e);
    }
    if (j >= j0) fa[j] = read_a(next_buf, h ^ 1, j);
    __builtin_amdgcn_sched_barrier(0);
  };
  // Bytes of the last stage past the end of the sum count for nothing, whatever
  // the rows hold there: zeros in the token operand, and, where a bf16 NaN
  // times zero would be one, in the channel operand.
  auto mask = [&](int s, int h) {
    const int left = static_cast<int>(a.kbytes) - (s * kBK + h * kStep + q * 16);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t m = byte_mask(left - 4 * d);
#pragma unroll
      for (int j = 0; j < FM; ++j) fa[j][d] &= m;
      if constexpr (!kI8) {
#pragma unroll
        for (int i = 0; i < FN; ++i) fw[h][i][d] &= m;
      }
    }
  };
  if (ns > 0) {
#pragma unroll
    for (int s = 0; s < kBuf; ++s)
      if (s < ns) stage(s, s);
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int i = 0; i < FN; ++i) fw[0][i] = read_w(0, 0, i);
#pragma unroll
    for (int j = 0; j < FM; ++j) fa[j] = read_a(0, 0, j);
    int buf = 0;
    for (int s = 0; s + 1 < ns; ++s) {
      const int next = buf + 1 == kBuf ? 0 : buf + 1;
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        group(0, j);
        reads(0, j, 0, buf);
      }
      // The second step's first group needs nothing of the next stage, and
      // covers the last of these reads.  Then stages s + 1 .. s + kBuf - 1 are
      // in flight (fewer near the end): wait for the first of them, for this
      // wavefront's own LDS reads and for the other wavefronts.  (The
      // compiler's barrier would wait for every load.)
      group(1, 0);
      if (s + kBuf - 1 >= ns) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NA + NW) * (kBuf - 2)) : "memory");
      if (s + kBuf < ns) stage(s + kBuf, buf);
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        if (j) group(1, j);
        reads(1, j, FM > 1 ? 1 : 0, next);
      }
      buf = next;
    }
    const bool tail = a.kbytes % kBK != 0;
    if (tail) mask(ns - 1, 0);
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      group(0, j);
      reads(0, j, 0, buf);
    }
    if (tail) mask(ns - 1, 1);
#pragma unroll
    for (int j = 0; j < FM; ++j) group(1, j);
  }

  // everyone has read the last stage
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  finish<kI8, kEpi, FM, FN, false>(a, acc, m0 + wm * FM * 16, n0 + wn * FN * 16, min(static_cast<int>(nv) - wn * FN * 16, FN * 16),
                            tile_n * WN + wn, smem + wave * (32 * FN * 16 * 2));
}

// How the channel operand lies in memory: a row for every channel, like the
// token operand, or a row for every term of the sum (bf16, or 8-bit integers
// that become bf16, which holds them exactly).
enum Lies { kRows, kAcross16, kAcross8 };

// Columns c .. c + 3 (c a multiple of 4) of a row of the head as they lie, and their values
template <bool k8>
__device__ __forceinline__ float head_value(u32x2_t v, int e) {
  if constexpr (k8) return static_cast<float>(static_cast<int8_t>(v[0] >> (8 * e)));
  else return __builtin_bit_cast(float, (e & 1) ? (v[e >> 1] & 0xFFFF0000u) : (v[e >> 1] << 16));
}
template <bool k8>
__device__ __forceinline__ u32x2_t head4(const char* row, int64_t c) {
  if constexpr (k8) return u32x2_t{*reinterpret_cast<const uint32_t*>(row + c), 0};
  else return *reinterpret_cast<const u32x2_t*>(row + 2 * c);
}

// Rows of 16 lanes 1 and 3 of x and 0 and 2 of y change places
__device__ __forceinline__ void exchange16(uint32_t& x, uint32_t& y) {
  const auto o = __builtin_amdgcn_permlane16_swap(x, y, false, false);
  x = o[0];
  y = o[1];
}

// 16 channels of one row of tiles of a wavefront that read its operand across:
// lane (q, r) holds token 16 j + r, channels 16 i + 4 q + 0..3.  Sums only.
template <int kLies, int FM, int FN>
__device__ __forceinline__ void finish_across(const NtArgs& a, f32x4_t (&acc)[FN][FM], int64_t m0, int64_t n0, int nv, int split, char* slab) {
  constexpr int kC = FN * 16;
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  const int q = lane >> 4, r = lane & 15;
  if (m0 >= a.m) return;
  const Slab<kC> sl{slab, lane};
  // Whole sums: the targets' rest times their rows of the head, which are on their
  // way while the 16 tokens before are put away.  A lane loads eight channels, for
  // itself and the lane 16 from it, of fragment 2 i or 2 i + 1, and they exchange
  // halves.  (4000 rows of 1024 under 600 words, one round of tiles: 28 us, 34 with
  // a lane's own four channels loaded where they are used, 23 without the rest.)
  constexpr bool k8 = kLies == kAcross8;
  int32_t target[FM];   // -1: no gradient
  float rest = 0.0f;
  using Chunk = std::conditional_t<k8, u32x2_t, u32x4_t>;
  Chunk hot[FN / 2];
  auto rows_of = [&](int j) {
    rest = a.rest[min(m0 + 16 * j + r, a.m - 1)];
#pragma unroll
    for (int i = 0; i < FN / 2; ++i) {
      const int c = 32 * i + 16 * (q & 1) + 8 * (q >> 1);
      hot[i] = Chunk{};
      if (target[j] >= 0 && c < nv)
        hot[i] = *reinterpret_cast<const Chunk*>(a.head + target[j] * a.ldw + (n0 + c) * (k8 ? 1 : 2));
    }
  };
  if (a.out) {
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int64_t tok = min(m0 + 16 * j + r, a.m - 1);
      const int32_t t = a.targets[tok];
      target[j] = no_gradient(t, a.vocab, a.lse[tok]) ? -1 : t;
    }
    rows_of(0);
  }
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    static_assert(FN == 8, "the operands of this statement");
    asm volatile("" : "+a"(acc[0][j]), "+a"(acc[1][j]), "+a"(acc[2][j]), "+a"(acc[3][j]), "+a"(acc[4][j]), "+a"(acc[5][j]),
                 "+a"(acc[6][j]), "+a"(acc[7][j]));
    const int64_t tok = m0 + 16 * j + r;
    f32x4_t v[FN];
#pragma unroll
    for (int i = 0; i < FN; ++i) v[i] = acc[i][j];
    float* const row = a.acc + (split * a.m + tok) * a.ld_acc + n0 + 4 * q;
    if (a.out) {   // whole rows, through LDS
#pragma unroll
      for (int i = 0; i < FN / 2; ++i) {
        u32x2_t w[2];
        if constexpr (k8) {
          uint32_t lo = hot[i][0], hi = hot[i][1];
          exchange16(lo, hi);
          w[0] = u32x2_t{lo, 0}, w[1] = u32x2_t{hi, 0};
        } else {
          uint32_t lo[2] = {hot[i][0], hot[i][1]}, hi[2] = {hot[i][2], hot[i][3]};
          exchange16(lo[0], hi[0]);
          exchange16(lo[1], hi[1]);
          w[0] = u32x2_t{lo[0], lo[1]}, w[1] = u32x2_t{hi[0], hi[1]};
        }
        // (zeros without a gradient, under an infinite head too, where dl = 0 gives NaN)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[2 * i + h][e] = target[j] < 0 ? 0.0f : fmaf(rest, head_value<k8>(w[h], e), v[2 * i + h][e]);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (j + 1 < FM) rows_of(j + 1);
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const int c = 16 * i + 4 * q;
        const uint32_t o[4] = {bf16_round(v[i][0]), bf16_round(v[i][1]), bf16_round(v[i][2]), bf16_round(v[i][3])};
        *reinterpret_cast<u32x2_t*>(sl.at(16 * (j & 1) + r, 2 * i + (q >> 1)) + (q & 1) * 8) = u32x2_t{o[0] | o[1] << 16, o[2] | o[3] << 16};
        // the last channels of an odd width belong to no whole chunk
        if (c >= (nv & ~7) && c < nv && tok < a.m) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < nv) a.out[tok * a.ld_out + n0 + c + e] = static_cast<uint16_t>(o[e]);
        }
      }
      if ((j & 1) || j + 1 == FM) {
        sl.fence();
        const int64_t t0 = m0 + 16 * (j & ~1);
        sl.store_rows(a.out + t0 * a.ld_out + n0, a.ld_out, static_cast<int>(min(static_cast<int64_t>(16 + 16 * (j & 1)), a.m - t0)), nv & ~7);
        sl.fence();
      }
    } else if (tok < a.m) {
#pragma unroll
      for (int i = 0; i < FN; ++i)
        if (16 * i + 4 * q < nv) *reinterpret_cast<f32x4_t*>(row + 16 * i) = v[i];
    }
  }
}

// 256 x 256 tiles: four wavefronts of 128 x 128, one a SIMD, so that an operand
// read from LDS serves eight products.  Nothing but its own order hides what
// such a wavefront waits for, so the order is written out: a product, then at
// most one LDS read of the next step's operands and one load.  The channel
// operand has three buffers: its loads run a stage and a half ahead, between
// the products of a stage's first step, the token operand's between those of
// the second; all in one step would queue for 1024 cycles behind each other.
// Workgroups stay and walk the tiles of their XCD; a tile's first loads start
// before the previous tile's sums are put away.  (4096 rows x 65536 words x
// 7168: 1.32 PFLOP/s with eight wavefronts of 128 x 64 and two buffers, 1.43
// with four, 1.46 with the third buffer.)
//
// A channel operand that lies across is read with the transposing LDS reads,
// 64 rows of 256 channels a stage; 8-bit integers become bf16 between the
// products, two and their packing at a time, so that three vector instructions
// follow a product at most, which is what one of 16 cycles hides.  (Gradient of
// 2048 rows under 131072 x 7168 in 8 bits: 4.4 ms, 5.0 with each piece of the
// head transposed in front of the product; of 4099 rows under 50021 x 7168 in
// bf16, both gradients: 6.8 and 7.2.)
template <bool kI8, int kEpi, int kLies>
__global__ __launch_bounds__(256, 1) void nt_wide_kernel(NtArgs a) {
  static_assert(kLies == kRows || (!kI8 && kEpi == kSum), "the gradient's products alone read across");
  constexpr int T = 256, F = 8, kLoads = 8, kProducts = F * F;
  constexpr int kRead0 = 3, kLoad0 = 4, kRead1 = 4, kLoad1 = 4;  // products between them
  static_assert(kRead0 * 2 * F <= kProducts && kRead1 * 2 * F <= kProducts && kLoad0 * kLoads <= kProducts, "a step's reads fit into it");
  constexpr bool kAcross = kLies != kRows;
  constexpr int kWStage = kLies == kAcross8 ? T * kBK / 2 : T * kBK, kWLoads = kWStage / 1024 / 4;
  constexpr int kWElem = kLies == kAcross8 ? 1 : 2, kWRow = T * kWElem;   // (across) bytes of an element and of a row in LDS
  constexpr int kSlabs = 4 * 32 * 128 * 2;
  // (two objects: the compiler then knows the transposing reads for reads of
  // one, and puts no wait for every load to LDS in front of each)
  __shared__ __align__(16) char sa[2][T * kBK];
  __shared__ __align__(16) char channel_mem[3 * kWStage > 2 * kWStage + kSlabs ? 3 * kWStage : 2 * kWStage + kSlabs];
  char(*const sw)[kWStage] = reinterpret_cast<char(*)[kWStage]>(channel_mem);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15, wm = wave >> 1, wn = wave & 1;
  // (across, the sum may be shared out: one part after the other, each with all its tiles)
  const int tiles = a.tm * a.tn, splits = kAcross ? a.splits : 1, all = tiles * splits;
  const int per = (all + kXcds - 1) / kXcds, last = min(all, static_cast<int>(blockIdx.x % kXcds + 1) * per);
  const int ns = static_cast<int>((a.kbytes + kBK - 1) / kBK), chunk = (ns + splits - 1) / splits;
  const uint32_t kpad = static_cast<uint32_t>((a.kbytes + 15) & ~15);
  uint32_t va[kLoads], vw[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int row = (wave + 4 * i) * 8 + (lane >> 3);
    va[i] = row * static_cast<uint32_t>(a.lda) + (((lane & 7) ^ token_swizzle(row)) << 4);
    if constexpr (!kAcross) vw[i] = row * static_cast<uint32_t>(a.ldw) + (((lane & 7) ^ channel_swizzle(row)) << 4);
  }
  // across: a row's 16-byte chunks are XORed by the row, so that the rows that
  // one transposing read takes (16, or 32 of 8 bits) fall on all banks evenly
  auto across_swizzle = [](int t) { return kLies == kAcross8 ? t & 15 : tile_swizzle(t); };
  uint32_t ow_across = 0;   // this lane's place in a stage: fragment 0 of the wavefront's eight
  if constexpr (kAcross) {
    constexpr int kChunks = kWRow / 16;
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) {
      const int t = (wave + 4 * i) * (64 / kChunks) + lane / kChunks;
      vw[i] = t * static_cast<uint32_t>(a.ldw) + ((lane % kChunks ^ across_swizzle(t)) << 4);
    }
    // bf16: 16 lanes give 4 rows' 16 channels, 8 bytes a lane, and each takes back 4 rows of one; 8-bit: 8 rows' 16
    const int t = 8 * q + (kLies == kAcross8 ? r >> 1 : r >> 2);
    const int chunk = kLies == kAcross8 ? wn * F : wn * 2 * F + ((r & 3) >> 1);
    ow_across = t * kWRow + ((chunk ^ across_swizzle(t)) << 4) + (r & 1) * 8;
  }
  int oa[2], ow[2];  // this lane's chunk of either step
  const int tok_row = wm * 128 + r, ch_row = wn * 128 + pair_channel(r, 0);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    oa[h] = tok_row * kBK + (((4 * h + q) ^ token_swizzle(tok_row)) << 4);
    ow[h] = ch_row * kBK + (((4 * h + q) ^ channel_swizzle(ch_row)) << 4);
  }
  struct Place {
    int64_t m0, n0;
    int tile_n, split, s0, s1;   // stages s0 .. s1 - 1
  };
  auto place = [&](int id) {
    const int split = kAcross ? id / tiles : 0;
    if constexpr (kAcross) id -= split * tiles;
    const int band = id / (8 * a.tn), rows = min(8, a.tm - band * 8), in = id - band * 8 * a.tn;
    return Place{static_cast<int64_t>(band * 8 + in % rows) * T, static_cast<int64_t>(in / rows) * T, in / rows, split,
                 kAcross ? split * chunk : 0, kAcross ? min(ns, (split + 1) * chunk) : ns};
  };
  auto tokens = [&](const Place& p, bool on) {
    const int mv = static_cast<int>(min(static_cast<int64_t>(T), a.m - p.m0));
    return make_rsrc(a.a + p.m0 * a.lda, on ? static_cast<uint32_t>((mv - 1) * a.lda) + kpad : 0);
  };
  auto channels = [&](const Place& p, bool on, int s) {
    if constexpr (kAcross) {
      constexpr int kStageRows = kBK / 2;
      const int64_t w0 = static_cast<int64_t>(s) * kStageRows;
      const int rows = static_cast<int>(min(static_cast<int64_t>(kStageRows), a.words - w0));
      const uint32_t width = static_cast<uint32_t>(((a.n * kWElem + 15) & ~int64_t{15}) - p.n0 * kWElem);
      return make_rsrc(a.w + (on ? w0 * a.ldw : 0) + p.n0 * kWElem, on ? static_cast<uint32_t>((rows - 1) * a.ldw) + width : 0);
    }
    const int nv = static_cast<int>(min(static_cast<int64_t>(T), a.n - p.n0));
    return make_rsrc(a.w + p.n0 * a.ldw, on ? static_cast<uint32_t>((nv - 1) * a.ldw) + kpad : 0);
  };
  // the first two stages (the second reads as zeros where there is none)
  auto begin = [&](const Place& p) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int s = p.s0 + b;
      const Rsrc ra = tokens(p, s < p.s1), rw = channels(p, s < p.s1, s);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) lds_load16(ra, sa[b] + (wave + 4 * i) * 1024, va[i] + s * kBK);
#pragma unroll
      for (int i = 0; i < kWLoads; ++i) lds_load16(rw, sw[b] + (wave + 4 * i) * 1024, vw[i] + (kAcross ? 0 : s * kBK));
    }
  };
  int id = static_cast<int>(blockIdx.x % kXcds) * per + static_cast<int>(blockIdx.x) / kXcds;
  if (id >= last) return;
  Place p = place(id);
  begin(p);
  for (;;) {
    typename Mfma<kI8>::acc_t acc[F][F];
    u32x4_t fa[2][F], fw[2][F];
    u32x2_t raw[F];   // 8-bit channels on their way to fw
    // Earlier pieces' sums are where these begin: read all at once, they cost one
    // latency (added at the end, 16 tokens at a time, they cost eight).
    if (kAcross && a.add) {
      if constexpr (kAcross) {
        const int64_t m = p.m0 + wm * 128;
        const int rows = static_cast<int>(max(int64_t{0}, min(int64_t{128}, a.m - m)));
        const Rsrc rs = make_rsrc(a.acc + (p.split * a.m + m) * a.ld_acc + p.n0, static_cast<uint32_t>(rows * a.ld_acc - (rows ? p.n0 : 0)) * 4);
        // (channels past a row's end are another row's, and nobody's results)
        const uint32_t at = (r * static_cast<uint32_t>(a.ld_acc) + wn * 128 + 4 * q) * 4;
#pragma unroll
        for (int j = 0; j < F; ++j)
#pragma unroll
          for (int i = 0; i < F; ++i)
            acc[i][j] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                rs, static_cast<int>(at + j * 64 * static_cast<uint32_t>(a.ld_acc) + i * 64), 0, 0));
      }
    } else {
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = typename Mfma<kI8>::acc_t{0, 0, 0, 0};
    }
    // The sums are all of the accumulation registers: left to the compiler, some
    // of them move to and fro around their products.
    auto product = [&](int h, int t) {
      if constexpr (kI8) asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc[t % F][t / F]) : "v"(fw[h][t % F]), "v"(fa[h][t / F]));
      else asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc[t % F][t / F]) : "v"(fw[h][t % F]), "v"(fa[h][t / F]));
    };
    // operand n of a step: the channels', then the tokens'
    auto read = [&](int ba, int bw, int h, int n) {
      if (n < F) {
        if constexpr (kAcross) {
          // (a wavefront's fragments lie in bits of the place that only the swizzle shares)
          const char* const at = sw[bw] + (ow_across ^ (n << (kLies == kAcross8 ? 4 : 5))) + h * (kBK / 4) * kWRow;
          if constexpr (kLies == kAcross8) {
            raw[n] = turned8(at);
          } else {
            const u32x2_t lo = turned16(at), hi = turned16(at + 4 * kWRow);
            fw[h][n] = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
          }
        } else {
          fw[h][n] = *reinterpret_cast<const u32x4_t*>(sw[bw] + ow[h] + ((n >> 1) * 32 + (n & 1) * 4) * kBK);
        }
      } else fa[h][n - F] = *reinterpret_cast<const u32x4_t*>(sa[ba] + oa[h] + (n - F) * 16 * kBK);
    };
    // words 2 c and 2 c + 1 of a fragment: whole numbers of at most 8 bits,
    // whose lower halves as fp32 are zeros
    auto widen8 = [&](int h, int n, int c) {
      const uint32_t v = raw[n][c >> 1] >> (16 * (c & 1));
      const float lo = static_cast<float>(static_cast<int8_t>(v)), hi = static_cast<float>(static_cast<int8_t>(v >> 8));
      fw[h][n][c] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
    };
    // Bytes of the last stage past the end of the sum count for nothing,
    // whatever the rows hold there: zeros in the token operand, and, where a
    // bf16 NaN times zero would be one, in the channel operand.
    auto mask = [&](int h) {
      const int left = static_cast<int>(a.kbytes) - ((ns - 1) * kBK + h * kStep + q * 16);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t m = byte_mask(left - 4 * d);
#pragma unroll
        for (int j = 0; j < F; ++j) fa[h][j][d] &= m;
        if constexpr (!kI8) {
#pragma unroll
          for (int i = 0; i < F; ++i) fw[h][i][d] &= m;
        }
      }
      asm volatile("s_nop 7" ::: "memory");  // the products that take these are not the compiler's to space
    };
    asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    // (written before the products that the compiler does not know as such)
#pragma unroll
    for (int j = 0; j < F; ++j)
      asm volatile("s_nop 3"
                   : "+a"(acc[0][j]), "+a"(acc[1][j]), "+a"(acc[2][j]), "+a"(acc[3][j]), "+a"(acc[4][j]), "+a"(acc[5][j]),
                     "+a"(acc[6][j]), "+a"(acc[7][j]));
#pragma unroll
    for (int n = 0; n < 2 * F; ++n) read(0, 0, 0, n);
    if constexpr (kLies == kAcross8) {
#pragma unroll
      for (int c = 0; c < 4 * F; ++c) widen8(0, c >> 2, c & 3);
      asm volatile("s_nop 7" ::: "memory");  // (as in mask)
    }
    int ba = 0, bw = 0;
    const bool tail = !kAcross && a.kbytes % kBK != 0;
    // what follows product t of a step: the next step's operands, one read every
    // `every` products; 8-bit channels first, then their conversions
    auto between = [&](int buf_a, int buf_w, int h, int t, int every, int at) {
      if constexpr (kLies == kAcross8) {
        if (t < 2 * F && (t & 1) == 0) read(buf_a, buf_w, h, t / 2);
        if (t >= 2 * F && t % 3 == 1 && (t - 2 * F) / 3 < F) read(buf_a, buf_w, h, F + (t - 2 * F) / 3);
        if (t >= F && t % 3 != 1 && t - F - (t - F) / 3 < 4 * F) {
          const int c = t - F - (t - F) / 3;
          widen8(h, c >> 2, c & 3);
        }
      } else {
        if (t % every == at && t / every < 2 * F) read(buf_a, buf_w, h, t / every);
      }
    };
    for (int s = p.s0; s < p.s1; ++s) {
      // past the last stage the loads have an empty range (they touch nothing)
      // and the reads bring what no product takes
      const Rsrc ra = tokens(p, s + 2 < p.s1), rw = channels(p, s + 2 < p.s1, s + 2);
      const uint32_t off = (s + 2) * kBK, off_w = kAcross ? 0 : off;
      const int bw1 = bw == 2 ? 0 : bw + 1, bw2 = bw1 == 2 ? 0 : bw1 + 1;
      if (tail && s + 1 == ns) mask(0);
#pragma unroll
      for (int t = 0; t < kProducts; ++t) {
        product(0, t);
        between(ba, bw, 1, t, kRead0, kRead0 - 1);
        if (t % kLoad0 == kLoad0 / 2 && t / kLoad0 < kWLoads) lds_load16(rw, sw[bw2] + (wave + t / kLoad0 * 4) * 1024, vw[t / kLoad0] + off_w);
        __builtin_amdgcn_sched_barrier(0);
      }
      // The next stage has landed (the channel operand's loads of this step are
      // the only ones that may still run), and everyone has read this one.
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kWLoads) : "memory");
      if (tail && s + 1 == ns) mask(1);
#pragma unroll
      for (int t = 0; t < kProducts; ++t) {
        product(1, t);
        if (t % kLoad1 == kLoad1 - 1 && t / kLoad1 < kLoads) lds_load16(ra, sa[ba] + (wave + t / kLoad1 * 4) * 1024, va[t / kLoad1] + off);
        between(ba ^ 1, bw1, 0, t, kRead1, kRead1 / 2);
        __builtin_amdgcn_sched_barrier(0);
      }
      ba ^= 1;
      bw = bw1;
    }
    // the last products' results are there after 19 wait states at most
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    // everyone has read the last stage, and no load is on its way
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const Place done = p;
    id += gridDim.x / kXcds;
    const bool more = id < last;
    if (more) {
      p = place(id);
      begin(p);
    }
    // (the next tile's stages lie in the first two buffers of either operand)
    const int nv = static_cast<int>(min(static_cast<int64_t>(T), a.n - done.n0)) - wn * 128;
    char* const slab = sw[2] + wave * (kSlabs / 4);
    if constexpr (kAcross) finish_across<kLies, F, F>(a, acc, done.m0 + wm * 128, done.n0 + wn * 128, nv, done.split, slab);
    else finish<kI8, kEpi, F, F, true>(a, acc, done.m0 + wm * 128, done.n0 + wn * 128, nv, done.tile_n * 2 + wn, slab);
    if (!more) return;
  }
}

// At most 16 tokens: the head's stream is the bound, or, under a short
// vocabulary, the chain along the sum.  A workgroup of 8 wavefronts owns 16
// channels and all tokens; the wavefronts share the sum, each loading its part
// of the head once, straight into matrix-core operands (16 bytes a lane, kBatch
// steps in flight), the tokens from cache the same way, and the eight sums are
// added through LDS.  (2 rows under a head of 566 x 5863: 11 us, 25 in tiles of
// 64 x 64.)
constexpr int kFewWaves = 8, kFewBatch = 8;

template <bool kI8, int kEpi>
__global__ __launch_bounds__(kFewWaves * 64, 2) void nt_few_kernel(NtArgs a) {
  typedef typename Mfma<kI8>::acc_t acc_t;
  __shared__ acc_t part[kFewWaves][64];
  __shared__ __align__(16) uint16_t turned[16][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int nv = static_cast<int>(min(int64_t{16}, a.n - n0));   // none in the padding of dl
  if (nv > 0) {
    const uint32_t kpad = static_cast<uint32_t>((a.kbytes + 15) & ~15);
    const Rsrc rw = make_rsrc(a.w + n0 * a.ldw, static_cast<uint32_t>((nv - 1) * a.ldw) + kpad);
    const Rsrc ra = make_rsrc(a.a, static_cast<uint32_t>((a.m - 1) * a.lda) + kpad);
    const int steps = static_cast<int>((a.kbytes + kStep - 1) / kStep);
    const int per = (steps + kFewWaves - 1) / kFewWaves, s0 = wave * per, s1 = min(steps, s0 + per);
    constexpr uint32_t kOut = 0xFFFFFFF0u;  // past every range: reads as 0, touches nothing
    const uint32_t vw = r < nv ? r * static_cast<uint32_t>(a.ldw) + q * 16 : kOut;
    const uint32_t va = r < a.m ? r * static_cast<uint32_t>(a.lda) + q * 16 : kOut;
    auto load = [&](Rsrc rs, uint32_t base, int s) {
      // a row's bytes from kpad on belong to the next row: not read
      const uint32_t off = base != kOut && s < s1 && s * kStep + q * 16 < static_cast<int>(kpad) ? base + s * kStep : kOut;
      return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, static_cast<int>(off), 0, 0));
    };
    acc_t acc = acc_t{0, 0, 0, 0};
    for (int s = s0; s < s1; s += kFewBatch) {
      u32x4_t w[kFewBatch], x[kFewBatch];
#pragma unroll
      for (int b = 0; b < kFewBatch; ++b) {
        w[b] = load(rw, vw, s + b);
        x[b] = load(ra, va, s + b);
      }
      if (s + kFewBatch >= steps && (a.kbytes & 15)) {
        // the last chunk's bytes behind the end count for nothing
#pragma unroll
        for (int b = 0; b < kFewBatch; ++b) {
          const int left = static_cast<int>(a.kbytes) - ((s + b) * kStep + q * 16);
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            x[b][d] &= byte_mask(left - 4 * d);
            if constexpr (!kI8) w[b][d] &= byte_mask(left - 4 * d);
          }
        }
      }
#pragma unroll
      for (int b = 0; b < kFewBatch; ++b) acc = Mfma<kI8>::run(w[b], x[b], acc);
    }
    part[wave][lane] = acc;
  }
  __syncthreads();
  if (wave) return;
  // token r, channels n0 + 4 q + 0..3
  float l[4], scale[4];
  const bool on = r < a.m;
  const float ts = kI8 && on ? a.as[r] : 1.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) scale[e] = kI8 && 4 * q + e < nv ? a.ws[n0 + 4 * q + e] : 1.0f;
  acc_t sum = acc_t{0, 0, 0, 0};
  if (nv > 0) {
    sum = part[0][lane];
#pragma unroll
    for (int i = 1; i < kFewWaves; ++i) sum += part[i][lane];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) l[e] = kI8 ? static_cast<float>(sum[e]) * ts * scale[e] : static_cast<float>(sum[e]);
  const int64_t target = on ? a.targets[r] : -1;
  const int64_t want = target - a.v0 - n0 - 4 * q;
  if constexpr (kEpi == kStats) {
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (4 * q + e >= nv) l[e] = -INFINITY;
      else if (target >= 0 && want == e) a.hit[r] = l[e];
      m = fmaxf(m, l[e]);
    }
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    const float base = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) s += exp_of(l[e] - base);
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (q == 0 && on) a.stats[static_cast<int64_t>(blockIdx.x) * a.m + r] = float2{m, s};
  } else {
    const float lse = on ? a.lse[r] : 0.0f;
    const bool dead = no_gradient(target, a.vocab, lse);
    const float g = dead ? 0.0f : a.g[r];
    float rest = 0.0f;
    uint32_t d[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = exp_of(l[e] - lse) - (want == e ? 1.0f : 0.0f);
      v *= g;
      if (kI8) v *= scale[e];
      d[e] = bf16_round(dead || 4 * q + e >= nv ? 0.0f : v);
      if (!dead && want == e && 4 * q + e < nv) a.rest[r] = rest = rounding_rest(v);
    }
    if (on) *reinterpret_cast<u32x2_t*>(a.dl + r * a.ld_dl + n0 + 4 * q) = u32x2_t{d[0] | d[1] << 16, d[2] | d[3] << 16};
    if (a.dlt) {
      // [channel][token], zeros for tokens up to a whole stage; from rest_at on the rest
      u32x4_t* const flat = reinterpret_cast<u32x4_t*>(&turned[0][0]);
#pragma unroll
      for (int i = 0; i < 2; ++i) flat[lane + 64 * i] = u32x4_t{0, 0, 0, 0};
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        turned[4 * q + e][r] = static_cast<uint16_t>(d[e]);
        if (!dead && want == e && 4 * q + e < nv) turned[4 * q + e][a.rest_at + r] = static_cast<uint16_t>(bf16_round(rest));
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = (lane + 64 * i) >> 3, t = (lane & 7) * 8;
        if (c < nv) *reinterpret_cast<u32x4_t*>(a.dlt + (n0 + c) * a.ld_dlt + t) = flat[lane + 64 * i];
      }
    }
  }
}

// dx of few rows under an 8-bit head, whose stream is then the bound: a
// workgroup adds dl[., v] w[v, c] for 128 columns c and its share of the words
// v, 64 at a time.  The matrix cores want eight words of one column, so the
// head's tile [word][column] becomes bf16, which holds 8-bit integers exactly,
// on its way through LDS and is read with the transposing LDS read.  Direct
// loads run three stages ahead.  (Gradient of 1 to 32 rows under 32000 x 4096:
// 67 to 74 us, 80 to 89 in tiles of 256 x 256; of 64 rows under 131072 x 7168:
// 606 and 476.)
constexpr int64_t kFewRows = 32;
constexpr int kDxWords = 64, kDxCols = 128;

struct DxFewArgs {
  const uint16_t* dl;   // [m][ld_dl], zeros from n to n_pad
  int64_t ld_dl;
  const char* w;
  int64_t ldw;          // bytes
  int64_t m, n, k;
  float* acc;           // [splits][m][ld_acc]
  int64_t ld_acc;
  int strips, per;      // column strips; stages of a split
};

__global__ __launch_bounds__(256) void head_dx_few_kernel(DxFewArgs a) {
  constexpr int NT = kFewRows / 16, kBuf = 4;
  constexpr int kWBytes = kDxWords * kDxCols, kTBytes = NT * 16 * kDxWords * 2;
  constexpr int kLW = kWBytes / 1024 / 4, kLT = kTBytes / 1024 / 4;  // load instructions a stage and wavefront
  static_assert(kLT >= 1, "every wavefront issues the same loads");
  __shared__ __align__(16) char sw[kBuf][kWBytes];
  __shared__ __align__(16) char st[kBuf][kTBytes];
  __shared__ __align__(16) char wide[2][kDxWords * kDxCols * 2];  // as bf16
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;
  const int strip = blockIdx.x % a.strips, split = blockIdx.x / a.strips;
  const int64_t c0 = static_cast<int64_t>(strip) * kDxCols;
  const int width = static_cast<int>(min(static_cast<int64_t>(kDxCols), ((a.k + 15) & ~int64_t{15}) - c0));  // bytes of a row here
  const int all = static_cast<int>((a.n + kDxWords - 1) / kDxWords);
  const int s_lo = split * a.per, ns = max(0, min(all - s_lo, a.per));
  auto stage = [&](int s) {
    const int buf = s % kBuf;
    const int64_t v0 = static_cast<int64_t>(s_lo + s) * kDxWords;
    const bool real = s < ns;
    const int vv = real ? static_cast<int>(min(static_cast<int64_t>(kDxWords), a.n - v0)) : 0;
    const Rsrc rw = make_rsrc(a.w + (real ? v0 * a.ldw + c0 : 0), real ? static_cast<uint32_t>((vv - 1) * a.ldw) + width : 0);
    const Rsrc rt = make_rsrc(a.dl + (real ? v0 : 0), real ? static_cast<uint32_t>((a.m - 1) * a.ld_dl * 2) + kDxWords * 2 : 0);
    constexpr int kPer = kDxCols / 16;  // 16-byte chunks of a word's row
#pragma unroll
    for (int i = 0; i < kLW; ++i) {
      const int ins = wave + 4 * i, t = ins * (64 / kPer) + lane / kPer;
      const int c = lane % kPer;
      lds_load16(rw, sw[buf] + ins * 1024, t < vv && c * 16 < width ? t * static_cast<uint32_t>(a.ldw) + c * 16 : 0xFFFFFFF0u);
    }
#pragma unroll
    for (int i = 0; i < kLT; ++i) {
      const int ins = wave + 4 * i, t = ins * 8 + (lane >> 3);
      lds_load16(rt, st[buf] + ins * 1024, t < a.m ? t * static_cast<uint32_t>(a.ld_dl * 2) + (((lane & 7) ^ token_swizzle(t)) << 4) : 0xFFFFFFF0u);
    }
  };
  f32x4_t acc[2][NT];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < kBuf - 1; ++s) stage(s);
  for (int s = 0; s < ns; ++s) {
    // stage s has landed, here and for everyone, and everyone has read stage s - 1
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((kLW + kLT) * (kBuf - 2)) : "memory");
    stage(s + kBuf - 1);
    const char* const from = sw[s % kBuf];
    char* const tile = wide[s & 1];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int idx = threadIdx.x + 256 * i, t = idx >> 3, c = idx & 7;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(from + idx * 16);
      float f[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] = static_cast<float>(static_cast<int8_t>(v[e >> 2] >> (8 * (e & 3))));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4_t o;
        // whole numbers of at most 8 bits: their lower halves are zeros
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, f[8 * h + 2 * e + 1]), __builtin_bit_cast(uint32_t, f[8 * h + 2 * e]), 0x07060302u);
        *reinterpret_cast<u32x4_t*>(tile + t * 256 + (((2 * c + h) ^ tile_swizzle(t)) << 4)) = o;
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = 32 * h + 8 * q + (r >> 2);
      u32x2_t lo[2], hi[2];
      uint32_t at[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        at[i] = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(tile)) + t * 256 +
                (((wave * 4 + 2 * i + ((r & 3) >> 1)) ^ tile_swizzle(t)) << 4) + (r & 1) * 8;
      asm volatile(
          "ds_read_b64_tr_b16 %0, %4\n\tds_read_b64_tr_b16 %1, %4 offset:1024\n\t"
          "ds_read_b64_tr_b16 %2, %5\n\tds_read_b64_tr_b16 %3, %5 offset:1024\n\ts_waitcnt lgkmcnt(0)"
          : "=&v"(lo[0]), "=&v"(hi[0]), "=&v"(lo[1]), "=&v"(hi[1])
          : "v"(at[0]), "v"(at[1])
          : "memory");
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int row = 16 * j + r;
        const u32x4_t x = *reinterpret_cast<const u32x4_t*>(st[s % kBuf] + row * kBK + (((4 * h + q) ^ token_swizzle(row)) << 4));
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[i][j] = Mfma<false>::run(u32x4_t{lo[i][0], lo[i][1], hi[i][0], hi[i][1]}, x, acc[i][j]);
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is on its way to LDS when it is given back
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t tok = 16 * j + r;
    if (tok >= a.m) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t c = c0 + wave * 32 + 16 * i + 4 * q;
      if (c < a.ld_acc) *reinterpret_cast<f32x4_t*>(a.acc + (split * a.m + tok) * a.ld_acc + c) = acc[i][j];
    }
  }
}

// (maximum, sum of exp(l - maximum)) of two sets of logits; a set without a
// maximum has sum 0, or NaN.
__device__ __forceinline__ float2 join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  return float2{m, (a.x == -INFINITY ? a.y : a.y * exp_of(a.x - m)) + (b.x == -INFINITY ? b.y : b.y * exp_of(b.x - m))};
}

// The parts of a token joined, kTok tokens a workgroup: 16 of them, whose
// parts lie side by side, or, up to 256 tokens, one (2048 parts of one token, from
// 131072 words: 4.7 us, 8.2 with 16; of 37 5.3 and 8.3, of 256 5.6 and 5.5).
template <int kTok>
__global__ __launch_bounds__(1024) void head_join_kernel(const float2* stats, const float* hit, const int32_t* targets, int64_t m,
                                                         int parts, int64_t vocab, float* loss, float* lse) {
  constexpr int kShare = 1024 / kTok;  // threads a token
  __shared__ float2 slot[16][kTok];
  const int tok = threadIdx.x % kTok, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTok + tok;
  float2 v = {-INFINITY, 0.0f};
  if (t < m) {
    int i = threadIdx.x / kTok;
    for (; i + 7 * kShare < parts; i += 8 * kShare) {
      float2 w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = stats[(i + e * kShare) * m + t];
#pragma unroll
      for (int e = 4; e >= 1; e >>= 1)
#pragma unroll
        for (int f = 0; f < e; ++f) w[f] = join(w[f], w[f + e]);
      v = join(v, w[0]);
    }
    for (; i < parts; i += kShare) v = join(v, stats[i * m + t]);
  }
  auto lanes = [&] {
#pragma unroll
    for (int o = kTok; o < 64; o <<= 1) v = join(v, float2{__shfl_xor(v.x, o), __shfl_xor(v.y, o)});
  };
  lanes();
  if (lane < kTok) slot[wave][lane] = v;
  __syncthreads();
  if (wave) return;
  v = float2{-INFINITY, 0.0f};
  for (int i = lane / kTok; i < 16; i += 64 / kTok) v = join(v, slot[i][tok]);
  lanes();
  if (lane >= kTok || t >= m) return;
  const float logs = __builtin_amdgcn_logf(v.y) * kLn2;
  const bool none = v.x == -INFINITY && v.y == 0.0f;
  lse[t] = none ? -INFINITY : v.x + logs;
  const int64_t target = targets[t];
  loss[t] = target < 0 ? 0.0f : none || target >= vocab ? NAN : logs - (hit[t] - v.x);
}

// out[c][r] = in[r][c] for r < n (zeros for r = n .. n_pad - 1 and for rows
// without a gradient, whatever they hold), c < k; 64 x 64 a workgroup.  The same
// again from column `again` on, if that is not 0.
__global__ __launch_bounds__(256) void transpose_kernel(const char* in, int64_t ld, int64_t n, int64_t k, const int32_t* targets,
                                                        const float* lse, int64_t vocab, uint16_t* out, int64_t ld_out,
                                                        int64_t n_pad, int64_t again) {
  __shared__ uint16_t tile[64][66];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 64, c0 = static_cast<int64_t>(blockIdx.y) * 64;
  const int row = threadIdx.x >> 3, c = (threadIdx.x & 7) * 8;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t rr = r0 + row + 32 * h;
    uint16_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0;
    if (rr < n && c0 + c < k && !no_gradient(targets[rr], vocab, lse[rr])) {
      // a row owns its bytes up to the next multiple of 16
      const u32x4_t w = *reinterpret_cast<const u32x4_t*>(in + rr * ld + (c0 + c) * 2);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) tile[c + e][row + 32 * h] = v[e];
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int col = row + 32 * h;
    if (c0 + col >= k || r0 + c >= n_pad) continue;
    u32x4_t w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = tile[col][c + 2 * e] | static_cast<uint32_t>(tile[col][c + 2 * e + 1]) << 16;
    *reinterpret_cast<u32x4_t*>(out + (c0 + col) * ld_out + r0 + c) = w;
    if (again) *reinterpret_cast<u32x4_t*>(out + (c0 + col) * ld_out + again + r0 + c) = w;
  }
}

struct JoinArgs {
  const float* acc;       // [splits][m][ld_acc]
  int64_t ld_acc;
  int splits;
  int64_t m, n, vocab;
  const int32_t* targets;
  const float* lse;
  const float* rest;
  const char* head;
  int64_t ldw;            // bytes
  uint16_t* out;
  int64_t ld_out;
};

// The parts of dx's sum and its targets' rest, rounded to bf16: four columns a
// thread, every fourth part a wavefront.  (9 parts of 256 x 7168: 46 us a column
// a thread.)
template <bool k8>
__global__ __launch_bounds__(256) void join_splits_kernel(JoinArgs a) {
  __shared__ f32x4_t part[4][64];
  const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 64 + lane, quads = a.ld_acc / 4;
  const int64_t row = i / quads, c = (i - row * quads) * 4;
  const bool on = row < a.m;
  f32x4_t s = {0, 0, 0, 0};
  auto add = [&](const f32x4_t& v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += v[e];
  };
  int32_t target = -1;
  float lse = 0.0f, rest = 0.0f;
  if (on) {
    // (on their way beside the sums)
    target = a.targets[row];
    lse = a.lse[row];
    rest = a.rest[row];
    const float* const at = a.acc + row * a.ld_acc + c;
    int p = g;
    for (; p + 12 < a.splits; p += 16) {
      f32x4_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const f32x4_t*>(at + (p + 4 * e) * a.m * a.ld_acc);
#pragma unroll
      for (int e = 0; e < 4; ++e) add(v[e]);
    }
    for (; p < a.splits; p += 4) add(*reinterpret_cast<const f32x4_t*>(at + p * a.m * a.ld_acc));
  }
  const bool dead = no_gradient(target, a.vocab, lse);   // (zeros as in finish_across)
  const u32x2_t hot = g || dead || c >= a.n ? u32x2_t{0, 0} : head4<k8>(a.head + target * a.ldw, c);
  part[g][lane] = s;
  __syncthreads();
  if (g || !on) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float v = fmaf(rest, head_value<k8>(hot, e), (part[0][lane][e] + part[1][lane][e]) + (part[2][lane][e] + part[3][lane][e]));
    if (c + e < a.n) a.out[row * a.ld_out + c + e] = static_cast<uint16_t>(dead ? 0u : bf16_round(v));
  }
}

__global__ __launch_bounds__(256) void zero_rows_kernel(uint16_t* out, int64_t ld, int64_t m, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < m * n; i += static_cast<int64_t>(gridDim.x) * 256)
    out[i / n * ld + i % n] = 0;
}

template <bool kI8, int kEpi, int TM, int TN, int WM, int WN, int kBuf, int kWavesPerSimd>
void launch_tile(NtArgs a, hipStream_t s) {
  a.tm = static_cast<int>((a.m + TM - 1) / TM);
  a.tn = static_cast<int>((a.n + TN - 1) / TN);
  const int64_t tiles = static_cast<int64_t>(a.tm) * a.tn;
  const dim3 grid(static_cast<unsigned>((tiles + kXcds - 1) / kXcds * kXcds));
  hipLaunchKernelGGL((nt_kernel<kI8, kEpi, TM, TN, WM, WN, kBuf, kWavesPerSimd>), grid, dim3(WM * WN * 64), 0, s, a);
}

// The tile for m tokens and n channels.
//  * Few tokens under a head: a workgroup for 16 channels, until there are as
//    many tiles of 64 as half the compute units (8 x 7168: 4000 words 17 us, 31 in
//    tiles of 64 x 64; 8000 words 28 and 32; 12000 words 38 and 33).
//  * Up to 64 tokens: the narrower of 64 and 128 channels whose tiles are two a CU
//    at most, else 256 (40 rows of 4096 in 8 bits, 50000 words: 41, 37 and 40 us in
//    tiles of 64, 128 and 256; 37 x 7168, 100003 words: 142, 147 and 133).
//  * More: the smallest of three estimates, in rounds of the chip (tiles of 64,
//    128 and 256: 300 x 1024 x 8000 words in bf16 15.0, 15.6, 32 us; 512 x 4096 x
//    32000 203, 134, 106).
enum Tile { kFew, k64x64, k64x128, k64x256, k128x128, k256x256 };

Tile pick_tile(int64_t m, int64_t n, int cus, bool few) {
  if (few && m <= 16 && n <= 32 * cus) return kFew;
  if (m <= 64) return n <= 128 * cus ? k64x64 : n <= 256 * cus ? k64x128 : k64x256;
  auto per_cu = [&](int64_t t) { return (((m + t - 1) / t) * ((n + t - 1) / t) + cus - 1) / cus; };
  const int64_t u256 = per_cu(256), u128 = per_cu(128), u64 = per_cu(64);
  constexpr int64_t k64[3] = {0, 17, 25};
  const int64_t t256 = 100 * u256, t128 = 64 * (u128 / 2) + 44 * (u128 % 2), t64 = 37 * (u64 / 3) + k64[u64 % 3];
  if (t256 <= t128 && t256 <= t64) return k256x256;
  return t128 <= t64 ? k128x128 : k64x64;
}
int tile_m(Tile t) { return t == k256x256 ? 256 : t == k128x128 ? 128 : t == kFew ? 16 : 64; }
int tile_n(Tile t) { return t == k256x256 || t == k64x256 ? 256 : t == k128x128 || t == k64x128 ? 128 : t == kFew ? 16 : 64; }
int tile_parts(Tile t) { return t == k64x256 || t == k64x128 ? 4 : t == kFew ? 1 : 2; }  // wavefronts along a tile's channels
int64_t stat_parts(Tile t, int64_t vocab) { return (vocab + tile_n(t) - 1) / tile_n(t) * tile_parts(t); }

template <bool kI8, int kEpi, int kLies>
void launch_wide(NtArgs a, int cus, hipStream_t s) {
  a.tm = static_cast<int>((a.m + 255) / 256);
  a.tn = static_cast<int>((a.n + 255) / 256);
  const int64_t tiles = static_cast<int64_t>(a.tm) * a.tn * (kLies == kRows ? 1 : a.splits);
  // a workgroup a compute unit (its LDS is all of one's), as many on every XCD
  const int64_t grid = std::min<int64_t>((tiles + kXcds - 1) / kXcds, std::max(1, cus / kXcds)) * kXcds;
  hipLaunchKernelGGL((nt_wide_kernel<kI8, kEpi, kLies>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a);
}

template <bool kI8, int kEpi>
void launch_nt(const NtArgs& a, Tile t, int cus, hipStream_t s) {
  switch (t) {
    case kFew:
      if constexpr (kEpi != kSum) {
        const int64_t n = kEpi == kGrad ? a.n_pad : a.n;
        hipLaunchKernelGGL((nt_few_kernel<kI8, kEpi>), dim3(static_cast<unsigned>((n + 15) / 16)), dim3(kFewWaves * 64), 0, s, a);
      }
      break;
    case k64x64: launch_tile<kI8, kEpi, 64, 64, 2, 2, 3, 2>(a, s); break;
    case k64x128: launch_tile<kI8, kEpi, 64, 128, 1, 4, 3, 2>(a, s); break;
    case k64x256: launch_tile<kI8, kEpi, 64, 256, 1, 4, 2, 2>(a, s); break;
    case k128x128: launch_tile<kI8, kEpi, 128, 128, 2, 2, 2, 2>(a, s); break;
    case k256x256: launch_wide<kI8, kEpi, kRows>(a, cus, s); break;
  }
}


int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

NtArgs logits_args(const HeadArgs& h) {
  NtArgs a{};
  a.a = static_cast<const char*>(h.x);
  a.lda = h.ldx;
  a.w = static_cast<const char*>(h.w);
  a.ldw = h.ldw;
  a.m = h.rows;
  a.n = h.vocab;
  a.kbytes = h.k * (h.i8 ? 1 : 2);
  a.as = h.x_scale;
  a.ws = h.w_scale;
  a.targets = h.targets;
  return a;
}

}  // namespace

HeadLayout head_layout(int64_t rows, int64_t vocab, int cus) {
  HeadLayout l{};
  l.hit = up(stat_parts(pick_tile(rows, vocab, cus, true), vocab) * rows * 8, 256);
  l.bytes = l.hit + up(rows * 4, 256);
  return l;
}

hipError_t launch_head(const HeadArgs& h, float* loss, float* lse, void* ws, int cus, hipStream_t s) {
  const Tile t = pick_tile(h.rows, h.vocab, cus, true);
  const HeadLayout l = head_layout(h.rows, h.vocab, cus);
  NtArgs a = logits_args(h);
  a.stats = static_cast<float2*>(ws);
  a.hit = reinterpret_cast<float*>(static_cast<char*>(ws) + l.hit);
  if (h.i8) launch_nt<true, kStats>(a, t, cus, s);
  else launch_nt<false, kStats>(a, t, cus, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int parts = static_cast<int>(stat_parts(t, h.vocab));
  if (h.rows <= 256)
    hipLaunchKernelGGL((head_join_kernel<1>), dim3(static_cast<unsigned>(h.rows)), dim3(1024), 0, s, a.stats, a.hit, h.targets, h.rows, parts,
                       h.vocab, loss, lse);
  else
    hipLaunchKernelGGL((head_join_kernel<16>), dim3(static_cast<unsigned>((h.rows + 15) / 16)), dim3(1024), 0, s, a.stats, a.hit, h.targets,
                       h.rows, parts, h.vocab, loss, lse);
  return hipGetLastError();
}

// Parts that dx's sum over `stages` x 64 words is shared out into when its tiles
// leave compute units idle: the fewest of what a tile's stages and its end (1.4
// us a stage, 8 stages an end) and the parts' store and join cost together.  Above
// 16 rounds there is nothing to gain (and the join's launch stays small).
static int dx_splits(int64_t rows, int64_t k, int64_t stages, int64_t pieces, int cus) {
  const int64_t tiles = (rows + 255) / 256 * ((k + 255) / 256);
  int best = 1;
  double best_us = 0;
  for (int64_t s = 1; s <= std::min<int64_t>(64, (stages + 3) / 4) && (s == 1 || tiles * s <= 16 * cus); ++s) {
    const double walk = 1.4 * pieces * ((tiles * s + cus - 1) / cus) * ((stages + s - 1) / s + 8);
    const double us = walk + (s > 1 ? s * rows * k * 8 / 4.7e6 : 0.0);
    if (s == 1 || us < best_us) best = static_cast<int>(s), best_us = us;
  }
  return best;
}

// Tokens along dW's sum: their dl, up to m_pad of them, and of up to 32 rows the
// targets' rest behind it, in the one stage that their sum takes anyway.  (A second
// stage for 33 to 64 rows: 64 under 131072 x 7168 1292 us, 1193 without.)
struct DwTokens {
  int64_t m_pad, rest_at, all;
};
static DwTokens dw_tokens(int64_t rows) {
  return rows <= 32 ? DwTokens{32, 32, 64} : DwTokens{up(rows, 64), 0, up(rows, 64)};
}

HeadBwdPlan plan_head_bwd(bool i8, int64_t rows, int64_t vocab, int64_t k, bool dx, bool dw, int cus) {
  HeadBwdPlan p{};
  if (i8 && rows <= kFewRows && rows * up(vocab, 64) <= int64_t{1} << 30) {
    // the whole vocabulary at once, up to 2^30 logits: dl is small beside the head (and its rows within 32-bit offsets)
    p.few = 1;
    p.width = up(vocab, 64);
    p.pieces = 1;
    int64_t at = up(rows * p.width * 2, 256);
    p.acc = at;
    // two workgroups a CU, of four stages of words at least
    const int64_t strips = (k + kDxCols - 1) / kDxCols, stages = (vocab + kDxWords - 1) / kDxWords;
    const int64_t want = std::max<int64_t>(1, std::min((2 * cus + strips - 1) / strips, (stages + 3) / 4));
    p.per = static_cast<int>((stages + want - 1) / want);
    p.splits = static_cast<int>((stages + p.per - 1) / p.per);
    if (dx) at += up(p.splits * rows * up(k, 8) * 4, 256);
    p.rest = at;
    p.bytes = at + up(rows * 4, 256);
    return p;
  }
  // pieces of the vocabulary: at most 2^26 logits, but 256 words at least, and of those
  // widths the one whose tiles fill whole rounds of the chip best
  const int64_t cap = std::max<int64_t>(1, (int64_t{1} << 26) / rows / 256);
  const int64_t cols = (vocab + 255) / 256;
  const int64_t tm = (rows + 255) / 256;
  auto rounds = [&](int64_t c) { return (tm * c + cus - 1) / cus; };
  int64_t best = -1, best_cost = 0;
  for (int64_t c = std::min(cap, cols); c >= 1 && c > std::min(cap, cols) - 64; --c) {
    const int64_t cost = cols / c * rounds(c) + (cols % c ? rounds(cols % c) : 0);
    if (best < 0 || cost < best_cost) best = c, best_cost = cost;
  }
  p.width = std::min(best * 256, up(vocab, 64));
  p.pieces = (vocab + p.width - 1) / p.width;
  int64_t at = up(rows * p.width * 2, 256);
  p.dlt = at;
  const int64_t tokens = dw_tokens(rows).all;
  if (dw) at += up(p.width * tokens * 2, 256);
  p.xt = at;
  if (dw) at += up(k * tokens * 2, 256);
  p.acc = at;
  p.splits = dx ? dx_splits(rows, k, std::min(p.width, up(vocab, 64)) / 64, p.pieces, cus) : 1;
  if (dx && (p.pieces > 1 || p.splits > 1)) at += up(p.splits * rows * up(k, 8) * 4, 256);
  p.rest = at;
  p.bytes = at + up(rows * 4, 256);
  return p;
}

hipError_t launch_head_bwd(const HeadArgs& h, const HeadBwdArgs& b, const HeadBwdPlan& p, void* ws, int cus, hipStream_t s) {
  char* base = static_cast<char*>(ws);
  uint16_t* dl = reinterpret_cast<uint16_t*>(base);
  float* rest = reinterpret_cast<float*>(base + p.rest);
  uint16_t* dlt = reinterpret_cast<uint16_t*>(base + p.dlt);
  uint16_t* xt = reinterpret_cast<uint16_t*>(base + p.xt);
  float* acc = p.few || p.pieces > 1 || p.splits > 1 ? reinterpret_cast<float*>(base + p.acc) : nullptr;
  const DwTokens tokens = dw_tokens(h.rows);
  if (b.dw)
    hipLaunchKernelGGL(transpose_kernel, dim3(static_cast<unsigned>((tokens.m_pad + 63) / 64), static_cast<unsigned>((h.k + 63) / 64)),
                       dim3(256), 0, s, static_cast<const char*>(h.x), h.ldx, h.rows, h.k, h.targets, b.lse, h.vocab, xt, tokens.all,
                       tokens.m_pad, tokens.rest_at);
  for (int64_t i = 0; i < p.pieces; ++i) {
    const int64_t v0 = i * p.width, n = std::min(p.width, h.vocab - v0), n_pad = up(n, 64);
    NtArgs a = logits_args(h);
    a.w += v0 * h.ldw;
    if (a.ws) a.ws += v0;
    a.v0 = v0;
    a.n = n;
    a.lse = b.lse;
    a.g = b.g;
    a.dl = dl;
    a.ld_dl = p.width;
    a.rest = rest;
    a.dlt = b.dw ? dlt : nullptr;
    a.ld_dlt = tokens.all;
    a.rest_at = tokens.rest_at;
    a.vocab = h.vocab;
    a.n_pad = n_pad;
    a.m_pad = tokens.m_pad;
    const Tile t = pick_tile(h.rows, n, cus, true);
    if (h.i8) launch_nt<true, kGrad>(a, t, cus, s);
    else launch_nt<false, kGrad>(a, t, cus, s);
    if (b.dx && p.few) {
      const int64_t strips = (h.k + kDxCols - 1) / kDxCols;
      const DxFewArgs d{dl, p.width, a.w, h.ldw, h.rows, n, h.k, acc, up(h.k, 8), static_cast<int>(strips), p.per};
      const dim3 grid(static_cast<unsigned>(strips * p.splits));
      hipLaunchKernelGGL(head_dx_few_kernel, grid, dim3(256), 0, s, d);
    } else if (b.dx) {
      NtArgs d{};
      d.a = reinterpret_cast<const char*>(dl);
      d.lda = p.width * 2;
      d.m = h.rows;
      d.n = h.k;
      d.kbytes = n_pad * 2;
      d.acc = acc;
      d.ld_acc = up(h.k, 8);
      d.add = i > 0;
      d.splits = p.splits;
      const bool last = p.splits == 1 && i + 1 == p.pieces;
      d.out = last ? b.dx : nullptr;
      d.ld_out = b.ld_dx;
      d.targets = h.targets;
      d.lse = b.lse;
      d.vocab = h.vocab;
      d.rest = rest;
      d.head = static_cast<const char*>(h.w);
      d.w = a.w;
      d.ldw = h.ldw;
      d.words = n;
      if (h.i8) launch_wide<false, kSum, kAcross8>(d, cus, s);
      else launch_wide<false, kSum, kAcross16>(d, cus, s);
    }
    if (b.dw) {
      NtArgs d{};
      d.a = reinterpret_cast<const char*>(dlt);
      d.lda = tokens.all * 2;
      d.w = reinterpret_cast<const char*>(xt);
      d.ldw = tokens.all * 2;
      d.m = n;
      d.n = h.k;
      d.kbytes = tokens.all * 2;
      d.out = b.dw + v0 * b.ld_dw;
      d.ld_out = b.ld_dw;
      launch_nt<false, kSum>(d, pick_tile(n, h.k, cus, false), cus, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (b.dx && (p.few || p.splits > 1)) {
    const JoinArgs j{acc, up(h.k, 8), p.splits, h.rows, h.k, h.vocab, h.targets, b.lse, rest, static_cast<const char*>(h.w), h.ldw, b.dx, b.ld_dx};
    const dim3 grid(static_cast<unsigned>((h.rows * (up(h.k, 8) / 4) + 63) / 64));
    if (h.i8) hipLaunchKernelGGL(join_splits_kernel<true>, grid, dim3(256), 0, s, j);
    else hipLaunchKernelGGL(join_splits_kernel<false>, grid, dim3(256), 0, s, j);
  }
  return hipGetLastError();
}

// dW of no tokens
hipError_t launch_head_zero(uint16_t* dw, int64_t ld, int64_t vocab, int64_t k, hipStream_t s) {
  const int64_t blocks = std::min<int64_t>((vocab * k + 255) / 256, 1 << 16);
  hipLaunchKernelGGL(zero_rows_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, dw, ld, vocab, k);
  return hipGetLastError();
}

}  // namespace stq
