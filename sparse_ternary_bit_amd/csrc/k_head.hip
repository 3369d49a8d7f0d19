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
// vocabulary at a time), or sums stored or added up (dx, dW).  The gradients'
// other operands are laid out along their sums first: W's piece and x
// transposed, and dl stored both ways from the tile in LDS.  A piece's dl, its
// transpose and W's piece stay near the 256 MB of the last-level cache.
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
  int tm, tn, step_n;     // tiles, and channels between tiles
  // logits
  const float* as;        // 8-bit rows: scales of tokens and channels
  const float* ws;
  const int32_t* targets;
  int64_t v0;             // vocabulary index of channel 0
  // kStats
  float2* stats;          // [tn][m]: maximum, sum of exp(l - maximum)
  float* hit;             // [m]: the target's logit
  // kGrad
  const float* lse;
  const float* g;
  int64_t vocab;          // the whole vocabulary
  uint16_t* dl;           // [m][ld_dl], zeros in channels n .. n_pad - 1
  int64_t ld_dl;
  uint16_t* dlt;          // [n][ld_dlt], zeros in tokens m .. m_pad - 1; may be NULL
  int64_t ld_dlt;
  int64_t n_pad, m_pad;
  // kSum
  float* acc;             // [splits][m][n]
  int add;                // add to acc
  int splits;             // parts of the sum, acc [m][n] each
  uint16_t* out;          // bf16 [m][ld_out] instead of acc's store (with add: acc is added first)
  int64_t ld_out;
  int vec;                // eight outputs may be stored at once
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

__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// Workgroup of WM x WN wavefronts, TM tokens x (at most) TN channels.  Both
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
  static_assert(kBuf * (TM + TN) * kBK >= TM * TN * 2, "the finished tile fits where the stages were");
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
  const int tiles = a.tm * a.tn, split = kEpi == kSum ? static_cast<int>(blockIdx.y) : 0;
  const int per = (tiles + kXcds - 1) / kXcds;
  const int id = (blockIdx.x % kXcds) * per + blockIdx.x / kXcds;
  if (id >= tiles) return;
  const int band = id / (8 * a.tn), rows = min(8, a.tm - band * 8), in = id - band * 8 * a.tn;
  const int tile_n = in / rows;
  const int64_t m0 = static_cast<int64_t>(band * 8 + in % rows) * TM, n0 = static_cast<int64_t>(tile_n) * a.step_n;
  const int mv = static_cast<int>(min(static_cast<int64_t>(TM), a.m - m0));
  const int nv = static_cast<int>(min(static_cast<int64_t>(a.step_n), a.n - n0));
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
  // this split's stages
  const int all = static_cast<int>((a.kbytes + kBK - 1) / kBK);
  const int s_per = kEpi == kSum ? (all + a.splits - 1) / a.splits : all;
  const int s_lo = split * s_per, ns = max(0, min(all - s_lo, s_per));
  auto stage = [&](int s, int buf) {
#pragma unroll
    for (int i = 0; i < NA; ++i) lds_load16(ra, sa[buf] + (wave + i * kNW) * 1024, va[i] + (s_lo + s) * kBK);
#pragma unroll
    for (int i = 0; i < NW; ++i) lds_load16(rw, sw[buf] + (wave + i * kNW) * 1024, vw[i] + (s_lo + s) * kBK);
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
    const int left = static_cast<int>(a.kbytes) - ((s_lo + s) * kBK + h * kStep + q * 16);
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
    const bool tail = a.kbytes % kBK != 0 && s_lo + ns == all;
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

  // token m0 + tok_row + 16 j, channels n0 + wn FN 16 + 32 p + 8 q + 0..7
  const int ch0 = wn * FN * 16 + 8 * q;
  auto value = [&](int j, int p, int e) -> float {
    const acc_t& v = acc[2 * p + (e >> 2)][j];
    return static_cast<float>(v[e & 3]);
  };
  if constexpr (kEpi == kSum) {
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int64_t tok = m0 + tok_row + j * 16;
      if (tok >= a.m) continue;
#pragma unroll
      for (int p = 0; p < FN / 2; ++p) {
        const int c = ch0 + 32 * p;
        if (c >= nv) continue;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = value(j, p, e);
        float* acc_row = a.acc ? a.acc + (static_cast<int64_t>(split) * a.m + tok) * a.n : nullptr;
        if (a.add) {
          float o[8];
          if (a.vec) load8f<float, true>(acc_row, n0 + c, a.n, o);
          else load8f<float, false>(acc_row, n0 + c, a.n, o);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        if (a.out) {
          bf16_t* row = reinterpret_cast<bf16_t*>(a.out) + tok * a.ld_out;
          if (a.vec) store8<bf16_t, true>(row, n0 + c, a.n, pack8<bf16_t>(v));
          else store8<bf16_t, false>(row, n0 + c, a.n, pack8<bf16_t>(v));
        } else {
          if (a.vec) store8<float, true>(acc_row, n0 + c, a.n, pack8<float>(v));
          else store8<float, false>(acc_row, n0 + c, a.n, pack8<float>(v));
        }
      }
    }
  }
  if constexpr (kEpi == kStats) {
    // a wavefront's maximum and sum of every token, then the wavefronts' of a token
    float wsc[FN / 2][8];
#pragma unroll
    for (int p = 0; p < FN / 2; ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e) wsc[p][e] = kI8 && ch0 + 32 * p + e < nv ? a.ws[n0 + ch0 + 32 * p + e] : 1.0f;
    float2* const part = reinterpret_cast<float2*>(smem);  // [WN][TM]
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // everyone has read the last stage
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int64_t tok = m0 + tok_row + j * 16;
      const bool on = tok < a.m;
      const float ts = kI8 && on ? a.as[tok] : 1.0f;
      const int64_t want = on ? a.targets[tok] - a.v0 - n0 - ch0 : -1;
      float l[FN / 2][8], m = -INFINITY;
#pragma unroll
      for (int p = 0; p < FN / 2; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          l[p][e] = kI8 ? value(j, p, e) * ts * wsc[p][e] : value(j, p, e);
          if (ch0 + 32 * p + e >= nv) l[p][e] = -INFINITY;
          else if (want == 32 * p + e) a.hit[tok] = l[p][e];
          m = fmaxf(m, l[p][e]);
        }
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float base = m == -INFINITY ? 0.0f : m;
      float s = 0.0f;
#pragma unroll
      for (int p = 0; p < FN / 2; ++p)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += exp_of(l[p][e] - base);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (q == 0) part[wn * TM + tok_row + j * 16] = float2{m, s};
    }
    __syncthreads();
    for (int t = threadIdx.x; t < mv; t += kNW * 64) {
      float m = part[t].x;
#pragma unroll
      for (int i = 1; i < WN; ++i) m = fmaxf(m, part[i * TM + t].x);
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < WN; ++i) {
        const float2 v = part[i * TM + t];
        s += v.x == -INFINITY ? v.y : v.y * exp_of(v.x - m);  // (without a maximum y is 0, or NaN)
      }
      a.stats[tile_n * a.m + m0 + t] = float2{m, s};
    }
  }
  if constexpr (kEpi == kGrad) {
    constexpr int kChunks = TN / 8;
    float wsc[FN / 2][8];
#pragma unroll
    for (int p = 0; p < FN / 2; ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e) wsc[p][e] = kI8 && ch0 + 32 * p + e < nv ? a.ws[n0 + ch0 + 32 * p + e] : 1.0f;
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // everyone has read the last stage
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int t = tok_row + j * 16;
      const int64_t tok = m0 + t;
      const bool on = tok < a.m;
      const float ts = kI8 && on ? a.as[tok] : 1.0f;
      const int64_t target = on ? a.targets[tok] : -1;
      const float lse = on ? a.lse[tok] : 0.0f;
      // no gradient: an ignored row, one without a distribution, a target past the vocabulary
      const bool dead = target < 0 || target >= a.vocab || lse == -INFINITY;
      const float g = dead ? 0.0f : a.g[tok];
      const int64_t want = target - a.v0 - n0 - ch0;
#pragma unroll
      for (int p = 0; p < FN / 2; ++p) {
        float d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float l = kI8 ? value(j, p, e) * ts * wsc[p][e] : value(j, p, e);
          float v = exp_of(l - lse);
          if (want == 32 * p + e) v -= 1.0f;
          v = g * v;
          if (kI8) v *= wsc[p][e];
          d[e] = dead || ch0 + 32 * p + e >= nv ? 0.0f : v;
        }
        const int chunk = (ch0 + 32 * p) / 8;
        *reinterpret_cast<u32x4_t*>(smem + t * TN * 2 + ((chunk ^ (tile_swizzle(t) & (kChunks - 1))) << 4)) = pack8<bf16_t>(d).w[0];
      }
    }
    __syncthreads();
    // the tile row by row ...
    const int64_t n_here = min(static_cast<int64_t>(TN), a.n_pad - n0);
    for (int i = threadIdx.x; i < TM * kChunks; i += kNW * 64) {
      const int t = i / kChunks, c = i % kChunks;
      if (t < mv && c * 8 < n_here)
        *reinterpret_cast<u32x4_t*>(a.dl + (m0 + t) * a.ld_dl + n0 + c * 8) =
            *reinterpret_cast<const u32x4_t*>(smem + t * TN * 2 + ((c ^ (tile_swizzle(t) & (kChunks - 1))) << 4));
    }
    // ... and column by column: 16 lanes give four tokens' 16 channels to the
    // transposing read and each takes back four tokens of one
    if (a.dlt) {
      const int64_t m_here = min(static_cast<int64_t>(TM), a.m_pad - m0);
      for (int i = wave; i < (TM / 32) * (TN / 16); i += kNW) {
        const int g0 = i % (TM / 32) * 32, c0 = i / (TM / 32) * 16;
        const int t = g0 + 8 * q + (r >> 2);
        const int chunk = c0 / 8 + ((r & 3) >> 1);
        const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem)) + t * TN * 2 +
                            ((chunk ^ (tile_swizzle(t) & (kChunks - 1))) << 4) + (r & 1) * 8;
        u32x2_t lo, hi;
        asm volatile("ds_read_b64_tr_b16 %0, %2\n\tds_read_b64_tr_b16 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(lo), "=&v"(hi)
                     : "v"(at), "n"(4 * TN * 2)
                     : "memory");
        if (g0 + 8 * q < m_here && c0 + r < nv)
          *reinterpret_cast<u32x4_t*>(a.dlt + (n0 + c0 + r) * a.ld_dlt + m0 + g0 + 8 * q) = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
      }
    }
  }
}

// The tiles' maxima and sums of a token joined; 64 tokens a workgroup, the
// tiles shared out over 16 wavefronts.
__global__ __launch_bounds__(1024) void head_join_kernel(const float2* stats, const float* hit, const int32_t* targets, int64_t m,
                                                         int tn, int64_t vocab, float* loss, float* lse) {
  __shared__ float2 part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  float top = -INFINITY, s = 0.0f;
  if (t < m) {
#pragma unroll 4
    for (int i = wave; i < tn; i += 16) {
      const float2 v = stats[i * m + t];
      const float m2 = fmaxf(top, v.x);
      // (a part without a maximum has sum 0, or NaN)
      s = (top == -INFINITY ? s : s * exp_of(top - m2)) + (v.x == -INFINITY ? v.y : v.y * exp_of(v.x - m2));
      top = m2;
    }
  }
  part[wave][lane] = float2{top, s};
  __syncthreads();
  if (wave || t >= m) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    const float2 v = part[i][lane];
    const float m2 = fmaxf(top, v.x);
    s = (top == -INFINITY ? s : s * exp_of(top - m2)) + (v.x == -INFINITY ? v.y : v.y * exp_of(v.x - m2));
    top = m2;
  }
  const float logs = __builtin_amdgcn_logf(s) * kLn2;
  const bool none = top == -INFINITY && s == 0.0f;
  lse[t] = none ? -INFINITY : top + logs;
  const int64_t target = targets[t];
  loss[t] = target < 0 ? 0.0f : none || target >= vocab ? NAN : logs - (hit[t] - top);
}

// out[c][r] = in[r][c] for r < n (zeros for r = n .. n_pad - 1 and for rows
// whose target is ignored), c < k: bf16 or 8-bit integers in, bf16 out; 64 x
// 64 a workgroup.
template <bool kI8>
__global__ __launch_bounds__(256) void transpose_kernel(const char* in, int64_t ld, int64_t n, int64_t k, const int32_t* targets,
                                                        uint16_t* out, int64_t ld_out, int64_t n_pad) {
  __shared__ uint16_t tile[64][66];
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 64, c0 = static_cast<int64_t>(blockIdx.y) * 64;
  const int row = threadIdx.x >> 3, c = (threadIdx.x & 7) * 8;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t rr = r0 + row + 32 * h;
    uint16_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0;
    if (rr < n && c0 + c < k && !(targets && targets[rr] < 0)) {
      // a row owns its bytes up to the next multiple of 16
      if constexpr (kI8) {
        const u32x2_t w = *reinterpret_cast<const u32x2_t*>(in + rr * ld + c0 + c);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = static_cast<uint16_t>(bf16_round(static_cast<float>(static_cast<int8_t>(w[e >> 2] >> (8 * (e & 3))))));
      } else {
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(in + rr * ld + (c0 + c) * 2);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
      }
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
  }
}

// The parts of a split sum, in order, rounded to bf16
__global__ __launch_bounds__(256) void join_splits_kernel(const float* acc, int splits, int64_t m, int64_t n, uint16_t* out,
                                                          int64_t ld_out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= m * n) return;
  float s = acc[i];
  for (int p = 1; p < splits; ++p) s += acc[p * m * n + i];
  out[i / n * ld_out + i % n] = static_cast<uint16_t>(bf16_round(s));
}

__global__ __launch_bounds__(256) void zero_rows_kernel(uint16_t* out, int64_t ld, int64_t m, int64_t n) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < m * n; i += static_cast<int64_t>(gridDim.x) * 256)
    out[i / n * ld + i % n] = 0;
}

template <bool kI8, int kEpi, int TM, int TN, int WM, int WN, int kBuf, int kWavesPerSimd>
void launch_tile(NtArgs a, int step_n, hipStream_t s) {
  a.step_n = step_n;
  a.tm = static_cast<int>((a.m + TM - 1) / TM);
  a.tn = static_cast<int>((a.n + step_n - 1) / step_n);
  const int64_t tiles = static_cast<int64_t>(a.tm) * a.tn;
  const dim3 grid(static_cast<unsigned>((tiles + kXcds - 1) / kXcds * kXcds), kEpi == kSum ? a.splits : 1);
  hipLaunchKernelGGL((nt_kernel<kI8, kEpi, TM, TN, WM, WN, kBuf, kWavesPerSimd>), grid, dim3(WM * WN * 64), 0, s, a);
}

// The tile for m tokens and n channels
enum Tile { k64x64, k64x256, k128x128, k256x256 };

Tile pick_tile(int64_t m, int64_t n, int cus) {
  if (m <= 64) return n <= 64 * cus ? k64x64 : k64x256;
  auto per_cu = [&](int64_t t) { return (((m + t - 1) / t) * ((n + t - 1) / t) + cus - 1) / cus; };
  const int64_t u256 = per_cu(256), u128 = per_cu(128), u64 = per_cu(64);
  constexpr int64_t k64[3] = {0, 17, 25};
  const int64_t t256 = 100 * u256, t128 = 64 * (u128 / 2) + 44 * (u128 % 2), t64 = 37 * (u64 / 3) + k64[u64 % 3];
  if (t256 <= t128 && t256 <= t64) return k256x256;
  return t128 <= t64 ? k128x128 : k64x64;
}
int tile_m(Tile t) { return t == k256x256 ? 256 : t == k128x128 ? 128 : 64; }
int tile_n(Tile t) { return t == k256x256 || t == k64x256 ? 256 : t == k128x128 ? 128 : 64; }

template <bool kI8, int kEpi>
void launch_nt(const NtArgs& a, Tile t, hipStream_t s) {
  switch (t) {
    case k64x64: launch_tile<kI8, kEpi, 64, 64, 2, 2, 3, 2>(a, 64, s); break;
    case k64x256: launch_tile<kI8, kEpi, 64, 256, 1, 4, 2, 2>(a, 256, s); break;
    case k128x128: launch_tile<kI8, kEpi, 128, 128, 2, 2, 2, 2>(a, 128, s); break;
    case k256x256: launch_tile<kI8, kEpi, 256, 256, 2, 4, 2, 2>(a, 256, s); break;
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
  const int64_t tn = (vocab + tile_n(pick_tile(rows, vocab, cus)) - 1) / tile_n(pick_tile(rows, vocab, cus));
  HeadLayout l{};
  l.hit = up(tn * rows * 8, 256);
  l.bytes = l.hit + up(rows * 4, 256);
  return l;
}

hipError_t launch_head(const HeadArgs& h, float* loss, float* lse, void* ws, int cus, hipStream_t s) {
  const Tile t = pick_tile(h.rows, h.vocab, cus);
  const HeadLayout l = head_layout(h.rows, h.vocab, cus);
  NtArgs a = logits_args(h);
  a.stats = static_cast<float2*>(ws);
  a.hit = reinterpret_cast<float*>(static_cast<char*>(ws) + l.hit);
  if (h.i8) launch_nt<true, kStats>(a, t, s);
  else launch_nt<false, kStats>(a, t, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(head_join_kernel, dim3(static_cast<unsigned>((h.rows + 63) / 64)), dim3(1024), 0, s, a.stats, a.hit, h.targets,
                     h.rows, static_cast<int>((h.vocab + tile_n(t) - 1) / tile_n(t)), h.vocab, loss, lse);
  return hipGetLastError();
}

// Pieces of the vocabulary: at most 2^26 logits and 2^27 weights each, and of
// those the width whose tiles fill whole rounds of the chip best.
HeadBwdPlan plan_head_bwd(int64_t rows, int64_t vocab, int64_t k, bool dx, bool dw, int cus) {
  HeadBwdPlan p{};
  const int64_t cap = std::max<int64_t>(1, std::min((int64_t{1} << 26) / rows, (int64_t{1} << 27) / k) / 256);
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
  const int64_t m_pad = up(rows, 64);
  int64_t at = up(rows * p.width * 2, 256);
  p.dlt = at;
  if (dw) at += up(p.width * m_pad * 2, 256);
  p.xt = at;
  if (dw) at += up(k * m_pad * 2, 256);
  p.wt = at;
  if (dx) at += up(k * p.width * 2, 256);
  p.acc = at;
  // few tokens leave few tiles: the sum over the vocabulary is shared out
  p.tile = pick_tile(rows, k, cus);
  const int64_t tiles = ((rows + tile_m(static_cast<Tile>(p.tile)) - 1) / tile_m(static_cast<Tile>(p.tile))) *
                        ((k + tile_n(static_cast<Tile>(p.tile)) - 1) / tile_n(static_cast<Tile>(p.tile)));
  p.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({cus / tiles, p.width / 1024, 16})));
  if (dx && (p.pieces > 1 || p.splits > 1)) at += up(p.splits * rows * k * 4, 256);
  p.bytes = at;
  return p;
}

hipError_t launch_head_bwd(const HeadArgs& h, const HeadBwdArgs& b, const HeadBwdPlan& p, void* ws, int cus, hipStream_t s) {
  char* base = static_cast<char*>(ws);
  uint16_t* dl = reinterpret_cast<uint16_t*>(base);
  uint16_t* dlt = reinterpret_cast<uint16_t*>(base + p.dlt);
  uint16_t* xt = reinterpret_cast<uint16_t*>(base + p.xt);
  uint16_t* wt = reinterpret_cast<uint16_t*>(base + p.wt);
  float* acc = p.pieces > 1 || p.splits > 1 ? reinterpret_cast<float*>(base + p.acc) : nullptr;
  const int64_t m_pad = up(h.rows, 64);
  auto vec = [](const void* q, int64_t ld_bytes) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0 && ld_bytes % 16 == 0; };
  auto blocks = [](int64_t n) { return static_cast<unsigned>((n + 255) / 256); };
  if (b.dw)
    hipLaunchKernelGGL((transpose_kernel<false>), dim3(static_cast<unsigned>(m_pad / 64), static_cast<unsigned>((h.k + 63) / 64)), dim3(256),
                       0, s, static_cast<const char*>(h.x), h.ldx, h.rows, h.k, h.targets, xt, m_pad, m_pad);
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
    a.dlt = b.dw ? dlt : nullptr;
    a.ld_dlt = m_pad;
    a.vocab = h.vocab;
    a.n_pad = n_pad;
    a.m_pad = m_pad;
    const Tile t = pick_tile(h.rows, n, cus);
    if (h.i8) launch_nt<true, kGrad>(a, t, s);
    else launch_nt<false, kGrad>(a, t, s);
    if (b.dx) {
      const dim3 grid(static_cast<unsigned>(n_pad / 64), static_cast<unsigned>((h.k + 63) / 64));
      if (h.i8) hipLaunchKernelGGL((transpose_kernel<true>), grid, dim3(256), 0, s, a.w, h.ldw, n, h.k, nullptr, wt, p.width, n_pad);
      else hipLaunchKernelGGL((transpose_kernel<false>), grid, dim3(256), 0, s, a.w, h.ldw, n, h.k, nullptr, wt, p.width, n_pad);
      NtArgs d{};
      d.a = reinterpret_cast<const char*>(dl);
      d.lda = p.width * 2;
      d.w = reinterpret_cast<const char*>(wt);
      d.ldw = p.width * 2;
      d.m = h.rows;
      d.n = h.k;
      d.kbytes = n_pad * 2;
      d.acc = acc;
      d.add = i > 0;
      d.splits = p.splits;
      const bool last = p.splits == 1 && i + 1 == p.pieces;
      d.out = last ? b.dx : nullptr;
      d.ld_out = b.ld_dx;
      d.vec = h.k % 4 == 0 && (!last || vec(b.dx, b.ld_dx * 2));
      launch_nt<false, kSum>(d, static_cast<Tile>(p.tile), s);
    }
    if (b.dw) {
      NtArgs d{};
      d.a = reinterpret_cast<const char*>(dlt);
      d.lda = m_pad * 2;
      d.w = reinterpret_cast<const char*>(xt);
      d.ldw = m_pad * 2;
      d.m = n;
      d.n = h.k;
      d.kbytes = m_pad * 2;
      d.splits = 1;
      d.out = b.dw + v0 * b.ld_dw;
      d.ld_out = b.ld_dw;
      d.vec = vec(d.out, b.ld_dw * 2);
      launch_nt<false, kSum>(d, pick_tile(n, h.k, cus), s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (b.dx && p.splits > 1)
    hipLaunchKernelGGL(join_splits_kernel, dim3(blocks(h.rows * h.k)), dim3(256), 0, s, acc, p.splits, h.rows, h.k, b.dx, b.ld_dx);
  return hipGetLastError();
}

// dW of no tokens
hipError_t launch_head_zero(uint16_t* dw, int64_t ld, int64_t vocab, int64_t k, hipStream_t s) {
  const int64_t blocks = std::min<int64_t>((vocab * k + 255) / 256, 1 << 16);
  hipLaunchKernelGGL(zero_rows_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, dw, ld, vocab, k);
  return hipGetLastError();
}

}  // namespace stq
