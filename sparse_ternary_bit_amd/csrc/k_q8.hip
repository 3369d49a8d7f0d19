// 8-bit integer matrix product with one scale per row of either operand, and
// the quantizer that makes such rows.
//
// Quantizer: s = fp32(max |x| / 127), q = the integer nearest the exact x / s
// (halves to even).  The nearest integer comes from an fp64 product and is
// put right by its exact remainder x - q s (q has 8 bits, s and x 24: the
// remainder is exact in fp64), so the result does not hang on how a division
// rounds.
//
// Product: y[i, j] = (sum_c a[i, c] w[j, c]) * a_scale[i] * w_scale[j] on the
// 8-bit matrix cores (v_mfma_i32_16x16x64_i8): integer sums are exact in 32
// bits for k <= 131071 whatever the order, so only the two scalings and the
// output's own rounding are rounded.
#include <algorithm>

#include "stq_device.hpp"
#include "stq_launch.hpp"
#include "stq_round8.hpp"

namespace stq {
namespace {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t bf16_bits(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

// ---------------------------------------------------------------------------
// quantizer
// ---------------------------------------------------------------------------

struct QuantArgs {
  const void* x;
  int64_t stride;   // elements
  int64_t k;
  int8_t* q;
  int64_t ldq;      // bytes
  float* scale;
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) {
  return __builtin_bit_cast(float, static_cast<uint32_t>(v) << 16);
}

// 16 elements from column c on; columns past k read as 0
template <typename T, bool kVec>
__device__ __forceinline__ void load16(const T* row, int64_t c, int64_t k, float (&v)[16]) {
  if (kVec && c + 16 <= k) {
    constexpr int kW = sizeof(T);  // 16-byte words: 2 (bf16) or 4 (fp32)
    u32x4_t w[kW];
#pragma unroll
    for (int i = 0; i < kW; ++i) w[i] = *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const char*>(row + c) + 16 * i);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t d = sizeof(T) == 4 ? w[i >> 2][i & 3] : w[i >> 3][(i >> 1) & 3];
      v[i] = __builtin_bit_cast(float, sizeof(T) == 4 ? d : (i & 1) ? (d & 0xFFFF0000u) : (d << 16));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = c + i < k ? to_f32<T>(row[c + i]) : 0.0f;
  }
}

__device__ __forceinline__ u32x4_t quantize16(const float (&v)[16], float scale, float inv, bool fast) {
  uint32_t o[4];
  quantize<16>(v, scale, inv, fast, o);
  return u32x4_t{o[0], o[1], o[2], o[3]};
}

// One workgroup a row.  Rows of up to 8192 values stay in registers between
// the maximum and the rounding; longer ones are read again, from cache.
// kVec: rows start on 16 bytes.
// A batch of rows fills the chip with workgroups of 256 (8192 rows of 7168:
// 43 us, 57 with 512); a few rows are latency, which more threads a row shorten
// (one row: 4.1 us against 6.1).
template <typename T, bool kVec, int kQuantThreads>
__global__ __launch_bounds__(kQuantThreads) void q8_quantize_kernel(QuantArgs a) {
  constexpr int kHeld = 512 / kQuantThreads;  // groups of 16 values a thread holds
  __shared__ uint32_t wmax[kQuantThreads / 64];
  const int64_t r = blockIdx.x;
  const T* row = static_cast<const T*>(a.x) + r * a.stride;
  const int64_t groups = (a.k + 15) / 16;
  // the largest magnitude as bits: a NaN orders above every number and so is kept
  uint32_t mx = 0;
  auto largest = [&](const float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = max(mx, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
  };
  float held[kHeld][16];
#pragma unroll
  for (int h = 0; h < kHeld; ++h) load16<T, kVec>(row, (threadIdx.x + h * kQuantThreads) * 16, a.k, held[h]);
#pragma unroll
  for (int h = 0; h < kHeld; ++h) largest(held[h]);
  for (int64_t g = threadIdx.x + kHeld * kQuantThreads; g < groups; g += kQuantThreads) {
    float v[16];
    load16<T, kVec>(row, g * 16, a.k, v);
    largest(v);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) mx = max(mx, static_cast<uint32_t>(__shfl_xor(static_cast<int>(mx), o)));
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = mx;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQuantThreads / 64; ++i) mx = max(mx, wmax[i]);
  const bool finite = mx < 0x7F800000u;
  const float scale = finite ? __builtin_bit_cast(float, mx) / 127.0f : NAN;
  if (threadIdx.x == 0) a.scale[r] = scale;
  const bool some = finite && scale > 0.0f;
  const float inv = some ? 1.0f / scale : 0.0f;
  const bool fast = scale > 0x1p-100f;  // far above where the reciprocal or the products leave the normal range
  auto put = [&](int64_t g, const float (&v)[16]) {
    *reinterpret_cast<u32x4_t*>(a.q + r * a.ldq + g * 16) = some ? quantize16(v, scale, inv, fast) : u32x4_t{0, 0, 0, 0};
  };
#pragma unroll
  for (int h = 0; h < kHeld; ++h)
    if (threadIdx.x + h * kQuantThreads < groups) put(threadIdx.x + h * kQuantThreads, held[h]);
  for (int64_t g = threadIdx.x + kHeld * kQuantThreads; g < groups; g += kQuantThreads) {
    float v[16];
    load16<T, kVec>(row, g * 16, a.k, v);
    put(g, v);
  }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------

struct QArgs {
  const int8_t* a;
  int64_t lda;
  const float* as;
  const int8_t* w;
  int64_t ldw;
  const float* ws;
  int64_t m, n, k;
  void* y;
  int64_t ldy;
  int bf16;
  int vec;  // eight outputs may be stored at once (16 bytes of bf16, 32 of fp32)
  int tm, tn;  // tiles along m and n
  int step_n;  // channels between tiles, a multiple of 8
};

// Output channels of a pair of 16-row MFMA tiles: row r of tile h stands for
// channel 8 (r >> 2) + 4 h + (r & 3) of the pair's 32, so that a lane, which
// holds rows 4q .. 4q+3 of both tiles, ends with eight neighbouring channels.
__device__ __forceinline__ int pair_channel(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }

// Eight channels from c on of token `tok`
__device__ __forceinline__ void store8(const QArgs& a, int64_t tok, int64_t c, const i32x4_t& lo, const i32x4_t& hi) {
  const float ts = a.as[tok];
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = c + e < a.n ? static_cast<float>(e < 4 ? lo[e] : hi[e - 4]) * ts * a.ws[c + e] : 0.0f;
  const bool whole = a.vec && c + 8 <= a.n;
  if (a.bf16) {
    uint16_t* y = static_cast<uint16_t*>(a.y) + tok * a.ldy + c;
    if (whole) {
      u32x4_t o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = bf16_bits(v[2 * e]) | bf16_bits(v[2 * e + 1]) << 16;
      *reinterpret_cast<u32x4_t*>(y) = o;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < a.n) y[e] = static_cast<uint16_t>(bf16_bits(v[e]));
    }
  } else {
    float* y = static_cast<float*>(a.y) + tok * a.ldy + c;
    if (whole) {
      *reinterpret_cast<f32x4_t*>(y) = f32x4_t{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4_t*>(y + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < a.n) y[e] = v[e];
    }
  }
}

__device__ __forceinline__ void lds_load16(Rsrc rs, void* lds, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      rs, reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(lds)), 16,
      static_cast<int>(voff), 0, 0, 0);
}

// All ones in the low `bytes` bytes of a word (none for bytes <= 0)
__device__ __forceinline__ uint32_t byte_mask(int bytes) {
  return bytes >= 4 ? 0xFFFFFFFFu : (1u << (8 * max(0, bytes))) - 1u;
}

constexpr int kStep = 64;         // bytes of k in one matrix-core step
constexpr int kBK = 2 * kStep;    // bytes of k per stage
constexpr int kXcds = 8;

// LDS slot of a row's 16-byte chunk (eight a row): the 16 rows that one
// operand read takes (16 neighbouring tokens, or the channels of one half of
// a pair) fall on 16 different 16-byte bank groups.
__device__ __forceinline__ int token_swizzle(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int channel_swizzle(int row) { return ((row >> 1) & 1) | ((row >> 2) & 6); }

// Workgroup of WM x WN wavefronts, TM tokens x (at most) TN channels; a.step_n
// channels lie between workgroups' tiles (TN, or less where that evens out the
// load).  Both operands stream into LDS 128 bytes of k at a time (direct
// 16-byte loads) through kBuf buffers.  While the matrix cores work on one
// 64-byte step, the operands of the next are read from LDS: a token operand
// into the registers that its last use has just freed, the channel operands
// into a second set.  Halfway through a stage a barrier says that the next
// stage has landed and that every wavefront has the rest of this one in
// registers; the loads of stage s + kBuf then start into its buffer.
template <int TM, int TN, int WM, int WN, int kBuf, int kWavesPerSimd>
__global__ __launch_bounds__(WM * WN * 64, kWavesPerSimd) void q8_gemm_kernel(QArgs a) {
  constexpr int kNW = WM * WN;
  constexpr int FM = TM / WM / 16, FN = TN / WN / 16;
  constexpr int NA = TM / 8 / kNW, NW = TN / 8 / kNW;  // load instructions a stage and wavefront, 8 rows each
  static_assert(FN % 2 == 0, "channel tiles come in pairs");
  static_assert(NA * 8 * kNW == TM && NW * 8 * kNW == TN, "every wavefront issues the same loads");
  __shared__ __align__(16) int8_t sa[kBuf][TM * kBK];
  __shared__ __align__(16) int8_t sw[kBuf][TN * kBK];
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
  const int64_t m0 = static_cast<int64_t>(band * 8 + in % rows) * TM, n0 = static_cast<int64_t>(in / rows) * a.step_n;
  const int mv = static_cast<int>(min(static_cast<int64_t>(TM), a.m - m0));
  const int nv = static_cast<int>(min(static_cast<int64_t>(a.step_n), a.n - n0));
  const uint32_t kpad = static_cast<uint32_t>((a.k + 15) & ~15);
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
  const int ns = static_cast<int>((a.k + kBK - 1) / kBK);
  auto stage = [&](int s, int buf) {
#pragma unroll
    for (int i = 0; i < NA; ++i) lds_load16(ra, sa[buf] + (wave + i * kNW) * 1024, va[i] + s * kBK);
#pragma unroll
    for (int i = 0; i < NW; ++i) lds_load16(rw, sw[buf] + (wave + i * kNW) * 1024, vw[i] + s * kBK);
  };
  i32x4_t acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  const int wm = wave / WN, wn = wave % WN;
  const int tok_row = wm * FM * 16 + r;
  const int ch_row = wn * FN * 16 + pair_channel(r, 0);
  int oa[2], ow[2];  // this lane's chunk of either step
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    oa[h] = tok_row * kBK + (((4 * h + q) ^ token_swizzle(tok_row)) << 4);
    ow[h] = ch_row * kBK + (((4 * h + q) ^ channel_swizzle(ch_row)) << 4);
  }
  i32x4_t fa[FM], fw[2][FN];
  auto read_w = [&](int buf, int h, int i) {
    return *reinterpret_cast<const i32x4_t*>(sw[buf] + ow[h] + ((i >> 1) * 32 + (i & 1) * 4) * kBK);
  };
  auto read_a = [&](int buf, int h, int j) { return *reinterpret_cast<const i32x4_t*>(sa[buf] + oa[h] + j * 16 * kBK); };
  // Product group j of a step (token operand j with every channel operand),
  // then the reads that its registers were waiting for: token operand j of
  // the next step, and with group j0 the channel operands and the token
  // operands of the groups before it.
  auto group = [&](int h, int j) {
#pragma unroll
    for (int i = 0; i < FN; ++i) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[h][i], fa[j], acc[i][j], 0, 0, 0);
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
  // bytes of the last stage past the end of k count for nothing, whatever the
  // rows hold there: zeros in the token operand
  auto mask = [&](int s, int h) {
    const int left = static_cast<int>(a.k) - (s * kBK + h * kStep + q * 16);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t m = byte_mask(left - 4 * d);
#pragma unroll
      for (int j = 0; j < FM; ++j) fa[j][d] = static_cast<int32_t>(static_cast<uint32_t>(fa[j][d]) & m);
    }
  };
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
    // The second step's first group needs nothing of the next stage, and covers
    // the last of these reads.  Then stages s + 1 .. s + kBuf - 1 are in flight
    // (fewer near the end): wait for the first of them, for this wavefront's
    // own LDS reads and for the other wavefronts.  (The compiler's barrier
    // would wait for every load.)
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
  if (a.k % kBK) mask(ns - 1, 0);
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    group(0, j);
    reads(0, j, 0, buf);
  }
  if (a.k % kBK) mask(ns - 1, 1);
#pragma unroll
  for (int j = 0; j < FM; ++j) group(1, j);
  // token m0 + wm FM 16 + 16 j + r, channels n0 + wn FN 16 + 32 p + 8 q + 0..7
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int64_t tok = m0 + tok_row + j * 16;
    if (tok >= a.m) continue;
#pragma unroll
    for (int p = 0; p < FN / 2; ++p) {
      const int c = wn * FN * 16 + 32 * p + 8 * q;
      if (c < nv) store8(a, tok, n0 + c, acc[2 * p][j], acc[2 * p + 1][j]);
    }
  }
}

// At most 16 tokens: the weights' stream is the bound.  A workgroup of 8
// wavefronts owns 16 channels and all tokens; the wavefronts share k, each
// loading its part of the weights once, straight into MFMA operands (16 bytes
// a lane, kBatch steps of 64 bytes of k in flight), the tokens from cache the
// same way, and the eight sums are added through LDS.
constexpr int kFewWaves = 8;
constexpr int kBatch = 8;

__global__ __launch_bounds__(kFewWaves * 64, 2) void q8_few_kernel(QArgs a) {
  __shared__ i32x4_t part[kFewWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int nv = static_cast<int>(min(int64_t{16}, a.n - n0));
  const uint32_t kpad = static_cast<uint32_t>((a.k + 15) & ~15);
  const Rsrc rw = make_rsrc(a.w + n0 * a.ldw, static_cast<uint32_t>((nv - 1) * a.ldw) + kpad);
  const Rsrc ra = make_rsrc(a.a, static_cast<uint32_t>((a.m - 1) * a.lda) + kpad);
  const int steps = static_cast<int>((a.k + kStep - 1) / kStep);
  const int per = (steps + kFewWaves - 1) / kFewWaves;
  const int s0 = wave * per, s1 = min(steps, s0 + per);
  constexpr uint32_t kOut = 0xFFFFFFF0u;  // past every range: reads as 0, touches nothing
  const uint32_t vw = r < nv ? r * static_cast<uint32_t>(a.ldw) + q * 16 : kOut;
  const uint32_t va = r < a.m ? r * static_cast<uint32_t>(a.lda) + q * 16 : kOut;
  i32x4_t acc = {0, 0, 0, 0};
  auto load = [&](Rsrc rs, uint32_t base, int s) {
    // a row's bytes from kpad on belong to the next row: not read
    const uint32_t off = base != kOut && s < s1 && s * kStep + q * 16 < static_cast<int>(kpad) ? base + s * kStep : kOut;
    return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, static_cast<int>(off), 0, 0));
  };
  for (int s = s0; s < s1; s += kBatch) {
    i32x4_t w[kBatch], x[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      w[b] = load(rw, vw, s + b);
      x[b] = load(ra, va, s + b);
    }
    if (s + kBatch >= steps && (a.k & 15)) {
      // the last chunk's bytes behind k count for nothing: zeros in the token operand
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int left = static_cast<int>(a.k) - ((s + b) * kStep + q * 16);  // bytes of this chunk inside k
#pragma unroll
        for (int d = 0; d < 4; ++d) x[b][d] = static_cast<int32_t>(static_cast<uint32_t>(x[b][d]) & byte_mask(left - 4 * d));
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[b], x[b], acc, 0, 0, 0);
  }
  part[wave][lane] = acc;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int i = 1; i < kFewWaves; ++i) acc += part[i][lane];
  if (r >= a.m) return;
  const float ts = a.as[r];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t c = n0 + 4 * q + e;
    if (c >= a.n) continue;
    const float v = static_cast<float>(acc[e]) * ts * a.ws[c];
    if (a.bf16) static_cast<uint16_t*>(a.y)[r * a.ldy + c] = static_cast<uint16_t>(bf16_bits(v));
    else static_cast<float*>(a.y)[r * a.ldy + c] = v;
  }
}

template <int TM, int TN, int WM, int WN, int kBuf, int kWavesPerSimd>
void launch_tile(QArgs a, int step_n, hipStream_t s) {
  a.step_n = step_n;
  a.tm = static_cast<int>((a.m + TM - 1) / TM);
  a.tn = static_cast<int>((a.n + step_n - 1) / step_n);
  const int64_t tiles = static_cast<int64_t>(a.tm) * a.tn;
  const dim3 grid(static_cast<unsigned>((tiles + kXcds - 1) / kXcds * kXcds));
  hipLaunchKernelGGL((q8_gemm_kernel<TM, TN, WM, WN, kBuf, kWavesPerSimd>), grid, dim3(WM * WN * 64), 0, s, a);
}

}  // namespace

hipError_t launch_q8_quantize(const Q8QuantArgs& g, hipStream_t s) {
  const QuantArgs a{g.x, g.x_stride, g.k, g.q, g.ldq, g.scale};
  const dim3 grid(static_cast<unsigned>(g.rows));
  const int esz = g.bf16 ? 2 : 4;
  const bool vec = (reinterpret_cast<uintptr_t>(g.x) & 15) == 0 && (g.x_stride * esz) % 16 == 0;
  const bool few = g.rows <= 1024;
  auto go = [&](auto kernel, int threads) { hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, s, a); };
  if (g.bf16) {
    if (vec) few ? go(q8_quantize_kernel<uint16_t, true, 512>, 512) : go(q8_quantize_kernel<uint16_t, true, 256>, 256);
    else few ? go(q8_quantize_kernel<uint16_t, false, 512>, 512) : go(q8_quantize_kernel<uint16_t, false, 256>, 256);
  } else {
    if (vec) few ? go(q8_quantize_kernel<float, true, 512>, 512) : go(q8_quantize_kernel<float, true, 256>, 256);
    else few ? go(q8_quantize_kernel<float, false, 512>, 512) : go(q8_quantize_kernel<float, false, 256>, 256);
  }
  return hipGetLastError();
}

// Which kernel, and which tile.  Times in us on 256 CUs, k = 7168 unless
// stated.
//  * Up to 16 tokens: q8_few_kernel, until its re-reads of the tokens (once
//    per 16 channels) weigh on a long channel list.  n = 4096: 8.2 for 1 token
//    and 10.3 for 16, against 17 for the 64 x 64 tiles; n = 32768, k = 4096: 27
//    and 36 against 33 (where the rule changes over: one token still gains
//    what 16 lose); n = 100003: 116 for 1 token and 178 for 16, against 122
//    and 125 for the 64 x 256 tiles.
//  * Up to 64 tokens: as wide a channel tile as leaves every CU two.  n =
//    16384, k = 4096: 21 with 64 channels, 27 with 128, 35 with 256; 50000, k =
//    4096: 53, 45, 50; 100003: 168, 150, 145.  Tiles of 128 and 256 are cut
//    narrower where that loads all CUs alike (100003 channels in whole tiles of
//    256: 177).
//  * More: the smallest of three estimates.  256 x 256 tiles take 100 a round
//    of one per CU; 128 x 128 tiles 64 a round of two, 44 where one is alone;
//    64 x 64 tiles 37 a round of three, 25 and 17 for two and one.  8192 x
//    4096: 203, 255 and 363; 2048 x 4096: 91, 65 and 93; 512 x 4096: 87, 43
//    and 25.
hipError_t launch_q8_matmul(const Q8MatmulArgs& g, hipStream_t s) {
  QArgs a{g.a, g.lda, g.a_scale, g.w, g.ldw, g.w_scale, g.m, g.n, g.k, g.y, g.ldy, g.bf16, 0, 0, 0, 0};
  const int esz = g.bf16 ? 2 : 4;
  a.vec = (reinterpret_cast<uintptr_t>(g.y) % 16) == 0 && (g.ldy * esz) % 16 == 0;
  const int64_t cus = g.cus;
  if (g.m <= 4 || (g.m <= 16 && g.n <= 128 * cus)) {
    hipLaunchKernelGGL(q8_few_kernel, dim3(static_cast<unsigned>((g.n + 15) / 16)), dim3(kFewWaves * 64), 0, s, a);
    return hipGetLastError();
  }
  if (g.m <= 64) {
    // channels a tile of at most tn so that whole rounds of two tiles a CU are evenly loaded
    auto even = [&](int64_t tn) {
      const int64_t rounds = (g.n + tn * 2 * cus - 1) / (tn * 2 * cus);
      return static_cast<int>(std::min(tn, ((g.n + rounds * 2 * cus - 1) / (rounds * 2 * cus) + 7) / 8 * 8));
    };
    if (g.n <= 64 * cus) launch_tile<64, 64, 2, 2, 3, 2>(a, 64, s);
    else if (g.n <= 256 * cus) launch_tile<64, 128, 1, 4, 3, 2>(a, even(128), s);
    else launch_tile<64, 256, 1, 4, 2, 2>(a, even(256), s);
    return hipGetLastError();
  }
  auto per_cu = [&](int64_t t) { return (((g.m + t - 1) / t) * ((g.n + t - 1) / t) + cus - 1) / cus; };
  const int64_t u256 = per_cu(256), u128 = per_cu(128), u64 = per_cu(64);
  constexpr int64_t k64[3] = {0, 17, 25};
  const int64_t t256 = 100 * u256, t128 = 64 * (u128 / 2) + 44 * (u128 % 2), t64 = 37 * (u64 / 3) + k64[u64 % 3];
  if (t256 <= t128 && t256 <= t64) launch_tile<256, 256, 2, 4, 2, 2>(a, 256, s);
  else if (t128 <= t64) launch_tile<128, 128, 2, 2, 2, 2>(a, 128, s);
  else launch_tile<64, 64, 2, 2, 3, 2>(a, 64, s);
  return hipGetLastError();
}

}  // namespace stq
