// The gated feed-forward over packed experts where rows are many: one pass is
// up to 160 rows of an expert against 128 gate rows and the same 128 up rows,
// h = silu(g) u formed where the sums are.
//
// What differs from the plain grouped product, whose passes stop at 80 rows:
// that kernel sums each 256-weight block apart and adds it, times the rows' d,
// to a second set of accumulators.  Here there is one set, held in units of
// the current block's d: between two blocks every sum is multiplied by
// d_before / d_now (one rounding to fp32 a block, as the other form's fused
// add has), and by the last d at the end.  A block whose d is 0 keeps the
// scale and gets codes of four zeros, the table's second half.  A sum is
// therefore held as sum / d, which leaves fp32 only for sums beyond 3e38 d.
// The registers that frees (64 weight rows x 160 tokens a wavefront take 160
// of 256) halve the decode per matrix product: 0.5 LDS reads and 2.2 VALU
// instructions an MFMA (itself counted) against 0.75 and 2.9.
//
// Weights are the products' rows where a pass is of up to 128 tokens: 1 to 2 %
// less time than as their columns (the card's power: a pattern has three
// values).  In longer ones they are the columns, so that a lane's sums share a
// weight row and a block's factors take four registers: sixteen do not fit
// beside 160 sums (spilled, 690 us become 930 for 2048 rows of 8 experts).
//
// Per block of 256 weights four stages of 64 activations; a stage's tokens
// stream into one of two LDS buffers while the other is multiplied. The
// stage's one barrier stands kAhead token tiles before its end, where every
// wavefront has read the last of the buffer: the tiles behind it are already
// in registers, so products go on while the next stage's first reads return,
// and the buffer's next fill starts at once. Token tiles are read kAhead
// ahead, the weights' operands of a k-step are decoded under the products of
// the one before, and the next block's records are made in six pieces between
// the last stage's token tiles (in one piece ahead of them: 905 us against 880
// for 64 rows of 256 experts). The loop has no branch: past the last block it
// stages the last one again, which nothing reads. (With branches the compiler
// moved accumulators through scratch memory, and a reload waits for every
// direct load in flight: 5 to 12 reloads a block cost 3 to 6 %.)
//
// Measured against passes of 80 rows of the plain kernel's form, us: 8 experts
// of 7168 x 2048, 16384 rows 819 -> 670 (1.43 PFLOP/s); 64 experts of 100 rows
// 381 -> 310; 32 uneven experts of 4096 x 1024, 8191 rows 155 -> 138; 256
// experts of 64 rows 915 -> 882. What bounds it: the matrix cores are busy 54
// % of the cycles at 64 rows a pass and the card runs at 1.9 of its 2.4 GHz
// under this load (a loop of these products alone reaches 1.97 PFLOP/s on such
// numbers); left out one at a time, the weights' stream, the records, the
// activations' stream, the pattern reads and the scale gave 9, 11, 8, 7 and 4
// %, and all of them together 34 %. Three wavefronts a SIMD (passes of 80 rows
// in 168 registers) and a ring of four stages changed nothing there.
#include <cstddef>
#include <type_traits>

#include "stq_device.hpp"
#include "stq_launch.hpp"
#include "stq_passes.hpp"

namespace stq {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;
constexpr int kCols = kWaves * 32;      // output columns of a workgroup: as many gate and up rows
constexpr int kStepK = 64;              // activations of a stage, 128 bytes a token
constexpr int kStageRow = kStepK * 2;
constexpr int kXcds = 8;
constexpr int kHalfRun = kTileRows / 2 * kBlockBytes;  // half a tile's run of one block, a multiple of 16
constexpr int kWLoads = 3;
constexpr int kWindow = kWLoads * 1024;
constexpr int kCodes = 64;              // the 32 codes, and with bit 5 set four zeros
constexpr int kAhead = 2;               // token tiles read ahead of their products
constexpr int kLonger = 64;             // rows of a pass that goes first
constexpr int kTiles = 10;              // token tiles of a pass

struct GatedArgs {
  const uint8_t* w;
  int64_t estride;
  int n_experts;
  int nb;
  int k;
  const uint16_t* x;
  const int32_t* offsets;
  int64_t total_m;
  int d_ff;
  int nslab;
  int max_tok;
  uint16_t* h;
  uint16_t* gu;
};

struct Smem {
  // lanes 0,1 of each code as bf16, then lanes 2,3; at byte 0, so that a code
  // times 4 is its address
  uint32_t lut[2 * kCodes];
  alignas(16) float ratio[kWaves][kTileRows];  // of each row's sums, into the next block's units
  alignas(16) float scale[kWaves][kTileRows];  // what they are in units of
  alignas(16) char x[2][kTiles * 16 * kStageRow];
  // code records, one word for a row and two k-steps: [k-step pair][quarter of
  // a k-step][row of its tile][tile], so a lane's four tiles are one read
  alignas(16) uint32_t rec[kWaves][4][4][16][4];
  alignas(16) char wraw[kWaves][kWindow];
};

__device__ __forceinline__ uint32_t pattern_word(uint32_t c, int lane) {
  auto bf = [&](int l) -> uint32_t {
    const int t = code_lane_value(c, l);
    return t == 0 ? 0u : (t > 0 ? 0x3F80u : 0xBF80u);
  };
  return bf(lane) | (bf(lane + 1) << 16);
}

__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v)); }

// the lane, opaque: what is derived from it is not kept over the loop in
// registers that the sums need
__device__ __forceinline__ int lane_now() {
  int t;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(t));
  return t;
}

// all but the last N of this wavefront's direct loads are in LDS, its reads
// have returned, and everyone is here
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int NT>
__device__ __forceinline__ void run_pass(const GatedArgs& a, Smem& sh, const uint8_t* wexp, int slab, int64_t row0,
                                         int mt) {
  static_assert(NT >= 2 && NT <= kTiles && kTiles % 2 == 0, "two tiles a wavefront's loads, and a stage longer than kAhead");
  const int lane = lane_now();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, r = lane & 15;

  // half a tile of gate rows and the half tile of the same up rows
  const int hrow0 = slab * kCols + wave * (kTileRows / 2);
  const int trow0 = hrow0 & ~(kTileRows - 1);
  const uint8_t* tb = wexp + static_cast<int64_t>(trow0) * a.nb * kBlockBytes;
  const uint32_t to_up = static_cast<uint32_t>(a.d_ff) * a.nb * kBlockBytes;
  const Rsrc rs = make_rsrc(tb, static_cast<uint32_t>(kTileRows) * a.nb * kBlockBytes + to_up);
  const uint32_t whalf = (hrow0 & (kTileRows / 2)) ? kHalfRun : 0u;

  // a stage: 8 tokens an instruction, chunk c of token t in slot c ^ (t & 7) of
  // its 128 bytes; tokens past the pass read zeros through the range check
  constexpr int kXLoads = (NT + 1) / 2;
  const uint32_t xrow = static_cast<uint32_t>(a.k) * 2;
  const Rsrc xs_rs = make_rsrc(a.x + row0 * a.k, static_cast<uint32_t>(mt) * xrow);
  const int t_first = 8 * wave + (lane >> 3);
  const uint32_t x_first = static_cast<uint32_t>(t_first) * xrow + (((lane & 7) ^ (t_first & 7)) * 16);
  auto stage_x = [&](int h, int buf) {
    uint32_t voff = x_first;
    asm volatile("" : "+v"(voff));  // the steps' offsets are not kept over the loop
#pragma unroll
    for (int j = 0; j < kXLoads; ++j, voff += 32 * xrow)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xs_rs, reinterpret_cast<__attribute__((address_space(3))) void*>(
                     reinterpret_cast<uintptr_t>(sh.x[buf] + (4 * j + wave) * 1024)),
          16, static_cast<int>(voff), h * kStageRow, 0, 0);
  };
  // this wavefront's runs of block b: pieces of 16 bytes, 84 of the gate rows
  // and 84 of the up rows
  auto stage_w = [&](int b) {
    const int lane = lane_now();
#pragma unroll
    for (int j = 0; j < kWLoads; ++j) {
      const int c = j * 64 + lane;
      const uint32_t off = c < kHalfRun / 16       ? whalf + c * 16u
                           : c < 2 * kHalfRun / 16 ? whalf + to_up + (c * 16u - kHalfRun)
                                                   : 0xFFFFFFF0u;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, reinterpret_cast<__attribute__((address_space(3))) void*>(
                  reinterpret_cast<uintptr_t>(sh.wraw[wave] + j * 1024)),
          16, static_cast<int>(off), b * kTileRows * kBlockBytes, 0, 0);
    }
  };

  // The block in the window: this lane's row's codes, each times 4, as records.
  // 42 bytes from an even byte: `sel` joins the halves of its words.  In pieces
  // that the products can hide: the words' reads run one piece ahead.
  constexpr bool kSpread = NT >= 4;  // room for the pieces between the stage's tiles
  struct Row {
    uint32_t v[3], sel, zero;  // words of the next k-step pair; 0x80808080 if d is 0
    uint32_t qh[2];
  } row;
  const char* const window = sh.wraw[wave];
  auto read_head = [&](int lane) {
    const uint32_t off = lane * kBlockBytes;
    const uint32_t* wv = reinterpret_cast<const uint32_t*>(window + (off & ~3u));
    row.v[0] = wv[0];
    row.qh[0] = wv[8];
    row.qh[1] = wv[9];
    row.v[2] = wv[10];
  };
  auto read_pair = [&](int lane, int s2) {
    const uint32_t off = lane * kBlockBytes;
    const uint32_t* wv = reinterpret_cast<const uint32_t*>(window + (off & ~3u)) + 2 * s2;
#pragma unroll
    for (int i = 0; i < 3; ++i) row.v[i] = wv[i];
  };
  auto put_head = [&](int lane) {
    const bool odd = lane & 1;  // starts in the middle of a word
    row.sel = odd ? 0x07060504u : 0x05040302u;
    const float d0 = half_bits_to_float(odd ? row.v[0] >> 16 : row.v[0]);
    const float was = sh.scale[wave][lane];
    const float d = d0 == 0.0f ? was : d0;
    row.zero = d0 == 0.0f ? 0x80808080u : 0u;
    sh.ratio[wave][lane] = was / d;
    sh.scale[wave][lane] = d;
    row.qh[0] = __builtin_amdgcn_perm(row.qh[1], row.qh[0], row.sel);
    row.qh[1] = __builtin_amdgcn_perm(row.v[2], row.qh[1], row.sel);
  };
  auto put_pair = [&](int lane, int s2) {
    const int ti = lane >> 4, tr = lane & 15;
    uint32_t cl[2], cu[2];
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const uint32_t W = __builtin_amdgcn_perm(row.v[o + 1], row.v[o], row.sel);
      const uint32_t QH = row.qh[s2 >> 1];
      const int sh6 = 6 - 2 * ((2 * s2 + o) & 3);
      cl[o] = ((W << 2) & 0x3C3C3C3Cu) | ((QH << sh6) & 0x40404040u) | row.zero;
      cu[o] = ((W >> 2) & 0x3C3C3C3Cu) | (((QH >> 1) << sh6) & 0x40404040u) | row.zero;
    }
    sh.rec[wave][s2][0][tr][ti] = __builtin_amdgcn_perm(cl[1], cl[0], 0x05040100u);
    sh.rec[wave][s2][1][tr][ti] = __builtin_amdgcn_perm(cl[1], cl[0], 0x07060302u);
    sh.rec[wave][s2][2][tr][ti] = __builtin_amdgcn_perm(cu[1], cu[0], 0x05040100u);
    sh.rec[wave][s2][3][tr][ti] = __builtin_amdgcn_perm(cu[1], cu[0], 0x07060302u);
  };
  // piece i of 0 .. 5; the first pair's records are there after piece 2
  auto records = [&](int lane, int i) {
    if (i == 0) read_head(lane);
    if (i == 1) {
      put_head(lane);
      read_pair(lane, 0);
    }
    if (i >= 2) {
      put_pair(lane, i - 2);
      if (i < 5) read_pair(lane, i - 1);
    }
  };

  // Weights as the products' rows (a lane's four sums are four weight rows of a
  // token) or as their columns (four tokens of one weight row)
  constexpr bool kRowsFirst = NT <= 8;
  auto multiply = [](const bf16x8_t& w, const bf16x8_t& x, const f32x4_t& c) {
    return kRowsFirst ? __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0)
                      : __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, w, c, 0, 0, 0);
  };
  // the factors, one a weight row, of a lane's sums of row tile i
  using Factors = std::conditional_t<kRowsFirst, f32x4_t, float>;
  auto factors = [](const float* row, int lane, int i) {
    return *reinterpret_cast<const Factors*>(row + 16 * i + (kRowsFirst ? 4 * (lane >> 4) : lane & 15));
  };
  auto scale_by = [](f32x4_t& c, const Factors& f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kRowsFirst) c[j] *= f[j];
      else c[j] *= f;
    }
  };
  f32x4_t acc[4][NT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  int xb[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) xb[ks] = r * kStageRow + ((4 * ks + q) ^ (r & 7)) * 16;

  // one code of row tile i: two words of the operand
  auto decode = [&](const u32x4_t& R, int ks, int half, u32x4_t (&A)[4]) {
    const int i = half >> 1;
    const uint32_t w = R[i];
    const uint32_t c = __builtin_amdgcn_ubfe(w, 16 * ks + 8 * (half & 1), 8);
    const char* lut = reinterpret_cast<const char*>(sh.lut);
    A[i][2 * (half & 1)] = *reinterpret_cast<const uint32_t*>(lut + c);
    A[i][2 * (half & 1) + 1] = *reinterpret_cast<const uint32_t*>(lut + c + 4 * kCodes);
  };

  sh.scale[wave][lane] = 1.0f;
  stage_x(0, 0);
  stage_w(0);
  stage_x(1, 1);
  wait_and_meet<kXLoads>();
#pragma unroll
  for (int i = 0; i < 6; ++i) records(lane, i);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the window has been read
  stage_w(min(1, a.nb - 1));

  u32x4_t A[2][4];
  bf16x8_t B[4];
  u32x4_t R = *reinterpret_cast<const u32x4_t*>(&sh.rec[wave][0][q][r][0]), Rn = R;
#pragma unroll
  for (int c = 0; c < 8; ++c) decode(R, 0, c, A[0]);
#pragma unroll
  for (int p = 0; p < kAhead; ++p)
    B[p] = *reinterpret_cast<const bf16x8_t*>(sh.x[0] + xb[p / NT] + (p % NT) * 16 * kStageRow);

  for (int b = 0; b < a.nb; ++b) {
    Factors up[4];
    const int ln = lane_now();
#pragma unroll
    for (int i = 0; i < 4; ++i) up[i] = factors(sh.ratio[wave], ln, i);
#pragma unroll
    for (int qt = 0; qt < 4; ++qt) {
      if (qt == 3 && !kSpread) {
        const int ln = lane_now();
#pragma unroll
        for (int i = 0; i < 6; ++i) records(ln, i);
      }
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int p = ks * NT + t, g = 2 * NT * qt + p;
          if (p == 2 * NT - kAhead) {
            // the next stage is in LDS (in a block's first stage the next
            // block's weights, issued after it, may still be on their way)
            if (qt == 0) wait_and_meet<kWLoads>();
            else wait_and_meet<0>();
            stage_x(min(4 * b + qt + 2, 4 * a.nb - 1), qt & 1);
            if (qt == 3) stage_w(min(b + 2, a.nb - 1));
          }
          const int ahead = (p + kAhead) % (2 * NT);
          B[(g + kAhead) & 3] = *reinterpret_cast<const bf16x8_t*>(
              sh.x[(p + kAhead < 2 * NT ? qt : qt + 1) & 1] + xb[ahead / NT] + (ahead % NT) * 16 * kStageRow);
          if (qt == 3 && kSpread && p < 6) records(lane, p);
          if (ks == 0 && t == NT - 1) Rn = *reinterpret_cast<const u32x4_t*>(&sh.rec[wave][(qt + 1) & 3][q][r][0]);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c * NT / 8 == t) decode(ks == 0 ? R : Rn, ks ^ 1, c, A[ks ^ 1]);
          if (qt == 0 && ks == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              scale_by(acc[i][t], up[i]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[i][t] = multiply(__builtin_bit_cast(bf16x8_t, A[ks][i]), B[g & 3], acc[i][t]);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (ks == 1) R = Rn;
      }
    }
  }

  // everyone is done with the stages: the outputs go through LDS as whole rows
  const int tid = wave * 64 + lane_now(), q1 = (tid >> 4) & 3, r1 = tid & 15;
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  Factors last[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) last[i] = factors(sh.scale[wave], tid & 63, i);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) scale_by(acc[i][t], last[i]);
  constexpr int kRowB = kCols * 2 + 16;
  static_assert(offsetof(Smem, x) + kTiles * 16 * kRowB <= sizeof(Smem), "the outputs fit");
  char* const tile = reinterpret_cast<char*>(&sh) + offsetof(Smem, x);
  auto put = [&](uint16_t* out, int64_t ld, auto value) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (kRowsFirst) {
          *reinterpret_cast<u32x2_t*>(tile + (16 * t + r1) * kRowB + (wave * 32 + 16 * i + 4 * q1) * 2) =
              u32x2_t{bf16_bits(value(t, i, 0)) | static_cast<uint32_t>(bf16_bits(value(t, i, 1))) << 16,
                      bf16_bits(value(t, i, 2)) | static_cast<uint32_t>(bf16_bits(value(t, i, 3))) << 16};
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint16_t*>(tile + (16 * t + 4 * q1 + j) * kRowB + (wave * 32 + 16 * i + r1) * 2) =
                bf16_bits(value(t, i, j));
        }
      }
    __syncthreads();
    for (int tok = tid >> 4; tok < mt; tok += kThreads / 16)
      *reinterpret_cast<u32x4_t*>(out + (row0 + tok) * ld + slab * kCols + 8 * (tid & 15)) =
          *reinterpret_cast<const u32x4_t*>(tile + tok * kRowB + 16 * (tid & 15));
  };
  // silu(g) u from the fp32 sums, rounded once; the saved sums too
  put(a.h, a.d_ff, [&](int t, int i, int j) {
    const float g = acc[i][t][j];
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * g)) * acc[i + 2][t][j];
  });
  if (a.gu) {
    __syncthreads();
    put(a.gu, 2 * a.d_ff, [&](int t, int i, int j) { return acc[i][t][j]; });
    __syncthreads();
    put(a.gu + a.d_ff, 2 * a.d_ff, [&](int t, int i, int j) { return acc[i + 2][t][j]; });
  }
}

__global__ __launch_bounds__(kThreads, 2) void gated_kernel(GatedArgs a) {
  __shared__ Smem sh;
  const int xcd = blockIdx.x % kXcds;
  const int local = blockIdx.x / kXcds;
  const int slab = local % a.nslab;
  const PassUnit u = find_pass(a.offsets, a.n_experts, a.total_m, (local / a.nslab) * kXcds + xcd, a.max_tok, kLonger);
  if (u.mt <= 0) return;
  if (threadIdx.x < kCodes) {
    sh.lut[threadIdx.x] = threadIdx.x < 32 ? pattern_word(threadIdx.x, 0) : 0u;
    sh.lut[kCodes + threadIdx.x] = threadIdx.x < 32 ? pattern_word(threadIdx.x, 2) : 0u;
  }
  __syncthreads();
  const uint8_t* wexp = a.w + static_cast<int64_t>(u.expert) * a.estride;
  const int nt = (u.mt + 15) >> 4;
  auto pass = [&](auto n) { run_pass<decltype(n)::value>(a, sh, wexp, slab, u.row0, u.mt); };
  using std::integral_constant;
  if (nt <= 2) pass(integral_constant<int, 2>{});
  else if (nt == 3) pass(integral_constant<int, 3>{});
  else if (nt == 4) pass(integral_constant<int, 4>{});
  else if (nt == 5) pass(integral_constant<int, 5>{});
  else if (nt == 6) pass(integral_constant<int, 6>{});
  else if (nt <= 8) pass(integral_constant<int, 8>{});
  else pass(integral_constant<int, 10>{});
}

}  // namespace

hipError_t launch_gated(const SwigluArgs& g, int max_tok, hipStream_t s) {
  GatedArgs a{};
  a.w = g.w_table;
  a.estride = g.expert_stride;
  a.n_experts = static_cast<int>(g.n_experts);
  a.nb = static_cast<int>(g.d_model / kQK);
  a.k = static_cast<int>(g.d_model);
  a.x = g.x;
  a.offsets = g.offsets;
  a.total_m = g.total_m;
  a.d_ff = static_cast<int>(g.d_ff);
  a.nslab = static_cast<int>(g.d_ff / kCols);
  a.h = g.h;
  a.gu = g.gate_up;
  a.max_tok = max_tok;
  const int64_t units = (pass_units(g.total_m, g.n_experts, max_tok) + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL(gated_kernel, dim3(static_cast<unsigned>(units * a.nslab)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace stq
