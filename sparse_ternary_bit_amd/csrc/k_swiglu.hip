// Gradients of the gated feed-forward h = silu(Wg x) * (Wu x) over the packed
// experts (its forward is the gated form of the grouped GEMM).
//
// With the saved pre-activations g, u, s = 1 / (1 + exp(-g)) and the gradient
// dh that arrives at h:
//     dg = dh u s (1 + g (1 - s)),   du = dh g s,   dz = [dg | du]
//     dx   = dz W        (W the expert's decoded [2 d_ff, d_model] matrix)
//     dW_e = dz_e^T x_e  over the expert's rows
//
// dz_kernel forms dz once per row in fp32.  The product with W takes it as
// fp16, each row scaled by a power of two that puts its largest magnitude in
// [2^14, 2^15), and folds the block scales into it, as d / D with D above every
// |d|: the weights' patterns enter the fp16 matrix cores exactly, and dz is
// rounded to 11 bits twice (itself, and its product with d / D) ahead of the
// fp32 sums.  Both keep their digits down to 2^-28 of the row's largest dz
// (times D); below, fp16's subnormal step leaves 2^-39 of it.  A bf16 operand
// would round to 8 bits everywhere.  The product with x takes dz as bf16, x's
// own type: fp16 has not the range for x, and dz as the sum of two bf16 numbers
// would double the products.
#include "stq_device.hpp"
#include "stq_launch.hpp"
#include "stq_passes.hpp"

namespace stq {
namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(a))) |
         static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(b))) << 16;
}
__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
  return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(a))) |
         static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(b))) << 16;
}
__device__ __forceinline__ void unpack_bf16(const u32x4_t& w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t d = w[i];
    v[2 * i] = __builtin_bit_cast(float, d << 16);
    v[2 * i + 1] = __builtin_bit_cast(float, d & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void* lds_at(void* base, int byte) { return static_cast<char*>(base) + byte; }
__device__ __forceinline__ void lds_load16(Rsrc rs, void* lds, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      rs, reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(lds)), 16,
      static_cast<int>(voff), 0, 0, 0);
}

// ---------------------------------------------------------------------------
// dz
// ---------------------------------------------------------------------------

struct DzArgs {
  const uint16_t* gu;  // [rows, 2 d_ff] bf16
  const uint16_t* dh;  // [rows, d_ff] bf16
  int d_ff;
  uint16_t* dz16;      // fp16 [rows, 2 d_ff], scaled, or NULL
  float* inv;          // [rows]: what undoes the row's scale
  uint16_t* dzb;       // bf16 [rows, 2 d_ff], or NULL
};

__device__ __forceinline__ void dz_of(const u32x4_t& gw, const u32x4_t& uw, const u32x4_t& hw, float (&dg)[8],
                                      float (&du)[8]) {
  float g[8], u[8], h[8];
  unpack_bf16(gw, g);
  unpack_bf16(uw, u);
  unpack_bf16(hw, h);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * g[i]));
    const float gs = g[i] * s;
    // 1 + g (1 - s) = 1 + g - g s; times s it is s + g s (1 - s)
    dg[i] = h[i] * u[i] * fmaf(gs, 1.0f - s, s);
    du[i] = h[i] * gs;
  }
}

// One workgroup a row; 8 columns of gate and up per thread and step.  The
// scaled form needs the row's largest magnitude first; the row is then read
// again (from cache) and formed again, which costs less than keeping it.
__global__ __launch_bounds__(256) void dz_kernel(DzArgs a) {
  __shared__ uint32_t wmax[4];
  const int64_t r = blockIdx.x;
  const u32x4_t* g = reinterpret_cast<const u32x4_t*>(a.gu + r * 2 * a.d_ff);
  const u32x4_t* u = reinterpret_cast<const u32x4_t*>(a.gu + r * 2 * a.d_ff + a.d_ff);
  const u32x4_t* h = reinterpret_cast<const u32x4_t*>(a.dh + r * a.d_ff);
  const int n8 = a.d_ff / 8;
  float scale = 1.0f;
  if (a.dz16) {
    uint32_t mx = 0;  // magnitudes as bits: infinities and NaN order above every number
    for (int i = threadIdx.x; i < n8; i += 256) {
      float dg[8], du[8];
      dz_of(g[i], u[i], h[i], dg, du);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        mx = max(mx, max(__builtin_bit_cast(uint32_t, dg[j]) & 0x7FFFFFFFu, __builtin_bit_cast(uint32_t, du[j]) & 0x7FFFFFFFu));
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) mx = max(mx, static_cast<uint32_t>(__shfl_xor(static_cast<int>(mx), o)));
    if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = mx;
    __syncthreads();
    mx = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
    // 2^e with e = 14 - floor(log2 max), held where 2^e and 2^-e are normal numbers; a row of
    // zeros, or one that is not finite, keeps 1
    const int ex = static_cast<int>(mx >> 23);
    const int e = (mx == 0 || ex == 255) ? 0 : max(-126, min(126, 14 + 127 - ex));
    scale = __builtin_bit_cast(float, static_cast<uint32_t>(127 + e) << 23);
    if (threadIdx.x == 0) a.inv[r] = __builtin_bit_cast(float, static_cast<uint32_t>(127 - e) << 23);
  }
  for (int i = threadIdx.x; i < n8; i += 256) {
    float dg[8], du[8];
    dz_of(g[i], u[i], h[i], dg, du);
    u32x4_t og, ou;
    if (a.dzb) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        og[j] = bf16_pair(dg[2 * j], dg[2 * j + 1]);
        ou[j] = bf16_pair(du[2 * j], du[2 * j + 1]);
      }
      reinterpret_cast<u32x4_t*>(a.dzb + r * 2 * a.d_ff)[i] = og;
      reinterpret_cast<u32x4_t*>(a.dzb + r * 2 * a.d_ff + a.d_ff)[i] = ou;
    }
    if (a.dz16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        og[j] = f16_pair(dg[2 * j] * scale, dg[2 * j + 1] * scale);
        ou[j] = f16_pair(du[2 * j] * scale, du[2 * j + 1] * scale);
      }
      reinterpret_cast<u32x4_t*>(a.dz16 + r * 2 * a.d_ff)[i] = og;
      reinterpret_cast<u32x4_t*>(a.dz16 + r * 2 * a.d_ff + a.d_ff)[i] = ou;
    }
  }
}

// ---------------------------------------------------------------------------
// dx = dz W
// ---------------------------------------------------------------------------
// A workgroup of 4 wavefronts owns one 256-weight block column of one expert
// (256 of dx's columns) and a pass of at most 96 of its rows; the sum runs
// over the matrix's 64-row tiles.  W enters transposed: an MFMA lane takes 8
// consecutive rows of one group of four columns.
//
//  * Codes: per tile a wavefront loads the words of its 16 groups (lane = row)
//    and writes the row's 16 code bytes to LDS; the transposing 8-byte LDS read
//    hands a lane its group's codes of 8 rows.  Each code is the offset of its
//    four fp16 lanes (+-1, 0) in a 32-entry table; byte permutes pair
//    neighbouring rows into the operands of four column sets (column 4 group +
//    j, j = 0..3), so a lane ends with 16 neighbouring columns of every token it
//    holds.
//  * Scales: d varies along the sum, so it goes into dz: a thread loads 8
//    columns of a token, multiplies them by the 8 rows' d / D (packed fp16) and
//    writes them to LDS.  D is a power of two above every |d| met so far, so
//    nothing leaves fp16's range; where a tile raises it the sums are scaled
//    down once.  d / D is exact unless it is a subnormal fp16 number, which
//    takes scales of 1 and more beside others 2^13 times smaller.  A pass that
//    meets such a pair starts over with the products formed in fp32 and rounded
//    once.  (Calls of the case below: 1210 us with all products in fp32, 1110
//    with packed ones and the watch for such pairs, 1097 without the watch.)
//
// All of it runs ahead of the matrix cores: while they multiply one 32-row
// step, the next step's table reads are in flight, and the next tile's codes
// and dz are written between a tile's two steps.  For 16384 rows of 256
// experts of 4096 x 7168 it takes 1050 us; the products alone would take about
// 700, the rest is the instructions of the decode (a form that multiplied d
// into the weights and transposed the codes in registers had 135 VALU
// instructions per tile and 34 products, and took 1270 us).  The same rows of
// 8 experts, in passes of 96, take 860 (passes of 80: 910).

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;
constexpr int kXcds = 8;
constexpr int kMaxTok = 96;
constexpr int kLonger = 64;         // rows of a pass that goes first
constexpr int kStageTok = (kMaxTok + 31) / 32 * 32;
constexpr int kRing = 8;            // a power of two, at least 5 (see the order of a tile)
constexpr int kRun = kTileRows * kBlockBytes;

struct DxArgs {
  const uint8_t* w;
  int64_t estride;
  int n_experts;
  int nb;            // blocks per matrix row
  int tiles;         // 64-row tiles of the matrix
  const int32_t* offsets;
  int64_t total_m;
  const uint16_t* dz;  // fp16 [total_m, 64 tiles]
  const float* inv;
  uint16_t* dx;        // bf16 [total_m, 256 nb]
  int max_tok;         // of a pass
};

struct DxSmem {
  uint64_t lut[32];                           // four fp16 lanes of each code; at byte 0
  // dz d / D: 64 columns of each token, 16-byte chunks swizzled; written 32
  // tokens at a time
  alignas(16) char a[2][kStageTok * 128];
  alignas(16) char w[kRing][3 * 1024];        // the tiles' runs of the block, here or on their way
  alignas(16) uint8_t rec[kWaves][kTileRows * 16];  // code bytes, [row][group of the wavefront]
  alignas(16) uint16_t d[2][kWaves][kTileRows];
};

// The largest of the lanes' values, as bits of non-negative numbers
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  auto step = [&](uint32_t o) { v = max(v, o); };
  step(__builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, v, 0x142, 0xF, 0xF, false));
  step(__builtin_amdgcn_update_dpp(0, v, 0x143, 0xF, 0xF, false));
  return __builtin_amdgcn_readlane(v, 63);
}

// kFar: products with d / D formed in fp32.  Without it the pass stops, the
// same in every wavefront, and returns true where a d lies so far below D that
// their fp16 quotient would lose digits.
template <int NT, bool kFar>
__device__ __forceinline__ bool dx_pass(const DxArgs& a, DxSmem& sh, const uint8_t* wexp, int b, int64_t row0, int mt) {
  // through an opaque move: what derives from the thread index is then computed
  // in each instantiation instead of being hoisted ahead of their choice, where
  // it would cost registers
  int tid;
  asm volatile("v_mov_b32 %0, %1" : "=v"(tid) : "v"(static_cast<int>(threadIdx.x)));
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, r = lane & 15;
  const uint32_t zrow = static_cast<uint32_t>(a.tiles) * 128u;  // bytes of a row of dz
  // rows past the pass lie past the descriptor's range and read as zeros
  const Rsrc rz = make_rsrc(a.dz + row0 * a.tiles * 64, static_cast<uint32_t>(mt) * zrow);
  // dz staging: this thread's chunk (8 columns) of tokens t0, t0 + 32, ...: 32
  // apart, so the chunk's place in a token's 128 bytes stays the same
  constexpr int NJ = (NT + 1) / 2;
  static_assert(NJ * 32 <= kStageTok, "every token written has its place");
  const int t0 = wave * 8 + (lane >> 3);
  const uint32_t z_first = t0 * zrow + (lane & 7) * 16;
  char* const z_put = sh.a[0] + t0 * 128 + (((lane & 7) ^ ((t0 >> 1) & 7)) << 4);
  struct Z {
    u32x4_t v[NJ];
  };
  auto load_z = [&](int t) {
    Z z;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      z.v[j] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rz, static_cast<int>(z_first + j * 32 * zrow + t * 128), 0, 0));
    return z;
  };
  // the tile's run of this block: 168 pieces of 16 bytes, 1 KB a wavefront
  auto stage_w = [&](int t) {
    const Rsrc rw = make_rsrc(wexp + (static_cast<int64_t>(t) * a.nb + b) * kRun, kRun);
    if (wave < 3) lds_load16(rw, sh.w[t % kRing] + wave * 1024, wave * 1024 + lane * 16);
  };
  // This wavefront's words of a tile, lane = row: code words 2w and 2w + 1 (12
  // aligned bytes around them) and select word w / 2 (8 bytes around it).  Rows
  // lie 42 bytes apart: even rows' words start 2 bytes into an aligned one.
  // (Loaded straight from memory, 42 bytes apart, they kept the L1's return
  // path busy 83 % of the time.)
  struct Raw {
    uint32_t w[3], h[2];
  };
  const int off_w = (lane * kBlockBytes + 2 + 8 * wave) & ~3, off_h = (lane * kBlockBytes + 34 + 4 * (wave >> 1)) & ~3;
  const uint32_t realign = (lane & 1) ? 0x03020100u : 0x05040302u;  // of (next, this)
  auto read_raw = [&](int t) {
    const char* base = sh.w[t % kRing];
    Raw x;
#pragma unroll
    for (int i = 0; i < 3; ++i) x.w[i] = *reinterpret_cast<const uint32_t*>(base + off_w + 4 * i);
#pragma unroll
    for (int i = 0; i < 2; ++i) x.h[i] = *reinterpret_cast<const uint32_t*>(base + off_h + 4 * i);
    return x;
  };
  auto read_d = [&](int t) { return *reinterpret_cast<const uint16_t*>(sh.w[t % kRing] + lane * kBlockBytes); };
  auto put_codes = [&](const Raw& x) {
    const uint32_t QH = __builtin_amdgcn_perm(x.h[1], x.h[0], realign);
    u32x4_t o;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t W = __builtin_amdgcn_perm(x.w[i + 1], x.w[i], realign);
      const int p = 2 * ((2 * wave + i) & 3);
      // byte j: 8 * code of local group 8i + j, then of 8i + 4 + j
      o[2 * i] = ((W << 3) & 0x78787878u) | ((QH << (7 - p)) & 0x80808080u);
      o[2 * i + 1] = ((W >> 1) & 0x78787878u) | ((QH << (6 - p)) & 0x80808080u);
    }
    *reinterpret_cast<u32x4_t*>(sh.rec[wave] + lane * 16) = o;
  };
  // D = 2^expo with 2^expo > every |d| so far; below 2^-15 there is nothing to
  // gain (1 / D has to be an fp16 number)
  int expo = -15;
  uint64_t far = 0;  // rows whose d / D is not a normal fp16 number (nor d itself, where D <= 1 loses nothing)
  auto raise = [&](uint16_t d, int e) {
    const uint32_t mag = d & 0x7FFFu;
    if (__ballot(mag >= static_cast<uint32_t>(e + 15) << 10) != 0)  // not every |d| < 2^e
      e = max(e, static_cast<int>(wave_umax(mag) >> 10) - 14);
    if constexpr (!kFar) far |= __ballot(mag - 1 < (e > 0 ? static_cast<uint32_t>(e + 1) << 10 : 1u) - 1);  // 0 < |d| < 2^(e-14)
    return e;
  };
  auto read_scales = [&](int slot) { return *reinterpret_cast<const u32x4_t*>(&sh.d[slot][wave][8 * (lane & 7)]); };
  auto put_z = [&](const Z& z, const u32x4_t& dw, int buf, int e) {
    const _Float16 f = __builtin_bit_cast(_Float16, static_cast<uint16_t>(e <= 14 ? (15 - e) << 10 : 0x0400 >> (e - 14)));  // 2^-e
    const float f32 = __builtin_bit_cast(float, (127 - e) << 23);  // the same
    f16x2_t d[4];
    float df[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = dw[i];
      if constexpr (kFar) {
        df[2 * i] = half_bits_to_float(w) * f32;
        df[2 * i + 1] = half_bits_to_float(w >> 16) * f32;
      } else {
        d[i] = __builtin_bit_cast(f16x2_t, w) * f;
      }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      u32x4_t o;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w = z.v[j][i];
        const f16x2_t v = __builtin_bit_cast(f16x2_t, w);
        if constexpr (kFar) o[i] = f16_pair(static_cast<float>(v[0]) * df[2 * i], static_cast<float>(v[1]) * df[2 * i + 1]);
        else o[i] = __builtin_bit_cast(uint32_t, v * d[i]);
      }
      *reinterpret_cast<u32x4_t*>(z_put + buf * (kStageTok * 128) + j * 32 * 128) = o;
    }
  };
  struct Step {
    u32x2_t v[8];  // four fp16 lanes of each of 8 rows
  };
  // The tile's codes of both steps: 16 lanes hand over 8 rows of 16 codes, lane
  // r takes group r's 8.  In one block with the wait for this wavefront's LDS
  // instructions and the barrier, both due here: the compiler cannot tell the
  // transposing read from the direct loads to LDS and would wait for those.
  const uint32_t get = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(sh.rec[wave] + lane * 8));
  auto take_codes = [&](u32x2_t (&c)[2]) {
    asm volatile(
        "ds_read_b64_tr_b8 %0, %2\n\t"
        "ds_read_b64_tr_b8 %1, %2 offset:512\n\t"
        "s_waitcnt lgkmcnt(0)\n\t"
        "s_barrier"
        : "=&v"(c[0]), "=&v"(c[1])
        : "v"(get)
        : "memory");
  };
  // rows 4h .. 4h + 3 of a lane's 8
  auto look_up = [&](const u32x2_t& codes, Step& p, int h) {
#pragma unroll
    for (int i = 4 * h; i < 4 * h + 4; ++i) {
      const uint32_t cw = codes[h];
      const uint32_t c = __builtin_amdgcn_ubfe(cw, 8 * (i & 3), 8);
      p.v[i] = *reinterpret_cast<const u32x2_t*>(reinterpret_cast<const char*>(sh.lut) + c);
    }
  };
  // their half of the four column sets' operands
  auto combine = [&](const Step& p, u32x4_t (&o)[4], int h) {
#pragma unroll
    for (int i = 2 * h; i < 2 * h + 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j][i] = __builtin_amdgcn_perm(p.v[2 * i + 1][j >> 1], p.v[2 * i][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
  };

  f32x4_t acc[4][NT];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[j][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int x = (r >> 1) & 7;
  int oa[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) oa[s] = r * 128 + (((4 * s + q) ^ x) << 4);
  f16x8_t A[NT];
  u32x4_t B[2][4];
  auto read_a = [&](int buf, int s, int i) { A[i] = *reinterpret_cast<const f16x8_t*>(sh.a[buf] + 16 * i * 128 + oa[s]); };
  // One step's products with B[s], the weights as the products' rows (as their
  // columns they take 3 % more time, and leave a lane 4 neighbouring outputs of
  // a token where it now has 16).  Each token operand is read for the step
  // (buf, s ^ 1) that follows as soon as its last use is issued, and `side`, the
  // work of the steps to come in four pieces, is spread between the products:
  // a wavefront can issue three other instructions while one product runs.
  auto multiply = [&](int buf, int s, auto side) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, B[s][j]), A[i], acc[j][i], 0, 0, 0);
      read_a(buf, s ^ 1, i);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k * NT / 4 == i) side(k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
        __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);  // up to three VALU instructions
        __builtin_amdgcn_sched_group_barrier(0x300, 2, 0);  // and two of LDS
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Prologue: the first five runs, the scales of tiles 0 and 1, tile 0's codes and dz
  const int last = a.tiles - 1;  // there are at least 8 tiles
#pragma unroll
  for (int t = 0; t < 5; ++t) stage_w(t);
  // dz is loaded two tiles ahead, or one where two would not fit the registers
  // (spilled, they cost 12 % at 96 rows)
  constexpr int kDepth = NT > 5 ? 1 : 2;
  Z z[2];
  z[0] = load_z(0);
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
  u32x2_t codes[2];
  int next;  // D's exponent with tile t + 1
  {
    const uint16_t d0 = read_d(0), d1 = read_d(1);
    sh.d[0][wave][lane] = d0;
    sh.d[1][wave][lane] = d1;
    put_codes(read_raw(0));
    expo = raise(d0, expo);
    next = raise(d1, expo);
    put_z(z[0], read_scales(0), 0, expo);
  }
  z[kDepth - 1] = load_z(1);
  if (kDepth == 2) z[0] = load_z(2);
  take_codes(codes);
  Step p;
#pragma unroll
  for (int i = 0; i < NT; ++i) read_a(0, 0, i);
  for (int h = 0; h < 2; ++h) {
    look_up(codes[0], p, h);
    combine(p, B[0], h);
  }
  // Tile t, its first step's operands ready.  nz holds dz of tile t + 1, on its
  // way since tile t - kDepth, and then takes t + 1 + kDepth.  The run of tile t
  // + 5 starts ahead of those loads, so when they have arrived (in tile t +
  // kDepth) it has too, and that tile's barrier shows it to every wavefront: its
  // scales are read in tile t + 3, its codes in tile t + 4.
  auto tile = [&](int t, int buf, Z& nz) {
    const Raw n = read_raw(t + 1);  // past the last tile: runs read before, not used
    const uint16_t d = read_d(t + 2);
    const u32x4_t dw = read_scales(buf ^ 1);
    multiply(buf, 0, [&](int k) {
      if (k < 2) look_up(codes[1], p, k);
      else combine(p, B[1], k - 2);
      if (k == 2) put_codes(n);
      if (k == 3) {
        put_z(nz, dw, buf ^ 1, next);
        sh.d[buf][wave][lane] = d;
      }
    });
    if (t + 5 <= last) stage_w(t + 5);
    __builtin_amdgcn_sched_barrier(0);
    nz = load_z(min(t + 1 + kDepth, last));
    // tile t + 1's dz is written and tile t's is read, by everyone
    take_codes(codes);
    multiply(buf ^ 1, 1, [&](int k) {
      if (k < 2) look_up(codes[0], p, k);
      else combine(p, B[0], k - 2);
    });
    if (next != expo && t < last) {
      const float f = ldexpf(1.0f, expo - next);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[j][i] *= f;
      expo = next;
    }
    if (t + 2 <= last) next = raise(d, next);
  };
  for (int t = 0; t < last && far == 0; t += 2) {  // an even number of tiles: the matrix has 512 rows or a multiple
    tile(t, 0, z[kDepth - 1]);
    tile(t + 1, 1, z[0]);
  }
  if (far != 0) return true;
  // dx[row0 + 16i + r, 256b + 64 wave + 16q + 4e + j]: 16 neighbouring columns
  const int64_t ld = static_cast<int64_t>(a.nb) * kQK;
  const float big = ldexpf(1.0f, expo);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int tok = 16 * i + r;
    if (tok >= mt) continue;
    const float inv = a.inv[row0 + tok];
    u32x2_t* out = reinterpret_cast<u32x2_t*>(a.dx + (row0 + tok) * ld + b * kQK + 64 * wave + 16 * q);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      out[e] = u32x2_t{bf16_pair(acc[0][i][e] * big * inv, acc[1][i][e] * big * inv),
                       bf16_pair(acc[2][i][e] * big * inv, acc[3][i][e] * big * inv)};
  }
  return false;
}

// One workgroup per (pass of an expert's tokens, block), passes found on the
// device and dealt to the XCDs as in the forward kernel: a pass's blocks share
// an XCD, and with it the pass's dz in that L2.
__global__ __launch_bounds__(kThreads, 2) void swiglu_dx_kernel(DxArgs a) {
  __shared__ DxSmem sh;
  const int xcd = blockIdx.x % kXcds;
  const int local = blockIdx.x / kXcds;
  const int b = local % a.nb;
  const PassUnit u = find_pass(a.offsets, a.n_experts, a.total_m, (local / a.nb) * kXcds + xcd, a.max_tok, kLonger);
  if (u.mt <= 0) return;
  if (threadIdx.x < 32) {
    uint64_t v = 0;
    for (int l = 0; l < 4; ++l) {
      const int t = code_lane_value(threadIdx.x, l);
      v |= static_cast<uint64_t>(t == 0 ? 0u : (t > 0 ? 0x3C00u : 0xBC00u)) << (16 * l);  // fp16 +-1
    }
    sh.lut[threadIdx.x] = v;
  }
  __syncthreads();
  const uint8_t* wexp = a.w + static_cast<int64_t>(u.expert) * a.estride;
  bool far;
  switch ((u.mt + 15) >> 4) {
    case 1: far = dx_pass<1, false>(a, sh, wexp, b, u.row0, u.mt); break;
    case 2: far = dx_pass<2, false>(a, sh, wexp, b, u.row0, u.mt); break;
    case 3: far = dx_pass<3, false>(a, sh, wexp, b, u.row0, u.mt); break;
    case 4: far = dx_pass<4, false>(a, sh, wexp, b, u.row0, u.mt); break;
    case 5: far = dx_pass<5, false>(a, sh, wexp, b, u.row0, u.mt); break;
    default: far = dx_pass<6, false>(a, sh, wexp, b, u.row0, u.mt); break;
  }
  if (!far) return;
  // what the pass had on its way to LDS has landed, for everyone
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if (u.mt <= 32) dx_pass<2, true>(a, sh, wexp, b, u.row0, u.mt);
  else dx_pass<6, true>(a, sh, wexp, b, u.row0, u.mt);
}

// ---------------------------------------------------------------------------
// dW_e = dz_e^T x_e
// ---------------------------------------------------------------------------
// A workgroup owns 256 rows x 128 columns of one expert's dW (a wavefront 64 x
// 128); the sum runs over the expert's tokens, 32 (one matrix-core step) at a
// time, through three LDS buffers.  Both operands lie [token][column] while
// the matrix cores want 8 consecutive tokens of one column, so they are read
// with the transposing 8-byte LDS read: 16 lanes give four tokens' 16 columns
// and each takes back four tokens of one.  The 16-byte pieces of a token are
// XORed by three bits of the token index, so the 16 tokens of one such read
// fall on different banks.  A step's 24 reads per 32 products are issued in
// one block that ends with their wait: left to the compiler, every one of them
// also waits for the direct loads to LDS in flight, which it cannot tell apart
// (439 us for 4099 rows of 8 experts of 4096 x 7168 in that form).

constexpr int kTR = 256, kTC = 128;  // rows and columns of a tile
constexpr int kTok = 32;             // tokens per stage
constexpr int kDwBuf = 3;

struct DwArgs {
  int n_experts;
  int n_r;           // matrix rows (2 d_ff)
  int n_c;           // d_model
  const int32_t* offsets;
  int64_t total_m;
  const uint16_t* dz;  // bf16 [total_m, n_r]
  const uint16_t* x;   // bf16 [total_m, n_c]
  uint16_t* dw;        // bf16 [n_experts, n_r, n_c]
};

__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int64_t total_m, int64_t* lo, int* m) {
  // clamped to [0, total_m], so that offsets outside the contract reach no row that is not there
  *lo = min(max(static_cast<int64_t>(offsets[e]), int64_t{0}), total_m);
  const int64_t hi = min(max(static_cast<int64_t>(offsets[e + 1]), *lo), total_m);
  *m = static_cast<int>(hi - *lo);
}

__device__ __forceinline__ int tok_swizzle(int t) { return 2 * ((t & 3) | ((t >> 1) & 4)); }

__global__ __launch_bounds__(kThreads, 2) void swiglu_dw_kernel(DwArgs a) {
  // three stages of dz and x, and after the last of them the outputs on their way
  __shared__ __align__(16) char smem[kDwBuf * kTok * (kTR + kTC) * 2];
  char(*const sz)[kTok * kTR * 2] = reinterpret_cast<char(*)[kTok * kTR * 2]>(smem);
  char(*const sx)[kTok * kTC * 2] = reinterpret_cast<char(*)[kTok * kTC * 2]>(smem + kDwBuf * kTok * kTR * 2);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, r = lane & 15;
  // Workgroups are dealt to the XCDs in turn: each takes one run of an
  // expert's tiles in bands of 8 rows of tiles, so that those at work together
  // share a compact block of dz and x in its L2 (4099 rows of 8 experts of
  // 4096 x 7168: 334 MB fetched and 267 us, 851 MB and 285 with rows fastest).
  const int tr = a.n_r / kTR, tc = a.n_c / kTC;
  const int per = (tr * tc + kXcds - 1) / kXcds;
  const int e = blockIdx.x / (per * kXcds), in = blockIdx.x % (per * kXcds);
  const int tile = (in % kXcds) * per + in / kXcds;
  if (tile >= tr * tc) return;
  const int band = tile / (8 * tc), rows = min(8, tr - band * 8), at = tile - band * 8 * tc;
  const int r0 = (band * 8 + at % rows) * kTR, c0 = (at / rows) * kTC;
  int64_t lo;
  int m;
  expert_rows(a.offsets, e, a.total_m, &lo, &m);
  const uint32_t zrow = static_cast<uint32_t>(a.n_r) * 2, xrow = static_cast<uint32_t>(a.n_c) * 2;
  // a wavefront instruction brings 2 tokens of dz (32 pieces each), 4 of x (16 each)
  constexpr int kLoads = kTok / 2 / kWaves + kTok / 4 / kWaves;
  auto stage = [&](int s) {
    const int buf = s % kDwBuf;
    const int64_t t0 = lo + static_cast<int64_t>(s) * kTok;
    const int tv = min(kTok, m - s * kTok);
    // tokens past the expert's rows lie past the descriptors' ranges and read as zeros
    const Rsrc rz = make_rsrc(a.dz + t0 * a.n_r + r0, (tv - 1) * zrow + kTR * 2);
    const Rsrc rx = make_rsrc(a.x + t0 * a.n_c + c0, (tv - 1) * xrow + kTC * 2);
#pragma unroll
    for (int j = 0; j < kTok / 2 / kWaves; ++j) {
      const int ins = wave + j * kWaves, t = ins * 2 + (lane >> 5);
      lds_load16(rz, sz[buf] + ins * 1024, t < tv ? t * zrow + ((lane & 31) ^ tok_swizzle(t)) * 16 : 0xFFFFFFF0u);
    }
#pragma unroll
    for (int j = 0; j < kTok / 4 / kWaves; ++j) {
      const int ins = wave + j * kWaves, t = ins * 4 + (lane >> 4);
      lds_load16(rx, sx[buf] + ins * 1024, t < tv ? t * xrow + ((lane & 15) ^ tok_swizzle(t)) * 16 : 0xFFFFFFF0u);
    }
  };
  f32x4_t acc[8][4];  // [column tile][row tile]
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // This lane's part of the transposing read of tokens 8q + 0..3 (the other
  // four lie four tokens' bytes on, in the same swizzle) and 16 columns: token
  // 8q + r / 4, columns 4 (r % 4) ..+3 of them.  Column tile i is 32 bytes on,
  // under the swizzle an XOR of 32 i, so one address a tile.
  const int t = 8 * q + (r >> 2);
  const int fz = t * kTR * 2, fx = t * kTC * 2, sw = tok_swizzle(t) * 16 + (r & 3) * 8;
  auto lds = [](const void* p) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)); };
  const int ns = (m + kTok - 1) / kTok;
#pragma unroll
  for (int s = 0; s < kDwBuf - 1; ++s)
    if (s < ns) stage(s);
  for (int s = 0; s < ns; ++s) {
    // stage s has landed (s + 1 may be on its way), here and for everyone, and
    // everyone has read stage s - 1, whose buffer the next loads take
    if (s + 1 < ns) asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kLoads) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    if (s + kDwBuf - 1 < ns) stage(s + kDwBuf - 1);
    const uint32_t bz = lds(sz[s % kDwBuf]) + fz, bx = lds(sx[s % kDwBuf]) + fx;
    u32x2_t z[4][2], x[8][2];
    uint32_t az[4], ax[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) az[j] = bz + (sw ^ (128 * wave + 32 * j));
#pragma unroll
    for (int i = 0; i < 8; ++i) ax[i] = bx + (sw ^ (32 * i));
    // tokens +4: 4 rows of 512 (dz) or 256 (x) bytes on
    asm volatile(
        "ds_read_b64_tr_b16 %0, %24\n\tds_read_b64_tr_b16 %1, %24 offset:2048\n\t"
        "ds_read_b64_tr_b16 %2, %25\n\tds_read_b64_tr_b16 %3, %25 offset:2048\n\t"
        "ds_read_b64_tr_b16 %4, %26\n\tds_read_b64_tr_b16 %5, %26 offset:2048\n\t"
        "ds_read_b64_tr_b16 %6, %27\n\tds_read_b64_tr_b16 %7, %27 offset:2048\n\t"
        "ds_read_b64_tr_b16 %8, %28\n\tds_read_b64_tr_b16 %9, %28 offset:1024\n\t"
        "ds_read_b64_tr_b16 %10, %29\n\tds_read_b64_tr_b16 %11, %29 offset:1024\n\t"
        "ds_read_b64_tr_b16 %12, %30\n\tds_read_b64_tr_b16 %13, %30 offset:1024\n\t"
        "ds_read_b64_tr_b16 %14, %31\n\tds_read_b64_tr_b16 %15, %31 offset:1024\n\t"
        "ds_read_b64_tr_b16 %16, %32\n\tds_read_b64_tr_b16 %17, %32 offset:1024\n\t"
        "ds_read_b64_tr_b16 %18, %33\n\tds_read_b64_tr_b16 %19, %33 offset:1024\n\t"
        "ds_read_b64_tr_b16 %20, %34\n\tds_read_b64_tr_b16 %21, %34 offset:1024\n\t"
        "ds_read_b64_tr_b16 %22, %35\n\tds_read_b64_tr_b16 %23, %35 offset:1024\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(z[0][0]), "=&v"(z[0][1]), "=&v"(z[1][0]), "=&v"(z[1][1]), "=&v"(z[2][0]), "=&v"(z[2][1]), "=&v"(z[3][0]),
          "=&v"(z[3][1]), "=&v"(x[0][0]), "=&v"(x[0][1]), "=&v"(x[1][0]), "=&v"(x[1][1]), "=&v"(x[2][0]), "=&v"(x[2][1]),
          "=&v"(x[3][0]), "=&v"(x[3][1]), "=&v"(x[4][0]), "=&v"(x[4][1]), "=&v"(x[5][0]), "=&v"(x[5][1]), "=&v"(x[6][0]),
          "=&v"(x[6][1]), "=&v"(x[7][0]), "=&v"(x[7][1])
        : "v"(az[0]), "v"(az[1]), "v"(az[2]), "v"(az[3]), "v"(ax[0]), "v"(ax[1]), "v"(ax[2]), "v"(ax[3]), "v"(ax[4]),
          "v"(ax[5]), "v"(ax[6]), "v"(ax[7])
        : "memory");
    bf16x8_t Z[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) Z[j] = __builtin_bit_cast(bf16x8_t, u32x4_t{z[j][0][0], z[j][0][1], z[j][1][0], z[j][1][1]});
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bf16x8_t X = __builtin_bit_cast(bf16x8_t, u32x4_t{x[i][0][0], x[i][0][1], x[i][1][0], x[i][1][1]});
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(X, Z[j], acc[i][j], 0, 0, 0);
    }
  }
  // A lane holds dw[e, r0 + 64 wave + 16j + r, c0 + 16i + 4q + 0..3], 8 bytes in
  // each of 16 rows an instruction: through LDS to whole rows of 256 bytes
  // (stored straight, the 470 MB of 8 experts cost 130 us more).  Every
  // wavefront has a part of its own, rows 16 bytes apart from a bank's period.
  constexpr int kRowB = kTC * 2 + 16;
  static_assert(kWaves * 64 * kRowB <= kDwBuf * kTok * (kTR + kTC) * 2, "the outputs fit where the stages were");
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // everyone has read the last stage
  char* const mine = smem + wave * 64 * kRowB;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      *reinterpret_cast<u32x2_t*>(mine + (16 * j + r) * kRowB + 32 * i + 8 * q) =
          u32x2_t{bf16_pair(acc[i][j][0], acc[i][j][1]), bf16_pair(acc[i][j][2], acc[i][j][3])};
  __builtin_amdgcn_wave_barrier();  // LDS serves a wavefront's instructions in order
  uint16_t* out = a.dw + (static_cast<int64_t>(e) * a.n_r + r0 + 64 * wave) * a.n_c + c0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int row = 4 * j + q;
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(mine + row * kRowB + r * 16);
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(out + static_cast<int64_t>(row) * a.n_c) + r);
  }
}

}  // namespace

SwigluBwdLayout swiglu_bwd_layout(int64_t d_ff, int64_t total_m, bool dx, bool dw) {
  auto up = [](int64_t b) { return (b + 255) / 256 * 256; };
  SwigluBwdLayout l{};
  const int64_t z = up(total_m * 2 * d_ff * 2);
  if (dx) {
    l.inv = z;
    l.dzb = z + up(total_m * 4);
  }
  l.bytes = l.dzb + (dw ? z : 0);
  return l;
}

// Rows of a pass: 96, or 32 where those would leave much of the chip idle.
// Measured, us of the whole call without dW, 96 / 32: one expert of 2 x 1024
// of 4096, 100 rows 33 / 28, 500 rows 41 / 30, 4000 rows 90 / 128; 2 x 2048 of
// 7168, 8 experts, 300 rows 57 / 61, 4096 rows 268 / 385.  (Passes of 80: 39
// for 500 rows, 97 for 4000, 285 for 4096 of 8 experts.)
int dx_rows_a_pass(const SwigluBwdArgs& g, int cus) {
  constexpr PassCost kCost{2.0, {0.5, 0.007}, {0.64, 0.0108}};  // a 64-row tile
  auto step = [&](int max_tok) { return pass_step_us(kCost, g.total_m, g.n_experts, max_tok, g.d_model / kQK, cus); };
  return step(32) < 0.95 * step(kMaxTok) ? 32 : kMaxTok;
}

hipError_t launch_swiglu_bwd(const SwigluBwdArgs& g, void* ws, int cus, hipStream_t s) {
  const SwigluBwdLayout l = swiglu_bwd_layout(g.d_ff, g.total_m, g.dx != nullptr, g.dw != nullptr);
  char* base = static_cast<char*>(ws);
  uint16_t* dz16 = g.dx ? reinterpret_cast<uint16_t*>(base) : nullptr;
  float* inv = g.dx ? reinterpret_cast<float*>(base + l.inv) : nullptr;
  uint16_t* dzb = g.dw ? reinterpret_cast<uint16_t*>(base + l.dzb) : nullptr;
  if (g.total_m > 0) {
    const DzArgs za{g.gate_up, g.dh, static_cast<int>(g.d_ff), dz16, inv, dzb};
    hipLaunchKernelGGL(dz_kernel, dim3(static_cast<unsigned>(g.total_m)), dim3(256), 0, s, za);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (g.dx && g.total_m > 0) {
    DxArgs a{g.w_table, g.expert_stride, static_cast<int>(g.n_experts), static_cast<int>(g.d_model / kQK),
             static_cast<int>(2 * g.d_ff / kTileRows), g.offsets, g.total_m, dz16, inv, g.dx, dx_rows_a_pass(g, cus)};
    const int64_t units = (pass_units(g.total_m, g.n_experts, a.max_tok) + kXcds - 1) / kXcds * kXcds;
    hipLaunchKernelGGL(swiglu_dx_kernel, dim3(static_cast<unsigned>(units * a.nb)), dim3(kThreads), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (g.dw) {
    DwArgs a{static_cast<int>(g.n_experts), static_cast<int>(2 * g.d_ff), static_cast<int>(g.d_model), g.offsets,
             g.total_m, dzb, g.x, g.dw};
    const int64_t tiles = (2 * g.d_ff / kTR) * (g.d_model / kTC);
    const int64_t grid = g.n_experts * ((tiles + kXcds - 1) / kXcds * kXcds);
    hipLaunchKernelGGL(swiglu_dw_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace stq
