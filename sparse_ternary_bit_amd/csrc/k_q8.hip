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
#include "stq_device.hpp"
#include "stq_launch.hpp"

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

// One workgroup a row.  The row is read twice, the second time from cache.
// kVec: rows start on 16 bytes.
template <typename T, bool kVec>
__global__ __launch_bounds__(256) void q8_quantize_kernel(QuantArgs a) {
  __shared__ uint32_t wmax[4];
  const int64_t r = blockIdx.x;
  const T* row = static_cast<const T*>(a.x) + r * a.stride;
  const int64_t groups = (a.k + 15) / 16;
  // the largest magnitude as bits: a NaN orders above every number and so is kept
  uint32_t mx = 0;
  for (int64_t g = threadIdx.x; g < groups; g += 256) {
    float v[16];
    load16<T, kVec>(row, g * 16, a.k, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = max(mx, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) mx = max(mx, static_cast<uint32_t>(__shfl_xor(static_cast<int>(mx), o)));
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = mx;
  __syncthreads();
  mx = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  const bool finite = mx < 0x7F800000u;
  const float scale = finite ? __builtin_bit_cast(float, mx) / 127.0f : NAN;
  if (threadIdx.x == 0) a.scale[r] = scale;
  const bool some = finite && scale > 0.0f;
  const double sd = some ? static_cast<double>(scale) : 0.0;
  const double inv = some ? 1.0 / sd : 0.0;
  const double half = 0.5 * sd;
  for (int64_t g = threadIdx.x; g < groups; g += 256) {
    float v[16];
    load16<T, kVec>(row, g * 16, a.k, v);
    u32x4_t o = {0, 0, 0, 0};
    if (some) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const double x = static_cast<double>(v[i]);
        double q = rint(x * inv);
        const double rem = fma(-q, sd, x);
        // the product can land on the wrong side only next to a half
        if (fabs(rem) > half) q += rem > 0.0 ? 1.0 : -1.0;
        else if (fabs(rem) == half) {
          const double other = q + (rem > 0.0 ? 1.0 : -1.0);
          if (static_cast<int>(q) & 1) q = other;
        }
        const int qi = max(-127, min(127, static_cast<int>(q)));
        o[i >> 2] |= (static_cast<uint32_t>(qi) & 0xFFu) << (8 * (i & 3));
      }
    }
    *reinterpret_cast<u32x4_t*>(a.q + r * a.ldq + g * 16) = o;
  }
}

// ---------------------------------------------------------------------------
// product
// ---------------------------------------------------------------------------

constexpr int kBK = 128;  // bytes of k per stage

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
  int vec;  // four outputs may be stored at once
};

__device__ __forceinline__ void lds_load16(Rsrc rs, void* lds, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      rs, reinterpret_cast<__attribute__((address_space(3))) void*>(reinterpret_cast<uintptr_t>(lds)), 16,
      static_cast<int>(voff), 0, 0, 0);
}

// Workgroup: TM tokens x TN channels, WM x WN wavefronts.  Both operands
// stream into LDS 128 bytes of k at a time (direct 16-byte loads, two
// buffers); a row's eight 16-byte chunks are XORed by half the row index, so
// the 16 rows of an operand read fall on 16 different 16-byte bank groups.
template <int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(WM * WN * 64) void q8_gemm_kernel(QArgs a) {
  constexpr int kNW = WM * WN;
  constexpr int FM = TM / WM / 16, FN = TN / WN / 16;
  __shared__ __align__(16) int8_t sa[2][TM * kBK];
  __shared__ __align__(16) int8_t sw[2][TN * kBK];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, r = lane & 15;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * TM, n0 = static_cast<int64_t>(blockIdx.x) * TN;
  const int mv = static_cast<int>(min(static_cast<int64_t>(TM), a.m - m0));
  const int nv = static_cast<int>(min(static_cast<int64_t>(TN), a.n - n0));
  const uint32_t kpad = static_cast<uint32_t>((a.k + 15) & ~15);
  const Rsrc ra = make_rsrc(a.a + m0 * a.lda, static_cast<uint32_t>((mv - 1) * a.lda) + kpad);
  const Rsrc rw = make_rsrc(a.w + n0 * a.ldw, static_cast<uint32_t>((nv - 1) * a.ldw) + kpad);
  auto stage = [&](int s, int buf) {
    const int row8 = lane >> 3, slot = lane & 7;
    for (int j = wave; j < TM / 8; j += kNW) {
      const int row = j * 8 + row8;
      lds_load16(ra, sa[buf] + j * 1024, row * static_cast<uint32_t>(a.lda) + s * kBK + ((slot ^ ((row >> 1) & 7)) << 4));
    }
    for (int j = wave; j < TN / 8; j += kNW) {
      const int row = j * 8 + row8;
      lds_load16(rw, sw[buf] + j * 1024, row * static_cast<uint32_t>(a.ldw) + s * kBK + ((slot ^ ((row >> 1) & 7)) << 4));
    }
  };
  i32x4_t acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  const int wm = wave / WN, wn = wave % WN;
  const int ns = static_cast<int>((a.k + kBK - 1) / kBK);
  const int tail = static_cast<int>(a.k % kBK);
  const int x = (r >> 1) & 7;
  stage(0, 0);
  for (int s = 0; s < ns; ++s) {
    const int buf = s & 1;
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
    if (s + 1 < ns) stage(s + 1, buf ^ 1);
    if (tail && s + 1 == ns) {
      // past the end of k: zeros in the token operand, whatever the rows hold there
      for (int i = tid; i < TM * kBK; i += kNW * 64) {
        const int row = i / kBK, c = i % kBK;
        if (c >= tail) sa[buf][row * kBK + (((c >> 4) ^ ((row >> 1) & 7)) << 4) + (c & 15)] = 0;
      }
      __syncthreads();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int so = ((4 * h + q) ^ x) << 4;
      i32x4_t fa[FM], fw[FN];
#pragma unroll
      for (int j = 0; j < FM; ++j) fa[j] = *reinterpret_cast<const i32x4_t*>(sa[buf] + (wm * FM * 16 + j * 16 + r) * kBK + so);
#pragma unroll
      for (int i = 0; i < FN; ++i) fw[i] = *reinterpret_cast<const i32x4_t*>(sw[buf] + (wn * FN * 16 + i * 16 + r) * kBK + so);
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[i], fa[j], acc[i][j], 0, 0, 0);
    }
  }
  // token m0 + ... + r, channels n0 + ... + 4q + 0..3
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int64_t tok = m0 + wm * FM * 16 + j * 16 + r;
    if (tok >= a.m) continue;
    const float ts = a.as[tok];
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      const int64_t c = n0 + wn * FN * 16 + i * 16 + 4 * q;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = c + e < a.n ? static_cast<float>(acc[i][j][e]) * ts * a.ws[c + e] : 0.0f;
      if (a.bf16) {
        uint16_t* y = static_cast<uint16_t*>(a.y) + tok * a.ldy + c;
        if (a.vec && c + 3 < a.n) {
          *reinterpret_cast<u32x2_t*>(y) = u32x2_t{bf16_bits(v[0]) | bf16_bits(v[1]) << 16, bf16_bits(v[2]) | bf16_bits(v[3]) << 16};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < a.n) y[e] = static_cast<uint16_t>(bf16_bits(v[e]));
        }
      } else {
        float* y = static_cast<float*>(a.y) + tok * a.ldy + c;
        if (a.vec && c + 3 < a.n) {
          *reinterpret_cast<f32x4_t*>(y) = f32x4_t{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < a.n) y[e] = v[e];
        }
      }
    }
  }
}

template <int TM, int TN, int WM, int WN>
void launch_tile(const QArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.n + TN - 1) / TN), static_cast<unsigned>((a.m + TM - 1) / TM));
  hipLaunchKernelGGL((q8_gemm_kernel<TM, TN, WM, WN>), grid, dim3(WM * WN * 64), 0, s, a);
}

}  // namespace

hipError_t launch_q8_quantize(const Q8QuantArgs& g, hipStream_t s) {
  const QuantArgs a{g.x, g.x_stride, g.k, g.q, g.ldq, g.scale};
  const dim3 grid(static_cast<unsigned>(g.rows));
  const int esz = g.bf16 ? 2 : 4;
  const bool vec = (reinterpret_cast<uintptr_t>(g.x) & 15) == 0 && (g.x_stride * esz) % 16 == 0;
  if (g.bf16) {
    if (vec) hipLaunchKernelGGL((q8_quantize_kernel<uint16_t, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((q8_quantize_kernel<uint16_t, false>), grid, dim3(256), 0, s, a);
  } else {
    if (vec) hipLaunchKernelGGL((q8_quantize_kernel<float, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((q8_quantize_kernel<float, false>), grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

int64_t q8_matmul_scratch_bytes(int64_t m, int64_t n, int64_t k, int cus) { return 0; }

hipError_t launch_q8_matmul(const Q8MatmulArgs& g, void* ws, hipStream_t s) {
  QArgs a{g.a, g.lda, g.a_scale, g.w, g.ldw, g.w_scale, g.m, g.n, g.k, g.y, g.ldy, g.bf16, 0};
  const int esz = g.bf16 ? 2 : 4;
  a.vec = (reinterpret_cast<uintptr_t>(g.y) % (4 * esz)) == 0 && g.ldy % 4 == 0;
  if (g.m <= 16) launch_tile<16, 64, 1, 4>(a, s);
  else if (g.m <= 64) launch_tile<64, 128, 1, 4>(a, s);
  else launch_tile<128, 128, 2, 2>(a, s);
  return hipGetLastError();
}

}  // namespace stq
