// Residual addition, root-mean-square norm and the rounding of the normed rows
// to 8-bit integers, in one pass, and the norm's gradients.
//
//     h = x + r (rounded to the stream's type)     rstd = 1 / sqrt(mean h^2 + eps)
//     y = h w rstd         q = nearest integer to y / scale,  scale = max |y| / 127
//
// rstd is the same for the whole row, so the integers do not depend on it:
// with v = h w and step = fp32(max |v| / 127), q is the integer nearest the
// exact v / step and scale = step rstd.  One pass over the row therefore
// gives the sum of squares and the largest |v| together, the row stays in
// registers, and the integers have one right value whatever the order of the
// sum.
//
// Gradients, with u = h rstd and g = dy w:
//     dx = dh + rstd (g - u mean(g u))            dw = sum over rows of dy u
#include <algorithm>
#include <type_traits>

#include "stq_launch.hpp"
#include "stq_round8.hpp"
#include "stq_rows.hpp"

namespace stq {
namespace {

struct None {};  // no residual

// Sum of `v` over a workgroup in a fixed order; `slot` holds one float a
// wavefront and is free again after the next barrier but one.
template <int kThreads>
__device__ __forceinline__ float block_sum(float v, float* slot) {
  v = sum64(v);
  if constexpr (kThreads == 64) return v;
  if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = slot[0];
#pragma unroll
  for (int i = 1; i < kThreads / 64; ++i) s += slot[i];
  return s;
}

// One workgroup a row; kHeld groups of 8 values a thread stay in registers,
// what lies beyond (rows of more than 8192 values) is read again.  HBM bounds
// it: 8192 rows of 7168, bf16 with a residual to 8 bits, 76 us for 411 MB, 5.4
// TB/s read and written.
template <typename TX, typename TR, int kThreads, int kHeld>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs a) {
  constexpr bool kRes = !__is_same(TR, None);
  __shared__ float ssum[kThreads / 64];
  __shared__ uint32_t smax[kThreads / 64];
  const int64_t r = blockIdx.x;
  const int64_t d = a.d, groups = (d + 7) / 8;
  const TX* x = static_cast<const TX*>(a.x) + r * a.x_stride;
  // the residual's type, or any where there is none
  using Res = std::conditional_t<kRes, TR, bf16_t>;
  auto load_res = [&](int64_t c) {
    if constexpr (kRes) return load8<TR>(static_cast<const TR*>(a.res) + r * a.res_stride, c, d);
    else return Raw8<Res>{};
  };
  float ss = 0.0f;
  uint32_t mx = 0;  // the largest |v| as bits: a NaN orders above every number and so is kept
  // the sum as it is stored, 8 values from column c on; columns past d are 0
  auto sum8 = [&](int64_t c, float (&f)[8], Raw8<TX> rx, Raw8<Res> rr) {
    settle8<TX>(rx, c, d);
    unpack8<TX>(rx, f);
    if constexpr (kRes) {
      float b[8];
      settle8<TR>(rr, c, d);
      unpack8<TR>(rr, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] += b[i];
      const Raw8<TR> o = pack8<TR>(f);
      store8<TR>(static_cast<TR*>(a.h) + r * a.h_stride, c, d, o);
      unpack8<TR>(o, f);
    }
  };
  auto weigh = [&](int64_t c, const float (&f)[8], float (&v)[8]) {
    float w[8];
    load8f<float>(a.weight, c, d, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = f[i] * w[i];
      ss = fmaf(f[i], f[i], ss);
      mx = max(mx, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
    }
  };
  float v[kHeld][8];
  {
    Raw8<TX> rx[kHeld];
    Raw8<Res> rr[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      rx[i] = load8<TX>(x, (threadIdx.x + i * kThreads) * 8, d);
      rr[i] = load_res((threadIdx.x + i * kThreads) * 8);
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (threadIdx.x + i * kThreads) * 8;
      float f[8];
      sum8(c, f, rx[i], rr[i]);
      weigh(c, f, v[i]);
    }
  }
  for (int64_t g = threadIdx.x + kHeld * kThreads; g < groups; g += kThreads) {
    float f[8], t[8];
    sum8(g * 8, f, load8<TX>(x, g * 8, d), load_res(g * 8));
    weigh(g * 8, f, t);
  }
  ss = sum64(ss);
  mx = max64(mx);
  if constexpr (kThreads > 64) {
    if ((threadIdx.x & 63) == 0) {
      ssum[threadIdx.x >> 6] = ss;
      smax[threadIdx.x >> 6] = mx;
    }
    __syncthreads();
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) {
      ss += ssum[i];
      mx = max(mx, smax[i]);
    }
  }
  const float rstd = 1.0f / sqrtf(ss / static_cast<float>(d) + a.eps);
  const bool finite = mx < 0x7F800000u;
  const float step = finite ? __builtin_bit_cast(float, mx) / 127.0f : NAN;
  if (threadIdx.x == 0) {
    if (a.rstd) a.rstd[r] = rstd;
    if (a.q) a.scale[r] = step == 0.0f ? 0.0f : step * rstd;   // (zeros without eps: rstd is infinite)
  }
  const bool some = finite && step > 0.0f;
  const float inv = some ? 1.0f / step : 0.0f;
  const bool fast = step > 0x1p-100f;
  auto put = [&](int64_t g, const float (&t)[8]) {
    if (a.q) {
      uint32_t o[2] = {0, 0};
      if (some) quantize<8>(t, step, inv, fast, o);
      *reinterpret_cast<u32x2_t*>(a.q + r * a.q_stride + g * 8) = u32x2_t{o[0], o[1]};
      // the row's last 16 bytes are its own: the half that no group covers is 0
      if (g == groups - 1 && (groups & 1)) *reinterpret_cast<u32x2_t*>(a.q + r * a.q_stride + g * 8 + 8) = u32x2_t{0, 0};
    }
    if (a.y) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = t[i] * rstd;
      store8<bf16_t>(reinterpret_cast<bf16_t*>(a.y) + r * a.y_stride, g * 8, d, pack8<bf16_t>(y));
    }
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (threadIdx.x + i * kThreads < groups) put(threadIdx.x + i * kThreads, v[i]);
  for (int64_t g = threadIdx.x + kHeld * kThreads; g < groups; g += kThreads) {
    float f[8], w[8], t[8];
    // this thread's own store of the sum, or x
    if constexpr (kRes) load8f<TR>(static_cast<const TR*>(a.h) + r * a.h_stride, g * 8, d, f);
    else load8f<TX>(x, g * 8, d, f);
    load8f<float>(a.weight, g * 8, d, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = f[i] * w[i];
    put(g, t);
  }
}

// dx, and each workgroup's part of dw: a workgroup walks the rows blockIdx.x,
// + gridDim.x, ..., and its threads add dy u for their columns in registers, so
// that dw costs no pass of its own.  kHeld * kThreads * 8 columns at most.  HBM
// bounds it: 4099 rows of 7168 with dh, all bf16, 47 us for 235 MB, 5.0 TB/s.
template <typename TH, typename TY, int kThreads, int kHeld>
__global__ __launch_bounds__(kThreads, 2) void norm_bwd_kernel(NormBwdArgs a, float* part) {
  // rows that are read at once: where a row is one group a thread, the latency of
  // its loads would stand alone (6845 rows of 87, cold: 43 us a row at a time, 24 so)
  constexpr int kBatch = kHeld == 1 ? 4 : 1, kWaves = kThreads / 64;
  __shared__ float slot[2][kBatch][kWaves];
  const int64_t d = a.d;
  float w[kHeld][8], acc[kHeld][8];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    load8f<float>(a.weight, (threadIdx.x + i * kThreads) * 8, d, w[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
  }
  int odd = 0;
  for (int64_t r0 = blockIdx.x; r0 < a.rows; r0 += kBatch * static_cast<int64_t>(gridDim.x), odd ^= 1) {
    float rstd[kBatch], dot[kBatch];
    Raw8<TH> rh[kBatch][kHeld], rd[kBatch][kHeld];
    Raw8<TY> ry[kBatch][kHeld];
    auto row = [&](int b) { return r0 + static_cast<int64_t>(b) * gridDim.x; };
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int64_t r = min(row(b), a.rows - 1);   // (past the last: read, and not looked at)
      rstd[b] = a.rstd[r];
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int64_t c = (threadIdx.x + i * kThreads) * 8;
        rh[b][i] = load8<TH>(static_cast<const TH*>(a.h) + r * a.h_stride, c, d);
        ry[b][i] = load8<TY>(static_cast<const TY*>(a.dy) + r * a.dy_stride, c, d);
        if (a.dh) rd[b][i] = load8<TH>(static_cast<const TH*>(a.dh) + r * a.dh_stride, c, d);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (row(b) >= a.rows) break;
      dot[b] = 0.0f;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        float f[8], g[8];
        settle8<TH>(rh[b][i], (threadIdx.x + i * kThreads) * 8, d);
        settle8<TY>(ry[b][i], (threadIdx.x + i * kThreads) * 8, d);
        unpack8<TH>(rh[b][i], f);
        unpack8<TY>(ry[b][i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float u = f[e] * rstd[b];
          acc[i][e] = fmaf(g[e], u, acc[i][e]);
          dot[b] = fmaf(g[e] * w[i][e], u, dot[b]);
        }
      }
      dot[b] = sum64(dot[b]);
      if (kWaves > 1 && (threadIdx.x & 63) == 0) slot[odd][b][threadIdx.x >> 6] = dot[b];
    }
    if constexpr (kWaves > 1) __syncthreads();
    if (!a.dx) continue;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (row(b) >= a.rows) break;
      if constexpr (kWaves > 1) {
        dot[b] = slot[odd][b][0];
#pragma unroll
        for (int i = 1; i < kWaves; ++i) dot[b] += slot[odd][b][i];
      }
      const float mean = dot[b] / static_cast<float>(d);
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const int64_t c = (threadIdx.x + i * kThreads) * 8;
        float f[8], g[8], o[8];
        unpack8<TH>(rh[b][i], f);
        unpack8<TY>(ry[b][i], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = rstd[b] * (g[e] * w[i][e] - f[e] * rstd[b] * mean);
        if (a.dh) {
          settle8<TH>(rd[b][i], c, d);
          unpack8<TH>(rd[b][i], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] += f[e];
        }
        if (c < d) store8<TH>(static_cast<TH*>(a.dx) + row(b) * a.dx_stride, c, d, pack8<TH>(o));
      }
    }
  }
  if (part) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int64_t c = (threadIdx.x + i * kThreads) * 8;
      if (c < d) store8<float>(part + static_cast<int64_t>(blockIdx.x) * d, c, d, pack8<float>(acc[i]));
    }
  }
}

// dx of row r by a workgroup, with a second read of the row
template <typename TH, typename TY, int kThreads>
__device__ __forceinline__ void dx_row(const NormBwdArgs& a, int64_t r, float* slot) {
  const int64_t d = a.d;
  const TH* h = static_cast<const TH*>(a.h) + r * a.h_stride;
  const TY* dy = static_cast<const TY*>(a.dy) + r * a.dy_stride;
  const float rstd = a.rstd[r];
  float dot = 0.0f;
  for (int64_t c = threadIdx.x * 8; c < d; c += kThreads * 8) {
    float f[8], g[8], w[8];
    load8f<TH>(h, c, d, f);
    load8f<TY>(dy, c, d, g);
    load8f<float>(a.weight, c, d, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) dot = fmaf(g[e] * w[e], f[e] * rstd, dot);
  }
  const float mean = block_sum<kThreads>(dot, slot) / static_cast<float>(d);
  for (int64_t c = threadIdx.x * 8; c < d; c += kThreads * 8) {
    float f[8], g[8], w[8], o[8];
    load8f<TH>(h, c, d, f);
    load8f<TY>(dy, c, d, g);
    load8f<float>(a.weight, c, d, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = rstd * (g[e] * w[e] - f[e] * rstd * mean);
    if (a.dh) {
      load8f<TH>(static_cast<const TH*>(a.dh) + r * a.dh_stride, c, d, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += f[e];
    }
    store8<TH>(static_cast<TH*>(a.dx) + r * a.dx_stride, c, d, pack8<TH>(o));
  }
}

// Few rows: a workgroup a row for dx, and one for 64 columns of dw, whose 32
// shares of the rows are joined through LDS.  One launch and no parts, for a
// second read of dy and h.  (Cold, events around the call: 64 x 878 12.0 us, 14.3
// with parts; 256 x 512 10.8 and 12.6, x 7168 14.9 and 19.6; 400 x 512 as one
// launch 14.1, with parts 13.3.)
template <typename TH, typename TY>
__global__ __launch_bounds__(256) void norm_bwd_few_kernel(NormBwdArgs a, int dx_rows) {
  __shared__ float part[32][64];
  if (static_cast<int>(blockIdx.x) < dx_rows) {
    dx_row<TH, TY, 256>(a, blockIdx.x, part[0]);
    return;
  }
  const int64_t c0 = static_cast<int64_t>(blockIdx.x - dx_rows) * 64, c = c0 + (threadIdx.x & 7) * 8;
  const int g = threadIdx.x >> 3;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  if (c < a.d) {
    constexpr int kAt = 4;   // rows in flight
    for (int64_t r0 = g; r0 < a.rows; r0 += 32 * kAt) {
      Raw8<TH> rh[kAt];
      Raw8<TY> ry[kAt];
      float rstd[kAt];
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        const int64_t r = min(r0 + 32 * i, a.rows - 1);
        rh[i] = load8<TH>(static_cast<const TH*>(a.h) + r * a.h_stride, c, a.d);
        ry[i] = load8<TY>(static_cast<const TY*>(a.dy) + r * a.dy_stride, c, a.d);
        rstd[i] = a.rstd[r];
      }
#pragma unroll
      for (int i = 0; i < kAt; ++i) {
        if (r0 + 32 * i >= a.rows) break;
        float f[8], y[8];
        settle8<TH>(rh[i], c, a.d);
        settle8<TY>(ry[i], c, a.d);
        unpack8<TH>(rh[i], f);
        unpack8<TY>(ry[i], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(y[e], f[e] * rstd[i], acc[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) part[g][(threadIdx.x & 7) * 8 + e] = acc[e];
  __syncthreads();
  if (threadIdx.x >= 64 || c0 + threadIdx.x >= a.d) return;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += part[i][threadIdx.x];
  a.dw[c0 + threadIdx.x] = s;
}

// Rows of more than 8192 values: dx a workgroup a row ...
template <typename TH, typename TY>
__global__ __launch_bounds__(512) void norm_bwd_wide_kernel(NormBwdArgs a) {
  __shared__ float slot[8];
  dx_row<TH, TY, 512>(a, blockIdx.x, slot);
}

// ... and dw column by column: workgroup (i, j) adds the rows j, j + gridDim.y,
// ... of 256 columns.
template <typename TH, typename TY>
__global__ __launch_bounds__(256) void norm_dweight_wide_kernel(NormBwdArgs a, float* part) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= a.d) return;
  float acc = 0.0f;
  for (int64_t r = blockIdx.y; r < a.rows; r += gridDim.y)
    acc = fmaf(widen(static_cast<const TY*>(a.dy)[r * a.dy_stride + c]),
               widen(static_cast<const TH*>(a.h)[r * a.h_stride + c]) * a.rstd[r], acc);
  part[static_cast<int64_t>(blockIdx.y) * a.d + c] = acc;
}

// The workgroups' parts added up: 32 columns a workgroup, 32 threads a column
__global__ __launch_bounds__(1024) void norm_dweight_sum_kernel(const float* part, int n, int64_t d, float* dw) {
  __shared__ float s[32][33];
  const int col = threadIdx.x & 31, lane = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + col;
  float acc = 0.0f;
  if (c < d) {
#pragma unroll 4
    for (int i = lane; i < n; i += 32) acc += part[static_cast<int64_t>(i) * d + c];
  }
  s[lane][col] = acc;
  __syncthreads();
  if (lane || c >= d) return;
  acc = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) acc += s[i][col];
  dw[c] = acc;
}


}  // namespace

// Threads a row.  Few rows are latency, which more threads shorten; a batch
// fills the chip with smaller workgroups.
hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  auto go = [&](auto x, auto res) {
    using TX = decltype(x);
    using TR = decltype(res);
    const dim3 grid(static_cast<unsigned>(a.rows));
    // one wavefront a short row, no barrier (8192 x 512: 8.1 us, 17 in four); a row
    // held in one group a thread while it fits (8192 x 2048: 23 us, 45 with four
    // groups); more rows than the chip takes at once in fewer, longer threads (7168
    // values by 1024 threads and by 256: 1 row 4.3 and 5.7 us, 512 rows 9.1 and 10.0,
    // 1024 rows 16.0 and 14.6, 8192 rows 107 and 82)
    if (a.d <= 512) hipLaunchKernelGGL((norm_kernel<TX, TR, 64, 1>), grid, dim3(64), 0, s, a);
    else if (a.d <= 2048) hipLaunchKernelGGL((norm_kernel<TX, TR, 256, 1>), grid, dim3(256), 0, s, a);
    else if (a.rows <= 512) hipLaunchKernelGGL((norm_kernel<TX, TR, 1024, 1>), grid, dim3(1024), 0, s, a);
    else hipLaunchKernelGGL((norm_kernel<TX, TR, 256, 4>), grid, dim3(256), 0, s, a);
  };
  auto with_res = [&](auto x) {
    if (!a.res) go(x, None{});
    else if (a.res_bf16) go(x, bf16_t{});
    else go(x, 0.0f);
  };
  a.x_bf16 ? with_res(bf16_t{}) : with_res(0.0f);
  return hipGetLastError();
}

constexpr int64_t kFewRows = 256;

// Workgroups that share the rows, each with a part of dw
int norm_bwd_parts(int64_t rows, int cus) { return rows <= kFewRows ? 0 : static_cast<int>(std::min<int64_t>(rows, 2 * cus)); }

hipError_t launch_norm_bwd(const NormBwdArgs& a, float* part, int cus, hipStream_t s) {
  const int parts = norm_bwd_parts(a.rows, cus);
  float* const pw = a.dw ? part : nullptr;
  auto go = [&](auto h, auto y) {
    using TH = decltype(h);
    using TY = decltype(y);
    const dim3 grid(static_cast<unsigned>(parts));
    if (a.rows <= kFewRows) {
      const unsigned rows = a.dx ? static_cast<unsigned>(a.rows) : 0, cols = a.dw ? static_cast<unsigned>((a.d + 63) / 64) : 0;
      auto few = [&](unsigned r, unsigned c) {
        hipLaunchKernelGGL((norm_bwd_few_kernel<TH, TY>), dim3(r + c), dim3(256), 0, s, a, static_cast<int>(r));
      };
      if (rows && cols && a.dx == a.dy) {   // dw first: dx takes dy's place
        few(0, cols);
        few(rows, 0);
      } else {
        few(rows, cols);
      }
      return;
    }
    // (as in the forward: 4099 x 512 9.8 us, 12.0 by 256 threads; x 2048 14.5 us, 27 with four groups)
    if (a.d <= 512) hipLaunchKernelGGL((norm_bwd_kernel<TH, TY, 64, 1>), grid, dim3(64), 0, s, a, pw);
    else if (a.d <= 2048) hipLaunchKernelGGL((norm_bwd_kernel<TH, TY, 256, 1>), grid, dim3(256), 0, s, a, pw);
    else if (a.d <= 8192) hipLaunchKernelGGL((norm_bwd_kernel<TH, TY, 256, 4>), grid, dim3(256), 0, s, a, pw);
    else {
      // dw first: dx may take dy's place
      if (pw)
        hipLaunchKernelGGL((norm_dweight_wide_kernel<TH, TY>),
                           dim3(static_cast<unsigned>((a.d + 255) / 256), static_cast<unsigned>(parts)), dim3(256), 0, s, a, pw);
      if (a.dx) hipLaunchKernelGGL((norm_bwd_wide_kernel<TH, TY>), dim3(static_cast<unsigned>(a.rows)), dim3(512), 0, s, a);
    }
  };
  auto with_y = [&](auto h) { a.dy_bf16 ? go(h, bf16_t{}) : go(h, 0.0f); };
  if (a.rows > 0) a.h_bf16 ? with_y(bf16_t{}) : with_y(0.0f);
  if (a.dw && (parts > 0 || a.rows == 0))
    hipLaunchKernelGGL(norm_dweight_sum_kernel, dim3(static_cast<unsigned>((a.d + 31) / 32)), dim3(1024), 0, s, part, parts, a.d, a.dw);
  return hipGetLastError();
}

}  // namespace stq
