// A token's expert rows added up with its weights, and the gradients of that:
//
//     y[t] = sum_j w[t, j] z[row(t, j)]
//     dz[row(t, j)] = w[t, j] dy[t]        dw[t, j] = <dy[t], z[row(t, j)]>
//
// row(t, j) < 0 (or outside z) is a pair without a row: it adds nothing, its
// dw is 0.  Sums run over j in order, in fp32: no atomics, the same bits every
// time.
#include <algorithm>
#include <type_traits>

#include "stq_launch.hpp"
#include "stq_rows.hpp"

namespace stq {
namespace {

constexpr int kBatch = 8;  // rows of a token in flight

// Workgroup: one token, blockDim.x * 8 columns.  HBM bounds it: 2048 tokens of 8
// fp32 rows of 7168, 105 us for 529 MB, 5.0 TB/s.
// Rows of whole chunks have a kernel without the others' ends (105 us against
// 107 to 108).
template <typename TZ, typename TY, bool kWhole>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a, int col_blocks) {
  const int64_t t = blockIdx.x / col_blocks;
  const int64_t c = (static_cast<int64_t>(blockIdx.x % col_blocks) * blockDim.x + threadIdx.x) * 8;
  if (c >= a.d) return;
  const TZ* z = static_cast<const TZ*>(a.z);
  const int32_t* rows = a.pair_row + t * a.top_k;
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = 0.0f;
  for (int j0 = 0; j0 < a.top_k; j0 += kBatch) {
    Raw8<TZ> raw[kBatch];
    float w[kBatch];
    int32_t row[kBatch];
    bool on[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int jj = min(j0 + j, a.top_k - 1);
      row[j] = rows[jj];
      on[j] = j0 + j < a.top_k && row[j] >= 0 && row[j] < a.n_rows;
      w[j] = a.weight ? a.weight[t * a.top_k + jj] : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (on[j]) raw[j] = load8<TZ, kWhole>(z + row[j] * a.z_stride, c, a.d);
    if (!kWhole && c + 8 > a.d) {   // (one branch for all of them)
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (on[j]) settle8<TZ>(raw[j], c, a.d);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (!on[j]) continue;
      float v[8];
      unpack8<TZ>(raw[j], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf(w[j], v[e], y[e]);
    }
  }
  store8<TY>(static_cast<TY*>(a.y) + t * a.y_stride, c, a.d, pack8<TY>(y));
}

// Workgroup: one token; its rows in batches of kBatch, dy read again for each
// batch (from cache).  HBM bounds it: 1021 tokens of 8 fp32 rows of 4096, dz in
// bf16, 40 us for 204 MB, 5.1 TB/s.
template <typename TY, typename TZ, typename TD, int kThreads>
__global__ __launch_bounds__(kThreads) void combine_bwd_kernel(CombineBwdArgs a) {
  __shared__ float part[kThreads / 64][kBatch];
  const int64_t t = blockIdx.x;
  const TY* dy = static_cast<const TY*>(a.dy) + t * a.dy_stride;
  const TZ* z = static_cast<const TZ*>(a.z);
  TD* dz = static_cast<TD*>(a.dz);
  for (int j0 = 0; j0 < a.top_k; j0 += kBatch) {
    const int n = min(kBatch, a.top_k - j0);
    int64_t row[kBatch];
    float w[kBatch], dot[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int64_t p = t * a.top_k + j0 + min(j, n - 1);
      const int32_t rr = a.pair_row[p];
      row[j] = j < n && rr >= 0 && rr < a.n_rows ? rr : -1;
      w[j] = a.weight ? a.weight[p] : 1.0f;
      dot[j] = 0.0f;
    }
    for (int64_t c = threadIdx.x * 8; c < a.d; c += kThreads * 8) {
      float g[8];
      Raw8<TZ> raw[kBatch];
      Raw8<TY> ry = load8<TY>(dy, c, a.d);
      if (a.dw) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (row[j] >= 0) raw[j] = load8<TZ>(z + row[j] * a.z_stride, c, a.d);
      }
      settle8<TY>(ry, c, a.d);
      unpack8<TY>(ry, g);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (row[j] < 0) continue;
        if (a.dw) {
          float v[8];
          settle8<TZ>(raw[j], c, a.d);
          unpack8<TZ>(raw[j], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) dot[j] = fmaf(g[e], v[e], dot[j]);
        }
        if (a.dz) {
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = w[j] * g[e];
          store8<TD>(dz + row[j] * a.dz_stride, c, a.d, pack8<TD>(o));
        }
      }
    }
    if (a.dw) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const float s = sum64(dot[j]);
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][j] = s;
      }
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < n) {
        float s = part[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < kThreads / 64; ++i) s += part[i][threadIdx.x];
        a.dw[t * a.top_k + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}


// One wavefront a short row (its gradient for 2048 x 8 x 512: 16 us, 27 in four)
int combine_threads(int64_t d) { return d <= 512 ? 64 : 256; }

}  // namespace

int64_t combine_col_blocks(int64_t d) {
  const int64_t per = combine_threads(d) * 8;
  return (d + per - 1) / per;
}

hipError_t launch_combine_rows(const CombineArgs& a, hipStream_t s) {
  const int64_t cb = combine_col_blocks(a.d);
  auto go = [&](auto z, auto y) {
    const dim3 grid(static_cast<unsigned>(a.tokens * cb)), block(combine_threads(a.d));
    if (a.d % 8 == 0) hipLaunchKernelGGL((combine_kernel<decltype(z), decltype(y), true>), grid, block, 0, s, a, static_cast<int>(cb));
    else hipLaunchKernelGGL((combine_kernel<decltype(z), decltype(y), false>), grid, block, 0, s, a, static_cast<int>(cb));
  };
  auto with_y = [&](auto z) { a.y_bf16 ? go(z, bf16_t{}) : go(z, 0.0f); };
  a.z_bf16 ? with_y(bf16_t{}) : with_y(0.0f);
  return hipGetLastError();
}

hipError_t launch_combine_rows_bwd(const CombineBwdArgs& a, hipStream_t s) {
  auto go = [&](auto y, auto z, auto dz) {
    const dim3 grid(static_cast<unsigned>(a.tokens));
    if (a.d <= 512) hipLaunchKernelGGL((combine_bwd_kernel<decltype(y), decltype(z), decltype(dz), 64>), grid, dim3(64), 0, s, a);
    else hipLaunchKernelGGL((combine_bwd_kernel<decltype(y), decltype(z), decltype(dz), 256>), grid, dim3(256), 0, s, a);
  };
  auto with_dz = [&](auto y, auto z) { a.dz_bf16 ? go(y, z, bf16_t{}) : go(y, z, 0.0f); };
  auto with_z = [&](auto y) { a.z_bf16 ? with_dz(y, bf16_t{}) : with_dz(y, 0.0f); };
  a.dy_bf16 ? with_z(bf16_t{}) : with_z(0.0f);
  return hipGetLastError();
}

}  // namespace stq
