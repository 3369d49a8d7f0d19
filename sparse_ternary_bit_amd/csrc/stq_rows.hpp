// Device-side helpers of the row operators: rows of fp32 or bf16 elements read
// and written eight at a time, and reductions inside a wavefront.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace stq {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

struct bf16_t {
  uint16_t bits;
};

__device__ __forceinline__ uint32_t bf16_round(float f) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(bf16_t v) { return __builtin_bit_cast(float, static_cast<uint32_t>(v.bits) << 16); }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16_t narrow<bf16_t>(float v) { return bf16_t{static_cast<uint16_t>(bf16_round(v))}; }

// Eight elements as they lie in memory
template <typename T>
struct Raw8 {
  static constexpr int kW = sizeof(T) / 2;  // 16-byte words
  u32x4_t w[kW];
};

// Sixteen bytes where elements lie, on any element's boundary: the memory takes
// such accesses as they are, and rows of odd length cost little more than
// aligned ones (783 rows of 6135: 44 us element by element).
struct __attribute__((packed, aligned(2))) Words16 {
  u32x4_t v;
};
struct __attribute__((packed, aligned(2))) Words8 {
  u32x2_t v;
};
__device__ __forceinline__ u32x4_t load16b(const void* p) { return static_cast<const Words16*>(p)->v; }
__device__ __forceinline__ void store16b(void* p, u32x4_t v) { static_cast<Words16*>(p)->v = v; }

// Elements c..c+7 of a row of n, as they are after settle8 below: where the row
// ends inside them, its last eight are read, and settle8 moves them into place.
// Two steps, so that every load of a batch is on its way before the first value
// is looked at (element by element the last columns were a chain of up to seven
// loads: gradients of 237 rows of 878 27 us).
// kWhole: n is a multiple of 8, and nothing is to settle.
template <typename T, bool kWhole = false>
__device__ __forceinline__ Raw8<T> load8(const T* row, int64_t c, int64_t n) {
  Raw8<T> r;
  if (kWhole || n >= 8) {
    const char* const at = reinterpret_cast<const char*>(row + min(c, n - 8));
#pragma unroll
    for (int i = 0; i < Raw8<T>::kW; ++i) r.w[i] = load16b(at + 16 * i);
  } else {
#pragma unroll
    for (int i = 0; i < Raw8<T>::kW; ++i) r.w[i] = u32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c + i >= n) continue;
      if constexpr (sizeof(T) == 4) r.w[i >> 2][i & 3] = __builtin_bit_cast(uint32_t, row[c + i]);
      else r.w[0][i >> 1] |= static_cast<uint32_t>(row[c + i].bits) << (16 * (i & 1));
    }
    // looked at here: nothing of this path is under way where the two meet, or
    // every load of the other would wait for it
#pragma unroll
    for (int i = 0; i < Raw8<T>::kW; ++i) asm("" : "+v"(r.w[i]));
  }
  return r;
}

// load8's elements in their places; columns past n become 0
template <typename T>
__device__ __forceinline__ void settle8(Raw8<T>& r, int64_t c, int64_t n) {
  if (n < 8 || c + 8 <= n) return;
  constexpr int kWords = 4 * Raw8<T>::kW;
  const int over = static_cast<int>(min(c + 8 - n, int64_t{8}));
  uint32_t w[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) w[i] = r.w[i >> 2][i & 3];
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __builtin_amdgcn_alignbit(i + 1 < kWords ? w[i + 1] : 0u, w[i], (over & 1) * 16);
  }
  const int words = sizeof(T) == 2 ? over >> 1 : over;
#pragma unroll
  for (int by = 1; by <= kWords; by *= 2)
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = words & by ? (i + by < kWords ? w[i + by] : 0u) : w[i];
#pragma unroll
  for (int i = 0; i < kWords; ++i) r.w[i >> 2][i & 3] = w[i];
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) v[i] = __builtin_bit_cast(float, static_cast<uint32_t>(r.w[i >> 2][i & 3]));
    else v[i] = __builtin_bit_cast(float, (i & 1) ? (r.w[0][i >> 1] & 0xFFFF0000u) : (r.w[0][i >> 1] << 16));
  }
}

template <typename T>
__device__ __forceinline__ void load8f(const T* row, int64_t c, int64_t n, float (&v)[8]) {
  Raw8<T> r = load8<T>(row, c, n);
  settle8<T>(r, c, n);
  unpack8<T>(r, v);
}

template <typename T>
__device__ __forceinline__ Raw8<T> pack8(const float (&v)[8]) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) r.w[i >> 2][i & 3] = __builtin_bit_cast(uint32_t, v[i]);
    else if ((i & 1) == 0) r.w[0][i >> 1] = bf16_round(v[i]) | bf16_round(v[i + 1]) << 16;
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void store8(T* row, int64_t c, int64_t n, const Raw8<T>& r) {
  if (c + 8 <= n) {
#pragma unroll
    for (int i = 0; i < Raw8<T>::kW; ++i) store16b(reinterpret_cast<char*>(row + c) + 16 * i, r.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c + i >= n) continue;
      if constexpr (sizeof(T) == 4) row[c + i] = __builtin_bit_cast(float, static_cast<uint32_t>(r.w[i >> 2][i & 3]));
      else row[c + i] = bf16_t{static_cast<uint16_t>(r.w[0][i >> 1] >> (16 * (i & 1)))};
    }
  }
}

// Reductions by DPP moves.  Inside 16 lanes by rotation: every lane gets the
// result, and the same bits, because each step adds the two halves of a set
// that both partners then hold.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), kCtrl, 0xF, 0xF, false));
}
template <int kCtrl>
__device__ __forceinline__ float dpp_move(float v) {
  return __builtin_bit_cast(float, dpp_move<kCtrl>(__builtin_bit_cast(uint32_t, v)));
}
template <typename T, typename F>
__device__ __forceinline__ T reduce16(T v, F f) {
  v = f(v, dpp_move<0x128>(v));  // row_ror:8, 4, 2, 1
  v = f(v, dpp_move<0x124>(v));
  v = f(v, dpp_move<0x122>(v));
  v = f(v, dpp_move<0x121>(v));
  return v;
}
template <typename T, typename F>
__device__ __forceinline__ T reduce64(T v, F f) {
  v = reduce16(v, f);
  v = f(v, __shfl_xor(v, 16));
  return f(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum16(float v) {
  return reduce16(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float sum64(float v) {
  return reduce64(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ uint32_t max64(uint32_t v) {
  return reduce64(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}

}  // namespace stq
