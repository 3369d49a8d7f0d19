// Passes over rows grouped by expert: every expert's rows are cut into passes
// of at most `max_tok`, and a workgroup finds the pass it has from the offsets
// on the device (the host does not know them).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

namespace stq {

// Most passes that total_m rows of n_experts can make: sum ceil(m_e / T) over
// k experts with rows is at most k + (total_m - k) / T, largest at the most
// experts that can have rows.
inline int64_t pass_units(int64_t total_m, int64_t n_experts, int64_t max_tok) {
  const int64_t k = n_experts < total_m ? n_experts : total_m;
  return k + (total_m - k) / max_tok;
}

// Experts that have rows, when `rows` rows choose among `experts` evenly.
inline double used_experts(double rows, double experts) { return experts * (1.0 - std::pow(1.0 - 1.0 / experts, rows)); }

// What a kernel of such passes takes for one step of its sum (a block, a
// tile), in us: a workgroup's step takes alone[0] + alone[1] t with a CU to
// itself and full[0] + full[1] t with `per_cu` on one, t the rows of a pass.
// A pass makes `slabs` workgroups; the rows' spread over the experts is the
// even one's (the host does not see the offsets).
struct PassCost {
  double per_cu, alone[2], full[2];
};
inline double pass_step_us(const PassCost& c, int64_t total_m, int64_t n_experts, int max_tok, int64_t slabs, int cus) {
  const double rows = static_cast<double>(total_m), used = used_experts(rows, static_cast<double>(n_experts));
  const double mean = rows / used, dev = std::sqrt(mean);
  auto cut = [&](double m) { return std::ceil(std::max(m, 1.0) / max_tok); };
  const double passes = used * (0.25 * cut(mean - dev) + 0.5 * cut(mean) + 0.25 * cut(mean + dev));
  const double tok = rows / passes;
  const double alone = c.alone[0] + c.alone[1] * tok, full = c.full[0] + c.full[1] * tok;
  const double load = passes * static_cast<double>(slabs) / cus;  // workgroups of a CU
  const double rounds = std::floor(load / c.per_cu), rest = load - rounds * c.per_cu;
  return rounds * full + (rest > 0.0 ? alone + (full - alone) * std::max(0.0, rest - 1.0) / (c.per_cu - 1.0) : 0.0);
}

struct PassUnit {
  int expert;
  int mt;        // rows of the pass; 0: there is no such pass
  int64_t row0;
};

// Pass `unit` counted over the experts in order, those with passes of more
// than `longer` rows first: a launch's last workgroups are then short ones
// (8191 uneven rows of 32 experts, one round of the chip: 142 to 150 us over
// four draws of the loads, 141 to 171 without).  An expert's rows are clamped
// to [0, total_m], so that offsets outside the contract reach no row that is
// not there, and its passes are of equal length.  Every wavefront does this
// for itself, 256 experts a step: a lane counts the passes of four experts,
// and a scan over the lanes finds the one that holds the unit.
__device__ __forceinline__ PassUnit find_pass(const int32_t* offsets, int n_experts, int64_t total_m, int unit,
                                              int max_tok, int longer) {
  const int lane = threadIdx.x & 63;
  int before = 0;  // passes of the experts ahead of this step's
  for (int first_class = 1; first_class >= 0; --first_class) {
    for (int e0 = 0; e0 < n_experts; e0 += 256) {
      int lo[5];
      const int e = e0 + 4 * lane;
#pragma unroll
      for (int i = 0; i < 5; ++i) lo[i] = offsets[min(e + i, n_experts)];
      int np[4], rows[4], sum = 0;
      int64_t first[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        first[i] = min(max(static_cast<int64_t>(lo[i]), int64_t{0}), total_m);
        const int64_t hi = min(max(static_cast<int64_t>(lo[i + 1]), first[i]), total_m);
        rows[i] = e + i < n_experts ? static_cast<int>(hi - first[i]) : 0;
        np[i] = (rows[i] + max_tok - 1) / max_tok;
        // rows > longer * np: its passes, of ceil(rows / np), are longer
        if ((rows[i] > static_cast<int64_t>(longer) * np[i]) != (first_class != 0)) np[i] = 0;
        sum += np[i];
      }
      int upto = sum;  // inclusive scan over the lanes
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(upto, o);
        if (lane >= o) upto += v;
      }
      const int want = unit - before;
      const uint64_t has = __ballot(upto > want);
      if (has) {
        const int src = __builtin_ctzll(has);
        int left = want - (upto - sum);  // meaningful in lane src
        int ei = 0, r = 0, n = 1;
        int64_t f = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (left >= 0 && left < np[i]) {
            ei = e + i;
            r = rows[i];
            n = np[i];
            f = first[i];
            break;
          }
          left -= np[i];
        }
        const int per = (r + n - 1) / n;
        const int base = left * per;
        PassUnit u;
        u.expert = __builtin_amdgcn_readfirstlane(__shfl(ei, src));
        u.mt = __builtin_amdgcn_readfirstlane(__shfl(max(0, min(per, r - base)), src));
        u.row0 = __builtin_amdgcn_readfirstlane(__shfl(static_cast<int>(f) + base, src));
        return u;
      }
      before += __shfl(upto, 63);
      if (before > (1 << 29)) break;  // offsets far outside the contract
    }
  }
  return PassUnit{0, 0, 0};
}

}  // namespace stq
