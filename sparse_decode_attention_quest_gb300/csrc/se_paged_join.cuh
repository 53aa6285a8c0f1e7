// How the partials of the dense paged decodes over separate K and V are joined, in the
// decode kernel or in one of its own, and the order of states staged in shared memory.
#pragma once

#include "se_paged.cuh"

namespace se {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kJoinWarps = 8;

// Where a state staged in shared memory keeps (head, dim): the dims of a row of D, turned by eight per pair of
// heads, so that the accumulators' lanes (four head pairs, eight dims) write to 32 banks.
template <int kD>
__device__ __forceinline__ int stage_at(int head, int dim) {
  return head * kD + (dim ^ (((head >> 1) & 3) << 3));
}

// Joins the partials of `parts` CTAs (first .. first + parts - 1) for the rows r0 .. of an item, by kW warps: a
// warp per row, or `share` of them when a row has many partials, joined in their order. With M the largest
// log-sum-exp of a row,
//     out = sum_i exp2(lse_i - M) o_i / sum_i exp2(lse_i - M).
// kBatch: partials in flight (a power of two). kLean: quotients and logarithms by the hardware approximations, which
// take less code: what a CTA runs once costs it the fetching of its instructions. kDown: weights and their sum are held
// 2^kDown lower (exact, but for weights below 2^-118), so that the sum of so many partials near fp32's largest is finite.
template <int kD, int kW>
struct JoinSmem {
  float acc[kW][kD];
  float m[kW], l[kW];
};
template <int kD, int kW, int kBatch, bool kLean, int kDown, typename Sync>
__device__ __forceinline__ void join_rows(const float* o_part, const float* lse_part, int first, int parts, int item,
                                          int rows, int r0, int share, JoinSmem<kD, kW>& sm, uint16_t* out,
                                          float* out_lse, Sync sync) {
  constexpr int kV = kD / 32;  // values per lane
  constexpr float kUp = 1 << kDown;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = min(r0 + warp / share, rows - 1), sub = warp % share;
  // Partial i is in slot 1 of the item's first CTA (i = 0), in slot 0 of the others. Other CTAs wrote it: past L1.
  auto part = [&](int i) { return (size_t)(2 * (first + i) + (i == 0)) * rows + r; };
  const int n = (parts - sub + share - 1) / share;
  float M = -INFINITY, l = 0.f, acc[kV];
#pragma unroll
  for (int x = 0; x < kV; ++x) acc[x] = 0.f;
  // Batches of partials, their loads in flight beside those of their log-sum-exps.
  for (int k0 = 0; k0 < n; k0 += kBatch) {
    float v[kBatch][kV];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (k0 + k >= n) continue;
      const float* p = o_part + part(sub + share * (k0 + k)) * kD + lane * kV;
      if constexpr (kV == 2) {
        const float2 t = __ldcg(reinterpret_cast<const float2*>(p));
        v[k][0] = t.x;
        v[k][1] = t.y;
      } else {
#pragma unroll
        for (int x = 0; x < kV; x += 4) {
          const float4 t = __ldcg(reinterpret_cast<const float4*>(p + x));
          v[k][x] = t.x;
          v[k][x + 1] = t.y;
          v[k][x + 2] = t.z;
          v[k][x + 3] = t.w;
        }
      }
    }
    const int mine = sub + share * (k0 + lane);
    const float ls = lane < kBatch && mine < parts ? __ldcg(lse_part + part(mine)) : -INFINITY;
    float top = ls;
#pragma unroll
    for (int o = kBatch / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = fmaxf(M, __shfl_sync(0xffffffffu, top, 0));
    const float base = finite_base(top), f0 = fast_exp2(M - base), w = fast_exp2(ls - base) * (1.f / kUp);
    M = top;
    l *= f0;
#pragma unroll
    for (int x = 0; x < kV; ++x) acc[x] *= f0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (k0 + k >= n) continue;
      const float f = __shfl_sync(0xffffffffu, w, k);
      l += f;
#pragma unroll
      for (int x = 0; x < kV; ++x) acc[x] += f * v[k][x];
    }
  }
  if (share == 1) {
    if (r0 + warp >= rows) return;
    const size_t orow = (size_t)item * rows + r;
    const bool none = l == 0.f;
    const float inv = kLean ? fast_rcp(l) : 1.f / l, log_l = kLean ? fast_log2(l * kUp) : log2f(l * kUp);
#pragma unroll
    for (int x = 0; x < kV; x += 2)
      *reinterpret_cast<uint32_t*>(out + orow * kD + lane * kV + x) =
          none ? 0u : pack_bf16x2(acc[x] * inv, acc[x + 1] * inv);
    if (out_lse && lane == 0) out_lse[orow] = none ? -INFINITY : (M + log_l) * kLn2;
    return;
  }
  sync();  // the previous rows' sums are read
#pragma unroll
  for (int x = 0; x < kV; ++x) sm.acc[warp][lane * kV + x] = acc[x];
  if (lane == 0) {
    sm.m[warp] = M;
    sm.l[warp] = l;
  }
  sync();
  // The rows' values, in pairs.
  for (int e = threadIdx.x; e < kW / share * (kD / 2); e += kW * 32) {
    const int w0 = e / (kD / 2) * share, d = e % (kD / 2) * 2, row = r0 + e / (kD / 2);
    if (row >= rows) continue;
    float top = -INFINITY;
    for (int k = 0; k < share; ++k) top = fmaxf(top, sm.m[w0 + k]);
    const float base = finite_base(top);
    float sum = 0.f, x = 0.f, y = 0.f;
    for (int k = 0; k < share; ++k) {
      const float f = fast_exp2(sm.m[w0 + k] - base);
      sum += f * sm.l[w0 + k];
      x += f * sm.acc[w0 + k][d];
      y += f * sm.acc[w0 + k][d + 1];
    }
    const size_t orow = (size_t)item * rows + row;
    const bool none = sum == 0.f;
    const float inv = kLean ? fast_rcp(sum) : 1.f / sum, log_l = kLean ? fast_log2(sum * kUp) : log2f(sum * kUp);
    *reinterpret_cast<uint32_t*>(out + orow * kD + d) = none ? 0u : pack_bf16x2(x * inv, y * inv);
    if (out_lse && d == 0) out_lse[orow] = none ? -INFINITY : (top + log_l) * kLn2;
  }
}

// The join of the items that span many CTAs, a CTA per few rows of an item.
template <int kD, int kDown>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const float* __restrict__ o_part,
                                                                    const float* __restrict__ lse_part,
                                                                    const int2* __restrict__ joins, int32_t ctas,
                                                                    int32_t rows, uint16_t* __restrict__ out,
                                                                    float* __restrict__ out_lse) {
  pdl_enter();
  static_assert(kMaxCtas <= kJoinWarps * 32, "a thread per item");
  __shared__ int4 todo[kMaxCtas];
  __shared__ int2 counts[kJoinWarps];
  __shared__ JoinSmem<kD, kJoinWarps> sm;
  const int2 n = list_joins(joins, ctas, rows, todo, counts);
  for (int u = blockIdx.x; u < n.y; u += gridDim.x) {
    const int4 j = join_of(todo, n.x, u);
    const int share = share_of(j.z);
    join_rows<kD, kJoinWarps, 8, false, kDown>(o_part, lse_part, j.x, j.z, j.y, rows,
                                               (u - j.w) * (kJoinWarps / share), share, sm, out, out_lse,
                                               [] { __syncthreads(); });
  }
}

}  // namespace
}  // namespace se
