// What the dense paged decodes share: which pages and tokens of a request are
// kept, the prefix of the kept pages over a batch, and the list of items whose
// partials are joined.
#pragma once

#include "se_ptx.cuh"

namespace se {

// The kept pages of a request: logical pages 0 .. sink_pages - 1, then recent_page .. (all pages: sink_pages = n).
struct Kept {
  int len;   // tokens (clipped to the table)
  int from;  // kept: j < sink or j >= from
  int n;     // kept pages
  int sink_pages;
  int recent_page;
  __device__ __forceinline__ int logical(int i) const { return i < sink_pages ? i : i - sink_pages + recent_page; }
};

__device__ __forceinline__ Kept kept_of(int L, int bt_stride, int sink, int recent, unsigned* err) {
  Kept k;
  if (L < 0 || L > (long long)bt_stride * kPageSize) {
    raise_error(err, SE_DEVERR_LENGTH);
    L = L < 0 ? 0 : bt_stride * kPageSize;
  }
  k.len = L;
  const int pages = L / kPageSize + (L % kPageSize != 0);
  k.from = recent > 0 && L > recent ? L - recent : 0;
  const int sp = sink / kPageSize + (sink % kPageSize != 0), rp = k.from / kPageSize;
  if (k.from <= sink || sp > rp) {  // no page is left out
    k.n = k.sink_pages = pages;
    k.recent_page = pages;
    if (k.from <= sink) k.from = 0;
  } else {
    k.sink_pages = sp;
    k.recent_page = rp;
    k.n = sp + pages - rp;
  }
  return k;
}

// Which of a page's 16 tokens are kept: t < hi and (t < a or t >= z), packed as hi | a << 8 | z << 16.
__device__ __forceinline__ uint32_t page_mask(const Kept& k, int sink, int page) {
  const int j0 = page * kPageSize;
  const int hi = min(kPageSize, k.len - j0);
  const int a = k.from == 0 ? kPageSize : max(0, min(kPageSize, sink - j0));
  const int z = max(0, min(kPageSize, k.from - j0));
  return (uint32_t)hi | (uint32_t)a << 8 | (uint32_t)z << 16;
}
__device__ __forceinline__ bool in_mask(uint32_t m, int t) {
  return t < (int)(m & 0xff) && (t < (int)(m >> 8 & 0xff) || t >= (int)(m >> 16));
}
__device__ __forceinline__ bool mask_is_full(uint32_t m) {
  return (m & 0xff) == kPageSize && ((m >> 8 & 0xff) == kPageSize || (m >> 16) == 0);
}

// Kept pages per request as an exclusive prefix (prefix[batch]: the total), by the whole CTA. Positions are
// 32-bit: requests that end behind page `most` are reported and cut short. sums: kThreads / 32 values.
template <int kThreads>
__device__ __forceinline__ void kept_prefix(const int32_t* seq_lens, int batch, int bt_stride, int sink, int recent,
                                            int most, int* prefix, long long* sums, unsigned* err) {
  constexpr int kWarps = kThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long at = 0;
  for (int base = 0; base < batch; base += kThreads) {
    const int b = base + threadIdx.x;
    long long incl = b < batch ? kept_of(seq_lens[b], bt_stride, sink, recent, err).n : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    long long before = at, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sums[w];
      all += sums[w];
    }
    __syncthreads();
    incl += before;
    if (b < batch) {
      if (incl > most) raise_error(err, SE_DEVERR_LENGTH);
      prefix[b + 1] = (int)(incl < most ? incl : most);
    }
    at += all;
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  __syncthreads();
}

// The items to join, as (first CTA, item, partials), from joins[c] = (item, partials) of every CTA c (0 partials:
// none), in the order of their CTAs: every CTA of the join kernel makes the same list. By the whole CTA, which has
// a thread per entry; returns the number of items. counts: one value per warp.
__device__ __forceinline__ int list_joins(const int2* joins, int ctas, int3* todo, int* counts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int2 j = threadIdx.x < ctas ? joins[threadIdx.x] : make_int2(0, 0);
  const uint32_t some = __ballot_sync(0xffffffffu, j.y > 0);
  if (lane == 0) counts[warp] = __popc(some);
  __syncthreads();
  int at = __popc(some & ((1u << lane) - 1)), all = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) {
    at += w < warp ? counts[w] : 0;
    all += counts[w];
  }
  if (j.y > 0) todo[at] = make_int3(threadIdx.x, j.x, j.y);
  __syncthreads();
  return all;
}

// Warps that share the partials of an item: each takes eight or fewer, until all eight warps of a CTA share.
__device__ __forceinline__ int share_of(int partials) { return partials <= 8 ? 1 : partials <= 16 ? 2 : partials <= 32 ? 4 : 8; }

// The base of exponentials whose largest argument is m: 0 where nothing but -inf has been seen.
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.f : m; }

}  // namespace se
