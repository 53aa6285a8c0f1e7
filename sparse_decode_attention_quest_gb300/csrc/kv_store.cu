// Write of a ragged batch of new K/V rows into their slots of the paged cache,
// with the Quest page summaries kept up to date (SparseEngine: Sparse-First
// Inference Engine, Figure 3 caption: the summaries stay with the KV blocks).
//
// Token t goes to slot s_t = slot_map[t]: page s_t / 16, row s_t % 16 of every KV
// head; a negative slot is padding. A run is a maximal sequence of tokens next
// to each other whose slots lie in one page; the page's summary becomes
//     min over the run's keys, and over the old minimum unless slot 0 is in the run,
// and likewise the maximum. One warp per (token, KV head): the warp of a run's
// first token copies the run's rows in order and sums up their bounds, the
// others leave at once. Bound by reading and writing every row once.
#include "se_ptx.cuh"

namespace se {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmin2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint4 min_bf16x8(uint4 a, uint4 b) {
  return make_uint4(min_bf16x2(a.x, b.x), min_bf16x2(a.y, b.y), min_bf16x2(a.z, b.z), min_bf16x2(a.w, b.w));
}
__device__ __forceinline__ uint4 max_bf16x8(uint4 a, uint4 b) {
  return make_uint4(max_bf16x2(a.x, b.x), max_bf16x2(a.y, b.y), max_bf16x2(a.z, b.z), max_bf16x2(a.w, b.w));
}

struct StoreArgs {
  KvView kv;
  uint16_t* k;
  uint16_t* v;
  const uint16_t* k_new;
  const uint16_t* v_new;  // NULL: latent cache
  long long k_stride;     // elements between tokens
  long long v_stride;
  const int32_t* slot_map;
  int32_t num_tokens;
  unsigned* err;
};

__global__ void __launch_bounds__(kWarps * 32) store_kernel(const StoreArgs a) {
  pdl_enter();
  const int H = a.kv.num_kv_heads;
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= (long long)a.num_tokens * H) return;
  const int t0 = (int)(w / H), h = (int)(w % H);
  const int s0 = a.slot_map[t0];
  if (s0 < 0) return;
  const int page = s0 / kPageSize;
  if (page >= a.kv.num_pages) {
    if (lane == 0) raise_error(a.err, SE_DEVERR_PAGE_RANGE);
    return;
  }
  const bool sums = a.kv.summary != nullptr;
  if (sums && t0 > 0) {
    const int prev = a.slot_map[t0 - 1];
    if (prev >= 0 && prev / kPageSize == page) return;  // inside a run
  }
  const int D = a.kv.head_dim, Dv = a.kv.head_dim_v;
  const size_t blk = (size_t)page * H + h;
  const uint32_t pinf = 0x7f807f80u, ninf = 0xff80ff80u;
  for (int c = lane; c < D / 8; c += 32) {
    uint4 mn = make_uint4(pinf, pinf, pinf, pinf), mx = make_uint4(ninf, ninf, ninf, ninf);
    bool opened = false;
    for (int t = t0; t < a.num_tokens; ++t) {
      const int s = a.slot_map[t];
      if (s < 0 || s / kPageSize != page || (!sums && t > t0)) break;
      const uint4 x = *reinterpret_cast<const uint4*>(a.k_new + (size_t)t * a.k_stride + (size_t)h * D + c * 8);
      *reinterpret_cast<uint4*>(a.k + (blk * kPageSize + s % kPageSize) * a.kv.row_stride_k + c * 8) = x;
      mn = min_bf16x8(mn, x);
      mx = max_bf16x8(mx, x);
      opened = opened || s % kPageSize == 0;
    }
    if (sums) {
      uint4* lo = reinterpret_cast<uint4*>(a.kv.summary + blk * 2 * D) + c;
      uint4* hi = lo + D / 8;
      if (!opened) {
        mn = min_bf16x8(mn, *lo);
        mx = max_bf16x8(mx, *hi);
      }
      *lo = mn;
      *hi = mx;
    }
  }
  if (a.v_new == nullptr) return;
  for (int t = t0; t < a.num_tokens; ++t) {
    const int s = a.slot_map[t];
    if (s < 0 || s / kPageSize != page || (!sums && t > t0)) break;
    for (int c = lane; c < Dv / 8; c += 32)
      *reinterpret_cast<uint4*>(a.v + (blk * kPageSize + s % kPageSize) * a.kv.row_stride_v + c * 8) =
          *reinterpret_cast<const uint4*>(a.v_new + (size_t)t * a.v_stride + (size_t)h * Dv + c * 8);
  }
}

}  // namespace

cudaError_t launch_kv_store(const KvView& kv, uint16_t* k_mut, uint16_t* v_mut, const uint16_t* k_new,
                            long long k_stride, const uint16_t* v_new, long long v_stride, const int32_t* slot_map,
                            int32_t num_tokens, unsigned* err, cudaStream_t stream) {
  StoreArgs a;
  a.kv = kv;
  a.k = k_mut;
  a.v = v_mut;
  a.k_new = k_new;
  a.v_new = v_new;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slot_map = slot_map;
  a.num_tokens = num_tokens;
  a.err = err;
  const long long warps = (long long)num_tokens * kv.num_kv_heads;
  const cudaError_t e = launch_pdl(store_kernel, dim3((unsigned)((warps + kWarps - 1) / kWarps)), dim3(kWarps * 32),
                                   0, stream, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace se
