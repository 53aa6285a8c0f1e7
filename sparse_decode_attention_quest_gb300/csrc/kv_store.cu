// Write of a ragged batch of new K/V rows into their slots of the paged cache,
// with the Quest page summaries kept up to date (SparseEngine: Sparse-First
// Inference Engine, Figure 3 caption: the summaries stay with the KV blocks).
//
// Token t goes to slot s_t = slot_map[t]: page s_t / 16, row s_t % 16 of every KV
// head; a negative slot is padding. A run is a maximal sequence of tokens next
// to each other whose slots lie in one page; the page's summary becomes
//     min over the run's keys, and over the old minimum unless slot 0 is in the run,
// and likewise the maximum.
//
// Bound by reading and writing every row once. A token's K and V rows are
// columns of 16 bytes; a warp takes 32 of them (512 bytes of a token's rows,
// read in one piece) and the runs that begin in its window of tokens, one
// run after another: a thread copies its column of the run's tokens, eight loads
// in flight, and holds the column's minimum and maximum in registers, so that
// nothing is exchanged between threads. What counts is bytes in flight: 80
// registers a thread (24 warps on an SM) without a spill carry 4 x 32K tokens of 8
// heads at 6.58 TB/s (168 us; 97% of the measured copy rate), 64 registers with
// 24 bytes spilled 183 us, and per-token row lookups in the loop 238 us.
// The window is 16 tokens, about a run of a prompt, for long batches, and shorter
// where there are fewer windows than warps, down to one token for a decode step,
// whose tokens lie in pages of their own.
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
  uint16_t* k;
  uint16_t* v;
  uint16_t* summary;
  int32_t num_pages, heads, dim, dim_v, row_k, row_v;
  const uint16_t* k_new;
  const uint16_t* v_new;  // not read when there are no V columns (latent cache)
  long long k_stride;     // elements between tokens
  long long v_stride;
  const int32_t* slot_map;
  int32_t num_tokens;
  int32_t k_cols;         // 16-byte columns of a token's K rows, of all its rows, and groups of 32 of them
  int32_t cols;
  int32_t col_groups;
  int32_t window;         // tokens whose runs a warp takes
  unsigned* err;
};

__global__ void __launch_bounds__(kWarps * 32, 3) store_kernel(const StoreArgs a) {
  pdl_enter();
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const long long win = w / a.col_groups;
  if (win * a.window >= a.num_tokens) return;
  const int t0 = (int)win * a.window, T = a.num_tokens;
  // Lane i holds the page of token t0 - 1 + i (-1: none) and its row.
  const int tl = t0 - 1 + lane;
  const int sl = tl >= 0 && tl < T ? a.slot_map[tl] : -1;
  int pg = sl < 0 ? -1 : sl / kPageSize;
  if (pg >= a.num_pages) {
    raise_error(a.err, SE_DEVERR_PAGE_RANGE);
    pg = -1;
  }
  const int prev = __shfl_up_sync(0xffffffffu, pg, 1);
  const bool begins = lane >= 1 && lane <= a.window && pg >= 0 && pg != prev;
  uint32_t runs = __ballot_sync(0xffffffffu, begins);

  const int col = (int)(w % a.col_groups) * 32 + lane;
  const bool on = col < a.cols, is_k = col < a.k_cols;
  const int c = is_k ? col : col - a.k_cols, width = is_k ? a.dim : a.dim_v;
  const int h = c / (width / 8), x0 = c % (width / 8) * 8;
  const long long src_stride = is_k ? a.k_stride : a.v_stride;
  const uint16_t* src = (is_k ? a.k_new : a.v_new) + c * 8;
  uint16_t* cache = is_k ? a.k : a.v;
  const int row_stride = is_k ? a.row_k : a.row_v;
  const bool sums = is_k && on && a.summary != nullptr;

  while (runs) {
    const int i0 = __ffs(runs) - 1;
    runs &= runs - 1;
    const int page = __shfl_sync(0xffffffffu, pg, i0);
    const size_t block = ((size_t)page * a.heads + h) * kPageSize;
    uint4 mn = make_uint4(0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u);  // +inf
    uint4 mx = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);  // -inf
    bool opened = false;
    // The run's length: as far as the lanes see it, and from memory behind them.
    const uint32_t same = __ballot_sync(0xffffffffu, pg == page) >> i0;
    const int seen = same == (0xffffffffu >> i0) ? 32 - i0 : __ffs(~same) - 1;
    const int first = t0 - 1 + i0, s0 = __shfl_sync(0xffffffffu, sl, i0);
    const uint32_t inrow = __ballot_sync(0xffffffffu, sl - s0 == lane - i0) >> i0;
    const uint16_t* from = src + (size_t)first * src_stride;
    int n = seen;
    if (i0 + seen == 32)
      while (first + n < T && a.slot_map[first + n] >= 0 && a.slot_map[first + n] / kPageSize == page) ++n;
    const bool ordered = n == seen && (inrow & ((1u << seen) - 1)) == (1u << seen) - 1;
    if (ordered) {
      // Rows one after another in the page, as a slot map built from lengths has them.
      const int r0 = s0 % kPageSize;
      opened = r0 == 0;
      uint16_t* to = cache + (block + r0) * row_stride + x0;
      if (on) {
        int k = 0;
        for (; k + 8 <= seen; k += 8) {
          uint4 x[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) x[u] = ld_stream_v4(reinterpret_cast<const uint4*>(from + u * src_stride));
          from += 8 * src_stride;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            *reinterpret_cast<uint4*>(to + u * row_stride) = x[u];
            mn = min_bf16x8(mn, x[u]);
            mx = max_bf16x8(mx, x[u]);
          }
          to += 8 * row_stride;
        }
        if (k < seen) {
          uint4 x[7];
#pragma unroll
          for (int u = 0; u < 7; ++u)
            if (k + u < seen) x[u] = ld_stream_v4(reinterpret_cast<const uint4*>(from + u * src_stride));
#pragma unroll
          for (int u = 0; u < 7; ++u)
            if (k + u < seen) {
              *reinterpret_cast<uint4*>(to + u * row_stride) = x[u];
              mn = min_bf16x8(mn, x[u]);
              mx = max_bf16x8(mx, x[u]);
            }
        }
      }
    } else {
      // Rows in any order, and a run of more tokens than a page has (slots named twice).
      for (int k = 0; k < n; ++k) {
        const int row = a.slot_map[first + k] % kPageSize;
        opened = opened || row == 0;
        if (!on) continue;
        const uint4 x = ld_stream_v4(reinterpret_cast<const uint4*>(from + (size_t)k * src_stride));
        *reinterpret_cast<uint4*>(cache + (block + row) * row_stride + x0) = x;
        mn = min_bf16x8(mn, x);
        mx = max_bf16x8(mx, x);
      }
    }
    if (sums) {
      uint4* lo = reinterpret_cast<uint4*>(a.summary + ((size_t)page * a.heads + h) * 2 * a.dim + x0);
      uint4* hi = lo + a.dim / 8;
      if (!opened) {
        mn = min_bf16x8(mn, *lo);
        mx = max_bf16x8(mx, *hi);
      }
      *lo = mn;
      *hi = mx;
    }
  }
}

}  // namespace

cudaError_t launch_kv_store(const KvView& kv, uint16_t* k_mut, uint16_t* v_mut, const uint16_t* k_new,
                            long long k_stride, const uint16_t* v_new, long long v_stride, const int32_t* slot_map,
                            int32_t num_tokens, int sm_count, unsigned* err, cudaStream_t stream) {
  StoreArgs a;
  a.k = k_mut;
  a.v = v_mut;
  a.summary = kv.summary;
  a.num_pages = kv.num_pages;
  a.heads = kv.num_kv_heads;
  a.dim = kv.head_dim;
  a.dim_v = kv.head_dim_v;
  a.row_k = kv.row_stride_k;
  a.row_v = kv.row_stride_v;
  a.k_new = k_new;
  a.v_new = v_new;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slot_map = slot_map;
  a.num_tokens = num_tokens;
  a.k_cols = kv.num_kv_heads * kv.head_dim / 8;
  a.cols = a.k_cols + (v_new ? kv.num_kv_heads * kv.head_dim_v / 8 : 0);
  a.col_groups = (a.cols + 31) / 32;
  a.err = err;
  // Windows of 16 tokens once they fill the SMs (32 warps each), shorter ones before.
  a.window = 16;
  while (a.window > 1 && (long long)num_tokens * a.col_groups < (long long)a.window * 32 * sm_count) a.window /= 2;
  const long long warps = (long long)((num_tokens + a.window - 1) / a.window) * a.col_groups;
  const cudaError_t e = launch_pdl(store_kernel, dim3((unsigned)((warps + kWarps - 1) / kWarps)), dim3(kWarps * 32),
                                   0, stream, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace se
