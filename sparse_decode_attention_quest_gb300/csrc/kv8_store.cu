// Write of a ragged batch of new K/V rows into an 8-bit paged cache, and rows of it
// read back.
//
// A page's 16 rows of one KV head share a scale s, a power of two with
// max |x| <= 448 s, and are held as e4m3 codes of x / s. e4m3 is a floating-point
// format: a power of two costs it no relative precision (half a step of 2^-4 from
// 2^-6 s on), and moving a page to a larger scale is exact but for the values that
// fall below that. A page begun earlier therefore takes later rows by
//     s' = max(s, need of the new rows),  c' = rne(c s / s')  where s' > s.
//
// Store: bound by reading 2 bytes and writing 1 of every value. A warp takes the runs
// (tokens next to each other whose slots lie in one page) that begin in its window of
// tokens, for one KV head of K or V or for several next to each other, 256 dims in all
// where the number of heads allows: it holds a run's rows in registers (256 dims wide,
// a row a load: sixteen 16-byte loads in flight per lane; 128 wide, two rows a load: eight),
// folds their magnitudes, exchanges them between the lanes of a head and of its other
// rows (three shuffles for four heads of 64 dims, four for two of 128, otherwise five or,
// for two of 64, four), and writes the codes, 8 bytes a lane. Windows as in the bf16
// store: 16 tokens for long batches, shorter ones down to one token where there are
// fewer windows than warps.
//
// Load: bound by reading 1 byte and writing 2. A CTA looks its window of rows up once
// (request by bisection, page from the table), then its warps take pieces of 16 codes.
#include "se_kv8.cuh"

namespace se {
namespace {

constexpr int kWarps = 8;
constexpr int kLoadThreads = 256;
constexpr int kMaxWindow = 64;  // rows of a load CTA

struct Kv8StoreArgs {
  Kv8View kv;
  const uint16_t* in[2];
  long long stride[2];  // elements between tokens
  const int32_t* slot_map;
  int32_t num_tokens;
  int32_t window;       // tokens whose runs a warp takes
  unsigned* err;
};

// Eight values times inv (at most 448, or NaN) as codes.
__device__ __forceinline__ uint2 quantise8(uint4 x, float inv) {
  return make_uint2(to_e4m3x4(bf16_lo(x.x) * inv, bf16_hi(x.x) * inv, bf16_lo(x.y) * inv, bf16_hi(x.y) * inv),
                    to_e4m3x4(bf16_lo(x.z) * inv, bf16_hi(x.z) * inv, bf16_lo(x.w) * inv, bf16_hi(x.w) * inv));
}
// Four codes moved to another scale.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  float f[4];
  from_e4m3x4(w, f);
  return to_e4m3x4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
}

// Eight values with NaN for infinities, which the conversion alone would take to 448.
__device__ __forceinline__ uint4 without_inf(uint4 x) {
  return make_uint4(x.x | not_finite_bf16x2(x.x), x.y | not_finite_bf16x2(x.y), x.z | not_finite_bf16x2(x.z),
                    x.w | not_finite_bf16x2(x.w));
}

// How a warp takes rows of kD dims, 8 dims a lane: those of kHeads KV heads next to each other as one.
template <int kD, int kHeads>
struct Lanes {
  static constexpr int kOfHead = kD / 8;            // lanes of a head's row
  static constexpr int kOfRow = kHeads * kOfHead;   // and of a row
  static constexpr int kRows = 32 / kOfRow;         // rows of a warp's load
  // Over the lanes of a head.
  static __device__ __forceinline__ uint32_t max_abs(uint32_t m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < kOfHead || o >= kOfRow) m = max_abs_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
    return max(m & 0xffffu, m >> 16);
  }
};

// A run of n tokens of one page, by a warp: a lane's columns of the page and of the first token's row.
template <int kD, int kHeads>
struct Run {
  uint8_t* rows;
  const uint16_t* from;
  long long stride;
  float* scale;
  int n, sub, lane;
  bool on;  // the lane has a head

  // The page's scale for rows whose largest magnitudes the lanes hold, and which slots they take (old: its present one,
  // where slot 0 is not among them); the other slots' codes follow. Returns its reciprocal; loud: a lane has infinities.
  __device__ __forceinline__ float take_scale(uint32_t amax, uint32_t written, float old, bool& loud) const {
    using L = Lanes<kD, kHeads>;
    uint32_t top = L::max_abs(amax);
    loud = __any_sync(0xffffffffu, top >= 0x7f80u);
    if (loud) {
      // The largest finite magnitudes instead.
      uint32_t m = 0;
      for (int k = sub; k < n && on; k += L::kRows) {
        const uint4 y = ld_stream_v4(reinterpret_cast<const uint4*>(from + k * stride));
        m = max_abs_bf16x8(m, make_uint4(y.x & ~not_finite_bf16x2(y.x), y.y & ~not_finite_bf16x2(y.y),
                                         y.z & ~not_finite_bf16x2(y.z), y.w & ~not_finite_bf16x2(y.w)));
      }
      __syncwarp();
      top = L::max_abs(m);
    }
    float s = scale_for(top);
    const bool opened = written & 1u;
    if (!opened) s = fmaxf(s, old);
    if (on && !opened && s != old) {
      const float ratio = old / s;
      for (int r = sub; r < kPageSize; r += L::kRows) {
        if (written >> r & 1u) continue;
        uint2* c = reinterpret_cast<uint2*>(rows + r * kD);
        *c = make_uint2(rescale4(c->x, ratio), rescale4(c->y, ratio));
      }
    }
    __syncwarp();  // every lane has the present scale
    if (on && lane % L::kOfHead == 0 && sub == 0 && (opened || s != old)) *scale = s;
    return 1.f / s;
  }
};

template <int kD, int kHeads>
__global__ void __launch_bounds__(kWarps * 32, kD * kHeads == 256 ? 2 : 3) kv8_store_kernel(const Kv8StoreArgs a) {
  using L = Lanes<kD, kHeads>;
  constexpr int kRows = L::kRows, kLoads = kPageSize / kRows;
  pdl_enter();
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, sub = lane / L::kOfRow, x0 = lane % L::kOfHead * 8;
  const int groups = 2 * ((a.kv.num_kv_heads + kHeads - 1) / kHeads);
  const long long win = w / groups;
  if (win * a.window >= a.num_tokens) return;
  const int t0 = (int)win * a.window, T = a.num_tokens;
  // Lane i holds the page of token t0 - 1 + i (-1: none).
  const int tl = t0 - 1 + lane;
  const int sl = tl >= 0 && tl < T ? a.slot_map[tl] : -1;
  int pg = sl < 0 ? -1 : sl / kPageSize;
  if (pg >= a.kv.num_pages) {
    raise_error(a.err, SE_DEVERR_PAGE_RANGE);
    pg = -1;
  }
  const int prev = __shfl_up_sync(0xffffffffu, pg, 1);
  uint32_t runs = __ballot_sync(0xffffffffu, lane >= 1 && lane <= a.window && pg >= 0 && pg != prev);

  const int cg = (int)(w % groups), is_v = cg & 1, mine = (cg >> 1) * kHeads + lane % L::kOfRow / L::kOfHead;
  const bool on = mine < a.kv.num_kv_heads;
  const int h = on ? mine : a.kv.num_kv_heads - 1;
  const uint16_t* src = (is_v ? a.in[1] : a.in[0]) + (long long)h * kD + x0;
  const long long stride = is_v ? a.stride[1] : a.stride[0];
  uint8_t* cache = is_v ? a.kv.v : a.kv.k;
  float* scales = is_v ? a.kv.v_scale : a.kv.k_scale;

  while (runs) {
    const int i0 = __ffs(runs) - 1;
    runs &= runs - 1;
    const int page = __shfl_sync(0xffffffffu, pg, i0);
    const size_t block = (size_t)page * a.kv.num_kv_heads + h;
    uint8_t* rows = cache + block * kPageSize * kD + x0;
    // The run's length: as far as the lanes see it, and from memory behind them.
    const uint32_t same = __ballot_sync(0xffffffffu, pg == page) >> i0;
    const int seen = same == (0xffffffffu >> i0) ? 32 - i0 : __ffs(~same) - 1;
    const int first = t0 - 1 + i0, s0 = __shfl_sync(0xffffffffu, sl, i0);
    const uint32_t inrow = __ballot_sync(0xffffffffu, sl - s0 == lane - i0) >> i0;
    const uint16_t* from = src + first * stride;
    int n = seen;
    if (i0 + seen == 32)
      while (first + n < T && a.slot_map[first + n] >= 0 && a.slot_map[first + n] / kPageSize == page) ++n;
    // Rows one after another in the page, as a slot map built from lengths has them.
    const bool ordered = n == seen && (inrow & ((1u << seen) - 1)) == (1u << seen) - 1;
    const int r0 = s0 % kPageSize;
    const Run<kD, kHeads> run{rows, from, stride, scales + block, n, sub, lane, on};
    const float old = r0 == 0 ? 0.f : scales[block];  // with the rows: it is needed where the run begins behind slot 0
    if (ordered && n == kPageSize) {
      uint4 x[kLoads];
      const uint16_t* p = from + sub * stride;
#pragma unroll
      for (int u = 0; u < kLoads; ++u, p += kRows * stride) x[u] = ld_stream_v4(reinterpret_cast<const uint4*>(p));
      uint32_t amax = 0;
#pragma unroll
      for (int u = 0; u < kLoads; ++u) amax = max_abs_bf16x8(amax, x[u]);
      bool loud;
      const float inv = run.take_scale(amax, 0xffffu, 0.f, loud);
      uint8_t* q = rows + sub * kD;
      if (loud)
#pragma unroll
        for (int u = 0; u < kLoads; ++u) x[u] = without_inf(x[u]);
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        if (on) *reinterpret_cast<uint2*>(q + u * kRows * kD) = quantise8(x[u], inv);
    } else if (ordered) {
      uint4 x[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        x[u] = make_uint4(0u, 0u, 0u, 0u);
        if (u * kRows + sub < n) x[u] = ld_stream_v4(reinterpret_cast<const uint4*>(from + (u * kRows + sub) * stride));
      }
      uint32_t amax = 0;
#pragma unroll
      for (int u = 0; u < kLoads; ++u) amax = max_abs_bf16x8(amax, x[u]);
      bool loud;
      const float inv = run.take_scale(amax, ((1u << n) - 1) << r0, old, loud);
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        if (on && u * kRows + sub < n)
          *reinterpret_cast<uint2*>(rows + (r0 + u * kRows + sub) * kD) = quantise8(loud ? without_inf(x[u]) : x[u], inv);
    } else {
      // Rows in any order, and a run of more tokens than a page has (slots named twice).
      uint32_t amax = 0, written = 0;
      for (int k = 0; k < n; ++k) {
        written |= 1u << a.slot_map[first + k] % kPageSize;
        if (sub == 0) amax = max_abs_bf16x8(amax, ld_stream_v4(reinterpret_cast<const uint4*>(from + k * stride)));
      }
      bool loud;
      const float inv = run.take_scale(amax, written, scales[block], loud);
      for (int k = 0; k < n && on && sub == 0; ++k) {
        const uint4 x = ld_stream_v4(reinterpret_cast<const uint4*>(from + k * stride));
        *reinterpret_cast<uint2*>(rows + a.slot_map[first + k] % kPageSize * kD) =
            quantise8(loud ? without_inf(x) : x, inv);
      }
    }
  }
}

struct Kv8LoadArgs {
  Kv8View kv;
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t* first;
  const int32_t* token_start;
  int32_t batch;
  int32_t num_rows;
  uint16_t* out[2];
  long long stride[2];
  int32_t window;  // rows of a CTA
  unsigned* err;
};

template <int kD>
__global__ void __launch_bounds__(kLoadThreads, 3) kv8_load_kernel(const Kv8LoadArgs a) {
  constexpr int kLanes = kD / 16;        // lanes of a row, 16 codes each
  constexpr int kRows = 32 / kLanes;     // rows of a warp's load
  constexpr int kLoads = 8;              // loads in flight
  __shared__ int slots[kMaxWindow];      // of the window's rows, -1: none
  pdl_enter();
  const int total = min(a.token_start[a.batch], a.num_rows), t0 = blockIdx.x * a.window;
  const int n = min(a.window, total - t0);
  if (n <= 0) return;
  if (threadIdx.x < n) {
    const int t = t0 + threadIdx.x;
    int l = 0, hi = a.batch;  // the last request that begins at or before row t
    while (hi - l > 1) {
      const int mid = (l + hi) >> 1;
      if (a.token_start[mid] <= t) l = mid; else hi = mid;
    }
    const long long pos = (long long)t - a.token_start[l] + (a.first ? a.first[l] : 0);
    int slot = -1;
    if (pos < 0 || pos >= (long long)a.bt_stride * kPageSize) {
      raise_error(a.err, SE_DEVERR_LENGTH);
    } else {
      const int page = a.block_table[(size_t)l * a.bt_stride + pos / kPageSize];
      if (page < 0 || page >= a.kv.num_pages)
        raise_error(a.err, SE_DEVERR_PAGE_RANGE);
      else
        slot = page * kPageSize + (int)(pos % kPageSize);
    }
    slots[threadIdx.x] = slot;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, sub = lane / kLanes, x0 = lane % kLanes * 16;
  const int chunks = (n + kRows * kLoads - 1) / (kRows * kLoads), tasks = chunks * 2 * a.kv.num_kv_heads;
  for (int task = threadIdx.x >> 5; task < tasks; task += kLoadThreads / 32) {
    const int cg = task / chunks, r0 = (task - cg * chunks) * kRows * kLoads + sub, is_v = cg & 1, h = cg >> 1;
    const uint8_t* cache = is_v ? a.kv.v : a.kv.k;
    const float* scales = is_v ? a.kv.v_scale : a.kv.k_scale;
    uint4 c[kLoads];
    float s[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int r = r0 + u * kRows, slot = r < n ? slots[r] : -1;
      s[u] = -1.f;
      if (slot < 0) continue;
      const size_t block = (size_t)(slot / kPageSize) * a.kv.num_kv_heads + h;
      c[u] = ld_stream_v4(reinterpret_cast<const uint4*>(cache + (block * kPageSize + slot % kPageSize) * kD + x0));
      s[u] = scales[block];
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int r = r0 + u * kRows;
      if (r >= n || slots[r] < 0) continue;
      uint16_t* out = (is_v ? a.out[1] : a.out[0]) + (t0 + r) * (is_v ? a.stride[1] : a.stride[0]) + (long long)h * kD + x0;
      const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
      uint32_t y[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[4];
        from_e4m3x4(w[i], f);
        y[2 * i] = pack_bf16x2(f[0] * s[u], f[1] * s[u]);
        y[2 * i + 1] = pack_bf16x2(f[2] * s[u], f[3] * s[u]);
      }
      reinterpret_cast<uint4*>(out)[0] = make_uint4(y[0], y[1], y[2], y[3]);
      reinterpret_cast<uint4*>(out)[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
}

template <int kD, int kHeads>
cudaError_t launch_store(Kv8StoreArgs& a, int sm_count, cudaStream_t stream) {
  const int groups = 2 * ((a.kv.num_kv_heads + kHeads - 1) / kHeads);
  // Windows of 16 tokens once they fill the SMs (16 warps each), shorter ones before.
  a.window = 16;
  while (a.window > 1 && (long long)a.num_tokens * groups < (long long)a.window * 16 * sm_count) a.window /= 2;
  const long long warps = ((long long)a.num_tokens + a.window - 1) / a.window * groups;
  return launch_pdl(kv8_store_kernel<kD, kHeads>, dim3((unsigned)((warps + kWarps - 1) / kWarps)), dim3(kWarps * 32), 0,
                    stream, a);
}
template <int kD>
cudaError_t launch_load(const Kv8LoadArgs& a, unsigned grid, cudaStream_t stream) {
  return launch_pdl(kv8_load_kernel<kD>, dim3(grid), dim3(kLoadThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_kv8_store(const Kv8View& kv, const uint16_t* k_new, long long k_stride, const uint16_t* v_new,
                             long long v_stride, const int32_t* slot_map, int32_t num_tokens, int sm_count,
                             unsigned* err, cudaStream_t stream) {
  Kv8StoreArgs a;
  a.kv = kv;
  a.in[0] = k_new;
  a.in[1] = v_new;
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.slot_map = slot_map;
  a.num_tokens = num_tokens;
  a.err = err;
  // Rows of 256 dims to a warp where the heads allow: 8 KB in flight for each.
  const int h = kv.num_kv_heads;
  switch (kv.head_dim) {
    case 64: return h % 4 ? launch_store<64, 2>(a, sm_count, stream) : launch_store<64, 4>(a, sm_count, stream);
    case 128: return h % 2 ? launch_store<128, 1>(a, sm_count, stream) : launch_store<128, 2>(a, sm_count, stream);
    default: return launch_store<256, 1>(a, sm_count, stream);
  }
}

cudaError_t launch_kv8_load(const Kv8View& kv, const int32_t* block_table, int32_t bt_stride, const int32_t* first,
                            const int32_t* token_start, int32_t batch, int32_t num_rows, uint16_t* k_out,
                            long long k_stride, uint16_t* v_out, long long v_stride, int sm_count, unsigned* err,
                            cudaStream_t stream) {
  Kv8LoadArgs a;
  a.kv = kv;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.first = first;
  a.token_start = token_start;
  a.batch = batch;
  a.num_rows = num_rows;
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  a.err = err;
  // Windows of 64 rows once they fill the SMs (four CTAs each), shorter ones before.
  a.window = kMaxWindow;
  while (a.window > 8 && (long long)num_rows < (long long)a.window * 4 * sm_count) a.window /= 2;
  const unsigned grid = (unsigned)(((long long)num_rows + a.window - 1) / a.window);
  switch (kv.head_dim) {
    case 64: return launch_load<64>(a, grid, stream);
    case 128: return launch_load<128>(a, grid, stream);
    default: return launch_load<256>(a, grid, stream);
  }
}

}  // namespace se
