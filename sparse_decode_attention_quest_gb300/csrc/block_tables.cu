// Block tables and slot maps built on the GPU from request lengths.
//
// A pool keeps its free pages as a stack: free_pages[0 .. count - 1], taken from
// the end. For request b with before_b cached and new_b incoming tokens
//     have_b = ceil(before_b / 16),  need_b = ceil((before_b + new_b) / 16) - have_b,
//     off_b  = sum of need over the requests before b,
//     page have_b + i of b (i < need_b) = free_pages[count - 1 - (off_b + i)],
//     slot of the token at position j of b = 16 * page(j / 16) + j % 16.
// The release is the mirror image (page i of b goes to
// free_pages[count + total - 1 - (off_b + i)]), so a release straight after an
// extension restores the stack exactly.
//
// The work is a prefix sum over the batch and one write per token: a few KB to a
// few MB, so a call is bound by its launch and by the latency of a chain of
// dependent loads (lengths, then a free page, then the stores): with cold caches
// 7.6 us for one token in each of 32 requests, 6.8 us for four prompts of 32K
// tokens (64 CTAs), 9.2 us for 312,000 tokens of 250 requests, 5.1 to 5.7 us for the
// releases of the three. Hence one launch: every CTA sums the prefixes of the whole batch by itself (the lengths
// are a few KB in L2) and fills its share of the slot map. A new page is taken
// from the stack by each of its tokens (the index is arithmetic on the
// prefixes); the token at slot 0 also writes the table entry, so no CTA waits for
// another's table entries. The CTA that arrives last, when every CTA has read
// the lengths and the count, writes the new lengths and the count back: the
// lengths may be updated in place, by a release (se_block_tables_release_ex) too.
#include "se_ptx.cuh"

namespace se {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// Inclusive prefixes over the CTA of two values per thread, and the CTA's totals (64 bits: lengths are 31-bit, and
// a batch of them needs more).
struct Pair {
  long long tokens, pages;
};
__device__ __forceinline__ Pair cta_inclusive(Pair x, Pair* sums, Pair* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, x.tokens, o), p = __shfl_up_sync(0xffffffffu, x.pages, o);
    if (lane >= o) {
      x.tokens += t;
      x.pages += p;
    }
  }
  __syncthreads();  // the previous use of sums is over
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  Pair before = {0, 0}, all = {0, 0};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const Pair s = sums[w];
    if (w < warp) {
      before.tokens += s.tokens;
      before.pages += s.pages;
    }
    all.tokens += s.tokens;
    all.pages += s.pages;
  }
  *total = all;
  return {x.tokens + before.tokens, x.pages + before.pages};
}

// The number of free pages, from the pool's state (a count outside [0, num_pages] is reported and clipped).
__device__ __forceinline__ int free_count(const int32_t* pool_state, int num_pages, unsigned* err) {
  int f = pool_state[0];
  if (f < 0 || f > num_pages) {
    if (threadIdx.x == 0) raise_error(err, SE_DEVERR_PAGE_RANGE);
    f = f < 0 ? 0 : num_pages;
  }
  return f;
}

// Counts this CTA in; true in the CTA that arrives last (which has reset the counter).
__device__ __forceinline__ bool arrive_last(int32_t* pool_state) {
  __shared__ int s_last;
  __syncthreads();
  if (gridDim.x == 1) return true;
  if (threadIdx.x == 0) {
    const uint32_t before = atomic_add_acq_rel_gpu(reinterpret_cast<uint32_t*>(pool_state) + 1, 1u);
    s_last = before == gridDim.x - 1;
    if (s_last) pool_state[1] = 0;
  }
  __syncthreads();
  return s_last != 0;
}

// Largest r with start[r] <= t (start ascending, start[0] = 0 <= t): the owner of element t.
__device__ __forceinline__ int owner(const int* start, int n, int t) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) extend_kernel(const int32_t* __restrict__ free_pages, int32_t* pool_state,
                                                          int32_t num_pages, int32_t* block_table, int32_t bt_stride,
                                                          const int32_t* seq_lens, const int32_t* new_lens,
                                                          int32_t batch, int32_t* seq_lens_after,
                                                          int32_t* token_start, int32_t* slot_map,
                                                          int32_t* positions, int32_t max_new_tokens, unsigned* err) {
  pdl_enter();
  extern __shared__ int smem[];
  __shared__ Pair sums[kWarps];
  __shared__ int s_taken;
  int* start = smem;              // [batch + 1] first new token of each request
  int* off = start + batch + 1;   // [batch] first page of its share of the stack, -1: not served
  int* before = off + batch;      // [batch]
  const int f = free_count(pool_state, num_pages, err);
  if (threadIdx.x == 0) s_taken = 0;
  long long tok0 = 0, page0 = 0;
  for (int base = 0; base < batch; base += kThreads) {
    const int b = base + threadIdx.x;
    int bf = 0, nw = 0;
    bool ok = false;
    if (b < batch) {
      bf = seq_lens[b];
      nw = new_lens[b];
      ok = bf >= 0 && nw >= 0 && (long long)bf + nw <= (long long)bt_stride * kPageSize;
      before[b] = bf;
    }
    // Requests from the first that ends behind the map on are not served, so that what they would take changes
    // nothing for those before.
    const int need = ok ? (bf + nw + kPageSize - 1) / kPageSize - (bf + kPageSize - 1) / kPageSize : 0;
    const long long tokens = nw > 0 ? nw : 0;
    Pair total;
    const Pair in = cta_inclusive({tokens, need}, sums, &total);
    const long long tok_incl = tok0 + in.tokens, incl = page0 + in.pages;
    if (b < batch && !(ok && tok_incl <= max_new_tokens) && blockIdx.x == 0) raise_error(err, SE_DEVERR_LENGTH);
    ok = ok && tok_incl <= max_new_tokens;
    if (b < batch) {
      // In batch order: once a request finds too few pages left, no later one gets any.
      const bool served = ok && (need == 0 || incl <= f);
      if (ok && !served && blockIdx.x == 0) raise_error(err, SE_DEVERR_NO_PAGES);
      const long long t0 = tok_incl - tokens;
      start[b] = (int)(t0 < max_new_tokens ? t0 : max_new_tokens);
      off[b] = served ? (int)(need == 0 ? 0 : incl - need) : -1;
      if (served && need > 0) atomicMax(&s_taken, (int)incl);
    }
    tok0 += total.tokens;
    page0 += total.pages;
  }
  if (threadIdx.x == 0) start[batch] = (int)(tok0 < max_new_tokens ? tok0 : max_new_tokens);
  __syncthreads();
  const int filled = start[batch];

  // Four entries of the map per thread and step.
  for (long long t0 = ((long long)blockIdx.x * kThreads + threadIdx.x) * 4; t0 < max_new_tokens;
       t0 += (long long)gridDim.x * kThreads * 4) {
    int sl[4], ps[4];
    int r = t0 < filled ? owner(start, batch, (int)t0) : 0;
    int page = -1, phys = -1, last_r = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = (int)t0 + i;
      sl[i] = -1;
      ps[i] = 0;
      if (t >= filled) continue;
      while (start[r + 1] <= t) ++r;
      if (off[r] < 0) continue;
      const int bf = before[r];
      const int pos = bf + t - start[r];
      const int p = pos / kPageSize;
      if (p != page || r != last_r) {
        const int have = (bf + kPageSize - 1) / kPageSize;
        page = p;
        last_r = r;
        phys = p < have ? block_table[(size_t)r * bt_stride + p] : free_pages[f - 1 - (off[r] + p - have)];
        if (phys < 0 || phys >= num_pages) {
          raise_error(err, SE_DEVERR_PAGE_RANGE);
          phys = -1;
        }
      }
      if (pos % kPageSize == 0) block_table[(size_t)r * bt_stride + p] = phys;
      ps[i] = pos;
      if (phys >= 0) sl[i] = phys * kPageSize + pos % kPageSize;
    }
    if (t0 + 4 <= max_new_tokens) {
      *reinterpret_cast<int4*>(slot_map + t0) = make_int4(sl[0], sl[1], sl[2], sl[3]);
      if (positions) *reinterpret_cast<int4*>(positions + t0) = make_int4(ps[0], ps[1], ps[2], ps[3]);
    } else {
      for (int i = 0; t0 + i < max_new_tokens; ++i) {
        slot_map[t0 + i] = sl[i];
        if (positions) positions[t0 + i] = ps[i];
      }
    }
  }
  if (!arrive_last(pool_state)) return;
  for (int b = threadIdx.x; b <= batch; b += kThreads) {
    token_start[b] = start[b];
    if (b < batch) seq_lens_after[b] = off[b] >= 0 ? before[b] + (start[b + 1] - start[b]) : before[b];
  }
  if (threadIdx.x == 0) pool_state[0] = f - s_taken;
}

// Whether lengths can shrink from len to keep.
__device__ __forceinline__ bool can_release(int len, int keep, int32_t bt_stride) {
  return keep >= 0 && keep <= len && len <= (long long)bt_stride * kPageSize;
}

__global__ void __launch_bounds__(kThreads) release_kernel(int32_t* free_pages, int32_t* pool_state,
                                                           int32_t num_pages,
                                                           const int32_t* __restrict__ block_table,
                                                           int32_t bt_stride, const int32_t* seq_lens,
                                                           const int32_t* keep_lens, int32_t batch,
                                                           int32_t* seq_lens_after, unsigned* err) {
  pdl_enter();
  extern __shared__ int smem[];
  __shared__ Pair sums[kWarps];
  int* start = smem;               // [batch + 1] first page of each request in the returned sequence
  int* first = start + batch + 1;  // [batch] its first returned logical page
  const int f = free_count(pool_state, num_pages, err);
  long long page0 = 0;
  for (int base = 0; base < batch; base += kThreads) {
    const int b = base + threadIdx.x;
    int n = 0, fp = 0;
    if (b < batch) {
      const int len = seq_lens[b], keep = keep_lens ? keep_lens[b] : 0;
      if (can_release(len, keep, bt_stride)) {
        fp = keep / kPageSize + (keep % kPageSize != 0);
        n = len / kPageSize + (len % kPageSize != 0) - fp;
      } else if (blockIdx.x == 0) {
        raise_error(err, SE_DEVERR_LENGTH);
      }
    }
    Pair total;
    const long long incl = page0 + cta_inclusive({0, n}, sums, &total).pages;
    if (b < batch) {
      const long long s = incl - n;
      start[b] = (int)(s < num_pages ? s : num_pages);
      first[b] = fp;
    }
    page0 += total.pages;
  }
  // More pages than the pool lacks cannot come back: nothing is returned.
  const bool sane = page0 <= num_pages - f;
  if (!sane && blockIdx.x == 0 && threadIdx.x == 0) raise_error(err, SE_DEVERR_PAGE_RANGE);
  const int total = sane ? (int)page0 : 0;
  if (threadIdx.x == 0) start[batch] = total;
  __syncthreads();
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total; i += (long long)gridDim.x * kThreads) {
    const int r = owner(start, batch, (int)i);
    int phys = block_table[(size_t)r * bt_stride + first[r] + ((int)i - start[r])];
    if (phys < 0 || phys >= num_pages) {
      raise_error(err, SE_DEVERR_PAGE_RANGE);
      phys = -1;
    }
    free_pages[f + total - 1 - (int)i] = phys;
  }
  if (!arrive_last(pool_state)) return;
  // Every CTA has read the lengths, and a thread reads a request's before it writes them: in place is fine.
  if (seq_lens_after)
    for (int b = threadIdx.x; b < batch; b += kThreads) {
      const int len = seq_lens[b], keep = keep_lens ? keep_lens[b] : 0;
      seq_lens_after[b] = sane && can_release(len, keep, bt_stride) ? keep : len;
    }
  if (threadIdx.x == 0) pool_state[0] = f + total;
}

int grid_for(long long elements, int per_thread, int sm_count) {
  const long long g = (elements + kThreads * per_thread - 1) / (kThreads * per_thread);
  return (int)(g < 1 ? 1 : g > sm_count ? sm_count : g);
}

}  // namespace

int block_tables_max_batch() { return 16384; }

cudaError_t launch_block_tables_extend(const int32_t* free_pages, int32_t* pool_state, int32_t num_pages,
                                       int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                       const int32_t* new_lens, int32_t batch, int32_t* seq_lens_after,
                                       int32_t* token_start, int32_t* slot_map, int32_t* positions,
                                       int32_t max_new_tokens, int sm_count, unsigned* err, cudaStream_t stream) {
  const size_t smem = (3 * (size_t)batch + 1) * sizeof(int);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(extend_kernel, (3 * block_tables_max_batch() + 1) * (int)sizeof(int), allowed);
  if (e != cudaSuccess) return e;
  e = launch_pdl(extend_kernel, dim3(grid_for(max_new_tokens, 4, sm_count)), dim3(kThreads), smem, stream, free_pages,
                 pool_state, num_pages, block_table, bt_stride, seq_lens, new_lens, batch, seq_lens_after,
                 token_start, slot_map, positions, max_new_tokens, err);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_block_tables_release(int32_t* free_pages, int32_t* pool_state, int32_t num_pages,
                                        const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                        const int32_t* keep_lens, int32_t batch, int32_t* seq_lens_after,
                                        int sm_count, unsigned* err, cudaStream_t stream) {
  const size_t smem = (2 * (size_t)batch + 1) * sizeof(int);
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(release_kernel, (2 * block_tables_max_batch() + 1) * (int)sizeof(int), allowed);
  if (e != cudaSuccess) return e;
  const long long most = (long long)batch * bt_stride < num_pages ? (long long)batch * bt_stride : num_pages;
  e = launch_pdl(release_kernel, dim3(grid_for(most, 1, sm_count)), dim3(kThreads), smem, stream, free_pages, pool_state,
                 num_pages, block_table, bt_stride, seq_lens, keep_lens, batch, seq_lens_after, err);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace se
