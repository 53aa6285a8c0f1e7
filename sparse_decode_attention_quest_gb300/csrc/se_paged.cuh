// What the dense paged decodes share: which pages and tokens of a request are
// kept, how the kept pages of a batch are shared among the CTAs, and the list of
// items whose partials are joined.
#pragma once

#include "se_ptx.cuh"

namespace se {

// The workspace of a dense paged decode: arrival counters of the items by their first CTA (zero between calls),
// the joins of every CTA, then the partials, two slots per CTA. The counters lie in the same place for every
// shape, and nothing else is written there, so that a workspace serves calls of all shapes that it is large
// enough for.
constexpr int kMaxCtas = 192;
constexpr size_t kArrivalBytes = kMaxCtas * sizeof(uint32_t);
constexpr size_t kCounterBytes = kArrivalBytes + kMaxCtas * sizeof(int2);
static_assert(kArrivalBytes % 16 == 0 && kCounterBytes % 16 == 0, "aligned for vector accesses");

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

// The longest line of items: places and the cuts beside them stay within 32 bits.
constexpr int kMaxPlaces = 0x7fffffff - 64;

// The share-out of a batch among the CTAs. An item is a request (or one of its `groups` groups of KV heads); it
// weighs its kept pages plus `over`, the pages' worth of time that starting and finishing an item costs a CTA, so
// that many short requests spread over the CTAs. The items' weights follow one another on a line of length
// `total`, cut every `span`. A cut within `over` of an item's end is moved there (a split costs a join), any
// other to a multiple of `unit` pages of its item. span > 2 over, so that the cuts keep their order and every CTA
// between an item's first and last holds pages of it.
//
// A batch that leaves CTAs over (kept_prefix decides) is cut into pieces instead: `piece` pages of one item, the last
// one of an item shorter, and each a CTA's whole slice. Then over = 0, an item weighs its pages rounded up to whole
// pieces, and span = piece.
struct Slices {
  const int* prefix;  // [batch + 1] weights of the requests before each (one group)
  int batch, groups, over, unit, span, total;

  // piece: as kept_prefix returned it.
  __device__ __forceinline__ void init(const int* pf, int n, int g, int overhead, int page_unit, int ctas, int piece) {
    prefix = pf;
    batch = n;
    groups = g;
    over = piece ? 0 : overhead;
    unit = page_unit;
    total = pf[n] * g;
    span = piece ? piece : max(2 * over + 1, (int)(((unsigned)total + (unsigned)ctas - 1) / (unsigned)ctas));
  }
  // The pages of request b, whose weight is w.
  __device__ __forceinline__ int pages_of(int b, int w) const {
    return over ? w - over : prefix[2 * batch + 1 + b];  // behind the prefix and the lengths
  }
  // The request whose weight covers place p < total.
  __device__ __forceinline__ int request_at(int p) const {
    int l = 0, h = batch;
    while (h - l > 1) {
      const int mid = (l + h) >> 1;
      if (prefix[mid] * groups <= p) l = mid; else h = mid;
    }
    return l;
  }
  // Where CTA k's slice begins (CTA k - 1's ends).
  __device__ __forceinline__ int cut(int k) const {
    if ((long long)k * span >= total) return total;
    const int p = k * span;
    if (over == 0) return p;
    const int b = request_at(p), base = prefix[b] * groups, w = prefix[b + 1] - prefix[b];
    const int s = groups == 1 ? base : p - (p - base) % w;  // the item's begin
    if (p - s <= over) return s;
    if (s + w - p <= over) return s + w;
    return s + over + (p - s - over + unit - 1) / unit * unit;
  }
};

// The slice [x, y) of a CTA. By a converged warp: a lane per cut.
__device__ __forceinline__ int2 slice_of(const Slices& sl, int cta) {
  const int mine = sl.cut(cta + (threadIdx.x & 1));
  return make_int2(__shfl_sync(0xffffffffu, mine, 0), __shfl_sync(0xffffffffu, mine, 1));
}

// Who else holds the items that reach beyond a CTA's slice [x, y): the item that began before it (partial slot 0;
// first0 the CTA where it begins, parts0 CTAs in all, 0: none) and the item that begins in it and goes on behind it
// (slot 1; parts1 CTAs from this one on, 0: none).
struct Neighbours {
  int first0, parts0, parts1;
};

// By a converged warp: the cuts are the long part, so the lanes take one each.
__device__ __forceinline__ Neighbours neighbours_of(const Slices& sl, int cta, int2 slice) {
  Neighbours h;
  const int lane = threadIdx.x & 31;
  // The item over the slice's first place (even lanes) and over its last (odd lanes).
  const int at = lane & 1 ? slice.y - 1 : slice.x;
  const int b = sl.request_at(at), base = sl.prefix[b] * sl.groups, w = sl.prefix[b + 1] - sl.prefix[b];
  const int s = sl.groups == 1 ? base : at - (at - base) % w;
  const int s0 = __shfl_sync(0xffffffffu, s, 0), e0 = __shfl_sync(0xffffffffu, s + w, 0);
  const int s1 = __shfl_sync(0xffffffffu, s, 1), e1 = __shfl_sync(0xffffffffu, s + w, 1);
  // Lane i: a place's span and the cuts beside it. Places: the first and the last page of the item that began
  // before, the last of the one that goes on behind.
  const int place = lane < 8 ? s0 + sl.over : lane < 16 ? e0 - 1 : e1 - 1;
  const int k = place / sl.span, c = sl.cut(k + (lane & 1));
  const int lo = __shfl_sync(0xffffffffu, c, lane & ~1), hi = __shfl_sync(0xffffffffu, c, lane | 1);
  const int owner = lo > place ? k - 1 : hi <= place ? k + 1 : k;
  const int f0 = __shfl_sync(0xffffffffu, owner, 0), l0 = __shfl_sync(0xffffffffu, owner, 8);
  const int l1 = __shfl_sync(0xffffffffu, owner, 16);
  h.first0 = f0;
  h.parts0 = s0 < slice.x ? l0 - f0 + 1 : 0;
  h.parts1 = e1 > slice.y && s1 >= slice.x ? l1 - cta + 1 : 0;
  return h;
}

// A CTA's slice, item by item: the pages [lo, hi) of the n of item (b, group).
struct Segments {
  Slices sl;
  int x, end;
  int b, group, lo, hi, n, item_start;
  __device__ __forceinline__ void init(const Slices& slices, int start, int stop) {
    sl = slices;
    x = start;
    end = stop;
    b = start < stop ? sl.request_at(start) : 0;
  }
  __device__ __forceinline__ bool next() {
    if (x >= end) return false;
    while (sl.prefix[b + 1] * sl.groups <= x) ++b;
    const int base = sl.prefix[b] * sl.groups, w = sl.prefix[b + 1] - sl.prefix[b];
    group = sl.groups == 1 ? 0 : (x - base) / w;
    item_start = base + group * w;
    n = sl.pages_of(b, w);
    lo = max(0, x - item_start - sl.over);
    x = min(item_start + w, end);
    hi = min(x - item_start - sl.over, n);
    return true;
  }
  __device__ __forceinline__ bool split() const { return lo > 0 || hi < n; }
};

constexpr int kPieceBatch = 160;  // a thread per request in every kernel

// Ints that kept_prefix writes.
constexpr size_t kept_ints(int batch) { return (size_t)(batch <= kPieceBatch ? 3 : 2) * batch + 1; }

// The requests' weights as an exclusive prefix (prefix[batch]: their sum), by the whole CTA. Places are 32-bit:
// requests that end behind place `most` are reported and left empty from there on. lens: the lengths as read, and
// for batches of up to kPieceBatch behind them the pages of each. sums: kThreads / 32 values.
//
// Returns the length of the pieces that the batch is cut into, 0: cut into slices of equal weight. Slices are at least
// 2 over + 1 long, so in a batch whose weight is less than that for every CTA some hold two items, or several steps of
// one, while others hold none. There pieces of one unit of pages are taken, or of two if they are no longer than the
// pages of such a slice, where every piece gets a CTA and the items have no more than `pieces` each on average (a
// join reads them all). 32 latent requests of up to 390 tokens: 16.4 us, 24.2 in slices; 100 requests of up to 200
// tokens, 4 heads of 128 dims: 9.1, 11.9.
template <int kThreads>
__device__ __forceinline__ int kept_prefix(const int32_t* seq_lens, int batch, int groups, int bt_stride, int sink,
                                           int recent, int over, int unit, int pieces, int ctas, int most, int* prefix,
                                           int* lens, long long* sums, unsigned* err) {
  static_assert(kPieceBatch <= kThreads, "one chunk");
  constexpr int kWarps = kThreads / 32;
  constexpr int kOne = 40;  // sums of pages, and from this bit on of requests that have any
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto weight = [&](long long v) { return (v & ((1ll << kOne) - 1)) + (int)(v >> kOne) * over; };
  // The sum of v over the threads up to this one, and over all. Of up to 32 requests every warp sums all itself.
  const bool alone = batch <= 32;
  const int me = alone ? lane : threadIdx.x;
  auto scan = [&](auto v, auto* part, auto& all) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const auto t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    if (alone) {
      all = __shfl_sync(0xffffffffu, v, 31);
      return v;
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) v += part[w];
      all += part[w];
    }
    __syncthreads();
    return v;
  };
  const bool writes = !alone || warp == 0;
  long long at = 0;
  int pages = 0;
  for (int base = 0; base < batch; base += kThreads) {
    const int b = base + me;
    const int L = b < batch ? seq_lens[b] : 0;
    if (writes && b < batch) lens[b] = L;
    pages = kept_of(L, bt_stride, sink, recent, err).n;
    long long all;
    const long long incl = weight(at + scan(pages > 0 ? pages + (1ll << kOne) : 0ll, sums, all));
    if (writes && b < batch) prefix[b + 1] = (int)(incl < most ? incl : -1);
    at += all;
  }
  if (threadIdx.x == 0) prefix[0] = 0;
  const long long total = weight(at);
  const int widest = 2 * unit <= over + 1 ? 2 * unit : unit, items = (int)(at >> kOne) * groups;
  const int bound = min(ctas, items * pieces);
  const long long places = min(total, 1ll << 20) * groups;  // many heads: beyond 32 bits
  int piece = 0;
  if (batch <= kPieceBatch && places <= (2 * over + 1) * ctas && places - items * over <= bound * widest) {
    // The requests' pieces of unit and of 2 unit pages, summed in the halves of a word.
    const int units = (pages + unit - 1) / unit;
    unsigned all;
    const unsigned incl =
        scan((unsigned)units | (unsigned)(units + 1) / 2 << 16, reinterpret_cast<unsigned*>(sums), all);
    if ((int)(all & 0xffff) * groups <= bound)
      piece = unit;
    else if (widest > unit && (int)(all >> 16) * groups <= bound)
      piece = widest;
    if (piece > 0 && writes && me < batch) {
      prefix[me + 1] = (piece == unit ? incl & 0xffff : incl >> 16) * piece;
      lens[batch + me] = pages;
    }
  }
  __syncthreads();
  if (total >= most) {
    // Too long a line: the requests from the first that does not fit on are left out.
    if (threadIdx.x == 0) {
      raise_error(err, SE_DEVERR_LENGTH);
      for (int b = 1; b <= batch; ++b)
        if (prefix[b] < 0) prefix[b] = prefix[b - 1];
    }
    __syncthreads();
  }
  return piece;
}

// Warps that share the partials of an item: each takes eight or fewer, until all eight warps of a CTA share.
__device__ __forceinline__ int share_of(int partials) {
  return partials <= 8 ? 1 : partials <= 16 ? 2 : partials <= 32 ? 4 : 8;
}

// The items to join, as (first CTA, item, partials, first unit), from joins[c] = (item, partials) of every CTA c (0
// partials: none), in the order of their CTAs: every CTA of a join kernel makes the same list. An item has
// ceil(tasks * share_of(partials) / warps) units, a CTA's work each: a task per warp, or per share_of warps. By the
// whole CTA (a thread per entry). counts: two values per warp. Returns (items, units).
__device__ __forceinline__ int2 list_joins(const int2* joins, int ctas, int tasks, int4* todo, int2* counts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int2 j = threadIdx.x < ctas ? joins[threadIdx.x] : make_int2(0, 0);
  const uint32_t some = __ballot_sync(0xffffffffu, j.y > 0);
  const int units = j.y > 0 ? (tasks * share_of(j.y) + warps - 1) / warps : 0;
  int incl = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) counts[warp] = make_int2(__popc(some), incl);
  __syncthreads();
  int at = __popc(some & ((1u << lane) - 1)), first = incl - units, items = 0, all = 0;
  for (int w = 0; w < warps; ++w) {
    const int2 c = counts[w];
    at += w < warp ? c.x : 0;
    first += w < warp ? c.y : 0;
    items += c.x;
    all += c.y;
  }
  if (j.y > 0) todo[at] = make_int4(threadIdx.x, j.x, j.y, first);
  __syncthreads();
  return make_int2(items, all);
}

// The item of unit u.
__device__ __forceinline__ int4 join_of(const int4* todo, int items, int u) {
  int l = 0, h = items;
  while (h - l > 1) {
    const int mid = (l + h) >> 1;
    if (todo[mid].w <= u) l = mid; else h = mid;
  }
  return todo[l];
}

// The base of exponentials whose largest argument is m: 0 where nothing but -inf has been seen.
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.f : m; }

}  // namespace se
