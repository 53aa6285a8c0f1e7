// Attention of one new token per request over its whole paged cache, or over
// its first sink and last recent tokens (SparseEngine: Sparse-First Inference
// Engine, Table 7: logit z and weight alpha over the history, the current token
// included; Tables 9-12: sink and recent tokens), for head dims 64, 128 and 256.
//
//     z_j = sm_scale q . k_j over the kept positions j < L,
//     out = sum_j exp(z_j - m) v_j / l,  l = sum_j exp(z_j - m),  lse = m + log l,
// in one pass over K and V with a running maximum m and sum l. Every kept K and V
// row is read once and serves all query heads of its KV head, a few flops per
// byte: the floor is the time of those bytes from HBM, and the design is about
// keeping copies in flight.
//
//  * Work: (request, KV head group) items follow one another on a line, each as
//    long as its kept pages and a step's worth of overhead; the CTAs (one per SM)
//    take equal slices (or, where those leave CTAs over, pieces of one step each):
//    ragged lengths balance, and a single long request spreads
//    over every SM. An item that spans CTAs leaves a partial (output,
//    log-sum-exp) per CTA; a CTA has at most two, for the item it starts inside
//    and the item it ends inside, so the workspace does not grow with the lengths.
//  * Join: where the partials that an item of the table's (or the windows') width
//    has in slices of the least length stay within kInlineBytes, if need be with
//    fewer KV heads per item, the CTA that publishes an item's last partial merges
//    them in the order of the pages. Otherwise a second kernel does, a warp per row:
//    one CTA reads partials from L2 at some 60 bytes a clock, and merging 32 of 16 KB
//    took it 25 of 46 us (4 requests of 2.5K tokens, 32 query heads). 48
//    windows of 1,064 tokens: 27.5 us, against 29.0 with the second kernel and 29.5
//    with a bound of 100 KB. The table's width is its capacity, so the same lengths
//    behind a wider one may take the second kernel: one request of 4K tokens 9.6 us
//    behind a table of 256 pages, 11.9 behind one of 8,192. In pieces an item can have
//    about twice the partials that the bound counts: one request of 4K tokens beside
//    19 of one token, 32 partials of 2 KB, takes 10.5 us joined here and 11.8 by the
//    second kernel.
//  * Copies: a page's rows of one KV head are 16 x D bf16, and the heads of a
//    group of Hc lie next to each other, so that one TMA box of 64 dims x
//    16 Hc rows x D / 64 brings a whole page of the group (16 to 32 KB for 4 to 8
//    heads). One warp issues them into a ring of five 32 KB slots, K and V of a
//    step in turn, 128-byte swizzled.
//  * Products: a consumer warp holds one (KV head, tile of query heads) state; R
//    warps share the pages of a step when the heads do not fill the warps. S^T =
//    K Q^T and O^T += V^T P^T are m16n8k16 bf16 MMAs with fp32 accumulators: the
//    page's 16 tokens, or 16 dims, are the rows, and up to 8 query heads the
//    columns (two column tiles where a warp takes 16), so that a group of up to eight heads
//    wastes no rows: the other way round, with heads as rows, half of the MMAs
//    and of the exponentials were for rows that do not exist, and a block took
//    a warp 450 instructions (8 x 16K tokens, 4 KV heads: 50.7 us). P^T goes from
//    accumulator to operand layout by two 8 x 8 transposes in registers.
//  * Rows that are not kept: their logits become -inf, and their value rows are
//    zeroed in shared memory first, since 0 * NaN is not 0.
#include <algorithm>

#include "se_paged_join.cuh"

namespace se {
namespace {

constexpr int kSlots = 5;
constexpr int kSlotBytes = 32 * 1024;
constexpr int kMetaRing = 4;     // steps whose page masks are held (at most three are in flight)
constexpr int kMaxPages = 16;    // pages of a step
constexpr int kMaxBatch = 4096;  // requests whose prefix fits beside the ring
constexpr int kInlineBytes = 48 * 1024;  // partials of an item, in slices, where one CTA merges them
constexpr int kInlineWidth = 32;          // pages of an item from which smaller boxes are taken for that

template <int kD>
struct Cfg {
  static constexpr int kWarps = kD == 256 ? 4 : 8;  // consumers
  static constexpr int kConsumers = kWarps * 32;
  static constexpr int kThreads = kConsumers + 32;
  static constexpr int kChunks = kD / 64;
  static constexpr int kBlocks = kSlotBytes / (kPageSize * kD * 2);  // (page, head) blocks of a slot
  static constexpr int kStageFloats = kWarps * 8 * kD;               // states handed over at a segment's end
  static constexpr int kFixed = 1024 + kSlots * kSlotBytes + kStageFloats * 4 + kWarps * 32 * 4 +
                                kMetaRing * kMaxPages * 4 + 2 * kSlots * 8 + 64;
  static constexpr int kMaxSmem = kFixed + kept_ints(kMaxBatch) * 4;
};

struct PagedArgs {
  const uint16_t* q;
  long long q_stride;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t group;        // query heads per KV head
  int32_t heads;        // KV heads of an item (Hc)
  int32_t head_groups;  // items per request
  int32_t mtiles;       // tiles of 8 or 16 query heads per KV head
  int32_t replicas;     // warps that share a (head, tile)
  int32_t step_pages;   // pages of a step
  int32_t num_pages;
  int32_t batch;
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t* seq_lens;
  int32_t sink, recent;
  float scale_log2;
  uint16_t* out;
  float* out_lse;
  float* o_part;        // [2 * CTAs][heads * group][D]
  float* lse_part;      // [2 * CTAs][heads * group], log2 domain
  // An item that spans CTAs is the only one to go on behind its first CTA, so that CTA's index names it.
  uint32_t* arrivals;   // [kMaxCtas] by first CTA, zero between calls
  int2* joins;          // [CTAs] by first CTA: item and partials for the join kernel (0 partials: nothing to do)
  bool deferred;        // the join kernel follows
  unsigned* err;
};

// kNt: column tiles of eight query heads; kSolo: no two warps share a (head, tile) (code of its own: as a branch
// beside the other it cost that one 0.8 us of 9.9).
template <int kD, int kNt, bool kSolo>
__global__ void __launch_bounds__(Cfg<kD>::kThreads, 1) paged_decode_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                           const __grid_constant__ CUtensorMap vmap,
                                                                           const PagedArgs a) {
  using C = Cfg<kD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* stage = reinterpret_cast<float*>(ring + kSlots * kSlotBytes);  // [warps][8][D]
  float* ml = stage + C::kStageFloats;                                  // [warps][(m, l)][8]
  uint32_t* meta = reinterpret_cast<uint32_t*>(ml + C::kWarps * 32);    // [kMetaRing][kMaxPages]
  uint64_t* full = reinterpret_cast<uint64_t*>(meta + kMetaRing * kMaxPages);
  uint64_t* empty = full + kSlots;
  int* flags = reinterpret_cast<int*>(empty + kSlots);  // [8]: joins to make, the items of slots 0 and 1, neighbours
  int* prefix = flags + 8;                              // [batch + 1]
  int* lens = prefix + a.batch + 1;                     // [batch], then the pages of each
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads = a.heads, G = a.group, rows = heads * G, HG = a.head_groups, Pg = a.step_pages;
  const int combos = heads * a.mtiles, active = combos * a.replicas;

  // What needs no input comes before the wait for the previous kernel; kept_prefix's barriers publish it.
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], active);
    }
    mbar_fence_init();
  }
  if (warp == C::kWarps && lane == 0) {
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
  }
  pdl_enter();
  // Pieces of a step: of up to eight query heads a CTA takes a second one in less time than more partials take to
  // join (1 x 1,000 tokens, 8 KV heads: 10.6 us with 32 partials an item, 10.0 with 16), of more it does not (1 x 4K,
  // 32 heads over one: 14.6 us with 32, 17.8 with 16).
  const int piece = kept_prefix<C::kThreads>(a.seq_lens, a.batch, HG, a.bt_stride, a.sink, a.recent, Pg, Pg,
                                             G > 8 ? 32 : 8, gridDim.x, kMaxPlaces / HG, prefix, lens,
                                             reinterpret_cast<long long*>(stage), a.err);
  // Requests without a kept token: the empty sum.
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    if (prefix[b + 1] != prefix[b]) continue;
    const size_t r0 = (size_t)b * a.num_q_heads;
    uint4* o = reinterpret_cast<uint4*>(a.out + r0 * kD);
    for (int i = threadIdx.x; i < a.num_q_heads * kD / 8; i += C::kThreads) o[i] = make_uint4(0, 0, 0, 0);
    if (a.out_lse)
      for (int i = threadIdx.x; i < a.num_q_heads; i += C::kThreads) a.out_lse[r0 + i] = -INFINITY;
  }
  Slices slices;
  slices.init(prefix, a.batch, HG, Pg, Pg, gridDim.x, piece);
  const int2 slice = slice_of(slices, blockIdx.x);
  if (slice.x >= slice.y) {
    if (a.deferred && threadIdx.x == 0) a.joins[blockIdx.x] = make_int2(0, 0);
    return;
  }

  Segments seg;
  seg.init(slices, slice.x, slice.y);
  bool dead = false;  // a bounded wait gave up: no further waits or products, but every barrier

  if (warp == C::kWarps) {
    // ------------------------------------------------------------ TMA producer
    const uint64_t policy = l2_evict_first_policy();
    const uint32_t page_bytes = (uint32_t)heads * kPageSize * kD * 2;
    int j = 0, step = 0;
    while (!dead && seg.next()) {
      const Kept k = kept_of(lens[seg.b], a.bt_stride, a.sink, a.recent, nullptr);
      const int32_t* bt = a.block_table + (size_t)seg.b * a.bt_stride;
      auto entry = [&](int i) { return i < seg.hi ? bt[k.logical(i)] : -1; };
      // Two windows of 32 table entries, one per lane: the second is loaded while the first is copied.
      int base = seg.lo, cur = entry(base + lane), nxt = entry(base + 32 + lane);
      for (int i0 = seg.lo; i0 < seg.hi && !dead; i0 += Pg, ++step) {
        if (i0 >= base + 32) {
          base += 32;
          cur = nxt;
          nxt = entry(base + 32 + lane);
        }
        const int i = i0 + lane;
        const int pc = __shfl_sync(0xffffffffu, cur, (i - base) & 31);
        const int pn = __shfl_sync(0xffffffffu, nxt, (i - base) & 31);
        const int phys = i < base + 32 ? pc : pn;
        const bool mine = lane < Pg && i < seg.hi;
        const bool ok = mine && phys >= 0 && phys < a.num_pages;
        if (mine && !ok) raise_error(a.err, SE_DEVERR_PAGE_RANGE);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, ok)) * page_bytes;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++j) {
          const int s = j % kSlots;
          if (lane == 0 && j >= kSlots && !mbar_wait(&empty[s], (j / kSlots - 1) & 1)) dead = true;
          dead = __shfl_sync(0xffffffffu, (int)dead, 0) != 0;
          if (dead) break;
          if (kv == 0 && lane < Pg)
            meta[(step % kMetaRing) * kMaxPages + lane] = ok ? page_mask(k, a.sink, k.logical(i)) : 0u;
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
          __syncwarp();
          if (ok)
            tma_load_3d(ring + s * kSlotBytes + lane * page_bytes, kv ? &vmap : &kmap, 0,
                        (phys * a.num_kv_heads + seg.group * heads) * kPageSize, 0, &full[s], policy);
        }
      }
    }
    // Every copy has landed before the CTA leaves.
    if (lane == 0) {
      for (int u = max(0, j - kSlots); u < j; ++u)
        if (!mbar_wait(&full[u % kSlots], (u / kSlots) & 1)) dead = true;
      if (dead) raise_error(a.err, SE_DEVERR_WAIT_TIMEOUT);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const bool works = warp < active;
  const int combo = warp % combos, replica = warp / combos;
  const int hc = combo / a.mtiles, mt = combo % a.mtiles;
  const int g = lane >> 2, t = lane & 3;
  const int tile_head = mt * 8 * kNt;  // first query head of the tile, in its KV head's group
  const uint32_t ring0 = smem_addr(ring);
  const uint32_t plane = (uint32_t)heads * kPageSize * 128;  // 64 dims of a page's rows
  const uint32_t page_bytes = plane * C::kChunks;
  const uint32_t k_off = swz128(lane & 15, lane >> 4);
  const uint32_t v_off = swz128((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
  int j = 0, step = 0;
  if (warp == 0) {  // while the first copies are on their way; in shared memory, as the loop needs its registers
    const Neighbours share = neighbours_of(slices, blockIdx.x, slice);
    if (lane == 0) {
      flags[2] = flags[3] = 0;
      flags[4] = share.first0;
      flags[5] = share.parts0;
      flags[6] = share.parts1;
    }
  }
  bool handed = false;

  while (seg.next()) {
    // Q^T as the B operand: head g of each column tile, dims 2 t, 2 t + 1 and 8 more.
    uint32_t qb[kD / 16][kNt][2];
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      const int hd = tile_head + nt * 8 + g;
      const bool real = works && hd < G;
      const int row = (seg.group * heads + hc) * G + (real ? hd : 0);
      const uint16_t* qr = a.q + (size_t)seg.b * a.q_stride + (size_t)row * kD;
#pragma unroll
      for (int ks = 0; ks < kD / 16; ++ks) {
        qb[ks][nt][0] = real ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * t) : 0u;
        qb[ks][nt][1] = real ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 2 * t + 8) : 0u;
      }
    }
    // O^T: dims 16 i + g (0, 1) and 8 more (2, 3), heads 2 t and 2 t + 1 of each column tile; m and l of those heads
    // (l: the thread's tokens only).
    float o[kD / 16][kNt][4], m[kNt][2], l[kNt][2];
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
#pragma unroll
      for (int i = 0; i < kD / 16; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    for (int i0 = seg.lo; i0 < seg.hi; i0 += Pg, ++step, j += 2) {
      if (!works) continue;
      const int sk = j % kSlots, sv = (j + 1) % kSlots;
      if (!dead && !__all_sync(0xffffffffu, mbar_wait(&full[sk], (j / kSlots) & 1))) dead = true;
      bool v_here = false, zeroed = false;
      for (int pg = replica; pg < Pg; pg += a.replicas) {
        const uint32_t mask = dead || i0 + pg >= seg.hi ? 0u : meta[(step % kMetaRing) * kMaxPages + pg];
        const bool last = pg + a.replicas >= Pg;
        const uint32_t blk = pg * page_bytes + (uint32_t)hc * kPageSize * 128;
        uint32_t pb[kNt][2];
        if (mask) {
          // The swizzle is an exclusive or of the 16-byte chunk with the row: two chunks further is one of bit 5 on.
          const uint32_t ka = ring0 + sk * kSlotBytes + blk + k_off;
          // S^T of one column tile in two accumulators: shorter chains of dependent products.
          constexpr int kAcc = kNt == 1 ? 2 : 1;
          float s2[kNt][kAcc][4];
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s2[nt][0][e] = s2[nt][kAcc - 1][e] = 0.f;
#pragma unroll
          for (int ks = 0; ks < kD / 16; ++ks) {
            uint32_t r0, r1, r2, r3;
            ldmatrix_x4(r0, r1, r2, r3, (ka ^ ((ks & 3) << 5)) + (ks >> 2) * plane);
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt)
              mma_bf16_16816(s2[nt][ks % kAcc], r0, r1, r2, r3, qb[ks][nt][0], qb[ks][nt][1]);
          }
          // Tokens g (0, 1) and g + 8 (2, 3), heads 2 t and 2 t + 1.
          float z[kNt][4];
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[nt][e] = (kAcc == 2 ? s2[nt][0][e] + s2[nt][1][e] : s2[nt][0][e]) * a.scale_log2;
          if (!mask_is_full(mask)) {
            const bool k0 = in_mask(mask, g), k1 = in_mask(mask, g + 8);
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) {
              z[nt][0] = k0 ? z[nt][0] : -INFINITY;
              z[nt][1] = k0 ? z[nt][1] : -INFINITY;
              z[nt][2] = k1 ? z[nt][2] : -INFINITY;
              z[nt][3] = k1 ? z[nt][3] : -INFINITY;
            }
          }
          float top[kNt][2];
          bool moved = false;
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              top[nt][e] = fmaxf(z[nt][e], z[nt][2 + e]);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1)
                top[nt][e] = fmaxf(top[nt][e], __shfl_xor_sync(0xffffffffu, top[nt][e], x));
              moved = moved || top[nt][e] > m[nt][e];
            }
          if (__any_sync(0xffffffffu, moved)) {
            // Some head's maximum moves: its sums follow.
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float mn = fmaxf(m[nt][e], top[nt][e]), f = fast_exp2(m[nt][e] - finite_base(mn));
                m[nt][e] = mn;
                l[nt][e] *= f;
#pragma unroll
                for (int i = 0; i < kD / 16; ++i) {
                  o[i][nt][e] *= f;
                  o[i][nt][2 + e] *= f;
                }
              }
          }
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) {
            // A head that has seen nothing but -inf keeps m = -inf and takes 0 as its base.
            const float b0 = finite_base(m[nt][0]), b1 = finite_base(m[nt][1]);
            const float p0 = fast_exp2(z[nt][0] - b0), p1 = fast_exp2(z[nt][1] - b1);
            const float p2 = fast_exp2(z[nt][2] - b0), p3 = fast_exp2(z[nt][3] - b1);
            l[nt][0] += p0 + p2;
            l[nt][1] += p1 + p3;
            // P meets V as bf16 (half a step, 2^-8 of each weight), as the MMA wants; l sums it unrounded.
            pb[nt][0] = transpose_8x8_b16(pack_bf16x2(p0, p1));
            pb[nt][1] = transpose_8x8_b16(pack_bf16x2(p2, p3));
          }
        }
        if (last) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[sk]);
        }
        if (!v_here) {
          if (!dead && !__all_sync(0xffffffffu, mbar_wait(&full[sv], ((j + 1) / kSlots) & 1))) dead = true;
          v_here = true;
        }
        if (mask && !dead) {
          const uint32_t vt = ring0 + sv * kSlotBytes + blk;
          if (!mask_is_full(mask)) {
            // Stale rows may hold NaN: zero them (two lanes per row).
            const int r = lane >> 1;
            if (!in_mask(mask, r))
              for (int c = lane & 1; c < kD / 8; c += 2)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + (c >> 3) * plane + swz128(r, c & 7)),
                             "r"(0u)
                             : "memory");
            zeroed = true;
            __syncwarp();
          }
          const uint32_t va = vt + v_off;
#pragma unroll
          for (int i = 0; i < kD / 16; ++i) {
            uint32_t r0, r1, r2, r3;
            ldmatrix_x4_trans(r0, r1, r2, r3, (va ^ ((i & 3) << 5)) + (i >> 2) * plane);
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) mma_bf16_16816(o[i][nt], r0, r1, r2, r3, pb[nt][0], pb[nt][1]);
          }
        }
      }
      if (zeroed) fence_proxy_async_smem();  // before the next copy into the slot
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[sv]);
    }

    // ---- the end of a segment: this CTA's share of item (b, hg) is done
    const bool split = seg.split();
    const int slot = seg.lo > 0 ? 0 : 1, item = seg.b * HG + seg.group;
    if (split && threadIdx.x == 0) flags[2 + slot] = item;
    const size_t out_row0 = (size_t)seg.b * a.num_q_heads + (size_t)seg.group * rows;
    const size_t part_row0 = (size_t)(2 * blockIdx.x + slot) * rows;
    // A whole row without a finite logit is 0 whatever its values hold (0 times them need not be); a partial of one
    // keeps that product, as the sum over a row with other tokens does.
    // The R warps of a (head, tile) stage their states, eight query heads at a time, and share the sums and the
    // output. Named barriers of the R warps: 2 + 2 combo, the states are there; 3 + 2 combo, they are read.
    if (!works) continue;
    const uint32_t threads = a.replicas * 32;
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      if (tile_head + nt * 8 >= G) continue;
      if (!kSolo && handed) named_bar_sync(3 + 2 * combo, threads);
      __syncwarp();
      handed = true;
      float* dst = stage + warp * 8 * kD;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
        const int hd = 2 * t + e;
        if constexpr (kSolo) {
          // No other states: the row is final.
          const bool none = l[nt][e] == 0.f;
          const float inv = none ? 0.f : 1.f / l[nt][e];
          const float lse2 = none ? -INFINITY : m[nt][e] + log2f(l[nt][e]);
          const int qr = tile_head + nt * 8 + hd, r = hc * G + qr;
#pragma unroll
          for (int i = 0; i < kD / 16; ++i) {
            o[i][nt][e] = none && !split ? 0.f : o[i][nt][e] * inv;
            o[i][nt][2 + e] = none && !split ? 0.f : o[i][nt][2 + e] * inv;
          }
          if (g == 0 && qr < G) {
            if (split)
              a.lse_part[part_row0 + r] = lse2;
            else if (a.out_lse)
              a.out_lse[out_row0 + r] = lse2 * kLn2;
          }
        }
#pragma unroll
        for (int i = 0; i < kD / 16; ++i) {
          dst[stage_at<kD>(hd, 16 * i + g)] = o[i][nt][e];
          dst[stage_at<kD>(hd, 16 * i + g + 8)] = o[i][nt][2 + e];
        }
        if (g == 0) {
          ml[warp * 16 + hd] = m[nt][e];
          ml[warp * 16 + 8 + hd] = l[nt][e];
        }
      }
      const int hds = min(8, G - tile_head - nt * 8);
      const size_t r0 = hc * G + tile_head + nt * 8;
      if constexpr (kSolo) {
        __syncwarp();
#pragma unroll 4
        for (int e = lane; e < hds * (kD / 4); e += 32) {
          const int d = e % (kD / 4) * 4, hd = e / (kD / 4);
          const float4 v = *reinterpret_cast<const float4*>(dst + stage_at<kD>(hd, d));
          if (split)
            *reinterpret_cast<float4*>(a.o_part + (part_row0 + r0 + hd) * kD + d) = v;
          else
            *reinterpret_cast<uint2*>(a.out + (out_row0 + r0 + hd) * kD + d) =
                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
        continue;
      }
      named_bar_sync(2 + 2 * combo, threads);
#pragma unroll 4
      for (int e = replica * 32 + lane; e < hds * (kD / 4); e += threads) {
        const int d = e % (kD / 4) * 4, hd = e / (kD / 4);
        float M = -INFINITY;
        for (int w = combo; w < active; w += combos) M = fmaxf(M, ml[w * 16 + hd]);
        const float base = finite_base(M);
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = combo; w < active; w += combos) {
          const float f = fast_exp2(ml[w * 16 + hd] - base);
          sum += f * ml[w * 16 + 8 + hd];
          const float4 v = *reinterpret_cast<const float4*>(stage + w * 8 * kD + stage_at<kD>(hd, d));
          acc = make_float4(acc.x + f * v.x, acc.y + f * v.y, acc.z + f * v.z, acc.w + f * v.w);
        }
        const bool none = sum == 0.f;
        const float inv = none ? 0.f : 1.f / sum, lse2 = none ? -INFINITY : M + log2f(sum);
        const size_t r = r0 + hd;
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (split)
          *reinterpret_cast<float4*>(a.o_part + (part_row0 + r) * kD + d) = acc;
        else
          *reinterpret_cast<uint2*>(a.out + (out_row0 + r) * kD + d) =
              none ? make_uint2(0u, 0u) : make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
        if (d == 0) {
          if (split)
            a.lse_part[part_row0 + r] = lse2;
          else if (a.out_lse)
            a.out_lse[out_row0 + r] = lse2 * kLn2;
        }
      }
    }
  }
  if (dead && lane == 0) raise_error(a.err, SE_DEVERR_WAIT_TIMEOUT);
  if (a.deferred && threadIdx.x == 0) a.joins[blockIdx.x] = make_int2(flags[3], flags[6]);

  // ---- Publish: count this CTA in on the (at most two) items it shares with few others; whoever completes
  // an item's count merges its partials (written by other CTAs: read past L1) and resets the counter.
  if (a.deferred) return;
  __threadfence();
  named_bar_sync(1, C::kConsumers);
  const int first0 = flags[4], parts0 = flags[5], parts1 = flags[6];
  if (parts0 == 0 && parts1 == 0) return;  // the same for all consumers
  if (threadIdx.x < 2) {
    const int parts = threadIdx.x ? parts1 : parts0;
    int last = 0;
    if (parts > 0) {
      uint32_t* cnt = a.arrivals + (threadIdx.x ? (int)blockIdx.x : first0);
      last = atomic_add_acq_rel_gpu(cnt, 1u) == (uint32_t)parts - 1;
      if (last) *cnt = 0;
    }
    flags[threadIdx.x] = last;
  }
  named_bar_sync(1, C::kConsumers);
  auto* join_smem = reinterpret_cast<JoinSmem<kD, C::kWarps>*>(stage);  // the states staged there are read
  static_assert(sizeof(JoinSmem<kD, C::kWarps>) <= (C::kStageFloats + C::kWarps * 32) * 4, "the join's sums fit");
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    if (!flags[s]) continue;
    const int first = s ? (int)blockIdx.x : first0, parts = s ? parts1 : parts0, item = flags[2 + s];
    const int warps = min(C::kWarps, share_of(parts));
    for (int r0 = 0; r0 < rows; r0 += C::kWarps / warps)
      join_rows<kD, C::kWarps, 8, false, 0>(a.o_part, a.lse_part, first, parts, item, rows, r0, warps, *join_smem,
                                            a.out, a.out_lse, [] { named_bar_sync(1, C::kConsumers); });
  }
}

// How the heads of a call are laid over the consumer warps, and where its joins run.
struct HeadPlan {
  int heads, head_groups, mtiles, replicas, step_pages;
  bool deferred;
};

// Query heads per KV head up to which a tile holds eight of them, above it sixteen. A warp of sixteen heads reads K
// and V once for both, but its state spills (nine warps leave 168 registers): it is the better one where shared
// memory or the tensor pipe would be read twice over at the full rate, that is in long caches of 64 dims (16 heads
// per KV head at 800 MB: 151 us, tiles of eight 176) and for many heads (128 dims, 32 heads: 182 against 222). Up to
// here eights are faster where latency counts (32 requests of 2.5K tokens, 4 KV heads of 128 dims with 16 heads
// each: 33.6 us against 40.8; 2 of 256 dims: 34.9 against 44.8) and even at 800 MB (131 against 135, 134 against 138;
// 32 heads of 256 dims: 223 against 217, and 32.5 against 41.8 for the 32 requests).
int eights_up_to(int head_dim) { return head_dim == 64 ? 8 : head_dim == 128 ? 16 : 32; }

// As many heads per box as leave at most an eighth of a slot empty (ten heads: boxes of two, not of five; 4 KB boxes
// of one head read at 91% of the measured copy rate, slots five eighths full at 73%), and no more than `most_heads`.
HeadPlan head_plan(int num_kv_heads, int group, int head_dim, int most_heads) {
  const int warps = head_dim == 256 ? Cfg<256>::kWarps : Cfg<128>::kWarps;
  const int blocks = kSlotBytes / (kPageSize * head_dim * 2);
  HeadPlan p;
  p.mtiles = group <= eights_up_to(head_dim) ? (group + 7) / 8 : (group + 15) / 16;
  for (int c = 1; c <= most_heads && c * p.mtiles <= warps; ++c) {
    if (num_kv_heads % c) continue;
    const int r = warps / (c * p.mtiles), pages = blocks / c / r * r;
    if (c > 1 && pages * c * 8 < blocks * 7) continue;
    p.heads = c;
    p.replicas = r;
    p.step_pages = pages;
  }
  p.head_groups = num_kv_heads / p.heads;
  p.deferred = true;
  return p;
}

// The largest boxes, unless the table's (or the windows') width keeps an item's partials, counted in slices of the
// least length, so few that smaller ones let the decode kernel join them: fewer heads per item are fewer rows to join and more CTAs that join. Not
// for short items, which are seldom split: more of them cost more than the join (64 requests of up to 19 pages, 8 KV
// heads of 64 dims: 16.8 us, 21.9 in boxes of four; up to 157 pages, 4 heads of 128 dims: 31.6, and 30.0 in boxes of
// one).
HeadPlan call_plan(int num_kv_heads, int group, int head_dim, int32_t bt_stride, int32_t sink_tokens,
                   int32_t recent_tokens, int ctas) {
  long long width = bt_stride;
  if (recent_tokens > 0)
    width = std::min(width, ((long long)sink_tokens + kPageSize - 1) / kPageSize + recent_tokens / kPageSize + 2);
  for (int c = 8; c > 0;) {
    HeadPlan p = head_plan(num_kv_heads, group, head_dim, c);
    if (c < 8 && width < kInlineWidth) break;
    const long long parts = std::min<long long>(ctas, (width + p.step_pages) / (2 * p.step_pages + 1) + 2);
    p.deferred = parts * p.heads * group * head_dim * (long long)sizeof(float) > kInlineBytes;
    if (!p.deferred) return p;
    c = p.heads - 1;
  }
  return head_plan(num_kv_heads, group, head_dim, 8);
}

int ctas_of(int sm_count) { return sm_count < kMaxCtas ? sm_count : kMaxCtas; }

template <int kD, int kNt, bool kSolo>
cudaError_t launch_as(const CUtensorMap& kmap, const CUtensorMap& vmap, const PagedArgs& a, int grid,
                   cudaStream_t stream) {
  const size_t smem = Cfg<kD>::kFixed + kept_ints(a.batch) * 4;
  static_assert(Cfg<kD>::kMaxSmem <= 227 * 1024, "the largest batch fits");
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(paged_decode_kernel<kD, kNt, kSolo>, Cfg<kD>::kMaxSmem, allowed);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_decode_kernel<kD, kNt, kSolo>, dim3(grid), dim3(Cfg<kD>::kThreads), smem, stream, kmap, vmap, a);
  if (e != cudaSuccess || !a.deferred) return e;
  const int rows = a.heads * a.group;
  // An item has at most `rows` units, and no more items than CTAs reach beyond a slice.
  const int units = std::min(grid, a.batch * a.head_groups) * rows;
  return launch_pdl(paged_join_kernel<kD, 0>, dim3(std::min(units, 8 * grid)), dim3(kJoinWarps * 32), 0, stream,
                    a.o_part, a.lse_part, a.joins, grid, rows, a.out, a.out_lse);
}

template <int kD>
cudaError_t launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const PagedArgs& a, int grid,
                   cudaStream_t stream) {
  const bool solo = a.replicas == 1;
  if (a.group <= 8 * a.mtiles)
    return solo ? launch_as<kD, 1, true>(kmap, vmap, a, grid, stream)
                : launch_as<kD, 1, false>(kmap, vmap, a, grid, stream);
  if constexpr (kD < 256)  // at 256 dims three or four tiles of sixteen leave no second warp to any
    if (!solo) return launch_as<kD, 2, false>(kmap, vmap, a, grid, stream);
  return launch_as<kD, 2, true>(kmap, vmap, a, grid, stream);
}

}  // namespace

int paged_decode_max_batch() { return kMaxBatch; }

bool paged_decode_supported(int num_kv_heads, int head_dim, int head_dim_v, int num_q_heads) {
  return head_dim == head_dim_v && (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
         num_q_heads / num_kv_heads <= 64;
}

int paged_decode_box_heads(int num_kv_heads, int num_q_heads, int head_dim, int32_t bt_stride, int32_t sink_tokens,
                           int32_t recent_tokens, int sm_count) {
  return call_plan(num_kv_heads, num_q_heads / num_kv_heads, head_dim, bt_stride, sink_tokens, recent_tokens,
                   ctas_of(sm_count)).heads;
}

size_t paged_decode_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  const HeadPlan p = head_plan(num_kv_heads, num_q_heads / num_kv_heads, head_dim, 8);  // the most rows of an item
  const size_t rows = (size_t)p.heads * (num_q_heads / num_kv_heads);
  return kCounterBytes + 2 * kMaxCtas * rows * (head_dim + 1) * sizeof(float);
}

cudaError_t launch_paged_decode(const CUtensorMap& kmap, const CUtensorMap& vmap, const KvView& kv, const uint16_t* q,
                                long long q_stride, int32_t num_q_heads, const int32_t* block_table,
                                int32_t bt_stride, const int32_t* seq_lens, int32_t batch, int32_t sink_tokens,
                                int32_t recent_tokens, float sm_scale, uint16_t* out, float* out_lse, void* workspace,
                                int sm_count, unsigned* err, cudaStream_t stream) {
  const int group = num_q_heads / kv.num_kv_heads;
  const int grid = ctas_of(sm_count);
  const HeadPlan p = call_plan(kv.num_kv_heads, group, kv.head_dim, bt_stride, sink_tokens, recent_tokens, grid);
  PagedArgs a;
  a.q = q;
  a.q_stride = q_stride;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = kv.num_kv_heads;
  a.group = group;
  a.heads = p.heads;
  a.head_groups = p.head_groups;
  a.mtiles = p.mtiles;
  a.replicas = p.replicas;
  a.step_pages = p.step_pages;
  a.num_pages = kv.num_pages;
  a.batch = batch;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.seq_lens = seq_lens;
  a.sink = sink_tokens;
  a.recent = recent_tokens;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.out = out;
  a.out_lse = out_lse;
  const size_t rows = (size_t)p.heads * group;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.arrivals = reinterpret_cast<uint32_t*>(ws);
  a.joins = reinterpret_cast<int2*>(ws + kArrivalBytes);
  a.o_part = reinterpret_cast<float*>(ws + kCounterBytes);
  a.lse_part = a.o_part + 2 * kMaxCtas * rows * kv.head_dim;
  a.err = err;
  a.deferred = p.deferred;
  switch (kv.head_dim) {
    case 64: return launch<64>(kmap, vmap, a, grid, stream);
    case 128: return launch<128>(kmap, vmap, a, grid, stream);
    default: return launch<256>(kmap, vmap, a, grid, stream);
  }
}

}  // namespace se
