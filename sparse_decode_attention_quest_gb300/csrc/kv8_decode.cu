// Attention of one new token per request over its whole 8-bit paged cache, or over its
// first sink and last recent tokens: se_paged_decode's computation with rows that are
// e4m3 codes, 16 tokens of a page and one KV head to a scale:
//
//     z_j = sm_scale s_k(page of j) q . c_j over the kept positions j < L,
//     out = sum_j exp(z_j - m) s_v(page of j) d_j / l,  l = sum_j exp(z_j - m),  lse = m + log l.
//
// The floor is the time of the codes from HBM, half that of the bf16 cache, and the
// share-out of the work, the joins and the ring of TMA boxes are its (paged_decode.cu). What
// differs is what has to happen to twice as many rows in the same time:
//
//  * Codes become fp16 (exact) on their way from shared memory, two conversions a word, and both products
//    are m16n8k16 fp16 MMAs. Neither operand's order matters as long as both have it: K's words keep
//    four dims of a token together, so Q^T is loaded in that order; V's, transposed as bytes, four tokens of a dim, so
//    P^T has them in that order, which the rows of K and V are read in such orders for (and without bank
//    conflicts): no bytes are moved in registers. (m16n8k32 e4m3 MMAs on K's codes as they lie, the query split into
//    two e4m3 numbers a dim, were slower: 454 instructions a block of 16 tokens and one head, 691 us for 3.2 GB.)
//  * A query row is scaled by a power of two to at most 448 and held as fp16: exact for dims down to 2^-24 of the
//    row's largest magnitude, within 2^-32 of it below (2^-125 where the power of two is the least, 2^-100).
//  * V's scales go into the weights before they are rounded to fp16: a weight enters as
//    w_j = exp2(z_j - m + log2 s_v - d + 14), with m + d a reference of their product's maximum, so that it is rounded
//    by half a step of 2^-11 down to 2^-28 of the largest, whatever the scales of pages that carry no weight. The
//    sum l takes the same exponentials, times exp2(d - log2 s_v - 14) for each page.
//  * m and m + d need not be the maxima: a weight may reach 2^15.9. A page whose weights stay below costs no exchange
//    between lanes, just a vote; any other (the first ones, mostly) moves both references to the maxima, and
//    the sums follow.
//  * A warp takes two pages at once where its registers allow: two independent chains of products.
//  * Scales travel with their slot: a 4-byte asynchronous copy per (page, head) that arrives on the slot's barrier.
//  * Rows that are not kept: their logits become -inf, and their value rows are
//    zeroed in shared memory first, since 0 * NaN is not 0.
#include <algorithm>

#include "se_kv8.cuh"
#include "se_paged_join.cuh"

namespace se {
namespace {

constexpr int kSlotBytes = 32 * 1024;
constexpr int kMetaRing = 4;     // steps whose page masks are held (at most three are in flight)
constexpr int kMaxPages = 32;    // pages of a step
constexpr int kMaxBatch = 4096;  // requests whose prefix fits beside the ring
constexpr float kWeightTop = 14.f;    // log2 of the weight at the reference
constexpr float kWeightMost = 15.9f;  // log2 of the largest weight, within fp16
constexpr float kLowest = -3.4e38f;   // m and d before any logit
constexpr int kLaunchRegs = 168;      // a thread's: a kernel that moves registers between warps gets as many as it may have
constexpr int kDown = 8;              // joins: up to 2^8 partials whose sum may pass fp32's largest
static_assert(kMaxCtas <= 1 << kDown, "an item has no more partials than CTAs");

// Four warps issue the boxes, every fourth page each: a warp takes some 65 clocks to issue one and 35 more per KB, so
// that one warp alone kept boxes of 1 KB to 48% of the copy rate and of 2 KB to 72% (32 x 32K tokens of one head: 64 dims,
// 0.13 GB, 49 us, so 31; 128 dims, 0.27 GB, 61 and 51; 32 x 16K tokens of 5 heads of 128 dims, 0.67 GB: 133 and 108).
//
// kMany: the kernel for many query heads per KV head. The twelve warps have 168 registers a thread at launch; here those of
// the issuers go to the consumers, for tiles of sixteen heads (256 dims: eight) and two pages at once, which 128 dims still
// spill 44 bytes a thread for and 256 dims 8 (64 x 16K tokens, 0.27 GB, 32 heads of 128 dims over one: 118 us before, 99
// so; 64: 201 and 166; 32 x 16K tokens, 0.27 GB, 16 over each of 4 of 64 dims: 80 and 72; 0.54 GB, 12 over each of 2 of
// 256 dims: 124 and 105). What bounds it is the time of the MMAs (8 clocks each) with the conversions, which hardly
// overlap.
template <int kD, bool kMany>
struct Cfg {
  static constexpr int kWarps = 8;  // consumers
  static constexpr int kConsumers = kWarps * 32;
  static constexpr int kIssuers = 4;
  static constexpr int kProducers = kIssuers * 32;
  static constexpr int kThreads = kConsumers + kProducers;
  static constexpr int kProducerRegs = 56, kConsumerRegs = 224;  // kMany: a thread's, of kLaunchRegs at launch
  // A consumer waits for registers that the launch does not have forever.
  static_assert(kProducerRegs * kProducers + kConsumerRegs * kConsumers <= kLaunchRegs * kThreads, "the shares");
  static_assert(kLaunchRegs * kThreads <= 65536, "registers of a launch");
  static constexpr int kSlots = kD == 256 ? 4 : 5;
  static constexpr int kBlocks = kSlotBytes / (kPageSize * kD);  // (page, head) blocks of a slot
  static constexpr int kStageFloats = kWarps * 8 * kD;           // states handed over at a segment's end
  static constexpr int kFixed = 1024 + kSlots * kSlotBytes + kStageFloats * 4 + kWarps * 8 * 4 +
                                kMetaRing * kMaxPages * 4 + kSlots * kBlocks * 4 + 2 * kSlots * 8 + 64;
  static constexpr int kMaxSmem = kFixed + kept_ints(kMaxBatch) * 4;
};

// Pages that a warp takes at once, and column tiles of eight query heads that it has.
__host__ __device__ constexpr int pages_at_once(int head_dim, bool many) {
  return many || head_dim == 128 ? 2 : head_dim == 64 ? 4 : 1;
}
__host__ __device__ constexpr int tiles_at_once(int head_dim, bool many) { return many && head_dim <= 128 ? 2 : 1; }

// The order in which the MMAs have a page's 16 tokens: row i of S^T is token k_row(i); V's rows are read as v_row(0),
// v_row(1) .., and a lane's word of them is tokens v_row(4 t) .. v_row(4 t + 3). The transposes of P^T put rows 2 t and
// 2 t + 1 of S^T's upper half into the first two of these places and of its lower half into the others, so
//     k_row(2 t + j) = v_row(4 t + j),  k_row(8 + 2 t + j) = v_row(4 t + 2 + j),  j = 0, 1,
// and any eight rows that are read at once have all residues modulo 8, which the swizzle spreads over all banks.
__device__ __forceinline__ int k_row(int i) { return i < 8 ? i : 8 + (i & 7 ^ 4); }
__device__ __forceinline__ int v_row(int i) { return k_row((i >> 2) * 2 + (i & 1) + (i & 2) * 4); }

// Byte offset of 16-byte chunk c of a block's row r: lines of 128 bytes, swizzled, `plane` bytes between the lines'
// first and second 128 bytes of a row; two rows of 64 dims share a line.
template <int kD>
__device__ __forceinline__ uint32_t row_chunk(int r, int c, uint32_t plane) {
  if constexpr (kD == 64) return swz128(r >> 1, (r & 1) * 4 + c);
  return (c >> 3) * plane + swz128(r, c & 7);
}

// A page's mask with its top bit set where all tokens are kept.
constexpr uint32_t kWhole = 0x80000000u;
__device__ __forceinline__ uint32_t tagged(uint32_t mask) { return mask_is_full(mask) ? mask | kWhole : mask; }

struct Kv8Args {
  const float* k_scale;
  const float* v_scale;
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

// kSolo: no two warps share a (head, tile) (code of its own: as a branch
// beside the other it cost that one 0.8 us of 9.9).
template <int kD, bool kMany, bool kSolo>
__global__ void __maxnreg__(kLaunchRegs) kv8_decode_kernel(const __grid_constant__ CUtensorMap kmap,
                                                           const __grid_constant__ CUtensorMap vmap,
                                                           const Kv8Args a) {
  using C = Cfg<kD, kMany>;
  constexpr int kSlots = C::kSlots, kNt = tiles_at_once(kD, kMany), kPp = pages_at_once(kD, kMany);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* stage = reinterpret_cast<float*>(ring + kSlots * kSlotBytes);  // [warps][8][D]
  float* lses = stage + C::kStageFloats;                                // [warps][8], log2 domain
  uint32_t* meta = reinterpret_cast<uint32_t*>(lses + C::kWarps * 8);   // [kMetaRing][kMaxPages]
  float* scales = reinterpret_cast<float*>(meta + kMetaRing * kMaxPages);  // [kSlots][kBlocks]
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + kSlots * C::kBlocks);
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
      mbar_init(&full[s], C::kIssuers + 32);  // each issuer's boxes, and each lane's scales of the last one
      mbar_init(&empty[s], active);
    }
    mbar_fence_init();
  }
  if (warp == C::kWarps && lane == 0) {
    tma_prefetch_map(&kmap);
    tma_prefetch_map(&vmap);
  }
  pdl_enter();
  // Pieces of a step: up to 32 partials an item, rather than two steps for a CTA (1 x 4K tokens, 4 heads over one: 9.5 us,
  // 10.6 in eights; 32 over 8: 10.5 and 13.2).
  const int piece = kept_prefix<C::kThreads>(a.seq_lens, a.batch, HG, a.bt_stride, a.sink, a.recent, Pg, Pg,
                                             32, gridDim.x, kMaxPlaces / HG, prefix, lens,
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

  if (warp >= C::kWarps) {
    // ------------------------------------------------------------ TMA producers: all go through all steps; the first
    // writes the masks, the last copies the scales
    if constexpr (kMany) set_max_registers<C::kProducerRegs, false>();
    const int issuer = warp - C::kWarps;
    const uint64_t policy = l2_evict_first_policy();
    const uint32_t page_bytes = (uint32_t)heads * kPageSize * kD;
    const int my_page = lane / heads, my_head = lane - my_page * heads;  // the block whose scales this lane copies
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
        const bool issues = ok && lane % C::kIssuers == issuer;
        if (mine && !ok) raise_error(a.err, SE_DEVERR_PAGE_RANGE);
        const int block_page = __shfl_sync(0xffffffffu, ok ? phys : -1, my_page);
        const bool scaled = lane < Pg * heads && block_page >= 0 && issuer == C::kIssuers - 1;
        const size_t block = (size_t)max(block_page, 0) * a.num_kv_heads + seg.group * heads + my_head;
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, issues)) * page_bytes;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++j) {
          const int s = j % kSlots;
          if (lane == 0 && j >= kSlots && !mbar_wait(&empty[s], (j / kSlots - 1) & 1)) dead = true;
          dead = __shfl_sync(0xffffffffu, (int)dead, 0) != 0;
          if (dead) break;
          if (kv == 0 && lane < Pg && issuer == 0)
            meta[(step % kMetaRing) * kMaxPages + lane] = ok ? tagged(page_mask(k, a.sink, k.logical(i))) : 0u;
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
          __syncwarp();
          if (issues)
            tma_load_3d(ring + s * kSlotBytes + lane * page_bytes, kv ? &vmap : &kmap, 0,
                        (phys * a.num_kv_heads + seg.group * heads) * (kPageSize * min(kD, 128) / 128), 0, &full[s],
                        policy);
          if (scaled) cp_async_4(smem_addr(scales + s * C::kBlocks + lane), (kv ? a.v_scale : a.k_scale) + block);
          if (issuer == C::kIssuers - 1) mbar_arrive_copies(&full[s]);
        }
      }
    }
    // Every copy has landed before the CTA leaves.
    cp_async_wait_all();
    if (lane == 0) {
      for (int u = max(0, j - kSlots); u < j; ++u)
        if (!mbar_wait(&full[u % kSlots], (u / kSlots) & 1)) dead = true;
      if (dead) raise_error(a.err, SE_DEVERR_WAIT_TIMEOUT);
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  if constexpr (kMany) set_max_registers<C::kConsumerRegs, true>();
  const bool works = warp < active;
  const int combo = warp % combos, replica = warp / combos;
  const int hc = combo / a.mtiles, mt = combo % a.mtiles;
  const int g = lane >> 2, t = lane & 3;
  const int tile_head = mt * 8 * kNt;  // first query head of the tile, in its KV head's group
  const uint32_t ring0 = smem_addr(ring);
  const uint32_t plane = (uint32_t)heads * kPageSize * 128;  // 128 dims of a page's rows
  const uint32_t page_bytes = (uint32_t)heads * kPageSize * kD;
  // Of ldmatrix: 16 rows, two chunks.
  const uint32_t off_k = row_chunk<kD>(k_row(lane & 15), lane >> 4, plane);
  const uint32_t off_v = row_chunk<kD>(v_row(lane & 15), lane >> 4, plane);
  int sk = 0, step = 0;   // K's slot of the step, and the parity of its use
  uint32_t phase = 0;
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
    // Q^T as the B operand: head g of each column tile, dims 4 t, 4 t + 1 and the next two of each sixteen.
    uint32_t qb[kD / 16][kNt][2];
    float zf[kNt][2];  // what turns the products of heads 2 t and 2 t + 1 into logits in base 2, but for K's scale
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      const int hd = tile_head + nt * 8 + g;
      const bool real = works && hd < G;
      const int row = (seg.group * heads + hc) * G + (real ? hd : 0);
      const uint16_t* qr = a.q + (size_t)seg.b * a.q_stride + (size_t)row * kD + 4 * t;
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < kD / 16; ++i) {
        const uint2 x = real ? *reinterpret_cast<const uint2*>(qr + i * 16) : make_uint2(0u, 0u);
        qb[i][nt][0] = x.x;
        qb[i][nt][1] = x.y;
        top = max_abs_nan_bf16x2(max_abs_nan_bf16x2(top, x.x), x.y);
      }
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) top = max_abs_nan_bf16x2(top, __shfl_xor_sync(0xffffffffu, top, x));
      top = max(top & 0xffffu, top >> 16);
      // A row that is not finite is NaN throughout.
      const float qs = scale_for(top < 0x7f80u ? top : 0u), inv = top < 0x7f80u ? fast_rcp(qs) : NAN;
#pragma unroll
      for (int i = 0; i < kD / 16; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          qb[i][nt][k] = pack_f16x2(bf16_lo(qb[i][nt][k]) * inv, bf16_hi(qb[i][nt][k]) * inv);
      zf[nt][0] = __shfl_sync(0xffffffffu, qs, 8 * t) * a.scale_log2;
      zf[nt][1] = __shfl_sync(0xffffffffu, qs, 8 * t + 4) * a.scale_log2;
    }
    // O^T: dims 16 i + g (0, 1) and 8 more (2, 3), heads 2 t and 2 t + 1 of each column tile, times
    // 2^(14 - m - d); m, d and l (times 2^-m, the thread's tokens only) of those heads.
    float o[kD / 16][kNt][4], m[kNt][2], d[kNt][2], l[kNt][2];
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
#pragma unroll
      for (int i = 0; i < kD / 16; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
      m[nt][0] = m[nt][1] = d[nt][0] = d[nt][1] = kLowest;
      l[nt][0] = l[nt][1] = 0.f;
    }

    for (int i0 = seg.lo; i0 < seg.hi && works; i0 += Pg, ++step) {
      const bool wraps = sk + 1 == kSlots;
      const int sv = wraps ? 0 : sk + 1;
      const uint32_t phase_v = phase ^ (uint32_t)wraps;
      if (!dead && !__all_sync(0xffffffffu, mbar_wait(&full[sk], phase))) dead = true;
      const uint32_t* masks = meta + (step % kMetaRing) * kMaxPages;
      bool v_here = false, zeroed = false;
      for (int pg0 = replica; pg0 < Pg; pg0 += kPp * a.replicas) {
        uint32_t mask[kPp], at[kPp];  // the page's kept tokens, and where its block begins in its slot
        int blk[kPp];
        bool any = false;
#pragma unroll
        for (int u = 0; u < kPp; ++u) {
          const int pg = pg0 + u * a.replicas;
          mask[u] = dead || pg >= Pg ? 0u : masks[pg];
          blk[u] = pg * heads + hc;
          at[u] = pg * page_bytes + hc * (kPageSize * min(kD, 128));
          any = any || mask[u];
        }
        if constexpr (kPp > 1) {
          // A page that is not there is another one over again, without a weight.
          int there = 0, there_at = 0;
#pragma unroll
          for (int u = kPp - 1; u >= 0; --u)
            if (mask[u]) there = blk[u], there_at = at[u];
#pragma unroll
          for (int u = 0; u < kPp; ++u)
            if (!mask[u]) blk[u] = there, at[u] = there_at;
        }
        const bool last = pg0 + kPp * a.replicas >= Pg;
        uint32_t all = kWhole;
#pragma unroll
        for (int u = 0; u < kPp; ++u) all &= mask[u];
        const bool whole = all != 0;
        // Products, then logits in base 2, of tokens k_row(g) (0, 1) and k_row(g + 8) (2, 3), heads 2 t and 2 t + 1.
        constexpr int kAcc = kPp * kNt == 1 ? 2 : 1;  // accumulators of a page's products where there is no other chain
        float s[kPp][kNt][4], more[kPp][kNt][4];
        if (any) {
#pragma unroll
          for (int u = 0; u < kPp; ++u)
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[u][nt][e] = more[u][nt][e] = 0.f;
#pragma unroll
          for (int c = 0; c < kD / 32; ++c) {
#pragma unroll
            for (int u = 0; u < kPp; ++u) {
              // The swizzle is an exclusive or of the 16-byte chunk with the line: two chunks further is one of bit 5 on.
              uint32_t r[4], lo[4], hi[4];
              ldmatrix_x4(r[0], r[1], r[2], r[3],
                          ((ring0 + sk * kSlotBytes + at[u] + off_k) ^ ((c & 3) << 5)) + (c >> 2) * plane);
#pragma unroll
              for (int k = 0; k < 4; ++k) e4m3x4_to_f16(r[k], lo[k], hi[k]);
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int nt = 0; nt < kNt; ++nt)
                  mma_f16_16816(kAcc == 2 && k ? more[u][nt] : s[u][nt], lo[2 * k], lo[2 * k + 1], hi[2 * k],
                                hi[2 * k + 1], qb[2 * c + k][nt][0], qb[2 * c + k][nt][1]);
            }
          }
#pragma unroll
          for (int u = 0; u < kPp; ++u) {
            // Both factors at once: the products times the query's alone pass fp32 where K's scale brings logits back.
            // Rounded here, not in a fused subtraction of a maximum: equal logits stay equal, however large.
            const float ks = scales[sk * C::kBlocks + blk[u]];
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                s[u][nt][e] = __fmul_rn(kAcc == 2 ? s[u][nt][e] + more[u][nt][e] : s[u][nt][e], zf[nt][e & 1] * ks);
            if (!whole) {
              const bool k0 = in_mask(mask[u] & ~kWhole, g), k1 = in_mask(mask[u] & ~kWhole, k_row(g + 8));
#pragma unroll
              for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[u][nt][e] = (e < 2 ? k0 : k1) ? s[u][nt][e] : -INFINITY;
            }
          }
        }
        if (last) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[sk]);
        }
        if (!v_here) {
          if (!dead && !__all_sync(0xffffffffu, mbar_wait(&full[sv], phase_v))) dead = true;
          v_here = true;
        }
        if (any && !dead) {
          float vs[kPp], x[kPp][kNt][4], lg[kPp][kNt][2];
          bool moved = false;
#pragma unroll
          for (int u = 0; u < kPp; ++u) {
            vs[u] = fast_log2(scales[sv * C::kBlocks + blk[u]]);
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float w = vs[u] + kWeightTop - d[nt][e];
                x[u][nt][e] = s[u][nt][e] - m[nt][e] + w;
                x[u][nt][2 + e] = s[u][nt][2 + e] - m[nt][e] + w;
                // l's exponentials over the weights; beyond 2^60 (a V scale far below the others') they have their own.
                lg[u][nt][e] = fast_exp2(-w);
                moved = moved || !(fmaxf(x[u][nt][e], x[u][nt][2 + e]) <= kWeightMost) || w < -60.f;
              }
          }
          if (__any_sync(0xffffffffu, moved)) {
            // References to the maxima; the sums follow. l takes its own exponentials here.
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float top = m[nt][e];
#pragma unroll
                for (int u = 0; u < kPp; ++u) top = fmaxf(top, fmaxf(s[u][nt][e], s[u][nt][2 + e]));
#pragma unroll
                for (int i = 4; i < 32; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
                const float back = m[nt][e] - top;
                float over = fmaxf(d[nt][e] + back, kLowest);
#pragma unroll
                for (int u = 0; u < kPp; ++u) over = fmaxf(over, fmaxf(s[u][nt][e], s[u][nt][2 + e]) - top + vs[u]);
#pragma unroll
                for (int i = 4; i < 32; i <<= 1) over = fmaxf(over, __shfl_xor_sync(0xffffffffu, over, i));
                const float f = fast_exp2(back + (d[nt][e] - over));
                l[nt][e] *= fast_exp2(back);
                m[nt][e] = top;
                d[nt][e] = over;
#pragma unroll
                for (int i = 0; i < kD / 16; ++i) {
                  o[i][nt][e] *= f;
                  o[i][nt][2 + e] *= f;
                }
#pragma unroll
                for (int u = 0; u < kPp; ++u) {
                  const float z0 = s[u][nt][e] - top, z1 = s[u][nt][2 + e] - top, w = vs[u] + kWeightTop - over;
                  x[u][nt][e] = z0 + w;
                  x[u][nt][2 + e] = z1 + w;
                  l[nt][e] += fast_exp2(z0) + fast_exp2(z1);
                  lg[u][nt][e] = 0.f;
                }
              }
          }
          uint32_t pb[kPp][kNt][2];
#pragma unroll
          for (int u = 0; u < kPp; ++u)
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) {
              const float w0 = fast_exp2(x[u][nt][0]), w1 = fast_exp2(x[u][nt][1]);
              const float w2 = fast_exp2(x[u][nt][2]), w3 = fast_exp2(x[u][nt][3]);
              l[nt][0] = fmaf(lg[u][nt][0], w0 + w2, l[nt][0]);
              l[nt][1] = fmaf(lg[u][nt][1], w1 + w3, l[nt][1]);
              // Weights meet V as fp16 (half a step, 2^-11 of each); l sums them unrounded.
              pb[u][nt][0] = transpose_8x8_b16(pack_f16x2(w0, w1));
              pb[u][nt][1] = transpose_8x8_b16(pack_f16x2(w2, w3));
            }
          if (!whole) {
#pragma unroll
            for (int u = 0; u < kPp; ++u) {
              if (!mask[u] || (mask[u] & kWhole)) continue;
              // Stale rows may hold NaN: zero them (two lanes per row).
              const int r = lane >> 1;
              if (!in_mask(mask[u], r))
                for (int c = lane & 1; c < kD / 16; c += 2)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                   ring0 + sv * kSlotBytes + at[u] + row_chunk<kD>(r, c, plane)),
                               "r"(0u)
                               : "memory");
              zeroed = true;
            }
            __syncwarp();
          }
#pragma unroll
          for (int c = 0; c < kD / 32; ++c) {
#pragma unroll
            for (int u = 0; u < kPp; ++u) {
              // Two chunks of 16 dims: four tokens of dims g and g + 8 of each.
              uint32_t r[4], lo[4], hi[4];
              ldmatrix_x2_trans_b8(r[0], r[1], r[2], r[3],
                                   ((ring0 + sv * kSlotBytes + at[u] + off_v) ^ ((c & 3) << 5)) + (c >> 2) * plane);
#pragma unroll
              for (int k = 0; k < 4; ++k) e4m3x4_to_f16(r[k], lo[k], hi[k]);
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int nt = 0; nt < kNt; ++nt)
                  mma_f16_16816(o[2 * c + k][nt], lo[2 * k], lo[2 * k + 1], hi[2 * k], hi[2 * k + 1], pb[u][nt][0],
                                pb[u][nt][1]);
            }
          }
        }
      }
      if (zeroed) fence_proxy_async_smem();  // before the next copy into the slot
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[sv]);
      sk = sv + 1 == kSlots ? 0 : sv + 1;
      phase = phase_v ^ (uint32_t)(sk == 0);
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
        // The average over the warp's own tokens (values near fp32's largest have no sum), 2^3 lower where it meets those
        // of up to 2^3 warps.
        const bool none = l[nt][e] == 0.f;
        const float inv = none ? 0.f : fast_rcp(l[nt][e]);
        const float f = fast_exp2(d[nt][e] - (kSolo ? kWeightTop : kWeightTop + 3.f));
        const float lse2 = none ? -INFINITY : m[nt][e] + fast_log2(l[nt][e]);
        if (kSolo && g == 0 && tile_head + nt * 8 + hd < G) {
          // No other states: the row is final.
          const int r = hc * G + tile_head + nt * 8 + hd;
          if (split)
            a.lse_part[part_row0 + r] = lse2;
          else if (a.out_lse)
            a.out_lse[out_row0 + r] = lse2 * kLn2;
        }
#pragma unroll
        for (int i = 0; i < kD / 16; ++i) {
          dst[stage_at<kD>(hd, 16 * i + g)] = kSolo && none && !split ? 0.f : o[i][nt][e] * inv * f;
          dst[stage_at<kD>(hd, 16 * i + g + 8)] = kSolo && none && !split ? 0.f : o[i][nt][2 + e] * inv * f;
        }
        if (!kSolo && g == 0) lses[warp * 8 + hd] = lse2;
      }
      const int hds = min(8, G - tile_head - nt * 8);
      const size_t r0 = hc * G + tile_head + nt * 8;
      if constexpr (kSolo) {
        __syncwarp();
#pragma unroll 1
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
#pragma unroll 1
      for (int e = replica * 32 + lane; e < hds * (kD / 4); e += threads) {
        const int d = e % (kD / 4) * 4, hd = e / (kD / 4);
        float M = -INFINITY;
        for (int w = combo; w < active; w += combos) M = fmaxf(M, lses[w * 8 + hd]);
        const float base = finite_base(M);
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = combo; w < active; w += combos) {
          const float f = fast_exp2(lses[w * 8 + hd] - base);
          sum += f;
          const float4 v = *reinterpret_cast<const float4*>(stage + w * 8 * kD + stage_at<kD>(hd, d));
          acc = make_float4(acc.x + f * v.x, acc.y + f * v.y, acc.z + f * v.z, acc.w + f * v.w);
        }
        const bool none = sum == 0.f;
        const float inv = none ? 0.f : 8.f * fast_rcp(sum), lse2 = none ? -INFINITY : M + fast_log2(sum);
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        const size_t r = r0 + hd;
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
  static_assert(sizeof(JoinSmem<kD, C::kWarps>) <= (C::kStageFloats + C::kWarps * 8) * 4, "the join's sums fit");
#pragma unroll 1
  for (int s = 0; s < 2; ++s) {
    if (!flags[s]) continue;
    const int first = s ? (int)blockIdx.x : first0, parts = s ? parts1 : parts0, item = flags[2 + s];
    const int warps = min(C::kWarps, share_of(parts));
    for (int r0 = 0; r0 < rows; r0 += C::kWarps / warps)
      join_rows<kD, C::kWarps, 4, true, kDown>(a.o_part, a.lse_part, first, parts, item, rows, r0, warps, *join_smem,
                                               a.out, a.out_lse, [] { named_bar_sync(1, C::kConsumers); });
  }
}

// How the heads of a call are laid over the consumer warps, and where its joins run.
struct HeadPlan {
  int heads, head_groups, mtiles, replicas, step_pages;
  bool deferred;
};

// Query heads per KV head from which the kernel for many is taken: 64 and 256 dims 9, 128 dims 17 (16 over each of 4, 16 x
// 16K tokens, 0.27 GB: 65 us against 68; but 32 requests of 2K tokens 30 against 28).
bool takes_many(int head_dim, int group) { return group > (head_dim == 128 ? 16 : 8); }

// The KV heads of a box, up to `most_heads`: the count for which most warps have pages, the larger of two alike (32 x
// 16K tokens: 5 heads of 64 dims, 0.34 GB, one to a box 61 us, five 86; 3 heads of 128 dims, 0.40 GB, 71 and 75). A
// warp's pages are whole sets of those it takes at once.
HeadPlan head_plan(int num_kv_heads, int group, int head_dim, int most_heads) {
  const int warps = Cfg<128, false>::kWarps, blocks = kSlotBytes / (kPageSize * head_dim);
  const bool many = takes_many(head_dim, group);
  const int once = pages_at_once(head_dim, many), tile = 8 * tiles_at_once(head_dim, many);
  HeadPlan p;
  p.mtiles = (group + tile - 1) / tile;
  int best = 0;
  for (int c = 1; c <= most_heads && c * p.mtiles <= warps; ++c) {
    if (num_kv_heads % c) continue;
    const int r = warps / (c * p.mtiles);
    int each = blocks / c / r;
    if (each > once) each -= each % once;
    if (each == 0 || c * p.mtiles * r < best) continue;
    best = c * p.mtiles * r;
    p.heads = c;
    p.replicas = r;
    p.step_pages = each * r;
  }
  p.head_groups = num_kv_heads / p.heads;
  p.deferred = true;
  return p;
}

// Largest boxes of which an item's partials, counted in slices of the least length over the table's (or the windows')
// width, have no more than 32 KB, so that the decode kernel joins them itself without delay; otherwise no more than 48
// KB; otherwise the largest of all and a second kernel (48 windows of 1,064 tokens, 32/4 heads: 21.6 us, 22.6 with 48 KB
// alone; 8 requests of 4K tokens, 64/8 heads of 64 dims: 15.6, 19.1, with 192 KB 34.3; but 1 request of 8K tokens, 32/8
// heads: 12.0, 14.8 with 32 KB alone). More items than two to a CTA are not made for that: 300 requests of up to 1,000
// tokens, 32/4 heads: 45 us, 63 in boxes of one head.
HeadPlan call_plan(int num_kv_heads, int group, int head_dim, int32_t bt_stride, int32_t sink_tokens,
                   int32_t recent_tokens, int batch, int ctas) {
  long long width = bt_stride;
  if (recent_tokens > 0)
    width = std::min(width, ((long long)sink_tokens + kPageSize - 1) / kPageSize + recent_tokens / kPageSize + 2);
  for (const int most : {32 * 1024, 48 * 1024})
    for (int c = 8; c > 0;) {
      HeadPlan p = head_plan(num_kv_heads, group, head_dim, c);
      if (c < 8 && (long long)batch * p.head_groups > 2 * ctas) break;
      const long long parts = std::min<long long>(ctas, (width + p.step_pages) / (2 * p.step_pages + 1) + 2);
      p.deferred = parts * p.heads * group * head_dim * (long long)sizeof(float) > most;
      if (!p.deferred) return p;
      c = p.heads - 1;
    }
  return head_plan(num_kv_heads, group, head_dim, 8);
}

int ctas_of(int sm_count) { return sm_count < kMaxCtas ? sm_count : kMaxCtas; }

template <int kD, bool kMany, bool kSolo>
cudaError_t launch_as(const CUtensorMap& kmap, const CUtensorMap& vmap, const Kv8Args& a, int grid,
                   cudaStream_t stream) {
  using C = Cfg<kD, kMany>;
  const size_t smem = C::kFixed + kept_ints(a.batch) * 4;
  static_assert(C::kMaxSmem <= 227 * 1024, "the largest batch fits");
  static std::atomic<uint64_t> allowed{0};
  if (kMany && !allowed.load(std::memory_order_acquire)) {
    // Were it built with fewer registers after all, no launch would end.
    cudaFuncAttributes at;
    const cudaError_t e = cudaFuncGetAttributes(&at, kv8_decode_kernel<kD, kMany, kSolo>);
    if (e != cudaSuccess) return e;
    if (at.numRegs * C::kThreads < C::kProducerRegs * C::kProducers + C::kConsumerRegs * C::kConsumers)
      return cudaErrorInvalidConfiguration;
  }
  cudaError_t e = allow_smem(kv8_decode_kernel<kD, kMany, kSolo>, C::kMaxSmem, allowed);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kv8_decode_kernel<kD, kMany, kSolo>, dim3(grid), dim3(C::kThreads), smem, stream, kmap, vmap, a);
  if (e != cudaSuccess || !a.deferred) return e;
  const int rows = a.heads * a.group;
  // An item has at most `rows` units, and no more items than CTAs reach beyond a slice.
  const int units = std::min(grid, a.batch * a.head_groups) * rows;
  return launch_pdl(paged_join_kernel<kD, kDown>, dim3(std::min(units, 8 * grid)), dim3(kJoinWarps * 32), 0, stream,
                    a.o_part, a.lse_part, a.joins, grid, rows, a.out, a.out_lse);
}

template <int kD>
cudaError_t launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const Kv8Args& a, int grid,
                   cudaStream_t stream) {
  const bool solo = a.replicas == 1;
  if (takes_many(kD, a.group))
    return solo ? launch_as<kD, true, true>(kmap, vmap, a, grid, stream)
                : launch_as<kD, true, false>(kmap, vmap, a, grid, stream);
  return solo ? launch_as<kD, false, true>(kmap, vmap, a, grid, stream)
              : launch_as<kD, false, false>(kmap, vmap, a, grid, stream);
}

}  // namespace

int kv8_decode_max_batch() { return kMaxBatch; }

bool kv8_decode_supported(int num_kv_heads, int head_dim, int num_q_heads) {
  return (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
         num_q_heads / num_kv_heads <= 64;
}

int kv8_decode_box_heads(int num_kv_heads, int num_q_heads, int head_dim, int32_t bt_stride, int32_t sink_tokens,
                         int32_t recent_tokens, int batch, int sm_count) {
  return call_plan(num_kv_heads, num_q_heads / num_kv_heads, head_dim, bt_stride, sink_tokens, recent_tokens, batch,
                   ctas_of(sm_count)).heads;
}

size_t kv8_decode_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  const HeadPlan p = head_plan(num_kv_heads, num_q_heads / num_kv_heads, head_dim, 8);  // the most rows of an item
  const size_t rows = (size_t)p.heads * (num_q_heads / num_kv_heads);
  return kCounterBytes + 2 * kMaxCtas * rows * (head_dim + 1) * sizeof(float);
}

cudaError_t launch_kv8_decode(const CUtensorMap& kmap, const CUtensorMap& vmap, const Kv8View& kv, const uint16_t* q,
                                long long q_stride, int32_t num_q_heads, const int32_t* block_table,
                                int32_t bt_stride, const int32_t* seq_lens, int32_t batch, int32_t sink_tokens,
                                int32_t recent_tokens, float sm_scale, uint16_t* out, float* out_lse, void* workspace,
                                int sm_count, unsigned* err, cudaStream_t stream) {
  const int group = num_q_heads / kv.num_kv_heads;
  const int grid = ctas_of(sm_count);
  const HeadPlan p = call_plan(kv.num_kv_heads, group, kv.head_dim, bt_stride, sink_tokens, recent_tokens, batch, grid);
  Kv8Args a;
  a.k_scale = kv.k_scale;
  a.v_scale = kv.v_scale;
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
