// Attention of one new token per request over its whole latent (MLA-style)
// paged cache, or over its first sink and last recent tokens (SparseEngine:
// Sparse-First Inference Engine, Figure 5 caption: an MLA model decoding at
// 32K/128K; Table 7: logit z and weight alpha; Tables 9-12: sink and recent).
//
// One cache row per token holds 576 dims (512 latent + 64 RoPE) and is the key;
// its first 512 dims are the value; all query heads (16..64) share it:
//     z_hj = sm_scale q_h . k_j,  out_h = sum_j softmax(z_h)_j k_j[0:512].
// A kept row (1152 bytes) is read once. With 64 heads it takes 139 kflop, 121
// flops a byte: at the copy rate a third of the tensor cores' time at full rate,
// but the products are small (64 heads) and bound by shared-memory reads: a
// 64-token tile takes 1200 clocks for S^T and 870 for PV measured alone, of the
// 3150 that its 72 KB take at the rate at which the 128-dim caches are read (7.1
// TB/s over 152 SMs at 2.07 GHz). So both must overlap the copies, and a tile's
// softmax must be short.
//
//  * Work: the requests follow one another on a line, each as long as its kept
//    pages and an overhead, which the CTAs share equally in tiles of 64 tokens (4
//    pages). An item that spans CTAs leaves a partial per CTA (at most two per
//    CTA, whatever the lengths), and a second kernel joins them. Batches that would
//    leave CTAs without work are cut into one or two tiles per CTA.
//  * A tile is eight groups of 8 rows, each group nine 64-dim chunks of 8 rows x
//    128 bytes, 128-byte swizzled: one 3-D TMA box per group. The queries (72 KB)
//    leave room for two tiles, 144 KB, which must cover the copies' latency as
//    well as the two products and the softmax: so the boxes of the tiles to come
//    are prefetched into L2 kPrefetch tiles ahead.
//  * S^T = K Q^T: M = 64 tokens, N = heads, 36 K steps in two accumulators; the
//    tile is the K-major A operand, the queries are B. O^T += V^T P^T: four M = 128
//    products per 16 tokens, A = the tile's first 512 dims read MN-major, B = P read
//    MN-major. Two warps issue S^T and one PV, all lanes converged with an elected
//    issuer: a lone lane's code moves every descriptor to the uniform registers
//    first and issues an S^T product every 49 clocks instead of 35. (One warp for
//    all products, PV first, was slower: 436 against 416 us for 64 x 32K tokens;
//    so was releasing a tile page by page, whose commits cost more than the earlier
//    copies gained.) The second S^T warp gained 16 us, logits scaled and shifted
//    in one FMA 20 us: 392 us.
//  * Eight softmax warps read S^T from TMEM (a thread one token x 16 heads), keep
//    a running maximum per head that moves only when a tile exceeds it by 2^8
//    (then the heads' output columns are rescaled in TMEM), and write P as bf16
//    over the tile's RoPE chunks, which S^T no longer needs.
//  * Rows that are not kept: logits -inf, value dims zeroed in shared memory.
#include <algorithm>

#include "se_paged.cuh"

namespace se {
namespace {

constexpr int kD = 576;
constexpr int kDv = 512;
constexpr int kChunks = kD / 64;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kTileTok = 64;
constexpr int kTilePages = kTileTok / kPageSize;
constexpr int kGroupRows = 8;                           // rows of a copy group (half a page)
constexpr int kChunkBytes = kGroupRows * 128;
constexpr int kGroupBytes = kChunks * kChunkBytes;      // 9 KB: one TMA box
constexpr int kStageBytes = (kTileTok / kGroupRows) * kGroupBytes;  // 72 KB
constexpr int kStages = 2;
constexpr int kPrefetch = 2;                            // tiles ahead in L2
constexpr int kQRows = 64;
constexpr int kQBytes = kChunks * kQRows * 128;
constexpr int kPOff = 8 * kChunkBytes;                  // P of a group: over its RoPE chunk
constexpr int kQOff = kStages * kStageBytes;
constexpr int kMiscOff = kQOff + kQBytes;
constexpr int kSoftThreads = 256;                       // warps 0-7: softmax + epilogue
constexpr int kSoftWarps = kSoftThreads / 32;
constexpr int kSWarp = 8;                               // issues S^T of chunks 0-4, owns TMEM
constexpr int kPvWarp = 9;                              // issues PV
constexpr int kLoadWarp = 10;                           // copies
constexpr int kSWarp2 = 11;                             // issues S^T of chunks 5-8
constexpr int kThreads = 384;
constexpr int kTmemCols = 512;
constexpr int kSCol = 0;                                // S^T of tile parity s: columns 128 s + those 64 further
constexpr int kOCol = 256;                              // O^T M-tile mt: columns 256 + 64 mt
constexpr float kRescaleLog2 = 8.f;
constexpr uint32_t kSoftBar = 1;
constexpr int kItemPages = 8;                           // what starting and finishing a request costs, in pages
constexpr int kPieces = 64;                             // of an item, where the batch leaves CTAs over
constexpr int kMaxBatch = 512;
constexpr int kJoinWarps = 8;
constexpr int kTaskDims = 128;                          // dims of a join task
constexpr int kOutRow = kDv * 2 + 16;                   // bytes between a whole item's output rows in shared memory
static_assert(kQRows * kOutRow <= kStageBytes, "the output rows fit into a stage");

// Shared memory behind the queries.
constexpr int kBarOff = 0;        // mbarriers
constexpr int kTmemSlotOff = 128;
constexpr int kMaskOff = 144;     // [2 stages][4 pages]
constexpr int kXmaxOff = 256;     // [2 tile parities][4 pages][64 heads] tile maxima
constexpr int kLsumOff = 2304;    // [4 pages][64]
constexpr int kMrowOff = 3328;    // [64]
constexpr int kLinvOff = 3584;    // [64]
constexpr int kLseOff = 3840;     // [64]
constexpr int kSumsOff = 4096;    // [12] 64-bit
constexpr int kPrefixOff = 4224;  // [batch + 1], and what kept_prefix puts behind it
constexpr int kSmemMax = 1024 + kMiscOff + kPrefixOff + kept_ints(kMaxBatch) * 4;
static_assert(kSmemMax <= 227 * 1024, "the largest batch fits");

struct LatentArgs {
  int32_t Hq;
  int32_t batch;
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t* seq_lens;
  int32_t num_pages;
  int32_t sink, recent;
  float scale_log2;
  uint16_t* out;     // [B][Hq][512]
  float* out_lse;
  int2* joins;       // [CTAs] by an item's first CTA: item and partials (0: nothing to join)
  float* o_part;     // [2 CTAs][Hq / 4][512][4]: four heads' partials per dim
  float* lse_part;   // [2 CTAs][Hq], log2 domain
  unsigned* err;
};

// D (+)= A B^T issued by one elected lane of a converged warp.
__device__ __forceinline__ void mma_elected(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrive on `bar` once every product the elected lane issued so far is done (the same lane each time).
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
      : "memory");
}

// The tiles of a CTA's slice in order: its segments, cut into tiles of 4 pages.
struct TileCursor {
  Segments sg;
  int ntiles, t, seg, j;
  bool valid;
  __device__ void open() {
    valid = sg.next();
    if (!valid) return;
    ntiles = (sg.hi - sg.lo + kTilePages - 1) / kTilePages;
    t = 0;
  }
  __device__ void init(const Slices& slices, int start, int stop) {
    sg.init(slices, start, stop);
    seg = j = 0;
    open();
  }
  __device__ bool last() const { return t == ntiles - 1; }
  __device__ void next() {
    ++j;
    if (++t == ntiles) {
      ++seg;
      open();
    }
  }
};

__global__ void __launch_bounds__(kThreads, 1) latent_decode_kernel(const __grid_constant__ CUtensorMap kvmap,
                                                                   const __grid_constant__ CUtensorMap qmap,
                                                                   const LatentArgs a) {
  pdl_enter();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* misc = smem + kMiscOff;
  uint64_t* bars = reinterpret_cast<uint64_t*>(misc + kBarOff);
  uint64_t* full = bars;         // [2] a tile landed
  uint64_t* empty = bars + 2;    // [2] the PV products of the stage's tile are done
  uint64_t* s_full = bars + 4;   // [2] S^T of a tile is in TMEM
  uint64_t* s_free = bars + 6;   // [2] S^T read by the softmax threads
  uint64_t* p_full = bars + 8;   // [2] P written, rows not kept zeroed, O^T rescaled
  uint64_t* o_free = bars + 11;  // O^T read by the epilogue
  uint64_t* q_full = bars + 12;  // the request's queries landed
  uint64_t* q_empty = bars + 13; // the last S^T product of a segment is done
  uint64_t* fin = bars + 14;     // every product of the CTA is done (all three issuers)
  // The PV products of a segment's last tile are done, one phase per segment: the epilogue cannot wait on
  // empty, which may be a phase behind (a parity wait names the current or the preceding phase only).
  uint64_t* o_last = bars + 15;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + kTmemSlotOff);
  uint32_t* masks = reinterpret_cast<uint32_t*>(misc + kMaskOff);
  float* xmax = reinterpret_cast<float*>(misc + kXmaxOff);
  float* lsum = reinterpret_cast<float*>(misc + kLsumOff);
  float* mrow = reinterpret_cast<float*>(misc + kMrowOff);
  float* linv = reinterpret_cast<float*>(misc + kLinvOff);
  float* lse_s = reinterpret_cast<float*>(misc + kLseOff);
  int* prefix = reinterpret_cast<int*>(misc + kPrefixOff);
  int* lens = prefix + a.batch + 1;  // [batch], then the pages of each
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hq = a.Hq;

  const int piece =
      kept_prefix<kThreads>(a.seq_lens, a.batch, 1, a.bt_stride, a.sink, a.recent, kItemPages, kTilePages, kPieces,
                            gridDim.x, kMaxPlaces, prefix, lens, reinterpret_cast<long long*>(misc + kSumsOff), a.err);
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    if (prefix[b + 1] != prefix[b]) continue;  // no kept token: the empty sum
    uint4* o = reinterpret_cast<uint4*>(a.out + (size_t)b * Hq * kDv);
    for (int i = threadIdx.x; i < Hq * kDv / 8; i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
    if (a.out_lse)
      for (int i = threadIdx.x; i < Hq; i += kThreads) a.out_lse[(size_t)b * Hq + i] = -INFINITY;
  }
  Slices slices;
  slices.init(prefix, a.batch, 1, kItemPages, kTilePages, gridDim.x, piece);
  const int2 slice = slice_of(slices, blockIdx.x);
  if (slice.x >= slice.y) {
    if (threadIdx.x == 0) a.joins[blockIdx.x] = make_int2(0, 0);
    return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&s_full[s], 2);
      mbar_init(&s_free[s], kSoftWarps);
      mbar_init(&p_full[s], kSoftWarps);
    }
    mbar_init(o_free, kSoftWarps);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    mbar_init(fin, 3);
    mbar_init(o_last, 1);
    mbar_fence_init();
  }
  if (warp == kSWarp) tmem_alloc(tmem_slot, kTmemCols);
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t smem0 = smem_addr(smem);
  bool dead = false;  // a bounded wait gave up: leave the loops, no further waits
  TileCursor c;
  c.init(slices, slice.x, slice.y);

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------ copies
    const uint64_t policy = l2_evict_first_policy();
    Kept k;
    int base = 0, cur = 0, nxt = 0;
    const int32_t* bt = nullptr;
    auto entry = [&](int i) {  // physical page of the segment's page i, -1: none
      if (i >= c.sg.hi) return -1;
      const int ph = bt[k.logical(i)];
      if (ph >= 0 && ph < a.num_pages) return ph;
      raise_error(a.err, SE_DEVERR_PAGE_RANGE);
      return -1;
    };
    // Lane l of a tile's first eight: half l % 2 of its page l / 2.
    const int pg = (lane >> 1) & 3, hf = lane & 1;
    auto page_of = [&](int i) {
      const int pc = __shfl_sync(0xffffffffu, cur, (i - base) & 31);
      const int pn = __shfl_sync(0xffffffffu, nxt, (i - base) & 31);
      return i < base + 32 ? pc : pn;
    };
    for (; c.valid; c.next()) {
      const int s = c.j & 1, i0 = c.sg.lo + c.t * kTilePages;
      if (c.t == 0) {
        k = kept_of(lens[c.sg.b], a.bt_stride, a.sink, a.recent, nullptr);
        bt = a.block_table + (size_t)c.sg.b * a.bt_stride;
        base = i0;
        cur = entry(base + lane);
        nxt = entry(base + 32 + lane);
      } else if (i0 == base + 32) {
        base += 32;
        cur = nxt;
        nxt = entry(base + 32 + lane);
      }
      const int i = i0 + pg;
      const int phys = page_of(i);
      if (lane == 0 && c.j >= 2 && !mbar_wait(&empty[s], ((c.j >> 1) - 1) & 1)) dead = true;
      dead = __shfl_sync(0xffffffffu, (int)dead, 0) != 0;
      if (dead) break;
      if (lane < 8 && hf == 0) masks[s * kTilePages + pg] = phys >= 0 ? page_mask(k, a.sink, k.logical(i)) : 0u;
      const uint32_t live = __popc(__ballot_sync(0xffffffffu, lane < 8 && phys >= 0));
      if (lane == 0) mbar_arrive_expect_tx(&full[s], live * kGroupBytes);
      __syncwarp();
      if (lane < 8 && phys >= 0)
        tma_load_3d(smem + s * kStageBytes + lane * kGroupBytes, &kvmap, 0, phys * kPageSize + hf * kGroupRows, 0,
                    &full[s], policy);
      if (c.t == 0) {
        // The request's queries, once the previous segment's S^T products are done with the buffer.
        if (lane == 0 && c.seg >= 1 && !mbar_wait(q_empty, (c.seg - 1) & 1)) dead = true;
        dead = __shfl_sync(0xffffffffu, (int)dead, 0) != 0;
        if (dead) {
          c.next();  // the tile's copies were issued
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(q_full, (uint32_t)Hq * kD * 2);
        __syncwarp();
        if (lane < kChunks)
          tma_load_3d(smem + kQOff + lane * kQRows * 128, &qmap, lane * 64, 0, c.sg.b, q_full, policy);
      }
      // L2 prefetch: the tile kPrefetch ahead (lanes 0-7), and at a segment's start those before it.
      for (int d = c.t == 0 ? 1 : kPrefetch; d <= kPrefetch; ++d) {
        const int ahead = page_of(i + d * kTilePages);
        if (lane < 8 && ahead >= 0) tma_prefetch_3d(&kvmap, 0, ahead * kPageSize + hf * kGroupRows, 0);
      }
    }
    // Every copy has landed before the CTA leaves.
    if (lane == 0) {
      for (int u = max(0, c.j - kStages); u < c.j; ++u)
        if (!mbar_wait(&full[u & 1], (u >> 1) & 1)) dead = true;
      if (dead) raise_error(a.err, SE_DEVERR_WAIT_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == kSWarp || warp == kSWarp2) {
    const int hf = warp == kSWarp2;  // the half of the K steps
    // ------------------------------------------------------------ S^T
    const uint32_t idesc = umma_idesc_bf16(64, Hq);
    const uint64_t dk0 = umma_desc_sw128_groups(smem0, kGroupBytes), dq = umma_desc_sw128(smem0 + kQOff);
    for (; c.valid; c.next()) {
      const int s = c.j & 1;
      bool ok = c.t != 0 || mbar_wait(q_full, c.seg & 1);
      ok = ok && (c.j < 2 || mbar_wait(&s_free[s], ((c.j >> 1) - 1) & 1)) && mbar_wait(&full[s], (c.j >> 1) & 1);
      if (!__all_sync(0xffffffffu, ok)) {
        dead = true;
        break;
      }
      tc05_fence_after();
      const uint32_t d = tmem + kSCol + s * 128 + hf * 64;
      const uint64_t dk = dk0 + (s ? (uint64_t)(kStageBytes >> 4) : 0);
      // 16 dims are 32 bytes of a 128-byte row; the next 64 dims are a chunk further.
#pragma unroll
      for (int ch = 0; ch < 5; ++ch) {
        if (ch == 4 && hf) break;  // 5 and 4 chunks
        const int cc = ch + 5 * hf;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          mma_elected(d, dk + cc * (kChunkBytes >> 4) + 2 * x, dq + cc * (kQRows * 128 >> 4) + 2 * x, idesc,
                      ch + x > 0 ? 1u : 0u);
      }
      commit_elected(&s_full[s]);
      if (c.last()) commit_elected(q_empty);
    }
    commit_elected(fin);
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------ O^T += V^T P^T
    const uint32_t idesc = umma_idesc_bf16_mn(128, 64);
    // MN-major: 64 dims (or heads) per 128-byte row, the next 64 dims a chunk further, the next 8 tokens a group.
    const uint64_t dv0 = umma_desc_sw128_mn_groups(smem0, kChunkBytes, kGroupBytes);
    for (; c.valid; c.next()) {
      const int s = c.j & 1;
      const bool first = c.t == 0;
      bool ok = mbar_wait(&p_full[s], (c.j >> 1) & 1);
      ok = ok && (!first || c.seg == 0 || mbar_wait(o_free, (c.seg - 1) & 1));
      if (!__all_sync(0xffffffffu, ok)) {
        dead = true;
        break;
      }
      tc05_fence_after();
      constexpr uint64_t kStep = (2 * kGroupBytes) >> 4, kMt = (2 * kChunkBytes) >> 4;
      const uint64_t dv = dv0 + (s ? (uint64_t)(kStageBytes >> 4) : 0), dp = dv + (kPOff >> 4);
      const uint32_t acc0 = first ? 0u : 1u;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
          mma_elected(tmem + kOCol + mt * 64, dv + mt * kMt + ks * kStep, dp + ks * kStep, idesc, ks > 0 ? 1u : acc0);
      // The epilogue of a whole item passes its rows through the stage and frees it.
      if (!c.last() || c.sg.split()) commit_elected(&empty[s]);
      if (c.last()) commit_elected(o_last);
    }
    commit_elected(fin);
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    // Warp w: page w % 4 of the tile (its TMEM lane quarter), heads 32 (w / 4) ..;
    // thread: token `tok` of the page, heads hh .. hh + 15.
    const int q4 = warp & 3;
    const int tok = lane & 15, hh = 32 * (warp >> 2) + 16 * (lane >> 4);
    const int hr = hh + reduced_index(lane);  // head of this thread's reduction results
    const int row = q4 * kPageSize + tok;     // token row of the tile
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const int parts1 = neighbours_of(slices, blockIdx.x, slice).parts1;
    int2 join = make_int2(0, 0);              // the item that goes on behind the slice
    float m_h[16], b_h[16], l_h[16];
    bool unset = false;                       // one of the heads has no finite maximum yet
#pragma unroll
    for (int i = 0; i < 16; ++i) m_h[i] = b_h[i] = l_h[i] = 0.f;
    for (; c.valid; c.next()) {
      const int j = c.j, t = c.t, s = j & 1;
      const bool ok_s = __all_sync(0xffffffffu, mbar_wait(&s_full[s], (j >> 1) & 1));
      uint32_t r[16];
      if (ok_s) {
        tc05_fence_after();
        uint32_t r2[16];
        tmem_ld16x2_16(tmem + lane_base + kSCol + s * 128 + 32 * (warp >> 2), r);
        tmem_ld16x2_16(tmem + lane_base + kSCol + s * 128 + 64 + 32 * (warp >> 2), r2);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) + __uint_as_float(r2[i]));
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = 0u;
      }
      tc05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_free[s]);
      const bool ok_f = __all_sync(0xffffffffu, mbar_wait(&full[s], (j >> 1) & 1));  // the masks of the tile
      dead = dead || !ok_s || !ok_f;
      const bool tok_ok = in_mask(masks[s * kTilePages + q4], tok);
      // Logits against the running maxima (0 for a head that has none yet).
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = fmaf(__uint_as_float(r[i]), a.scale_log2, -b_h[i]);
      if (!tok_ok || hh + 16 > Hq) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!tok_ok || hh + i >= Hq) x[i] = -INFINITY;
      }
      if (!tok_ok && (warp >> 2) == 0) {
        // Rows that are not kept (or not copied) may hold NaN: zero their value dims, as 0 * NaN is not 0.
        const uint32_t st = smem0 + s * kStageBytes + (row / kGroupRows) * kGroupBytes;
#pragma unroll 1
        for (int ch = 4 * (lane >> 4); ch < 4 * (lane >> 4) + 4; ++ch)
#pragma unroll
          for (int k = 0; k < 8; ++k) st_shared_v4(st + ch * kChunkBytes + swz128(row % kGroupRows, k), 0u, 0u, 0u, 0u);
      }
      // After the segment's first tile, a tile whose scores all stay within 2^8 of the running maxima changes
      // nothing but P and l. Otherwise, and while a head has seen nothing but -inf (its base of 0 is no maximum),
      // the tile maxima are exchanged and the running maxima recomputed.
      bool need = dead || unset;
#pragma unroll
      for (int i = 0; i < 16; ++i) need = need || x[i] > kRescaleLog2;
      if (t == 0 || bar_red_or(kSoftBar, kSoftThreads, need)) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = tok_ok && hh + i < Hq ? __uint_as_float(r[i]) * a.scale_log2 : -INFINITY;
        half_warp_reduce16<true>(v, lane);
        // Two buffers by tile parity: the barriers keep every thread within one tile of the others.
        float* xm = xmax + s * 256;
        xm[q4 * 64 + hr] = v[0];
        if (bar_red_or(kSoftBar, kSoftThreads, dead)) {  // also publishes xmax
          dead = true;
          break;
        }
        float f[16];
        bool moved = false;
        unset = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 w0 = *reinterpret_cast<const float4*>(xm + hh + 4 * k);
          const float4 w1 = *reinterpret_cast<const float4*>(xm + 64 + hh + 4 * k);
          const float4 w2 = *reinterpret_cast<const float4*>(xm + 128 + hh + 4 * k);
          const float4 w3 = *reinterpret_cast<const float4*>(xm + 192 + hh + 4 * k);
          const float tm[4] = {fmaxf(fmaxf(w0.x, w1.x), fmaxf(w2.x, w3.x)), fmaxf(fmaxf(w0.y, w1.y), fmaxf(w2.y, w3.y)),
                               fmaxf(fmaxf(w0.z, w1.z), fmaxf(w2.z, w3.z)), fmaxf(fmaxf(w0.w, w1.w), fmaxf(w2.w, w3.w))};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 4 * k + e;
            const float mo = m_h[i];
            const float mn = (t == 0 || tm[e] > mo + kRescaleLog2) ? tm[e] : mo;
            const bool mv = t > 0 && mn != mo;
            f[i] = mv ? fast_exp2(mo - mn) : 1.f;
            moved = moved || mv;
            m_h[i] = mn;
            unset = unset || (mn == -INFINITY && hh + i < Hq);
            l_h[i] = t == 0 ? 0.f : l_h[i] * f[i];
            b_h[i] = finite_base(mn);
            x[i] = tok_ok && hh + i < Hq ? fmaf(__uint_as_float(r[i]), a.scale_log2, -b_h[i]) : -INFINITY;
          }
        }
        if (__any_sync(0xffffffffu, moved)) {
          // The O^T columns of this warp's head half (its lane quarter) to the new maxima.
          const bool ok_o = __all_sync(0xffffffffu, mbar_wait(&empty[s ^ 1], ((j - 1) >> 1) & 1));
          if (ok_o) {
            float fc[32];  // factor of column cc of the half: lanes 0-15 hold heads 0-15, lanes 16-31 heads 16-31
#pragma unroll
            for (int cc = 0; cc < 32; ++cc) fc[cc] = __shfl_sync(0xffffffffu, f[cc & 15], (cc >> 4) * 16);
            tc05_fence_after();
#pragma unroll 1
            for (int mt = 0; mt < 4; ++mt) {
              const uint32_t ta = tmem + lane_base + kOCol + mt * 64 + 32 * (warp >> 2);
              uint32_t o[32];
              tmem_ld32(ta, o);
              tmem_ld_wait();
#pragma unroll
              for (int cc = 0; cc < 32; ++cc) o[cc] = __float_as_uint(__uint_as_float(o[cc]) * fc[cc]);
              tmem_st32(ta, o);
            }
            tmem_st_wait();
          } else {
            dead = true;
          }
        }
      }
      // P of this token for heads hh .. hh + 15, rounded to bf16 (half a step, 2^-8 of each weight, as the MMA
      // wants; l sums it unrounded), into its row of its group's RoPE chunk (64 heads per 128-byte row).
      uint32_t pk[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float pa = fast_exp2(x[2 * i]), pb = fast_exp2(x[2 * i + 1]);
        l_h[2 * i] += pa;
        l_h[2 * i + 1] += pb;
        pk[i] = pack_bf16x2(pa, pb);
      }
      const uint32_t prow = smem0 + s * kStageBytes + (row / kGroupRows) * kGroupBytes + kPOff;
      st_shared_v4(prow + swz128(row % kGroupRows, hh >> 3), pk[0], pk[1], pk[2], pk[3]);
      st_shared_v4(prow + swz128(row % kGroupRows, (hh >> 3) + 1), pk[4], pk[5], pk[6], pk[7]);
      fence_proxy_async_smem();
      tc05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[s]);

      if (c.last()) {
        // ---- epilogue of the segment: O = O^T / l per head, or a partial
        const int b = c.sg.b;
        float w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = l_h[i];
        half_warp_reduce16<false>(w, lane);
        lsum[q4 * 64 + hr] = w[0];
        if (q4 == 0 && tok == 0)
#pragma unroll
          for (int i = 0; i < 16; ++i) mrow[hh + i] = m_h[i];
        named_bar_sync(kSoftBar, kSoftThreads);
        if (threadIdx.x < 64) {
          const int h = threadIdx.x;
          const float l = (lsum[h] + lsum[64 + h]) + (lsum[128 + h] + lsum[192 + h]);
          linv[h] = l == 0.f ? 0.f : 1.f / l;
          lse_s[h] = l == 0.f ? -INFINITY : mrow[h] + log2f(l);
        }
        named_bar_sync(kSoftBar, kSoftThreads);
        const bool ok_e = __all_sync(0xffffffffu, mbar_wait(o_last, c.seg & 1));
        dead = dead || !ok_e;
        const bool split = c.sg.split();
        const int slot = 2 * blockIdx.x + (c.sg.lo > 0 ? 0 : 1);
        if (c.sg.lo == 0 && split) join = make_int2(b, parts1);
        if (ok_e && !split) {
          // Whole rows: transposed in pairs of 8 x 8 tiles into rows of the last tile's stage, which no product reads
          // any more, and from there by bulk copies of a row each.
          tc05_fence_after();
          const int h0 = 32 * (warp >> 2);
          float2 inv[4];  // of this thread's columns: heads h0 + 8 i + 2 (lane % 4) and the next
#pragma unroll
          for (int i = 0; i < 4; ++i) inv[i] = *reinterpret_cast<const float2*>(linv + h0 + 8 * i + 2 * (lane & 3));
          const uint32_t to = smem0 + s * kStageBytes + (h0 + 8 * (lane >> 4) + (lane & 7)) * kOutRow +
                              (32 * q4 + (lane & 8)) * 2;
          if (h0 < Hq) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt)
#pragma unroll
              for (int x = 0; x < 2; ++x) {  // 16 dims
                uint32_t o[16];
                tmem_ld16x256b_x4(tmem + lane_base + ((uint32_t)(16 * x) << 16) + kOCol + mt * 64 + h0, o);
                tmem_ld_wait();
                uint32_t y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  y[i] = pack_bf16x2(__uint_as_float(o[2 * i]) * inv[i >> 1].x,
                                     __uint_as_float(o[2 * i + 1]) * inv[i >> 1].y);
                const uint32_t at = to + (mt * 128 + 16 * x) * 2;
                stmatrix_x4_trans(at, y[0], y[1], y[2], y[3]);
                stmatrix_x4_trans(at + 16 * kOutRow, y[4], y[5], y[6], y[7]);
              }
          }
          fence_proxy_async_smem();
        }
        if (ok_e && split) {
          tc05_fence_after();
#pragma unroll 1
          for (int mt = 0; mt < 4; ++mt) {
            uint32_t o[32];
            tmem_ld32(tmem + lane_base + kOCol + mt * 64 + 32 * (warp >> 2), o);
            tmem_ld_wait();
            const int d = mt * 128 + 32 * q4 + lane;
            // Four heads of a dim in one 16-byte store.
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int h = 32 * (warp >> 2) + 4 * k;
              if (h < Hq) {
                const float4 val =
                    make_float4(__uint_as_float(o[4 * k]) * linv[h], __uint_as_float(o[4 * k + 1]) * linv[h + 1],
                                __uint_as_float(o[4 * k + 2]) * linv[h + 2], __uint_as_float(o[4 * k + 3]) * linv[h + 3]);
                *reinterpret_cast<float4*>(a.o_part + (((size_t)slot * (Hq / 4) + h / 4) * kDv + d) * 4) = val;
              }
            }
          }
        }
        if (threadIdx.x < Hq) {
          if (split)
            a.lse_part[(size_t)slot * Hq + threadIdx.x] = lse_s[threadIdx.x];
          else if (a.out_lse)
            a.out_lse[(size_t)b * Hq + threadIdx.x] = lse_s[threadIdx.x] * kLn2;
        }
        tc05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);
        if (!split) {
          named_bar_sync(kSoftBar, kSoftThreads);  // the rows are complete
          if (warp == 0) {
            if (ok_e)
              for (int h = lane; h < Hq; h += 32) {
                const uint32_t from = smem0 + s * kStageBytes + h * kOutRow;
                if (linv[h] == 0.f) {
                  // No finite logit: 0 whatever the values hold (0 times them need not be; a partial keeps that
                  // product, as the sum over a row with other tokens does).
#pragma unroll 1
                  for (int i = 0; i < kDv * 2; i += 16) st_shared_v4(from + i, 0u, 0u, 0u, 0u);
                  fence_proxy_async_smem();
                }
                tma_store_bulk(a.out + ((size_t)b * Hq + h) * kDv, from, kDv * 2);
              }
            tma_store_commit();
            tma_store_wait_read();
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
          }
        }
      }
    }
    if (warp == 0) tma_store_wait();
    if (threadIdx.x == 0) a.joins[blockIdx.x] = join;
  }
  if (dead && lane == 0) raise_error(a.err, SE_DEVERR_WAIT_TIMEOUT);
  if (warp == kSWarp && !__all_sync(0xffffffffu, mbar_wait(fin, 0)) && lane == 0)
    raise_error(a.err, SE_DEVERR_WAIT_TIMEOUT);
  tc05_fence_before();
  __syncthreads();
  tc05_fence_after();
  if (warp == kSWarp) tmem_dealloc(tmem, kTmemCols);
}

// Joins the partials of the items that span CTAs. With M_h the largest log-sum-exp of head h,
//     out_h = sum_i exp2(lse_hi - M_h) o_hi / sum_i exp2(lse_hi - M_h).
// A warp takes four heads and 128 dims of an item, four consecutive dims per lane; share_of(partials) warps share
// the partials of an item that has many, and are joined in their order.
__global__ void __launch_bounds__(kJoinWarps * 32) latent_join_kernel(const float* __restrict__ o_part,
                                                                     const float* __restrict__ lse_part,
                                                                     const int2* __restrict__ joins, int32_t ctas,
                                                                     int32_t Hq, uint16_t* __restrict__ out,
                                                                     float* __restrict__ out_lse) {
  pdl_enter();
  static_assert(kMaxCtas <= kJoinWarps * 32, "a thread per item");
  __shared__ int4 todo[kMaxCtas];
  __shared__ int2 counts[kJoinWarps];
  __shared__ float4 acc_s[kJoinWarps][4][32], m_s[kJoinWarps], l_s[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tasks = (Hq / 4) * (kDv / kTaskDims);  // a multiple of the warps
  const int2 todos = list_joins(joins, ctas, tasks, todo, counts);
  auto scale4 = [](const float4& a, const float4& f) {
    return make_float4(a.x * f.x, a.y * f.y, a.z * f.z, a.w * f.w);
  };
  auto fma4 = [](const float4& f, const float4& v, const float4& a) {
    return make_float4(a.x + f.x * v.x, a.y + f.y * v.y, a.z + f.z * v.z, a.w + f.w * v.w);
  };
  auto max4 = [](const float4& a, const float4& b) {
    return make_float4(fmaxf(a.x, b.x), fmaxf(a.y, b.y), fmaxf(a.z, b.z), fmaxf(a.w, b.w));
  };
  // exp2(a - m), 0 where nothing but -inf has been seen.
  auto weight4 = [](const float4& a, const float4& m) {
    return make_float4(fast_exp2(a.x - finite_base(m.x)), fast_exp2(a.y - finite_base(m.y)),
                       fast_exp2(a.z - finite_base(m.z)), fast_exp2(a.w - finite_base(m.w)));
  };
  for (int u = blockIdx.x; u < todos.y; u += gridDim.x) {
    const int4 jn = join_of(todo, todos.x, u);
    const int share = share_of(jn.z), task = (u - jn.w) * (kJoinWarps / share) + warp / share, sub = warp % share;
    const int blk = task / (kDv / kTaskDims), d = task % (kDv / kTaskDims) * kTaskDims + 4 * lane;
    // Partial i is in slot 1 of the item's first CTA (i = 0), in slot 0 of the others.
    auto part = [&](int i) { return (size_t)(2 * (jn.x + i) + (i == 0)) * (Hq / 4) + blk; };
    const int n = (jn.z - sub + share - 1) / share;
    float4 M = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY), l = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 acc[4] = {l, l, l, l};  // dims d .. d + 3 of the four heads
    // Batches of four partials, their loads in flight beside those of their log-sum-exps.
    for (int k0 = 0; k0 < n; k0 += 4) {
      float4 v[4][4], ls[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ls[k] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (k0 + k >= n) continue;
        const size_t p = part(sub + share * (k0 + k));
        ls[k] = *reinterpret_cast<const float4*>(lse_part + p * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = *reinterpret_cast<const float4*>(o_part + (p * kDv + d + e) * 4);
      }
      const float4 top = max4(M, max4(max4(ls[0], ls[1]), max4(ls[2], ls[3])));
      const float4 f0 = weight4(M, top);
      M = top;
      l = scale4(l, f0);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = scale4(acc[e], f0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k0 + k >= n) continue;
        const float4 w = weight4(ls[k], M);
        l = make_float4(l.x + w.x, l.y + w.y, l.z + w.z, l.w + w.w);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fma4(w, v[k][e], acc[e]);
      }
    }
    if (share > 1) {
      __syncthreads();  // the previous unit's sums are read
#pragma unroll
      for (int e = 0; e < 4; ++e) acc_s[warp][e][lane] = acc[e];
      if (lane == 0) {
        m_s[warp] = M;
        l_s[warp] = l;
      }
      __syncthreads();
      if (sub > 0) continue;  // the first of the warps that share adds the others
      for (int k = 1; k < share; ++k) {
        const float4 mk = m_s[warp + k], top = max4(M, mk), f0 = weight4(M, top), fk = weight4(mk, top);
        M = top;
        l = fma4(fk, l_s[warp + k], scale4(l, f0));
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = fma4(fk, acc_s[warp + k][e][lane], scale4(acc[e], f0));
      }
    }
    const size_t row = (size_t)jn.y * Hq + blk * 4;
    const float ll[4] = {l.x, l.y, l.z, l.w}, mm[4] = {M.x, M.y, M.z, M.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      auto at = [&](const float4& v) { return h == 0 ? v.x : h == 1 ? v.y : h == 2 ? v.z : v.w; };
      const bool none = ll[h] == 0.f;
      const float inv = 1.f / ll[h];
      *reinterpret_cast<uint2*>(out + (row + h) * kDv + d) =
          none ? make_uint2(0u, 0u)
               : make_uint2(pack_bf16x2(at(acc[0]) * inv, at(acc[1]) * inv),
                            pack_bf16x2(at(acc[2]) * inv, at(acc[3]) * inv));
      if (out_lse && d == 0) out_lse[row + h] = none ? -INFINITY : (mm[h] + log2f(ll[h])) * kLn2;
    }
  }
}

}  // namespace

int paged_latent_max_batch() { return kMaxBatch; }

bool paged_latent_supported(int num_kv_heads, int head_dim, int head_dim_v, int num_q_heads) {
  return num_kv_heads == 1 && head_dim == kD && head_dim_v == kDv && num_q_heads % 16 == 0 && num_q_heads >= 16 &&
         num_q_heads <= 64;
}

size_t paged_latent_workspace_bytes(int32_t num_q_heads) {
  return kCounterBytes + 2 * kMaxCtas * (size_t)num_q_heads * (kDv + 1) * sizeof(float);
}

cudaError_t launch_paged_latent(const CUtensorMap& kvmap, const CUtensorMap& qmap, const KvView& kv,
                                int32_t num_q_heads, const int32_t* block_table, int32_t bt_stride,
                                const int32_t* seq_lens, int32_t batch, int32_t sink_tokens, int32_t recent_tokens,
                                float sm_scale, uint16_t* out, float* out_lse, void* workspace, int sm_count,
                                unsigned* err, cudaStream_t stream) {
  LatentArgs a;
  a.Hq = num_q_heads;
  a.batch = batch;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.seq_lens = seq_lens;
  a.num_pages = kv.num_pages;
  a.sink = sink_tokens;
  a.recent = recent_tokens;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.out = out;
  a.out_lse = out_lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.joins = reinterpret_cast<int2*>(ws + kArrivalBytes);  // the arrival counters before them are not used here
  a.o_part = reinterpret_cast<float*>(ws + kCounterBytes);
  a.lse_part = a.o_part + 2 * kMaxCtas * (size_t)num_q_heads * kDv;
  a.err = err;
  const int grid = std::min(sm_count, kMaxCtas);
  const size_t smem = 1024 + kMiscOff + kPrefixOff + kept_ints(batch) * 4;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(latent_decode_kernel, kSmemMax, allowed);
  if (e != cudaSuccess) return e;
  e = launch_pdl(latent_decode_kernel, dim3(grid), dim3(kThreads), smem, stream, kvmap, qmap, a);
  if (e != cudaSuccess) return e;
  // An item has at most as many units as tasks, and no more items than CTAs reach beyond a slice.
  const int units = std::min(grid, batch) * (num_q_heads / 4) * (kDv / kTaskDims);
  return launch_pdl(latent_join_kernel, dim3(std::min(units, 8 * grid)), dim3(kJoinWarps * 32), 0, stream, a.o_part,
                    a.lse_part, a.joins, grid, num_q_heads, out, out_lse);
}

}  // namespace se
