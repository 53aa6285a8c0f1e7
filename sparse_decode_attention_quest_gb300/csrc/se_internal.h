// Internal declarations shared by the host entry points (api.cu) and the
// kernel translation units. Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "../../include/sparse_engine.h"

namespace se {

// Launch with programmatic stream serialization: the kernel may be scheduled
// while the previous kernel in the stream finishes; it waits (pdl_wait) before
// touching memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Raises a kernel's dynamic shared memory limit once per device (`done`: one bit per device, a static
// of the kernel's launcher).
template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_acq_rel);
  return e;
}

constexpr int kPageSize = 16;
// Bounded waits: an mbarrier wait gives up after this much wall time or polls.
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr uint32_t kWaitLimitIters = 1u << 28;

// Device-visible copy of the cache layout (plain values, passed by value).
struct KvView {
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* summary;
  int32_t num_pages;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t head_dim_v;
  int32_t row_stride_k;
  int32_t row_stride_v;
};

// The same of an 8-bit cache.
struct Kv8View {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int32_t num_pages;
  int32_t num_kv_heads;
  int32_t head_dim;
};

// ---- quest_summary.cu
cudaError_t launch_build_summaries(const KvView& kv, const int32_t* block_table, int32_t bt_stride,
                                   const int32_t* seq_lens, int32_t batch, int32_t max_seq_len, unsigned* err,
                                   cudaStream_t stream);
// overlap_previous: the kernel may run alongside the previous kernel of the
// stream (it must touch nothing that kernel reads or writes) and completes after it.
cudaError_t launch_append_update(const KvView& kv, uint16_t* k_mut, uint16_t* v_mut, const uint16_t* k_new,
                                 const uint16_t* v_new, const int32_t* block_table, int32_t bt_stride,
                                 const int32_t* seq_lens_before, int32_t batch, bool overlap_previous,
                                 unsigned* err, cudaStream_t stream);

// ---- quest_score.cu
bool score_pages_supported(int num_kv_heads, int head_dim);
// Bytes of the per-request multipliers (P and N) that pn_ws holds.
size_t score_pn_bytes(int32_t batch, int32_t num_kv_heads, int32_t head_dim);
// pn_ws (score_pn_bytes, 16-byte aligned) or null: with it, a first kernel
// reduces every request's queries once and the scoring kernel reads the result;
// without it, every CTA reduces the queries of the requests it scores.
cudaError_t launch_score_pages(const KvView& kv, const uint16_t* q, int32_t num_q_heads,
                               const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                               int32_t batch, int32_t max_seq_len, float* scores, int32_t score_stride,
                               float* pn_ws, int sm_count, unsigned* err, cudaStream_t stream);
// ---- quest_topk.cu
// Top-k of the candidate pages: those holding none of the first sink_tokens and
// none of the last recent_tokens tokens (the last page always kept); the kept
// windows are written around the selection.
cudaError_t launch_topk_pages(const float* scores, int32_t score_stride, const int32_t* seq_lens, int32_t batch,
                              int32_t num_kv_heads, int32_t max_seq_len, int32_t topk, int32_t sink_tokens,
                              int32_t recent_tokens, int32_t* out_pages, int32_t* out_counts, int32_t sel_stride,
                              unsigned* err, cudaStream_t stream);
size_t topk_smem_bytes(int32_t max_seq_len);

// ---- sparse_decode.cu
struct DecodePlan {
  int32_t nsplit;           // most CTAs whose slices one item's pages can span (partial slots per row)
  int32_t pages_per_split;  // fewest selected pages per CTA slice
  int32_t grid;             // CTAs launched
};
DecodePlan plan_gqa_decode(int32_t batch, int32_t num_kv_heads, int32_t sel_stride, int sm_count);
size_t gqa_decode_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t head_dim_v, const DecodePlan& plan);
// Byte offset in the workspace of the per-item arrival counters (batch x KV heads
// uint32, zero between calls: every call leaves them as it found them).
size_t gqa_decode_arrivals_offset(int32_t batch, int32_t num_q_heads, int32_t head_dim_v, const DecodePlan& plan);
size_t gqa_decode_max_items();
cudaError_t launch_gqa_decode(const KvView& kv, const uint16_t* q, int32_t num_q_heads, const int32_t* block_table,
                              int32_t bt_stride, const int32_t* seq_lens, int32_t batch, const int32_t* sel_pages,
                              const int32_t* sel_counts, int32_t sel_stride, float sm_scale, uint16_t* out,
                              float* out_lse, void* workspace, const DecodePlan& plan, unsigned* err,
                              cudaStream_t stream);

// ---- mla_decode.cu (latent cache: head_dim 576, value = first 512 dims, one KV head)
bool mla_decode_supported(int num_kv_heads, int head_dim, int head_dim_v, int num_q_heads);
DecodePlan plan_mla_decode(int32_t sel_stride, int sm_count);
size_t mla_decode_workspace_bytes(int32_t batch, int32_t num_q_heads, const DecodePlan& plan);
size_t mla_decode_max_items();
// kvmap: the cache as rows of 576 bf16, boxes of 64 x 16; qmap: the queries as
// batch x num_q_heads rows of 576, boxes of 64 x num_q_heads (both 128-byte swizzle).
cudaError_t launch_mla_decode(const CUtensorMap& kvmap, const CUtensorMap& qmap, const KvView& kv, const uint16_t* q,
                              int32_t num_q_heads, const int32_t* block_table,
                              int32_t bt_stride, const int32_t* seq_lens, int32_t batch, const int32_t* sel_pages,
                              const int32_t* sel_counts, int32_t sel_stride, float sm_scale, uint16_t* out,
                              float* out_lse, void* workspace, const DecodePlan& plan, unsigned* err,
                              cudaStream_t stream);

// ---- quest_fused.cu: append + score + top-k + decode in one launch (a cluster per item)
int fused_max_candidates();
int fused_max_kept();
int fused_cluster_size(int items, int sm_count);
cudaError_t launch_quest_fused(const KvView& kv, uint16_t* k_mut, uint16_t* v_mut, const uint16_t* k_new,
                               const uint16_t* v_new, const uint16_t* q, int32_t num_q_heads,
                               const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens, int32_t batch,
                               int32_t max_seq_len, int32_t topk, int32_t sink_tokens, int32_t recent_tokens,
                               float sm_scale, uint16_t* out, float* out_lse, int32_t* sel, int32_t* sel_counts,
                               int32_t sel_stride, int sm_count, unsigned* err, cudaStream_t stream);

// ---- snapkv.cu
int snapkv_max_slices(int max_len);
size_t snapkv_part_bytes(int pairs, int max_len);
int snapkv_select_max_candidates();
// kmap: the key cache as rows of 128 bf16, boxes of 64 x 16; qmap: the window
// queries as [B][W][Hq][128], boxes of 64 dims x G heads x W positions x 1
// (both 128-byte swizzle).
cudaError_t launch_snapkv_scores(const CUtensorMap& kmap, const CUtensorMap& qmap, const KvView& kv, const uint16_t* qwin,
                                 int32_t num_q_heads,
                                 int32_t window, const int32_t* bt, int32_t bt_stride, const int32_t* lens,
                                 int32_t batch, int32_t max_len, float sm_scale, float* scores, int32_t score_stride,
                                 float* row_lse, void* part_ws, int sm_count, unsigned* err, cudaStream_t stream);
// The next launch_snapkv_scores of this host thread runs as a wait probe (limit in us).
void set_snapkv_wait_probe(uint32_t limit_us);
// Keeps positions 0 .. sink - 1 and n - recent .. n - 1 (recent >= window) and the keep best
// pooled candidates between them.
cudaError_t launch_snapkv_select(const float* scores, int32_t score_stride, const int32_t* lens, int32_t batch,
                                 int32_t num_kv_heads, int32_t window, int32_t max_len, int32_t pool, int32_t keep,
                                 int32_t sink, int32_t recent, int32_t* kept, int32_t kept_stride,
                                 int32_t* kept_counts, unsigned* err, cudaStream_t stream);
cudaError_t launch_snapkv_gather(const KvView& src, uint16_t* dk, uint16_t* dv, int32_t dst_num_pages,
                                 const int32_t* src_bt, int32_t src_bt_stride, const int32_t* dst_bt,
                                 int32_t dst_bt_stride, const int32_t* lens, int32_t batch, const int32_t* kept,
                                 int32_t kept_stride, const int32_t* kept_counts, unsigned* err, cudaStream_t stream);

// ---- block_tables.cu: page pool, block tables and slot maps
int block_tables_max_batch();
cudaError_t launch_block_tables_extend(const int32_t* free_pages, int32_t* pool_state, int32_t num_pages,
                                       int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                       const int32_t* new_lens, int32_t batch, int32_t* seq_lens_after,
                                       int32_t* token_start, int32_t* slot_map, int32_t* positions,
                                       int32_t max_new_tokens, int sm_count, unsigned* err, cudaStream_t stream);
cudaError_t launch_block_tables_release(int32_t* free_pages, int32_t* pool_state, int32_t num_pages,
                                        const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                                        const int32_t* keep_lens, int32_t batch, int32_t* seq_lens_after,
                                        int sm_count, unsigned* err, cudaStream_t stream);

// ---- kv_store.cu: rows of new tokens into their slots (+ summaries when kv.summary is set)
cudaError_t launch_kv_store(const KvView& kv, uint16_t* k_mut, uint16_t* v_mut, const uint16_t* k_new,
                            long long k_stride, const uint16_t* v_new, long long v_stride, const int32_t* slot_map,
                            int32_t num_tokens, int sm_count, unsigned* err, cudaStream_t stream);

// ---- paged_decode.cu: one new token over the whole cache, or over a sink and a recent window
int paged_decode_max_batch();
bool paged_decode_supported(int num_kv_heads, int head_dim, int head_dim_v, int num_q_heads);
// KV heads per TMA box of a call.
int paged_decode_box_heads(int num_kv_heads, int num_q_heads, int head_dim, int32_t bt_stride, int32_t sink_tokens,
                           int32_t recent_tokens, int sm_count);
size_t paged_decode_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim);
// kmap, vmap: the caches as (64 dims, row, 64-dim chunk), boxes of 64 x 16 paged_decode_box_heads x all
// chunks, 128-byte swizzle.
cudaError_t launch_paged_decode(const CUtensorMap& kmap, const CUtensorMap& vmap, const KvView& kv, const uint16_t* q,
                                long long q_stride, int32_t num_q_heads, const int32_t* block_table,
                                int32_t bt_stride, const int32_t* seq_lens, int32_t batch, int32_t sink_tokens,
                                int32_t recent_tokens, float sm_scale, uint16_t* out, float* out_lse, void* workspace,
                                int sm_count, unsigned* err, cudaStream_t stream);

// ---- latent_decode.cu: the same over a latent cache (576-dim rows, value = first 512 dims)
bool paged_latent_supported(int num_kv_heads, int head_dim, int head_dim_v, int num_q_heads);
int paged_latent_max_batch();
size_t paged_latent_workspace_bytes(int32_t num_q_heads);
// kvmap: the cache as (64 dims, row, 64-dim chunk), boxes of 64 x 8 x 9; qmap: the queries as
// [batch][num_q_heads][576], boxes of 64 x num_q_heads x 1 (both 128-byte swizzle).
cudaError_t launch_paged_latent(const CUtensorMap& kvmap, const CUtensorMap& qmap, const KvView& kv,
                                int32_t num_q_heads, const int32_t* block_table, int32_t bt_stride,
                                const int32_t* seq_lens, int32_t batch, int32_t sink_tokens, int32_t recent_tokens,
                                float sm_scale, uint16_t* out, float* out_lse, void* workspace, int sm_count,
                                unsigned* err, cudaStream_t stream);

// ---- rotary.cu: positions into query and key rows
cudaError_t launch_rotary(const uint16_t* q, long long q_stride, int32_t q_heads, const uint16_t* k, long long k_stride,
                          int32_t kv_heads, int32_t dim, int32_t offset, int32_t rot, bool interleaved, bool inverse,
                          const uint64_t* freqs, float amplitude, const int32_t* positions, const int32_t* num_valid,
                          int32_t num_tokens, uint16_t* q_out, long long q_out_stride, uint16_t* k_out,
                          long long k_out_stride, int sm_count, cudaStream_t stream);

// ---- kv8_store.cu: rows of new tokens into an 8-bit cache, and rows of it back
cudaError_t launch_kv8_store(const Kv8View& kv, const uint16_t* k_new, long long k_stride, const uint16_t* v_new,
                             long long v_stride, const int32_t* slot_map, int32_t num_tokens, int sm_count,
                             unsigned* err, cudaStream_t stream);
cudaError_t launch_kv8_load(const Kv8View& kv, const int32_t* block_table, int32_t bt_stride, const int32_t* first,
                            const int32_t* token_start, int32_t batch, int32_t num_rows, uint16_t* k_out,
                            long long k_stride, uint16_t* v_out, long long v_stride, int sm_count, unsigned* err,
                            cudaStream_t stream);

// ---- kv8_decode.cu: one new token over an 8-bit cache
int kv8_decode_max_batch();
bool kv8_decode_supported(int num_kv_heads, int head_dim, int num_q_heads);
// KV heads per TMA box of a call.
int kv8_decode_box_heads(int num_kv_heads, int num_q_heads, int head_dim, int32_t bt_stride, int32_t sink_tokens,
                         int32_t recent_tokens, int batch, int sm_count);
size_t kv8_decode_workspace_bytes(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim);
// kmap, vmap: the caches as (128 bytes, line, 128-byte chunk of a row), 128-byte swizzle; a line is a row (two rows of
// 64 dims), a box the lines of a page's kv8_decode_box_heads heads, all chunks.
cudaError_t launch_kv8_decode(const CUtensorMap& kmap, const CUtensorMap& vmap, const Kv8View& kv, const uint16_t* q,
                              long long q_stride, int32_t num_q_heads, const int32_t* block_table, int32_t bt_stride,
                              const int32_t* seq_lens, int32_t batch, int32_t sink_tokens, int32_t recent_tokens,
                              float sm_scale, uint16_t* out, float* out_lse, void* workspace, int sm_count,
                              unsigned* err, cudaStream_t stream);

// ---- api.cu: per-device context and helpers shared with other entry points
cudaError_t device_context(int* sm_count, unsigned** err);
void set_error_detail(const char* fn, const char* what);
// Argument checks of a sparse paged decode call (everything but the workspace),
// before any launch; *latent tells which kernel serves the shape.
se_status_t check_decode_call(const char* fn, const se_paged_kv_t* kv, const void* q, int32_t num_q_heads,
                              const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens, int32_t batch,
                              const int32_t* sel_pages, const int32_t* sel_counts, int32_t sel_stride,
                              float sm_scale, const void* out, const float* out_lse, bool* latent);

}  // namespace se
