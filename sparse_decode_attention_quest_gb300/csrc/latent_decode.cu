// Attention of one new token per request over its whole latent (MLA-style)
// paged cache, or over its first sink and last recent tokens: one 576-dim row per
// token is the key, its first 512 dims the value, shared by all query heads.
//
//     z_j = sm_scale q . k_j over the kept positions j < L,
//     out = sum_j exp(z_j - m) v_j / l,  l = sum_j exp(z_j - m),  lse = m + log l,
// in one pass with a running maximum m and sum l. One CTA per (request, query head).
#include "se_ptx.cuh"

namespace se {
namespace {

constexpr int kThreads = 128;
constexpr float kLn2 = 0.6931471805599453f;

struct LatentArgs {
  KvView kv;
  const uint16_t* q;
  long long q_stride;
  int32_t num_q_heads;
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t* seq_lens;
  int32_t sink, recent;
  float scale_log2;
  uint16_t* out;
  float* out_lse;
  unsigned* err;
};

__global__ void __launch_bounds__(kThreads) paged_latent_kernel(const LatentArgs a) {
  pdl_enter();
  __shared__ float qs[576], sc[kPageSize];
  const int b = blockIdx.x / a.num_q_heads, hq = blockIdx.x % a.num_q_heads;
  const int H = a.kv.num_kv_heads, h = hq / (a.num_q_heads / H), D = a.kv.head_dim, Dv = a.kv.head_dim_v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int c = threadIdx.x; c < D; c += kThreads)
    qs[c] = __uint_as_float((uint32_t)a.q[(size_t)b * a.q_stride + (size_t)hq * D + c] << 16);
  int L = a.seq_lens[b];
  if (L < 0 || L > (long long)a.bt_stride * kPageSize) {
    if (threadIdx.x == 0) raise_error(a.err, SE_DEVERR_LENGTH);
    L = L < 0 ? 0 : a.bt_stride * kPageSize;
  }
  const int lo = a.recent > 0 ? max(0, L - a.recent) : 0;  // kept: j < sink or j >= lo
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p * kPageSize < L; ++p) {
    if (p * kPageSize >= a.sink && (p + 1) * kPageSize <= lo) continue;
    const int phys = a.block_table[(size_t)b * a.bt_stride + p];
    if (phys < 0 || phys >= a.kv.num_pages) {
      if (threadIdx.x == 0) raise_error(a.err, SE_DEVERR_PAGE_RANGE);
      continue;
    }
    const size_t row0 = ((size_t)phys * H + h) * kPageSize;
    for (int i = warp; i < kPageSize; i += kThreads / 32) {
      const int j = p * kPageSize + i;
      const bool kept = j < L && (j < a.sink || j >= lo);
      float s = 0.f;
      if (kept)
        for (int c = lane; c < D; c += 32)
          s += qs[c] * __uint_as_float((uint32_t)a.kv.k[(row0 + i) * a.kv.row_stride_k + c] << 16);
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      if (lane == 0) sc[i] = kept ? s * a.scale_log2 : -INFINITY;
    }
    __syncthreads();
    float n = m;
    for (int i = 0; i < kPageSize; ++i) n = fmaxf(n, sc[i]);
    const float base = n == -INFINITY ? 0.f : n, f = exp2f(m - base);
    m = n;
    l *= f;
    for (int k = 0; k < 4; ++k) o[k] *= f;
    for (int i = 0; i < kPageSize; ++i) {
      const int j = p * kPageSize + i;
      if (!(j < L && (j < a.sink || j >= lo))) continue;
      const float w = exp2f(sc[i] - base);
      l += w;
      for (int k = 0, d = threadIdx.x; d < Dv; ++k, d += kThreads)
        o[k] += w * __uint_as_float((uint32_t)a.kv.v[(row0 + i) * a.kv.row_stride_v + d] << 16);
    }
    __syncthreads();
  }
  const size_t row = (size_t)b * a.num_q_heads + hq;
  const bool empty = l == 0.f;
  for (int k = 0, d = threadIdx.x; d < Dv; ++k, d += kThreads)
    a.out[row * Dv + d] = (uint16_t)(pack_bf16x2(empty ? 0.f : o[k] / l, 0.f) & 0xffffu);
  if (a.out_lse && threadIdx.x == 0) a.out_lse[row] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

bool paged_latent_supported(int num_kv_heads, int head_dim, int head_dim_v, int num_q_heads) {
  return num_kv_heads == 1 && head_dim == 576 && head_dim_v == 512 && num_q_heads % 16 == 0 && num_q_heads >= 16 &&
         num_q_heads <= 64;
}

size_t paged_latent_workspace_bytes(int32_t batch, int32_t num_q_heads) { return 16; }

cudaError_t launch_paged_latent(const KvView& kv, const uint16_t* q, long long q_stride, int32_t num_q_heads,
                                const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens, int32_t batch,
                                int32_t sink_tokens, int32_t recent_tokens, float sm_scale, uint16_t* out,
                                float* out_lse, void* workspace, int sm_count, unsigned* err, cudaStream_t stream) {
  LatentArgs a;
  a.kv = kv;
  a.q = q;
  a.q_stride = q_stride;
  a.num_q_heads = num_q_heads;
  a.block_table = block_table;
  a.bt_stride = bt_stride;
  a.seq_lens = seq_lens;
  a.sink = sink_tokens;
  a.recent = recent_tokens;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.out = out;
  a.out_lse = out_lse;
  a.err = err;
  const cudaError_t e = launch_pdl(paged_latent_kernel, dim3((unsigned)(batch * num_q_heads)), dim3(kThreads), 0, stream, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace se
