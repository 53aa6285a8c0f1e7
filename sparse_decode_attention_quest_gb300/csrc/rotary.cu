// Rotary positions of query and key rows (the positions are those that the page
// tables give a batch's new tokens). For pair i of a row at position p,
//     y0 = A (x0 cos a - x1 sin a),  y1 = A (x1 cos a + x0 sin a),  a = p w_i.
//
// Angles: a position far out times a frequency in fp32 loses the angle (p = 10^6:
// a 16th of a radian), and 64-bit floating point is slow here. The frequencies come as
// 64-bit fractions of a turn instead, f_i = w_i / 2 pi * 2^64, and p f_i modulo 2^64
// is the angle's fraction of a turn: the reduction is the integer product's own wrap,
// exact, and its upper 32 bits go to sincospif.
//
// Bound by reading and writing the rows once. A CTA takes a few tokens: it computes
// their cosines and sines once into shared memory (every head of a token uses
// the same ones), then each thread takes pieces of the rows, two 16-byte vectors each:
// both halves of eight pairs, or a vector of the first and one of the second half of
// the interleaved pairs, so that the lanes' vectors lie next to each other, a batch
// of them in flight. Dims that are not turned are copied in a loop of their own
// (beside the others, in the same one, a row of 128 dims with 64 turned took
// 4 x 32K tokens of 40 heads 519 us for a floor of 401).
#include <algorithm>

#include "se_ptx.cuh"

namespace se {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;          // units a thread has in flight
constexpr int kMaxAngles = 2304;   // of a CTA: eight tokens of the widest rows
constexpr int kMaxTile = 64;       // tokens of a CTA

struct RotaryArgs {
  const uint16_t* in[2];   // queries, keys
  uint16_t* out[2];
  long long in_stride[2];
  long long out_stride[2];
  int32_t q_heads, heads;  // of queries, of both
  int32_t dim, offset, pairs;
  int32_t units;           // pieces of a row's turned dims
  int32_t copies;          // vectors of a row that are not turned but written
  uint32_t units_magic;    // of the divisions by units, by copies and by the heads of a CTA (magic_of)
  uint32_t copies_magic;
  uint32_t heads_magic;
  int32_t tile;            // tokens of a CTA
  int32_t tile_heads;      // heads of a CTA
  float amplitude, sign;
  const uint64_t* freqs;
  const int32_t* positions;
  const int32_t* num_valid;
  int32_t num_tokens;
};

// Loads of rows that the same thread may overwrite: not the read-only path.
__device__ __forceinline__ uint4 ld_row_v4(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_row_v2(const uint16_t* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}

// Two pairs, halves apart: words a and b hold x0 and x1 of both.
__device__ __forceinline__ void turn_halves(uint32_t& a, uint32_t& b, float2 c, float2 s) {
  const float a0 = bf16_lo(a), a1 = bf16_hi(a), b0 = bf16_lo(b), b1 = bf16_hi(b);
  a = pack_bf16x2(a0 * c.x - b0 * s.x, a1 * c.y - b1 * s.y);
  b = pack_bf16x2(b0 * c.x + a0 * s.x, b1 * c.y + a1 * s.y);
}
// One pair in a word.
__device__ __forceinline__ uint32_t turn_pair(uint32_t w, float c, float s) {
  const float x0 = bf16_lo(w), x1 = bf16_hi(w);
  return pack_bf16x2(x0 * c - x1 * s, x1 * c + x0 * s);
}

__device__ __forceinline__ uint4 turn_pairs(uint4 x, float4 c, float4 s) {
  return make_uint4(turn_pair(x.x, c.x, s.x), turn_pair(x.y, c.y, s.y), turn_pair(x.z, c.z, s.z),
                    turn_pair(x.w, c.w, s.w));
}
// The first dim of vector v (eight dims) of those that are not turned.
__device__ __forceinline__ int beside(const RotaryArgs& a, int v) {
  return v * 8 < a.offset ? v * 8 : v * 8 + 2 * a.pairs;
}

// n / d by its magic_of(d).
__device__ __forceinline__ int quotient(int n, uint32_t magic) { return magic ? (int)__umulhi((uint32_t)n, magic) : n; }

// Pieces of eight pairs, and of four (8-byte vectors, and one vector) where the pairs are no multiple of eight.
enum Layout { kHalf8, kHalf4, kInterleaved8, kInterleaved4 };

template <int kLayout>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
  __shared__ __align__(16) float cosines[kMaxAngles];
  __shared__ __align__(16) float sines[kMaxAngles];
  __shared__ bool live[kMaxTile];
  pdl_enter();
  const int t0 = blockIdx.x * a.tile;
  const int valid = a.num_valid ? min(*a.num_valid, a.num_tokens) : a.num_tokens;
  const int tokens = min(a.tile, valid - t0);
  if (tokens <= 0) return;
  const int h0 = blockIdx.y * a.tile_heads, heads = min(a.tile_heads, a.heads - h0);
  // Piece e of `each` a row: where it is, and its place in the row.
  struct Place {
    int token, piece, is_k;
    long long in, out;
  };
  auto place_of = [&](int e, int each, uint32_t magic) {
    Place p;
    const int row = quotient(e, magic);
    p.piece = e - row * each;
    p.token = heads == a.tile_heads ? quotient(row, a.heads_magic) : row / heads;
    const int h = h0 + row - p.token * heads, t = t0 + p.token;
    p.is_k = h >= a.q_heads;
    const long long head = (long long)(p.is_k ? h - a.q_heads : h) * a.dim;
    p.in = t * a.in_stride[p.is_k] + head;
    p.out = t * a.out_stride[p.is_k] + head;
    return p;
  };

  // The first pieces are on their way while the angles are computed.
  constexpr int kDims = kLayout == kHalf4 ? 4 : 8;  // of a vector
  const int total = tokens * heads * a.units;
  uint4 x[kBatch], y[kBatch];
  Place at[kBatch];
  auto load = [&](int first) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (first + u * kThreads >= total) continue;
      at[u] = place_of(first + u * kThreads, a.units, a.units_magic);
      const int d = a.offset + at[u].piece * kDims;
      const uint16_t* from = a.in[at[u].is_k] + at[u].in + d;
      at[u].out += d;
      if (kLayout == kHalf4) {
        const uint2 lo = ld_row_v2(from), hi = ld_row_v2(from + a.pairs);
        x[u] = make_uint4(lo.x, lo.y, 0u, 0u);
        y[u] = make_uint4(hi.x, hi.y, 0u, 0u);
      } else {
        x[u] = ld_row_v4(from);
        if (kLayout != kInterleaved4) y[u] = ld_row_v4(from + a.pairs);
      }
    }
  };
  load(threadIdx.x);

  if (threadIdx.x < tokens) live[threadIdx.x] = a.positions[t0 + threadIdx.x] >= 0;
  for (int e = threadIdx.x; e < tokens * a.pairs; e += kThreads) {
    const int tk = e / a.pairs, i = e - tk * a.pairs;
    const uint64_t turns = (uint64_t)(uint32_t)max(a.positions[t0 + tk], 0) * a.freqs[i];
    float s, c;
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
    cosines[e] = c * a.amplitude;
    sines[e] = s * a.amplitude * a.sign;
  }
  __syncthreads();

  for (int first = threadIdx.x; first < total; first += kBatch * kThreads) {
    if (first != threadIdx.x) load(first);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (first + u * kThreads >= total || !live[at[u].token]) continue;
      uint16_t* out = a.out[at[u].is_k] + at[u].out;
      constexpr int kPairs = kLayout == kHalf8 ? 8 : 4;
      const float* cs = cosines + at[u].token * a.pairs + at[u].piece * kPairs;
      const float* sn = sines + at[u].token * a.pairs + at[u].piece * kPairs;
      const float4 c0 = *reinterpret_cast<const float4*>(cs), s0 = *reinterpret_cast<const float4*>(sn);
      if constexpr (kLayout == kInterleaved8 || kLayout == kInterleaved4) {
        *reinterpret_cast<uint4*>(out) = turn_pairs(x[u], c0, s0);
        if constexpr (kLayout == kInterleaved8)
          *reinterpret_cast<uint4*>(out + a.pairs) =
              turn_pairs(y[u], *reinterpret_cast<const float4*>(cs + a.pairs / 2),
                         *reinterpret_cast<const float4*>(sn + a.pairs / 2));
      } else {
        turn_halves(x[u].x, y[u].x, make_float2(c0.x, c0.y), make_float2(s0.x, s0.y));
        turn_halves(x[u].y, y[u].y, make_float2(c0.z, c0.w), make_float2(s0.z, s0.w));
        if constexpr (kLayout == kHalf8) {
          const float4 c1 = *reinterpret_cast<const float4*>(cs + 4), s1 = *reinterpret_cast<const float4*>(sn + 4);
          turn_halves(x[u].z, y[u].z, make_float2(c1.x, c1.y), make_float2(s1.x, s1.y));
          turn_halves(x[u].w, y[u].w, make_float2(c1.z, c1.w), make_float2(s1.z, s1.w));
          *reinterpret_cast<uint4*>(out) = x[u];
          *reinterpret_cast<uint4*>(out + a.pairs) = y[u];
        } else {
          *reinterpret_cast<uint2*>(out) = make_uint2(x[u].x, x[u].y);
          *reinterpret_cast<uint2*>(out + a.pairs) = make_uint2(y[u].x, y[u].y);
        }
      }
    }
  }

  const int copied = tokens * heads * a.copies;
  for (int first = threadIdx.x; first < copied; first += kBatch * kThreads) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (first + u * kThreads >= copied) continue;
      at[u] = place_of(first + u * kThreads, a.copies, a.copies_magic);
      const int d = beside(a, at[u].piece);
      x[u] = ld_row_v4(a.in[at[u].is_k] + at[u].in + d);
      at[u].out += d;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (first + u * kThreads < copied && live[at[u].token])
        *reinterpret_cast<uint4*>(a.out[at[u].is_k] + at[u].out) = x[u];
  }
}

// ceil(2^32 / d), and 0 for d = 1: quotient is exact for n < 2^32 / d.
uint32_t magic_of(int d) { return d == 1 ? 0u : (uint32_t)((0x100000000ull + d - 1) / d); }

}  // namespace

cudaError_t launch_rotary(const uint16_t* q, long long q_stride, int32_t q_heads, const uint16_t* k, long long k_stride,
                          int32_t kv_heads, int32_t dim, int32_t offset, int32_t rot, bool interleaved, bool inverse,
                          const uint64_t* freqs, float amplitude, const int32_t* positions, const int32_t* num_valid,
                          int32_t num_tokens, uint16_t* q_out, long long q_out_stride, uint16_t* k_out,
                          long long k_out_stride, int sm_count, cudaStream_t stream) {
  RotaryArgs a;
  a.in[0] = q;
  a.in[1] = k;
  a.out[0] = q_out;
  a.out[1] = k_out;
  a.in_stride[0] = q_stride;
  a.in_stride[1] = k_stride;
  a.out_stride[0] = q_out_stride;
  a.out_stride[1] = k_out_stride;
  a.q_heads = q_heads;
  a.heads = q_heads + kv_heads;
  a.dim = dim;
  a.offset = offset;
  a.pairs = rot / 2;
  const int layout = interleaved ? (a.pairs % 8 == 0 ? kInterleaved8 : kInterleaved4) : a.pairs % 8 == 0 ? kHalf8 : kHalf4;
  a.units = a.pairs / (a.pairs % 8 == 0 ? 8 : 4);
  // In place nothing else is written. (Queries in place and keys not, or the other way round: copied onto themselves.)
  const bool in_place = (q_heads == 0 || q_out == q) && (kv_heads == 0 || k_out == k);
  a.copies = in_place ? 0 : (dim - rot) / 8;
  a.units_magic = magic_of(a.units);
  a.copies_magic = a.copies ? magic_of(a.copies) : 0u;
  // A few tokens per CTA where there are many; one, its heads shared by several CTAs, where there are few.
  a.tile = 1;
  a.tile_heads = a.heads;
  if (num_tokens >= 16 * sm_count) {
    a.tile = std::max(1, std::min({kMaxTile, kMaxAngles / a.pairs, kBatch * kThreads / (a.heads * a.units)}));
  } else {
    while (a.tile_heads > 1 && a.tile_heads * a.units > kThreads &&
           (long long)num_tokens * ((a.heads + a.tile_heads - 1) / a.tile_heads) < 2 * sm_count)
      a.tile_heads = (a.tile_heads + 1) / 2;
  }
  a.heads_magic = magic_of(a.tile_heads);
  a.amplitude = amplitude;
  a.sign = inverse ? -1.f : 1.f;
  a.freqs = freqs;
  a.positions = positions;
  a.num_valid = num_valid;
  a.num_tokens = num_tokens;
  const dim3 grid((num_tokens + a.tile - 1) / a.tile, (a.heads + a.tile_heads - 1) / a.tile_heads);
  switch (layout) {
    case kHalf8: return launch_pdl(rotary_kernel<kHalf8>, grid, dim3(kThreads), 0, stream, a);
    case kHalf4: return launch_pdl(rotary_kernel<kHalf4>, grid, dim3(kThreads), 0, stream, a);
    case kInterleaved8: return launch_pdl(rotary_kernel<kInterleaved8>, grid, dim3(kThreads), 0, stream, a);
    default: return launch_pdl(rotary_kernel<kInterleaved4>, grid, dim3(kThreads), 0, stream, a);
  }
}

}  // namespace se
