// The expanded attention for fp32 outputs: keys, values and probabilities stay in
// fp32, on the CUDA cores.  (bf16 outputs: latent_prefill.cu, on the tensor cores.)
//
// A CTA takes 64 queries of a head and walks the keys 32 at a time through shared
// memory.  A warp owns eight queries: a lane forms the eight scores of one key
// (its row against eight broadcast ones), the warp their maxima and sums by
// shuffles, and then a lane the outputs of four dims of the eight rows.
// Shared memory bounds it: 12 of its cycles for the scores of 4 dims against 8 of
// multiplications.
// Measured: 2 x 300 tokens over 8000, 32 heads 6.5 ms (15 TFLOP/s); some 30 times as
// slow as bf16 outputs.  Where queries are few the keys are split: 16 tokens over
// 8000, 16 heads 0.24 ms (2.6 with a CTA for all keys), 783 over 2000, 3 heads 0.24
// (1.3).
#include <cuda_bf16.h>
#include <math_constants.h>

#include "decode.cuh"
#include "fp4.cuh"
#include "latent.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kQueries = 64, kKeys = 32, kRows = 8;  // of a CTA; of a step; of a warp
constexpr int kPitch = 196;                          // floats of a key's row: lanes read 16 bytes a row each, four banks apart
constexpr int kSmemFloats = kQueries * 192 + kKeys * kPitch + kKeys * 128 + kThreads / 32 * kKeys * kRows;

__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
  s = fmaf(a.x, b.x, s);
  s = fmaf(a.y, b.y, s);
  s = fmaf(a.z, b.z, s);
  return fmaf(a.w, b.w, s);
}

// Where the queries do not fill the SMs their keys are split: a CTA leaves its rows
// unnormalised, maxima and sums before them, and a second kernel adds them up.
struct Split {
  int n;      // of a row's keys
  int tiles;  // query tiles of a chunk
  float* ml;  // [sequence][head][tile][split][64][2] maximum (log2), sum
  float* o;   // the same [128]
};
__device__ __forceinline__ int64_t part_row(const Split& c, int heads, int seq, int head, int tile, int split) {
  return (((static_cast<int64_t>(seq) * heads + head) * c.tiles + tile) * c.n + split) * kQueries;
}

__global__ void __launch_bounds__(kThreads, 2) attend_f32_kernel(const LatentPrefillParams p, const LatentExpanded x,
                                                                 const Split c) {
  const int seq = blockIdx.z, head = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = p.cu_q[seq], n = p.cu_q[seq + 1] - b;
  // the longest rows first
  const int split = static_cast<int>(blockIdx.x) % c.n;
  const int q0 = (c.tiles - 1 - static_cast<int>(blockIdx.x) / c.n) * kQueries;
  if (x.tile0[seq + 1] == x.tile0[seq] || q0 >= n) return;
  extern __shared__ __align__(16) float smem[];
  float* sq = smem;
  float* sk = sq + kQueries * 192;
  float* sv = sk + kKeys * kPitch;
  float* sp = sv + kKeys * 128 + warp * kKeys * kRows;  // [key][row] of this warp
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
  const int here = min(kQueries, n - q0);
  for (int i = tid; i < kQueries * 192; i += kThreads) {
    const int r = i / 192;
    const int64_t at = (static_cast<int64_t>(b + q0 + min(r, here - 1)) * p.num_heads + x.head0 + head) * 192 + i % 192;
    sq[i] = r < here ? __bfloat162float(q[at]) * p.scale_log2 : 0.f;
  }
  const int64_t base = static_cast<int64_t>(x.tile0[seq]) * 128;
  const float* gk = reinterpret_cast<const float*>(x.k) + (head * x.rows + base) * 128;
  const float* gv = reinterpret_cast<const float*>(x.v) + (head * x.rows + base) * 128;
  const __nv_bfloat16* gr = reinterpret_cast<const __nv_bfloat16*>(x.rope) + base * 64;
  const int first = p.q_start[seq] + q0;  // position of the first query
  const int steps = (first + here + kKeys - 1) / kKeys;
  const int kbegin = static_cast<int>(static_cast<int64_t>(steps) * split / c.n) * kKeys;
  const int kend = static_cast<int>(static_cast<int64_t>(steps) * (split + 1) / c.n) * kKeys;
  float m[kRows], l[kRows];
  float4 acc[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) m[r] = -CUDART_INF_F, l[r] = 0.f, acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t0 = kbegin; t0 < kend; t0 += kKeys) {
    __syncthreads();
    // (a context's last tile of 128 rows is whole)
    for (int i = tid; i < kKeys * 32; i += kThreads) {
      const int r = i >> 5, c = (i & 31) * 4;
      *reinterpret_cast<float4*>(sk + r * kPitch + c) = __ldg(reinterpret_cast<const float4*>(gk + static_cast<int64_t>(t0 + r) * 128 + c));
      *reinterpret_cast<float4*>(sv + r * 128 + c) = __ldg(reinterpret_cast<const float4*>(gv + static_cast<int64_t>(t0 + r) * 128 + c));
    }
    for (int i = tid; i < kKeys * 64; i += kThreads)
      sk[(i >> 6) * kPitch + 128 + (i & 63)] = __bfloat162float(gr[static_cast<int64_t>(t0 + (i >> 6)) * 64 + (i & 63)]);
    __syncthreads();
    if (warp * kRows >= here) continue;
    float s[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) s[r] = 0.f;
#pragma unroll 4
    for (int d = 0; d < 192; d += 4) {
      const float4 k = *reinterpret_cast<const float4*>(sk + lane * kPitch + d);
#pragma unroll
      for (int r = 0; r < kRows; ++r) s[r] = dot4(*reinterpret_cast<const float4*>(sq + (warp * kRows + r) * 192 + d), k, s[r]);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (t0 + lane > first + warp * kRows + r) s[r] = -CUDART_INF_F;
      float top = s[r];
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float now = fmaxf(m[r], top), ref = now == -CUDART_INF_F ? 0.f : now;
      const float e = exp2f(s[r] - ref), alpha = exp2f(m[r] - ref);
      float sum = e;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[r] = fmaf(l[r], alpha, sum);
      m[r] = now;
      acc[r].x *= alpha, acc[r].y *= alpha, acc[r].z *= alpha, acc[r].w *= alpha;
      s[r] = e;
    }
    *reinterpret_cast<float4*>(sp + lane * kRows) = make_float4(s[0], s[1], s[2], s[3]);
    *reinterpret_cast<float4*>(sp + lane * kRows + 4) = make_float4(s[4], s[5], s[6], s[7]);
    __syncwarp();
#pragma unroll 4
    for (int j = 0; j < kKeys; ++j) {
      const float4 v = *reinterpret_cast<const float4*>(sv + j * 128 + lane * 4);
      const float4 a = *reinterpret_cast<const float4*>(sp + j * kRows), z = *reinterpret_cast<const float4*>(sp + j * kRows + 4);
      const float w[kRows] = {a.x, a.y, a.z, a.w, z.x, z.y, z.z, z.w};
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        acc[r].x = fmaf(w[r], v.x, acc[r].x);
        acc[r].y = fmaf(w[r], v.y, acc[r].y);
        acc[r].z = fmaf(w[r], v.z, acc[r].z);
        acc[r].w = fmaf(w[r], v.w, acc[r].w);
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int j = warp * kRows + r;
    if (j >= here) break;
    if (c.n > 1) {
      const int64_t at = part_row(c, x.heads, seq, head, q0 / kQueries, split) + j;
      if (lane == 0) *reinterpret_cast<float2*>(c.ml + at * 2) = make_float2(m[r], l[r]);
      *reinterpret_cast<float4*>(c.o + at * 128 + lane * 4) = acc[r];
      continue;
    }
    const float inv = l[r] != 0.f ? 1.f / l[r] : 0.f;
    const int64_t at = (static_cast<int64_t>(b + q0 + j) * p.num_heads + x.head0 + head) * 128 + lane * 4;
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) =
        make_float4(acc[r].x * inv, acc[r].y * inv, acc[r].z * inv, acc[r].w * inv);
  }
}

// A warp: a row's parts added up, in the order of the keys.
__global__ void __launch_bounds__(kThreads) join_f32_kernel(const LatentPrefillParams p, const LatentExpanded x, const Split c) {
  const int seq = blockIdx.z, head = blockIdx.y, lane = threadIdx.x & 31;
  const int b = p.cu_q[seq], n = p.cu_q[seq + 1] - b;
  const int row = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (x.tile0[seq + 1] == x.tile0[seq] || row >= n) return;
  float ref = -CUDART_INF_F, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < c.n; ++i) {
    const int64_t at = part_row(c, x.heads, seq, head, row / kQueries, i) + row % kQueries;
    const float2 e = *reinterpret_cast<const float2*>(c.ml + at * 2);
    const float4 y = *reinterpret_cast<const float4*>(c.o + at * 128 + lane * 4);
    if (e.y == 0.f) continue;  // keys that this row does not see
    const float now = fmaxf(ref, e.x), w = exp2f(e.x - now), old = exp2f(ref - now);
    ref = now;
    sum = fmaf(w, e.y, sum * old);
    acc.x = fmaf(w, y.x, acc.x * old);
    acc.y = fmaf(w, y.y, acc.y * old);
    acc.z = fmaf(w, y.z, acc.z * old);
    acc.w = fmaf(w, y.w, acc.w * old);
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  const int64_t at = (static_cast<int64_t>(b + row) * p.num_heads + x.head0 + head) * 128 + lane * 4;
  *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
}

}  // namespace

cudaError_t launch_latent_attend_f32(const LatentPrefillParams& p, const LatentExpanded& x, cudaStream_t stream) {
  const int longest = p.max_q_len < p.num_tokens ? p.max_q_len : p.num_tokens;
  int per_sm = 0;
  const cudaError_t e = fp4_occupancy(reinterpret_cast<const void*>(&attend_f32_kernel), kThreads, kSmemFloats * 4, &per_sm);
  if (e != cudaSuccess) return e;
  Split c{};
  c.n = 1;
  c.tiles = (longest + kQueries - 1) / kQueries;
  // two CTAs an SM; their parts take a quarter of the room that the other form's parts have
  const int64_t ctas = static_cast<int64_t>(c.tiles) * x.heads * p.num_seqs, most = 2 * device_sm_count();
  if (ctas * 2 <= most) {
    const int64_t by_keys = (static_cast<int64_t>(p.max_context_len) + 4 * kKeys - 1) / (4 * kKeys);
    c.n = static_cast<int>(most / ctas < by_keys ? most / ctas : by_keys < 1 ? 1 : by_keys);
    c.ml = x.parts;
    c.o = x.parts + ctas * c.n * kQueries * 2;
  }
  for (int s0 = 0; s0 < p.num_seqs; s0 += 65535) {  // what a grid's third dimension holds
    LatentPrefillParams q = p;
    LatentExpanded y = x;
    q.cu_q += s0, q.q_start += s0, y.tile0 += s0;
    const unsigned seqs = static_cast<unsigned>(p.num_seqs - s0 < 65535 ? p.num_seqs - s0 : 65535);
    attend_f32_kernel<<<dim3(static_cast<unsigned>(c.tiles * c.n), x.heads, seqs), kThreads, kSmemFloats * 4, stream>>>(q, y, c);
    cudaError_t f = cudaGetLastError();
    if (f != cudaSuccess) return f;
    if (c.n == 1) continue;
    join_f32_kernel<<<dim3(static_cast<unsigned>((longest + kThreads / 32 - 1) / (kThreads / 32)), x.heads, seqs), kThreads, 0, stream>>>(q, y, c);
    if ((f = cudaGetLastError()) != cudaSuccess) return f;
  }
  return cudaSuccess;
}

}  // namespace pa
