// Causal attention of chunks of queries over the latent cache in its expanded
// form: k[h,t] = (w_k[h] c[t], rope[t]), v[h,t] = w_v[h] c[t], c the latent part
// of a row.  First the keys and values of every head, then the attention.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "decode.cuh"
#include "fp4.cuh"
#include "latent.cuh"
#include "ptx.cuh"

namespace pa {
namespace {

// The first place of each chunk's context in the expanded arrays, a multiple of
// 128; -1 for an empty chunk and for one that is refused.  One CTA; the contexts
// of the chunks before count in 64 bits.
constexpr int kPlanThreads = 512;
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const LatentPrefillParams p, int32_t* base) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int64_t sums[2][kPlanThreads / 32];
  const int64_t table_tokens = static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
  int64_t seen = 0, place = 0;  // contexts and places of the sequences before this round of kPlanThreads
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int64_t len = 0;
    bool bad = false;
    if (s < p.num_seqs) {
      const int64_t b = p.cu_q[s], n = static_cast<int64_t>(p.cu_q[s + 1]) - b, q0 = p.q_start[s];
      bad = n != 0;
      if (n > 0 && n <= p.max_q_len && b >= 0 && b + n <= p.num_tokens && q0 >= 0 && q0 + n <= p.max_context_len &&
          q0 + n <= table_tokens)
        len = q0 + n, bad = false;
    }
    const int64_t padded = (len + 127) / 128 * 128;
    int64_t x = len, y = padded;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) x += u, y += v;
    }
    if (lane == 31) sums[0][warp] = x, sums[1][warp] = y;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += sums[0][w], y += sums[1][w];
    if (s < p.num_seqs) {
      if (seen + x > p.total_context) bad = bad || len > 0, len = 0;
      base[s] = len > 0 ? static_cast<int32_t>(place + y - padded) : -1;
      if (bad && p.status) atomicExch(p.status, kDevErrInvalidArg);
    }
    for (int w = 0; w < kPlanThreads / 32; ++w) seen += sums[0][w], place += sums[1][w];
    __syncthreads();
  }
}

// a block: 8 tokens of a sequence, a head; a thread: a dim of the head's key and value
__global__ void __launch_bounds__(128) expand_kernel(const LatentPrefillParams p, const int32_t* bases, __nv_bfloat16* k, __nv_bfloat16* v) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int seq = blockIdx.z, h = blockIdx.y, t0 = blockIdx.x * 8;
  const int64_t base = bases[seq];
  if (base < 0) return;
  const int len = p.q_start[seq] + p.cu_q[seq + 1] - p.cu_q[seq];
  if (t0 >= len) return;
  __shared__ float c[8][512];
  const int dim = p.latent_dim + p.rope_dim;
  for (int i = threadIdx.x; i < 8 * p.latent_dim; i += 128) {
    const int t = t0 + i / p.latent_dim;
    float x = 0.f;
    if (t < len) {
      int phys = p.block_tables[static_cast<int64_t>(seq) * p.max_blocks_per_seq + t / p.block_size];
      if (phys < 0 || phys >= p.num_blocks) {
        if (p.status) atomicExch(p.status, kDevErrInvalidArg);
        phys = 0;
      }
      x = __bfloat162float(static_cast<const __nv_bfloat16*>(
          p.cache)[(static_cast<int64_t>(phys) * p.block_size + t % p.block_size) * dim + i % p.latent_dim]);
    }
    c[i / p.latent_dim][i % p.latent_dim] = x;
  }
  __syncthreads();
  const int64_t w_at = (static_cast<int64_t>(h) * p.head_dim + threadIdx.x) * p.latent_dim;
  const __nv_bfloat16* wk = static_cast<const __nv_bfloat16*>(p.w_k) + w_at;
  const __nv_bfloat16* wv = static_cast<const __nv_bfloat16*>(p.w_v) + w_at;
  float ak[8] = {}, av[8] = {};
  for (int i = 0; i < p.latent_dim; ++i) {
    const float a = __bfloat162float(wk[i]), b = __bfloat162float(wv[i]);
    for (int j = 0; j < 8; ++j) ak[j] = fmaf(a, c[j][i], ak[j]), av[j] = fmaf(b, c[j][i], av[j]);
  }
  for (int j = 0; j < 8 && t0 + j < len; ++j) {
    const int64_t at = ((base + t0 + j) * p.num_heads + h) * 128 + threadIdx.x;
    k[at] = __float2bfloat16(ak[j]);
    v[at] = __float2bfloat16(av[j]);
  }
}

// a warp: one query row
__global__ void __launch_bounds__(128) attend_kernel(const LatentPrefillParams p, const int32_t* bases, const __nv_bfloat16* k,
                                                     const __nv_bfloat16* v) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int seq = blockIdx.z, h = blockIdx.y, j = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int b = p.cu_q[seq], n = p.cu_q[seq + 1] - b;
  const int64_t base = bases[seq];
  if (base < 0 || j >= n) return;
  const int limit = p.q_start[seq] + j + 1;
  const int64_t row = static_cast<int64_t>(b + j) * p.num_heads + h;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row * 192;
  float qv[6], acc[4] = {};
  for (int i = 0; i < 6; ++i) qv[i] = __bfloat162float(q[i * 32 + lane]) * p.scale_log2;
  float m = -CUDART_INF_F, l = 0.f;
  for (int t = 0; t < limit; ++t) {
    int phys = p.block_tables[static_cast<int64_t>(seq) * p.max_blocks_per_seq + t / p.block_size];
    if (phys < 0 || phys >= p.num_blocks) phys = 0;
    const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(p.cache) +
                             (static_cast<int64_t>(phys) * p.block_size + t % p.block_size) * 576 + 512;
    const int64_t at = ((base + t) * p.num_heads + h) * 128;
    float s = 0.f;
    for (int i = 0; i < 4; ++i) s = fmaf(qv[i], __bfloat162float(k[at + i * 32 + lane]), s);
    for (int i = 0; i < 2; ++i) s = fmaf(qv[4 + i], __bfloat162float(r[i * 32 + lane]), s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mn = fmaxf(m, s), ref = mn == -CUDART_INF_F ? 0.f : mn;
    const float a = exp2f(m - ref), e = exp2f(s - ref);
    l = l * a + e;
    for (int i = 0; i < 4; ++i) acc[i] = fmaf(e, __bfloat162float(v[at + i * 32 + lane]), acc[i] * a);
    m = mn;
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  for (int i = 0; i < 4; ++i) {
    const int64_t at = row * 128 + i * 32 + lane;
    if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(acc[i] * inv);
    else static_cast<float*>(p.out)[at] = acc[i] * inv;
  }
}

}  // namespace

namespace {
int64_t padded_rows(int num_seqs, int64_t total_context) { return (total_context + static_cast<int64_t>(num_seqs) * 127) / 128 * 128; }
int64_t plan_bytes(int num_seqs) { return (static_cast<int64_t>(num_seqs) * 4 + 255) / 256 * 256; }
}  // namespace

size_t latent_prefill_workspace(int num_seqs, int num_heads, int, int, int head_dim, int64_t total_context) {
  return static_cast<size_t>(plan_bytes(num_seqs) + padded_rows(num_seqs, total_context) * num_heads * head_dim * 4);
}

cudaError_t launch_latent_prefill(const LatentPrefillParams& p, cudaStream_t stream) {
  int32_t* base = reinterpret_cast<int32_t*>(p.ws);
  __nv_bfloat16* k = reinterpret_cast<__nv_bfloat16*>(p.ws + plan_bytes(p.num_seqs));
  __nv_bfloat16* v = k + padded_rows(p.num_seqs, p.total_context) * p.num_heads * 128;
  cudaError_t e = launch_early(plan_kernel, dim3(1), kPlanThreads, stream, p, base);
  if (e != cudaSuccess) return e;
  e = launch_early(expand_kernel, dim3((p.max_context_len + 7) / 8, p.num_heads, p.num_seqs), 128, stream, p,
                   static_cast<const int32_t*>(base), k, v);
  if (e != cudaSuccess) return e;
  return launch_early(attend_kernel, dim3((p.max_q_len + 3) / 4, p.num_heads, p.num_seqs), 128, stream, p,
                      static_cast<const int32_t*>(base), static_cast<const __nv_bfloat16*>(k),
                      static_cast<const __nv_bfloat16*>(v));
}

}  // namespace pa
