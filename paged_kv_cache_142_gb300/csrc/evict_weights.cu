// Accumulated attention weights: weights[t] += sum over a window's queries and
// heads of softmax_t(scale q . k[t]).  First each row's maximum and sum, then
// each token's probabilities added up.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "decode.cuh"
#include "fp4.cuh"
#include "latent.cuh"
#include "ptx.cuh"

namespace pa {
namespace {

__device__ __forceinline__ const __nv_bfloat16* key_at(const WeightsParams& p, int seq, int kvh, int t, bool report) {
  int phys = p.block_tables[static_cast<int64_t>(seq) * p.max_blocks_per_seq + t / p.block_size];
  if (phys < 0 || phys >= p.num_blocks) {
    if (report) atomicExch(p.err, kDevErrInvalidArg);
    phys = 0;
  }
  return static_cast<const __nv_bfloat16*>(p.k_cache) +
         ((static_cast<int64_t>(phys) * p.num_kv_heads + kvh) * p.block_size + t % p.block_size) * p.head_dim;
}
__device__ __forceinline__ int length_of(const WeightsParams& p, int seq) {
  const int len = p.context_lens[seq];
  if (len >= 0 && len <= p.max_context_len) return len;
  atomicExch(p.err, kDevErrInvalidArg);
  return 0;
}

// a warp: a query row's log2 of its sum of exponentials
__global__ void __launch_bounds__(128) stats_kernel(const WeightsParams p, float* lse) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t per_seq = static_cast<int64_t>(p.window) * p.num_q_heads;
  if (row >= per_seq * p.num_seqs) return;
  const int seq = static_cast<int>(row / per_seq), r = static_cast<int>(row % per_seq);
  const int w = r / p.num_q_heads, h = r % p.num_q_heads, kvh = h / (p.num_q_heads / p.num_kv_heads);
  const int mine = p.head_dim / 32;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row * p.head_dim;
  float qv[18];
  for (int i = 0; i < mine; ++i) qv[i] = __bfloat162float(q[i * 32 + lane]) * p.scale_log2;
  const int limit = length_of(p, seq) - p.window + 1 + w;
  float m = -CUDART_INF_F, l = 0.f;
  for (int t = 0; t < limit; ++t) {
    const __nv_bfloat16* k = key_at(p, seq, kvh, t, lane == 0);
    float s = 0.f;
    for (int i = 0; i < mine; ++i) s = fmaf(qv[i], __bfloat162float(k[i * 32 + lane]), s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mn = fmaxf(m, s), ref = mn == -CUDART_INF_F ? 0.f : mn;
    l = l * exp2f(m - ref) + exp2f(s - ref);
    m = mn;
  }
  if (lane == 0) lse[row] = limit > 0 ? m + log2f(l) : CUDART_INF_F;
}

// a warp: a token, row after row
__global__ void __launch_bounds__(128) add_kernel(const WeightsParams p, const float* lse) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, seq = blockIdx.y, t = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int len = length_of(p, seq);
  if (t >= len) return;
  const int mine = p.head_dim / 32, group = p.num_q_heads / p.num_kv_heads;
  float total = 0.f;
  for (int kvh = 0; kvh < p.num_kv_heads; ++kvh) {
    const __nv_bfloat16* k = key_at(p, seq, kvh, t, false);
    float kv[18];
    for (int i = 0; i < mine; ++i) kv[i] = __bfloat162float(k[i * 32 + lane]) * p.scale_log2;
    for (int w = max(0, t + p.window - len); w < p.window; ++w)
      for (int g = 0; g < group; ++g) {
        const int64_t row = (static_cast<int64_t>(seq) * p.window + w) * p.num_q_heads + kvh * group + g;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row * p.head_dim;
        float s = 0.f;
        for (int i = 0; i < mine; ++i) s = fmaf(kv[i], __bfloat162float(q[i * 32 + lane]), s);
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        total += exp2f(s - lse[row]);
      }
  }
  if (lane == 0) p.weights[seq * p.weights_stride + t] += total;
}

}  // namespace

size_t weights_workspace(int num_seqs, int window, int num_q_heads, int, int, int) {
  return 256 + static_cast<size_t>(num_seqs) * window * num_q_heads * 4;
}

cudaError_t launch_weights(const WeightsParams& p, cudaStream_t stream) {
  float* lse = reinterpret_cast<float*>(p.ws + 256);
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.window * p.num_q_heads;
  const cudaError_t e = launch_early(stats_kernel, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, stream, p, lse);
  if (e != cudaSuccess) return e;
  return launch_early(add_kernel, dim3((p.max_context_len + 3) / 4, p.num_seqs), 128, stream, p,
                      static_cast<const float*>(lse));
}

}  // namespace pa
