// Attention over the latent cache in its absorbed form.
//   s[h,t] = scale q[h] . row[t],  out[h] = sum_t softmax(s)[t] row[t][:latent]
// A warp for each query row; its lanes share the row's dims.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "decode.cuh"
#include "fp4.cuh"
#include "latent.cuh"
#include "ptx.cuh"

namespace pa {
namespace {

__global__ void __launch_bounds__(128) latent_decode_kernel(const LatentDecodeParams p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int64_t per_seq = static_cast<int64_t>(p.q_len) * p.num_heads;
  if (row >= per_seq * p.num_seqs) return;
  const int seq = static_cast<int>(row / per_seq);
  const int j = static_cast<int>(row % per_seq) / p.num_heads;
  const int dim = p.latent_dim + p.rope_dim, mine = dim / 32;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row * dim;
  float qv[18], acc[18];
  for (int i = 0; i < mine; ++i) qv[i] = __bfloat162float(q[i * 32 + lane]) * p.scale_log2, acc[i] = 0.f;
  float m = -CUDART_INF_F, l = 0.f;
  int len = p.context_lens[seq];
  if (len > p.max_context_len || len < 0) {
    if (lane == 0) atomicExch(p.err, kDevErrInvalidArg);
    len = 0;
  }
  const int limit = len - p.q_len + 1 + j;
  const int32_t* table = p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq;
  for (int t = 0; t < limit; ++t) {
    int phys = table[t / p.block_size];
    if (phys < 0 || phys >= p.num_blocks) {
      if (lane == 0) atomicExch(p.err, kDevErrInvalidArg);
      phys = 0;
    }
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(p.cache) +
                             (static_cast<int64_t>(phys) * p.block_size + t % p.block_size) * dim;
    float s = 0.f, kv[18];
    for (int i = 0; i < mine; ++i) kv[i] = __bfloat162float(k[i * 32 + lane]), s = fmaf(qv[i], kv[i], s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mn = fmaxf(m, s), ref = mn == -CUDART_INF_F ? 0.f : mn;
    const float a = exp2f(m - ref), e = exp2f(s - ref);
    l = l * a + e;
    for (int i = 0; i < mine; ++i) acc[i] = fmaf(e, kv[i], acc[i] * a);
    m = mn;
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  for (int i = 0; i < p.latent_dim / 32; ++i) {
    const int64_t at = row * p.latent_dim + i * 32 + lane;
    if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(acc[i] * inv);
    else static_cast<float*>(p.out)[at] = acc[i] * inv;
  }
}

}  // namespace

size_t latent_decode_workspace(int, int, int, int) { return 256; }

cudaError_t launch_latent_decode(const LatentDecodeParams& p, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.q_len * p.num_heads;
  return launch_early(latent_decode_kernel, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, stream, p);
}

}  // namespace pa
