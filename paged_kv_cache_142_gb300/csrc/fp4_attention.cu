// Attention over the 4-bit pages, one CTA per (query row, query head): every
// thread scores one key of a 128-key tile, then owns dims of the output.  The
// softmax is online (running maximum and sum in fp32, log2 domain).
#include <cuda_bf16.h>
#include <math_constants.h>

#include "decode.cuh"
#include "fp4.cuh"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float warp_max(float v) {
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D>
__device__ void attend(const Fp4AttnParams& p, int64_t row, int head, const int32_t* table, int n) {
  __shared__ float qs[D], ps[kThreads], red[4];
  __shared__ int64_t tile_at[kThreads];
  const int tid = threadIdx.x;
  const int bs = p.block_size;
  const int kvh = head / (p.num_q_heads / p.num_kv_heads);
  const int64_t tile_bytes = fp4_tile_bytes(bs, D);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (row * p.num_q_heads + head) * D;
  for (int d = tid; d < D; d += kThreads) qs[d] = __bfloat162float(q[d]);
  __syncthreads();
  constexpr int kPer = (D + kThreads - 1) / kThreads;
  float m = -CUDART_INF_F, l = 0.f, o[kPer];
  for (int e = 0; e < kPer; ++e) o[e] = 0.f;
  for (int t0 = 0; t0 < n; t0 += kThreads) {
    const int t = t0 + tid;
    float s = -CUDART_INF_F;
    int64_t at = 0;
    if (t < n) {
      int phys = table[t / bs];
      if (phys < 0 || phys >= p.num_blocks) {
        if (p.err) atomicExch(p.err, kDevErrInvalidArg);
        phys = 0;
      }
      at = (static_cast<int64_t>(phys) * p.num_kv_heads + kvh) * tile_bytes;
      const int off = t % bs;
      const uint8_t* codes = p.k_cache + at + off * (D / 2);
      const uint8_t* scales = p.k_cache + at + bs * (D / 2) + off * (D / 16);
      float sum = 0.f;
      for (int g = 0; g < D / 16; ++g) {
        const float sc = fp4::scale_to_f32(scales[g]);
        float part = 0.f;
        for (int w = 0; w < 2; ++w) {
          uint32_t h[4];
          fp4::codes_to_f16(*reinterpret_cast<const uint32_t*>(codes + g * 8 + w * 4), h);
          for (int e = 0; e < 4; ++e) {
            const float2 f = fp4::f16x2_to_f32(h[e]);
            part = fmaf(qs[g * 16 + w * 8 + 2 * e], f.x, part);
            part = fmaf(qs[g * 16 + w * 8 + 2 * e + 1], f.y, part);
          }
        }
        sum = fmaf(part, sc, sum);
      }
      s = sum * p.scale_log2;
    }
    float tm = warp_max(s);
    if ((tid & 31) == 0) red[tid >> 5] = tm;
    __syncthreads();
    tm = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float mn = fmaxf(m, tm);
    const float ref = mn == -CUDART_INF_F ? 0.f : mn;
    const float pr = t < n ? exp2f(s - ref) : 0.f;
    const float corr = exp2f(m - ref);
    ps[tid] = pr;
    tile_at[tid] = at;
    float ts = warp_sum(pr);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = ts;
    __syncthreads();
    l = l * corr + red[0] + red[1] + red[2] + red[3];
    m = mn;
    const int cnt = min(kThreads, n - t0);
    for (int e = 0; e < kPer; ++e) {
      const int d = tid + e * kThreads;
      if (d >= D) continue;
      float acc = o[e] * corr;
      for (int j = 0; j < cnt; ++j) {
        const int off = (t0 + j) % bs;
        const uint8_t* tile = p.v_cache + tile_at[j];
        const uint32_t byte = tile[off * (D / 2) + d / 2];
        const float sc = fp4::scale_to_f32(tile[bs * (D / 2) + off * (D / 16) + d / 16]);
        uint32_t h[4];
        fp4::codes_to_f16(byte, h);
        const float2 f = fp4::f16x2_to_f32(h[0]);
        acc = fmaf(ps[j], ((d & 1) ? f.y : f.x) * sc, acc);
      }
      o[e] = acc;
    }
    __syncthreads();
  }
  for (int e = 0; e < kPer; ++e) {
    const int d = tid + e * kThreads;
    if (d >= D) continue;
    const float v = n > 0 ? o[e] / l * p.v_scale : 0.f;
    const int64_t i = (row * p.num_q_heads + head) * D + d;
    if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[i] = __float2bfloat16_rn(v);
    else static_cast<float*>(p.out)[i] = v;
  }
}

__global__ void __launch_bounds__(kThreads) fp4_prefill_kernel(const Fp4AttnParams p) {
  const int head = blockIdx.x % p.num_q_heads;
  const int j = blockIdx.x / p.num_q_heads, seq = blockIdx.y;
  const int b = p.cu_q[seq], n = p.cu_q[seq + 1] - b, q0 = p.q_start[seq];
  if (j >= n) return;
  const int64_t table_tokens = static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
  const int64_t last = static_cast<int64_t>(q0) + n;
  if (b < 0 || b + n > p.num_tokens || q0 < 0 || last > table_tokens || last > p.max_context_len) {
    if (p.err && threadIdx.x == 0) atomicExch(p.err, kDevErrInvalidArg);
    return;
  }
  attend<128>(p, b + j, head, p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq, q0 + j + 1);
}

}  // namespace

cudaError_t launch_fp4_prefill(const Fp4AttnParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.max_q_len) * static_cast<unsigned>(p.num_q_heads),
                  static_cast<unsigned>(p.num_seqs));
  fp4_prefill_kernel<<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
