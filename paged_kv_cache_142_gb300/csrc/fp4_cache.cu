// Write to and read back from the pages of the 4-bit K/V cache (the format:
// fp4.cuh).  One thread quantises, or restores, one 16-value group of one
// token's row of one head; blockIdx.y picks K or V.  Both are bound by the
// bytes they move.
#include <cuda_bf16.h>

#include "decode.cuh"
#include "fp4.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;

struct Fp4RowParams {
  const int64_t* slots;
  int64_t num_slots, tile_bytes;
  int32_t num_tokens, bs_log, hkv, groups;  // groups: head_dim / 16
  int32_t* status;
};

// The group of work item i: its tile's offset in the pool, its row's place,
// or false for padding and for slots past the pool.
__device__ __forceinline__ bool locate(const Fp4RowParams& p, int64_t i, int64_t& codes, int64_t& scales) {
  const int64_t row = i / p.groups;  // token * hkv + head
  const int g = static_cast<int>(i - row * p.groups);
  const int64_t t = row / p.hkv;
  const int h = static_cast<int>(row - t * p.hkv);
  const int64_t slot = p.slots[t];
  if (slot < 0) return false;
  if (slot >= p.num_slots) {
    if (p.status && g == 0 && h == 0 && blockIdx.y == 0) atomicExch(p.status, kDevErrInvalidArg);
    return false;
  }
  const int64_t blk = slot >> p.bs_log;
  const int off = static_cast<int>(slot - (blk << p.bs_log));
  const int64_t tile = (blk * p.hkv + h) * p.tile_bytes;
  codes = tile + (static_cast<int64_t>(off) * p.groups + g) * 8;
  scales = tile + (static_cast<int64_t>(p.groups * 8) << p.bs_log) + static_cast<int64_t>(off) * p.groups + g;
  return true;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    fp4_append_kernel(Fp4RowParams p, const void* __restrict__ key, const void* __restrict__ value,
                      uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache, float k_inv, float v_inv) {
  const void* src = blockIdx.y ? value : key;
  uint8_t* cache = blockIdx.y ? v_cache : k_cache;
  const float inv = blockIdx.y ? v_inv : k_inv;
  const int64_t total = static_cast<int64_t>(p.num_tokens) * p.hkv * p.groups;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    int64_t codes, scales;
    if (!locate(p, i, codes, scales)) continue;
    uint32_t w[16];  // the values' fp32 bits
    if (BF16) {
      const uint4* s = static_cast<const uint4*>(src) + i * 2;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint4 r = s[v];
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[v * 8 + 2 * e] = u[e] << 16;
          w[v * 8 + 2 * e + 1] = u[e] & 0xffff0000u;
        }
      }
    } else {
      const uint4* s = static_cast<const uint4*>(src) + i * 4;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint4 r = s[v];
        w[4 * v] = r.x;
        w[4 * v + 1] = r.y;
        w[4 * v + 2] = r.z;
        w[4 * v + 3] = r.w;
      }
    }
    uint32_t top = 0;
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      top = max(top, w[e] & 0x7fffffffu);
      x[e] = __uint_as_float(w[e]) * inv;
    }
    uint2 c;
    uint32_t sc;
    fp4::quantise16(x, top, c, sc);
    *reinterpret_cast<uint2*>(cache + codes) = c;
    cache[scales] = static_cast<uint8_t>(sc);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    fp4_gather_kernel(Fp4RowParams p, void* __restrict__ key, void* __restrict__ value,
                      const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache, float k_scale,
                      float v_scale) {
  void* dst = blockIdx.y ? value : key;
  const uint8_t* cache = blockIdx.y ? v_cache : k_cache;
  const float gs = blockIdx.y ? v_scale : k_scale;
  const int64_t total = static_cast<int64_t>(p.num_tokens) * p.hkv * p.groups;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    int64_t codes, scales;
    if (!locate(p, i, codes, scales)) continue;
    const uint2 c = *reinterpret_cast<const uint2*>(cache + codes);
    const float s = fp4::scale_to_f32(cache[scales]) * gs;
    uint32_t h[8];
    fp4::codes_to_f16(c.x, reinterpret_cast<uint32_t(&)[4]>(h[0]));
    fp4::codes_to_f16(c.y, reinterpret_cast<uint32_t(&)[4]>(h[4]));
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 f = fp4::f16x2_to_f32(h[e]);
      w[2 * e] = __float_as_uint(f.x * s);
      w[2 * e + 1] = __float_as_uint(f.y * s);
    }
    if (BF16) {  // exact: the values' low 16 bits are zero (NaN keeps its high bits)
      uint4* d = static_cast<uint4*>(dst) + i * 2;
#pragma unroll
      for (int v = 0; v < 2; ++v)
        d[v] = make_uint4(__byte_perm(w[8 * v], w[8 * v + 1], 0x7632), __byte_perm(w[8 * v + 2], w[8 * v + 3], 0x7632),
                          __byte_perm(w[8 * v + 4], w[8 * v + 5], 0x7632),
                          __byte_perm(w[8 * v + 6], w[8 * v + 7], 0x7632));
    } else {
      uint4* d = static_cast<uint4*>(dst) + i * 4;
#pragma unroll
      for (int v = 0; v < 4; ++v) d[v] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
    }
  }
}

Fp4RowParams row_params(const int64_t* slots, int32_t num_tokens, int32_t num_blocks, int32_t block_size,
                        int32_t num_kv_heads, int32_t head_dim, int32_t* status) {
  Fp4RowParams p{};
  p.slots = slots;
  p.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  p.tile_bytes = fp4_tile_bytes(block_size, head_dim);
  p.num_tokens = num_tokens;
  p.bs_log = __builtin_ctz(static_cast<unsigned>(block_size));
  p.hkv = num_kv_heads;
  p.groups = head_dim / kFp4Group;
  p.status = status;
  return p;
}

dim3 row_grid(const Fp4RowParams& p) {
  const int64_t total = static_cast<int64_t>(p.num_tokens) * p.hkv * p.groups;
  int64_t blocks = (total + kThreads - 1) / kThreads;
  const int64_t cap = device_sm_count() * 32;
  return dim3(static_cast<unsigned>(blocks < cap ? blocks : cap), 2);
}

}  // namespace

cudaError_t launch_fp4_append(const void* key, const void* value, bool src_bf16, int32_t num_tokens,
                              const int64_t* slots, void* k_cache, void* v_cache, int32_t num_blocks,
                              int32_t block_size, int32_t num_kv_heads, int32_t head_dim, float k_scale,
                              float v_scale, int32_t* status, cudaStream_t stream) {
  const Fp4RowParams p = row_params(slots, num_tokens, num_blocks, block_size, num_kv_heads, head_dim, status);
  auto kc = static_cast<uint8_t*>(k_cache), vc = static_cast<uint8_t*>(v_cache);
  if (src_bf16)
    fp4_append_kernel<true><<<row_grid(p), kThreads, 0, stream>>>(p, key, value, kc, vc, 1.f / k_scale, 1.f / v_scale);
  else
    fp4_append_kernel<false><<<row_grid(p), kThreads, 0, stream>>>(p, key, value, kc, vc, 1.f / k_scale, 1.f / v_scale);
  return cudaGetLastError();
}

cudaError_t launch_fp4_gather(void* key, void* value, bool dst_bf16, int32_t num_tokens, const int64_t* slots,
                              const void* k_cache, const void* v_cache, int32_t num_blocks, int32_t block_size,
                              int32_t num_kv_heads, int32_t head_dim, float k_scale, float v_scale, int32_t* status,
                              cudaStream_t stream) {
  const Fp4RowParams p = row_params(slots, num_tokens, num_blocks, block_size, num_kv_heads, head_dim, status);
  auto kc = static_cast<const uint8_t*>(k_cache), vc = static_cast<const uint8_t*>(v_cache);
  if (dst_bf16)
    fp4_gather_kernel<true><<<row_grid(p), kThreads, 0, stream>>>(p, key, value, kc, vc, k_scale, v_scale);
  else
    fp4_gather_kernel<false><<<row_grid(p), kThreads, 0, stream>>>(p, key, value, kc, vc, k_scale, v_scale);
  return cudaGetLastError();
}

}  // namespace pa
