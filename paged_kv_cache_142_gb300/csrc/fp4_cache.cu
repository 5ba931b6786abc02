// Write to and read back from the pages of the 4-bit K/V cache (the format:
// fp4.cuh).  One thread quantises, or restores, the 16 values of one group of
// one token's row of one head; blockIdx.y picks K or V.  The bytes moved bound
// both, once each thread keeps the loads of several tokens in flight and no
// index costs a division: a thread's place in a token's row is found once.
// 32768 tokens of 8 heads x 128 (172 MB): append 36.5 us (4.7 TB/s, 68% of its
// issue slots filled: 105 instructions a group), gather 28 us (6.1 TB/s); one behind the
// other, the gather's start within the append's end, 67 us (72 without).
#include <cuda_bf16.h>

#include "decode.cuh"
#include "fp4.cuh"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;
constexpr int kAppendUnroll = 2, kGatherUnroll = 4;  // tokens a thread works on at a time

struct Fp4RowParams {
  const int64_t* slots;
  int64_t num_slots, tile_bytes;
  int32_t num_tokens, bs_log, hkv, groups_log, groups;  // groups of a token's row of all heads
  int32_t* status;
};

// 32 bytes of global memory
__device__ __forceinline__ void load32(uint32_t (&w)[8], const void* p) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}

// Walks this thread's groups, kUnroll tokens at a time: early(e, row) for
// each, then early2(e, codes, scales) and last(e, row, codes, scales) for those
// whose slot is in the pool.  `row` is the group's number in the tensors of
// rows, codes and scales are its places in the pool.
template <int kUnroll, typename EARLY, typename EARLY2, typename LAST>
__device__ __forceinline__ void each_group(const Fp4RowParams& p, EARLY early, EARLY2 early2, LAST last) {
  const int per_block = p.groups < kThreads ? kThreads / p.groups : 1;  // tokens
  const int tok = p.groups < kThreads ? threadIdx.x / p.groups : 0;
  const int first = p.groups < kThreads ? threadIdx.x - tok * p.groups : threadIdx.x;
  if (tok >= per_block) return;
  const int group_mask = (1 << p.groups_log) - 1;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
  for (int r = first; r < p.groups; r += kThreads) {  // once, unless a token has more groups than the block threads
    const int h = r >> p.groups_log, g = r & group_mask;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * per_block + tok; t0 < p.num_tokens; t0 += step * kUnroll) {
      int64_t slot[kUnroll], codes[kUnroll], scales[kUnroll];
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) {
        const int64_t t = t0 + e * step;
        slot[e] = -1;
        if (t < p.num_tokens) {
          slot[e] = p.slots[t];
          early(e, t * p.groups + r);
        }
      }
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) {
        if (slot[e] >= p.num_slots) {  // past the pool: reported, neither written nor read
          if (p.status && r == 0 && blockIdx.y == 0) atomicExch(p.status, kDevErrInvalidArg);
          slot[e] = -1;
        }
        const int64_t blk = slot[e] >> p.bs_log;
        const int64_t off = slot[e] - (blk << p.bs_log);
        const int64_t tile = (blk * p.hkv + h) * p.tile_bytes;
        codes[e] = tile + (((off << p.groups_log) + g) << 3);
        scales[e] = tile + (int64_t(8) << (p.groups_log + p.bs_log)) + (off << p.groups_log) + g;
        if (slot[e] >= 0) early2(e, codes[e], scales[e]);
      }
#pragma unroll
      for (int e = 0; e < kUnroll; ++e)
        if (slot[e] >= 0) last(e, (t0 + e * step) * p.groups + r, codes[e], scales[e]);
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, BF16 ? 4 : 3)
    fp4_append_kernel(const Fp4RowParams p, const void* __restrict__ key, const void* __restrict__ value,
                      uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache, float k_scale, float v_scale,
                      float k_inv, float v_inv) {
  // a call launched behind this one may begin; it waits for this grid's writes
  // before it reads the cache, as this one waits for the kernel before
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const unsigned char* src = static_cast<const unsigned char*>(blockIdx.y ? value : key);
  uint8_t* cache = blockIdx.y ? v_cache : k_cache;
  const float k = blockIdx.y ? v_scale : k_scale, inv = blockIdx.y ? v_inv : k_inv;
  constexpr int kWords = BF16 ? 1 : 2;  // in eights
  uint32_t w[kAppendUnroll][kWords][8];
  each_group<kAppendUnroll>(
      p,
      [&](int e, int64_t row) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) load32(w[e][i], src + (row * kWords + i) * 32);
      },
      [](int, int64_t, int64_t) {},
      [&](int e, int64_t, int64_t codes, int64_t scales) {
        float x[16];
        uint32_t top = 0;  // largest magnitude's bits
        if (BF16) {
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t u = w[e][0][i];
            m = __vmaxu2(m, u & 0x7fff7fffu);
            x[2 * i] = __uint_as_float(u << 16);
            x[2 * i + 1] = __uint_as_float(u & 0xffff0000u);
          }
          top = max(m << 16, m & 0xffff0000u);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t u = w[e][BF16 ? 0 : i >> 3][i & 7];
            top = max(top, u & 0x7fffffffu);
            x[i] = __uint_as_float(u);
          }
        }
        uint2 c;
        uint32_t sc;
        fp4::quantise16(x, top, k, inv, c, sc);
        *reinterpret_cast<uint2*>(cache + codes) = c;
        cache[scales] = static_cast<uint8_t>(sc);
      });
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    fp4_gather_kernel(const Fp4RowParams p, void* __restrict__ key, void* __restrict__ value,
                      const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache, float k_scale,
                      float v_scale) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  unsigned char* dst = static_cast<unsigned char*>(blockIdx.y ? value : key);
  const uint8_t* cache = blockIdx.y ? v_cache : k_cache;
  const float k = blockIdx.y ? v_scale : k_scale;
  uint2 c[kGatherUnroll];
  uint32_t sc[kGatherUnroll];
  each_group<kGatherUnroll>(
      p, [](int, int64_t) {},
      [&](int e, int64_t codes, int64_t scales) {
        c[e] = *reinterpret_cast<const uint2*>(cache + codes);
        sc[e] = cache[scales];
      },
      [&](int e, int64_t row, int64_t, int64_t) {
        const float s = fp4::scale_to_f32(sc[e]) * k;
        uint32_t h[8], w[16];
        fp4::codes_to_f16(c[e].x, reinterpret_cast<uint32_t(&)[4]>(h[0]));
        fp4::codes_to_f16(c[e].y, reinterpret_cast<uint32_t(&)[4]>(h[4]));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = fp4::f16x2_to_f32(h[i]);
          w[2 * i] = __float_as_uint(f.x * s);
          w[2 * i + 1] = __float_as_uint(f.y * s);
        }
        if (BF16) {  // exact: the values' low 16 bits are zero (NaN keeps its high bits)
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = __byte_perm(w[2 * i], w[2 * i + 1], 0x7632);
          fp4::store32(dst + row * 32, o);
        } else {
          fp4::store32(dst + row * 64, reinterpret_cast<uint32_t(&)[8]>(w[0]));
          fp4::store32(dst + row * 64 + 32, reinterpret_cast<uint32_t(&)[8]>(w[8]));
        }
      });
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
  p.groups_log = __builtin_ctz(static_cast<unsigned>(head_dim / kFp4Group));
  p.groups = num_kv_heads * (head_dim / kFp4Group);
  p.status = status;
  return p;
}

dim3 row_grid(const Fp4RowParams& p, int unroll) {
  const int64_t per_block = p.groups < kThreads ? kThreads / p.groups : 1;
  // every token its own block while that fills the card; then unroll and more
  int64_t blocks = (p.num_tokens + per_block - 1) / per_block;
  const int64_t few = device_sm_count() * 8;
  if (blocks > few) blocks = (blocks + unroll - 1) / unroll > few ? (blocks + unroll - 1) / unroll : few;
  const int64_t cap = device_sm_count() * 64;
  return dim3(static_cast<unsigned>(blocks < cap ? blocks : cap), 2);
}

}  // namespace

cudaError_t launch_fp4_append(const void* key, const void* value, bool src_bf16, int32_t num_tokens,
                              const int64_t* slots, void* k_cache, void* v_cache, int32_t num_blocks,
                              int32_t block_size, int32_t num_kv_heads, int32_t head_dim, float k_scale,
                              float v_scale, int32_t* status, cudaStream_t stream) {
  const Fp4RowParams p = row_params(slots, num_tokens, num_blocks, block_size, num_kv_heads, head_dim, status);
  auto kc = static_cast<uint8_t*>(k_cache), vc = static_cast<uint8_t*>(v_cache);
  return launch_early(src_bf16 ? fp4_append_kernel<true> : fp4_append_kernel<false>, row_grid(p, kAppendUnroll), kThreads,
                      stream, p, key, value, kc, vc, k_scale, v_scale, 1.f / k_scale, 1.f / v_scale);
}

cudaError_t launch_fp4_gather(void* key, void* value, bool dst_bf16, int32_t num_tokens, const int64_t* slots,
                              const void* k_cache, const void* v_cache, int32_t num_blocks, int32_t block_size,
                              int32_t num_kv_heads, int32_t head_dim, float k_scale, float v_scale, int32_t* status,
                              cudaStream_t stream) {
  const Fp4RowParams p = row_params(slots, num_tokens, num_blocks, block_size, num_kv_heads, head_dim, status);
  auto kc = static_cast<const uint8_t*>(k_cache), vc = static_cast<const uint8_t*>(v_cache);
  return launch_early(dst_bf16 ? fp4_gather_kernel<true> : fp4_gather_kernel<false>, row_grid(p, kGatherUnroll), kThreads,
                      stream, p, key, value, kc, vc, k_scale, v_scale);
}

}  // namespace pa
