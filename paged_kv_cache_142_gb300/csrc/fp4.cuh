// The 4-bit K/V page format and the internal interface of its kernels.
//
// A row of head_dim values is cut into groups of 16.  With k the call's global
// scale (a power of two) and a = max |x| / k over a group,
//   s    = a / 6 rounded to e4m3 (nearest even, at most 448)    one byte
//   code = x / k / s rounded to e2m1 (nearest even, at most 6)  four bits
//   the value read back is code * s * k.
// code has 2 significant bits and s has 4, so code * s has at most 6: it is
// exact in bf16 and in f16 (at most 6 * 448, at least 2^-10), and the
// attention kernels multiply exactly the stored values.  A group with a
// non-finite element gets the NaN scale: it reads back as NaN.
//
// A (block, kv head) tile is one run of bytes: block_size rows of D / 2 code
// bytes (element 2i in the low nibble of byte i), block_size rows of D / 16
// scale bytes, padding up to a multiple of 16 bytes.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace pa {

constexpr int kFp4Group = 16;

inline __host__ __device__ int64_t fp4_tile_bytes(int bs, int d) {
  return (static_cast<int64_t>(bs) * (d / 2 + d / kFp4Group) + 15) & ~static_cast<int64_t>(15);
}

struct Fp4AttnParams {
  void* out;
  const void* q;  // bf16
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;  // decode
  const int32_t* cu_q;          // prefill
  const int32_t* q_start;
  int32_t num_seqs, num_q_heads, num_kv_heads, num_blocks, block_size, max_blocks_per_seq;
  int32_t max_context_len;
  int32_t num_tokens, max_q_len;  // prefill
  int32_t out_bf16;
  float scale_log2;  // softmax scale * log2(e) * k_scale
  float v_scale;
  int32_t* err;      // device error word (may be null in prefill)
  uint64_t test_stall_ns;  // decode, timeout-path test hook (0 = off): a wait for what never comes, this long
  unsigned char* ws;
};

// Launches a kernel whose CTAs may start while the one before still drains: it
// calls griddep_wait before it touches memory.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

cudaError_t launch_fp4_append(const void* key, const void* value, bool src_bf16, int32_t num_tokens,
                              const int64_t* slots, void* k_cache, void* v_cache, int32_t num_blocks,
                              int32_t block_size, int32_t num_kv_heads, int32_t head_dim, float k_scale,
                              float v_scale, int32_t* status, cudaStream_t stream);
cudaError_t launch_fp4_gather(void* key, void* value, bool dst_bf16, int32_t num_tokens, const int64_t* slots,
                              const void* k_cache, const void* v_cache, int32_t num_blocks, int32_t block_size,
                              int32_t num_kv_heads, int32_t head_dim, float k_scale, float v_scale, int32_t* status,
                              cudaStream_t stream);
cudaError_t fp4_occupancy(const void* fn, int threads, int smem, int* per_sm);
int64_t fp4_counter_bytes();
size_t fp4_decode_workspace(int num_q_heads, int num_kv_heads, int head_dim);
cudaError_t launch_fp4_decode(const Fp4AttnParams& p, int head_dim, cudaStream_t stream);
size_t fp4_prefill_workspace(int num_seqs, int num_q_heads, int num_kv_heads, int max_q_len, int max_context_len);
cudaError_t launch_fp4_prefill(const Fp4AttnParams& p, cudaStream_t stream);

struct CompactParams {
  // plane i: (i even: k_cache, odd: v_cache) + i / 2 * layer_bytes
  unsigned char* k_cache;
  unsigned char* v_cache;
  int64_t layer_bytes;
  const int32_t* block_tables;
  const int32_t* dst_start;
  const int32_t* keep;
  const int32_t* cu_keep;
  int32_t* status;
  int32_t num_planes, num_blocks, block_size, num_kv_heads, max_blocks_per_seq, num_seqs, max_keep;
  int32_t num_keep;     // entries of keep; -1: what cu_keep says
  int32_t row_bytes;    // one token's row of one head (4-bit pages: its codes)
  int32_t scale_bytes;  // 4-bit pages: its scales, else 0
  int64_t tile_bytes;
};
cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream);

#ifdef __CUDACC__
namespace fp4 {

// 8 codes of a word -> four f16 pairs (element 2i in the low half)
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// two e4m3 scales -> f16 pair (low byte in the low half)
__device__ __forceinline__ uint32_t scales_to_f16(uint32_t two) {
  uint32_t r;
  const uint16_t v = static_cast<uint16_t>(two);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// both halves of a f16 pair as floats
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t v) {
  float2 r;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(v));
  return r;
}
__device__ __forceinline__ float scale_to_f32(uint32_t byte) { return f16x2_to_f32(scales_to_f16(byte)).x; }

// x (>= 0) to the nearest e4m3, ties to even, at most 448
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
// eight values to the nearest e2m1, ties to even, at most 6: their codes, the first in the lowest nibble
__device__ __forceinline__ uint32_t to_e2m1x8(const uint64_t (&t)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .f32 l, h;\n\t"
      "mov.b64 {l, h}, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 a, h, l;\n\t"
      "mov.b64 {l, h}, %2;\n\tcvt.rn.satfinite.e2m1x2.f32 b, h, l;\n\t"
      "mov.b64 {l, h}, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 c, h, l;\n\t"
      "mov.b64 {l, h}, %4;\n\tcvt.rn.satfinite.e2m1x2.f32 d, h, l;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "l"(t[0]), "l"(t[1]), "l"(t[2]), "l"(t[3]));
  return r;
}
// pairs of fp32
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 2^x, and two values rounded to a f16 pair (lo in the low half)
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// 32 bytes of global memory, aligned to as many
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 16 fp32 values -> 8 code bytes and the scale byte, under the global scale k
// (a power of two) with 1 / k = inv.  `top`: the bits of their largest magnitude.
//
// Both roundings are those of the exact quotients.  A quotient x / y is formed
// as q + (x - q y) r, with q = x r and r an approximate 1 / y: the remainder is
// exact, so the result is x / y to within 2^-40 of it, rounded once to fp32.
// A border between two targets is representable, so a quotient that equals one
// comes out equal.  One that does not is off by more than half an fp32 step: the
// border times y has at most 7 significant bits, x differs from it by an fp32
// step at least, and divided by y (below 2^(e+1) by 1/16 or more) that is 0.53
// of a step of the border or more.  So it cannot round onto the border either.
__device__ __forceinline__ void quantise16(float (&x)[16], uint32_t top, float k, float inv, uint2& codes,
                                           uint32_t& scale) {
  if (top >= 0x7f800000u) {  // infinity or NaN among them: the group reads back as NaN
    codes = make_uint2(0, 0);
    scale = 0x7fu;
    return;
  }
  const float a = __uint_as_float(top) * inv;
  if (a > 1e6f) {  // the scale is at its largest, and past 2688 so is the code: no overflow below
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fminf(fmaxf(x[i], -1e6f * k), 1e6f * k);
  }
  const float a6 = fminf(a, 1e6f), q6 = a6 * (1.f / 6.f);
  scale = to_e4m3(fmaf(fmaf(-q6, 6.f, a6), 1.f / 6.f, q6));
  const float s = scale_to_f32(scale);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  r = scale ? r * inv : 0.f;  // k scales exactly
  const uint64_t r2 = pair(r, r), nsk = pair(-s * k, -s * k);
  uint64_t t[2][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t v = pair(x[2 * i], x[2 * i + 1]);
    const uint64_t q = mul2(v, r2);
    t[i >> 2][i & 3] = fma2(fma2(q, nsk, v), r2, q);
  }
  codes.x = to_e2m1x8(t[0]);
  codes.y = to_e2m1x8(t[1]);
}

}  // namespace fp4
#endif

}  // namespace pa
