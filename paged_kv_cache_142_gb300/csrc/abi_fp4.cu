// C ABI of the 4-bit cache and of token compaction: argument validation and
// launches.  Declarations and contracts: include/pa.h.
#include <cmath>

#include "decode.cuh"
#include "fp4.cuh"
#include "pa.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool is_float(pa_dtype d) { return d == PA_DTYPE_F32 || d == PA_DTYPE_BF16; }

// a power of two of moderate size: dividing by it and multiplying by it is exact
bool global_scale_ok(float s) {
  int e = 0;
  return s > 0.f && std::isfinite(s) && std::frexp(s, &e) == 0.5f && e >= -31 && e <= 33;
}

pa_status check_pool(int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim) {
  if (num_blocks <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0) return PA_ERR_INVALID_ARG;
  if ((block_size & (block_size - 1)) != 0 || block_size > 256) return PA_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return PA_ERR_UNSUPPORTED;
  // tiles are numbered in 32 bits by the attention kernels
  if (static_cast<int64_t>(num_blocks) * num_kv_heads >= (int64_t(1) << 31)) return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

pa_status check_rows(const void* key, const void* value, pa_dtype dtype, int32_t num_tokens,
                     const int64_t* slot_mapping, const void* k_cache, const void* v_cache, int32_t num_blocks,
                     int32_t block_size, int32_t num_kv_heads, int32_t head_dim, float k_scale, float v_scale,
                     const int32_t* status) {
  const pa_status st = check_pool(num_blocks, block_size, num_kv_heads, head_dim);
  if (st != PA_OK) return st;
  if (num_tokens < 0 || !is_float(dtype) || !global_scale_ok(k_scale) || !global_scale_ok(v_scale))
    return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (!key || !value || !slot_mapping || !k_cache || !v_cache) return PA_ERR_INVALID_ARG;
  if (!aligned(key, 32) || !aligned(value, 32) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(slot_mapping, 8) || !aligned(status, 4))
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

// Positions, and what the kernels round up from them, fit 32 bits.
constexpr int32_t kMaxContext = 1 << 30;

bool group_ok(int32_t num_q_heads, int32_t num_kv_heads) {
  const int g = num_q_heads / num_kv_heads;
  return g == 1 || g == 2 || g == 4 || g == 8 || g == 16;
}

// num_keep: entries of keep, or -1 for what cu_keep says
pa_status compact_impl(void* k_cache, void* v_cache, int64_t cache_layer_stride, int32_t num_layers,
                       int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim, pa_dtype dtype,
                       const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* dst_start,
                       const int32_t* keep, int32_t num_keep, const int32_t* cu_keep, int32_t num_seqs,
                       int32_t max_keep, int32_t* status, void* stream) {
  if (num_blocks <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      (dtype != PA_DTYPE_FP4 && !is_float(dtype)))
    return PA_ERR_INVALID_ARG;
  if ((block_size & (block_size - 1)) != 0 || block_size > 256) return PA_ERR_UNSUPPORTED;
  if (dtype == PA_DTYPE_FP4 && check_pool(num_blocks, block_size, num_kv_heads, head_dim) != PA_OK)
    return PA_ERR_UNSUPPORTED;
  const int64_t e = dtype == PA_DTYPE_F32 ? 4 : (dtype == PA_DTYPE_BF16 ? 2 : 1);
  const int64_t row = dtype == PA_DTYPE_FP4 ? head_dim / 2 : head_dim * e;
  if (dtype != PA_DTYPE_FP4 && (row % 16 != 0 || row > 8192)) return PA_ERR_UNSUPPORTED;
  const int64_t tile = dtype == PA_DTYPE_FP4 ? pa::fp4_tile_bytes(block_size, head_dim) : row * block_size;
  const int64_t layer = tile * num_kv_heads * num_blocks;
  if (num_seqs < 0 || max_keep < 0 || num_keep < -1 || max_blocks_per_seq <= 0 || num_layers < 1 || num_layers > 32767)
    return PA_ERR_INVALID_ARG;
  if (num_layers > 1 && (cache_layer_stride * e < layer || (cache_layer_stride * e) % 16 != 0))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || max_keep == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !dst_start || !keep || !cu_keep) return PA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_tables, 4) || !aligned(dst_start, 4) ||
      !aligned(keep, 4) || !aligned(cu_keep, 4) || !aligned(status, 4))
    return PA_ERR_INVALID_ARG;
  pa::CompactParams p{};
  p.k_cache = static_cast<unsigned char*>(k_cache);
  p.v_cache = static_cast<unsigned char*>(v_cache);
  p.layer_bytes = num_layers > 1 ? cache_layer_stride * e : 0;
  p.block_tables = block_tables;
  p.dst_start = dst_start;
  p.keep = keep;
  p.cu_keep = cu_keep;
  p.status = status;
  p.num_layers = num_layers;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.max_keep = max_keep;
  p.num_keep = num_keep;
  p.row_bytes = static_cast<int32_t>(row);
  p.scale_bytes = dtype == PA_DTYPE_FP4 ? head_dim / 16 : 0;
  p.tile_bytes = tile;
  return pa::launch_compact(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t pa_fp4_tile_bytes(int32_t block_size, int32_t head_dim) {
  return check_pool(1, block_size, 1, head_dim) == PA_OK ? static_cast<size_t>(pa::fp4_tile_bytes(block_size, head_dim))
                                                         : 0;
}

pa_status pa_reshape_and_cache_fp4(const void* key, const void* value, pa_dtype src_dtype, int32_t num_tokens,
                                   const int64_t* slot_mapping, void* k_cache, void* v_cache, int32_t num_blocks,
                                   int32_t block_size, int32_t num_kv_heads, int32_t head_dim, float k_scale,
                                   float v_scale, int32_t* status, void* stream) {
  const pa_status st = check_rows(key, value, src_dtype, num_tokens, slot_mapping, k_cache, v_cache, num_blocks,
                                  block_size, num_kv_heads, head_dim, k_scale, v_scale, status);
  if (st != PA_OK || num_tokens == 0) return st;
  return pa::launch_fp4_append(key, value, src_dtype == PA_DTYPE_BF16, num_tokens, slot_mapping, k_cache, v_cache,
                               num_blocks, block_size, num_kv_heads, head_dim, k_scale, v_scale, status,
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

pa_status pa_gather_cache_fp4(void* key, void* value, pa_dtype dst_dtype, int32_t num_tokens,
                              const int64_t* slot_mapping, const void* k_cache, const void* v_cache,
                              int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                              float k_scale, float v_scale, int32_t* status, void* stream) {
  const pa_status st = check_rows(key, value, dst_dtype, num_tokens, slot_mapping, k_cache, v_cache, num_blocks,
                                  block_size, num_kv_heads, head_dim, k_scale, v_scale, status);
  if (st != PA_OK || num_tokens == 0) return st;
  return pa::launch_fp4_gather(key, value, dst_dtype == PA_DTYPE_BF16, num_tokens, slot_mapping, k_cache, v_cache,
                               num_blocks, block_size, num_kv_heads, head_dim, k_scale, v_scale, status,
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

size_t pa_decode_fp4_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                    int32_t block_size, int32_t max_context_len) {
  if (num_seqs < 0 || num_q_heads <= 0 || max_context_len < 0 ||
      check_pool(1, block_size, num_kv_heads, head_dim) != PA_OK || num_q_heads % num_kv_heads ||
      !group_ok(num_q_heads, num_kv_heads) || max_context_len > kMaxContext)
    return 0;
  return pa::fp4_decode_workspace(num_q_heads, num_kv_heads, head_dim);
}

pa_status pa_decode_fp4(void* out, pa_dtype out_dtype, const void* q, int32_t num_seqs, int32_t num_q_heads,
                        const void* k_cache, const void* v_cache, int32_t num_blocks, int32_t block_size,
                        int32_t num_kv_heads, int32_t head_dim, const int32_t* block_tables,
                        int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t max_context_len, float scale,
                        float k_scale, float v_scale, void* workspace, size_t workspace_bytes, void* stream) {
  const pa_status st = check_pool(num_blocks, block_size, num_kv_heads, head_dim);
  if (st != PA_OK) return st;
  if (!is_float(out_dtype) || !std::isfinite(scale) || !global_scale_ok(k_scale) || !global_scale_ok(v_scale) ||
      num_seqs < 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads || max_blocks_per_seq <= 0 ||
      max_context_len < 0 || static_cast<int64_t>(max_blocks_per_seq) * block_size < max_context_len ||
      !std::isfinite(scale * 1.4426950408889634f * k_scale))
    return PA_ERR_INVALID_ARG;
  if (!group_ok(num_q_heads, num_kv_heads) || max_context_len > kMaxContext) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens) return PA_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4))
    return PA_ERR_INVALID_ARG;
  const size_t need =
      pa_decode_fp4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, max_context_len);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return PA_ERR_WORKSPACE;
  pa::Fp4AttnParams p{};
  p.out = out;
  p.q = q;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.out_bf16 = out_dtype == PA_DTYPE_BF16 ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f * k_scale;
  p.v_scale = v_scale;
  p.err = static_cast<int32_t*>(workspace);
  p.test_stall_ns = pa::test_stall_ns();
  p.ws = static_cast<unsigned char*>(workspace);
  return pa::launch_fp4_decode(p, head_dim, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_prefill_fp4_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                     int32_t block_size, int32_t max_q_len, int32_t max_context_len) {
  if (num_seqs < 0 || num_q_heads <= 0 || max_q_len < 0 || max_context_len < 0 ||
      check_pool(1, block_size, num_kv_heads, head_dim) != PA_OK || num_q_heads % num_kv_heads || head_dim != 128 ||
      !group_ok(num_q_heads, num_kv_heads) || max_context_len > kMaxContext)
    return 0;
  return pa::fp4_prefill_workspace(num_seqs, num_q_heads, num_kv_heads, max_q_len, max_context_len);
}

pa_status pa_prefill_fp4(void* out, pa_dtype out_dtype, const void* q, int32_t num_tokens, const int32_t* cu_q,
                         const int32_t* q_start, int32_t num_seqs, int32_t max_q_len, int32_t max_context_len,
                         int32_t num_q_heads, const void* k_cache, const void* v_cache, int32_t num_blocks,
                         int32_t block_size, int32_t num_kv_heads, int32_t head_dim, const int32_t* block_tables,
                         int32_t max_blocks_per_seq, float scale, float k_scale, float v_scale, int32_t* status,
                         void* workspace, size_t workspace_bytes, void* stream) {
  const pa_status st = check_pool(num_blocks, block_size, num_kv_heads, head_dim);
  if (st != PA_OK) return st;
  if (!is_float(out_dtype) || !(scale > 0.f) || !std::isfinite(scale) || !global_scale_ok(k_scale) ||
      !global_scale_ok(v_scale) || num_tokens < 0 || num_seqs < 0 || max_q_len < 0 || num_q_heads <= 0 ||
      num_q_heads % num_kv_heads || max_blocks_per_seq <= 0 || max_context_len < 0 ||
      static_cast<int64_t>(max_blocks_per_seq) * block_size < max_context_len ||
      !std::isfinite(scale * 1.4426950408889634f * k_scale))
    return PA_ERR_INVALID_ARG;
  if (head_dim != 128 || !group_ok(num_q_heads, num_kv_heads) || max_context_len > kMaxContext)
    return PA_ERR_UNSUPPORTED;
  if (num_tokens == 0 || num_seqs == 0 || max_q_len == 0) return PA_OK;
  if (!out || !q || !cu_q || !q_start || !k_cache || !v_cache || !block_tables) return PA_ERR_INVALID_ARG;
  if (!aligned(out, 32) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(cu_q, 4) ||
      !aligned(q_start, 4) || !aligned(block_tables, 4) || !aligned(status, 4))
    return PA_ERR_INVALID_ARG;
  const size_t need = pa_prefill_fp4_workspace_size(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                                    max_q_len, max_context_len);
  if (need == 0) return PA_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return PA_ERR_WORKSPACE;
  pa::Fp4AttnParams p{};
  p.out = out;
  p.q = q;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.block_tables = block_tables;
  p.cu_q = cu_q;
  p.q_start = q_start;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.num_tokens = num_tokens;
  p.max_q_len = max_q_len;
  p.out_bf16 = out_dtype == PA_DTYPE_BF16 ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f * k_scale;
  p.v_scale = v_scale;
  p.err = status;
  p.ws = static_cast<unsigned char*>(workspace);
  return pa::launch_fp4_prefill(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_compact_tokens(void* k_cache, void* v_cache, int64_t cache_layer_stride, int32_t num_layers,
                            int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                            pa_dtype dtype, const int32_t* block_tables, int32_t max_blocks_per_seq,
                            const int32_t* dst_start, const int32_t* keep, const int32_t* cu_keep, int32_t num_seqs,
                            int32_t max_keep, int32_t* status, void* stream) {
  return compact_impl(k_cache, v_cache, cache_layer_stride, num_layers, num_blocks, block_size, num_kv_heads, head_dim,
                      dtype, block_tables, max_blocks_per_seq, dst_start, keep, -1, cu_keep, num_seqs, max_keep, status,
                      stream);
}

pa_status pa_compact_tokens_checked(void* k_cache, void* v_cache, int64_t cache_layer_stride, int32_t num_layers,
                                    int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                                    pa_dtype dtype, const int32_t* block_tables, int32_t max_blocks_per_seq,
                                    const int32_t* dst_start, const int32_t* keep, int32_t num_keep,
                                    const int32_t* cu_keep, int32_t num_seqs, int32_t max_keep, int32_t* status,
                                    void* stream) {
  if (num_keep < 0) return PA_ERR_INVALID_ARG;
  return compact_impl(k_cache, v_cache, cache_layer_stride, num_layers, num_blocks, block_size, num_kv_heads, head_dim,
                      dtype, block_tables, max_blocks_per_seq, dst_start, keep, num_keep, cu_keep, num_seqs, max_keep,
                      status, stream);
}

}  // extern "C"
