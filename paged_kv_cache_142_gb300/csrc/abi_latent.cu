// C ABI of the latent cache and of eviction by attention weight: argument
// validation and launches.  Declarations and contracts: include/pa.h.
#include <cmath>

#include "decode.cuh"
#include "fp4.cuh"
#include "latent.cuh"
#include "pa.h"

namespace {

constexpr float kLog2e = 1.4426950408889634f;
// Positions, and what the kernels round up from them, fit 32 bits.
constexpr int32_t kMaxContext = 1 << 30;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool is_float(pa_dtype d) { return d == PA_DTYPE_F32 || d == PA_DTYPE_BF16; }
int64_t bytes_of(pa_dtype d) { return d == PA_DTYPE_F32 ? 4 : 2; }

// a pool of latent rows for copies: any dims whose parts are whole 16-byte pieces
pa_status check_rows(int32_t num_blocks, int32_t block_size, int32_t latent_dim, int32_t rope_dim, pa_dtype dtype) {
  if (num_blocks <= 0 || block_size <= 0 || latent_dim <= 0 || rope_dim <= 0 || !is_float(dtype))
    return PA_ERR_INVALID_ARG;
  if ((block_size & (block_size - 1)) != 0 || block_size > 256) return PA_ERR_UNSUPPORTED;
  const int64_t e = bytes_of(dtype);
  if (latent_dim * e % 16 || rope_dim * e % 16 || (static_cast<int64_t>(latent_dim) + rope_dim) * e > 8192)
    return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

// what the attention kernels take
pa_status check_attention(int32_t num_blocks, int32_t block_size, int32_t latent_dim, int32_t rope_dim) {
  const pa_status st = check_rows(num_blocks, block_size, latent_dim, rope_dim, PA_DTYPE_BF16);
  if (st != PA_OK) return st;
  return latent_dim == 512 && rope_dim == 64 && block_size >= 8 ? PA_OK : PA_ERR_UNSUPPORTED;
}

// a pool's rows are numbered in 32 bits by the tensor loads
bool pool_ok(int64_t tiles, int32_t block_size) { return tiles * block_size < (int64_t(1) << 31); }

bool table_ok(int32_t max_blocks_per_seq, int32_t block_size, int32_t max_context_len) {
  return max_blocks_per_seq > 0 && max_context_len >= 0 &&
         static_cast<int64_t>(max_blocks_per_seq) * block_size >= max_context_len;
}

}  // namespace

extern "C" {

pa_status pa_reshape_and_cache_latent(const void* latent, int64_t latent_stride, const void* rope, int64_t rope_stride,
                                      int32_t num_tokens, const int64_t* slot_mapping, void* cache, int32_t num_blocks,
                                      int32_t block_size, int32_t latent_dim, int32_t rope_dim, pa_dtype dtype,
                                      int32_t* status, void* stream) {
  const pa_status st = check_rows(num_blocks, block_size, latent_dim, rope_dim, dtype);
  if (st != PA_OK) return st;
  const int64_t e = bytes_of(dtype);
  if (num_tokens < 0) return PA_ERR_INVALID_ARG;
  if (num_tokens > 1 && (latent_stride < latent_dim || rope_stride < rope_dim || latent_stride * e % 16 ||
                         rope_stride * e % 16))
    return PA_ERR_INVALID_ARG;
  if (num_tokens == 0) return PA_OK;
  if (!latent || !rope || !slot_mapping || !cache) return PA_ERR_INVALID_ARG;
  if (!aligned(latent, 16) || !aligned(rope, 16) || !aligned(cache, 16) || !aligned(slot_mapping, 8) ||
      !aligned(status, 4))
    return PA_ERR_INVALID_ARG;
  return pa::launch_latent_append(latent, latent_stride * e, rope, rope_stride * e, num_tokens, slot_mapping, cache,
                                  static_cast<int64_t>(num_blocks) * block_size, static_cast<int32_t>(latent_dim * e),
                                  static_cast<int32_t>(rope_dim * e), status,
                                  static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

pa_status pa_copy_blocks_latent(void* cache, int64_t cache_layer_stride, int32_t num_layers, int32_t num_blocks,
                                int32_t block_size, int32_t latent_dim, int32_t rope_dim, pa_dtype dtype,
                                const int64_t* block_pairs, int32_t num_pairs, int32_t* status, void* stream) {
  const pa_status st = check_rows(num_blocks, block_size, latent_dim, rope_dim, dtype);
  if (st != PA_OK) return st;
  const int64_t e = bytes_of(dtype);
  const int64_t block = (static_cast<int64_t>(latent_dim) + rope_dim) * block_size * e;
  if (num_pairs < 0 || num_layers < 1 || num_layers > 32767) return PA_ERR_INVALID_ARG;
  if (num_layers > 1 && (cache_layer_stride * e < block * num_blocks || cache_layer_stride * e % 16 != 0))
    return PA_ERR_INVALID_ARG;
  if (num_pairs == 0) return PA_OK;
  if (!cache || !block_pairs) return PA_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || !aligned(block_pairs, 8) || !aligned(status, 4)) return PA_ERR_INVALID_ARG;
  const int64_t layer = num_layers > 1 ? cache_layer_stride * e : 0;
  return pa::launch_copy_blocks(cache, static_cast<unsigned char*>(cache) + layer, 2 * layer, num_layers, num_blocks,
                                block, block_pairs, num_pairs, status,
                                static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

pa_status pa_compact_tokens_latent(void* cache, int64_t cache_layer_stride, int32_t num_layers, int32_t num_blocks,
                                   int32_t block_size, int32_t latent_dim, int32_t rope_dim, pa_dtype dtype,
                                   const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* dst_start,
                                   const int32_t* keep, int32_t num_keep, const int32_t* cu_keep, int32_t num_seqs,
                                   int32_t max_keep, int32_t* status, void* stream) {
  const pa_status st = check_rows(num_blocks, block_size, latent_dim, rope_dim, dtype);
  if (st != PA_OK) return st;
  const int64_t e = bytes_of(dtype), row = (static_cast<int64_t>(latent_dim) + rope_dim) * e;
  if (num_seqs < 0 || max_keep < 0 || num_keep < 0 || max_blocks_per_seq <= 0 || num_layers < 1 || num_layers > 32767)
    return PA_ERR_INVALID_ARG;
  if (num_layers > 1 && (cache_layer_stride * e < row * block_size * num_blocks || cache_layer_stride * e % 16 != 0))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  // no sequence may keep a token: a launch moves nothing and only reports those that do
  const bool nothing = max_keep == 0;
  if (nothing && !status) return PA_OK;
  if (!dst_start || !cu_keep || (!nothing && (!cache || !block_tables || !keep))) return PA_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || !aligned(block_tables, 4) || !aligned(dst_start, 4) || !aligned(keep, 4) ||
      !aligned(cu_keep, 4) || !aligned(status, 4))
    return PA_ERR_INVALID_ARG;
  const int64_t layer = num_layers > 1 ? cache_layer_stride * e : 0;
  pa::CompactParams p{};
  p.k_cache = static_cast<unsigned char*>(cache);
  p.v_cache = p.k_cache + layer;
  p.layer_bytes = 2 * layer;
  p.num_planes = num_layers;
  p.block_tables = block_tables;
  p.dst_start = dst_start;
  p.keep = keep;
  p.cu_keep = cu_keep;
  p.status = status;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.num_kv_heads = 1;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.max_keep = max_keep;
  p.num_keep = num_keep;
  p.row_bytes = static_cast<int32_t>(row);
  p.tile_bytes = row * block_size;
  return pa::launch_compact(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_decode_latent_workspace_size(int32_t num_seqs, int32_t q_len, int32_t num_heads, int32_t latent_dim,
                                       int32_t rope_dim, int32_t block_size, int32_t max_context_len) {
  if (num_seqs < 0 || q_len <= 0 || num_heads <= 0 || num_heads > 128 || max_context_len < 0 ||
      max_context_len > kMaxContext || check_attention(1, block_size, latent_dim, rope_dim) != PA_OK ||
      static_cast<int64_t>(num_seqs) * q_len * num_heads >= (int64_t(1) << 31))
    return 0;
  return pa::latent_decode_workspace(num_seqs, q_len, num_heads, max_context_len);
}

pa_status pa_decode_latent(void* out, pa_dtype out_dtype, const void* q, int32_t num_seqs, int32_t q_len,
                           int32_t num_heads, const void* cache, int32_t num_blocks, int32_t block_size,
                           int32_t latent_dim, int32_t rope_dim, const int32_t* block_tables,
                           int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t max_context_len,
                           float scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (num_blocks <= 0 || block_size <= 0 || latent_dim <= 0 || rope_dim <= 0 || !is_float(out_dtype) ||
      !std::isfinite(scale * kLog2e) || num_seqs < 0 || q_len <= 0 || num_heads <= 0 ||
      !table_ok(max_blocks_per_seq, block_size, max_context_len))
    return PA_ERR_INVALID_ARG;
  const size_t need = pa_decode_latent_workspace_size(num_seqs, q_len, num_heads, latent_dim, rope_dim, block_size,
                                                      max_context_len);
  if (need == 0 || !pool_ok(num_blocks, block_size)) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  if (!out || !q || !cache || !block_tables || !context_lens) return PA_ERR_INVALID_ARG;
  if (!aligned(out, 32) || !aligned(q, 16) || !aligned(cache, 16) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4))
    return PA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return PA_ERR_WORKSPACE;
  pa::LatentDecodeParams p{};
  p.out = out;
  p.q = q;
  p.cache = cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.num_seqs = num_seqs;
  p.q_len = q_len;
  p.num_heads = num_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.out_bf16 = out_dtype == PA_DTYPE_BF16 ? 1 : 0;
  p.scale_log2 = scale * kLog2e;
  p.err = static_cast<int32_t*>(workspace);
  p.ws = static_cast<unsigned char*>(workspace);
  p.test_stall_ns = pa::test_stall_ns();
  return pa::launch_latent_decode(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_prefill_latent_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t latent_dim, int32_t rope_dim,
                                        int32_t head_dim, int32_t block_size, int32_t max_q_len,
                                        int32_t max_context_len, int64_t total_context) {
  if (num_seqs < 0 || num_heads <= 0 || num_heads > 65535 || max_q_len < 0 || max_context_len < 0 ||
      max_context_len > kMaxContext || total_context < 0 || head_dim != 128 ||
      total_context + static_cast<int64_t>(num_seqs) * 128 >= (int64_t(1) << 31) ||
      check_attention(1, block_size, latent_dim, rope_dim) != PA_OK)
    return 0;
  return pa::latent_prefill_workspace(num_seqs, num_heads, head_dim, total_context);
}

pa_status pa_prefill_latent(void* out, pa_dtype out_dtype, const void* q, int32_t num_tokens, const int32_t* cu_q,
                            const int32_t* q_start, int32_t num_seqs, int32_t max_q_len, int32_t max_context_len,
                            int64_t total_context, int32_t num_heads, const void* cache, int32_t num_blocks,
                            int32_t block_size, int32_t latent_dim, int32_t rope_dim, const void* w_k, const void* w_v,
                            int32_t head_dim, const int32_t* block_tables, int32_t max_blocks_per_seq, float scale,
                            int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  if (num_blocks <= 0 || block_size <= 0 || latent_dim <= 0 || rope_dim <= 0 || head_dim <= 0 ||
      !is_float(out_dtype) || !(scale > 0.f) || !std::isfinite(scale * kLog2e) || num_tokens < 0 || num_seqs < 0 ||
      max_q_len < 0 || num_heads <= 0 || total_context < 0 ||
      !table_ok(max_blocks_per_seq, block_size, max_context_len))
    return PA_ERR_INVALID_ARG;
  const size_t need = pa_prefill_latent_workspace_size(num_seqs, num_heads, latent_dim, rope_dim, head_dim, block_size,
                                                       max_q_len, max_context_len, total_context);
  if (need == 0 || !pool_ok(num_blocks, block_size)) return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  // no chunk may have a token: the plan alone runs, and reports those that do
  const bool nothing = num_tokens == 0 || max_q_len == 0;
  if (nothing && !status) return PA_OK;
  if (!cu_q || !q_start || (!nothing && (!out || !q || !cache || !w_k || !w_v || !block_tables)))
    return PA_ERR_INVALID_ARG;
  if (!aligned(out, 32) || !aligned(q, 16) || !aligned(cache, 16) || !aligned(w_k, 16) || !aligned(w_v, 16) ||
      !aligned(cu_q, 4) || !aligned(q_start, 4) || !aligned(block_tables, 4) || !aligned(status, 4))
    return PA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return PA_ERR_WORKSPACE;
  pa::LatentPrefillParams p{};
  p.out = out;
  p.q = q;
  p.cache = cache;
  p.w_k = w_k;
  p.w_v = w_v;
  p.cu_q = cu_q;
  p.q_start = q_start;
  p.block_tables = block_tables;
  p.total_context = total_context;
  p.num_tokens = num_tokens;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_q_len = max_q_len;
  p.max_context_len = max_context_len;
  p.out_bf16 = out_dtype == PA_DTYPE_BF16 ? 1 : 0;
  p.scale_log2 = scale * kLog2e;
  p.status = status;
  p.ws = static_cast<unsigned char*>(workspace);
  p.test_stall_ns = pa::test_stall_ns();
  return pa::launch_latent_prefill(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t pa_accumulate_weights_workspace_size(int32_t num_seqs, int32_t window, int32_t num_q_heads,
                                            int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                            int32_t max_context_len) {
  if (num_seqs < 0 || num_seqs > 65535 || window <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      num_q_heads % num_kv_heads || max_context_len < 0 || max_context_len > kMaxContext || block_size < 8 ||
      block_size > 256 || (block_size & (block_size - 1)) != 0 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256 && head_dim != 576) || num_q_heads / num_kv_heads > 128 ||
      static_cast<int64_t>(num_seqs) * window * num_q_heads >= (int64_t(1) << 31))
    return 0;
  return pa::weights_workspace(num_seqs, window, num_q_heads, num_kv_heads, head_dim, max_context_len);
}

pa_status pa_accumulate_weights(float* weights, int64_t weights_stride, const void* q, int32_t num_seqs,
                                int32_t window, int32_t num_q_heads, const void* k_cache, int32_t num_blocks,
                                int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                                const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
                                int32_t max_context_len, float scale, void* workspace, size_t workspace_bytes,
                                void* stream) {
  if (num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0 || !std::isfinite(scale * kLog2e) ||
      num_seqs < 0 || window <= 0 || num_q_heads <= 0 || num_q_heads % num_kv_heads ||
      !table_ok(max_blocks_per_seq, block_size, max_context_len) || (num_seqs > 1 && weights_stride < max_context_len))
    return PA_ERR_INVALID_ARG;
  const size_t need = pa_accumulate_weights_workspace_size(num_seqs, window, num_q_heads, num_kv_heads, head_dim,
                                                           block_size, max_context_len);
  if (need == 0 || !pool_ok(static_cast<int64_t>(num_blocks) * num_kv_heads, block_size)) return PA_ERR_UNSUPPORTED;
  // (bounds of 0: nothing is added, and the call only reports lengths that pass them)
  if (num_seqs == 0 || (max_context_len == 0 && !weights)) return PA_OK;
  if (!weights || !q || !k_cache || !block_tables || !context_lens) return PA_ERR_INVALID_ARG;
  if (!aligned(weights, 4) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4))
    return PA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return PA_ERR_WORKSPACE;
  pa::WeightsParams p{};
  p.weights = weights;
  p.weights_stride = weights_stride;
  p.q = q;
  p.k_cache = k_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.num_seqs = num_seqs;
  p.window = window;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.head_dim = head_dim;
  p.scale_log2 = scale * kLog2e;
  p.err = static_cast<int32_t*>(workspace);
  p.ws = static_cast<unsigned char*>(workspace);
  p.test_stall_ns = pa::test_stall_ns();
  return pa::launch_weights(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_select_tokens(int32_t* keep, int32_t num_keep, const int32_t* cu_keep, float* weights,
                           int64_t weights_stride, const int32_t* dst_start, const int32_t* context_lens,
                           int32_t num_seqs, int32_t recent, int32_t max_context_len, int32_t* status, void* stream) {
  if (num_keep < 0 || num_seqs < 0 || recent < 0 || max_context_len < 0 ||
      (num_seqs > 1 && weights_stride < max_context_len))
    return PA_ERR_INVALID_ARG;
  if (max_context_len > kMaxContext || static_cast<int64_t>(num_seqs) * 8 >= (int64_t(1) << 31))
    return PA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PA_OK;
  // no sequence may have a token: a launch writes nothing and only reports those that do
  if (max_context_len == 0 && !status) return PA_OK;
  if ((!keep && num_keep > 0) || !cu_keep || (!weights && max_context_len > 0) || !dst_start || !context_lens)
    return PA_ERR_INVALID_ARG;
  if (!aligned(keep, 4) || !aligned(cu_keep, 4) || !aligned(weights, 4) || !aligned(dst_start, 4) ||
      !aligned(context_lens, 4) || !aligned(status, 4))
    return PA_ERR_INVALID_ARG;
  pa::SelectParams p{};
  p.keep = keep;
  p.cu_keep = cu_keep;
  p.weights = weights;
  p.weights_stride = weights_stride;
  p.dst_start = dst_start;
  p.context_lens = context_lens;
  p.status = status;
  p.num_keep = num_keep;
  p.num_seqs = num_seqs;
  p.recent = recent;
  p.max_context_len = max_context_len;
  return pa::launch_select(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
