// The latent cache and eviction by attention weight: internal interface of
// their kernels.
//
// A latent cache holds one row a token, shared by every head: [num_blocks]
// [block_size][latent_dim + rope_dim], the vector that keys and values derive
// from and then the part of the key that carries the position.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace pa {

struct LatentDecodeParams {
  void* out;       // [num_seqs][q_len][num_heads][latent_dim]
  const void* q;   // bf16 [num_seqs][q_len][num_heads][latent_dim + rope_dim]
  const void* cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int32_t num_seqs, q_len, num_heads, num_blocks, block_size, max_blocks_per_seq, max_context_len;
  int32_t out_bf16;
  float scale_log2;  // softmax scale * log2(e)
  int32_t* err;      // the workspace's error word
  unsigned char* ws;
  uint64_t test_stall_ns;  // timeout-path test hook (0 = off): scores begin with a wait for what never comes, this long
};

struct LatentPrefillParams {
  void* out;       // [num_tokens][num_heads][head_dim]
  const void* q;   // bf16 [num_tokens][num_heads][head_dim + rope_dim]
  const void* cache;
  const void* w_k;  // bf16 [num_heads][head_dim][latent_dim]
  const void* w_v;
  const int32_t* cu_q;
  const int32_t* q_start;
  const int32_t* block_tables;
  int64_t total_context;
  int32_t num_tokens, num_seqs, num_heads, num_blocks, block_size, max_blocks_per_seq, max_q_len, max_context_len;
  int32_t out_bf16;
  float scale_log2;
  int32_t* status;  // may be null
  unsigned char* ws;
  uint64_t test_stall_ns;  // as in decode, in the expansion's and the attention's results
};

// What the kernels of one pa_prefill_latent call share, in its workspace.  Tokens
// of the contexts lie one behind the other, each context from a multiple of 128 on.
struct LatentExpanded {
  int32_t* tile0;        // [num_seqs + 1] 128-token tiles before a sequence; one without any is empty or refused
  int64_t* place0;       // [num_seqs + 1] places before a sequence, for one head (latent_prefill.cu)
  int32_t* counters;     // [CTAs], zeroed by every call
  float* parts;          // maxima, sums and rows that CTAs leave for one another
  unsigned char* rope;   // [rows][64] bf16
  unsigned char* k;      // [heads][rows][128]
  unsigned char* v;
  int64_t rows;          // of a head: whole tiles
  int32_t head0, heads;  // of this pass
  bool f32;              // keys and values in fp32 (fp32 outputs), else bf16
};

// How the expanded attention's work is counted: an item is a pair of 128-token
// tiles of a sequence for one head, and has kLatentLead places (what starting and
// ending it costs a CTA, in steps) and one for each step of 128 keys.
constexpr int kLatentLead = 2, kLatentPair = 256;
// steps of pair j of n query tokens behind q0 others
__host__ __device__ __forceinline__ int latent_steps(int n, int q0, int j) {
  return (q0 + (n < (j + 1) * kLatentPair ? n : (j + 1) * kLatentPair) + 127) / 128;
}
// places of pairs 0 .. j - 1, all whole, for one head: two more steps for every pair
__host__ __device__ __forceinline__ int64_t latent_places_before(int q0, int j) {
  return static_cast<int64_t>(j) * (kLatentLead + (q0 + 127) / 128) + static_cast<int64_t>(j) * (j + 1);
}
__host__ __device__ __forceinline__ int64_t latent_places(int n, int q0) {
  if (n <= 0) return 0;
  const int j = (n + kLatentPair - 1) / kLatentPair - 1;
  return latent_places_before(q0, j) + kLatentLead + latent_steps(n, q0, j);
}

struct WeightsParams {
  float* weights;  // [num_seqs], rows weights_stride apart
  int64_t weights_stride;
  const void* q;   // bf16 [num_seqs][window][num_q_heads][head_dim]
  const void* k_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int32_t num_seqs, window, num_q_heads, num_kv_heads, num_blocks, block_size, max_blocks_per_seq, max_context_len;
  int32_t head_dim;
  float scale_log2;
  int32_t* err;
  unsigned char* ws;
  uint64_t test_stall_ns;  // as in decode
};

struct SelectParams {
  int32_t* keep;
  const int32_t* cu_keep;
  float* weights;
  int64_t weights_stride;
  const int32_t* dst_start;
  const int32_t* context_lens;
  int32_t* status;  // may be null
  int32_t num_keep, num_seqs, recent, max_context_len;
};

cudaError_t launch_latent_append(const void* latent, int64_t latent_stride_bytes, const void* rope,
                                 int64_t rope_stride_bytes, int32_t num_tokens, const int64_t* slots, void* cache,
                                 int64_t num_slots, int32_t latent_bytes, int32_t rope_bytes, int32_t* status,
                                 cudaStream_t stream);
size_t latent_decode_workspace(int num_seqs, int q_len, int num_heads, int max_context_len);
cudaError_t launch_latent_decode(const LatentDecodeParams& p, cudaStream_t stream);
size_t latent_prefill_workspace(int num_seqs, int num_heads, int head_dim, int64_t total_context);
cudaError_t launch_latent_prefill(const LatentPrefillParams& p, cudaStream_t stream);
cudaError_t launch_latent_plan(const LatentPrefillParams& p, const LatentExpanded& x, cudaStream_t stream);
cudaError_t launch_latent_expand(const LatentPrefillParams& p, const LatentExpanded& x, cudaStream_t stream);
cudaError_t launch_latent_attend_f32(const LatentPrefillParams& p, const LatentExpanded& x, cudaStream_t stream);
size_t weights_workspace(int num_seqs, int window, int num_q_heads, int num_kv_heads, int head_dim,
                         int max_context_len);
cudaError_t launch_weights(const WeightsParams& p, cudaStream_t stream);
cudaError_t launch_select(const SelectParams& p, cudaStream_t stream);

// cuTensorMapEncodeTiled for bf16 data (abi.cu): dims and box innermost first, strides in bytes from the second on;
// swizzle: the span in bytes (128 or 64)
bool encode_bf16_tiles(CUtensorMap* m, int rank, const void* base, const uint64_t* dims, const uint64_t* strides,
                       const uint32_t* box, int swizzle);

}  // namespace pa
