// Token compaction inside the pages of a paged cache: of each sequence, the
// kept tokens behind position dst_start move to the front, in order:
//   position dst_start + j  :=  position keep[j],   keep[j] >= dst_start + j.
//
// One CTA owns the rows of one (sequence, head group, layer, K or V), so no
// other CTA reads or writes them.  It walks the kept tokens in chunks: all of
// a chunk's rows are read into registers, the CTA synchronises, then they are
// written.  keep ascends, so every later source lies at or behind its own
// destination and so behind every destination written so far: nothing is
// overwritten before it is read, and the next chunk may be read before this
// one is written.  Bound by the bytes moved.
#include "decode.cuh"
#include "fp4.cuh"

namespace pa {
namespace {

constexpr int kThreads = 256;

// VEC: the unit of a move (16 bytes; 4-bit pages with head_dim 64: 4 bytes,
// their scale rows' size).
template <typename VEC>
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactParams p, int heads_per_cta, int units_per_row,
                                                           int code_units) {
  const int seq = blockIdx.x;
  const int h0 = blockIdx.y * heads_per_cta;
  const int64_t layer = blockIdx.z >> 1;
  unsigned char* cache = ((blockIdx.z & 1) ? p.v_cache : p.k_cache) + layer * p.layer_bytes;
  const int b = p.cu_keep[seq], n = p.cu_keep[seq + 1] - b;
  const int dst0 = p.dst_start[seq];
  const int64_t table_tokens = static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
  const bool report = p.status && blockIdx.y == 0 && blockIdx.z == 0;
  if (n <= 0) {
    if (n < 0 && report && threadIdx.x == 0) atomicExch(p.status, kDevErrInvalidArg);
    return;
  }
  if (b < 0 || n > p.max_keep || dst0 < 0 || dst0 + static_cast<int64_t>(n) > table_tokens) {
    if (report && threadIdx.x == 0) atomicExch(p.status, kDevErrInvalidArg);
    return;
  }
  const int32_t* table = p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq;
  const int per_token = heads_per_cta * units_per_row;
  const int64_t total = static_cast<int64_t>(n) * per_token;
  const int bs = p.block_size;
  for (int64_t i0 = 0; i0 < total; i0 += kThreads) {
    const int64_t i = i0 + threadIdx.x;
    VEC v;
    VEC* dst = nullptr;
    if (i < total) {
      const int j = static_cast<int>(i / per_token);
      const int r = static_cast<int>(i - static_cast<int64_t>(j) * per_token);
      const int h = h0 + r / units_per_row, u = r % units_per_row;
      const int src_pos = p.keep[b + j], dst_pos = dst0 + j;
      const bool ok = src_pos >= dst_pos && src_pos < table_tokens && (j == 0 || src_pos > p.keep[b + j - 1]);
      int sb = -1, db = -1;
      if (ok) {
        sb = table[src_pos / bs];
        db = table[dst_pos / bs];
      }
      if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
        if (report && r == 0) atomicExch(p.status, kDevErrInvalidArg);
      } else if (src_pos != dst_pos && h < p.num_kv_heads) {
        const int64_t st = (static_cast<int64_t>(sb) * p.num_kv_heads + h) * p.tile_bytes;
        const int64_t dt = (static_cast<int64_t>(db) * p.num_kv_heads + h) * p.tile_bytes;
        const int so = src_pos % bs, dof = dst_pos % bs;
        int64_t in_s, in_d;
        if (u < code_units) {
          in_s = static_cast<int64_t>(so) * p.row_bytes + u * static_cast<int>(sizeof(VEC));
          in_d = static_cast<int64_t>(dof) * p.row_bytes + u * static_cast<int>(sizeof(VEC));
        } else {
          const int64_t base = static_cast<int64_t>(bs) * p.row_bytes + (u - code_units) * static_cast<int>(sizeof(VEC));
          in_s = base + static_cast<int64_t>(so) * p.scale_bytes;
          in_d = base + static_cast<int64_t>(dof) * p.scale_bytes;
        }
        v = *reinterpret_cast<const VEC*>(cache + st + in_s);
        dst = reinterpret_cast<VEC*>(cache + dt + in_d);
      }
    }
    __syncthreads();
    if (dst) *dst = v;
  }
}

template <typename VEC>
cudaError_t launch(const CompactParams& p, cudaStream_t stream) {
  const int code_units = p.row_bytes / static_cast<int>(sizeof(VEC));
  const int units = code_units + p.scale_bytes / static_cast<int>(sizeof(VEC));
  const int hpc = 1;
  const dim3 grid(static_cast<unsigned>(p.num_seqs), static_cast<unsigned>((p.num_kv_heads + hpc - 1) / hpc),
                  static_cast<unsigned>(2 * p.num_layers));
  compact_kernel<VEC><<<grid, kThreads, 0, stream>>>(p, hpc, units, code_units);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  if (p.scale_bytes == 0 || p.scale_bytes % 16 == 0) return launch<uint4>(p, stream);
  return p.scale_bytes % 8 == 0 ? launch<uint2>(p, stream) : launch<uint32_t>(p, stream);
}

}  // namespace pa
