// Token compaction inside the pages of a paged cache: of each sequence, the
// kept tokens behind position dst_start move to the front, in order:
//   position dst_start + j  :=  position keep[j],   keep[j] >= dst_start + j.
//
// One CTA owns the rows of one (sequence, head group) in a few planes (a plane:
// the K or V cache of a layer, or a layer of a latent cache), so no other CTA reads or writes them.  It walks
// the kept tokens in chunks, and a chunk plane by plane: all of its rows are
// read into registers, the CTA synchronises, then they are written.  keep
// ascends, so every later source lies at or behind its own destination and so
// behind every destination written so far: nothing is overwritten before it is
// read, and the next chunk, or plane, may be read before this one is written.
//
// What bounds it is the chain keep -> block table -> row, three dependent
// loads a chunk, more than the bytes: so a chunk is as long as the CTA's
// registers allow (four pieces a thread, 512 threads for long lists), its
// places serve several planes, the next plane's rows load before this one's
// are written, and few kept tokens (accepted drafts) take all heads in one CTA.
// 64 sequences x up to 8 tokens in 32 layers (78 MB): 23.4 us; 16 sequences x
// 2000 of 4096 tokens in 4 bits (74 MB): 27.6 us, call behind call (one piece a
// thread and a CTA a plane and head: 49 and 104 us).
#include "decode.cuh"
#include "fp4.cuh"
#include "ptx.cuh"

namespace pa {
namespace {

constexpr int kUnroll = 4;       // pieces a thread holds
constexpr int kMaxThreads = 512;

struct Piece {
  uint32_t w[4];
};
__device__ __forceinline__ void load_piece(Piece& v, const unsigned char* p, int bytes) {
  if (bytes == 16) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    v.w[0] = r.x, v.w[1] = r.y, v.w[2] = r.z, v.w[3] = r.w;
  } else if (bytes == 8) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    v.w[0] = r.x, v.w[1] = r.y;
  } else {
    v.w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
__device__ __forceinline__ void store_piece(const Piece& v, unsigned char* p, int bytes) {
  if (bytes == 16) *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  else if (bytes == 8) *reinterpret_cast<uint2*>(p) = make_uint2(v.w[0], v.w[1]);
  else *reinterpret_cast<uint32_t*>(p) = v.w[0];
}

// MANY: several planes, each loaded while the one before is written; else one,
// with the next chunk's places found meanwhile.
template <bool MANY>
__global__ void __launch_bounds__(kMaxThreads, 2)
    compact_kernel(const CompactParams p, int heads_per_cta, int units, int planes) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int seq = blockIdx.x;
  const int plane0 = blockIdx.z * planes, plane1 = min(p.num_planes, plane0 + planes);
  auto cache_of = [&](int plane) {
    return ((plane & 1) ? p.v_cache : p.k_cache) + (plane >> 1) * p.layer_bytes;
  };
  const int b = p.cu_keep[seq], n = p.cu_keep[seq + 1] - b;
  const int dst0 = p.dst_start[seq];
  // positions are 32-bit numbers
  const int64_t table_tokens = min(static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size, int64_t(0x7fffffff));
  const int num_keep = p.num_keep >= 0 ? p.num_keep : p.cu_keep[p.num_seqs];  // entries that may be read
  const bool report = p.status && blockIdx.y == 0 && blockIdx.z == 0;
  if (n == 0) return;
  if (b < 0 || n < 0 || n > p.max_keep || b + static_cast<int64_t>(n) > num_keep || dst0 < 0 ||
      dst0 + static_cast<int64_t>(n) > table_tokens) {
    if (report && threadIdx.x == 0) atomicExch(p.status, kDevErrInvalidArg);
    return;
  }
  const int32_t* table = p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq;
  const int bs_log = __ffs(p.block_size) - 1, bs_mask = p.block_size - 1;
  // this thread's piece: token `tok` of every step of `tokens` tokens, unit u of head h.
  // Units of a row: 16-byte pieces (4-bit pages: of its codes, then its scales)
  const int per_token = heads_per_cta * units;
  const int tokens = blockDim.x / per_token;
  const int tok = threadIdx.x / per_token;
  const int r = threadIdx.x - tok * per_token;
  const int h = blockIdx.y * heads_per_cta + r / units, u = r % units;
  const bool scales = p.scale_bytes && u == units - 1;
  const int bytes = scales ? p.scale_bytes : 16;
  const int stride = scales ? p.scale_bytes : p.row_bytes;  // from row to row of a tile
  const int64_t first = h * p.tile_bytes + (scales ? static_cast<int64_t>(p.row_bytes) << bs_log : u * 16);
  const bool mine = tok < tokens && h < p.num_kv_heads;
  const int64_t block_bytes = p.tile_bytes * p.num_kv_heads;
  const int chunk = tokens * kUnroll;

  // where a chunk's pieces come from and go to (src < 0: nothing to move)
  int64_t src[kUnroll], dst[kUnroll];
  auto locate = [&](int j0) {
#pragma unroll
    for (int e = 0; e < kUnroll; ++e) {
      const int j = j0 + e * tokens + tok;
      src[e] = -1;
      if (!mine || j >= n) continue;
      const int sp = p.keep[b + j], dp = dst0 + j;
      int sb = -1, db = -1;
      if (sp >= dp && sp < table_tokens && (j == 0 || sp > p.keep[b + j - 1])) {
        sb = table[sp >> bs_log];
        db = table[dp >> bs_log];
      }
      if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
        if (report && r == 0) atomicExch(p.status, kDevErrInvalidArg);
        continue;
      }
      if (sp == dp) continue;
      src[e] = sb * block_bytes + first + static_cast<int64_t>(sp & bs_mask) * stride;
      dst[e] = db * block_bytes + first + static_cast<int64_t>(dp & bs_mask) * stride;
    }
  };
  auto load = [&](Piece (&x)[kUnroll], const unsigned char* cache) {
#pragma unroll
    for (int e = 0; e < kUnroll; ++e)
      if (src[e] >= 0) load_piece(x[e], cache + src[e], bytes);
  };
  if (MANY) {
    Piece v[2][kUnroll];
    auto store = [&](const Piece (&x)[kUnroll], unsigned char* cache) {
#pragma unroll
      for (int e = 0; e < kUnroll; ++e)
        if (src[e] >= 0) store_piece(x[e], cache + dst[e], bytes);
    };
    for (int j0 = 0; j0 < n; j0 += chunk) {
      locate(j0);
      load(v[0], cache_of(plane0));
      for (int plane = plane0; plane < plane1; plane += 2) {
        if (plane + 1 < plane1) load(v[1], cache_of(plane + 1));
        __syncthreads();
        store(v[0], cache_of(plane));
        if (plane + 2 < plane1) load(v[0], cache_of(plane + 2));
        __syncthreads();
        if (plane + 1 < plane1) store(v[1], cache_of(plane + 1));
      }
    }
  } else {
    unsigned char* cache = cache_of(plane0);
    locate(0);
    for (int j0 = 0; j0 < n; j0 += chunk) {
      Piece v[kUnroll];
      int64_t to[kUnroll];
      load(v, cache);
#pragma unroll
      for (int e = 0; e < kUnroll; ++e) to[e] = src[e] >= 0 ? dst[e] : -1;
      if (j0 + chunk < n) locate(j0 + chunk);
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kUnroll; ++e)
        if (to[e] >= 0) store_piece(v[e], cache + to[e], bytes);
    }
  }
}

}  // namespace

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  const int units = p.row_bytes / 16 + (p.scale_bytes ? 1 : 0);
  // few kept tokens: as many heads a CTA as one chunk of 256 threads moves at once
  int heads = 1;
  for (int h = 2; h <= p.num_kv_heads; ++h)
    if (h * units <= 256 && static_cast<int64_t>(p.max_keep) * h * units <= 256 * kUnroll) heads = h;
  int threads = 256;
  while (threads < kMaxThreads && (threads < units || static_cast<int64_t>(p.max_keep) * heads * units > threads * kUnroll))
    threads *= 2;
  const int64_t groups = (p.num_kv_heads + heads - 1) / heads;
  // as few planes a CTA as let all CTAs run at once (an SM holds 1024 threads of them)
  const int64_t room = device_sm_count() * (1024 / threads), per_plane = static_cast<int64_t>(p.num_seqs) * groups;
  int planes = 1;
  while (planes < p.num_planes && per_plane * ((p.num_planes + planes - 1) / planes) > room) ++planes;
  const dim3 grid(static_cast<unsigned>(p.num_seqs), static_cast<unsigned>(groups),
                  static_cast<unsigned>((p.num_planes + planes - 1) / planes));
  return launch_early(planes > 1 ? compact_kernel<true> : compact_kernel<false>, grid, threads, stream, p, heads, units,
                      planes);
}

}  // namespace pa
