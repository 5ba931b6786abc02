// Keys and values of every head from the latent rows:
//   K[h][t] = w_k[h] c_t,   V[h][t] = w_v[h] c_t,   D[128 x 256] = C[128 x 512] W[h]^T
// for 128-token tiles of the contexts, and the position parts of the rows packed
// beside them.  Rounded to bf16 (the products that follow take bf16; 2^-8, as the
// output: a row that sees few keys is then a value rounded twice, 0.0027 relative
// against 64 bits with its probabilities', where one rounding gives 0.0017, and over
// a long history 0.0018; a second part of the values would be two pieces of a step
// more beside five and 128 multiplications beside 320), or left in fp32 where the
// outputs are.  Rows behind a context are zeros.  A token whose
// value is not finite gets a value of zero and a key of NaN: whoever sees it puts
// out NaN, and 0 * NaN does not reach the rows that do not.
//
// A CTA holds its tile's rows (128 KB, gathered through the block table by TMA)
// and walks the heads; their weights stream.  4096 clocks of products need 256 KB
// of weights, 64 bytes a clock, more than the second-level cache feeds every SM
// with: so two CTAs with two tiles form one product of 256 rows, for which each
// holds half of the weights (the first the keys', the second the values').
// Six warps: 0-3 write out (a token a thread; bf16 through shared memory by TMA),
// 4 loads, 5 of the first CTA issues the pair's products; the results of two heads
// alternate in tensor memory.
// Measured, 4 x 2048 tokens of 128 heads (275 GFLOP, 0.5 GB written): 203 us, 1350
// TFLOP/s; 228 with stores from registers, 32 bytes of its own row a lane.  The
// weights' way from the second-level cache bounds it: 3 stages cost 20 us more
// than 4, 5 with half the room for results gain nothing.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "decode.cuh"
#include "fp4.cuh"
#include "latent.cuh"
#include "ptx.cuh"
#include "umma.cuh"

namespace pa {
namespace latent_expand_detail {

using namespace um;

// ---------------------------------------------------------------- the plan
// Tiles and places before every sequence; one CTA.  The contexts of the chunks
// before count in 64 bits, and the counters of the attention start at zero.
constexpr int kPlanThreads = 512;
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const LatentPrefillParams p, const LatentExpanded x, int num_counters) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int64_t sums[3][kPlanThreads / 32];
  const int64_t table_tokens = static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
  int64_t seen = 0, tiles = 0, places = 0;  // before this round of kPlanThreads sequences
  for (int i = tid; i < num_counters; i += kPlanThreads) x.counters[i] = 0;
  if (tid == 0) x.tile0[0] = 0, x.place0[0] = 0;
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int64_t n = 0, q0 = 0;
    bool ok = false, bad = false;
    if (s < p.num_seqs) {
      const int64_t b = p.cu_q[s];
      n = static_cast<int64_t>(p.cu_q[s + 1]) - b, q0 = p.q_start[s];
      ok = n > 0 && n <= p.max_q_len && b >= 0 && b + n <= p.num_tokens && q0 >= 0 && q0 + n <= p.max_context_len &&
           q0 + n <= table_tokens;
      bad = n != 0 && !ok;
    }
    auto scan = [&](int64_t v, int which) {  // inclusive, over the block
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (lane == 31) sums[which][warp] = v;
      __syncthreads();
      for (int w = 0; w < warp; ++w) v += sums[which][w];
      return v;
    };
    auto all = [&](int which) {
      int64_t v = 0;
      for (int w = 0; w < kPlanThreads / 32; ++w) v += sums[which][w];
      return v;
    };
    const int64_t upto = seen + scan(ok ? q0 + n : 0, 0);
    seen += all(0);
    if (ok && upto > p.total_context) ok = false, bad = true;
    const int64_t t = tiles + scan(ok ? (q0 + n + 127) / 128 : 0, 1);
    const int64_t u = places + scan(ok ? latent_places(static_cast<int>(n), static_cast<int>(q0)) : 0, 2);
    tiles += all(1);
    places += all(2);
    if (s < p.num_seqs) {
      x.tile0[s + 1] = static_cast<int32_t>(t);
      x.place0[s + 1] = u;
      if (bad && p.status) atomicExch(p.status, kDevErrInvalidArg);
    }
    __syncthreads();
  }
}

// ----------------------------------------------------------- the expansion
constexpr int kThreads = 6 * 32;
constexpr int kABytes = 8 * 16384;   // [8 chunks of 64 columns][128 rows x 128 bytes]
constexpr int kBBytes = 16384;       // a chunk of a head's weights: 128 rows of w_k, or of w_v
constexpr int kStages = 4;
constexpr int kOutBytes = 4096;      // 64 columns of a warp's 32 tokens
constexpr int kOffB = kABytes, kOffOut = kOffB + kStages * kBBytes, kOffBar = kOffOut + 4 * 2 * kOutBytes;
constexpr int kSmemBytes = 1024 + kOffBar + 256;
enum : int {
  kAFull = 0, kAFree = 1, kBFull = 2, kBFree = kBFull + kStages, kDFull = kBFree + kStages, kDFree = kDFull + 2,
  kDrain = kDFree + 2, kNever, kNumBars
};
static_assert(kNumBars * 8 + 16 <= 256, "barrier area");
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

struct Launch {
  LatentPrefillParams p;
  LatentExpanded x;
  int bs_log;
};

// 16 columns of a token's key or value in fp32
__device__ __forceinline__ void store16(unsigned char* dst, int64_t at, const float (&y)[16]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = __float_as_uint(y[8 * q + e]);
    fp4::store32(dst + at * 4 + 32 * q, h);
  }
}
// 128 columns of a row of the results as bf16 pairs
__device__ __forceinline__ void load_row(uint32_t at, uint32_t (&w)[64]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t v[32];
    load_now(at + c * 32, v);
#pragma unroll
    for (int j = 0; j < 16; ++j) w[c * 16 + j] = pack_bf16(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    expand_kernel(const __grid_constant__ Launch L, const __grid_constant__ CUtensorMap tm_pool,
                  const __grid_constant__ CUtensorMap tm_wk, const __grid_constant__ CUtensorMap tm_wv,
                  const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  const LatentPrefillParams& p = L.p;
  const LatentExpanded& x = L.x;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  volatile int* gave_up = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();

  if (tid == 0) {
    ptx::mbar_init(&bars[kAFull], 1);
    ptx::mbar_init(&bars[kAFree], 1);
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&bars[kBFull + i], 1);
      ptx::mbar_init(&bars[kBFree + i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars[kDFull + i], 1);
      ptx::mbar_init(&bars[kDFree + i], 8);
    }
    ptx::mbar_init(&bars[kDrain], 1);
    ptx::mbar_init(&bars[kNever], 1);
    *gave_up = 0;
    ptx::mbar_init_fence();
  }
  if (warp == 5) {
    tmem_alloc_pair(tmem_slot, 512);
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool aborted = false;
  cluster_sync();  // both CTAs' barriers are ready

  // units (pair of tiles, head), equal runs of them for the clusters
  const int tiles = x.tile0[p.num_seqs];
  const int64_t units = static_cast<int64_t>((tiles + 1) / 2) * x.heads;
  const int64_t clusters = gridDim.x / 2, c = blockIdx.x / 2;
  const int64_t u0 = units * c / clusters, u1 = units * (c + 1) / clusters;

  // a tile's sequence, first token and tokens (none for a tile behind the last)
  struct Tile {
    int seq, tok, n;
  };
  auto tile_of = [&](int64_t unit, uint32_t which) {
    Tile t{0, 0, 0};
    const int i = static_cast<int>(unit / x.heads) * 2 + static_cast<int>(which);
    if (i >= tiles) return t;
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {  // the last sequence that starts at or before it
      const int mid = (lo + hi + 1) >> 1;
      if (x.tile0[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    t.seq = lo;
    t.tok = (i - x.tile0[lo]) * 128;
    t.n = min(128, p.q_start[lo] + p.cu_q[lo + 1] - p.cu_q[lo] - t.tok);
    return t;
  };

  // the first CTA's barrier at this place: it issues the pair's products
  auto first_of = [](uint64_t* bar) { return remote(bar, 0); };

  if (warp == 4) {
    // ============================== loads ==============================
    const int page_rows = min(128, 1 << L.bs_log);
    uint32_t kb = 0, ka = 0;
    const uint64_t keep = ptx::policy_evict_last();
    for (int64_t u = u0; u < u1 && !aborted; ++u) {
      const int h = x.head0 + static_cast<int>(u % x.heads);
      if (u == u0 || u % x.heads == 0) {
        const Tile t = tile_of(u, rank);
        wait(&bars[kAFree], (ka & 1u) ^ 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) break;
        ++ka;
        auto pages_of = [&](const Tile& y) { return (y.n + page_rows - 1) / page_rows; };
        const int pages = pages_of(t);
        if (rank == 0) {
          const int both = pages + pages_of(tile_of(u, 1));
          if (lane == 0) ptx::mbar_arrive_expect_tx(&bars[kAFull], static_cast<uint32_t>(both * page_rows) * 1024u);
        }
        __syncwarp();
        if (lane < pages) {
          const int tok = t.tok + lane * page_rows;
          int phys = __ldg(p.block_tables + static_cast<int64_t>(t.seq) * p.max_blocks_per_seq + (tok >> L.bs_log));
          if (phys < 0 || phys >= p.num_blocks) {  // never read outside the pool
            if (p.status) atomicExch(p.status, kDevErrInvalidArg);
            phys = 0;
          }
          const int at = static_cast<int>((static_cast<int64_t>(phys) << L.bs_log) + (tok & ((1 << L.bs_log) - 1)));
          for (int ch = 0; ch < 8; ++ch)
            tma_load_2d_pair(smem + ch * 16384 + lane * page_rows * 128, &tm_pool, ch * 64, at, first_of(&bars[kAFull]), keep);
        }
        __syncwarp();
      }
      for (int ch = 0; ch < 8 && !aborted; ++ch, ++kb) {
        const uint32_t slot = kb % kStages;
        wait(&bars[kBFree + slot], ((kb / kStages) & 1u) ^ 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) break;
        if (lane == 0) {
          if (rank == 0) ptx::mbar_arrive_expect_tx(&bars[kBFull + slot], 2 * kBBytes);
          tma_load_2d_pair(smem + kOffB + slot * kBBytes, rank ? &tm_wv : &tm_wk, ch * 64, h * 128,
                           first_of(&bars[kBFull + slot]), keep);
        }
        __syncwarp();
      }
    }
    // The products signal these barriers of both CTAs when they complete, which
    // no thread's order covers: a CTA stays until the last signals are here (one
    // that arrives where its CTA has gone is a fault).
    for (uint32_t k = kb > kStages ? kb - kStages : 0; k < kb; ++k)
      wait(&bars[kBFree + k % kStages], (k / kStages) & 1u, aborted);
    if (ka) wait(&bars[kAFree], (ka - 1) & 1u, aborted);
    aborted = __any_sync(0xffffffffu, aborted);
    if (aborted && rank == 0) {  // (both CTAs' loads are counted here)
      wait_for_loads(&bars[kAFull], 1, ka);
      wait_for_loads(&bars[kBFull], kStages, kb);
    }
  } else if (warp == 5) {
    // ============================ products ============================
    const bool leader = elect_one();
    constexpr uint32_t kId = ptx::idesc_bf16_f32(256, 256, 0, 0);
    const uint64_t desc_a = ptx::smem_desc(smem, 16, 1024, ptx::kLayoutSw128);
    const uint64_t desc_b = ptx::smem_desc(smem + kOffB, 16, 1024, ptx::kLayoutSw128);
    uint32_t kb = 0, ka = 0, kd = 0;
    for (int64_t u = u0; u < u1 && !aborted && rank == 0; ++u, ++kd) {
      if (u == u0 || u % x.heads == 0) wait(&bars[kAFull], ka++ & 1u, aborted);
      wait(&bars[kDFree + (kd & 1u)], ((kd >> 1) & 1u) ^ 1u, aborted);
      const uint32_t d = tmem + (kd & 1u) * 256;
      for (int ch = 0; ch < 8; ++ch, ++kb) {
        const uint32_t slot = kb % kStages;
        wait(&bars[kBFull + slot], (kb / kStages) & 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) break;
        ptx::tc_fence_after();
        if (leader) {
          const uint64_t da = desc_a + ch * (16384 >> 4), db = desc_b + slot * (kBBytes >> 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) umma_pair(d, da + j * 2, db + j * 2, kId, ch + j > 0);
          umma_commit_pair(&bars[kBFree + slot]);
          if (ch == 7) {
            umma_commit_pair(&bars[kDFull + (kd & 1u)]);
            if (u + 1 == u1 || (u + 1) % x.heads == 0) umma_commit_pair(&bars[kAFree]);
          }
        }
        __syncwarp();
      }
    }
    if (leader) {  // nothing may be in flight when tensor memory is freed
      if (rank == 0) umma_commit_pair(&bars[kDrain]);
      bool late = false;
      wait(&bars[kDrain], 0, late);
      if (late) aborted = true;
    }
    aborted = __any_sync(0xffffffffu, aborted);
  } else {
    // ===================== results: a token a thread =====================
    const uint32_t lanes = static_cast<uint32_t>(32 * warp) << 16;
    const bool f32 = x.f32;
    uint32_t kd = 0;
    Tile t{0, 0, 0};
    if (p.test_stall_ns && !ptx::mbar_wait(&bars[kNever], 0, p.test_stall_ns)) aborted = true;  // pa_test_stall_decode
    aborted = __any_sync(0xffffffffu, aborted);
    for (int64_t u = u0; u < u1 && !aborted; ++u, ++kd) {
      if (u == u0 || u % x.heads == 0) t = tile_of(u, rank);
      const int h = static_cast<int>(u % x.heads);
      const int tile = static_cast<int>(u / x.heads) * 2 + static_cast<int>(rank);
      const int64_t row = static_cast<int64_t>(tile) * 128 + tid;
      const bool there = tile < tiles, valid = tid < t.n;
      if (h == 0 && there) {  // the position part, packed
        uint4 r[8];
        const int tok = t.tok + tid;
        if (valid) {
          int phys = __ldg(p.block_tables + static_cast<int64_t>(t.seq) * p.max_blocks_per_seq + (tok >> L.bs_log));
          if (phys < 0 || phys >= p.num_blocks) phys = 0;
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const __nv_bfloat16*>(p.cache) +
              ((static_cast<int64_t>(phys) << L.bs_log) + (tok & ((1 << L.bs_log) - 1))) * 576 + 512);
#pragma unroll
          for (int e = 0; e < 8; ++e) r[e] = __ldg(src + e);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          reinterpret_cast<uint4*>(x.rope)[row * 8 + e] = valid ? r[e] : make_uint4(0, 0, 0, 0);
      }
      wait(&bars[kDFull + (kd & 1u)], (kd >> 1) & 1u, aborted);
      aborted = __any_sync(0xffffffffu, aborted);
      if (aborted) break;
      ptx::tc_fence_after();
      const uint32_t d = tmem + lanes + (kd & 1u) * 256;
      auto all_read = [&]() {
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) remote_arrive(first_of(&bars[kDFree + (kd & 1u)]));
      };
      bool odd = false;  // the value is not finite somewhere
      if (!f32) {
        // bf16 rows leave by TMA, 64 columns of the warp's 32 tokens at a time
        // (stored from registers, 32 bytes of its own row a lane, they took longer than the products)
        uint32_t w[64];
        auto put = [&](const CUtensorMap* map) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            unsigned char* box = smem + kOffOut + (warp * 2 + half) * kOutBytes;
            if (lane == 0) tma_stores_read<1>();  // the box before in the same place
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const uint32_t* y = w + half * 32 + c * 4;
              *reinterpret_cast<uint4*>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tma_store_2d(map, half * 64, static_cast<int>(h * x.rows + row), box);
            __syncwarp();  // loads of tensor memory are the whole warp's
          }
        };
        load_row(d + 128, w);  // values first
#pragma unroll
        for (int j = 0; j < 64; ++j) odd |= (w[j] & 0x7f80u) == 0x7f80u || (w[j] & 0x7f800000u) == 0x7f800000u;
        if (odd || !valid) {
#pragma unroll
          for (int j = 0; j < 64; ++j) w[j] = 0u;
        }
        if (there) put(&tm_v);
        load_row(d, w);
        all_read();
        if (odd || !valid) {
#pragma unroll
          for (int j = 0; j < 64; ++j) w[j] = valid ? 0x7fff7fffu : 0u;
        }
        if (there) put(&tm_k);
        continue;
      }
      const int64_t at = (static_cast<int64_t>(h) * x.rows + row) * 128;
#pragma unroll 1
      for (int col = 0; col < 256; col += 32) {
        const int from = (col + 128) & 255;  // values first
        uint32_t v[32];
        load_now(d + from, v);
        if (col == 224) all_read();
        if (!there) continue;
        if (from >= 128) {
#pragma unroll
          for (int j = 0; j < 32; ++j) odd |= (v[j] & 0x7f800000u) == 0x7f800000u;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float y[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            y[j] = !valid ? 0.f : (from < 128 && odd ? __uint_as_float(0x7fffffffu) : __uint_as_float(v[16 * q + j]));
          store16(from < 128 ? x.k : x.v, at + (from & 127) + 16 * q, y);
        }
      }
      if (odd && valid && there) {  // no value, in place of what was stored
        const float none[16] = {};
        for (int col = 0; col < 128; col += 16) store16(x.v, at + col, none);
      }
    }
    tma_stores_done();
  }

  if (aborted) *gave_up = 1;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  cluster_sync();  // the other CTA may still load, read and signal here
  if (*gave_up) let_arrive();
  __syncwarp();
  if (warp == 5) tmem_dealloc_pair(tmem, 512);
  if (tid == 0 && *gave_up && p.status) atomicExch(p.status, kDevErrTimeout);
}

}  // namespace latent_expand_detail

cudaError_t launch_latent_plan(const LatentPrefillParams& p, const LatentExpanded& x, cudaStream_t stream) {
  using namespace latent_expand_detail;
  plan_kernel<<<1, kPlanThreads, 0, stream>>>(p, x, static_cast<int>(device_sm_count()));
  return cudaGetLastError();
}

cudaError_t launch_latent_expand(const LatentPrefillParams& p, const LatentExpanded& x, cudaStream_t stream) {
  using namespace latent_expand_detail;
  Launch L{};
  L.p = p;
  L.x = x;
  L.bs_log = __builtin_ctz(static_cast<unsigned>(p.block_size));
  CUtensorMap tm_pool, tm_wk, tm_wv, tm_k, tm_v;
  const uint64_t pool[2] = {576, static_cast<uint64_t>(p.num_blocks) * p.block_size}, pool_stride[1] = {1152};
  const uint32_t pool_box[2] = {64, static_cast<uint32_t>(p.block_size < 128 ? p.block_size : 128)};
  const uint64_t w[2] = {512, static_cast<uint64_t>(p.num_heads) * 128}, w_stride[1] = {1024};
  const uint32_t w_box[2] = {64, 128}, out_box[2] = {64, 32};
  const uint64_t out[2] = {128, static_cast<uint64_t>(x.rows) * x.heads}, out_stride[1] = {256};
  if (!encode_bf16_tiles(&tm_pool, 2, p.cache, pool, pool_stride, pool_box, 128) ||
      !encode_bf16_tiles(&tm_wk, 2, p.w_k, w, w_stride, w_box, 128) ||
      !encode_bf16_tiles(&tm_wv, 2, p.w_v, w, w_stride, w_box, 128) ||
      !encode_bf16_tiles(&tm_k, 2, x.k, out, out_stride, out_box, 128) ||
      !encode_bf16_tiles(&tm_v, 2, x.v, out, out_stride, out_box, 128))
    return cudaErrorInvalidValue;
  const void* fn = reinterpret_cast<const void*>(&expand_kernel);
  int per_sm = 0;
  cudaError_t e = fp4_occupancy(fn, kThreads, kSmemBytes, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t units = (x.rows / 128 + 1) / 2 * x.heads, most = device_sm_count() / 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (units < 1 ? 1 : (units < most ? units : most))));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&L, &tm_pool, &tm_wk, &tm_wv, &tm_k, &tm_v};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace pa
