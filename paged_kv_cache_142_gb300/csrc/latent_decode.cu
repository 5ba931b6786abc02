// Attention over the latent cache in its absorbed form, on the 5th-generation
// tensor cores; latent_dim 512, rope_dim 64.
//
//   S[128 rows x 64 tokens] = Q K^T,   P = 2^(S f - m),   O[128 x 512] += P V
// A row is one head of one query token; K is the cached row (576 values), V its
// first 512.  Every head shares the rows, so a step does 4.4 MFLOP a token for
// 1152 bytes (128 heads): bytes and products are in balance, and both have to
// stream.
//
// O alone is 256 KB in fp32, all of an SM's tensor memory, so a cluster of two
// CTAs shares an item by columns: CTA c holds columns 256 c .. of the latent
// part and half of the position part, of all rows and all tokens.  No byte of
// the cache is loaded twice.
// Each forms S over its own 288 columns; the two add their partial sums up
// through distributed shared memory (32 KB a tile each way at 128 rows), and both
// form the same probabilities, each for its columns of O: handing P over instead
// halves the exponentials, but puts a second exchange into a tile's chain.
// A row's reference is raised only when its maximum passes it by 2^8.
// The queries lie in tensor memory as the A operand (144 columns), so that
// shared memory holds four tiles of K and V.
//
// fp32 outputs take the probabilities in two bf16 parts, P and what its
// rounding left (2^-16 in all); bf16 outputs take one (2^-8, as the output): off by
// 0.0020 relative against 64 bits, where one rounding of the output gives 0.0017.
// Two parts would give that, for 13% of the time (the fp32 form takes 79.5 us where
// this one takes 70, batch of 256, and 90 where it takes 79.5, 128 heads).
//
// The work is cut into equal runs of tiles, one for each cluster, across the
// borders of sequences; a cluster that takes part of an item leaves its rows
// unnormalised in the workspace, and a second kernel adds the parts up.
//
// One CTA per SM, 19 warps: 0-15 scores and outputs, 16 loads, 17 and 18 issue
// the products of S and of O (one warp for both would hold back the next S while
// it waits for P).  A tile's chain (scores, exchange, maximum, probabilities)
// takes 2000 clocks, nearly all of them latency, whatever the width: so several
// tiles are in it at a time, and only the reference passes from one group of
// warps to the next.  More than 32 rows: two groups of eight warps, half of a
// row's tokens a thread; a warp whose rows nobody has does nothing.  At most 32
// rows would leave three quarters of tensor memory, and so of the warps (a warp
// reaches the lanes of its own quarter), without work: there the queries stand
// in all four quarters, each of the last three has every third tile's scores, a
// quarter of a row's tokens a thread, and the first's warps keep the outputs
// (16 rows, batch of 256 with 900 tokens or so: 64 us; two groups of two warps: 71).
//
// Measured: the batch of 256 with 16 heads reads 259 MB in 64 us, 4.0 TB/s (60%
// of a plain copy): what is left is the start and the end of an item, where the
// chain has fewer tiles than it could.  The batch of 64 with 128 heads takes 73 us
// (2.3 TB/s, 500 TFLOP/s): the exchange of 32 KB of partial sums a tile and the
// merge of the parts (10 us) bound it.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "decode.cuh"
#include "fp4.cuh"
#include "latent.cuh"
#include "ptx.cuh"
#include "umma.cuh"

namespace pa {
namespace latent_decode_detail {

using namespace um;

constexpr int kThreads = 19 * 32;
constexpr int kTile = 64;                      // tokens
constexpr int kLatBytes = kTile * 512;         // [8-token group][4 chunks of 64 columns][8 rows x 128 bytes]
constexpr int kRopeBytes = kTile * 64;         // [8-token group][8 rows x 64 bytes]
constexpr int kStageBytes = kLatBytes + kRopeBytes;
__host__ __device__ constexpr int p_bytes(bool narrow) { return (narrow ? 32 : 128) * 128; }  // [half of the tokens][rows x 32 bf16]
// the other CTA's partial sums: [half of the tokens][4-token group][row][4]
__host__ __device__ constexpr int x_bytes(bool narrow) { return (narrow ? 32 : 128) * kTile * 4; }
constexpr uint32_t kColQ = 256, kColS = 400;   // tensor memory: O at 0
constexpr float kSlack = 8.f;
constexpr int kMaxSeqs = 2048;  // of one launch: their places lie in shared memory
constexpr int kMostLead = 8;
constexpr int kMinTiles = 4;  // of a cluster's run, where there are enough clusters

// narrow: at most 32 rows, whose probabilities and sums leave room for another tile
// and whose scores every quarter of tensor memory can have (see below)
__host__ __device__ constexpr int groups_of(bool narrow) { return narrow ? 3 : 2; }
__host__ __device__ constexpr int stages_of(bool hi, bool narrow) { return narrow ? 5 : hi ? 3 : 4; }

// barriers
enum : int {
  kFull = 0, kEmpty = 5, kQFull = 10, kSFree = 11, kSFull = 12, kXFull = 15, kXFree = 18, kPFull = 21, kPFree = 24,
  kODone = 27, kOFree = 30, kDrain = 31, kLFull = 33, kLFree = 34, kRef = 35, kNever = 43, kNumBars = 44
};
// shared memory, behind the stages: P slots, the exchange, then
constexpr int kOffBar = 0;
constexpr int kOffTops = 512;                  // [2 turns][group][part of the tokens][rows] maxima of a part of a row
constexpr int kOffRefs = kOffTops + 4096;      // [group][rows] the rows' references
constexpr int kOffPrefix = kOffRefs + 1024;

struct Launch {
  LatentDecodeParams p;
  int rows, row_tiles;   // of a sequence; tiles of 128
  int quarters;          // of the 128 rows that any tile has
  int bs_log, part_rows;
  int num_clusters;
  int lead;              // what starting and ending an item costs a cluster, in tiles: places before its first
  int4* desc;            // [clusters] the item that a cluster's run begins inside of: sequence (or -1), row tile, first and last cluster
  float* ml;             // [2 * clusters][part_rows][2] maximum (log2), sum
  float* o;              // [2 * clusters][part_rows][512]
};

// An item (a row tile of a sequence) and this cluster's part of it.
struct Item {
  int seq, rt, len, tiles;
  int start, end;  // places: the lead's, then the tiles'
  int t0, t1;
  bool whole;
};

struct Walk {
  const Launch& L;
  const int* prefix;
  int c_begin, c_end;
  __device__ __forceinline__ int length(int seq) const {
    const int n = L.p.context_lens[seq];
    return n > 0 && n <= L.p.max_context_len ? n : 0;
  }
  __device__ __forceinline__ void derive(Item& it) const {
    it.end = it.start + L.lead + it.tiles;
    const int first = it.start + L.lead;
    it.t0 = max(c_begin, first) - first;
    it.t1 = min(c_end, it.end) - first;
    it.whole = it.t0 == 0 && it.t1 == it.tiles;
  }
  __device__ __forceinline__ void open(Item& it) const {
    it.len = length(it.seq);
    it.tiles = (it.len + kTile - 1) / kTile;
  }
  // the item at c_begin
  __device__ __noinline__ void find(Item& it) const {
    int lo = 0, hi = L.p.num_seqs - 1;
    while (lo < hi) {  // the last sequence that starts at or before it
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= c_begin) lo = mid;
      else hi = mid - 1;
    }
    it.seq = lo;
    open(it);
    const int r = c_begin - prefix[lo];
    it.rt = r / (L.lead + it.tiles);
    it.start = c_begin - r % (L.lead + it.tiles);
    derive(it);
  }
  __device__ __forceinline__ void next(Item& it) const {
    it.start = it.end;
    if (++it.rt == L.row_tiles) {
      it.rt = 0;
      do ++it.seq;
      while (prefix[it.seq + 1] == it.start);  // sequences without places
      open(it);
    }
    derive(it);
  }
  // calls f(item, the one behind it, whether there is one) for every item with tiles of this cluster's
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if (c_begin >= c_end) return;
    Item it, nxt;
    find(it);
    for (;;) {
      bool more = it.end < c_end;
      nxt = it;
      if (more) {
        next(nxt);
        more = nxt.t1 > nxt.t0;
      }
      if (it.t1 > it.t0) f(it, nxt, more);
      if (!more) return;
      it = nxt;
    }
  }
};

// keys that the last (first) row of a row tile sees
__device__ __forceinline__ int seen_by(const Launch& L, const Item& it, int row) {
  return it.len - L.p.q_len + 1 + row / L.p.num_heads;
}

// 16 outputs of a row
__device__ __forceinline__ void store16(const LatentDecodeParams& p, int64_t at, const float (&v)[16]) {
  uint32_t h[8];
  if (p.out_bf16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    fp4::store32(static_cast<__nv_bfloat16*>(p.out) + at, h);
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = __float_as_uint(v[8 * q + e]);
      fp4::store32(static_cast<float*>(p.out) + at + 8 * q, h);
    }
  }
}

// Of the tokens from .. upto - 1 of a stretch of staged rows, those of `odd` whose
// latent columns are not all finite become zero.  By a whole warp, 8 columns a lane.
__device__ __forceinline__ void clear_odd(unsigned char* rows, uint32_t odd, int from, int upto, int lane) {
  for (int j = from; j < upto; ++j) {
    if (!((odd >> j) & 1u)) continue;
    uint4* at = reinterpret_cast<uint4*>(rows + (j >> 3) * 4096 + (lane >> 3) * 1024 + (j & 7) * 128 + (lane & 7) * 16);
    const uint4 x = *at;
    auto bad = [](uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; };
    if (__any_sync(0xffffffffu, bad(x.x) || bad(x.y) || bad(x.z) || bad(x.w))) *at = make_uint4(0, 0, 0, 0);
  }
}

template <bool HI, bool NARROW>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ Launch L, const __grid_constant__ CUtensorMap tm_lat,
                  const __grid_constant__ CUtensorMap tm_rope) {
  constexpr int kStages = stages_of(HI, NARROW), kParts = HI ? 2 : 1, kRows = NARROW ? 32 : 128;
  constexpr uint32_t kGroups = groups_of(NARROW);  // tiles in the chain of scores and probabilities
  constexpr int kPBytes = p_bytes(NARROW), kXBytes = x_bytes(NARROW);
  const LatentDecodeParams& p = L.p;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  // [groups][parts]; of fewer than 128 rows the products read on, into rows of nobody's
  unsigned char* smem_p = smem + kStages * kStageBytes;
  unsigned char* smem_x = smem_p + kGroups * kParts * kPBytes;
  unsigned char* rest = smem_x + kXBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(rest + kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  volatile int* gave_up = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* tops = reinterpret_cast<float*>(rest + kOffTops);
  float* refs = NARROW ? tops + 768 : reinterpret_cast<float*>(rest + kOffRefs);
  float* sums = tops + 864;  // narrow: [group][part of the tokens][32], up to kOffPrefix
  int* prefix = reinterpret_cast<int*>(rest + kOffPrefix);
  __shared__ int warp_sums[kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
  const int cluster = blockIdx.x >> 1;

  ptx::griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&bars[kFull + i], 1);
      ptx::mbar_init(&bars[kEmpty + i], 1);
    }
    const int warps = NARROW ? 4 : 2 * L.quarters;  // of a group
    ptx::mbar_init(&bars[kQFull], kGroups * warps);
    ptx::mbar_init(&bars[kSFree], warps);
    for (uint32_t i = 0; i < kGroups; ++i) {
      ptx::mbar_init(&bars[kSFull + i], 1);
      ptx::mbar_init(&bars[kXFull + i], 1);
      ptx::mbar_init(&bars[kXFree + i], warps);
      ptx::mbar_init(&bars[kPFull + i], NARROW ? 8 : warps);
      ptx::mbar_init(&bars[kPFree + i], 1);
      ptx::mbar_init(&bars[kODone + i], 1);
    }
    ptx::mbar_init(&bars[kOFree], NARROW ? 4 : 2 * warps);
    ptx::mbar_init(&bars[kLFull], 12);
    ptx::mbar_init(&bars[kLFree], 4);
    for (int i = 0; i < 8; ++i) ptx::mbar_init(&bars[kRef + i], NARROW ? 4 : 2);
    ptx::mbar_init(&bars[kDrain], 1);
    ptx::mbar_init(&bars[kDrain + 1], 1);
    ptx::mbar_init(&bars[kNever], 1);
    *gave_up = 0;
    ptx::mbar_init_fence();
  }
  if (warp == 17) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool aborted = false;
  ptx::griddep_wait();

  // ---- places before every sequence; sequences without tokens: zeros ----
  {
    const int per = (p.num_seqs + kThreads - 1) / kThreads;
    const int beg = min(p.num_seqs, tid * per), end = min(p.num_seqs, beg + per);
    int local = 0;
    for (int s = beg; s < end; ++s) {
      const int n = p.context_lens[s];
      int places = 0;
      if (n > 0 && n <= p.max_context_len) places = (L.lead + (n + kTile - 1) / kTile) * L.row_tiles;
      else if (n != 0 && blockIdx.x == 0) atomicExch(p.err, kDevErrInvalidArg);
      prefix[s + 1] = places;
      local += places;
    }
    int x = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int run = x - local;
    for (int w = 0; w < warp; ++w) run += warp_sums[w];
    if (tid == 0) prefix[0] = 0;
    for (int s = beg; s < end; ++s) prefix[s + 1] = run += prefix[s + 1];
    __syncthreads();
    const float zero[16] = {};
    for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x)
      if (prefix[s + 1] == prefix[s])
        for (int64_t i = tid; i < static_cast<int64_t>(L.rows) * 32; i += kThreads)
          store16(p, static_cast<int64_t>(s) * L.rows * 512 + i * 16, zero);
  }
  if (tid == 0 && rank == 0) L.desc[cluster] = make_int4(-1, 0, 0, 0);  // until it reports an item
  cluster_sync();  // both CTAs' barriers are ready
  const int total = prefix[p.num_seqs];
  const int share = total / L.num_clusters, extra = total - share * L.num_clusters;
  auto run_begin = [&](int c) { return c * share + min(c, extra); };
  const Walk walk{L, prefix, run_begin(cluster), run_begin(cluster + 1)};

  // no product may be in flight when tensor memory is freed
  auto drain = [&](int bar, bool leader) {
    if (leader) {
      ptx::umma_commit(&bars[bar]);
      bool late = false;
      wait(&bars[bar], 0, late);
      if (late) aborted = true;
    }
    aborted = __any_sync(0xffffffffu, aborted);
  };

  auto stall = [&]() {  // pa_test_stall_decode
    if (p.test_stall_ns && !ptx::mbar_wait(&bars[kNever], 0, p.test_stall_ns)) aborted = true;
    __syncwarp();
  };
  // a quarter of an item's queries into tensor memory, once all scores of the item before are formed
  auto load_queries = [&](const Item& it, uint32_t lanes, int r, int quad) {
    const int row = it.rt * 128 + r;
    const bool valid = row < L.rows;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                      (static_cast<int64_t>(it.seq) * L.rows + row) * 576);
    uint32_t v[32];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint4 x = valid ? __ldg(src + rank * 32 + quad * 8 + e) : make_uint4(0, 0, 0, 0);
      v[4 * e] = x.x, v[4 * e + 1] = x.y, v[4 * e + 2] = x.z, v[4 * e + 3] = x.w;
    }
    const uint4 y = valid ? __ldg(src + 64 + rank * 4 + quad) : make_uint4(0, 0, 0, 0);
    __syncwarp();  // the stores are the whole warp's
    ptx::tmem_st32(tmem + lanes + kColQ + quad * 32, v);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(tmem + lanes + kColQ + 128 + quad * 4),
                 "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w)
                 : "memory");
    ptx::tmem_wait_st();
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&bars[kQFull]);
  };
  // the next item's queries, on their way
  auto fetch_queries = [&](const Item& it, int r, int quad) {
    const int row = it.rt * 128 + r;
    const char* src = static_cast<const char*>(p.q) + (static_cast<int64_t>(it.seq) * L.rows + row) * 1152;
    if (row < L.rows) {
      asm volatile("prefetch.global.L2 [%0];" ::"l"(src + rank * 512 + quad * 128));
      if (quad == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 1024 + rank * 64));
    }
  };
  // a quarter of the columns of a row's outputs: normalised, or as a part
  auto put_out = [&](const Item& it, int r, int quad, float m, float l) {
    const int row = it.rt * 128 + r;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const int64_t out_row = static_cast<int64_t>(it.seq) * L.rows + row;
    const int64_t part = (static_cast<int64_t>(cluster) * 2 + (it.t0 > 0 ? 0 : 1)) * L.part_rows + r;
    const bool store = row < L.rows && r < L.part_rows;
    if (!it.whole && rank == 0 && store && quad == 0) *reinterpret_cast<float2*>(L.ml + part * 2) = make_float2(m, l);
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      uint32_t v[32];
      __syncwarp();  // the load is the whole warp's, lanes without a row among it
      load_now(tmem + lanes + quad * 64 + c * 32, v);
      if (c == 1) {  // O is read: the next item's P V may write it
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars[kOFree]);
      }
      if (!store) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(v[16 * h + j]);
        const int64_t col = static_cast<int64_t>(rank) * 256 + quad * 64 + c * 32 + h * 16;
        if (it.whole) {
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] = inv != 0.f ? y[j] * inv : 0.f;
          store16(p, out_row * 512 + col, y);
        } else {
          uint32_t w[8];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(y[8 * q + e]);
            fp4::store32(L.o + part * 512 + col + 8 * q, w);
          }
        }
      }
    }
    // a cluster that begins inside an item's tiles reports it
    if (it.t0 > 0 && rank == 0 && tid == 0) {
      const int wide = extra * (share + 1);
      auto cluster_of = [&](int u) { return u < wide ? u / (share + 1) : extra + (u - wide) / share; };
      L.desc[cluster] = make_int4(it.seq, it.rt, cluster_of(it.start + L.lead), cluster_of(it.end - 1));
    }
  };

  if (warp == 16) {
    // ============================== loads ==============================
    // lane i: the latent part of the tile's page i; lane 16 + i: its position part
    const int page_rows = min(kTile, 1 << L.bs_log), pages = kTile / page_rows;
    const int page = lane & 15;
    const uint64_t policy = L.row_tiles == 1 ? ptx::policy_evict_first() : ptx::policy_evict_normal();
    uint32_t kt = 0;
    if (lane == 0) {
      ptx::prefetch_tensormap(&tm_lat);
      ptx::prefetch_tensormap(&tm_rope);
    }
    walk.each([&](const Item& it, const Item&, bool) {
      const int32_t* table = p.block_tables + static_cast<int64_t>(it.seq) * p.max_blocks_per_seq;
      const int kend = seen_by(L, it, min(L.rows, it.rt * 128 + 128) - 1);  // nobody sees what lies behind it
      auto row_of = [&](int t) -> int {  // the page's first row in the pool, in 8-row groups; -1: nothing to load
        const int tok = t * kTile + page * page_rows;
        if (page >= pages || tok >= kend) return -1;
        int phys = __ldg(table + (tok >> L.bs_log));
        if (phys < 0 || phys >= p.num_blocks) {  // never read outside the pool
          atomicExch(p.err, kDevErrInvalidArg);
          phys = 0;
        }
        return static_cast<int>((static_cast<int64_t>(phys) << L.bs_log) / 8) + (tok & ((1 << L.bs_log) - 1)) / 8;
      };
      int at = row_of(it.t0);
      for (int t = it.t0; t < it.t1 && !aborted; ++t, ++kt) {
        const int now = at;
        if (t + 1 < it.t1) at = row_of(t + 1);
        const int slot = kt % kStages;
        wait(&bars[kEmpty + slot], ((kt / kStages) & 1u) ^ 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) return;
        const uint32_t have = __popc(__ballot_sync(0xffffffffu, now >= 0) & 0xffffu);
        unsigned char* stage = smem + slot * kStageBytes;
        if (lane == 0) ptx::mbar_arrive_expect_tx(&bars[kFull + slot], have * page_rows * (512 + 64));
        __syncwarp();
        if (now >= 0) {
          if (lane < 16)
            ptx::tma_load_4d(stage + page * page_rows * 512, &tm_lat, 0, 0, static_cast<int>(rank) * 4, now,
                             &bars[kFull + slot], policy);
          else
            ptx::tma_load_2d(stage + kLatBytes + page * page_rows * 64, &tm_rope, static_cast<int>(rank) * 32, now * 8,
                             &bars[kFull + slot], policy);
        }
        __syncwarp();
      }
    });
    if (aborted) wait_for_loads(&bars[kFull], kStages, kt);
  } else if (warp == 17) {
    // ===================== products of the scores =====================
    const bool leader = elect_one();
    constexpr uint32_t kIdS = ptx::idesc_bf16_f32(128, kTile, 0, 0);
    const uint64_t desc_k = ptx::smem_desc(smem, 16, 4096, ptx::kLayoutSw128);
    const uint64_t desc_r = ptx::smem_desc(smem + kLatBytes, 16, 512, kLayoutSw64);
    uint32_t kt = 0, items = 0;
    walk.each([&](const Item& it, const Item&, bool) {
      const int kend = seen_by(L, it, min(L.rows, it.rt * 128 + 128) - 1);
      for (int t = it.t0; t < it.t1 && !aborted; ++t, ++kt) {
        const uint32_t slot = kt % kStages;
        wait(&bars[kFull + slot], (kt / kStages) & 1u, aborted);
        if (t == it.t0) wait(&bars[kQFull], items & 1u, aborted);
        wait(&bars[kSFree], (kt & 1u) ^ 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) return;
        unsigned char* stage = smem + slot * kStageBytes;
        const int there = max(0, kend - t * kTile);
        if (there < kTile) {
          // rows behind the last token: zeros, whatever the page or an earlier
          // tile left there (0 * NaN would reach O)
          for (int i = there * 32 + lane; i < kTile * 32; i += 32) {
            const int row = i >> 5, c = i & 31;
            *reinterpret_cast<uint4*>(stage + (row >> 3) * 4096 + (c >> 3) * 1024 + (row & 7) * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
        }
        ptx::tc_fence_after();
        if (leader) {
          const uint64_t dk = desc_k + slot * (kStageBytes >> 4), dr = desc_r + slot * (kStageBytes >> 4);
#pragma unroll
          for (int j = 0; j < 16; ++j)  // chunks of 64 columns, 16 of them (32 bytes) each
            umma_ts(tmem + kColS, tmem + kColQ + j * 8, dk + (j >> 2) * (1024 >> 4) + (j & 3) * 2, kIdS, j > 0);
#pragma unroll
          for (int j = 0; j < 2; ++j) umma_ts(tmem + kColS, tmem + kColQ + 128 + j * 8, dr + j * 2, kIdS, 1);
          ptx::umma_commit(&bars[kSFull + kt % kGroups]);
        }
        __syncwarp();
      }
      ++items;
    });
    drain(kDrain + 1, leader);
  } else if (warp == 18) {
    // ===================== products with the values =====================
    const bool leader = elect_one();
    constexpr uint32_t kIdO = ptx::idesc_bf16_f32(128, 256, 0, 1);
    const uint64_t desc_v = ptx::smem_desc(smem, 1024, 4096, ptx::kLayoutSw128);
    const uint64_t desc_p = ptx::smem_desc(smem_p, 16, 512, kLayoutSw64);
    uint32_t kt = 0, items = 0;
    walk.each([&](const Item& it, const Item&, bool) {
      for (int t = it.t0; t < it.t1 && !aborted; ++t, ++kt) {
        const uint32_t slot = kt % kGroups;
        if (t == it.t0) wait(&bars[kOFree], (items & 1u) ^ 1u, aborted);
        wait(&bars[kPFull + slot], (kt / kGroups) & 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) return;
        ptx::tc_fence_after();
        if (leader) {
          const uint64_t dv = desc_v + (kt % kStages) * (kStageBytes >> 4);
          const uint64_t dp = desc_p + slot * (kParts * kPBytes >> 4);
#pragma unroll
          for (int h = 0; h < kParts; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)  // 16 tokens each
              ptx::umma_bf16(tmem, dp + h * (kPBytes >> 4) + (j >> 1) * (kPBytes / 2 >> 4) + (j & 1) * 2,
                             dv + j * (8192 >> 4), kIdO, h + j > 0 || t > it.t0 ? 1u : 0u);
          ptx::umma_commit(&bars[kEmpty + kt % kStages]);
          ptx::umma_commit(&bars[kPFree + slot]);
          ptx::umma_commit(&bars[kODone + slot]);
        }
        __syncwarp();
      }
      ++items;
    });
    drain(kDrain, leader);
  } else if (NARROW && (warp & 3) == 0) {
    // ========= outputs of few rows: references, then a quarter of the columns =========
    // Lanes 0-31 hold the rows' outputs; the lanes of the other quarters of tensor
    // memory have the same rows' scores, a tile each.
    const int part = warp >> 2;
    uint32_t kt = 0, items = 0;
    walk.each([&](const Item& it, const Item&, bool) {
      const uint32_t k1 = kt + (it.t1 - it.t0);
      float m = -CUDART_INF_F;
      for (uint32_t k = kt; k < k1 && !aborted; ++k) {
        const uint32_t g = k % kGroups;
        wait(&bars[kRef + g], (k / kGroups) & 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) break;
        const float now = refs[g * 32 + lane];
        const float alpha = now != m ? fp4::fast_exp2(m - now) : 1.f;
        m = now;
        if (k > kt && __any_sync(0xffffffffu, alpha != 1.f)) {
          const uint32_t b = (k - 1) % kGroups;
          wait(&bars[kODone + b], ((k - 1) / kGroups) & 1u, aborted);
          aborted = __any_sync(0xffffffffu, aborted);
          if (aborted) break;
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t v[32];
            load_now(tmem + part * 64 + c * 32, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
            ptx::tmem_st32(tmem + part * 64 + c * 32, v);
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars[kPFull + g]);
      }
      const uint32_t kl = k1 - 1;
      kt = k1;
      wait(&bars[kLFull], items & 1u, aborted);
      aborted = __any_sync(0xffffffffu, aborted);
      if (aborted) return;
      float l = 0.f;
#pragma unroll
      for (int i = 0; i < 12; ++i) l += sums[i * 32 + lane];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars[kLFree]);
      ++items;
      wait(&bars[kODone + kl % kGroups], (kl / kGroups) & 1u, aborted);
      aborted = __any_sync(0xffffffffu, aborted);
      if (aborted) return;
      ptx::tc_fence_after();
      put_out(it, lane, part, m, l);
    });
  } else if (NARROW && warp < 16) {
    // ===== scores of few rows: every third tile, a quarter of a row's tokens per thread =====
    const uint32_t group = static_cast<uint32_t>(warp & 3) - 1;  // the tiles k = group mod 3
    const int part = warp >> 2, r = lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    auto all_parts = [&]() { ptx::bar_sync(1 + static_cast<int>(group), 128); };
    uint32_t kt = 0, items = 0;
    bool first = true;
    const float f = p.scale_log2;
    stall();
    walk.each([&](const Item& it, const Item& nxt, bool more) {
      const int row = it.rt * 128 + r;
      const int limit = row < L.rows ? seen_by(L, it, row) : 0;
      const int limit_min = seen_by(L, it, it.rt * 128), limit_max = seen_by(L, it, L.rows - 1);
      const uint32_t k1 = kt + (it.t1 - it.t0);  // behind the last tile
      if (first) load_queries(it, lanes, r, part);
      first = false;
      if (more) fetch_queries(nxt, r, part);
      float m = -CUDART_INF_F, l = 0.f;  // l: of this thread's tokens, on the reference m
      // (a warp that gave up goes on, without waiting, to meet the others at the named barriers)
      for (uint32_t k = kt + (group + 2 * kt) % kGroups; k < k1; k += kGroups) {
        const uint32_t ph = (k / kGroups) & 1u, before_g = (group + 2) % kGroups;
        const int t = it.t0 + static_cast<int>(k - kt);
        wait(&bars[kSFull + group], ph, aborted);
        if (k > 0) wait(&bars[kXFree + before_g], ((k - 1) / kGroups) & 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        ptx::tc_fence_after();
        uint32_t s[16];
        load_now(tmem + lanes + kColS + part * 16, s);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars[kSFree]);
        if (!aborted) {
          const uint32_t dst = remote(smem_x + part * (kXBytes / 4), peer), bar = remote(&bars[kXFull + group], peer);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            store_async4(dst + (j * 32 + r) * 16, __uint_as_float(s[4 * j]), __uint_as_float(s[4 * j + 1]),
                         __uint_as_float(s[4 * j + 2]), __uint_as_float(s[4 * j + 3]), bar);
        }
        // (not once this warp gave up: the bytes of a tile that never comes would be added to the next one's)
        if (r == 0 && part == 0 && !aborted) ptx::mbar_arrive_expect_tx(&bars[kXFull + group], kXBytes);
        if (limit_min < limit_max && limit_min < (t + 1) * kTile) {  // as below
          uint32_t odd = 0;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if ((s[j] & 0x7f800000u) == 0x7f800000u) odd |= 1u << j;
          odd = __shfl_sync(0xffffffffu, odd, 0);
          const int from = max(0, limit_min - t * kTile - part * 16), upto = min(16, limit_max - t * kTile - part * 16);
          if (odd) wait(&bars[kFull + k % kStages], (k / kStages) & 1u, aborted);
          clear_odd(smem + (k % kStages) * kStageBytes + part * 2 * 4096, odd, from, upto, lane);
        }
        wait(&bars[kXFull + group], ph, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        float x[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 y = *reinterpret_cast<const float4*>(smem_x + part * (kXBytes / 4) + (j * 32 + r) * 16);
          x[4 * j] = (__uint_as_float(s[4 * j]) + y.x) * f;
          x[4 * j + 1] = (__uint_as_float(s[4 * j + 1]) + y.y) * f;
          x[4 * j + 2] = (__uint_as_float(s[4 * j + 2]) + y.z) * f;
          x[4 * j + 3] = (__uint_as_float(s[4 * j + 3]) + y.w) * f;
        }
        const int nvis = limit - t * kTile - part * 16;
        if (!__all_sync(0xffffffffu, nvis >= 16)) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j >= nvis) x[j] = -CUDART_INF_F;
        }
        float top = fmaxf(x[0], x[1]);
#pragma unroll
        for (int j = 2; j < 16; j += 2) top = max3(top, x[j], x[j + 1]);
        __syncwarp();  // every lane has read its sums
        if (lane == 0 && !aborted) remote_arrive(remote(&bars[kXFree + group], peer), top);
        float* four = tops + ((ph * kGroups + group) * 4) * 32 + r;
        four[part * 32] = top;
        all_parts();
        top = fmaxf(fmaxf(four[0], four[32]), fmaxf(four[64], four[96]));
        float before = -CUDART_INF_F;  // the reference of the tile before, which another group had
        if (k > kt) wait(&bars[kRef + before_g], ((k - 1) / kGroups) & 1u, aborted);
        // this group's P, and its references, are free once P V of its tile before is complete
        wait(&bars[kPFree + group], ph ^ 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (k > kt) before = refs[before_g * 32 + r];
        const bool raise = top > before + kSlack || (before == -CUDART_INF_F && top > before);
        const float now = raise ? top : before;
        if (part == 0) refs[group * 32 + r] = now;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars[kRef + group]);
        if (m != now) l *= fp4::fast_exp2(m - now);
        m = now;
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        if (aborted) continue;
        unsigned char* prow = smem_p + group * kParts * kPBytes + (part >> 1) * (kPBytes / 2) + (r >> 3) * 512 + (r & 7) * 64;
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[4], w2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = fp4::fast_exp2(x[8 * c + 2 * e] - ref), b = fp4::fast_exp2(x[8 * c + 2 * e + 1] - ref);
            sum0 += a;
            sum1 += b;
            w[e] = pack_bf16(a, b);
            if (HI) w2[e] = pack_bf16(a - __uint_as_float(w[e] << 16), b - __uint_as_float(w[e] & 0xffff0000u));
          }
          const int at = (((part & 1) * 2 + c) ^ ((r >> 1) & 3)) << 4;
          *reinterpret_cast<uint4*>(prow + at) = make_uint4(w[0], w[1], w[2], w[3]);
          if (HI) *reinterpret_cast<uint4*>(prow + kPBytes + at) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
        }
        l += sum0 + sum1;
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars[kPFull + group]);
      }
      const uint32_t kl = k1 - 1;
      if (more) {  // the next item's scores begin beside this one's last product and outputs
        wait(&bars[kSFull + kl % kGroups], (kl / kGroups) & 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        ptx::tc_fence_after();
        load_queries(nxt, lanes, r, part);
      }
      // ---- the rows' sums, on the last reference ----
      wait(&bars[kRef + kl % kGroups], (kl / kGroups) & 1u, aborted);
      wait(&bars[kLFree], (items & 1u) ^ 1u, aborted);
      aborted = __any_sync(0xffffffffu, aborted);
      const float last = refs[(kl % kGroups) * 32 + r];
      if (m != last) l *= fp4::fast_exp2(m - last);
      sums[(group * 4 + part) * 32 + r] = l;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars[kLFull]);
      kt = k1;
      ++items;
    });
  } else if (!NARROW && (warp & 3) < L.quarters) {
    // ===== scores and outputs: every other tile, half of a row's tokens per thread =====
    const int r = tid & 127;  // row of the tile, tensor-memory lane
    const int half = (warp >> 2) & 1;
    const uint32_t group = warp >> 3;  // the tiles k = group mod 2
    const int quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    auto both_halves = [&]() { ptx::bar_sync(1 + 4 * static_cast<int>(group) + quarter, 64); };
    auto everybody = [&]() { ptx::bar_sync(9, L.quarters * 128); };
    const int quad = 2 * static_cast<int>(group) + half;  // a quarter of the columns of Q and O
    uint32_t kt = 0;
    bool first = true;
    const float f = p.scale_log2;
    stall();
    walk.each([&](const Item& it, const Item& nxt, bool more) {
      const int row = it.rt * 128 + r;
      const bool valid = row < L.rows;
      const int last_row = min(L.rows, it.rt * 128 + 128) - 1;
      const int limit = valid ? seen_by(L, it, row) : 0;
      const int limit_min = seen_by(L, it, it.rt * 128), limit_max = seen_by(L, it, last_row);
      const uint32_t k1 = kt + (it.t1 - it.t0);  // behind the last tile
      if (first) load_queries(it, lanes, r, quad);
      first = false;
      if (more) fetch_queries(nxt, r, quad);
      float m = -CUDART_INF_F, l = 0.f;  // l: of this thread's tokens, on the reference m
      // (a warp that gave up goes on, without waiting, to meet the others at the named barriers)
      for (uint32_t k = kt + ((kt ^ group) & 1u); k < k1; k += 2) {
        const uint32_t ph = (k >> 1) & 1u;
        const int t = it.t0 + static_cast<int>(k - kt);
        wait(&bars[kSFull + group], ph, aborted);
        if (k > 0) wait(&bars[kXFree + (group ^ 1u)], ((k - 1) >> 1) & 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        ptx::tc_fence_after();
        uint32_t s[32];
        load_now(tmem + lanes + kColS + half * 32, s);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars[kSFree]);
        // ---- this CTA's partial sums to the other, and the other's ----
        if (!aborted) {
          const uint32_t dst = remote(smem_x + half * (kXBytes / 2), peer), bar = remote(&bars[kXFull + group], peer);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            store_async4(dst + (j * kRows + r) * 16, __uint_as_float(s[4 * j]), __uint_as_float(s[4 * j + 1]),
                         __uint_as_float(s[4 * j + 2]), __uint_as_float(s[4 * j + 3]), bar);
        }
        if (r == 0 && half == 0 && !aborted)
          ptx::mbar_arrive_expect_tx(&bars[kXFull + group], L.quarters * 32 * kTile * 4);
        // Tokens that some rows of the tile see and others do not: a value among
        // this CTA's columns that is not finite becomes zero, so that 0 * NaN does
        // not reach the rows that do not see it; the others have the score.  Such a
        // value makes every row's partial sum not finite, so row 0's says which
        // tokens to look at (its query may be what is not finite, or its sum may
        // have overflowed: the value itself decides).
        if (quarter == 0 && limit_min < limit_max && limit_min < (t + 1) * kTile) {
          uint32_t odd = 0;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if ((s[j] & 0x7f800000u) == 0x7f800000u) odd |= 1u << j;
          odd = __shfl_sync(0xffffffffu, odd, 0);
          const int from = max(0, limit_min - t * kTile - half * 32), upto = min(32, limit_max - t * kTile - half * 32);
          if (odd) wait(&bars[kFull + k % kStages], (k / kStages) & 1u, aborted);
          clear_odd(smem + (k % kStages) * kStageBytes + half * 4 * 4096, odd, from, upto, lane);
        }
        wait(&bars[kXFull + group], ph, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        float x[32];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 y = *reinterpret_cast<const float4*>(smem_x + half * (kXBytes / 2) + (j * kRows + r) * 16);
          x[4 * j] = (__uint_as_float(s[4 * j]) + y.x) * f;
          x[4 * j + 1] = (__uint_as_float(s[4 * j + 1]) + y.y) * f;
          x[4 * j + 2] = (__uint_as_float(s[4 * j + 2]) + y.z) * f;
          x[4 * j + 3] = (__uint_as_float(s[4 * j + 3]) + y.w) * f;
        }
        const int nvis = limit - t * kTile - half * 32;
        if (!__all_sync(0xffffffffu, nvis >= 32)) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j >= nvis) x[j] = -CUDART_INF_F;
        }
        float m0 = x[0], m1 = x[1];
#pragma unroll
        for (int j = 2; j < 32; j += 4) {
          m0 = max3(m0, x[j], x[j + 1]);
          if (j + 3 < 32) m1 = max3(m1, x[j + 2], x[j + 3]);
        }
        float top = fmaxf(m0, m1);
        __syncwarp();  // every lane has read its sums
        if (lane == 0 && !aborted) remote_arrive(remote(&bars[kXFree + group], peer), top);
        float* pair = tops + ((ph * 2 + group) * 2) * 128 + r;
        pair[half * 128] = top;
        both_halves();
        top = fmaxf(top, pair[(half ^ 1) * 128]);
        // the reference of the tile before, which the other group had
        float before = -CUDART_INF_F;
        if (k > kt) {
          wait(&bars[kRef + (group ^ 1u) * 4 + quarter], ((k - 1) >> 1) & 1u, aborted);
          aborted = __any_sync(0xffffffffu, aborted);
          before = refs[(group ^ 1u) * 128 + r];
        }
        const bool raise = top > before + kSlack || (before == -CUDART_INF_F && top > before);
        const float now = raise ? top : before;
        const float alpha = raise && k > kt ? fp4::fast_exp2(before - now) : 1.f;
        if (half == 0) refs[group * 128 + r] = now;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars[kRef + group * 4 + quarter]);
        if (m != now) l *= fp4::fast_exp2(m - now);
        m = now;
        const float ref = m == -CUDART_INF_F ? 0.f : m;
        wait(&bars[kPFree + group], ph ^ 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) continue;
        // [half][128 rows x 64 bytes], 64-byte swizzle
        unsigned char* prow = smem_p + group * kParts * kPBytes + half * (kPBytes / 2) + (r >> 3) * 512 + (r & 7) * 64;
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[4], w2[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a = fp4::fast_exp2(x[8 * c + 2 * e] - ref), b = fp4::fast_exp2(x[8 * c + 2 * e + 1] - ref);
            sum0 += a;
            sum1 += b;
            w[e] = pack_bf16(a, b);
            if (HI) w2[e] = pack_bf16(a - __uint_as_float(w[e] << 16), b - __uint_as_float(w[e] & 0xffff0000u));
          }
          const int at = (c ^ ((r >> 1) & 3)) << 4;
          *reinterpret_cast<uint4*>(prow + at) = make_uint4(w[0], w[1], w[2], w[3]);
          if (HI) *reinterpret_cast<uint4*>(prow + kPBytes + at) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
        }
        l += sum0 + sum1;
        ptx::fence_proxy_async_smem();
        if (k > kt && __any_sync(0xffffffffu, alpha != 1.f)) {
          // this half's columns of O on the new reference, once P V of the tile
          // before is in them (a barrier for every other tile: with one, its
          // phase could be two behind this row's, which looks like done)
          wait(&bars[kODone + (group ^ 1u)], ((k - 1) >> 1) & 1u, aborted);
          aborted = __any_sync(0xffffffffu, aborted);
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            load_now(tmem + lanes + half * 128 + c * 32, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
            ptx::tmem_st32(tmem + lanes + half * 128 + c * 32, v);
          }
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
        }
        __syncwarp();
        if (lane == 0 && !aborted) ptx::mbar_arrive(&bars[kPFull + group]);
      }
      const uint32_t kl = k1 - 1;
      if (more) {  // the next item's scores begin beside this one's last product and outputs
        wait(&bars[kSFull + (kl & 1u)], (kl >> 1) & 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        ptx::tc_fence_after();
        load_queries(nxt, lanes, r, quad);
      }
      // ---- the rows' sums, then the outputs ----
      everybody();
      const float last = refs[(kl & 1u) * 128 + r];
      if (m != last) l *= fp4::fast_exp2(m - last);
      m = last;
      tops[quad * 128 + r] = l;
      everybody();
      l = (tops[r] + tops[128 + r]) + (tops[256 + r] + tops[384 + r]);
      everybody();  // read before the next tile writes there
      wait(&bars[kODone + (kl & 1u)], (kl >> 1) & 1u, aborted);
      aborted = __any_sync(0xffffffffu, aborted);
      kt = k1;
      if (aborted) return;
      ptx::tc_fence_after();
      put_out(it, r, quad, m, l);
    });
  }

  if (aborted) *gave_up = 1;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 17) ptx::tmem_dealloc(tmem, 512);
  if (tid == 0 && *gave_up) atomicExch(p.err, kDevErrTimeout);
  cluster_sync();  // the other CTA may still signal this one's barriers
  if (*gave_up) let_arrive();
}

// Parts of items added up.  The first cluster behind an item's start reports the
// item, and the rows of a cluster that reports none, or a later one of an item, are
// nobody's.  A warp takes a row, or (MANY parts each: few items) a quarter of its
// columns and every eighth part, and the CTA's warps join; there a CTA looks for its
// item's report, since hardly any cluster has one.
constexpr int kMergeThreads = 256;
template <bool MANY>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const Launch L) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  constexpr int N = MANY ? 1 : 4, kStep = MANY ? 8 : 1;  // columns lane * 4 + 128 i; parts of a warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int u = MANY ? blockIdx.x >> 2 : blockIdx.x * (kMergeThreads / 32) + warp;
  const int r = u % L.part_rows, col = (MANY ? (blockIdx.x & 3) * 128 : 0) + lane * 4;
  int b = 1 + u / L.part_rows;
  if (MANY) {  // the report of this rank
    int left = u / L.part_rows;
    b = L.num_clusters;
    for (int i = 1 + lane; i - lane < L.num_clusters && b == L.num_clusters; i += 32) {
      const int4 d = i < L.num_clusters ? L.desc[i] : make_int4(-1, 0, 0, 0);
      const uint32_t those = __ballot_sync(0xffffffffu, d.x >= 0 && d.z == i - 1);
      const int n = __popc(those);
      if (left < n) b = i - lane + static_cast<int>(__fns(those, 0, left + 1));
      left -= n;
    }
  }
  if (b >= L.num_clusters) return;
  const int4 d = L.desc[b];
  const int row = d.y * 128 + r;
  if (d.x < 0 || d.z != b - 1 || row >= L.rows) return;
  // the part that begins the item lies in its cluster's second place, the others in their first
  auto part_of = [&](int c) { return (static_cast<int64_t>(c) * 2 + (c == d.z ? 1 : 0)) * L.part_rows + r; };
  float4 acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float ref = -CUDART_INF_F, sum = 0.f;
  auto add = [&](float2 e, const float4 (&x)[N]) {
    if (e.y == 0.f) return;  // a part that this row sees nothing of
    const float now = fmaxf(ref, e.x), w = fp4::fast_exp2(e.x - now), old = fp4::fast_exp2(ref - now);
    ref = now;
    sum = fmaf(w, e.y, sum * old);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      acc[i].x = fmaf(w, x[i].x, acc[i].x * old);
      acc[i].y = fmaf(w, x[i].y, acc[i].y * old);
      acc[i].z = fmaf(w, x[i].z, acc[i].z * old);
      acc[i].w = fmaf(w, x[i].w, acc[i].w * old);
    }
  };
#pragma unroll MANY ? 4 : 2
  for (int c = d.z + (MANY ? warp : 0); c <= d.w; c += kStep) {
    const float2 e = __ldcg(reinterpret_cast<const float2*>(L.ml + part_of(c) * 2));
    float4 x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __ldcg(reinterpret_cast<const float4*>(L.o + part_of(c) * 512 + col + 128 * i));
    add(e, x);
  }
  if (MANY) {
    __shared__ float2 ml[8];
    __shared__ float4 rows[8][32];
    if (lane == 0) ml[warp] = make_float2(ref, sum);
    rows[warp][lane] = acc[0];
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      const float4 x[1] = {rows[w][lane]};
      add(ml[w], reinterpret_cast<const float4(&)[N]>(x));
    }
  }
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t at = (static_cast<int64_t>(d.x) * L.rows + row) * 512 + col + 128 * i;
    const float4 y = make_float4(acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv);
    if (L.p.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(L.p.out) + at) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(L.p.out) + at) = y;
  }
}

int smem_bytes(bool hi, bool narrow, int seqs) {
  return 1024 + stages_of(hi, narrow) * kStageBytes + groups_of(narrow) * (hi ? 2 : 1) * p_bytes(narrow) + x_bytes(narrow) + kOffPrefix +
         (seqs + 64) / 64 * 256;
}

// Sequences of one launch: their places fit an int.  0: not even one's do.
int seqs_of(int num_seqs, int64_t row_tiles, int max_context_len) {
  const int64_t places = (kMostLead + (static_cast<int64_t>(max_context_len) + kTile - 1) / kTile) * row_tiles;
  const int64_t fit = ((int64_t(1) << 31) - 1) / places;
  const int64_t most = fit < kMaxSeqs ? fit : kMaxSeqs;
  return static_cast<int>(num_seqs < most ? num_seqs : most);
}

int max_clusters() { return static_cast<int>(device_sm_count() / 2); }
int part_rows_of(int64_t rows) { return static_cast<int>(rows < 128 ? rows : 128); }

}  // namespace latent_decode_detail

size_t latent_decode_workspace(int num_seqs, int q_len, int num_heads, int max_context_len) {
  using namespace latent_decode_detail;
  const int64_t rows = static_cast<int64_t>(q_len) * num_heads;
  if (num_seqs > 0 && seqs_of(num_seqs, (rows + 127) / 128, max_context_len) == 0) return 0;
  // header | reports | maxima and sums | parts
  const int64_t n = max_clusters();
  return static_cast<size_t>(256 + (n * 16 + 255) / 256 * 256 + 2 * n * part_rows_of(rows) * (512 + 2) * 4);
}

cudaError_t launch_latent_decode(const LatentDecodeParams& p, cudaStream_t stream) {
  using namespace latent_decode_detail;
  const int64_t rows = static_cast<int64_t>(p.q_len) * p.num_heads, row_tiles = (rows + 127) / 128;
  const int seqs = seqs_of(p.num_seqs, row_tiles, p.max_context_len);
  const int n = max_clusters();
  const bool hi = !p.out_bf16;
  // the pool as groups of 8 rows of 8 chunks of 64 columns, and as rows of position columns
  CUtensorMap tm_lat, tm_rope;
  const uint64_t pool_rows = static_cast<uint64_t>(p.num_blocks) * p.block_size;
  const uint32_t box_rows = p.block_size < kTile ? p.block_size : kTile;
  {
    const uint64_t dims[4] = {64, 8, 8, pool_rows / 8}, strides[3] = {1152, 128, 9216};
    const uint32_t box[4] = {64, 8, 4, box_rows / 8};
    if (!encode_bf16_tiles(&tm_lat, 4, p.cache, dims, strides, box, 128)) return cudaErrorInvalidValue;
  }
  {
    const uint64_t dims[2] = {64, pool_rows}, strides[1] = {1152};
    const uint32_t box[2] = {32, box_rows};
    if (!encode_bf16_tiles(&tm_rope, 2, static_cast<const __nv_bfloat16*>(p.cache) + 512, dims, strides, box, 64))
      return cudaErrorInvalidValue;
  }
  for (int seq0 = 0; seq0 < p.num_seqs; seq0 += seqs) {
    Launch L{};
    L.p = p;
    L.p.num_seqs = p.num_seqs - seq0 < seqs ? p.num_seqs - seq0 : seqs;
    L.p.q = static_cast<const __nv_bfloat16*>(p.q) + static_cast<int64_t>(seq0) * rows * 576;
    L.p.out = static_cast<unsigned char*>(p.out) + static_cast<int64_t>(seq0) * rows * 512 * (p.out_bf16 ? 2 : 4);
    L.p.context_lens += seq0;
    L.p.block_tables += static_cast<int64_t>(seq0) * p.max_blocks_per_seq;
    L.rows = static_cast<int>(rows);
    L.row_tiles = static_cast<int>(row_tiles);
    L.quarters = row_tiles > 1 ? 4 : static_cast<int>((rows + 31) / 32);
    L.bs_log = __builtin_ctz(static_cast<unsigned>(p.block_size));
    L.part_rows = part_rows_of(rows);
    // 16 rows: 2 tiles (64 us the batch of 256; 3: 64, 4: 66, 6: 70); 128 rows, whose outputs and queries are
    // eight times as much: 7 (batch of 64: 73 us; 3: 81, 5: 75)
    L.lead = 2 + 5 * L.part_rows / 128;
    // every SM, while a cluster gets a few tiles
    const int64_t tiles = static_cast<int64_t>(L.p.num_seqs) * row_tiles * ((static_cast<int64_t>(p.max_context_len) + kTile - 1) / kTile);
    const int64_t want = (tiles + kMinTiles - 1) / kMinTiles;
    L.num_clusters = static_cast<int>(want < 1 ? 1 : (want < n ? want : n));
    L.desc = reinterpret_cast<int4*>(p.ws + 256);
    L.ml = reinterpret_cast<float*>(p.ws + 256 + (static_cast<int64_t>(n) * 16 + 255) / 256 * 256);
    L.o = L.ml + static_cast<int64_t>(2) * n * L.part_rows * 2;
    const bool narrow = rows <= 32;
    const int smem = smem_bytes(hi, narrow, L.p.num_seqs);
    const void* fn = narrow ? (hi ? reinterpret_cast<const void*>(&decode_kernel<true, true>)
                                  : reinterpret_cast<const void*>(&decode_kernel<false, true>))
                            : (hi ? reinterpret_cast<const void*>(&decode_kernel<true, false>)
                                  : reinterpret_cast<const void*>(&decode_kernel<false, false>));
    int per_sm = 0;
    cudaError_t e = fp4_occupancy(fn, kThreads, smem, &per_sm);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * L.num_clusters));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    void* args[] = {&L, &tm_lat, &tm_rope};
    e = cudaLaunchKernelExC(&cfg, fn, args);
    if (e != cudaSuccess) return e;
    if (L.num_clusters > 1) {
      // Parts of a row spread over warps, and a warp a row: 1 x 30000 tokens with 16 heads 31 and 62 us, with
      // 128 heads 39 and 76; 4 x 8192 with 128 heads 43 and 45, 8 x 4096 45 and 41 (its CTAs are too many);
      // with 16 heads 8 x 4096 29 and 31, 15 x 4000 the same
      const int64_t items = static_cast<int64_t>(L.p.num_seqs) * row_tiles;
      const bool many = items < 16 && items * L.part_rows <= 512;
      const dim3 ctas(static_cast<unsigned>(
          many ? items * L.part_rows * 4 : (static_cast<int64_t>(L.num_clusters - 1) * L.part_rows + 7) / 8));
      e = many ? launch_early(merge_kernel<true>, ctas, kMergeThreads, stream, L)
               : launch_early(merge_kernel<false>, ctas, kMergeThreads, stream, L);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

}  // namespace pa
