// Accumulated attention weights: weights[t] += sum over a window's queries and
// heads of softmax_t(scale q . k[t]).
//
// Three steps.  (1) scores: S = Q K^T on the 5th-generation tensor cores, with each
// tile's maximum and sum of exponentials per row; of few rows written out in fp32
// (log2 domain, -inf where a row does not see a token).  (2) a row's logarithm of
// its sum from its tiles'.  (3) a token's 2^(s - lse) added up over the rows in a
// fixed order, and into its weight: from the stored scores, or of many rows from
// scores formed a second time.
//
// Stored scores cost 8 bytes a row and token, written and read: 32 of a decode
// step's four rows against 256 of the key, but 1024 of 128 rows, four times the key.
//
// Measured: a decode step of 256 sequences, 32 q / 8 kv heads (448 MB of keys) 96 us,
// of them the scores 78 (5.8 TB/s, 85% of a plain copy), the sums 6, the tokens 12;
// a window of 32 queries over 4 x 9000 to 16384 tokens 64 us, 29 and 33 of them the
// two times that the scores are formed.  No unit bounds those (special functions 28
// and 25% busy, issue slots 49 and 37%, tensor pipe 21 and 19%, memory 52 and 46%):
// a tile's chain does, product, tensor-memory load, maximum, exponentials, with two
// tiles in it (half of the warps for the scores: 74; stored scores: 132).  A step of
// 128 heads over 44 MB of latent rows 33 us, 21 of them the scores: 147 KB of
// queries leave room for two tiles of 32 tokens, whose loads, products and scores
// hardly overlap (special functions 4%, memory 26%); the rest is the two kernels
// behind.  Windows of many rows over latent rows or heads of 256 store all scores:
// 32 queries of 128 heads over 4 x 16384 latent rows 1.2 ms, a sequence a launch.
//
// Step 1: a CTA walks an equal run of units (token tile of a sequence, kv head and
// row tile).  The rows of a tile are the heads of a kv head's group, query after
// query.  Warps 0-3 and 4-7 take the scores of every other unit (a row a thread), 8
// loads, 9 issues products; where a tile has 64 tokens or more, eight further warps
// take its second half.  A page is one TMA box: [8-token group]
// [chunk of 64 dims][8 rows x 128 bytes] of its kv head.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "decode.cuh"
#include "fp4.cuh"
#include "latent.cuh"
#include "ptx.cuh"
#include "umma.cuh"

namespace pa {
namespace weights_detail {

using namespace um;

constexpr int kThreads = 10 * 32;
// warps that take scores: a row's tokens in two halves where a tile has two of 32
__host__ __device__ constexpr int halves_of(int nc, bool few) { return !few && nc <= 4 ? 2 : 1; }
__host__ __device__ constexpr int threads_of(int nc, bool few) { return (2 + 8 * halves_of(nc, few)) * 32; }
constexpr int kMaxSeqs = 1024;  // of one launch: their units lie in shared memory
constexpr int64_t kScoreBytes = int64_t(512) << 20;  // of one launch, where a sequence does not need more

// NC: chunks of 64 dims; tokens of a tile, tiles and query tiles in shared memory
template <int NC>
struct Shape {
  static constexpr int kTokens = NC <= 2 ? 128 : NC <= 4 ? 64 : 32;
  static constexpr int kStageBytes = kTokens * NC * 128;
  static constexpr int kStages = NC == 1 ? 8 : NC <= 4 ? 4 : 2;
  static constexpr int kQBytes = NC * 16384;  // [chunk][128 rows x 128 bytes]
  static constexpr int kQSlots = NC <= 2 ? 2 : 1;
  static constexpr int kOffQ = kStages * kStageBytes;
  static constexpr int kOffBar = kOffQ + kQSlots * kQBytes;
  static constexpr int kOffPrefix = kOffBar + 256;
};

enum : int { kFull = 0, kFree = 8, kQFull = 16, kQFree = 18, kSFull = 20, kSFree = 22, kDrain = 24, kNever = 25, kNumBars = 26 };

struct Launch {
  WeightsParams p;
  int group;        // query heads of a kv head
  int rows;         // of a kv head: window * group
  int tile_queries; // queries of a row tile; its rows are tile_queries * group <= 128
  int row_tiles;
  int bs_log;
  int64_t pitch;    // scores of a row
  int tiles_pitch;  // tiles of a row
  float* lse;       // [seqs][kv heads * rows]
  float2* tile_ml;  // [seqs][kv heads * rows][tiles_pitch] maximum (log2), sum
  float* scores;    // [seqs][kv heads * rows][pitch]; null: formed a second time instead
};

__device__ __forceinline__ int length_of(const WeightsParams& p, int seq) {
  const int n = p.context_lens[seq];
  return n > 0 && n <= p.max_context_len ? n : 0;
}

// prefix[s]: units before sequence s, `each` of them a tile of `tokens`
template <int THREADS>
__device__ __forceinline__ void count_units(const WeightsParams& p, int* prefix, int* warp_sums, int tokens, int each) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (p.num_seqs + THREADS - 1) / THREADS;
  const int beg = min(p.num_seqs, tid * per), end = min(p.num_seqs, beg + per);
  int local = 0;
  for (int s = beg; s < end; ++s) {
    const int n = length_of(p, s);
    if (n != p.context_lens[s] && blockIdx.x == 0) atomicExch(p.err, kDevErrInvalidArg);
    const int units = (n + tokens - 1) / tokens * each;
    prefix[s + 1] = units;
    local += units;
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
}

// A unit: a token tile of (sequence, kv head, row tile).
struct Unit {
  int seq, len, tiles;
  int kvh, rt, tile;
};

template <int NC>
struct Walk {
  const Launch& L;
  const int* prefix;
  int u0, u1;
  __device__ __forceinline__ void open(Unit& x) const {
    x.len = length_of(L.p, x.seq);
    x.tiles = (x.len + Shape<NC>::kTokens - 1) / Shape<NC>::kTokens;
  }
  __device__ __forceinline__ void find(Unit& x) const {
    int lo = 0, hi = L.p.num_seqs - 1;
    while (lo < hi) {  // the last sequence that starts at or before it
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= u0) lo = mid;
      else hi = mid - 1;
    }
    x.seq = lo;
    open(x);
    const int r = u0 - prefix[lo], at = r / x.tiles;
    x.tile = r - at * x.tiles;
    x.kvh = at / L.row_tiles;
    x.rt = at - x.kvh * L.row_tiles;
  }
  // f(unit, first of its queries here, last of its queries here)
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if (u0 >= u1) return;
    Unit x;
    find(x);
    bool first = true;
    for (int u = u0; u < u1; ++u) {
      const bool last = x.tile + 1 == x.tiles;
      f(x, first, last || u + 1 == u1);
      first = last;
      if (!last) {
        ++x.tile;
        continue;
      }
      x.tile = 0;
      if (++x.rt < L.row_tiles) continue;
      x.rt = 0;
      if (++x.kvh < L.p.num_kv_heads) continue;
      x.kvh = 0;
      if (u + 1 == u1) continue;
      do ++x.seq;
      while (prefix[x.seq + 1] == u + 1);  // sequences without units
      open(x);
    }
  }
};

// FEW: at most 16 rows.  Then tokens are the product's rows and queries its
// columns: a thread has one token's scores of all rows instead of one row's of all
// tokens, so that four warps share the exponentials that a quarter of the lanes
// of one would form, and a row's maximum and sum go through shuffles.
template <int NC, bool FEW>
__global__ void __launch_bounds__(threads_of(NC, FEW), 1)
    scores_kernel(const __grid_constant__ Launch L, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_q) {
  using S = Shape<NC>;
  constexpr int kHalves = halves_of(NC, FEW);
  const WeightsParams& p = L.p;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  volatile int* gave_up = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* prefix = reinterpret_cast<int*>(smem + S::kOffPrefix);
  __shared__ int warp_sums[threads_of(NC, FEW) / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  ptx::griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      ptx::mbar_init(&bars[kFull + i], 1);
      ptx::mbar_init(&bars[kFree + i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars[kQFull + i], 1);
      ptx::mbar_init(&bars[kQFree + i], 1);
      ptx::mbar_init(&bars[kSFull + i], 1);
      ptx::mbar_init(&bars[kSFree + i], 4 * kHalves);
    }
    ptx::mbar_init(&bars[kDrain], 1);
    ptx::mbar_init(&bars[kNever], 1);
    *gave_up = 0;
    ptx::mbar_init_fence();
  }
  if (warp == 9) {
    ptx::tmem_alloc(tmem_slot, 256);
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool aborted = false;
  ptx::griddep_wait();

  count_units<threads_of(NC, FEW)>(p, prefix, warp_sums, S::kTokens, p.num_kv_heads * L.row_tiles);
  const int total = prefix[p.num_seqs];
  const int share = total / gridDim.x, extra = total - share * gridDim.x;
  auto run_begin = [&](int c) { return c * share + min(c, extra); };
  const Walk<NC> walk{L, prefix, run_begin(blockIdx.x), run_begin(blockIdx.x + 1)};

  if (warp == 8) {
    // ============================== loads ==============================
    // lane i: the unit's page i
    const int page_rows = min(S::kTokens, 1 << L.bs_log), pages = S::kTokens / page_rows;  // at most 16
    const uint64_t policy = L.row_tiles == 1 ? ptx::policy_evict_first() : ptx::policy_evict_normal();
    uint32_t k = 0, qk = 0;
    // a unit's pages are looked up while the one before is loaded
    struct {
      int at, q_head, q_row;
      bool first;
    } ahead{-1, 0, 0, false};
    auto issue = [&]() {
      if (aborted) return;
      if (ahead.first) {  // the row tile's queries; rows past them are nobody's
        const uint32_t slot = qk % S::kQSlots;
        wait(&bars[kQFree + slot], ((qk / S::kQSlots) & 1u) ^ 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) return;
        ++qk;
        if (lane == 0) {
          const uint32_t rows = static_cast<uint32_t>(min(L.tile_queries, p.window) * L.group);
          ptx::mbar_arrive_expect_tx(&bars[kQFull + slot], rows * 128u * NC);
          for (int c = 0; c < NC; ++c)
            tma_load_3d(smem + S::kOffQ + slot * S::kQBytes + c * 16384, &tm_q, c * 64, ahead.q_head, ahead.q_row,
                        &bars[kQFull + slot], ptx::policy_evict_normal());
        }
        __syncwarp();
      }
      const uint32_t slot = k % S::kStages;
      wait(&bars[kFree + slot], ((k / S::kStages) & 1u) ^ 1u, aborted);
      aborted = __any_sync(0xffffffffu, aborted);
      if (aborted) return;
      const uint32_t have = __popc(__ballot_sync(0xffffffffu, ahead.at >= 0));
      if (lane == 0) ptx::mbar_arrive_expect_tx(&bars[kFull + slot], have * page_rows * 128u * NC);
      __syncwarp();
      if (ahead.at >= 0)
        ptx::tma_load_4d(smem + slot * S::kStageBytes + lane * page_rows * 128 * NC, &tm_k, 0, 0, 0, ahead.at,
                         &bars[kFull + slot], policy);
      __syncwarp();
      ++k;
    };
    bool any = false;
    walk.each([&](const Unit& x, bool first, bool) {
      const int tok = x.tile * S::kTokens + lane * page_rows;
      int phys = -1;
      const bool there = lane < pages && tok < x.len;
      if (there) phys = __ldg(p.block_tables + static_cast<int64_t>(x.seq) * p.max_blocks_per_seq + (tok >> L.bs_log));
      if (any) issue();
      any = true;
      if (there && (phys < 0 || phys >= p.num_blocks)) {  // never read outside the pool
        atomicExch(p.err, kDevErrInvalidArg);
        phys = 0;
      }
      // the page's first row in the pool, in 8-row groups
      ahead.at = there ? static_cast<int>(((static_cast<int64_t>(phys) * p.num_kv_heads + x.kvh) << L.bs_log) / 8) +
                             (tok & ((1 << L.bs_log) - 1)) / 8
                       : -1;
      ahead.q_head = x.kvh * L.group;
      ahead.q_row = x.seq * p.window + x.rt * L.tile_queries;
      ahead.first = first;
    });
    if (any) issue();
    if (aborted) {
      wait_for_loads(&bars[kFull], S::kStages, k);
      wait_for_loads(&bars[kQFull], S::kQSlots, qk);
    }
  } else if (warp == 9) {
    // ============================ products ============================
    const bool leader = elect_one();
    constexpr uint32_t kId = ptx::idesc_bf16_f32(128, FEW ? 16 : S::kTokens, 0, 0);
    const uint64_t desc_k = ptx::smem_desc(smem, 16, 1024 * NC, ptx::kLayoutSw128);
    const uint64_t desc_q = ptx::smem_desc(smem + S::kOffQ, 16, 1024, ptx::kLayoutSw128);
    uint32_t k = 0, qk = 0;
    walk.each([&](const Unit&, bool first, bool last) {
      if (aborted) return;
      const uint32_t slot = k % S::kStages, qslot = qk % S::kQSlots;
      if (first) wait(&bars[kQFull + qslot], (qk / S::kQSlots) & 1u, aborted);
      wait(&bars[kSFree + (k & 1u)], ((k >> 1) & 1u) ^ 1u, aborted);
      wait(&bars[kFull + slot], (k / S::kStages) & 1u, aborted);
      aborted = __any_sync(0xffffffffu, aborted);
      if (aborted) return;
      ptx::tc_fence_after();
      if (leader) {
        const uint64_t dk = desc_k + slot * (S::kStageBytes >> 4), dq = desc_q + qslot * (S::kQBytes >> 4);
#pragma unroll
        for (int c = 0; c < 4 * NC; ++c) {
          const uint64_t q = dq + (c >> 2) * (16384 >> 4) + (c & 3) * 2, t = dk + (c >> 2) * (1024 >> 4) + (c & 3) * 2;
          ptx::umma_bf16(tmem + (k & 1u) * 128, FEW ? t : q, FEW ? q : t, kId, c > 0);
        }
        ptx::umma_commit(&bars[kSFull + (k & 1u)]);
        ptx::umma_commit(&bars[kFree + slot]);
        if (last) ptx::umma_commit(&bars[kQFree + qslot]);
      }
      __syncwarp();
      ++k;
      qk += last;
    });
    if (leader) {  // nothing may be in flight when tensor memory is freed
      ptx::umma_commit(&bars[kDrain]);
      bool late = false;
      wait(&bars[kDrain], 0, late);
      if (late) aborted = true;
    }
    aborted = __any_sync(0xffffffffu, aborted);
  } else {
    // ==================== scores: one row per thread ====================
    // warps 0-7 the first half of a tile's tokens, 10-17 the second; lanes by the warp's number mod 4
    const uint32_t buffer = warp < 8 ? warp >> 2 : (warp - 10) >> 2;  // the units k = buffer mod 2
    const int half = warp < 8 ? 0 : 1;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + buffer * 128;
    uint32_t k = 0;
    const int64_t all_rows = static_cast<int64_t>(p.num_kv_heads) * L.rows;
    if (p.test_stall_ns && !ptx::mbar_wait(&bars[kNever], 0, p.test_stall_ns)) aborted = true;  // pa_test_stall_decode
    __syncwarp();
    walk.each([&](const Unit& x, bool, bool) {
      const uint32_t mine = k++;
      if (aborted || (mine & 1u) != buffer) return;
      wait(&bars[kSFull + buffer], (mine >> 1) & 1u, aborted);
      aborted = __any_sync(0xffffffffu, aborted);
      if (aborted) return;
      ptx::tc_fence_after();
      if constexpr (FEW) {
        uint32_t v[16];
        load_now(at, v);
        const int64_t row0 = x.seq * all_rows + static_cast<int64_t>(x.kvh) * L.rows;
        float* dst = L.scores + row0 * L.pitch + x.tile * S::kTokens + r;
        const int tok = x.tile * S::kTokens + r;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (j >= L.rows) break;
          const int seen = x.len - p.window + 1 + j / L.group;  // tokens that this row sees
          const float y = tok < seen ? __uint_as_float(v[j]) * p.scale_log2 : -CUDART_INF_F;
          dst[j * L.pitch] = y;
          float top = y;
#pragma unroll
          for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          float e = fp4::fast_exp2(y - (top == -CUDART_INF_F ? 0.f : top));
#pragma unroll
          for (int o = 16; o; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
          // a warp's 32 tokens have statistics of their own
          if (lane == 0) L.tile_ml[(row0 + j) * L.tiles_pitch + x.tile * 4 + (warp & 3)] = make_float2(top, e);
        }
      } else {
        const int tile_rows = min(L.tile_queries * L.group, L.rows - x.rt * L.tile_queries * L.group);
        const int row = x.rt * L.tile_queries * L.group + r;
        const bool valid = r < tile_rows;
        if ((warp & 3) * 32 < tile_rows) {
          const int seen = x.len - p.window + 1 + row / L.group;  // tokens that this row sees
          const int from = half * (S::kTokens / kHalves);
          const int nvis = seen - x.tile * S::kTokens - from;
          const int64_t grow = x.seq * all_rows + static_cast<int64_t>(x.kvh) * L.rows + row;
          float* dst = L.scores + grow * L.pitch + x.tile * S::kTokens + from;
          const uint64_t ff = fp4::pair(p.scale_log2, p.scale_log2);
          float top = -CUDART_INF_F, sum = 0.f;
#pragma unroll 1
          for (int c = 0; c < S::kTokens / kHalves; c += 32) {
            uint32_t v[32];
            load_now(at + from + c, v);
            uint64_t y[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              y[j] = fp4::mul2(fp4::pair(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), ff);
            if (!__all_sync(0xffffffffu, nvis >= c + 32)) {
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float2 t = fp4::unpair(y[j]);
                y[j] = fp4::pair(c + 2 * j < nvis ? t.x : -CUDART_INF_F, c + 2 * j + 1 < nvis ? t.y : -CUDART_INF_F);
              }
            }
            float m0 = top, m1 = -CUDART_INF_F;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float2 t = fp4::unpair(y[j]), u = fp4::unpair(y[j + 1]);
              m0 = max3(m0, t.x, t.y);
              m1 = max3(m1, u.x, u.y);
            }
            const float now = fmaxf(m0, m1), ref = now == -CUDART_INF_F ? 0.f : now;
            const uint64_t less = fp4::pair(-ref, -ref);
            uint64_t s0 = 0, s1 = 0;
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float2 t = fp4::unpair(fp4::add2(y[j], less)), u = fp4::unpair(fp4::add2(y[j + 1], less));
              s0 = fp4::add2(s0, fp4::pair(fp4::fast_exp2(t.x), fp4::fast_exp2(t.y)));
              s1 = fp4::add2(s1, fp4::pair(fp4::fast_exp2(u.x), fp4::fast_exp2(u.y)));
            }
            const float2 t = fp4::unpair(fp4::add2(s0, s1));
            sum = fmaf(sum, fp4::fast_exp2(top - ref), t.x + t.y);
            top = now;
            if (valid && L.scores) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 z = fp4::unpair(y[4 * q + e]);
                  w[2 * e] = __float_as_uint(z.x), w[2 * e + 1] = __float_as_uint(z.y);
                }
                fp4::store32(dst + c + 8 * q, w);
              }
            }
            __syncwarp();  // the next load is the whole warp's
          }
          if (valid) L.tile_ml[grow * L.tiles_pitch + x.tile * kHalves + half] = make_float2(top, sum);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars[kSFree + buffer]);
    });
  }

  if (aborted) *gave_up = 1;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 9) ptx::tmem_dealloc(tmem, 256);
  if (tid == 0 && *gave_up) atomicExch(p.err, kDevErrTimeout);
}

// A warp: a row's log2 of its sum over its tiles (infinity where it sees nothing).
__global__ void __launch_bounds__(256) lse_kernel(const Launch L, int tokens) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t all_rows = static_cast<int64_t>(L.p.num_kv_heads) * L.rows;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  if (row >= all_rows * L.p.num_seqs) return;
  const int len = length_of(L.p, static_cast<int>(row / all_rows));
  const int seen = len - L.p.window + 1 + static_cast<int>(row % all_rows) % L.rows / L.group;
  const int tiles = (len + tokens - 1) / tokens;  // (what a row's statistics stand for)
  float m = -CUDART_INF_F, s = 0.f;
  for (int i = lane; i < tiles; i += 32) {
    const float2 e = __ldcg(L.tile_ml + row * L.tiles_pitch + i);
    const float now = fmaxf(m, e.x), ref = now == -CUDART_INF_F ? 0.f : now;
    s = fmaf(s, fp4::fast_exp2(m - ref), e.y * fp4::fast_exp2(e.x - ref));
    m = now;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    const float now = fmaxf(m, m2), ref = now == -CUDART_INF_F ? 0.f : now;
    s = fmaf(s, fp4::fast_exp2(m - ref), s2 * fp4::fast_exp2(m2 - ref));
    m = now;
  }
  if (lane == 0) L.lse[row] = seen > 0 ? m + log2f(s) : CUDART_INF_F;
}

// A CTA: 128 tokens of a sequence; its warps share the rows, four tokens a lane.
constexpr int kAddWarps = 8;
__global__ void __launch_bounds__(32 * kAddWarps) add_kernel(const Launch L) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int seq = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = length_of(L.p, seq), t0 = blockIdx.x * 128;
  if (t0 >= len) return;
  const int rows = L.p.num_kv_heads * L.rows;
  const float* lse = L.lse + static_cast<int64_t>(seq) * rows;
  const float* s = L.scores + static_cast<int64_t>(seq) * rows * L.pitch + t0 + lane * 4;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  if (t0 + lane * 4 < len) {
#pragma unroll 8
    for (int r = warp; r < rows; r += kAddWarps) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(s + r * L.pitch));
      const float l = __ldcg(lse + r);
      sum.x += fp4::fast_exp2(x.x - l);
      sum.y += fp4::fast_exp2(x.y - l);
      sum.z += fp4::fast_exp2(x.z - l);
      sum.w += fp4::fast_exp2(x.w - l);
    }
  }
  __shared__ float4 part[kAddWarps][32];
  part[warp][lane] = sum;
  __syncthreads();
  if (threadIdx.x < 128 && t0 + static_cast<int>(threadIdx.x) < len) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kAddWarps; ++w) v += reinterpret_cast<const float*>(part[w])[threadIdx.x];
    L.p.weights[seq * L.p.weights_stride + t0 + threadIdx.x] += v;
  }
}

// Step 3 without stored scores: a token tile's products with every row tile again,
// tokens as the product's rows (128) and queries as its columns, so that a thread
// adds up one token's probabilities of half a row tile and needs only its partner's
// in the end.  Warps 0-3 add the first halves, 4-7 the second ones, 8 loads, 9
// issues products.
template <int NC>
__global__ void __launch_bounds__(kThreads, 1)
    again_kernel(const __grid_constant__ Launch L, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_q) {
  using S = Shape<NC>;
  static_assert(S::kTokens == 128 && S::kQSlots == 2, "a tile's tokens are the product's rows");
  const WeightsParams& p = L.p;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  volatile int* gave_up = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* prefix = reinterpret_cast<int*>(smem + S::kOffPrefix);
  __shared__ int warp_sums[kThreads / 32];
  __shared__ __align__(16) float row_lse[2][128];
  __shared__ float other[128];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  ptx::griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      ptx::mbar_init(&bars[kFull + i], 1);
      ptx::mbar_init(&bars[kFree + i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars[kQFull + i], 1);
      ptx::mbar_init(&bars[kQFree + i], 1);
      ptx::mbar_init(&bars[kSFull + i], 1);
      ptx::mbar_init(&bars[kSFree + i], 8);
    }
    ptx::mbar_init(&bars[kDrain], 1);
    ptx::mbar_init(&bars[kNever], 1);
    *gave_up = 0;
    ptx::mbar_init_fence();
  }
  if (warp == 9) {
    ptx::tmem_alloc(tmem_slot, 256);
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool aborted = false;
  ptx::griddep_wait();
  count_units<kThreads>(p, prefix, warp_sums, S::kTokens, 1);
  const int total = prefix[p.num_seqs];
  const int share = total / gridDim.x, extra = total - share * gridDim.x;
  auto run_begin = [&](int c) { return c * share + min(c, extra); };
  const int u0 = run_begin(blockIdx.x), u1 = run_begin(blockIdx.x + 1);
  const int inner = p.num_kv_heads * L.row_tiles;
  const int64_t all_rows = static_cast<int64_t>(p.num_kv_heads) * L.rows;

  // f(sequence, its length, tile) for the tiles of this CTA
  auto tiles = [&](auto f) {
    if (u0 >= u1) return;
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {  // the last sequence that starts at or before it
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= u0) lo = mid;
      else hi = mid - 1;
    }
    for (int u = u0; u < u1; ++u) {
      while (prefix[lo + 1] == u) ++lo;  // the next sequence with tiles
      f(lo, length_of(p, lo), u - prefix[lo]);
    }
  };

  if (warp == 8) {
    // ============================== loads ==============================
    const int page_rows = min(128, 1 << L.bs_log), pages = 128 / page_rows;
    const uint64_t normal = ptx::policy_evict_normal();
    uint32_t k = 0;
    tiles([&](int seq, int len, int tile) {
      const int tok = tile * 128 + lane * page_rows;
      int phys = -1;
      if (lane < pages && tok < len) {
        phys = __ldg(p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq + (tok >> L.bs_log));
        if (phys < 0 || phys >= p.num_blocks) phys = 0;  // (reported by the first step)
      }
      const uint32_t have = __popc(__ballot_sync(0xffffffffu, phys >= 0));
      for (int i = 0; i < inner && !aborted; ++i, ++k) {
        const int kvh = i / L.row_tiles, rt = i - kvh * L.row_tiles;
        const uint32_t slot = k % S::kStages, qslot = k & 1u;
        wait(&bars[kQFree + qslot], ((k >> 1) & 1u) ^ 1u, aborted);
        wait(&bars[kFree + slot], ((k / S::kStages) & 1u) ^ 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) return;
        if (lane == 0) {
          const uint32_t rows = static_cast<uint32_t>(min(L.tile_queries, p.window) * L.group);
          ptx::mbar_arrive_expect_tx(&bars[kQFull + qslot], rows * 128u * NC);
          ptx::mbar_arrive_expect_tx(&bars[kFull + slot], have * page_rows * 128u * NC);
          for (int c = 0; c < NC; ++c)
            tma_load_3d(smem + S::kOffQ + qslot * S::kQBytes + c * 16384, &tm_q, c * 64, kvh * L.group,
                        seq * p.window + rt * L.tile_queries, &bars[kQFull + qslot], normal);
        }
        __syncwarp();
        if (phys >= 0)
          ptx::tma_load_4d(smem + slot * S::kStageBytes + lane * page_rows * 128 * NC, &tm_k, 0, 0, 0,
                           static_cast<int>(((static_cast<int64_t>(phys) * p.num_kv_heads + kvh) << L.bs_log) / 8) +
                               (tok & ((1 << L.bs_log) - 1)) / 8,
                           &bars[kFull + slot], normal);
        __syncwarp();
      }
    });
    if (aborted) {
      wait_for_loads(&bars[kFull], S::kStages, k);
      wait_for_loads(&bars[kQFull], 2, k);
    }
  } else if (warp == 9) {
    // ============================ products ============================
    const bool leader = elect_one();
    constexpr uint32_t kId = ptx::idesc_bf16_f32(128, 128, 0, 0);
    const uint64_t desc_k = ptx::smem_desc(smem, 16, 1024 * NC, ptx::kLayoutSw128);
    const uint64_t desc_q = ptx::smem_desc(smem + S::kOffQ, 16, 1024, ptx::kLayoutSw128);
    uint32_t k = 0;
    tiles([&](int, int, int) {
      for (int i = 0; i < inner && !aborted; ++i, ++k) {
        const uint32_t slot = k % S::kStages, two = k & 1u, ph = (k >> 1) & 1u;
        wait(&bars[kQFull + two], ph, aborted);
        wait(&bars[kFull + slot], (k / S::kStages) & 1u, aborted);
        wait(&bars[kSFree + two], ph ^ 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) return;
        ptx::tc_fence_after();
        if (leader) {
          const uint64_t dk = desc_k + slot * (S::kStageBytes >> 4), dq = desc_q + two * (S::kQBytes >> 4);
#pragma unroll
          for (int c = 0; c < 4 * NC; ++c)
            ptx::umma_bf16(tmem + two * 128, dk + (c >> 2) * (1024 >> 4) + (c & 3) * 2,
                           dq + (c >> 2) * (16384 >> 4) + (c & 3) * 2, kId, c > 0);
          ptx::umma_commit(&bars[kSFull + two]);
          ptx::umma_commit(&bars[kFree + slot]);
          ptx::umma_commit(&bars[kQFree + two]);
        }
        __syncwarp();
      }
    });
    if (leader) {  // nothing may be in flight when tensor memory is freed
      ptx::umma_commit(&bars[kDrain]);
      bool late = false;
      wait(&bars[kDrain], 0, late);
      if (late) aborted = true;
    }
    aborted = __any_sync(0xffffffffu, aborted);
  } else {
    // ============ sums: one token and half of a row tile per thread ============
    const int half = warp >> 2, r = tid & 127;
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    uint32_t k = 0;
    if (p.test_stall_ns && !ptx::mbar_wait(&bars[kNever], 0, p.test_stall_ns)) aborted = true;  // pa_test_stall_decode
    __syncwarp();
    tiles([&](int seq, int len, int tile) {
      const int tok = tile * 128 + r;
      float s0 = 0.f, s1 = 0.f;
      // rows that are nobody's, or see nothing: 2^(s - inf) = 0
      auto lse_of = [&](int i) {
        const int kvh = i / L.row_tiles, first = (i - kvh * L.row_tiles) * L.tile_queries * L.group;
        const int rows = min(L.tile_queries * L.group, L.rows - first);
        return half == 0 && r < rows ? __ldcg(L.lse + seq * all_rows + static_cast<int64_t>(kvh) * L.rows + first + r)
                                     : CUDART_INF_F;
      };
      float ahead = lse_of(0);
      for (int i = 0; i < inner; ++i, ++k) {  // (a warp that gave up still meets the others at the barrier)
        const int rt = i % L.row_tiles;
        const uint32_t two = k & 1u;
        const int rows = min(L.tile_queries * L.group, L.rows - rt * L.tile_queries * L.group);
        if (half == 0) row_lse[two][r] = ahead;
        ptx::bar_sync(1, 256);
        if (i + 1 < inner) ahead = lse_of(i + 1);
        wait(&bars[kSFull + two], (k >> 1) & 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        ptx::tc_fence_after();
        // queries from which on (by row of the tile) this token is seen: its first such query's first row
        const int q0 = tok - (len - p.window) - rt * L.tile_queries;
        const int from = q0 > 0 ? q0 * L.group : 0;
        const bool all = __all_sync(0xffffffffu, from == 0) && rows == 128;
#pragma unroll 1
        for (int c = half * 64; c < half * 64 + 64; c += 32) {
          uint32_t v[32];
          load_now(at + two * 128 + c, v);
          if (all) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 l = *reinterpret_cast<const float4*>(&row_lse[two][c + j]);
              s0 += fp4::fast_exp2(fmaf(__uint_as_float(v[j]), p.scale_log2, -l.x));
              s1 += fp4::fast_exp2(fmaf(__uint_as_float(v[j + 1]), p.scale_log2, -l.y));
              s0 += fp4::fast_exp2(fmaf(__uint_as_float(v[j + 2]), p.scale_log2, -l.z));
              s1 += fp4::fast_exp2(fmaf(__uint_as_float(v[j + 3]), p.scale_log2, -l.w));
            }
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              s0 += c + j >= from && c + j < rows
                        ? fp4::fast_exp2(fmaf(__uint_as_float(v[j]), p.scale_log2, -row_lse[two][c + j]))
                        : 0.f;
            __syncwarp();  // the next load is the whole warp's
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0 && !aborted) ptx::mbar_arrive(&bars[kSFree + two]);
      }
      if (half) other[r] = s0 + s1;
      ptx::bar_sync(1, 256);
      if (!half && tok < len && !aborted) p.weights[seq * p.weights_stride + tok] += s0 + s1 + other[r];
    });
  }

  if (aborted) *gave_up = 1;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 9) ptx::tmem_dealloc(tmem, 256);
  if (tid == 0 && *gave_up) atomicExch(p.err, kDevErrTimeout);
}

int tokens_of(int head_dim) {
  return head_dim <= 128 ? 128 : head_dim <= 256 ? 64 : 32;
}
constexpr int kStatTokens = 32;  // the least that a row's statistics stand for
int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
// Scores stored or formed again, by a kv head's rows.  Stored they cost 8 bytes a row
// and token, and an exponential; again a product of 128 rows, whatever number of
// them there are, and the keys once more.  4 x 8192 tokens, 8 kv heads of 128 dims,
// stored and again: 48 rows 52 and 54 us, 64 rows 60 and 54, 128 rows 101 and 52 (64
// dims: 48 rows 45 and 50, 64 rows 52 and 50; 64 x 1000 tokens, 64 rows: 101 and 99).
constexpr int kStoredRows = 56;
bool again(int64_t rows, int head_dim) { return head_dim <= 128 && rows > kStoredRows; }
// of one sequence: its rows' logarithms, tiles' statistics and scores
int64_t seq_bytes(int64_t rows, bool stored, int max_context_len) {
  return rows * (4 + up(max_context_len, 128) / kStatTokens * 8 + (stored ? up(max_context_len, 128) * 4 : 0));
}
// sequences of one launch; 0: not even one's units fit an int
int seqs_of(int num_seqs, int64_t rows, int num_kv_heads, int head_dim, int max_context_len) {
  const int64_t units = up(max_context_len, 128) / tokens_of(head_dim) * (rows < num_kv_heads ? num_kv_heads : rows);
  const int64_t fit = units > 0 ? ((int64_t(1) << 31) - 1) / units : kMaxSeqs;
  if (fit == 0) return 0;
  int64_t n = kScoreBytes / (seq_bytes(rows, !again(rows / num_kv_heads, head_dim), max_context_len) + 1);
  if (n < 1) n = 1;
  if (n > fit) n = fit;
  if (n > kMaxSeqs) n = kMaxSeqs;
  return static_cast<int>(n < num_seqs ? n : num_seqs);
}

// one CTA per SM, launched while the kernel before drains
cudaError_t launch_walk(const void* fn, int threads, int smem, const Launch& L, const CUtensorMap& tm_k, const CUtensorMap& tm_q,
                        int64_t most_units, cudaStream_t stream) {
  int per_sm = 0;
  const cudaError_t e = fp4_occupancy(fn, threads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t sms = device_sm_count();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(most_units < 1 ? 1 : (most_units < sms ? most_units : sms)));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<Launch*>(&L), const_cast<CUtensorMap*>(&tm_k), const_cast<CUtensorMap*>(&tm_q)};
  return cudaLaunchKernelExC(&cfg, fn, args);
}
template <int NC>
int smem_of(int num_seqs) {
  return 1024 + Shape<NC>::kOffPrefix + (num_seqs + 64) / 64 * 256;
}

}  // namespace weights_detail

// What a launch needs grows and shrinks with the window and the context: many rows
// store no scores, and fewer long sequences fit one launch.  The size grows with
// each argument, so that a workspace serves every smaller call: at least what any
// launch of as many rows or fewer takes, which is one sequence or kScoreBytes.
size_t weights_workspace(int num_seqs, int window, int num_q_heads, int num_kv_heads, int head_dim, int max_context_len) {
  using namespace weights_detail;
  const int64_t rows = static_cast<int64_t>(window) * num_q_heads;
  if (num_seqs == 0) return 256;
  if (rows >= (int64_t(1) << 31) || seqs_of(num_seqs, rows, num_kv_heads, head_dim, max_context_len) == 0) return 0;
  auto bound = [&](int64_t n, bool stored) {
    const int64_t one = seq_bytes(n, stored, max_context_len), all = one * num_seqs;
    const int64_t most = one > kScoreBytes ? one : kScoreBytes;
    return all < most ? all : most;
  };
  const int64_t store = head_dim <= 128 ? static_cast<int64_t>(kStoredRows) * num_kv_heads : rows;
  int64_t bytes = bound(rows < store ? rows : store, true);
  if (rows > store && bound(rows, false) > bytes) bytes = bound(rows, false);
  return static_cast<size_t>(256 + 3 * 256 + bytes);
}

cudaError_t launch_weights(const WeightsParams& p, cudaStream_t stream) {
  using namespace weights_detail;
  const int64_t rows = static_cast<int64_t>(p.window) * p.num_q_heads;
  const int seqs = seqs_of(p.num_seqs, rows, p.num_kv_heads, p.head_dim, p.max_context_len);
  const int NC = p.head_dim / 64, tokens = tokens_of(p.head_dim), group = p.num_q_heads / p.num_kv_heads;
  Launch L{};
  L.group = group;
  L.rows = p.window * group;
  L.tile_queries = 128 / group;
  L.row_tiles = (p.window + L.tile_queries - 1) / L.tile_queries;
  L.bs_log = __builtin_ctz(static_cast<unsigned>(p.block_size));
  L.pitch = up(p.max_context_len, 128);
  const bool few = L.rows <= 16 && tokens == 128;
  const int stat_tokens = few ? kStatTokens : tokens / halves_of(NC, false);
  L.tiles_pitch = static_cast<int>(L.pitch / stat_tokens);
  unsigned char* at = p.ws + 256;
  const bool twice = again(L.rows, p.head_dim);
  if (!twice) {
    L.scores = reinterpret_cast<float*>(at);
    at += up(static_cast<int64_t>(seqs) * rows * L.pitch * 4, 256);
  }
  L.tile_ml = reinterpret_cast<float2*>(at);
  at += up(static_cast<int64_t>(seqs) * rows * L.tiles_pitch * 8, 256);
  L.lse = reinterpret_cast<float*>(at);
  CUtensorMap tm_k, tm_q;
  // K as groups of 8 rows of NC chunks of 64 dims; queries as (dims, heads, queries)
  const uint64_t row = static_cast<uint64_t>(p.head_dim) * 2;
  const uint64_t kd[4] = {64, 8, static_cast<uint64_t>(NC), static_cast<uint64_t>(p.num_blocks) * p.num_kv_heads * p.block_size / 8};
  const uint64_t ks[3] = {row, 128, 8 * row};
  const uint32_t kb[4] = {64, 8, static_cast<uint32_t>(NC), static_cast<uint32_t>(p.block_size < tokens ? p.block_size : tokens) / 8};
  if (!encode_bf16_tiles(&tm_k, 4, p.k_cache, kd, ks, kb, 128)) return cudaErrorInvalidValue;
  const uint64_t qs[2] = {row, row * p.num_q_heads};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(group), static_cast<uint32_t>(p.window < L.tile_queries ? p.window : L.tile_queries)};
  for (int s0 = 0; s0 < p.num_seqs; s0 += seqs) {
    L.p = p;
    L.p.num_seqs = p.num_seqs - s0 < seqs ? p.num_seqs - s0 : seqs;
    L.p.weights += s0 * p.weights_stride;
    L.p.q = static_cast<const __nv_bfloat16*>(p.q) + static_cast<int64_t>(s0) * rows * p.head_dim;
    L.p.block_tables += static_cast<int64_t>(s0) * p.max_blocks_per_seq;
    L.p.context_lens += s0;
    const uint64_t qd[3] = {static_cast<uint64_t>(p.head_dim), static_cast<uint64_t>(p.num_q_heads),
                            static_cast<uint64_t>(L.p.num_seqs) * p.window};
    if (!encode_bf16_tiles(&tm_q, 3, L.p.q, qd, qs, qb, 128)) return cudaErrorInvalidValue;
    const int64_t tiles = L.pitch / tokens * L.p.num_seqs;
    const void* fn = NC == 1   ? (few ? reinterpret_cast<const void*>(&scores_kernel<1, true>) : reinterpret_cast<const void*>(&scores_kernel<1, false>))
                     : NC == 2 ? (few ? reinterpret_cast<const void*>(&scores_kernel<2, true>) : reinterpret_cast<const void*>(&scores_kernel<2, false>))
                     : NC == 4 ? reinterpret_cast<const void*>(&scores_kernel<4, false>)
                               : reinterpret_cast<const void*>(&scores_kernel<9, false>);
    const int n = L.p.num_seqs;
    const int smem = NC == 1 ? smem_of<1>(n) : NC == 2 ? smem_of<2>(n) : NC == 4 ? smem_of<4>(n) : smem_of<9>(n);
    cudaError_t e = launch_walk(fn, threads_of(NC, few), smem, L, tm_k, tm_q, tiles * p.num_kv_heads * L.row_tiles, stream);
    if (e != cudaSuccess) return e;
    if (p.max_context_len == 0) continue;  // it has reported the lengths; no token has a weight
    const int64_t warps = rows * L.p.num_seqs;
    e = launch_early(lse_kernel, dim3(static_cast<unsigned>((warps + 7) / 8)), 256, stream, L, stat_tokens);
    if (e != cudaSuccess) return e;
    if (twice)
      e = launch_walk(NC == 1 ? reinterpret_cast<const void*>(&again_kernel<1>) : reinterpret_cast<const void*>(&again_kernel<2>),
                      kThreads, smem, L, tm_k, tm_q, tiles, stream);
    else
      e = launch_early(add_kernel, dim3(static_cast<unsigned>(L.pitch / 128), static_cast<unsigned>(L.p.num_seqs)),
                     32 * kAddWarps, stream, L);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pa
