// Causal attention of chunks of queries over the latent cache in its expanded
// form, on the 5th-generation tensor cores: keys of 128 + 64 dims, values of 128.
//
//   S[128 rows x 128 keys] = Q K^T,   P = 2^(S f - m),   O[128 x 128] += P V
// The keys and values of every head are expanded first (latent_expand.cu), so
// that a query and key pair costs 320 multiplications instead of the absorbed
// form's 1088, and a key's 131072 for its two projections are shared by all
// queries.  A row is one token of one head; a CTA takes two tiles of 128 tokens,
// so that every key and value loaded serves 256 rows.  Accumulators are fp32 in
// tensor memory: S of both tiles, O of both.  P is written over its S and read
// from there as the A operand, in bf16 (2^-8, as the output).  fp32 outputs need
// more than that and have a kernel of their own (latent_prefill_f32.cu).
//
// Queries take 96 KB of shared memory; the rest is a ring of eight 16 KB pieces (64
// dims of a step's keys; 64 of its values' tokens), each freed as both tiles have
// used it.
//
// The work is cut into equal runs of steps (128 keys of a tile pair), one for
// each CTA, across the borders of heads, pairs and sequences; an item is a
// (sequence, tile pair, head).  A CTA that takes part of an item's keys leaves its
// rows unnormalised in the workspace with their maximum and sum, and the last CTA
// of the item adds the parts up in the order of the keys.
//
// One CTA per SM, 11 warps, each role walking the same items: 0-3 and 4-7 the
// softmax of the first and the second tile (a row a thread), 8 loads, 9 and 10
// issue the products of the first and the second tile.
//
// A row's reference is raised only when its maximum passes it by 2^8, so that O is
// rarely rescaled.  Measured, 4 x 2048 tokens of 128 heads (687 GFLOP): 630 us, 1090
// TFLOP/s (57% of the products' rate); 2 x 200 to 512 tokens over 8000 to 16000, 32
// heads: 267 us.  A tile's softmax (tensor memory, 128 exponentials a thread, P)
// bounds it: two tiles' products fill half of the time that it takes.  A head's
// pairs follow one another, so that some of its keys come from the second-level
// cache (heads inside pairs: 16 us more).
#include <cuda_bf16.h>
#include <math_constants.h>

#include "decode.cuh"
#include "fp4.cuh"
#include "latent.cuh"
#include "ptx.cuh"
#include "umma.cuh"

namespace pa {
namespace latent_prefill_detail {

using namespace um;

constexpr int kThreads = 11 * 32;
constexpr int kPiece = 16384;
constexpr int kSlots = 8;
constexpr int kOffRing = 6 * kPiece;  // behind the queries: [tile][3 chunks of 64 dims][128 rows x 128 bytes]
constexpr int kOffBar = kOffRing + kSlots * kPiece;
constexpr int kSmemBytes = 1024 + kOffBar + 512;
constexpr float kSlack = 8.f;  // the reference is raised past 2^8

// barriers
enum : int {
  kFull = 0, kFree = kSlots, kQFull = 2 * kSlots, kQFree, kSFull, kPFull = kSFull + 2, kODone = kPFull + 2,
  kOFree = kODone + 2, kDrain = kOFree + 2, kNever, kNumBars
};
static_assert(kNumBars * 8 + 32 <= 512, "barrier area");
constexpr uint32_t kColO = 256;  // tensor memory: S of the tiles at 0 and 128, then O of the tiles

constexpr int kLead = kLatentLead, kPair = kLatentPair;

struct Launch {
  LatentPrefillParams p;
  LatentExpanded x;
};

// A sequence's items, head after head with the pairs inside.
struct Chunk {
  int b, n, q0;
  int64_t row0;  // of its context in the expanded arrays
  __device__ __forceinline__ int pairs() const { return (n + kPair - 1) / kPair; }
  __device__ __forceinline__ int tiles(int j) const { return latent_steps(n, q0, j); }
  __device__ __forceinline__ int64_t before(int j) const { return latent_places_before(q0, j); }
};

__device__ __forceinline__ Chunk chunk_of(const Launch& L, int seq) {
  Chunk c;
  c.b = L.p.cu_q[seq];
  c.n = L.p.cu_q[seq + 1] - c.b;
  c.q0 = L.p.q_start[seq];
  c.row0 = static_cast<int64_t>(L.x.tile0[seq]) * 128;
  return c;
}

// The item at a place: its sequence, pair, head and how far behind its first place
// it lies.  One copy for every kind of warp, its result in registers.
__device__ __noinline__ int4 item_at(const int64_t* place0, const int32_t* cu_q, const int32_t* q_start, int num_seqs,
                                     int heads, int64_t u) {
  int lo = 0, hi = num_seqs - 1;
  while (lo < hi) {  // the last sequence that starts at or before it
    const int mid = (lo + hi + 1) >> 1;
    if (place0[mid] * heads <= u) lo = mid;
    else hi = mid - 1;
  }
  const Chunk c{0, cu_q[lo + 1] - cu_q[lo], q_start[lo], 0};
  const int64_t of_head = place0[lo + 1] - place0[lo];
  int64_t r = u - place0[lo] * heads;
  const int head = static_cast<int>(r / of_head);
  r -= head * of_head;
  int a = 0, b = c.pairs() - 1;
  while (a < b) {
    const int mid = (a + b + 1) >> 1;
    if (c.before(mid) <= r) a = mid;
    else b = mid - 1;
  }
  return make_int4(lo, a, head, static_cast<int>(r - c.before(a)));
}

// An item and this CTA's part of it.
struct Item {
  Chunk c;
  int seq, pair, head;  // the head among this pass's
  int64_t start, end;   // places: kLead, then the steps
  int tok0, pos0, ntok; // first token in the chunk; its position; tokens of the two tiles
  int t0, t1;           // this CTA's steps
  int n0, n1;           // this CTA's steps of each tile
  bool whole;
  __device__ __forceinline__ int kend() const { return pos0 + ntok; }  // keys that the last token sees
  __device__ __forceinline__ int steps_of(int tile) const { return tile ? n1 : n0; }
};

struct Walk {
  const Launch& L;
  int64_t c_begin, c_end;
  __device__ __forceinline__ void derive(Item& it) const {
    const int tiles = it.c.tiles(it.pair);
    it.end = it.start + kLead + tiles;
    it.tok0 = it.pair * kPair;
    it.ntok = min(kPair, it.c.n - it.tok0);
    it.pos0 = it.c.q0 + it.tok0;
    const int64_t first = it.start + kLead;
    it.t0 = static_cast<int>((c_begin > first ? c_begin : first) - first);
    it.t1 = static_cast<int>((c_end < it.end ? c_end : it.end) - first);
    it.whole = it.t0 == 0 && it.t1 == tiles;
    // the first tile's last token may see fewer keys than the second's
    const int seen0 = (it.pos0 + min(128, it.ntok) + 127) / 128;
    it.n0 = max(0, min(it.t1, seen0) - it.t0);
    it.n1 = it.ntok > 128 ? max(0, it.t1 - it.t0) : 0;
  }
  __device__ __forceinline__ void find(Item& it) const;
  __device__ __forceinline__ void next(Item& it) const {
    it.start = it.end;
    if (++it.pair * kPair >= it.c.n) {
      it.pair = 0;
      if (++it.head == L.x.heads) {
        it.head = 0;
        do ++it.seq;
        while (L.x.place0[it.seq + 1] * L.x.heads == it.start);  // sequences without places
        it.c = chunk_of(L, it.seq);
      }
    }
    derive(it);
  }
  // calls f for every item with steps of this CTA's
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    Item it;
    it.end = c_begin;
    for (bool more = c_begin < c_end; more;) {
      if (it.end == c_begin) find(it);
      else next(it);
      more = it.end < c_end;
      if (it.t1 > it.t0) f(it);
    }
  }
};

__device__ __forceinline__ void Walk::find(Item& it) const {
  const int4 x = item_at(L.x.place0, L.p.cu_q, L.p.q_start, L.p.num_seqs, L.x.heads, c_begin);
  it.seq = x.x, it.pair = x.y, it.head = x.z, it.start = c_begin - x.w;
  it.c = chunk_of(L, it.seq);
  derive(it);
}

// A row's probabilities 2^(s f + bias) of a step's 128 keys as 64 bf16 pairs, their
// sum, and the largest s; MASK: keys from nvis on do not count.
template <bool MASK>
__device__ __forceinline__ void probabilities(uint32_t s_at, int nvis, float f, float bias, uint32_t (&pk)[64], float& top,
                                              float& sum) {
  const uint64_t ff = fp4::pair(f, f), bb = fp4::pair(bias, bias);
  uint64_t s0 = 0, s1 = 0;
  float m0 = -CUDART_INF_F, m1 = m0;
#pragma unroll
  for (int c = 0; c < 128; c += 16) {
    uint32_t v[16];
    load_now(s_at + c, v);
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = __uint_as_float(v[j + e]);
        if (MASK && c + j + e >= nvis) x[e] = -CUDART_INF_F;
      }
      m0 = max3(m0, x[0], x[1]);
      m1 = max3(m1, x[2], x[3]);
      const float2 a = fp4::unpair(fp4::fma2(fp4::pair(x[0], x[1]), ff, bb));
      const float2 b = fp4::unpair(fp4::fma2(fp4::pair(x[2], x[3]), ff, bb));
      const float e0 = fp4::fast_exp2(a.x), e1 = fp4::fast_exp2(a.y), e2 = fp4::fast_exp2(b.x), e3 = fp4::fast_exp2(b.y);
      s0 = fp4::add2(s0, fp4::pair(e0, e1));
      s1 = fp4::add2(s1, fp4::pair(e2, e3));
      pk[(c + j) / 2] = pack_bf16(e0, e1);
      pk[(c + j) / 2 + 1] = pack_bf16(e2, e3);
    }
  }
  top = fmaxf(m0, m1);
  const float2 t = fp4::unpair(fp4::add2(s0, s1));
  sum = t.x + t.y;
}
// the largest of a row's first nvis scores of a step
template <bool MASK>
__device__ __forceinline__ float row_max(uint32_t s_at, int nvis) {
  float m0 = -CUDART_INF_F, m1 = m0;
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    uint32_t v[32];
    load_now(s_at + c, v);
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = MASK && c + j + e >= nvis ? -CUDART_INF_F : __uint_as_float(v[j + e]);
      m0 = max3(m0, x[0], x[1]);
      m1 = max3(m1, x[2], x[3]);
    }
  }
  return fmaxf(m0, m1);
}

// 16 outputs of a row, times inv, in a whole 32-byte sector
__device__ __forceinline__ void store_out(const LatentPrefillParams& p, int64_t at, const uint32_t (&v)[16], float inv) {
  uint32_t h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = pack_bf16(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv);
  fp4::store32(static_cast<__nv_bfloat16*>(p.out) + at, h);
}

__global__ void __launch_bounds__(kThreads, 1)
    attend_kernel(const __grid_constant__ Launch L, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_rope, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v) {
  constexpr int kKeys = 3, kValues = 2;  // pieces of a step
  const LatentPrefillParams& p = L.p;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* ring = smem + kOffRing;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  volatile int* gave_up = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* last_flag = gave_up + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(&bars[kFull + i], 1);
      ptx::mbar_init(&bars[kFree + i], 2);
    }
    ptx::mbar_init(&bars[kQFull], 1);
    ptx::mbar_init(&bars[kQFree], 2);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars[kSFull + i], 1);
      ptx::mbar_init(&bars[kPFull + i], 4);
      ptx::mbar_init(&bars[kODone + i], 1);
      ptx::mbar_init(&bars[kOFree + i], 4);
    }
    ptx::mbar_init(&bars[kDrain], 2);
    ptx::mbar_init(&bars[kNever], 1);
    *gave_up = 0;
    ptx::mbar_init_fence();
  }
  if (warp == 9) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool aborted = false;

  const int64_t total = L.x.place0[p.num_seqs] * L.x.heads;
  const int64_t share = total / gridDim.x, extra = total - share * gridDim.x;
  auto cta_begin = [&](int64_t c) { return c * share + (c < extra ? c : extra); };
  const Walk walk{L, cta_begin(blockIdx.x), cta_begin(blockIdx.x + 1)};

  if (warp == 8) {
    // ============================== loads ==============================
    uint32_t ic = 0, uc = 0;  // items, pieces
    const uint64_t first = ptx::policy_evict_first(), normal = ptx::policy_evict_normal();
    auto piece = [&]() -> unsigned char* {  // the next piece's place, once it is free
      const uint32_t slot = uc % kSlots;
      wait(&bars[kFree + slot], ((uc / kSlots) & 1u) ^ 1u, aborted);
      if (aborted) return nullptr;
      ptx::mbar_arrive_expect_tx(&bars[kFull + slot], kPiece);
      return ring + slot * kPiece;
    };
    if (lane == 0)
      walk.each([&](const Item& it) {
        if (aborted) return;
        const int n = max(it.n0, it.n1);
        const int row0 = static_cast<int>(it.c.row0), at0 = static_cast<int>(it.head * L.x.rows + it.c.row0);
        // the queries; rows past the chunk are other rows' or zeros, and nobody's
        wait(&bars[kQFree], (ic & 1u) ^ 1u, aborted);
        if (aborted) return;
        ++ic;
        const int tiles = it.ntok > 128 ? 2 : 1;
        ptx::mbar_arrive_expect_tx(&bars[kQFull], static_cast<uint32_t>(tiles * 3 * kPiece));
        for (int i = 0; i < tiles; ++i)
          for (int c = 0; c < 3; ++c)
            ptx::tma_load_2d(smem + (i * 3 + c) * kPiece, &tm_q, (L.x.head0 + it.head) * 192 + c * 64,
                             it.c.b + it.tok0 + i * 128, &bars[kQFull], first);
        auto keys = [&](int t) {
          for (int k = 0; k < kKeys; ++k, ++uc) {
            unsigned char* dst = piece();
            if (!dst) return;
            uint64_t* bar = &bars[kFull + uc % kSlots];
            if (k == kKeys - 1) ptx::tma_load_2d(dst, &tm_rope, 0, row0 + t * 128, bar, normal);
            else ptx::tma_load_2d(dst, &tm_k, k * 64, at0 + t * 128, bar, normal);
          }
        };
        keys(it.t0);
        for (int t = 0; t < n && !aborted; ++t) {
          for (int k = 0; k < kValues; ++k, ++uc) {
            unsigned char* dst = piece();
            if (!dst) return;
            uint64_t* bar = &bars[kFull + uc % kSlots];
            const int y = at0 + (it.t0 + t) * 128 + k * 64;
            for (int h = 0; h < 2; ++h) ptx::tma_load_2d(dst + h * kPiece / 2, &tm_v, h * 64, y, bar, normal);
          }
          if (t + 1 < n) keys(it.t0 + t + 1);
        }
      });
    if (aborted) {  // (lane 0)
      wait_for_loads(&bars[kFull], kSlots, uc);
      wait_for_loads(&bars[kQFull], 1, ic);
    }
    __syncwarp();
    aborted = __any_sync(0xffffffffu, aborted);
  } else if (warp >= 9) {
    // ============================ products ============================
    // A warp for each tile, so that one's waits pass while the other's products
    // run.  The whole warp runs this and descriptors stay in uniform registers;
    // one elected lane issues.
    const int i = warp - 9;
    const bool leader = elect_one();
    constexpr uint32_t kIdS = ptx::idesc_bf16_f32(128, 128, 0, 0), kIdO = ptx::idesc_bf16_f32(128, 128, 0, 1);
    const uint64_t desc_q = ptx::smem_desc(smem + i * 3 * kPiece, 16, 1024, ptx::kLayoutSw128);
    const uint64_t desc_k = ptx::smem_desc(ring, 16, 1024, ptx::kLayoutSw128);
    const uint64_t desc_v = ptx::smem_desc(ring, kPiece / 2, 1024, ptx::kLayoutSw128);
    const uint32_t s_at = tmem + i * 128, o_at = tmem + kColO + i * 128;
    uint32_t ic = 0, uc = 0, pc = 0, oc = 0;  // items; pieces; steps and items of the tile
    uint32_t turns = 0;
    walk.each([&](const Item& it) {
      const int n = max(it.n0, it.n1), mine = it.steps_of(i);
      for (int t = -1; t < n; ++t) {
        // P V of step t (none before the first), Q K^T of step t + 1
        const bool do_pv = t >= 0 && t < mine, next = t + 1 < n, do_qk = t + 1 < mine;
        uint64_t* bar = nullptr;
        uint32_t parity = 0;
        if (lane == 0 && do_pv) bar = &bars[kPFull + i], parity = pc & 1u;
        if (lane == 1 && t == 0 && do_pv) bar = &bars[kOFree + i], parity = (oc & 1u) ^ 1u;
        if (lane == 2 && t == -1) bar = &bars[kQFull], parity = ic & 1u;
        if (bar) wait(bar, parity, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        // the tiles' turns: whole steps alternate, so that the tiles' softmaxes
        // and products do too (a warp that gave up goes on taking turns).  The
        // ring holds a step's pieces, so that the tile ahead never waits for one
        // that the other has to free first.
        if (i) ptx::bar_sync(1, 64);
        else if (turns++) ptx::bar_sync(2, 64);
        ptx::tc_fence_after();
        if (t >= 0) {
#pragma unroll
          for (int k = 0; k < kValues; ++k, ++uc) {
            const uint32_t slot = uc % kSlots;
            wait(&bars[kFull + slot], (uc / kSlots) & 1u, aborted);
            aborted = __any_sync(0xffffffffu, aborted);
            if (aborted) continue;
            if (leader) {
              if (do_pv) {
                const uint64_t dv = desc_v + slot * (kPiece >> 4);
#pragma unroll
                for (int j = 0; j < 4; ++j)  // 16 keys each
                  umma_ts(o_at, s_at + k * 32 + j * 8, dv + j * (2048 >> 4), kIdO, k + j > 0 || t > 0);
                ptx::umma_commit(&bars[kFree + slot]);
              } else {
                ptx::mbar_arrive(&bars[kFree + slot]);  // a step of the other tile alone
              }
            }
            __syncwarp();
          }
          if (do_pv && !aborted) {
            if (leader) ptx::umma_commit(&bars[kODone + i]);
            ++pc;
            oc += t == 0;
          }
        }
        if (next) {
#pragma unroll
          for (int k = 0; k < kKeys; ++k, ++uc) {
            const uint32_t slot = uc % kSlots;
            wait(&bars[kFull + slot], (uc / kSlots) & 1u, aborted);
            aborted = __any_sync(0xffffffffu, aborted);
            if (aborted) continue;
            if (leader) {
              if (do_qk) {
                const uint64_t dk = desc_k + slot * (kPiece >> 4);
                const uint64_t dq = desc_q + k * (kPiece >> 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) ptx::umma_bf16(s_at, dq + j * 2, dk + j * 2, kIdS, k + j > 0);
                ptx::umma_commit(&bars[kFree + slot]);
              } else {
                ptx::mbar_arrive(&bars[kFree + slot]);
              }
            }
            __syncwarp();
          }
          if (leader && !aborted) {
            if (do_qk) ptx::umma_commit(&bars[kSFull + i]);
            if (t + 2 == n) ptx::umma_commit(&bars[kQFree]);  // the last Q K^T is issued
          }
        }
        __syncwarp();
        asm volatile("bar.arrive %0, 64;" ::"r"(i ? 2 : 1) : "memory");
      }
      ++ic;
    });
    if (i == 0 && turns) ptx::bar_sync(2, 64);
    // nothing may be in flight when tensor memory is freed
    if (leader) {
      ptx::umma_commit(&bars[kDrain]);
      bool late = false;
      wait(&bars[kDrain], 0, late);
      if (late) aborted = true;
    }
    aborted = __any_sync(0xffffffffu, aborted);
  } else {
    // ============ softmax and output: one query row per thread ============
    const int i = warp >> 2;  // tile
    const int r = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_at = tmem + lanes + i * 128, o_at = tmem + lanes + kColO + i * 128;
    const int trow = i * 128 + r;
    uint32_t sc = 0;  // steps of the tile
    const float f = fmaxf(p.scale_log2, 1.2e-38f);  // not zero: a masked -inf times it stays -inf
    if (p.test_stall_ns && !ptx::mbar_wait(&bars[kNever], 0, p.test_stall_ns)) aborted = true;  // pa_test_stall_decode
    aborted = __any_sync(0xffffffffu, aborted);
    walk.each([&](const Item& it) {  // a warp that gave up still meets the others below
      const int64_t row = static_cast<int64_t>(it.c.b + it.tok0 + trow) * p.num_heads + L.x.head0 + it.head;
      const bool valid = trow < it.ntok;
      const int steps = it.steps_of(i);
      // keys that this row sees (one that is nobody's: as the last, so that it needs no mask of its own)
      const int limit = valid ? it.pos0 + trow + 1 : it.kend();
      float m = -CUDART_INF_F, l = 0.f;
      for (int t = 0; t < steps && !aborted; ++t, ++sc) {
        wait(&bars[kSFull + i], sc & 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) break;
        ptx::tc_fence_after();
        const int nvis = limit - (it.t0 + t) * 128;
        const bool all = __all_sync(0xffffffffu, nvis >= 128);
        // a row's new reference, for its sum and for its O once P V of the step before is in it
        auto raise_to = [&](bool raise, float now) {
          const float alpha = raise ? fp4::fast_exp2(m - now) : 1.f;
          if (raise) m = now;
          l *= alpha;
          if (t == 0) return;
          wait(&bars[kODone + i], (sc - 1) & 1u, aborted);
          aborted = __any_sync(0xffffffffu, aborted);
          if (aborted) return;
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            load_now(o_at + c * 32, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
            ptx::tmem_st32(o_at + c * 32, v);
          }
        };
        // The probabilities are formed on the reference as it is; a row whose
        // maximum turns out to pass it by more than 2^8 raises it, and the step
        // is formed again (its scores are still there).  The first step starts
        // from its own maximum.
        if (t == 0) {
          const float mx = (all ? row_max<false>(s_at, nvis) : row_max<true>(s_at, nvis)) * f;
          if (nvis > 0 && mx > -CUDART_INF_F) m = mx;
        }
        uint32_t pk[64];
        float top, sum;
        auto form = [&]() {
          const float bias = m == -CUDART_INF_F ? 0.f : -m;
          if (all) probabilities<false>(s_at, nvis, f, bias, pk, top, sum);
          else probabilities<true>(s_at, nvis, f, bias, pk, top, sum);
        };
        form();
        const bool raise = top * f > m + kSlack;
        if (__any_sync(0xffffffffu, raise)) {
          raise_to(raise, top * f);
          form();
        }
        ptx::tmem_st32(s_at, *reinterpret_cast<uint32_t(*)[32]>(pk));
        ptx::tmem_st32(s_at + 32, *reinterpret_cast<uint32_t(*)[32]>(pk + 32));
        if (aborted) break;
        l += sum;
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars[kPFull + i]);
      }
      // a part's place
      auto part_of = [&](int64_t c) { return (c * 2 + (cta_begin(c) >= it.start ? 0 : 1)) * kPair; };
      float* const ml = L.x.parts;
      float* const po = L.x.parts + static_cast<int64_t>(gridDim.x) * 2 * kPair * 2;
      const int64_t prow = part_of(blockIdx.x) + trow;
      if (steps > 0 && !aborted) {
        wait(&bars[kODone + i], (sc - 1) & 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
      }
      if (steps > 0 && !aborted) {
        ptx::tc_fence_after();
        const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t v[2][16];
          load_now(o_at + c, v[0]);
          load_now(o_at + c + 16, v[1]);
          if (c == 96) {  // O is read: the next item's P V may write it
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars[kOFree + i]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!valid) {
            } else if (it.whole) {
              store_out(p, row * 128 + c + h * 16, v[h], inv);
            } else {
              float4* dst = reinterpret_cast<float4*>(po + prow * 128 + c + h * 16);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                dst[q] = make_float4(__uint_as_float(v[h][4 * q]), __uint_as_float(v[h][4 * q + 1]),
                                     __uint_as_float(v[h][4 * q + 2]), __uint_as_float(v[h][4 * q + 3]));
            }
          }
          __syncwarp();  // the next load is the whole warp's
        }
      }
      if (it.whole) return;
      // the last CTA of the item adds its parts up
      if (valid && !aborted) *reinterpret_cast<float2*>(ml + prow * 2) = make_float2(m, l);
      auto cta_of = [&](int64_t u) {
        const int64_t wide = extra * (share + 1);
        return u < wide ? u / (share + 1) : extra + (u - wide) / share;
      };
      const int64_t c0 = cta_of(it.start + kLead), c1 = cta_of(it.end - 1);
      __threadfence();
      ptx::bar_sync(3, 256);
      if (tid == 0) {
        int32_t* counter = L.x.counters + c0;
        const int before = atomicAdd(counter, 1);
        *last_flag = before == c1 - c0;
        if (before == c1 - c0) *counter = 0;
        __threadfence();
      }
      ptx::bar_sync(3, 256);
      if (*last_flag) {
        // 16 outputs a thread, eight threads a row: a warp reads whole rows
        for (int k = tid; k < it.ntok * 8; k += 256) {
          const int pr = k >> 3, d = (k & 7) * 16;
          float M = -CUDART_INF_F;
#pragma unroll 4
          for (int64_t c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(ml + (part_of(c) + pr) * 2));
          const float ref = M == -CUDART_INF_F ? 0.f : M;
          float acc[16], sum = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[j] = 0.f;
#pragma unroll 2
          for (int64_t c = c0; c <= c1; ++c) {
            const int64_t at = part_of(c) + pr;
            const float2 e = __ldcg(reinterpret_cast<const float2*>(ml + at * 2));
            const float4* src = reinterpret_cast<const float4*>(po + at * 128 + d);
            float4 y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = __ldcg(src + j);
            if (e.y == 0.f) continue;  // a part that this row sees nothing of: its O may be anything
            const float w = fp4::fast_exp2(e.x - ref);
            sum = fmaf(w, e.y, sum);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              acc[4 * j] = fmaf(w, y[j].x, acc[4 * j]);
              acc[4 * j + 1] = fmaf(w, y[j].y, acc[4 * j + 1]);
              acc[4 * j + 2] = fmaf(w, y[j].z, acc[4 * j + 2]);
              acc[4 * j + 3] = fmaf(w, y[j].w, acc[4 * j + 3]);
            }
          }
          const int64_t orow = static_cast<int64_t>(it.c.b + it.tok0 + pr) * p.num_heads + L.x.head0 + it.head;
          store_out(p, orow * 128 + d, reinterpret_cast<uint32_t(&)[16]>(acc), sum != 0.f ? 1.f / sum : 0.f);
        }
      }
      ptx::bar_sync(3, 256);  // the flag is free again
    });
  }

  if (aborted) *gave_up = 1;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 9) ptx::tmem_dealloc(tmem, 512);
  if (tid == 0 && *gave_up && p.status) atomicExch(p.status, kDevErrTimeout);
}

int64_t rows_of(int64_t num_seqs, int64_t total_context) { return (total_context + num_seqs * 127) / 128 * 128; }
int64_t up(int64_t n) { return (n + 1023) / 1024 * 1024; }
int64_t parts_bytes(int64_t ctas) { return ctas * 2 * kPair * (128 + 2) * 4; }

}  // namespace latent_prefill_detail

size_t latent_prefill_workspace(int num_seqs, int num_heads, int head_dim, int64_t total_context) {
  using namespace latent_prefill_detail;
  const int64_t sms = device_sm_count(), rows = rows_of(num_seqs, total_context);
  // tiles and places before the sequences | counters | parts | position parts | keys | values.  Room for an even number
  // of heads: fp32 outputs take half of them at a time.
  const int64_t heads = (static_cast<int64_t>(num_heads) + 1) / 2 * 2;
  if (rows * heads >= (int64_t(1) << 31)) return 0;  // rows are numbered in 32 bits by the tensor loads
  return static_cast<size_t>(1024 + up((static_cast<int64_t>(num_seqs) + 1) * 12 + 8) + up(sms * 4) + up(parts_bytes(sms)) +
                             up(rows * 128) + 2 * up(rows * heads * head_dim * 2));
}

cudaError_t launch_latent_prefill(const LatentPrefillParams& p, cudaStream_t stream) {
  using namespace latent_prefill_detail;
  const int64_t sms = device_sm_count();
  const int all = (p.num_heads + 1) / 2 * 2, pass = p.out_bf16 ? p.num_heads : all / 2;
  LatentExpanded x{};
  x.rows = rows_of(p.num_seqs, p.total_context);
  x.f32 = !p.out_bf16;
  unsigned char* at = reinterpret_cast<unsigned char*>(up(reinterpret_cast<int64_t>(p.ws)));
  auto take = [&](int64_t bytes) {
    unsigned char* r = at;
    at += up(bytes);
    return r;
  };
  x.place0 = reinterpret_cast<int64_t*>(take((static_cast<int64_t>(p.num_seqs) + 1) * 12 + 8));
  x.tile0 = reinterpret_cast<int32_t*>(x.place0 + p.num_seqs + 1);
  x.counters = reinterpret_cast<int32_t*>(take(sms * 4));
  x.parts = reinterpret_cast<float*>(take(parts_bytes(sms)));
  x.rope = take(x.rows * 128);
  x.k = take(x.rows * all * 256);
  x.v = take(x.rows * all * 256);
  x.heads = pass;
  cudaError_t e = launch_latent_plan(p, x, stream);
  if (e != cudaSuccess || x.rows == 0 || p.num_tokens == 0 || p.max_q_len == 0) return e;
  if (x.f32) {
    for (int h = 0; h < p.num_heads; h += pass) {
      x.head0 = h;
      x.heads = p.num_heads - h < pass ? p.num_heads - h : pass;
      if ((e = launch_latent_expand(p, x, stream)) != cudaSuccess) return e;
      if ((e = launch_latent_attend_f32(p, x, stream)) != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  if ((e = launch_latent_expand(p, x, stream)) != cudaSuccess) return e;
  Launch L{};
  L.p = p;
  L.x = x;
  CUtensorMap tq, tr, tk, tv;
  const uint64_t q[2] = {static_cast<uint64_t>(p.num_heads) * 192, static_cast<uint64_t>(p.num_tokens)};
  const uint64_t q_stride[1] = {static_cast<uint64_t>(p.num_heads) * 384};
  const uint64_t r[2] = {64, static_cast<uint64_t>(x.rows)}, r_stride[1] = {128};
  const uint64_t k[2] = {128, static_cast<uint64_t>(x.rows) * x.heads}, k_stride[1] = {256};
  const uint32_t box[2] = {64, 128}, box_v[2] = {64, 64};
  if (!encode_bf16_tiles(&tq, 2, p.q, q, q_stride, box, 128) || !encode_bf16_tiles(&tr, 2, x.rope, r, r_stride, box, 128) ||
      !encode_bf16_tiles(&tk, 2, x.k, k, k_stride, box, 128) || !encode_bf16_tiles(&tv, 2, x.v, k, k_stride, box_v, 128))
    return cudaErrorInvalidValue;
  const void* fn = reinterpret_cast<const void*>(&attend_kernel);
  int per_sm = 0;
  if ((e = fp4_occupancy(fn, kThreads, kSmemBytes, &per_sm)) != cudaSuccess) return e;
  // every SM, while the items are not cut into too many parts to add up
  const int64_t items = (static_cast<int64_t>(p.num_tokens) / kPair + p.num_seqs) * x.heads;
  const int64_t ctas = items * 32 < sms ? items * 32 : sms;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  void* args[] = {&L, &tq, &tr, &tk, &tv};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace pa
