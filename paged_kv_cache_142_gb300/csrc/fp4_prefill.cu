// Causal attention of chunks of queries over the 4-bit K/V pages (the format:
// fp4.cuh) on the 5th-generation tensor cores; head_dim 128.
//
//   S[128 rows x 128 keys]  = Q K^T,   P = 2^(S f - m),   O[128 x 128] += P V
// A row is one query head of one token; a CTA takes two tiles of 128 rows
// (TQ = 128 / G tokens x the G heads of a kv head, each), so every key and
// value that it restores from 4 bits serves 256 rows.  code * scale is exact in
// bf16 and in f16.  Keys become bf16, so that the queries enter as they are, by
// TMA; values become f16, so that the probabilities are rounded to 11 bits
// (2^-12 each, where bf16 would leave 2^-9).  Accumulators are fp32 in tensor
// memory: S of both tiles, O of both.  P is written over its S and read from
// there as the A operand.
//
// The work is cut into equal runs of steps (128 keys of a tile pair), one for
// each CTA, across the borders of heads, tile pairs and sequences; an item is
// a (sequence, tile pair, kv head).  A CTA that takes part of an item's keys
// leaves its rows unnormalised in the workspace with their maximum and sum, and
// the last CTA of the item adds the parts up in the order of the keys.
//
// One CTA per SM, 14 warps, each role walking the same items:
//  * warps 8-11 restore: a thread owns one key of a tile.  It reads the key's
//    64 code bytes and 8 scales through the block table, one tile ahead, and
//    writes the 128 values in the 128-byte-swizzled layout that the tensor core
//    reads; then the same for the value row.  A value group that stands for NaN
//    enters the product as zero, and its key's place is noted: rows that see
//    the key put NaN out, while 0 * NaN must not reach the others.  Warp 8 loads
//    the queries too
//    (turning them to f16 here instead, with a power of two for each row, cost
//    12000 clocks an item: four warps of long dependent chains);
//  * warps 12 and 13 issue the products of the first and the second tile.
//    Q.K^T of a tile's next step is issued right behind P.V of its last one,
//    which read P from the same columns (the tensor core runs a thread's
//    products in order); while one tile's softmax runs the tensor core works
//    for the other;
//  * warps 0-3 and 4-7 run the softmax of the first and the second tile, one
//    row a thread: maximum, exponentials and sum in fp32 (log2 domain).  The
//    reference of a row is raised only when its maximum passes it by 2^8.
// What bounds it is a tile's chain: 128 rows' exponentials (1000 clocks; 512 of
// them the exponential unit's), P.V and Q.K^T (550 each), and 900 of barriers and
// tensor-memory waits, 3150 a step in all; the other tile's products fill its
// gaps, 2250 of the 3150 clocks.  16 prompts of 2048 tokens, 32 q / 8 kv heads:
// 519 us, 1060 TFLOP/s, 55% of the measured bf16 rate; chunks of 200 to 512 tokens
// over 8000 to 16000: 177 us, 1208 TFLOP/s.  What it took: one elected lane of a uniform warp issues
// unrolled products (a rolled loop of one lane: 130 clocks an instruction, 987 us
// instead of 730), one pass over the scores on the reference as it is, a warp for
// each tile's products taking turns (720 to 692 us), equal runs and TMA queries
// (678), items walked instead of searched and whole-sector stores (592), kLead
// of 2 (530), NaN values kept from the rows that do not see them (548), and the
// search for the first item out of line (519).  P.V in two halves, one beside the
// other half's softmax, took 612 us, and one copy of the probabilities' code for
// first and second tries 526.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math_constants.h>

#include <type_traits>

#include "decode.cuh"
#include "fp4.cuh"
#include "ptx.cuh"

namespace pa {
namespace fp4_prefill_detail {

constexpr int kThreads = 14 * 32;
constexpr int kTileBytes = 32768;  // 128 rows x 128 f16
constexpr int kOffQ = 0;           // two tiles: [half of the dims][128 rows][128 bytes]
constexpr int kOffK = 2 * kTileBytes;
constexpr int kOffV = kOffK + 2 * kTileBytes;
constexpr int kOffBar = kOffV + 2 * kTileBytes;
constexpr int kOffNan = kOffBar + 256;            // [8 items][8 groups] the first key whose value is NaN
constexpr int kOffPrefix = kOffNan + 256;         // [sequences + 1] places before a sequence
constexpr int kSmemBytes = kOffPrefix + 1024;     // with slack to align the base, then the places
constexpr float kSlack = 8.f;     // the reference is raised past 2^8
constexpr float kPShift = 6.f;    // probabilities enter P.V times 2^6: below 2^14, none lost before 2^-30

// barriers ([2] each where they have a number)
enum : int {
  kQFull = 0, kQFree = 1, kKFull = 2, kKFree = 4, kVFull = 6, kVFree = 8,
  kSFull = 10, kPFull = 12, kODone = 14, kOFree = 16, kDrain = 18, kNumBars = 19
};
static_assert(kNumBars * 8 + 16 <= 256, "barrier area");
constexpr uint32_t kColO = 256;  // tensor memory: S of the tiles at 0 and 128, then O of the tiles

// What starting and ending an item costs a CTA, in steps: the shares count it,
// as places before the item's first step.
constexpr int kLead = 2;
constexpr int kMaxSeqs = 4096;   // of one launch: their places lie in shared memory
constexpr int kMostParts = 32;   // CTAs for each item on the average, at most (a long one among short ones has more)

struct Launch {
  Fp4AttnParams p;      // of this launch's sequences
  int rows;             // of a part: the most that a tile pair has
  uint32_t tile_bytes;
  int bs_log;
  int32_t* counters;    // [CTAs], zero between launches: of the item that CTA is the first of several to work on
  float* ml;            // [2 * CTAs][rows][2] maximum (log2), sum
  float* o;             // [2 * CTAs][rows][128]
};

// A sequence's items, pair after pair with the kv heads inside.  Pair j has
// kLead + ceil((q0 + tokens up to its end) / 128) places for each head.
template <int G>
struct Chunk {
  static constexpr int S = 256 / G;  // tokens of a pair
  int b, n, q0;
  __device__ __forceinline__ int pairs() const { return (n + S - 1) / S; }
  __device__ __forceinline__ int tiles(int j) const { return (q0 + min(n, (j + 1) * S) + 127) / 128; }
  // places of pairs 0 .. j - 1, all whole, for one head
  __device__ __forceinline__ int before(int j) const {
    if (S > 128) return j * (kLead + (q0 + 127) / 128) + j * (j + 1);  // two more tiles for every pair
    // sum of ceil((a + t) / per) over t = 1 .. j, with q0 rounded up to pairs a
    constexpr int per = S > 128 ? 1 : 128 / S;
    const int a = (q0 + S - 1) / S;
    // (modulo 2^32: the sums may pass it where their difference does not)
    auto f = [](uint32_t x) {
      const uint32_t k = x / per, r = x % per;
      return per * ((k & 1) ? k * ((k + 1) / 2) : k / 2 * (k + 1)) + r * (k + 1);
    };
    return static_cast<int>(static_cast<uint32_t>(j * kLead) + f(a + j) - f(a));
  }
  __device__ __forceinline__ int places() const {  // of one head
    if (n <= 0) return 0;
    const int j = pairs() - 1;
    return before(j) + kLead + tiles(j);
  }
};

template <int G>
__device__ __forceinline__ Chunk<G> chunk_of(const Launch& L, int seq) {
  Chunk<G> c;
  c.b = L.p.cu_q[seq];
  c.n = L.p.cu_q[seq + 1] - c.b;
  c.q0 = L.p.q_start[seq];
  return c;
}

// The item at a place: its sequence, pair, kv head and first place.  One copy
// for the three kinds of warps, once each: inlined in each of them it pushed
// code that runs out of the instruction cache (16 x 2048 prompts 549 us, so 519).
template <int G>
__device__ __noinline__ int4 item_at(const Launch& L, const int* prefix, int u) {
  const int hkv = L.p.num_kv_heads;
  int lo = 0, hi = L.p.num_seqs - 1;
  while (lo < hi) {  // the last sequence that starts at or before it
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  const Chunk<G> c = chunk_of<G>(L, lo);
  int r = u - prefix[lo];
  int a = 0, b = c.pairs() - 1;
  while (a < b) {
    const int mid = (a + b + 1) >> 1;
    if (hkv * c.before(mid) <= r) a = mid;
    else b = mid - 1;
  }
  r -= hkv * c.before(a);
  const int places = kLead + c.tiles(a);
  return make_int4(lo, a, r / places, u - r % places);
}

// An item and this CTA's part of it.
template <int G>
struct Item {
  static constexpr int TQ = 128 / G;
  Chunk<G> c;
  int seq, pair, kvh;
  int start, end;  // places: kLead, then the steps
  // derived: first token in the chunk; position of tok0; tokens of the two tiles
  int tok0, pos0, ntok;
  int t0, t1;      // this CTA's steps
  int n0, n1;      // this CTA's steps of each tile
  bool whole;      // all steps are this CTA's
  __device__ __forceinline__ int kend() const { return pos0 + ntok; }  // keys that the last token sees
  __device__ __forceinline__ int steps_of(int tile) const { return tile ? n1 : n0; }

  __device__ __forceinline__ void derive(int c_begin, int c_end) {
    const int tiles = c.tiles(pair);
    end = start + kLead + tiles;
    tok0 = pair * 2 * TQ;
    ntok = min(2 * TQ, c.n - tok0);
    pos0 = c.q0 + tok0;
    const int first = start + kLead;
    t0 = max(c_begin, first) - first;
    t1 = min(c_end, end) - first;
    whole = t0 == 0 && t1 == tiles;
    // the first tile's last token may see fewer keys than the second's
    const int seen0 = (pos0 + min(TQ, ntok) + 127) / 128;
    n0 = max(0, min(t1, seen0) - t0);
    n1 = ntok > TQ ? max(0, t1 - t0) : 0;
  }
  // the item at place c_begin
  __device__ __forceinline__ void find(const Launch& L, const int* prefix, int c_begin, int c_end) {
    const int4 x = item_at<G>(L, prefix, c_begin);
    seq = x.x, pair = x.y, kvh = x.z, start = x.w;
    c = chunk_of<G>(L, seq);
    derive(c_begin, c_end);
  }
  // the next one (there is one before c_end)
  __device__ __forceinline__ void next(const Launch& L, const int* prefix, int c_begin, int c_end) {
    start = end;
    if (++kvh == L.p.num_kv_heads) {
      kvh = 0;
      if (++pair * 2 * TQ >= c.n) {
        pair = 0;
        do ++seq;
        while (prefix[seq + 1] == start);  // sequences without places
        c = chunk_of<G>(L, seq);
      }
    }
    derive(c_begin, c_end);
  }
};

__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, bool& aborted) {
  if (!aborted && !ptx::mbar_wait(bar, parity, kWaitLimitNs)) aborted = true;
}
// one lane of the warp, the same each time
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
  return yes != 0;
}
using fp4::fast_exp2;
using fp4::pack_f16;
// kind::f16, f16 operands, fp32 accumulator, M = N = 128; b_mn: B is N-major
__host__ __device__ constexpr uint32_t idesc_f16(int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (16u << 17) | (8u << 24);
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// waits for this warp's tensor-memory loads; what uses v comes after it
__device__ __forceinline__ void wait_ld16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// A row's probabilities 2^(s f + bias) of a step's 128 keys as 64 f16 pairs,
// their sum, and the largest s; MASK: keys from nvis on do not count.  The
// next 16 scores load while 16 are worked on.
template <bool MASK>
__device__ __forceinline__ void probabilities(uint32_t s_at, int nvis, float f, float bias, uint32_t (&pk)[64],
                                              float& top, float& sum) {
  const uint64_t ff = fp4::pair(f, f), bb = fp4::pair(bias, bias);
  uint64_t s0 = 0, s1 = 0;
  float m0 = -CUDART_INF_F, m1 = m0;
  uint32_t v[2][16];
  ptx::TmemLd<16>::run(s_at, v[0]);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    wait_ld16(v[c & 1]);
    if (c < 7) ptx::TmemLd<16>::run(s_at + (c + 1) * 16, v[(c + 1) & 1]);
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = __uint_as_float(v[c & 1][j + e]);
        if (MASK && c * 16 + j + e >= nvis) x[e] = -CUDART_INF_F;
      }
      m0 = max3(m0, x[0], x[1]);
      m1 = max3(m1, x[2], x[3]);
      const float2 a = fp4::unpair(fp4::fma2(fp4::pair(x[0], x[1]), ff, bb)), b = fp4::unpair(fp4::fma2(fp4::pair(x[2], x[3]), ff, bb));
      const float e0 = fast_exp2(a.x), e1 = fast_exp2(a.y), e2 = fast_exp2(b.x), e3 = fast_exp2(b.y);
      s0 = fp4::add2(s0, fp4::pair(e0, e1));
      s1 = fp4::add2(s1, fp4::pair(e2, e3));
      pk[(c * 16 + j) / 2] = pack_f16(e0, e1);
      pk[(c * 16 + j) / 2 + 1] = pack_f16(e2, e3);
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
  for (int c = 0; c < 128; c += 64) {
    uint32_t v[4][16];
#pragma unroll
    for (int h = 0; h < 4; ++h) ptx::TmemLd<16>::run(s_at + c + h * 16, v[h]);
#pragma unroll
    for (int h = 0; h < 4; ++h) wait_ld16(v[h]);
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[e] = MASK && c + h * 16 + j + e >= nvis ? -CUDART_INF_F : __uint_as_float(v[h][j + e]);
        m0 = max3(m0, x[0], x[1]);
        m1 = max3(m1, x[2], x[3]);
      }
  }
  return fmaxf(m0, m1);
}

// A key's or value's row: 64 code bytes and 8 scales.
struct Row {
  uint4 c[4];
  uint2 s;
};

using fp4::store32;
// 16 outputs of a row, times inv, in whole 32-byte sectors
__device__ __forceinline__ void store_out(const Fp4AttnParams& p, int64_t at, const uint32_t (&v)[16], float inv) {
  uint32_t h[8];
  if (p.out_bf16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const __nv_bfloat162 x =
          __floats2bfloat162_rn(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv);
      h[e] = *reinterpret_cast<const uint32_t*>(&x);
    }
    store32(static_cast<__nv_bfloat16*>(p.out) + at, h);
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = __float_as_uint(__uint_as_float(v[8 * q + e]) * inv);
      store32(static_cast<float*>(p.out) + at + 8 * q, h);
    }
  }
}
}  // namespace fp4_prefill_detail

template <int G>
__global__ void __launch_bounds__(fp4_prefill_detail::kThreads, 1)
    fp4_prefill_kernel(const __grid_constant__ fp4_prefill_detail::Launch L, const __grid_constant__ CUtensorMap tm_q) {
  using namespace fp4_prefill_detail;
  constexpr int TQ = 128 / G;
  const Fp4AttnParams& p = L.p;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  volatile int* gave_up = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* prefix = reinterpret_cast<int*>(smem + kOffPrefix);
  int* first_nan = reinterpret_cast<int*>(smem + kOffNan);
  __shared__ int warp_sums[kThreads / 32];
  __shared__ int last_flag;

  ptx::griddep_launch_dependents();
  if (tid == 0) {
    ptx::mbar_init(&bars[kQFull], 1);
    ptx::mbar_init(&bars[kQFree], 2);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars[kKFull + i], 4);
      ptx::mbar_init(&bars[kKFree + i], 2);
      ptx::mbar_init(&bars[kVFull + i], 4);
      ptx::mbar_init(&bars[kVFree + i], 2);
      ptx::mbar_init(&bars[kSFull + i], 1);
      ptx::mbar_init(&bars[kPFull + i], 4);
      ptx::mbar_init(&bars[kODone + i], 1);
      ptx::mbar_init(&bars[kOFree + i], 4);
    }
    ptx::mbar_init(&bars[kDrain], 2);
    *gave_up = 0;
    ptx::mbar_init_fence();
  }
  if (tid < 64) first_nan[tid] = 0x7fffffff;
  if (warp == 12) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool aborted = false;
  ptx::griddep_wait();

  // ---- places before every sequence; a chunk that is refused has none ----
  {
    const int per = (p.num_seqs + kThreads - 1) / kThreads;
    const int beg = min(p.num_seqs, tid * per), end = min(p.num_seqs, beg + per);
    const int64_t table_tokens = static_cast<int64_t>(p.max_blocks_per_seq) << L.bs_log;
    int local = 0;
    for (int s = beg; s < end; ++s) {
      const Chunk<G> c = chunk_of<G>(L, s);
      const int64_t last = static_cast<int64_t>(c.q0) + c.n;
      int places = 0;
      if (c.n > 0 && c.b >= 0 && static_cast<int64_t>(c.b) + c.n <= p.num_tokens && c.q0 >= 0 && c.n <= p.max_q_len &&
          last <= table_tokens && last <= p.max_context_len)
        places = c.places() * p.num_kv_heads;
      else if (c.n != 0 && blockIdx.x == 0 && p.err)
        atomicExch(p.err, kDevErrInvalidArg);
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
  }
  const int total = prefix[p.num_seqs];
  const int share = total / gridDim.x, extra = total - share * gridDim.x;
  auto cta_begin = [&](int c) { return c * share + min(c, extra); };
  const int c_begin = cta_begin(blockIdx.x), c_end = cta_begin(blockIdx.x + 1);

  if (warp >= 8 && warp < 12) {
    // ======================= restoring, queries =======================
    const int r = tid - 256;  // this thread's key of a tile, and query row of both
    const int bs = 1 << L.bs_log;
    const uint32_t sw = r & 7;
    uint32_t ic = 0, kc = 0;
    auto locate = [&](const Item<G>& it, const int32_t* table, int t) -> int64_t {
      const int key = t * 128 + r;
      if (key >= it.kend()) return -1;
      const int lb = key >> L.bs_log;
      int phys = __ldg(table + lb);
      if (phys < 0 || phys >= p.num_blocks) {  // never read outside the pool
        if (p.err) atomicExch(p.err, kDevErrInvalidArg);
        phys = 0;
      }
      return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(phys) * p.num_kv_heads + it.kvh) *
                                  L.tile_bytes);
    };
    // NaN scales of a value row out of it, and noted
    auto take_nan = [&](Row& x, int key, int* noted) {
      uint32_t w[2] = {x.s.x, x.s.y};
      if ((((w[0] & 0x7f7f7f7fu) + 0x01010101u) | ((w[1] & 0x7f7f7f7fu) + 0x01010101u)) & 0x80808080u) {
        for (int g = 0; g < 8; ++g)
          if (((w[g >> 2] >> (8 * (g & 3))) & 0x7fu) == 0x7fu) {
            atomicMin(&noted[g], key);
            w[g >> 2] &= ~(0xffu << (8 * (g & 3)));
          }
        x.s = make_uint2(w[0], w[1]);
      }
    };
    auto load = [&](Row& x, const uint8_t* cache, int64_t at, int t) {
      if (at < 0) {  // past the last key: zeros
#pragma unroll
        for (int i = 0; i < 4; ++i) x.c[i] = make_uint4(0, 0, 0, 0);
        x.s = make_uint2(0, 0);
        return;
      }
      const int off = (t * 128 + r) & (bs - 1);
      const uint4* c = reinterpret_cast<const uint4*>(cache + at + off * 64);
#pragma unroll
      for (int i = 0; i < 4; ++i) x.c[i] = __ldg(c + i);
      x.s = __ldg(reinterpret_cast<const uint2*>(cache + at + bs * 64 + off * 8));
    };
    // a row restored, K to bf16 and V to f16, in 16-byte chunks of 8 dims
    auto store = [&](unsigned char* tile, const Row& x, auto bf16) {
      unsigned char* row = tile + (r >> 3) * 2048 + sw * 128;
      const uint32_t w[16] = {x.c[0].x, x.c[0].y, x.c[0].z, x.c[0].w, x.c[1].x, x.c[1].y, x.c[1].z, x.c[1].w,
                              x.c[2].x, x.c[2].y, x.c[2].z, x.c[2].w, x.c[3].x, x.c[3].y, x.c[3].z, x.c[3].w};
#pragma unroll
      for (int g = 0; g < 8; ++g) {  // scale groups: 16 dims
        const uint32_t two = fp4::scales_to_f16((g < 4 ? x.s.x : x.s.y) >> (16 * ((g >> 1) & 1)));
        const uint32_t sc = (g & 1) ? __byte_perm(two, 0, 0x3232) : __byte_perm(two, 0, 0x1010);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t h[4];
          fp4::codes_to_f16(w[2 * g + e], h);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            h[k] = fp4::mul_f16x2(h[k], sc);
            if (decltype(bf16)::value) {  // exact: 6 significant bits, so the fp32 value's low half is zero
              const float2 f = fp4::f16x2_to_f32(h[k]);
              h[k] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
            }
          }
          const int chunk = 2 * g + e;
          *reinterpret_cast<uint4*>(row + (chunk >> 3) * 1024 + (((chunk & 7) ^ sw) << 4)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
    };
    if (warp == 8 && lane == 0) ptx::prefetch_tensormap(&tm_q);
    Item<G> it;
    it.end = c_begin;
    for (bool more = c_begin < c_end; more && !aborted;) {
      if (it.end == c_begin) it.find(L, prefix, c_begin, c_end);
      else it.next(L, prefix, c_begin, c_end);
      more = it.end < c_end;
      if (it.t1 <= it.t0) continue;  // its first step is the next CTA's
      const int n = max(it.n0, it.n1);
      const int32_t* table = p.block_tables + static_cast<int64_t>(it.seq) * p.max_blocks_per_seq;
      Row kx, vx;
      int64_t at = -1;
      if (n > 0) {
        at = locate(it, table, it.t0);
        load(kx, p.k_cache, at, it.t0);
        load(vx, p.v_cache, at, it.t0);
      }
      // the queries of the item, a box for every head and half of the dims;
      // rows past the chunk are other rows' or zeros, and nobody's
      if (warp == 8 && lane == 0) {
        wait(&bars[kQFree], (ic & 1u) ^ 1u, aborted);
        if (!aborted) {
          const int tiles = it.ntok > TQ ? 2 : 1;
          ptx::mbar_arrive_expect_tx(&bars[kQFull], static_cast<uint32_t>(tiles * kTileBytes));
          for (int i = 0; i < tiles; ++i)
            for (int g = 0; g < G; ++g)
              for (int h = 0; h < 2; ++h)
                ptx::tma_load_2d(smem + kOffQ + i * kTileBytes + h * 16384 + g * TQ * 128, &tm_q,
                                 (it.kvh * G + g) * 128 + h * 64, it.c.b + it.tok0 + i * TQ, &bars[kQFull],
                                 ptx::policy_evict_first());
        }
      }
      aborted = __any_sync(0xffffffffu, aborted);
      const uint32_t item_no = ic++;
      // Three items ahead the notes start afresh, in the place of those of five
      // items ago.  A warp gets no further than two steps, so two items, ahead of
      // another: nobody writes them yet.  And both tiles have read the old ones:
      // the last value stored waited until both product warps had released the
      // one of two steps before, of item J >= item_no - 3, and a product warp
      // begins J only when its tile's outputs of the items before J, notes
      // included, are read (kOFree, whether the tile has steps in J or not).
      if (tid >= 256 && tid < 264) first_nan[((item_no + 3) & 7u) * 8 + tid - 256] = 0x7fffffff;
      for (int t = 0; t < n && !aborted; ++t, ++kc) {
        const int slot = kc & 1u;
        const uint32_t ph = (kc >> 1) & 1u;
        const bool next = t + 1 < n;
        if (next) at = locate(it, table, it.t0 + t + 1);
        wait(&bars[kKFree + slot], ph ^ 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) break;
        store(smem + kOffK + slot * kTileBytes, kx, std::true_type{});
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars[kKFull + slot]);
        if (next) load(kx, p.k_cache, at, it.t0 + t + 1);
        wait(&bars[kVFree + slot], ph ^ 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) break;
        take_nan(vx, (it.t0 + t) * 128 + r, first_nan + (item_no & 7u) * 8);
        store(smem + kOffV + slot * kTileBytes, vx, std::false_type{});
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars[kVFull + slot]);
        if (next) load(vx, p.v_cache, at, it.t0 + t + 1);
      }
    }
  } else if (warp >= 12) {
    // ============================ products ============================
    // A warp for each tile, so that one's waits pass while the other's products
    // run.  The whole warp runs this and descriptors stay in uniform registers;
    // one elected lane issues.  The eight instructions of a product are
    // unrolled: a rolled loop of one lane took 130 clocks each.
    const int i = warp - 12;
    const bool leader = elect_one();
    constexpr uint32_t kIdQK = ptx::idesc_bf16_f32(128, 128, 0, 0), kIdPV = idesc_f16(1);
    const uint64_t desc_q = ptx::smem_desc(smem + kOffQ + i * kTileBytes, 16, 1024, ptx::kLayoutSw128);
    const uint64_t desc_k = ptx::smem_desc(smem + kOffK, 16, 2048, ptx::kLayoutSw128);
    const uint64_t desc_v = ptx::smem_desc(smem + kOffV, 1024, 2048, ptx::kLayoutSw128);
    const uint32_t s_at = tmem + i * 128, o_at = tmem + kColO + i * 128;
    uint32_t ic = 0, kc = 0, pc = 0, oc = 0;  // items; steps of keys; steps and items of the tile
    auto qk = [&](uint32_t slot) {
      const uint64_t dk = desc_k + slot * (kTileBytes >> 4);
      if (leader) {
#pragma unroll
        for (int k = 0; k < 8; ++k)  // halves of 64 dims, 16 dims (32 bytes) each
          ptx::umma_bf16(s_at, desc_q + (k >> 2) * (16384 >> 4) + (k & 3) * 2,
                         dk + (k >> 2) * (1024 >> 4) + (k & 3) * 2, kIdQK, k > 0);
        ptx::umma_commit(&bars[kSFull + i]);
        ptx::umma_commit(&bars[kKFree + slot]);
      }
    };
    auto pv = [&](uint32_t slot, bool first) {
      const uint64_t dv = desc_v + slot * (kTileBytes >> 4);
      if (leader) {
#pragma unroll
        for (int k = 0; k < 8; ++k)  // 16 keys (4096 bytes) each
          umma_ts(o_at, s_at + k * 8, dv + k * (4096 >> 4), kIdPV, k > 0 ? 1u : !first);
        ptx::umma_commit(&bars[kODone + i]);
        ptx::umma_commit(&bars[kVFree + slot]);
      }
    };
    uint32_t turns = 0;
    Item<G> it;
    it.end = c_begin;
    for (bool more = c_begin < c_end; more;) {
      if (it.end == c_begin) it.find(L, prefix, c_begin, c_end);
      else it.next(L, prefix, c_begin, c_end);
      more = it.end < c_end;
      if (it.t1 <= it.t0) continue;
      const int n = max(it.n0, it.n1), mine = it.steps_of(i);
      for (int t = -1; t < n; ++t) {
        // P.V of step t (none before the first), Q.K^T of step t + 1; a lane
        // polls each of the barriers that this needs
        const uint32_t vslot = (kc + t) & 1u, kslot = (kc + t + 1) & 1u;
        const bool do_pv = t >= 0 && t < mine, next = t + 1 < n, do_qk = t + 1 < mine;
        uint64_t* bar = nullptr;
        uint32_t parity = 0;
        if (lane == 0 && do_pv) bar = &bars[kPFull + i], parity = pc & 1u;
        if (lane == 1 && t >= 0) bar = &bars[kVFull + vslot], parity = ((kc + t) >> 1) & 1u;
        if (lane == 2 && next) bar = &bars[kKFull + kslot], parity = ((kc + t + 1) >> 1) & 1u;
        if (lane == 3 && t == 0) bar = &bars[kOFree + i], parity = (oc & 1u) ^ 1u;  // also where P.V is none: see the notes
        if (lane == 4 && t == -1) bar = &bars[kQFull], parity = ic & 1u;
        if (bar) wait(bar, parity, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        // the tiles' turns: whole steps alternate, so that the tiles' softmaxes
        // and products do too (a warp that gave up goes on taking turns)
        if (i) ptx::bar_sync(1, 64);
        else if (turns++) ptx::bar_sync(2, 64);
        ptx::tc_fence_after();
        if (aborted) {
        } else if (do_pv) {
          pv(vslot, t == 0);
          ++pc;
          oc += t == 0;
        } else if (t >= 0 && leader) {
          ptx::mbar_arrive(&bars[kVFree + vslot]);  // a step of the other tile alone
        }
        if (aborted) {
        } else if (do_qk) {
          qk(kslot);
        } else if (next && leader) {
          ptx::mbar_arrive(&bars[kKFree + kslot]);
        }
        if (!aborted && leader && next && t + 2 == n) ptx::umma_commit(&bars[kQFree]);  // the last Q.K^T is issued
        __syncwarp();
        asm volatile("bar.arrive %0, 64;" ::"r"(i ? 2 : 1) : "memory");
      }
      kc += n;
      ++ic;
    }
    if (i == 0 && turns) ptx::bar_sync(2, 64);
    // nothing may be in flight when tensor memory is freed
    if (leader) {
      ptx::umma_commit(&bars[kDrain]);
      bool drain = false;
      wait(&bars[kDrain], 0, drain);
      if (aborted || drain) *gave_up = 1;
    }
    __syncwarp();
  } else {
    // ============ softmax and output: one query row per thread ============
    const int i = warp >> 2;  // tile
    const int quarter = warp & 3;
    const int r = 32 * quarter + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t s_at = tmem + lanes + i * 128, o_at = tmem + lanes + kColO + i * 128;
    const int g = r / TQ, trow = i * TQ + r % TQ;
    uint32_t sc = 0, ic = 0;  // steps of the tile, items
    const float f = fmaxf(p.scale_log2, 1.2e-38f);  // not zero: a masked -inf times it stays -inf
    Item<G> it;
    it.end = c_begin;
    for (bool more = c_begin < c_end; more;) {  // a warp that gave up still meets the others below
      if (it.end == c_begin) it.find(L, prefix, c_begin, c_end);
      else it.next(L, prefix, c_begin, c_end);
      more = it.end < c_end;
      if (it.t1 <= it.t0) continue;  // its first step is the next CTA's
      const int64_t row = static_cast<int64_t>(it.c.b + it.tok0 + trow) * p.num_q_heads + it.kvh * G + g;
      const bool valid = trow < it.ntok;
      const int steps = it.steps_of(i);
      const uint32_t item_no = ic++;
      // keys that this row sees (one that is nobody's: as the last, so that it needs no mask of its own)
      const int limit = valid ? it.pos0 + trow + 1 : it.kend();
      float m = -CUDART_INF_F, l = 0.f;
      for (int t = 0; t < steps && !aborted; ++t, ++sc) {
        wait(&bars[kSFull + i], sc & 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
        if (aborted) break;
        ptx::tc_fence_after();
        const int nvis = limit - (it.t0 + t) * 128;
        // The probabilities are formed on the reference as it is; a row whose
        // maximum turns out to pass it by more than 2^8 raises it, and the step
        // is formed again (its scores are still there).  The first step starts
        // from its own maximum.
        if (t == 0) {
          const float mx =
              (__all_sync(0xffffffffu, nvis >= 128) ? row_max<false>(s_at, nvis) : row_max<true>(s_at, nvis)) * f;
          if (nvis > 0 && mx > -CUDART_INF_F) m = mx;
        }
        uint32_t pk[64];
        float top, sum;
        auto form = [&]() {
          const float bias = m == -CUDART_INF_F ? 0.f : kPShift - m;
          if (__all_sync(0xffffffffu, nvis >= 128)) probabilities<false>(s_at, nvis, f, bias, pk, top, sum);
          else probabilities<true>(s_at, nvis, f, bias, pk, top, sum);
        };
        form();
        const bool raise = top * f > m + kSlack;
        if (__any_sync(0xffffffffu, raise)) {
          const float alpha = raise ? fast_exp2(m - top * f) : 1.f;
          if (raise) m = top * f;
          l *= alpha;
          if (t > 0) {  // O, once P.V of the step before is in it
            wait(&bars[kODone + i], (sc - 1) & 1u, aborted);
            aborted = __any_sync(0xffffffffu, aborted);
            if (aborted) break;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t v[32];
              ptx::TmemLd<32>::run(o_at + c * 32, v);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
              ptx::tmem_st32(o_at + c * 32, v);
            }
          }
          form();
        }
        l += sum;
        ptx::tmem_st32(s_at, *reinterpret_cast<uint32_t(*)[32]>(pk));
        ptx::tmem_st32(s_at + 32, *reinterpret_cast<uint32_t(*)[32]>(pk + 32));
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars[kPFull + i]);
      }
      // a part's place; its row: token of the pair, then head
      auto part_of = [&](int c) { return static_cast<int64_t>(c * 2 + (cta_begin(c) >= it.start ? 0 : 1)) * L.rows; };
      const int64_t prow = part_of(blockIdx.x) + trow * G + g;
      if (steps > 0 && !aborted) {
        wait(&bars[kODone + i], (sc - 1) & 1u, aborted);
        aborted = __any_sync(0xffffffffu, aborted);
      }
      if (steps > 0 && !aborted) {
        ptx::tc_fence_after();
        const float inv = l != 0.f ? p.v_scale / l : 0.f;
        // the first key with a NaN in this lane's group (read before O is handed on, which frees the notes)
        const int nan_key = first_nan[(item_no & 7u) * 8 + (lane & 7)];
#pragma unroll 1
        for (int c = 0; c < 128; c += 64) {
          uint32_t v[4][16];
#pragma unroll
          for (int h = 0; h < 4; ++h) ptx::TmemLd<16>::run(o_at + c + h * 16, v[h]);
#pragma unroll
          for (int h = 0; h < 4; ++h) wait_ld16(v[h]);
          if (c == 64) {  // O is read: the next item's P.V may write it
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&bars[kOFree + i]);
          }
          if (!valid) continue;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            if (it.whole) {
              store_out(p, row * 128 + c + h * 16, v[h], inv);
            } else {
              float4* dst = reinterpret_cast<float4*>(L.o + prow * 128 + c + h * 16);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                dst[q] = make_float4(__uint_as_float(v[h][4 * q]), __uint_as_float(v[h][4 * q + 1]),
                                     __uint_as_float(v[h][4 * q + 2]), __uint_as_float(v[h][4 * q + 3]));
            }
          }
        }
        if (__any_sync(0xffffffffu, nan_key != 0x7fffffff)) {  // groups of which the row sees a NaN, over what was stored
#pragma unroll 1
          for (int k = 0; k < 8; ++k) {
            if (__shfl_sync(0xffffffffu, nan_key, k) >= limit || !valid) continue;
            if (it.whole) {
              uint32_t v[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = 0x7fffffffu;
              store_out(p, row * 128 + k * 16, v, 1.f);
            } else {
              for (int j = 0; j < 16; ++j) L.o[prow * 128 + k * 16 + j] = __uint_as_float(0x7fffffffu);
            }
          }
        }
      }
      if (!it.whole) {
        // the last CTA of the item adds its parts up
        if (valid && !aborted) *reinterpret_cast<float2*>(L.ml + prow * 2) = make_float2(m, l);
        auto cta_of = [&](int u) {
          const int wide = extra * (share + 1);
          return u < wide ? u / (share + 1) : extra + (u - wide) / share;
        };
        const int c0 = cta_of(it.start + kLead), c1 = cta_of(it.end - 1);
        __threadfence();
        ptx::bar_sync(3, 256);
        if (tid == 0) {
          int32_t* counter = L.counters + c0;
          const int before = atomicAdd(counter, 1);
          last_flag = before == c1 - c0;
          if (before == c1 - c0) *counter = 0;
          __threadfence();
        }
        ptx::bar_sync(3, 256);
        if (last_flag) {
          // 16 outputs a thread, eight threads a row: a warp reads whole rows
          for (int k = tid; k < it.ntok * G * 8; k += 256) {
            const int pr = k >> 3, d = (k & 7) * 16;  // token of the pair * G + head
            float M = -CUDART_INF_F;
#pragma unroll 4
            for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(L.ml + (part_of(c) + pr) * 2));
            const float ref = M == -CUDART_INF_F ? 0.f : M;
            float acc[16], sum = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[j] = 0.f;
#pragma unroll 2
            for (int c = c0; c <= c1; ++c) {
              const int64_t at = part_of(c) + pr;
              const float2 e = __ldcg(reinterpret_cast<const float2*>(L.ml + at * 2));
              const float4* src = reinterpret_cast<const float4*>(L.o + at * 128 + d);
              float4 x[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = __ldcg(src + j);
              if (e.y == 0.f) continue;  // a part that this row sees nothing of: its O may be anything
              const float w = fast_exp2(e.x - ref);
              sum = fmaf(w, e.y, sum);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                acc[4 * j] = fmaf(w, x[j].x, acc[4 * j]);
                acc[4 * j + 1] = fmaf(w, x[j].y, acc[4 * j + 1]);
                acc[4 * j + 2] = fmaf(w, x[j].z, acc[4 * j + 2]);
                acc[4 * j + 3] = fmaf(w, x[j].w, acc[4 * j + 3]);
              }
            }
            const int64_t orow = static_cast<int64_t>(it.c.b + it.tok0 + pr / G) * p.num_q_heads + it.kvh * G + pr % G;
            store_out(p, orow * 128 + d, reinterpret_cast<uint32_t(&)[16]>(acc), sum != 0.f ? p.v_scale / sum : 0.f);
          }
        }
        ptx::bar_sync(3, 256);  // the flag is free again
      }
    }
  }

  if (aborted) *gave_up = 1;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 12) ptx::tmem_dealloc(tmem, 512);
  if (tid == 0 && *gave_up && p.err) atomicExch(p.err, kDevErrTimeout);
}

}  // namespace pa

extern "C" bool encode_q_tokens(CUtensorMap* m, const void* base, uint64_t tokens, uint64_t row_elems, uint32_t box_rows);

namespace pa {
namespace {

const void* kernel_for(int group) {
  switch (group) {
    case 1: return reinterpret_cast<const void*>(&fp4_prefill_kernel<1>);
    case 2: return reinterpret_cast<const void*>(&fp4_prefill_kernel<2>);
    case 4: return reinterpret_cast<const void*>(&fp4_prefill_kernel<4>);
    case 8: return reinterpret_cast<const void*>(&fp4_prefill_kernel<8>);
    default: return reinterpret_cast<const void*>(&fp4_prefill_kernel<16>);
  }
}

// A chunk is no longer than the context that it ends in, however loose the
// caller's bound (and one token at least, so that a launch has a CTA to report
// what it refuses).
int longest_of(int max_q_len, int max_context_len) {
  const int n = max_q_len < max_context_len ? max_q_len : max_context_len;
  return n > 1 ? n : 1;
}
// Of chunks of up to n tokens: a chunk's tile pairs, and the rows of a pair (a
// pair has 256 / group tokens).  Neither forms a product that could pass 32 bits.
int64_t pairs_of(int group, int n) { return (static_cast<int64_t>(n) + 256 / group - 1) / (256 / group); }
int rows_of(int group, int n) { return n < 256 / group ? n * group : 256; }

// Sequences of one launch: their places fit an int.  0: not even one's do.
int seqs_of(int num_seqs, int num_kv_heads, int group, int longest, int max_context_len) {
  using namespace fp4_prefill_detail;
  constexpr int64_t kMost = (int64_t(1) << 31) - 1;
  // of one head: below 2^50, as a context has at most 2^30 tokens
  const int64_t places = (kLead + (static_cast<int64_t>(max_context_len) + 127) / 128) * pairs_of(group, longest);
  const int64_t fit = kMost / places / num_kv_heads;
  const int64_t most = fit < kMaxSeqs ? fit : kMaxSeqs;
  return static_cast<int>(num_seqs < most ? num_seqs : most);
}

}  // namespace

size_t fp4_prefill_workspace(int num_seqs, int num_q_heads, int num_kv_heads, int max_q_len, int max_context_len) {
  const int G = num_q_heads / num_kv_heads;
  const int longest = longest_of(max_q_len, max_context_len);
  if (num_seqs > 0 && max_q_len > 0 && seqs_of(num_seqs, num_kv_heads, G, longest, max_context_len) == 0) return 0;
  // header | counters | parts: the first two lie where they lie for every shape
  return static_cast<size_t>(256 + fp4_counter_bytes() + 2 * device_sm_count() * rows_of(G, longest) * (128 + 2) * 4);
}

cudaError_t launch_fp4_prefill(const Fp4AttnParams& p, cudaStream_t stream) {
  using namespace fp4_prefill_detail;
  const int G = p.num_q_heads / p.num_kv_heads;
  const int longest = longest_of(p.max_q_len, p.max_context_len);
  const int seqs = seqs_of(p.num_seqs, p.num_kv_heads, G, longest, p.max_context_len);
  const int64_t sms = device_sm_count();
  CUtensorMap tm_q;
  if (!encode_q_tokens(&tm_q, p.q, static_cast<uint64_t>(p.num_tokens), static_cast<uint64_t>(p.num_q_heads) * 128,
                       static_cast<uint32_t>(128 / G)))
    return cudaErrorInvalidValue;
  for (int seq0 = 0; seq0 < p.num_seqs; seq0 += seqs) {
    Launch L{};
    L.p = p;
    L.p.num_seqs = p.num_seqs - seq0 < seqs ? p.num_seqs - seq0 : seqs;
    L.p.cu_q += seq0;
    L.p.q_start += seq0;
    L.p.block_tables += static_cast<int64_t>(seq0) * p.max_blocks_per_seq;
    L.rows = rows_of(G, longest);
    L.tile_bytes = static_cast<uint32_t>(fp4_tile_bytes(p.block_size, 128));
    L.bs_log = __builtin_ctz(static_cast<unsigned>(p.block_size));
    L.counters = reinterpret_cast<int32_t*>(p.ws + 256);
    L.o = reinterpret_cast<float*>(p.ws + 256 + fp4_counter_bytes());
    L.ml = L.o + 2 * sms * L.rows * 128;
    const void* fn = kernel_for(G);
    const int smem = kSmemBytes + (L.p.num_seqs + 64) / 64 * 256;  // few different sizes
    int per_sm = 0;
    cudaError_t e = fp4_occupancy(fn, kThreads, smem, &per_sm);
    if (e != cudaSuccess) return e;
    // every SM, while the items are not cut into too many parts to add up
    const int64_t items = static_cast<int64_t>(L.p.num_seqs) * pairs_of(G, longest) * p.num_kv_heads;
    const int64_t ctas = items * kMostParts < sms ? items * kMostParts : sms;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&L, &tm_q};
    e = cudaLaunchKernelExC(&cfg, fn, args);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pa
