// Decode attention over the 4-bit K/V pages (the format: fp4.cuh).
//
// For every (sequence, kv head), with its G query heads,
//   S[t][h] = scale q[h].K[t],  O[h] = sum_t softmax_t(S)[t][h] V[t].
// A token costs 9/16 byte an element where bf16 costs 2, so the memory leaves
// an SM about 780 clocks for 128 tokens of one kv head (K and V, D = 128), and
// what bounds the kernel next is the instructions that turn codes into
// operands: 2 per 2 elements (cvt e2m1x2 -> f16x2, times the scale).  Hence:
//  * the products run on mma.sync m16n8k16 (f16 in, fp32 out), whose operands
//    come from registers: a converted value goes straight into the instruction
//    that uses it, and never to shared or tensor memory.  Both products put
//    the cache on the 16-row side and the heads on the 8-column side,
//      S^T[16 tokens x 8 heads]  = K[16 x D] . Q^T
//      O^T[16 dims x 8 heads]   += V^T[16 x 16 tokens] . P^T,
//    so with G = 4 half of the columns are idle, not three quarters;
//  * the indices a product sums over may come in any order.  In Q.K^T a thread
//    takes D / 4 consecutive dims of a token (one 16-byte load for D = 128);
//    in P.V it takes D / 8 consecutive dims of four tokens, and two tokens'
//    nibbles are interleaved before the conversion, which then yields the
//    (token, token') pairs that the instruction wants;
//  * codes * scale is exact in f16.  The queries are scaled by a power of two
//    per head (their largest magnitude to 2^14) and are exact in f16 down to
//    2^-28 of it.  The probabilities, times 2^10, are rounded to f16: 2^-12
//    each, against 2^-9 in bf16, and none is lost before 2^-34 of the largest;
//  * every warp streams its own 32-token units, K and V, through a ring of its
//    own with cp.async, the table entries of the next unit loaded one unit
//    ahead.  (Bulk copies of the pages' tiles were right too, but the hardware
//    takes them lane by lane: 25 instructions each, four a unit.)  Blocks of 8 (from
//    128 dims on), of 16 and of 32 and more tokens have kernels with their layout
//    as constants: 700 instructions a unit instead of 900 (32 sequences of 4096
//    tokens in blocks of 8: 55.7 us, 69 without; in blocks of 4, which have none,
//    84).  Warps meet only at the end of a (sequence, kv head), to add up their
//    sums.  Units of 64 tokens, which halve what a unit costs besides its tokens,
//    gave 70.3 / 76.8 / 65.0 us against 65.2 / 72.2 / 69.7 (the three sizes below):
//    too few units for the warps of a short sequence;
//  * the work is cut into equal runs of units, one for each CTA, across the
//    borders of heads and sequences, counting what a head's start and end cost
//    (kLead).  A (sequence, kv head) that several CTAs share is joined by the
//    last of them, in the order of its tokens, so results do not depend on which
//    CTA is last.
//
// Four CTAs of four warps an SM (128 registers): three of 168 registers gave
// 66.6 / 78.9 / 66.3 us where four gave 64.4 / 73.9 / 69.4 (batch 256 GQA, batch
// 64 MHA, 8 x 32768 tokens); 8 warps a CTA 76 / 121 / 75, since more warps share
// a head's start and end.  At 65 us the batch-256 step (253 MB) runs at 3.9 TB/s,
// 57% of the measured copy rate: the loads alone took 58 us of a 73 us version
// and the instructions alone 60, with 57% of the issue slots filled by 16 warps.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <mutex>

#include "decode.cuh"
#include "fp4.cuh"
#include "ptx.cuh"

namespace pa {
namespace fp4_decode_detail {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnit = 32;    // tokens a warp takes at a time
// Units in a warp's ring: what an SM's shared memory holds for 16 warps (8
// with 16 heads or 256 dims), so that a warp has the next one or three in
// flight while it works on one.
__host__ __device__ constexpr int ring_stages(int D, int NT) { return D == 64 || (D == 128 && NT == 2) ? 4 : 2; }
constexpr int kMergeHeads = 4;  // heads whose sums are joined at a time
// What starting and joining a (sequence, kv head) costs a CTA, in units: the
// shares of the CTAs count it, as places before the first unit.
constexpr int kLead = 6;
constexpr float kPShift = 10.f;  // probabilities enter P.V times 2^10
// The reference of the probabilities is raised only when a score passes it by
// more than 2^4: they stay below 2^14 in f16, and most units leave O alone.
constexpr float kSlack = 4.f;

// Sequences of one launch: their lengths and unit counts live in shared memory.
constexpr int kMaxSeqs = 1024;

struct Launch {
  Fp4AttnParams p;
  int seq0, nseq;          // this launch's sequences
  int hkv, group, cache_heads, per_cache_head;  // (virtual) kv heads, their query heads; see launch_fp4_decode
  int eff_log;             // log2 of the tokens of a piece (a page's, at most a unit's)
  int bs_log;
  int piece_bytes;         // of one piece in shared memory
  int kv_bytes;            // of one unit's K (or V) in shared memory
  int off_merge, off_stat, off_qraw, off_q, off_qfac, off_prefix, off_lens, off_bar;
  uint32_t tile_bytes;
  int32_t* counters;       // [CTAs], zero between launches: of the head that CTA is the first of several to work on
  float* part;             // [2 * CTAs][G * (D + 2)]
};

using fp4::fast_exp2;
using fp4::pack_f16;
// the 8 x 8 matrix of 16-bit elements spread over the warp, transposed
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// four outputs, times inv
__device__ __forceinline__ void store4(const Fp4AttnParams& p, int64_t at, const float4& v, float inv) {
  if (p.out_bf16) {
    __nv_bfloat162 r[2] = {__floats2bfloat162_rn(v.x * inv, v.y * inv), __floats2bfloat162_rn(v.z * inv, v.w * inv)};
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + at) = *reinterpret_cast<const uint2*>(r);
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  }
}
template <int BYTES>
struct Words;  // BYTES consecutive bytes of shared memory as 32-bit words
template <>
struct Words<4> {
  uint32_t w[1];
  __device__ __forceinline__ void load(const unsigned char* p) { w[0] = *reinterpret_cast<const uint32_t*>(p); }
};
template <>
struct Words<8> {
  uint32_t w[2];
  __device__ __forceinline__ void load(const unsigned char* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
};
template <>
struct Words<16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const unsigned char* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
};
template <>
struct Words<32> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const unsigned char* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 16);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
};

// A place of the launch: a unit, 32 tokens of a (sequence, kv head), or one of
// the kLead places before its first unit (st < 0), which hold no work.
struct Cursor {
  int seq, head, st, nst;  // st of the nst units of this (sequence, kv head)
};

}  // namespace fp4_decode_detail

// D: head_dim; NT: columns of heads in eights (G <= 8 * NT); EL: log2 of the
// tokens of a piece (blocks of 8 tokens: 3, of 16: 4, of 32 and more: 5), or -1
// for smaller blocks, whose layout is then read from L
template <int D, int NT, int EL>
__global__ void __launch_bounds__(fp4_decode_detail::kThreads, (D <= 128 && NT == 1) ? 4 : 2)
    fp4_decode_kernel(const __grid_constant__ fp4_decode_detail::Launch L) {
  using namespace fp4_decode_detail;
  constexpr int kStages = ring_stages(D, NT);
  const int eff_log = EL >= 0 ? EL : L.eff_log;
  const int eff = 1 << eff_log, npieces = kUnit >> eff_log;
  const int piece_bytes = EL >= 0 ? (1 << (EL >= 0 ? EL : 0)) * (D / 2 + D / 16) : L.piece_bytes;
  const int kv_bytes = EL >= 0 ? kUnit * (D / 2 + D / 16) : L.kv_bytes;
  constexpr int kMma = D / 16;        // instructions of Q.K^T a slice of 16 tokens, and of P.V
  constexpr int kKWords = D / 32;     // words of codes of a thread's dims in Q.K^T (D / 4)
  constexpr int kVWords = D / 64;     // and in P.V (D / 8)
  const Fp4AttnParams& p = L.p;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, tig = lane & 3;  // the thread's row and column group in an instruction's operands
  const int hkv = L.hkv, G = L.group;
  unsigned char* ring = smem + warp * (kStages * 2 * kv_bytes);
  float* merge = reinterpret_cast<float*>(smem + L.off_merge);     // [warp][G][D + pad]
  float2* stat = reinterpret_cast<float2*>(smem + L.off_stat);     // [warp][8]: maximum, sum
  __nv_bfloat16* qraw = reinterpret_cast<__nv_bfloat16*>(smem + L.off_qraw);  // [G * D], the next segment's
  uint4* qf16 = reinterpret_cast<uint4*>(smem + L.off_q);  // [2][NT][D / 32][32 lanes]: operands of Q.K^T
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + L.off_prefix);       // [nseq + 1] places before a sequence
  int32_t* lens = reinterpret_cast<int32_t*>(smem + L.off_lens);
  float* qfac = reinterpret_cast<float*>(smem + L.off_qfac);               // [2][16] score factors
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + L.off_bar);         // the next segment's queries
  uint64_t* merge_free = q_full + 1;  // the merge area and stat have been read
  uint64_t* never = q_full + 2;       // no one arrives: for pa_test_stall_decode
  __shared__ int warp_sums[kWarps];
  __shared__ int last_flag;

  ptx::griddep_launch_dependents();
  if (tid == 0) {
    ptx::mbar_init(q_full, 1);
    ptx::mbar_init(merge_free, kWarps);
    ptx::mbar_init(never, 1);
    ptx::mbar_init_fence();
  }
  for (int i = tid; i < 2 * NT * (D / 32) * 32; i += kThreads) qf16[i] = make_uint4(0, 0, 0, 0);  // heads past G
  ptx::griddep_wait();

  // ---- places before every sequence: kLead and one for every unit of each of
  // its kv heads (an empty sequence has a unit of no tokens) ----
  {
    const int per = (L.nseq + kThreads - 1) / kThreads;
    const int beg = min(L.nseq, tid * per), end = min(L.nseq, beg + per);
    int local = 0;
    for (int i = beg; i < end; ++i) {
      int n = p.context_lens[L.seq0 + i];
      if (n < 0 || n > p.max_context_len) {
        if (blockIdx.x == 0) atomicExch(p.err, kDevErrInvalidArg);
        n = n < 0 ? 0 : p.max_context_len;
      }
      lens[i] = n;
      local += (kLead + max(1, (n + kUnit - 1) / kUnit)) * hkv;
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
    for (int i = beg; i < end; ++i) {
      prefix[i] = run;
      run += (kLead + max(1, (lens[i] + kUnit - 1) / kUnit)) * hkv;
    }
    if (tid == kThreads - 1) prefix[L.nseq] = run;
    __syncthreads();
  }
  const int total = prefix[L.nseq];
  // CTA c takes places [c * share + min(c, extra), ...): share or share + 1 of them
  const int share = total / gridDim.x, extra = total - share * gridDim.x;
  auto cta_begin = [&](int c) { return c * share + min(c, extra); };
  auto cta_of = [&](int u) {
    const int wide = extra * (share + 1);
    return u < wide ? u / (share + 1) : extra + (u - wide) / share;
  };
  const int c_begin = cta_begin(blockIdx.x), c_end = cta_begin(blockIdx.x + 1);
  if (c_begin >= c_end) return;

  auto locate = [&](int u, Cursor& c) {
    int lo = 0, hi = L.nseq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    c.seq = lo;
    const int places = (prefix[lo + 1] - prefix[lo]) / hkv;
    const int r = u - prefix[lo];
    c.nst = places - kLead;
    c.head = r / places;
    c.st = r - c.head * places - kLead;
  };
  auto advance = [&](Cursor& c, int by) {
    c.st += by;
    while (c.st >= c.nst) {
      c.st -= c.nst + kLead;
      if (++c.head == hkv) {
        c.head = 0;
        if (++c.seq >= L.nseq) return;
        c.nst = (prefix[c.seq + 1] - prefix[c.seq]) / hkv - kLead;
      }
    }
  };

  // ---- this warp's stream of units: c_begin + warp, + kWarps, ... ----
  const int bs = 1 << L.bs_log;
  Cursor ic{};              // the next unit to be fetched
  int iu = c_begin + warp;  // its place
  int ilen = 0;             // its sequence's length
  const int32_t* itable = nullptr;
  int32_t phys = 0;         // its page, this lane's piece
  auto fetch_table = [&]() {
    const int tok = ic.st * kUnit + (lane << eff_log);
    if (lane < npieces && tok < ilen) phys = __ldg(itable + (tok >> L.bs_log));
  };
  auto enter = [&]() {  // ic is in another sequence
    ilen = lens[ic.seq];
    itable = p.block_tables + static_cast<int64_t>(L.seq0 + ic.seq) * p.max_blocks_per_seq;
  };
  auto next_unit = [&]() {
    iu += kWarps;
    if (iu >= c_end) return;
    ic.st += kWarps;
    if (ic.st >= ic.nst) {  // into the next (sequence, kv head), past its lead
      ic.st -= kWarps;
      advance(ic, kWarps);
      while (ic.st < 0) {
        iu += kWarps;
        if (iu >= c_end) return;
        advance(ic, kWarps);
      }
      enter();
    }
    fetch_table();
  };
  auto copy16 = [](uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  };
  const uint32_t ring_lane = ptx::smem_addr(ring) + lane * 16;
  const uint8_t* const k_lane = p.k_cache + lane * 16;
  const uint8_t* const v_lane = p.v_cache + lane * 16;
  const uint32_t tile_bytes = L.tile_bytes;
  uint32_t issue_at = 0;  // the ring place to be filled
  int use_slot = 0;
  // fetches the next unit, or nothing at the end: one group of copies each time
  auto issue = [&]() {
    if (iu < c_end) {
      const int nv = (ilen - ic.st * kUnit + eff - 1) >> eff_log;  // pieces that hold tokens, or more
      if (lane < min(nv, npieces) && static_cast<uint32_t>(phys) >= static_cast<uint32_t>(p.num_blocks)) {
        atomicExch(p.err, kDevErrInvalidArg);  // never read outside the pool
        phys = 0;
      }
      const uint32_t dst = ring_lane + issue_at;
      const uint32_t cache_head = L.per_cache_head == 1 ? ic.head : ic.head / L.per_cache_head;
      // this lane's piece's tile (fewer than 2^31 of them in a pool)
      const uint32_t mine = static_cast<uint32_t>(phys) * L.cache_heads + cache_head;
      if constexpr (EL >= 0) {
        // 16-byte chunks: kPerPiece a lane of a piece's codes, then one of the
        // unit's scales in the first kScales lanes
        constexpr int kEff = 1 << EL, kPieces = kUnit / kEff, kPieceBytes = kEff * (D / 2 + D / 16);
        constexpr int kPerPiece = kEff * (D / 2) / 512, kScales = kUnit * (D / 16) / 16;
        static_assert(kPerPiece > 0 && kPerPiece * 512 == kEff * (D / 2), "whole rounds of the lanes");
        const int row = EL == 5 ? (ic.st * kUnit) & (bs - 1) : 0;  // of the piece in its tile
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          const uint64_t at = static_cast<uint64_t>(__shfl_sync(0xffffffffu, mine, j)) * tile_bytes + row * (D / 2);
          if (j < nv) {
#pragma unroll
            for (int i = 0; i < kPerPiece; ++i) {
              copy16(dst + j * kPieceBytes + i * 512, k_lane + at + i * 512);
              copy16(dst + j * kPieceBytes + kv_bytes + i * 512, v_lane + at + i * 512);
            }
          }
        }
        // a piece's scale chunks: lanes c of kScales / kPieces
        constexpr int kSc = kScales / kPieces;
        const int j = (lane / kSc) & (kPieces - 1);
        const uint64_t at = static_cast<uint64_t>(__shfl_sync(0xffffffffu, mine, j)) * tile_bytes + bs * (D / 2) +
                            row * (D / 16) - j * (kSc * 16);
        if (lane < kScales && j < nv) {
          const uint32_t d = dst + j * (kPieceBytes - kSc * 16) + kEff * (D / 2);
          copy16(d, k_lane + at);
          copy16(d + kv_bytes, v_lane + at);
        }
      } else {
        const int n = min(nv, npieces);
#pragma unroll 1
        for (int j = 0; j < n; ++j) {  // whole tiles of a few hundred bytes
          const uint64_t at = static_cast<uint64_t>(__shfl_sync(0xffffffffu, mine, j)) * tile_bytes;
          for (int c = 0; c + lane * 16 < piece_bytes; c += 512) {
            copy16(dst + j * piece_bytes + c, k_lane + at + c);
            copy16(dst + j * piece_bytes + kv_bytes + c, v_lane + at + c);
          }
        }
      }
      issue_at = issue_at + 2 * kv_bytes == kStages * 2 * kv_bytes ? 0 : issue_at + 2 * kv_bytes;
      next_unit();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (iu < c_end) {
    locate(iu, ic);
    while (ic.st < 0 && iu < c_end) {
      iu += kWarps;
      if (iu < c_end) advance(ic, kWarps);
    }
    if (iu < c_end) {
      enter();
      fetch_table();
    }
  }
  for (int s = 0; s < kStages; ++s) issue();

  // ---- where this thread's tokens lie in a unit ----
  // Row r of a slice (and index r of the sum in P.V) is token 2a + (e ^ (a & 1))
  // for r = 2a + e: of the rows 0, 2, 4, 6 that a load of V touches together
  // two then lie in even and two in odd 64-byte rows (D = 128).
  auto row_token = [](int r) { return (r & ~1) + ((r & 1) ^ ((r >> 1) & 1)); };
  auto place = [&](int t, int& codes, int& scales) {
    const int piece = t >> eff_log, o = t & (eff - 1);
    codes = piece * piece_bytes + o * (D / 2);
    scales = piece * piece_bytes + eff * (D / 2) + o * (D / 16);
  };
  int k_c0, k_s0, v_c0, v_s0, v_c1, v_s1, c8, s8, c16, s16;
  place(row_token(g), k_c0, k_s0);
  place(row_token(2 * tig), v_c0, v_s0);
  place(row_token(2 * tig + 1), v_c1, v_s1);
  {
    int z0, z1;
    place(0, z0, z1);
    place(8, c8, s8);
    place(16, c16, s16);
    s8 -= z1;
    s16 -= z1;
  }
  k_c0 += tig * (D / 8);
  k_s0 += tig * (D / 64);
  v_c0 += g * (D / 16);
  v_c1 += g * (D / 16);
  v_s0 += g * D / 128;
  v_s1 += g * D / 128;

  // ---- queries: a (sequence, kv head)'s rows, fetched one segment ahead ----
  // They are turned into f16, in the order of the operands, before the segment
  // before is joined (its own are in the other buffer).
  const int q_chunks = G * D / 8;
  auto fetch_q = [&](const Cursor& c) {  // one run of bytes
    if (tid == 0) {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) +
                                 (static_cast<int64_t>(L.seq0 + c.seq) * p.num_q_heads + c.head * G) * D;
      ptx::mbar_arrive_expect_tx(q_full, G * D * 2);
      ptx::bulk_g2s(qraw, src, G * D * 2, q_full, ptx::policy_evict_first());
    }
  };
  // A wait that gives up ends the whole CTA's work at its next barrier: no later
  // wait begins, no query copy either, and the end reports it.
  bool aborted = false;
  uint32_t q_parity = 0;
  auto convert_q = [&](int b) {
    if (!ptx::mbar_wait(q_full, q_parity, kWaitLimitNs)) aborted = true;
    q_parity ^= 1u;
    for (int i0 = 0; i0 < q_chunks; i0 += kThreads) {
      const int i = i0 + tid;
      const uint4 v = i < q_chunks ? *reinterpret_cast<const uint4*>(qraw + i * 8) : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
#pragma unroll
      for (int x = 1; x < D / 8; x *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
      // exponent that takes the head's largest magnitude to [2^14, 2^15); 0
      // for a zero, subnormal or non-finite row.  A negative softmax scale
      // goes into the sign of the query: the score factor is not negative.
      const int ex = static_cast<int>(top >> 7);
      const int shift = ex == 0 || ex == 255 ? 0 : max(-126, min(126, 14 - (ex - 127)));
      const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 + shift) << 23), p.scale_log2);
      uint32_t r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        r[e] = pack_f16(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xffff0000u) * up);
      if (i < q_chunks) {
        const int h = i / (D / 8), c = i % (D / 8);  // head, eight dims of it
        qf16[((b * NT + (h >> 3)) * (D / 32) + c % (D / 32)) * 32 + (h & 7) * 4 + c / (D / 32)] = make_uint4(r[0], r[1], r[2], r[3]);
        if (c == 0)
          // (not zero: a masked -inf times it stays -inf)
          qfac[b * 16 + h] =
              fmaxf(fabsf(p.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 - shift) << 23), 1.2e-38f);
      }
    }
  };

  Cursor sc;  // the segment: this CTA's units of one (sequence, kv head)
  locate(c_begin, sc);
  const int s_begin = sc.st < 0 ? c_begin - sc.st : c_begin;  // its first unit
  if (sc.st < 0) sc.st = 0;
  if (s_begin >= c_end) return;
  fetch_q(sc);
  convert_q(0);
  aborted = __syncthreads_or(aborted);
  int qb = 0;
  uint32_t merge_parity = 1;  // free at the start
  for (int sb = s_begin; sb < c_end && !aborted;) {
    const int item_b = sb - sc.st;                    // the item's first unit
    const int se = min(c_end, item_b + sc.nst);       // the segment's end
    Cursor next = sc;
    const bool more = se + kLead < c_end;             // another segment with a unit follows
    if (more) {
      next.st = sc.nst - 1;
      advance(next, 1 + kLead);
      fetch_q(next);
    }
    const int len = lens[sc.seq];

    float fac[NT][2];  // score factor of the thread's columns, heads 2 tig and 2 tig + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) fac[nt][c] = nt * 8 + 2 * tig + c < G ? qfac[qb * 16 + nt * 8 + 2 * tig + c] : 1.f;

    float o[NT][kMma][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) m[nt][e] = -CUDART_INF_F, l[nt][e] = 0.f;
#pragma unroll
      for (int j = 0; j < kMma; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
    }

    // the warp's units of the segment
    const int first = sb + ((c_begin + warp - sb) % kWarps + kWarps) % kWarps;
    for (int u = first; u < se; u += kWarps) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      __syncwarp();
      const int slot = use_slot;
      if (++use_slot == kStages) use_slot = 0;
      const unsigned char* kb = ring + slot * 2 * kv_bytes;
      const unsigned char* vb = kb + kv_bytes;
      const int left = len - (u - item_b) * kUnit;  // tokens from this unit on

      // S^T of two slices of 16 tokens, side by side
      float s[2][NT][4];
      Words<D / 8> kw[2][2];  // [slice][rows g, g + 8]: the codes of the thread's dims
      uint32_t ks[2][2];      // their scales: D / 64 bytes
#pragma unroll
      for (int sl = 0; sl < 2; ++sl)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          kw[sl][r].load(kb + k_c0 + sl * c16 + r * c8);
          const unsigned char* ps = kb + k_s0 + sl * s16 + r * s8;
          if (D == 64) ks[sl][r] = ps[0];
          else if (D == 128) ks[sl][r] = *reinterpret_cast<const uint16_t*>(ps);
          else ks[sl][r] = *reinterpret_cast<const uint32_t*>(ps);
        }
#pragma unroll
      for (int sl = 0; sl < 2; ++sl)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[sl][nt][e] = 0.f;
#pragma unroll
      for (int w = 0; w < kKWords; ++w) {
        uint4 q[NT];  // head g (and g + 8), eight dims
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) q[nt] = qf16[((qb * NT + nt) * (D / 32) + w) * 32 + lane];
#pragma unroll
        for (int sl = 0; sl < 2; ++sl) {
          uint32_t h[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            // words 2i and 2i + 1 are group i of the thread's dims
            const uint32_t pair = fp4::scales_to_f16(ks[sl][r] >> (16 * (w >> 2)));
            const uint32_t sc2 = (w & 2) ? __byte_perm(pair, 0, 0x3232) : __byte_perm(pair, 0, 0x1010);
            fp4::codes_to_f16(kw[sl][r].w[w], h[r]);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[r][e] = fp4::mul_f16x2(h[r][e], sc2);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma(s[sl][nt], h[0][0], h[1][0], h[0][1], h[1][1], q[nt].x, q[nt].y);
            mma(s[sl][nt], h[0][2], h[1][2], h[0][3], h[1][3], q[nt].z, q[nt].w);
          }
        }
      }
      if (left < kUnit) {  // tokens past the end
        const int t = row_token(g);
#pragma unroll
        for (int sl = 0; sl < 2; ++sl)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (sl * 16 + (e >> 1) * 8 + t >= left) s[sl][nt][e] = -CUDART_INF_F;
      }
      // m: the reference of the probabilities (log2), the same in the four
      // lanes' column of a head; l: the sum of this thread's own rows
      float mx[NT][2];
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          mx[nt][c] = fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2]));
          mx[nt][c] *= fac[nt][c];
          over |= mx[nt][c] > m[nt][c] + kSlack;
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = mx[nt][c];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            const float mn = fmaxf(m[nt][c], v);
            const float corr = mn == -CUDART_INF_F ? 1.f : fast_exp2(m[nt][c] - mn);
            m[nt][c] = mn;
            l[nt][c] *= corr;
#pragma unroll
            for (int j = 0; j < kMma; ++j) o[nt][j][c] *= corr, o[nt][j][c + 2] *= corr;
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float bias = m[nt][c] == -CUDART_INF_F ? 0.f : kPShift - m[nt][c];
#pragma unroll
          for (int sl = 0; sl < 2; ++sl)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float e = fast_exp2(fmaf(s[sl][nt][c + 2 * r], fac[nt][c], bias));
              s[sl][nt][c + 2 * r] = e;
              l[nt][c] += e;
            }
        }
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int sl = 0; sl < 2; ++sl)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            pb[sl][nt][r] = transpose8x8(pack_f16(s[sl][nt][2 * r], s[sl][nt][2 * r + 1]));

      // O^T += V^T P^T
#pragma unroll
      for (int sl = 0; sl < 2; ++sl) {
        Words<D / 16> v[4];  // tokens of indices 2 tig, 2 tig + 1, and + 8
        uint32_t vs[4][D == 256 ? 2 : 1];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int co = ((t & 1) ? v_c1 : v_c0) + sl * c16 + (t >> 1) * c8;
          const int so = ((t & 1) ? v_s1 : v_s0) + sl * s16 + (t >> 1) * s8;
          v[t].load(vb + co);
          vs[t][0] = vb[so];
          if (D == 256) vs[t][D == 256 ? 1 : 0] = vb[so + 1];
        }
        if (left < kUnit) {  // the scales of what lies past the end may be NaN: 0 * NaN must not reach the sums
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (sl * 16 + (t >> 1) * 8 + row_token(2 * tig + (t & 1)) >= left) {
              vs[t][0] = 0;
              if (D == 256) vs[t][D == 256 ? 1 : 0] = 0;
            }
        }
#pragma unroll
        for (int w = 0; w < kVWords; ++w) {
          const int sg = D == 256 ? (w >> 1) : 0;
          const uint32_t m0 = fp4::scales_to_f16(vs[0][sg] | (vs[1][sg] << 8));
          const uint32_t m1 = fp4::scales_to_f16(vs[2][sg] | (vs[3][sg] << 8));
          uint32_t a0[4], a1[4], a2[4], a3[4];  // even dims, odd dims of tokens 0, 1; the same of tokens 2, 3
          const uint32_t x0 = v[0].w[w], x1 = v[1].w[w], x2 = v[2].w[w], x3 = v[3].w[w];
          fp4::codes_to_f16((x0 & 0x0f0f0f0fu) | ((x1 << 4) & 0xf0f0f0f0u), a0);
          fp4::codes_to_f16(((x0 >> 4) & 0x0f0f0f0fu) | (x1 & 0xf0f0f0f0u), a1);
          fp4::codes_to_f16((x2 & 0x0f0f0f0fu) | ((x3 << 4) & 0xf0f0f0f0u), a2);
          fp4::codes_to_f16(((x2 >> 4) & 0x0f0f0f0fu) | (x3 & 0xf0f0f0f0u), a3);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t b0 = fp4::mul_f16x2(a0[e], m0), b1 = fp4::mul_f16x2(a1[e], m0);
            const uint32_t b2 = fp4::mul_f16x2(a2[e], m1), b3 = fp4::mul_f16x2(a3[e], m1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma(o[nt][4 * w + e], b0, b1, b2, b3, pb[sl][nt][0], pb[sl][nt][1]);
          }
        }
      }
      __syncwarp();
      issue();
    }

    // ---- the warps' sums of the segment joined, a few heads at a time ----
    // Head pairs at a distance of 2 D + 4 floats, and the floats of row group g
    // turned by a multiple of 8, so that a store touches every bank once.
    constexpr int kPair = 2 * D + 4, kRow = D / 8, kHeads = kMergeHeads;
    const int gpairs = (min(G, kHeads) + 1) / 2;
    const int turn = D == 64 ? 0 : (D == 128 ? 8 * ((g >> 1) & 1) : 8 * (g & 3));
    const bool active = first < se;
    const bool complete = item_b >= sb && item_b + sc.nst <= se;
    const int64_t out_row = static_cast<int64_t>(L.seq0 + sc.seq) * p.num_q_heads + sc.head * G;
    const int part_slot = sb == s_begin ? 0 : 1;
    float* part = L.part + (static_cast<int64_t>(blockIdx.x) * 2 + part_slot) * (G * (D + 2));
    if (more) convert_q(qb ^ 1);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 4);
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 8);
        l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], 16);
      }
#pragma unroll
      for (int h0 = 0; h0 < 8; h0 += kHeads) {
        const int heads = min(kHeads, G - nt * 8 - h0);  // of this round
        if (heads <= 0) break;
        // the round before, of this segment or the last, is read
        if (!ptx::mbar_wait(merge_free, merge_parity, kWaitLimitNs)) aborted = true;
        if (p.test_stall_ns && !ptx::mbar_wait(never, 0, p.test_stall_ns)) aborted = true;
        merge_parity ^= 1u;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int h = 2 * tig + c - h0;
          if (!aborted && h >= 0 && h < kHeads) {
            if (g == 0) stat[warp * 8 + h] = active ? make_float2(m[nt][c], l[nt][c]) : make_float2(-CUDART_INF_F, 0.f);
            if (active && h < heads) {
              float* row = merge + warp * (gpairs * kPair) + (h >> 1) * kPair + c * D + g * kRow;
#pragma unroll
              for (int j = 0; j < kMma; ++j)
                *reinterpret_cast<float2*>(row + ((2 * j + turn) & (kRow - 1))) =
                    make_float2(o[nt][j][c], o[nt][j][c + 2]);
            }
          }
        }
        aborted = __syncthreads_or(aborted);
        if (aborted) goto stop;
        for (int i = tid; i < heads * D / 4; i += kThreads) {
          const int h = i / (D / 4), d = (i - h * (D / 4)) * 4;
          float2 st[kWarps];
          float M = -CUDART_INF_F;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            st[w] = stat[w * 8 + h];
            M = fmaxf(M, st[w].x);
          }
          const float ref = M == -CUDART_INF_F ? 0.f : M;
          const int rg = d / kRow;
          const int rt = D == 64 ? 0 : (D == 128 ? 8 * ((rg >> 1) & 1) : 8 * (rg & 3));
          const float* at = merge + (h >> 1) * kPair + (h & 1) * D + rg * kRow + ((d - rg * kRow + rt) & (kRow - 1));
          float lsum = 0.f;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            if (st[w].y != 0.f) {  // a warp without tokens wrote nothing
              const float f = fast_exp2(st[w].x - ref);
              const float4 v = *reinterpret_cast<const float4*>(at + w * (gpairs * kPair));
              lsum = fmaf(f, st[w].y, lsum);
              x.x = fmaf(f, v.x, x.x);
              x.y = fmaf(f, v.y, x.y);
              x.z = fmaf(f, v.z, x.z);
              x.w = fmaf(f, v.w, x.w);
            }
          }
          const int head = nt * 8 + h0 + h;
          if (complete) {
            const float inv = lsum != 0.f ? p.v_scale / lsum : 0.f;
            store4(p, (out_row + head) * D + d, x, inv);
          } else {
            float* q = part + 2 * G + head * D + d;
            *reinterpret_cast<float2*>(q) = make_float2(x.x, x.y);
            *reinterpret_cast<float2*>(q + 2) = make_float2(x.z, x.w);
            if (d == 0) *reinterpret_cast<float2*>(part + 2 * head) = make_float2(M, lsum);
          }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(merge_free);
      }
    }
    if (!complete) {
      // the last CTA of the item joins the CTAs' parts, in the order of the tokens
      __threadfence();
      __syncthreads();  // and nobody reads the merge area any more
      const int c0 = cta_of(item_b), c1 = cta_of(item_b + sc.nst - 1);
      if (tid == 0) {
        int32_t* counter = L.counters + c0;
        const int before = atomicAdd(counter, 1);
        last_flag = before == c1 - c0;
        if (before == c1 - c0) *counter = 0;
        __threadfence();
      }
      __syncthreads();
      if (last_flag) {
        const int n = c1 - c0 + 1;
        const float* base = L.part;
        auto part_of = [&](int k) {
          const int c = c0 + k;
          return base + (static_cast<int64_t>(c) * 2 + (cta_begin(c) >= item_b - kLead ? 0 : 1)) * (G * (D + 2));
        };
        // groups of threads take every ngroups-th part; then the groups are added
        const int width = min(kThreads, G * D / 4);  // threads that cover the item's outputs, 4 each
        const int ngroups = kThreads / width, grp = tid / width;
        for (int i0 = 0; i0 < G * D / 4; i0 += width) {
          const int i = i0 + tid % width;
          const int h = i / (D / 4), d = (i - h * (D / 4)) * 4;
          float M = -CUDART_INF_F;
#pragma unroll 8
          for (int k = 0; k < n; ++k) M = fmaxf(M, __ldcg(part_of(k) + 2 * h));
          const float ref = M == -CUDART_INF_F ? 0.f : M;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          float lsum = 0.f;
#pragma unroll 4
          for (int k = grp; k < n; k += ngroups) {
            const float* q = part_of(k);
            const float2 st = __ldcg(reinterpret_cast<const float2*>(q + 2 * h));
            const float2 v0 = __ldcg(reinterpret_cast<const float2*>(q + 2 * G + h * D + d));
            const float2 v1 = __ldcg(reinterpret_cast<const float2*>(q + 2 * G + h * D + d + 2));
            const float f = st.y != 0.f ? fast_exp2(st.x - ref) : 0.f;
            lsum = fmaf(f, st.y, lsum);
            acc.x = fmaf(f, v0.x, acc.x);
            acc.y = fmaf(f, v0.y, acc.y);
            acc.z = fmaf(f, v1.x, acc.z);
            acc.w = fmaf(f, v1.y, acc.w);
          }
          if (ngroups > 1) {
            float* red = merge + tid * 5;  // 5 floats a thread
            red[0] = acc.x, red[1] = acc.y, red[2] = acc.z, red[3] = acc.w, red[4] = lsum;
            __syncthreads();
            if (grp == 0) {
              for (int r = 1; r < ngroups; ++r) {
                const float* o2 = merge + (tid + r * width) * 5;
                acc.x += o2[0], acc.y += o2[1], acc.z += o2[2], acc.w += o2[3], lsum += o2[4];
              }
            }
          }
          if (grp == 0) {
            const float inv = lsum != 0.f ? p.v_scale / lsum : 0.f;
            store4(p, (out_row + h) * D + d, acc, inv);
          }
        }
      }
      __syncthreads();  // the merge area and the flag are free again
    }
    if (!more) break;
    sb = se + kLead;
    sc = next;
    qb ^= 1;
  }
stop:
  if (aborted) {  // the whole CTA; the output is undefined, and the heads that it shares are left unjoined
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (tid == 0) {
      atomicExch(p.err, kDevErrTimeout);
      // a query copy whose wait of 2 s gave up is given another 2 s to land
      (void)ptx::mbar_wait(q_full, q_parity ^ 1u, kWaitLimitNs);
    }
    __syncthreads();
  }
}

namespace {

using fp4_decode_detail::Launch;

template <int D, int NT>
const void* kernel_of(int eff_log) {
  if (eff_log == 5) return reinterpret_cast<const void*>(&fp4_decode_kernel<D, NT, 5>);
  if (eff_log == 4) return reinterpret_cast<const void*>(&fp4_decode_kernel<D, NT, 4>);
  if constexpr (D >= 128)  // a round of the lanes copies 512 bytes: 8 rows of codes
    if (eff_log == 3) return reinterpret_cast<const void*>(&fp4_decode_kernel<D, NT, 3>);
  return reinterpret_cast<const void*>(&fp4_decode_kernel<D, NT, -1>);
}
const void* kernel_for(int head_dim, int group, int eff_log) {
  if (head_dim == 64) return group <= 8 ? kernel_of<64, 1>(eff_log) : kernel_of<64, 2>(eff_log);
  if (head_dim == 128) return group <= 8 ? kernel_of<128, 1>(eff_log) : kernel_of<128, 2>(eff_log);
  return kernel_of<256, 1>(eff_log);
}

// CTAs that a launch has at most: what its part slots are sized for.
int64_t max_ctas(int head_dim, int group) { return device_sm_count() * (head_dim <= 128 && group <= 8 ? 4 : 2); }

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

}  // namespace

// 16 query heads of 256 dims would need more registers than a thread has:
// they are taken as two kv heads of 8 that share their pages.
int per_cache_head(int head_dim, int group) { return head_dim == 256 && group == 16 ? 2 : 1; }

int64_t fp4_counter_bytes() { return round_up(4 * device_sm_count() * 4, 256); }

// CTAs of a kernel that an SM holds with this much dynamic shared memory, the
// answers kept for the devices and sizes that come by.
cudaError_t fp4_occupancy(const void* fn, int threads, int smem, int* per_sm) {
  struct Entry {
    const void* fn;
    int device, smem, per_sm;
  };
  static std::mutex mu;
  static Entry kept[64];
  static int n = 0, next = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  for (int i = 0; i < n; ++i)
    if (kept[i].fn == fn && kept[i].device == dev && kept[i].smem == smem) {
      *per_sm = kept[i].per_sm;
      return cudaSuccess;
    }
  // the attribute only ever grows: another thread's launch may count on it
  cudaFuncAttributes at{};
  if ((e = cudaFuncGetAttributes(&at, fn)) != cudaSuccess) return e;
  if (smem > at.maxDynamicSharedSizeBytes &&
      (e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
    return e;
  if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, fn, threads, smem)) != cudaSuccess) return e;
  if (*per_sm < 1) return cudaErrorInvalidConfiguration;
  kept[next] = Entry{fn, dev, smem, *per_sm};
  next = (next + 1) % 64;
  if (n < 64) ++n;
  return cudaSuccess;
}

size_t fp4_decode_workspace(int num_q_heads, int num_kv_heads, int head_dim) {
  using namespace fp4_decode_detail;
  const int split = per_cache_head(head_dim, num_q_heads / num_kv_heads);
  const int G = num_q_heads / num_kv_heads / split;
  // header | counters | parts: the first two lie where they lie for every shape
  return static_cast<size_t>(256 + fp4_counter_bytes() + max_ctas(head_dim, G) * 2 * G * (head_dim + 2) * 4);
}

cudaError_t launch_fp4_decode(const Fp4AttnParams& p, int head_dim, cudaStream_t stream) {
  using namespace fp4_decode_detail;
  const int split = per_cache_head(head_dim, p.num_q_heads / p.num_kv_heads);
  const int hkv = p.num_kv_heads * split;
  const int G = p.num_q_heads / hkv;
  const int eff = p.block_size < kUnit ? p.block_size : kUnit;
  const int eff_log = __builtin_ctz(static_cast<unsigned>(eff));
  const void* fn = kernel_for(head_dim, G, eff_log);
  // sequences of one launch: their places fit an int
  const int64_t places = (static_cast<int64_t>(p.max_context_len) + kUnit - 1) / kUnit + 1 + kLead;
  const int64_t fit = ((int64_t(1) << 31) - 1) / (places * hkv);
  const int seqs = static_cast<int>(fit < kMaxSeqs ? fit : kMaxSeqs);
  if (seqs < 1) return cudaErrorInvalidValue;
  for (int seq0 = 0; seq0 < p.num_seqs; seq0 += seqs) {
    Launch L{};
    L.p = p;
    L.seq0 = seq0;
    L.nseq = p.num_seqs - seq0 < seqs ? p.num_seqs - seq0 : seqs;
    L.hkv = hkv;
    L.group = G;
    L.cache_heads = p.num_kv_heads;
    L.per_cache_head = split;
    L.bs_log = __builtin_ctz(static_cast<unsigned>(p.block_size));
    L.eff_log = eff_log;
    L.tile_bytes = static_cast<uint32_t>(fp4_tile_bytes(p.block_size, head_dim));
    L.piece_bytes = static_cast<int>(fp4_tile_bytes(eff, head_dim));
    L.kv_bytes = (kUnit / eff) * L.piece_bytes;
    const int64_t merge =
        static_cast<int64_t>(kWarps) * (((G < kMergeHeads ? G : kMergeHeads) + 1) / 2) * (2 * head_dim + 4) * 4;
    int64_t off = static_cast<int64_t>(kWarps) * ring_stages(head_dim, G <= 8 ? 1 : 2) * 2 * L.kv_bytes;
    auto take = [&](int64_t bytes) {
      const int64_t at = off;
      off += round_up(bytes, 16);
      return static_cast<int>(at);
    };
    L.off_merge = take(merge > kThreads * 20 ? merge : kThreads * 20);
    L.off_stat = take(kWarps * 8 * 8);
    L.off_qraw = take(G * head_dim * 2);
    L.off_q = take(2 * (G <= 8 ? 8 : 16) * head_dim * 2);
    L.off_qfac = take(2 * 16 * 4);
    const int64_t held = round_up(L.nseq + 1, 64);  // few different sizes
    L.off_prefix = take(held * 4);
    L.off_lens = take(held * 4);
    L.off_bar = take(3 * 8);
    L.counters = reinterpret_cast<int32_t*>(p.ws + 256);
    L.part = reinterpret_cast<float*>(p.ws + 256 + fp4_counter_bytes());
    // at least a unit for every warp, as far as the longest context allows
    const int64_t most = static_cast<int64_t>(L.nseq) * hkv * ((p.max_context_len + kUnit - 1) / kUnit);
    int64_t ctas = (most + kWarps - 1) / kWarps;
    const int64_t items = static_cast<int64_t>(L.nseq) * hkv;
    if (ctas < items) ctas = items;
    int per_sm = 0;
    cudaError_t e = fp4_occupancy(fn, kThreads, static_cast<int>(off), &per_sm);
    if (e != cudaSuccess) return e;
    int64_t cap = device_sm_count() * per_sm;  // all of them at work at once: their shares are equal
    if (cap > max_ctas(head_dim, G)) cap = max_ctas(head_dim, G);
    if (ctas > cap) ctas = cap;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(off);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {&L};
    e = cudaLaunchKernelExC(&cfg, fn, args);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pa
