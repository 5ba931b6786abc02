// The tokens that stay when a cache is thinned out: of the positions
// [dst_start, len) of a sequence the last `recent`, and of the others those with
// the largest weights (ties: the lowest position first), in ascending order, and
// the weights moved to the places that token compaction gives their tokens.
//
// The threshold is found by radix selection on the weights' order-preserving
// bit patterns: up to four passes, each counts the 8-bit digits of the candidates
// that agree with the digits found so far, until all of those stay.  Then one sweep
// in order of the positions numbers what is above it, and as many of what equals
// it as are still wanted.  Counts are integers, so the result does not depend on
// the order of anything.
//
// A cluster of 1 to 8 CTAs shares a sequence: each holds a slice of its weights
// in shared memory, counts it there, and adds up the others' counts through
// distributed shared memory.  A digit that many weights share (zeros, the
// exponents of small numbers) would serialise a warp's additions, so every CTA
// counts in 16 copies, by lane, each a bank further.
//
// The work is a chain of passes with a barrier of the cluster after each; its
// bytes (8 a candidate) hardly count.  Measured: 32 sequences of 150 to 700 tokens
// 7.5 us (14 with rounds of the whole CTA and always four passes), 8 of 20000 to
// 32768 9.9 us (37 before).
#include <cooperative_groups.h>

#include "decode.cuh"
#include "fp4.cuh"
#include "latent.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCopies = 16, kPitch = 257;
constexpr int kMostCached = 48 * 1024;  // weights of a slice in shared memory

// ascending with the value; -0 as 0, NaN below everything
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p, int cap) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int seq = blockIdx.x / C, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c0 = p.cu_keep[seq], c1 = p.cu_keep[seq + 1];
  const int a = p.dst_start[seq], b = p.context_lens[seq], n = c1 - c0;
  // (every bound by comparison first: differences of values that are out of range may wrap)
  if (c0 == c1 && a >= 0 && a <= b && b <= p.max_context_len) {
    // nothing stays: the weights are cleared below
  } else if (c0 < 0 || c1 < c0 || c1 > p.num_keep || a < 0 || b < a || b > p.max_context_len || n > b - a) {
    if (p.status && rank == 0 && tid == 0) atomicExch(p.status, kDevErrInvalidArg);
    return;  // the whole cluster
  }
  const int late = min(max(p.recent, 0), n), need = n - late;
  const int last = b - late, m = last - a;  // candidates: [a, last)
  const int per = (m + C - 1) / C;
  const int lo = a + min(m, rank * per), hi = a + min(m, (rank + 1) * per), mine = hi - lo;
  float* row = p.weights + seq * p.weights_stride;
  const bool cached = per <= cap;

  extern __shared__ float slice[];
  __shared__ int hist[kCopies * kPitch];
  __shared__ int total[2][256], sums[256];
  __shared__ int shared_digit[3];
  __shared__ int2 counts;          // above, equal: of this CTA's slice
  __shared__ int2 warp_counts[kWarps];
  // a warp's stretch of the slice
  const int seg = (mine + kWarps * 32 - 1) / (kWarps * 32) * 32;
  const int w0 = min(mine, warp * seg), w1 = min(mine, w0 + seg);
  if (cached)
    for (int i = w0 + lane; i < w1; i += 32) slice[i] = row[lo + i];
  const float* w = cached ? slice : row + lo;

  // ---- the threshold, digit by digit ----
  uint32_t prefix = 0, mask = 0;
  int want = need;  // of the candidates that agree with prefix
  if (need > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      for (int i = tid; i < kCopies * kPitch; i += kThreads) hist[i] = 0;
      __syncthreads();
      int* mine_hist = hist + (lane & (kCopies - 1)) * kPitch;
#pragma unroll 4
      for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t k = order_of(w[i]);
        if ((k & mask) == prefix) atomicAdd(mine_hist + ((k >> shift) & 255u), 1);
      }
      __syncthreads();
      if (tid < 256) {
        int s = 0;
#pragma unroll
        for (int c = 0; c < kCopies; ++c) s += hist[c * kPitch + tid];
        total[pass & 1][tid] = s;
      }
      if (C > 1) cluster.sync();
      if (tid < 256) {
        int s = 0;
        if (C > 1) {
          int v[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) v[c] = c < C ? cluster.map_shared_rank(&total[pass & 1][0], c)[tid] : 0;
#pragma unroll
          for (int c = 0; c < 8; ++c) s += v[c];
        } else {
          s = total[pass & 1][tid];
        }
        sums[255 - tid] = s;
      }
      __syncthreads();
      if (warp == 0) {
        // lane: digits 255 - 8 lane and the seven below
        int cnt[8], sum = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += cnt[e] = sums[8 * lane + e];
        int above = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, above, o);
          if (lane >= o) above += y;
        }
        above -= sum;
        if (above < want && want <= above + sum) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (want > above && want <= above + cnt[e]) {
              shared_digit[0] = 255 - 8 * lane - e;
              shared_digit[1] = want - above;
              shared_digit[2] = cnt[e];
            }
            above += cnt[e];
          }
        }
      }
      __syncthreads();
      prefix |= static_cast<uint32_t>(shared_digit[0]) << shift;
      mask |= 255u << shift;
      want = shared_digit[1];
      if (want == shared_digit[2] && prefix) {  // all that agree so far stay: they are what lies above prefix - 1
        prefix -= 1;
        want = 0;
        break;
      }
    }
  } else {
    prefix = 0xffffffffu;  // no weight is as large
  }

  // ---- how many of each slice stay ----
  int gt = 0, eq = 0;
#pragma unroll 4
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = order_of(w[i]);
    gt += k > prefix;
    eq += k == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt), eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) warp_counts[warp] = make_int2(gt, eq);
  __syncthreads();
  if (tid == 0) {
    int2 s = make_int2(0, 0);
    for (int i = 0; i < kWarps; ++i) s.x += warp_counts[i].x, s.y += warp_counts[i].y;
    counts = s;
  }
  cluster.sync();  // also: every slice has been read
  int base = 0, take = want;  // places before this stretch; of its equal ones the first `take` stay
  auto pass_over = [&](int2 s) {
    base += s.x + min(s.y, take);
    take -= min(s.y, take);
  };
  for (int c = 0; c < rank; ++c) pass_over(*cluster.map_shared_rank(&counts, c));
  for (int v = 0; v < warp; ++v) pass_over(warp_counts[v]);

  // ---- positions in order, and the weights behind them ----
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const float x = i < w1 ? w[i] : 0.f;
    const uint32_t k = order_of(x);
    const bool is_gt = i < w1 && k > prefix, is_eq = i < w1 && k == prefix;
    const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
    const uint32_t below = (1u << lane) - 1u;
    const int g = __popc(bg & below), e = __popc(be & below);
    if (is_gt || (is_eq && e < take)) {
      const int at = base + g + min(e, take);
      p.keep[c0 + at] = lo + i;
      if (cached) row[a + at] = x;
    }
    pass_over(make_int2(__popc(bg), __popc(be)));
  }
  for (int j = rank * kThreads + tid; j < late; j += C * kThreads) p.keep[c0 + need + j] = last + j;
  if (cached) {
    // the rest of the candidates' places is cleared by everybody, the recent tokens' weights are moved by one CTA
    for (int t = max(a + n, lo) + tid; t < hi; t += kThreads) row[t] = 0.f;
    if (rank) {
      cluster.sync();  // nobody leaves while its counts may be read
      return;
    }
    if (last != a + need) {
      for (int j0 = 0; j0 < late; j0 += kThreads) {  // to places at or before their own, in order
        const int j = j0 + tid;
        const float x = j < late ? row[last + j] : 0.f;
        __syncthreads();
        if (j < late) row[a + need + j] = x;
      }
      __syncthreads();
      for (int t = max(a + n, last) + tid; t < b; t += kThreads) row[t] = 0.f;
    }
    cluster.sync();
    return;
  }
  // slices too long for shared memory: one CTA moves all weights, in order
  __threadfence();
  cluster.sync();
  if (rank) return;
  for (int j0 = 0; j0 < n; j0 += kThreads) {
    const int j = j0 + tid;
    const float x = j < n ? __ldcg(row + __ldcg(p.keep + c0 + j)) : 0.f;
    __syncthreads();
    if (j < n) row[a + j] = x;
    __syncthreads();
  }
  for (int t = a + n + tid; t < b; t += kThreads) row[t] = 0.f;
}

}  // namespace

cudaError_t launch_select(const SelectParams& p, cudaStream_t stream) {
  // CTAs a sequence: a slice of some 2048 weights each while they all run at once, two an SM (one CTA
  // alone sweeps 32768 weights 64 to a thread)
  int ctas = 1;
  while (ctas < 8 && static_cast<int64_t>(ctas) * 2048 < p.max_context_len &&
         static_cast<int64_t>(p.num_seqs) * ctas * 2 <= 2 * device_sm_count())
    ctas *= 2;
  const int per = (p.max_context_len + ctas - 1) / ctas;
  const int cap = per < kMostCached ? per : kMostCached;
  const int smem = (cap + 1023) / 1024 * 4096;
  int per_sm = 0;
  cudaError_t e = fp4_occupancy(reinterpret_cast<const void*>(&select_kernel), kThreads, smem, &per_sm);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.num_seqs) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_kernel, SelectParams(p), cap);
}

}  // namespace pa
