// blockmean.cuh - key blocks of each query block chosen by the mean score of
// the tile, for the block-sparse attention.
//
// The mean of the scores <q, k> over all pairs of a query block i and a key
// block j is the product of the blocks' means,
//   s(i, j) = <mean of q over i, mean of k over j>,
// so a row of scores costs one product of d per tile instead of the tile's
// 128 x 128.  Kept for row i: its own neighbourhood |i - j| <= local, then
// the largest s, at equal scores the lower j first, up to `keep` blocks.
//
// A border between kept and dropped must not depend on rounding: means and
// the scores that decide are 64-bit.  Three steps:
//  1. blockmean_pool_kernel: means, one read of q and k (the bound: HBM).
//  2. (rows' scores)
//  3. blockmean_select_kernel: one warp per row.
#pragma once
#include "ptx.cuh"

namespace bsa {

constexpr int kMeanMaxBlocks = 8192;
constexpr int kPoolThreads = 256;
constexpr int kPoolWarps = kPoolThreads / 32;

// grid (nB, ceil(H * d / 256), 2): one 128-token block of 256 neighbouring
// channels (whole heads) of q or k.  A warp reads 512 contiguous bytes per
// token, 8 channels a lane; its 16 tokens are added in 64 bits in order, then
// the eight warps' sums in order: bf16 values are 8 bits wide, so such a sum
// is exact unless the block spans more than 2^38, and equal blocks always
// give equal means.
// mean: [2][H][nB][d] double.
__global__ void __launch_bounds__(kPoolThreads) blockmean_pool_kernel(
    const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k, int N, int H, int d, int nB,
    double* __restrict__ mean) {
  __shared__ double s_sum[kPoolWarps][256];
  const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t row = static_cast<size_t>(H) * d;
  const int c0 = blockIdx.y * 256 + lane * 8;
  const __nv_bfloat16* x = blockIdx.z ? k : q;
  const int rows = min(128, N - b * 128);
  double acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0;
  if (c0 < static_cast<int>(row)) {
    const __nv_bfloat16* p = x + (static_cast<size_t>(b) * 128 + warp * 16) * row + c0;
    uint4 v[16];
#pragma unroll
    for (int t = 0; t < 16; ++t)
      v[t] = (warp * 16 + t < rows) ? __ldg(reinterpret_cast<const uint4*>(p + t * row)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const uint32_t w[4] = {v[t].x, v[t].y, v[t].z, v[t].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] += static_cast<double>(__uint_as_float(w[i] << 16));
        acc[2 * i + 1] += static_cast<double>(__uint_as_float(w[i] & 0xFFFF0000u));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s_sum[warp][lane * 8 + i] = acc[i];
  __syncthreads();
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c < static_cast<int>(row)) {
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kPoolWarps; ++w) s += s_sum[w][threadIdx.x];
    const int h = c / d;
    mean[((static_cast<size_t>(blockIdx.z) * H + h) * nB + b) * d + (c - h * d)] = s / rows;
  }
}

// 64-bit order of scores: larger key = larger score, -0 = +0, not-a-number
// with the smallest (it counts as minus infinity).
__device__ __forceinline__ unsigned long long score_key(double s) {
  if (!(s == s)) s = -INFINITY;
  s += 0.0;                                           // -0 becomes +0
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(s));
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

__device__ __forceinline__ unsigned long long warp_min_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = w < v ? w : v;
  }
  return v;
}

// One warp per row (grid (rows of a head in groups of warps, heads)); dynamic
// shared memory per warp: nB keys (8 bytes) and nB bits of candidates.
// A row's candidates are the blocks whose score has to be known in 64 bits;
// `take` of them are kept, found by bisection over their keys.
template <int D>
__global__ void __launch_bounds__(256) blockmean_select_kernel(const double* __restrict__ mean, int H, int nB, int keep,
                                                               int local, int32_t* __restrict__ idx,
                                                               int32_t* __restrict__ cnt) {
  extern __shared__ unsigned long long s_mean_keys[];
  constexpr int E = D / 64;                           // double2 per lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wpc = blockDim.x >> 5;
  const int qb = blockIdx.x * wpc + warp, h = blockIdx.y;
  if (qb >= nB) return;
  unsigned long long* key = s_mean_keys + static_cast<size_t>(warp) * nB;
  const double* mq = mean + (static_cast<size_t>(h) * nB + qb) * D;
  const double* mk = mean + (static_cast<size_t>(H) + h) * nB * D;
  const int f0 = max(0, qb - local), f1 = local < 0 ? f0 : min(nB, qb + local + 1);   // own neighbourhood
  const int forced = f1 - f0;
  const int total = min(nB, max(keep, forced));
  const int take = total - forced;                    // blocks chosen by score
  double2 qv[E];
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = *reinterpret_cast<const double2*>(mq + e * 64 + 2 * lane);
  unsigned long long pivot = 0, kmin = ~0ull, kmax = 0;
  int rest = nB - forced;                             // blocks with a key >= pivot
  if (take > 0 && take < rest) {
    for (int j = 0; j < nB; ++j) {
      double s = 0.0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const double2 kv = *reinterpret_cast<const double2*>(mk + static_cast<size_t>(j) * D + e * 64 + 2 * lane);
        s = fma(qv[e].x, kv.x, s);
        s = fma(qv[e].y, kv.y, s);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      const unsigned long long u = score_key(s);
      if (lane == 0) key[j] = u;
      if (j < f0 || j >= f1) {
        kmin = min(kmin, u);
        kmax = max(kmax, u);
      }
    }
    __syncwarp();
    // pivot = the take-th largest key: bisection below the bits all keys share
    pivot = kmin;
    if (kmax != kmin) {
      const int top = 63 - __clzll(static_cast<long long>(kmax ^ kmin));
      pivot = kmin >> top >> 1 << top << 1;
      for (int bit = top; bit >= 0; --bit) {
        const unsigned long long c = pivot | (1ull << bit);
        int n = 0;
        for (int j = lane; j < nB; j += 32) n += (key[j] >= c && (j < f0 || j >= f1)) ? 1 : 0;
        if (__reduce_add_sync(0xFFFFFFFFu, n) >= take) pivot = c;
      }
    }
  }
  // blocks above the pivot are kept, of those at the pivot the first ones
  const bool all = take == rest, none = take == 0;
  int ties = 0;
  if (!all && !none) {
    int above = 0;
    for (int j = lane; j < nB; j += 32) above += (key[j] > pivot && (j < f0 || j >= f1)) ? 1 : 0;
    ties = take - __reduce_add_sync(0xFFFFFFFFu, above);
  }
  int32_t* out = idx + (static_cast<size_t>(h) * nB + qb) * nB;
  int n = 0, seen = 0;
  for (int base = 0; base < nB; base += 32) {
    const int j = base + lane;
    const bool own = j >= f0 && j < f1;
    bool kept = j < nB && (own || all);
    const bool score = j < nB && !own && !all && !none;
    const bool tie = score && key[j] == pivot;
    const uint32_t tmask = __ballot_sync(0xFFFFFFFFu, tie);
    if (score && key[j] > pivot) kept = true;
    if (tie && seen + __popc(tmask & ((1u << lane) - 1u)) < ties) kept = true;
    seen += __popc(tmask);
    const uint32_t kmask = __ballot_sync(0xFFFFFFFFu, kept);
    if (kept) out[n + __popc(kmask & ((1u << lane) - 1u))] = j;
    n += __popc(kmask);
  }
  for (int j = n + lane; j < nB; j += 32) out[j] = -1;
  if (lane == 0) cnt[static_cast<size_t>(h) * nB + qb] = n;
}

}  // namespace bsa
