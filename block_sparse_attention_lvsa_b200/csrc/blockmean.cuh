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
// A border between kept and dropped must not depend on rounding: the means and
// the scores that decide are 64-bit.  64-bit scores of every tile would cost
// far more than reading q and k (9.5 ms against 0.2 ms at 1536 blocks and 12
// heads of 128), so they are taken only near the border:
//  1. blockmean_pool_kernel: means in 64 bits, split in two bf16 parts
//     (m = hi + lo + rest, |rest| <= 2^-16 |m|), and their norms; one read of q
//     and k, the HBM bound of the operator.
//  2. blockmean_score_kernel: hi hi + hi lo + lo hi on the tensor cores, off by
//     less than E = 2^-13 |mean q| max_j |mean k_j|: the parts leave out at most
//     3 * 2^-16 sum |q_c k_c|, and 3 d <= 384 additions in 32 bits at most
//     384 * 2^-23 of it, together 9.2e-5 < 2^-13 = 1.22e-4 of |q| |k|.
//  3. blockmean_select_kernel: the take-th largest rough score t of a row is
//     within E of the take-th largest exact one, so a block above t + 2E is
//     kept, one below t - 2E is not, and only those between (a few of 1536)
//     get 64-bit scores.  Rows whose norms leave the range where these bounds
//     hold (32-bit products near the ends of the exponent, values that are not
//     finite) get 64-bit scores throughout.
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
// mean: [2][H][nB][d] double; hi, lo: bf16 [2][H][nB][d]; norm: [2][H][nB] double.
__global__ void __launch_bounds__(kPoolThreads) blockmean_pool_kernel(
    const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k, int N, int H, int d, int nB,
    double* __restrict__ mean, __nv_bfloat16* __restrict__ hi, __nv_bfloat16* __restrict__ lo,
    double* __restrict__ norm) {
  __shared__ double s_sum[kPoolWarps][256];
  __shared__ double s_sq[kPoolWarps];
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
  double m = 0.0;
  if (c < static_cast<int>(row)) {
#pragma unroll
    for (int w = 0; w < kPoolWarps; ++w) m += s_sum[w][threadIdx.x];
    m /= rows;
    const int h = c / d;
    const size_t at = ((static_cast<size_t>(blockIdx.z) * H + h) * nB + b) * d + (c - h * d);
    mean[at] = m;
    const __nv_bfloat16 x = __float2bfloat16(static_cast<float>(m));
    hi[at] = x;
    lo[at] = __float2bfloat16(static_cast<float>(m - static_cast<double>(__bfloat162float(x))));
  }
  double sq = m * m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
  if (lane == 0) s_sq[warp] = sq;
  __syncthreads();
  const int wph = d / 32;                             // warps whose channels form one head
  if (lane == 0 && warp % wph == 0 && c < static_cast<int>(row)) {
    sq = 0.0;
    for (int w = 0; w < wph; ++w) sq += s_sq[warp + w];
    norm[(static_cast<size_t>(blockIdx.z) * H + c / d) * nB + b] = sqrt(sq);
  }
}

constexpr int kScoreThreads = 128;

template <int D>
struct ScoreSmem {
  static constexpr uint32_t kBox = 128 * 128;         // 128 rows x 64 bf16, or 128 rows x 32 floats
  static constexpr uint32_t kTile = (D / 64) * kBox;
  static constexpr uint32_t kQh = 0, kKh = kTile, kKl = 2 * kTile, kQl = 3 * kTile;
  static constexpr uint32_t kBar = 4 * kTile;         // the f32 tile (4 boxes) lies over the operands
  static constexpr uint32_t kHolder = kBar + 32;
  static constexpr uint32_t kAlloc = kHolder + 16 + 1024;
};

// Rough scores of 128 query blocks x 128 key blocks of one head.  hi and lo
// are mapped (d, nB, 2 H): heads of q, then heads of k; scores (nB, nB, heads).
template <int D>
__global__ void __launch_bounds__(kScoreThreads)
blockmean_score_kernel(const __grid_constant__ CUtensorMap tmHi, const __grid_constant__ CUtensorMap tmLo,
                       const __grid_constant__ CUtensorMap tmS, int H, int h0, int nB, long long limit) {
  using L = ScoreSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  volatile uint32_t* holder = reinterpret_cast<volatile uint32_t*>(smem_raw + (base - raw) + L::kHolder);
  auto bar = [&](int i) -> uint32_t { return base + L::kBar + 8u * static_cast<uint32_t>(i); };   // hi, lo loaded; done
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k0 = blockIdx.x * 128, q0 = blockIdx.y * 128, h = h0 + blockIdx.z;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(bar(i), 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(base + L::kHolder, 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *holder;
  bool ok = true;
  if (threadIdx.x == 0) {
    mbar_arrive_expect_tx(bar(0), 2 * L::kTile);
    mbar_arrive_expect_tx(bar(1), 2 * L::kTile);
#pragma unroll
    for (int b = 0; b < D / 64; ++b) {
      tma_load_3d(base + L::kQh + b * L::kBox, &tmHi, bar(0), b * 64, q0, h);
      tma_load_3d(base + L::kKh + b * L::kBox, &tmHi, bar(0), b * 64, k0, H + h);
    }
#pragma unroll
    for (int b = 0; b < D / 64; ++b) {
      tma_load_3d(base + L::kKl + b * L::kBox, &tmLo, bar(1), b * 64, k0, H + h);
      tma_load_3d(base + L::kQl + b * L::kBox, &tmLo, bar(1), b * 64, q0, h);
    }
  }
  if (warp == 1) {
    constexpr uint32_t kIdesc = idesc_bf16_f32(128, 128, false, false);
    const uint32_t a[3] = {L::kQh, L::kQh, L::kQl}, b[3] = {L::kKh, L::kKl, L::kKh};
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      if (t < 2) ok = mbar_wait_warp(bar(t), 0, limit) && ok;
      tc_fence_after();
      const uint64_t da = desc64(sw128_desc(base + a[t], 16, 1024)), db = desc64(sw128_desc(base + b[t], 16, 1024));
#pragma unroll
      for (int g = 0; g < D / 64; ++g)
        if (ok)
          mma4_ss_warp(tbase, da + g * (L::kBox >> 4), db + g * (L::kBox >> 4), kIdesc, (t > 0 || g > 0) ? 1u : 0u);
    }
    tc_commit_warp(bar(2));
  }
  // the copies have landed and the products are done: the operands' room is free
  ok = mbar_wait(bar(0), 0, limit) && mbar_wait(bar(1), 0, limit);
  ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(2), 0, limit) && ok);
  tc_fence_after();
  __syncthreads();
  const int r = threadIdx.x;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    uint32_t v[32];
    tmem_ld_x32(tbase + (static_cast<uint32_t>(32 * warp) << 16) + 32 * b, v);
#pragma unroll
    for (int c = 0; c < 8; ++c)
      st_shared_v4(base + b * L::kBox + r * 128 + ((c ^ (r & 7)) * 16), v[4 * c], v[4 * c + 1], v[4 * c + 2],
                   v[4 * c + 3]);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && ok) {
    for (int b = 0; b < 4; ++b)
      if (k0 + 32 * b < nB) tma_store_3d(&tmS, base + b * L::kBox, k0 + 32 * b, q0, blockIdx.z);
    bulk_commit();
    bulk_wait_read_all();
  }
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tbase, 128);
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

__device__ __forceinline__ float warp_max_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

constexpr int kSelWarps = 4;
constexpr float kRoughError = 1.0f / 8192.0f;         // E / (|q| max |k|), see above

// One warp per row (grid (groups of rows, heads of the pass)).  Lane l holds
// the rough scores of blocks l, l + 32, ... in registers (KPL of them; KPL = 0:
// rows of more than 2048 blocks stay in shared memory).  Shared memory per
// warp: nB 64-bit keys of candidates and, for KPL = 0, nB floats.
template <int D, int KPL>
__global__ void __launch_bounds__(kSelWarps * 32)
blockmean_select_kernel(const double* __restrict__ mean, const double* __restrict__ norm,
                        const float* __restrict__ scores, int ldS, int H, int h0, int nB, int keep, int local,
                        int32_t* __restrict__ idx, int32_t* __restrict__ cnt) {
  extern __shared__ unsigned long long s_mean_keys[];
  __shared__ double s_max[kSelWarps];
  constexpr int E2 = D / 64;                          // double2 of a mean per lane
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wpc = blockDim.x >> 5;
  const int qb = blockIdx.x * wpc + warp, h = h0 + blockIdx.y;
  // largest norm of the head's key means; one that is not finite shows as such
  double kmax = 0.0;
  bool kfin = true;
  for (int j = threadIdx.x; j < nB; j += blockDim.x) {
    const double x = norm[(static_cast<size_t>(H) + h) * nB + j];
    kfin = kfin && isfinite(x);
    kmax = x > kmax ? x : kmax;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double x = __shfl_xor_sync(kAll, kmax, o);
    kmax = x > kmax ? x : kmax;
  }
  if (lane == 0) s_max[warp] = kmax;
  kfin = __syncthreads_and(kfin);
  for (int w = 0; w < wpc; ++w) kmax = s_max[w] > kmax ? s_max[w] : kmax;
  if (qb >= nB) return;

  const size_t per_warp = static_cast<size_t>(nB) + (KPL == 0 ? (nB + 1) / 2 : 0);
  unsigned long long* key = s_mean_keys + warp * per_warp;
  float* srow = reinterpret_cast<float*>(key + nB);
  const double* mq = mean + (static_cast<size_t>(h) * nB + qb) * D;
  const double* mk = mean + (static_cast<size_t>(H) + h) * nB * D;
  const int chunks = KPL ? KPL : (nB + 31) / 32;
  const int f0 = max(0, qb - local), f1 = local < 0 ? f0 : min(nB, qb + local + 1);   // own neighbourhood
  const int forced = f1 - f0, rest = nB - forced;
  const int take = min(nB, max(keep, forced)) - forced;        // blocks chosen by score

  // rough scores; out of the choice: -infinity
  float v[KPL ? KPL : 1];
  float lo = INFINITY, hi = -INFINITY;
  {
    const float* row = scores + (static_cast<size_t>(blockIdx.y) * nB + qb) * ldS;
#pragma unroll
    for (int i = 0; i < chunks; ++i) {
      const int j = i * 32 + lane;
      const bool on = j < nB && (j < f0 || j >= f1);
      const float x = on ? __ldg(row + j) : -INFINITY;
      if (on) lo = fminf(lo, x);
      hi = fmaxf(hi, x);
      if (KPL) v[KPL ? i : 0] = x;
      else if (j < nB) srow[j] = x;
    }
  }
  lo = -warp_max_f(-lo);
  hi = warp_max_f(hi);
  __syncwarp();
  auto score = [&](int i) -> float { return KPL ? v[KPL ? i : 0] : (i * 32 + lane < nB ? srow[i * 32 + lane] : -INFINITY); };
  auto count = [&](float t) -> int {                  // blocks with a rough score >= t > -infinity
    int n = 0;
#pragma unroll
    for (int i = 0; i < chunks; ++i) n += score(i) >= t ? 1 : 0;
    return __reduce_add_sync(kAll, n);
  };

  // sure: kept for certain (> top); candidates: in [bottom, top]
  float bottom = -INFINITY, top = INFINITY;
  const double qn = norm[static_cast<size_t>(h) * nB + qb], scale = qn * kmax;
  const bool choose = take > 0 && take < rest;
  const bool rough = choose && kfin && isfinite(qn) && qn >= 1e-25 && kmax >= 1e-25 && scale >= 1e-25 && scale <= 1e30;
  if (rough) {
    const float e = static_cast<float>(scale) * kRoughError;
    // count(lo) >= take > count(hi): the take-th largest lies in [lo, hi)
    int nlo = rest, nhi = 0;
    hi = hi + fmaxf(e, 1e-6f * fabsf(hi));
    while (nlo - nhi > 1 && hi - lo > e) {
      const float mid = lo + 0.5f * (hi - lo);
      if (!(mid > lo && mid < hi)) break;
      const int n = count(mid);
      if (n >= take) {
        lo = mid;
        nlo = n;
      } else {
        hi = mid;
        nhi = n;
      }
    }
    if (nlo - nhi == 1) {                             // the one score in [lo, hi)
      float t = -INFINITY;
#pragma unroll
      for (int i = 0; i < chunks; ++i) {
        const float x = score(i);
        if (x >= lo && x < hi) t = x;
      }
      lo = hi = warp_max_f(t);
    }
    top = hi + 2.01f * e;
    bottom = lo - 2.01f * e;
  }
  // every block outside the neighbourhood is kept, sure, candidate, or dropped
  int sure = 0, cand = 0;
  if (rough) {
#pragma unroll
    for (int i = 0; i < chunks; ++i) {
      const float x = score(i);
      sure += x > top ? 1 : 0;
      cand += (x >= bottom && x <= top) ? 1 : 0;
    }
    sure = __reduce_add_sync(kAll, sure);
    cand = __reduce_add_sync(kAll, cand);
  } else if (choose) {
    cand = rest;
  }
  const int want = take - sure;                       // candidates to keep
  const bool weigh = choose && want < cand;
  auto is_cand = [&](int i) -> bool {
    const int j = i * 32 + lane;
    if (rough) {
      const float x = score(i);
      return x >= bottom && x <= top;
    }
    return choose && j < nB && (j < f0 || j >= f1);
  };
  // 64-bit scores of the candidates in ascending order; the want-th largest
  // key by bisection, ties to the first
  unsigned long long pivot = 0;
  int ties = cand;
  if (weigh) {
    double2 qv[E2];
#pragma unroll
    for (int u = 0; u < E2; ++u) qv[u] = *reinterpret_cast<const double2*>(mq + u * 64 + 2 * lane);
    unsigned long long kmin = ~0ull, kmx = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < chunks; ++i) {
      uint32_t m = __ballot_sync(kAll, is_cand(i));
      while (m) {
        const int j = i * 32 + __ffs(m) - 1;
        m &= m - 1;
        double s = 0.0;
#pragma unroll
        for (int u = 0; u < E2; ++u) {
          const double2 kv = *reinterpret_cast<const double2*>(mk + static_cast<size_t>(j) * D + u * 64 + 2 * lane);
          s = fma(qv[u].x, kv.x, s);
          s = fma(qv[u].y, kv.y, s);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
        const unsigned long long k = score_key(s);
        kmin = k < kmin ? k : kmin;
        kmx = k > kmx ? k : kmx;
        if (lane == 0) key[at] = k;
        ++at;
      }
    }
    __syncwarp();
    pivot = kmin;
    if (kmx != kmin) {                                // below the bits that all keys share
      const int bits = 63 - __clzll(static_cast<long long>(kmx ^ kmin));
      pivot = kmin >> bits >> 1 << bits << 1;
      for (int bit = bits; bit >= 0; --bit) {
        const unsigned long long c = pivot | (1ull << bit);
        int n = 0;
        for (int u = lane; u < cand; u += 32) n += key[u] >= c ? 1 : 0;
        if (__reduce_add_sync(kAll, n) >= want) pivot = c;
      }
    }
    int above = 0;
    for (int u = lane; u < cand; u += 32) above += key[u] > pivot ? 1 : 0;
    ties = want - __reduce_add_sync(kAll, above);
  }
  int32_t* out = idx + (static_cast<size_t>(h) * nB + qb) * nB;
  int n = 0, at = 0, seen = 0;
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int i = 0; i < chunks; ++i) {
    const int j = i * 32 + lane;
    const bool in = j < nB;
    bool kept = in && ((j >= f0 && j < f1) || (take > 0 && take == rest) || (rough && score(i) > top));
    const bool c = is_cand(i);
    const uint32_t cm = __ballot_sync(kAll, c);
    if (weigh && cm) {
      const unsigned long long k = c ? key[at + __popc(cm & below)] : 0ull;
      const bool tie = c && k == pivot;
      const uint32_t tm = __ballot_sync(kAll, tie);
      kept = kept || (c && k > pivot) || (tie && seen + __popc(tm & below) < ties);
      seen += __popc(tm);
      at += __popc(cm);
    } else if (c) {
      kept = true;
    }
    const uint32_t km = __ballot_sync(kAll, kept);
    if (kept) out[n + __popc(km & below)] = j;
    n += __popc(km);
  }
  for (int j = n + lane; j < nB; j += 32) out[j] = -1;
  if (lane == 0) cnt[static_cast<size_t>(h) * nB + qb] = n;
}

}  // namespace bsa
