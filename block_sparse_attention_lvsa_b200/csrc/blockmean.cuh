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
// The rounding of 32-bit sums must not decide between kept and dropped: the means
// and the scores that decide are 64-bit, a score within 2^-49 |mean q| |mean k| of
// the exact one (up to 4 products and 5 additions a lane and two means, half a
// step of 2^-53 each).  Blocks of equal means have equal scores and go by their
// index; blocks whose scores are closer than that without being the same may be
// ordered by rounding.  64-bit scores of every tile would cost far more than
// reading q and k (9.5 ms against 0.2 ms at 1536 blocks and 12 heads of 128), so
// they are taken only near the border:
//  1. blockmean_pool_kernel: means in 64 bits, split in two bf16 parts
//     (m = hi + lo + rest, |rest| <= 2^-16 |m|), and their norms; one read of q
//     and k, the HBM bound of the operator.
//  2. blockmean_score_kernel: hi hi + hi lo + lo hi on the tensor cores, off by
//     less than E = 2^-13 |mean q| max_j |mean k_j|: the parts leave out at most
//     3 * 2^-16 sum |q_c k_c|, and 3 d <= 384 additions in 32 bits at most
//     384 * 2^-23 of it, together 9.2e-5 < 2^-13 = 1.22e-4 of |q| |k|.  (This
//     takes the tensor cores to lose at most a step of 2^-23 of the magnitudes
//     with each product that they add; measured, sums of 128 products of one sign
//     are low by 2.8 * 2^-24 on average and 7.3 * 2^-24 at most.)
//  3. blockmean_select_kernel: the take-th largest rough score t of a row is
//     within E of the take-th largest exact one, so a block above t + 2E is
//     kept, one below t - 2E is not, and only those between (a few of 1536)
//     get 64-bit scores.  E grows with what all key blocks share, although that
//     changes no ranking: the whole call takes 409 us for 12 heads of 1536 blocks
//     of unrelated tokens, 427, 1,382 and 3,087 us where every key has a common
//     part of norm 3, 10 and 30 (more than kSelKeys candidates: see below).
//     Rows whose norms leave the range where these bounds hold (32-bit products
//     near the ends of the exponent, values that are not finite), and calls with
//     so few blocks that there are no rough scores, get 64-bit scores throughout.
#pragma once
#include "rope.cuh"   // packed pairs of float

namespace bsa {

constexpr int kMeanMaxBlocks = 8192;
constexpr int kPoolWarps = 8;                          // adding warps; one more loads
constexpr int kPoolThreads = 32 * (kPoolWarps + 1);
constexpr int kPoolStages = 3;                         // 32 tokens x 256 channels each
constexpr int kPoolCtas = 3;                           // per SM

struct PoolSmem {
  static constexpr uint32_t kStage = 32 * 512;
  static constexpr uint32_t kSum = kPoolStages * kStage;             // [8 warps][256] double
  static constexpr uint32_t kSq = kSum + kPoolWarps * 256 * 8;       // [8] double
  static constexpr uint32_t kBar = kSq + kPoolWarps * 8;
  static constexpr uint32_t kAlloc = kBar + 2 * kPoolStages * 8 + 128;
};

// Means of 128-token blocks.  A tile is one block of 256 neighbouring channels
// (whole heads) of q or k, in four TMA boxes of 32 tokens; the blocks of the grid
// stride over the tiles, slabs of the same tokens first.  One warp keeps
// kPoolStages boxes in flight (with three blocks an SM 144 KB, against the 43 KB
// that the memory's latency asks for), so that the loads do not wait for the
// adds.  The other warps add 4 tokens of each box, 8 channels a lane, in 64 bits
// in order, then the eight warps' sums in order: bf16 values are 8 bits wide, so
// such a sum is exact unless the block spans more than 2^38, and equal blocks
// always give equal means.
// 225 us under ncu for q and k of 196560 x 12 x 128 (1.21 GB, 5.4 TB/s); the unit
// that converts to 64 bits is 69% busy.  Loads and adds in the same warps: 272 us;
// half of the conversions by moving bits in the integer pipe: 246 us; half of
// them by adding two tokens in 32 bits first, where that is exact: 226 us; four
// adding warps with twice the tokens each: 285 us; two or four blocks an SM: the
// whole call 9 to 14 us slower.
// mean: [2][H][nB][d] double; hi, lo: bf16 [2][H][nB][d]; norm: [2][H][nB] double.
__global__ void __launch_bounds__(kPoolThreads, kPoolCtas) blockmean_pool_kernel(
    const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
    const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k, int N, int H, int d, int nB,
    double* __restrict__ mean, __nv_bfloat16* __restrict__ hi, __nv_bfloat16* __restrict__ lo,
    double* __restrict__ norm, long long limit) {
  using L = PoolSmem;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 127u) & ~127u;
  uint8_t* gbase = smem_raw + (base - raw);
  double* s_sum = reinterpret_cast<double*>(gbase + L::kSum);
  double* s_sq = reinterpret_cast<double*>(gbase + L::kSq);
  auto full = [&](int i) -> uint32_t { return base + L::kBar + 8u * static_cast<uint32_t>(i); };
  auto empty = [&](int i) -> uint32_t { return full(kPoolStages + i); };
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = H * d, slabs = (row + 255) / 256;
  const long long tiles = 2LL * nB * slabs;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPoolStages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), kPoolWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == kPoolWarps) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (long long t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
        const int slab = static_cast<int>(t % slabs);
        const int zb = static_cast<int>(t / slabs), z = zb >= nB, b = zb - z * nB;
        for (int u = 0; u < 4; ++u, ++it) {
          const int slot = it % kPoolStages;
          if (it >= kPoolStages) ok = mbar_wait(empty(slot), (it / kPoolStages - 1) & 1, limit);
          if (!ok) break;
          mbar_arrive_expect_tx(full(slot), L::kStage);
          tma_load_2d(base + slot * L::kStage, z ? &tmK : &tmQ, full(slot), slab * 256, b * 128 + u * 32);
        }
      }
      // wait (bounded) for this thread's own copies still in flight
      for (int u = max(0, it - kPoolStages); u < it; ++u) mbar_wait(full(u % kPoolStages), (u / kPoolStages) & 1, limit);
    }
    return;
  }

  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int slab = static_cast<int>(t % slabs);
    const int zb = static_cast<int>(t / slabs), z = zb >= nB, b = zb - z * nB;
    const int rows = min(128, N - b * 128);
    double acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0;
#pragma unroll 1
    for (int u = 0; u < 4; ++u) {
      if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(full(slot), phase, limit));
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = *reinterpret_cast<const uint4*>(gbase + slot * L::kStage + (warp * 4 + i) * 512 + lane * 16);
      mbar_arrive_after(empty(slot), v[0].x | v[1].x | v[2].x | v[3].x, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          acc[2 * c] += static_cast<double>(__uint_as_float(w[c] << 16));
          acc[2 * c + 1] += static_cast<double>(__uint_as_float(w[c] & 0xFFFF0000u));
        }
      }
      if (++slot == kPoolStages) {
        slot = 0;
        phase ^= 1;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      *reinterpret_cast<double2*>(s_sum + warp * 256 + lane * 8 + i) = make_double2(acc[i], acc[i + 1]);
    named_barrier_sync(1, kPoolWarps * 32);
    const int c = slab * 256 + threadIdx.x;
    double m = 0.0;
    const int h = c / d;
    const size_t at = ((static_cast<size_t>(z) * H + h) * nB + b) * d + (c - h * d);
    if (c < row) {
#pragma unroll
      for (int w = 0; w < kPoolWarps; ++w) m += s_sum[w * 256 + threadIdx.x];
      m = rows == 128 ? m * (1.0 / 128) : m / rows;
      mean[at] = m;
      const __nv_bfloat16 x = __float2bfloat16(static_cast<float>(m));
      hi[at] = x;
      lo[at] = __float2bfloat16(static_cast<float>(m - static_cast<double>(__bfloat162float(x))));
    }
    double sq = m * m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
    if (lane == 0) s_sq[warp] = sq;
    named_barrier_sync(1, kPoolWarps * 32);           // also: the sums have been read
    const int wph = d / 32;                           // warps whose channels form one head
    if (lane == 0 && warp % wph == 0 && c < row) {
      sq = 0.0;
      for (int w = 0; w < wph; ++w) sq += s_sq[warp + w];
      norm[(static_cast<size_t>(z) * H + h) * nB + b] = sqrt(sq);
    }
  }
}

constexpr int kScoreThreads = 256;
constexpr int kScoreTiles = 4;                         // key tiles of a block

template <int D>
struct ScoreSmem {
  static constexpr uint32_t kBox = 128 * 128;         // 128 rows x 64 bf16
  static constexpr uint32_t kTile = (D / 64) * kBox;
  static constexpr uint32_t kQh = 0, kQl = kTile, kRing = 2 * kTile;   // two stages of Kh, Kl
  static constexpr uint32_t kBar = 6 * kTile;
  static constexpr uint32_t kHolder = kBar + 16 * 8;
  static constexpr uint32_t kAlloc = kHolder + 16 + 1024;
};
enum : int { Y_QFULL = 0, Y_KFULL = 1, Y_KEMPTY = 3, Y_SFULL = 5, Y_SFREE = 7, Y_COUNT = 9 };

// 32 bytes, 32-byte aligned
__device__ __forceinline__ void st_global_v8(float* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Rough scores of 128 query blocks x up to kScoreTiles * 128 key blocks of one
// head.  hi and lo are mapped (d, nB, 2 H): heads of q, then heads of k.  The
// query parts are loaded once, the key parts through a ring of two, and the
// accumulators alternate, so that a tile's loads, its products and the stores
// of the one before overlap.  A thread stores whole 32-byte sectors of its own
// row.  57 us under ncu (cold cache) for 12 heads of 1536 x 1536 at d = 128, 21.7
// GFLOP in three products; with one tile a block, staged in shared memory for a
// TMA store, the call took 413 instead of 405 us.
// Warps: 0 TMA, 1 tcgen05.mma, 4..7 stores.
template <int D>
__global__ void __launch_bounds__(kScoreThreads)
blockmean_score_kernel(const __grid_constant__ CUtensorMap tmHi, const __grid_constant__ CUtensorMap tmLo,
                       float* __restrict__ scores, int ldS, int H, int h0, int nB, long long limit) {
  using L = ScoreSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  volatile uint32_t* holder = reinterpret_cast<volatile uint32_t*>(smem_raw + (base - raw) + L::kHolder);
  auto bar = [&](int i) -> uint32_t { return base + L::kBar + 8u * static_cast<uint32_t>(i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = blockIdx.x * kScoreTiles, q0 = blockIdx.y * 128, h = h0 + blockIdx.z;
  const int n = min(kScoreTiles, (nB + 127) / 128 - first);
  if (threadIdx.x == 0) {
    for (int i = 0; i < Y_COUNT; ++i) mbar_init(bar(i), i >= Y_SFREE ? 4 : 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(base + L::kHolder, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *holder;
  if (warp == 0) {
    if (lane == 0) {
      mbar_arrive_expect_tx(bar(Y_QFULL), 2 * L::kTile);
#pragma unroll
      for (int b = 0; b < D / 64; ++b) {
        tma_load_3d(base + L::kQh + b * L::kBox, &tmHi, bar(Y_QFULL), b * 64, q0, h);
        tma_load_3d(base + L::kQl + b * L::kBox, &tmLo, bar(Y_QFULL), b * 64, q0, h);
      }
      int j = 0;
      for (; j < n; ++j) {
        if (j >= 2 && !mbar_wait(bar(Y_KEMPTY + (j & 1)), ((j >> 1) - 1) & 1, limit)) break;
        const uint32_t dst = base + L::kRing + (j & 1) * 2 * L::kTile;
        mbar_arrive_expect_tx(bar(Y_KFULL + (j & 1)), 2 * L::kTile);
#pragma unroll
        for (int b = 0; b < D / 64; ++b) {
          tma_load_3d(dst + b * L::kBox, &tmHi, bar(Y_KFULL + (j & 1)), b * 64, (first + j) * 128, H + h);
          tma_load_3d(dst + L::kTile + b * L::kBox, &tmLo, bar(Y_KFULL + (j & 1)), b * 64, (first + j) * 128, H + h);
        }
      }
      // wait (bounded) for this thread's own copies still in flight
      mbar_wait(bar(Y_QFULL), 0, limit);
      for (int u = max(0, j - 2); u < j; ++u) mbar_wait(bar(Y_KFULL + (u & 1)), (u >> 1) & 1, limit);
    }
  } else if (warp == 1) {
    constexpr uint32_t kIdesc = idesc_bf16_f32(128, 128, false, false);
    bool ok = mbar_wait_warp(bar(Y_QFULL), 0, limit);
    int j = 0;
    for (; ok && j < n; ++j) {
      if (!(ok = mbar_wait_warp(bar(Y_KFULL + (j & 1)), (j >> 1) & 1, limit))) break;
      if (j >= 2 && !(ok = mbar_wait_warp(bar(Y_SFREE + (j & 1)), ((j >> 1) - 1) & 1, limit))) break;
      tc_fence_after();
      const uint32_t k = base + L::kRing + (j & 1) * 2 * L::kTile;
      const uint32_t a[3] = {base + L::kQh, base + L::kQh, base + L::kQl}, b[3] = {k, k + L::kTile, k};
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        const uint64_t da = desc64(sw128_desc(a[t], 16, 1024)), db = desc64(sw128_desc(b[t], 16, 1024));
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
          mma4_ss_warp(tbase + (j & 1) * 128, da + g * (L::kBox >> 4), db + g * (L::kBox >> 4), kIdesc,
                       (t > 0 || g > 0) ? 1u : 0u);
      }
      tc_commit2_warp(bar(Y_SFULL + (j & 1)), bar(Y_KEMPTY + (j & 1)));
    }
    // the products have completed before TMEM may be released
    if (j > 0) mbar_wait_warp(bar(Y_SFULL + ((j - 1) & 1)), ((j - 1) >> 1) & 1, limit);
  } else if (warp >= 4) {
    const int q = q0 + threadIdx.x - 128;
    const uint32_t tS = tbase + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    float* row = scores + (static_cast<size_t>(blockIdx.z) * nB + q) * ldS;
    for (int j = 0; j < n; ++j) {
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(bar(Y_SFULL + (j & 1)), (j >> 1) & 1, limit))) break;
      tc_fence_after();
      const int k0 = (first + j) * 128;
#pragma unroll
      for (int c = 0; c < 128; c += 32) {
        uint32_t v[32];
        tmem_ld_x32(tS + (j & 1) * 128 + c, v);
#pragma unroll
        for (int u = 0; u < 32; u += 8)
          if (q < nB && k0 + c + u < ldS) st_global_v8(row + k0 + c + u, v + u);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Y_SFREE + (j & 1)));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tbase, 256);
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

// warps (rows) per block; four long rows fill shared memory
__host__ __device__ constexpr int sel_warps(int c4) { return c4 ? 8 : 4; }
constexpr int kSelKeys = 32;
__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
constexpr float kRoughError = 1.0f / 8192.0f;         // E / (|q| max |k|), see above

// One warp per row (grid (groups of rows, heads of the pass)).  Block j sits
// in lane (j % 128) / 4, component j % 4 of chunk j / 128, so that a lane reads
// four neighbouring scores at once; C4 chunks are kept in registers, because
// the bisection reads them again and again (C4 = 0: rows of more than 2048
// blocks, in shared memory).  One pass then turns the scores into a bit per
// block (sure, candidate; 8 chunks a word); what follows loops over those words:
// code that is unrolled over the row more often does not fit the instruction
// cache (640 against 305 us for 12 x 1536 rows of 1536 blocks; 130 us as it is,
// half of it issue slots, the rest waits for the few 64-bit means).  A few candidates are ranked directly, a lane each; more than kSelKeys
// (rows of equal scores) by bisection over their keys, which then lie in memory
// that is the row's own: the rough scores, no longer needed, and the output
// list, not yet written.
template <int D, int C4>
__global__ void __launch_bounds__(sel_warps(C4) * 32)
blockmean_select_kernel(const double* __restrict__ mean, const double* __restrict__ norm,
                        float* scores, int ldS, int H, int h0, int nB, int keep, int local, int32_t* idx,
                        int32_t* __restrict__ cnt) {
  extern __shared__ float4 s_rows[];
  constexpr int kW = sel_warps(C4);
  constexpr int kWords = C4 ? (C4 + 7) / 8 : kMeanMaxBlocks / 1024;
  __shared__ uint32_t s_sure[kW][kWords][32], s_cand[kW][kWords][32];
  __shared__ unsigned long long s_key[kW][kSelKeys];
  __shared__ int s_at[kW][kSelKeys];
  __shared__ uint32_t s_max[kW];
  constexpr int E2 = D / 64;                          // double2 of a mean per lane
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int qb = blockIdx.x * kW + warp, h = h0 + blockIdx.y;
  // an upper bound of the head's key norms: the upper words of non-negative
  // 64-bit floats order like them (not finite: above all others), plus one step
  uint32_t top_word = 0;
  const uint32_t* kn = reinterpret_cast<const uint32_t*>(norm + (static_cast<size_t>(H) + h) * nB);
  for (int j = threadIdx.x; j < nB; j += kW * 32) top_word = max(top_word, kn[2 * j + 1]);
  top_word = __reduce_max_sync(kAll, top_word);
  if (lane == 0) s_max[warp] = top_word;
  __syncthreads();
  if (qb >= nB) return;
  for (int w = 0; w < kW; ++w) top_word = max(top_word, s_max[w]);
  const bool kfin = top_word < 0x7FE00000u;
  const double kmax = __hiloint2double(static_cast<int>(top_word + 1), 0);

  float4* srow = s_rows + static_cast<size_t>(warp) * (ldS / 4);
  float* row = scores + (static_cast<size_t>(blockIdx.y) * nB + qb) * ldS;
  int32_t* out = idx + (static_cast<size_t>(h) * nB + qb) * nB;
  uint32_t(*sure)[32] = s_sure[warp];
  uint32_t(*cand)[32] = s_cand[warp];
  const double* mq = mean + (static_cast<size_t>(h) * nB + qb) * D;
  const double* mk = mean + (static_cast<size_t>(H) + h) * nB * D;
  const int used = (nB + 127) / 128;                  // chunks
  const int chunks = C4 ? C4 : used;
  const int words = (used + 7) / 8;
  const int f0 = max(0, qb - local), f1 = local < 0 ? f0 : min(nB, qb + local + 1);   // own neighbourhood
  const int forced = f1 - f0, rest = nB - forced;
  const int take = min(nB, max(keep, forced)) - forced;        // blocks chosen by score
  const double qn = norm[static_cast<size_t>(h) * nB + qb], scale = qn * kmax;
  const bool choose = take > 0 && take < rest;
  const bool rough = choose && scores != nullptr && kfin && isfinite(qn) && qn >= 1e-25 && kmax >= 1e-25 && scale >= 1e-25 && scale <= 1e30;
  auto own = [&](int j) -> bool { return j >= f0 && j < f1; };
  // chunk i holds blocks that take no part in the choice
  auto mixed = [&](int i) -> bool { return 128 * i + 128 > nB || (128 * i + 128 > f0 && 128 * i < f1); };

  if (rough) {
    // rough scores; out of the choice: -infinity.  Their extremes, and mean and
    // deviation from one of them (which keeps the digits of close scores)
    float4 v[C4 ? C4 : 1];
    float lo = INFINITY, hi = -INFINITY;
    const float x0 = __ldcg(row + (f0 > 0 ? 0 : f1));
    const uint64_t nx0 = f2pack(-x0, -x0);
    uint64_t s1 = f2pack(0.f, 0.f), s2 = s1;
#pragma unroll
    for (int i = 0; i < chunks; ++i) {
      const int j = 128 * i + 4 * lane;
      float4 x = make_float4(x0, x0, x0, x0);
      if (j < nB) x = __ldcg(reinterpret_cast<const float4*>(row + j));
      if (mixed(i)) {                                 // blocks that do not count stand at x0 for a moment
        const bool a = j >= nB || own(j), b = j + 1 >= nB || own(j + 1), c = j + 2 >= nB || own(j + 2),
                   e = j + 3 >= nB || own(j + 3);
        x = make_float4(a ? x0 : x.x, b ? x0 : x.y, c ? x0 : x.z, e ? x0 : x.w);
      }
      lo = fminf(lo, fminf(fminf(x.x, x.y), fminf(x.z, x.w)));
      hi = fmaxf(hi, fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)));
      const uint64_t d0 = fadd2(f2pack(x.x, x.y), nx0), d1 = fadd2(f2pack(x.z, x.w), nx0);
      s1 = fadd2(s1, fadd2(d0, d1));
      s2 = ffma2(d1, d1, ffma2(d0, d0, s2));
      if (mixed(i)) {
        const bool a = j >= nB || own(j), b = j + 1 >= nB || own(j + 1), c = j + 2 >= nB || own(j + 2),
                   e = j + 3 >= nB || own(j + 3);
        x = make_float4(a ? -INFINITY : x.x, b ? -INFINITY : x.y, c ? -INFINITY : x.z, e ? -INFINITY : x.w);
      }
      if (C4) v[C4 ? i : 0] = x;
      else if (j < nB) srow[j / 4] = x;
    }
    lo = -warp_max_f(-lo);
    hi = warp_max_f(hi);
    const float mean_d = warp_sum_f(f2sum(s1)) / rest;
    const float sd = sqrtf(fmaxf(warp_sum_f(f2sum(s2)) / rest - mean_d * mean_d, 0.f));
    __syncwarp();
    auto score = [&](int i) -> float4 {
      if (C4) return v[C4 ? i : 0];
      if (128 * i + 4 * lane < nB) return srow[32 * i + lane];
      return make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    };
    // blocks with a score >= t: all positions less those whose difference has
    // its sign bit set (one packed subtraction and an add for each)
    auto count = [&](float t) -> int {
      const uint64_t nt = f2pack(-t, -t);
      uint32_t below = 0;
#pragma unroll
      for (int i = 0; i < chunks; ++i) {
        const float4 x = score(i);
        float a, b, c, e;
        f2unpack(fadd2(f2pack(x.x, x.y), nt), a, b);
        f2unpack(fadd2(f2pack(x.z, x.w), nt), c, e);
        below += __float_as_uint(a) >> 31;
        below += __float_as_uint(b) >> 31;
        below += __float_as_uint(c) >> 31;
        below += __float_as_uint(e) >> 31;
      }
      return 128 * chunks - static_cast<int>(__reduce_add_sync(kAll, below));
    };
    const float e = static_cast<float>(scale) * kRoughError;
    // count(lo) >= take > count(hi): the take-th largest lies in [lo, hi).  The
    // first steps go where a normal distribution of the row's mean and deviation
    // would put it, each then by the density there and a little beyond; later
    // ones by the counts' proportion, every third in the middle.  (6 steps on
    // average over normal rows of 1536, where halving takes 12.)
    int nlo = rest, nhi = 0;
    hi = hi + fmaxf(e, 1e-6f * fabsf(hi));
    float z = normcdfinvf(1.f - static_cast<float>(take) / rest);
    for (int step = 0; nlo - nhi > 1 && hi - lo > e; ++step) {
      const float mean_x = x0 + mean_d;
      float mid = fmaf(z, sd, mean_x);
      if (step > 5 || !(mid > lo && mid < hi)) {
        const float part = step % 3 == 2 ? 0.5f : (nlo - take + 0.5f) / (nlo - nhi);
        mid = lo + fminf(fmaxf(part, 0.02f), 0.98f) * (hi - lo);
      }
      if (!(mid > lo && mid < hi)) break;
      const int n = count(mid);
      if (n >= take) {
        lo = mid;
        nlo = n;
      } else {
        hi = mid;
        nhi = n;
      }
      if (step <= 5) {
        const float miss = static_cast<float>(n - take);            // > 0: the threshold is higher
        const float zz = (mid - mean_x) / sd;
        const float density = rest * 0.3989423f * __expf(-0.5f * zz * zz);
        z = zz + (miss + (miss >= 0.f ? 1.f : -1.f) * fmaf(0.05f, fabsf(miss), 1.f)) / density;
      }
    }
    // the take-th largest rough score is within [lo, hi), the exact one within
    // E of it
    const float top = hi + 2.01f * e, bottom = lo - 2.01f * e;
    uint32_t sm = 0, cm = 0;
#pragma unroll
    for (int i = 0; i < chunks; ++i) {
      const float4 x = score(i);
      const int b = 4 * (i & 7);
      sm |= (x.x > top ? 1u << b : 0u) | (x.y > top ? 2u << b : 0u) | (x.z > top ? 4u << b : 0u) | (x.w > top ? 8u << b : 0u);
      cm |= (x.x >= bottom ? 1u << b : 0u) | (x.y >= bottom ? 2u << b : 0u) | (x.z >= bottom ? 4u << b : 0u) |
            (x.w >= bottom ? 8u << b : 0u);
      if ((i & 7) == 7 || i == chunks - 1) {
        sure[i >> 3][lane] = sm;
        cand[i >> 3][lane] = cm & ~sm;
        sm = cm = 0;
      }
    }
  } else {
    // no rough scores: nothing is sure; when there is a choice every block
    // outside the neighbourhood is weighed
    for (int w = 0; w < words; ++w) {
      uint32_t cm = 0;
      for (int b = 0; b < 32; ++b) {
        const int j = 128 * (8 * w + b / 4) + 4 * lane + b % 4;
        if (choose && j < nB && !own(j)) cm |= 1u << b;
      }
      sure[w][lane] = 0u;
      cand[w][lane] = cm;
    }
  }
  __syncwarp();
  const bool all = take == rest;                      // (with forced blocks: every block)
  if (choose) {
    int n_sure = 0, n_cand = 0;
    for (int w = 0; w < words; ++w) {
      n_sure += __popc(sure[w][lane]);
      n_cand += __popc(cand[w][lane]);
    }
    n_sure = __reduce_add_sync(kAll, n_sure);
    n_cand = __reduce_add_sync(kAll, n_cand);
    const int want = take - n_sure;                   // candidates to keep
    const bool few = n_cand <= kSelKeys;
    if (want == n_cand) {
      for (int w = 0; w < words; ++w) sure[w][lane] |= cand[w][lane];
    } else {
      // 64-bit scores of the candidates
      double2 qv[E2];
#pragma unroll
      for (int u = 0; u < E2; ++u) qv[u] = *reinterpret_cast<const double2*>(mq + u * 64 + 2 * lane);
      int at = 0;
#pragma unroll 1
      for (int w = 0; w < words; ++w) {
        const uint32_t mine = cand[w][lane];
        for (uint32_t lanes = __ballot_sync(kAll, mine != 0u); lanes; lanes &= lanes - 1) {
          const int src = __ffs(lanes) - 1;
          for (uint32_t m = __shfl_sync(kAll, mine, src); m; m &= m - 1) {
            const int b = __ffs(m) - 1;
            const int j = 128 * (8 * w + (b >> 2)) + 4 * src + (b & 3);
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
            if (lane == 0) {
              if (few) {
                s_key[warp][at] = k;
                s_at[warp][at] = j;
              } else {
                __stcg(out + j, static_cast<int32_t>(k >> 32));
                __stcg(row + j, __uint_as_float(static_cast<uint32_t>(k)));
              }
            }
            ++at;
          }
        }
      }
      __syncwarp();
      auto keep_block = [&](int j) {
        atomicOr(&sure[j >> 10][(j >> 2) & 31], 1u << (4 * ((j >> 7) & 7) + (j & 3)));
      };
      if (few) {
        // a lane's candidate is kept if fewer than `want` come before it
        const unsigned long long k = lane < n_cand ? s_key[warp][lane] : 0ull;
        const int j = lane < n_cand ? s_at[warp][lane] : 0;
        int before = 0;
        for (int u = 0; u < n_cand; ++u) {
          const unsigned long long ku = s_key[warp][u];
          before += (ku > k || (ku == k && s_at[warp][u] < j)) ? 1 : 0;
        }
        if (lane < n_cand && before < want) keep_block(j);
      } else {
        // bisection over the 64 bits of the want-th largest key, then over the
        // position of the last tie that is kept
        auto key = [&](int j) -> unsigned long long {
          return static_cast<unsigned long long>(static_cast<uint32_t>(__ldcg(out + j))) << 32 |
                 __float_as_uint(__ldcg(row + j));
        };
        auto is_cand = [&](int j) -> bool {
          return (cand[j >> 10][(j >> 2) & 31] >> (4 * ((j >> 7) & 7) + (j & 3))) & 1u;
        };
        unsigned long long pivot = 0;
#pragma unroll 1
        for (int bit = 63; bit >= 0; --bit) {
          const unsigned long long c = pivot | (1ull << bit);
          int n = 0;
          for (int j = lane; j < nB; j += 32) n += is_cand(j) && key(j) >= c ? 1 : 0;
          if (__reduce_add_sync(kAll, n) >= want) pivot = c;
        }
        int above = 0;
        for (int j = lane; j < nB; j += 32) above += is_cand(j) && key(j) > pivot ? 1 : 0;
        const int ties = want - __reduce_add_sync(kAll, above);
        int last = nB - 1;                            // smallest j with enough ties up to it
        for (int lo_j = 0; lo_j < last;) {
          const int mid = (lo_j + last) / 2;
          int n = 0;
          for (int j = lane; j <= mid; j += 32) n += is_cand(j) && key(j) == pivot ? 1 : 0;
          if (__reduce_add_sync(kAll, n) >= ties) last = mid;
          else lo_j = mid + 1;
        }
        for (int j = lane; j < nB; j += 32) {
          if (!is_cand(j)) continue;
          const unsigned long long k = key(j);
          if (k > pivot || (k == pivot && j <= last)) keep_block(j);
        }
      }
    }
    __syncwarp();
  }
  // kept blocks in ascending order, -1 behind them
  const uint32_t below = (1u << lane) - 1u;
  int n = 0;
#pragma unroll 2
  for (int i = 0; i < used; ++i) {
    const int j = 128 * i + 4 * lane;
    uint32_t bits = all ? 15u : (sure[i >> 3][lane] >> (4 * (i & 7))) & 15u;
    if (mixed(i)) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (own(j + c)) bits |= 1u << c;
        if (j + c >= nB) bits &= ~(1u << c);
      }
    }
    const int own_count = __popc(bits);
    const uint32_t b0 = __ballot_sync(kAll, own_count & 1), b1 = __ballot_sync(kAll, own_count & 2),
                   b2 = __ballot_sync(kAll, own_count & 4);
    int32_t* p = out + n + __popc(b0 & below) + 2 * __popc(b1 & below) + 4 * __popc(b2 & below);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (bits & (1u << c)) *p++ = j + c;
    n += __popc(b0) + 2 * __popc(b1) + 4 * __popc(b2);
  }
  if (nB % 4 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0) {
    const int a = min(nB, (n + 3) & ~3);
    if (n + lane < a) out[n + lane] = -1;
    for (int j = a + 4 * lane; j < nB; j += 128) *reinterpret_cast<int4*>(out + j) = make_int4(-1, -1, -1, -1);
  } else {
    for (int j = n + lane; j < nB; j += 32) out[j] = -1;
  }
  if (lane == 0) cnt[static_cast<size_t>(h) * nB + qb] = n;
}

}  // namespace bsa
