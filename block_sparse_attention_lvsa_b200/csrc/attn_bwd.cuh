// attn_bwd.cuh - gradient of the block-sparse softmax attention on sm_100a
// tensor cores (tcgen05 + TMEM + TMA).
//
// With s = scale <q, k>, p = exp(s - lse) the forward's probabilities and
// D_q = <do_q, o_q> = sum_k p <do_q, v_k> (the second form for rows of few keys):
//   dv_k = sum_q p do_q
//   ds   = p (<do_q, v_k> - D_q)
//   dq_q = scale sum_k ds k_k,     dk_k = scale sum_q ds q_q
// over the pairs that the index admits.  lse comes from the forward, so a
// tile needs no running maximum and tiles can be taken in any grouping.
//
// Two kinds of CTA in one launch, each with every sum of its outputs inside the
// CTA (no atomics: the result does not change from run to run), at the price of
// forming s and <do, v> twice (7 products of 128 x 128 x d a tile instead of 5):
//   bwd_dkv  one CTA per 128-key tile and head, over the query
//     tiles that list it (the index transposed on the device).  Tiles are
//     held transposed, S^T = K Q^T and dP^T = V dO^T, so that P^T and dS^T
//     (bf16, in TMEM) are the A operands of dV += P^T dO and dK += dS^T Q and
//     never touch shared memory.  TMEM is full (S, dP, dV, dK, 128 columns
//     each at d = 128): P and dS both lie over dP, so that S is free again as
//     soon as its scores are in registers and the next tile's S runs during
//     the exponentials.
//   bwd_dq   one CTA per 128-query tile and head, over its own
//     list: S = Q K^T, dP = dO V^T, dQ += dS K.
//
// Warp roles (640 threads):
//   warp 0         TMA producer          warp 1   tcgen05.mma issuer
//   warps 4..19    four groups of 4 warps; group g turns columns
//                  32 g .. 32 g + 31 of every tile, thread = TMEM lane = row
// What a thread does with a tile (read S, 32 exponentials, read dP, form ds,
// write P and dS) is a chain of latencies; with two groups of 64 columns it
// took ~3,300 cycles a tile against 2,048 of tensor work (clock trace), with
// four groups the chains are half as long and twice as many overlap.
// setmaxnreg gives the groups 104 registers a thread and the other warps 56.
//   tensor order, dkv:  S(i+1), dV(i), dK(i), dP(i+1)
//                 dq:   dP(j+1), dQ(j), S(j+2)
// P and dS are rounded to bf16 for the products (half a step, at most 2^-8
// of each term, as P is in the forward); all sums are 32-bit.  Each group
// writes over its own columns, so the groups never wait for one another.
#pragma once
#include "rope.cuh"   // fmul2
#include "attn_fwd.cuh"

namespace bsa {

struct BwdParams {
  int N, H, nB;
  float sl2;                        // scale * log2(e)
  float scale;
  // dq: key-tile lists of the query tiles (see AttnParams)
  const int32_t* list;
  const int32_t* count;
  const uint8_t* flags;
  long long lhs;
  int lrs, chs;
  // dkv: bit sets of the lists [heads or 1][nW][nB] (part: null without flags)
  // and room for the query-tile lists of the key tiles [H][nB][nB]
  const uint32_t* bits;
  const uint32_t* part;
  long long bhs;                    // head stride of the bit sets (0: shared by all heads)
  int32_t* tlist;
  // element mask (LVSA)
  const uint32_t* fbits;
  int TW, P;
  // per (head, token), padded to nB * 128: -lse * log2(e) (-inf: no key) and -D
  const float* nl;
  const float* nd;
  long long wait_limit_ns;
};

constexpr int kBwdGroups = 4;                      // of 128 threads
constexpr int kBwdCols = 128 / kBwdGroups;         // columns of a tile per group
constexpr int kBwdThreads = 128 + 128 * kBwdGroups;
// launched with at most 96 registers a thread (640 x 96 = 61,440)
constexpr int kBwdRegsLow = 56, kBwdRegsHigh = 104;
static_assert(kBwdRegsLow * 128 + kBwdRegsHigh * 128 * kBwdGroups <= 96 * kBwdThreads, "register split");
constexpr int kPartialBit = 1 << 30;

// D[tmem] (+)= A[tmem] * B[smem] for two consecutive K-steps of 16 (see
// mma4_ts_warp).
__device__ __forceinline__ void mma2_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                             uint32_t accumulate_first) {
  asm volatile(
      "{\n\t.reg .pred e, p, t;\n\t.reg .b64 b1;\n\t.reg .b32 a1;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 t, %5, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.u32 a1, %1, 8;\n\tadd.s64 b1, %2, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, t;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate_first), "r"(1u)
      : "memory");
}
// 16 consecutive columns of the thread's TMEM lane, complete on return
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr) : "memory");
}
// 16 columns written and complete on return
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n\t"
               "tcgen05.wait::st.sync.aligned;"
               :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]) : "memory");
}

// untiled copy global -> shared (16-byte aligned addresses and size), completes on `bar`
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint32_t bits32(int a, int b) {          // bits a .. b - 1, 0 <= a < b <= 32
  return (b - a == 32 ? 0xFFFFFFFFu : (1u << (b - a)) - 1u) << a;
}
__device__ __forceinline__ bool frame_bit(const BwdParams& p, int fq, int fk) {
  return (__ldg(p.fbits + static_cast<size_t>(fq) * p.TW + (fk >> 5)) >> (fk & 31)) & 1u;
}
// Element mask of 32 query columns for key frame fk: bit c set iff query q0+c
// < N may attend it.
__device__ __forceinline__ uint32_t query_mask(const BwdParams& p, int fk, int q0) {
  uint32_t m = 0u;
  const int qend = min(q0 + kBwdCols, p.N);
  for (int f = q0 / p.P; f * p.P < qend; ++f)
    if (frame_bit(p, f, fk)) m |= bits32(max(f * p.P, q0) - q0, min((f + 1) * p.P, qend) - q0);
  return m;
}
// Element mask of 32 key columns for query frame fq (no frames: every key < N).
__device__ __forceinline__ uint32_t key_mask(const BwdParams& p, int fq, int k0) {
  uint32_t m = 0u;
  const int kend = min(k0 + kBwdCols, p.N);
  if (p.fbits == nullptr) return k0 < kend ? bits32(0, kend - k0) : 0u;
  for (int f = k0 / p.P; f * p.P < kend; ++f)
    if (frame_bit(p, fq, f)) m |= bits32(max(f * p.P, k0) - k0, min((f + 1) * p.P, kend) - k0);
  return m;
}

// Rows of few keys.  <do, o> with o rounded to bf16 is off by up to 2^-8 of
// sum |do| |o|, next to differences <do, v_k> - D that, with two or three keys,
// can all be small: dq and dk of 2 tokens were off by up to 6e-2 of their norm.
// Up to kFewKeys keys D is therefore formed anew in 32 bits,
//   D = sum p <do, v_k> / sum p,
// from which the sum of ds over the row vanishes as it should, whatever factor
// lse is off by (its 32 bits leave 2^-22 |lse| of the exponent: p of a row with
// scores near 8,000 sums to 1 only within 4e-3).  The rounding of o averages out
// over the keys: with 32 or more it adds less to the error of the gradients
// (3.1e-3 to 3.6e-3 of their norm with 16 keys, 2.6e-3 to 3.0e-3 with 64) than
// the rounding of p and ds (2.4e-3).
// That D is right only where o and lse are of this list, not of one with more
// keys.  They are taken to be where it is as near to <do, o> as o's rounding and
// that of the forward's p leave it,
//   |D - <do, o>| <= 2^-8 (<|do|, |o|> + sum p <|do|, |v_k|>)
// (and an eighth more for the 32-bit sums): rows of the forward's own list meet
// that whatever the factor is (tested up to scores of 8,000), and where another
// row meets it the one D is as good as the other.  The sum of p does not tell them
// apart: with |sum p - 1| <= 2^-12 most rows at scores of 2,000 were missed.
// A row of one key has p = 1 and ds = 0 whatever dP is; where such rows can fill
// the input (`ones`: frames of one token, a last block of one key) they get the
// mark kOneKey in place of -D, a NaN that no arithmetic gives, at which ds is set
// to 0.  Elsewhere the check would cost 5% (947 against 889 us, 161 blocks, 12
// heads, d = 128).
constexpr int kFewKeys = 32;
constexpr uint32_t kOneKey = 0x7FC00001u;
// What it costs the whole gradient: 10.6 -> 16.6 us where every row has 32 keys
// (32 tokens, 6 heads, d = 128; 20.8 with 8 keys in flight, and blocks of 256
// threads leave SMs idle), 36.7 -> 38.4 us where a short last block only may make
// such rows (4,104 tokens); nothing where the sizes exclude them.
constexpr int prep_threads(bool few) { return few ? 64 : 256; }

// The keys of query n of head h by its list, if there are 1 to kFewKeys, into
// `keys`: their number, or 0.  Called by a group of G lanes (mask `gm`, lane l
// of it): lanes 0..3 take 32 columns of a tile each.
template <int G>
__device__ __forceinline__ int few_keys(const BwdParams& p, int n, int h, unsigned gm, int l, int32_t* keys) {
  const int qt = n >> 7;
  const int m = min(max(p.count[static_cast<size_t>(h) * p.chs + qt], 0), p.lrs);
  const size_t off = static_cast<size_t>(h) * p.lhs + static_cast<size_t>(qt) * p.lrs;
  const int fq = p.fbits != nullptr ? n / p.P : 0;
  int total = 0;
  for (int j = 0; j < m; ++j) {
    const int kt = p.list[off + j];
    if (kt < 0 || kt >= p.nB) continue;
    const int k0 = kt * 128 + 32 * l;
    uint32_t w = 0u;
    if (l < 4 && k0 < p.N) {
      // a tile that is not partial holds 128 keys
      const bool part = p.flags != nullptr ? p.flags[off + j] != 0 : kt * 128 + 128 > p.N;
      w = part ? key_mask(p, fq, k0) : 0xFFFFFFFFu;
    }
    const int c = __popc(w);
    int before = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ci = __shfl_sync(gm, c, i, G);
      before += i < l ? ci : 0;
      sum += ci;
    }
    if (total + sum > kFewKeys) return 0;
    for (int at = total + before; w != 0u; w &= w - 1u) keys[at++] = k0 + __ffs(w) - 1;
    total += sum;
  }
  __syncwarp(gm);
  return total;
}

// a 16-byte load that stays where the call stands (several in flight)
__device__ __forceinline__ uint4 ld_pinned_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
constexpr float kRoundedO = 1.125f / 256.f;        // 2^-8 and an eighth
// <|x|, |y|> over 8 channels in bf16
__device__ __forceinline__ float abs_dot8(const uint4& a, const uint4& b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum = fmaf(fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(y[i] << 16)), sum);
    sum = fmaf(fabsf(__uint_as_float(x[i] & 0xFFFF0000u)), fabsf(__uint_as_float(y[i] & 0xFFFF0000u)), sum);
  }
  return sum;
}
// <x, y> over 8 channels in bf16
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float sum) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), sum);
    sum = fmaf(__uint_as_float(x[i] & 0xFFFF0000u), __uint_as_float(y[i] & 0xFFFF0000u), sum);
  }
  return sum;
}

// Two independent preparations in one launch, 256 threads a block (FEW: 64).
// Blocks below `bit_blocks`: bit sets of the rows' lists, bits[h][w][qb] bit b =
// key tile 32 w + b is listed by query tile qb, and the same of the partial
// ones.  One warp per row; 8192 tiles at a time in shared memory.  Entries out
// of range are skipped and, like repeated ones, reported.
// The others: nl = -lse * log2(e) and nd = -D per (head, token),
// [H][nB * 128]; tokens past N and rows without a key get nl = -inf (p = 0);
// d/8 lanes a row.  FEW: rows of at most kFewKeys keys may occur.
template <int D, bool FEW>
__global__ void __launch_bounds__(prep_threads(FEW)) attn_bwd_prep_kernel(
    const int32_t* __restrict__ list, const int32_t* __restrict__ count, const uint8_t* __restrict__ flags,
    long long lhs, int lrs, int chs, int nB, int list_heads, unsigned bit_blocks, uint32_t* __restrict__ bits,
    uint32_t* __restrict__ part, const __nv_bfloat16* __restrict__ o, long long o_ts, long long o_hs,
    const __nv_bfloat16* __restrict__ go, const float* __restrict__ lse, int N, int H, float* __restrict__ nl,
    float* __restrict__ nd, bool ones, const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ k,
    const __nv_bfloat16* __restrict__ v, const BwdParams p) {
  constexpr int kWords = 256;
  constexpr int kThreads = prep_threads(FEW), kWarps = kThreads / 32;
  __shared__ uint32_t s_on[kWarps][kWords], s_part[kWarps][kWords];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x < bit_blocks) {
    const long long row = static_cast<long long>(blockIdx.x) * kWarps + warp;              // h * nB + query tile
    if (row >= static_cast<long long>(list_heads) * nB) return;
    const int h = static_cast<int>(row / nB), qb = static_cast<int>(row - static_cast<long long>(h) * nB);
    const int nW = (nB + 31) / 32;
    int n = count[static_cast<size_t>(h) * chs + qb];
    bool bad = n < 0 || n > lrs;
    n = min(max(n, 0), lrs);
    const size_t off = static_cast<size_t>(h) * lhs + static_cast<size_t>(qb) * lrs;
    for (int w0 = 0; w0 < nW; w0 += kWords) {
      const int words = min(kWords, nW - w0);
      for (int w = lane; w < words; w += 32) s_on[warp][w] = s_part[warp][w] = 0u;
      __syncwarp();
      for (int j = lane; j < n; j += 32) {
        const int kt = list[off + j];
        if (kt < 0 || kt >= nB) {
          bad = true;
          continue;
        }
        const int w = (kt >> 5) - w0;
        if (w < 0 || w >= words) continue;
        const uint32_t b = 1u << (kt & 31);
        if (atomicOr(&s_on[warp][w], b) & b) bad = true;
        if (flags != nullptr && flags[off + j]) atomicOr(&s_part[warp][w], b);
      }
      __syncwarp();
      for (int w = lane; w < words; w += 32) {
        const size_t at = (static_cast<size_t>(h) * nW + w0 + w) * nB + qb;
        bits[at] = s_on[warp][w];
        if (part != nullptr) part[at] = s_part[warp][w];
      }
      __syncwarp();
    }
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) set_status(BSA_ERR_INDEX_RANGE);
    return;
  }
  constexpr int G = D / 8;
  const int NP = nB * 128;
  const long long row = (static_cast<long long>(blockIdx.x - bit_blocks) * kThreads + threadIdx.x) / G;   // n * H + h
  const int l = threadIdx.x % G;
  const int n = static_cast<int>(row / H);
  const int h = static_cast<int>(row - static_cast<long long>(n) * H);
  const bool on = n < N;
  uint4 g = make_uint4(0u, 0u, 0u, 0u);
  float sum = 0.f, size = 0.f;                        // size: <|do|, |o|> + sum p <|do|, |v_k|>, of the lane's channels
  if (on) {
    g = __ldg(reinterpret_cast<const uint4*>(go + row * D + 8 * l));
    const uint4 ov = __ldg(reinterpret_cast<const uint4*>(o + n * o_ts + h * o_hs + 8 * l));
    sum = dot8(ov, g, 0.f);
    if (FEW) size = abs_dot8(ov, g);
  }
#pragma unroll
  for (int s = G / 2; s > 0; s >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
  const float e = on ? lse[static_cast<size_t>(h) * N + n] : -INFINITY;
  const float nle = (e == -INFINITY) ? -INFINITY : -e * 1.4426950408889634f;
  bool one = false;
  if constexpr (FEW) {
    __shared__ int32_t s_keys[kThreads / G][kFewKeys];
    const unsigned gm = ((1u << G) - 1u) << (lane & ~(G - 1));
    int32_t* keys = s_keys[threadIdx.x / G];
    const int t = on ? few_keys<G>(p, n, h, gm, l, keys) : 0;
    if (t > 0) {
      const uint4 qr = __ldg(reinterpret_cast<const uint4*>(q + row * D + 8 * l));
      float all = 0.f, acc = 0.f;
      constexpr int kBatch = 4;                     // keys in flight
      for (int j0 = 0; j0 < t; j0 += kBatch) {
        uint4 kr[kBatch], vr[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const size_t at = (static_cast<size_t>(keys[min(j0 + u, t - 1)]) * H + h) * D + 8 * l;
          kr[u] = ld_pinned_v4(k + at);
          vr[u] = ld_pinned_v4(v + at);
        }
        float s[kBatch], dp[kBatch], sz[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          s[u] = dot8(qr, kr[u], 0.f);
          dp[u] = dot8(g, vr[u], 0.f);
          sz[u] = abs_dot8(g, vr[u]);
        }
#pragma unroll
        for (int i = G / 2; i > 0; i >>= 1) {
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            s[u] += __shfl_xor_sync(gm, s[u], i);
            dp[u] += __shfl_xor_sync(gm, dp[u], i);
          }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const float pj = j0 + u < t ? ex2_approx(fmaf(s[u], p.sl2, nle)) : 0.f;
          all += pj;
          acc = fmaf(pj, dp[u], acc);
          size = fmaf(pj, sz[u], size);
        }
      }
#pragma unroll
      for (int i = G / 2; i > 0; i >>= 1) size += __shfl_xor_sync(gm, size, i);
      const float own = acc / all;                    // no key of any weight: not a number, not taken
      if (fabsf(own - sum) <= kRoundedO * size) {
        sum = own;
        one = ones && t == 1;
      }
    }
  }
  if (l == 0 && n < NP) {
    const size_t at = static_cast<size_t>(h) * NP + n;
    nl[at] = nle;
    nd[at] = one ? __uint_as_float(kOneKey) : -sum;
  }
}

// The query tiles that list key tile kt, ascending, entry = tile | partial <<
// 30, by one warp from the bit sets (`bits`, `part`: the head's).  Returns
// their number.
__device__ __forceinline__ int listed_by(const uint32_t* bits, const uint32_t* part, int nB, int kt, int32_t* out,
                                         int lane) {
  const size_t at = static_cast<size_t>(kt >> 5) * nB;
  int n = 0;
#pragma unroll 4
  for (int q0 = 0; q0 < nB; q0 += 32) {
    const int qb = q0 + lane;
    const uint32_t a = qb < nB ? __ldg(bits + at + qb) : 0u;
    const uint32_t b = (part != nullptr && qb < nB) ? __ldg(part + at + qb) : 0u;
    const bool on = (a >> (kt & 31)) & 1u;
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, on);
    if (on) out[n + __popc(m & ((1u << lane) - 1u))] = qb | (((b >> (kt & 31)) & 1u) ? kPartialBit : 0);
    n += __popc(m);
  }
  return n;
}
// a list entry written by this block (not through the read-only path), loaded
// where the call stands
__device__ __forceinline__ int32_t ld_entry(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// COLS columns of one row of an f32 accumulator (TMEM) to bf16 in a
// 128-byte-swizzled box in shared memory, from its column `col`, times `mul`;
// zeros when !have.
template <int COLS>
__device__ __forceinline__ void store_rows(uint32_t tAcc, uint32_t sBox, int col, int r, float mul, bool have) {
#pragma unroll
  for (int c0 = 0; c0 < COLS; c0 += 16) {
    uint32_t ov[16];
    __syncwarp();
    if (have) {
      tmem_ld_x16(tAcc + c0, ov);
    } else {
#pragma unroll
      for (int c = 0; c < 16; ++c) ov[c] = 0u;
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const uint32_t dst = sBox + r * 128 + ((((col + c0) / 8 + v) ^ (r & 7)) * 16);
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = pack_bf16x2(__uint_as_float(ov[8 * v + 2 * i]) * mul, __uint_as_float(ov[8 * v + 2 * i + 1]) * mul);
      st_shared_v4(dst, w[0], w[1], w[2], w[3]);
    }
  }
}

template <int D>
struct BwdSmem {
  static constexpr uint32_t kBox = 128 * 128;
  static constexpr uint32_t kTile = (D / 64) * kBox;
  // dkv: K, V, three Q and two dO tiles, nl and nd beside each dO (128 floats
  // each); dq: Q, dO, three K and two V tiles
  static constexpr uint32_t kA = 0, kB = kTile, kRing3 = 2 * kTile, kRing2 = 5 * kTile;
  static constexpr uint32_t kRows = 7 * kTile;
  static constexpr uint32_t kBar = kRows + 2 * 1024;
  static constexpr uint32_t kHolder = kBar + 32 * 8;
  // declared 1,024-byte aligned: at d = 128 there is no room for slack
  static constexpr uint32_t kAlloc = kHolder + 16;
};
static_assert(BwdSmem<128>::kAlloc <= 232448, "shared memory of one block");

enum : int {
  W_AB = 0,                           // K and V loaded
  W_QFULL = 1, W_QEMPTY = 4,          // [3]
  W_OFULL = 7, W_OEMPTY = 9,          // [2] dO, nl, nd
  W_SFULL = 11, W_SFREE = 12,
  W_DPFULL = 13,                      // [2]
  // [tile parity][group]: with two dP a group may store tile i+1 before the
  // issuer has looked at another group's tile i
  W_P = 15, W_DS = W_P + 2 * kBwdGroups,
  W_FINAL = W_DS + 2 * kBwdGroups,
  W_COUNT
};
static_assert(W_COUNT <= 32, "barrier slots");

// dK and dV of key tile kt of head h.
template <int D, bool ONE>
__device__ __forceinline__ void bwd_dkv(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                        const CUtensorMap& tmG, const CUtensorMap& tmDK, const CUtensorMap& tmDV,
                                        const BwdParams& p, const int kt, const int h) {
  using L = BwdSmem<D>;
  extern __shared__ __align__(1024) uint8_t smem_bwd[];
  const uint32_t base = smem_u32(smem_bwd);
  if (base & 1023u) {                                   // the swizzled tiles need the declared alignment
    set_status(BSA_ERR_CUDA);
    return;
  }
  const uint32_t bar0 = base + L::kBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* holder = reinterpret_cast<volatile uint32_t*>(smem_bwd + L::kHolder);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long limit = p.wait_limit_ns;
  int32_t* lst = p.tlist + (static_cast<size_t>(h) * p.nB + kt) * p.nB;
  const int NP = p.nB * 128;

  if (threadIdx.x == 0) {
    for (int i = 0; i < W_COUNT; ++i)
      mbar_init(bar(i), i == W_SFREE ? 4 * kBwdGroups : ((i >= W_P && i < W_FINAL) ? 4 : 1));
    fence_mbar_init();
    // K and V are on their way while TMEM is allocated and the list is looked up
    mbar_arrive_expect_tx(bar(W_AB), 2 * L::kTile);
#pragma unroll
    for (int b = 0; b < D / 64; ++b) {
      tma_load_3d(base + L::kA + b * L::kBox, &tmK, bar(W_AB), b * 64, h, kt * 128);
      tma_load_3d(base + L::kB + b * L::kBox, &tmV, bar(W_AB), b * 64, h, kt * 128);
    }
  }
  if (warp == 1) {
    tmem_alloc(base + L::kHolder, 512);
    tmem_relinquish();
  }
  if (warp == 2) {
    const size_t off = static_cast<size_t>(h) * p.bhs;
    const int c = listed_by(p.bits + off, p.part != nullptr ? p.part + off : nullptr, p.nB, kt, lst, lane);
    if (lane == 0) holder[1] = static_cast<uint32_t>(c);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = holder[0];
  const int n = static_cast<int>(holder[1]);
  // d = 64 leaves room for two dP, so that dP(i+1) need not wait for dK(i)
  constexpr int kDP = D == 64 ? 2 : 1;
  constexpr uint32_t kTS = 0, kTDP = 128, kTDV = 128 + 128 * kDP, kTDK = kTDV + D;
  auto tdp = [&](int i) -> uint32_t { return tbase + kTDP + (kDP == 2 ? (i & 1) * 128u : 0u); };
  constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t kIdescD = idesc_bf16_f32(128, D, false, true);
  auto sQ = [&](int i) -> uint32_t { return base + L::kRing3 + (i % 3) * L::kTile; };
  auto sG = [&](int i) -> uint32_t { return base + L::kRing2 + (i & 1) * L::kTile; };
  auto sRow = [&](int i) -> uint32_t { return base + L::kRows + (i & 1) * 1024; };

  if (warp == 0) {
    regs_dec<kBwdRegsLow>();
    if (lane == 0) {
      int nq = 0, no = 0;                               // copies started
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int qt = ld_entry(lst + i) & ~kPartialBit;
        if (i >= 3) ok = mbar_wait(bar(W_QEMPTY + i % 3), (i / 3 - 1) & 1, limit);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(W_QFULL + i % 3), L::kTile);
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
          tma_load_3d(sQ(i) + b * L::kBox, &tmQ, bar(W_QFULL + i % 3), b * 64, h, qt * 128);
        ++nq;
        if (i >= 2) ok = mbar_wait(bar(W_OEMPTY + (i & 1)), ((i >> 1) - 1) & 1, limit);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(W_OFULL + (i & 1)), L::kTile + 1024);
        const size_t at = static_cast<size_t>(h) * NP + static_cast<size_t>(qt) * 128;
        bulk_load(sRow(i), p.nl + at, 512, bar(W_OFULL + (i & 1)));
        bulk_load(sRow(i) + 512, p.nd + at, 512, bar(W_OFULL + (i & 1)));
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
          tma_load_3d(sG(i) + b * L::kBox, &tmG, bar(W_OFULL + (i & 1)), b * 64, h, qt * 128);
        ++no;
      }
      // drain: wait (bounded) for this thread's own copies still in flight
      mbar_wait(bar(W_AB), 0, limit);
      for (int u = max(0, nq - 3); u < nq; ++u) mbar_wait(bar(W_QFULL + u % 3), (u / 3) & 1, limit);
      for (int u = max(0, no - 2); u < no; ++u) mbar_wait(bar(W_OFULL + (u & 1)), (u >> 1) & 1, limit);
    }
  } else if (warp == 1) {
    regs_dec<kBwdRegsLow>();
    if (n > 0) {
      const uint64_t dK = desc64(sw128_desc(base + L::kA, 16, 1024)), dV = desc64(sw128_desc(base + L::kB, 16, 1024));
      // S^T = K Q_i^T
      auto s_mma = [&](int i) {
        const uint64_t dq = desc64(sw128_desc(sQ(i), 16, 1024));
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
          mma4_ss_warp(tbase + kTS, dK + g * (L::kBox >> 4), dq + g * (L::kBox >> 4), kIdescS, g > 0);
        tc_commit_warp(bar(W_SFULL));
      };
      // dP^T = V dO_i^T
      auto dp_mma = [&](int i) {
        const uint64_t dg = desc64(sw128_desc(sG(i), 16, 1024));
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
          mma4_ss_warp(tdp(i), dV + g * (L::kBox >> 4), dg + g * (L::kBox >> 4), kIdescS, g > 0);
        tc_commit_warp(bar(W_DPFULL + (kDP == 2 ? (i & 1) : 0)));
      };
      // dst += A^T B, 32 queries of A (in dP's columns from `off`) as each group stores them
      auto grad_mma = [&](uint32_t dst, uint32_t off, uint32_t tile, int first_bar, int i) -> bool {
        const uint64_t db = desc64(sw128_desc(tile, L::kBox, 1024));
#pragma unroll
        for (int g = 0; g < kBwdGroups; ++g) {
          if (!mbar_wait_warp(bar(first_bar + (i & 1) * kBwdGroups + g), (i >> 1) & 1, limit)) return false;
          tc_fence_after();
          mma2_ts_warp(tbase + dst, tdp(i) + off + g * kBwdCols, db + g * (kBwdCols * 128 >> 4), kIdescD,
                       (i > 0 || g > 0) ? 1u : 0u);
        }
        return true;
      };
      bool ok = mbar_wait_warp(bar(W_AB), 0, limit) && mbar_wait_warp(bar(W_QFULL), 0, limit);
      tc_fence_after();
      if (ok) s_mma(0);
      ok = ok && mbar_wait_warp(bar(W_OFULL), 0, limit);
      tc_fence_after();
      if (ok) dp_mma(0);
      for (int i = 0; ok && i < n; ++i) {
        const int nx = i + 1;
        // S of the next tile as soon as this one's scores are in registers
        if (nx < n) {
          if (!(ok = mbar_wait_warp(bar(W_QFULL + nx % 3), (nx / 3) & 1, limit))) break;
          if (!(ok = mbar_wait_warp(bar(W_SFREE), i & 1, limit))) break;
          tc_fence_after();
          s_mma(nx);
          if (kDP == 2) {
            if (!(ok = mbar_wait_warp(bar(W_OFULL + (nx & 1)), (nx >> 1) & 1, limit))) break;
            tc_fence_after();
            dp_mma(nx);
          }
        }
        if (!(ok = grad_mma(kTDV, 0, sG(i), W_P, i))) break;                       // dV += P^T dO_i
        tc_commit_warp(bar(W_OEMPTY + (i & 1)));
        if (kDP == 1 && nx < n && !(ok = mbar_wait_warp(bar(W_OFULL + (nx & 1)), (nx >> 1) & 1, limit))) break;
        if (!(ok = grad_mma(kTDK, kBwdCols / 2, sQ(i), W_DS, i))) break;           // dK += dS^T Q_i
        tc_commit_warp(bar(W_QEMPTY + i % 3));
        if (kDP == 1 && nx < n) dp_mma(nx);
      }
      tc_commit_warp(bar(W_FINAL));
      mbar_wait_warp(bar(W_FINAL), 0, limit);
    }
  } else if (warp < 4) {
    regs_dec<kBwdRegsLow>();
  } else {
    regs_inc<kBwdRegsHigh>();
    const int g = (warp - 4) >> 2;
    const int r = (threadIdx.x - 128) & 127;
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tS = tbase + lane_off + kTS + kBwdCols * g, tDP0 = lane_off + kBwdCols * g;
    const int fk = p.fbits != nullptr ? min(kt * 128 + r, p.N - 1) / p.P : 0;
    const uint64_t sl2p = f2pack(p.sl2, p.sl2);
    bool ok = true;
    int e_next = n > 0 ? ld_entry(lst) : 0;
    for (int i = 0; ok && i < n; ++i) {
      const int e = e_next;
      if (i + 1 < n) e_next = ld_entry(lst + i + 1);
      const bool part = (e & kPartialBit) != 0 && p.fbits != nullptr;
      uint32_t mw = 0xFFFFFFFFu;
      if (part) mw = query_mask(p, fk, (e & ~kPartialBit) * 128 + kBwdCols * g);
      ok = mbar_wait(bar(W_OFULL + (i & 1)), (i >> 1) & 1, limit);
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(W_SFULL), i & 1, limit) && ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t rowv = sRow(i) + 4 * kBwdCols * g;
      uint32_t sr[32];
      float* pv = reinterpret_cast<float*>(sr);
      tmem_ld_x32(tS, sr);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(W_SFREE));
      uint32_t pk[16];
#pragma unroll
      for (int c = 0; c < kBwdCols; c += 4) {
        const float4 nl = ld_shared_f4(rowv + 4 * c);
        const uint64_t x01 = ffma2(f2pack(pv[c], pv[c + 1]), sl2p, f2pack(nl.x, nl.y));
        const uint64_t x23 = ffma2(f2pack(pv[c + 2], pv[c + 3]), sl2p, f2pack(nl.z, nl.w));
        f2unpack(x01, pv[c], pv[c + 1]);
        f2unpack(x23, pv[c + 2], pv[c + 3]);
#pragma unroll
        for (int u = 0; u < 4; ++u) pv[c + u] = ex2_approx(pv[c + u]);
      }
      if (part) {
#pragma unroll
        for (int c = 0; c < kBwdCols; ++c)
          if (!((mw >> c) & 1u)) pv[c] = 0.f;
      }
#pragma unroll
      for (int c = 0; c < kBwdCols; c += 2) pk[c / 2] = pack_bf16x2(pv[c], pv[c + 1]);
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(W_DPFULL + (kDP == 2 ? (i & 1) : 0)), (kDP == 2 ? i >> 1 : i) & 1, limit));
      if (!ok) break;
      tc_fence_after();
      // dP of these columns goes to registers, P takes the first half of them,
      // dS the second; nd is read before P is signalled, which lets go of the rows
      const uint32_t tDP = tdp(i) + tDP0;
      uint32_t dr[32];
      float* dv = reinterpret_cast<float*>(dr);
      tmem_ld_x32(tDP, dr);
#pragma unroll
      for (int c = 0; c < kBwdCols; c += 4) {
        const float4 nd = ld_shared_f4(rowv + 512 + 4 * c);
        f2unpack(fadd2(f2pack(dv[c], dv[c + 1]), f2pack(nd.x, nd.y)), dv[c], dv[c + 1]);
        f2unpack(fadd2(f2pack(dv[c + 2], dv[c + 3]), f2pack(nd.z, nd.w)), dv[c + 2], dv[c + 3]);
        if constexpr (ONE) {
          if (__float_as_uint(nd.x) == kOneKey) dv[c] = 0.f;
          if (__float_as_uint(nd.y) == kOneKey) dv[c + 1] = 0.f;
          if (__float_as_uint(nd.z) == kOneKey) dv[c + 2] = 0.f;
          if (__float_as_uint(nd.w) == kOneKey) dv[c + 3] = 0.f;
        }
      }
      uint32_t rows = 0u;                             // of every load of nd
#pragma unroll
      for (int c = 0; c < kBwdCols; c += 4) rows |= __float_as_uint(dv[c]);
      tmem_st_x16(tDP, pk);
      tc_fence_before();
      __syncwarp();
      mbar_arrive_after(bar(W_P + (i & 1) * kBwdGroups + g), rows, lane);
#pragma unroll
      for (int c = 0; c < kBwdCols; c += 2) {
        float y0, y1;
        f2unpack(fmul2(f2pack(pv[c], pv[c + 1]), f2pack(dv[c], dv[c + 1])), y0, y1);
        pk[c / 2] = pack_bf16x2(y0, y1);
      }
      tmem_st_x16(tDP + kBwdCols / 2, pk);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(W_DS + (i & 1) * kBwdGroups + g));
    }
    // epilogue: groups 0 and 1 write dV (through V's tile), 2 and 3 dK (through
    // K's), 64 channels each
    if (n > 0) {
      ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(bar(W_FINAL), 0, limit));
      tc_fence_after();
    }
    __all_sync(0xFFFFFFFFu, mbar_wait(bar(W_AB), 0, limit));   // the tile has landed before it is written over
    const bool have = __all_sync(0xFFFFFFFFu, ok && n > 0);
    const int acc = g >> 1, b = g & 1;
    if (b * 64 < D) {
      const uint32_t sOut = base + (acc ? L::kA : L::kB) + b * L::kBox;
      store_rows<64>(tbase + lane_off + (acc ? kTDK : kTDV) + b * 64, sOut, 0, r, acc ? p.scale : 1.f, have);
      fence_proxy_async_smem();
      named_barrier_sync(1 + g, 128);
      if (r == 0) {
        tma_store_3d(acc ? &tmDK : &tmDV, sOut, b * 64, h, kt * 128);
        bulk_commit();
        bulk_wait_read_all();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tbase, 512);
  }
}

enum : int {
  X_AB = 0,                           // Q and dO loaded
  X_KFULL = 1, X_KEMPTY = 4,          // [3]
  X_VFULL = 7, X_VEMPTY = 9,          // [2]
  X_SFULL = 11,                       // [2]
  X_DPFULL = 13,
  X_DS = 14,
  X_FINAL = 15,
  X_COUNT
};

// dQ of query tile qt of head h.
template <int D, bool ONE>
__device__ __forceinline__ void bwd_dq(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                       const CUtensorMap& tmG, const CUtensorMap& tmDQ, const BwdParams& p,
                                       const int qt, const int h) {
  using L = BwdSmem<D>;
  extern __shared__ __align__(1024) uint8_t smem_bwd[];
  const uint32_t base = smem_u32(smem_bwd);
  if (base & 1023u) {                                   // the swizzled tiles need the declared alignment
    set_status(BSA_ERR_CUDA);
    return;
  }
  const uint32_t bar0 = base + L::kBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  volatile uint32_t* holder = reinterpret_cast<volatile uint32_t*>(smem_bwd + L::kHolder);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long limit = p.wait_limit_ns;
  const int NP = p.nB * 128;
  if (threadIdx.x == 0) {
    for (int i = 0; i < X_COUNT; ++i) mbar_init(bar(i), i == X_DS ? 4 * kBwdGroups : 1);
    fence_mbar_init();
    // Q and dO are on their way while the list is looked up
    mbar_arrive_expect_tx(bar(X_AB), 2 * L::kTile);
#pragma unroll
    for (int b = 0; b < D / 64; ++b) {
      tma_load_3d(base + L::kA + b * L::kBox, &tmQ, bar(X_AB), b * 64, h, qt * 128);
      tma_load_3d(base + L::kB + b * L::kBox, &tmG, bar(X_AB), b * 64, h, qt * 128);
    }
  }
  int m = p.count[static_cast<size_t>(h) * p.chs + qt];       // entries; n: those in range
  m = min(max(m, 0), p.lrs);
  const size_t off = static_cast<size_t>(h) * p.lhs + static_cast<size_t>(qt) * p.lrs;
  const int32_t* lst = p.list + off;
  const uint8_t* flg = p.flags != nullptr ? p.flags + off : nullptr;
  int n = 0;
  for (int j0 = 0; j0 < m; j0 += 32) {
    const int e = j0 + lane < m ? lst[j0 + lane] : -1;
    n += __popc(__ballot_sync(0xFFFFFFFFu, e >= 0 && e < p.nB));
  }

  if (warp == 1) {
    tmem_alloc(base + L::kHolder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *holder;
  constexpr uint32_t kTDP = 256, kTDQ = 384;                  // S_0 at 0, S_1 at 128
  constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
  constexpr uint32_t kIdescD = idesc_bf16_f32(128, D, false, true);
  auto sK = [&](int j) -> uint32_t { return base + L::kRing3 + (j % 3) * L::kTile; };
  auto sV = [&](int j) -> uint32_t { return base + L::kRing2 + (j & 1) * L::kTile; };

  if (warp == 0) {
    regs_dec<kBwdRegsLow>();
    if (lane == 0) {
      int jk = 0, jv = 0;
      bool ok = true;
      for (int u = 0; u < m; ++u) {
        const int kt = lst[u];
        if (kt < 0 || kt >= p.nB) continue;
        if (jk >= 3) ok = mbar_wait(bar(X_KEMPTY + jk % 3), (jk / 3 - 1) & 1, limit);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(X_KFULL + jk % 3), L::kTile);
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
          tma_load_3d(sK(jk) + b * L::kBox, &tmK, bar(X_KFULL + jk % 3), b * 64, h, kt * 128);
        ++jk;
        if (jv >= 2) ok = mbar_wait(bar(X_VEMPTY + (jv & 1)), ((jv >> 1) - 1) & 1, limit);
        if (!ok) break;
        mbar_arrive_expect_tx(bar(X_VFULL + (jv & 1)), L::kTile);
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
          tma_load_3d(sV(jv) + b * L::kBox, &tmV, bar(X_VFULL + (jv & 1)), b * 64, h, kt * 128);
        ++jv;
      }
      mbar_wait(bar(X_AB), 0, limit);
      for (int u = max(0, jk - 3); u < jk; ++u) mbar_wait(bar(X_KFULL + u % 3), (u / 3) & 1, limit);
      for (int u = max(0, jv - 2); u < jv; ++u) mbar_wait(bar(X_VFULL + (u & 1)), (u >> 1) & 1, limit);
    }
  } else if (warp == 1) {
    regs_dec<kBwdRegsLow>();
    if (n > 0) {
      const uint64_t dQ = desc64(sw128_desc(base + L::kA, 16, 1024)), dG = desc64(sw128_desc(base + L::kB, 16, 1024));
      // S = Q K_j^T into buffer j % 2
      auto s_mma = [&](int j) {
        const uint64_t dk = desc64(sw128_desc(sK(j), 16, 1024));
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
          mma4_ss_warp(tbase + (j & 1) * 128, dQ + g * (L::kBox >> 4), dk + g * (L::kBox >> 4), kIdescS, g > 0);
        tc_commit_warp(bar(X_SFULL + (j & 1)));
      };
      // dP = dO V_j^T; V_j is free after it
      auto dp_mma = [&](int j) {
        const uint64_t dv = desc64(sw128_desc(sV(j), 16, 1024));
#pragma unroll
        for (int g = 0; g < D / 64; ++g)
          mma4_ss_warp(tbase + kTDP, dG + g * (L::kBox >> 4), dv + g * (L::kBox >> 4), kIdescS, g > 0);
        tc_commit2_warp(bar(X_DPFULL), bar(X_VEMPTY + (j & 1)));
      };
      auto k_wait = [&](int j) -> bool {
        const bool w = mbar_wait_warp(bar(X_KFULL + j % 3), (j / 3) & 1, limit);
        tc_fence_after();
        return w;
      };
      auto v_wait = [&](int j) -> bool {
        const bool w = mbar_wait_warp(bar(X_VFULL + (j & 1)), (j >> 1) & 1, limit);
        tc_fence_after();
        return w;
      };
      bool ok = mbar_wait_warp(bar(X_AB), 0, limit) && k_wait(0);
      if (ok) s_mma(0);
      ok = ok && v_wait(0);
      if (ok) dp_mma(0);
      if (ok && n > 1 && (ok = k_wait(1))) s_mma(1);
      for (int j = 0; ok && j < n; ++j) {
        if (j + 1 < n && !(ok = v_wait(j + 1))) break;
        const uint64_t dk = desc64(sw128_desc(sK(j), L::kBox, 1024));
        const uint32_t tA = tbase + (j & 1) * 128;
        // dS_j of every group: dP has been read and S_j is done with
        if (!(ok = mbar_wait_warp(bar(X_DS), j & 1, limit))) break;
        tc_fence_after();
        if (j + 1 < n) dp_mma(j + 1);
        // dQ += dS K_j
#pragma unroll
        for (int g = 0; g < kBwdGroups; ++g)
          mma2_ts_warp(tbase + kTDQ, tA + g * kBwdCols, dk + g * (kBwdCols * 128 >> 4), kIdescD, (j > 0 || g > 0) ? 1u : 0u);
        tc_commit_warp(bar(X_KEMPTY + j % 3));
        if (j + 2 < n && (ok = k_wait(j + 2))) s_mma(j + 2);
      }
      tc_commit_warp(bar(X_FINAL));
      mbar_wait_warp(bar(X_FINAL), 0, limit);
    }
  } else if (warp < 4) {
    regs_dec<kBwdRegsLow>();
  } else {
    regs_inc<kBwdRegsHigh>();
    const int g = (warp - 4) >> 2;
    const int r = (threadIdx.x - 128) & 127;
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tDP = tbase + lane_off + kTDP + kBwdCols * g;
    const int fq = p.fbits != nullptr ? min(qt * 128 + r, p.N - 1) / p.P : 0;
    const float nl = p.nl[static_cast<size_t>(h) * NP + qt * 128 + r], nd = p.nd[static_cast<size_t>(h) * NP + qt * 128 + r];
    const uint64_t sl2p = f2pack(p.sl2, p.sl2), nlp = f2pack(nl, nl), ndp = f2pack(nd, nd);
    bool ok = true;
    int j = 0;
    int kt_next = m > 0 ? ld_pinned_s32(lst) : 0;
    uint32_t f_next = (m > 0 && flg != nullptr) ? ld_pinned_u8(flg) : 0u;
    for (int u = 0; ok && u < m; ++u) {
      const int kt = kt_next;
      const uint32_t fl = f_next;
      if (u + 1 < m) {
        kt_next = ld_pinned_s32(lst + u + 1);
        if (flg != nullptr) f_next = ld_pinned_u8(flg + u + 1);
      }
      if (kt < 0 || kt >= p.nB) continue;
      const bool part = flg != nullptr ? fl != 0u : kt * 128 + 128 > p.N;
      uint32_t mw = 0xFFFFFFFFu;
      if (part) mw = key_mask(p, fq, kt * 128 + kBwdCols * g);
      const uint32_t tS = tbase + lane_off + (j & 1) * 128 + kBwdCols * g;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(X_SFULL + (j & 1)), (j >> 1) & 1, limit));
      if (!ok) break;
      tc_fence_after();
      uint32_t sr[32];
      float* pv = reinterpret_cast<float*>(sr);
      tmem_ld_x32(tS, sr);
#pragma unroll
      for (int c = 0; c < kBwdCols; c += 2) {
        float x0, x1;
        f2unpack(ffma2(f2pack(pv[c], pv[c + 1]), sl2p, nlp), x0, x1);
        pv[c] = ex2_approx(x0);
        pv[c + 1] = ex2_approx(x1);
      }
      if (part) {
#pragma unroll
        for (int c = 0; c < kBwdCols; ++c)
          if (!((mw >> c) & 1u)) pv[c] = 0.f;
      }
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar(X_DPFULL), j & 1, limit));
      if (!ok) break;
      tc_fence_after();
      uint32_t dr[32], pk[16];
      const float* dv = reinterpret_cast<const float*>(dr);
      tmem_ld_x32(tDP, dr);
#pragma unroll
      for (int c = 0; c < kBwdCols; c += 2) {
        float y0, y1;
        f2unpack(fmul2(f2pack(pv[c], pv[c + 1]), fadd2(f2pack(dv[c], dv[c + 1]), ndp)), y0, y1);
        pk[c / 2] = pack_bf16x2(y0, y1);
      }
      if constexpr (ONE) {
        const bool one = __float_as_uint(nd) == kOneKey;
#pragma unroll
        for (int c = 0; c < kBwdCols / 2; ++c) pk[c] = one ? 0u : pk[c];
      }
      tmem_st_x16(tS, pk);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(X_DS));
      ++j;
    }
    // epilogue: every group writes D / 4 channels of dQ through Q's tile
    if (n > 0) {
      ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait(bar(X_FINAL), 0, limit));
      tc_fence_after();
    }
    __all_sync(0xFFFFFFFFu, mbar_wait(bar(X_AB), 0, limit));
    const bool have = __all_sync(0xFFFFFFFFu, ok && n > 0);
    constexpr int kCols = D / kBwdGroups;
    const int c0 = g * kCols, b = c0 / 64;
    const uint32_t sOut = base + L::kA + b * L::kBox;
    store_rows<kCols>(tbase + lane_off + kTDQ + c0, sOut, c0 % 64, r, p.scale, have);
    fence_proxy_async_smem();
    constexpr int kPerBox = 64 / kCols;                 // groups that fill one box
    named_barrier_sync(1 + b, 128 * kPerBox);
    if (r == 0 && c0 % 64 == 0) {
      tma_store_3d(&tmDQ, sOut, b * 64, h, qt * 128);
      bulk_commit();
      bulk_wait_read_all();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tbase, 512);
  }
}

// Key tiles and query tiles in one launch, so that one kind fills the SMs that
// the other's last blocks leave.  Grid (2 nB, heads): the key tiles of a head,
// then its query tiles (they share K, V, Q and dO in L2); or (nB, heads, 2): all
// key tiles first, then all query tiles, whose shorter blocks even out the end.
// The second order where the blocks fill the SMs only a few times (see
// launch_bwd): 45.0 against 49.3 us for 208 blocks (26 tiles, 4 heads, d = 64),
// but 2,466 against 2,409 us for 6,144 blocks (256 tiles, 12 heads, d = 128).
template <int D, bool ONE>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmG,
                const __grid_constant__ CUtensorMap tmDQ, const __grid_constant__ CUtensorMap tmDK,
                const __grid_constant__ CUtensorMap tmDV, const BwdParams p) {
  const int t = blockIdx.x + blockIdx.z * p.nB, h = blockIdx.y;
  if (t < p.nB)
    bwd_dkv<D, ONE>(tmQ, tmK, tmV, tmG, tmDK, tmDV, p, t, h);
  else
    bwd_dq<D, ONE>(tmQ, tmK, tmV, tmG, tmDQ, p, t - p.nB, h);
}

}  // namespace bsa
