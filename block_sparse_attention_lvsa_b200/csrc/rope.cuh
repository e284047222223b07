// rope.cuh - rotary positions over up to three axes (time, height, width),
// alone or in one pass with the per-head RMS norm of queries and keys, and
// the gradient of that pass.
//
// Forward, per token n and head h (one row of d channels):
//   z = x * r * w,  r = (mean_c x_c^2 + eps)^-1/2        (norm; else z = x)
//   pair j of the row is turned by the angle of its axis' position:
//   (y_a, y_b) = (z_a cos - z_b sin, z_a sin + z_b cos)
// Pairs are dealt to the axes in order (the first pairs[0] to axis 0, and so
// on); pairs beyond the last axis stay as they are.  cos and sin come from
// one table per axis, built once in 64-bit arithmetic.
// Backward, with g = the output gradient turned by minus the angle and
// xh = x r:
//   dw = sum over rows of g xh
//   dx = r (g w - xh mean_c(g w xh))
// (without the norm the gradient of the rotation is the rotation by minus
// the angle).  r is recomputed from x, which the backward pass reads anyway.
//
// Bound by memory traffic: each row is read once and written once.  d/8
// neighbouring lanes own one row, four pairs (eight channels) a lane, so both
// members of a pair, the table entries and the weights of a lane's channels
// stay in that lane; the row sums are butterflies over d/8 lanes.  A group of
// d/8 lanes takes up to kRopeHeads heads of one token: their loads are all
// issued before the first use, and the lane's four (cos, sin) are read once
// for all of them.  All arithmetic is float32; the one rounding is the
// store.
#pragma once
#include <cuda_fp16.h>
#include "ptx.cuh"

namespace bsa {

constexpr int kRopeHeads = 8;        // most heads per group and step
constexpr int kRopeThreads = 256;

// Device view of bsa_rope.
struct RopeDev {
  const float* table[3];
  int pairs[3];
  int len[3];
  int first[3];
  int gh, gw;                        // grid height and width
  long long ngrid;                   // tokens inside the grid
  const int32_t* pos;                // [N][3] or null (grid)
  float sign;                        // +1 forward, -1 inverse
};

// One [N, H, d] tensor pair (input, output) with element strides.
struct RopeTensor {
  const void* x;                     // input
  const void* g;                     // output gradient (backward)
  void* y;                           // output / input gradient
  long long xt, xh, gt, gh, yt, yh;  // token and head strides
  int H;
  int chunks;                        // groups a token's heads are dealt to
  int per;                           // heads per group: ceil(H / chunks)
  const void* w;                     // norm weight [d] or null
};

struct RopeParams {
  RopeTensor t[2];                   // q, k (blockIdx.y)
  long long N;
  RopeDev r;
  int w_f32;                         // weights are float32 (else the tensors' type)
  float eps;
  float* partial;                    // backward: [2][gridDim.x][d] weight-gradient partial sums
};

// eight channels of a row as float: adjacent layout = 8 consecutive channels,
// split layout = 4 at c and 4 at c + d/2; member a of pair u is v[2u], b v[2u+1]
template <typename T> struct Vec8;
template <> struct Vec8<float> {
  float4 a, b;
};
template <> struct Vec8<__nv_bfloat16> {
  uint2 a, b;
};
template <> struct Vec8<__half> {
  uint2 a, b;
};

template <bool SPLIT, int D>
__device__ __forceinline__ void load8(const float* row, int l, Vec8<float>& v) {
  v.a = *reinterpret_cast<const float4*>(row + (SPLIT ? 4 * l : 8 * l));
  v.b = *reinterpret_cast<const float4*>(row + (SPLIT ? D / 2 + 4 * l : 8 * l + 4));
}
template <bool SPLIT, int D, typename T>
__device__ __forceinline__ void load8(const T* row, int l, Vec8<T>& v) {
  if (SPLIT) {
    v.a = *reinterpret_cast<const uint2*>(row + 4 * l);
    v.b = *reinterpret_cast<const uint2*>(row + D / 2 + 4 * l);
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(row + 8 * l);
    v.a = make_uint2(w.x, w.y);
    v.b = make_uint2(w.z, w.w);
  }
}

__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) { return pack_bf16x2(a, b); }
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// f[0..7] in pair order: f[2u], f[2u+1] are the two members of pair u
template <bool SPLIT>
__device__ __forceinline__ void to_pairs(const Vec8<float>& v, float (&f)[8]) {
  const float x[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    f[2 * u] = SPLIT ? x[u] : x[2 * u];
    f[2 * u + 1] = SPLIT ? x[4 + u] : x[2 * u + 1];
  }
}
template <bool SPLIT, typename T>
__device__ __forceinline__ void to_pairs(const Vec8<T>& v, float (&f)[8]) {
  const float2 p[4] = {unpack2(v.a.x, T()), unpack2(v.a.y, T()), unpack2(v.b.x, T()), unpack2(v.b.y, T())};
  const float x[8] = {p[0].x, p[0].y, p[1].x, p[1].y, p[2].x, p[2].y, p[3].x, p[3].y};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    f[2 * u] = SPLIT ? x[u] : x[2 * u];
    f[2 * u + 1] = SPLIT ? x[4 + u] : x[2 * u + 1];
  }
}

template <bool SPLIT, int D>
__device__ __forceinline__ void store8(float* row, int l, const float (&f)[8]) {
  float x[8];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    x[SPLIT ? u : 2 * u] = f[2 * u];
    x[SPLIT ? 4 + u : 2 * u + 1] = f[2 * u + 1];
  }
  *reinterpret_cast<float4*>(row + (SPLIT ? 4 * l : 8 * l)) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(row + (SPLIT ? D / 2 + 4 * l : 8 * l + 4)) = make_float4(x[4], x[5], x[6], x[7]);
}
template <bool SPLIT, int D, typename T>
__device__ __forceinline__ void store8(T* row, int l, const float (&f)[8]) {
  if (SPLIT) {
    *reinterpret_cast<uint2*>(row + 4 * l) = make_uint2(pack2(f[0], f[2], T()), pack2(f[4], f[6], T()));
    *reinterpret_cast<uint2*>(row + D / 2 + 4 * l) = make_uint2(pack2(f[1], f[3], T()), pack2(f[5], f[7], T()));
  } else {
    *reinterpret_cast<uint4*>(row + 8 * l) = make_uint4(pack2(f[0], f[1], T()), pack2(f[2], f[3], T()),
                                                        pack2(f[4], f[5], T()), pack2(f[6], f[7], T()));
  }
}

// The four pairs of a lane: which axis each belongs to and where its column
// of that axis' table starts.
struct LanePairs {
  const float* col[4];
  int stride[4];                     // floats per position; 0: the pair is not rotated
  int axis[4];
};
__device__ __forceinline__ void lane_pairs(const RopeDev& r, int l, LanePairs& lp) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    int j = 4 * l + u;
    lp.axis[u] = 0;
    lp.stride[u] = 0;
    lp.col[u] = nullptr;
#pragma unroll
    for (int a = 0; a < 3; ++a) {
      if (j >= 0 && j < r.pairs[a]) {
        lp.axis[u] = a;
        lp.stride[u] = 2 * r.pairs[a];
        lp.col[u] = r.table[a] + 2 * j;
      }
      j -= r.pairs[a];               // negative once an axis took the pair
    }
  }
}

// cos and sign * sin of the lane's pairs for token n
__device__ __forceinline__ void lane_angles(const RopeDev& r, const LanePairs& lp, long long n, float (&c)[4],
                                            float (&s)[4]) {
  int p[3] = {-1, -1, -1};
  if (r.pos != nullptr) {
    const int32_t* q = r.pos + 3 * n;
#pragma unroll
    for (int a = 0; a < 3; ++a) {
      p[a] = __ldg(q + a);
      if (r.pairs[a] > 0 && p[a] >= r.len[a]) {     // past the table: reported, not rotated
        set_status(BSA_ERR_INDEX_RANGE);
        p[a] = -1;
      }
    }
  } else if (n < r.ngrid) {
    const int i = static_cast<int>(n);              // the grid has fewer than 2^31 tokens
    const int row = i / r.gw;
    p[2] = r.first[2] + (i - row * r.gw);
    const int fr = row / r.gh;
    p[1] = r.first[1] + (row - fr * r.gh);
    p[0] = r.first[0] + fr;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int pa = lp.axis[u] == 0 ? p[0] : (lp.axis[u] == 1 ? p[1] : p[2]);
    c[u] = 1.f;
    s[u] = 0.f;
    if (lp.stride[u] > 0 && pa >= 0) {
      const float2 cs = __ldg(reinterpret_cast<const float2*>(lp.col[u] + static_cast<long long>(pa) * lp.stride[u]));
      c[u] = cs.x;
      s[u] = r.sign * cs.y;
    }
  }
}

// Pairs of a row turned in place.  A pair with sin = 0 leaves its members
// apart, so that an unturned pair is a copy even next to an infinity.
__device__ __forceinline__ void turn(float (&f)[8], const float (&c)[4], const float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = f[2 * i], b = f[2 * i + 1];
    const bool on = s[i] != 0.f;
    f[2 * i] = on ? a * c[i] - b * s[i] : a * c[i];
    f[2 * i + 1] = on ? a * s[i] + b * c[i] : b * c[i];
  }
}

template <bool SPLIT, int D, typename T>
__device__ __forceinline__ void lane_weight(const void* w, int w_f32, int l, float (&f)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
  } else if (w_f32) {
    Vec8<float> v;
    load8<SPLIT, D>(static_cast<const float*>(w), l, v);
    to_pairs<SPLIT>(v, f);
  } else {
    Vec8<T> v;
    load8<SPLIT, D>(static_cast<const T*>(w), l, v);
    to_pairs<SPLIT>(v, f);
  }
}

template <int D>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Forward: rotation, with the norm before it when NORM.
template <typename T, int D, bool SPLIT, bool NORM>
__global__ void __launch_bounds__(kRopeThreads) rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int G = D / 8;                            // lanes per row
  const RopeTensor& t = p.t[blockIdx.y];
  const int l = threadIdx.x % G;
  LanePairs lp;
  lane_pairs(p.r, l, lp);
  float w[8];
  if (NORM) lane_weight<SPLIT, D, T>(t.w, p.w_f32, l, w);
  const long long items = p.N * t.chunks;
  constexpr int kGroups = kRopeThreads / G;
  // every lane of a warp runs the same number of steps (the butterflies take
  // the whole warp); groups past the end work on no head
  for (long long base = static_cast<long long>(blockIdx.x) * kGroups; base < items;
       base += static_cast<long long>(gridDim.x) * kGroups) {
    const long long it = base + threadIdx.x / G;
    const long long n = it / t.chunks;
    const int h0 = static_cast<int>(it - n * t.chunks) * t.per;
    const int nh = it < items ? min(t.per, t.H - h0) : 0;
    const T* x = static_cast<const T*>(t.x) + n * t.xt + h0 * t.xh;
    T* y = static_cast<T*>(t.y) + n * t.yt + h0 * t.yh;
    Vec8<T> v[kRopeHeads];
#pragma unroll
    for (int u = 0; u < kRopeHeads; ++u)
      if (u < nh) load8<SPLIT, D>(x + u * t.xh, l, v[u]);
    float c[4], s[4];
    if (nh > 0) lane_angles(p.r, lp, n, c, s);
#pragma unroll
    for (int u = 0; u < kRopeHeads; ++u) {
      if (NORM) {
        if (u >= t.per) break;                        // the same for the whole grid
      } else if (u >= nh) {
        break;
      }
      float f[8];
      to_pairs<SPLIT>(v[u], f);
      if (NORM) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
        ss = group_sum<D>(ss);
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= r * w[i];
      }
      turn(f, c, s);
      if (u < nh) store8<SPLIT, D>(y + u * t.yh, l, f);
    }
  }
}

// Backward of the norm and rotation.  Weight gradients: every lane sums its
// channels over its rows, a block's groups are added in a fixed order, and
// rope_dw_kernel adds the blocks' partial sums, again in a fixed order, so
// that the result does not change from run to run.
template <typename T, int D, bool SPLIT>
__global__ void __launch_bounds__(kRopeThreads) rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int G = D / 8;
  constexpr int kGroups = kRopeThreads / G;
  __shared__ float s_dw[kGroups][D];
  const RopeTensor& t = p.t[blockIdx.y];
  const int l = threadIdx.x % G;
  LanePairs lp;
  lane_pairs(p.r, l, lp);
  float w[8], dw[8];
  lane_weight<SPLIT, D, T>(t.w, p.w_f32, l, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = 0.f;
  const long long items = p.N * t.chunks;
  for (long long base = static_cast<long long>(blockIdx.x) * kGroups; base < items;
       base += static_cast<long long>(gridDim.x) * kGroups) {
    const long long it = base + threadIdx.x / G;
    const long long n = it / t.chunks;
    const int h0 = static_cast<int>(it - n * t.chunks) * t.per;
    const int nh = it < items ? min(t.per, t.H - h0) : 0;
    const T* x = static_cast<const T*>(t.x) + n * t.xt + h0 * t.xh;
    const T* g = static_cast<const T*>(t.g) + n * t.gt + h0 * t.gh;
    T* y = static_cast<T*>(t.y) + n * t.yt + h0 * t.yh;
    float c[4], s[4];
    bool have = false;
#pragma unroll 1
    for (int b = 0; b < t.per; b += 4) {              // four heads' loads in flight
      Vec8<T> vx[4], vg[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (b + u < nh) {
          load8<SPLIT, D>(x + (b + u) * t.xh, l, vx[u]);
          load8<SPLIT, D>(g + (b + u) * t.gh, l, vg[u]);
        }
      }
      if (!have && nh > 0) lane_angles(p.r, lp, n, c, s);
      have = true;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (b + u >= t.per) break;                    // the same for the whole grid
        float fx[8], fg[8];
        to_pairs<SPLIT>(vx[u], fx);
        to_pairs<SPLIT>(vg[u], fg);
        float ss = 0.f, dot = 0.f;
        turn(fg, c, s);                               // back: the sign is in s
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(fx[i], fx[i], ss);
          dot = fmaf(fg[i] * w[i], fx[i], dot);
        }
        ss = group_sum<D>(ss);
        dot = group_sum<D>(dot);
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        const float m = dot * r * (1.f / D);          // mean(g w xh)
        if (b + u < nh) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float xh = fx[i] * r;
            dw[i] = fmaf(fg[i], xh, dw[i]);
            f[i] = r * (fg[i] * w[i] - xh * m);
          }
          store8<SPLIT, D>(y + (b + u) * t.yh, l, f);
        }
      }
    }
  }
  // channel of dw[i]: the inverse of the pair order
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s_dw[threadIdx.x / G][SPLIT ? 4 * l + i : 8 * l + 2 * i] = dw[2 * i];
    s_dw[threadIdx.x / G][SPLIT ? D / 2 + 4 * l + i : 8 * l + 2 * i + 1] = dw[2 * i + 1];
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f;
#pragma unroll
    for (int gr = 0; gr < kGroups; ++gr) sum += s_dw[gr][threadIdx.x];
    p.partial[(static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * D + threadIdx.x] = sum;
  }
}

// dw[c] = sum over blocks of partial[tensor][block][c]; one block per tensor
// (blockIdx.x), 1024 threads: 1024 / d slices of the blocks, added in order.
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* __restrict__ partial, int blocks, int d,
                                                       float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float s[1024];
  const int c = threadIdx.x % d, slice = threadIdx.x / d, slices = 1024 / d;
  const float* src = partial + static_cast<size_t>(blockIdx.x) * blocks * d + c;
  float sum = 0.f;
#pragma unroll 8
  for (int b = slice; b < blocks; b += slices) sum += src[static_cast<size_t>(b) * d];
  s[threadIdx.x] = sum;
  __syncthreads();
  float* dw = blockIdx.x ? dwk : dwq;
  if (slice == 0 && dw != nullptr) {
    for (int i = 1; i < slices; ++i) sum += s[i * d + c];
    dw[c] = sum;
  }
}

// table[i][j] = (cos, sin) of (start + i * step) * theta^(-j / pairs), angles
// and functions in 64 bits (a far position's angle keeps ~1e-16 of itself,
// where 32 bits would be off by whole digits of the turn), rounded once.
__global__ void rope_table_kernel(int len, int pairs, double theta, double start, double step,
                                  float* __restrict__ table) {
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<long long>(len) * pairs) return;
  const int p = static_cast<int>(i / pairs), j = static_cast<int>(i % pairs);
  const double a = (start + p * step) * pow(theta, -static_cast<double>(j) / pairs);
  double sn, cs;
  sincos(a, &sn, &cs);
  table[2 * i] = static_cast<float>(cs);
  table[2 * i + 1] = static_cast<float>(sn);
}

}  // namespace bsa
