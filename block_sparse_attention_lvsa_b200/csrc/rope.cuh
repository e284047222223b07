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
// d/8 lanes goes through the heads of one token, four rows' loads at a time,
// with the token's cos and sin (times the weights) in registers, and the blocks
// stride over the tokens, so that a lane finds its pairs once.  The arithmetic
// is in packed pairs of float32 (half the instructions: with scalar ones, and
// the angles looked up again for every eight heads, the kernel was bound by
// instruction issue); the one rounding is the store.  One B200, bf16, q and k of
// 196560 x 12 x 128 (2.42 GB): 400 us, 0.92 of the measured copy bandwidth
// (first form 571 us); the rotation alone of one of them 191 us, 0.96.
// The backward pass has three streams and more to compute per row; its loads go
// through a ring in shared memory, two steps ahead: 340 us at 32760 x 40 x 128,
// 0.90 (loads in registers 415 us; the forward pass is slower with a ring, 437
// against 391 us).
#pragma once
#include <cuda_fp16.h>
#include "attn_fwd.cuh"

namespace bsa {

constexpr int kRopeHeads = 4;        // rows of a group per step (32-bit types: half)
constexpr int kRopeThreads = 256;
constexpr int kRopeBwdStages = 3;    // steps of the backward kernel's load ring
constexpr int kRopeFwdCtas = 3, kRopeBwdCtas = 2;          // blocks per SM
template <typename T>
constexpr int rope_rows() { return sizeof(T) == 4 ? kRopeHeads / 2 : kRopeHeads; }
// ring bytes: 16 (32) bytes a lane of every row of x and g
constexpr int kRopeRing = kRopeBwdStages * 2 * kRopeHeads * 16 * kRopeThreads;

__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Device view of bsa_rope.
struct RopeDev {
  const float* table[3];
  int pairs[3];
  int len[3];
  int first[3];
  uint32_t gh, gw;                   // grid height and width
  uint32_t mh, mw;                   // n / gh = (n * mh) >> sh for 0 <= n < 2^31, and so for gw
  int sh, sw;
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
  const void* w;                     // norm weight [d] or null
};

struct RopeParams {
  RopeTensor t[2];                   // q, k (blockIdx.y)
  long long N;
  RopeDev r;
  int per;                           // heads per block of a token (blockIdx.z counts them)
  int w_f32;                         // weights are float32 (else the tensors' type)
  float eps;
  float* partial;                    // backward: [2][gridDim.x * gridDim.z][d] weight-gradient partial sums
};

// A lane's eight channels as loaded: adjacent layout 8 consecutive channels,
// split layout 4 at c and 4 at c + d/2.
template <typename T> struct Vec8 {
  uint2 a, b;
};
template <> struct Vec8<float> {
  float4 a, b;
};

// Ring in shared memory: every lane copies its channels of the next rows
// asynchronously into a slot of its own (so that nobody else waits for them)
// and reads them back two steps later.  `slot` is the lane's slot of a row; a
// row of 32-bit values takes a second one behind all lanes'.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
constexpr uint32_t kRopeSlots = 16 * kRopeThreads;
template <bool SPLIT, int D, typename T>
__device__ __forceinline__ void copy8(uint32_t slot, const T* row, int l) {
  if constexpr (sizeof(T) == 4) {
    cp_async16(slot, row + (SPLIT ? 4 * l : 8 * l));
    cp_async16(slot + kRopeSlots, row + (SPLIT ? D / 2 + 4 * l : 8 * l + 4));
  } else if constexpr (SPLIT) {
    cp_async8(slot, row + 4 * l);
    cp_async8(slot + 8, row + D / 2 + 4 * l);
  } else {
    cp_async16(slot, row + 8 * l);
  }
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void read8(uint32_t slot, Vec8<float>& v) {
  const uint4 a = ld_shared_u4(slot), b = ld_shared_u4(slot + kRopeSlots);
  v.a = make_float4(__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w));
  v.b = make_float4(__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w));
}
template <typename T>
__device__ __forceinline__ void read8(uint32_t slot, Vec8<T>& v) {
  const uint4 a = ld_shared_u4(slot);
  v.a = make_uint2(a.x, a.y);
  v.b = make_uint2(a.z, a.w);
}
// The same as packed pairs of float: members a of pairs (0, 1) and (2, 3),
// members b of the same pairs.
struct Row8 {
  uint64_t a[2], b[2];
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

template <bool SPLIT>
__device__ __forceinline__ Row8 to_row(const Vec8<float>& v) {
  Row8 r;
  if (SPLIT) {
    r.a[0] = f2pack(v.a.x, v.a.y);
    r.a[1] = f2pack(v.a.z, v.a.w);
    r.b[0] = f2pack(v.b.x, v.b.y);
    r.b[1] = f2pack(v.b.z, v.b.w);
  } else {
    r.a[0] = f2pack(v.a.x, v.a.z);
    r.a[1] = f2pack(v.b.x, v.b.z);
    r.b[0] = f2pack(v.a.y, v.a.w);
    r.b[1] = f2pack(v.b.y, v.b.w);
  }
  return r;
}
template <bool SPLIT, typename T>
__device__ __forceinline__ Row8 to_row(const Vec8<T>& v) {
  const float2 p = unpack2(v.a.x, T()), q = unpack2(v.a.y, T()), s = unpack2(v.b.x, T()), t = unpack2(v.b.y, T());
  Row8 r;
  if (SPLIT) {
    r.a[0] = f2pack(p.x, p.y);
    r.a[1] = f2pack(q.x, q.y);
    r.b[0] = f2pack(s.x, s.y);
    r.b[1] = f2pack(t.x, t.y);
  } else {
    r.a[0] = f2pack(p.x, q.x);
    r.a[1] = f2pack(s.x, t.x);
    r.b[0] = f2pack(p.y, q.y);
    r.b[1] = f2pack(s.y, t.y);
  }
  return r;
}

template <bool SPLIT, int D, typename T>
__device__ __forceinline__ void store8(T* row, int l, const Row8& r) {
  float a[4], b[4];
  f2unpack(r.a[0], a[0], a[1]);
  f2unpack(r.a[1], a[2], a[3]);
  f2unpack(r.b[0], b[0], b[1]);
  f2unpack(r.b[1], b[2], b[3]);
  if constexpr (sizeof(T) == 4) {
    float4* p = reinterpret_cast<float4*>(row + (SPLIT ? 4 * l : 8 * l));
    float4* q = reinterpret_cast<float4*>(row + (SPLIT ? D / 2 + 4 * l : 8 * l + 4));
    *p = SPLIT ? make_float4(a[0], a[1], a[2], a[3]) : make_float4(a[0], b[0], a[1], b[1]);
    *q = SPLIT ? make_float4(b[0], b[1], b[2], b[3]) : make_float4(a[2], b[2], a[3], b[3]);
  } else if constexpr (SPLIT) {
    *reinterpret_cast<uint2*>(row + 4 * l) = make_uint2(pack2(a[0], a[1], T()), pack2(a[2], a[3], T()));
    *reinterpret_cast<uint2*>(row + D / 2 + 4 * l) = make_uint2(pack2(b[0], b[1], T()), pack2(b[2], b[3], T()));
  } else {
    *reinterpret_cast<uint4*>(row + 8 * l) = make_uint4(pack2(a[0], b[0], T()), pack2(a[1], b[1], T()),
                                                        pack2(a[2], b[2], T()), pack2(a[3], b[3], T()));
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
    const uint32_t i = static_cast<uint32_t>(n);    // the grid has fewer than 2^31 tokens
    const uint32_t row = static_cast<uint32_t>((static_cast<uint64_t>(i) * r.mw) >> r.sw);
    const uint32_t fr = static_cast<uint32_t>((static_cast<uint64_t>(row) * r.mh) >> r.sh);
    p[2] = r.first[2] + static_cast<int>(i - row * r.gw);
    p[1] = r.first[1] + static_cast<int>(row - fr * r.gh);
    p[0] = r.first[0] + static_cast<int>(fr);
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

// (x, y) = (u c + v s, w c + z s) forms below are fused multiply-adds in packed
// pairs: -v for a subtraction is a sign flip of both halves.
__device__ __forceinline__ uint64_t f2neg(uint64_t v) { return v ^ 0x8000000080000000ull; }

template <bool SPLIT, int D, typename T>
__device__ __forceinline__ Row8 lane_weight(const void* w, int w_f32, int l) {
  if (w == nullptr) {
    const uint64_t one = f2pack(1.f, 1.f);
    return Row8{{one, one}, {one, one}};
  }
  if (w_f32) {
    Vec8<float> v;
    load8<SPLIT, D>(static_cast<const float*>(w), l, v);
    return to_row<SPLIT>(v);
  }
  Vec8<T> v;
  load8<SPLIT, D>(static_cast<const T*>(w), l, v);
  return to_row<SPLIT>(v);
}

template <int D>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float f2sum(uint64_t v) {
  float a, b;
  f2unpack(v, a, b);
  return a + b;
}

// Forward: rotation, with the norm before it when NORM.  Grid (blocks over the
// tokens, tensors, parts of the heads).
template <typename T, int D, bool SPLIT, bool NORM>
__global__ void __launch_bounds__(kRopeThreads, kRopeFwdCtas) rope_fwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int G = D / 8;                            // lanes per row
  constexpr int kGroups = kRopeThreads / G, kRows = rope_rows<T>();
  const RopeTensor& t = p.t[blockIdx.y];
  const int h0 = blockIdx.z * p.per, heads = min(p.per, t.H - h0);
  if (heads <= 0) return;
  const int l = threadIdx.x % G;
  LanePairs lp;
  lane_pairs(p.r, l, lp);
  Row8 w;
  if (NORM) w = lane_weight<SPLIT, D, T>(t.w, p.w_f32, l);
  // every lane of a warp runs the same number of steps (the butterflies take
  // the whole warp); groups past the last token load and store nothing
  for (long long base = static_cast<long long>(blockIdx.x) * kGroups; base < p.N;
       base += static_cast<long long>(gridDim.x) * kGroups) {
    const long long n = base + threadIdx.x / G;
    const bool on = n < p.N;
    const T* x = static_cast<const T*>(t.x) + n * t.xt + h0 * t.xh;
    T* y = static_cast<T*>(t.y) + n * t.yt + h0 * t.yh;
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (on) lane_angles(p.r, lp, n, c, s);
    // y_a = a ca + b sb, y_b = a sa + b cb, with the weights of a and b inside
    uint64_t ca[2], sb[2], sa[2], cb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t cc = f2pack(c[2 * i], c[2 * i + 1]), ss = f2pack(s[2 * i], s[2 * i + 1]);
      ca[i] = NORM ? fmul2(cc, w.a[i]) : cc;
      cb[i] = NORM ? fmul2(cc, w.b[i]) : cc;
      sa[i] = NORM ? fmul2(ss, w.a[i]) : ss;
      sb[i] = f2neg(NORM ? fmul2(ss, w.b[i]) : ss);
    }
    // an unturned pair is a copy, even next to an infinity
    const bool turned = s[0] != 0.f && s[1] != 0.f && s[2] != 0.f && s[3] != 0.f;
#pragma unroll 1
    for (int b = 0; b < heads; b += kRows) {
      Vec8<T> v[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u)
        if (on && b + u < heads) load8<SPLIT, D>(x + (b + u) * t.xh, l, v[u]);
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (b + u >= heads) break;                    // the same for the whole block
        const Row8 f = to_row<SPLIT>(v[u]);
        Row8 o;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          o.a[i] = ffma2(f.b[i], sb[i], fmul2(f.a[i], ca[i]));
          o.b[i] = ffma2(f.a[i], sa[i], fmul2(f.b[i], cb[i]));
        }
        if (NORM) {
          const uint64_t q = ffma2(f.b[1], f.b[1], ffma2(f.a[1], f.a[1], ffma2(f.b[0], f.b[0], fmul2(f.a[0], f.a[0]))));
          const float ss = group_sum<D>(f2sum(q));
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          const uint64_t rr = f2pack(r, r);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            o.a[i] = fmul2(o.a[i], rr);
            o.b[i] = fmul2(o.b[i], rr);
          }
        } else if (!turned) {
          float a[4], e[4], oa[4], oe[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            f2unpack(f.a[i], a[2 * i], a[2 * i + 1]);
            f2unpack(f.b[i], e[2 * i], e[2 * i + 1]);
            f2unpack(o.a[i], oa[2 * i], oa[2 * i + 1]);
            f2unpack(o.b[i], oe[2 * i], oe[2 * i + 1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            oa[i] = s[i] != 0.f ? oa[i] : a[i] * c[i];
            oe[i] = s[i] != 0.f ? oe[i] : e[i] * c[i];
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            o.a[i] = f2pack(oa[2 * i], oa[2 * i + 1]);
            o.b[i] = f2pack(oe[2 * i], oe[2 * i + 1]);
          }
        }
        if (on) store8<SPLIT, D>(y + (b + u) * t.yh, l, o);
      }
    }
  }
}

// Backward of the norm and rotation.  Weight gradients: every lane sums its
// channels over its rows, a block's groups are added in a fixed order, and
// rope_dw_kernel adds the blocks' partial sums, again in a fixed order, so
// that the result does not change from run to run.
template <typename T, int D, bool SPLIT>
__global__ void __launch_bounds__(kRopeThreads, kRopeBwdCtas) rope_bwd_kernel(const __grid_constant__ RopeParams p) {
  constexpr int G = D / 8;
  constexpr int kGroups = kRopeThreads / G, kRows = rope_rows<T>(), kStages = kRopeBwdStages;
  constexpr uint32_t kRow = sizeof(T) == 4 ? 2 * kRopeSlots : kRopeSlots, kStage = 2 * kRows * kRow;   // x, g
  extern __shared__ __align__(128) uint8_t smem_rope[];
  __shared__ __align__(16) float s_dw[kGroups][D];
  const RopeTensor& t = p.t[blockIdx.y];
  const int h0 = blockIdx.z * p.per, heads = min(p.per, t.H - h0);
  const int l = threadIdx.x % G;
  const uint32_t slot = smem_u32(smem_rope) + threadIdx.x * 16;
  const long long first = static_cast<long long>(blockIdx.x) * kGroups, stride = static_cast<long long>(gridDim.x) * kGroups;
  long long ahead = first;
  int ahead_b = 0;
  const T* xa = static_cast<const T*>(t.x) + (first + threadIdx.x / G) * t.xt + h0 * t.xh;
  const T* ga = static_cast<const T*>(t.g) + (first + threadIdx.x / G) * t.gt + h0 * t.gh;
  auto load = [&](int stage) {
    if (ahead + threadIdx.x / G < p.N) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (ahead_b + u < heads) {
          copy8<SPLIT, D>(slot + stage * kStage + 2 * u * kRow, xa + (ahead_b + u) * t.xh, l);
          copy8<SPLIT, D>(slot + stage * kStage + (2 * u + 1) * kRow, ga + (ahead_b + u) * t.gh, l);
        }
      }
    }
    cp_async_commit();
    ahead_b += kRows;
    if (ahead_b >= heads) {
      ahead_b = 0;
      ahead += stride;
      xa += stride * t.xt;
      ga += stride * t.gt;
    }
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(i);
  LanePairs lp;
  lane_pairs(p.r, l, lp);
  const Row8 w = lane_weight<SPLIT, D, T>(t.w, p.w_f32, l);
  const uint64_t zero = f2pack(0.f, 0.f);
  Row8 dw{{zero, zero}, {zero, zero}};
  int stage = 0;
  for (long long base = first; base < p.N; base += stride) {
    const long long n = base + threadIdx.x / G;
    const bool on = n < p.N;
    T* y = static_cast<T*>(t.y) + n * t.yt + h0 * t.yh;
    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (on) lane_angles(p.r, lp, n, c, s);            // s: of the angle turned back
    const uint64_t cc[2] = {f2pack(c[0], c[1]), f2pack(c[2], c[3])};
    const uint64_t ss[2] = {f2pack(s[0], s[1]), f2pack(s[2], s[3])};
#pragma unroll 1
    for (int b = 0; b < heads; b += kRows) {
      cp_async_wait<kStages - 2>();
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (b + u >= heads) break;                    // the same for the whole block
        Vec8<T> vx, vg;
        read8(slot + stage * kStage + 2 * u * kRow, vx);
        read8(slot + stage * kStage + (2 * u + 1) * kRow, vg);
        const Row8 fx = to_row<SPLIT>(vx), fg = to_row<SPLIT>(vg);
        Row8 z, zx;                                   // g turned back, and times x
        uint64_t q = zero, dot = zero;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          z.a[i] = ffma2(f2neg(fg.b[i]), ss[i], fmul2(fg.a[i], cc[i]));
          z.b[i] = ffma2(fg.a[i], ss[i], fmul2(fg.b[i], cc[i]));
          zx.a[i] = fmul2(z.a[i], fx.a[i]);
          zx.b[i] = fmul2(z.b[i], fx.b[i]);
          q = ffma2(fx.b[i], fx.b[i], ffma2(fx.a[i], fx.a[i], q));
          dot = ffma2(zx.b[i], w.b[i], ffma2(zx.a[i], w.a[i], dot));
        }
        const float sq = group_sum<D>(f2sum(q));
        const float sd = group_sum<D>(f2sum(dot));
        const float r = rsqrtf(sq * (1.f / D) + p.eps);
        const float m = -(sd * r) * (1.f / D) * r * r;   // -mean(g w xh) r^2: dx = r g w + x m
        const uint64_t rr = f2pack(r, r), mm = f2pack(m, m);
        if (on) {
          Row8 o;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            dw.a[i] = ffma2(zx.a[i], rr, dw.a[i]);
            dw.b[i] = ffma2(zx.b[i], rr, dw.b[i]);
            o.a[i] = ffma2(fx.a[i], mm, fmul2(fmul2(z.a[i], w.a[i]), rr));
            o.b[i] = ffma2(fx.b[i], mm, fmul2(fmul2(z.b[i], w.b[i]), rr));
          }
          store8<SPLIT, D>(y + (b + u) * t.yh, l, o);
        }
      }
      load(stage == 0 ? kStages - 1 : stage - 1);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }
  }
  cp_async_wait<0>();
  // channels of the pairs
  store8<SPLIT, D>(s_dw[threadIdx.x / G], l, dw);
  __syncthreads();
  if (threadIdx.x < D) {
    float sum = 0.f;
#pragma unroll
    for (int gr = 0; gr < kGroups; ++gr) sum += s_dw[gr][threadIdx.x];
    const size_t block = (static_cast<size_t>(blockIdx.y) * gridDim.z + blockIdx.z) * gridDim.x + blockIdx.x;
    p.partial[block * D + threadIdx.x] = sum;
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
