// bsa_lib.cu - C ABI of libbsa.so (declared in include/bsa.h).
//
// Host side of every call: argument validation (before anything is
// enqueued), TMA tensor-map encoding, workspace carving and kernel launches
// on the caller's stream.  The library allocates no memory and never
// synchronises except in bsa_get_device_status.  Everything is one
// translation unit so the per-device status word is a single symbol.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <algorithm>
#include <atomic>
#include <mutex>
#include <numeric>

#include "ptx.cuh"
#include "lvsa_index.cuh"
#include "losa_select.cuh"
#include "attn_fwd.cuh"
#include "blockmass.cuh"
#include "rope.cuh"
#include "blockmean.cuh"
#include "attn_bwd.cuh"

namespace {

using namespace bsa;

constexpr long long kWaitLimitNs = 1500000000LL;   // 1.5 s per device-side wait
constexpr int kMaxDevices = 64;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 3-D view (d, H, N) of a bf16 [N, H, d] tensor; box (64, 1, rows), 128B swizzle.
bool make_qkv_map(CUtensorMap* m, const void* ptr, int N, int H, int d, int rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(N)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(H) * d * 2};
  cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int n_tiles(int N) { return (N + 127) / 128; }

int check_qkv(const void* q, const void* k, const void* v, int N, int H, int d, const void* o, const float* lse) {
  if (!q || !k || !v || !o || !lse) return BSA_ERR_ARG;
  if (N < 1 || H < 1 || H > 65535) return BSA_ERR_ARG;
  if (d != 64 && d != 128) return BSA_ERR_UNSUPPORTED;
  if (static_cast<long long>(N) * H * d >= (1LL << 31)) return BSA_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4))
    return BSA_ERR_ARG;
  return BSA_OK;
}

// grid over query-tile pairs x `grid_heads` heads, from head prm.h_off
template <int D, bool MASS>
int launch_attn(const void* q, const void* k, const void* v, int N, int H, int grid_heads, const AttnParams& prm,
                cudaStream_t st) {
  using L = AttnSmem<D, MASS>;
  // set once per device; concurrent first calls may both set it (idempotent)
  static std::atomic<bool> attr_set[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return BSA_ERR_CUDA;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(attn_tile_kernel<D, MASS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(L::kAlloc)) != cudaSuccess)
      return BSA_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  CUtensorMap mq, mk, mv, mo;
  // query, key, value and output tiles are all 128 rows (boxes of 128 rows x 64 channels)
  if (!make_qkv_map(&mq, q, N, H, D, 128) || !make_qkv_map(&mk, k, N, H, D, 128) ||
      !make_qkv_map(&mv, v, N, H, D, 128) || !make_qkv_map(&mo, prm.o, N, H, D, 128))
    return BSA_ERR_CUDA;
  dim3 grid((prm.nB + kQTilesPerCta - 1) / kQTilesPerCta, grid_heads);
  attn_tile_kernel<D, MASS><<<grid, kAttnThreads, L::kAlloc, st>>>(mq, mk, mv, mo, prm);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

int launch_attn_any(int d, bool mass, const void* q, const void* k, const void* v, int N, int H, int grid_heads,
                    const AttnParams& prm, cudaStream_t st) {
  if (d == 128) return mass ? launch_attn<128, true>(q, k, v, N, H, grid_heads, prm, st)
                            : launch_attn<128, false>(q, k, v, N, H, grid_heads, prm, st);
  return mass ? launch_attn<64, true>(q, k, v, N, H, grid_heads, prm, st)
              : launch_attn<64, false>(q, k, v, N, H, grid_heads, prm, st);
}

AttnParams base_params(int N, int H, float scale, void* o, float* lse) {
  AttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.N = N;
  p.H = H;
  p.nB = n_tiles(N);
  p.sl2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.wait_limit_ns = kWaitLimitNs;
  return p;
}

// Workspace of the one-pass dense measuring step, per head: log2 partial
// sums [nB key tiles][N rows] float32.
size_t dense_mass_head_bytes(int N) { return static_cast<size_t>(n_tiles(N)) * static_cast<size_t>(N) * 4; }

// Forward in mass mode over head passes of `hc` heads, each followed by the
// block-mass reduction.  With `unvisited`, the log partial sums are first
// set to NaN (all bytes 0xFF): entries of tiles the index never reaches keep
// it and the reduction counts them as no mass.
int blockmass_passes(const void* q, const void* k, const void* v, int N, int H, int d, AttnParams p, float* lpart,
                     int hc, bool unvisited, const float* lse, float* mass, cudaStream_t st) {
  const int nB = n_tiles(N);
  const size_t per_head = dense_mass_head_bytes(N);
  for (int h0 = 0; h0 < H; h0 += hc) {
    const int hn = std::min(hc, H - h0);
    if (unvisited && cudaMemsetAsync(lpart, 0xFF, per_head * hn, st) != cudaSuccess) return BSA_ERR_CUDA;
    p.lpart = lpart;
    p.h_off = h0;
    int rc = launch_attn_any(d, true, q, k, v, N, H, hn, p, st);
    if (rc != BSA_OK) return rc;
    const dim3 grid((nB + kMassWarps - 1) / kMassWarps, (nB + kMassKt - 1) / kMassKt, hn);
    blockmass_reduce_kernel<<<grid, kMassThreads, 0, st>>>(lpart, lse, mass, N, nB, h0);
    if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
  }
  return BSA_OK;
}

// Workspace layout for LVSA frame indexes.
struct LvsaWs {
  size_t fbits, cnt, idx, flag, total;
};
LvsaWs lvsa_ws_layout(int N, int T) {
  const size_t nB = static_cast<size_t>(n_tiles(N));
  const size_t TW = static_cast<size_t>((T + 31) / 32);
  LvsaWs w;
  w.fbits = 0;
  w.cnt = round_up(w.fbits + static_cast<size_t>(T) * TW * 4, 256);
  w.idx = round_up(w.cnt + nB * 4, 256);
  w.flag = round_up(w.idx + nB * nB * 4, 256);
  w.total = round_up(w.flag + nB * nB, 256);
  return w;
}

// Workspace bytes an index needs (LVSA tile lists; for the intersection also
// its per-entry flags [H][nB][nB]); (size_t)-1 for an invalid index.
size_t index_ws_bytes(const bsa_index* index, int N, int H) {
  if (!index) return static_cast<size_t>(-1);
  if (index->kind == BSA_INDEX_BLOCKS) return 0;
  if (index->kind != BSA_INDEX_LVSA_FRAMES && index->kind != BSA_INDEX_LVSA_BLOCKS) return static_cast<size_t>(-1);
  if (index->T < 1 || index->T > kMaxFrames || N % index->T) return static_cast<size_t>(-1);
  const size_t nB = static_cast<size_t>(n_tiles(N));
  size_t t = lvsa_ws_layout(N, index->T).total;
  if (index->kind == BSA_INDEX_LVSA_BLOCKS) t += round_up(static_cast<size_t>(H) * nB * nB, 256);
  return t;
}

// Workspace of the attention's gradient: the index's own part, the padded
// per-row values, the bit sets of the lists (shared by all heads for LVSA frame
// indexes) and room for the lists the other way round.
struct BwdWs {
  size_t nl, nd, bits, part, tlist, total;
  int lists;                        // heads with lists of their own (1: shared)
};
BwdWs bwd_ws_layout(const bsa_index* index, int N, int H) {
  BwdWs w;
  std::memset(&w, 0, sizeof(w));
  const size_t ix = index_ws_bytes(index, N, H);
  if (ix == static_cast<size_t>(-1)) {
    w.total = ix;
    return w;
  }
  const size_t nB = static_cast<size_t>(n_tiles(N)), nW = (nB + 31) / 32;
  const size_t lists = index->kind == BSA_INDEX_LVSA_FRAMES ? 1 : static_cast<size_t>(H);
  w.lists = static_cast<int>(lists);
  w.nl = round_up(ix, 256);
  w.nd = w.nl + static_cast<size_t>(H) * nB * 128 * 4;
  w.bits = w.nd + static_cast<size_t>(H) * nB * 128 * 4;
  w.part = round_up(w.bits + lists * nW * nB * 4, 256);
  w.tlist = index->kind == BSA_INDEX_BLOCKS ? w.part : round_up(w.part + lists * nW * nB * 4, 256);
  w.total = round_up(w.tlist + static_cast<size_t>(H) * nB * nB * 4, 256);
  return w;
}

// Validates `index`, enqueues its expansion (LVSA frame sets -> tile lists,
// flags of the intersection) and fills the list fields of `p`; *used = the
// workspace bytes taken from its start.
int setup_index(const bsa_index* index, int N, int H, void* workspace, size_t ws_bytes, AttnParams& p,
                size_t* used, cudaStream_t st) {
  const int nB = p.nB;
  *used = 0;
  const bool lvsa = index->kind == BSA_INDEX_LVSA_FRAMES || index->kind == BSA_INDEX_LVSA_BLOCKS;
  const bool blocks = index->kind == BSA_INDEX_BLOCKS || index->kind == BSA_INDEX_LVSA_BLOCKS;
  if (!lvsa && !blocks) return BSA_ERR_ARG;
  if (blocks) {
    if (index->block != 128) return BSA_ERR_UNSUPPORTED;
    if (index->H != H || index->nQB != nB || index->nKB != nB) return BSA_ERR_SHAPE;
    if (!index->idx || !index->cnt) return BSA_ERR_ARG;
    p.list = index->idx;
    p.count = index->cnt;
    p.flags = nullptr;
    p.lhs = static_cast<long long>(index->nQB) * index->nKB;
    p.lrs = index->nKB;
    p.chs = index->nQB;
  }
  if (lvsa) {
    const int T = index->T;
    if (T < 1 || T > kMaxFrames) return BSA_ERR_ARG;
    if (N % T) return BSA_ERR_SHAPE;
    if (!index->frames || !index->counts) return BSA_ERR_ARG;
    const LvsaWs w = lvsa_ws_layout(N, T);
    const size_t need = index_ws_bytes(index, N, H);
    if (!workspace || ws_bytes < need || !aligned(workspace, 256)) return BSA_ERR_WORKSPACE;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    uint32_t* fbits = reinterpret_cast<uint32_t*>(ws + w.fbits);
    int32_t* tcnt = reinterpret_cast<int32_t*>(ws + w.cnt);
    int32_t* tidx = reinterpret_cast<int32_t*>(ws + w.idx);
    uint8_t* tflag = ws + w.flag;
    lvsa_frame_bits_kernel<<<(T + 3) / 4, 128, 0, st>>>(T, index->frames, index->counts, fbits);
    lvsa_tiles_kernel<<<(nB + 3) / 4, 128, 0, st>>>(N, T, N / T, nB, fbits, tcnt, tidx, tflag);
    p.fbits = fbits;
    p.TW = (T + 31) / 32;
    p.P = N / T;
    if (blocks) {
      uint8_t* cflag = ws + w.total;
      compose_flags_kernel<<<static_cast<unsigned>(H) * nB, 256, 0, st>>>(nB, index->idx, index->cnt, tcnt, tidx,
                                                                        tflag, cflag);
      p.flags = cflag;
    } else {
      p.list = tidx;
      p.count = tcnt;
      p.flags = tflag;
      p.lhs = 0;
      p.lrs = nB;
      p.chs = 0;
    }
    if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
    *used = need;
  }
  return BSA_OK;
}

}  // namespace

extern "C" {

const char* bsa_version(void) { return "bsa-b200 0.1 (sm_100a)"; }

const char* bsa_status_string(int s) {
  switch (s) {
    case BSA_OK: return "BSA_OK";
    case BSA_WARN_OVER_BUDGET: return "BSA_WARN_OVER_BUDGET";
    case BSA_ERR_ARG: return "BSA_ERR_ARG";
    case BSA_ERR_SHAPE: return "BSA_ERR_SHAPE";
    case BSA_ERR_CUDA: return "BSA_ERR_CUDA";
    case BSA_ERR_INDEX_RANGE: return "BSA_ERR_INDEX_RANGE";
    case BSA_ERR_TIMEOUT: return "BSA_ERR_TIMEOUT";
    case BSA_ERR_UNSUPPORTED: return "BSA_ERR_UNSUPPORTED";
    case BSA_ERR_WORKSPACE: return "BSA_ERR_WORKSPACE";
    default: return "BSA_UNKNOWN_STATUS";
  }
}

int lvsa_build_index(int T, int T_per, int W, int C, int step, int32_t* frames, int32_t* counts, void* stream) {
  if (T < 1 || T > kMaxFrames || T_per < 1 || W < 1 || C < 1 || step < 0) return BSA_ERR_ARG;
  if (!frames || !counts || !aligned(frames, 4) || !aligned(counts, 4)) return BSA_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int threads = 128;
  lvsa_build_index_kernel<<<(T + threads - 1) / threads, threads, 0, st>>>(T, T_per, C, step, frames, counts);
  if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
  // over budget iff some t has |G_s u {t}| > C (pure function of the scalars)
  const int s_mod = step % T_per;
  const int nG = (s_mod < T) ? (T - 1 - s_mod) / T_per + 1 : 0;
  const bool has_non_anchor = nG < T;
  const bool over = (nG > C) || (has_non_anchor && nG + 1 > C);
  return over ? BSA_WARN_OVER_BUDGET : BSA_OK;
}

int lvsa_build_index_window(int T, int T_per, int W, int step, int32_t* frames, int32_t* counts, void* stream) {
  if (T < 1 || T > kMaxFrames || T_per < 1 || W < 1 || step < 0) return BSA_ERR_ARG;
  // |G_s| = number of f in [0, T) with f = step mod T_per (mod T_per)
  const int s_mod = step % T_per;
  const int nG = (s_mod < T) ? (T - 1 - s_mod) / T_per + 1 : 0;
  const int C = static_cast<int>(std::min<long long>(T, static_cast<long long>(nG) + W));
  // |G_s u {t}| <= min(T, nG + 1) <= C, so the fill never reports over budget
  return lvsa_build_index(T, T_per, W, C, step, frames, counts, stream);
}

size_t bsa_workspace_bytes(int op, int N, int H, int d, const bsa_index* index) {
  if (N < 1 || H < 1 || (d != 64 && d != 128)) return static_cast<size_t>(-1);
  const size_t per_head = dense_mass_head_bytes(N);
  // head shares of log partial sums: every head in one pass, up to 4 GiB
  const size_t heads = std::max<size_t>(1, std::min<size_t>(static_cast<size_t>(H), (size_t(4) << 30) / per_head));
  if (op == BSA_OP_DENSE_BLOCKMASS) return per_head * heads;
  if (op == BSA_OP_BLOCKSPARSE_BWD) return bwd_ws_layout(index, N, H).total;
  if (op != BSA_OP_BLOCKSPARSE_FWD && op != BSA_OP_BLOCKMASS) return static_cast<size_t>(-1);
  const size_t ix = index_ws_bytes(index, N, H);
  if (ix == static_cast<size_t>(-1)) return ix;
  return op == BSA_OP_BLOCKSPARSE_FWD ? ix : round_up(ix, 256) + per_head * heads;
}

int blocksparse_attn_fwd(const void* q, const void* k, const void* v, int N, int H, int d, float scale,
                         const bsa_index* index, void* o, float* lse, void* workspace, size_t ws_bytes,
                         void* stream) {
  int rc = check_qkv(q, k, v, N, H, d, o, lse);
  if (rc != BSA_OK) return rc;
  if (!index || !std::isfinite(scale)) return BSA_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  AttnParams p = base_params(N, H, scale, o, lse);
  size_t used = 0;
  rc = setup_index(index, N, H, workspace, ws_bytes, p, &used, st);
  if (rc != BSA_OK) return rc;
  return launch_attn_any(d, false, q, k, v, N, H, H, p, st);
}

int attn_blockmass(const void* q, const void* k, const void* v, int N, int H, int d, float scale,
                   const bsa_index* index, void* o, float* lse, float* mass, void* workspace, size_t ws_bytes,
                   void* stream) {
  int rc = check_qkv(q, k, v, N, H, d, o, lse);
  if (rc != BSA_OK) return rc;
  if (!index || !mass || !aligned(mass, 4) || !std::isfinite(scale)) return BSA_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  AttnParams p = base_params(N, H, scale, o, lse);
  size_t used = 0;
  rc = setup_index(index, N, H, workspace, ws_bytes, p, &used, st);
  if (rc != BSA_OK) return rc;
  const size_t off = round_up(used, 256);
  const size_t per_head = dense_mass_head_bytes(N);
  if (!workspace || ws_bytes < off || ws_bytes - off < per_head) return BSA_ERR_WORKSPACE;
  float* lpart = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + off);
  const int hc = static_cast<int>(std::min<size_t>(static_cast<size_t>(H), (ws_bytes - off) / per_head));
  return blockmass_passes(q, k, v, N, H, d, p, lpart, hc, /*unvisited=*/true, lse, mass, st);
}

int attn_dense_blockmass(const void* q, const void* k, const void* v, int N, int H, int d, int block, float scale,
                         void* o, float* lse, float* mass, void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_qkv(q, k, v, N, H, d, o, lse);
  if (rc != BSA_OK) return rc;
  if (!mass || !aligned(mass, 4) || !std::isfinite(scale)) return BSA_ERR_ARG;
  if (block != 128) return BSA_ERR_UNSUPPORTED;
  const size_t per_head = dense_mass_head_bytes(N);
  if (!workspace || !aligned(workspace, 256) || ws_bytes < per_head) return BSA_ERR_WORKSPACE;
  AttnParams p = base_params(N, H, scale, o, lse);
  p.dense = 1;
  const int hc = static_cast<int>(std::min<size_t>(static_cast<size_t>(H), ws_bytes / per_head));
  // every (row, key tile) is visited: no need to mark the workspace first
  return blockmass_passes(q, k, v, N, H, d, p, static_cast<float*>(workspace), hc, false, lse, mass,
                          static_cast<cudaStream_t>(stream));
}

int losa_select(const float* mass, int H, int nQB, int nKB, double tau, int32_t* idx, int32_t* cnt, void* stream) {
  if (!mass || !idx || !cnt || !aligned(mass, 4) || !aligned(idx, 4) || !aligned(cnt, 4)) return BSA_ERR_ARG;
  if (H < 1 || nQB < 1 || nKB < 1) return BSA_ERR_ARG;
  if (nKB > kSelectMaxBlocks) return BSA_ERR_UNSUPPORTED;
  if (!(tau > 0.0 && tau <= 1.0)) return BSA_ERR_ARG;
  const long long rows = static_cast<long long>(H) * nQB;
  if (rows > 0x7FFFFFFFLL) return BSA_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // rows of up to 2048 blocks: keys in registers, 8 warps (one row each) per CTA
  if (nKB <= 2048) {
    const int wpc = 8;
    const long long ctas = std::min<long long>((rows + wpc - 1) / wpc, 1LL << 20);
    const dim3 grid(static_cast<unsigned>(ctas)), block(wpc * 32);
    const int r = static_cast<int>(rows);
    if (nKB <= 256)
      losa_select_reg_kernel<8><<<grid, block, 0, st>>>(mass, r, nKB, tau, idx, cnt);
    else if (nKB <= 512)
      losa_select_reg_kernel<16><<<grid, block, 0, st>>>(mass, r, nKB, tau, idx, cnt);
    else if (nKB <= 1024)
      losa_select_reg_kernel<32><<<grid, block, 0, st>>>(mass, r, nKB, tau, idx, cnt);
    else
      losa_select_reg_kernel<64><<<grid, block, 0, st>>>(mass, r, nKB, tau, idx, cnt);
    return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
  }
  // longer rows: keys in shared memory, warps per CTA sized to <= 96 KB
  const size_t row_bytes = static_cast<size_t>(nKB) * 8;
  const int wpc = static_cast<int>(std::min<size_t>(8, std::max<size_t>(1, (96 * 1024) / row_bytes)));
  const size_t smem = row_bytes * wpc;
  static std::atomic<bool> attr_set[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return BSA_ERR_CUDA;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    // largest request: 96 KB (several warps) or one row of kSelectMaxBlocks keys (64 KB)
    if (cudaFuncSetAttribute(losa_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024) !=
        cudaSuccess)
      return BSA_ERR_CUDA;
    attr_set[dev].store(true, std::memory_order_release);
  }
  const long long ctas = std::min<long long>((rows + wpc - 1) / wpc, 1LL << 20);
  losa_select_kernel<<<static_cast<unsigned>(ctas), wpc * 32, smem, st>>>(mass, static_cast<int>(rows), nKB, tau,
                                                                         idx, cnt);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

int bsa_get_device_status(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return BSA_ERR_CUDA;
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_bsa_status, sizeof(int)) != cudaSuccess) return BSA_ERR_CUDA;
  if (cudaMemcpyToSymbol(g_bsa_status, &zero, sizeof(int)) != cudaSuccess) return BSA_ERR_CUDA;
  return v;
}

}  // extern "C"

namespace {
__global__ void debug_expired_wait_kernel(long long limit_ns, int form) {
  __shared__ alignas(8) unsigned long long bar;
  const uint32_t b = smem_u32(&bar);
  if (threadIdx.x == 0) {
    mbar_init(b, 1);
    fence_mbar_init();
  }
  __syncthreads();
  // nothing ever arrives on this barrier: the wait must give up by itself
  if (form == 0) {
    if (threadIdx.x == 0) mbar_wait(b, 0, limit_ns);
  } else {
    // the whole-warp form: every lane must see the same (false) result
    const bool ok = mbar_wait_warp(b, 0, limit_ns);
    if (__any_sync(0xFFFFFFFFu, ok) && threadIdx.x == 0) atomicExch(&g_bsa_status, BSA_ERR_ARG);
  }
}
}  // namespace

extern "C" int bsa_debug_expired_wait(long long limit_ns, int form, void* stream) {
  if (limit_ns < 100000LL || limit_ns > 10000000000LL || form < 0 || form > 1) return BSA_ERR_ARG;
  debug_expired_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(limit_ns, form);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// blocksparse_attn_fwd_noalloc: the workspace of blocksparse_attn_fwd placed in
// a file-scope device array, for callers that cannot allocate device memory.
// Host code must not use the array's name as a device address: the address
// is looked up once per device with cudaGetSymbolAddress (that device
// current) and passed on like a caller-owned workspace.
namespace {
constexpr size_t kNoAllocScratchBytes = BSA_NOALLOC_SCRATCH_BYTES;
__device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];
void* g_noalloc_ptr[kMaxDevices] = {};
std::mutex g_noalloc_mu;
}  // namespace

extern "C" int blocksparse_attn_fwd_noalloc(const void* q, const void* k, const void* v, int N, int H, int d,
                                            float scale, const bsa_index* index, void* o, float* lse,
                                            void* stream) {
  if (!index || N < 1 || H < 1) return BSA_ERR_ARG;
  if (index->kind == BSA_INDEX_LVSA_FRAMES || index->kind == BSA_INDEX_LVSA_BLOCKS) {
    // frame lists need the tile lists; the intersection also H * nB * nB flag bytes
    if (index->T < 1 || index->T > kMaxFrames) return BSA_ERR_ARG;
    if (N % index->T) return BSA_ERR_SHAPE;
    if (index_ws_bytes(index, N, H) > kNoAllocScratchBytes) return BSA_ERR_WORKSPACE;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return BSA_ERR_CUDA;
  void* scratch = nullptr;
  {
    std::lock_guard<std::mutex> lock(g_noalloc_mu);
    if (!g_noalloc_ptr[dev]) {
      void* p = nullptr;
      if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) return BSA_ERR_CUDA;
      g_noalloc_ptr[dev] = p;
    }
    scratch = g_noalloc_ptr[dev];
  }
  return blocksparse_attn_fwd(q, k, v, N, H, d, scale, index, o, lse, scratch, kNoAllocScratchBytes, stream);
}

// ---------------------------------------------------------------------------
// Rotary positions and the normed rotation of queries and keys.
namespace {

// per-device opt-in to large dynamic shared memory, set once per kernel
template <typename K>
int allow_smem(K* kernel, int bytes, std::atomic<bool>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return BSA_ERR_CUDA;
  if (!done[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
      return BSA_ERR_CUDA;
    done[dev].store(true, std::memory_order_release);
  }
  return BSA_OK;
}

int esize(int dtype) { return dtype == BSA_F32 ? 4 : 2; }

// rows of an output tensor must not overlap
bool rows_apart(const bsa_heads* t, long long N, int d) {
  const long long lo = std::min(t->token_stride, t->head_stride), hi = std::max(t->token_stride, t->head_stride);
  if (N == 1) return t->H == 1 || t->head_stride >= d;
  if (t->H == 1) return t->token_stride >= d;
  const long long inner = t->token_stride < t->head_stride ? N : t->H;
  return lo >= d && hi / lo >= inner;
}

int check_heads(const bsa_heads* t, int dtype, long long N, int d, bool out) {
  if (!t || !t->data || t->H < 1 || t->H > 65535 || t->token_stride < 0 || t->head_stride < 0) return BSA_ERR_ARG;
  const size_t es = esize(dtype);
  if (!aligned(t->data, 16) || (t->token_stride * es) % 16 || (t->head_stride * es) % 16) return BSA_ERR_ARG;
  // byte offsets stay far below 2^63
  if (t->token_stride > (1LL << 60) / N || t->head_stride > (1LL << 60) / t->H) return BSA_ERR_UNSUPPORTED;
  if (out && !rows_apart(t, N, d)) return BSA_ERR_ARG;
  return BSA_OK;
}

// Whether two tensors share memory: for tokens the same stride apart in both (as
// slices of one projection are) the exact answer; with token strides of their own,
// or more than 2^20 pairs of heads to go through, any common range counts.
bool share_memory(const bsa_heads* a, const bsa_heads* b, int dtype, long long N, int d) {
  const long long ats = N > 1 ? a->token_stride : 0, bts = N > 1 ? b->token_stride : 0;
  const long long ahs = a->H > 1 ? a->head_stride : 0, bhs = b->H > 1 ? b->head_stride : 0;
  const long long aw = (a->H - 1) * ahs + d, bw = (b->H - 1) * bhs + d;         // a token's range
  const long long diff = (reinterpret_cast<intptr_t>(b->data) - reinterpret_cast<intptr_t>(a->data)) / esize(dtype);
  if (diff >= (N - 1) * ats + aw || -diff >= (N - 1) * bts + bw) return false;
  if (ats != bts) return true;
  auto apart = [&](long long period, long long wa, long long wb) {              // modulo `period`
    if (period == 0) return false;
    const long long r = (diff % period + period) % period;
    return r >= wa && r + wb <= period;
  };
  if (apart(ats, aw, bw) || apart(std::gcd(std::gcd(ats, ahs), bhs), d, d)) return false;
  // rows h of a and g of b meet where |x + n ats| < d for a number n of tokens between them
  auto meet = [&](long long x) {
    if (ats == 0) return -d < x && x < d;
    auto floor_div = [&](long long y) { return y / ats - (y % ats < 0 ? 1 : 0); };
    return std::max(-floor_div(x + d - 1), 1 - N) <= std::min(floor_div(d - 1 - x), N - 1);
  };
  if (ahs == bhs || a->H == 1 || b->H == 1) {
    const long long hs = std::max(ahs, bhs);
    for (long long h = 1 - a->H; h < b->H; ++h)
      if (meet(diff + h * hs)) return true;
    return false;
  }
  if (static_cast<long long>(a->H) * b->H > (1 << 20)) return true;
  for (long long h = 0; h < a->H; ++h)
    for (long long g = 0; g < b->H; ++g)
      if (meet(diff + g * bhs - h * ahs)) return true;
  return false;
}

// An output next to a tensor that it may replace (its own input or gradient, with
// the same layout) or, without `own`, to any other.
bool in_the_way(const bsa_heads* out, const bsa_heads* t, int dtype, long long N, int d, bool own) {
  if (own && out->data == t->data && out->H == t->H && (N == 1 || out->token_stride == t->token_stride) &&
      (t->H == 1 || out->head_stride == t->head_stride))
    return false;
  return share_memory(out, t, dtype, N, d);
}

int check_sizes(int dtype, long long N, int d) {
  if (dtype != BSA_BF16 && dtype != BSA_F16 && dtype != BSA_F32) return BSA_ERR_ARG;
  if (N < 1) return BSA_ERR_ARG;
  if (d != 64 && d != 128) return BSA_ERR_UNSUPPORTED;
  if (N > (1LL << 40)) return BSA_ERR_UNSUPPORTED;
  return BSA_OK;
}

// n / d = (n * m) >> s for 0 <= n < 2^31 and 1 <= d < 2^31: with 2^(l-1) < d <= 2^l
// and m = floor(2^(31+l) / d) + 1 (33 bits at most; 32 because d > 2^(l-1)), m d
// is above 2^(31+l) by at most 2^l, so that n m / 2^(31+l) is above n / d by less
// than 1 / d.
void division(uint32_t d, uint32_t* m, int* s) {
  int l = 0;
  while ((1u << l) < d) ++l;
  *m = static_cast<uint32_t>((1ull << (31 + l)) / d + 1);
  *s = 31 + l;
}

// rope may be null: nothing is turned
int rope_dev(const bsa_rope* rope, long long N, int d, bool inverse, RopeDev* r) {
  std::memset(r, 0, sizeof(*r));
  r->sign = inverse ? -1.f : 1.f;
  r->gh = r->gw = 1;
  division(1, &r->mh, &r->sh);
  division(1, &r->mw, &r->sw);
  if (!rope) return BSA_OK;
  if (rope->pairing != BSA_ROPE_ADJACENT && rope->pairing != BSA_ROPE_SPLIT) return BSA_ERR_ARG;
  long long sum = 0;
  for (int a = 0; a < 3; ++a) {
    if (rope->pairs[a] < 0) return BSA_ERR_ARG;
    sum += rope->pairs[a];
    if (rope->pairs[a] == 0) continue;
    if (rope->len[a] < 1 || !rope->table[a] || !aligned(rope->table[a], 8)) return BSA_ERR_ARG;
    r->table[a] = rope->table[a];
    r->pairs[a] = rope->pairs[a];
    r->len[a] = rope->len[a];
  }
  if (sum < 1 || sum > d / 2) return BSA_ERR_SHAPE;
  if (rope->pos) {
    if (!aligned(rope->pos, 4)) return BSA_ERR_ARG;
    r->pos = rope->pos;
    return BSA_OK;
  }
  long long n = 1;
  for (int a = 0; a < 3; ++a) {
    if (rope->grid[a] < 1 || rope->first[a] < 0) return BSA_ERR_ARG;
    n *= rope->grid[a];
    if (n > N || n >= (1LL << 31)) return BSA_ERR_SHAPE;
    if (rope->pairs[a] > 0 && static_cast<long long>(rope->first[a]) + rope->grid[a] > rope->len[a])
      return BSA_ERR_SHAPE;
    r->first[a] = rope->first[a];
  }
  r->gh = rope->grid[1];
  r->gw = rope->grid[2];
  division(r->gh, &r->mh, &r->sh);
  division(r->gw, &r->mw, &r->sw);
  r->ngrid = n;
  return BSA_OK;
}

void set_tensor(RopeTensor* t, const bsa_heads* x, const bsa_heads* g, const bsa_heads* y, const void* w) {
  t->x = x ? x->data : nullptr;
  t->xt = x ? x->token_stride : 0;
  t->xh = x ? x->head_stride : 0;
  t->g = g ? g->data : nullptr;
  t->gt = g ? g->token_stride : 0;
  t->gh = g ? g->head_stride : 0;
  t->y = y->data;
  t->yt = y->token_stride;
  t->yh = y->head_stride;
  t->H = y->H;
  t->w = w;
}

// Grid of a rotation: blocks over the tokens (at most `most` in all, as many as
// are resident; each strides), tensors, parts of the heads.  A block takes all heads of its tokens,
// so that their angles are looked up once; with too few tokens to fill the
// SMs the heads are dealt to several blocks, kRopeHeads at the least.
dim3 rope_grid(RopeParams* p, int tensors, int d, long long most) {
  const int groups = kRopeThreads / (d / 8);
  int H = 1;
  for (int i = 0; i < tensors; ++i) H = std::max(H, p->t[i].H);
  const long long blocks = (p->N + groups - 1) / groups;
  p->per = H;
  int parts = 1;
  while (p->per > kRopeHeads && blocks * tensors * parts < 2 * 148) {
    p->per = std::max(kRopeHeads, (p->per / 2 + kRopeHeads - 1) / kRopeHeads * kRopeHeads);
    parts = (H + p->per - 1) / p->per;
  }
  const long long x = std::max(1LL, std::min(blocks, most / (static_cast<long long>(tensors) * parts)));
  return dim3(static_cast<unsigned>(x), tensors, parts);
}

template <typename T, int D, bool SPLIT, bool NORM>
int launch_rope_fwd(RopeParams& p, int tensors, cudaStream_t st) {
  const dim3 grid = rope_grid(&p, tensors, D, 148 * kRopeFwdCtas);
  rope_fwd_kernel<T, D, SPLIT, NORM><<<grid, kRopeThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

template <typename T, int D>
int launch_rope_fwd(RopeParams& p, int tensors, bool split, bool norm, cudaStream_t st) {
  if (split) return norm ? launch_rope_fwd<T, D, true, true>(p, tensors, st) : launch_rope_fwd<T, D, true, false>(p, tensors, st);
  return norm ? launch_rope_fwd<T, D, false, true>(p, tensors, st) : launch_rope_fwd<T, D, false, false>(p, tensors, st);
}

int launch_rope_fwd_any(RopeParams& p, int dtype, int d, int tensors, bool split, bool norm, cudaStream_t st) {
  if (d == 128) {
    if (dtype == BSA_BF16) return launch_rope_fwd<__nv_bfloat16, 128>(p, tensors, split, norm, st);
    if (dtype == BSA_F16) return launch_rope_fwd<__half, 128>(p, tensors, split, norm, st);
    return launch_rope_fwd<float, 128>(p, tensors, split, norm, st);
  }
  if (dtype == BSA_BF16) return launch_rope_fwd<__nv_bfloat16, 64>(p, tensors, split, norm, st);
  if (dtype == BSA_F16) return launch_rope_fwd<__half, 64>(p, tensors, split, norm, st);
  return launch_rope_fwd<float, 64>(p, tensors, split, norm, st);
}

// most blocks of the backward pass (all tensors and parts of the heads): their
// weight-gradient partial sums are added by one block per tensor afterwards
constexpr long long kRopeBwdBlocks = 148 * kRopeBwdCtas;

template <typename T, int D, bool SPLIT>
int launch_rope_bwd(const RopeParams& p, dim3 grid, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  const int rc = allow_smem(rope_bwd_kernel<T, D, SPLIT>, kRopeRing, done);
  if (rc != BSA_OK) return rc;
  rope_bwd_kernel<T, D, SPLIT><<<grid, kRopeThreads, kRopeRing, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

template <typename T, int D>
int launch_rope_bwd(const RopeParams& p, bool split, dim3 grid, cudaStream_t st) {
  return split ? launch_rope_bwd<T, D, true>(p, grid, st) : launch_rope_bwd<T, D, false>(p, grid, st);
}

int launch_rope_bwd_any(const RopeParams& p, int dtype, int d, bool split, dim3 grid, cudaStream_t st) {
  if (d == 128) {
    if (dtype == BSA_BF16) return launch_rope_bwd<__nv_bfloat16, 128>(p, split, grid, st);
    if (dtype == BSA_F16) return launch_rope_bwd<__half, 128>(p, split, grid, st);
    return launch_rope_bwd<float, 128>(p, split, grid, st);
  }
  if (dtype == BSA_BF16) return launch_rope_bwd<__nv_bfloat16, 64>(p, split, grid, st);
  if (dtype == BSA_F16) return launch_rope_bwd<__half, 64>(p, split, grid, st);
  return launch_rope_bwd<float, 64>(p, split, grid, st);
}

// weight type and pointers of the norm
int check_weights(const void* wq, const void* wk, int dtype, int wtype, float eps) {
  if (wtype != BSA_F32 && wtype != dtype) return BSA_ERR_ARG;
  if ((wq && !aligned(wq, 16)) || (wk && !aligned(wk, 16))) return BSA_ERR_ARG;
  if (!std::isfinite(eps) || !(eps > 0.f)) return BSA_ERR_ARG;
  return BSA_OK;
}

}  // namespace

extern "C" {

int rope_build_table(int len, int pairs, double theta, double start, double step, float* table, void* stream) {
  if (len < 1 || pairs < 1 || !table || !aligned(table, 8)) return BSA_ERR_ARG;
  if (!std::isfinite(theta) || !(theta > 0.0) || !std::isfinite(start) || !std::isfinite(step)) return BSA_ERR_ARG;
  const long long n = static_cast<long long>(len) * pairs;
  if (n > (1LL << 37)) return BSA_ERR_UNSUPPORTED;
  rope_table_kernel<<<static_cast<unsigned>((n + 127) / 128), 128, 0, static_cast<cudaStream_t>(stream)>>>(
      len, pairs, theta, start, step, table);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

int rope_apply(const bsa_heads* x, const bsa_heads* y, int dtype, long long N, int d, const bsa_rope* rope,
               int inverse, void* stream) {
  int rc = check_sizes(dtype, N, d);
  if (rc != BSA_OK) return rc;
  if (!rope) return BSA_ERR_ARG;
  if ((rc = check_heads(x, dtype, N, d, false)) != BSA_OK) return rc;
  if ((rc = check_heads(y, dtype, N, d, true)) != BSA_OK) return rc;
  if (x->H != y->H) return BSA_ERR_SHAPE;
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.N = N;
  if ((rc = rope_dev(rope, N, d, inverse != 0, &p.r)) != BSA_OK) return rc;
  if (in_the_way(y, x, dtype, N, d, true)) return BSA_ERR_ARG;
  set_tensor(&p.t[0], x, nullptr, y, nullptr);
  return launch_rope_fwd_any(p, dtype, d, 1, rope->pairing == BSA_ROPE_SPLIT, false,
                             static_cast<cudaStream_t>(stream));
}

int qk_norm_rope_fwd(const bsa_heads* q, const bsa_heads* k, const bsa_heads* qo, const bsa_heads* ko, int dtype,
                     long long N, int d, const void* wq, const void* wk, int wtype, float eps, const bsa_rope* rope,
                     void* stream) {
  int rc = check_sizes(dtype, N, d);
  if (rc != BSA_OK) return rc;
  if ((rc = check_weights(wq, wk, dtype, wtype, eps)) != BSA_OK) return rc;
  if ((k == nullptr) != (ko == nullptr)) return BSA_ERR_ARG;
  const int tensors = k ? 2 : 1;
  for (int i = 0; i < tensors; ++i) {
    const bsa_heads* x = i ? k : q;
    const bsa_heads* y = i ? ko : qo;
    if ((rc = check_heads(x, dtype, N, d, false)) != BSA_OK) return rc;
    if ((rc = check_heads(y, dtype, N, d, true)) != BSA_OK) return rc;
    if (x->H != y->H) return BSA_ERR_SHAPE;
  }
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.N = N;
  p.eps = eps;
  p.w_f32 = wtype == BSA_F32;
  if ((rc = rope_dev(rope, N, d, false, &p.r)) != BSA_OK) return rc;
  if (in_the_way(qo, q, dtype, N, d, true)) return BSA_ERR_ARG;
  if (k && (in_the_way(ko, k, dtype, N, d, true) || in_the_way(qo, k, dtype, N, d, false) ||
            in_the_way(ko, q, dtype, N, d, false) || in_the_way(qo, ko, dtype, N, d, false)))
    return BSA_ERR_ARG;
  set_tensor(&p.t[0], q, nullptr, qo, wq);
  if (k) set_tensor(&p.t[1], k, nullptr, ko, wk);
  return launch_rope_fwd_any(p, dtype, d, tensors, rope && rope->pairing == BSA_ROPE_SPLIT, true,
                             static_cast<cudaStream_t>(stream));
}

size_t qk_norm_rope_bwd_workspace_bytes(long long N, int Hq, int Hk, int d) {
  if (N < 1 || Hq < 1 || Hk < 0 || (d != 64 && d != 128)) return static_cast<size_t>(-1);
  // the grid's parts of the heads number at most ceil(H / kRopeHeads), a tensor's
  // blocks at least one each
  const size_t parts = static_cast<size_t>(std::max(Hq, Hk) + kRopeHeads - 1) / kRopeHeads;
  return std::max<size_t>(kRopeBwdBlocks, 2 * parts) * d * sizeof(float);
}

int qk_norm_rope_bwd(const bsa_heads* gq, const bsa_heads* gk, const bsa_heads* q, const bsa_heads* k,
                     const bsa_heads* dq, const bsa_heads* dk, int dtype, long long N, int d, const void* wq,
                     const void* wk, int wtype, float eps, const bsa_rope* rope, float* dwq, float* dwk,
                     void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_sizes(dtype, N, d);
  if (rc != BSA_OK) return rc;
  if ((rc = check_weights(wq, wk, dtype, wtype, eps)) != BSA_OK) return rc;
  if ((k == nullptr) != (gk == nullptr) || (k == nullptr) != (dk == nullptr)) return BSA_ERR_ARG;
  if (!k && dwk) return BSA_ERR_ARG;
  if ((dwq && !aligned(dwq, 4)) || (dwk && !aligned(dwk, 4))) return BSA_ERR_ARG;
  const int tensors = k ? 2 : 1;
  for (int i = 0; i < tensors; ++i) {
    const bsa_heads* x = i ? k : q;
    const bsa_heads* g = i ? gk : gq;
    const bsa_heads* y = i ? dk : dq;
    if ((rc = check_heads(x, dtype, N, d, false)) != BSA_OK) return rc;
    if ((rc = check_heads(g, dtype, N, d, false)) != BSA_OK) return rc;
    if ((rc = check_heads(y, dtype, N, d, true)) != BSA_OK) return rc;
    if (x->H != y->H || g->H != y->H) return BSA_ERR_SHAPE;
  }
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  p.N = N;
  p.eps = eps;
  p.w_f32 = wtype == BSA_F32;
  if ((rc = rope_dev(rope, N, d, true, &p.r)) != BSA_OK) return rc;
  if (!workspace || !aligned(workspace, 256) ||
      ws_bytes < qk_norm_rope_bwd_workspace_bytes(N, q->H, k ? k->H : 0, d))
    return BSA_ERR_WORKSPACE;
  for (const bsa_heads* t : {q, gq})
    if (in_the_way(dq, t, dtype, N, d, true) || (k && in_the_way(dk, t, dtype, N, d, false))) return BSA_ERR_ARG;
  if (k) {
    for (const bsa_heads* t : {k, gk})
      if (in_the_way(dk, t, dtype, N, d, true) || in_the_way(dq, t, dtype, N, d, false)) return BSA_ERR_ARG;
    if (in_the_way(dq, dk, dtype, N, d, false)) return BSA_ERR_ARG;
  }
  set_tensor(&p.t[0], q, gq, dq, wq);
  if (k) set_tensor(&p.t[1], k, gk, dk, wk);
  p.partial = static_cast<float*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid = rope_grid(&p, tensors, d, kRopeBwdBlocks);
  rc = launch_rope_bwd_any(p, dtype, d, rope && rope->pairing == BSA_ROPE_SPLIT, grid, st);
  if (rc != BSA_OK || (!dwq && !dwk)) return rc;
  rope_dw_kernel<<<tensors, 1024, 0, st>>>(p.partial, static_cast<int>(grid.x * grid.z), d, dwq, dwk);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Key blocks by block means.
namespace {

// Workspace: means (64-bit), norms, the two bf16 parts, rough scores of the
// heads of one pass.
struct MeanWs {
  size_t mean, norm, hi, lo, scores, total;
  size_t per_head;                  // scores of one head
  int ldS;                          // floats per row of scores
  int heads;                        // heads per pass
};
// Scores of one pass: small enough to stay in L2 (126 MB) between the kernel
// that writes them and the one that reads them.
constexpr size_t kMeanPassBytes = size_t(64) << 20;
constexpr int kMeanExactBlocks = 8;                   // at most kSelKeys: the keys stay in shared memory
static_assert(kMeanExactBlocks <= kSelKeys, "keys of a row without rough scores");

MeanWs mean_ws_layout(int N, int H, int d) {
  const size_t nB = static_cast<size_t>(n_tiles(N)), elems = static_cast<size_t>(2) * H * nB * d;
  MeanWs w;
  w.ldS = static_cast<int>(round_up(nB, 8));          // rows of whole 32-byte sectors
  w.per_head = nB * w.ldS * 4;
  w.heads = static_cast<int>(std::max<size_t>(1, std::min<size_t>(H, kMeanPassBytes / w.per_head)));
  w.mean = 0;
  w.norm = elems * 8;
  w.hi = round_up(w.norm + static_cast<size_t>(2) * H * nB * 8, 256);
  w.lo = round_up(w.hi + elems * 2, 256);
  w.scores = round_up(w.lo + elems * 2, 256);
  w.total = round_up(w.scores + w.per_head * w.heads, 256);
  return w;
}

// (d, nB, heads) of a bf16 [heads][nB][d] array, boxes of 64 x 128 x 1
bool make_means_map(CUtensorMap* m, const void* ptr, int d, int nB, int heads) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(nB), static_cast<cuuint64_t>(heads)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(nB) * d * 2};
  cuuint32_t box[3] = {64, 128, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int C4>
int launch_mean_select(const MeanWs& w, uint8_t* ws, int H, int h0, int heads, int nB, int keep, int local,
                       int32_t* idx, int32_t* cnt, cudaStream_t st, bool rough = true) {
  size_t smem = 0;
  if (C4 == 0) {                                      // rows in shared memory
    static std::atomic<bool> done[kMaxDevices];
    smem = static_cast<size_t>(sel_warps(C4)) * w.ldS * 4;
    int rc = allow_smem(blockmean_select_kernel<D, C4>, sel_warps(C4) * kMeanMaxBlocks * 4, done);
    if (rc != BSA_OK) return rc;
  }
  const dim3 grid((nB + sel_warps(C4) - 1) / sel_warps(C4), heads);
  blockmean_select_kernel<D, C4><<<grid, sel_warps(C4) * 32, smem, st>>>(
      reinterpret_cast<const double*>(ws + w.mean), reinterpret_cast<const double*>(ws + w.norm),
      rough ? reinterpret_cast<float*>(ws + w.scores) : nullptr, w.ldS, H, h0, nB, keep, local, idx, cnt);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

// [N, H * d] bf16 as rows, boxes of 32 tokens x 256 channels
bool make_rows_map(CUtensorMap* m, const void* ptr, int N, int row) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(N)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(row) * 2};
  cuuint32_t box[2] = {256, 32};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launch_pool(const MeanWs& w, uint8_t* ws, const void* q, const void* k, int N, int H, int d, int nB,
                cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  int rc = allow_smem(blockmean_pool_kernel, static_cast<int>(PoolSmem::kAlloc), done);
  if (rc != BSA_OK) return rc;
  CUtensorMap mq, mk;
  if (!make_rows_map(&mq, q, N, H * d) || !make_rows_map(&mk, k, N, H * d)) return BSA_ERR_CUDA;
  const long long tiles = 2LL * nB * ((H * d + 255) / 256);
  const unsigned blocks = static_cast<unsigned>(std::min<long long>(tiles, 148 * kPoolCtas));
  blockmean_pool_kernel<<<blocks, kPoolThreads, PoolSmem::kAlloc, st>>>(
      mq, mk, static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), N, H, d, nB,
      reinterpret_cast<double*>(ws + w.mean), reinterpret_cast<__nv_bfloat16*>(ws + w.hi),
      reinterpret_cast<__nv_bfloat16*>(ws + w.lo), reinterpret_cast<double*>(ws + w.norm), kWaitLimitNs);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

template <int D>
int launch_mean(const MeanWs& w, uint8_t* ws, int H, int nB, int keep, int local, int32_t* idx, int32_t* cnt,
                cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  int rc = allow_smem(blockmean_score_kernel<D>, static_cast<int>(ScoreSmem<D>::kAlloc), done);
  if (rc != BSA_OK) return rc;
  // few blocks: 64-bit scores of all cost less than the rough ones' launch (8
  // blocks: 31.2 against 36.5 us for a call alone with 2 heads, 36.4 against 42.7
  // with 40)
  if (nB <= kMeanExactBlocks) return launch_mean_select<D, 2>(w, ws, H, 0, H, nB, keep, local, idx, cnt, st, false);
  CUtensorMap mh, ml;
  if (!make_means_map(&mh, ws + w.hi, D, nB, 2 * H) || !make_means_map(&ml, ws + w.lo, D, nB, 2 * H))
    return BSA_ERR_CUDA;
  const unsigned tiles = static_cast<unsigned>((nB + 127) / 128);
  for (int h0 = 0; h0 < H; h0 += w.heads) {
    const int hn = std::min(w.heads, H - h0);
    const dim3 grid((tiles + kScoreTiles - 1) / kScoreTiles, tiles, hn);
    blockmean_score_kernel<D><<<grid, kScoreThreads, ScoreSmem<D>::kAlloc, st>>>(
        mh, ml, reinterpret_cast<float*>(ws + w.scores), w.ldS, H, h0, nB, kWaitLimitNs);
    if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
    // the fewest chunks of 128 blocks that hold the row: every step of the search
    // goes through all of them (1025, 1280, 1536 blocks, 12 heads of 128, whole call:
    // 250, 335, 408 us with 12 chunks, 273, 371, 444 us with 16)
    if (nB <= 256) rc = launch_mean_select<D, 2>(w, ws, H, h0, hn, nB, keep, local, idx, cnt, st);
    else if (nB <= 512) rc = launch_mean_select<D, 4>(w, ws, H, h0, hn, nB, keep, local, idx, cnt, st);
    else if (nB <= 1024) rc = launch_mean_select<D, 8>(w, ws, H, h0, hn, nB, keep, local, idx, cnt, st);
    else if (nB <= 1536) rc = launch_mean_select<D, 12>(w, ws, H, h0, hn, nB, keep, local, idx, cnt, st);
    else if (nB <= 2048) rc = launch_mean_select<D, 16>(w, ws, H, h0, hn, nB, keep, local, idx, cnt, st);
    else rc = launch_mean_select<D, 0>(w, ws, H, h0, hn, nB, keep, local, idx, cnt, st);
    if (rc != BSA_OK) return rc;
  }
  return BSA_OK;
}

}  // namespace

extern "C" {

size_t blockmean_select_workspace_bytes(int N, int H, int d) {
  if (N < 1 || H < 1 || H > 32767 || (d != 64 && d != 128) || n_tiles(N) > kMeanMaxBlocks)
    return static_cast<size_t>(-1);
  return mean_ws_layout(N, H, d).total;
}

int blockmean_select(const void* q, const void* k, int N, int H, int d, int block, int keep, int local, int32_t* idx,
                     int32_t* cnt, void* workspace, size_t ws_bytes, void* stream) {
  if (!q || !k || !idx || !cnt || !aligned(q, 16) || !aligned(k, 16) || !aligned(idx, 4) || !aligned(cnt, 4))
    return BSA_ERR_ARG;
  if (N < 1 || H < 1 || keep < 1 || local < -1) return BSA_ERR_ARG;
  if (block != 128 || (d != 64 && d != 128) || H > 32767) return BSA_ERR_UNSUPPORTED;
  if (static_cast<long long>(N) * H * d >= (1LL << 31) || n_tiles(N) > kMeanMaxBlocks) return BSA_ERR_UNSUPPORTED;
  const MeanWs w = mean_ws_layout(N, H, d);
  if (!workspace || !aligned(workspace, 256) || ws_bytes < w.total) return BSA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int nB = n_tiles(N);
  local = std::min(local, nB);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int rc = launch_pool(w, ws, q, k, N, H, d, nB, st);
  if (rc != BSA_OK) return rc;
  rc = d == 128 ? launch_mean<128>(w, ws, H, nB, keep, local, idx, cnt, st)
                          : launch_mean<64>(w, ws, H, nB, keep, local, idx, cnt, st);
  if (rc != BSA_OK) return rc;
  // the widest neighbourhood of any row
  return std::min<long long>(nB, 2LL * local + 1) > keep ? BSA_WARN_OVER_BUDGET : BSA_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Gradient of the block-sparse attention.
namespace {

template <int D, bool ONE>
int launch_bwd(const void* go, const void* q, const void* k, const void* v, int N, int H, const BwdParams& p,
               void* dq, void* dk, void* dv, cudaStream_t st) {
  static std::atomic<bool> done[kMaxDevices];
  const int rc = allow_smem(attn_bwd_kernel<D, ONE>, static_cast<int>(BwdSmem<D>::kAlloc), done);
  if (rc != BSA_OK) return rc;
  CUtensorMap mq, mk, mv, mg, mdq, mdk, mdv;
  if (!make_qkv_map(&mq, q, N, H, D, 128) || !make_qkv_map(&mk, k, N, H, D, 128) ||
      !make_qkv_map(&mv, v, N, H, D, 128) || !make_qkv_map(&mg, go, N, H, D, 128) ||
      !make_qkv_map(&mdq, dq, N, H, D, 128) || !make_qkv_map(&mdk, dk, N, H, D, 128) ||
      !make_qkv_map(&mdv, dv, N, H, D, 128))
    return BSA_ERR_CUDA;
  // all key tiles first where the blocks fill the SMs fewer than eight times
  const bool apart = 2LL * p.nB * H < 8 * 148;
  const dim3 grid(apart ? p.nB : 2 * p.nB, H, apart ? 2 : 1);
  attn_bwd_kernel<D, ONE><<<grid, kBwdThreads, BwdSmem<D>::kAlloc, st>>>(mq, mk, mv, mg, mdq, mdk, mdv, p);
  return cudaGetLastError() == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace

extern "C" int blocksparse_attn_bwd(const void* go, const void* q, const void* k, const void* v, const bsa_heads* o,
                                    const float* lse, int N, int H, int d, float scale, const bsa_index* index,
                                    void* dq, void* dk, void* dv, void* workspace, size_t ws_bytes, void* stream) {
  int rc = check_qkv(q, k, v, N, H, d, go, lse);
  if (rc != BSA_OK) return rc;
  if (!dq || !dk || !dv || !index || !std::isfinite(scale) || !(scale > 0.f)) return BSA_ERR_ARG;
  if (!aligned(dq, 16) || !aligned(dk, 16) || !aligned(dv, 16)) return BSA_ERR_ARG;
  if ((rc = check_heads(o, BSA_BF16, N, d, false)) != BSA_OK) return rc;
  if (o->H != H) return BSA_ERR_SHAPE;
  const size_t bytes = static_cast<size_t>(N) * H * d * 2;
  const size_t obytes = (static_cast<size_t>(N - 1) * o->token_stride + static_cast<size_t>(H - 1) * o->head_stride + d) * 2;
  const void* outs[3] = {dq, dk, dv};
  const void* ins[4] = {go, q, k, v};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 4; ++j)
      if (overlap(outs[i], bytes, ins[j], bytes)) return BSA_ERR_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], bytes, outs[j], bytes)) return BSA_ERR_ARG;
    if (overlap(outs[i], bytes, o->data, obytes)) return BSA_ERR_ARG;
    if (overlap(outs[i], bytes, lse, static_cast<size_t>(H) * N * 4)) return BSA_ERR_ARG;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  AttnParams a = base_params(N, H, scale, nullptr, nullptr);
  const BwdWs w = bwd_ws_layout(index, N, H);
  size_t used = 0;
  // what setup_index enqueues must fit too: check the whole workspace first
  if (w.total != static_cast<size_t>(-1) && (!workspace || !aligned(workspace, 256) || ws_bytes < w.total)) {
    const bool blocks = index->kind == BSA_INDEX_BLOCKS || index->kind == BSA_INDEX_LVSA_BLOCKS;
    if (blocks && index->block != 128) return BSA_ERR_UNSUPPORTED;
    if (blocks && (index->H != H || index->nQB != a.nB || index->nKB != a.nB)) return BSA_ERR_SHAPE;
    return BSA_ERR_WORKSPACE;
  }
  rc = setup_index(index, N, H, workspace, ws_bytes, a, &used, st);
  if (rc != BSA_OK) return rc;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int nB = a.nB;
  BwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.N = N;
  p.H = H;
  p.nB = nB;
  p.sl2 = a.sl2;
  p.scale = scale;
  p.list = a.list;
  p.count = a.count;
  p.flags = a.flags;
  p.lhs = a.lhs;
  p.lrs = a.lrs;
  p.chs = a.chs;
  p.fbits = a.fbits;
  p.TW = a.TW;
  p.P = a.P;
  p.wait_limit_ns = a.wait_limit_ns;
  float* nl = reinterpret_cast<float*>(ws + w.nl);
  float* nd = reinterpret_cast<float*>(ws + w.nd);
  uint32_t* bits = reinterpret_cast<uint32_t*>(ws + w.bits);
  uint32_t* part = a.flags ? reinterpret_cast<uint32_t*>(ws + w.part) : nullptr;
  p.nl = nl;
  p.nd = nd;
  p.bits = bits;
  p.part = part;
  p.bhs = w.lists == 1 ? 0 : static_cast<long long>((nB + 31) / 32) * nB;
  p.tlist = reinterpret_cast<int32_t*>(ws + w.tlist);
  const __nv_bfloat16* ob = static_cast<const __nv_bfloat16*>(o->data);
  const __nv_bfloat16* gb = static_cast<const __nv_bfloat16*>(go);
  // Whether a row can have as few keys as kFewKeys, or one: whole frames have P
  // each, listed blocks 128, but the last one what is left.
  const int last = N - 128 * (nB - 1);
  const int least = index->kind == BSA_INDEX_LVSA_FRAMES ? a.P : a.fbits != nullptr ? std::min(a.P, last) : last;
  const bool ones = least == 1;
  const bool few = index->kind == BSA_INDEX_LVSA_BLOCKS || least <= kFewKeys;   // parts of frames in blocks: any number
  const int threads = prep_threads(few), warps = threads / 32;
  const unsigned bit_blocks = static_cast<unsigned>((static_cast<long long>(w.lists) * nB + warps - 1) / warps);
  const long long lanes = static_cast<long long>(nB) * 128 * H * (d / 8);
  const unsigned blocks = bit_blocks + static_cast<unsigned>((lanes + threads - 1) / threads);
  auto* prep = d == 128 ? (few ? attn_bwd_prep_kernel<128, true> : attn_bwd_prep_kernel<128, false>)
                        : (few ? attn_bwd_prep_kernel<64, true> : attn_bwd_prep_kernel<64, false>);
  prep<<<blocks, threads, 0, st>>>(a.list, a.count, a.flags, a.lhs, a.lrs, a.chs, nB, w.lists, bit_blocks, bits, part, ob,
                               o->token_stride, o->head_stride, gb, lse, N, H, nl, nd, ones, static_cast<const __nv_bfloat16*>(q),
                               static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), p);
  if (cudaGetLastError() != cudaSuccess) return BSA_ERR_CUDA;
  auto* launch = d == 128 ? (ones ? launch_bwd<128, true> : launch_bwd<128, false>)
                          : (ones ? launch_bwd<64, true> : launch_bwd<64, false>);
  return launch(go, q, k, v, N, H, p, dq, dk, dv, st);
}
