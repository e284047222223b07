"""Python binding of libbsa.so: frame/block-sparse video attention on B200.

Argument marshalling only.  Every computation runs in the CUDA kernels of
``libbsa.so`` (see include/bsa.h for the contract of each call); torch is
used for device memory and streams.  The library must have been built
(``python -m block_sparse_attention_lvsa_b200.build``); importing this
package raises if it is missing - there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import Optional, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbsa.so")

BSA_OK = 0
BSA_WARN_OVER_BUDGET = 1
BSA_ERR_ARG = -1
BSA_ERR_SHAPE = -2
BSA_ERR_CUDA = -3
BSA_ERR_INDEX_RANGE = -4
BSA_ERR_TIMEOUT = -5
BSA_ERR_UNSUPPORTED = -6
BSA_ERR_WORKSPACE = -7

BSA_INDEX_LVSA_FRAMES = 1
BSA_INDEX_BLOCKS = 2
BSA_INDEX_LVSA_BLOCKS = 3
BSA_OP_BLOCKSPARSE_FWD = 1
BSA_OP_DENSE_BLOCKMASS = 2
BSA_OP_BLOCKMASS = 3
BSA_OP_BLOCKSPARSE_BWD = 4

BSA_BF16 = 0
BSA_F16 = 1
BSA_F32 = 2
BSA_ROPE_ADJACENT = 0
BSA_ROPE_SPLIT = 1

EXPORTED = ("lvsa_build_index", "lvsa_build_index_window", "attn_dense_blockmass", "attn_blockmass", "losa_select", "blocksparse_attn_fwd",
            "bsa_workspace_bytes", "bsa_get_device_status", "bsa_status_string",
            "bsa_debug_expired_wait", "bsa_version", "blocksparse_attn_fwd_noalloc",
            "rope_build_table", "rope_apply", "qk_norm_rope_fwd", "qk_norm_rope_bwd",
            "qk_norm_rope_bwd_workspace_bytes", "blockmean_select", "blockmean_select_workspace_bytes",
            "blocksparse_attn_bwd")


class BsaError(RuntimeError):
    def __init__(self, call: str, status: int):
        self.status = status
        super().__init__(f"{call} failed: {status_string(status)} ({status})")


class bsa_index(ctypes.Structure):
    """Mirror of ``struct bsa_index`` in include/bsa.h."""
    _fields_ = [
        ("kind", ctypes.c_int),
        ("T", ctypes.c_int),
        ("frames", ctypes.c_void_p),
        ("counts", ctypes.c_void_p),
        ("block", ctypes.c_int),
        ("H", ctypes.c_int),
        ("nQB", ctypes.c_int),
        ("nKB", ctypes.c_int),
        ("idx", ctypes.c_void_p),
        ("cnt", ctypes.c_void_p),
    ]


class bsa_heads(ctypes.Structure):
    """Mirror of ``struct bsa_heads`` in include/bsa.h."""
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("H", ctypes.c_int),
        ("token_stride", ctypes.c_longlong),
        ("head_stride", ctypes.c_longlong),
    ]


class bsa_rope(ctypes.Structure):
    """Mirror of ``struct bsa_rope`` in include/bsa.h."""
    _fields_ = [
        ("pairing", ctypes.c_int),
        ("pairs", ctypes.c_int * 3),
        ("len", ctypes.c_int * 3),
        ("table", ctypes.c_void_p * 3),
        ("grid", ctypes.c_int * 3),
        ("first", ctypes.c_int * 3),
        ("pos", ctypes.c_void_p),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m block_sparse_attention_lvsa_b200.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, D, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_double, ctypes.c_float, ctypes.c_size_t
    L, HP, RP = ctypes.c_longlong, ctypes.POINTER(bsa_heads), ctypes.POINTER(bsa_rope)
    sig = {
        "lvsa_build_index": (I, [I, I, I, I, I, P, P, P]),
        "lvsa_build_index_window": (I, [I, I, I, I, P, P, P]),
        "attn_dense_blockmass": (I, [P, P, P, I, I, I, I, F, P, P, P, P, SZ, P]),
        "attn_blockmass": (I, [P, P, P, I, I, I, F, ctypes.POINTER(bsa_index), P, P, P, P, SZ, P]),
        "losa_select": (I, [P, I, I, I, D, P, P, P]),
        "blocksparse_attn_fwd": (I, [P, P, P, I, I, I, F, ctypes.POINTER(bsa_index), P, P, P, SZ, P]),
        "bsa_workspace_bytes": (SZ, [I, I, I, I, ctypes.POINTER(bsa_index)]),
        "bsa_get_device_status": (I, [P]),
        "bsa_status_string": (ctypes.c_char_p, [I]),
        "bsa_debug_expired_wait": (I, [ctypes.c_longlong, I, P]),
        "bsa_version": (ctypes.c_char_p, []),
        "blocksparse_attn_fwd_noalloc": (I, [P, P, P, I, I, I, F, ctypes.POINTER(bsa_index), P, P, P]),
        "rope_build_table": (I, [I, I, D, D, D, P, P]),
        "rope_apply": (I, [HP, HP, I, L, I, RP, I, P]),
        "qk_norm_rope_fwd": (I, [HP, HP, HP, HP, I, L, I, P, P, I, F, RP, P]),
        "qk_norm_rope_bwd": (I, [HP, HP, HP, HP, HP, HP, I, L, I, P, P, I, F, RP, P, P, P, SZ, P]),
        "qk_norm_rope_bwd_workspace_bytes": (SZ, [L, I, I, I]),
        "blockmean_select": (I, [P, P, I, I, I, I, I, I, P, P, P, SZ, P]),
        "blockmean_select_workspace_bytes": (SZ, [I, I, I]),
        "blocksparse_attn_bwd": (I, [P, P, P, P, HP, P, I, I, I, F, ctypes.POINTER(bsa_index), P, P, P, P, SZ, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def lib():
    return _lib


def status_string(status: int) -> str:
    return _lib.bsa_status_string(int(status)).decode()


def version() -> str:
    return _lib.bsa_version().decode()


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _check(call: str, rc: int, allow=(BSA_OK,)) -> int:
    if rc not in allow:
        raise BsaError(call, rc)
    return rc


def _check_qkv(q, k, v):
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 3:
            raise ValueError("q, k, v must be contiguous bf16 CUDA tensors of shape [N, H, d]")
    if not (q.shape == k.shape == v.shape):
        raise ValueError("q, k, v shapes differ")


def _check_tensor(name: str, t: Optional[torch.Tensor], shape, dtype, device) -> None:
    """A caller-supplied buffer the library writes or reads by pointer: the C
    side cannot see its size, so dtype, shape, contiguity and device are
    checked here, before the call (a wrong one would mean out-of-bounds
    device accesses)."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != torch.device(device):
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _check_out(q: torch.Tensor, o: Optional[torch.Tensor], lse: Optional[torch.Tensor],
               mass: Optional[torch.Tensor] = None) -> None:
    """o like q (bf16 [N, H, d]), lse float32 [H, N], mass float32 [H, nB, nB]; same device as q."""
    N, H, _ = q.shape
    nB = math.ceil(N / 128)
    _check_tensor("o", o, q.shape, torch.bfloat16, q.device)
    _check_tensor("lse", lse, (H, N), torch.float32, q.device)
    _check_tensor("mass", mass, (H, nB, nB), torch.float32, q.device)


def _check_workspace(ws: Optional[torch.Tensor], device) -> None:
    if ws is None:
        return
    if not isinstance(ws, torch.Tensor) or not ws.is_contiguous() or ws.device != torch.device(device):
        raise ValueError(f"workspace must be a contiguous tensor on {device}")


# ----------------------------------------------------------------- calls ---
def lvsa_build_index(T: int, T_per: int, W: int, C: int, step: int,
                     frames: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                     device=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, bool]:
    """A(t) for every frame at ``step``: (frames [T,T] int32, counts [T] int32, over_budget)."""
    dev = device if device is not None else (frames.device if frames is not None else "cuda")
    _check_tensor("frames", frames, (T, T), torch.int32, dev)
    _check_tensor("counts", counts, (T,), torch.int32, dev)
    if frames is None:
        frames = torch.empty((T, T), dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty((T,), dtype=torch.int32, device=dev)
    rc = _lib.lvsa_build_index(T, T_per, W, C, step, _ptr(frames), _ptr(counts), _stream(stream))
    _check("lvsa_build_index", rc, (BSA_OK, BSA_WARN_OVER_BUDGET))
    return frames, counts, rc == BSA_WARN_OVER_BUDGET


def lvsa_build_index_window(T: int, T_per: int, W: int, step: int,
                            frames: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                            device=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """A(t) under the fixed-window reading (W non-anchor frames): (frames [T,T] int32, counts [T] int32)."""
    dev = device if device is not None else (frames.device if frames is not None else "cuda")
    _check_tensor("frames", frames, (T, T), torch.int32, dev)
    _check_tensor("counts", counts, (T,), torch.int32, dev)
    if frames is None:
        frames = torch.empty((T, T), dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty((T,), dtype=torch.int32, device=dev)
    rc = _lib.lvsa_build_index_window(T, T_per, W, step, _ptr(frames), _ptr(counts), _stream(stream))
    _check("lvsa_build_index_window", rc)
    return frames, counts


def lvsa_index(T: int, frames: torch.Tensor, counts: torch.Tensor) -> bsa_index:
    """Index of kind BSA_INDEX_LVSA_FRAMES over device frames [T, T] and counts [T] (int32)."""
    _check_tensor("frames", frames, (T, T), torch.int32, frames.device)
    _check_tensor("counts", counts, (T,), torch.int32, frames.device)
    ix = bsa_index()
    ix.kind = BSA_INDEX_LVSA_FRAMES
    ix.T = T
    ix.frames = frames.data_ptr()
    ix.counts = counts.data_ptr()
    ix._tensors = (frames, counts)         # the struct holds raw pointers: keep the tensors alive with it
    return ix


def block_index(idx: torch.Tensor, cnt: torch.Tensor, block: int = 128) -> bsa_index:
    """Index of kind BSA_INDEX_BLOCKS over device idx [H, nQB, nKB] and cnt [H, nQB] (int32)."""
    if not isinstance(idx, torch.Tensor) or idx.dim() != 3:
        raise ValueError("idx must be an int32 tensor [H, nQB, nKB]")
    H, nQB, nKB = idx.shape
    _check_tensor("idx", idx, (H, nQB, nKB), torch.int32, idx.device)
    _check_tensor("cnt", cnt, (H, nQB), torch.int32, idx.device)
    ix = bsa_index()
    ix.kind = BSA_INDEX_BLOCKS
    ix.block, ix.H, ix.nQB, ix.nKB = block, H, nQB, nKB
    ix.idx = idx.data_ptr()
    ix.cnt = cnt.data_ptr()
    ix._tensors = (idx, cnt)               # the struct holds raw pointers: keep the tensors alive with it
    return ix


def lvsa_block_index(T: int, frames: torch.Tensor, counts: torch.Tensor, idx: torch.Tensor, cnt: torch.Tensor,
                     block: int = 128) -> bsa_index:
    """Intersection index: LVSA frame sets (frames, counts) within per-head key-block lists (idx, cnt)."""
    ix = block_index(idx, cnt, block)
    ix.kind = BSA_INDEX_LVSA_BLOCKS
    ix.T = T
    ix.frames = frames.data_ptr()
    ix.counts = counts.data_ptr()
    ix._tensors = (frames, counts, idx, cnt)
    return ix


def workspace_bytes(op: int, N: int, H: int, d: int, index: Optional[bsa_index] = None) -> int:
    n = _lib.bsa_workspace_bytes(op, N, H, d, ctypes.byref(index) if index is not None else None)
    if n == ctypes.c_size_t(-1).value:
        raise BsaError("bsa_workspace_bytes", BSA_ERR_ARG)
    return int(n)


def blocksparse_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, index: bsa_index,
                         scale: Optional[float] = None, o: Optional[torch.Tensor] = None,
                         lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                         stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Masked attention restricted to ``index``; returns (o [N,H,d] bf16, lse [H,N] f32)."""
    _check_qkv(q, k, v)
    _check_out(q, o, lse)
    _check_workspace(workspace, q.device)
    N, H, d = q.shape
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((H, N), dtype=torch.float32, device=q.device)
    need = workspace_bytes(BSA_OP_BLOCKSPARSE_FWD, N, H, d, index)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.blocksparse_attn_fwd(_ptr(q), _ptr(k), _ptr(v), N, H, d, float(scale), ctypes.byref(index),
                                   _ptr(o), _ptr(lse), _ptr(workspace), ws_bytes, _stream(stream))
    _check("blocksparse_attn_fwd", rc)
    return o, lse


def blocksparse_attn_fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, index: bsa_index,
                                 o: torch.Tensor, lse: torch.Tensor, scale: Optional[float] = None,
                                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """blocksparse_attn_fwd without a workspace: the library's static scratch array is
    used instead, so the call allocates nothing (o and lse are the caller's)."""
    if o is None or lse is None:
        raise ValueError("blocksparse_attn_fwd_noalloc writes into the caller's o and lse")
    _check_qkv(q, k, v)
    _check_out(q, o, lse)
    N, H, d = q.shape
    if scale is None:
        scale = d ** -0.5
    rc = _lib.blocksparse_attn_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), N, H, d, float(scale), ctypes.byref(index),
                                           _ptr(o), _ptr(lse), _stream(stream))
    _check("blocksparse_attn_fwd_noalloc", rc)
    return o, lse


def attn_dense_blockmass(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block: int = 128,
                         scale: Optional[float] = None, o=None, lse=None, mass=None,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """Dense attention plus LoSA block mass; returns (o, lse, mass [H, nB, nB] f32).

    ``workspace`` (uint8 CUDA tensor, 256-byte aligned) holds at least one
    head's log partial sums, nB * N * 4 bytes; more heads per pass when larger.
    When omitted, ``workspace_bytes(BSA_OP_DENSE_BLOCKMASS, ...)`` bytes are allocated.
    """
    _check_qkv(q, k, v)
    _check_out(q, o, lse, mass)
    _check_workspace(workspace, q.device)
    N, H, d = q.shape
    nB = math.ceil(N / 128)
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((H, N), dtype=torch.float32, device=q.device)
    if mass is None:
        mass = torch.empty((H, nB, nB), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(workspace_bytes(BSA_OP_DENSE_BLOCKMASS, N, H, d), dtype=torch.uint8,
                                device=q.device)
    rc = _lib.attn_dense_blockmass(_ptr(q), _ptr(k), _ptr(v), N, H, d, block, float(scale),
                                   _ptr(o), _ptr(lse), _ptr(mass), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream))
    _check("attn_dense_blockmass", rc)
    return o, lse, mass


def attn_blockmass(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, index: bsa_index,
                   scale: Optional[float] = None, o=None, lse=None, mass=None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention restricted to ``index`` plus its LoSA block mass; returns (o, lse, mass [H, nB, nB] f32)."""
    _check_qkv(q, k, v)
    _check_out(q, o, lse, mass)
    _check_workspace(workspace, q.device)
    N, H, d = q.shape
    nB = math.ceil(N / 128)
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((H, N), dtype=torch.float32, device=q.device)
    if mass is None:
        mass = torch.empty((H, nB, nB), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(workspace_bytes(BSA_OP_BLOCKMASS, N, H, d, index), dtype=torch.uint8,
                                device=q.device)
    rc = _lib.attn_blockmass(_ptr(q), _ptr(k), _ptr(v), N, H, d, float(scale), ctypes.byref(index),
                             _ptr(o), _ptr(lse), _ptr(mass), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check("attn_blockmass", rc)
    return o, lse, mass


def losa_select(mass: torch.Tensor, tau: float = 0.99, idx=None, cnt=None, stream=None):
    """Minimal tau-mass key-block sets; returns (idx [H,nQB,nKB] int32 (-1 padded), cnt [H,nQB] int32)."""
    if mass.dtype != torch.float32 or not mass.is_cuda or not mass.is_contiguous() or mass.dim() != 3:
        raise ValueError("mass must be a contiguous float32 CUDA tensor [H, nQB, nKB]")
    H, nQB, nKB = mass.shape
    _check_tensor("idx", idx, (H, nQB, nKB), torch.int32, mass.device)
    _check_tensor("cnt", cnt, (H, nQB), torch.int32, mass.device)
    if idx is None:
        idx = torch.empty((H, nQB, nKB), dtype=torch.int32, device=mass.device)
    if cnt is None:
        cnt = torch.empty((H, nQB), dtype=torch.int32, device=mass.device)
    rc = _lib.losa_select(_ptr(mass), H, nQB, nKB, float(tau), _ptr(idx), _ptr(cnt), _stream(stream))
    _check("losa_select", rc)
    return idx, cnt


# ------------------------------------------- rotary positions, normed q and k ---
_DTYPES = {torch.bfloat16: BSA_BF16, torch.float16: BSA_F16, torch.float32: BSA_F32}
_PAIRINGS = {"adjacent": BSA_ROPE_ADJACENT, "split": BSA_ROPE_SPLIT}
_ROPE = struct.Struct("@i3i3i3P3i3iP")         # bsa_rope, packed in one go
# handle of a device's current stream, without a Stream object where torch's C module offers
# that (it has no such name in builds without CUDA, where the host checks still serve)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _enter(device: torch.device, stream):
    """Makes the tensors' device, and ``stream`` if given, current for a call; None where
    they are already.  What a call allocates then comes from that stream's pool and is
    not handed to other work while the call still uses it.  To be closed with _leave."""
    if stream is None:
        if device.index == torch.cuda.current_device():
            return None
        guard = torch.cuda.device(device)
    else:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        guard = torch.cuda.stream(stream)
    guard.__enter__()
    return guard


def _leave(guard) -> None:
    if guard is not None:
        guard.__exit__(None, None, None)


def _heads(name: str, t: torch.Tensor, like: Optional[torch.Tensor] = None, any_heads: bool = False) -> bsa_heads:
    """bsa_heads of a CUDA tensor [N, H, d] with unit channel stride (of the
    type, device and sizes of ``like``, but for H with ``any_heads``)."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES or not t.is_cuda or t.dim() != 3:
        raise ValueError(f"{name} must be a bf16, fp16 or fp32 CUDA tensor of shape [N, H, d]")
    shape = t.shape
    if like is not None:
        want = like.shape
        same = (shape[0] == want[0] and shape[2] == want[2]) if any_heads else shape == want
        if not same or t.dtype != like.dtype or t.device != like.device:
            raise ValueError(f"{name} must be {like.dtype} of shape {tuple(want)} on {like.device}, "
                             f"got {t.dtype} {tuple(shape)} on {t.device}")
    ts, hs, cs = t.stride()
    if cs != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have unit channel stride")
    return bsa_heads(t.data_ptr(), shape[1], ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0)


def _fresh(like: torch.Tensor):
    """A new contiguous [N, H, d] tensor of ``like``'s type and device, and its bsa_heads."""
    t = torch.empty_like(like, memory_format=torch.contiguous_format)
    _, H, d = t.shape
    return t, bsa_heads(t.data_ptr(), H, H * d, d)


def _weight(name: str, w: Optional[torch.Tensor], x: torch.Tensor):
    """The address of a norm weight [d], None without one."""
    if w is None:
        return None
    if not isinstance(w, torch.Tensor) or w.dtype not in (torch.float32, x.dtype):
        raise ValueError(f"{name} must be float32 or {x.dtype}")
    if w.dim() != 1 or w.shape[0] != x.shape[2] or not w.is_contiguous() or w.device != x.device:
        raise ValueError(f"{name} must be a contiguous [{x.shape[2]}] on {x.device}")
    return w.data_ptr()


def _weight_type(wq, wk, x) -> int:
    if wq is not None and wk is not None and wq.dtype != wk.dtype:
        raise ValueError("wq and wk must have the same dtype")
    w = wq if wq is not None else wk
    return BSA_F32 if w is None else _DTYPES[w.dtype]


def _rope_for(rope: Optional[bsa_rope], x: torch.Tensor):
    """The tables and positions are read by pointer: they must be on x's device and hold x's tokens."""
    if rope is None:
        return None
    if not isinstance(rope, bsa_rope):
        raise ValueError("rope must come from rope_axes")
    if rope._device != x.device:
        raise ValueError(f"the rotation's tables are on {rope._device}, the tensor on {x.device}")
    if rope._pos is not None and rope._pos.shape[0] != x.shape[0]:
        raise ValueError(f"pos holds {rope._pos.shape[0]} tokens, the tensor {x.shape[0]}")
    return rope


def rope_build_table(length: int, pairs: int, theta: float = 10000.0, start: float = 0.0, step: float = 1.0,
                     table: Optional[torch.Tensor] = None, device=None, stream=None) -> torch.Tensor:
    """cos and sin of one axis, float32 [length, pairs, 2]: row i, pair j holds the
    angle (start + i * step) * theta ** (-j / pairs)."""
    if length < 1 or pairs < 1:
        raise ValueError("length and pairs must be at least 1")
    if table is not None:
        device = table.device
        _check_tensor("table", table, (length, pairs, 2), torch.float32, device)
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError("the table must be on a CUDA device")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    guard = _enter(device, stream)
    try:
        if table is None:
            table = torch.empty((length, pairs, 2), dtype=torch.float32, device=device)
        rc = _lib.rope_build_table(length, pairs, theta, start, step, table.data_ptr(), _raw_stream(device.index))
    finally:
        _leave(guard)
    _check("rope_build_table", rc)
    return table


def rope_axes(tables, grid=None, first=(0, 0, 0), pos: Optional[torch.Tensor] = None,
              pairing: str = "adjacent") -> bsa_rope:
    """Rotary positions over up to three axes, for rope_apply and qk_norm_rope_*.

    ``tables``: one float32 [len, pairs, 2] per axis (rope_build_table), the
    outermost axis (time) first.  Either ``grid`` gives the extent of every
    axis (tokens row-major, starting at ``first``; tokens behind the grid are
    not turned), or ``pos`` (int32 [N, 3]) lists the positions (negative: not
    turned along that axis).  ``pairing``: "adjacent" channels 2j, 2j+1 or
    "split" channels j, j+d/2 form a pair."""
    n = len(tables)
    if not 1 <= n <= 3:
        raise ValueError("rope_axes takes one to three tables")
    if pairing not in _PAIRINGS:
        raise ValueError(f"pairing must be one of {tuple(_PAIRINGS)}")
    if (grid is None) == (pos is None):
        raise ValueError("give either grid or pos")
    dev = None
    pairs, lens, ptrs = [0, 0, 0], [0, 0, 0], [0, 0, 0]
    for a, t in enumerate(tables):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or t.dim() != 3 or not t.is_cuda or \
                t.shape[2] != 2 or not t.is_contiguous():
            raise ValueError("a table must be a contiguous float32 CUDA tensor [len, pairs, 2]")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"the tables are on {dev} and {t.device}")
        lens[a], pairs[a], _ = t.shape
        ptrs[a] = t.data_ptr()
    g, f = (1, 1, 1), (0, 0, 0)
    if pos is not None:
        _check_tensor("pos", pos, (pos.shape[0], 3), torch.int32, dev)
    else:
        grid, first = tuple(grid), tuple(first)
        if len(grid) != n or len(first) < n:
            raise ValueError("grid and first must give every axis")
        g, f = grid + (1,) * (3 - n), first[:n] + (0,) * (3 - n)
    try:
        r = bsa_rope.from_buffer_copy(_ROPE.pack(_PAIRINGS[pairing], *pairs, *lens, *ptrs, *g, *f,
                                                 0 if pos is None else pos.data_ptr()))
    except struct.error as e:
        raise ValueError(f"grid and first must be whole numbers of 32 bits, got {grid} and {first}") from e
    r._device, r._pos = dev, pos
    r._tensors = (tuple(tables), pos)      # the struct holds raw pointers: keep the tensors alive with it
    return r


def rope_apply(x: torch.Tensor, rope: bsa_rope, inverse: bool = False, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """x [N, H, d] turned by its tokens' positions (``inverse``: turned back, which is
    also the gradient).  ``out`` may be x itself; x may be a strided slice."""
    hx = _heads("x", x)
    if _rope_for(rope, x) is None:
        raise ValueError("rope must come from rope_axes")
    dev = x.device
    guard = _enter(dev, stream)
    try:
        if out is None:
            out, ho = _fresh(x)
        else:
            ho = _heads("out", out, x)
        rc = _lib.rope_apply(hx, ho, _DTYPES[x.dtype], x.shape[0], x.shape[2], rope, bool(inverse),
                             _raw_stream(dev.index))
    finally:
        _leave(guard)
    _check("rope_apply", rc)
    return out


def qk_norm_rope_fwd(q: torch.Tensor, k: Optional[torch.Tensor], wq: Optional[torch.Tensor] = None,
                     wk: Optional[torch.Tensor] = None, rope: Optional[bsa_rope] = None, eps: float = 1e-6,
                     qo: Optional[torch.Tensor] = None, ko: Optional[torch.Tensor] = None, stream=None):
    """RMS norm of every head of q [N, Hq, d] and k [N, Hk, d] (weights wq, wk [d] or
    None), then the rotation (None: none), in one pass; returns (qo, ko).  k may be
    None (then ko is).  An output may be its own input."""
    hq = _heads("q", q)
    if k is None and (wk is not None or ko is not None):
        raise ValueError("wk and ko need k")
    hk = None if k is None else _heads("k", k, q, True)
    pq, pk = _weight("wq", wq, q), _weight("wk", wk, q)
    wtype = _weight_type(wq, wk, q)
    rope = _rope_for(rope, q)
    dev = q.device
    guard = _enter(dev, stream)
    try:
        if qo is None:
            qo, hqo = _fresh(q)
        else:
            hqo = _heads("qo", qo, q)
        hko = None
        if k is not None:
            if ko is None:
                ko, hko = _fresh(k)
            else:
                hko = _heads("ko", ko, k)
        rc = _lib.qk_norm_rope_fwd(hq, hk, hqo, hko, _DTYPES[q.dtype], q.shape[0], q.shape[2], pq, pk, wtype, eps,
                                   rope, _raw_stream(dev.index))
    finally:
        _leave(guard)
    _check("qk_norm_rope_fwd", rc)
    return qo, ko


def qk_norm_rope_bwd(gq: torch.Tensor, gk: Optional[torch.Tensor], q: torch.Tensor, k: Optional[torch.Tensor],
                     wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None,
                     rope: Optional[bsa_rope] = None, eps: float = 1e-6, dq: Optional[torch.Tensor] = None,
                     dk: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of qk_norm_rope_fwd: (dq, dk, dwq, dwk) for the output gradients gq, gk.
    dwq and dwk are float32 [d], None where the weight is None; dk is None where k is."""
    hq = _heads("q", q)
    hgq = _heads("gq", gq, q)
    if (gk is None) != (k is None) or (k is None and (wk is not None or dk is not None)):
        raise ValueError("gk, wk and dk need k, and k needs gk")
    hk = hgk = None
    if k is not None:
        hk, hgk = _heads("k", k, q, True), _heads("gk", gk, k)
    pq, pk = _weight("wq", wq, q), _weight("wk", wk, q)
    wtype = _weight_type(wq, wk, q)
    rope = _rope_for(rope, q)
    dev = q.device
    _check_workspace(workspace, dev)
    N, H, d = q.shape
    need = _lib.qk_norm_rope_bwd_workspace_bytes(N, H, 0 if k is None else k.shape[1], d)
    if need == ctypes.c_size_t(-1).value:
        raise BsaError("qk_norm_rope_bwd_workspace_bytes", BSA_ERR_UNSUPPORTED)
    guard = _enter(dev, stream)
    try:
        if dq is None:
            dq, hdq = _fresh(q)
        else:
            hdq = _heads("dq", dq, q)
        hdk = None
        if k is not None:
            if dk is None:
                dk, hdk = _fresh(k)
            else:
                hdk = _heads("dk", dk, k)
        if workspace is None:
            workspace = q.new_empty(need, dtype=torch.uint8)
        dwq = None if wq is None else torch.empty_like(wq, dtype=torch.float32)
        dwk = None if wk is None else torch.empty_like(wk, dtype=torch.float32)
        rc = _lib.qk_norm_rope_bwd(hgq, hgk, hq, hk, hdq, hdk, _DTYPES[q.dtype], N, d, pq, pk, wtype, eps, rope,
                                   None if dwq is None else dwq.data_ptr(), None if dwk is None else dwk.data_ptr(),
                                   workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                   _raw_stream(dev.index))
    finally:
        _leave(guard)
    _check("qk_norm_rope_bwd", rc)
    return dq, dk, dwq, dwk


# ------------------------------------------------ key blocks by block means ---
def blockmean_select(q: torch.Tensor, k: torch.Tensor, keep: int, local: int = 0, block: int = 128, idx=None, cnt=None,
                     workspace: Optional[torch.Tensor] = None, stream=None, return_over_budget: bool = False):
    """Per (head, query block) the ``keep`` key blocks of the largest mean score, the blocks
    within ``local`` of the own one always among them (-1: none forced); returns
    (idx [H,nB,nB] int32 ascending, -1 padded, cnt [H,nB] int32) for block_index.
    A neighbourhood of more than ``keep`` blocks is kept whole (cnt says so); with
    ``return_over_budget`` a third value tells whether there is one."""
    _check_qkv(q, k, k)
    if k.device != q.device:
        raise ValueError(f"k must be on {q.device}, got {k.device}")
    _check_workspace(workspace, q.device)
    N, H, d = q.shape
    nB = math.ceil(N / 128)
    _check_tensor("idx", idx, (H, nB, nB), torch.int32, q.device)
    _check_tensor("cnt", cnt, (H, nB), torch.int32, q.device)
    need = _lib.blockmean_select_workspace_bytes(N, H, d)
    if need == ctypes.c_size_t(-1).value:
        raise BsaError("blockmean_select", BSA_ERR_UNSUPPORTED)
    dev = q.device
    guard = _enter(dev, stream)
    try:
        if idx is None:
            idx = q.new_empty((H, nB, nB), dtype=torch.int32)
        if cnt is None:
            cnt = q.new_empty((H, nB), dtype=torch.int32)
        if workspace is None:
            workspace = q.new_empty(need, dtype=torch.uint8)
        rc = _lib.blockmean_select(q.data_ptr(), k.data_ptr(), N, H, d, int(block), int(keep), int(local),
                                   idx.data_ptr(), cnt.data_ptr(), workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), _raw_stream(dev.index))
    finally:
        _leave(guard)
    _check("blockmean_select", rc, (BSA_OK, BSA_WARN_OVER_BUDGET))
    return (idx, cnt, rc == BSA_WARN_OVER_BUDGET) if return_over_budget else (idx, cnt)


# ------------------------------------------------- gradient of the attention ---
def blocksparse_attn_bwd(go: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                         lse: torch.Tensor, index: bsa_index, scale: Optional[float] = None,
                         dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                         dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of blocksparse_attn_fwd: (dq, dk, dv), each bf16 [N,H,d], for the gradient go of o.
    o and lse are the forward call's results for the same q, k, v, index and scale (o may be
    a strided copy)."""
    _check_qkv(q, k, v)
    N, H, d = q.shape
    dev = q.device
    for name, t in (("k", k), ("v", v), ("go", go), ("dq", dq), ("dk", dk), ("dv", dv)):
        _check_tensor(name, t, q.shape, torch.bfloat16, dev)
    for name, t in (("go", go), ("o", o), ("lse", lse)):
        if t is None:
            raise ValueError(f"{name} must be given")
    ho = _heads("o", o, q)
    _check_tensor("lse", lse, (H, N), torch.float32, dev)
    _check_workspace(workspace, dev)
    for t in getattr(index, "_tensors", ()):
        if t.device != dev:
            raise ValueError(f"the index is on {t.device}, the tensors on {dev}")
    if scale is None:
        scale = d ** -0.5
    need = workspace_bytes(BSA_OP_BLOCKSPARSE_BWD, N, H, d, index)
    guard = _enter(dev, stream)
    try:
        if workspace is None:
            workspace = q.new_empty(need, dtype=torch.uint8)
        dq, dk, dv = (torch.empty_like(q) if t is None else t for t in (dq, dk, dv))
        rc = _lib.blocksparse_attn_bwd(go.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), ho, lse.data_ptr(),
                                       N, H, d, scale, index, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                       workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                       _raw_stream(dev.index))
    finally:
        _leave(guard)
    _check("blocksparse_attn_bwd", rc)
    return dq, dk, dv


def get_device_status(stream=None) -> int:
    """Synchronise the stream and return + clear the device status word."""
    return int(_lib.bsa_get_device_status(_stream(stream)))


def debug_expired_wait(limit_ns: int, form: int = 0, stream=None) -> int:
    """Enqueue the expired-wait diagnostic (form 0: one thread waits, 1: the whole warp)."""
    return int(_lib.bsa_debug_expired_wait(int(limit_ns), int(form), _stream(stream)))


def lvsa_workspace_views(workspace: torch.Tensor, N: int, T: int):
    """Views of the LVSA workspace written by blocksparse_attn_fwd (layout of bsa_lib.cu).

    Returns (fbits [T, TW] int32 bit rows, tile_cnt [nB], tile_idx [nB, nB], tile_flag [nB, nB] uint8);
    row qt of tile_idx/tile_flag is valid in its first tile_cnt[qt] entries.
    """
    def up(x, a=256):
        return (x + a - 1) // a * a
    nB = math.ceil(N / 128)
    TW = (T + 31) // 32
    o_cnt = up(T * TW * 4)
    o_idx = up(o_cnt + nB * 4)
    o_flag = up(o_idx + nB * nB * 4)
    ws = workspace.view(torch.uint8)
    fbits = ws[:T * TW * 4].view(torch.int32).view(T, TW)
    cnt = ws[o_cnt:o_cnt + nB * 4].view(torch.int32)
    idx = ws[o_idx:o_idx + nB * nB * 4].view(torch.int32).view(nB, nB)
    flag = ws[o_flag:o_flag + nB * nB].view(nB, nB)
    return fbits, cnt, idx, flag
