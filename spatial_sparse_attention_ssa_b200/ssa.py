"""ctypes binding of libssa.so (argument marshalling only).

Each call here converts torch tensors to device pointers, sizes and the
current CUDA stream, allocates the caller-owned outputs and workspace with
torch, and calls the C ABI of include/ssa.h.  Every step of the attention
runs in the library's CUDA kernels; there is no CPU path.  A missing or
unloadable library raises immediately.
"""
from __future__ import annotations

import ctypes
import dataclasses
import math
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libssa.so")

SSA_OK = 0
STATUS_NAMES = {0: "SSA_OK", 1: "SSA_ERR_INVALID_ARG", 2: "SSA_ERR_UNSUPPORTED", 3: "SSA_ERR_WORKSPACE",
                4: "SSA_ERR_COORD_RANGE", 5: "SSA_ERR_CUDA", 6: "SSA_ERR_TIMEOUT"}
DTYPE_BF16, DTYPE_F32 = 0, 1
GATE_WEIGHTS, GATE_LOGITS = 0, 1
OP_BIN, OP_FORWARD, OP_BACKWARD, OP_GEO_SELECT, OP_CROSS_FORWARD, OP_CROSS_BACKWARD = 0, 1, 2, 3, 4, 5
OP_SP_FORWARD, OP_SP_BACKWARD = 6, 7
OP_WINDOW_BACKWARD, OP_DIFF_BACKWARD, OP_WINDOW_BACKWARD_TENSORS, OP_DIFF_BACKWARD_TENSORS = 8, 9, 10, 11
WINDOW_MAX_EDGE, WINDOW_TILE = 16, 16
SEL_SCORES, SEL_GIVEN = 0, 1

EXPORTS = ("ssa_bin", "ssa_forward", "ssa_backward", "ssa_workspace_size", "ssa_error_string",
           "ssa_get_device_status", "ssa_version", "ssa_launch_count", "ssa_profile_enable",
           "ssa_profile_read", "ssa_geo_select", "ssa_cross_forward", "ssa_cross_backward", "ssa_pool",
           "ssa_diag_wait_timeout", "ssa_diag_ex2", "ssa_sp_forward", "ssa_sp_backward",
           "ssa_window_plan", "ssa_window_forward", "ssa_window_backward", "ssa_window_workspace_size",
           "ssa_diff_forward", "ssa_diff_backward", "ssa_act8_pack", "ssa_act8_unpack")


class SSAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (%s)" % (where, STATUS_NAMES.get(status, status),
                                                 _lib().ssa_error_string(status).decode()))


class Conv(ctypes.Structure):
    _fields_ = [("coords", ctypes.c_void_p), ("wk", ctypes.c_void_p), ("bk", ctypes.c_void_p),
                ("wv", ctypes.c_void_p), ("bv", ctypes.c_void_p), ("dwk", ctypes.c_void_p),
                ("dbk", ctypes.c_void_p), ("dwv", ctypes.c_void_p), ("dbv", ctypes.c_void_p)]


class Params(ctypes.Structure):
    _fields_ = [("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("m_cmp", ctypes.c_int32), ("m_win", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int32), ("gate_mode", ctypes.c_int32),
                ("selection", ctypes.c_int32), ("conv", ctypes.POINTER(Conv)), ("deterministic", ctypes.c_int32)]


class Partition(ctypes.Structure):
    _fields_ = [("id", ctypes.c_void_p), ("perm", ctypes.c_void_p), ("ptr", ctypes.c_void_p),
                ("cu", ctypes.c_void_p), ("key", ctypes.c_void_p), ("count", ctypes.c_int64)]


class SpLocalC(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("cu_seqlens", ctypes.c_void_p), ("tokens", ctypes.c_void_p),
                ("win", ctypes.POINTER(Partition)), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("ks", ctypes.c_void_p), ("vs", ctypes.c_void_p)]


class Saved(ctypes.Structure):
    _fields_ = [("kc", ctypes.c_void_p), ("vc", ctypes.c_void_p), ("ks", ctypes.c_void_p),
                ("vs", ctypes.c_void_p), ("o_branch", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("sel", ctypes.c_void_p)]


class WinPlanC(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("tiles", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("count", ctypes.c_int64), ("m", ctypes.c_int32)]


_TORCH_DTYPE = {DTYPE_BF16: torch.bfloat16, DTYPE_F32: torch.float32}


class WindowParams(ctypes.Structure):
    _fields_ = [("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]

    @property
    def _dtype(self) -> torch.dtype:
        """The type of the tensors, from the field that the library reads."""
        dt = _TORCH_DTYPE.get(self.dtype)
        if dt is None:
            raise ValueError("dtype must be DTYPE_BF16 or DTYPE_F32")
        return dt


class WindowBiasC(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("bucket", ctypes.c_void_p), ("nb", ctypes.c_int32)]


class Act8C(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libssa.so is not built (python -m spatial_sparse_attention_ssa_b200.build)")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        pp = ctypes.POINTER(Partition)
        lib.ssa_bin.argtypes = [vp, vp, i32, i64, i32, i32, i32, pp, pp, vp, sz, vp]
        lib.ssa_bin.restype = ctypes.c_int
        lib.ssa_forward.argtypes = [ctypes.POINTER(Params), vp, i32, i64, pp, pp, vp, vp, vp, vp, vp,
                                    ctypes.POINTER(Saved), vp, sz, vp]
        lib.ssa_forward.restype = ctypes.c_int
        lib.ssa_backward.argtypes = [ctypes.POINTER(Params), vp, i32, i64, pp, pp, vp, vp, vp, vp,
                                     ctypes.POINTER(Saved), vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ssa_backward.restype = ctypes.c_int
        lib.ssa_cross_forward.argtypes = [ctypes.POINTER(Params), vp, i32, i64, i64, pp, vp, vp, vp, vp, vp,
                                          ctypes.POINTER(Saved), vp, sz, vp]
        lib.ssa_cross_forward.restype = ctypes.c_int
        lib.ssa_cross_backward.argtypes = [ctypes.POINTER(Params), vp, i32, i64, i64, pp, vp, vp, vp, vp,
                                           ctypes.POINTER(Saved), vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ssa_cross_backward.restype = ctypes.c_int
        spp = ctypes.POINTER(SpLocalC)
        lib.ssa_sp_forward.argtypes = [ctypes.POINTER(Params), i32, i64, pp, spp, vp, vp, vp, vp, vp,
                                       ctypes.POINTER(Saved), vp, sz, vp]
        lib.ssa_sp_forward.restype = ctypes.c_int
        lib.ssa_sp_backward.argtypes = [ctypes.POINTER(Params), i32, i64, pp, spp, vp, vp, vp, vp,
                                        ctypes.POINTER(Saved), vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ssa_sp_backward.restype = ctypes.c_int
        lib.ssa_diag_wait_timeout.argtypes = [vp, vp]
        lib.ssa_diag_wait_timeout.restype = ctypes.c_int
        lib.ssa_diag_ex2.argtypes = [vp, vp, vp, i64, vp]
        lib.ssa_diag_ex2.restype = ctypes.c_int
        lib.ssa_pool.argtypes = [i32, i32, i32, i64, pp, vp, vp, vp, vp, vp, vp, vp]
        lib.ssa_pool.restype = ctypes.c_int
        lib.ssa_geo_select.argtypes = [vp, vp, i32, i64, i32, pp, i32, i32, i32, vp, vp, sz, vp]
        lib.ssa_geo_select.restype = ctypes.c_int
        wp, pl, wb, a8 = (ctypes.POINTER(x) for x in (WindowParams, WinPlanC, WindowBiasC, Act8C))
        lib.ssa_window_plan.argtypes = [vp, i64, i32, pp, pl, vp]
        lib.ssa_window_plan.restype = ctypes.c_int
        lib.ssa_window_workspace_size.argtypes = [i32, wp, pl]
        lib.ssa_window_workspace_size.restype = sz
        lib.ssa_window_forward.argtypes = [wp, pl, wb, vp, vp, vp, vp, vp, vp]
        lib.ssa_window_forward.restype = ctypes.c_int
        lib.ssa_window_backward.argtypes = [wp, pl, wb, vp, vp, vp, a8, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ssa_window_backward.restype = ctypes.c_int
        f32 = ctypes.c_float
        lib.ssa_diff_forward.argtypes = [wp, pl, vp, f32, vp, vp, vp, vp, vp]
        lib.ssa_diff_forward.restype = ctypes.c_int
        lib.ssa_diff_backward.argtypes = [wp, pl, vp, f32, vp, vp, vp, a8, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.ssa_diff_backward.restype = ctypes.c_int
        lib.ssa_act8_pack.argtypes = [i32, i64, i32, vp, vp, vp, vp]
        lib.ssa_act8_pack.restype = ctypes.c_int
        lib.ssa_act8_unpack.argtypes = [i32, i64, i32, vp, vp, vp, vp]
        lib.ssa_act8_unpack.restype = ctypes.c_int
        lib.ssa_workspace_size.argtypes = [i32, ctypes.POINTER(Params), i32, i64, i64, i64]
        lib.ssa_workspace_size.restype = sz
        lib.ssa_error_string.argtypes = [ctypes.c_int]
        lib.ssa_error_string.restype = ctypes.c_char_p
        lib.ssa_get_device_status.argtypes = [vp]
        lib.ssa_get_device_status.restype = ctypes.c_int
        lib.ssa_version.argtypes = []
        lib.ssa_version.restype = i32
        lib.ssa_launch_count.argtypes = []
        lib.ssa_launch_count.restype = ctypes.c_uint64
        lib.ssa_profile_enable.argtypes = [i32]
        lib.ssa_profile_enable.restype = None
        lib.ssa_profile_read.argtypes = [ctypes.c_char_p, i32, ctypes.POINTER(ctypes.c_float),
                                         ctypes.POINTER(ctypes.c_int32), i32]
        lib.ssa_profile_read.restype = i32
        _LIB = lib
    return _LIB


def lib():
    """The loaded ctypes library (raises if it is not built)."""
    return _lib()


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


# the current stream's handle without building a Stream object, where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device | None = None) -> int:
    if _raw_stream is not None and device is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _check(status: int, where: str) -> None:
    if status != SSA_OK:
        raise SSAError(status, where)


def _require_cuda(*ts: torch.Tensor) -> None:
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("SSA tensors must be contiguous CUDA tensors")


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# binning
# ---------------------------------------------------------------------------


@dataclass
class Bins:
    """One partition (blocks or windows): device int32 tensors + count."""
    id: torch.Tensor
    perm: torch.Tensor
    ptr: torch.Tensor
    cu: torch.Tensor
    key: torch.Tensor
    count: int

    @staticmethod
    def empty(n: int, s: int, device) -> "Bins":
        z = lambda *shape: torch.empty(*shape, dtype=torch.int32, device=device)  # noqa: E731
        return Bins(z(n), z(n), z(n + 1), z(s + 1), z(max(n, 1), 3), 0)

    def c(self) -> Partition:
        return Partition(_ptr(self.id), _ptr(self.perm), _ptr(self.ptr), _ptr(self.cu), _ptr(self.key),
                         self.count)


def ssa_bin(coords: torch.Tensor, cu_seqlens: torch.Tensor, R: int, m_cmp: int, m_win: int,
            out: tuple[Bins, Bins] | None = None, workspace: torch.Tensor | None = None):
    """Step 1: block and window partitions of the tokens.  Returns (blk, win)."""
    _require_cuda(coords, cu_seqlens)
    n = int(coords.shape[0])
    s = int(cu_seqlens.shape[0]) - 1
    dev = coords.device
    blk, win = out if out is not None else (Bins.empty(n, s, dev), Bins.empty(n, s, dev))
    L = _lib()
    need = L.ssa_workspace_size(OP_BIN, None, s, n, n, n)
    ws = workspace if workspace is not None and workspace.numel() >= need else _workspace(need, dev)
    pb, pw = blk.c(), win.c()
    st = L.ssa_bin(_ptr(coords), _ptr(cu_seqlens), s, n, int(R), int(m_cmp), int(m_win),
                   ctypes.byref(pb), ctypes.byref(pw), _ptr(ws), ws.numel(), _stream(dev))
    _check(st, "ssa_bin")
    blk.count = int(pb.count)
    win.count = int(pw.count)
    return blk, win


def ssa_pool(blk: "Bins", k: torch.Tensor, v: torch.Tensor, out=None):
    """Step 2 alone: (ks, vs, kc, vc) -- K and V gathered in block order, head-major
    [Hkv, N, d], and the block means [Hkv, B, d], in the dtype of k."""
    _require_cuda(k, v)
    n, hkv, d = (int(x) for x in k.shape)
    dt = DTYPE_BF16 if k.dtype == torch.bfloat16 else DTYPE_F32
    if out is None:
        e = lambda *shape: torch.empty(*shape, dtype=k.dtype, device=k.device)  # noqa: E731
        out = (e(hkv, n, d), e(hkv, n, d), e(hkv, max(blk.count, 1), d), e(hkv, max(blk.count, 1), d))
    ks, vs, kc, vc = out
    pb = blk.c()
    st = _lib().ssa_pool(dt, hkv, d, n, ctypes.byref(pb), _ptr(k), _ptr(v), _ptr(ks), _ptr(vs), _ptr(kc), _ptr(vc),
                         _stream(k.device))
    _check(st, "ssa_pool")
    return ks, vs, kc, vc


def ssa_geo_select(coords: torch.Tensor, cu_seqlens: torch.Tensor, R: int, blk: "Bins", m_cmp: int, topk: int,
                   hkv: int, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """3D-aware block routing: the topk blocks nearest to each token (shortest
    distance between voxel centres; ties to the lower id), int32 [N, hkv, topk]
    global block ids, ascending, padded with -1, the same for every KV group."""
    _require_cuda(coords, cu_seqlens)
    n = int(coords.shape[0])
    s = int(cu_seqlens.shape[0]) - 1
    dev = coords.device
    sel = out if out is not None else torch.empty((n, hkv, topk), dtype=torch.int32, device=dev)
    L = _lib()
    need = L.ssa_workspace_size(OP_GEO_SELECT, None, s, n, blk.count, 0)
    ws = workspace if workspace is not None and workspace.numel() >= need else _workspace(need, dev)
    pb = blk.c()
    st = L.ssa_geo_select(_ptr(coords), _ptr(cu_seqlens), s, n, int(R), ctypes.byref(pb), int(m_cmp), int(topk),
                          int(hkv), _ptr(sel), _ptr(ws), ws.numel(), _stream(dev))
    _check(st, "ssa_geo_select")
    return sel


def ssa_bin_noalloc(coords: torch.Tensor, cu_seqlens: torch.Tensor, R: int, m_cmp: int, m_win: int,
                    out: tuple[Bins, Bins] | None = None):
    """ssa_bin with the library's fixed internal scratch instead of a workspace,
    for callers that cannot allocate device memory at binning time (up to
    SSA_BIN_NOALLOC_MAX_TOKENS tokens; calls that overlap on the GPU race).
    `out` must be preallocated by such callers; without it this wrapper
    allocates the output tensors itself with torch."""
    _require_cuda(coords, cu_seqlens)
    n = int(coords.shape[0])
    s = int(cu_seqlens.shape[0]) - 1
    dev = coords.device
    blk, win = out if out is not None else (Bins.empty(n, s, dev), Bins.empty(n, s, dev))
    L = _lib()
    fn = L.ssa_bin_noalloc
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                   ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(Partition), ctypes.POINTER(Partition),
                   ctypes.c_void_p]
    fn.restype = ctypes.c_int
    pb, pw = blk.c(), win.c()
    st = fn(_ptr(coords), _ptr(cu_seqlens), s, n, int(R), int(m_cmp), int(m_win), ctypes.byref(pb),
            ctypes.byref(pw), _stream(dev))
    _check(st, "ssa_bin_noalloc")
    blk.count = int(pb.count)
    win.count = int(pw.count)
    return blk, win


# ---------------------------------------------------------------------------
# forward / backward
# ---------------------------------------------------------------------------


@dataclass
class ConvWeights:
    """Learned compression: a sparse 3x3x3 convolution of K and V before the block
    mean.  coords int32 [N, 3]; wk / wv fp32 [Hkv, 27, d, d] (offset, in, out); bk /
    bv fp32 [Hkv, d]; the gradients dwk, dbk, dwv, dbv (same shapes) are written by
    ssa_backward."""
    coords: torch.Tensor
    wk: torch.Tensor
    bk: torch.Tensor
    wv: torch.Tensor
    bv: torch.Tensor
    dwk: torch.Tensor | None = None
    dbk: torch.Tensor | None = None
    dwv: torch.Tensor | None = None
    dbv: torch.Tensor | None = None

    def __post_init__(self):
        for name in ("dwk", "dbk", "dwv", "dbv"):
            if getattr(self, name) is None:
                setattr(self, name, torch.zeros_like(getattr(self, name[1:])))
        self._c = Conv(*(_ptr(getattr(self, f)) for f, _ in Conv._fields_))


def make_params(hq, hkv, d, m_cmp, m_win, topk, dtype: torch.dtype, gate_mode: int,
                scale: float = 0.0, selection: int = SEL_SCORES, conv: ConvWeights | None = None,
                deterministic: bool = False) -> Params:
    dt = DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32 if dtype == torch.float32 else None
    if dt is None:
        raise ValueError("dtype must be torch.bfloat16 or torch.float32")
    prm = Params(hq, hkv, d, m_cmp, m_win, topk, scale, dt, gate_mode, selection,
                 ctypes.pointer(conv._c) if conv is not None else None, 1 if deterministic else 0)
    prm._conv = conv  # keeps the weights (and the struct the pointer refers to) alive
    return prm


@dataclass
class SavedTensors:
    kc: torch.Tensor
    vc: torch.Tensor
    ks: torch.Tensor
    vs: torch.Tensor
    o_branch: torch.Tensor
    lse: torch.Tensor
    sel: torch.Tensor

    @staticmethod
    def empty(p: Params, n: int, btot: int, dtype, device) -> "SavedTensors":
        return SavedTensors(
            torch.empty(p.hkv, max(btot, 1), p.d, dtype=dtype, device=device),
            torch.empty(p.hkv, max(btot, 1), p.d, dtype=dtype, device=device),
            torch.empty(p.hkv, n, p.d, dtype=dtype, device=device),
            torch.empty(p.hkv, n, p.d, dtype=dtype, device=device),
            torch.empty(3, n, p.hq, p.d, dtype=torch.float32, device=device),
            torch.empty(3, n, p.hq, dtype=torch.float32, device=device),
            torch.empty(n, p.hkv, p.topk, dtype=torch.int32, device=device))

    @staticmethod
    def empty_cross(p: Params, nq: int, nkv: int, btot: int, dtype, device) -> "SavedTensors":
        """Buffers of ssa_cross_forward: two branches, keys / values of the voxel tokens."""
        return SavedTensors(
            torch.empty(p.hkv, max(btot, 1), p.d, dtype=dtype, device=device),
            torch.empty(p.hkv, max(btot, 1), p.d, dtype=dtype, device=device),
            torch.empty(p.hkv, nkv, p.d, dtype=dtype, device=device),
            torch.empty(p.hkv, nkv, p.d, dtype=dtype, device=device),
            torch.empty(2, nq, p.hq, p.d, dtype=torch.float32, device=device),
            torch.empty(2, nq, p.hq, dtype=torch.float32, device=device),
            torch.empty(nq, p.hkv, p.topk, dtype=torch.int32, device=device))

    def c(self) -> Saved:
        return Saved(_ptr(self.kc), _ptr(self.vc), _ptr(self.ks), _ptr(self.vs), _ptr(self.o_branch),
                     _ptr(self.lse), _ptr(self.sel))


def workspace_size(op: int, p: Params, s: int, n: int, btot: int, wtot: int) -> int:
    return int(_lib().ssa_workspace_size(op, ctypes.byref(p), s, n, btot, wtot))


def ssa_forward(p: Params, cu_seqlens: torch.Tensor, blk: Bins, win: Bins, q: torch.Tensor,
                k: torch.Tensor, v: torch.Tensor, gates: torch.Tensor, out: torch.Tensor | None = None,
                saved: SavedTensors | None = None, workspace: torch.Tensor | None = None,
                sel: torch.Tensor | None = None):
    """Steps 2-6.  Returns (out [N, Hq, d], saved).  With p.selection == SEL_GIVEN,
    `sel` (int32 [N, Hkv, topk], e.g. from ssa_geo_select) becomes saved.sel and is
    read instead of the score top-k; entries outside the token's sequence are set
    to -1 on the device and reported by device_status()."""
    _require_cuda(cu_seqlens, q, k, v, gates)
    n = int(q.shape[0])
    s = int(cu_seqlens.shape[0]) - 1
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    if saved is None:
        saved = SavedTensors.empty(p, n, blk.count, q.dtype, dev)
    if p.selection == SEL_GIVEN:
        if sel is not None:
            if sel.dtype != torch.int32 or not sel.is_contiguous() or tuple(sel.shape) != (n, p.hkv, p.topk):
                raise ValueError("sel must be a contiguous int32 tensor [N, Hkv, topk]")
            saved = dataclasses.replace(saved, sel=sel)
    elif sel is not None:
        raise ValueError("sel is only read with selection=SEL_GIVEN")
    need = workspace_size(OP_FORWARD, p, s, n, blk.count, win.count)
    ws = workspace if workspace is not None and workspace.numel() >= need else _workspace(need, dev)
    pb, pw, sv = blk.c(), win.c(), saved.c()
    st = _lib().ssa_forward(ctypes.byref(p), _ptr(cu_seqlens), s, n, ctypes.byref(pb), ctypes.byref(pw),
                            _ptr(q), _ptr(k), _ptr(v), _ptr(gates), _ptr(out), ctypes.byref(sv), _ptr(ws),
                            ws.numel(), _stream(dev))
    _check(st, "ssa_forward")
    return out, saved


def ssa_backward(p: Params, cu_seqlens: torch.Tensor, blk: Bins, win: Bins, q, k, v, gates,
                 saved: SavedTensors, dout: torch.Tensor, grads=None, workspace: torch.Tensor | None = None):
    """Step 7.  Returns (dq, dk, dv, dgates), all fp32."""
    _require_cuda(cu_seqlens, q, k, v, gates, dout)
    n = int(q.shape[0])
    s = int(cu_seqlens.shape[0]) - 1
    dev = q.device
    if grads is None:
        f32 = dict(dtype=torch.float32, device=dev)
        grads = (torch.empty(q.shape, **f32), torch.empty(k.shape, **f32), torch.empty(v.shape, **f32),
                 torch.empty(gates.shape, **f32))
    dq, dk, dv, dg = grads
    need = workspace_size(OP_BACKWARD, p, s, n, blk.count, win.count)
    ws = workspace if workspace is not None and workspace.numel() >= need else _workspace(need, dev)
    pb, pw, sv = blk.c(), win.c(), saved.c()
    st = _lib().ssa_backward(ctypes.byref(p), _ptr(cu_seqlens), s, n, ctypes.byref(pb), ctypes.byref(pw),
                             _ptr(q), _ptr(k), _ptr(v), _ptr(gates), ctypes.byref(sv), _ptr(dout), _ptr(dq),
                             _ptr(dk), _ptr(dv), _ptr(dg), _ptr(ws), ws.numel(), _stream(dev))
    _check(st, "ssa_backward")
    return dq, dk, dv, dg


@dataclass
class SpLocal:
    """One rank's tokens of a batch split by whole blocks (see ssa_sp_forward in
    include/ssa.h): their per-sequence offsets, their rows among all tokens, their own
    window partition and K / V, and room for their window-ordered K / V copies."""
    cu_seqlens: torch.Tensor  # int32 [S+1]
    tokens: torch.Tensor      # int32 [Nr]
    win: Bins                 # ssa_bin of the rank's coordinates (edge m_win)
    k: torch.Tensor           # [Nr, Hkv, d]
    v: torch.Tensor
    ks: torch.Tensor          # [Hkv, Nr, d]
    vs: torch.Tensor

    @staticmethod
    def make(cu_seqlens, tokens, win: Bins, k, v) -> "SpLocal":
        n, hkv, d = (int(x) for x in k.shape)
        e = lambda: torch.empty(hkv, n, d, dtype=k.dtype, device=k.device)  # noqa: E731
        return SpLocal(cu_seqlens, tokens, win, k, v, e(), e())

    def c(self):
        pw = self.win.c()
        return SpLocalC(int(self.k.shape[0]), _ptr(self.cu_seqlens), _ptr(self.tokens), ctypes.pointer(pw),
                        _ptr(self.k), _ptr(self.v), _ptr(self.ks), _ptr(self.vs)), pw


def ssa_sp_forward(p: Params, blk: Bins, n_all: int, loc: SpLocal, q: torch.Tensor, k: torch.Tensor,
                   v: torch.Tensor, gates: torch.Tensor, out: torch.Tensor | None = None,
                   saved: SavedTensors | None = None, workspace: torch.Tensor | None = None):
    """One rank's forward (sequences split by whole blocks): its query rows q / gates
    [Nr, Hq, *] against all N tokens' k / v binned into `blk`; returns (out, saved)."""
    _require_cuda(q, k, v, gates, loc.cu_seqlens, loc.tokens, loc.k, loc.v)
    nr, s = int(q.shape[0]), int(loc.cu_seqlens.shape[0]) - 1
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    if saved is None:  # the cross-attention buffers, with room for the third (window) branch
        saved = dataclasses.replace(SavedTensors.empty_cross(p, nr, n_all, blk.count, q.dtype, dev),
                                    o_branch=torch.empty(3, nr, p.hq, p.d, dtype=torch.float32, device=dev),
                                    lse=torch.empty(3, nr, p.hq, dtype=torch.float32, device=dev))
    need = workspace_size(OP_SP_FORWARD, p, s, nr, blk.count, loc.win.count)
    ws = workspace if workspace is not None and workspace.numel() >= need else _workspace(need, dev)
    pb, sv = blk.c(), saved.c()
    lc, _keep = loc.c()
    st = _lib().ssa_sp_forward(ctypes.byref(p), s, int(n_all), ctypes.byref(pb), ctypes.byref(lc), _ptr(q), _ptr(k),
                               _ptr(v), _ptr(gates), _ptr(out), ctypes.byref(sv), _ptr(ws), ws.numel(),
                               _stream(dev))
    _check(st, "ssa_sp_forward")
    return out, saved


def ssa_sp_backward(p: Params, blk: Bins, n_all: int, loc: SpLocal, q, k, v, gates, saved: SavedTensors,
                    dout, grads=None, workspace: torch.Tensor | None = None):
    """One rank's backward: (dq [Nr, Hq, d], dk, dv [N, Hkv, d] = its rows' contributions to every
    token's key gradients, dgates [Nr, Hq, 3])."""
    _require_cuda(q, k, v, gates, dout)
    nr, s = int(q.shape[0]), int(loc.cu_seqlens.shape[0]) - 1
    dev = q.device
    if grads is None:
        grads = (torch.empty(q.shape, dtype=torch.float32, device=dev),
                 torch.empty(k.shape, dtype=torch.float32, device=dev),
                 torch.empty(v.shape, dtype=torch.float32, device=dev),
                 torch.empty(gates.shape, dtype=torch.float32, device=dev))
    dq, dk, dv, dg = grads
    need = workspace_size(OP_SP_BACKWARD, p, s, nr, blk.count, loc.win.count)
    ws = workspace if workspace is not None and workspace.numel() >= need else _workspace(need, dev)
    pb, sv = blk.c(), saved.c()
    lc, _keep = loc.c()
    st = _lib().ssa_sp_backward(ctypes.byref(p), s, int(n_all), ctypes.byref(pb), ctypes.byref(lc), _ptr(q), _ptr(k),
                                _ptr(v), _ptr(gates), ctypes.byref(sv), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                                _ptr(dg), _ptr(ws), ws.numel(), _stream(dev))
    _check(st, "ssa_sp_backward")
    return dq, dk, dv, dg


def ssa_cross_forward(p: Params, q_cu: torch.Tensor, blk: Bins, q: torch.Tensor, k: torch.Tensor,
                      v: torch.Tensor, gates: torch.Tensor, out: torch.Tensor | None = None,
                      saved: SavedTensors | None = None, workspace: torch.Tensor | None = None,
                      sel: torch.Tensor | None = None):
    """Cross-attention SSA: queries q [Nq, Hq, d] (sequence s = rows q_cu[s] ..
    q_cu[s+1]-1) attend the voxel tokens k / v [Nkv, Hkv, d] binned into `blk`
    through the compressed and selected branches; gates [Nq, Hq, 2].
    Returns (out [Nq, Hq, d], saved)."""
    _require_cuda(q_cu, q, k, v, gates)
    nq, nkv = int(q.shape[0]), int(k.shape[0])
    s = int(q_cu.shape[0]) - 1
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    if saved is None:
        saved = SavedTensors.empty_cross(p, nq, nkv, blk.count, q.dtype, dev)
    if p.selection == SEL_GIVEN:
        if sel is not None:
            if sel.dtype != torch.int32 or not sel.is_contiguous() or tuple(sel.shape) != (nq, p.hkv, p.topk):
                raise ValueError("sel must be a contiguous int32 tensor [Nq, Hkv, topk]")
            saved = dataclasses.replace(saved, sel=sel)
    elif sel is not None:
        raise ValueError("sel is only read with selection=SEL_GIVEN")
    need = workspace_size(OP_CROSS_FORWARD, p, s, nq, blk.count, 0)
    ws = workspace if workspace is not None and workspace.numel() >= need else _workspace(need, dev)
    pb, sv = blk.c(), saved.c()
    st = _lib().ssa_cross_forward(ctypes.byref(p), _ptr(q_cu), s, nq, nkv, ctypes.byref(pb), _ptr(q), _ptr(k),
                                  _ptr(v), _ptr(gates), _ptr(out), ctypes.byref(sv), _ptr(ws), ws.numel(),
                                  _stream(dev))
    _check(st, "ssa_cross_forward")
    return out, saved


def ssa_cross_backward(p: Params, q_cu: torch.Tensor, blk: Bins, q, k, v, gates, saved: SavedTensors,
                       dout: torch.Tensor, grads=None, workspace: torch.Tensor | None = None):
    """Gradients of ssa_cross_forward: (dq, dk, dv, dgates), all fp32."""
    _require_cuda(q_cu, q, k, v, gates, dout)
    nq, nkv = int(q.shape[0]), int(k.shape[0])
    s = int(q_cu.shape[0]) - 1
    dev = q.device
    if grads is None:
        f32 = dict(dtype=torch.float32, device=dev)
        grads = (torch.empty(q.shape, **f32), torch.empty(k.shape, **f32), torch.empty(v.shape, **f32),
                 torch.empty(gates.shape, **f32))
    dq, dk, dv, dg = grads
    need = workspace_size(OP_CROSS_BACKWARD, p, s, nq, blk.count, 0)
    ws = workspace if workspace is not None and workspace.numel() >= need else _workspace(need, dev)
    pb, sv = blk.c(), saved.c()
    st = _lib().ssa_cross_backward(ctypes.byref(p), _ptr(q_cu), s, nq, nkv, ctypes.byref(pb), _ptr(q), _ptr(k),
                                   _ptr(v), _ptr(gates), ctypes.byref(sv), _ptr(dout), _ptr(dq), _ptr(dk),
                                   _ptr(dv), _ptr(dg), _ptr(ws), ws.numel(), _stream(dev))
    _check(st, "ssa_cross_backward")
    return dq, dk, dv, dg


# ---------------------------------------------------------------------------
# attention inside the cells of a partition
# ---------------------------------------------------------------------------


def _on_one_device(*ts: torch.Tensor | None) -> torch.device:
    """The device that all tensors share (contiguous CUDA tensors, as every call wants)."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("SSA tensors must be contiguous CUDA tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("SSA tensors must be on one device")
    return dev


def _call(device: torch.device, name: str, *args) -> None:
    """One library call on the device's current stream, with that device current."""
    fn = getattr(_lib(), name)
    if torch.cuda.current_device() == device.index:
        st = fn(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _stream(device))
    if st != SSA_OK:
        raise SSAError(st, name)


def _want(t: torch.Tensor, shape: tuple, dtype: torch.dtype, name: str) -> None:
    if t.dtype != dtype or t.shape != shape:
        raise ValueError("%s must be %s %s, got %s %s" % (name, dtype, tuple(shape), t.dtype, tuple(t.shape)))


@dataclass(frozen=True)
class WindowPlan:
    """Work plan of one partition (see ssa_win_plan in include/ssa.h): made once per voxel
    set, read by every layer and both passes of the window and differential calls."""
    rows: torch.Tensor   # int32 [n, 2]
    tiles: torch.Tensor  # int32 [n // 16 + count + 1, 4]
    n: int
    count: int
    m: int

    def __post_init__(self):
        put = lambda name, x: object.__setattr__(self, name, x)  # noqa: E731
        put("_c", WinPlanC(_ptr(self.rows), _ptr(self.tiles), self.n, self.count, self.m))
        put("_ref", ctypes.byref(self._c))
        put("_ws", {})  # workspace bytes by call and heads
        put("_sizes", (tuple(self.rows.shape), self.rows.dtype, tuple(self.tiles.shape), self.tiles.dtype) == (
            (self.n, 2), torch.int32, (self.n // WINDOW_TILE + self.count + 1, 4), torch.int32))
        put("_dev", self.rows.device if all(x.is_cuda and x.is_contiguous() and x.device == self.rows.device
                                            for x in (self.rows, self.tiles)) else None)

    def device(self, *ts: torch.Tensor | None) -> torch.device:
        """The device of the plan and of `ts`."""
        dev = _on_one_device(*ts)
        if dev != self._dev:
            raise ValueError("the plan's arrays must be contiguous CUDA tensors on the device of the others")
        if not self._sizes:
            raise ValueError("the plan's rows must be int32 [n, 2], its tiles int32 [n // 16 + count + 1, 4]")
        return dev

    def workspace_size(self, op: int, p: "WindowParams") -> int:
        """Bytes that OP_WINDOW_BACKWARD or OP_DIFF_BACKWARD needs for these heads, or their
        _TENSORS forms for calls whose q, k, v are not Act8."""
        key = (op, p.hq, p.hkv, p.d, p.dtype)
        if key not in self._ws:
            self._ws[key] = int(_lib().ssa_window_workspace_size(op, p, self._ref))
        return self._ws[key]


def ssa_window_plan(coords: torch.Tensor | None, win: Bins, m: int = 0) -> WindowPlan:
    """Plan of the partition `win` (from ssa_bin; `blk` serves as well).  With the binned
    coordinates and the window edge m (at most WINDOW_MAX_EDGE) it carries the offset codes
    that a bias reads; coords = None makes a plan without them, for any partition."""
    n = int(win.perm.shape[0])
    for name, x in (("win.perm", win.perm), ("win.id", win.id)):
        _want(x, (n,), torch.int32, name)
    if win.ptr.dtype != torch.int32 or win.ptr.dim() != 1 or win.ptr.shape[0] < win.count + 1:
        raise ValueError("win.ptr must be int32 of win.count + 1 entries at least")
    if coords is not None:
        _want(coords, (n, 3), torch.int32, "coords")
    dev = _on_one_device(win.perm, win.id, win.ptr, coords)
    e = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)  # noqa: E731
    plan = WindowPlan(e(n, 2), e(n // WINDOW_TILE + win.count + 1, 4), n, int(win.count), int(m) if coords is not None else 0)
    pb = win.c()
    _call(dev, "ssa_window_plan", _ptr(coords), n, int(m), ctypes.byref(pb), plan._ref)
    return plan


def make_window_params(hq: int, hkv: int, d: int, dtype: torch.dtype, scale: float = 0.0) -> WindowParams:
    """Heads and type of the window and differential calls (scale 0: 1/sqrt(d))."""
    dt = DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32 if dtype == torch.float32 else None
    if dt is None:
        raise ValueError("dtype must be torch.bfloat16 or torch.float32")
    return WindowParams(hq, hkv, d, dt, scale)


@dataclass
class WindowBias:
    """Learned relative position bias: table fp32 [hq, nb]; bucket int32 [(2m-1)^3] maps an
    offset to its bucket (None: every offset its own, nb = (2m-1)^3)."""
    table: torch.Tensor
    bucket: torch.Tensor | None = None


def window_log_buckets(m: int, device="cuda") -> tuple[torch.Tensor, int]:
    """(bucket, nb) of logarithmic buckets: per axis the sign of the offset and the power of
    two that holds its magnitude (0, 1, 2-3, 4-7, 8-15)."""
    a = torch.arange(-(m - 1), m, device=device)
    axis = torch.floor(torch.log2(a.abs().clamp_min(1).double())).long().add(1).mul(a.sign())
    top = int(axis.max())
    k = 2 * top + 1
    x = axis + top
    return ((x[:, None, None] * k + x[None, :, None]) * k + x[None, None, :]).reshape(-1).to(torch.int32), k ** 3


@dataclass
class Act8:
    """Rows in 8 bits: codes int8 [..., d], scale fp32 [...] (a power of two per row)."""
    codes: torch.Tensor
    scale: torch.Tensor


def _bias_c(bias: WindowBias | None, p: WindowParams, plan: WindowPlan):
    if bias is None:
        return None, 0
    if bias.table.dim() != 2:
        raise ValueError("bias.table must be [hq, nb]")
    nb = int(bias.table.shape[1])
    _want(bias.table, (p.hq, nb), torch.float32, "bias.table")
    if bias.bucket is not None:
        _want(bias.bucket, ((2 * plan.m - 1) ** 3,), torch.int32, "bias.bucket")
    return WindowBiasC(_ptr(bias.table), _ptr(bias.bucket), nb), nb


def _qkv(p: WindowParams, plan: WindowPlan, q, k, v):
    """(pointers of q, k, v, the Act8C array or None, their tensors)."""
    n = plan.n
    names = (("q", q, p.hq), ("k", k, p.hkv), ("v", v, p.hkv))
    if all(isinstance(x, Act8) for x in (q, k, v)):
        for name, x, h in names:
            _want(x.codes, (n, h, p.d), torch.int8, name + ".codes")
            _want(x.scale, (n, h), torch.float32, name + ".scale")
        arr = (Act8C * 3)(*((_ptr(x.codes), _ptr(x.scale)) for x in (q, k, v)))
        return (None, None, None), arr, [t for x in (q, k, v) for t in (x.codes, x.scale)]
    if any(isinstance(x, Act8) for x in (q, k, v)):
        raise ValueError("q, k, v must be three tensors or three Act8")
    dt = p._dtype
    for name, x, h in names:
        _want(x, (n, h, p.d), dt, name)
    return (_ptr(q), _ptr(k), _ptr(v)), None, [q, k, v]


def ssa_window_forward(p: WindowParams, plan: WindowPlan, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       bias: WindowBias | None = None, out: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of every token over the tokens of its cell, with an optional learned relative
    position bias: out [N, hq, d].  `lse` (fp32 [N, hq]) receives the softmax normalisers."""
    ptrs, a8, ts = _qkv(p, plan, q, k, v)
    if a8 is not None:
        raise ValueError("the forward reads tensors, not Act8")
    bc, _ = _bias_c(bias, p, plan)
    dev = plan.device(*ts, out, lse, *((bias.table, bias.bucket) if bias else ()))
    if out is None:
        out = torch.empty_like(q)
    else:
        _want(out, q.shape, q.dtype, "out")
    if lse is not None:
        _want(lse, (plan.n, p.hq), torch.float32, "lse")
    _call(dev, "ssa_window_forward", p, plan._ref, bc, *ptrs, _ptr(out), _ptr(lse))
    return out


# the backward calls whose q, k, v are tensors
_TENSORS_OP = {OP_WINDOW_BACKWARD: OP_WINDOW_BACKWARD_TENSORS, OP_DIFF_BACKWARD: OP_DIFF_BACKWARD_TENSORS}


def _window_backward(op: int, name: str, p: WindowParams, plan: WindowPlan, extra, extra_tensors, q, k, v, dout,
                     last: torch.Tensor | None, grads, workspace):
    ptrs, a8, ts = _qkv(p, plan, q, k, v)
    _want(dout, (plan.n, p.hq, p.d), p._dtype, "dout")
    dev = plan.device(*ts, dout, last, workspace, *extra_tensors, *(grads or ()))
    if workspace is not None and workspace.dtype != torch.uint8:
        raise ValueError("workspace must be uint8")
    shapes = ((plan.n, p.hq, p.d), (plan.n, p.hkv, p.d), (plan.n, p.hkv, p.d))
    if grads is None:
        grads = tuple(torch.empty(s, dtype=p._dtype, device=dev) for s in shapes)
    else:
        for g, s in zip(grads, shapes):
            _want(g, s, p._dtype, "grads")
    need = plan.workspace_size(op if a8 is not None else _TENSORS_OP[op], p)
    ws = workspace if workspace is not None and workspace.numel() >= need else _workspace(need, dev)
    _call(dev, name, p, plan._ref, *extra, *ptrs, a8, _ptr(dout), *(_ptr(g) for g in grads), _ptr(last), _ptr(ws),
          ws.numel())
    return (*grads, last)


def ssa_window_backward(p: WindowParams, plan: WindowPlan, q, k, v, dout: torch.Tensor,
                        bias: WindowBias | None = None, grads=None, dbias: torch.Tensor | bool | None = None,
                        workspace: torch.Tensor | None = None):
    """Gradients of ssa_window_forward: (dq, dk, dv, dbias), dq, dk, dv in the dtype of the
    inputs, dbias fp32 [hq, nb] (None without a bias, or with dbias = False: a bias that is not
    trained, whose gradient is not computed).  q, k, v are the forward's, or three Act8 of
    them."""
    bc, nb = _bias_c(bias, p, plan)
    if dbias is False:
        dbias, wanted = None, False
    else:
        wanted = bias is not None
    if bias is None and dbias is not None:
        raise ValueError("dbias without a bias")
    if wanted and dbias is None:
        dbias = torch.empty(p.hq, nb, dtype=torch.float32, device=dout.device)
    elif dbias is not None:
        _want(dbias, (p.hq, nb), torch.float32, "dbias")
    return _window_backward(OP_WINDOW_BACKWARD, "ssa_window_backward", p, plan, (bc,),
                            (bias.table, bias.bucket) if bias else (), q, k, v, dout, dbias, grads, workspace)


def ssa_diff_forward(p: WindowParams, plan: WindowPlan, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     lam: torch.Tensor, lam_init: float, out: torch.Tensor | None = None) -> torch.Tensor:
    """Differential attention inside the cells: the difference of the softmax maps of heads
    2h and 2h+1 over the value heads 2h, 2h+1 side by side; lam fp32 [4, hq/2, d] holds the
    weights' vectors (see ssa_diff_forward in include/ssa.h).  Returns out [N, hq, d]."""
    ptrs, a8, ts = _qkv(p, plan, q, k, v)
    if a8 is not None:
        raise ValueError("the forward reads tensors, not Act8")
    _want(lam, (4, p.hq // 2, p.d), torch.float32, "lam")
    dev = plan.device(*ts, lam, out)
    if out is None:
        out = torch.empty_like(q)
    else:
        _want(out, q.shape, q.dtype, "out")
    _call(dev, "ssa_diff_forward", p, plan._ref, _ptr(lam), float(lam_init), *ptrs, _ptr(out))
    return out


def ssa_diff_backward(p: WindowParams, plan: WindowPlan, q, k, v, lam: torch.Tensor, lam_init: float,
                      dout: torch.Tensor, grads=None, dlam: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None):
    """Gradients of ssa_diff_forward: (dq, dk, dv, dlam), dlam fp32 [4, hq/2, d].  q, k, v are
    the forward's, or three Act8 of them."""
    _want(lam, (4, p.hq // 2, p.d), torch.float32, "lam")
    if dlam is None:
        dlam = torch.empty_like(lam)
    else:
        _want(dlam, lam.shape, torch.float32, "dlam")
    return _window_backward(OP_DIFF_BACKWARD, "ssa_diff_backward", p, plan, (_ptr(lam), float(lam_init)), (lam,), q, k, v,
                            dout, dlam, grads, workspace)


def ssa_act8_pack(x: torch.Tensor, out: Act8 | None = None) -> Act8:
    """Rows x [..., d] (bf16 or fp32, d 32, 64 or 128) in 8 bits with a power-of-two scale each."""
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("x must be bfloat16 or float32")
    if out is None:
        dev = _on_one_device(x)
        out = Act8(torch.empty(x.shape, dtype=torch.int8, device=dev),
                   torch.empty(x.shape[:-1], dtype=torch.float32, device=dev))
    else:
        _want(out.codes, x.shape, torch.int8, "codes")
        _want(out.scale, x.shape[:-1], torch.float32, "scale")
        dev = _on_one_device(x, out.codes, out.scale)
    _call(dev, "ssa_act8_pack", DTYPE_BF16 if x.dtype == torch.bfloat16 else DTYPE_F32, out.scale.numel(),
          x.shape[-1], _ptr(x), _ptr(out.codes), _ptr(out.scale))
    return out


def ssa_act8_unpack(held: Act8, dtype: torch.dtype, out: torch.Tensor | None = None) -> torch.Tensor:
    """The values that `held` stands for, in bf16 (exact) or fp32."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("dtype must be torch.bfloat16 or torch.float32")
    shape = held.codes.shape
    _want(held.codes, shape, torch.int8, "codes")
    _want(held.scale, shape[:-1], torch.float32, "scale")
    if out is not None:
        _want(out, shape, dtype, "out")
    dev = _on_one_device(held.codes, held.scale, out)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    _call(dev, "ssa_act8_unpack", DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32, held.scale.numel(),
          shape[-1], _ptr(held.codes), _ptr(held.scale), _ptr(out))
    return out


def device_status(stream: int | None = None) -> int:
    return int(_lib().ssa_get_device_status(stream if stream is not None else _stream()))


def launch_count() -> int:
    """Kernels this library has launched in this process."""
    return int(_lib().ssa_launch_count())


def profile_enable(on: bool) -> None:
    _lib().ssa_profile_enable(1 if on else 0)


def profile_read(max_entries: int = 128) -> dict:
    """{kernel name: (total ms, launches)} recorded since the last read."""
    L = _lib()
    name_len = 64
    names = ctypes.create_string_buffer(name_len * max_entries)
    ms = (ctypes.c_float * max_entries)()
    cnt = (ctypes.c_int32 * max_entries)()
    n = min(L.ssa_profile_read(names, name_len, ms, cnt, max_entries), max_entries)
    out = {}
    for i in range(n):
        nm = names.raw[i * name_len:(i + 1) * name_len].split(b"\0", 1)[0].decode()
        out[nm] = (float(ms[i]), int(cnt[i]))
    return out


def diag_wait_timeout(device=None) -> tuple[int, int]:
    """Runs the bounded-wait diagnostic; returns (lane wait gave up, warp wait gave up)."""
    out = torch.zeros(2, dtype=torch.int32, device=device or "cuda")
    _check(_lib().ssa_diag_wait_timeout(_ptr(out), _stream(out.device)), "ssa_diag_wait_timeout")
    o = out.cpu().tolist()
    return int(o[0]), int(o[1])


def diag_ex2(x: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(2^x on the FMA pipe as the kernels evaluate it, 2^x from ex2.approx) for fp32 x."""
    _require_cuda(x)
    yp, ym = torch.empty_like(x), torch.empty_like(x)
    _check(_lib().ssa_diag_ex2(_ptr(x), _ptr(yp), _ptr(ym), x.numel(), _stream(x.device)), "ssa_diag_ex2")
    return yp, ym


def default_scale(d: int) -> float:
    return 1.0 / math.sqrt(d)
