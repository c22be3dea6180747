"""ctypes binding of libmoeq (include/moeq.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. PyTorch supplies device memory (outputs, workspaces) and the current
stream. There is no CPU fallback: if the library is not built, or no CUDA
device is present, every call raises.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from dataclasses import dataclass

import torch

from .synth import QWeightT

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libmoeq.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_MISALIGNED",
                3: "MOE_ERR_UNSUPPORTED", 4: "MOE_ERR_WORKSPACE", 5: "MOE_ERR_CUDA",
                6: "MOE_ERR_DEVICE"}
W_INT4 = 1
W_MXFP4 = 2
FMT = {"int4": W_INT4, "mxfp4": W_MXFP4}
EPI_NONE, EPI_SWIGLU, EPI_SWIGLU_BWD = 0, 1, 2
DEVERR_NONE, DEVERR_WAIT_TIMEOUT, DEVERR_BAD_OFFSETS = 0, 1, 2

EXPORTED = ("moe_route_permute", "moe_route_permute_noalloc", "moe_grouped_qgemm_fwd", "moe_grouped_qgemm_bwd_dx",
            "moe_unpermute_combine", "moe_get_device_error", "moe_status_string",
            "moe_abi_version", "moe_test_dequant", "moe_test_set_wait_budget",
            "moe_dequant_experts", "moe_ep_regroup", "moe_nvtx_enabled", "moe_route_scored",
            "moe_route_scored_bwd", "moe_combine_bwd", "moe_quantize_fp8_rows",
            "moe_dequantize_fp8_rows", "moe_grouped_fp8_gemm_fwd", "moe_grouped_fp8_gemm_bwd_dx")
SCORE = {"softmax": 1, "sigmoid": 2}
FP8_BLOCK128_F32, FP8_BLOCK32_E8M0 = 1, 2


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what} failed: {STATUS_NAMES.get(status, status)}")
        self.status = status


class QWeightC(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("fmt", ctypes.c_int32)]


class GroupsC(ctypes.Structure):
    _fields_ = [("expert_offsets", ctypes.c_void_p), ("active", ctypes.c_void_p),
                ("num_active", ctypes.c_void_p), ("chunk_offsets", ctypes.c_void_p),
                ("num_chunks", ctypes.c_void_p), ("E", ctypes.c_int32)]


class RouterC(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


class Fp8WeightC(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("E", ctypes.c_int32),
                ("N", ctypes.c_int32), ("K", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libmoeq.so is not built ({LIB_PATH}); run "
                           "`python -m quantized_rl_fine_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)
    L.moe_route_permute.argtypes = [vp, vp, i64, i32, i32, i64, i32, vp, vp, vp, vp, vp, vp, vp,
                                    vp, vp, vp, vp, sz, vp]
    L.moe_route_permute_noalloc.argtypes = [vp, vp, i64, i32, i32, i64, i32, vp, vp, vp, vp, vp,
                                            vp, vp, vp, vp, vp, vp]
    L.moe_grouped_qgemm_fwd.argtypes = [vp, vp, i64, ctypes.POINTER(QWeightC),
                                        ctypes.POINTER(GroupsC), vp, i32, vp, vp, vp, sz, vp]
    L.moe_grouped_qgemm_bwd_dx.argtypes = [vp, i64, ctypes.POINTER(QWeightC),
                                           ctypes.POINTER(GroupsC), i32, vp, vp, vp, vp, vp, vp,
                                           vp, sz, vp]
    L.moe_unpermute_combine.argtypes = [vp, vp, vp, i64, i32, i64, vp, i32, vp]
    L.moe_get_device_error.argtypes = [ctypes.POINTER(i32), vp]
    L.moe_status_string.argtypes = [i32]
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_abi_version.argtypes = []
    L.moe_test_dequant.argtypes = [vp, vp, i64, i32, i32, vp, vp]
    L.moe_test_set_wait_budget.argtypes = [i64]
    L.moe_dequant_experts.argtypes = [ctypes.POINTER(QWeightC), vp, i32, vp, vp]
    L.moe_ep_regroup.argtypes = [vp, i32, i32, i64, vp, vp, i64, i32, i32, vp, vp, vp, vp, vp, vp]
    rp, fp = ctypes.POINTER(RouterC), ctypes.POINTER(Fp8WeightC)
    gp = ctypes.POINTER(GroupsC)
    L.moe_route_scored.argtypes = [vp, vp, vp, i64, i32, i32, i64, rp, i32, vp, vp, vp, vp, vp, vp, vp,
                                   vp, vp, vp, vp, sz, vp]
    L.moe_route_scored_bwd.argtypes = [vp, vp, vp, vp, i64, i32, i32, rp, vp, vp]
    L.moe_combine_bwd.argtypes = [vp, vp, vp, vp, i64, i32, i64, vp, vp, vp]
    L.moe_quantize_fp8_rows.argtypes = [vp, i64, i64, vp, i32, vp, vp, vp]
    L.moe_dequantize_fp8_rows.argtypes = [vp, vp, i64, i64, i32, vp, vp]
    L.moe_grouped_fp8_gemm_fwd.argtypes = [vp, vp, i64, fp, gp, i32, vp, vp, vp, vp, vp]
    L.moe_grouped_fp8_gemm_bwd_dx.argtypes = [vp, vp, i64, fp, gp, i32, vp, vp, vp, vp, vp]
    for name in EXPORTED:
        if name not in ("moe_status_string",):
            getattr(L, name).restype = ctypes.c_int32
    _lib = L
    return L


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoeError(status, what)


def _p(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libmoeq takes CUDA tensors only")


def _workspace(nbytes: int, device):
    """(tensor or None, pointer or None, size argument) for a queried workspace size."""
    if int(nbytes) == 0:
        return None, None, None
    ws = torch.empty(int(nbytes), dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), ctypes.byref(ctypes.c_size_t(ws.numel()))


# --------------------------------------------------------------------------
# Routing
# --------------------------------------------------------------------------

@dataclass
class Routing:
    topk_idx: torch.Tensor        # [T, k] int32
    gates: torch.Tensor           # [T, k] fp32
    expert_offsets: torch.Tensor  # [E+1] int32
    active: torch.Tensor          # [E] int32
    num_active: torch.Tensor      # [1] int32
    chunk_offsets: torch.Tensor   # [E+1] int32
    num_chunks: torch.Tensor      # [1] int32
    perm_token: torch.Tensor      # [T*k] int32
    inv_perm: torch.Tensor        # [T*k] int32
    x_perm: torch.Tensor | None   # [T*k, d] bf16
    E: int
    k: int

    def groups(self) -> GroupsC:
        return GroupsC(_p(self.expert_offsets), _p(self.active), _p(self.num_active),
                       _p(self.chunk_offsets), _p(self.num_chunks), self.E)


def moe_route_permute(logits: torch.Tensor, x: torch.Tensor | None, k: int, chunk_size: int,
                      stream=None, out: Routing | None = None) -> Routing:
    _require_cuda(logits, x)
    T, E = logits.shape
    dev = logits.device
    if out is None:
        i32 = dict(dtype=torch.int32, device=dev)
        out = Routing(
            topk_idx=torch.empty((T, k), **i32), gates=torch.empty((T, k), dtype=torch.float32, device=dev),
            expert_offsets=torch.empty(E + 1, **i32), active=torch.empty(E, **i32),
            num_active=torch.empty(1, **i32), chunk_offsets=torch.empty(E + 1, **i32),
            num_chunks=torch.empty(1, **i32), perm_token=torch.empty(T * k, **i32),
            inv_perm=torch.empty(T * k, **i32),
            x_perm=None if x is None else torch.empty((T * k, x.shape[1]), dtype=torch.bfloat16, device=dev),
            E=E, k=k)
    L = lib()
    d = 0 if x is None else x.shape[1]
    wsb = ctypes.c_size_t(0)
    args = lambda ws, wsz: (_p(logits), _p(x), T, E, k, d, chunk_size, _p(out.topk_idx),
                            _p(out.gates), _p(out.expert_offsets), _p(out.active),
                            _p(out.num_active), _p(out.chunk_offsets), _p(out.num_chunks),
                            _p(out.perm_token), _p(out.inv_perm), _p(out.x_perm), ws, wsz,
                            _stream(stream))
    _check(L.moe_route_permute(*args(None, ctypes.byref(wsb))), "moe_route_permute (workspace query)")
    ws, wsp, wsz = _workspace(wsb.value, dev)
    _check(L.moe_route_permute(*args(wsp, wsz)), "moe_route_permute")
    return out


# --------------------------------------------------------------------------
# Grouped GEMMs
# --------------------------------------------------------------------------

def qweight_c(w: QWeightT) -> QWeightC:
    _require_cuda(w.packed, w.scales)
    return QWeightC(_p(w.packed), _p(w.scales), w.E, w.N, w.K, FMT[w.fmt])


def moe_grouped_qgemm_fwd(a: torch.Tensor, w: QWeightT, routing: Routing, epi: int = EPI_NONE,
                          adapter: torch.Tensor | None = None, save_gu: bool = False,
                          stream=None, out: torch.Tensor | None = None,
                          saved: torch.Tensor | None = None, a_rows: torch.Tensor | None = None):
    """Returns out [M, N] (none) or (out [M, N/2], saved [M, N] or None) (swiglu).
    With a_rows (int32 [M], e.g. routing.perm_token), row p of the input is a[a_rows[p]]."""
    _require_cuda(a, adapter, a_rows)
    M = a_rows.shape[0] if a_rows is not None else a.shape[0]
    F = w.N // 2 if epi == EPI_SWIGLU else w.N
    if out is None:
        out = torch.empty((M, F), dtype=torch.bfloat16, device=a.device)
    if save_gu and saved is None:
        saved = torch.empty((M, w.N), dtype=torch.bfloat16, device=a.device)
    qw, g = qweight_c(w), routing.groups()
    wsb = ctypes.c_size_t(0)
    L = lib()
    args = lambda ws, wsz: (_p(a), _p(a_rows), M, ctypes.byref(qw), ctypes.byref(g), _p(adapter),
                            epi, _p(out), _p(saved) if save_gu else None, ws, wsz, _stream(stream))
    _check(L.moe_grouped_qgemm_fwd(*args(None, ctypes.byref(wsb))),
           "moe_grouped_qgemm_fwd (workspace query)")
    ws, wsp, wsz = _workspace(wsb.value, a.device)
    _check(L.moe_grouped_qgemm_fwd(*args(wsp, wsz)), "moe_grouped_qgemm_fwd")
    if epi == EPI_SWIGLU:
        return out, (saved if save_gu else None)
    return out


def moe_grouped_qgemm_bwd_dx(dout: torch.Tensor, w: QWeightT, routing: Routing,
                             epi: int = EPI_NONE, saved_gu: torch.Tensor | None = None,
                             adapter: torch.Tensor | None = None, a: torch.Tensor | None = None,
                             stream=None, out: torch.Tensor | None = None,
                             a_rows: torch.Tensor | None = None):
    """Returns din ([M, K], or [M, 2K] for swiglu_bwd), plus d_adapter when an adapter is given.
    With a_rows, row p of the adapter's input a is a[a_rows[p]]."""
    _require_cuda(dout, saved_gu, adapter, a, a_rows)
    M = dout.shape[0]
    width = 2 * w.K if epi == EPI_SWIGLU_BWD else w.K
    if out is None:
        out = torch.empty((M, width), dtype=torch.bfloat16, device=dout.device)
    d_adapter = None
    if adapter is not None:
        d_adapter = torch.empty((w.E, w.K // 32, 32, 32), dtype=torch.float32, device=dout.device)
    qw, g = qweight_c(w), routing.groups()
    wsb = ctypes.c_size_t(0)
    L = lib()
    args = lambda ws, wsz: (_p(dout), M, ctypes.byref(qw), ctypes.byref(g), epi, _p(saved_gu),
                            _p(adapter), _p(a), _p(a_rows), _p(out), _p(d_adapter), ws, wsz,
                            _stream(stream))
    _check(L.moe_grouped_qgemm_bwd_dx(*args(None, ctypes.byref(wsb))),
           "moe_grouped_qgemm_bwd_dx (workspace query)")
    ws, wsp, wsz = _workspace(wsb.value, dout.device)
    _check(L.moe_grouped_qgemm_bwd_dx(*args(wsp, wsz)), "moe_grouped_qgemm_bwd_dx")
    return (out, d_adapter) if adapter is not None else out


def moe_unpermute_combine(rows: torch.Tensor, routing: Routing, gates: torch.Tensor | None,
                          T: int, mode: int = 0, stream=None, out: torch.Tensor | None = None):
    """mode 0: [T*k, D] -> [T, D] gate-weighted sum; mode 1: [T, D] -> [T*k, D] gate-scaled scatter."""
    _require_cuda(rows, gates)
    k = routing.k
    D = rows.shape[1]
    if out is None:
        shape = (T, D) if mode == 0 else (T * k, D)
        out = torch.empty(shape, dtype=torch.bfloat16, device=rows.device)
    _check(lib().moe_unpermute_combine(_p(rows), _p(routing.inv_perm), _p(gates), T, k, D,
                                       _p(out), mode, _stream(stream)), "moe_unpermute_combine")
    return out


def moe_get_device_error(stream=None) -> int:
    code = ctypes.c_int32(0)
    _check(lib().moe_get_device_error(ctypes.byref(code), _stream(stream)), "moe_get_device_error")
    return code.value


def moe_test_dequant(packed: torch.Tensor, scales: torch.Tensor, fmt: str, stream=None) -> torch.Tensor:
    """packed [R, K/2] uint8, scales [K/32, R] -> bf16 [R, K] with the GEMM's dequant functions."""
    _require_cuda(packed, scales)
    R, half = packed.shape
    out = torch.empty((R, 2 * half), dtype=torch.bfloat16, device=packed.device)
    _check(lib().moe_test_dequant(_p(packed), _p(scales), R, 2 * half, FMT[fmt], _p(out),
                                  _stream(stream)), "moe_test_dequant")
    return out


def moe_dequant_experts(w: QWeightT, experts: torch.Tensor, stream=None,
                        out: torch.Tensor | None = None) -> torch.Tensor:
    """Whole experts dequantized to BF16: out [count, N, K] = W[experts]."""
    _require_cuda(experts)
    count = int(experts.numel())
    if out is None:
        out = torch.empty((count, w.N, w.K), dtype=torch.bfloat16, device=experts.device)
    qw = qweight_c(w)
    _check(lib().moe_dequant_experts(ctypes.byref(qw), _p(experts), count, _p(out), _stream(stream)),
           "moe_dequant_experts")
    return out


def moe_ep_regroup(counts: torch.Tensor, rows: torch.Tensor, direction: int, chunk_size: int = 8,
                   stream=None, out: torch.Tensor | None = None):
    """Expert parallelism: received rows [R, D] reordered source-major -> local
    expert-major (direction 0, returns (rows, local Routing tables)) or back
    (direction 1, returns rows). counts: device int32 [W, E_loc]."""
    _require_cuda(counts, rows)
    W, E_loc = counts.shape
    R, D = rows.shape
    if out is None:
        out = torch.empty_like(rows)
    dev = rows.device
    i32 = dict(dtype=torch.int32, device=dev)
    if direction == 0:
        t = dict(expert_offsets=torch.empty(E_loc + 1, **i32), active=torch.empty(E_loc, **i32),
                 num_active=torch.empty(1, **i32), chunk_offsets=torch.empty(E_loc + 1, **i32),
                 num_chunks=torch.empty(1, **i32))
    else:
        t = dict(expert_offsets=None, active=None, num_active=None, chunk_offsets=None, num_chunks=None)
    _check(lib().moe_ep_regroup(_p(counts), W, E_loc, R, _p(rows), _p(out), D, direction, chunk_size,
                                _p(t["expert_offsets"]), _p(t["active"]), _p(t["num_active"]),
                                _p(t["chunk_offsets"]), _p(t["num_chunks"]), _stream(stream)),
           "moe_ep_regroup")
    if direction == 1:
        return out
    groups = Routing(topk_idx=None, gates=None, perm_token=None, inv_perm=None, x_perm=out,
                     E=E_loc, k=1, **t)
    return out, groups


# --------------------------------------------------------------------------
# Scored routing, router gradient, FP8 rows and FP8 expert products
#
# These calls check dtype, shape, layout (contiguous) and device of every
# tensor, run on the tensors' own device, and allocate their outputs and
# workspaces on the stream they launch on. For small batches the host is the
# bound (a launch takes 3 us of a call's 8 to 20), hence sizes passed to
# torch.empty one by one (a tuple costs 0.8 us) and few Python objects.
# --------------------------------------------------------------------------

def _need(t, name: str, dtype, shape, device=None):
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.shape == shape
            and t.is_contiguous() and (device is None or t.device == device)):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: libmoeq takes CUDA tensors only")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    raise ValueError(f"{name}: on {t.device}, expected {device}")


# The raw handle of a device's current stream; building a Stream object for it costs 4 us a call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _here(device) -> int:
    """The current stream of the tensors' device (which is the current one inside _on)."""
    return _raw_stream(device.index)


@contextlib.contextmanager
def _switch(device, stream):
    with torch.cuda.device(device):
        with torch.cuda.stream(stream):       # None: the device's current stream
            yield


_HERE = contextlib.nullcontext()


def _on(device, stream):
    """The tensors' device, and `stream` (if any) as its current stream."""
    if device.type != "cuda":
        raise ValueError("libmoeq takes CUDA tensors only")
    if stream is not None and stream.device != device:
        raise ValueError(f"stream: of {stream.device}, but the tensors are on {device}")
    if stream is None and device.index == torch.cuda.current_device():
        return _HERE
    return _switch(device, stream)


@dataclass(frozen=True)
class RouterSpec:
    """How moe_route_scored selects experts and forms gates (moe_router in moeq.h)."""
    score: str = "softmax"        # "softmax" (over all experts) or "sigmoid"
    groups: int = 1               # expert groups of E / groups consecutive experts
    topk_groups: int = 1          # groups a token may choose from
    group_top: int = 1            # a group's score: sum of its 1 or 2 largest keys
    renorm: bool = True           # gates divided by the sum of the selected scores
    scale: float = 1.0            # factor of every gate

    @functools.lru_cache(maxsize=256)
    def c(self) -> RouterC:
        if self.score not in SCORE:
            raise ValueError(f"score {self.score!r}: expected one of {sorted(SCORE)}")
        return RouterC(SCORE[self.score], self.groups, self.topk_groups, self.group_top,
                       1 if self.renorm else 0, self.scale)


@functools.lru_cache(maxsize=256)
def _scored_ws_bytes(T: int, E: int, k: int, router: RouterSpec, chunk_size: int) -> int:
    """Workspace of moe_route_scored (a function of the sizes alone)."""
    wsb = ctypes.c_size_t(0)
    _check(lib().moe_route_scored(None, None, None, T, E, k, 0, ctypes.byref(router.c()), chunk_size, None,
                                  None, None, None, None, None, None, None, None, None, None,
                                  ctypes.byref(wsb), None), "moe_route_scored (workspace query)")
    return wsb.value


@functools.lru_cache(maxsize=256)
def _routing_layout(T: int, E: int, k: int) -> tuple[list[int], list[int], list[int]]:
    """Split sizes of one 32-bit buffer into the gates and the eight tables (each starting on 16
    bytes) and the padding between them, which of the pieces are these nine, and their byte offsets."""
    sizes, pieces, at = [], [], []
    for n in (T * k, T * k, E + 1, E, 1, E + 1, 1, T * k, T * k):
        pieces.append(len(sizes))
        at.append(4 * sum(sizes))
        sizes.append(n)
        if n % 4:
            sizes.append(-n % 4)
    return sizes, pieces, at


def _split_routing(buf: torch.Tensor, x_perm: torch.Tensor | None, T: int, E: int, k: int) -> Routing:
    sizes, pieces, _ = _routing_layout(T, E, k)
    parts = buf.split_with_sizes(sizes)
    gates, idx, off, act, nact, chunk, nchunk, perm, inv = [parts[i] for i in pieces]
    return Routing(topk_idx=idx.view(T, k), gates=gates.view(torch.float32).view(T, k), expert_offsets=off,
                   active=act, num_active=nact, chunk_offsets=chunk, num_chunks=nchunk, perm_token=perm,
                   inv_perm=inv, x_perm=x_perm, E=E, k=k)


def _need_routing(r: Routing, T: int, E: int, k: int, d: int | None, dev):
    i32 = torch.int32
    for name, n in (("expert_offsets", E + 1), ("active", E), ("num_active", 1),
                    ("chunk_offsets", E + 1), ("num_chunks", 1), ("perm_token", T * k),
                    ("inv_perm", T * k)):
        _need(getattr(r, name), "out." + name, i32, (n,), dev)
    _need(r.topk_idx, "out.topk_idx", i32, (T, k), dev)
    _need(r.gates, "out.gates", torch.float32, (T, k), dev)
    if d is not None:
        _need(r.x_perm, "out.x_perm", torch.bfloat16, (T * k, d), dev)


def moe_route_scored(logits: torch.Tensor, x: torch.Tensor | None, k: int, chunk_size: int,
                     router: RouterSpec, bias: torch.Tensor | None = None, stream=None,
                     out: Routing | None = None) -> Routing:
    """moe_route_permute with softmax or sigmoid scores, a selection bias [E], expert groups and
    renormalised or plain gates."""
    if logits.dim() != 2:
        raise ValueError("logits: expected [T, E]")
    T, E = logits.shape
    dev = logits.device
    _need(logits, "logits", torch.float32, (T, E))
    if bias is not None:
        _need(bias, "bias", torch.float32, (E,), dev)
    d = None
    if x is not None:
        d = x.shape[-1]
        _need(x, "x", torch.bfloat16, (T, d), dev)
    with _on(dev, stream):
        need = _scored_ws_bytes(T, E, k, router, chunk_size)
        if out is None:
            sizes, _, at = _routing_layout(T, E, k)
            buf = torch.empty(sum(sizes), dtype=torch.int32, device=dev)
            base = buf.data_ptr()
            gates, idx, *tables = [base + o for o in at]
            x_perm = None if d is None else torch.empty(T * k, d, dtype=torch.bfloat16, device=dev)
        else:
            _need_routing(out, T, E, k, d, dev)
            gates, idx = _p(out.gates), _p(out.topk_idx)
            tables = [_p(t) for t in (out.expert_offsets, out.active, out.num_active, out.chunk_offsets,
                                      out.num_chunks, out.perm_token, out.inv_perm)]
            x_perm = out.x_perm
        ws, wsp, wsz = _workspace(need, dev)
        _check(lib().moe_route_scored(
            _p(logits), _p(bias), _p(x), T, E, k, d or 0, ctypes.byref(router.c()), chunk_size, idx, gates,
            *tables, None if d is None else _p(x_perm), wsp, wsz, _here(dev)), "moe_route_scored")
        # The tensors of the tables are made behind the launch (9 us of host work).
        return _split_routing(buf, x_perm, T, E, k) if out is None else out


def moe_route_scored_bwd(d_gates: torch.Tensor, logits: torch.Tensor, routing: Routing,
                         router: RouterSpec, stream=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """d_logits [T, E] from the gates' gradient [T, k] and the selection (and gates, if kept) in
    `routing`."""
    if logits.dim() != 2:
        raise ValueError("logits: expected [T, E]")
    T, E = logits.shape
    k, dev = routing.k, logits.device
    _need(logits, "logits", torch.float32, (T, E))
    _need(d_gates, "d_gates", torch.float32, (T, k), dev)
    _need(routing.topk_idx, "routing.topk_idx", torch.int32, (T, k), dev)
    if routing.gates is not None:
        _need(routing.gates, "routing.gates", torch.float32, (T, k), dev)
    rc = router.c()
    with _on(dev, stream):
        if out is None:
            out = torch.empty(T, E, dtype=torch.float32, device=dev)
        else:
            _need(out, "out", torch.float32, (T, E), dev)
        _check(lib().moe_route_scored_bwd(_p(d_gates), _p(routing.gates), _p(logits), _p(routing.topk_idx),
                                          T, E, k, ctypes.byref(rc), _p(out), _here(dev)), "moe_route_scored_bwd")
    return out


def moe_combine_bwd(dy: torch.Tensor, rows: torch.Tensor, routing: Routing, stream=None,
                    out: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Backward of the combine: (d_rows [T*k, D] = gate * dy per slot, d_gates [T, k] = dy . rows)."""
    if dy.dim() != 2:
        raise ValueError("dy: expected [T, D]")
    T, D = dy.shape
    k, dev = routing.k, dy.device
    _need(dy, "dy", torch.bfloat16, (T, D))
    _need(rows, "rows", torch.bfloat16, (T * k, D), dev)
    _need(routing.inv_perm, "routing.inv_perm", torch.int32, (T * k,), dev)
    if routing.gates is not None:
        _need(routing.gates, "routing.gates", torch.float32, (T, k), dev)
    with _on(dev, stream):
        if out is None:
            out = torch.empty(T * k, D, dtype=torch.bfloat16, device=dev)
        else:
            _need(out, "out", torch.bfloat16, (T * k, D), dev)
        d_gates = torch.empty(T, k, dtype=torch.float32, device=dev)
        _check(lib().moe_combine_bwd(_p(dy), _p(rows), _p(routing.inv_perm), _p(routing.gates), T, k, D,
                                     _p(out), _p(d_gates), _here(dev)), "moe_combine_bwd")
    return out, d_gates


@dataclass
class Fp8Rows:
    """e4m3 rows and their block scales: fp32 [ceil(K/128), M] (FP8 rows) or uint8 E8M0
    [K/32, M] (8-bit checkpoint of saved activations)."""
    q: torch.Tensor               # [M, K] float8_e4m3fn
    scales: torch.Tensor

    @property
    def fmt(self) -> int:
        return FP8_BLOCK32_E8M0 if self.scales.dtype == torch.uint8 else FP8_BLOCK128_F32

    def nbytes(self) -> int:
        return self.q.numel() + self.scales.numel() * self.scales.element_size()


@dataclass
class Fp8WeightT:
    """FP8 expert stack: e4m3 [E, N, K] and one fp32 scale per 128 x 128 block."""
    q: torch.Tensor               # [E, N, K] float8_e4m3fn
    scales: torch.Tensor          # [E, ceil(N/128), ceil(K/128)] float32

    @property
    def E(self):
        return self.q.shape[0]

    @property
    def N(self):
        return self.q.shape[1]

    @property
    def K(self):
        return self.q.shape[2]

    def to(self, device) -> "Fp8WeightT":
        return Fp8WeightT(self.q.to(device), self.scales.to(device))

    def nbytes(self) -> int:
        return self.q.numel() + 4 * self.scales.numel()


def _need_fp8_rows(r: Fp8Rows, name: str, M: int, K: int, device, e8m0: bool = False):
    _need(r.q, name + ".q", torch.float8_e4m3fn, (M, K), device)
    if e8m0:
        _need(r.scales, name + ".scales", torch.uint8, (-(-K // 32), M), device)
    else:
        _need(r.scales, name + ".scales", torch.float32, (-(-K // 128), M), device)


def _new_fp8_rows(M: int, K: int, device, e8m0: bool = False) -> Fp8Rows:
    scales = (torch.empty(-(-K // 32), M, dtype=torch.uint8, device=device) if e8m0 else
              torch.empty(-(-K // 128), M, dtype=torch.float32, device=device))
    return Fp8Rows(torch.empty(M, K, dtype=torch.float8_e4m3fn, device=device), scales)


def _fp8_weight_c(w: Fp8WeightT, device) -> Fp8WeightC:
    q = w.q
    if q.dim() != 3:
        raise ValueError("w.q: expected [E, N, K]")
    E, N, K = q.shape
    _need(q, "w.q", torch.float8_e4m3fn, (E, N, K), device)
    _need(w.scales, "w.scales", torch.float32, (E, -(-N // 128), -(-K // 128)), device)
    return Fp8WeightC(q.data_ptr(), w.scales.data_ptr(), E, N, K)


def _groups_c(routing: Routing, E: int, device) -> GroupsC:
    i32 = torch.int32
    _need(routing.expert_offsets, "routing.expert_offsets", i32, (E + 1,), device)
    _need(routing.active, "routing.active", i32, (E,), device)
    _need(routing.num_active, "routing.num_active", i32, (1,), device)
    return GroupsC(routing.expert_offsets.data_ptr(), routing.active.data_ptr(),
                   routing.num_active.data_ptr(), None, None, E)


def moe_quantize_fp8_rows(x: torch.Tensor, routing: Routing | None = None, stream=None,
                          out: Fp8Rows | None = None) -> Fp8Rows:
    """BF16 rows [T, K] to FP8 rows; with a routing, token t is written to its k permuted rows
    (the grouped product's input, [T*k, K])."""
    if x.dim() != 2:
        raise ValueError("x: expected [T, K]")
    T, K = x.shape
    dev = x.device
    _need(x, "x", torch.bfloat16, (T, K))
    k = 1 if routing is None else routing.k
    if routing is not None:
        _need(routing.inv_perm, "routing.inv_perm", torch.int32, (T * k,), dev)
    with _on(dev, stream):
        if out is None:
            out = _new_fp8_rows(T * k, K, dev)
        else:
            _need_fp8_rows(out, "out", T * k, K, dev)
        _check(lib().moe_quantize_fp8_rows(_p(x), T, K, None if routing is None else _p(routing.inv_perm),
                                           k, _p(out.q), _p(out.scales), _here(dev)),
               "moe_quantize_fp8_rows")
    return out


def moe_dequantize_fp8_rows(rows: Fp8Rows, stream=None, out: torch.Tensor | None = None) -> torch.Tensor:
    """FP8 rows or an 8-bit checkpoint as BF16 [M, K]."""
    if rows.q.dim() != 2:
        raise ValueError("rows.q: expected [M, K]")
    M, K = rows.q.shape
    dev = rows.q.device
    _need_fp8_rows(rows, "rows", M, K, dev, rows.fmt == FP8_BLOCK32_E8M0)
    with _on(dev, stream):
        if out is None:
            out = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
        else:
            _need(out, "out", torch.bfloat16, (M, K), dev)
        _check(lib().moe_dequantize_fp8_rows(_p(rows.q), _p(rows.scales), M, K, rows.fmt, _p(out),
                                             _here(dev)), "moe_dequantize_fp8_rows")
    return out


def moe_grouped_fp8_gemm_fwd(a: Fp8Rows, w: Fp8WeightT, routing: Routing, epi: int = EPI_NONE,
                             save_gu: bool = False, stream=None):
    """EPI_NONE: BF16 [M, N]. EPI_SWIGLU: (h as Fp8Rows [M, N/2], the 8-bit checkpoint of
    gate|up as Fp8Rows [M, N], or None without save_gu)."""
    if a.q.dim() != 2:
        raise ValueError("a.q: expected [M, K]")
    M, dev = a.q.shape[0], a.q.device
    wc = _fp8_weight_c(w, dev)
    g, N = _groups_c(routing, wc.E, dev), wc.N
    _need_fp8_rows(a, "a", M, wc.K, dev)
    if save_gu and epi != EPI_SWIGLU:
        raise ValueError("save_gu: only with EPI_SWIGLU")
    with _on(dev, stream):
        if epi == EPI_SWIGLU:
            h = _new_fp8_rows(M, N // 2, dev)
            saved = _new_fp8_rows(M, N, dev, e8m0=True) if save_gu else None
            outs = (_p(h.q), _p(h.scales), _p(saved.q) if save_gu else None,
                    _p(saved.scales) if save_gu else None)
        else:
            out = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
            outs = (_p(out), None, None, None)
        _check(lib().moe_grouped_fp8_gemm_fwd(_p(a.q), _p(a.scales), M, ctypes.byref(wc), ctypes.byref(g),
                                              epi, *outs, _here(dev)), "moe_grouped_fp8_gemm_fwd")
    return (h, saved) if epi == EPI_SWIGLU else out


def moe_grouped_fp8_gemm_bwd_dx(dout: Fp8Rows, w: Fp8WeightT, routing: Routing, epi: int = EPI_NONE,
                                saved: Fp8Rows | None = None, stream=None):
    """EPI_NONE: din, BF16 [M, K]. EPI_SWIGLU_BWD: [dg | du] as Fp8Rows [M, 2K] from the 8-bit
    checkpoint `saved` [M, 2K]."""
    if dout.q.dim() != 2:
        raise ValueError("dout.q: expected [M, N]")
    M, dev = dout.q.shape[0], dout.q.device
    wc = _fp8_weight_c(w, dev)
    g, K = _groups_c(routing, wc.E, dev), wc.K
    _need_fp8_rows(dout, "dout", M, wc.N, dev)
    glu = epi == EPI_SWIGLU_BWD
    if glu != (saved is not None):
        raise ValueError("saved: exactly with EPI_SWIGLU_BWD")
    if glu:
        _need_fp8_rows(saved, "saved", M, 2 * K, dev, e8m0=True)
    with _on(dev, stream):
        if glu:
            out = _new_fp8_rows(M, 2 * K, dev)
            outs = (_p(saved.q), _p(saved.scales), _p(out.q), _p(out.scales))
        else:
            out = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
            outs = (None, None, _p(out), None)
        _check(lib().moe_grouped_fp8_gemm_bwd_dx(_p(dout.q), _p(dout.scales), M, ctypes.byref(wc),
                                                 ctypes.byref(g), epi, *outs, _here(dev)),
               "moe_grouped_fp8_gemm_bwd_dx")
    return out


def moe_test_set_wait_budget(cycles: int):
    _check(lib().moe_test_set_wait_budget(int(cycles)), "moe_test_set_wait_budget")
