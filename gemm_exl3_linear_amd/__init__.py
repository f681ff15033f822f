"""Python binding of the MI355X EXL3 library (libexl3.so, C ABI in include/exl3.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  PyTorch supplies device memory and the current stream.  The library
must have been built (``python -m gemm_exl3_linear_amd.build`` or
``__graft_entry__.build()``); importing this package does not load it, the
first call does, and a missing library raises instead of falling back.
"""
from __future__ import annotations

import ctypes
import operator
import os
import re
from dataclasses import dataclass
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB_PATH = os.path.join(HERE, "libexl3.so")
HEADER_PATH = os.path.join(ROOT, "include", "exl3.h")

EXL3_OK = 0
EXL3_E_INVALID = 1
EXL3_E_UNSUPPORTED = 2
EXL3_E_WORKSPACE = 3
EXL3_E_HIP = 4
EXL3_F16 = 0
EXL3_F32 = 1
CODEBOOK_MUL1 = 2
MAX_TOPK = 16
MAX_MULTI = 8
SCRATCH_BYTES = 32 << 20  # EXL3_SCRATCH_BYTES
MX4_BLOCK = 32
MX4_LINEAR_MAX_ROWS = 64
MX4_MOE_MAX_TOKENS = 16
MX4_MOE_MAX_EXPERTS = 1024
ROUTE_SOFTMAX = 0
ROUTE_SIGMOID = 1
ROUTE_MAX_EXPERTS = 1024
ROUTE_MAX_GROUPS = 64
GROUP_MAX = 0
GROUP_TOP2 = 1
LORA_MAX_RANK = 256
LORA_MAX_ADAPTERS = 4096


class Exl3Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} (status {status})")


class _Weight(ctypes.Structure):
    _fields_ = [("trellis", ctypes.c_void_p), ("suh", ctypes.c_void_p), ("svh", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("k", ctypes.c_int32), ("n", ctypes.c_int32),
                ("bits", ctypes.c_int32), ("codebook", ctypes.c_int32)]


class _Arena(ctypes.Structure):
    _fields_ = [("trellis", ctypes.c_void_p), ("suh", ctypes.c_void_p), ("svh", ctypes.c_void_p),
                ("experts", ctypes.c_int32), ("slots", ctypes.c_int32), ("k", ctypes.c_int32),
                ("n", ctypes.c_int32), ("bits", ctypes.c_int32), ("codebook", ctypes.c_int32)]


class _Widths(ctypes.Structure):
    _fields_ = [("bits_host", ctypes.c_void_p), ("bits", ctypes.c_void_p), ("offsets", ctypes.c_void_p)]


class _Mx4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("k", ctypes.c_int64)]


class _Mx4Experts(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("experts", ctypes.c_int32),
                ("slots", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32)]


class _Mx4MoeLayer(ctypes.Structure):
    _fields_ = [("router", ctypes.c_void_p), ("router_bias", ctypes.c_void_p), ("scoring", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float), ("gate_up", _Mx4Experts),
                ("down", _Mx4Experts), ("shared_gate_up", _Mx4Experts), ("shared_down", _Mx4Experts),
                ("shared_gate", ctypes.c_void_p)]


class _RouteRule(ctypes.Structure):
    _fields_ = [("balance", ctypes.c_void_p), ("experts", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("scoring", ctypes.c_int32), ("groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]


class _RouterWeight(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("experts", ctypes.c_int32),
                ("hidden", ctypes.c_int32)]


class _LoraStack(ctypes.Structure):
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("ranks", ctypes.c_void_p), ("adapters", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("k", ctypes.c_int64), ("n", ctypes.c_int64)]


_lib = None


def header_functions() -> list[str]:
    """Names of the functions include/exl3.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(exl3_[a-z_0-9]+)\s*\(", text)))


def lib() -> ctypes.CDLL:
    """Load libexl3.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it first (python -m gemm_exl3_linear_amd.build)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L.exl3_abi_version.restype = i32
    L.exl3_abi_version.argtypes = []
    L.exl3_status_str.restype = ctypes.c_char_p
    L.exl3_status_str.argtypes = [i32]
    L.exl3_reconstruct.restype = i32
    L.exl3_reconstruct.argtypes = [ctypes.POINTER(_Weight), vp, vp]
    L.exl3_hadamard.restype = i32
    L.exl3_hadamard.argtypes = [vp, vp, i32, i64, i64, i64, i64, vp, vp, vp]
    L.exl3_linear_workspace_size.restype = sz
    L.exl3_linear_workspace_size.argtypes = [ctypes.POINTER(_Weight), i64]
    L.exl3_linear.restype = i32
    L.exl3_linear.argtypes = [ctypes.POINTER(_Weight), vp, i64, i64, vp, i64, i32, vp, sz, vp]
    L.exl3_linear_no_workspace.restype = i32
    L.exl3_linear_no_workspace.argtypes = [ctypes.POINTER(_Weight), vp, i64, i64, vp, i64, i32, vp]
    L.exl3_reconstruct_int8.restype = i32
    L.exl3_reconstruct_int8.argtypes = [ctypes.POINTER(_Weight), vp, vp]
    L.exl3_linear_int8_workspace_size.restype = sz
    L.exl3_linear_int8_workspace_size.argtypes = [ctypes.POINTER(_Weight), i64]
    L.exl3_linear_int8.restype = i32
    L.exl3_linear_int8.argtypes = [ctypes.POINTER(_Weight), vp, i64, i64, vp, i64, i32, vp, sz, vp]
    L.exl3_linear_multi_workspace_size.restype = sz
    L.exl3_linear_multi_workspace_size.argtypes = [ctypes.POINTER(ctypes.POINTER(_Weight)), i32, i64]
    L.exl3_linear_multi.restype = i32
    L.exl3_linear_multi.argtypes = [ctypes.POINTER(ctypes.POINTER(_Weight)), i32, vp, i64, i64,
                                    ctypes.POINTER(vp), ctypes.POINTER(i64), i32, vp, sz, vp]
    L.exl3_grouped_experts_workspace_size.restype = sz
    L.exl3_grouped_experts_workspace_size.argtypes = [ctypes.POINTER(_Arena), ctypes.POINTER(_Arena), i64, i32]
    L.exl3_grouped_experts.restype = i32
    L.exl3_grouped_experts.argtypes = [ctypes.POINTER(_Arena), ctypes.POINTER(_Arena), vp, vp, vp, i64, i32,
                                       vp, vp, sz, vp]
    Wp = ctypes.POINTER(_Widths)
    L.exl3_grouped_experts_mixed_workspace_size.restype = sz
    L.exl3_grouped_experts_mixed_workspace_size.argtypes = [ctypes.POINTER(_Arena), Wp, ctypes.POINTER(_Arena),
                                                            Wp, i64, i32]
    L.exl3_grouped_experts_mixed.restype = i32
    L.exl3_grouped_experts_mixed.argtypes = [ctypes.POINTER(_Arena), Wp, ctypes.POINTER(_Arena), Wp, vp, vp, vp,
                                             i64, i32, vp, vp, sz, vp]
    Mp, Lp = ctypes.POINTER(_Mx4), ctypes.POINTER(_Mx4MoeLayer)
    L.exl3_mx4_quantize.restype = i32
    L.exl3_mx4_quantize.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp]
    L.exl3_mx4_reconstruct.restype = i32
    L.exl3_mx4_reconstruct.argtypes = [Mp, vp, i32, i64, vp]
    L.exl3_mx4_matmul_workspace_size.restype = sz
    L.exl3_mx4_matmul_workspace_size.argtypes = [Mp, Mp]
    L.exl3_mx4_matmul.restype = i32
    L.exl3_mx4_matmul.argtypes = [Mp, Mp, vp, vp, i64, i32, vp, sz, vp]
    L.exl3_mx4_linear_workspace_size.restype = sz
    L.exl3_mx4_linear_workspace_size.argtypes = [Mp, i64]
    L.exl3_mx4_linear.restype = i32
    L.exl3_mx4_linear.argtypes = [Mp, vp, vp, i64, i64, vp, i64, i32, vp, sz, vp]
    L.exl3_mx4_moe_workspace_size.restype = sz
    L.exl3_mx4_moe_workspace_size.argtypes = [Lp, i64, i32]
    L.exl3_mx4_moe.restype = i32
    L.exl3_mx4_moe.argtypes = [Lp, vp, i64, i64, i32, vp, i64, i32, vp, vp, vp, sz, vp]
    rule, router, lora = ctypes.POINTER(_RouteRule), ctypes.POINTER(_RouterWeight), ctypes.POINTER(_LoraStack)
    L.exl3_route_topk.restype = i32
    L.exl3_route_topk.argtypes = [rule, vp, i32, i64, i64, vp, vp, vp]
    L.exl3_router_linear_workspace_size.restype = sz
    L.exl3_router_linear_workspace_size.argtypes = [router, i64]
    L.exl3_router_linear.restype = i32
    L.exl3_router_linear.argtypes = [router, vp, i64, i64, vp, i64, vp, sz, vp]
    L.exl3_router_workspace_size.restype = sz
    L.exl3_router_workspace_size.argtypes = [router, i64, i32]
    L.exl3_router.restype = i32
    L.exl3_router.argtypes = [router, rule, vp, i64, i64, vp, i64, vp, vp, vp, sz, vp]
    L.exl3_lora_workspace_size.restype = sz
    L.exl3_lora_workspace_size.argtypes = [lora, i64]
    L.exl3_lora.restype = i32
    L.exl3_lora.argtypes = [lora, vp, i64, i64, vp, vp, i64, vp, i64, i32, vp, sz, vp]
    _lib = L
    return L


def status_str(status: int) -> str:
    return lib().exl3_status_str(int(status)).decode()


def abi_version() -> int:
    return int(lib().exl3_abi_version())


def _check(status: int, what: str):
    if status != EXL3_OK:
        raise Exl3Error(status, what)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream(stream=None) -> int:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


# ---------------------------------------------------------------------------
# tensors
# ---------------------------------------------------------------------------
@dataclass
class Exl3Weight:
    """One EXL3 tensor on the GPU: trellis int16/uint16 [k/16, n/16, 16*bits],
    suh fp16 [k], svh fp16 [n], optional bias fp16 [n]."""
    trellis: "object"
    suh: "object"
    svh: "object"
    bits: int
    bias: Optional["object"] = None
    codebook: int = CODEBOOK_MUL1

    @property
    def k(self) -> int:
        return int(self.trellis.shape[0]) * 16

    @property
    def n(self) -> int:
        return int(self.trellis.shape[1]) * 16

    def _c(self) -> _Weight:
        return _Weight(_ptr(self.trellis), _ptr(self.suh), _ptr(self.svh), _ptr(self.bias),
                       self.k, self.n, int(self.bits), int(self.codebook))

    @staticmethod
    def from_numpy(trellis, suh, svh, bits, bias=None, device="cuda"):
        import torch
        t = torch.from_numpy(trellis.view("int16").copy()).to(device)
        s1 = torch.from_numpy(suh.astype("float16")).to(device)
        s2 = torch.from_numpy(svh.astype("float16")).to(device)
        b = None if bias is None else torch.from_numpy(bias.astype("float16")).to(device)
        return Exl3Weight(t, s1, s2, bits, b)


@dataclass
class Exl3Arena:
    """Packed expert arena on the GPU: trellis [E, slots, k/16, n/16, 16*bits],
    suh fp16 [E, slots, k], svh fp16 [E, slots, n]."""
    trellis: "object"
    suh: "object"
    svh: "object"
    bits: int
    codebook: int = CODEBOOK_MUL1

    @property
    def experts(self) -> int:
        return int(self.trellis.shape[0])

    @property
    def slots(self) -> int:
        return int(self.trellis.shape[1])

    @property
    def k(self) -> int:
        return int(self.trellis.shape[2]) * 16

    @property
    def n(self) -> int:
        return int(self.trellis.shape[3]) * 16

    def _c(self) -> _Arena:
        return _Arena(_ptr(self.trellis), _ptr(self.suh), _ptr(self.svh), self.experts, self.slots,
                      self.k, self.n, int(self.bits), int(self.codebook))

    @staticmethod
    def from_numpy(arena: dict, device="cuda"):
        import torch
        return Exl3Arena(torch.from_numpy(arena["trellis"].view("int16").copy()).to(device),
                         torch.from_numpy(arena["suh"].astype("float16")).to(device),
                         torch.from_numpy(arena["svh"].astype("float16")).to(device),
                         int(arena["bits"]))


@dataclass
class Exl3MixedArena:
    """Expert arena with a width per expert on the GPU: trellis int16/uint16
    [total words] with expert e's slots at word offsets[e] on, widths int32
    [E] both on the host (``bits_host``, a ctypes array the record points to)
    and on the GPU (``bits``), offsets int64 [E] on the GPU, suh fp16
    [E, slots, k], svh fp16 [E, slots, n]."""
    trellis: "object"
    suh: "object"
    svh: "object"
    bits: "object"
    offsets: "object"
    bits_host: "object"
    codebook: int = CODEBOOK_MUL1

    @property
    def experts(self) -> int:
        return int(self.suh.shape[0])

    @property
    def slots(self) -> int:
        return int(self.suh.shape[1])

    @property
    def k(self) -> int:
        return int(self.suh.shape[2])

    @property
    def n(self) -> int:
        return int(self.svh.shape[2])

    def _c(self) -> _Arena:
        return _Arena(_ptr(self.trellis), _ptr(self.suh), _ptr(self.svh), self.experts, self.slots,
                      self.k, self.n, 0, int(self.codebook))

    def _w(self) -> _Widths:
        return _Widths(ctypes.addressof(self.bits_host), _ptr(self.bits), _ptr(self.offsets))

    @staticmethod
    def from_numpy(arena: dict, device="cuda"):
        """Packs the per-expert trellis arrays (entry e [slots, k/16, n/16,
        16*bits[e]]) one after the other into one allocation."""
        import numpy as np
        import torch
        widths = [int(b) for b in arena["bits"]]
        sizes = [int(t.size) for t in arena["trellis"]]
        offsets = np.concatenate([[0], np.cumsum(sizes)[:-1]]).astype(np.int64)
        flat = np.concatenate([np.ascontiguousarray(t).reshape(-1) for t in arena["trellis"]])
        host = (ctypes.c_int32 * len(widths))(*widths)
        return Exl3MixedArena(torch.from_numpy(flat.view("int16").copy()).to(device),
                              torch.from_numpy(arena["suh"].astype("float16")).to(device),
                              torch.from_numpy(arena["svh"].astype("float16")).to(device),
                              torch.tensor(widths, dtype=torch.int32, device=device),
                              torch.from_numpy(offsets).to(device), host)


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def exl3_reconstruct(w: Exl3Weight, out=None, stream=None):
    import torch
    if out is None:
        out = torch.empty((w.k, w.n), dtype=torch.float16, device=w.trellis.device)
    cw = w._c()
    _check(lib().exl3_reconstruct(ctypes.byref(cw), _ptr(out), _stream(stream)), "exl3_reconstruct")
    return out


def exl3_hadamard(x, sign_before=None, sign_after=None, out=None, stream=None):
    import torch
    assert x.dim() == 2 and x.stride(1) == 1
    dtype = {torch.float16: EXL3_F16, torch.float32: EXL3_F32}[x.dtype]
    if out is None:
        out = torch.empty_like(x)
    rows, dim = x.shape
    _check(lib().exl3_hadamard(_ptr(x), _ptr(out), dtype, rows, dim, x.stride(0), out.stride(0),
                               _ptr(sign_before), _ptr(sign_after), _stream(stream)), "exl3_hadamard")
    return out


def exl3_linear_workspace_size(w: Exl3Weight, m: int) -> int:
    cw = w._c()
    return int(lib().exl3_linear_workspace_size(ctypes.byref(cw), int(m)))


def _ydt(dtype) -> int:
    import torch
    if dtype == torch.float16:
        return EXL3_F16
    if dtype == torch.float32:
        return EXL3_F32
    raise ValueError(f"output dtype {dtype} is not fp16 or fp32")


def exl3_linear(x, w: Exl3Weight, out_dtype=None, out=None, workspace=None, stream=None):
    import torch
    assert x.dim() == 2 and x.dtype == torch.float16 and x.stride(1) == 1
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, w.n), dtype=out_dtype or torch.float16, device=x.device)
    ydt = _ydt(out.dtype)
    cw = w._c()
    if workspace is None:  # a caller's workspace is checked against the size by the library
        need = int(lib().exl3_linear_workspace_size(ctypes.byref(cw), int(m)))
        if need:  # scratch only: no clearing needed
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().exl3_linear(ctypes.byref(cw), _ptr(x), m, x.stride(0), _ptr(out), out.stride(0), ydt,
                             _ptr(workspace), wsb, _stream(stream)), "exl3_linear")
    return out


def exl3_linear_no_workspace(x, w: Exl3Weight, out, stream=None):
    """exl3_linear_no_workspace: exl3_linear with the library's own device
    array as workspace; the caller passes the output (nothing is allocated
    here or in the library)."""
    import torch
    assert x.dim() == 2 and x.dtype == torch.float16 and x.stride(1) == 1
    assert out.dim() == 2 and out.shape[0] == x.shape[0]
    cw = w._c()
    _check(lib().exl3_linear_no_workspace(ctypes.byref(cw), _ptr(x), x.shape[0], x.stride(0), _ptr(out),
                                          out.stride(0), _ydt(out.dtype), _stream(stream)),
           "exl3_linear_no_workspace")
    return out


def exl3_reconstruct_int8(w: Exl3Weight, out=None, stream=None):
    """int8 weights W_q [k, n] of the int8 prefill (exl3_reconstruct_int8)."""
    import torch
    if out is None:
        out = torch.empty((w.k, w.n), dtype=torch.int8, device=w.trellis.device)
    cw = w._c()
    _check(lib().exl3_reconstruct_int8(ctypes.byref(cw), _ptr(out), _stream(stream)),
           "exl3_reconstruct_int8")
    return out


def exl3_linear_int8_workspace_size(w: Exl3Weight, m: int) -> int:
    cw = w._c()
    return int(lib().exl3_linear_int8_workspace_size(ctypes.byref(cw), int(m)))


def exl3_linear_int8(x, w: Exl3Weight, out_dtype=None, out=None, workspace=None, stream=None):
    """The int8 prefill linear (exl3_linear_int8): x fp16 [m, k] -> y [m, n]."""
    import torch
    assert x.dim() == 2 and x.dtype == torch.float16 and x.stride(1) == 1
    m = x.shape[0]
    if out is None:
        out = torch.empty((m, w.n), dtype=out_dtype or torch.float16, device=x.device)
    ydt = _ydt(out.dtype)
    cw = w._c()
    if workspace is None:
        need = int(lib().exl3_linear_int8_workspace_size(ctypes.byref(cw), int(m)))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().exl3_linear_int8(ctypes.byref(cw), _ptr(x), m, x.stride(0), _ptr(out), out.stride(0),
                                  ydt, _ptr(workspace), wsb, _stream(stream)), "exl3_linear_int8")
    return out


def _weight_array(ws):
    """ctypes array of pointers to the tensors' C records (records kept alive)."""
    recs = [w._c() for w in ws]
    arr = (ctypes.POINTER(_Weight) * len(recs))(*[ctypes.pointer(r) for r in recs])
    return arr, recs


def exl3_linear_multi_workspace_size(ws, m: int) -> int:
    arr, _recs = _weight_array(ws)
    return int(lib().exl3_linear_multi_workspace_size(arr, len(ws), int(m)))


def exl3_linear_multi(x, ws, out_dtype=None, outs=None, workspace=None, stream=None):
    """y[i] = exl3_linear(x, ws[i]) for tensors that share the input x (same k)."""
    import torch
    assert x.dim() == 2 and x.dtype == torch.float16 and x.stride(1) == 1
    m = x.shape[0]
    if outs is None:
        outs = [torch.empty((m, w.n), dtype=out_dtype or torch.float16, device=x.device) for w in ws]
    ydt = _ydt(outs[0].dtype)
    arr, _recs = _weight_array(ws)
    if workspace is None:
        need = int(lib().exl3_linear_multi_workspace_size(arr, len(ws), int(m)))
        if need:  # scratch only: no clearing needed
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    yp = (ctypes.c_void_p * len(outs))(*[_ptr(o) for o in outs])
    ld = (ctypes.c_int64 * len(outs))(*[o.stride(0) for o in outs])
    _check(lib().exl3_linear_multi(arr, len(ws), _ptr(x), m, x.stride(0), yp, ld, ydt, _ptr(workspace), wsb,
                                   _stream(stream)), "exl3_linear_multi")
    return outs


def exl3_grouped_experts_workspace_size(gate_up: Exl3Arena, down: Exl3Arena, t: int, topk: int) -> int:
    a, b = gate_up._c(), down._c()
    return int(lib().exl3_grouped_experts_workspace_size(ctypes.byref(a), ctypes.byref(b), int(t), int(topk)))


def exl3_grouped_experts(x, topk_ids, topk_weights, gate_up: Exl3Arena, down: Exl3Arena, out=None,
                         workspace=None, stream=None):
    import torch
    assert x.dtype == torch.float16 and x.is_contiguous()
    assert topk_ids.dtype == torch.int32 and topk_ids.is_contiguous()
    assert topk_weights.dtype == torch.float32 and topk_weights.is_contiguous()
    t, topk = topk_ids.shape
    if out is None:
        out = torch.empty((t, down.n), dtype=torch.float32, device=x.device)
    a, b = gate_up._c(), down._c()
    if workspace is None:
        need = int(lib().exl3_grouped_experts_workspace_size(ctypes.byref(a), ctypes.byref(b), int(t), int(topk)))
        if need:
            workspace = torch.zeros(need, dtype=torch.uint8, device=x.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().exl3_grouped_experts(ctypes.byref(a), ctypes.byref(b), _ptr(x), _ptr(topk_ids),
                                      _ptr(topk_weights), t, topk, _ptr(out), _ptr(workspace), wsb,
                                      _stream(stream)), "exl3_grouped_experts")
    return out


def exl3_grouped_experts_mixed_workspace_size(gate_up: Exl3MixedArena, down: Exl3MixedArena, t: int,
                                              topk: int) -> int:
    a, b = gate_up._c(), down._c()
    wa, wb = gate_up._w(), down._w()
    return int(lib().exl3_grouped_experts_mixed_workspace_size(ctypes.byref(a), ctypes.byref(wa), ctypes.byref(b),
                                                               ctypes.byref(wb), int(t), int(topk)))


def exl3_grouped_experts_mixed(x, topk_ids, topk_weights, gate_up: Exl3MixedArena, down: Exl3MixedArena,
                               out=None, workspace=None, stream=None):
    """exl3_grouped_experts over arenas whose experts each have their own width."""
    import torch
    assert x.dtype == torch.float16 and x.is_contiguous()
    assert topk_ids.dtype == torch.int32 and topk_ids.is_contiguous()
    assert topk_weights.dtype == torch.float32 and topk_weights.is_contiguous()
    t, topk = topk_ids.shape
    if out is None:
        out = torch.empty((t, down.n), dtype=torch.float32, device=x.device)
    a, b = gate_up._c(), down._c()
    wa, wb = gate_up._w(), down._w()
    if workspace is None:
        need = int(lib().exl3_grouped_experts_mixed_workspace_size(ctypes.byref(a), ctypes.byref(wa),
                                                                   ctypes.byref(b), ctypes.byref(wb), int(t),
                                                                   int(topk)))
        if need:
            workspace = torch.zeros(need, dtype=torch.uint8, device=x.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().exl3_grouped_experts_mixed(ctypes.byref(a), ctypes.byref(wa), ctypes.byref(b), ctypes.byref(wb),
                                            _ptr(x), _ptr(topk_ids), _ptr(topk_weights), t, topk, _ptr(out),
                                            _ptr(workspace), wsb, _stream(stream)), "exl3_grouped_experts_mixed")
    return out


# ---------------------------------------------------------------------------
# MXFP4 (microscaled 4-bit floating point)
# ---------------------------------------------------------------------------
def _refuse(what: str):
    raise ValueError(what)


# Host time counts for single tokens (a launch takes 3.7 us): what the calls below
# look up each time is kept here, since an import inside a function costs 0.2 us.
_dtype_codes = {}    # torch dtype -> EXL3_F16, EXL3_F32
_cuda_queries = []   # current device, current stream of a device
_number_types = []   # torch.int32, torch.float32 (from the first _place on)
_shape = operator.attrgetter("shape")


def _place(t, what: str, stream):
    """Device index and stream handle (the current stream's if None) of a call on
    t, which has to be on the current device: the library launches there.  The raw
    query costs 0.1 us of host time where torch.cuda.current_stream() costs 2.9."""
    i = t.get_device()
    if i < 0:
        _refuse(f"{what} is not on a GPU")
    if not _cuda_queries:
        import torch
        _number_types[:] = (torch.int32, torch.float32)
        _cuda_queries.extend((torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream))
    if i != _cuda_queries[0]():
        _refuse(f"{what} is on GPU {i}, not on the current device")
    if stream is None:
        return i, _cuda_queries[1](i)
    if stream.device_index != i:
        _refuse(f"the stream is of GPU {stream.device_index}, {what} is on GPU {i}")
    return i, int(stream.cuda_stream)


def _tensor(t, what: str, dtype, shape):
    """t, checked: dtype, shape (None entries are free), contiguous."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t
    if t.dtype != dtype:
        _refuse(f"{what} is {t.dtype}, not {dtype}")
    if t.shape != shape and (t.dim() != len(shape) or any(s is not None and s != d for s, d in zip(shape, t.shape))):
        _refuse(f"{what} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous():
        _refuse(f"{what} is not contiguous")
    return t


def _f16_f32(t, what: str) -> int:
    if not _dtype_codes:
        import torch
        _dtype_codes.update({torch.float16: EXL3_F16, torch.float32: EXL3_F32})
    code = _dtype_codes.get(t.dtype)
    if code is None:
        _refuse(f"{what} is {t.dtype}, not fp16 or fp32")
    return code


def _f16_rows(x, cols: int):
    """Rows and row stride of the fp16 matrix x, checked."""
    if _f16_f32(x, "x") != EXL3_F16:
        _refuse(f"x is {x.dtype}, not fp16")
    m, _, ld = _matrix(x, "x", None, cols)
    return m, ld


def _matrix(t, what: str, rows: Optional[int], cols: Optional[int]):
    """Rows, columns and row stride of t, checked as a matrix of contiguous rows.
    With fewer than two rows the stride says nothing and the width, rounded up to
    8, stands in."""
    stride = t.stride()
    if len(stride) != 2:
        _refuse(f"{what} is not a matrix")
    m, n = t.shape
    if (rows is not None and m != rows) or (cols is not None and n != cols):
        _refuse(f"{what} has shape {(m, n)}, not {(rows, cols)}")
    if stride[1] != 1 and n > 1 and m:  # of no elements strides say nothing
        _refuse(f"{what} does not have contiguous rows")
    return m, n, stride[0] if m > 1 else -(-n // 8) * 8


def _new(make, shape, dtype, device, stream):
    """make(shape, ...): a tensor of the stream that the call runs on, so that
    its memory is not another stream's, cleared or handed on too early."""
    import torch
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _scratch(workspace, zeroed: bool, need, args, device: int, stream):
    """Address and bytes of the caller's workspace, or of a new one (need(*args)
    bytes), and the tensor that holds it."""
    if workspace is None:
        n = need(*args)
        if not n:
            return 0, 0, None
        import torch
        workspace = _new(torch.zeros if zeroed else torch.empty, n, torch.uint8, device, stream)
        return workspace.data_ptr(), n, workspace
    n = workspace.nbytes
    if n and (workspace.get_device() != device or not workspace.is_contiguous()):
        _refuse("the workspace is on another device than the operands, or not contiguous")
    return workspace.data_ptr(), n, workspace


@dataclass(frozen=True)
class Exl3Mx4:
    """An MXFP4 matrix on the GPU: codes uint8 [rows, k/2] (the even element in
    a byte's low half), scales uint8 [rows, k/32] (2^(s - 127), 255 is NaN)."""
    codes: "object"
    scales: "object"

    def __post_init__(self):
        import torch
        _tensor(self.codes, "codes", torch.uint8, (None, None))
        if self.codes.shape[1] == 0 or self.codes.shape[1] % (MX4_BLOCK // 2):
            _refuse(f"codes have {self.codes.shape[1]} bytes a row, not a multiple of {MX4_BLOCK // 2}")
        _tensor(self.scales, "scales", torch.uint8, (self.codes.shape[0], self.codes.shape[1] // (MX4_BLOCK // 2)))
        if self.codes.device != self.scales.device:
            _refuse("codes and scales are on different devices")
        record = _Mx4(_ptr(self.codes), _ptr(self.scales), self.rows, self.k)
        object.__setattr__(self, "_record", record)
        object.__setattr__(self, "_ref", ctypes.byref(record))
        object.__setattr__(self, "_seen", (_ptr(self.codes), _ptr(self.scales), self.codes.shape))
        object.__setattr__(self, "_fields", (_ptr(self.codes), _ptr(self.scales), self.rows, self.k))

    def _now(self):
        """Addresses of codes and scales, rows and k, with the record of the same
        at _ref: of the tensors as they are.  If their memory or shape was changed
        under them (`.data =`, set_, resize_), they are checked and read again."""
        c, s = self.codes, self.scales
        if (c.data_ptr(), s.data_ptr(), c.shape) != self._seen:
            self.__post_init__()
        return self._fields

    def __reduce__(self):  # copies and pickles take the tensors, not the record's pointers
        return Exl3Mx4, (self.codes, self.scales)

    @property
    def rows(self) -> int:
        return int(self.codes.shape[0])

    @property
    def k(self) -> int:
        return int(self.codes.shape[1]) * 2

    @staticmethod
    def empty(rows: int, k: int, device="cuda"):
        import torch
        return Exl3Mx4(torch.empty((rows, k // 2), dtype=torch.uint8, device=device),
                       torch.empty((rows, k // MX4_BLOCK), dtype=torch.uint8, device=device))


@dataclass(frozen=True)
class Exl3Mx4Arena:
    """MXFP4 tensors of experts on the GPU: codes uint8 [E, slots, n, k/2],
    scales uint8 [E, slots, n, k/32]."""
    codes: "object"
    scales: "object"

    def __post_init__(self):
        import torch
        _tensor(self.codes, "codes", torch.uint8, (None, None, None, None))
        e, slots, n, half = self.codes.shape
        _tensor(self.scales, "scales", torch.uint8, (e, slots, n, half // (MX4_BLOCK // 2)))
        if half == 0 or half % (MX4_BLOCK // 2):
            _refuse(f"codes have {half} bytes a row, not a multiple of {MX4_BLOCK // 2}")
        if self.codes.device != self.scales.device:
            _refuse("codes and scales are on different devices")

    def _c(self) -> _Mx4Experts:
        self.__post_init__()  # the tensors as they are now
        e, slots, n, half = self.codes.shape
        return _Mx4Experts(_ptr(self.codes), _ptr(self.scales), e, slots, n, 2 * half)


@dataclass(frozen=True)
class Exl3MoeRouter:
    """Router of a mixture-of-experts layer: weight fp16 [E, hidden], bias fp32
    [E] or None, scoring "softmax" (chosen and weighted by softmax(l + bias)) or
    "sigmoid" (chosen by sigmoid(l) + bias, weighted by sigmoid(l)); weights are
    divided by their sum if `renormalize`, then multiplied by `scale`."""
    weight: "object"
    bias: Optional["object"] = None
    scoring: str = "softmax"
    renormalize: bool = True
    scale: float = 1.0


@dataclass(frozen=True)
class Exl3Mx4Shared:
    """Shared expert: arenas of one expert, and optionally gate fp16 [hidden]
    (its weight is sigmoid(x . gate), else 1)."""
    gate_up: Exl3Mx4Arena
    down: Exl3Mx4Arena
    gate: Optional["object"] = None


@dataclass(frozen=True)
class Exl3Mx4Moe:
    """A mixture-of-experts layer with MXFP4 experts: gate_up [E, 2, inter, .],
    down [E, 1, hidden, .], and optionally a shared expert."""
    router: Exl3MoeRouter
    gate_up: Exl3Mx4Arena
    down: Exl3Mx4Arena
    shared: Optional[Exl3Mx4Shared] = None

    def __post_init__(self):
        import torch
        gu, dn, sh, r = self.gate_up._c(), self.down._c(), self.shared, self.router
        dev = self.gate_up.codes.device
        tensors = [self.down.codes, _tensor(r.weight, "router weight", torch.float16, (gu.experts, gu.k))]
        if r.bias is not None:
            tensors.append(_tensor(r.bias, "router bias", torch.float32, (gu.experts,)))
        if r.scoring not in ("softmax", "sigmoid"):
            _refuse(f"scoring {r.scoring!r} is not softmax or sigmoid")
        sgu, sdn, gate = _Mx4Experts(), _Mx4Experts(), None
        if sh is not None:
            sgu, sdn, gate = sh.gate_up._c(), sh.down._c(), sh.gate
            tensors += [sh.gate_up.codes, sh.down.codes]
            if gate is not None:
                tensors.append(_tensor(gate, "shared gate", torch.float16, (gu.k,)))
        if any(t.device != dev for t in tensors):
            _refuse("the layer's tensors are on different devices")
        scoring = ROUTE_SOFTMAX if r.scoring == "softmax" else ROUTE_SIGMOID
        record = _Mx4MoeLayer(_ptr(r.weight), _ptr(r.bias), scoring, int(r.renormalize), float(r.scale), gu, dn,
                              sgu, sdn, _ptr(gate))
        arenas = [self.gate_up, self.down] + ([sh.gate_up, sh.down] if sh is not None else [])
        parts = tuple(t for a in arenas for t in (a.codes, a.scales)) + tuple(
            t for t in (r.weight, r.bias, gate) if t is not None)
        widths = tuple(a.codes for a in arenas[::2])  # the others' shapes follow from these
        object.__setattr__(self, "_record", record)
        object.__setattr__(self, "_ref", ctypes.byref(record))
        object.__setattr__(self, "_parts", (parts, widths, torch.Tensor.data_ptr))
        object.__setattr__(self, "_seen", (list(map(_ptr, parts)), list(map(_shape, widths))))

    def _now(self) -> _Mx4MoeLayer:
        """The record of the tensors as they are (Exl3Mx4._now)."""
        parts, widths, data_ptr = self._parts
        if (list(map(data_ptr, parts)), list(map(_shape, widths))) != self._seen:
            self.__post_init__()
        return self._record

    def __reduce__(self):  # copies and pickles take the tensors, not the record's pointers
        return Exl3Mx4Moe, (self.router, self.gate_up, self.down, self.shared)


def exl3_mx4_quantize(x, out: Optional[Exl3Mx4] = None, stream=None) -> Exl3Mx4:
    """MXFP4 of fp16 or fp32 rows x [rows, k], k a multiple of 32."""
    rows, k, ldx = _matrix(x, "x", None, None)
    dtype = _f16_f32(x, "x")
    device, on = _place(x, "x", stream)
    if out is None:
        if k == 0 or k % MX4_BLOCK:
            _refuse(f"x has {k} columns, not a multiple of {MX4_BLOCK}")
        import torch
        out = Exl3Mx4(_new(torch.empty, (rows, k // 2), torch.uint8, device, stream),
                      _new(torch.empty, (rows, k // MX4_BLOCK), torch.uint8, device, stream))
    codes, scales, n, nk = out._now()
    if n != rows or nk != k or out.codes.get_device() != device:
        _refuse("out does not match x")
    _check(lib().exl3_mx4_quantize(x.data_ptr(), dtype, rows, k, ldx, codes, scales, on),
           "exl3_mx4_quantize")
    return out


def exl3_mx4_reconstruct(w: Exl3Mx4, dtype=None, out=None, stream=None):
    """The values w stands for, fp16 (the default) or fp32 [rows, k]."""
    device, on = _place(w.codes, "w", stream)
    _, _, n, k = w._now()
    if out is None:
        import torch
        out = _new(torch.empty, (n, k), dtype or torch.float16, device, stream)
    elif out.get_device() != device:
        _refuse("out is on another device than w")
    ldo = _matrix(out, "out", n, k)[2]
    _check(lib().exl3_mx4_reconstruct(w._ref, out.data_ptr(), _f16_f32(out, "out"), ldo, on),
           "exl3_mx4_reconstruct")
    return out


def _product_out(out, out_dtype, m: int, n: int, device: int, bias, stream):
    """The output of a product (a new one if none is given), its row stride and
    type."""
    if out is None:
        import torch
        out, ldy = _new(torch.empty, (m, n), out_dtype or torch.float16, device, stream), n
    elif out.get_device() != device:
        _refuse("out is on another device than the operands")
    else:
        ldy = _matrix(out, "out", m, n)[2]
    if bias is not None:
        import torch
        _tensor(bias, "bias", torch.float16, (n,))
        if bias.get_device() != device:
            _refuse("bias is on another device than the operands")
    return out, ldy, _f16_f32(out, "out")


def exl3_mx4_matmul_workspace_size(a: Exl3Mx4, b: Exl3Mx4) -> int:
    a._now(), b._now()
    return int(lib().exl3_mx4_matmul_workspace_size(a._ref, b._ref))


def exl3_mx4_matmul(a: Exl3Mx4, b: Exl3Mx4, bias=None, out_dtype=None, out=None, workspace=None, stream=None):
    """y [m, n] = a [m, k] b [n, k]^T (+ bias fp16 [n]), both MXFP4."""
    device, on = _place(a.codes, "a", stream)
    if b.codes.get_device() != device:
        _refuse("a and b are on different devices")
    out, ldy, ydt = _product_out(out, out_dtype, a._now()[2], b._now()[2], device, bias, stream)
    ws, nws, _keep = _scratch(workspace, False, lib().exl3_mx4_matmul_workspace_size, (a._ref, b._ref), device, stream)
    _check(lib().exl3_mx4_matmul(a._ref, b._ref, _ptr(bias), out.data_ptr(), ldy, ydt, ws, nws, on),
           "exl3_mx4_matmul")
    return out


def exl3_mx4_linear_workspace_size(w: Exl3Mx4, m: int) -> int:
    w._now()
    return int(lib().exl3_mx4_linear_workspace_size(w._ref, int(m)))


def exl3_mx4_linear(x, w: Exl3Mx4, bias=None, out_dtype=None, out=None, workspace=None, stream=None):
    """y [m, n] = x w^T (+ bias fp16 [n]): fp16 rows x [m, k], m up to 64,
    against MXFP4 weights w [n, k]."""
    _, _, n, k = w._now()
    m, ldx = _f16_rows(x, k)
    device, on = _place(x, "x", stream)
    if w.codes.get_device() != device:
        _refuse("x and w are on different devices")
    out, ldy, ydt = _product_out(out, out_dtype, m, n, device, bias, stream)
    ws, nws, _keep = _scratch(workspace, False, lib().exl3_mx4_linear_workspace_size, (w._ref, m), device, stream)
    _check(lib().exl3_mx4_linear(w._ref, _ptr(bias), x.data_ptr(), m, ldx, out.data_ptr(), ldy, ydt, ws, nws,
                                 on), "exl3_mx4_linear")
    return out


def exl3_mx4_moe_workspace_size(layer: Exl3Mx4Moe, t: int, topk: int) -> int:
    layer._now()
    return int(lib().exl3_mx4_moe_workspace_size(layer._ref, int(t), int(topk)))


def exl3_mx4_moe(x, layer: Exl3Mx4Moe, topk: int, out_dtype=None, out=None, topk_ids=None, topk_weights=None,
                 workspace=None, stream=None):
    """A whole mixture-of-experts layer for up to 16 tokens x fp16 [t, hidden]:
    router, top-k, SwiGLU experts, shared expert.  topk_ids int32 and
    topk_weights fp32 [t, topk] receive the routing if given.  A workspace
    passed in has to be zero-filled before its first use and is then left to
    this function."""
    import torch
    hidden = layer._now().gate_up.k
    t, ldx = _f16_rows(x, hidden)
    device, on = _place(x, "x", stream)
    if layer.gate_up.codes.get_device() != device:
        _refuse("x and the layer are on different devices")
    out, ldy, ydt = _product_out(out, out_dtype, t, hidden, device, None, stream)
    for v, what, dt in ((topk_ids, "topk_ids", torch.int32), (topk_weights, "topk_weights", torch.float32)):
        if v is not None and _tensor(v, what, dt, (t, topk)).get_device() != device:
            _refuse(f"{what} is on another device than x")
    ws, nws, _keep = _scratch(workspace, True, lib().exl3_mx4_moe_workspace_size, (layer._ref, t, topk), device, stream)
    _check(lib().exl3_mx4_moe(layer._ref, x.data_ptr(), t, ldx, topk, out.data_ptr(), ldy, ydt, _ptr(topk_ids),
                              _ptr(topk_weights), ws, nws, on), "exl3_mx4_moe")
    return out


# ---------------------------------------------------------------------------
# Routing to experts
# ---------------------------------------------------------------------------
def _int32(v, what: str) -> int:
    """v as a C int, which a record's field would else take modulo 2^32."""
    i = operator.index(v)
    if not -(1 << 31) <= i < 1 << 31:
        _refuse(f"{what} is {i}, past 32 bits")
    return i


class _Record:
    """A record of tensors: subclasses give `_tensors()` (the checked tensors, None
    left out) and `_make(...)`, the C record of them."""

    def __post_init__(self):
        import torch
        parts = self._tensors()
        if any(t.device != parts[0].device for t in parts):
            _refuse("the tensors are on different devices")
        record = self._make()
        object.__setattr__(self, "_record", record)
        object.__setattr__(self, "_ref", ctypes.byref(record))
        object.__setattr__(self, "_parts", (parts, torch.Tensor.data_ptr))
        object.__setattr__(self, "_seen", (list(map(_ptr, parts)), list(map(_shape, parts))))

    def _now(self):
        """The record of the tensors as they are: checked and read again if their
        memory or shape was changed under them (`.data =`, set_, resize_).  A change of
        strides alone, as by t_() of a square matrix, is not seen: asking each tensor
        costs every call 0.1 to 0.2 us."""
        parts, data_ptr = self._parts
        if parts and (list(map(data_ptr, parts)), list(map(_shape, parts))) != self._seen:
            self.__post_init__()
        return self._record

    def __reduce__(self):  # copies and pickles take the tensors, not the record's pointers
        return type(self), tuple(getattr(self, f) for f in self.__dataclass_fields__)


@dataclass(frozen=True)
class Exl3Router(_Record):
    """A router's linear: weight fp16 [experts, hidden], bias fp32 [experts] or None."""
    weight: "object"
    bias: Optional["object"] = None

    def _tensors(self):
        import torch
        parts = [_tensor(self.weight, "router weight", torch.float16, (None, None))]
        if self.bias is not None:
            parts.append(_tensor(self.bias, "router bias", torch.float32, (self.experts,)))
        return parts

    def _make(self):
        return _RouterWeight(_ptr(self.weight), _ptr(self.bias), _int32(self.experts, "experts"),
                             _int32(self.hidden, "hidden"))

    @property
    def experts(self) -> int:
        return int(self.weight.shape[0])

    @property
    def hidden(self) -> int:
        return int(self.weight.shape[1])


@dataclass(frozen=True)
class Exl3RouteRule(_Record):
    """How logits become choices and weights: scoring "softmax" or "sigmoid"; balance
    fp32 [experts], added to the scores for the choice alone, or None; `groups` groups
    of consecutive experts of which `topk_groups` (all if None) are kept, graded by
    group_score "max" (their best) or "top2" (the sum of their two best); weights
    divided by their sum if `renormalize`, then multiplied by `scale`."""
    experts: int
    topk: int
    scoring: str = "softmax"
    balance: Optional["object"] = None
    groups: int = 1
    topk_groups: Optional[int] = None
    group_score: str = "max"
    renormalize: bool = True
    scale: float = 1.0

    def _tensors(self):
        if self.balance is None:
            return []
        import torch
        return [_tensor(self.balance, "balance", torch.float32, (self.experts,))]

    def _make(self):
        if self.scoring not in ("softmax", "sigmoid"):
            _refuse(f"scoring {self.scoring!r} is not softmax or sigmoid")
        if self.group_score not in ("max", "top2"):
            _refuse(f"group_score {self.group_score!r} is not max or top2")
        topk_groups = self.groups if self.topk_groups is None else self.topk_groups
        return _RouteRule(_ptr(self.balance), _int32(self.experts, "experts"), _int32(self.topk, "topk"),
                          ROUTE_SOFTMAX if self.scoring == "softmax" else ROUTE_SIGMOID,
                          _int32(self.groups, "groups"), _int32(topk_groups, "topk_groups"),
                          GROUP_MAX if self.group_score == "max" else GROUP_TOP2, int(bool(self.renormalize)),
                          float(self.scale))


def _choices(rule: Exl3RouteRule, t: int, topk_ids, topk_weights, device: int, stream):
    """The tensors that take the choices (new ones where none are given), checked."""
    int32, float32 = _number_types
    if rule.balance is not None and rule.balance.get_device() != device:
        _refuse("the balance is on another device than the operands")
    shape = (t, rule.topk)
    if topk_ids is None or topk_weights is None:
        import torch
    if topk_ids is None:
        topk_ids = _new(torch.empty, shape, int32, device, stream)
    elif _tensor(topk_ids, "topk_ids", int32, shape).get_device() != device:
        _refuse("topk_ids is on another device than the operands")
    if topk_weights is None:
        topk_weights = _new(torch.empty, shape, float32, device, stream)
    elif _tensor(topk_weights, "topk_weights", float32, shape).get_device() != device:
        _refuse("topk_weights is on another device than the operands")
    return topk_ids, topk_weights


def exl3_route_topk(logits, rule: Exl3RouteRule, topk_ids=None, topk_weights=None, stream=None):
    """Choices int32 [t, topk] and weights fp32 [t, topk] of tokens with the logits
    fp16 or fp32 [t, experts]."""
    rule._now()
    t, _, ldl = _matrix(logits, "logits", None, rule.experts)
    device, on = _place(logits, "logits", stream)
    topk_ids, topk_weights = _choices(rule, t, topk_ids, topk_weights, device, stream)
    _check(lib().exl3_route_topk(rule._ref, logits.data_ptr(), _f16_f32(logits, "logits"), t, ldl,
                                 topk_ids.data_ptr(), topk_weights.data_ptr(), on), "exl3_route_topk")
    return topk_ids, topk_weights


def exl3_router_linear_workspace_size(router: Exl3Router, t: int) -> int:
    router._now()
    return int(lib().exl3_router_linear_workspace_size(router._ref, int(t)))


def _logits(out, t: int, router: Exl3Router, device: int):
    """Row stride of the logits' tensor, checked."""
    if _f16_f32(out, "the logits' tensor") != EXL3_F32:
        _refuse(f"the logits' tensor is {out.dtype}, not fp32")
    if out.get_device() != device:
        _refuse("the logits' tensor is on another device than x")
    return _matrix(out, "the logits' tensor", t, router.experts)[2]


def _router_rows(x, router: Exl3Router, stream):
    hidden = router._now().hidden
    t, ldx = _f16_rows(x, hidden)
    device, on = _place(x, "x", stream)
    if router.weight.get_device() != device:
        _refuse("x and the router are on different devices")
    return t, ldx, device, on


def exl3_router_linear(x, router: Exl3Router, out=None, workspace=None, stream=None):
    """Logits fp32 [t, experts] of fp16 rows x [t, hidden].  A workspace passed in has to
    be zero-filled before its first use and is then left to the router's functions."""
    t, ldx, device, on = _router_rows(x, router, stream)
    if out is None:
        import torch
        out = _new(torch.empty, (t, router.experts), torch.float32, device, stream)
    ldl = _logits(out, t, router, device)
    ws, nws, _keep = _scratch(workspace, True, lib().exl3_router_linear_workspace_size, (router._ref, t), device,
                              stream)
    _check(lib().exl3_router_linear(router._ref, x.data_ptr(), t, ldx, out.data_ptr(), ldl, ws, nws, on),
           "exl3_router_linear")
    return out


def exl3_router_workspace_size(router: Exl3Router, t: int, logits: bool = True) -> int:
    """Bytes exl3_router needs; logits: whether the call gets a tensor for them."""
    router._now()
    return int(lib().exl3_router_workspace_size(router._ref, int(t), int(logits)))


def exl3_router(x, router: Exl3Router, rule: Exl3RouteRule, logits=None, topk_ids=None, topk_weights=None,
                workspace=None, stream=None):
    """Choices int32 [t, topk] and weights fp32 [t, topk] of fp16 rows x [t, hidden]:
    a router's linear and exl3_route_topk of its logits in one call.  logits fp32
    [t, experts] receives the logits if given; they are exl3_router_linear's to rounding.
    The workspace is exl3_router_linear's."""
    rule._now()
    t, ldx, device, on = _router_rows(x, router, stream)
    ldl, ptr = (0, 0) if logits is None else (_logits(logits, t, router, device), logits.data_ptr())
    topk_ids, topk_weights = _choices(rule, t, topk_ids, topk_weights, device, stream)
    ws, nws, _keep = _scratch(workspace, True, lib().exl3_router_workspace_size,
                              (router._ref, t, logits is not None), device, stream)
    _check(lib().exl3_router(router._ref, rule._ref, x.data_ptr(), t, ldx, ptr, ldl, topk_ids.data_ptr(),
                             topk_weights.data_ptr(), ws, nws, on), "exl3_router")
    return topk_ids, topk_weights


# ---------------------------------------------------------------------------
# Low-rank adapters
# ---------------------------------------------------------------------------
@dataclass(frozen=True)
class Exl3Lora(_Record):
    """Adapters of one projection: a fp16 [adapters, rank, k], b fp16 [adapters, n,
    rank], scales fp32 [adapters] or None (1), ranks int32 [adapters] (each adapter's own
    rank) or None."""
    a: "object"
    b: "object"
    scales: Optional["object"] = None
    ranks: Optional["object"] = None

    def _tensors(self):
        import torch
        parts = [_tensor(self.a, "a", torch.float16, (None, None, None))]
        count, rank, _ = self.a.shape
        parts.append(_tensor(self.b, "b", torch.float16, (count, None, rank)))
        if self.scales is not None:
            parts.append(_tensor(self.scales, "scales", torch.float32, (count,)))
        if self.ranks is not None:
            parts.append(_tensor(self.ranks, "ranks", torch.int32, (count,)))
        return parts

    def _make(self):
        return _LoraStack(_ptr(self.a), _ptr(self.b), _ptr(self.scales), _ptr(self.ranks),
                          _int32(self.adapters, "adapters"), _int32(self.rank, "rank"), self.k, self.n)

    @property
    def adapters(self) -> int:
        return int(self.a.shape[0])

    @property
    def rank(self) -> int:
        return int(self.a.shape[1])

    @property
    def k(self) -> int:
        return int(self.a.shape[2])

    @property
    def n(self) -> int:
        return int(self.b.shape[1])


def exl3_lora_workspace_size(lora: Exl3Lora, m: int) -> int:
    lora._now()
    return int(lib().exl3_lora_workspace_size(lora._ref, int(m)))


def exl3_lora(x, lora: Exl3Lora, rows, base=None, out_dtype=None, out=None, workspace=None, stream=None):
    """y [m, n] = base + scale_a B_a (A_a x) with a = rows[i] (int32 [m]) for row i;
    rows whose value is no adapter (-1) get base, or zeros without one.  x fp16 [m, k],
    base and y of one type, fp16 or fp32.  `out=base` adds in place."""
    record = lora._now()
    m, ldx = _f16_rows(x, record.k)
    device, on = _place(x, "x", stream)
    if lora.a.get_device() != device:
        _refuse("x and the adapters are on different devices")
    if _tensor(rows, "rows", _number_types[0], (m,)).get_device() != device:
        _refuse("rows is on another device than x")
    if out_dtype is None and base is not None:
        out_dtype = base.dtype
    out, ldy, ydt = _product_out(out, out_dtype, m, record.n, device, None, stream)
    ldb, ptr = 0, 0
    if base is not None:
        if base.dtype != out.dtype:
            _refuse(f"base is {base.dtype}, the output {out.dtype}")
        if base.get_device() != device:
            _refuse("base is on another device than x")
        ldb, ptr = _matrix(base, "base", m, record.n)[2], base.data_ptr()
    ws, nws, _keep = _scratch(workspace, False, lib().exl3_lora_workspace_size, (lora._ref, m), device, stream)
    _check(lib().exl3_lora(lora._ref, x.data_ptr(), m, ldx, rows.data_ptr(), ptr, ldb, out.data_ptr(), ldy, ydt, ws,
                           nws, on), "exl3_lora")
    return out
