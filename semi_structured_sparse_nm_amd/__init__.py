"""MI355X (gfx950) N:M semi-structured sparse weight x dense activation product.

Thin Python binding of libnmsparse.so (C ABI in include/nm_sparse.h): it only
marshals torch tensors to device pointers and the current HIP stream; every
step of the computation runs in the library's HIP kernels.  PyTorch provides
device memory and streams.  There is no CPU fallback: without the built
library every call raises.

    p = pack(W, N, M)                      # W: [R, K] int8 / float16 / bfloat16 on the GPU
    Y = spmm(p, X, bias=None, scale=None, out_dtype=None)   # X: [K, T]  ->  Y: [R, T]

    # the gated feed-forward block on two packed weights, and its gradients
    H = glu(pg, pu, Xt, act="silu", pre=None)               # Xt: [T, K]  ->  H: [T, R]
    dX, dWg, dWu = glu_backward(pg, pu, Xt, pre, dH, act="silu")

    # microscaled 4-bit weights: their product and gated block
    m = mx_quantize(W)                                      # W: [R, K] float16 / bfloat16 / float32
    Y = mx_linear(m, Xt)                                    # Xt: [T, K]  ->  Y: [T, R]
    H = mx_glu(mg, mu, Xt, act="silu")

Operation: paper "Realizable N:M Sparse Transformer Inference via
Search-Kernel Co-Design" (arXiv 2607.12505) -- Sec. 2.1 N:M constraint,
Sec. 4.2 packed windows and micro-dense execution.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnmsparse.so")

NM_OK, NM_EINVAL, NM_EUNSUPPORTED, NM_EHIP = 0, 1, 2, 3
NM_I8, NM_F16, NM_BF16, NM_I32, NM_F32 = 0, 1, 2, 3, 4
FORMAT_VERSION = 1

_TORCH_TO_NM = {torch.int8: NM_I8, torch.float16: NM_F16, torch.bfloat16: NM_BF16,
                torch.int32: NM_I32, torch.float32: NM_F32}
_NM_TO_TORCH = {v: k for k, v in _TORCH_TO_NM.items()}


class NmPacked(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("K", ctypes.c_int64), ("N", ctypes.c_int32),
                ("M", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("format_version", ctypes.c_uint32), ("values", ctypes.c_void_p),
                ("values_bytes", ctypes.c_size_t), ("meta", ctypes.c_void_p),
                ("meta_bytes", ctypes.c_size_t)]


class NmHybrid(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("K", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("format_version", ctypes.c_uint32),
                ("values", ctypes.c_void_p), ("values_bytes", ctypes.c_size_t),
                ("meta", ctypes.c_void_p), ("meta_bytes", ctypes.c_size_t),
                ("codes", ctypes.c_void_p), ("codes_bytes", ctypes.c_size_t),
                ("res_ptr", ctypes.c_void_p), ("res_ptr_bytes", ctypes.c_size_t),
                ("res_ent", ctypes.c_void_p), ("res_ent_bytes", ctypes.c_size_t),
                ("n_fill", ctypes.c_int64), ("n_res", ctypes.c_int64)]


class NmMx(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("K", ctypes.c_int64), ("format_version", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("codes", ctypes.c_void_p), ("codes_bytes", ctypes.c_size_t),
                ("scales", ctypes.c_void_p), ("scales_bytes", ctypes.c_size_t)]


HYBRID_BUFFERS = ("values", "meta", "codes", "res_ptr", "res_ent")


class NmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)}")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libnmsparse.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m semi_structured_sparse_nm_amd._build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        PP = ctypes.POINTER(NmPacked)
        L.nm_pack_size.argtypes = [I64, I64, I32, I32, I32, ctypes.POINTER(SZ), ctypes.POINTER(SZ)]
        L.nm_pack.argtypes = [P, I64, PP, P]
        L.nm_spmm_workspace_size.argtypes = [PP, I64, I32, ctypes.POINTER(SZ)]
        L.nm_spmm_tk_workspace_size.argtypes = [PP, I64, I32, ctypes.POINTER(SZ)]
        L.nm_spmm.argtypes = [PP, P, I64, I64, P, I64, I32, P, P, P, SZ, P]
        L.nm_status_str.argtypes = [ctypes.c_int]
        L.nm_status_str.restype = ctypes.c_char_p
        L.nm_spmm_variant.argtypes = [PP, I64, I32]
        L.nm_spmm_variant.restype = ctypes.c_char_p
        L.nm_spmm_ksplit.argtypes = [PP, I64, I32, I32]
        L.nm_spmm_ksplit.restype = I32
        L.nm_spmm_variant_act.argtypes = [PP, I64, I32, I32]
        L.nm_spmm_variant_act.restype = ctypes.c_char_p
        L.nm_spmm_act.argtypes = [PP, P, I64, I64, P, I64, I32, P, P, I32, ctypes.c_float, P, SZ, P]
        L.nm_spmm_act.restype = ctypes.c_int
        L.nm_spmm_tk.argtypes = [PP, P, I64, I64, P, I64, I32, P, P, I32, ctypes.c_float, P, SZ, P]
        L.nm_spmm_tk.restype = ctypes.c_int
        L.nm_spmm_variant_tk.argtypes = [PP, I64, I32, I32]
        L.nm_spmm_variant_tk.restype = ctypes.c_char_p
        L.nm_spmm_noalloc.argtypes = [PP, P, I64, I64, P, I64, I32, P, P, I32, ctypes.c_float, P]
        L.nm_spmm_noalloc.restype = ctypes.c_int
        L.nm_spmm_noalloc_max_bytes.argtypes = []
        L.nm_spmm_noalloc_max_bytes.restype = SZ
        HP = ctypes.POINTER(NmHybrid)
        L.nm_hybrid_pack_size.argtypes = [P, I64, I64, I64, I32, HP]
        L.nm_hybrid_pack.argtypes = [P, I64, HP]
        L.nm_hybrid_spmm.argtypes = [HP, P, I64, I64, P, I64, I32, P, I32, P]
        L.nm_glu_workspace_size.argtypes = [PP, PP, P, I64, I64, ctypes.POINTER(SZ)]
        L.nm_glu.argtypes = [PP, PP, P, I64, I64, P, I64, I32, P, P, I64, P, SZ, P]
        L.nm_glu_kept.argtypes = [PP, PP, P, I64, I64, P, I64, I32, P, P, I64, I32, P, SZ, P]
        L.nm_glu_backward_workspace_size.argtypes = [PP, PP, I64, ctypes.POINTER(SZ)]
        L.nm_glu_backward.argtypes = [PP, PP, P, I64, I64, P, P, I64, P, I64, I32, P, I64, P, P, I64, P, SZ, P]
        L.nm_glu_backward_kept.argtypes = [PP, PP, P, I64, I64, P, P, I64, I32, P, I64, I32, P, I64, P, P, I64, P, SZ,
                                           P]
        MP = ctypes.POINTER(NmMx)
        L.nm_mx_size.argtypes = [I64, I64, ctypes.POINTER(SZ), ctypes.POINTER(SZ)]
        L.nm_mx_quantize.argtypes = [P, I64, I32, MP, P]
        L.nm_mx_dequantize.argtypes = [MP, P, I64, I32, P]
        L.nm_mx_workspace_size.argtypes = [MP, MP, I64, I32, ctypes.POINTER(SZ)]
        L.nm_mx_linear.argtypes = [MP, MP, P, I64, I32, I64, P, I64, I32, P, I32, P, SZ, P]
        L.nm_mx_glu.argtypes = [MP, MP, MP, P, I64, I32, I64, P, I64, I32, I32, P, SZ, P]
        for f in ("nm_pack_size", "nm_pack", "nm_spmm_workspace_size", "nm_spmm", "nm_hybrid_pack_size",
                  "nm_hybrid_pack", "nm_hybrid_spmm", "nm_glu_workspace_size", "nm_glu", "nm_glu_kept",
                  "nm_glu_backward_workspace_size", "nm_glu_backward", "nm_glu_backward_kept", "nm_mx_size", "nm_mx_quantize",
                  "nm_mx_dequantize", "nm_mx_workspace_size", "nm_mx_linear", "nm_mx_glu"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def status_str(s: int) -> str:
    return lib().nm_status_str(int(s)).decode()


def _check(st: int, what: str):
    if st != NM_OK:
        raise NmError(st, what)


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def pack_size(rows: int, K: int, N: int, M: int, dtype: int):
    vb, mb = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().nm_pack_size(rows, K, N, M, dtype, ctypes.byref(vb), ctypes.byref(mb)),
           "nm_pack_size")
    return vb.value, mb.value


def _fields_of(p) -> dict:
    """What a copy or a pickle of p holds: not its cached C descriptor."""
    return {k: v for k, v in p.__dict__.items() if k != "_c_desc"}


@dataclass
class Packed:
    """Packed N:M weights on the GPU (two uint8 device buffers + shape)."""
    rows: int
    K: int
    N: int
    M: int
    dtype: int
    values: torch.Tensor
    meta: torch.Tensor | None
    format_version: int = FORMAT_VERSION

    def desc(self) -> NmPacked:
        d = NmPacked()
        d.rows, d.K, d.N, d.M, d.dtype = self.rows, self.K, self.N, self.M, self.dtype
        d.format_version = self.format_version
        d.values, d.values_bytes = self.values.data_ptr(), self.values.numel()
        if self.meta is not None:
            d.meta, d.meta_bytes = self.meta.data_ptr(), self.meta.numel()
        else:
            d.meta, d.meta_bytes = None, 0
        return d

    def __getstate__(self):
        return _fields_of(self)

    @property
    def torch_dtype(self):
        return _NM_TO_TORCH[self.dtype]


def pack(W: torch.Tensor, N: int, M: int) -> Packed:
    """nm_pack: keep the N largest-|w| of every M consecutive K-elements of each row."""
    if W.dim() != 2 or W.stride(1) != 1:
        raise ValueError("W must be a 2-D tensor with unit stride along K")
    dt = _TORCH_TO_NM.get(W.dtype)
    if dt not in (NM_I8, NM_F16, NM_BF16):
        raise TypeError(f"unsupported weight dtype {W.dtype}")
    if W.device.type != "cuda":
        raise ValueError(f"W is on {W.device}, not on a GPU")
    R, K = W.shape
    vb, mb = pack_size(R, K, N, M, dt)
    values = torch.empty(vb, dtype=torch.uint8, device=W.device)
    meta = torch.empty(mb, dtype=torch.uint8, device=W.device) if mb else None
    p = Packed(R, K, N, M, dt, values, meta, 0)
    d = p.desc()
    _check(lib().nm_pack(W.data_ptr(), W.stride(0), ctypes.byref(d), _stream(W.device)), "nm_pack")
    p.format_version = d.format_version
    return p


def _check_operands(p: Packed, X: torch.Tensor, out: torch.Tensor, out_dtype: torch.dtype,
                    bias: torch.Tensor | None, scale: torch.Tensor | None,
                    workspace: torch.Tensor | None) -> None:
    """Type, length and device checks of one product's operands, before any
    launch: the kernels size every buffer range from the requested dtypes and
    R, so a mismatch here would read or write past a tensor's end."""
    wdt = p.torch_dtype
    if X.dtype != wdt:
        raise TypeError(f"activation dtype {X.dtype} does not match the weight dtype {wdt}")
    if out.dtype != out_dtype:
        raise TypeError(f"out has dtype {out.dtype}, the call asks for {out_dtype}")
    if _TORCH_TO_NM.get(out_dtype) is None:
        raise TypeError(f"unsupported output dtype {out_dtype}")
    want_bias = torch.int32 if p.dtype == NM_I8 else torch.float32
    for name, t, dt in (("bias", bias, want_bias), ("scale", scale, torch.float32)):
        if t is None:
            continue
        if t.dtype != dt:
            raise TypeError(f"{name} must be {dt} for {wdt} weights, got {t.dtype}")
        if t.dim() != 1 or t.numel() != p.rows or (t.numel() > 1 and t.stride(0) != 1):
            raise ValueError(f"{name} must be a contiguous vector of length R={p.rows}, got {tuple(t.shape)}")
    if out_dtype == torch.int8 and scale is None:
        raise ValueError("int8 output needs a float32 scale of length R")
    dev = p.values.device
    if dev.type != "cuda":
        raise ValueError(f"the packed weight is on {dev}, not on a GPU")
    for name, t in (("X", X), ("out", out), ("bias", bias), ("scale", scale), ("workspace", workspace),
                    ("meta", p.meta)):
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the packed weight on {dev}")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")


def default_out_dtype(wdt: int) -> torch.dtype:
    return {NM_I8: torch.int32, NM_F16: torch.float16, NM_BF16: torch.bfloat16}[wdt]


def workspace_size(p: Packed, T: int, out_dtype: torch.dtype) -> int:
    n = ctypes.c_size_t()
    d = p.desc()
    _check(lib().nm_spmm_workspace_size(ctypes.byref(d), T, _TORCH_TO_NM[out_dtype], ctypes.byref(n)),
           "nm_spmm_workspace_size")
    return n.value


def workspace_size_tk(p: Packed, T: int, out_dtype: torch.dtype) -> int:
    """nm_spmm_tk_workspace_size: the workspace linear() needs."""
    n = ctypes.c_size_t()
    d = p.desc()
    _check(lib().nm_spmm_tk_workspace_size(ctypes.byref(d), T, _TORCH_TO_NM[out_dtype], ctypes.byref(n)),
           "nm_spmm_tk_workspace_size")
    return n.value


ACTS = {"none": 0, "gelu": 1}


def variant(p: Packed, T: int, out_dtype: torch.dtype, act: str = "none") -> str:
    d = p.desc()
    return lib().nm_spmm_variant_act(ctypes.byref(d), T, _TORCH_TO_NM[out_dtype], ACTS[act]).decode()


def variant_tk(p: Packed, T: int, out_dtype: torch.dtype, act: str = "none") -> str:
    d = p.desc()
    return lib().nm_spmm_variant_tk(ctypes.byref(d), T, _TORCH_TO_NM[out_dtype], ACTS[act]).decode()


def ksplit(p: Packed, T: int, out_dtype: torch.dtype, act: str = "none") -> int:
    """K slices (workgroup-level split of K) nm_spmm would use; 1 = none."""
    d = p.desc()
    return int(lib().nm_spmm_ksplit(ctypes.byref(d), T, _TORCH_TO_NM[out_dtype], ACTS[act]))


def spmm(p: Packed, X: torch.Tensor, bias: torch.Tensor | None = None,
         scale: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
         out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
         act: str = "none", out_scale: float = 1.0) -> torch.Tensor:
    """nm_spmm (nm_spmm_act with `act` != "none"): Y[R, T] =
    epilogue((mask . W) @ X) with X [K, T] (tokens contiguous); act "gelu"
    fuses GELU into the epilogue (int8 output: out_scale requantises it)."""
    if X.dim() != 2 or X.stride(1) != 1:
        raise ValueError("X must be a 2-D tensor with unit stride along T")
    if X.shape[0] != p.K:
        raise ValueError(f"X has {X.shape[0]} rows, the weight has K={p.K}")
    T = X.shape[1]
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else default_out_dtype(p.dtype)
    if out is None:
        out = torch.empty((p.rows, T), dtype=out_dtype, device=X.device)
    if out.dim() != 2 or out.stride(1) != 1 or tuple(out.shape) != (p.rows, T):
        raise ValueError("out must be [R, T] with unit stride along T")
    _check_operands(p, X, out, out_dtype, bias, scale, workspace)
    need = workspace_size(p, T, out_dtype)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    d = p.desc()
    st = lib().nm_spmm_act(ctypes.byref(d), X.data_ptr(), X.stride(0), T, out.data_ptr(), out.stride(0),
                           _TORCH_TO_NM[out_dtype], None if bias is None else bias.data_ptr(),
                           None if scale is None else scale.data_ptr(), ACTS[act], float(out_scale),
                           None if workspace is None else workspace.data_ptr(),
                           0 if workspace is None else workspace.numel() * workspace.element_size(),
                           _stream(X.device))
    _check(st, "nm_spmm_act" if act != "none" else "nm_spmm")
    return out


def spmm_noalloc(p: Packed, X: torch.Tensor, out: torch.Tensor, bias: torch.Tensor | None = None,
                 scale: torch.Tensor | None = None, act: str = "none", out_scale: float = 1.0) -> torch.Tensor:
    """nm_spmm_noalloc: spmm() into a caller-given `out` with no allocation
    at all (the library's per-device scratch replaces the workspace), for
    code that cannot allocate, such as HIP graph capture."""
    if X.dim() != 2 or X.stride(1) != 1 or X.shape[0] != p.K:
        raise ValueError("X must be [K, T] with unit stride along T")
    T = X.shape[1]
    if out.dim() != 2 or out.stride(1) != 1 or tuple(out.shape) != (p.rows, T):
        raise ValueError("out must be [R, T] with unit stride along T")
    _check_operands(p, X, out, out.dtype, bias, scale, None)
    d = p.desc()
    st = lib().nm_spmm_noalloc(ctypes.byref(d), X.data_ptr(), X.stride(0), T, out.data_ptr(), out.stride(0),
                               _TORCH_TO_NM[out.dtype], None if bias is None else bias.data_ptr(),
                               None if scale is None else scale.data_ptr(), ACTS[act], float(out_scale),
                               _stream(X.device))
    _check(st, "nm_spmm_noalloc")
    return out


def noalloc_max_bytes() -> int:
    return int(lib().nm_spmm_noalloc_max_bytes())


def linear(p: Packed, Xt: torch.Tensor, bias: torch.Tensor | None = None,
           scale: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
           out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
           act: str = "none", out_scale: float = 1.0) -> torch.Tensor:
    """nm_spmm_tk, the PyTorch-linear layout: Yt[T, R] = epilogue(Xt @ (mask . W)^T)
    with Xt [T, K] (K contiguous), as torch.nn.functional.linear takes it."""
    if Xt.dim() != 2 or Xt.stride(1) != 1:
        raise ValueError("Xt must be a 2-D tensor with unit stride along K")
    if Xt.shape[1] != p.K:
        raise ValueError(f"Xt has {Xt.shape[1]} columns, the weight has K={p.K}")
    T = Xt.shape[0]
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else default_out_dtype(p.dtype)
    if out is None:
        out = torch.empty((T, p.rows), dtype=out_dtype, device=Xt.device)
    if out.dim() != 2 or out.stride(1) != 1 or tuple(out.shape) != (T, p.rows):
        raise ValueError("out must be [T, R] with unit stride along R")
    _check_operands(p, Xt, out, out_dtype, bias, scale, workspace)
    need = workspace_size_tk(p, T, out_dtype)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=Xt.device)
    d = p.desc()
    st = lib().nm_spmm_tk(ctypes.byref(d), Xt.data_ptr(), Xt.stride(0), T, out.data_ptr(), out.stride(0),
                          _TORCH_TO_NM[out_dtype], None if bias is None else bias.data_ptr(),
                          None if scale is None else scale.data_ptr(), ACTS[act], float(out_scale),
                          None if workspace is None else workspace.data_ptr(),
                          0 if workspace is None else workspace.numel() * workspace.element_size(),
                          _stream(Xt.device))
    _check(st, "nm_spmm_tk")
    return out


# ---------------------------------------------------------------- three-layer format
@dataclass
class Hybrid:
    """A weight in the three-layer format (Sparse-TC 2:4, slot filling with
    PDD codes, CSR residual) as five uint8 buffers on one device."""
    rows: int
    K: int
    dtype: int
    values: torch.Tensor
    meta: torch.Tensor
    codes: torch.Tensor
    res_ptr: torch.Tensor
    res_ent: torch.Tensor | None
    n_fill: int
    n_res: int
    format_version: int = FORMAT_VERSION

    def desc(self) -> NmHybrid:
        d = NmHybrid()
        d.rows, d.K, d.dtype, d.format_version = self.rows, self.K, self.dtype, self.format_version
        d.n_fill, d.n_res = self.n_fill, self.n_res
        for name in HYBRID_BUFFERS:
            t = getattr(self, name)
            setattr(d, name, None if t is None else t.data_ptr())
            setattr(d, name + "_bytes", 0 if t is None else t.numel())
        return d

    @property
    def torch_dtype(self):
        return _NM_TO_TORCH[self.dtype]

    def nbytes(self) -> int:
        return sum(0 if getattr(self, n) is None else getattr(self, n).numel() for n in HYBRID_BUFFERS)


def hybrid_pack_host(W: torch.Tensor) -> Hybrid:
    """nm_hybrid_pack on the host: W (float16 / bfloat16, any device) is
    copied to host memory and packed there; the buffers are CPU tensors."""
    if W.dim() != 2:
        raise ValueError("W must be 2-D")
    dt = _TORCH_TO_NM.get(W.dtype)
    if dt not in (NM_F16, NM_BF16):
        raise TypeError(f"the three-layer format takes float16 / bfloat16 weights, not {W.dtype}")
    Wh = W.detach().to("cpu").contiguous()
    R, K = Wh.shape
    d = NmHybrid()
    _check(lib().nm_hybrid_pack_size(Wh.data_ptr(), K, R, K, dt, ctypes.byref(d)), "nm_hybrid_pack_size")
    bufs = {n: torch.empty(getattr(d, n + "_bytes"), dtype=torch.uint8) for n in HYBRID_BUFFERS}
    h = Hybrid(R, K, dt, bufs["values"], bufs["meta"], bufs["codes"], bufs["res_ptr"],
               bufs["res_ent"] if d.n_res else None, d.n_fill, d.n_res, 0)
    dd = h.desc()
    _check(lib().nm_hybrid_pack(Wh.data_ptr(), K, ctypes.byref(dd)), "nm_hybrid_pack")
    h.format_version = dd.format_version
    return h


def pack_hybrid(W: torch.Tensor, device=None) -> Hybrid:
    """Pack W into the three-layer format (host packer, offline) and place the
    buffers on `device` (default: W's device, which must be a GPU)."""
    device = torch.device(device) if device is not None else W.device
    if device.type != "cuda":
        raise ValueError(f"target device {device} is not a GPU")
    h = hybrid_pack_host(W)
    for n in HYBRID_BUFFERS:
        t = getattr(h, n)
        if t is not None:
            setattr(h, n, t.to(device))
    return h


def spmm_hybrid(h: Hybrid, X: torch.Tensor, bias: torch.Tensor | None = None,
                out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                act: str = "none") -> torch.Tensor:
    """nm_hybrid_spmm: Y[R, T] = epilogue(W @ X) for a three-layer weight,
    X [K, T] (tokens contiguous)."""
    if X.dim() != 2 or X.stride(1) != 1 or X.shape[0] != h.K:
        raise ValueError("X must be [K, T] with unit stride along T")
    if X.dtype != h.torch_dtype:
        raise TypeError(f"X is {X.dtype}, the weight is {h.torch_dtype}")
    T = X.shape[1]
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else h.torch_dtype
    if out is None:
        out = torch.empty((h.rows, T), dtype=out_dtype, device=X.device)
    if out.dim() != 2 or out.stride(1) != 1 or tuple(out.shape) != (h.rows, T) or out.dtype != out_dtype:
        raise ValueError("out must be [R, T] of out_dtype with unit stride along T")
    tensors = [X, out] + [getattr(h, n) for n in HYBRID_BUFFERS if getattr(h, n) is not None]
    if bias is not None:
        if bias.dtype != torch.float32 or bias.numel() != h.rows or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous float32 [R] tensor")
        tensors.append(bias)
    for t in tensors:
        if t.device != X.device:
            raise ValueError(f"operand on {t.device}, X on {X.device}")
    d = h.desc()
    st = lib().nm_hybrid_spmm(ctypes.byref(d), X.data_ptr(), X.stride(0), T, out.data_ptr(), out.stride(0),
                              _TORCH_TO_NM[out_dtype], None if bias is None else bias.data_ptr(),
                              ACTS[act], _stream(X.device))
    _check(st, "nm_hybrid_spmm")
    return out


# ---------------------------------------------------------------- gated feed-forward block
GLU_ACTS = {"gelu": 1, "silu": 2}

# The smallest of the calls below take a few microseconds on the GPU, so their
# host side is kept short: descriptors and workspace sizes are remembered per
# weight and shape, devices compared by index, streams taken as raw handles.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_ws_sizes: dict = {}
# NM_FFN_TILE as it is now, or None; from the mapping behind os.environ (50 ns
# against 550, in calls of 9 us)
_forced_path = functools.partial(os.environ._data.get, os.environ.encodekey("NM_FFN_TILE"))


def _descriptor(p):
    """byref of p's C descriptor, built again whenever a field changed."""
    if type(p) is Packed:
        v, m = p.values, p.meta
        key = (v.data_ptr(), v.numel(), p.rows, p.K, p.N, p.M, p.dtype, p.format_version)
    else:
        v, m = p.codes, p.scales
        key = (v.data_ptr(), v.numel(), p.rows, p.K, p.format_version)
    if m is not None:
        key += (m.data_ptr(), m.numel())
    c = p.__dict__.get("_c_desc")
    if c is None or c[0] != key:
        d = p.desc()
        c = p.__dict__["_c_desc"] = (key, d, ctypes.byref(d))
    return c[2]


def _sized(f, what: str, key: tuple, *args) -> int:
    """A workspace size of the library, remembered by shape and device; asked
    for again where the environment forces a path, which decides it too."""
    forced = _forced_path() is not None
    n = None if forced else _ws_sizes.get(key)
    if n is None:
        b = ctypes.c_size_t()
        with torch.cuda.device(key[-1]):                  # the plan depends on the device
            _check(f(*args, ctypes.byref(b)), what)
        n = b.value
        if not forced:
            if len(_ws_sizes) > 4096:
                _ws_sizes.clear()
            _ws_sizes[key] = n
    return n


def _one_gpu(names: str, t0: torch.Tensor, *rest) -> int:
    """The index of the one GPU t0 and the other tensors live on (None ones are
    skipped); names: of all of them, for the error."""
    i = t0.get_device()
    if i < 0:
        raise ValueError(f"{names.split(', ')[0]} is on {t0.device}, not on a GPU")
    for t in rest:
        if t is not None and t.get_device() != i:
            first, *others = names.split(", ")
            name = others[next(k for k, r in enumerate(rest) if r is t)]
            raise ValueError(f"{name} is on {t.device}, {first} on {t0.device}")
    return i


def _row_pitch(name: str, t: torch.Tensor, rows: int, cols: int) -> int:
    """Elements between the rows of a [rows, cols] tensor with unit stride
    along its columns, as the library takes them (rows may not overlap)."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {tuple(t.shape)}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name} must have unit stride along its second dimension")
    if rows == 1:
        return cols
    if s0 < cols:
        raise ValueError(f"{name} has overlapping rows (stride {s0} for {cols} columns)")
    return s0


def _workspace(workspace: torch.Tensor | None, need: int, dev: int):
    """(tensor, pointer, bytes): the caller's workspace where it is large
    enough, else a new one; the tensor is held by the caller of the library."""
    if workspace is not None:
        if workspace.get_device() != dev:
            raise ValueError(f"workspace is on {workspace.device}, the operands on cuda:{dev}")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        n = workspace.numel() * workspace.element_size()
        if n >= need:
            return workspace, workspace.data_ptr(), n
    if not need:
        return None, None, 0
    workspace = torch.empty(need, dtype=torch.uint8, device=f"cuda:{dev}")
    return workspace, workspace.data_ptr(), need


def _glu_act(act: str) -> int:
    a = GLU_ACTS.get(act)
    if a is None:
        raise ValueError(f"act must be one of {sorted(GLU_ACTS)}, got {act!r}")
    return a


def _check_dtype(name: str, t: torch.Tensor, want: torch.dtype) -> None:
    if t.dtype != want:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {want}")


def _call(dev: int, f, what: str, *args) -> None:
    """One library call with the operands' device current and its current
    stream as the last argument."""
    if dev == _current_device():
        st = f(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = f(*args, _raw_stream(dev))
    if st != NM_OK:
        raise NmError(st, what)


def _glu_operands(gate: Packed, up: Packed, Xt: torch.Tensor):
    if gate.dtype not in (NM_F16, NM_BF16):
        raise TypeError(f"the gated block takes float16 / bfloat16 weights, not {gate.torch_dtype}")
    if (gate.rows, gate.K, gate.N, gate.M, gate.dtype) != (up.rows, up.K, up.N, up.M, up.dtype):
        f = next(f for f in ("rows", "K", "N", "M", "dtype") if getattr(gate, f) != getattr(up, f))
        raise ValueError(f"gate and up differ in {f}: {getattr(gate, f)} and {getattr(up, f)}")
    if Xt.dim() != 2:
        raise ValueError("Xt must be a 2-D tensor")
    T = Xt.shape[0]
    ldx = _row_pitch("Xt", Xt, T, gate.K)
    _check_dtype("Xt", Xt, gate.torch_dtype)
    return T, ldx


def _check_pre(pre: torch.Tensor, T: int, p: Packed):
    """(elements between pre's rows, its type)"""
    if pre.shape != (2, T, p.rows):
        raise ValueError(f"pre must be [2, {T}, {p.rows}], got {tuple(pre.shape)}")
    dt = _TORCH_TO_NM.get(pre.dtype)
    if dt != p.dtype and dt != NM_F32:
        raise TypeError(f"pre has dtype {pre.dtype}, expected {p.torch_dtype} or {torch.float32}")
    half, ld, s2 = pre.stride()
    if s2 != 1 and p.rows > 1:
        raise ValueError("pre must have unit stride along its last dimension")
    if T == 1:
        ld = p.rows
    elif ld < p.rows:
        raise ValueError(f"pre has overlapping rows (stride {ld} for {p.rows} columns)")
    # one half behind the other, or their rows in turn
    if half < (T - 1) * ld + p.rows and not (T > 1 and p.rows <= half <= ld - p.rows):
        raise ValueError("the two halves of pre overlap")
    return ld, dt


def _glu_key(what: str, p: Packed, T: int, rows, dev: int) -> tuple:
    return what, p.rows, p.K, p.N, p.M, p.dtype, T, rows, dev


def glu_workspace_size(gate: Packed, up: Packed, T: int) -> int:
    """nm_glu_workspace_size: bytes of workspace glu() may need for T rows of
    any stride and alignment."""
    n = ctypes.c_size_t()
    _check(lib().nm_glu_workspace_size(_descriptor(gate), _descriptor(up), None, 0, T, ctypes.byref(n)),
           "nm_glu_workspace_size")
    return n.value


def glu(gate: Packed, up: Packed, Xt: torch.Tensor, act: str = "silu", out: torch.Tensor | None = None,
        pre: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """nm_glu, the gated feed-forward block on two packed weights of one
    shape, N:M and dtype (float16 / bfloat16): H[T, R] = act(G) * U with
    G = Xt @ (mask . Wg)^T, U = Xt @ (mask . Wu)^T, Xt [T, K] (K contiguous).
    act: "silu" or "gelu".  pre: a [2, T, R] tensor that receives G and U,
    which glu_backward() takes, in float32 as they are summed or rounded to
    the weights' dtype (half the memory; the gradients' distance from unrounded
    ones grows from 1.4 to 1.8 times that of the output's rounding alone).  Not
    part of autograd's graph."""
    T, ldx = _glu_operands(gate, up, Xt)
    a = _glu_act(act)
    R = gate.rows
    if out is None:
        out = Xt.new_empty((T, R))
    else:
        _check_dtype("out", out, Xt.dtype)
    ldh = _row_pitch("out", out, T, R)
    ldp, pdt, g, u = 0, 0, None, None
    if pre is not None:
        ldp, pdt = _check_pre(pre, T, gate)
        g = pre.data_ptr()
        u = g + pre.stride(0) * pre.element_size()
    dev = _one_gpu("Xt, gate, gate meta, up, up meta, out, pre", Xt, gate.values, gate.meta, up.values, up.meta, out,
                   pre)
    L, dg, du = lib(), _descriptor(gate), _descriptor(up)
    x = Xt.data_ptr()
    need = _sized(L.nm_glu_workspace_size, "nm_glu_workspace_size", _glu_key("glu", gate, T, (x % 16, ldx), dev), dg,
                  du, x, ldx, T)
    ws, wp, wn = _workspace(workspace, need, dev)
    _call(dev, L.nm_glu_kept, "nm_glu", dg, du, x, ldx, T, out.data_ptr(), ldh, a, g, u, ldp, pdt, wp, wn)
    return out


def glu_backward_workspace_size(gate: Packed, up: Packed, T: int) -> int:
    """nm_glu_backward_workspace_size: bytes of workspace glu_backward() needs."""
    n = ctypes.c_size_t()
    _check(lib().nm_glu_backward_workspace_size(_descriptor(gate), _descriptor(up), T, ctypes.byref(n)),
           "nm_glu_backward_workspace_size")
    return n.value


def glu_backward(gate: Packed, up: Packed, Xt: torch.Tensor, pre: torch.Tensor, dH: torch.Tensor, act: str = "silu",
                 need_dx: bool = True, need_dw: bool = True, workspace: torch.Tensor | None = None):
    """nm_glu_backward: the gradients of glu() for a fixed mask, from dH
    [T, R] and the products glu() kept in `pre`.  Returns (dX [T, K],
    dWg [R, K], dWu [R, K]) in the weights' dtype; the weight gradients are
    dense and zero where the weight is pruned.  need_dx / need_dw = False
    leaves that part out (None in its place).  The gradients of G and U are
    operands of the weights' type: float16 ones beyond 65504 are infinite and
    below 2^-25 zero, so losses are scaled as for any float16 gradient.
    Neither call is part of autograd's graph."""
    T, ldx = _glu_operands(gate, up, Xt)
    a = _glu_act(act)
    if not need_dx and not need_dw:
        raise ValueError("glu_backward needs need_dx or need_dw")
    ldp, pdt = _check_pre(pre, T, gate)
    R, K = gate.rows, gate.K
    lddh = _row_pitch("dH", dH, T, R)
    _check_dtype("dH", dH, Xt.dtype)
    dev = _one_gpu("Xt, gate, gate meta, up, up meta, pre, dH", Xt, gate.values, gate.meta, up.values, up.meta, pre,
                   dH)
    L, dg, du = lib(), _descriptor(gate), _descriptor(up)
    need = _sized(L.nm_glu_backward_workspace_size, "nm_glu_backward_workspace_size",
                  _glu_key("glu_backward", gate, T, None, dev), dg, du, T)
    ws, wp, wn = _workspace(workspace, need, dev)
    dX = Xt.new_empty((T, K)) if need_dx else None
    dWg = Xt.new_empty((R, K)) if need_dw else None
    dWu = Xt.new_empty((R, K)) if need_dw else None
    g = pre.data_ptr()
    _call(dev, L.nm_glu_backward_kept, "nm_glu_backward", dg, du, Xt.data_ptr(), ldx, T, g,
          g + pre.stride(0) * pre.element_size(), ldp, pdt, dH.data_ptr(), lddh, a,
          dX.data_ptr() if need_dx else None, K, dWg.data_ptr() if need_dw else None,
          dWu.data_ptr() if need_dw else None, K, wp, wn)
    return dX, dWg, dWu


# ---------------------------------------------------------------- microscaled 4-bit format
@dataclass
class Mx:
    """rows x K values in the microscaled 4-bit format (E2M1 elements, one
    E8M0 scale for each block of 32 along K) as two uint8 device buffers."""
    rows: int
    K: int
    codes: torch.Tensor
    scales: torch.Tensor
    format_version: int = FORMAT_VERSION

    def desc(self) -> NmMx:
        return NmMx(self.rows, self.K, self.format_version, 0, self.codes.data_ptr(), self.codes.numel(),
                    self.scales.data_ptr(), self.scales.numel())

    def __getstate__(self):
        return _fields_of(self)

    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


_FLOATS = {torch.float16: NM_F16, torch.bfloat16: NM_BF16, torch.float32: NM_F32}


def _float_type(name: str, dt: torch.dtype) -> int:
    n = _FLOATS.get(dt)
    if n is None:
        raise TypeError(f"{name} must be float16, bfloat16 or float32, got {dt}")
    return n


def mx_size(rows: int, K: int):
    """nm_mx_size: bytes of an Mx's codes and scales."""
    n = _ws_sizes.get((rows, K))
    if n is None:
        c, s = ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().nm_mx_size(rows, K, ctypes.byref(c), ctypes.byref(s)), "nm_mx_size")
        if len(_ws_sizes) > 4096:
            _ws_sizes.clear()
        n = _ws_sizes[(rows, K)] = (c.value, s.value)
    return n


def mx_quantize(X: torch.Tensor) -> Mx:
    """nm_mx_quantize: X [rows, K] (float16, bfloat16 or float32) in the
    microscaled 4-bit format: blocks of 32 along K, scale
    2^(floor(log2(amax)) - 2), elements rounded half to even and saturated."""
    if X.dim() != 2:
        raise ValueError("X must be a 2-D tensor")
    xdt = _float_type("X", X.dtype)
    rows, K = X.shape
    ldx = _row_pitch("X", X, rows, K)
    dev = _one_gpu("X", X)
    c, s = mx_size(rows, K)
    m = Mx(rows, K, X.new_empty((c,), dtype=torch.uint8), X.new_empty((s,), dtype=torch.uint8))
    _call(dev, lib().nm_mx_quantize, "nm_mx_quantize", X.data_ptr(), ldx, xdt, _descriptor(m))
    return m


def mx_dequantize(m: Mx, out_dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """nm_mx_dequantize: the [rows, K] values m stands for."""
    if out is None:
        out = m.codes.new_empty((m.rows, m.K), dtype=out_dtype)
    ydt = _float_type("out", out.dtype)
    ld = _row_pitch("out", out, m.rows, m.K)
    dev = _one_gpu("codes, scales, out", m.codes, m.scales, out)
    _call(dev, lib().nm_mx_dequantize, "nm_mx_dequantize", _descriptor(m), out.data_ptr(), ld, ydt)
    return out


def mx_workspace_size(w: Mx, T: int, glu: bool = False) -> int:
    """nm_mx_workspace_size: bytes of workspace mx_linear() / mx_glu() may need
    for T tokens."""
    n = ctypes.c_size_t()
    _check(lib().nm_mx_workspace_size(_descriptor(w), None, T, int(glu), ctypes.byref(n)), "nm_mx_workspace_size")
    return n.value


def _mx_operands(w: Mx, X, out_dtype, out, workspace, glu: bool, names: str, *others):
    """Checks shared by mx_linear and mx_glu: (device, T, xq, x pointer, ldx,
    x dtype, out, ldy, y dtype, workspace triple)."""
    if type(X) is Mx:
        if X.K != w.K:
            raise ValueError(f"X has K={X.K}, the weight has K={w.K}")
        T, xq, xp, ldx, xdt = X.rows, _descriptor(X), None, 0, 0
        x0, xs, default = X.codes, X.scales, torch.bfloat16
    else:
        if X.dim() != 2:
            raise ValueError("X must be a 2-D tensor or an Mx")
        xdt = _float_type("X", X.dtype)
        T = X.shape[0]
        ldx = _row_pitch("X", X, T, w.K)
        xq, xp = None, X.data_ptr()
        x0, xs, default = X, None, X.dtype
    if out is None:
        out = x0.new_empty((T, w.rows), dtype=default if out_dtype is None else out_dtype)
    elif out_dtype is not None:
        _check_dtype("out", out, out_dtype)
    ydt = _float_type("out", out.dtype)
    ldy = _row_pitch("out", out, T, w.rows)
    dev = _one_gpu(names, x0, xs, w.codes, w.scales, out, *others)
    need = _sized(lib().nm_mx_workspace_size, "nm_mx_workspace_size", ("mx", w.rows, w.K, T, glu, xq is None, dev),
                  _descriptor(w), xq, T, int(glu))
    return dev, T, xq, xp, ldx, xdt, out, ldy, ydt, _workspace(workspace, need, dev)


def mx_linear(w: Mx, X, bias: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
              out: torch.Tensor | None = None, act: str = "none",
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    """nm_mx_linear: Y[T, R] = act(X @ W^T + bias) with W and X in the
    microscaled 4-bit format.  X: a [T, K] float16 / bfloat16 / float32 tensor,
    quantised by the call, or an Mx; Y has X's dtype (an Mx: bfloat16) unless
    out_dtype says otherwise; act "none" or "gelu"."""
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    bp = None
    if bias is not None:
        _check_dtype("bias", bias, torch.float32)
        if bias.shape != (w.rows,) or (w.rows > 1 and bias.stride(0) != 1):
            raise ValueError(f"bias must be a contiguous vector of length R={w.rows}, got {tuple(bias.shape)}")
        bp = bias.data_ptr()
    dev, T, xq, xp, ldx, xdt, out, ldy, ydt, ws = _mx_operands(
        w, X, out_dtype, out, workspace, False, "X, X scales, weight codes, weight scales, out, bias", bias)
    _call(dev, lib().nm_mx_linear, "nm_mx_linear", _descriptor(w), xq, xp, ldx, xdt, T, out.data_ptr(), ldy, ydt, bp,
          ACTS[act], ws[1], ws[2])
    return out


def mx_glu(gate: Mx, up: Mx, X, act: str = "silu", out_dtype: torch.dtype | None = None,
           out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """nm_mx_glu: the gated feed-forward block with both weights (and the
    activations, as in mx_linear) in the microscaled 4-bit format:
    H[T, R] = act(X @ Wg^T) * (X @ Wu^T); act "silu" or "gelu"."""
    a = _glu_act(act)
    if gate.rows != up.rows or gate.K != up.K:
        raise ValueError(f"gate is {gate.rows} x {gate.K}, up is {up.rows} x {up.K}")
    dev, T, xq, xp, ldx, xdt, out, ldy, ydt, ws = _mx_operands(
        gate, X, out_dtype, out, workspace, True,
        "X, X scales, gate codes, gate scales, out, up codes, up scales", up.codes, up.scales)
    _call(dev, lib().nm_mx_glu, "nm_mx_glu", _descriptor(gate), _descriptor(up), xq, xp, ldx, xdt, T, out.data_ptr(),
          ldy, ydt, a, ws[1], ws[2])
    return out
