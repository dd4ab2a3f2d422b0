"""Thin ctypes binding of the C ABI in include/exl3.h.

Functions keep the C names and only marshal arguments (torch tensors -> device
pointers, torch streams -> cudaStream_t).  Every step of the layer runs in the
CUDA library; if it is not built, importing this module raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libexl3_gb300.so")

EXL3_F16, EXL3_BF16, EXL3_F32, EXL3_I32, EXL3_I64, EXL3_E4M3, EXL3_E4M3_RANDOM = 0, 1, 2, 3, 4, 5, 6
EXL3_CB_MUL1, EXL3_CB_MCG, EXL3_CB_3INST = 0, 1, 2
STATUS = {0: "OK", -1: "E_NULL", -2: "E_DEVICE", -3: "E_DTYPE", -4: "E_SHAPE", -5: "E_ALIGN",
          -6: "E_WORKSPACE", -7: "E_ROUTING", -8: "E_CODEBOOK", -9: "E_CUDA",
          -10: "E_VALUE"}
ADAMW_BLOCK = 256          # elements that share a scale of an 8-bit state
DERR_ROUTE_ID, DERR_TABLE, DERR_TIMEOUT, DERR_PLAN = 1, 2, 4, 8

_DTYPE = {torch.float16: EXL3_F16, torch.bfloat16: EXL3_BF16, torch.float32: EXL3_F32,
          torch.int32: EXL3_I32, torch.int64: EXL3_I64}


class Exl3Error(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} returned {code} ({STATUS.get(code, '?')})")
        self.code = code


class exl3_proj(ctypes.Structure):
    _fields_ = [("trellis", ctypes.c_void_p), ("suh", ctypes.c_void_p),
                ("svh", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32),
                ("K", ctypes.c_int32), ("codebook", ctypes.c_int32)]


class exl3_experts(ctypes.Structure):
    _fields_ = [("trellis", ctypes.c_void_p), ("suh", ctypes.c_void_p),
                ("svh", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("K", ctypes.c_void_p), ("codebook", ctypes.c_void_p)]


class exl3_stages(ctypes.Structure):
    _fields_ = [("num_stages", ctypes.c_int32), ("trellis", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("K", ctypes.c_void_p)]


class exl3_adapters(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("rank", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("N", ctypes.c_int32), ("max_rank", ctypes.c_int32),
                ("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32)]


class exl3_adamw_tensors(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("numel", ctypes.c_void_p), ("first", ctypes.c_void_p),
                ("blocks", ctypes.c_int64), ("N", ctypes.c_int32), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("state_dtype", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                          "(the library has no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    V, I, Z, P = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER
    lib.exl3_abi_version.restype = I
    lib.exl3_moe_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.exl3_moe_workspace_bytes.restype = Z
    lib.exl3_linear_workspace_bytes.argtypes = [I, I, I]
    lib.exl3_linear_workspace_bytes.restype = Z
    lib.exl3_route_pack_max_tiles.argtypes = [I, I, I, I]
    lib.exl3_route_pack_max_tiles.restype = I
    lib.exl3_route_pack.argtypes = [V, I, I, I, I, I, V, V, V, V, V]
    lib.exl3_route_pack.restype = I
    lib.exl3_linear.argtypes = [V, I, I, P(exl3_proj), V, V, Z, V]
    lib.exl3_linear.restype = I
    lib.exl3_moe_forward.argtypes = [V, I, I, I, I, I, I, V, I, V, I, P(exl3_experts), I, V, Z, V, V]
    lib.exl3_moe_forward.restype = I
    lib.exl3_moe_additive.argtypes = [V, I, I, I, I, I, I, V, I, V, I, P(exl3_experts),
                                      P(exl3_stages), I, V, Z, V, V]
    lib.exl3_moe_additive.restype = I
    lib.exl3_profile_events.argtypes = [V]
    lib.exl3_profile_events.restype = I
    lib.exl3_workspace_error.argtypes = [V, P(ctypes.c_int32), V]
    lib.exl3_workspace_error.restype = I
    lib.exl3_router_workspace_bytes.argtypes = [I, I]
    lib.exl3_router_workspace_bytes.restype = Z
    lib.exl3_router_forward.argtypes = [V, I, I, I, I, I, V, V, I, V, V, V, V, V, Z, V]
    lib.exl3_router_forward.restype = I
    lib.exl3_router_backward.argtypes = [V, I, I, I, I, I, V, V, V, I, V, V, V, V, V]
    lib.exl3_router_backward.restype = I
    lib.exl3_lora_plan_bytes.argtypes = [I, I]
    lib.exl3_lora_plan_bytes.restype = Z
    lib.exl3_lora_plan.argtypes = [V, I, I, I, V, Z, V]
    lib.exl3_lora_plan.restype = I
    lib.exl3_lora_h_cols.argtypes = [I]
    lib.exl3_lora_h_cols.restype = I
    lib.exl3_lora_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.exl3_lora_workspace_bytes.restype = Z
    lib.exl3_lora_forward.argtypes = [V, I, I, V, V, Z, V, V, V, V, Z, V]
    lib.exl3_lora_forward.restype = I
    lib.exl3_lora_backward.argtypes = [V, V, V, I, I, V, V, Z, V, V, V, V, Z, V]
    lib.exl3_lora_backward.restype = I
    D = ctypes.c_double
    lib.exl3_dispatch_workspace_bytes.argtypes = [I, I, I]
    lib.exl3_dispatch_workspace_bytes.restype = Z
    lib.exl3_dispatch_plan.argtypes = [V, I, I, I, I, V, V, V, V, V, Z, V]
    lib.exl3_dispatch_plan.restype = I
    lib.exl3_dispatch.argtypes = [V, I, I, I, I, V, V, V]
    lib.exl3_dispatch.restype = I
    lib.exl3_combine.argtypes = [V, I, I, I, I, V, V, I, V, V, V]
    lib.exl3_combine.restype = I
    lib.exl3_combine_backward.argtypes = [V, V, I, I, I, I, V, V, I, V, V, V]
    lib.exl3_combine_backward.restype = I
    lib.exl3_adamw_workspace_bytes.argtypes = []
    lib.exl3_adamw_workspace_bytes.restype = Z
    lib.exl3_adamw.argtypes = [V, D, D, D, D, D, V, V, V, V, Z, V]
    lib.exl3_adamw.restype = I
    return lib


_lib = _load()
EXPORTED = ["exl3_abi_version", "exl3_moe_workspace_bytes", "exl3_linear_workspace_bytes",
            "exl3_route_pack_max_tiles", "exl3_route_pack", "exl3_linear", "exl3_moe_forward",
            "exl3_moe_additive", "exl3_profile_events", "exl3_workspace_error",
            "exl3_router_workspace_bytes", "exl3_router_forward", "exl3_router_backward",
            "exl3_lora_plan_bytes", "exl3_lora_plan", "exl3_lora_h_cols", "exl3_lora_workspace_bytes",
            "exl3_lora_forward", "exl3_lora_backward", "exl3_dispatch_workspace_bytes",
            "exl3_dispatch_plan", "exl3_dispatch", "exl3_combine", "exl3_combine_backward",
            "exl3_adamw_workspace_bytes", "exl3_adamw"]


def lib():
    return _lib


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _bytes(t):
    return 0 if t is None else t.nbytes


def _check(fn, rc, raise_on_error):
    if rc != 0 and raise_on_error:
        raise Exl3Error(fn, rc)
    return rc


# --------------------------------------------------------------------------- sizes
def exl3_abi_version() -> int:
    return _lib.exl3_abi_version()


def exl3_moe_workspace_bytes(M, topk, E, hidden, inter, capacity) -> int:
    return _lib.exl3_moe_workspace_bytes(M, topk, E, hidden, inter, capacity)


def exl3_linear_workspace_bytes(M, in_features, out_features) -> int:
    return _lib.exl3_linear_workspace_bytes(M, in_features, out_features)


def exl3_route_pack_max_tiles(M, topk, E, capacity) -> int:
    return _lib.exl3_route_pack_max_tiles(M, topk, E, capacity)


def exl3_router_workspace_bytes(M, E) -> int:
    return _lib.exl3_router_workspace_bytes(M, E)


def exl3_lora_plan_bytes(M, N) -> int:
    return _lib.exl3_lora_plan_bytes(M, N)


def exl3_lora_h_cols(max_rank) -> int:
    return _lib.exl3_lora_h_cols(max_rank)


def exl3_lora_workspace_bytes(M, N, in_features, out_features, max_rank) -> int:
    return _lib.exl3_lora_workspace_bytes(M, N, in_features, out_features, max_rank)


def exl3_dispatch_workspace_bytes(M, topk, E) -> int:
    return _lib.exl3_dispatch_workspace_bytes(M, topk, E)


def exl3_adamw_workspace_bytes() -> int:
    return _lib.exl3_adamw_workspace_bytes()


# --------------------------------------------------------------------------- device weights
def _to_dev(a: np.ndarray, device) -> torch.Tensor:
    if a.dtype == np.uint32:
        a = a.view(np.int32)
    elif a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


class DeviceProjection:
    """One projection in device memory (from a workloads.Projection)."""

    def __init__(self, proj, device="cuda"):
        self.trellis = _to_dev(proj.trellis.reshape(-1), device)
        self.suh = _to_dev(proj.suh, device)
        self.svh = _to_dev(proj.svh, device)
        self.scale = _to_dev(proj.scale, device)
        self.K, self.codebook = int(proj.K), int(proj.codebook)
        self.in_features, self.out_features = proj.in_features, proj.out_features

    def struct(self) -> exl3_proj:
        return exl3_proj(self.trellis.data_ptr(), self.suh.data_ptr(), self.svh.data_ptr(),
                         self.scale.data_ptr(), self.in_features, self.out_features, self.K,
                         self.codebook)


class DeviceExperts:
    """All experts of a layer: one trellis arena, one fp16 vector arena and the
    int64 pointer / int32 width and codebook tables of exl3_experts.

    get_proj(e, p) returns a workloads.Projection; K_of(e, p) its width (used to
    size the arena before any projection is generated)."""

    def __init__(self, get_proj, E, hidden, inter, K_of, device="cuda"):
        shape = {0: (hidden, inter), 1: (hidden, inter), 2: (inter, hidden)}
        words = [[(shape[p][0] // 16) * (shape[p][1] // 16) * 8 * int(K_of(e, p))
                  for p in range(3)] for e in range(E)]
        host = np.empty(sum(sum(r) for r in words), np.uint32)
        vec = np.empty(E * (2 * (2 * hidden + 2 * inter) + 2 * hidden + inter), np.float16)
        toff, voff, Ks, cbs = [], [], [], []
        o = v = 0
        for e in range(E):
            for p in range(3):
                pr = get_proj(e, p)
                n = pr.trellis.size
                assert n == words[e][p] and (pr.in_features, pr.out_features) == shape[p]
                host[o:o + n] = pr.trellis.reshape(-1)
                toff.append(o)
                o += n
                offs = []
                for arr in (pr.suh, pr.svh, pr.scale):
                    vec[v:v + arr.size] = arr
                    offs.append(v)
                    v += arr.size
                voff.append(offs)
                Ks.append(pr.K)
                cbs.append(pr.codebook)
        self.arena = _to_dev(host, device)
        self.vectors = torch.from_numpy(vec[:v]).to(device)
        base, vb = self.arena.data_ptr(), self.vectors.data_ptr()
        i64 = dict(dtype=torch.int64, device=device)
        self.t_trellis = torch.tensor([base + 4 * x for x in toff], **i64)
        self.t_suh = torch.tensor([vb + 2 * x[0] for x in voff], **i64)
        self.t_svh = torch.tensor([vb + 2 * x[1] for x in voff], **i64)
        self.t_scale = torch.tensor([vb + 2 * x[2] for x in voff], **i64)
        self.t_K = torch.tensor(Ks, dtype=torch.int32, device=device)
        self.t_cb = torch.tensor(cbs, dtype=torch.int32, device=device)
        self.E, self.hidden, self.inter = E, hidden, inter
        self.trellis_words = [w for r in words for w in r]

    @classmethod
    def from_workload(cls, w, device="cuda"):
        s = w.spec
        return cls(w.projection, s.E, s.hidden, s.inter, lambda e, p: s.K[e], device)

    def struct(self) -> exl3_experts:
        return exl3_experts(self.t_trellis.data_ptr(), self.t_suh.data_ptr(),
                            self.t_svh.data_ptr(), self.t_scale.data_ptr(),
                            self.t_K.data_ptr(), self.t_cb.data_ptr())


class DeviceStages:
    """Stage-major residual tables of exl3_stages (stages 1..S-1)."""

    def __init__(self, get_residual, alpha: np.ndarray, Ks, E, device="cuda"):
        nres = alpha.shape[0]
        self.num_stages = 1 + nres
        arrays, ptr_index = [], []
        for s in range(nres):
            for e in range(E):
                for p in range(3):
                    t = get_residual(s + 1, e, p)
                    ptr_index.append(None if t is None else len(arrays))
                    if t is not None:
                        arrays.append(t.reshape(-1))
        total = sum(a.size for a in arrays)
        host = np.empty(max(total, 4), np.uint32)
        offs, o = [], 0
        for a in arrays:
            host[o:o + a.size] = a
            offs.append(o)
            o += a.size
        self.arena = _to_dev(host, device)
        base = self.arena.data_ptr()
        ptrs = [0 if i is None else base + 4 * offs[i] for i in ptr_index]
        self.t_trellis = torch.tensor(ptrs, dtype=torch.int64, device=device)
        self.t_scale = torch.from_numpy(np.ascontiguousarray(alpha, np.float32).reshape(-1)).to(device)
        self.t_K = torch.tensor(np.repeat(np.asarray(Ks, np.int32), E * 3), device=device)
        self.trellis_bytes = 4 * total

    def struct(self) -> exl3_stages:
        return exl3_stages(self.num_stages, self.t_trellis.data_ptr(), self.t_scale.data_ptr(),
                           self.t_K.data_ptr())


class DeviceAdapters:
    """The tables of exl3_adapters over N adapters' device tensors: A[i] is
    [rank][in], B[i] [rank][out], all of one 16-bit dtype; scales[i] multiplies
    the update.  The same class over gradient tensors is what
    exl3_lora_backward writes through.  Keeps the tensors alive."""

    def __init__(self, A, B, scales, max_rank=None):
        self.A, self.B = list(A), list(B)
        if not self.A or len(self.A) != len(self.B) or len(self.A) != len(scales):
            raise ValueError("one A, one B and one scale per adapter")
        self.N, self.dtype, device = len(self.A), self.A[0].dtype, self.A[0].device
        self.in_features, self.out_features = self.A[0].shape[1], self.B[0].shape[1]
        for a, b in zip(self.A, self.B):
            if (a.shape != (b.shape[0], self.in_features) or b.shape[1] != self.out_features or
                    a.dtype != self.dtype or b.dtype != self.dtype or a.device != device or
                    b.device != device or not a.is_contiguous() or not b.is_contiguous()):
                raise ValueError("A must be [rank][in] and B [rank][out], contiguous, of one "
                                 "dtype and device")
        self.ranks = [a.shape[0] for a in self.A]
        self.max_rank = max(1, max(self.ranks)) if max_rank is None else int(max_rank)
        self.h_cols = exl3_lora_h_cols(self.max_rank)
        self.t_A = torch.tensor([a.data_ptr() for a in self.A], dtype=torch.int64, device=device)
        self.t_B = torch.tensor([b.data_ptr() for b in self.B], dtype=torch.int64, device=device)
        self.t_rank = torch.tensor(self.ranks, dtype=torch.int32, device=device)
        self.t_scale = torch.tensor(list(scales), dtype=torch.float32, device=device)
        self._struct = exl3_adapters(self.t_A.data_ptr(), self.t_B.data_ptr(),
                                     self.t_rank.data_ptr(), self.t_scale.data_ptr(), self.N,
                                     self.max_rank, self.in_features, self.out_features)
        self._ref = ctypes.byref(self._struct)     # built once: a decode call is short

    def struct(self) -> exl3_adapters:
        return self._struct


class DeviceAdamW:
    """The tables of exl3_adamw_tensors over lists of device tensors: parameters
    of one dtype, their gradients (of that dtype or float32) and the states m
    and v, float32 or float8_e4m3fn.  e4m3 states need m_scale and v_scale (one
    float32 per 256 elements; v then holds codes of sqrt(v)); master: float32
    copies of 16-bit parameters.  rounding, of e4m3 states: "nearest", or "random" for
    runs of more than some hundred steps, over which only that one's moments follow
    the gradients.  Zeroed states are a fresh optimiser's.  Keeps the tensors alive;
    their storage must stay where it is: building the tables takes some 2.5 us a
    tensor, so they are for buffers that stay, and gradients that move from step to
    step (set to none in between) are copied into such buffers, or get new tables."""

    def __init__(self, params, grads, m, v, m_scale=None, v_scale=None, master=None, rounding="nearest"):
        opt = lambda l: None if l is None else list(l)
        self.params, self.grads, self.m, self.v = list(params), list(grads), list(m), list(v)
        self.m_scale, self.v_scale, self.master = opt(m_scale), opt(v_scale), opt(master)
        if not self.params or not self.m:
            raise ValueError("at least one tensor")
        p0, state = self.params[0], self.m[0].dtype
        numel = [p.numel() for p in self.params]
        blocks = [-(-n // ADAMW_BLOCK) for n in numel]
        codes = state is torch.float8_e4m3fn
        if codes == (self.m_scale is None) or codes == (self.v_scale is None):
            raise ValueError("m_scale and v_scale belong to float8_e4m3fn states")
        if rounding not in ("nearest", "random") or (rounding == "random" and not codes):
            raise ValueError("rounding is nearest or, of float8_e4m3fn states, random")
        if self.master is not None and p0.dtype is torch.float32:
            raise ValueError("float32 parameters have no masters")
        grad = self.grads[0].dtype if self.grads else None
        if grad not in (p0.dtype, torch.float32) or state not in (torch.float32, torch.float8_e4m3fn):
            raise ValueError("gradients are of the parameters' dtype or float32, states float32 or float8_e4m3fn")
        for what, l, dtype, sizes in (("params", self.params, p0.dtype, numel), ("grads", self.grads, grad, numel),
                                      ("m", self.m, state, numel), ("v", self.v, state, numel),
                                      ("m_scale", self.m_scale, torch.float32, blocks),
                                      ("v_scale", self.v_scale, torch.float32, blocks),
                                      ("master", self.master, torch.float32, numel)):
            if l is None:
                continue
            if len(l) != len(self.params):
                raise ValueError(f"{what}: one per parameter")
            for t, n in zip(l, sizes):
                if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.device != p0.device:
                    raise ValueError(f"{what} must be contiguous, of one dtype and device, and of the parameters' sizes")
                if l is not self.m_scale and l is not self.v_scale and t.data_ptr() % 16:
                    raise ValueError(f"{what} must be 16-byte aligned")
        first = [0]
        for b in blocks:
            first.append(first[-1] + b)
        table = lambda l: None if l is None else torch.tensor(l, dtype=torch.int64, device=p0.device)
        ptrs = lambda l: None if l is None else table([t.data_ptr() for t in l])
        self._tables = [ptrs(self.params), ptrs(self.grads), ptrs(self.m), ptrs(self.v), ptrs(self.m_scale),
                        ptrs(self.v_scale), ptrs(self.master), table(numel), table(first)]
        self._struct = exl3_adamw_tensors(*[_ptr(t) for t in self._tables], first[-1], len(numel),
                                          _DTYPE[p0.dtype], _DTYPE[grad],
                                          EXL3_F32 if not codes else EXL3_E4M3_RANDOM if rounding == "random" else EXL3_E4M3)
        self._ref = ctypes.byref(self._struct)

    def struct(self) -> exl3_adamw_tensors:
        return self._struct


# --------------------------------------------------------------------------- entry points
def exl3_route_pack(ids, E, capacity, offsets, packed, tiles, info, stream=None,
                    raise_on_error=True) -> int:
    M, topk = ids.shape
    rc = _lib.exl3_route_pack(_ptr(ids), _DTYPE[ids.dtype], M, topk, E, capacity, _ptr(offsets),
                              _ptr(packed), _ptr(tiles), _ptr(info), _stream(stream))
    return _check("exl3_route_pack", rc, raise_on_error)


def exl3_linear(x, proj: DeviceProjection, y, workspace, stream=None, raise_on_error=True) -> int:
    st = proj.struct()
    rc = _lib.exl3_linear(_ptr(x), _DTYPE[x.dtype], x.shape[0], ctypes.byref(st), _ptr(y),
                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                          _stream(stream))
    return _check("exl3_linear", rc, raise_on_error)


def exl3_moe_forward(x, ids, rw, experts: DeviceExperts, capacity, workspace, out, stream=None,
                     raise_on_error=True) -> int:
    st = experts.struct()
    M, topk = ids.shape
    rc = _lib.exl3_moe_forward(_ptr(x), _DTYPE[x.dtype], M, experts.hidden, experts.inter,
                               experts.E, topk, _ptr(ids), _DTYPE[ids.dtype], _ptr(rw),
                               _DTYPE[rw.dtype], ctypes.byref(st), capacity, _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _ptr(out),
                               _stream(stream))
    return _check("exl3_moe_forward", rc, raise_on_error)


def exl3_moe_additive(x, ids, rw, experts: DeviceExperts, stages: DeviceStages, capacity,
                      workspace, out, stream=None, raise_on_error=True) -> int:
    st = experts.struct()
    ss = stages.struct()
    M, topk = ids.shape
    rc = _lib.exl3_moe_additive(_ptr(x), _DTYPE[x.dtype], M, experts.hidden, experts.inter,
                                experts.E, topk, _ptr(ids), _DTYPE[ids.dtype], _ptr(rw),
                                _DTYPE[rw.dtype], ctypes.byref(st), ctypes.byref(ss), capacity,
                                _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _ptr(out), _stream(stream))
    return _check("exl3_moe_additive", rc, raise_on_error)


def _shaped(what, t, shape, dtype=None):
    if t is not None and (t.shape != shape or not t.is_contiguous() or
                          (dtype is not None and t.dtype is not dtype)):
        raise ValueError(f"{what} must be a contiguous {shape} tensor"
                         f"{'' if dtype is None else ' of ' + str(dtype)}")


def _as_bytes(mask):
    """A bool mask's bytes, 0 and 1."""
    return mask.view(torch.uint8) if mask is not None and mask.dtype is torch.bool else mask


def exl3_router_forward(logits, ids, rw, renorm=False, stats=None, valid=None, counts=None, loss=None,
                        workspace=None, stream=None, raise_on_error=True) -> int:
    M, E = logits.shape
    topk = ids.shape[1]
    _shaped("logits", logits, (M, E))
    _shaped("ids", ids, (M, topk), torch.int32)
    _shaped("rw", rw, (M, topk))
    if stats is not None:
        _shaped("stats", stats, (M, 2), torch.float32)
    if counts is not None or loss is not None:
        _shaped("counts", counts, (E + 1,), torch.int32)
        _shaped("loss", loss, (1,), torch.float32)
    valid = _as_bytes(valid)
    _shaped("valid", valid, (M,), torch.uint8)
    rc = _lib.exl3_router_forward(logits.data_ptr(), _DTYPE[logits.dtype], M, E, topk, renorm,
                                  ids.data_ptr(), rw.data_ptr(), _DTYPE[rw.dtype], _ptr(stats),
                                  _ptr(valid), _ptr(counts), _ptr(loss), _ptr(workspace),
                                  _bytes(workspace), _stream(stream))
    return _check("exl3_router_forward", rc, raise_on_error)


def exl3_router_backward(logits, ids, stats, d_logits, renorm=False, d_rw=None, valid=None,
                         counts=None, d_loss=None, stream=None, raise_on_error=True) -> int:
    M, E = logits.shape
    topk = ids.shape[1]
    _shaped("logits", logits, (M, E))
    _shaped("ids", ids, (M, topk), torch.int32)
    _shaped("stats", stats, (M, 2), torch.float32)
    _shaped("d_logits", d_logits, (M, E), logits.dtype)
    if d_rw is not None:
        _shaped("d_rw", d_rw, (M, topk))
    valid = _as_bytes(valid)
    _shaped("valid", valid, (M,), torch.uint8)
    if counts is not None or d_loss is not None:
        _shaped("counts", counts, (E + 1,), torch.int32)
        _shaped("d_loss", d_loss, (1,), torch.float32)
    rw_dtype = EXL3_F32 if d_rw is None else _DTYPE[d_rw.dtype]
    rc = _lib.exl3_router_backward(logits.data_ptr(), _DTYPE[logits.dtype], M, E, topk, renorm,
                                   ids.data_ptr(), stats.data_ptr(), _ptr(d_rw), rw_dtype,
                                   _ptr(valid), _ptr(counts), _ptr(d_loss), d_logits.data_ptr(),
                                   _stream(stream))
    return _check("exl3_router_backward", rc, raise_on_error)


def exl3_lora_plan(ids, N, plan, stream=None, raise_on_error=True) -> int:
    M = ids.shape[0]
    _shaped("ids", ids, (M,))
    rc = _lib.exl3_lora_plan(_ptr(ids), _DTYPE[ids.dtype], M, N, _ptr(plan), _bytes(plan),
                             _stream(stream))
    return _check("exl3_lora_plan", rc, raise_on_error)


def exl3_lora_forward(x, plan, adapters: DeviceAdapters, y, workspace, base=None, h=None,
                      stream=None, raise_on_error=True) -> int:
    M, dt = x.shape[0], adapters.dtype
    out = (M, adapters.out_features)
    _shaped("x", x, (M, adapters.in_features), dt)
    _shaped("y", y, out, dt)
    if base is not None:
        _shaped("base", base, out, dt)
    if h is not None:
        _shaped("h", h, (M, adapters.h_cols), dt)
    rc = _lib.exl3_lora_forward(x.data_ptr(), _DTYPE[dt], M, adapters._ref, plan.data_ptr(),
                                _bytes(plan), _ptr(base), y.data_ptr(), _ptr(h),
                                workspace.data_ptr(), _bytes(workspace), _stream(stream))
    return _check("exl3_lora_forward", rc, raise_on_error)


def exl3_lora_backward(dy, x, h, plan, adapters: DeviceAdapters, grads, workspace, dx=None,
                       dx_base=None, stream=None, raise_on_error=True) -> int:
    M, dt = dy.shape[0], adapters.dtype
    inp = (M, adapters.in_features)
    _shaped("dy", dy, (M, adapters.out_features), dt)
    if x is not None:
        _shaped("x", x, inp, dt)
    if h is not None:
        _shaped("h", h, (M, adapters.h_cols), dt)
    if dx is not None:
        _shaped("dx", dx, inp, dt)
    if dx_base is not None:
        _shaped("dx_base", dx_base, inp, dt)
    if grads is not None and (grads.ranks != adapters.ranks or grads.dtype is not dt):
        raise ValueError("grads must hold a tensor like A and one like B for every adapter")
    rc = _lib.exl3_lora_backward(dy.data_ptr(), _ptr(x), _ptr(h), _DTYPE[dt], M, adapters._ref,
                                 plan.data_ptr(), _bytes(plan), _ptr(dx_base), _ptr(dx),
                                 None if grads is None else grads._ref, workspace.data_ptr(),
                                 _bytes(workspace), _stream(stream))
    return _check("exl3_lora_backward", rc, raise_on_error)


def _arg(what, t, shape, dtype=None):
    """The address of a tensor that has to be contiguous and of this shape (and dtype); None for None."""
    if t is None:
        return None
    if t.shape != shape or not t.is_contiguous() or (dtype is not None and t.dtype is not dtype):
        _shaped(what, t, shape, dtype)
    return t.data_ptr()


def exl3_dispatch_plan(ids, E, offsets, packed, slots, workspace, experts=None, stream=None,
                       raise_on_error=True) -> int:
    M, topk = shape = ids.shape
    i32, routes = torch.int32, (M * topk,)
    rc = _lib.exl3_dispatch_plan(_arg("ids", ids, shape), _DTYPE[ids.dtype], M, topk, E,
                                 _arg("offsets", offsets, (E + 1,), i32), _arg("packed", packed, routes, i32),
                                 _arg("slots", slots, shape, i32), _arg("experts", experts, routes, i32),
                                 _ptr(workspace), _bytes(workspace), _stream(stream))
    return _check("exl3_dispatch_plan", rc, raise_on_error)


def exl3_dispatch(x, slots, xp, stream=None, raise_on_error=True) -> int:
    M, topk = shape = slots.shape
    width, dt = x.shape[1], x.dtype
    rc = _lib.exl3_dispatch(_arg("x", x, (M, width)), _DTYPE[dt], M, topk, width,
                            _arg("slots", slots, shape, torch.int32), _arg("xp", xp, (M * topk, width), dt),
                            _stream(stream))
    return _check("exl3_dispatch", rc, raise_on_error)


def exl3_combine(y, slots, out, rw=None, base=None, stream=None, raise_on_error=True) -> int:
    M, topk = shape = slots.shape
    width, dt = out.shape[1], out.dtype
    row = (M, width)
    rc = _lib.exl3_combine(_arg("y", y, (M * topk, width), dt), _DTYPE[dt], M, topk, width,
                           _arg("slots", slots, shape, torch.int32), _arg("rw", rw, shape),
                           EXL3_F32 if rw is None else _DTYPE[rw.dtype], _arg("base", base, row, dt),
                           _arg("out", out, row), _stream(stream))
    return _check("exl3_combine", rc, raise_on_error)


def exl3_combine_backward(d_out, y, slots, rw, dy=None, d_rw=None, stream=None, raise_on_error=True) -> int:
    M, topk = shape = slots.shape
    width, dt = d_out.shape[1], d_out.dtype
    rows, of = (M * topk, width), d_rw if rw is None else rw
    rc = _lib.exl3_combine_backward(_arg("d_out", d_out, (M, width)), _arg("y", y, rows, dt), _DTYPE[dt], M, topk,
                                    width, _arg("slots", slots, shape, torch.int32), _arg("rw", rw, shape),
                                    EXL3_F32 if of is None else _DTYPE[of.dtype], _arg("dy", dy, rows, dt),
                                    _arg("d_rw", d_rw, shape, None if rw is None else rw.dtype), _stream(stream))
    return _check("exl3_combine_backward", rc, raise_on_error)


def exl3_adamw(tensors: DeviceAdamW, step, workspace, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
               lr_scale=None, grad_scale=None, stream=None, raise_on_error=True) -> int:
    f32 = torch.float32
    rc = _lib.exl3_adamw(tensors._ref, lr, betas[0], betas[1], eps, weight_decay,
                         _arg("lr_scale", lr_scale, (1,), f32), _arg("grad_scale", grad_scale, (1,), f32),
                         _arg("step", step, (1,), torch.int32), _ptr(workspace), _bytes(workspace),
                         _stream(stream))
    return _check("exl3_adamw", rc, raise_on_error)


class ProfileEvents:
    """Five torch CUDA events recorded between the fused layer's kernels
    (route pack | rotation | gate/up GEMM | down GEMM + combine)."""

    def __init__(self):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(5)]
        for e in self.events:          # creates the underlying cudaEvent_t
            e.record()
        torch.cuda.synchronize()
        self._arr = (ctypes.c_void_p * 5)(*[ctypes.c_void_p(e.cuda_event) for e in self.events])

    def __enter__(self):
        _lib.exl3_profile_events(ctypes.cast(self._arr, ctypes.c_void_p))
        return self

    def __exit__(self, *exc):
        _lib.exl3_profile_events(None)

    def times_ms(self):
        """(route pack, rotation, gate/up, down + combine) in ms for the last call."""
        e = self.events
        return [e[i].elapsed_time(e[i + 1]) for i in range(4)]


def exl3_workspace_error(workspace, stream=None) -> int:
    err = ctypes.c_int32(0)
    rc = _lib.exl3_workspace_error(_ptr(workspace), ctypes.byref(err), _stream(stream))
    _check("exl3_workspace_error", rc, True)
    return int(err.value)
