"""Binding of libbeam_moe.so (include/beam_moe.h): ctypes, and for the calls that
check whole tensors the compiled module _marshal.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  Tensors are torch tensors on the current CUDA device; streams default
to torch's current stream.  Loading fails loudly when the library is missing:
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbeam_moe.so")

BEAM_BF16 = 0
BEAM_F32 = 1
FORWARD_STAGES = 7

STATUS = {0: "BEAM_OK", 1: "BEAM_ERR_INVALID_ARG", 2: "BEAM_ERR_UNSUPPORTED_SHAPE",
          3: "BEAM_ERR_WORKSPACE", 4: "BEAM_ERR_CUDA", 5: "BEAM_ERR_TIMEOUT",
          6: "BEAM_ERR_INTERNAL"}


class BeamError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class Desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("d", ctypes.c_int), ("E", ctypes.c_int),
                ("I", ctypes.c_int), ("K", ctypes.c_int), ("dtype", ctypes.c_int),
                ("renorm_topk", ctypes.c_int), ("mask_logit_threshold", ctypes.c_float),
                ("n_shared", ctypes.c_int), ("I_shared", ctypes.c_int)]


class Mx4Desc(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("E", ctypes.c_int), ("n", ctypes.c_int),
                ("k", ctypes.c_int), ("swiglu", ctypes.c_int), ("out_dtype", ctypes.c_int)]


class BlockDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("d", ctypes.c_int), ("dtype", ctypes.c_int),
                ("eps", ctypes.c_float), ("res_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("accumulate", ctypes.c_int)]


class BalanceDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("E", ctypes.c_int), ("K", ctypes.c_int),
                ("n_seq", ctypes.c_int), ("logits_ld", ctypes.c_int), ("has_mask", ctypes.c_int),
                ("count_kept", ctypes.c_int), ("mask_logit_threshold", ctypes.c_float),
                ("coef", ctypes.c_float)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("BN", ctypes.c_int), ("router_bn", ctypes.c_int),
                ("router_splits", ctypes.c_int), ("p_cap", ctypes.c_int),
                ("tiles_cap", ctypes.c_int), ("sub_bn", ctypes.c_int),
                ("one_launch", ctypes.c_int), ("sh_bn", ctypes.c_int),
                ("sh_split1", ctypes.c_int), ("sh_split2", ctypes.c_int)] + \
               [(n, ctypes.c_size_t) for n in (
                   "off_err", "off_meta", "off_counts", "off_hist", "off_partial", "off_idx",
                   "off_w", "off_pair", "off_pair_pos", "off_tiles", "off_xp", "off_h", "off_y",
                   "off_tile_done", "off_hs", "off_ys", "off_tiles_sub", "off_ctl", "off_sp",
                   "workspace_bytes")]


_lib = None


def lib():
    """The loaded library; raises if it was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m dynamic_expert_routing_router_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        pd = ctypes.POINTER(Desc)
        L.beam_moe_workspace_size.argtypes = [pd]
        L.beam_moe_workspace_size.restype = sz
        L.beam_moe_plan.argtypes = [pd, ctypes.POINTER(PlanInfo)]
        L.beam_moe_route.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_moe_forward.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_moe_forward_shared.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                              vp]
        L.beam_moe_forward_shared.restype = i32
        L.beam_moe_forward_profiled.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp,
                                                ctypes.POINTER(vp)]
        L.beam_moe_check.argtypes = [pd, vp, vp]
        L.beam_moe_route_noalloc.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.beam_moe_route_noalloc.restype = i32
        L.beam_moe_set_one_launch_tokens.argtypes = [i32]
        L.beam_moe_set_one_launch_tokens.restype = i32
        L.beam_moe_forward_kernel_count.argtypes = [pd]
        L.beam_moe_forward_kernel_count.restype = i32
        L.beam_moe_backward_workspace_size.argtypes = [pd]
        L.beam_moe_backward_workspace_size.restype = sz
        L.beam_moe_backward.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp,
                                        vp, vp, vp, vp, sz, vp]
        L.beam_moe_backward.restype = i32
        L.beam_moe_backward_aux.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp,
                                            vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_moe_backward_aux.restype = i32
        L.beam_moe_backward_kernel_count.argtypes = [pd]
        L.beam_moe_backward_kernel_count.restype = i32
        L.beam_moe_ep_dispatch.argtypes = [pd, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_moe_ep_dispatch.restype = i32
        L.beam_moe_expert_rows.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_moe_expert_rows.restype = i32
        L.beam_moe_ep_combine.argtypes = [pd, vp, vp, vp, vp, vp, vp]
        L.beam_moe_ep_combine.restype = i32
        L.beam_moe_route_noalloc_check.argtypes = [vp]
        L.beam_moe_route_noalloc_check.restype = i32
        L.beam_moe_tau_to_logit.argtypes = [ctypes.c_float]
        L.beam_moe_tau_to_logit.restype = ctypes.c_float
        L.beam_moe_set_fault_injection.argtypes = [i32, ctypes.c_ulonglong]
        L.beam_moe_set_fault_injection.restype = i32
        pb = ctypes.POINTER(BlockDesc)
        L.beam_block_enter.argtypes = [pb, vp, vp, vp, vp]
        L.beam_block_exit.argtypes = [pb, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.beam_block_workspace_size.argtypes = [pb]
        L.beam_block_workspace_size.restype = sz
        L.beam_block_enter_backward.argtypes = [pb, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_block_exit_backward.argtypes = [pb] + [vp] * 15 + [sz, vp]
        pl = ctypes.POINTER(BalanceDesc)
        L.beam_moe_balance_workspace_size.argtypes = [pl]
        L.beam_moe_balance_workspace_size.restype = sz
        L.beam_moe_balance.argtypes = [pl, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_moe_balance_backward.argtypes = [pl, vp, vp, vp, vp, vp, vp]
        for f in ("beam_block_enter", "beam_block_exit", "beam_block_enter_backward",
                  "beam_block_exit_backward", "beam_moe_balance", "beam_moe_balance_backward"):
            getattr(L, f).restype = i32
        i64 = ctypes.c_longlong
        L.beam_mx4_quantize.argtypes = [i32, i64, i32, vp, vp, vp, vp, i32, vp]
        L.beam_mx4_dequantize.argtypes = [i32, i64, i32, vp, vp, i32, vp, vp]
        pm = ctypes.POINTER(Mx4Desc)
        L.beam_mx4_workspace_size.argtypes = [pm]
        L.beam_mx4_workspace_size.restype = sz
        L.beam_mx4_expert_product.argtypes = [pm, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.beam_mx4_check.argtypes = [pm, vp, vp]
        for f in ("beam_mx4_quantize", "beam_mx4_dequantize", "beam_mx4_expert_product",
                  "beam_mx4_check"):
            getattr(L, f).restype = i32
        L.beam_status_str.argtypes = [i32]
        L.beam_status_str.restype = ctypes.c_char_p
        L.beam_moe_stage_name.argtypes = [i32]
        L.beam_moe_stage_name.restype = ctypes.c_char_p
        for f in ("beam_moe_plan", "beam_moe_route", "beam_moe_forward",
                  "beam_moe_forward_profiled", "beam_moe_check"):
            getattr(L, f).restype = i32
        _lib = L
    return _lib


def tau_logit(tau: float) -> float:
    """The descriptor's mask threshold for sigmoid(z) >= tau (beam_moe_tau_to_logit)."""
    return float(lib().beam_moe_tau_to_logit(ctypes.c_float(tau)))


def desc(T, d, E, I, K, dtype="bf16", renorm=1, tau=0.5, n_shared=0, I_shared=0) -> Desc:
    """Layer descriptor; `tau` is the mask threshold of sigmoid(x W_mask);
    n_shared always-on shared experts of width I_shared."""
    code = dtype if isinstance(dtype, int) else (BEAM_BF16 if dtype == "bf16" else BEAM_F32)
    return Desc(int(T), int(d), int(E), int(I), int(K), int(code), int(renorm),
                tau_logit(tau), int(n_shared), int(I_shared))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ok(status, what):
    if status != 0:
        raise BeamError(status, what)


def status_str(status: int) -> str:
    return lib().beam_status_str(int(status)).decode()


def stage_name(i: int):
    s = lib().beam_moe_stage_name(int(i))
    return None if s is None else s.decode()


def workspace_size(dsc: Desc) -> int:
    return int(lib().beam_moe_workspace_size(ctypes.byref(dsc)))


def set_one_launch_tokens(max_tokens: int) -> int:
    """Largest batch run as one launch (0 = never); returns the previous value."""
    return int(lib().beam_moe_set_one_launch_tokens(int(max_tokens)))


def kernel_count(dsc: Desc) -> int:
    """Kernel launches of one forward call for this descriptor."""
    return int(lib().beam_moe_forward_kernel_count(ctypes.byref(dsc)))


def backward_workspace_size(dsc: Desc) -> int:
    return int(lib().beam_moe_backward_workspace_size(ctypes.byref(dsc)))


def backward_kernel_count(dsc: Desc) -> int:
    """Kernel launches of one backward call for this descriptor."""
    return int(lib().beam_moe_backward_kernel_count(ctypes.byref(dsc)))


def alloc_backward_workspace(dsc: Desc, device=None):
    """A uint8 torch tensor of backward_workspace_size(dsc) bytes on `device`."""
    import torch
    n = backward_workspace_size(dsc)
    if n == 0:
        raise BeamError(1, "beam_moe_backward_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def backward(dsc, x, W_gate, W_mask, W1, W3, W2, dy, beta, dx, dW_gate, dW_mask, dW1, dW3, dW2,
             workspace, stream=None, dlogits=None):
    """Training-mode gradients (straight-through estimator, beta-weighted
    penalty on the candidates' mask scores).  dx is overwritten; the weight
    gradients (fp32, shaped like their weights) are accumulated into.
    dlogits: a further gradient of the main router's logits, f32 [T, E]
    (balance_backward), that goes on to dx and dW_gate."""
    if dlogits is not None:
        import torch
        aux = _arg("beam_moe_backward_aux", "dlogits", dlogits, torch.float32, (dsc.T, dsc.E),
                   _current_device())
        _ok(lib().beam_moe_backward_aux(
            ctypes.byref(dsc), _ptr(x), _ptr(W_gate), _ptr(W_mask), _ptr(W1), _ptr(W3), _ptr(W2),
            _ptr(dy), aux, ctypes.c_float(beta), _ptr(dx), _ptr(dW_gate), _ptr(dW_mask),
            _ptr(dW1), _ptr(dW3), _ptr(dW2), _ptr(workspace), workspace.numel(),
            _stream(stream)), "beam_moe_backward_aux")
        return
    _ok(lib().beam_moe_backward(ctypes.byref(dsc), _ptr(x), _ptr(W_gate), _ptr(W_mask),
                                _ptr(W1), _ptr(W3), _ptr(W2), _ptr(dy), ctypes.c_float(beta),
                                _ptr(dx), _ptr(dW_gate), _ptr(dW_mask), _ptr(dW1), _ptr(dW3),
                                _ptr(dW2), _ptr(workspace), workspace.numel(), _stream(stream)),
        "beam_moe_backward")


def plan(dsc: Desc) -> dict:
    info = PlanInfo()
    _ok(lib().beam_moe_plan(ctypes.byref(dsc), ctypes.byref(info)), "beam_moe_plan")
    return {name: getattr(info, name) for name, _ in PlanInfo._fields_}


def alloc_workspace(dsc: Desc, device=None):
    """A uint8 torch tensor of workspace_size(dsc) bytes on `device`."""
    import torch
    n = workspace_size(dsc)
    if n == 0:
        raise BeamError(1, "beam_moe_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def route(dsc, x, W_gate, W_mask, topk_idx, topk_w, counts, hist=None, logits=None,
          workspace=None, stream=None):
    _ok(lib().beam_moe_route(ctypes.byref(dsc), _ptr(x), _ptr(W_gate), _ptr(W_mask),
                             _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(hist),
                             _ptr(logits), _ptr(workspace),
                             workspace.numel() if workspace is not None else 0,
                             _stream(stream)), "beam_moe_route")


NOALLOC_SCRATCH_BYTES = 16 << 20


def route_noalloc(dsc, x, W_gate, W_mask, topk_idx, topk_w, counts, hist=None, logits=None,
                  stream=None):
    """beam_moe_route without a caller workspace (scratch in the library's own
    fixed device array); for callers that cannot allocate device memory."""
    _ok(lib().beam_moe_route_noalloc(ctypes.byref(dsc), _ptr(x), _ptr(W_gate), _ptr(W_mask),
                                     _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(hist),
                                     _ptr(logits), _stream(stream)), "beam_moe_route_noalloc")


def route_noalloc_check(stream=None):
    """Synchronise and read the error word of the last route_noalloc call."""
    _ok(lib().beam_moe_route_noalloc_check(_stream(stream)), "beam_moe_route_noalloc_check")


FAULT_NONE, FAULT_EXPERT_STAGE, FAULT_ROUTER_STAGE, FAULT_SHARED_STAGE = 0, 1, 2, 3
FAULT_MX4_STAGE = 4


def set_fault_injection(mode: int, wait_limit_ns: int = 0):
    """Testing aid (beam_moe_set_fault_injection): make a bounded device wait
    expire in later calls; mode 0 and wait_limit_ns 0 restore the defaults."""
    _ok(lib().beam_moe_set_fault_injection(int(mode), int(wait_limit_ns)),
        "beam_moe_set_fault_injection")


def forward(dsc, x, W_gate, W_mask, W1, W3, W2, out, workspace, stream=None):
    _ok(lib().beam_moe_forward(ctypes.byref(dsc), _ptr(x), _ptr(W_gate), _ptr(W_mask),
                               _ptr(W1), _ptr(W3), _ptr(W2), _ptr(out), _ptr(workspace),
                               workspace.numel(), _stream(stream)), "beam_moe_forward")


def forward_shared(dsc, x, W_gate, W_mask, W1, W3, W2, W1s, W3s, W2s, out, workspace,
                   stream=None):
    """The layer with dsc.n_shared always-on shared experts (weights W1s, W3s
    [S, I_shared, d], W2s [S, d, I_shared])."""
    _ok(lib().beam_moe_forward_shared(ctypes.byref(dsc), _ptr(x), _ptr(W_gate), _ptr(W_mask),
                                      _ptr(W1), _ptr(W3), _ptr(W2), _ptr(W1s), _ptr(W3s),
                                      _ptr(W2s), _ptr(out), _ptr(workspace), workspace.numel(),
                                      _stream(stream)), "beam_moe_forward_shared")


def forward_profiled(dsc, x, W_gate, W_mask, W1, W3, W2, out, workspace, events, stream=None):
    """`events`: FORWARD_STAGES + 1 torch.cuda.Event(enable_timing=True) or None
    (None records nothing at that point)."""
    arr = (ctypes.c_void_p * len(events))(*[None if e is None else e.cuda_event
                                             for e in events])
    _ok(lib().beam_moe_forward_profiled(ctypes.byref(dsc), _ptr(x), _ptr(W_gate), _ptr(W_mask),
                                        _ptr(W1), _ptr(W3), _ptr(W2), _ptr(out),
                                        _ptr(workspace), workspace.numel(), _stream(stream),
                                        arr), "beam_moe_forward_profiled")


def ep_dispatch(dsc, n_ranks, x, topk_idx, counts, send_rows, send_pair, send_expert,
                send_counts, pair_pos, workspace, stream=None):
    """Kept pairs grouped by destination rank (expert-parallel dispatch)."""
    _ok(lib().beam_moe_ep_dispatch(ctypes.byref(dsc), int(n_ranks), _ptr(x), _ptr(topk_idx),
                                   _ptr(counts), _ptr(send_rows), _ptr(send_pair),
                                   _ptr(send_expert), _ptr(send_counts), _ptr(pair_pos),
                                   _ptr(workspace), workspace.numel(), _stream(stream)),
        "beam_moe_ep_dispatch")


def expert_rows(dsc, x_rows, expert_id, W1, W3, W2, y_rows, workspace, stream=None):
    """y_rows[i] = E_{expert_id[i]}(x_rows[i]) in fp32 (dsc.K == 1, dsc.T rows)."""
    _ok(lib().beam_moe_expert_rows(ctypes.byref(dsc), _ptr(x_rows), _ptr(expert_id), _ptr(W1),
                                   _ptr(W3), _ptr(W2), _ptr(y_rows), _ptr(workspace),
                                   workspace.numel(), _stream(stream)), "beam_moe_expert_rows")


def ep_combine(dsc, y_rows, topk_idx, topk_w, pair_pos, out, stream=None):
    """out_t = sum over kept k of topk_w[t,k] * y_rows[pair_pos[t,k]] (slot order)."""
    _ok(lib().beam_moe_ep_combine(ctypes.byref(dsc), _ptr(y_rows), _ptr(topk_idx),
                                  _ptr(topk_w), _ptr(pair_pos), _ptr(out), _stream(stream)),
        "beam_moe_ep_combine")


# ------------------------------------------------------ checked arguments --
# The calls below take whole tensors, not buffers with a descriptor's word for
# their size, so the binding refuses what the library cannot see: another
# dtype or shape, strides, another device than the current one.  The checks and
# the call run in the compiled module _marshal (csrc/marshal.cpp), from one
# description of each entry point; errors are worded here.

def _code(dtype):
    return dtype if isinstance(dtype, int) else (BEAM_BF16 if dtype == "bf16" else BEAM_F32)


_torch_module = None
_marshal_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _marshal():
    """The compiled half of the binding; raises if it was not built, or only for
    another torch or Python."""
    global _marshal_module
    if _marshal_module is None:
        from importlib import machinery, util

        from . import build
        _torch()  # its libraries come first
        path, name = build.marshal_path(), __package__ + "._marshal"
        try:
            spec = util.spec_from_loader(name, machinery.ExtensionFileLoader(name, path), origin=path)
            m = util.module_from_spec(spec)
            spec.loader.exec_module(m)
        except ImportError as e:
            raise RuntimeError(f"the module {os.path.basename(path)} is missing: build it with "
                               "`python -m dynamic_expert_routing_router_b200.build`") from e
        _marshal_module = m
    return _marshal_module


def _torch_dtype(code):
    return _torch().bfloat16 if code == BEAM_BF16 else _torch().float32


def _arg(what, name, t, dtype, shape, dev, optional=False):
    """The address of tensor `t`, which has to be a contiguous `dtype` tensor
    of `shape` on device `dev` (_current_device(); None: anywhere); None where
    it may be left out."""
    if t is None:
        if optional:
            return None
        raise BeamError(1, f"{what}: {name} is missing")
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise BeamError(1, f"{what}: {name} has to be a contiguous {dtype} tensor of shape "
                           f"{tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if dev is not None and t.get_device() != dev:
        raise BeamError(1, f"{what}: {name} is on {t.device}, not the current CUDA device")
    return t.data_ptr()


_ROWS, _F32, _I32, _U8, _WORKSPACE = range(5)


class _Entry:
    """An entry point f(desc, tensors..., stream) and what its tensors have to
    be: "name dtype dim ..." each, dtype "rows" (by the descriptor's field
    `rows`), f32, i32, u8 or "workspace" (an address and a size), dims products
    of descriptor fields ("E*n", "k/32", "n_seq+1"); a "?" behind the name:
    may be left out."""

    _KINDS = {"rows": _ROWS, "f32": _F32, "i32": _I32, "u8": _U8, "workspace": _WORKSPACE}

    def __init__(self, name, desc, rows, *tensors):
        self.name, self.rows = name, rows
        self.run = self._first  # (desc, stream, tensors...) -> status
        self.fields = [f for f, _ in desc._fields_]
        self.tensors = []
        for t in tensors:
            label, kind, *dims = t.split()
            self.tensors.append((label.rstrip("?"), self._KINDS[kind], label.endswith("?"),
                                 [self._dim(d) for d in dims]))

    def _dim(self, text):
        """(field a or -1, field b or -1, divisor, addend) of a size."""
        if text.isdigit():
            return (-1, -1, 1, int(text))
        text, _, add = text.partition("+")
        text, _, div = text.partition("/")
        a, _, b = text.partition("*")
        at = self.fields.index
        return (at(a), at(b) if b else -1, int(div or 1), int(add or 0))

    def _first(self, *args):
        address = ctypes.cast(getattr(lib(), self.name), ctypes.c_void_p).value
        rows = self.fields.index(self.rows) if self.rows else -1
        m = _marshal()
        self.run = functools.partial(m.run, m.spec(
            address, len(self.fields), rows,
            [(kind, opt, dims) for _, kind, opt, dims in self.tensors]))
        return self.run(*args)

    def refuse(self, status, dsc, tensors):
        """Raise for a status, or for the tensor that is not as described."""
        if status > 0:
            raise BeamError(status, self.name)
        torch = _torch()
        f = [getattr(dsc, x) for x in self.fields]
        kinds = {_F32: torch.float32, _I32: torch.int32, _U8: torch.uint8,
                 _WORKSPACE: torch.uint8}
        if self.rows:
            kinds[_ROWS] = _torch_dtype(getattr(dsc, self.rows))
        for (_, kind, _, _), t in zip(self.tensors, tensors):
            if kind == _WORKSPACE and t is None:
                raise BeamError(3, f"{self.name}: the workspace is missing")
        for dev in (None, _current_device()):
            for (name, kind, opt, dims), t in zip(self.tensors, tensors):
                if kind == _WORKSPACE:
                    shape = t.shape
                else:
                    shape = tuple((0 if a < 0 else f[a]) * (1 if b < 0 else f[b]) // div + add
                                  for a, b, div, add in dims)
                _arg(self.name, name, t, kinds[kind], shape, dev, opt)
        raise BeamError(1, self.name)


def _alloc(what, n, device):
    if n == 0:
        raise BeamError(1, what)
    return _torch().empty(n, dtype=_torch().uint8, device=device or "cuda")


def _current_device():
    """Index of the current CUDA device.  Before CUDA is up no tensor can be on
    one: -2, which no tensor's get_device() gives."""
    torch = _torch()
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -2


# ------------------------------------------------- the residual block around --

_BLOCK_ENTER = _Entry("beam_block_enter", BlockDesc, "dtype", "x rows T d", "w rows d",
                      "n rows T d")
_BLOCK_EXIT = _Entry("beam_block_exit", BlockDesc, "dtype", "res rows T d", "y rows T d",
                     "w_out? rows d", "gate_c? rows d", "gate_t? rows T", "out rows T d",
                     "w_next? rows d", "n_next? rows T d")
_BLOCK_ENTER_BACKWARD = _Entry("beam_block_enter_backward", BlockDesc, "dtype", "x rows T d",
                               "w rows d", "dn f32 T d", "dskip? rows T d", "dx rows T d",
                               "dw f32 d", "workspace workspace")
_BLOCK_EXIT_BACKWARD = _Entry("beam_block_exit_backward", BlockDesc, "dtype", "y rows T d",
                              "out? rows T d", "w_out? rows d", "gate_c? rows d",
                              "gate_t? rows T", "w_next? rows d", "dout rows T d",
                              "dn_next? f32 T d", "dres rows T d", "dy rows T d", "dw_out? f32 d",
                              "dgate_c? f32 d", "dgate_t? f32 T", "dw_next? f32 d",
                              "workspace workspace")


def block_desc(T, d, dtype="bf16", eps=1e-6, res_scale=1.0, branch_scale=1.0,
               accumulate=False) -> BlockDesc:
    """T rows of width d around the layer; out = res_scale res + branch_scale
    (gated, normed y).  accumulate: the backward adds to the weights' gradients."""
    return BlockDesc(int(T), int(d), _code(dtype), float(eps), float(res_scale),
                     float(branch_scale), int(accumulate))


def block_workspace_size(dsc: BlockDesc) -> int:
    return int(lib().beam_block_workspace_size(ctypes.byref(dsc)))


def alloc_block_workspace(dsc: BlockDesc, device=None):
    """A uint8 torch tensor of block_workspace_size(dsc) bytes on `device`."""
    return _alloc("beam_block_workspace_size", block_workspace_size(dsc), device)


def block_enter(dsc, x, w, n, stream=None):
    """n = x r(x) w, r(x) = 1 / sqrt(mean x^2 + eps) per row: what the layer reads."""
    status = _BLOCK_ENTER.run(dsc, stream, x, w, n)
    if status:
        _BLOCK_ENTER.refuse(status, dsc, (x, w, n))


def block_exit(dsc, res, y, out, w_out=None, gate_c=None, gate_t=None, w_next=None, n_next=None,
               stream=None):
    """out = res_scale res + branch_scale sigmoid(gate_t) gate_c w_out y r(y)
    (each of w_out [d], gate_c [d], gate_t [T] may be left out; without w_out y
    is not normed); with w_next also n_next = out r(out) w_next."""
    if (w_next is None) != (n_next is None):
        raise BeamError(1, "beam_block_exit: w_next and n_next go together")
    status = _BLOCK_EXIT.run(dsc, stream, res, y, w_out, gate_c, gate_t, out, w_next, n_next)
    if status:
        _BLOCK_EXIT.refuse(status, dsc, (res, y, w_out, gate_c, gate_t, out, w_next, n_next))


def block_enter_backward(dsc, x, w, dn, dx, dw, workspace, dskip=None, stream=None):
    """dx = dskip + dn (f32, as backward's dx) through the norm; dw f32 [d]."""
    status = _BLOCK_ENTER_BACKWARD.run(dsc, stream, x, w, dn, dskip, dx, dw, workspace)
    if status:
        _BLOCK_ENTER_BACKWARD.refuse(status, dsc, (x, w, dn, dskip, dx, dw, workspace))


def block_exit_backward(dsc, y, dout, dres, dy, workspace, out=None, dn_next=None, w_out=None,
                        gate_c=None, gate_t=None, w_next=None, dw_out=None, dgate_c=None,
                        dgate_t=None, dw_next=None, stream=None):
    """Gradients of block_exit for dout and, with w_next, dn_next (f32): dres
    and dy in the rows' dtype, and in f32 that of each weight and gate that is
    given (dw_out, dgate_c, dw_next [d], dgate_t [T])."""
    if ((w_out is None) != (dw_out is None) or (gate_c is None) != (dgate_c is None)
            or (gate_t is None) != (dgate_t is None) or (w_next is None) != (dw_next is None)
            or (w_next is None) != (dn_next is None)):
        raise BeamError(1, "beam_block_exit_backward: a weight or gate and its gradient go together")
    status = _BLOCK_EXIT_BACKWARD.run(dsc, stream, y, out, w_out, gate_c, gate_t, w_next, dout,
                                      dn_next, dres, dy, dw_out, dgate_c, dgate_t, dw_next,
                                      workspace)
    if status:
        _BLOCK_EXIT_BACKWARD.refuse(status, dsc, (y, out, w_out, gate_c, gate_t, w_next, dout,
                                    dn_next, dres, dy, dw_out, dgate_c, dgate_t, dw_next,
                                    workspace))


# ------------------------------------------------------------ balance loss --

_BALANCE = _Entry("beam_moe_balance", BalanceDesc, None, "logits f32 T logits_ld",
                  "seq_begin? i32 n_seq+1", "loss f32 1", "cand_counts i32 n_seq E",
                  "kept_counts? i32 n_seq E", "mean_prob? f32 n_seq E", "workspace workspace")
_BALANCE_BACKWARD = _Entry("beam_moe_balance_backward", BalanceDesc, None,
                           "logits f32 T logits_ld", "seq_begin? i32 n_seq+1",
                           "counts i32 n_seq E", "dloss? f32 1", "dlogits f32 T E")


def balance_desc(T, E, K, n_seq=1, logits_ld=None, has_mask=False, count_kept=False, tau=0.5,
                 coef=1.0) -> BalanceDesc:
    """Balance loss over n_seq sequences of T tokens in all.  logits_ld: floats
    per row of the logits (default E, or 2 E with has_mask: route's)."""
    ld = (2 * E if has_mask else E) if logits_ld is None else logits_ld
    return BalanceDesc(int(T), int(E), int(K), int(n_seq), int(ld), int(has_mask),
                       int(count_kept), tau_logit(tau), float(coef))


def balance_workspace_size(dsc: BalanceDesc) -> int:
    return int(lib().beam_moe_balance_workspace_size(ctypes.byref(dsc)))


def alloc_balance_workspace(dsc: BalanceDesc, device=None):
    """A uint8 torch tensor of balance_workspace_size(dsc) bytes on `device`."""
    return _alloc("beam_moe_balance_workspace_size", balance_workspace_size(dsc), device)


def balance(dsc, logits, loss, cand_counts, workspace, kept_counts=None, mean_prob=None,
            seq_begin=None, stream=None):
    """loss f32 [1] = coef / n_seq sum_s sum_e f_se P_se from logits f32
    [T, logits_ld]; cand_counts (kept_counts) int32 [n_seq, E]: how many tokens
    of a sequence have (keep) expert e among their K candidates; mean_prob f32
    [n_seq, E] = P.  seq_begin int32 [n_seq + 1] (device)."""
    if kept_counts is not None and not dsc.has_mask:
        raise BeamError(1, "beam_moe_balance: kept_counts without a mask")
    status = _BALANCE.run(dsc, stream, logits, seq_begin, loss, cand_counts, kept_counts,
                          mean_prob, workspace)
    if status:
        _BALANCE.refuse(status, dsc, (logits, seq_begin, loss, cand_counts, kept_counts,
                        mean_prob, workspace))


def balance_backward(dsc, logits, counts, dlogits, seq_begin=None, dloss=None, stream=None):
    """dlogits f32 [T, E] of the balance loss, times dloss f32 [1] (device; 1 if
    left out).  counts: the forward's cand_counts, or kept_counts with
    count_kept.  backward(..., dlogits=) carries it on."""
    status = _BALANCE_BACKWARD.run(dsc, stream, logits, seq_begin, counts, dloss, dlogits)
    if status:
        _BALANCE_BACKWARD.refuse(status, dsc, (logits, seq_begin, counts, dloss, dlogits))


# ------------------------------------------- experts in 4-bit floating point --

_MX4_PRODUCT = _Entry("beam_mx4_expert_product", Mx4Desc, "out_dtype", "a_codes u8 N k/2",
                      "a_scales u8 N k/32", "counts i32 E", "w_codes u8 E*n k/2",
                      "w_scales u8 E*n k/32", "w3_codes? u8 E*n k/2", "w3_scales? u8 E*n k/32",
                      "out rows N n", "workspace workspace")


def _rows_call(name, quantize):
    """A call that finds its entry point when it first runs."""
    def first(*args):
        address = ctypes.cast(getattr(lib(), name), ctypes.c_void_p).value
        _rows_run[quantize] = functools.partial(_marshal().rows, address, quantize)
        return _rows_run[quantize](*args)
    return first


_rows_run = {True: _rows_call("beam_mx4_quantize", True),
             False: _rows_call("beam_mx4_dequantize", False)}


def _refuse_rows(what, status, x, codes, scales, n_rows):
    """Raise for a status, or for the tensor that is not as it has to be."""
    if status > 0:
        raise BeamError(status, what)
    torch = _torch()
    if x.dim() != 2 or x.dtype not in (torch.bfloat16, torch.float32):
        raise BeamError(1, f"{what}: a bf16 or f32 matrix is wanted, got {x.dtype} "
                           f"{tuple(x.shape)}")
    rows, cols = x.shape
    if cols % 32:
        raise BeamError(2, f"{what}: {cols} columns are no multiple of 32")
    for dev in (None, _current_device()):
        _arg(what, "values", x, x.dtype, (rows, cols), dev)
        _arg(what, "codes", codes, torch.uint8, (rows, cols // 2), dev)
        _arg(what, "scales", scales, torch.uint8, (rows, cols // 32), dev)
        _arg(what, "n_rows", n_rows, torch.int32, (1,), dev, True)
    raise BeamError(1, what)


def mx4_quantize(x, codes, scales, n_rows=None, tiled=False, stream=None):
    """x [rows, cols] (bf16 or f32) to MXFP4: codes uint8 [rows, cols / 2],
    scales uint8 [rows, cols / 32]; tiled: the scales in the tiles the product
    reads its weights' from.  n_rows: int32 [1] on the device, the rows that
    are there (the others are left as they are)."""
    status = _rows_run[True](x, codes, scales, n_rows, tiled, stream)
    if status:
        _refuse_rows("beam_mx4_quantize", status, x, codes, scales, n_rows)


def mx4_dequantize(codes, scales, out, tiled=False, stream=None):
    """The values of an MXFP4 matrix, out [rows, cols] bf16 or f32."""
    status = _rows_run[False](out, codes, scales, None, tiled, stream)
    if status:
        _refuse_rows("beam_mx4_dequantize", status, out, codes, scales, None)


def mx4_desc(N, E, n, k, swiglu=False, out="bf16") -> Mx4Desc:
    """One grouped projection: capacity of N token rows of width k, E experts
    of n weight rows; swiglu: gate and up; out: the output's dtype."""
    return Mx4Desc(int(N), int(E), int(n), int(k), int(swiglu), _code(out))


def mx4_workspace_size(dsc: Mx4Desc) -> int:
    return int(lib().beam_mx4_workspace_size(ctypes.byref(dsc)))


def alloc_mx4_workspace(dsc: Mx4Desc, device=None):
    """A uint8 torch tensor of mx4_workspace_size(dsc) bytes on `device`."""
    return _alloc("beam_mx4_workspace_size", mx4_workspace_size(dsc), device).zero_()


def mx4_expert_product(dsc, a_codes, a_scales, counts, w_codes, w_scales, out, workspace,
                       w3_codes=None, w3_scales=None, stream=None):
    """out[i] = a_i w_e^T for the rows i of expert e (grouped by expert, counts
    int32 [E] on the device), or SiLU(a_i w_e^T) * (a_i w3_e^T) when
    dsc.swiglu.  w_scales, w3_scales: tiled (mx4_quantize(..., tiled=True))."""
    if not dsc.swiglu and (w3_codes is not None or w3_scales is not None):
        raise BeamError(1, "beam_mx4_expert_product: a second weight without swiglu")
    status = _MX4_PRODUCT.run(dsc, stream, a_codes, a_scales, counts, w_codes, w_scales, w3_codes,
                              w3_scales, out, workspace)
    if status:
        _MX4_PRODUCT.refuse(status, dsc, (a_codes, a_scales, counts, w_codes, w_scales, w3_codes,
                            w3_scales, out, workspace))


def mx4_check(dsc, workspace, stream=None):
    """Synchronise and read the status of the last product on `workspace`."""
    _ok(lib().beam_mx4_check(ctypes.byref(dsc), _ptr(workspace), _stream(stream)),
        "beam_mx4_check")


def check(dsc, workspace, stream=None):
    _ok(lib().beam_moe_check(ctypes.byref(dsc), _ptr(workspace), _stream(stream)),
        "beam_moe_check")


def workspace_views(dsc, workspace) -> dict:
    """Typed views of the intermediate arrays inside a forward workspace."""
    import torch
    P = plan(dsc)
    T, K, E = dsc.T, dsc.K, dsc.E
    dt = torch.bfloat16 if dsc.dtype == BEAM_BF16 else torch.float32
    es = 2 if dsc.dtype == BEAM_BF16 else 4

    def view(off, n, dtype, size):
        return workspace[off: off + n * size].view(dtype)

    return dict(
        err=view(P["off_err"], 1, torch.int32, 4),
        meta=view(P["off_meta"], 4, torch.int32, 4),
        counts=view(P["off_counts"], E, torch.int32, 4),
        hist=view(P["off_hist"], K + 1, torch.int32, 4),
        partial=view(P["off_partial"], P["router_splits"] * T * 2 * E, torch.float32, 4).view(
            P["router_splits"], T, 2 * E),
        idx=view(P["off_idx"], T * K, torch.int32, 4).view(T, K),
        w=view(P["off_w"], T * K, torch.float32, 4).view(T, K),
        pair=view(P["off_pair"], P["p_cap"], torch.int32, 4),
        pair_pos=view(P["off_pair_pos"], T * K, torch.int32, 4).view(T, K),
        tiles=view(P["off_tiles"], 4 * P["tiles_cap"], torch.int32, 4).view(-1, 4),
        xp=view(P["off_xp"], P["p_cap"] * dsc.d, dt, es).view(P["p_cap"], dsc.d),
        h=view(P["off_h"], P["p_cap"] * dsc.I, dt, es).view(P["p_cap"], dsc.I),
        y=view(P["off_y"], P["p_cap"] * dsc.d, torch.float32, 4).view(P["p_cap"], dsc.d),
        ys=view(P["off_ys"], max(1, P["sh_split2"]) * dsc.n_shared * T * dsc.d, torch.float32,
                4).view(max(1, P["sh_split2"]) * dsc.n_shared * T, dsc.d),
        plan=P,
    )
