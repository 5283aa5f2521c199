"""Thin ctypes binding of libcgtp (include/cgtp.h): same names, argument marshalling only.

Every step runs in the library's HIP kernels.  Torch supplies device memory
and the stream (``torch.cuda.current_stream().cuda_stream``); when an output
tensor is not given, it is allocated here with ``torch.empty`` -- the only
allocation on the path, and one the library itself never makes.  If
``libcgtp.so`` is missing the first call raises: there is no fallback.

The block and optimizer calls (norm, join, AdamW) go through a small compiled module
(``csrc/torch/calls.cpp``) when their outputs are all new: the same checks, outputs and entry points
at half the cost of a call.  What it does not take comes back here.
"""
import ctypes
import os
from functools import lru_cache

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcgtp.so")

CGTP_UVU, CGTP_UVW = 0, 1
CGTP_F32, CGTP_F64, CGTP_BF16, CGTP_F16 = 0, 1, 2, 3
DTYPES = {"f32": CGTP_F32, "f64": CGTP_F64, "bf16": CGTP_BF16, "f16": CGTP_F16}
GATES = {None: 0, "row": 1, "channel": 2}
ACTS = {"identity": 0, "sigmoid": 1, "silu": 2, "tanh": 3}
STATUS = {0: "CGTP_OK", 1: "CGTP_ERR_INVALID_ARG", 2: "CGTP_ERR_IRREPS", 3: "CGTP_ERR_UNSUPPORTED",
          4: "CGTP_ERR_COMPILE", 5: "CGTP_ERR_HIP", 6: "CGTP_ERR_INTERNAL"}
STATUS_CODES = {v: k for k, v in STATUS.items()}

EXPORTS = ("cgtp_plan_create", "cgtp_plan_destroy", "cgtp_plan_info_get", "cgtp_plan_path",
           "cgtp_plan_path_coefficients", "cgtp_plan_source", "cgtp_tp_forward", "cgtp_conv_forward",
           "cgtp_graph_transpose", "cgtp_conv_backward", "cgtp_spherical_harmonics", "cgtp_last_error",
           "cgtp_conv_forward_ordered", "cgtp_graph_order", "cgtp_conv_double_backward", "cgtp_tp_backward",
           "cgtp_conv_forward_radial", "cgtp_plan_radial_prepare", "cgtp_plan_radial_source",
           "cgtp_tp_backward_workspace_size", "cgtp_plan_uvw_backward_prepare", "cgtp_plan_uvw_backward_source",
           "cgtp_conv_backward_workspace_size", "cgtp_conv_backward_ws", "cgtp_plan_conv_uvw_backward_prepare",
           "cgtp_plan_conv_uvw_backward_source", "cgtp_conv_backward_radial", "cgtp_conv_backward_radial_workspace_size",
           "cgtp_conv_row_split", "cgtp_tp_backward_noalloc", "cgtp_conv_backward_receiver",
           "cgtp_conv_backward_receiver_workspace_size", "cgtp_conv_double_backward_workspace_size",
           "cgtp_conv_double_backward_ws",
           "cgtp_block_create", "cgtp_block_destroy", "cgtp_block_info_get", "cgtp_block_source",
           "cgtp_block_workspace_size", "cgtp_norm_forward", "cgtp_norm_backward", "cgtp_join_forward",
           "cgtp_join_backward", "cgtp_adamw_create", "cgtp_adamw_destroy", "cgtp_adamw_info_get", "cgtp_adamw_offset",
           "cgtp_grad_norm", "cgtp_adamw_step", "cgtp_adamw_schedule", "cgtp_adamw_schedule_norm",
           "cgtp_adamw_state_read", "cgtp_adamw_state_write")
_STRING_RESULTS = ("cgtp_last_error", "cgtp_plan_source", "cgtp_plan_radial_source", "cgtp_plan_uvw_backward_source",
                   "cgtp_plan_conv_uvw_backward_source", "cgtp_block_source")


class CgtpError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class PlanInfo(ctypes.Structure):
    _fields_ = [("d_x", ctypes.c_int32), ("d_sh", ctypes.c_int32), ("d_out", ctypes.c_int32),
                ("num_paths", ctypes.c_int32), ("weight_numel", ctypes.c_int64),
                ("nnz_total", ctypes.c_int32), ("mode", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("fwd_tasks", ctypes.c_int32)]


class PathInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("i1", "i2", "slot", "l1", "l2", "l3", "p3", "x_off", "y_off",
                                              "out_off", "mul_in", "mul_out")] + \
               [("w_off", ctypes.c_int64), ("nnz", ctypes.c_int32)]


class BlockConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "gate", "act", "post_norm", "next_norm")] + \
               [("eps", ctypes.c_double), ("alpha", ctypes.c_double)]


class BlockInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("d", "channels", "gate_width", "dtype", "lanes", "elements")]


class AdamWConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "state_bits", "master")]


class AdamWInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("elements", "blocks", "norm_workspace")] + [("n_tensors", ctypes.c_int32)]


class AdamWHyper(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay", "max_norm",
                                               "grad_scale")] + [("step", ctypes.c_int64)]


_lib = None


def lib():
    """Load libcgtp.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m clebsch_gordan_tensor_cgtp_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        L.cgtp_last_error.restype = ctypes.c_char_p
        L.cgtp_plan_source.restype = ctypes.c_char_p
        L.cgtp_plan_radial_source.restype = ctypes.c_char_p
        L.cgtp_plan_uvw_backward_source.restype = ctypes.c_char_p
        L.cgtp_plan_conv_uvw_backward_source.restype = ctypes.c_char_p
        L.cgtp_plan_conv_uvw_backward_source.argtypes = [vp, i32]
        L.cgtp_conv_backward_workspace_size.argtypes = [vp, i64, i64, ctypes.POINTER(ctypes.c_size_t)]
        L.cgtp_conv_backward_ws.argtypes = [vp, i64, i64] + [vp] * 14 + [ctypes.c_size_t, vp]
        L.cgtp_conv_backward_radial_workspace_size.argtypes = [vp, i64, i64, i32, ctypes.POINTER(ctypes.c_size_t)]
        L.cgtp_conv_backward_radial.argtypes = [vp, i64, i64] + [vp] * 7 + [i32] + [vp] * 8 + [ctypes.c_size_t, vp]
        L.cgtp_plan_source.argtypes = [vp]
        L.cgtp_conv_row_split.argtypes = [vp, i64, i64, i32, ctypes.POINTER(i32)]
        L.cgtp_plan_create.argtypes = [ctypes.c_char_p] * 3 + [ctypes.c_int, ctypes.c_int, ctypes.POINTER(vp)]
        L.cgtp_plan_destroy.argtypes = [vp]
        L.cgtp_plan_info_get.argtypes = [vp, ctypes.POINTER(PlanInfo)]
        L.cgtp_plan_path.argtypes = [vp, i32, ctypes.POINTER(PathInfo)]
        L.cgtp_plan_path_coefficients.argtypes = [vp, i32, i32, vp, vp, ctypes.POINTER(i32)]
        L.cgtp_tp_forward.argtypes = [vp, i64, vp, vp, vp, ctypes.c_int, vp, vp]
        L.cgtp_tp_backward.argtypes = [vp, i64, vp, vp, vp, ctypes.c_int, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.cgtp_tp_backward_noalloc.argtypes = [vp, i64, vp, vp, vp, ctypes.c_int, vp, vp, vp, vp, vp]
        L.cgtp_tp_backward_workspace_size.argtypes = [vp, i64, ctypes.POINTER(ctypes.c_size_t)]
        L.cgtp_conv_backward_receiver.argtypes = [vp, i64, i64] + [vp] * 12 + [ctypes.c_size_t, vp]
        L.cgtp_conv_backward_receiver_workspace_size.argtypes = [vp, i64, i64, ctypes.POINTER(ctypes.c_size_t),
                                                                 ctypes.POINTER(ctypes.c_size_t)]
        L.cgtp_plan_uvw_backward_prepare.argtypes = [vp]
        L.cgtp_plan_uvw_backward_source.argtypes = [vp]
        L.cgtp_plan_conv_uvw_backward_prepare.argtypes = [vp]
        L.cgtp_plan_radial_prepare.argtypes = [vp, i32]
        L.cgtp_plan_radial_source.argtypes = [vp, i32]
        L.cgtp_conv_forward_radial.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp]
        L.cgtp_conv_double_backward.argtypes = [vp, i64, i64] + [vp] * 18
        L.cgtp_conv_double_backward_workspace_size.argtypes = [vp, i64, i64, ctypes.POINTER(ctypes.c_size_t)]
        L.cgtp_conv_double_backward_ws.argtypes = [vp, i64, i64] + [vp] * 18 + [ctypes.c_size_t, vp]
        L.cgtp_conv_forward.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, vp, vp]
        L.cgtp_conv_forward_ordered.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp]
        L.cgtp_graph_order.argtypes = [i64, vp, vp, vp]
        L.cgtp_graph_transpose.argtypes = [i64, i64, vp, vp, vp, vp, vp, vp]
        L.cgtp_conv_backward.argtypes = [vp, i64, i64] + [vp] * 13
        L.cgtp_spherical_harmonics.argtypes = [i32, ctypes.c_int, i64, vp, vp, vp]
        sz, dbl, szp = ctypes.c_size_t, ctypes.c_double, ctypes.POINTER(ctypes.c_size_t)
        L.cgtp_block_source.restype = ctypes.c_char_p
        L.cgtp_block_source.argtypes = [vp]
        L.cgtp_block_create.argtypes = [ctypes.c_char_p, ctypes.POINTER(BlockConfig), ctypes.POINTER(vp)]
        L.cgtp_block_destroy.argtypes = [vp]
        L.cgtp_block_info_get.argtypes = [vp, ctypes.POINTER(BlockInfo)]
        L.cgtp_block_workspace_size.argtypes = [vp, i64, szp]
        L.cgtp_norm_forward.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp]
        L.cgtp_norm_backward.argtypes = [vp, i64, vp, i64] + [vp] * 7 + [sz, vp]
        L.cgtp_join_forward.argtypes = [vp, i64, vp, vp, i64, vp, i64] + [vp] * 8
        L.cgtp_join_backward.argtypes = [vp, i64, vp, vp, vp, vp, i64, vp, i64] + [vp] * 7 + [i64, vp, i64] + \
            [vp] * 4 + [sz, vp]
        L.cgtp_adamw_create.argtypes = [i32, vp, ctypes.POINTER(AdamWConfig), ctypes.POINTER(vp)]
        L.cgtp_adamw_destroy.argtypes = [vp]
        L.cgtp_adamw_info_get.argtypes = [vp, ctypes.POINTER(AdamWInfo)]
        L.cgtp_adamw_offset.argtypes = [vp, i32, ctypes.POINTER(i64)]
        L.cgtp_grad_norm.argtypes = [vp, vp, vp, vp, sz, vp]
        L.cgtp_adamw_step.argtypes = [vp] * 7 + [ctypes.POINTER(AdamWHyper), vp, vp, vp]
        L.cgtp_adamw_schedule.argtypes = [vp, dbl, dbl, vp]
        L.cgtp_adamw_schedule_norm.argtypes = [vp, dbl, dbl, vp, dbl, vp]
        L.cgtp_adamw_state_read.argtypes = [vp] * 7
        L.cgtp_adamw_state_write.argtypes = [vp] * 7
        for name in EXPORTS:
            if name not in _STRING_RESULTS:
                getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


_compiled = None


def _calls():
    """The compiled calls (csrc/torch/calls.cpp): checks, new outputs and the entry point of the block
    and optimizer calls (raises if they have not been built)."""
    global _compiled
    if _compiled is None:
        import torch  # noqa: F401  (whose libraries the module links)
        lib()
        try:
            from . import _calls as module
        except ImportError as e:
            raise ImportError(f"{HERE}/_calls.so is missing or does not load ({e}): "
                              "run `python -m clebsch_gordan_tensor_cgtp_amd.build`") from e
        _compiled = module
    return _compiled


def last_error() -> str:
    return lib().cgtp_last_error().decode()


def _check(status):
    if status != 0:
        raise CgtpError(status, last_error())


def _answer(got):
    """What a compiled call returns: its outputs, or the status of a failure."""
    if type(got) is int:
        _check(got)
    return got


# ------------------------------------------------------------------------------------ plans

class Plan:
    def __init__(self, in_irreps, sh_irreps, out_irreps, mode="uvu", dtype="f32"):
        self._h = None
        self.mode, self.dtype = mode, dtype
        self.irreps = (in_irreps, sh_irreps, out_irreps)
        h = ctypes.c_void_p()
        _check(lib().cgtp_plan_create(in_irreps.encode(), sh_irreps.encode(), out_irreps.encode(),
                                      {"uvu": CGTP_UVU, "uvw": CGTP_UVW}[mode],
                                      {"f32": CGTP_F32, "f64": CGTP_F64}[dtype], ctypes.byref(h)))
        self._h = h
        info = PlanInfo()
        _check(lib().cgtp_plan_info_get(h, ctypes.byref(info)))
        self.info = info
        self.d_x, self.d_sh, self.d_out = info.d_x, info.d_sh, info.d_out
        self.num_paths, self.weight_numel, self.nnz_total = info.num_paths, info.weight_numel, info.nnz_total

    @property
    def handle(self):
        return self._h

    @property
    def wide_uvw(self) -> bool:
        """A uvw plan with a multiplicity above 16: its batched backward runs the uvw convolution
        backward on the identity graph (computed once per plan)."""
        if not hasattr(self, "_wide_uvw"):
            self._wide_uvw = self.mode == "uvw" and any(
                max(self.path(p)["mul_in"], self.path(p)["mul_out"]) > 16 for p in range(self.num_paths))
        return self._wide_uvw

    @property
    def torch_dtype(self):
        import torch
        return torch.float32 if self.dtype == "f32" else torch.float64

    def path(self, p: int) -> dict:
        pi = PathInfo()
        _check(lib().cgtp_plan_path(self._h, p, ctypes.byref(pi)))
        return {f: getattr(pi, f) for f, _ in PathInfo._fields_}

    def coefficients(self, p: int):
        """(ijk int32 [nnz,3], values float64 [nnz]) of path p, as the planner computed them."""
        import numpy as np
        n = ctypes.c_int32()
        _check(lib().cgtp_plan_path_coefficients(self._h, p, 0, None, None, ctypes.byref(n)))
        ijk = np.zeros((n.value, 3), dtype=np.int32)
        vals = np.zeros(n.value, dtype=np.float64)
        _check(lib().cgtp_plan_path_coefficients(self._h, p, n.value, ijk.ctypes.data, vals.ctypes.data,
                                                 ctypes.byref(n)))
        return ijk, vals

    def row_split(self, n_nodes: int, n_edges: int, double_backward: bool = False) -> int:
        """Waves per receiver row (1, 2 or 4) of the forward (or of the double backward's receiver
        pass) for a graph of this size; kernels of split rows carry the suffix _split2/_split4."""
        v = ctypes.c_int32()
        _check(lib().cgtp_conv_row_split(self._h, n_nodes, n_edges, 1 if double_backward else 0, ctypes.byref(v)))
        return v.value

    @property
    def source(self) -> str:
        return lib().cgtp_plan_source(self._h).decode()

    def uvw_backward_source(self) -> str:
        """Generate and compile the uvw batched-backward module (host only); its source."""
        _check(lib().cgtp_plan_uvw_backward_prepare(self._h))
        return lib().cgtp_plan_uvw_backward_source(self._h).decode()

    def conv_uvw_backward_source(self, module: int = 0) -> str:
        """Generate and compile the uvw convolution-backward modules (host only); the source of
        module 0 (G and dW kernels) or 1 (the unit-weight sender pass)."""
        _check(lib().cgtp_plan_conv_uvw_backward_prepare(self._h))
        return lib().cgtp_plan_conv_uvw_backward_source(self._h, module).decode()

    def radial_source(self, R: int) -> str:
        """Generate and compile the radial-projection module for R (host only); its source."""
        _check(lib().cgtp_plan_radial_prepare(self._h, R))
        return lib().cgtp_plan_radial_source(self._h, R).decode()

    def close(self):
        if self._h is not None and _lib is not None:
            lib().cgtp_plan_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def plan_create(in_irreps, sh_irreps, out_irreps, mode="uvu", dtype="f32") -> Plan:
    return Plan(in_irreps, sh_irreps, out_irreps, mode, dtype)


def sh_irreps(lmax: int) -> str:
    return "+".join(f"1x{l}{'e' if l % 2 == 0 else 'o'}" for l in range(lmax + 1))


def per_path_out_irreps(in_irreps: str, lmax_sh: int, lmax_out: int) -> str:
    """One output block per coupling path, in path order (string bookkeeping only)."""
    terms = []
    for term in in_irreps.replace(" ", "").split("+"):
        mul, lp = term.split("x")
        l1, p1 = int(lp[:-1]), (1 if lp[-1] == "e" else -1)
        for l2 in range(lmax_sh + 1):
            p3 = p1 * (1 if l2 % 2 == 0 else -1)
            for l3 in range(abs(l1 - l2), min(l1 + l2, lmax_out) + 1):
                terms.append(f"{mul}x{l3}{'e' if p3 == 1 else 'o'}")
    return "+".join(terms)


@lru_cache(maxsize=None)
def plan_for(spec, dtype="f32") -> Plan:
    """The plan of a workload from ``synth.WORKLOADS`` (cached per process)."""
    if hasattr(spec, "n_edges"):
        if spec.mode == "uvw":
            return Plan(spec.in_irreps, sh_irreps(spec.lmax_sh), spec.out_irreps, "uvw", dtype)
        out = per_path_out_irreps(spec.in_irreps, spec.lmax_sh, spec.lmax_out)
        return Plan(spec.in_irreps, sh_irreps(spec.lmax_sh), out, "uvu", dtype)
    if spec.mode == "uvu":
        out = per_path_out_irreps(spec.in_irreps, spec.lmax_sh, spec.lmax_sh)
        return Plan(spec.in_irreps, sh_irreps(spec.lmax_sh), out, "uvu", dtype)
    return Plan(spec.in_irreps, sh_irreps(spec.lmax_sh), spec.out_irreps, "uvw", dtype)


# ------------------------------------------------------------------------------------ calls

def _stream(stream, device=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, name, dtype=None, shape=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


def _ptr_or_null(t, name, dtype=None, shape=None):
    return ctypes.c_void_p(0) if t is None else _dev(t, name, dtype, shape)


def tp_forward(plan: Plan, x, y, w, out=None, stream=None):
    import torch
    B = x.shape[0]
    dt = plan.torch_dtype
    if out is None:
        out = torch.empty((B, plan.d_out), dtype=dt, device=x.device)
    shared = 1 if plan.mode == "uvw" else 0
    wshape = (plan.weight_numel,) if shared else (B, plan.weight_numel)
    _check(lib().cgtp_tp_forward(plan.handle, B, _dev(x, "x", dt, (B, plan.d_x)), _dev(y, "y", dt, (B, plan.d_sh)),
                                 _dev(w, "w", dt, wshape), shared, _dev(out, "out", dt, (B, plan.d_out)),
                                 _stream(stream, x.device)))
    return out


def tp_backward_workspace_size(plan: Plan, B: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().cgtp_tp_backward_workspace_size(plan.handle, B, ctypes.byref(n)))
    return n.value


def tp_backward(plan: Plan, x, y, w, grad_out, grad_x=None, grad_y=None, grad_w=None, need=(True, True, True),
                workspace=None, stream=None):
    """Batched product backward: returns (grad_x, grad_y, grad_w); entries not in ``need`` are None.
    uvu: per-row weights; uvw: shared weights (a workspace is allocated here unless given)."""
    import torch
    B = x.shape[0]
    dt = plan.torch_dtype
    dev = x.device
    shared = 1 if plan.mode == "uvw" else 0
    wshape = (plan.weight_numel,) if shared else (B, plan.weight_numel)
    shapes = ((B, plan.d_x), (B, plan.d_sh), wshape)
    res = [None if not nd else (torch.empty(sh, dtype=dt, device=dev) if o is None else o)
           for o, nd, sh in zip((grad_x, grad_y, grad_w), need, shapes)]
    # uvw with every multiplicity <= 16 needs the workspace for grad_w only; wider uvw plans run
    # the convolution backward on the identity graph, which needs it for every gradient
    wide = plan.wide_uvw
    wanted = res[2] is not None or (wide and any(r is not None for r in res))
    nbytes = tp_backward_workspace_size(plan, B) if wanted else 0
    if workspace is None and nbytes:
        es = 4 if plan.dtype == "f32" else 8
        workspace = torch.empty(-(-nbytes // es), dtype=dt, device=dev)
    ws = ctypes.c_void_p(0) if workspace is None else ctypes.c_void_p(workspace.data_ptr())
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().cgtp_tp_backward(plan.handle, B, _dev(x, "x", dt, shapes[0]), _dev(y, "y", dt, shapes[1]),
                                  _dev(w, "w", dt, wshape), shared, _dev(grad_out, "grad_out", dt, (B, plan.d_out)),
                                  *[_ptr_or_null(r, n, dt, sh) for r, n, sh in zip(res, ("grad_x", "grad_y", "grad_w"),
                                                                                   shapes)],
                                  ws, ctypes.c_size_t(wsb), _stream(stream, dev)))
    return tuple(res)


def tp_backward_noalloc(plan: Plan, x, y, w, grad_out, grad_x, grad_y, grad_w, stream=None):
    """cgtp_tp_backward_noalloc: the batched backward with its temporary memory in the library's
    fixed device scratch.  Every output (or None to skip it) is given by the caller; nothing is
    allocated here or in the library."""
    B = x.shape[0]
    dt = plan.torch_dtype
    shared = 1 if plan.mode == "uvw" else 0
    wshape = (plan.weight_numel,) if shared else (B, plan.weight_numel)
    shapes = ((B, plan.d_x), (B, plan.d_sh), wshape)
    _check(lib().cgtp_tp_backward_noalloc(
        plan.handle, B, _dev(x, "x", dt, shapes[0]), _dev(y, "y", dt, shapes[1]), _dev(w, "w", dt, wshape), shared,
        _dev(grad_out, "grad_out", dt, (B, plan.d_out)),
        *[_ptr_or_null(r, n, dt, sh) for r, n, sh in zip((grad_x, grad_y, grad_w), ("grad_x", "grad_y", "grad_w"),
                                                         shapes)], _stream(stream, x.device)))
    return grad_x, grad_y, grad_w


def graph_order(row_ptr, order=None, stream=None):
    """Heavy-first receiver schedule (stable by log2 degree bucket, descending)."""
    import torch
    N = row_ptr.shape[0] - 1
    order = torch.empty(N, dtype=torch.int32, device=row_ptr.device) if order is None else order
    _check(lib().cgtp_graph_order(N, _dev(row_ptr, "row_ptr", torch.int32), _dev(order, "order", torch.int32, (N,)),
                                  _stream(stream, row_ptr.device)))
    return order


def conv_forward(plan: Plan, row_ptr, col, x, y, w, out=None, order=None, stream=None):
    import torch
    N, E = row_ptr.shape[0] - 1, col.shape[0]
    dt = plan.torch_dtype
    if out is None:
        out = torch.empty((N, plan.d_out), dtype=dt, device=x.device)
    wshape = (plan.weight_numel,) if plan.mode == "uvw" else (E, plan.weight_numel)  # uvw: shared weights
    _check(lib().cgtp_conv_forward_ordered(plan.handle, N, E, _dev(row_ptr, "row_ptr", torch.int32),
                                   _dev(col, "col", torch.int32), _ptr_or_null(order, "order", torch.int32, (N,)),
                                   _dev(x, "x", dt, (N, plan.d_x)),
                                   _dev(y, "y", dt, (E, plan.d_sh)), _dev(w, "w", dt, wshape),
                                   _dev(out, "out", dt, (N, plan.d_out)), _stream(stream, x.device)))
    return out


def conv_forward_radial(plan: Plan, row_ptr, col, x, y, rho, theta, out=None, order=None, stream=None):
    """Convolution with W_e = rho[e] @ theta built in the kernel (rho [E][R], theta [R][weight_numel])."""
    import torch
    N, E = row_ptr.shape[0] - 1, col.shape[0]
    R = theta.shape[0]
    dt = plan.torch_dtype
    if out is None:
        out = torch.empty((N, plan.d_out), dtype=dt, device=x.device)
    _check(lib().cgtp_conv_forward_radial(plan.handle, N, E, _dev(row_ptr, "row_ptr", torch.int32),
                                          _dev(col, "col", torch.int32), _ptr_or_null(order, "order", torch.int32, (N,)),
                                          _dev(x, "x", dt, (N, plan.d_x)), _dev(y, "y", dt, (E, plan.d_sh)), R,
                                          _dev(rho, "rho", dt, (E, R)), _dev(theta, "theta", dt, (R, plan.weight_numel)),
                                          _dev(out, "out", dt, (N, plan.d_out)), _stream(stream, x.device)))
    return out


def conv_backward_radial_workspace_size(plan: Plan, N: int, E: int, R: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().cgtp_conv_backward_radial_workspace_size(plan.handle, N, E, R, ctypes.byref(n)))
    return n.value


def conv_backward_radial(plan: Plan, row_ptr, col, transpose, x, y, rho, theta, grad_out, outs=(None, None, None, None),
                         need=(True, True, True, True), workspace=None, stream=None):
    """Backward of the radial-projection convolution: (grad_x, grad_y, grad_rho, grad_theta); entries
    not in ``need`` are None and not computed.  The workspace (uvu: dTheta partials; uvw: those,
    G and two SH-sized rows per edge) is allocated here unless given."""
    import torch
    N, E = row_ptr.shape[0] - 1, col.shape[0]
    R = theta.shape[0]
    dt = plan.torch_dtype
    dev = x.device
    shapes = ((N, plan.d_x), (E, plan.d_sh), (E, R), (R, plan.weight_numel))
    res = [None if not nd else (torch.empty(sh, dtype=dt, device=dev) if o is None else o)
           for o, nd, sh in zip(outs, need, shapes)]
    nbytes = conv_backward_radial_workspace_size(plan, N, E, R) if res[3] is not None or plan.mode == "uvw" else 0
    if workspace is None and nbytes:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    ws = ctypes.c_void_p(0) if workspace is None else ctypes.c_void_p(workspace.data_ptr())
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    t_row_ptr, t_edge, t_dst = transpose
    names = ("grad_x", "grad_y", "grad_rho", "grad_theta")
    _check(lib().cgtp_conv_backward_radial(
        plan.handle, N, E, _dev(row_ptr, "row_ptr", torch.int32), _dev(col, "col", torch.int32),
        _dev(t_row_ptr, "t_row_ptr", torch.int32, (N + 1,)), _dev(t_edge, "t_edge", torch.int32, (E,)),
        _dev(t_dst, "t_dst", torch.int32, (E,)), _dev(x, "x", dt, (N, plan.d_x)), _dev(y, "y", dt, (E, plan.d_sh)), R,
        _dev(rho, "rho", dt, (E, R)), _dev(theta, "theta", dt, (R, plan.weight_numel)),
        _dev(grad_out, "grad_out", dt, (N, plan.d_out)),
        *[_ptr_or_null(r, nm, dt, sh) for r, nm, sh in zip(res, names, shapes)],
        ws, ctypes.c_size_t(wsb), _stream(stream, dev)))
    return tuple(res)


def graph_transpose(row_ptr, col, t_row_ptr=None, t_edge=None, t_dst=None, stream=None):
    import torch
    N, E = row_ptr.shape[0] - 1, col.shape[0]
    dev = row_ptr.device
    t_row_ptr = torch.empty(N + 1, dtype=torch.int32, device=dev) if t_row_ptr is None else t_row_ptr
    t_edge = torch.empty(E, dtype=torch.int32, device=dev) if t_edge is None else t_edge
    t_dst = torch.empty(E, dtype=torch.int32, device=dev) if t_dst is None else t_dst
    _check(lib().cgtp_graph_transpose(N, E, _dev(row_ptr, "row_ptr", torch.int32), _dev(col, "col", torch.int32),
                                      _dev(t_row_ptr, "t_row_ptr", torch.int32, (N + 1,)),
                                      _dev(t_edge, "t_edge", torch.int32, (E,)),
                                      _dev(t_dst, "t_dst", torch.int32, (E,)), _stream(stream, dev)))
    return t_row_ptr, t_edge, t_dst


def conv_backward_workspace_size(plan: Plan, N: int, E: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().cgtp_conv_backward_workspace_size(plan.handle, N, E, ctypes.byref(n)))
    return n.value


def conv_backward(plan: Plan, row_ptr, col, transpose, x, y, w, grad_out, grad_x=None, grad_y=None, grad_w=None,
                  need=(True, True, True), order=None, workspace=None, stream=None):
    """Returns (grad_x, grad_y, grad_w); entries not in ``need`` are None and not computed.
    uvw plans: shared weights, a workspace (allocated here unless given) and an optional
    receiver schedule ``order`` for the weight-gradient pass."""
    import torch
    N, E = row_ptr.shape[0] - 1, col.shape[0]
    dt = plan.torch_dtype
    dev = x.device
    t_row_ptr, t_edge, t_dst = transpose
    uvw = plan.mode == "uvw"
    wshape = (plan.weight_numel,) if uvw else (E, plan.weight_numel)
    if need[0] and grad_x is None:
        grad_x = torch.empty((N, plan.d_x), dtype=dt, device=dev)
    if need[1] and grad_y is None:
        grad_y = torch.empty((E, plan.d_sh), dtype=dt, device=dev)
    if need[2] and grad_w is None:
        grad_w = torch.empty(wshape, dtype=dt, device=dev)
    gx = grad_x if need[0] else None
    gy = grad_y if need[1] else None
    gw = grad_w if need[2] else None
    if uvw:
        nbytes = conv_backward_workspace_size(plan, N, E)
        if workspace is None and nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        ws = ctypes.c_void_p(0) if workspace is None else ctypes.c_void_p(workspace.data_ptr())
        wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(lib().cgtp_conv_backward_ws(
            plan.handle, N, E, _dev(row_ptr, "row_ptr", torch.int32), _dev(col, "col", torch.int32),
            _ptr_or_null(order, "order", torch.int32, (N,)),
            _dev(t_row_ptr, "t_row_ptr", torch.int32, (N + 1,)), _dev(t_edge, "t_edge", torch.int32, (E,)),
            _dev(t_dst, "t_dst", torch.int32, (E,)), _dev(x, "x", dt, (N, plan.d_x)),
            _dev(y, "y", dt, (E, plan.d_sh)), _dev(w, "w", dt, wshape), _dev(grad_out, "grad_out", dt, (N, plan.d_out)),
            _ptr_or_null(gx, "grad_x", dt, (N, plan.d_x)), _ptr_or_null(gy, "grad_y", dt, (E, plan.d_sh)),
            _ptr_or_null(gw, "grad_w", dt, wshape), ws, ctypes.c_size_t(wsb), _stream(stream, dev)))
        return gx, gy, gw
    _check(lib().cgtp_conv_backward(
        plan.handle, N, E, _dev(row_ptr, "row_ptr", torch.int32), _dev(col, "col", torch.int32),
        _dev(t_row_ptr, "t_row_ptr", torch.int32, (N + 1,)), _dev(t_edge, "t_edge", torch.int32, (E,)),
        _dev(t_dst, "t_dst", torch.int32, (E,)), _dev(x, "x", dt, (N, plan.d_x)), _dev(y, "y", dt, (E, plan.d_sh)),
        _dev(w, "w", dt, (E, plan.weight_numel)), _dev(grad_out, "grad_out", dt, (N, plan.d_out)),
        _ptr_or_null(gx, "grad_x", dt, (N, plan.d_x)), _ptr_or_null(gy, "grad_y", dt, (E, plan.d_sh)),
        _ptr_or_null(gw, "grad_w", dt, (E, plan.weight_numel)), _stream(stream, dev)))
    return gx, gy, gw


def conv_backward_receiver_workspace_size(plan: Plan, N: int, E: int):
    """(bytes for one edge range holding every edge, the least workspace the call accepts)."""
    full, least = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().cgtp_conv_backward_receiver_workspace_size(plan.handle, N, E, ctypes.byref(full), ctypes.byref(least)))
    return full.value, least.value


def conv_backward_receiver(plan: Plan, row_ptr, col, transpose, x, y, w, grad_out, grad_x=None, grad_y=None,
                           grad_w=None, need=(True, True, True), workspace=None, stream=None):
    """The convolution backward in receiver order (cgtp_conv_backward_receiver): returns (grad_x,
    grad_y, grad_w); entries not in ``need`` are None and not computed.  grad_x needs a workspace
    (uint8 device tensor); the edges are taken in ranges of as many dx rows as it holds.  One that
    holds every edge is allocated here unless given."""
    import torch
    N, E = row_ptr.shape[0] - 1, col.shape[0]
    dt = plan.torch_dtype
    dev = x.device
    t_row_ptr, t_edge, _ = transpose
    if need[0] and grad_x is None:
        grad_x = torch.empty((N, plan.d_x), dtype=dt, device=dev)
    if need[1] and grad_y is None:
        grad_y = torch.empty((E, plan.d_sh), dtype=dt, device=dev)
    if need[2] and grad_w is None:
        grad_w = torch.empty((E, plan.weight_numel), dtype=dt, device=dev)
    gx = grad_x if need[0] else None
    gy = grad_y if need[1] else None
    gw = grad_w if need[2] else None
    if gx is not None and workspace is None and E > 0:
        workspace = torch.empty(conv_backward_receiver_workspace_size(plan, N, E)[0], dtype=torch.uint8, device=dev)
    ws = ctypes.c_void_p(0) if workspace is None else ctypes.c_void_p(workspace.data_ptr())
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().cgtp_conv_backward_receiver(
        plan.handle, N, E, _dev(row_ptr, "row_ptr", torch.int32), _dev(col, "col", torch.int32),
        _dev(t_row_ptr, "t_row_ptr", torch.int32, (N + 1,)), _dev(t_edge, "t_edge", torch.int32, (E,)),
        _dev(x, "x", dt, (N, plan.d_x)), _dev(y, "y", dt, (E, plan.d_sh)), _dev(w, "w", dt, (E, plan.weight_numel)),
        _dev(grad_out, "grad_out", dt, (N, plan.d_out)), _ptr_or_null(gx, "grad_x", dt, (N, plan.d_x)),
        _ptr_or_null(gy, "grad_y", dt, (E, plan.d_sh)), _ptr_or_null(gw, "grad_w", dt, (E, plan.weight_numel)),
        ws, ctypes.c_size_t(wsb), _stream(stream, dev)))
    return gx, gy, gw


def conv_double_backward_workspace_size(plan: Plan, N: int, E: int) -> int:
    n = ctypes.c_size_t()
    _check(lib().cgtp_conv_double_backward_workspace_size(plan.handle, N, E, ctypes.byref(n)))
    return n.value


def conv_double_backward(plan: Plan, row_ptr, col, transpose, x, y, w, grad_out, gg_x, gg_y, gg_w, order=None,
                         outs=(None, None, None, None), need=(True, True, True, True), workspace=None, stream=None):
    """Second-order gradients (grad_x, grad_y, grad_w, grad_grad_out) of
    <gg_x, dx> + <gg_y, dy> + <gg_w, dW>, where (dx, dy, dW) = conv_backward(x, y, w, grad_out).
    An upstream gradient given as None is passed as zeros.  Entries not in ``need`` are None
    and not computed.  uvw plans (shared weights) run cgtp_conv_double_backward_ws with a
    workspace, allocated here unless given."""
    import torch
    N, E = row_ptr.shape[0] - 1, col.shape[0]
    dt = plan.torch_dtype
    dev = x.device
    wshape = (plan.weight_numel,) if plan.mode == "uvw" else (E, plan.weight_numel)
    shapes = ((N, plan.d_x), (E, plan.d_sh), wshape, (N, plan.d_out))
    gg = [torch.zeros(sh, dtype=dt, device=dev) if t is None else t for t, sh in zip((gg_x, gg_y, gg_w), shapes)]
    res = [None if not nd else (torch.empty(sh, dtype=dt, device=dev) if o is None else o)
           for o, nd, sh in zip(outs, need, shapes)]
    t_row_ptr, t_edge, t_dst = transpose
    names = ("grad_x", "grad_y", "grad_w", "grad_grad_out")
    if plan.mode == "uvw":
        nbytes = conv_double_backward_workspace_size(plan, N, E)
        if workspace is None and nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        ws = ctypes.c_void_p(0) if workspace is None else ctypes.c_void_p(workspace.data_ptr())
        wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(lib().cgtp_conv_double_backward_ws(
            plan.handle, N, E, _dev(row_ptr, "row_ptr", torch.int32), _dev(col, "col", torch.int32),
            _ptr_or_null(order, "order", torch.int32, (N,)),
            _dev(t_row_ptr, "t_row_ptr", torch.int32, (N + 1,)), _dev(t_edge, "t_edge", torch.int32, (E,)),
            _dev(t_dst, "t_dst", torch.int32, (E,)), _dev(x, "x", dt, shapes[0]), _dev(y, "y", dt, shapes[1]),
            _dev(w, "w", dt, shapes[2]), _dev(grad_out, "grad_out", dt, shapes[3]),
            _dev(gg[0], "gg_x", dt, shapes[0]), _dev(gg[1], "gg_y", dt, shapes[1]), _dev(gg[2], "gg_w", dt, shapes[2]),
            *[_ptr_or_null(r, nm, dt, sh) for r, nm, sh in zip(res, names, shapes)], ws, ctypes.c_size_t(wsb),
            _stream(stream, dev)))
        return tuple(res)
    _check(lib().cgtp_conv_double_backward(
        plan.handle, N, E, _dev(row_ptr, "row_ptr", torch.int32), _dev(col, "col", torch.int32),
        _ptr_or_null(order, "order", torch.int32, (N,)),
        _dev(t_row_ptr, "t_row_ptr", torch.int32, (N + 1,)), _dev(t_edge, "t_edge", torch.int32, (E,)),
        _dev(t_dst, "t_dst", torch.int32, (E,)), _dev(x, "x", dt, shapes[0]), _dev(y, "y", dt, shapes[1]),
        _dev(w, "w", dt, shapes[2]), _dev(grad_out, "grad_out", dt, shapes[3]),
        _dev(gg[0], "gg_x", dt, shapes[0]), _dev(gg[1], "gg_y", dt, shapes[1]), _dev(gg[2], "gg_w", dt, shapes[2]),
        *[_ptr_or_null(r, nm, dt, sh) for r, nm, sh in zip(res, names, shapes)], _stream(stream, dev)))
    return tuple(res)


def spherical_harmonics(lmax: int, vec, out=None, stream=None):
    import torch
    E = vec.shape[0]
    dt = vec.dtype
    if dt not in (torch.float32, torch.float64):
        raise TypeError("vec must be float32 or float64")
    if out is None:
        out = torch.empty((E, (lmax + 1) ** 2), dtype=dt, device=vec.device)
    _check(lib().cgtp_spherical_harmonics(lmax, CGTP_F64 if dt == torch.float64 else CGTP_F32, E,
                                          _dev(vec, "vec", dt, (E, 3)), _dev(out, "y", dt, (E, (lmax + 1) ** 2)),
                                          _stream(stream, vec.device)))
    return out


# ------------------------------------------------------------------------------------ blocks

def _torch_dtype(dtype: str):
    import torch
    return {"f32": torch.float32, "f64": torch.float64, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]


class Block:
    """The row norm at a block's entry and the join at its end (norm, gate, residual sum, the next
    block's norm) for one irreps row and configuration; compiled when it is created.  Like a Plan, it is
    closed (or dropped) only after the kernels launched with it have finished; block_for keeps it."""

    def __init__(self, irreps, dtype="f32", gate=None, act="sigmoid", post_norm=False, next_norm=False, eps=1e-6,
                 alpha=1.0):
        self._h = None
        self.irreps, self.dtype = irreps, dtype
        self.gate, self.act, self.post_norm, self.next_norm = gate, act, bool(post_norm), bool(next_norm)
        self.eps, self.alpha = float(eps), float(alpha)
        cfg = BlockConfig(DTYPES[dtype], GATES[gate], ACTS[act], int(self.post_norm), int(self.next_norm), self.eps,
                          self.alpha)
        h = ctypes.c_void_p()
        _check(lib().cgtp_block_create(irreps.encode(), ctypes.byref(cfg), ctypes.byref(h)))
        self._h = h
        info = BlockInfo()
        _check(lib().cgtp_block_info_get(h, ctypes.byref(info)))
        self.d, self.channels, self.gate_width = info.d, info.channels, info.gate_width
        self.lanes, self.lane_elements = info.lanes, info.elements
        self.torch_dtype = _torch_dtype(dtype)                              # of rows
        self.real_dtype = _torch_dtype("f64" if dtype == "f64" else "f32")  # of statistics and weights
        self._calls = _calls()
        self._meta = self._calls.block(h.value, self.d, self.channels, self.gate_width, self.post_norm, self.next_norm,
                                       DTYPES[dtype])

    @property
    def handle(self):
        return self._h

    @property
    def source(self) -> str:
        return lib().cgtp_block_source(self._h).decode()

    def close(self):
        self._meta = None
        if self._h is not None and _lib is not None:
            lib().cgtp_block_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


@lru_cache(maxsize=None)
def block_for(irreps, dtype="f32", gate=None, act="sigmoid", post_norm=False, next_norm=False, eps=1e-6,
              alpha=1.0) -> Block:
    """The block of a configuration (cached per process)."""
    return Block(irreps, dtype, gate, act, post_norm, next_norm, eps, alpha)


def _device_index(t, name):
    try:
        if t.is_cuda:
            return t.get_device()
    except AttributeError:
        pass
    raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")


_current_raw_stream = None


def _in_stream(stream, call, *args, **kw):
    """The call with `stream` as the current one, so that what it allocates belongs to that stream."""
    import torch
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def _current(index):
    """The tensors' device as the current one: launches go there, and a block's code is loaded there."""
    import torch
    return torch.cuda.device(index)


def _raw_stream(index):
    global _current_raw_stream
    if _current_raw_stream is None:
        import torch
        _current_raw_stream = torch._C._cuda_getCurrentRawStream
    return _current_raw_stream(index)


def _refuse(t, name, dtype, shape, index):
    """Raise what is wrong with a tensor that _addr did not take."""
    _dev(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _addr(t, name, dtype, shape, index):
    """Address of a contiguous tensor of this type, shape and device."""
    try:
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index:
            return t.data_ptr()
    except AttributeError:
        pass
    return _refuse(t, name, dtype, shape, index)


def _addr_or_null(t, name, dtype, shape, index):
    return None if t is None else _addr(t, name, dtype, shape, index)


def _rows(t, name, dtype, shape, index):
    """(address, row pitch) of n rows of `width` consecutive elements, any pitch of at least that."""
    n, width = shape
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index:
            ld, one = t.stride()
            if n <= 1:
                ld = width
            if ld >= width and (one == 1 or width <= 1):
                return t.data_ptr(), ld
    except AttributeError:
        pass
    _device_index(t, name)
    if t.dtype == dtype and tuple(t.shape) == tuple(shape) and t.get_device() == index:
        if width > 1 and t.stride(1) != 1:
            raise ValueError(f"{name}: the elements of a row must be consecutive")
        raise ValueError(f"{name}: rows overlap (row pitch {t.stride(0)} of {width} elements)")
    return _refuse(t.contiguous(), name, dtype, shape, index)


def _rows_or_null(t, name, dtype, shape, index):
    return (None, shape[1]) if t is None else _rows(t, name, dtype, shape, index)


def _output(t, wanted, name, dtype, shape, like, index):
    """(tensor, address) of an output: the caller's, or a new one where it is wanted."""
    if t is not None:
        return t, _addr(t, name, dtype, shape, index)
    if not wanted:
        return None, None
    t = like.new_empty(shape, dtype=dtype)
    return t, t.data_ptr()


def _row_output(t, wanted, name, dtype, shape, like, index):
    """(tensor, address, row pitch) of an output of rows."""
    if t is not None:
        return (t,) + _rows(t, name, dtype, shape, index)
    return _output(None, wanted, name, dtype, shape, like, index) + (shape[1],)


def block_workspace_size(block: Block, n: int) -> int:
    v = ctypes.c_size_t()
    _check(lib().cgtp_block_workspace_size(block.handle, n, ctypes.byref(v)))
    return v.value


def _workspace(t, name, nbytes, like, index):
    """(address, bytes, tensor) of the caller's workspace, or of a new one."""
    if t is None:
        import torch
        t = like.new_empty(nbytes, dtype=torch.uint8)
        return t.data_ptr(), nbytes, t
    return _addr(t, name, t.dtype, t.shape, index), t.numel() * t.element_size(), t


def norm_forward(block: Block, x, w, u=None, rstd=None, need_rstd=True, stream=None):
    """(u, rstd): u = x * rstd(x) * w per channel.  x may have a row pitch; w None stands for ones."""
    if u is None and rstd is None and stream is None:
        got = block._calls.norm_forward(block._meta, x, w, need_rstd)
        if got is not None:
            return _answer(got)
    if stream is not None:
        return _in_stream(stream, norm_forward, block, x, w, u, rstd, need_rstd)
    dev = _device_index(x, "x")
    n, dt, rt = x.shape[0], block.torch_dtype, block.real_dtype
    rows = (n, block.d)
    xp, x_ld = _rows(x, "x", dt, rows, dev)
    u, up = _output(u, True, "u", dt, rows, x, dev)
    rstd, rp = _output(rstd, need_rstd, "rstd", rt, (n,), x, dev)
    with _current(dev):
        _check(lib().cgtp_norm_forward(block.handle, n, xp, x_ld, _addr_or_null(w, "w", rt, (block.channels,), dev), up,
                                       rp, _raw_stream(dev)))
    return u, rstd


def norm_backward(block: Block, x, w, rstd, grad_u, grad_add=None, grad_x=None, grad_w=None, need=(True, True),
                  workspace=None, stream=None):
    """(grad_x, grad_w); entries not in ``need`` are None and not computed.  grad_add, when given,
    is added to grad_x (the gradient that reaches x past the norm)."""
    if grad_x is None and grad_w is None and workspace is None and stream is None:
        got = block._calls.norm_backward(block._meta, x, w, rstd, grad_u, grad_add, *need)
        if got is not None:
            return _answer(got)
    if stream is not None:
        return _in_stream(stream, norm_backward, block, x, w, rstd, grad_u, grad_add, grad_x, grad_w, need, workspace)
    dev = _device_index(x, "x")
    n, dt, rt, cs = x.shape[0], block.torch_dtype, block.real_dtype, (block.channels,)
    rows = (n, block.d)
    xp, x_ld = _rows(x, "x", dt, rows, dev)
    gx, gxp = _output(grad_x if need[0] else None, need[0], "grad_x", dt, rows, x, dev)
    gw, gwp = _output(grad_w if need[1] else None, need[1], "grad_w", rt, cs, x, dev)
    ws, ws_bytes = None, 0
    if gw is not None:
        ws, ws_bytes, workspace = _workspace(workspace, "workspace", block_workspace_size(block, n), x, dev)
    with _current(dev):
        _check(lib().cgtp_norm_backward(block.handle, n, xp, x_ld, _addr_or_null(w, "w", rt, cs, dev),
                                        _addr(rstd, "rstd", rt, (n,), dev), _addr(grad_u, "grad_u", dt, rows, dev),
                                        _addr_or_null(grad_add, "grad_add", dt, rows, dev), gxp, gwp, ws, ws_bytes,
                                        _raw_stream(dev)))
    return gx, gw


def join_forward(block: Block, res, f, gate, w_post, scale, w_next, h=None, u=None, rstd_f=None, rstd_h=None,
                 need_rstd=True, stream=None):
    """(h, u, rstd_f, rstd_h): h = alpha*res + scale*act(gate)*w_post*f*rstd(f), u = h*rstd(h)*w_next.
    f and gate may have a row pitch (both in one buffer, say); weights given as None are ones; what
    the block's configuration leaves out is None."""
    if h is None and u is None and rstd_f is None and rstd_h is None and stream is None:
        got = block._calls.join_forward(block._meta, res, f, gate, w_post, scale, w_next, need_rstd)
        if got is not None:
            return _answer(got)
    if stream is not None:
        return _in_stream(stream, join_forward, block, res, f, gate, w_post, scale, w_next, h, u, rstd_f, rstd_h, need_rstd)
    dev = _device_index(f, "f")
    n, dt, rt, cs = f.shape[0], block.torch_dtype, block.real_dtype, (block.channels,)
    rows, stat = (n, block.d), (n,)
    fp, f_ld = _rows(f, "f", dt, rows, dev)
    gp, g_ld = _rows_or_null(gate, "gate", dt, (n, block.gate_width), dev)
    h, hp = _output(h, True, "h", dt, rows, f, dev)
    u, up = _output(u, block.next_norm, "u", dt, rows, f, dev)
    rstd_f, rfp = _output(rstd_f, need_rstd and block.post_norm, "rstd_f", rt, stat, f, dev)
    rstd_h, rhp = _output(rstd_h, need_rstd and block.next_norm, "rstd_h", rt, stat, f, dev)
    with _current(dev):
        _check(lib().cgtp_join_forward(
            block.handle, n, _addr(res, "res", dt, rows, dev), fp, f_ld, gp, g_ld,
            _addr_or_null(w_post, "w_post", rt, cs, dev), _addr_or_null(scale, "scale", rt, cs, dev),
            _addr_or_null(w_next, "w_next", rt, cs, dev), hp, up, rfp, rhp, _raw_stream(dev)))
    return h, u, rstd_f, rstd_h


_NO_OUTS = (None,) * 6


def join_backward(block: Block, grad_h, grad_u, h, f, gate, w_post, scale, w_next, rstd_f, rstd_h,
                  outs=_NO_OUTS, need=(True,) * 6, workspace=None, stream=None):
    """(grad_res, grad_f, grad_gate, grad_w_post, grad_scale, grad_w_next) from the gradients of h
    (None: zero) and u and the forward's h and statistics; entries not in ``need``, or that the
    block's configuration leaves out, are None and not computed.  grad_f and grad_gate given in
    ``outs`` may have a row pitch."""
    if outs is _NO_OUTS and workspace is None and stream is None:
        got = block._calls.join_backward(block._meta, grad_h, grad_u, h, f, gate, w_post, scale, w_next, rstd_f, rstd_h,
                                         need)
        if got is not None:
            return _answer(got)
    if stream is not None:
        return _in_stream(stream, join_backward, block, grad_h, grad_u, h, f, gate, w_post, scale, w_next, rstd_f,
                          rstd_h, outs, need, workspace)
    dev = _device_index(f, "f")
    n, dt, rt, cs = f.shape[0], block.torch_dtype, block.real_dtype, (block.channels,)
    rows, gates, stat = (n, block.d), (n, block.gate_width), (n,)
    fp, f_ld = _rows(f, "f", dt, rows, dev)
    gp, g_ld = _rows_or_null(gate, "gate", dt, gates, dev)
    has_gate, post, nxt = block.gate_width > 0, block.post_norm, block.next_norm
    o0, o1, o2, o3, o4, o5 = [o if nd else None for o, nd in zip(outs, need)]
    gr, grp = _output(o0, need[0], "grad_res", dt, rows, f, dev)
    gf, gfp, gf_ld = _row_output(o1, need[1], "grad_f", dt, rows, f, dev)
    gg, ggp, gg_ld = _row_output(o2, need[2] and has_gate, "grad_gate", dt, gates, f, dev)
    gp3, g3 = _output(o3, need[3] and post, "grad_w_post", rt, cs, f, dev)
    gp4, g4 = _output(o4, need[4], "grad_scale", rt, cs, f, dev)
    gp5, g5 = _output(o5, need[5] and nxt, "grad_w_next", rt, cs, f, dev)
    ws, ws_bytes = None, 0
    if g3 is not None or g4 is not None or g5 is not None:
        ws, ws_bytes, workspace = _workspace(workspace, "workspace", block_workspace_size(block, n), f, dev)
    with _current(dev):
        _check(lib().cgtp_join_backward(
            block.handle, n, _addr_or_null(grad_h, "grad_h", dt, rows, dev),
            _addr_or_null(grad_u, "grad_u", dt, rows, dev), _addr_or_null(h, "h", dt, rows, dev), fp, f_ld, gp, g_ld, _addr_or_null(w_post, "w_post", rt, cs, dev),
            _addr_or_null(scale, "scale", rt, cs, dev), _addr_or_null(w_next, "w_next", rt, cs, dev),
            _addr_or_null(rstd_f, "rstd_f", rt, stat, dev), _addr_or_null(rstd_h, "rstd_h", rt, stat, dev),
            grp, gfp, gf_ld, ggp, gg_ld, g3, g4, g5, ws, ws_bytes, _raw_stream(dev)))
    return gr, gf, gg, gp3, gp4, gp5


# ------------------------------------------------------------------------------------ optimizer

class AdamW:
    """The layout of an AdamW step over tensors of these sizes (host only).  Moments are flat tensors
    of ``elements`` values, tensor t's at ``offsets[t]``; ``state`` makes them."""

    def __init__(self, sizes, dtype="f32", state_bits=32, master=False):
        self._h = None
        self.sizes, self.dtype, self.state_bits, self.master = tuple(int(n) for n in sizes), dtype, state_bits, master
        arr = (ctypes.c_int64 * max(1, len(self.sizes)))(*self.sizes)
        cfg = AdamWConfig(DTYPES[dtype], state_bits, int(bool(master)))
        h = ctypes.c_void_p()
        _check(lib().cgtp_adamw_create(len(self.sizes), arr, ctypes.byref(cfg), ctypes.byref(h)))
        self._h = h
        info = AdamWInfo()
        _check(lib().cgtp_adamw_info_get(h, ctypes.byref(info)))
        self.elements, self.blocks, self.norm_workspace = info.elements, info.blocks, info.norm_workspace
        self._offsets = None
        self.torch_dtype = _torch_dtype(dtype)
        self.real_dtype = _torch_dtype("f64" if dtype == "f64" else "f32")
        import torch
        self.moment_dtypes = (torch.int8, torch.uint8) if state_bits == 8 else (self.real_dtype, self.real_dtype)
        self._calls = _calls()
        self._meta = self._calls.adamw(h.value, self.sizes, self.elements, self.blocks, self.norm_workspace, state_bits,
                                       DTYPES[dtype])

    @property
    def handle(self):
        return self._h

    @property
    def offsets(self):
        if self._offsets is None:
            at, off = ctypes.c_int64(), []
            for t in range(len(self.sizes)):
                _check(lib().cgtp_adamw_offset(self._h, t, ctypes.byref(at)))
                off.append(at.value)
            self._offsets = tuple(off)
        return self._offsets

    def state(self, device, params=None):
        """(m, v, scales, master) at the start: zero moments, and master copies of ``params``."""
        import torch
        mt, vt = self.moment_dtypes
        m = torch.zeros(self.elements, dtype=mt, device=device)
        v = torch.zeros(self.elements, dtype=vt, device=device)
        scales = torch.zeros((2, self.blocks), device=device) if self.state_bits == 8 else None
        master = None
        if self.master:
            master = torch.zeros(self.elements, device=device)
            for p, at in zip(params, self.offsets):
                master[at:at + p.numel()].copy_(p.detach().reshape(-1))
        return m, v, scales, master

    def close(self):
        self._meta = None
        if self._h is not None and _lib is not None:
            lib().cgtp_adamw_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class TensorList:
    """Tensors of an AdamW layout (parameters or gradients, None where a gradient is absent), checked
    when they are listed and again at every use."""

    def __init__(self, opt: AdamW, tensors):
        self.opt, self.tensors = opt, tuple(tensors)
        if len(self.tensors) != len(opt.sizes):
            raise ValueError(f"{len(self.tensors)} tensors, the layout has {len(opt.sizes)}")
        self._given = [t for t in self.tensors if t is not None]
        self.device_index = _device_index(self._given[0], "tensor") if self._given else None
        if self._given and not opt._calls.takes_tensors(opt._meta, self.tensors):
            self.pointers()

    def pointers(self):
        """The tensors' addresses as the entry points take them."""
        for i, (t, n) in enumerate(zip(self.tensors, self.opt.sizes)):
            if t is None:
                continue
            _dev(t, f"tensor {i}", self.opt.torch_dtype)
            if t.numel() != n:
                raise ValueError(f"tensor {i} has {t.numel()} elements, the layout {n}")
            if t.get_device() != self.device_index:
                raise ValueError(f"tensor {i} is on {t.device}, expected cuda:{self.device_index}")
        at = [None if t is None else t.data_ptr() for t in self.tensors]
        return (ctypes.c_void_p * max(1, len(at)))(*at)


def tensor_list(opt: AdamW, tensors) -> TensorList:
    return TensorList(opt, tensors)


def _list(opt, tensors):
    if not isinstance(tensors, TensorList):
        return TensorList(opt, tensors)
    if tensors.opt is not opt:
        raise ValueError("the tensors were listed for another layout")
    return tensors


def _held(tensors):
    """A TensorList, or the tensors of any iterable, which may be read once only."""
    return tensors if isinstance(tensors, TensorList) else tuple(tensors)


def _tuple(opt, tensors):
    if not isinstance(tensors, TensorList):
        return tuple(tensors)
    if tensors.opt is not opt:
        raise ValueError("the tensors were listed for another layout")
    return tensors.tensors


def grad_norm(opt: AdamW, grads, norm=None, workspace=None, stream=None):
    """The global norm of the gradients (a TensorList or tensors; None ones are left out): a device
    float64 tensor of one element."""
    if stream is not None:
        return _in_stream(stream, grad_norm, opt, grads, norm, workspace)
    grads = _held(grads)
    if norm is None and workspace is None:
        got = opt._calls.grad_norm(opt._meta, _tuple(opt, grads))
        if got is not None:
            return _answer(got)[0]
    import torch
    grads = _list(opt, grads)
    dev = grads.device_index
    if dev is None:
        raise ValueError("there is no gradient")
    like = grads._given[0]
    norm = like.new_empty(1, dtype=torch.float64) if norm is None else norm
    ws, ws_bytes, workspace = _workspace(workspace, "workspace", opt.norm_workspace, like, dev)
    with _current(dev):
        _check(lib().cgtp_grad_norm(opt.handle, grads.pointers(), _addr(norm, "norm", torch.float64, (1,), dev), ws,
                                    ws_bytes, _raw_stream(dev)))
    return norm


def adamw_step(opt: AdamW, params, grads, m, v, scales=None, master=None, *, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
               weight_decay=0.01, step=0, max_norm=0.0, grad_scale=1.0, norm=None, schedule=None, stream=None):
    """One AdamW step in place: params, m, v (and scales, master).  ``step`` counts from 1; with
    ``norm`` (as of grad_norm) a step whose norm is not finite changes nothing, and max_norm > 0
    clips by it.  ``schedule``: a device float64 tensor {step, lr, 1 - beta1^step, 1 - beta2^step}
    in the place of ``step`` and ``lr`` (adamw_schedule advances it; where steps may be skipped, give it
    the same ``norm`` and ``grad_scale``)."""
    if stream is not None:
        return _in_stream(stream, adamw_step, opt, params, grads, m, v, scales, master, lr=lr, beta1=beta1, beta2=beta2,
                          eps=eps, weight_decay=weight_decay, step=step, max_norm=max_norm, grad_scale=grad_scale,
                          norm=norm, schedule=schedule)
    params, grads = _held(params), _held(grads)
    got = opt._calls.adamw_step(opt._meta, _tuple(opt, params), _tuple(opt, grads), m, v, scales, master, norm,
                                schedule, step, lr, beta1, beta2, eps, weight_decay, max_norm, grad_scale)
    if got is not None:
        _answer(got)
        return
    import torch
    params, grads = _list(opt, params), _list(opt, grads)
    if len(params._given) != len(opt.sizes):
        raise ValueError("a parameter is None")
    dev, el, (mt, vt) = params.device_index, (opt.elements,), opt.moment_dtypes
    if dev is None or grads.device_index not in (None, dev):
        raise ValueError("parameters and gradients are not on one device" if params._given else "there is no parameter")
    hyper = AdamWHyper(lr, beta1, beta2, eps, weight_decay, max_norm, grad_scale, step)
    with _current(dev):
        _check(lib().cgtp_adamw_step(
            opt.handle, params.pointers(), grads.pointers(), _addr(m, "m", mt, el, dev), _addr(v, "v", vt, el, dev),
            _addr_or_null(scales, "scales", torch.float32, (2, opt.blocks), dev),
            _addr_or_null(master, "master", torch.float32, el, dev), ctypes.byref(hyper),
            _addr_or_null(norm, "norm", torch.float64, (1,), dev),
            _addr_or_null(schedule, "schedule", torch.float64, (4,), dev), _raw_stream(dev)))


def adamw_schedule(schedule, beta1=0.9, beta2=0.999, stream=None, norm=None, grad_scale=1.0):
    """Advance a device schedule {step, lr, 1 - beta1^step, 1 - beta2^step} by one step.  With the ``norm``
    and ``grad_scale`` that the step is given after it, a step that changes nothing is not counted."""
    if stream is not None:
        return _in_stream(stream, adamw_schedule, schedule, beta1, beta2, norm=norm, grad_scale=grad_scale)
    import torch
    dev = _device_index(schedule, "schedule")
    with _current(dev):
        _check(lib().cgtp_adamw_schedule_norm(_addr(schedule, "schedule", torch.float64, (4,), dev), beta1, beta2,
                                              _addr_or_null(norm, "norm", torch.float64, (1,), dev), grad_scale,
                                              _raw_stream(dev)))
    return schedule


def adamw_state_read(opt: AdamW, m, v, scales, m_out=None, v_out=None, stream=None):
    """The values that 8-bit moments stand for: (m, v) in float32."""
    if m_out is None and v_out is None and stream is None:
        got = opt._calls.adamw_state_read(opt._meta, m, v, scales)
        if got is not None:
            return _answer(got)
    if stream is not None:
        return _in_stream(stream, adamw_state_read, opt, m, v, scales, m_out, v_out)
    import torch
    dev, el, (mt, vt), f32 = _device_index(m, "m"), (opt.elements,), opt.moment_dtypes, torch.float32
    m_out = m.new_empty(el, dtype=f32) if m_out is None else m_out
    v_out = m.new_empty(el, dtype=f32) if v_out is None else v_out
    with _current(dev):
        _check(lib().cgtp_adamw_state_read(opt.handle, _addr(m, "m", mt, el, dev), _addr(v, "v", vt, el, dev),
                                           _addr_or_null(scales, "scales", f32, (2, opt.blocks), dev),
                                           _addr(m_out, "m_out", f32, el, dev), _addr(v_out, "v_out", f32, el, dev),
                                           _raw_stream(dev)))
    return m_out, v_out


def adamw_state_write(opt: AdamW, m_in, v_in, m, v, scales, stream=None):
    """8-bit moments from float32 values (both in the flat layout)."""
    if stream is not None:
        return _in_stream(stream, adamw_state_write, opt, m_in, v_in, m, v, scales)
    import torch
    dev, el, (mt, vt), f32 = _device_index(m, "m"), (opt.elements,), opt.moment_dtypes, torch.float32
    with _current(dev):
        _check(lib().cgtp_adamw_state_write(opt.handle, _addr(m_in, "m_in", f32, el, dev),
                                            _addr(v_in, "v_in", f32, el, dev), _addr(m, "m", mt, el, dev),
                                            _addr(v, "v", vt, el, dev),
                                            _addr_or_null(scales, "scales", f32, (2, opt.blocks), dev),
                                            _raw_stream(dev)))
    return m, v, scales
