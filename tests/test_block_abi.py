"""Blocks and the optimizer step on the CPU: layouts, sizes, generated sources, and refusals, all
before any GPU call (the addresses below are never dereferenced)."""
import ctypes
import re

import numpy as np
import pytest

from clebsch_gordan_tensor_cgtp_amd import binding as cg

INVAL, UNSUP = cg.STATUS_CODES["CGTP_ERR_INVALID_ARG"], cg.STATUS_CODES["CGTP_ERR_UNSUPPORTED"]
IRREPS = cg.STATUS_CODES["CGTP_ERR_IRREPS"]
NULL = ctypes.c_void_p(0)
MB = 1 << 20


def at(mb, off=0):
    return ctypes.c_void_p(mb * MB + off)


@pytest.mark.parametrize("irreps, d, channels", [
    ("1x0e", 1, 1), ("32x0e+32x1o+32x2e", 288, 96), ("19x0e+7x1o+5x2e", 65, 31), ("3x0e+2x0o+1x7o", 20, 6),
    ("4096x0e", 4096, 4096)])
@pytest.mark.parametrize("dtype", ["f32", "f64", "bf16", "f16"])
def test_block_layout(irreps, d, channels, dtype):
    for gate, width in (("channel", channels), ("row", 1), (None, 0)):
        b = cg.Block(irreps, dtype, gate=gate, act="silu", post_norm=True, next_norm=True)
        assert (b.d, b.channels, b.gate_width) == (d, channels, width)
        check_layout(b, d)


def check_layout(b, d):
    assert b.lanes & (b.lanes - 1) == 0 and 1 <= b.lanes <= 1024
    assert b.lanes * b.lane_elements >= d and b.lane_elements <= 128
    # the source's slots cover every column once
    const = {m[0]: [int(v) for v in m[1].split(",")] for m in
             re.findall(r"constexpr int (\w+)(?:\[\w+\])? = \{?([-\d, ]+)\}?;", b.source)}
    cv, seen = const["CV"][0], []
    for j in range(const["NSLOT"][0]):
        k = const["S_K"][j]
        for lane in range(b.lanes):
            first = (const["S_UNIT"][j] + lane) * cv
            for c in range(first, min(first + cv, const["S_MUL"][j])):
                seen += range(const["S_COL"][j] + c * k, const["S_COL"][j] + c * k + k)
    assert sorted(seen) == list(range(d))
    for name in ("cgtp_norm_fwd", "cgtp_norm_bwd", "cgtp_join_fwd", "cgtp_join_bwd", "cgtp_block_reduce"):
        assert name + "(" in b.source
    assert "atomic" not in b.source.lower().replace("__atomic_acq_rel", "")


def test_block_workspace_is_one_partial_per_workgroup():
    b = cg.Block("32x0e+32x1o+32x2e", "f32", gate="channel", post_norm=True, next_norm=True)
    one = cg.block_workspace_size(b, 1)
    assert one == 2 * 96 * 4                       # P and Q of one workgroup
    assert cg.block_workspace_size(b, 0) == 0
    sizes = [cg.block_workspace_size(b, n) for n in (10, 1000, 100_000, 1_000_000)]
    assert all(s % one == 0 for s in sizes) and sizes == sorted(sizes) and sizes[-1] == sizes[-2]


def test_block_creation_refusals():
    L, h = cg.lib(), ctypes.c_void_p()

    def create(irreps=b"4x0e", **over):
        v = dict(dtype=0, gate=0, act=0, post_norm=0, next_norm=0, eps=1e-6, alpha=1.0)
        v.update(over)
        return L.cgtp_block_create(irreps, ctypes.byref(cg.BlockConfig(*v.values())), ctypes.byref(h))
    assert create(b"4x0q") == IRREPS and create(b"") == IRREPS and create(b"0x0e") == IRREPS
    assert create(b"4x8e") == IRREPS
    for bad in (dict(dtype=4), dict(dtype=-1), dict(gate=3), dict(act=4), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=1e-40), dict(alpha=float("inf"))):
        assert create(**bad) == INVAL, bad
        assert cg.last_error()
    assert create(None) == INVAL
    assert L.cgtp_block_create(b"4x0e", None, ctypes.byref(h)) == INVAL
    assert create(b"131073x0e") == UNSUP                      # over 1024 lanes x 128 elements
    many = b"+".join([b"1x0e+1x1o"] * 33)   # with a gate per channel, 132 elements in a lane
    assert create(many, gate=2) == UNSUP and create(many, gate=1) == 0 and L.cgtp_block_destroy(h) == 0
    assert create(b"+".join([b"1x0e+1x1o"] * 65), gate=1) == UNSUP   # 130 runs of equal degrees
    assert create(b"30000x0e+6000x1o") == UNSUP               # 48,000 sums over columns: 192 KB of LDS
    assert L.cgtp_block_destroy(None) == 0
    with pytest.raises(cg.CgtpError, match="irreps"):
        cg.Block("nonsense")


def test_norm_refusals():
    L, b = cg.lib(), cg.Block("32x0e", "f32")
    s = NULL

    def fwd(n=4, x=at(1), ld=32, w=at(2), u=at(3), rstd=at(4)):
        return L.cgtp_norm_forward(b.handle, n, x, ld, w, u, rstd, s)
    assert fwd(n=0, x=NULL, u=NULL) == 0
    assert L.cgtp_norm_forward(None, 4, at(1), 32, at(2), at(3), at(4), s) == INVAL
    assert fwd(n=-1) == INVAL and fwd(n=1 << 31) == INVAL
    assert fwd(x=NULL) == INVAL and fwd(u=NULL) == INVAL
    assert fwd(x=at(1, 2)) == INVAL and fwd(w=at(2, 2)) == INVAL and fwd(rstd=at(4, 1)) == INVAL
    assert fwd(ld=31) == INVAL and fwd(ld=1 << 31) == INVAL
    assert fwd(u=at(1, 64)) == INVAL and cg.last_error() == "u overlaps x"
    assert fwd(w=at(3, 128)) == INVAL and fwd(rstd=at(3, 128)) == INVAL and fwd(rstd=at(2)) == INVAL

    def bwd(n=4, x=at(1), ld=32, w=at(2), rstd=at(4), du=at(5), add=NULL, dx=at(6), dw=at(7), ws=at(8), nb=1 << 20):
        return L.cgtp_norm_backward(b.handle, n, x, ld, w, rstd, du, add, dx, dw, ws, nb, s)
    assert bwd(dx=NULL, dw=NULL) == 0
    assert bwd(rstd=NULL) == INVAL and bwd(du=NULL) == INVAL and bwd(x=NULL) == INVAL
    assert bwd(ws=NULL) == INVAL and bwd(ws=at(8, 64)) == INVAL
    assert bwd(nb=31) == INVAL and "workspace too small" in cg.last_error()
    assert bwd(dx=at(5)) == INVAL and bwd(dw=at(8)) == INVAL and bwd(add=at(6, 4)) == INVAL


def test_join_refusals():
    L = cg.lib()
    full = cg.Block("32x0e", "f32", gate="channel", post_norm=True, next_norm=True)
    bare = cg.Block("32x0e", "f32")

    def fwd(b=full, n=4, res=at(1), f=at(2), fl=32, g=at(3), gl=32, wp=at(4), sc=at(5), wn=at(6), h=at(7), u=at(8),
            rf=at(9), rh=at(10)):
        return L.cgtp_join_forward(b.handle, n, res, f, fl, g, gl, wp, sc, wn, h, u, rf, rh, NULL)
    assert fwd(n=0) == 0 and fwd(n=-1) == INVAL
    for miss in ("res", "f", "g", "h", "u"):
        assert fwd(**{miss: NULL}) == INVAL, miss
    assert fwd(fl=31) == INVAL and fwd(gl=31) == INVAL
    assert fwd(h=at(1)) == INVAL and fwd(u=at(7, 256)) == INVAL and fwd(rf=at(2, 8)) == INVAL
    assert fwd(rf=at(9), rh=at(9)) == INVAL
    # what the configuration leaves out is not given
    none = dict(b=bare, g=NULL, wp=NULL, wn=NULL, u=NULL, rf=NULL, rh=NULL)
    for extra in (dict(g=at(3)), dict(wp=at(4)), dict(wn=at(6)), dict(u=at(8)), dict(rf=at(9)), dict(rh=at(10))):
        assert fwd(**{**none, **extra}) == INVAL, extra

    def bwd(b=full, n=4, dh=at(1), du=at(2), h=at(3), f=at(4), fl=32, g=at(5), gl=32, wp=at(6), sc=at(7), wn=at(8),
            rf=at(9), rh=at(10), dr=at(11), df=at(12), dfl=32, dg=at(13), dgl=32, gp=at(14), gs=at(15), gn=at(16),
            ws=at(17), nb=1 << 20):
        return L.cgtp_join_backward(b.handle, n, dh, du, h, f, fl, g, gl, wp, sc, wn, rf, rh, dr, df, dfl, dg, dgl, gp,
                                    gs, gn, ws, nb, NULL)
    assert bwd(dr=NULL, df=NULL, dg=NULL, gp=NULL, gs=NULL, gn=NULL) == 0
    for miss in ("du", "h", "f", "g", "rf", "rh", "ws"):
        assert bwd(**{miss: NULL}) == INVAL, miss
    assert bwd(nb=8) == INVAL and bwd(dfl=8) == INVAL and bwd(dgl=8) == INVAL
    # side by side in one buffer is fine up to the check that follows (the workspace is too small),
    # any overlap of the rows is not
    side = dict(df=at(12), dfl=64, dg=at(12, 128), dgl=64)
    assert bwd(**side, nb=8) == INVAL and "workspace" in cg.last_error()
    assert bwd(df=at(12), dfl=64, dg=at(12, 124), dgl=64) == INVAL and "overlaps" in cg.last_error()
    assert bwd(df=at(12), dfl=64, dg=at(12, 132), dgl=64) == INVAL and "overlaps" in cg.last_error()
    assert bwd(df=at(12), dfl=64, dg=at(12, 128), dgl=65) == INVAL and "overlaps" in cg.last_error()
    assert bwd(gp=at(15)) == INVAL and bwd(ws=at(16)) == INVAL and bwd(dr=at(1)) == INVAL
    assert bwd(b=bare, du=NULL, h=NULL, g=NULL, wp=NULL, wn=NULL, rf=NULL, rh=NULL, dh=NULL, dg=NULL, gp=NULL,
               gn=NULL) == INVAL and "grad_h" in cg.last_error()


def test_adamw_layout():
    o = cg.AdamW([5, 2048, 0, 2049, 1], "f32", 8)
    assert o.offsets == (0, 2048, 4096, 4096, 8192) and o.elements == 10240 and o.blocks == 160
    assert cg.AdamW([], "f32").elements == 0
    with pytest.raises(cg.CgtpError, match="CGTP_ERR_UNSUPPORTED"):
        cg.AdamW([4], "f64", 8)
    for bad in (dict(state_bits=16), dict(master=True), dict(dtype="f64", master=True)):
        with pytest.raises(cg.CgtpError, match="CGTP_ERR_INVALID_ARG"):
            cg.AdamW([4], **bad)
    with pytest.raises(cg.CgtpError, match="out of range"):
        cg.AdamW([-1])


def test_adamw_refusals():
    L = cg.lib()
    o32, o8 = cg.AdamW([100, 50]), cg.AdamW([100, 50], "bf16", 8, True)

    def hyper(**over):
        v = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, max_norm=0.0, grad_scale=1.0, step=1)
        v.update(over)
        return cg.AdamWHyper(*v.values())

    def arr(*p):
        return (ctypes.c_void_p * 2)(*[x.value for x in p])

    def step(o=o32, p=(at(1), at(2)), g=(at(3), at(4)), m=at(5), v=at(6), sc=NULL, ma=NULL, hy=None, norm=NULL, sch=NULL):
        hy = hyper() if hy is None else hy
        return L.cgtp_adamw_step(o.handle, None if p is None else arr(*p), None if g is None else arr(*g), m, v, sc, ma,
                                 ctypes.byref(hy), norm, sch, NULL)
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(eps=1e-50),
                dict(weight_decay=-1.0), dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=1.0),
                dict(grad_scale=float("inf")), dict(step=0)):
        assert step(hy=hyper(**bad)) == INVAL, bad
    assert step(p=None) == INVAL and step(g=None) == INVAL
    assert step(p=(at(1), NULL)) == INVAL and step(p=(at(1, 2), at(2))) == INVAL and step(g=(at(3, 1), at(4))) == INVAL
    assert step(m=NULL) == INVAL and step(v=at(6, 8)) == INVAL
    assert step(sc=at(7)) == INVAL and step(ma=at(8)) == INVAL
    # what is written overlaps nothing: tied tensors, moments, another tensor's gradient
    assert step(p=(at(1), at(1, 396))) == INVAL and "overlaps" in cg.last_error()
    assert step(g=(at(3), at(1, 16))) == INVAL and step(m=at(1)) == INVAL and step(m=at(6)) == INVAL
    assert step(norm=at(5, 8)) == INVAL and step(sch=at(2, 8)) == INVAL
    # 8-bit moments need their scales, master copies their buffer
    assert step(o=o8, sc=NULL, ma=at(8)) == INVAL and step(o=o8, sc=at(7), ma=NULL) == INVAL
    nb = cg.AdamW([100, 50]).norm_workspace
    gn = lambda g=arr(at(3), at(4)), n=at(5), ws=at(6), b=nb: L.cgtp_grad_norm(o32.handle, g, n, ws, b, NULL)  # noqa: E731
    assert gn(n=NULL) == INVAL and gn(ws=NULL) == INVAL and gn(b=nb - 1) == INVAL and gn(n=at(3, 8)) == INVAL
    assert gn(ws=at(6, 8)) == INVAL and gn(g=arr(at(3, 1), at(4))) == INVAL
    assert L.cgtp_adamw_schedule(None, 0.9, 0.999, NULL) == INVAL
    assert L.cgtp_adamw_schedule(at(1), 1.0, 0.999, NULL) == INVAL
    rd = lambda o, mo=at(5), vo=at(6): L.cgtp_adamw_state_read(o.handle, at(1), at(2), at(3), mo, vo, NULL)  # noqa: E731
    assert rd(o32) == UNSUP and rd(o8, mo=at(1)) == INVAL and rd(o8, mo=NULL, vo=NULL) == 0
    assert L.cgtp_adamw_state_write(o32.handle, at(1), at(2), at(3), at(4), at(5), NULL) == UNSUP
    assert L.cgtp_adamw_state_write(o8.handle, at(1), at(2), at(3), at(4), NULL, NULL) == INVAL


def test_binding_refuses_what_is_not_a_device_tensor():
    torch = pytest.importorskip("torch")
    o, b = cg.AdamW([4, 3]), cg.Block("4x0e")
    with pytest.raises(TypeError, match="CUDA"):
        cg.tensor_list(o, [torch.zeros(4), torch.zeros(3)])
    with pytest.raises(ValueError, match="layout has 2"):
        cg.tensor_list(o, [torch.zeros(4)])
    with pytest.raises(TypeError):
        cg.norm_forward(b, torch.zeros(2, 4), None)
    with pytest.raises(KeyError):
        cg.Block("4x0e", "f8")
    assert np.isclose(b.eps, 1e-6)


def test_compiled_calls_leave_what_they_do_not_take_to_the_binding():
    """They answer None, and the binding says what is wrong; wrong use of the module itself raises."""
    torch = pytest.importorskip("torch")
    b, o = cg.Block("4x0e+2x1o", gate="channel", post_norm=True, next_norm=True), cg.AdamW([4, 3])
    calls, x, g = b._calls, torch.zeros(2, 10), torch.zeros(2, 6)
    assert calls.norm_forward(b._meta, x, None, True) is None          # not on a device
    assert calls.norm_forward(b._meta, "x", None, True) is None
    assert calls.join_forward(b._meta, x, x, g, None, None, None, True) is None
    assert calls.join_backward(b._meta, x, x, x, x, g, None, None, None, None, None, (True,) * 6) is None
    assert calls.norm_backward(b._meta, x, None, None, x, None, True, True) is None
    assert calls.grad_norm(o._meta, (torch.zeros(4), torch.zeros(3))) is None
    assert calls.takes_tensors(o._meta, (torch.zeros(4), torch.zeros(3))) is False
    assert calls.grad_norm(o._meta, (None, None)) is None and calls.grad_norm(o._meta, "ab") is None
    assert calls.adamw_step(o._meta, (torch.zeros(4),), (None,), x, x, None, None, None, None, 1, *[0.5] * 7) is None
    assert calls.adamw_state_read(o._meta, x, x, x) is None
    for bad in (lambda: calls.norm_forward(b._meta, x, None), lambda: calls.block(1, 2), lambda: calls.adamw(1)):
        with pytest.raises(TypeError, match="wanted"):
            bad()
    with pytest.raises(ValueError):
        calls.norm_forward(o._meta, x, None, True)                     # another kind of handle
    with pytest.raises(TypeError, match="CUDA"):
        cg.join_forward(b, x, x, g, None, None, None)
    with pytest.raises(ValueError, match="no gradient"):
        cg.grad_norm(o, [None, None])
