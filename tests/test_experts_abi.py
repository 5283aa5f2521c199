"""Group norm, routing and experts' products on the CPU: layouts, sizes, generated sources, and refusals, all before
any GPU call (the addresses below are never dereferenced)."""
import ctypes
import re

import pytest

from clebsch_gordan_tensor_cgtp_amd import binding as cg
from oracle import experts as ox

from expert_cases import DTYPES, LINEAR_CASES, NORM_SHAPES

INVAL, UNSUP = cg.STATUS_CODES["CGTP_ERR_INVALID_ARG"], cg.STATUS_CODES["CGTP_ERR_UNSUPPORTED"]
IRREPS = cg.STATUS_CODES["CGTP_ERR_IRREPS"]
NULL = ctypes.c_void_p(0)
MB = 1 << 20


def at(mb, off=0):
    return ctypes.c_void_p(mb * MB + off)


def constants(source):
    return {m[0]: [int(v) for v in m[1].split(",")] for m in
            re.findall(r"constexpr int (\w+)(?:\[\w+\])? = \{?([-\d, ]+)\}?;", source)}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("channels, groups", sorted({s[:2] for s in NORM_SHAPES}))
def test_group_norm_layout(channels, groups, dtype):
    norm = cg.group_norm_for(channels, groups, dtype, act="silu", eps=1e-5)
    c = {k: v[0] for k, v in constants(norm.source).items()}
    # the lanes' slots cover a row's channels, and no lane holds more than 32
    assert c["P"] * c["RW"] <= 64 and c["NS"] * c["CV"] <= 32 and c["GP"] // 2 < groups <= c["GP"] and c["BF"] >= 1
    assert (c["NS"] - 1) * 64 * c["CV"] < channels <= ((c["NS"] - 1) * 64 + c["P"]) * c["CV"]
    assert c["NS"] == 1 or c["P"] == 64
    assert "atomic" not in norm.source.lower()
    # bounded whatever the rows: partial sums of 1,024 chunks and 1,024 graphs' workgroups
    most = 8 * (2048 * 2 * channels + (1024 + 10) * 2 * groups) + 3 * 256
    for n in (0, 1, 1000, 1_000_000, 100_000_000):
        for backward in (False, True):
            assert 0 < cg.group_norm_workspace_size(norm, n, 10, backward) <= most
    assert cg.group_norm_workspace_size(norm, 100, 0) == 0


def test_group_norm_creation_refusals():
    L, h = cg.lib(), ctypes.c_void_p()

    def create(**over):
        v = dict(dtype=0, channels=8, groups=2, act=0, eps=1e-6)
        v.update(over)
        return L.cgtp_group_norm_create(ctypes.byref(cg.GroupNormConfig(*v.values())), ctypes.byref(h))
    for bad in (dict(dtype=4), dict(dtype=-1), dict(channels=0), dict(groups=0), dict(groups=3), dict(groups=16), dict(act=4),
                dict(act=-1), dict(eps=0.0), dict(eps=float("nan")), dict(eps=1e-40)):
        assert create(**bad) == INVAL and cg.last_error(), bad
    assert create(channels=2049, groups=1) == UNSUP
    assert L.cgtp_group_norm_create(None, ctypes.byref(h)) == INVAL
    assert L.cgtp_group_norm_destroy(None) == 0 and L.cgtp_group_norm_source(None) is None


def test_group_norm_refusals():
    L, g = cg.lib(), cg.group_norm_for(32, 4, "f32", act="silu", eps=1e-5)

    def fwd(n=100, s=3, ptr=at(1), x=at(2), ld=32, w=at(3), b=at(4), y=at(5), yl=32, fill=0, m=at(6), r=at(7), ws=at(8), nb=MB):
        return L.cgtp_group_norm_forward(g.handle, n, s, ptr, x, ld, w, b, y, yl, fill, m, r, ws, nb, NULL)
    assert fwd(s=0) == 0 and L.cgtp_group_norm_forward(None, 1, 1, *[at(1)] * 2, 32, *[at(1)] * 3, 32, 0, *[at(1)] * 3, 9, NULL) == INVAL
    assert fwd(n=-1) == INVAL and fwd(n=1 << 31) == INVAL and fwd(s=-1) == INVAL and fwd(s=1 << 31) == INVAL
    for miss in ("ptr", "x", "y", "ws", "m", "r"):
        assert fwd(**{miss: NULL}) == INVAL, miss
    for odd in ("ptr", "x", "w", "b", "y", "m", "r"):
        assert fwd(**{odd: at(20, 2)}) == INVAL, odd
    assert fwd(ld=31) == INVAL and fwd(yl=31) == INVAL and fwd(ws=at(8, 64)) == INVAL
    assert fwd(nb=cg.group_norm_workspace_size(g, 100, 3) - 1) == INVAL and "workspace too small" in cg.last_error()
    for a, b in (("y", "x"), ("y", "w"), ("m", "y"), ("r", "m"), ("ws", "x"), ("ws", "r"), ("m", "ptr")):
        addr = dict(ptr=1, x=2, w=3, b=4, y=5, m=6, r=7, ws=8)
        assert fwd(**{a: at(addr[b])}) == INVAL and "overlaps" in cg.last_error(), (a, b)

    def bwd(n=100, s=3, ptr=at(1), x=at(2), ld=32, w=at(3), b=at(4), m=at(6), r=at(7), dy=at(9), dyl=32, dx=at(10), dxl=32,
            dw=at(11), db=at(12), ws=at(8), nb=MB):
        return L.cgtp_group_norm_backward(g.handle, n, s, ptr, x, ld, w, b, m, r, dy, dyl, dx, dxl, 0, dw, db, ws, nb, NULL)
    assert bwd(dx=NULL, dw=NULL, db=NULL) == 0
    for miss in ("ptr", "x", "m", "r", "dy", "ws"):
        assert bwd(**{miss: NULL}) == INVAL, miss
    assert bwd(dyl=31) == INVAL and bwd(dxl=31) == INVAL and bwd(nb=100) == INVAL
    for a, b in ((dict(dx=at(9)), "grad_y"), (dict(dw=at(3)), "w"), (dict(db=at(11)), "grad_w"), (dict(dx=at(2)), "x")):
        assert bwd(**a) == INVAL and "overlaps" in cg.last_error(), b


def test_router_creation_refusals():
    L, h = cg.lib(), ctypes.c_void_p()

    def create(**over):
        v = dict(dtype=0, score=0, experts=8, top_k=2, groups=1, top_groups=1, renormalise=1, scale=1.0)
        v.update(over)
        return L.cgtp_router_create(ctypes.byref(cg.RouterConfig(*v.values())), ctypes.byref(h))
    for bad in (dict(dtype=4), dict(score=2), dict(experts=0), dict(top_k=0), dict(top_k=9), dict(groups=3), dict(groups=0),
                dict(top_groups=2), dict(top_groups=0), dict(groups=4, top_groups=1, top_k=3), dict(scale=float("inf"))):
        assert create(**bad) == INVAL and cg.last_error(), bad
    assert create(experts=513) == UNSUP and create(experts=64, top_k=33) == UNSUP
    assert create(experts=130, groups=65, top_groups=2) == UNSUP          # over a wave's lanes
    for e, groups in ((510, 15), (504, 18), (495, 33), (510, 17), (512, 64)):
        assert create(experts=e, groups=groups, top_groups=2) == 0 and L.cgtp_router_destroy(h) == 0
    assert create(experts=130, groups=65, top_groups=65) == 0 and L.cgtp_router_destroy(h) == 0  # every group: none
    assert L.cgtp_router_create(None, ctypes.byref(h)) == INVAL and L.cgtp_router_destroy(None) == 0


def test_route_refusals():
    L, r = cg.lib(), cg.router_for(8, 2, "f32")

    def fwd(n=4, l=at(1), ld=8, b=at(2), e=at(3), w=at(4)):
        return L.cgtp_route_forward(r.handle, n, l, ld, b, e, w, NULL)
    assert fwd(n=0, l=NULL, e=NULL) == 0 and L.cgtp_route_forward(None, 4, at(1), 8, *[at(2)] * 3, NULL) == INVAL
    assert fwd(n=-1) == INVAL and fwd(n=1 << 30) == INVAL                  # 2^31 slots
    assert fwd(l=NULL) == INVAL and fwd(e=NULL) == INVAL and fwd(w=NULL) == INVAL and fwd(ld=7) == INVAL
    assert fwd(l=at(1, 2)) == INVAL and fwd(b=at(2, 1)) == INVAL and fwd(e=at(3, 2)) == INVAL and fwd(w=at(4, 2)) == INVAL
    assert fwd(e=at(1, 64)) == INVAL and fwd(w=at(3)) == INVAL and fwd(w=at(2, 16)) == INVAL

    def bwd(n=4, l=at(1), ld=8, e=at(3), g=at(4), o=at(5)):
        return L.cgtp_route_backward(r.handle, n, l, ld, e, g, o, NULL)
    assert bwd(n=0) == 0 and bwd(l=NULL) == INVAL and bwd(e=NULL) == INVAL and bwd(g=NULL) == INVAL and bwd(o=NULL) == INVAL
    assert bwd(o=at(1)) == INVAL and bwd(o=at(3)) == INVAL and bwd(o=at(4, 16)) == INVAL and bwd(ld=3) == INVAL

    big = 100_000
    need = cg.route_order_workspace_size(r, big)
    assert cg.route_order_workspace_size(r, 1000) == 0 < need

    def order(n=big, e=at(1), rows=at(2), s=at(3), o=at(4), ws=at(5), nb=need):
        return L.cgtp_route_order(r.handle, n, e, rows, s, o, ws, nb, NULL)
    for miss in ("e", "rows", "s", "o", "ws"):
        assert order(**{miss: NULL}) == INVAL, miss
    assert order(nb=need - 1) == INVAL and order(ws=at(5, 16)) == INVAL and order(n=-1) == INVAL
    assert order(rows=at(1)) == INVAL and order(s=at(2)) == INVAL and order(o=at(3)) == INVAL and order(ws=at(4)) == INVAL


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("a, b, e, k, n", LINEAR_CASES)
def test_linear_layout(a, b, e, k, n, dtype):
    linear = cg.linear_for(a, b, dtype, experts=e, top_k=k)
    found, numel, d_in, d_out = ox.paths(a, b)
    assert (linear.d_in, linear.d_out, linear.num_paths, linear.weight_numel) == (d_in, d_out, len(found), numel)
    c = constants(linear.source)
    assert [c[n] for n in ("W_MI", "W_XC", "W_MO", "W_GC", "W_K", "W_OFF")] == [list(v) for v in zip(*found)]
    # the gradients' tiles cover every weight once
    seen = []
    for p, v, u, bv, bu, wv, wu, nodes in zip(*[c["T_" + n] for n in ("PATH", "V", "U", "BV", "BU", "WV", "WU", "NODES")]):
        mi, _, mo, _, _, off = found[p]
        seen += [off + i * mi + j for i in range(v, min(mo, v + 16 * bv)) for j in range(u, min(mi, u + 16 * bu))]
        assert wv * wu <= 4 and nodes % 4 == 0
    assert sorted(seen) == list(range(numel))
    # the units of each direction cover every 16-block of every irrep once, in waves that exist
    for name in ("Forward", "Backward", "ForwardFew", "BackwardFew"):
        d = constants(re.search(r"struct %s \{\n(.*?)\n\};\n" % name, linear.source, re.S).group(1))
        blocks = [(o, i) for o, f, m in zip(d["U_OUT"], d["U_N0"], d["U_NN"]) for i in range(f, f + m)]
        assert sorted(blocks) == [(o, i) for o, mul in enumerate(d["O_MUL"]) for i in range(-(-mul // 16))]
        assert sorted(set(d["U_WAVE"])) == list(range(d["WAVES"][0])) and d["WAVES"][0] <= 12
    assert "atomic" not in linear.source.lower()


def test_linear_creation_refusals():
    L, h = cg.lib(), ctypes.c_void_p()

    def create(a=b"4x0e", b=b"4x0e", **over):
        v = dict(dtype=0, experts=4, top_k=2)
        v.update(over)
        return L.cgtp_linear_create(a, b, ctypes.byref(cg.LinearConfig(*v.values())), ctypes.byref(h))
    assert create(b"4x0q") == IRREPS and create(b=b"") == IRREPS
    assert create(b"4x0e", b"4x0o") == IRREPS and "no irrep" in cg.last_error()
    for bad in (dict(dtype=4), dict(experts=0), dict(top_k=-1), dict(top_k=5), dict(top_k=0)):
        assert create(**bad) == INVAL and cg.last_error(), bad
    assert create(None) == INVAL and create(b=None) == INVAL
    assert L.cgtp_linear_create(b"4x0e", b"4x0e", None, ctypes.byref(h)) == INVAL
    assert create(experts=513) == UNSUP and create(experts=64, top_k=33) == UNSUP
    assert create(b"600x1o", b"40x1o", dtype=1) == UNSUP and "LDS" in cg.last_error()
    assert create(b"9000x0e", b"9000x0e") == UNSUP and create(b"+".join([b"1x0e"] * 9), b"+".join([b"1x0e"] * 9)) == UNSUP
    assert L.cgtp_linear_destroy(None) == 0


def test_linear_refusals():
    L, q = cg.lib(), cg.linear_for("8x0e", "12x0e", "f32", experts=4, top_k=2)

    def fwd(h=q.handle, n=4, x=at(1), xl=8, w=at(2), e=at(3), p=at(4), rows=at(5), o=at(6), ol=12):
        return L.cgtp_linear_forward(h, n, x, xl, w, e, p, rows, o, ol, NULL)
    assert fwd(n=0, x=NULL, e=NULL, p=NULL) == 0 and fwd(h=None) == INVAL
    assert fwd(n=-1) == INVAL and fwd(n=1 << 30) == INVAL
    for miss in ("x", "w", "e", "p", "o"):
        assert fwd(**{miss: NULL}) == INVAL, miss
    for odd in ("x", "w", "e", "p", "rows", "o"):
        assert fwd(**{odd: at(9, 2)}) == INVAL, odd
    assert fwd(xl=7) == INVAL and fwd(ol=11) == INVAL
    for other in (1, 2, 3, 4, 5):
        assert fwd(o=at(other)) == INVAL and "overlaps" in cg.last_error()
    plain = cg.linear_for("8x0e", "12x0e", "f32")
    assert fwd(h=plain.handle, e=at(3), p=NULL) == INVAL and fwd(h=plain.handle, e=NULL, p=at(4)) == INVAL

    def bwd(h=q.handle, n=4, x=at(1), w=at(2), e=at(3), p=at(4), rows=at(5), s=at(6), off=at(7), g=at(8), gl=12, dx=at(9), dxl=8,
            dw=at(10), dp=at(11), ws=at(12), nb=MB):
        return L.cgtp_linear_backward(h, n, x, 8, w, e, p, rows, s, off, g, gl, dx, dxl, dw, dp, ws, nb, NULL)
    assert bwd(dx=NULL, dw=NULL, dp=NULL) == 0
    for miss in ("x", "w", "e", "p", "s", "off", "g", "ws"):
        assert bwd(**{miss: NULL}) == INVAL, miss
    assert bwd(gl=11) == INVAL and bwd(dxl=7) == INVAL and bwd(ws=at(12, 16)) == INVAL
    assert bwd(nb=cg.linear_workspace_size(q, 4) - 1) == INVAL and "workspace too small" in cg.last_error()
    for kw in (dict(dx=at(1)), dict(dx=at(8)), dict(dw=at(2)), dict(dp=at(4)), dict(dw=at(9)), dict(ws=at(6)), dict(dp=at(3))):
        assert bwd(**kw) == INVAL and "overlaps" in cg.last_error(), kw
    assert bwd(h=plain.handle, e=NULL, p=NULL, s=at(6), off=NULL, dp=NULL) == INVAL
    assert bwd(h=plain.handle, e=NULL, p=NULL, s=NULL, off=NULL, dp=at(11)) == INVAL


def test_binding_refusals():
    import torch
    norm, router = cg.group_norm_for(4, 2, "f32"), cg.router_for(4, 2, "f32")
    linear, x = cg.linear_for("4x0e", "4x0e", "f32", experts=4, top_k=2), torch.zeros(3, 4)
    with pytest.raises(TypeError, match="must be a CUDA"):
        cg.group_norm_forward(norm, x, torch.zeros(2, dtype=torch.int32), None, None)
    with pytest.raises(TypeError, match="must be a CUDA"):
        cg.route_forward(router, x)
    with pytest.raises(TypeError, match="must be a CUDA"):
        cg.route_order(router, torch.zeros(3, 2, dtype=torch.int32))
    with pytest.raises(TypeError, match="must be a CUDA"):
        cg.linear_forward(linear, x, torch.zeros(4, 16))
    with pytest.raises(cg.CgtpError, match="no irrep"):
        cg.Linear("4x0e", "4x1o")
    closed = cg.Router(4, 2)
    closed.close()
    closed.close()
    with pytest.raises(cg.CgtpError, match="NULL"):
        cg.route_order_workspace_size(closed, 5)
