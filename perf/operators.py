"""Cases and plain forms of the operators around the convolution in a training step.

Three operators of a residual equivariant network, each row-wise over irreps rows (element
(channel u, component m) of an irrep at offset + u*(2l+1) + (m + l); "Dx0e" is an ordinary row):

norm   u = x * rstd(x) * w[c],  rstd(x) = (mean(x^2) + eps)^(-1/2) over the whole row, which a
       rotation leaves alone; w has one entry per channel, shared by its 2l+1 components.
join   the end of a block and the start of the next in one pass:
       h = alpha * r + s[c] * act(gate) * w_post[c] * f * rstd(f),   u = h * rstd(h) * w_next[c];
       r the residual row, f the block's output, gate one logit per channel or per row.
adamw  decoupled-decay Adam over many tensors at once, moments in 32 bits or in 8-bit codes, with
       the gradient's global norm and its clipping.

``run`` computes a case in elementary torch operations, or by the library where ``own`` is true.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-5
TORCH = {"f32": torch.float32, "f64": torch.float64, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "f64": 8, "bf16": 2, "f16": 2}
# Moments lie in flat buffers, every tensor padded with zeros to whole units; an 8-bit moment has
# one scale per block.
UNIT, BLOCK = 2048, 64
HYPER = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01, "max_norm": 1.0}


# ------------------------------------------------------------------------------------ cases

def listed():
    ladder = {n: "+".join("%dx%d%s" % (n, l, "eo"[l % 2]) for l in range(4)) for n in (32, 64, 128)}
    to2 = {n: t.rsplit("+", 1)[0] for n, t in ladder.items()}
    return [
        # the rows of the small batched product: a launch's latency
        {"name": "norm-fwd-1024x16-f32", "op": "norm", "dir": "fwd", "rows": 1024, "irreps": "4x0e+4x1o",
         "dtype": "f32"},
        # double precision features of the MACE-like graph
        {"name": "norm-fwd-20000x2048-f64", "op": "norm", "dir": "fwd", "rows": 20000, "irreps": ladder[128],
         "dtype": "f64"},
        # every node of the power-law graph, the gradient added to the residual's
        {"name": "norm-bwd-200000x576-f32", "op": "norm", "dir": "bwd", "rows": 200000, "irreps": to2[64],
         "dtype": "f32", "add": True},
        # a wide scalar stream in 16 bits, as a readout trunk has it
        {"name": "norm-bwd-8192x4096-bf16", "op": "norm", "dir": "bwd", "rows": 8192, "irreps": "4096x0e",
         "dtype": "bf16", "add": False},
        # one row alone: inference on a single node
        {"name": "join-fwd-1x8192-bf16", "op": "join", "dir": "fwd", "rows": 1, "irreps": "8192x0e", "dtype": "bf16",
         "gate": "channel", "act": "silu", "post": True, "next": True, "packed": False},
        # the NequIP-like graph's nodes, a gate logit for each channel
        {"name": "join-fwd-5000x288-f32", "op": "join", "dir": "fwd", "rows": 5000, "irreps": to2[32], "dtype": "f32",
         "gate": "channel", "act": "sigmoid", "post": True, "next": True, "packed": True},
        # a large graph's features in 16 bits, the block's output and its gates in one row
        {"name": "join-fwd-200000x576-bf16", "op": "join", "dir": "fwd", "rows": 200000, "irreps": to2[64],
         "dtype": "bf16", "gate": "channel", "act": "silu", "post": True, "next": True, "packed": True},
        # odd multiplicities, one gate for a row, no norm after the block
        {"name": "join-bwd-4999x65-f16", "op": "join", "dir": "bwd", "rows": 4999, "irreps": "19x0e+7x1o+5x2e",
         "dtype": "f16", "gate": "row", "act": "tanh", "post": False, "next": True, "packed": True},
        # the MACE-like graph's nodes: every gradient of the join
        {"name": "join-bwd-20000x2048-f32", "op": "join", "dir": "bwd", "rows": 20000, "irreps": ladder[128],
         "dtype": "f32", "gate": "channel", "act": "sigmoid", "post": True, "next": True, "packed": True},
        # a small network's many small tensors, with clipping: latency
        {"name": "adamw-6x32-f32", "op": "adamw", "layers": 6, "mul": 32, "dtype": "f32", "bits": 32, "master": False,
         "clip": True, "shift": 0},
        # a wide network in single precision, moments in 8 bits, with clipping
        {"name": "adamw-3x3500-f32-8bit", "op": "adamw", "layers": 3, "mul": 3500, "dtype": "f32", "bits": 8,
         "master": False, "clip": True, "shift": 0},
        # 16-bit weights with single precision copies, odd sizes, views that are not aligned
        {"name": "adamw-4x2501-bf16-master", "op": "adamw", "layers": 4, "mul": 2501, "dtype": "bf16", "bits": 32,
         "master": True, "clip": False, "shift": 3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    if rng.random() < 0.35:
        layers = rng.randint(1, 8)
        dtype = rng.choice(["f32", "f32", "bf16", "f16", "f64"])
        return {"op": "adamw", "layers": layers, "mul": _log(rng, 8, 3800 / math.sqrt(layers)), "dtype": dtype,
                "bits": 32 if dtype == "f64" else rng.choice([32, 8]),
                "master": dtype in ("bf16", "f16") and rng.random() < 0.5, "clip": rng.random() < 0.5,
                "shift": rng.randint(0, 7)}
    dtype = rng.choice(["f32", "f32", "bf16", "f16", "f64"])
    if rng.random() < 0.4:
        irreps = "%dx0e" % _log(rng, 1, 8192)
    else:
        top = _log(rng, 1, 128)
        terms = ["%dx%d%s" % (rng.randint(1, top), rng.randint(0, 4), rng.choice("eo"))
                 for _ in range(rng.randint(1, 5))]
        irreps = "+".join(terms)
    width = sum(_degrees(irreps))
    most = 20000 * 2048 * 4 // (width * BYTES[dtype])
    case = {"op": rng.choice(["norm", "join", "join"]), "dir": rng.choice(["fwd", "bwd"]),
            "rows": _log(rng, 1, min(200000, most)), "irreps": irreps, "dtype": dtype}
    if case["op"] == "norm":
        case["add"] = rng.random() < 0.5
    else:
        case.update(gate=rng.choice(["none", "row", "channel", "channel"]),
                    act=rng.choice(["identity", "sigmoid", "silu", "tanh"]), post=rng.random() < 0.8,
                    next=rng.random() < 0.8, packed=rng.random() < 0.5)
    return case


# ------------------------------------------------------------------------------------ layouts

def _degrees(irreps):
    """Components of each channel, in order: their sum is the row's width."""
    out = []
    for term in irreps.split("+"):
        mul, lp = term.split("x")
        out += [2 * int(lp[:-1]) + 1] * int(mul)
    return out


def _sizes(case):
    """A network's tensors: per layer three norm weights and a scale per channel, a radial
    projection, three mixing matrices and a small radial network; then a readout."""
    m = case["mul"]
    layer = [3 * m, 3 * m, 3 * m, 8 * 15 * m, m * m, m * m, m * m, 8 * 64, 64 * 64, 64]
    return layer * case["layers"] + [m, 1]


def _layout(case):
    sizes = _sizes(case)
    units = [-(-n // UNIT) for n in sizes]
    starts = [UNIT * u for u in np.concatenate([[0], np.cumsum(units)]).tolist()]
    return sizes, starts[:-1], starts[-1]


# ------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, dtype=dtype, device="cuda")

    if case["op"] == "adamw":
        return _prepare_adamw(case, normal)
    n, dt = case["rows"], TORCH[case["dtype"]]
    real = torch.float64 if case["dtype"] == "f64" else torch.float32
    deg = _degrees(case["irreps"])
    c, d = len(deg), sum(deg)
    chan = np.repeat(np.arange(c), deg)
    first = np.cumsum([0] + deg[:-1])
    # the columns of each channel, the row's end (a zero) standing for what shorter ones lack
    cols = np.where(np.arange(max(deg)) < np.array(deg)[:, None], first[:, None] + np.arange(max(deg)), d)
    st = {"case": case, "chan": torch.from_numpy(chan).cuda(), "cols": torch.from_numpy(cols).cuda()}

    def weight():
        return 1 + 0.1 * normal(c, dtype=real)

    def rows(width=d):
        return normal(n, width, dtype=real).to(dt)

    if own:
        st["block"] = _block(case)
    if case["op"] == "norm":
        st["x"], st["w"] = (normal(n, d, dtype=real) * torch.exp(normal(n, 1, dtype=real))).to(dt), weight()
        if case["dir"] == "bwd":
            st["grad_u"] = rows()
            st["grad_add"] = rows() if case["add"] else None
            st["rstd"] = _rstd(st["x"], EPS)
        return st
    gates = {"none": 0, "row": 1, "channel": c}[case["gate"]]
    buf = torch.empty(n, d + gates, dtype=dt, device="cuda") if case["packed"] else None
    f = normal(n, d, dtype=real) * torch.exp(0.5 * normal(n, 1, dtype=real))
    # receivers without edges have a row of zeros
    f = (f * (torch.rand(n, 1, generator=gen, device="cuda") > 0.01)).to(dt)
    gate = rows(gates) if gates else None
    if buf is not None:
        buf[:, :d] = f
        f = buf[:, :d]
        if gates:
            buf[:, d:] = gate
            gate = buf[:, d:]
    st.update(r=rows(), f=f, gate=gate, w_post=weight() if case["post"] else None, scale=0.2 * weight(),
              w_next=weight() if case["next"] else None, alpha=1.0)
    if case["dir"] == "bwd":
        h, _, st["rstd_f"], st["rstd_h"] = _join(st)
        st["h"], st["r"] = h, None
        st["grad_h"], st["grad_u"] = rows(), rows() if case["next"] else None
    return st


def _prepare_adamw(case, normal):
    sizes, starts, total = _layout(case)
    dt = TORCH[case["dtype"]]
    real = torch.float64 if case["dtype"] == "f64" else torch.float32
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    for n, s in zip(sizes, starts):
        live[s:s + n] = True

    def flat(values, dtype):
        buf = torch.zeros(total + case["shift"], dtype=dtype, device="cuda")[case["shift"]:]
        buf.copy_(values * live)
        return buf

    weights = normal(total, dtype=real) * 0.05
    st = {"case": case, "step": 100, "p": flat(weights, dt), "g": flat(normal(total, dtype=real) * 1e-3, dt),
          "master": weights * live if case["master"] else None}
    m, s = normal(total, dtype=real) * 3e-4 * live, 1e-3 * torch.exp(0.5 * normal(total, dtype=real)) * live
    if case["bits"] == 8:
        (st["m"], am), (st["v"], as_) = _encode(m, 127, torch.int8), _encode(s, 255, torch.uint8)
        st["scales"] = torch.stack([am, as_])
    else:
        st["m"], st["v"], st["scales"] = m, s * s, None
    if own:
        from clebsch_gordan_tensor_cgtp_amd import binding as cg
        st["opt"] = cg.AdamW(sizes, dtype=case["dtype"], state_bits=case["bits"], master=case["master"])
        st["params"] = cg.tensor_list(st["opt"], [st["p"][s:s + n] for n, s in zip(sizes, starts)])
        st["grads"] = cg.tensor_list(st["opt"], [st["g"][s:s + n] for n, s in zip(sizes, starts)])
    return st


def _block(case):
    from clebsch_gordan_tensor_cgtp_amd import binding as cg
    if case["op"] == "norm":
        return cg.block_for(case["irreps"], case["dtype"], eps=EPS)
    return cg.block_for(case["irreps"], case["dtype"], gate=None if case["gate"] == "none" else case["gate"],
                        act=case["act"], post_norm=case["post"], next_norm=case["next"], eps=EPS, alpha=1.0)


# ------------------------------------------------------------------------------------ plain forms

def _wide(t):
    return t if t is None or t.dtype == torch.float64 else t.float()


def _rstd(x, eps):
    return torch.rsqrt(_wide(x).square().mean(1) + eps)


def _act(kind, g):
    """The gate's activation and its derivative."""
    if kind == "identity":
        return g, torch.ones_like(g)
    if kind == "tanh":
        a = torch.tanh(g)
        return a, 1 - a * a
    s = torch.sigmoid(g)
    return (s, s * (1 - s)) if kind == "sigmoid" else (g * s, s * (1 + g * (1 - s)))


def _norm_grad(wdu, xhat, rstd):
    return rstd[:, None] * (wdu - xhat * (wdu * xhat).mean(1, keepdim=True))


def _per_channel(st, t):
    """[N][D] to [N][C]: the sum over each channel's components."""
    if st["cols"].shape[1] == 1:
        return t
    return torch.cat([t, t.new_zeros(t.shape[0], 1)], 1)[:, st["cols"]].sum(2)


def _weight_grad(t, like):
    return t.sum(0, dtype=torch.float64).to(like.dtype)


def _post_scale(st):
    return st["scale"] if st["w_post"] is None else st["scale"] * st["w_post"]


def _join(st):
    chan, dt = st["chan"], st["f"].dtype
    f, gate = _wide(st["f"]), _wide(st["gate"])
    y, rstd_f = f, None
    if st["w_post"] is not None:
        rstd_f = _rstd(f, EPS)
        y = f * rstd_f[:, None]
    y = y * _post_scale(st)[chan]
    if gate is not None:
        a = _act(st["case"]["act"], gate)[0]
        y = y * (a if a.shape[1] == 1 else a[:, chan])
    h = st["alpha"] * _wide(st["r"]) + y
    u, rstd_h = None, None
    if st["w_next"] is not None:
        rstd_h = _rstd(h, EPS)
        u = (h * rstd_h[:, None] * st["w_next"][chan]).to(dt)
    return h.to(dt), u, rstd_f, rstd_h


def _join_grad(st):
    chan, dt = st["chan"], st["f"].dtype
    f, gate, dh = _wide(st["f"]), _wide(st["gate"]), _wide(st["grad_h"])
    out = {}
    if st["w_next"] is not None:
        du, hhat = _wide(st["grad_u"]), _wide(st["h"]) * st["rstd_h"][:, None]
        dh = dh + _norm_grad(du * st["w_next"][chan], hhat, st["rstd_h"])
        out["w_next"] = _weight_grad(_per_channel(st, du * hhat), st["w_next"])
    out["r"] = (st["alpha"] * dh).to(dt)
    fhat = f if st["w_post"] is None else f * st["rstd_f"][:, None]
    ws = _post_scale(st)
    t = _per_channel(st, dh * fhat)
    dy = dh * ws[chan]
    if gate is not None:
        a, da = _act(st["case"]["act"], gate)
        dy = dy * (a if a.shape[1] == 1 else a[:, chan])
        dgate = t * ws
        out["gate"] = (da * (dgate.sum(1, keepdim=True) if a.shape[1] == 1 else dgate)).to(dt)
        t = t * a
    t = t.sum(0, dtype=torch.float64)
    if st["w_post"] is not None:
        out["w_post"] = (t * st["scale"]).to(st["scale"].dtype)
        out["scale"] = (t * st["w_post"]).to(st["scale"].dtype)
        dy = _norm_grad(dy, fhat, st["rstd_f"])
    else:
        out["scale"] = t.to(st["scale"].dtype)
    out["f"] = dy.to(dt)
    return out


def _encode(x, top, dtype):
    """8-bit codes of a block's values by the root of their share of its largest, and that value;
    a value of the unsigned kind that is not zero gets no code of zero."""
    a = x.abs().view(-1, BLOCK)
    most = a.amax(1)
    most = torch.where(most < torch.finfo(torch.float32).tiny, torch.zeros_like(most), most)
    inv = torch.where(most > 0, 1 / most, torch.zeros_like(most))
    q = torch.round(torch.sqrt(a * inv[:, None]) * top).clamp(0, top)
    if dtype == torch.uint8:
        q = torch.where((a > 0) & (most > 0)[:, None], q.clamp(min=1), q)
    q = q.view(-1)
    return (q if dtype == torch.uint8 else torch.where(x < 0, -q, q)).to(dtype), most


def _decode(q, most, top):
    t = q.float() * (1 / top)
    return ((t * t.abs()).view(-1, BLOCK) * most[:, None]).view(-1)


def _adamw(st):
    case, hy = st["case"], HYPER
    st["step"] += 1
    g = _wide(st["g"])
    norm = None
    if case["clip"]:
        norm = g.double().square().sum().sqrt()
        g = g * torch.clamp(hy["max_norm"] / norm, max=1.0).to(g.dtype)
    m, v = st["m"], st["v"]
    if case["bits"] == 8:
        m = _decode(m, st["scales"][0], 127)
        v = _decode(v, st["scales"][1], 255).square()
    m = m * hy["beta1"] + g * (1 - hy["beta1"])
    v = v * hy["beta2"] + g * g * (1 - hy["beta2"])
    s = torch.sqrt(v)
    p = _wide(st["p"]) if st["master"] is None else st["master"]
    p = p * (1 - hy["lr"] * hy["weight_decay"])
    bias1, bias2 = 1 - hy["beta1"] ** st["step"], 1 - hy["beta2"] ** st["step"]
    p = p - m * (hy["lr"] / bias1) / (s * (1 / math.sqrt(bias2)) + hy["eps"])
    st["p"].copy_(p)
    if st["master"] is not None:
        st["master"].copy_(p)
    out = {"p": st["p"], "master": st["master"], "norm": None if norm is None else norm.view(1)}
    if case["bits"] == 8:
        (st["m"], am), (st["v"], as_) = _encode(m, 127, torch.int8), _encode(s, 255, torch.uint8)
        st["scales"] = torch.stack([am, as_])
        out["m"], out["v"] = _decode(st["m"], am, 127), _decode(st["v"], as_, 255).square()
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
        out["m"], out["v"] = st["m"], st["v"]
    return out


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "adamw":
        return _adamw(state)
    if case["op"] == "join":
        if case["dir"] == "bwd":
            return _join_grad(state)
        h, u, rstd_f, rstd_h = _join(state)
        return {"h": h, "u": u, "rstd_f": rstd_f, "rstd_h": rstd_h}
    x, dt, w = _wide(state["x"]), state["x"].dtype, state["w"]
    if case["dir"] == "fwd":
        rstd = _rstd(x, EPS)
        return {"u": (x * rstd[:, None] * w[state["chan"]]).to(dt), "rstd": rstd}
    xhat, du = x * state["rstd"][:, None], _wide(state["grad_u"])
    dx = _norm_grad(du * w[state["chan"]], xhat, state["rstd"])
    if state["grad_add"] is not None:
        dx = dx + _wide(state["grad_add"])
    return {"x": dx.to(dt), "w": _weight_grad(_per_channel(state, du * xhat), w)}


# ------------------------------------------------------------------------------------ the library

def _run_own(st):
    from clebsch_gordan_tensor_cgtp_amd import binding as cg
    case = st["case"]
    if case["op"] == "adamw":
        st["step"] += 1
        norm = cg.grad_norm(st["opt"], st["grads"]) if case["clip"] else None
        hyper = dict(HYPER)
        if not case["clip"]:
            hyper.pop("max_norm")
        cg.adamw_step(st["opt"], st["params"], st["grads"], st["m"], st["v"], st["scales"], st["master"],
                      step=st["step"], norm=norm, **hyper)
        m, v = st["m"], st["v"]
        if case["bits"] == 8:
            m, v = cg.adamw_state_read(st["opt"], m, v, st["scales"])
        return {"p": st["p"], "master": st["master"], "norm": norm, "m": m, "v": v}
    if case["op"] == "norm":
        if case["dir"] == "fwd":
            u, rstd = cg.norm_forward(st["block"], st["x"], st["w"])
            return {"u": u, "rstd": rstd}
        dx, dw = cg.norm_backward(st["block"], st["x"], st["w"], st["rstd"], st["grad_u"], grad_add=st["grad_add"])
        return {"x": dx, "w": dw}
    if case["dir"] == "fwd":
        h, u, rstd_f, rstd_h = cg.join_forward(st["block"], st["r"], st["f"], st["gate"], st["w_post"], st["scale"],
                                               st["w_next"])
        return {"h": h, "u": u, "rstd_f": rstd_f, "rstd_h": rstd_h}
    got = cg.join_backward(st["block"], st["grad_h"], st["grad_u"], st["h"], st["f"], st["gate"], st["w_post"],
                           st["scale"], st["w_next"], st["rstd_f"], st["rstd_h"])
    names = ("r", "f", "gate", "w_post", "scale", "w_next")
    return {k: t for k, t in zip(names, got) if t is not None}


# ------------------------------------------------------------------------------------ work

def work(case):
    """Every input read once, every output written once."""
    if case["op"] == "adamw":
        n, b = sum(_sizes(case)), BYTES[case["dtype"]]
        moment = 1 if case["bits"] == 8 else max(4, b)
        per = 3 * b + 4 * moment + (8 if case["master"] else 0)
        if case["master"]:
            per -= b  # the 16-bit weight is only written
        if case["bits"] == 8:
            per += 16 / BLOCK + 8  # scales both ways; the decoded moments that come back
        return {"bytes": n * per, "flops": 20 * n}
    deg = _degrees(case["irreps"])
    n, c, d, b = case["rows"], len(deg), sum(deg), BYTES[case["dtype"]]
    w = 8 if case["dtype"] == "f64" else 4
    if case["op"] == "norm":
        if case["dir"] == "fwd":
            return {"bytes": 2 * n * d * b + (n + c) * w, "flops": 4 * n * d}
        return {"bytes": (4 if case["add"] else 3) * n * d * b + (n + 2 * c) * w, "flops": 9 * n * d}
    gates = {"none": 0, "row": 1, "channel": c}[case["gate"]]
    stats, weights = int(case["post"]) + int(case["next"]), 1 + int(case["post"]) + int(case["next"])
    if case["dir"] == "fwd":
        return {"bytes": n * b * ((4 if case["next"] else 3) * d + gates) + (n * stats + c * weights) * w,
                "flops": 10 * n * d}
    return {"bytes": n * b * ((6 if case["next"] else 4) * d + 2 * gates) + (n * stats + 2 * c * weights) * w,
            "flops": 20 * n * d}


# ------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, st)
    deg = torch.tensor(_degrees(case["irreps"]), device="cuda")

    def wide(name):
        return None if st.get(name) is None else st[name].double()

    def spread(c):  # a value per channel to one per column
        return torch.repeat_interleave(c, deg, dim=-1)

    def gather(t):  # the sum of each channel's columns, irrep by irrep
        parts, at = [], 0
        for term in case["irreps"].split("+"):
            mul, k = int(term.split("x")[0]), 2 * int(term.split("x")[1][:-1]) + 1
            parts.append(t[:, at:at + mul * k].reshape(-1, mul, k).sum(2))
            at += mul * k
        return torch.cat(parts, 1)

    def normed(x):
        return x / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + EPS)

    def through_norm(x, g):  # d/dx of <g, normed(x)>
        q = (x * x).sum(1, keepdim=True) / x.shape[1] + EPS
        return g / q.sqrt() - x * (g * x).sum(1, keepdim=True) / (x.shape[1] * q.pow(1.5))

    if case["op"] == "norm":
        x, w = wide("x"), wide("w")
        if case["dir"] == "fwd":
            return {"u": normed(x) * spread(w), "rstd": 1 / torch.sqrt((x * x).sum(1) / x.shape[1] + EPS)}
        du = wide("grad_u")
        dx = through_norm(x, du * spread(w))
        if case["add"]:
            dx += wide("grad_add")
        return {"x": dx, "w": gather(du * normed(x)).sum(0)}
    f, gate, scale, w_post, w_next = wide("f"), wide("gate"), wide("scale"), wide("w_post"), wide("w_next")
    fhat = f if w_post is None else normed(f)
    both = scale if w_post is None else scale * w_post
    act = {"identity": lambda g: g, "tanh": torch.tanh, "sigmoid": lambda g: 1 / (1 + torch.exp(-g)),
           "silu": lambda g: g / (1 + torch.exp(-g))}[case["act"]]
    slope = {"identity": torch.ones_like, "tanh": lambda g: torch.cosh(g).pow(-2),
             "sigmoid": lambda g: (2 * torch.cosh(g / 2)).pow(-2),
             "silu": lambda g: 1 / (1 + torch.exp(-g)) + g * (2 * torch.cosh(g / 2)).pow(-2)}[case["act"]]
    a = torch.ones(1, 1, dtype=torch.float64, device="cuda") if gate is None else act(gate)
    a_cols = a if a.shape[1] == 1 else spread(a)
    if case["dir"] == "fwd":
        h = wide("r") + a_cols * spread(both) * fhat
        return {"h": h, "u": None if w_next is None else normed(h) * spread(w_next),
                "rstd_f": None if w_post is None else 1 / torch.sqrt((f * f).sum(1) / f.shape[1] + EPS),
                "rstd_h": None if w_next is None else 1 / torch.sqrt((h * h).sum(1) / f.shape[1] + EPS)}
    dh, out = wide("grad_h"), {}
    if w_next is not None:
        h, du = wide("h"), wide("grad_u")
        # the statistic is an input: it was taken from the sum before its rounding
        hhat = h * wide("rstd_h")[:, None]
        g = du * spread(w_next)
        dh = dh + wide("rstd_h")[:, None] * (g - hhat * (g * hhat).sum(1, keepdim=True) / h.shape[1])
        out["w_next"] = gather(du * hhat).sum(0)
    out["r"] = dh
    t = gather(dh * fhat)
    if gate is not None:
        out["gate"] = slope(gate) * ((t * both).sum(1, keepdim=True) if gate.shape[1] == 1 else t * both)
    t = (t * a).sum(0)
    out["scale"] = t if w_post is None else t * w_post
    dy = dh * a_cols * spread(both)
    if w_post is not None:
        out["w_post"] = t * scale
        dy = through_norm(f, dy)
    out["f"] = dy
    return out


def _exact_adamw(case, st):
    hy, step = HYPER, st["step"] + 1
    g, norm = st["g"].double(), None
    if case["clip"]:
        norm = torch.linalg.vector_norm(g)
        g = g * min(1.0, hy["max_norm"] / float(norm))
    m, v = st["m"].double(), st["v"].double()
    if case["bits"] == 8:
        by = st["scales"].double().repeat_interleave(BLOCK, dim=1)
        m, v = by[0] * m.sign() * (m / 127) ** 2, (by[1] * (v / 255) ** 2) ** 2
    m = hy["beta1"] * m + (1 - hy["beta1"]) * g
    v = hy["beta2"] * v + (1 - hy["beta2"]) * g ** 2
    p = st["p"].double() if st["master"] is None else st["master"].double()
    mhat, vhat = m / (1 - hy["beta1"] ** step), v / (1 - hy["beta2"] ** step)
    p = p - hy["lr"] * (mhat / (vhat.sqrt() + hy["eps"]) + hy["weight_decay"] * p)
    eight = case["bits"] == 8  # a code next to a border goes by the last bit of 32
    return {"p": p, "master": None if st["master"] is None else p, "norm": None if norm is None else norm.view(1),
            "m": None if eight else m, "v": None if eight else v}
