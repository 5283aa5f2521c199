"""Cases and plain forms of the operators of a mixture of experts over node features.

Rows are nodes; element (channel u, component m) of an irrep at offset + u*(2l+1) + (m + l).

gnorm   group norm and activation over a batch of graphs, channels last: graph b holds the rows
        ptr[b]..ptr[b+1]; over its rows and a group's channels, m and v are mean and variance,
        y = act((x - m) (v + eps)^(-1/2) w[c] + b[c]).
route   the experts of each row: scores s = softmax(logits) or sigmoid(logits), choice by s + bias: the
        groups of experts with the largest sums of their best two, in them the top_k; weights
        scale s or scale s / (sum of the chosen s).  With it the lists that products and gradients of
        the experts go by: rows by the pair of their lowest experts, slots (row * top_k + choice) by
        expert, each expert's first slot.
linear  out[n] = sum_j p[n, j] W[e(n, j)] x[n], a matrix [mul_out][mul_in] for each pair of equal
        irreps (inputs' order, then outputs'), every component of a channel mixed alike.

``run`` computes a case in elementary torch operations, or by the library where ``own`` is true.
"""
import math
import random

import torch

own = False

EPS = 1e-5
TORCH = {"f32": torch.float32, "f64": torch.float64, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "f64": 8, "bf16": 2, "f16": 2}
BINS = 4096  # of the rows' order


# ------------------------------------------------------------------------------------ cases

def _ladder(mul, lmax):
    return "+".join("%dx%d%s" % (mul, l, "eo"[l % 2]) for l in range(lmax + 1))


def listed():
    return [
        # two dozen small molecules, a narrow network: a launch's latency
        {"name": "gnorm-fwd-504x32-f32", "op": "gnorm", "dir": "fwd", "rows": 504, "graphs": 24, "channels": 32,
         "groups": 4, "act": "silu", "dtype": "f32"},
        # a large batch of molecules of all sizes, 16-bit features
        {"name": "gnorm-fwd-200000x64-bf16", "op": "gnorm", "dir": "fwd", "rows": 200000, "graphs": 4000,
         "channels": 64, "groups": 8, "act": "silu", "dtype": "bf16"},
        # training on the MACE-like graph's nodes, a batch of mid-sized graphs
        {"name": "gnorm-bwd-20000x128-f32", "op": "gnorm", "dir": "bwd", "rows": 20000, "graphs": 160,
         "channels": 128, "groups": 8, "act": "silu", "dtype": "f32"},
        # a few huge graphs, odd widths
        {"name": "gnorm-bwd-199999x95-f16", "op": "gnorm", "dir": "bwd", "rows": 199999, "graphs": 3,
         "channels": 95, "groups": 5, "act": "tanh", "dtype": "f16"},
        # the rows of the small batched product, a handful of experts
        {"name": "route-fwd-1024x8-f32", "op": "route", "dir": "fwd", "rows": 1024, "experts": 8, "top_k": 2,
         "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "renorm": True, "scale": 1.0,
         "dtype": "f32"},
        # every node of the power-law graph, many experts in groups, balanced by a bias
        {"name": "route-fwd-200000x64-bf16", "op": "route", "dir": "fwd", "rows": 200000, "experts": 64, "top_k": 6,
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "renorm": True, "scale": 2.5,
         "dtype": "bf16"},
        # training: scores that are not renormalised send a gradient to every logit
        {"name": "route-bwd-20000x128-f32", "op": "route", "dir": "bwd", "rows": 20000, "experts": 128, "top_k": 4,
         "score": "softmax", "bias": True, "groups": 1, "top_groups": 1, "renorm": False, "scale": 1.0,
         "dtype": "f32"},
        # inference on one small molecule
        {"name": "linear-fwd-21x576-bf16", "op": "linear", "dir": "fwd", "rows": 21, "in": _ladder(64, 2),
         "out": _ladder(64, 2), "experts": 8, "top_k": 2, "dtype": "bf16"},
        # the NequIP-like graph's nodes
        {"name": "linear-fwd-5000x288-f32", "op": "linear", "dir": "fwd", "rows": 5000, "in": _ladder(32, 2),
         "out": _ladder(32, 2), "experts": 8, "top_k": 2, "dtype": "f32"},
        # every node of the power-law graph in 16 bits
        {"name": "linear-fwd-200000x576-bf16", "op": "linear", "dir": "fwd", "rows": 200000, "in": _ladder(64, 2),
         "out": _ladder(64, 2), "experts": 16, "top_k": 2, "dtype": "bf16"},
        # training on the MACE-like graph's nodes, every gradient
        {"name": "linear-bwd-20000x2048-f32", "op": "linear", "dir": "bwd", "rows": 20000, "in": _ladder(128, 3),
         "out": _ladder(128, 3), "experts": 8, "top_k": 2, "dtype": "f32"},
        # odd multiplicities into other ones, double precision
        {"name": "linear-bwd-4999x65-f64", "op": "linear", "dir": "bwd", "rows": 4999, "in": "19x0e+7x1o+5x2e",
         "out": "11x0e+13x1o+3x2e", "experts": 5, "top_k": 3, "dtype": "f64"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng: random.Random):
    op = rng.choice(["gnorm", "route", "linear", "linear"])
    dtype = rng.choice(["f32", "f32", "bf16", "f16", "f64"])
    case = {"op": op, "dir": rng.choice(["fwd", "bwd"]), "dtype": dtype}
    if op == "gnorm":
        groups, width = _log(rng, 1, 16), _log(rng, 1, 32)
        rows = _log(rng, 1, min(200000, 60_000_000 // (groups * width * BYTES[dtype])))
        case.update(rows=rows, graphs=_log(rng, 1, max(1, rows // 8)), channels=groups * width, groups=groups,
                    act=rng.choice(["identity", "sigmoid", "silu", "tanh"]))
    elif op == "route":
        groups, width = rng.choice([1, 1, 2, 4, 8, 5]), _log(rng, 1, 32)
        experts, top = groups * width, rng.randint(1, groups)
        case.update(rows=_log(rng, 1, min(200000, 16_000_000 // experts)), experts=experts,
                    top_k=rng.randint(1, min(8, top * width)), score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top, renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]))
    else:
        irreps = ["%d%s" % (l, p) for l in range(4) for p in "eo"]
        rng.shuffle(irreps)
        top = _log(rng, 2, 128)
        kept = irreps[:rng.randint(1, 4)]
        case["in"] = "+".join("%dx%s" % (rng.randint(1, top), t) for t in kept)
        case["out"] = "+".join("%dx%s" % (rng.randint(1, top), t) for t in rng.sample(kept, len(kept)))
        experts = _log(rng, 1, 64)
        case.update(experts=experts, top_k=rng.randint(1, min(4, experts)))
        one = work({**case, "rows": 1000})
        none = work({**case, "rows": 0})
        per = {k: (one[k] - none[k]) / 1000 for k in one}
        most = min(200e6 / per["bytes"], 20e9 / per["flops"])
        case["rows"] = _log(rng, 1, min(200000, most))
    return case


# ------------------------------------------------------------------------------------ layouts

def _irreps(text):
    """(mul, degree and parity, components, first column) of each term."""
    out, at = [], 0
    for term in text.split("+"):
        mul, lp = term.split("x")
        k = 2 * int(lp[:-1]) + 1
        out.append((int(mul), lp, k, at))
        at += int(mul) * k
    return out, at


def _paths(case):
    """(mul_in, first column, mul_out, first column, components, first weight) of each pair of equal irreps."""
    (ins, d_in), (outs, d_out) = _irreps(case["in"]), _irreps(case["out"])
    paths, at = [], 0
    for mi, ti, k, xi in ins:
        for mo, to, _, yo in outs:
            if ti == to:
                paths.append((mi, xi, mo, yo, k, at))
                at += mi * mo
    return paths, d_in, d_out, at


# ------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n, dt = case["rows"], TORCH[case["dtype"]]
    real = torch.float64 if case["dtype"] == "f64" else torch.float32

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=real, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, dtype=torch.float64, device="cuda")

    st = {"case": case, "real": real}
    if case["op"] == "gnorm":
        c = case["channels"]
        # graphs' sizes spread by a factor of a few, some of them empty where there are many
        share = torch.cumsum(torch.exp(0.7 * uniform(case["graphs"]) * 2), 0)
        ends = torch.round(share / share[-1] * n).to(torch.int32)
        st["ptr"] = torch.cat([ends.new_zeros(1), ends])
        st["x"] = (normal(n, c) * torch.exp(0.3 * normal(1, c)) + 0.5 * normal(1, c)).to(dt)
        st["w"], st["b"] = 1 + 0.1 * normal(c), 0.1 * normal(c)
        if case["dir"] == "bwd":
            st["grad_y"] = normal(n, c).to(dt)
            st["mean"], st["rstd"] = (t.contiguous() for t in _stats(st))  # as the forward leaves them
        if own:
            from clebsch_gordan_tensor_cgtp_amd import binding as cg
            st["plan"] = cg.group_norm_for(c, case["groups"], case["dtype"], act=case["act"], eps=EPS)
        return st
    e, k = case["experts"], case["top_k"]
    # some experts are liked more than others
    st["logits"] = (normal(n, e) + 0.5 * normal(1, e)).to(dt if case["op"] == "route" else real)
    if case["op"] == "route":
        st["bias"] = 0.1 * normal(e) if case["bias"] else None
        if case["dir"] == "bwd":
            st["experts"] = _choose(st)[0]
            st["grad_p"] = normal(n, k)
        if own:
            st["router"] = _router(case)
        return st
    paths, d_in, d_out, numel = _paths(case)
    st["experts"] = torch.sort(st.pop("logits"), dim=1, descending=True, stable=True)[1][:, :k].int().contiguous()
    p = uniform(n, k) + 0.1
    st["p"] = (p / p.sum(1, keepdim=True)).to(real)
    st["x"] = normal(n, d_in).to(dt)
    w = normal(e, numel)
    for mi, _, mo, _, _, at in paths:
        w[:, at:at + mi * mo] /= math.sqrt(mi)
    st["w"] = w.to(dt)
    if case["dir"] == "bwd":
        st["g"] = normal(n, d_out).to(dt)
    if own:
        from clebsch_gordan_tensor_cgtp_amd import binding as cg
        st["plan"] = cg.linear_for(case["in"], case["out"], case["dtype"], experts=e, top_k=k)
        # made with the choice of experts, whose cases count it
        st["order"] = cg.route_order(cg.router_for(e, k, "f32"), st["experts"])
    return st


def _router(case):
    from clebsch_gordan_tensor_cgtp_amd import binding as cg
    return cg.router_for(case["experts"], case["top_k"], case["dtype"], score=case["score"], groups=case["groups"],
                         top_groups=case["top_groups"], renormalise=case["renorm"], scale=case["scale"])


# ------------------------------------------------------------------------------------ plain forms

def _wide(t):
    return t if t.dtype == torch.float64 else t.float()


def _graph_of(st):
    ptr = st["ptr"].long()
    return torch.repeat_interleave(ptr[1:] - ptr[:-1], output_size=st["case"]["rows"])


def _graph_sums(st, t):
    """Sums over a graph's rows and a group's channels: [N][C] to [graphs][groups], in 64 bits, as
    differences of running sums."""
    c = st["case"]
    rows = t.view(c["rows"], c["groups"], -1).sum(2, dtype=torch.float64)
    running = torch.zeros(c["groups"], c["rows"] + 1, dtype=torch.float64, device=t.device)
    torch.cumsum(rows.t().contiguous(), 1, out=running[:, 1:])
    at = running[:, st["ptr"].long()]
    return (at[:, 1:] - at[:, :-1]).t()


def _counts(st):
    ptr = st["ptr"].long()
    return ((ptr[1:] - ptr[:-1]) * (st["case"]["channels"] // st["case"]["groups"])).clamp(min=1).double()[:, None]


def _columns(st, graph, t):
    """A value per graph and group to one per row and channel."""
    c = st["case"]
    return t[graph].repeat_interleave(c["channels"] // c["groups"], 1)


def _stats(st):
    graph, n, x = _graph_of(st), _counts(st), _wide(st["x"])
    mean = _graph_sums(st, x) / n
    off = x - _columns(st, graph, mean.to(x.dtype))
    var = _graph_sums(st, off * off) / n
    return mean.to(x.dtype), torch.rsqrt(var + EPS).to(x.dtype)


def _act(kind, z):
    """The activation and its derivative."""
    if kind == "identity":
        return z, torch.ones_like(z)
    if kind == "tanh":
        a = torch.tanh(z)
        return a, 1 - a * a
    s = torch.sigmoid(z)
    return (s, s * (1 - s)) if kind == "sigmoid" else (z * s, s * (1 + z * (1 - s)))


def _gnorm(st):
    case, dt = st["case"], st["x"].dtype
    graph, x = _graph_of(st), _wide(st["x"])
    if case["dir"] == "fwd":
        mean, rstd = _stats(st)
        z = (x - _columns(st, graph, mean)) * _columns(st, graph, rstd) * st["w"] + st["b"]
        return {"y": _act(case["act"], z)[0].to(dt), "mean": mean, "rstd": rstd}
    r = _columns(st, graph, st["rstd"])
    xh = (x - _columns(st, graph, st["mean"])) * r
    dz = _wide(st["grad_y"]) * _act(case["act"], xh * st["w"] + st["b"])[1]
    q, n = dz * st["w"], _counts(st)
    a = _columns(st, graph, (_graph_sums(st, q) / n).to(x.dtype))
    b = _columns(st, graph, (_graph_sums(st, q * xh) / n).to(x.dtype))
    return {"x": (r * (q - a - xh * b)).to(dt), "w": (dz * xh).sum(0, dtype=torch.float64).to(x.dtype),
            "b": dz.sum(0, dtype=torch.float64).to(x.dtype)}


def _scores(st):
    x = st["logits"].double()
    return torch.softmax(x, 1) if st["case"]["score"] == "softmax" else torch.sigmoid(x)


def _choose(st):
    """(experts, scores): in 64 bits, as a choice between neighbours must not hang on a rounding."""
    case, s = st["case"], _scores(st)
    c = s if st["bias"] is None else s + st["bias"].double()
    if case["top_groups"] < case["groups"]:
        in_groups = c.view(c.shape[0], case["groups"], -1)
        best = torch.sort(in_groups, dim=2, descending=True)[0][:, :, :2].sum(2)
        taken = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, taken, True)
        c = torch.where(keep[:, :, None], in_groups, -math.inf).view_as(c)
    return torch.sort(c, dim=1, descending=True, stable=True)[1][:, :case["top_k"]].int().contiguous(), s


def _route(st):
    case, real = st["case"], st["real"]
    if case["dir"] == "fwd":
        experts, s = _choose(st)
        p = s.gather(1, experts.long())
        if case["renorm"]:
            p = p / p.sum(1, keepdim=True)
        rows, slots, offsets = _lists(case, experts)
        return {"experts": experts, "p": (p * case["scale"]).to(real), "rows": rows, "slots": slots,
                "offsets": offsets}
    dt, idx, dp = st["logits"].dtype, st["experts"].long(), st["grad_p"] * case["scale"]
    s = _scores(st).to(real)
    p = s.gather(1, idx)
    if case["renorm"]:
        total = p.sum(1, keepdim=True)
        dp = (dp - (dp * p).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, idx, dp)
    if case["score"] == "sigmoid":
        return (ds * s * (1 - s)).to(dt)
    return (s * (ds - (ds * s).sum(1, keepdim=True))).to(dt)


def _lists(case, experts):
    """Rows by the pair of their lowest experts (as many bins of the second as there is room for), slots
    by expert, each expert's first slot."""
    e, k = case["experts"], case["top_k"]
    low = torch.sort(experts, dim=1)[0].long()
    key = low[:, 0]
    if k > 1:
        bins = min(e, BINS // e)
        key = key * bins + low[:, 1] * bins // e
    slots = torch.sort(experts.reshape(-1), stable=True)[1].int()
    count = torch.bincount(experts.reshape(-1).long(), minlength=e)
    offsets = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)]).int()
    return torch.sort(key, stable=True)[1].int(), slots, offsets


def _linear(st):
    case, dt = st["case"], st["x"].dtype
    paths, d_in, d_out, numel = _paths(case)
    x, w, n, k = _wide(st["x"]), _wide(st["w"]), case["rows"], case["top_k"]
    backward = case["dir"] == "bwd"
    g = _wide(st["g"]) if backward else None
    out = x.new_zeros(n, d_in if backward else d_out)
    dw, dp = torch.zeros_like(w), torch.zeros_like(st["p"])
    for e in range(case["experts"]):
        row, choice = torch.nonzero(st["experts"] == e, as_tuple=True)
        p = st["p"][row, choice][:, None]
        xe = x[row]
        if not backward:
            part = x.new_zeros(len(row), d_out)
            for mi, xi, mo, yo, c, at in paths:
                a = xe[:, xi:xi + mi * c].view(-1, mi, c).transpose(1, 2).reshape(-1, mi)
                y = a @ w[e, at:at + mi * mo].view(mo, mi).t()
                part[:, yo:yo + mo * c] += y.view(-1, c, mo).transpose(1, 2).reshape(-1, mo * c)
            out.index_add_(0, row, part * p)
            continue
        ge, part = g[row], x.new_zeros(len(row), d_in)
        for mi, xi, mo, yo, c, at in paths:
            a = xe[:, xi:xi + mi * c].view(-1, mi, c).transpose(1, 2)
            b = ge[:, yo:yo + mo * c].view(-1, mo, c).transpose(1, 2)
            t = b.reshape(-1, mo) @ w[e, at:at + mi * mo].view(mo, mi)
            part[:, xi:xi + mi * c] += t.view(-1, c, mi).transpose(1, 2).reshape(-1, mi * c)
            dw[e, at:at + mi * mo] = ((b * p[:, :, None]).reshape(-1, mo).t() @ a.reshape(-1, mi)).reshape(-1)
        dp[row, choice] = (part * xe).sum(1)
        out.index_add_(0, row, part * p)
    return {"x": out.to(dt), "w": dw.to(dt), "p": dp} if backward else out.to(dt)


def run(state):
    if own:
        return _run_own(state)
    return {"gnorm": _gnorm, "route": _route, "linear": _linear}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------ the library

def _run_own(st):
    from clebsch_gordan_tensor_cgtp_amd import binding as cg
    case = st["case"]
    if case["op"] == "gnorm":
        if case["dir"] == "fwd":
            y, mean, rstd = cg.group_norm_forward(st["plan"], st["x"], st["ptr"], st["w"], st["b"])
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dw, db = cg.group_norm_backward(st["plan"], st["x"], st["ptr"], st["w"], st["b"], st["mean"], st["rstd"],
                                            st["grad_y"])
        return {"x": dx, "w": dw, "b": db}
    if case["op"] == "route":
        if case["dir"] == "fwd":
            experts, p = cg.route_forward(st["router"], st["logits"], st["bias"])
            order = cg.route_order(st["router"], experts)
            return {"experts": experts, "p": p, "rows": order.rows, "slots": order.slots, "offsets": order.offsets}
        return cg.route_backward(st["router"], st["logits"], st["experts"], st["grad_p"])
    if case["dir"] == "fwd":
        return cg.linear_forward(st["plan"], st["x"], st["w"], st["experts"], st["p"], st["order"])
    dx, dw, dp = cg.linear_backward(st["plan"], st["x"], st["w"], st["g"], st["experts"], st["p"], st["order"])
    return {"x": dx, "w": dw, "p": dp}


# ------------------------------------------------------------------------------------ work

def work(case):
    """Every input read once, every output written once."""
    n, b = case["rows"], BYTES[case["dtype"]]
    real = 8 if case["dtype"] == "f64" else 4
    if case["op"] == "gnorm":
        c, stats = case["channels"], 2 * case["graphs"] * case["groups"] * real
        if case["dir"] == "fwd":
            return {"bytes": 2 * n * c * b + stats + 2 * c * real + 4 * case["graphs"], "flops": 15 * n * c}
        return {"bytes": 3 * n * c * b + stats + 4 * c * real + 4 * case["graphs"], "flops": 30 * n * c}
    e, k = case["experts"], case["top_k"]
    if case["op"] == "route":
        if case["dir"] == "fwd":
            return {"bytes": n * (e * b + k * (4 + real) + 4 + 4 * k) + 4 * e, "flops": n * e * 15}
        reads = e if case["score"] == "softmax" and not case["renorm"] else k
        return {"bytes": n * ((e + reads) * b + k * (4 + real)), "flops": n * reads * 15}
    paths, d_in, d_out, numel = _paths(case)
    flops = 2 * n * k * sum(mi * mo * c for mi, _, mo, _, c, _ in paths)
    used = min(e, n * k)  # experts that some row may take; a gradient is written for every one
    if case["dir"] == "fwd":
        return {"bytes": n * ((d_in + d_out) * b + k * (4 + real)) + used * numel * b, "flops": flops}
    return {"bytes": n * ((2 * d_in + d_out) * b + k * (4 + 2 * real)) + (used + e) * numel * b, "flops": 2 * flops}


# ------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"gnorm": _exact_gnorm, "route": _exact_route, "linear": _exact_linear}[case["op"]](case, st)


def _exact_gnorm(case, st):
    x, w, b = st["x"].double(), st["w"].double(), st["b"].double()
    ends, g = st["ptr"].tolist(), case["groups"]
    act = {"identity": lambda z: z, "tanh": torch.tanh, "sigmoid": lambda z: 1 / (1 + torch.exp(-z)),
           "silu": lambda z: z / (1 + torch.exp(-z))}[case["act"]]
    slope = {"identity": torch.ones_like, "tanh": lambda z: torch.cosh(z).pow(-2),
             "sigmoid": lambda z: (2 * torch.cosh(z / 2)).pow(-2),
             "silu": lambda z: 1 / (1 + torch.exp(-z)) + z * (2 * torch.cosh(z / 2)).pow(-2)}[case["act"]]
    if case["graphs"] > 8000:
        return None
    out, mean, rstd, dw, db = torch.zeros_like(x), [], [], torch.zeros_like(w), torch.zeros_like(b)
    wg, bg = w.view(1, g, -1), b.view(1, g, -1)
    for i, (lo, hi) in enumerate(zip(ends, ends[1:])):
        xs = x[lo:hi].view(hi - lo, g, -1)
        if case["dir"] == "fwd":
            if hi == lo:
                mean.append(x.new_zeros(g))
                rstd.append(x.new_full((g,), EPS ** -0.5))
                continue
            m = xs.mean((0, 2))
            r = 1 / torch.sqrt(xs.var((0, 2), unbiased=False) + EPS)
            mean.append(m)
            rstd.append(r)
            out[lo:hi] = act((xs - m[:, None]) * r[:, None] * wg + bg).view(hi - lo, -1)
            continue
        if hi == lo:
            continue
        # the statistics are inputs here: they were rounded when the forward stored them
        r = st["rstd"][i].double()[:, None]
        xh = (xs - st["mean"][i].double()[:, None]) * r
        dz = st["grad_y"][lo:hi].double().view_as(xs) * slope(xh * wg + bg)
        dw += (dz * xh).sum(0).view(-1)
        db += dz.sum(0).view(-1)
        q = dz * wg
        out[lo:hi] = (r * (q - q.mean((0, 2))[:, None] - xh * (q * xh).mean((0, 2))[:, None])).view(hi - lo, -1)
    if case["dir"] == "fwd":
        return {"y": out, "mean": torch.stack(mean), "rstd": torch.stack(rstd)}
    return {"x": out, "w": dw, "b": db}


def _exact_route(case, st):
    x, k, e, scale = st["logits"].double(), case["top_k"], case["experts"], case["scale"]
    if case["score"] == "softmax":
        s = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    else:
        s = 1 / (1 + torch.exp(-x))
    if case["dir"] == "bwd":
        # the chain rule through every step, by differentiating the definition
        leaf = x.clone().requires_grad_(True)
        s = torch.exp(leaf - torch.logsumexp(leaf, 1, keepdim=True)) if case["score"] == "softmax" else \
            1 / (1 + torch.exp(-leaf))
        p = torch.gather(s, 1, st["experts"].long())
        p = scale * (p / p.sum(1, keepdim=True) if case["renorm"] else p)
        return torch.autograd.grad((p * st["grad_p"].double()).sum(), leaf)[0]
    c = s.clone() if st["bias"] is None else s + st["bias"].double()
    if case["top_groups"] < case["groups"]:
        width, cols = e // case["groups"], []
        for g in range(case["groups"]):
            own_cols = c[:, g * width:(g + 1) * width]
            first = own_cols.max(1)
            if width > 1:
                rest = own_cols.scatter(1, first[1][:, None], -math.inf)
                cols.append(first[0] + rest.max(1)[0])
            else:
                cols.append(first[0])
        best = torch.stack(cols, 1)
        # a group stays where fewer than top_groups others beat it (an equal one before it does)
        i = torch.arange(case["groups"], device=x.device)
        beats = (best[:, None, :] > best[:, :, None]) | ((best[:, None, :] == best[:, :, None]) & (i[None, :] < i[:, None]))
        keep = beats.sum(2) < case["top_groups"]
        c = torch.where(keep.repeat_interleave(width, 1), c, torch.full_like(c, -math.inf))
    picks = []
    for _ in range(k):
        most = c.max(1, keepdim=True)[0]
        i = torch.where(c == most, torch.arange(e, device=x.device), e).min(1)[0]  # the first of equals
        picks.append(i)
        c = c.scatter(1, i[:, None], -math.inf)
    experts = torch.stack(picks, 1)
    p = torch.gather(s, 1, experts)
    p = scale * (p / p.sum(1, keepdim=True) if case["renorm"] else p)
    # sorting by a key that holds the place as well leaves no ties
    n, big = case["rows"], case["rows"] * k
    flat = experts.reshape(-1)
    slots = torch.argsort(flat * big + torch.arange(big, device=x.device))
    offsets = torch.stack([(flat < i).sum() for i in range(e + 1)])
    lowest = experts.min(1)[0]
    key = lowest
    if k > 1:
        second = torch.where(experts == lowest[:, None], e, experts).min(1)[0]
        bins = min(e, BINS // e)
        key = lowest * bins + torch.div(second * bins, e, rounding_mode="floor")
    rows = torch.argsort(key * n + torch.arange(n, device=x.device))
    return {"experts": experts.int(), "p": p, "rows": rows.int(), "slots": slots.int(), "offsets": offsets.int()}


def _exact_linear(case, st):
    paths, d_in, d_out, numel = _paths(case)
    x, w, p, n = st["x"].double(), st["w"].double(), st["p"].double(), case["rows"]
    # each row's weight for each expert
    mix = torch.zeros(n, case["experts"], dtype=torch.float64, device="cuda").scatter_(1, st["experts"].long(), p)
    out = x.new_zeros(n, d_in if case["dir"] == "bwd" else d_out)
    dw, dmix = torch.zeros_like(w), torch.zeros_like(mix)
    for mi, xi, mo, yo, c, at in paths:
        xs = x[:, xi:xi + mi * c].view(n, mi, c)
        gs = st["g"].double()[:, yo:yo + mo * c].view(n, mo, c) if case["dir"] == "bwd" else None
        for e in range(case["experts"]):
            we, some = w[e, at:at + mi * mo].view(mo, mi), torch.nonzero(mix[:, e])[:, 0]
            xe, pe = xs[some], mix[some, e]
            for m in range(c):
                if gs is None:
                    cols = yo + m + c * torch.arange(mo, device="cuda")
                    out[some[:, None], cols] += pe[:, None] * (xe[:, :, m] @ we.t())
                    continue
                ge = gs[some][:, :, m]
                back = ge @ we
                out[some[:, None], xi + m + c * torch.arange(mi, device="cuda")] += pe[:, None] * back
                dw[e, at:at + mi * mo] += ((ge * pe[:, None]).t() @ xe[:, :, m]).reshape(-1)
                dmix[some, e] += (back * xe[:, :, m]).sum(1)
    if case["dir"] == "fwd":
        return out
    return {"x": out, "w": dw, "p": dmix.gather(1, st["experts"].long())}
