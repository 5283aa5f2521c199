"""Train two residual convolution blocks to match a teacher of the same shape.

    python examples/train_blocks.py [--steps 60] [--bits 8] [--experts 8]

Each block: the row norm, the fully connected (uvw) convolution over the graph, and the join, which
norms the convolution's output, gates it per channel by scalars that the convolution makes beside it
(both stay in one buffer, side by side), adds the residual and norms the sum for the next block.  With experts
a mixture of linear layers follows: the scalars' group norm over the graph, a linear head on it, two experts for each
node by the head's logits, and their products of the node's features.  The step
is captured into a HIP graph once and replayed: forward, backward, the gradients' global norm, clipping and
AdamW with the step's number on the device.  Everything runs in the library's kernels; torch holds the memory.
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402

from clebsch_gordan_tensor_cgtp_amd import binding as cg  # noqa: E402
from clebsch_gordan_tensor_cgtp_amd import synth  # noqa: E402

MUL, LMAX, BLOCKS = 16, 2, 2
FEATURES = f"{MUL}x0e+{MUL}x1o+{MUL}x2e"
GATES = 3 * MUL                                            # one per channel of the features
OUT = f"{GATES + MUL}x0e+{MUL}x1o+{MUL}x2e"                 # gates first, then the features


class Net:
    """Weights, their gradients and the buffers of one graph's forward and backward."""

    def __init__(self, graph, vec, seed, device, experts=0, dtype="f32"):
        import torch
        self.row_ptr, self.col = graph
        self.n = self.row_ptr.shape[0] - 1
        self.plan = cg.Plan(FEATURES, cg.sh_irreps(LMAX), OUT, "uvw", dtype)
        self.entry = cg.block_for(FEATURES, dtype)
        self.block = cg.block_for(FEATURES, dtype, gate="channel", act="sigmoid", post_norm=True, next_norm=True)
        self.y = cg.spherical_harmonics(LMAX, vec)
        self.transpose = cg.graph_transpose(self.row_ptr, self.col)
        c = self.block.channels
        gen = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=gen, device=device, dtype=vec.dtype)  # noqa: E731
        one = lambda: 1 + 0.1 * normal(c)  # noqa: E731
        self.params = [one()]                              # the entry norm's
        for _ in range(BLOCKS):                            # W, post, scale, next
            w = normal(self.plan.weight_numel) * 0.1
            self.params += [w, one(), 0.5 * one(), one()]
        self.experts = experts
        if experts:                                        # the group norm's weight and bias, the head, the experts
            self.norm = cg.group_norm_for(MUL, 4, dtype, act="silu", eps=1e-5)
            self.head = cg.linear_for(f"{MUL}x0e", f"{experts}x0e", dtype)
            self.router = cg.router_for(experts, 2, dtype)
            self.linear = cg.linear_for(FEATURES, FEATURES, dtype, experts=experts, top_k=2)
            self.graphs = torch.tensor([0, self.n], dtype=torch.int32, device=device)
            self.params += [1 + 0.1 * normal(MUL), 0.1 * normal(MUL), 0.5 * normal(1, self.head.weight_numel),
                            normal(experts, self.linear.weight_numel) / MUL ** 0.5]
        self.grads = [torch.zeros_like(p) for p in self.params]

    def forward(self, x):
        """The last norm's rows, and what the backward reads."""
        u, rstd = cg.norm_forward(self.entry, x, self.params[0])
        kept, h = [(x, rstd)], x
        for b in range(BLOCKS):
            w, post, scale, nxt = self.params[1 + 4 * b:5 + 4 * b]
            out = cg.conv_forward(self.plan, self.row_ptr, self.col, u, self.y, w)
            f, gate = out[:, GATES:], out[:, :GATES]
            before = u
            h, u, rf, rh = cg.join_forward(self.block, h, f, gate, post, scale, nxt)
            kept.append((before, f, gate, h, rf, rh))
        if self.experts:
            w, bias, head, experts = self.params[-4:]
            z, mean, rstd = cg.group_norm_forward(self.norm, u[:, :MUL], self.graphs, w, bias)
            logits = cg.linear_forward(self.head, z, head)
            e, p = cg.route_forward(self.router, logits)
            order = cg.route_order(self.router, e)
            kept.append((u, z, mean, rstd, logits, e, p, order))
            u = cg.linear_forward(self.linear, u, experts, e, p, order)
        return u, kept

    def backward(self, grad_u, kept):
        """The gradients of every weight, into self.grads."""
        import torch
        grad_h = None
        if self.experts:
            w, bias, head, experts = self.params[-4:]
            gw, gbias, ghead, gexperts = self.grads[-4:]
            u, z, mean, rstd, logits, e, p, order = kept[-1]
            grad_u, _, gp = cg.linear_backward(self.linear, u, experts, grad_u, e, p, order, outs=(None, gexperts, None))
            gl = cg.route_backward(self.router, logits, e, gp)
            gz = cg.linear_backward(self.head, z, head, gl, outs=(None, ghead, None))[0]
            gs = cg.group_norm_backward(self.norm, u[:, :MUL], self.graphs, w, bias, mean, rstd, gz, grad_w=gw,
                                        grad_bias=gbias)[0]
            grad_u[:, :MUL] += gs
        for b in reversed(range(BLOCKS)):
            w, post, scale, nxt = self.params[1 + 4 * b:5 + 4 * b]
            gw, gpost, gscale, gnxt = self.grads[1 + 4 * b:5 + 4 * b]
            before, f, gate, h, rf, rh = kept[1 + b]
            packed = torch.empty((self.n, self.plan.d_out), device=f.device, dtype=f.dtype)
            grad_h = cg.join_backward(self.block, grad_h, grad_u, h, f, gate, post, scale, nxt, rf, rh,
                                      outs=(None, packed[:, GATES:], packed[:, :GATES], gpost, gscale, gnxt))[0]
            grad_u, _, _ = cg.conv_backward(self.plan, self.row_ptr, self.col, self.transpose, before, self.y, w, packed,
                                            grad_w=gw, need=(True, False, True))
        x, rstd = kept[0]
        cg.norm_backward(self.entry, x, self.params[0], rstd, grad_u, grad_w=self.grads[0], need=(False, True))


def setup(device="cuda:0", nodes=2000, edges=40_000, seed=0, experts=0, dtype="f32"):
    """A graph, node features, a student and the teacher's answer."""
    import torch
    st = synth.streams(seed)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    graph = tuple(up(a) for a in synth.uniform_graph(nodes, edges, synth.rng(st["graph"])))
    real = np.float64 if dtype == "f64" else np.float32
    vec = up(synth.normal(st["vec"], (edges, 3), dtype=real))
    student, teacher = (Net(graph, vec, s, device, experts, dtype) for s in (1, 2))
    x = up(synth.normal(st["x"], (nodes, student.plan.d_x), dtype=real))
    return student, x, teacher.forward(x)[0]


def train(steps=60, bits=32, lr=1e-2, max_norm=1.0, graph=True, device="cuda:0", **kw):
    """Losses, one per step (mean squared difference from the teacher's rows)."""
    import torch
    net, x, want = setup(device, **kw)
    opt = cg.AdamW([p.numel() for p in net.params], "f32", bits)
    m, v, scales, master = opt.state(device)
    params, grads = cg.tensor_list(opt, net.params), cg.tensor_list(opt, net.grads)
    schedule = torch.tensor([0.0, lr, 0.0, 0.0], dtype=torch.float64, device=device)
    off = torch.empty_like(want)

    def step():
        u, kept = net.forward(x)
        torch.sub(u, want, out=off)
        net.backward(off * (2.0 / off.numel()), kept)
        norm = cg.grad_norm(opt, grads)
        cg.adamw_schedule(schedule, norm=norm)
        cg.adamw_step(opt, params, grads, m, v, scales, master, weight_decay=1e-4, max_norm=max_norm, norm=norm,
                      schedule=schedule)

    loss = lambda: off.square().mean().item()  # noqa: E731  (outside the graph: it is only shown)
    step()                                                 # also loads the kernels before a capture
    losses = [loss()]
    run = step
    if graph:
        captured = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(captured):
            step()
        run = captured.replay
    for _ in range(steps - 1):
        run()
        losses.append(loss())
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--bits", type=int, default=32, choices=(32, 8), help="of AdamW's moments")
    ap.add_argument("--experts", type=int, default=0, help="of the mixture behind the blocks, two to a node (0: none)")
    ap.add_argument("--eager", action="store_true", help="no captured graph")
    a = ap.parse_args()
    losses = train(a.steps, a.bits, graph=not a.eager, experts=a.experts)
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i + 1:4d}  loss {losses[i]:.5f}")
    print(f"step {len(losses):4d}  loss {losses[-1]:.5f}")


if __name__ == "__main__":
    main()
