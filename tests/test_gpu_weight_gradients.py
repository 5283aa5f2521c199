"""Weight gradients over many rows, which a lane adds in its own precision one after the other: against the
float64 oracle, within the roundings that the block's geometry makes."""
import math

import numpy as np
import pytest

from clebsch_gordan_tensor_cgtp_amd import binding as cg
from oracle import block as ob

from block_cases import CONFIGS, EPS, inputs, wide, work_unit

pytestmark = pytest.mark.gpu


def roundings(block, rows):
    """Of a row's term: three sums over the row (a lane's elements one after the other, the lanes by
    halves, a product and the mean), 20 for the gate and the products.  Of the sum: the rows that a lane
    takes, a channel's columns, the workgroup's row groups; the partials are added in double and rounded."""
    per_row = 3 * (block.lane_elements + math.ceil(math.log2(block.lanes)) + 2) + 20
    groups = cg.block_workspace_size(block, rows) // (block.channels * (2 if block.next_norm else 1) *
                                                      block.real_dtype.itemsize)
    at_once = groups * max(1, 256 // block.lanes)
    return per_row + math.ceil(rows / at_once) + 15 + 256 // min(block.lanes, 256) + 2


@pytest.mark.parametrize("irreps, rows, dtype", [
    ("64x0e+64x1o+64x2e", 40_001, "f32"), ("64x0e+64x1o+64x2e", 40_001, "bf16"), ("8192x0e", 1501, "f32"),
    ("1x0e+1x1o", 300_007, "f16"), ("512x0e", 9001, "f64")])
def test_weight_gradients_over_many_rows(device, irreps, rows, dtype):
    import torch
    config = CONFIGS[0]
    t = inputs(irreps, rows, dtype, config, 29)
    d = {k: None if v is None else v.to(device) for k, v in t.items()}
    n = {k: wide(v) for k, v in t.items()}
    block = cg.block_for(irreps, dtype, gate="channel", act="sigmoid", post_norm=True, next_norm=True, eps=EPS)
    host = lambda x: x.double().cpu().numpy()  # noqa: E731

    def check(got, want, of):
        value, size = want
        off, most = np.abs(host(got) - value), roundings(of, rows) * work_unit(dtype) * size
        assert np.all(off <= most), np.max(off / most)
    plain = cg.block_for(irreps, dtype, eps=EPS)
    rstd = cg.norm_forward(plain, d["x"], d["w"])[1]
    dw = cg.norm_backward(plain, d["x"], d["w"], rstd, d["du"], need=(False, True))[1]
    check(dw, ob.norm_grad(irreps, n["x"], n["w"], host(rstd), n["du"])["grad_w"], plain)
    h, _, rf, rh = cg.join_forward(block, d["res"], d["f"], d["gate"], d["w_post"], d["scale"], d["w_next"])
    grads = cg.join_backward(block, d["dh"], d["du"], h, d["f"], d["gate"], d["w_post"], d["scale"], d["w_next"], rf, rh,
                             need=(False, False, False, True, True, True))
    want = ob.join_grad(irreps, n["dh"], n["du"], host(h), n["f"], n["gate"], n["w_post"], n["scale"], n["w_next"],
                        host(rf), host(rh), 1.0)
    for g, name in zip(grads[3:], ("grad_w_post", "grad_scale", "grad_w_next")):
        check(g, want[name], block)
    # partials in a fixed order: the same bits again
    again = cg.join_backward(block, d["dh"], d["du"], h, d["f"], d["gate"], d["w_post"], d["scale"], d["w_next"], rf, rh)
    assert all(torch.equal(a, b) for a, b in zip(grads[3:], again[3:]))
