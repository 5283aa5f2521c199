"""Refusals of the schedule that counts only the steps taken, before any GPU call (the addresses are
never dereferenced)."""
import ctypes

from clebsch_gordan_tensor_cgtp_amd import binding as cg

INVAL = cg.STATUS_CODES["CGTP_ERR_INVALID_ARG"]


def test_schedule_with_a_norm_refusals():
    L, at = cg.lib(), lambda n: ctypes.c_void_p((1 << 20) + n)
    go = lambda sch=at(0), b1=0.9, b2=0.999, norm=at(64), scale=1.0: L.cgtp_adamw_schedule_norm(  # noqa: E731
        sch, b1, b2, norm, scale, None)
    assert go(sch=None) == INVAL and go(sch=at(4)) == INVAL and go(norm=at(68)) == INVAL
    assert go(b1=1.0) == INVAL and go(b1=-0.1) == INVAL and go(b2=float("nan")) == INVAL
    for bad in (float("nan"), float("inf")):
        assert go(scale=bad) == INVAL and "grad_scale" in cg.last_error()
    assert go(norm=at(24)) == INVAL and "overlaps" in cg.last_error()
