"""What `info` of an operator's plan gives: the library's answer each time, in a
structure of its own, and an error once the plan is gone."""
import ctypes

import pytest
import torch

from warp_specialized_pipelined_amd import migemm

PLANS = {
    "norm": lambda: migemm.NormPlan(4, 64, 1e-5, x_rs=64, y_rs=64),
    "scaled": lambda: migemm.ScaledPlan(4, 64, 64, a_rs=64, b_cs=64, d_rs=64),
    "vocab_loss": lambda: migemm.VocabLossPlan(4, 64, 64, x_rs=64, w_rs=64),
    "int8": lambda: migemm.Int8Plan(4, 64, 64, a_rs=64, b_cs=64, d_rs=64),
    "quantize": lambda: migemm.QuantizePlan(4, 64, x_rs=64, q_rs=64),
    "block_norm": lambda: migemm.BlockNormPlan(4, 64, 1e-5, x_rs=64, r_rs=64, h_rs=64, y_rs=64),
    "checkpoint": lambda: migemm.CheckpointPlan(4, 64, x_rs=64),
}


def check(plan, destroy):
    first = plan.info
    want = [getattr(first, name) for name, _ in first._fields_]
    setattr(first, first._fields_[0][0], want[0] + 5)          # the caller's own copy
    again = plan.info
    assert again is not first and [getattr(again, name) for name, _ in again._fields_] == want
    destroy(plan.handle)
    with pytest.raises(migemm.MigemmError):
        plan.info
    plan.handle = None
    with pytest.raises(migemm.MigemmError):
        plan.info


class OnePlan:
    """A library with one plan of each kind, for a machine without a GPU."""

    def __init__(self):
        self.alive = False

    def __getattr__(self, name):
        if name.endswith("_plan_create"):
            def create(desc, out):
                out._obj.value, self.alive = 4096, True
                return migemm.MIGEMM_OK
            return create
        if name.endswith("_plan_destroy"):
            def destroy(handle):
                self.alive = False
                return migemm.MIGEMM_OK
            return destroy
        if name.endswith("_plan_get_info"):
            def get_info(handle, out):
                if not self.alive or handle is None:
                    return migemm.MIGEMM_ERR_INVALID_ARG
                ctypes.memset(ctypes.byref(out._obj), 1, ctypes.sizeof(out._obj))
                return migemm.MIGEMM_OK
            return get_info
        if name == "gemm_status_string":
            return lambda status: b"refused"
        raise AttributeError(name)


@pytest.mark.parametrize("kind", sorted(PLANS))
def test_info_without_a_gpu(kind, monkeypatch):
    lib = OnePlan()
    monkeypatch.setattr(migemm, "load", lambda: lib)
    plan = PLANS[kind]()
    check(plan, getattr(lib, "gemm_%s_plan_destroy" % kind))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", sorted(PLANS))
def test_info(kind):
    assert torch.cuda.is_available()
    plan = PLANS[kind]()
    check(plan, getattr(migemm.load(), "gemm_%s_plan_destroy" % kind))
