"""Every kernel of the norm, each at widths that reach it: the plan says which
one it is, so that a rule which moves the widths to another kernel fails here
instead of leaving one without a test (tolerances: test_norm.py's)."""
import ctypes

import pytest
import torch

from tests.test_norm import BF16, E4M3, EPS, Norm, check, check_backward, untouched
from warp_specialized_pipelined_amd import migemm

BAD = migemm.MIGEMM_ERR_INVALID_ARG


def test_info_refuses_what_is_not_a_norm_plan():
    lib = migemm.load()
    junk = ctypes.create_string_buffer(b"\xff" * 4096)
    info = migemm.migemm_norm_info()
    for p in (None, ctypes.addressof(junk)):
        assert lib.gemm_norm_plan_get_info(p, ctypes.byref(info)) == BAD
    assert bytes(info) == bytes(ctypes.sizeof(info))


# Rows, columns, and the waves a row and vectors a lane, forward and backward:
# the first and the last width of each, and one that ends inside a vector.
SIZES = [
    ((256, 512), (1, 1)), ((256, 513), (4, 1)), ((256, 2048), (4, 1)), ((256, 2049), (16, 1)),
    ((100, 8192), (16, 1)), ((100, 8193), (16, 2)), ((50, 16384), (16, 2)), ((50, 16385), (16, 4)),
    ((257, 512), (1, 1)), ((1029, 513), (1, 2)), ((1200, 1021), (1, 2)), ((700, 1024), (1, 2)),
    ((1100, 1025), (1, 4)), ((2053, 1531), (1, 4)), ((300, 2048), (1, 4)),
    ((300, 2049), (4, 2)), ((1031, 3333), (4, 2)), ((257, 4096), (4, 2)),
    ((300, 4097), (4, 4)), ((1050, 5000), (4, 4)), ((513, 8001), (4, 4)), ((260, 8192), (4, 4)),
    ((300, 8193), (16, 2)), ((257, 16384), (16, 2)), ((270, 16391), (16, 4)), ((257, 32768), (16, 4)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("size,shape", SIZES, ids=["x".join(map(str, s)) for s, _ in SIZES])
@pytest.mark.parametrize("y_type", [BF16, E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("residual", [True, False], ids=["residual", "plain"])
def test_kernel(size, shape, y_type, residual):
    p = Norm(*size, y_type, residual, seed=size[0] + 3 * size[1])
    i = p.plan.info
    assert (i.forward_waves, i.forward_vectors) == shape == (i.backward_waves, i.backward_vectors)
    p.forward()
    p.backward()
    torch.cuda.synchronize()
    check(p)
    check_backward(p)
    untouched(p, ["y", "dx"] + (["h"] if residual else []))


@pytest.mark.gpu
def test_info_of_other_plans():
    i = migemm.NormPlan(700, 5000, EPS, x_rs=5000, y_rs=5000).info
    assert (i.forward_waves, i.forward_vectors) == (4, 4)
    assert (i.backward_waves, i.backward_vectors, i.backward_workgroups) == (0, 0, 0)
    assert i.cu_count == torch.cuda.get_device_properties(0).multi_processor_count
    lib, info = migemm.load(), migemm.migemm_norm_info()
    s = migemm.ScaledPlan(4, 64, 64, a_rs=64, b_cs=64, d_rs=64)
    assert lib.gemm_norm_plan_get_info(s.handle, ctypes.byref(info)) == BAD
    n = Norm(4, 64)
    assert lib.gemm_norm_plan_get_info(n.plan.handle, None) == BAD
    # one workgroup walks few rows; two a compute unit walk many
    assert n.plan.info.backward_workgroups == 1
    assert Norm(5000, 64).plan.info.backward_workgroups == min(5000 // 4, 2 * i.cu_count)
