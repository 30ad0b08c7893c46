"""examples/eight_bit_block.py against fp32, and the operators that it runs
together on two streams at once and in captured graphs."""
import importlib.util
import os

import pytest
import torch

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "eight_bit_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("eight_bit_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hidden,wide", [(512, 1024, 4096), (1, 256, 512), (77, 512, 1040)])
def test_the_example_agrees_with_fp32(example, tokens, hidden, wide):
    errors = example.main(["--tokens", str(tokens), "--hidden", str(hidden), "--wide", str(wide)])
    # A value rounded to bf16 is off by 2^-8 at most: the outputs, and y and dy
    # on their way (with the stored h, three such roundings a path).
    for k in ("h", "p", "dx", "dz", "dr", "dpost_weight", "dweight"):
        assert errors[k] < 3 * 2.0 ** -8, (k, errors)
    # int8 rows: half a code of 127 for a row's largest, which is at most the
    # square root of the columns times the row's root mean square; two products,
    # rows and weights of each.
    assert errors["out"] < 4 * 0.5 / 127 * max(hidden, wide) ** 0.5 + 2.0 ** -6, errors
    # The gradient from the kept form is exact but for fp32 sums of 2 tokens; what
    # the form itself is off by is half a step of e4m3, 2^-4.
    assert errors["dup_kept"] < 2 * (tokens + 4) * 2.0 ** -23, errors
    assert errors["dup"] < 2.0 ** -4 + 2.0 ** -8, errors


@pytest.mark.gpu
def test_two_streams_at_once(example):
    """Two programs with plans and workspaces of their own."""
    inputs = [example.Inputs(300, 512, 1040, seed) for seed in (3, 4)]
    alone = []
    for i in inputs:
        s, t = example.Serving(i), example.Training(i)
        s.run(i)
        t.forward(i)
        t.backward(i)
        torch.cuda.synchronize()
        alone.append([u.clone() for u in (s.h, s.out, t.p, t.dup, t.dx, t.dz, t.dr, t.dw, t.dpw)])
    programs = [(example.Serving(i), example.Training(i), torch.cuda.Stream()) for i in inputs]
    torch.cuda.synchronize()
    for _ in range(3):
        for (s, t, stream), i in zip(programs, inputs):
            t.dup.zero_()
            torch.cuda.synchronize()
        for (s, t, stream), i in zip(programs, inputs):
            s.run(i, stream)
            t.forward(i, stream)
            t.backward(i, stream)
        torch.cuda.synchronize()
        for (s, t, _), want in zip(programs, alone):
            for u, v in zip((s.h, s.out, t.p, t.dup, t.dx, t.dz, t.dr, t.dw, t.dpw), want):
                assert torch.equal(u, v)


@pytest.mark.gpu
def test_a_captured_step(example):
    i = example.Inputs(200, 512, 1040, 5)
    s, t = example.Serving(i), example.Training(i)

    def step():
        t.dup.zero_()
        s.run(i)
        t.forward(i)
        t.backward(i)

    step()
    torch.cuda.synchronize()
    outputs = (s.h, s.out, t.p, t.dup, t.dx, t.dz, t.dr, t.dw, t.dpw)
    want = [u.clone() for u in outputs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for u in outputs:
            u.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(outputs, want))
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(outputs, want))
