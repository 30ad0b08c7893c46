"""What calls of the block's operators may share: a workspace between graphs and
eager calls that run one after another, a matrix between several arguments that
are read, and the library between host threads with plans of their own."""
import threading

import pytest
import torch

from tests.test_block_norm import INT8, Block
from tests.test_checkpoint import FP32, Checkpoint
from tests.test_int8 import Int8
from tests.test_quantize import Rows
from warp_specialized_pipelined_amd import migemm

pytestmark = pytest.mark.gpu


def test_graphs_that_share_a_workspace():
    a, b = Int8(2205, 18, 13802, seed=1), Int8(34, 2802, 15899, seed=2)
    c, n = Checkpoint(1421, 18, 19, FP32, seed=3), Block(700, 4100, seed=4)
    c.pack()
    n.forward()
    assert a.plan.info.splits > 1 and b.plan.info.splits > 1 and c.plan.info.splits > 1
    sizes = [p.plan.workspace_size for p in (a, b, c, n)]
    ws = torch.full((max(sizes),), 0xFF, dtype=torch.uint8, device="cuda")
    for p in (a, b, c, n):
        p.ws = ws
    calls = [(a.run, lambda: [a.d]), (b.run, lambda: [b.d]), (c.gradient, lambda: [c.dw]),
             (n.backward, lambda: [n.dx, n.dz, n.dr, n.dweight, n.dpost_weight])]
    want, graphs = [], []
    for call, out in calls:
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in out()])
    a.check()
    b.check()
    c.check_gradient()
    for call, _ in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for turn in range(3):
        for _, out in calls:
            for t in out():
                t.fill_(7)
        ws.fill_(turn)
        for k in range(4):
            graphs[(k + turn) % 4].replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(calls, want):
            assert all(torch.equal(x, y) for x, y in zip(out(), w))
        for k, (call, out) in enumerate(calls):
            graphs[(k + 1) % 4].replay()
            call()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(out(), want[k]))


def test_one_matrix_for_several_arguments():
    p, q = Block(300, 1999, seed=5), Block(300, 1999, seed=5)
    for t in (p.z, p.r):
        t.copy_(p.x)
    p.dh.copy_(p.dy)
    p.weight.copy_(p.post_weight)
    p.forward()
    p.backward()
    q.x.copy_(p.x)
    q.dy.copy_(p.dy)
    q.post_weight.copy_(p.post_weight)
    q.z, q.r, q.dh, q.weight = q.x, q.x, q.dy, q.post_weight
    q.forward()
    q.backward()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(p.outputs(), q.outputs()))
    a = Int8(300, 300, 1000, seed=6)
    a.b, a.sb = a.a, a.sa
    a.run()
    torch.cuda.synchronize()
    a.check()


def test_host_threads():
    """Plans made, run and destroyed on four threads, each on its own stream."""
    kinds = [lambda: Int8(300, 500, 2000, seed=1), lambda: Block(300, 2001, INT8, seed=2),
             lambda: Checkpoint(700, 300, 200, FP32, seed=3), lambda: Rows(torch.randn(
                 300, 9001, generator=torch.Generator().manual_seed(4)).bfloat16())]

    def run(p, stream=None):
        if isinstance(p, Block):
            p.forward(stream)
            p.backward(stream)
            return p.outputs()
        if isinstance(p, Checkpoint):
            p.pack(stream)
            p.gradient(stream)
            return [p.dw, p.kept]
        p.run(stream)
        return [p.d] if isinstance(p, Int8) else [p.q_full, p.scale]

    sets = [[make() for make in kinds] for _ in range(4)]
    want = [[t.clone() for t in run(p)] for p in sets[0]]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    errors = []

    def work(problems, stream):
        try:
            for _ in range(20):
                for p in problems:
                    d = p.plan.desc
                    again = object.__new__(type(p.plan))
                    migemm._OperatorPlan.__init__(again, d)
                    p.plan = again
                    run(p, stream)
            stream.synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(sets, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for problems in sets:
        for p, w in zip(problems, want):
            got = p.outputs() if isinstance(p, Block) else (
                [p.dw, p.kept] if isinstance(p, Checkpoint) else ([p.d] if isinstance(p, Int8) else [p.q_full, p.scale]))
            assert all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
                       for x, y in zip(got, w))
