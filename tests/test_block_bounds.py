"""What the block's operators touch: every buffer lies inside a larger one that is
filled with NaN codes, on the least alignment that a call takes (matrices on 16
bytes, vectors of fp32 on 4, where the header allows it).  The results are those
of buffers of their own, bit for bit, so nothing around an input counts; around
the outputs, before the first row, between the columns and the stride, and behind
the last row, nothing changes, nor does any input."""
import pytest
import torch

from tests.test_block_kernels import INT8, KEPT
from tests.test_block_norm import BF16, E4M3, Block
from tests.test_block_norm import INT8 as INT8_ROWS
from tests.test_block_norm_in_place import GIVEN, KERNELS
from tests.test_checkpoint import FP32, Checkpoint
from tests.test_int8 import Int8
from tests.test_quantize import Rows

pytestmark = pytest.mark.gpu

AROUND = 1 << 16  # bytes before and behind


class Inside:
    """A copy of t (a vector, or a matrix with its row stride) inside NaN codes,
    `past` bytes past a multiple of 256."""

    def __init__(self, t, past=16, copy=True):
        rows, ld = (1, t.numel()) if t.dim() == 1 else (t.shape[0], t.stride(0))
        size = t.element_size()
        self.buffer = torch.full((2 * AROUND + rows * ld * size,), 0xFF, dtype=torch.uint8, device="cuda")
        first = AROUND + past
        assert self.buffer.data_ptr() % 256 == 0
        full = self.buffer[first:first + rows * ld * size].view(t.dtype)
        self.t = full if t.dim() == 1 else full.view(rows, ld)[:, :t.shape[1]]
        if copy:
            self.t.copy_(t)
        self.before = self.buffer.clone()

    def is_as_it_was(self):
        return torch.equal(self.buffer, self.before)

    def rest_is_as_it_was(self, got):
        """The result is `got`, and putting what was there back leaves what was there."""
        same = torch.equal(self.t.contiguous().view(torch.uint8), got.contiguous().view(torch.uint8))
        self.t.copy_(Inside.of(self.before, self))
        return same and self.is_as_it_was()

    @staticmethod
    def of(buffer, like):
        """The place of `like`'s tensor in another buffer."""
        first = like.t.data_ptr() - like.buffer.data_ptr()
        t = like.t
        n = t.numel() if t.dim() == 1 else t.shape[0] * t.stride(0)
        full = buffer[first:first + n * t.element_size()].view(t.dtype)
        return full if t.dim() == 1 else full.view(t.shape[0], t.stride(0))[:, :t.shape[1]]


def inside(t, past=16, copy=True):
    return None if t is None else Inside(t, past, copy)


def tensor(i):
    return None if i is None else i.t


def check(inputs, outputs):
    """outputs: (where, what it has to be)."""
    torch.cuda.synchronize()
    for i in inputs:
        assert i is None or i.is_as_it_was()
    for o, want in outputs:
        assert o is None or o.rest_is_as_it_was(want)


def workspace(ws):
    return None if ws is None else Inside(ws, 0)


def workspace_is_inside(w):
    if w is not None:
        w.t.fill_(0xFF)
        assert (w.buffer == 0xFF).all()


@pytest.mark.parametrize("M,N,K", [s for _, sizes in INT8 for s in sizes] + [(3, 5, 129), (300, 500, 2000)])
def test_int8(M, N, K):
    p = Int8(M, N, K, seed=M + N + K)
    p.run()
    torch.cuda.synchronize()
    a = [inside(t) for t in (p.a, p.sa, p.b, p.sb, p.bias)]
    d, ws = inside(p.d, copy=False), workspace(p.ws)
    p.plan.run(*[tensor(i) for i in a], d.t, tensor(ws))
    check(a, [(d, p.d)])
    workspace_is_inside(ws)


@pytest.mark.parametrize("rows,cols", [(5, 511), (2000, 1000), (2000, 1999), (5, 2047), (300, 4001), (300, 8191),
                                       (3, 8001), (3, 16001), (3, 32001), (300, 12001), (300, 16383), (300, 16385)])
@pytest.mark.parametrize("q_type", [INT8_ROWS, E4M3], ids=["int8", "e4m3"])
def test_quantize(rows, cols, q_type):
    g = torch.Generator().manual_seed(rows + cols)
    p = Rows(torch.randn(rows, cols, generator=g).bfloat16(), q_type)
    p.run()
    torch.cuda.synchronize()
    x, q, scale = inside(p.x), inside(p.q, copy=False), inside(p.scale, 4, copy=False)
    p.plan.run(x.t, q.t, scale.t)
    check([x], [(q, p.q), (scale, p.scale)])


@pytest.mark.parametrize("rows,cols", [s for _, _, sizes in KERNELS for s in sizes] + [(1, 9), (3, 16383)])
@pytest.mark.parametrize("gate,post", GIVEN, ids=["gate-post", "gate-bare", "open-post", "open-bare"])
def test_block_norm(rows, cols, gate, post):
    for y_type in (BF16, E4M3, INT8_ROWS) if gate == post else (BF16,):
        p = Block(rows, cols, y_type, post=post, gate=gate, seed=rows + cols)
        p.forward()
        p.backward()
        torch.cuda.synchronize()
        i = {n: inside(getattr(p, n)) for n in ("x", "z", "r", "post_weight", "weight")}
        o = {n: inside(getattr(p, n), copy=False) for n in ("h", "y")}
        o.update({n: inside(getattr(p, n), 4, copy=False) for n in ("scale", "post_rstd", "rstd")})
        p.plan.run(*[tensor(v) for v in (*i.values(), *o.values())])
        check(i.values(), [(v, getattr(p, n)) for n, v in o.items()])
        i = {n: inside(getattr(p, n)) for n in ("dy", "dh", "x", "z", "h", "post_weight", "weight")}
        i.update({n: inside(getattr(p, n), 4) for n in ("post_rstd", "rstd")})
        o = {n: inside(getattr(p, n), copy=False) for n in ("dx", "dz", "dr")}
        o.update({n: inside(getattr(p, n), 4, copy=False) for n in ("dpost_weight", "dweight")})
        ws = workspace(p.ws)
        p.plan.run_backward(*[tensor(v) for v in (*i.values(), *o.values())], tensor(ws))
        check(i.values(), [(v, getattr(p, n)) for n, v in o.items()])
        workspace_is_inside(ws)


@pytest.mark.parametrize("tokens,cols,out_cols", [s for _, sizes in KEPT for s in sizes] + [(31, 33, 65), (65, 200, 300)])
@pytest.mark.parametrize("dw_type,accumulate", [(BF16, False), (FP32, False), (FP32, True)],
                         ids=["bf16", "fp32", "accumulate"])
def test_checkpoint(tokens, cols, out_cols, dw_type, accumulate):
    p = Checkpoint(tokens, cols, out_cols, dw_type, accumulate, seed=tokens + cols + out_cols)
    p.pack()
    p.gradient()
    back = torch.empty_like(p.x.as_strided((tokens, p.x.stride(0)), (p.x.stride(0), 1)))[:, :cols]
    p.plan.unpack(p.kept, back)
    torch.cuda.synchronize()
    n = p.plan.checkpoint_size
    x, kept = inside(p.x), inside(p.kept[:n], copy=False)
    p.plan.pack(x.t, kept.t)
    check([x], [(kept, p.kept[:n])])
    kept, dy, dw, ws = inside(p.kept[:n]), inside(p.dy), inside(p.dw, copy=False), workspace(p.ws)
    if accumulate:
        dw.t.copy_(p.before)
    p.plan.weight_gradient(dy.t, kept.t, dw.t, tensor(ws))
    check([kept, dy], [(dw, p.dw)])
    workspace_is_inside(ws)
    x = inside(back, copy=False)
    p.plan.unpack(kept.t, x.t)
    check([kept], [(x, back)])
