"""The block norm in place, on every kernel pair that a plan chooses: h over x, z
or r and a bf16 y over another of them; dx, dr and dz over any three of the bf16
matrices that come in.  Rows enough that a walker takes several, so that the
next row is on its way while one is written.  What comes out is what separate
buffers get, bit for bit, and nothing past the columns is written."""
import itertools

import pytest
import torch

from tests.test_block_norm import Block

pytestmark = pytest.mark.gpu

# (forward, backward) waves and vectors, and rows and columns that reach them.
KERNELS = [
    ((1, 1), (1, 1), [(200, 511), (5003, 512), (5003, 77)]),
    ((1, 2), (1, 2), [(5003, 1001), (5003, 1000)]),
    ((1, 4), (4, 1), [(1301, 1999), (1301, 2000)]),
    ((4, 1), (4, 1), [(200, 2047), (200, 2048)]),
    ((4, 2), (4, 2), [(1301, 4001), (1301, 4000)]),
    ((4, 4), (8, 2), [(701, 8191), (701, 8190)]),
    ((16, 1), (16, 1), [(200, 8001), (200, 8000)]),
    ((8, 4), (8, 4), [(701, 16383), (701, 16382), (40, 9001)]),
]
GIVEN = [(True, True), (True, False), (False, True), (False, False)]


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def whole(view, cols):
    """The storage of a matrix of Block's, with what lies past the columns."""
    return view.as_strided((view.shape[0], view.stride(0)), (view.stride(0), 1))


def keep(p, names):
    """Copies of those matrices, on storage of their own with the same stride."""
    out = {}
    for n in names:
        full = whole(getattr(p, n), p.cols).clone()
        out[n] = full[:, :p.cols]
    return out


@pytest.mark.parametrize("forward,backward,rows,cols",
                         [(f, b, *size) for f, b, sizes in KERNELS for size in sizes])
@pytest.mark.parametrize("gate,post", GIVEN, ids=["gate-post", "gate-bare", "open-post", "open-bare"])
def test_in_place(forward, backward, rows, cols, gate, post):
    p = Block(rows, cols, post=post, gate=gate, seed=rows + cols)
    i = p.plan.info
    assert (i.forward_waves, i.forward_vectors) == forward and (i.backward_waves, i.backward_vectors) == backward
    p.forward()
    p.backward()
    torch.cuda.synchronize()

    come_in = ("x", "z", "r") if gate else ("x", "r")
    for over_h, over_y in itertools.permutations(come_in, 2):
        m = keep(p, come_in)
        rstd, post_rstd = torch.full_like(p.rstd, 7), torch.full_like(p.rstd, 7) if post else None
        p.plan.run(m["x"], m.get("z"), m["r"], p.post_weight, p.weight, m[over_h], m[over_y], None, post_rstd, rstd)
        torch.cuda.synchronize()
        assert same(m[over_h], p.h) and same(m[over_y], p.y) and same(rstd, p.rstd), (over_h, over_y)
        assert not post or same(post_rstd, p.post_rstd)
        for t in m.values():
            assert torch.isnan(whole(t, cols)[:, cols:].float()).all()

    come_in = ("dy", "dh", "x", "z", "h") if gate else ("dy", "dh", "x", "h")
    for k in range(len(come_in)):
        over = dict(zip(("dx", "dr", "dz") if gate else ("dx", "dr"), come_in[k:] + come_in[:k]))
        m = keep(p, come_in)
        out = {n: m[o] for n, o in over.items()}
        dw, dpw = torch.full_like(p.dweight, 7), torch.full_like(p.dweight, 7) if post else None
        p.ws.fill_(0xFF)
        p.plan.run_backward(m["dy"], m["dh"], m["x"], m.get("z"), m["h"], p.post_weight, p.weight, p.post_rstd, p.rstd,
                            out["dx"], out.get("dz"), out["dr"], dpw, dw, p.ws)
        torch.cuda.synchronize()
        for n in out:
            assert same(out[n], getattr(p, n)), (n, over)
        assert same(dw, p.dweight) and (not post or same(dpw, p.dpost_weight)), over
        for t in m.values():
            assert torch.isnan(whole(t, cols)[:, cols:].float()).all()
