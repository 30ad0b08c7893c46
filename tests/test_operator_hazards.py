"""Wait states in front of the LDS-DMA loads of the operators' kernels, and no
scratch access in their K loops (CPU: compiles to gfx950 assembly, runs
nothing).  The rules and their check are test_asm_hazards.py's."""
import re

import pytest

from tests.test_asm_hazards import LDS_LOAD, check_load
from warp_specialized_pipelined_amd import build as _build


@pytest.fixture(scope="module", params=["scaled_kernels", "loss_kernels"])
def kernels(request, tmp_path_factory):
    text = open(_build.dump_asm(str(tmp_path_factory.mktemp("asm")), request.param)).read()
    out = {}
    for m in re.finditer(r"^(_ZN6migemm\S*):[^\n]*\n(.*?)^\.Lfunc_end", text, re.S | re.M):
        lines = m.group(2).split("\n")
        if any(LDS_LOAD.match(x) for x in lines):
            out[m.group(1)] = lines
    assert out
    assert request.param != "scaled_kernels" or sum("scaled_mid" in n for n in out) == 5
    return out


def test_lds_dma_loads_have_their_wait_states(kernels):
    bad = ["%s line %d: %s" % (name[:80], i, p) for name, lines in kernels.items()
           for i, line in enumerate(lines) if LDS_LOAD.match(line) for p in check_load(lines, i)]
    assert not bad, "\n".join(bad[:20])


def _innermost_loops(lines):
    """(first, last) line of every innermost loop with matrix instructions: a
    backward branch to a label closes a loop."""
    labels = {m.group(1): i for i, l in enumerate(lines) if (m := re.match(r"^(\.LBB\w+):", l))}
    loops = [(labels[m.group(1)], i) for i, l in enumerate(lines)
             if (m := re.search(r"s_c?branch\w*\s+(\.LBB\w+)", l)) and labels.get(m.group(1), i) < i]
    loops = [(a, b) for a, b in loops if any("v_mfma" in x for x in lines[a:b])]
    inner = [(a, b) for a, b in loops
             if not any(a <= c and d <= b and (c, d) != (a, b) for c, d in loops)]
    return inner


def test_no_scratch_access_inside_a_k_loop(kernels):
    bad = {}
    for name, lines in kernels.items():
        loops = _innermost_loops(lines)
        assert loops, name
        hits = [lines[i].strip() for a, b in loops for i in range(a, b) if "scratch_" in lines[i]]
        if hits:
            bad[name] = hits[:3]
    assert not bad, bad
