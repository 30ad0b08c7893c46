"""Wait states in front of the LDS-DMA loads of the int8 product's and the
checkpoint gradient's kernels, and no scratch access in their K loops (CPU:
compiles to gfx950 assembly, runs nothing).  The rules are
test_asm_hazards.py's; its check takes a load's text, so the gradient's loads of
four bytes are read as those of sixteen."""
import re

import pytest

from tests.test_asm_hazards import LDS_LOAD, check_load
from tests.test_operator_hazards import _innermost_loops
from warp_specialized_pipelined_amd import build as _build

KERNELS = {"int8_kernels": ("scaled_", 5), "checkpoint_kernels": ("kept_gradient", 4)}


@pytest.fixture(scope="module", params=sorted(KERNELS))
def kernels(request, tmp_path_factory):
    text = open(_build.dump_asm(str(tmp_path_factory.mktemp("asm")), request.param)).read()
    text = re.sub(r"buffer_load_dword (v\d+, s\[\d+:\d+\], 0 offen lds)", r"buffer_load_dwordx4 \1", text)
    out = {}
    for m in re.finditer(r"^(_ZN6migemm\S*):[^\n]*\n(.*?)^\.Lfunc_end", text, re.S | re.M):
        lines = m.group(2).split("\n")
        if any(LDS_LOAD.match(x) for x in lines):
            out[m.group(1)] = lines
    name, count = KERNELS[request.param]
    assert len(out) == count and all(name in n for n in out), sorted(out)
    return out


def test_lds_dma_loads_have_their_wait_states(kernels):
    bad = ["%s line %d: %s" % (name[:80], i, p) for name, lines in kernels.items()
           for i, line in enumerate(lines) if LDS_LOAD.match(line) for p in check_load(lines, i)]
    assert not bad, "\n".join(bad[:20])


def test_no_scratch_access_inside_a_k_loop(kernels):
    bad = {}
    for name, lines in kernels.items():
        loops = _innermost_loops(lines)
        assert loops, name
        hits = [lines[i].strip() for a, b in loops for i in range(a, b) if "scratch_" in lines[i]]
        if hits:
            bad[name] = hits[:3]
    assert not bad, bad
