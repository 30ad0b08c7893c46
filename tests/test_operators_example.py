"""examples/projection_and_loss.py against its fp32 form."""
import importlib.util
import os

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "projection_and_loss.py")


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hidden,vocab", [(512, 1024, 32000), (1, 256, 1000), (100, 512, 5000)])
def test_the_example_agrees_with_fp32(tokens, hidden, vocab):
    spec = importlib.util.spec_from_file_location("projection_and_loss", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    errors = example.main(["--tokens", str(tokens), "--hidden", str(hidden), "--vocab", str(vocab)])
    # The fp32 form rounds where the operators do, but a value on the border of
    # two e4m3 or bf16 ones may fall to the other side, by a step of 2^-3 or
    # 2^-7: few do.  What is left is the rounding of y2, g and the gradients to
    # bf16, 2^-8 / sqrt(3) of each at most.
    assert errors["loss"] < 2.0 ** -7
    for k in ("dhead", "dw2", "dh2"):
        assert errors[k] < 2.0 ** -6, errors
