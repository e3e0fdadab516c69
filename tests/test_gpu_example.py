"""The example block runs, and is as far from fp32 activations as two e4m3 roundings leave it.

Each activation is rounded to e4m3 twice (the norm, the SwiGLU): relative steps uniform in +-2^-4 at worst and over
the octave about 2^-4 / sqrt(3) * 0.75 = 2.7e-2 in the root mean square, so two of them give 3.8e-2 of the output's norm
(sums of independent terms keep the ratio; the SwiGLU takes the first rounding through two factors, sqrt(2) of it):
under 2.7e-2 * (1 + sqrt(2)) = 6.5e-2.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_moe_block.py")


@pytest.mark.parametrize("args", [[], ["--tokens", "1"], ["--tokens", "700", "--experts", "16", "--ffn", "768", "--hidden", "1024"]])
def test_fp8_moe_block(args):
    spec = importlib.util.spec_from_file_location("fp8_moe_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main([*args, "--steps", "2"]) <= 6.5e-2
