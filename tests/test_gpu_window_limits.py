"""Attention inside the cells at the limits of its numbers."""
import pytest
import torch

from test_gpu_window import Problem, run_window, shell

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shift", [120, -95])
@pytest.mark.parametrize("m", [5, 14])
def test_bias_gradient_scales_with_the_size_of_dp(m, shift):
    """dout and v times powers of two: dP, D and dS are the same numbers times a power of two (the
    largest |dP| here is near 2^125 and 2^-90), so dbias is, bit for bit."""
    coords, cu = shell(71, 300, r=9)
    pr = Problem(coords, cu, m, 4, 2, 32, torch.bfloat16, seed=72, bias="offset")
    want = run_window(pr)["dbias"].double() * 2.0 ** shift
    pr.dout *= 2.0 ** (shift // 2)
    pr.v *= 2.0 ** (shift - shift // 2)
    got = run_window(pr)["dbias"]
    assert bool(torch.isfinite(got).all())
    assert torch.equal(got.double(), want)
