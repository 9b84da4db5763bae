"""The dense block at the width of a dense layer, several times an expert's, by
the tests of the narrower sizes: one token, few tokens (more tiles of features
than SMs), and pairs of CTAs with many tiles each."""
import pytest

import test_gpu_ffn
from test_gpu_ffn import DT

pytestmark = test_gpu_ffn.pytestmark
WIDE = [(1, 1024, 18432), (16, 1024, 18432), (60, 520, 10952), (300, 512, 18432), (1500, 264, 10944)]


@pytest.mark.parametrize("keep", ["none", "fp8", "full"])
@pytest.mark.parametrize("t", list(DT))
@pytest.mark.parametrize("T,d,I", WIDE)
def test_forward(T, d, I, t, keep):
    test_gpu_ffn.test_forward(T, d, I, t, keep)


@pytest.mark.parametrize("keep", ["fp8", "full"])
@pytest.mark.parametrize("t", list(DT))
@pytest.mark.parametrize("T,d,I", WIDE)
def test_backward(T, d, I, t, keep):
    test_gpu_ffn.test_backward(T, d, I, t, keep)
