"""Attention at the ends of what its arguments may be: windows, lengths and launches next to
the ends of 32 bits. Tolerances are those of test_gpu_kv.py."""

import numpy as np
import pytest
import torch

import block_quantized_matmul_q4_amd as qmm
from test_gpu_kv import Setup, device, gpu  # noqa: F401  (device: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 3])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("news", [(5, 9), (60, 70)])
def test_the_largest_windows_hide_nothing(window, causal, news):
    """... not even of requests with more new rows than tokens, whose first rows stand before 0."""
    s = Setup([50, 3], list(news), 1, 4, 128, 16)
    want = s.check(causal=causal)
    got = s.check(causal=causal, window=window)
    assert all(np.array_equal(a, b) for a, b in zip(want, got))
