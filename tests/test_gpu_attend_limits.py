"""Attention at the ends of what its arguments may be: windows, lengths and launches next to
the ends of 32 bits. Tolerances are those of test_gpu_kv.py."""

import numpy as np
import pytest
import torch

import block_quantized_matmul_q4_amd as qmm
import kv_reference as ref
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


LONGEST = 2**31 - 16                                    # tokens, the most that a table of 16-token pages holds


@pytest.mark.parametrize("new,group", [(1, 1), (4, 4), (40, 2)])
@pytest.mark.parametrize("window", [200, 3000])
@pytest.mark.parametrize("causal", [True, False])
def test_the_last_tokens_of_the_longest_request(new, group, window, causal):
    """A step from there would start past 2^31 - 1. The same as a short request's last tokens, bit
    for bit: the window hides the others, whose pages do not exist."""
    s = Setup([4096 - 16], [new], 1, group, 64, 16)
    hints = {"max_q": new, "max_len": 4096, "causal": causal, "window": window}
    want = s.check(**hints)
    table = torch.full((1, LONGEST // 16), -1, dtype=torch.int32, device="cuda")
    table[0, -s.table.shape[1]:] = gpu(s.table[0])
    lens = torch.tensor([LONGEST], dtype=torch.int32, device="cuda")
    got = qmm.attend_q4_0(gpu(s.q), gpu(s.cache), table, lens, gpu(s.cu), return_lse=True, **hints)
    assert all(np.array_equal(a, b.cpu().numpy()) for a, b in zip(want, got))


@pytest.mark.parametrize("new", [1, 20])
def test_all_tokens_of_the_longest_request(new):
    """Every page is the same one, so each of its 16 tokens counts 2^27 - 1 times and the result is
    theirs. A lane adds up 2^16 weights and an accumulator 2^18 products (at most: 2048 parts, four
    waves), which round to 2^-8 and 2^-6 of their sums; the rest is the bounds of test_gpu_kv.py."""
    s = Setup([16], [1], 1, 1, 64, 16)
    o, lse, size, reach = ref.attend(s.q, s.cache, 16, s.table, s.lens, s.cu, 64 ** -0.5)
    table = torch.full((1, LONGEST // 16), int(s.table[0, 0]), dtype=torch.int32, device="cuda")
    lens = torch.tensor([LONGEST], dtype=torch.int32, device="cuda")
    q = gpu(s.q).expand(new, 1, 64).contiguous()
    cu = torch.tensor([0, new], dtype=torch.int32, device="cuda")
    got, got_lse = (x.cpu().numpy() for x in qmm.attend_q4_0(q, gpu(s.cache), table, lens, cu, causal=False,
                                                             max_q=new, return_lse=True))
    e = 1e-4 * reach
    want = lse + np.log(2.0**27 - 1)
    assert (np.abs(got_lse - want) <= e + 2.0**-8 + 1e-6 * (1 + np.abs(want))).all()
    assert (np.abs(got - o) <= (2 * e[..., None] + 2.0**-6 + 2.0**-8) * size + 2.0**-29).all()
