"""Attention at the ends of what its arguments may be: windows, lengths and launches next to
the ends of 32 bits. Tolerances are those of test_gpu_kv.py."""

import copy

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


def same_as_reference(s, b, o, lse, **args):
    """Checks request b's rows of a batch whose results are o, lse."""
    one, rows = copy.copy(s), slice(int(s.cu[b]), int(s.cu[b + 1]))
    one.q, one.table, one.lens = s.q[rows], s.table[b:b + 1], s.lens[b:b + 1]
    one.cu = s.cu[b:b + 2] - s.cu[b]
    one.run = lambda **_: (o[rows].cpu().numpy().astype(np.float64), lse[rows].cpu().numpy().astype(np.float64))
    one.check(**args)


def test_default_hints_of_a_large_batch():
    """512 requests of 32 rows, each of them launched for all 16384: as many tiles as 2^32 threads."""
    rng = np.random.default_rng(5)
    s = Setup([int(n) for n in rng.integers(20, 120, 512)], [32] * 512, 8, 8, 64, 16)
    args = [gpu(x) for x in (s.q, s.cache, s.table, s.lens, s.cu)]
    o, lse = qmm.attend_q4_0(*args, return_lse=True)
    want = qmm.attend_q4_0(*args, max_q=32, return_lse=True)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    for b in (0, 300, 511):
        same_as_reference(s, b, o, lse)


@pytest.mark.parametrize("news,group", [([2, 1, 2, 1, 1, 2], 1), ([20, 3, 19, 1, 0, 20], 2)])
def test_more_requests_than_one_launch_takes(news, group):
    """600000 requests of 8 heads; those with rows are at the ends of the launches."""
    batch, at = 600000, [0, 262143, 262144, 524287, 524288, 599999]
    s = Setup([100, 37, 64, 5, 20, 111], news, 8, group, 64, 16)
    table = torch.zeros(batch, s.table.shape[1], dtype=torch.int32, device="cuda")
    lens, rows = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(2))
    table[at], lens[at] = gpu(s.table), gpu(s.lens)
    rows[at] = torch.tensor(news, dtype=torch.int32, device="cuda")
    cu = torch.cat([rows.new_zeros(1), rows.cumsum(0).int()])
    s.run = lambda **args: [x.cpu().numpy().astype(np.float64) for x in qmm.attend_q4_0(
        gpu(s.q), gpu(s.cache), table, lens, cu, max_q=max(news), return_lse=True, **args)]
    s.check()


@pytest.mark.parametrize("max_q", [1, 3])               # more than 16 parts, and fewer
def test_more_rows_than_one_join_takes(max_q):
    """16395 rows of 64 heads in 15 and 20 parts; all but five belong to a request without tokens."""
    s = Setup([5000, 5000], [2, 3], 1, 64, 64, 16)
    q = torch.randn(16395, 64, 64, device="cuda")
    q[:2], q[-3:] = gpu(s.q[:2]), gpu(s.q[2:])
    table, lens = gpu(s.table[[0, 0, 1]]), torch.tensor([5000, 0, 5000], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2, 16392, 16395], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((16395, 64), 7.0, device="cuda")
    qmm.attend_q4_0(q, gpu(s.cache), table, lens, cu, max_q=max_q, out=out, lse=lse)
    assert not out[2:-3].any() and (lse[2:-3] == -np.inf).all()
    s.run = lambda **_: [torch.cat([x[:2], x[-3:]]).cpu().numpy().astype(np.float64) for x in (out, lse)]
    s.check()


def test_a_cache_without_heads_or_pages_is_refused():
    s = Setup([10], [1], 1, 1, 64, 16)
    rest = [gpu(x) for x in (s.table, s.lens, s.cu)]
    for pages, heads in ((3, 0), (0, 1), (0, 0)):
        cache = torch.empty(pages, heads, 1152, dtype=torch.uint8, device="cuda")
        with pytest.raises((ValueError, qmm.QmmError), match="multiple|num_pages"):
            qmm.attend_q4_0(gpu(s.q), cache, *rest)
