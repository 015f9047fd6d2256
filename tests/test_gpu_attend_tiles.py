"""Attention whose workgroups take two tiles of 16 rows against the same decoded keys
(up to 128 dims, where there is work for every workgroup slot: here requests
without tokens or rows make up the number), on the GPU against the 64-bit
reference. tests/test_kv_tiles.py checks on the host that these calls are launched
that way. Tolerances are those derived in test_gpu_kv.py and test_gpu_kv_prompt.py.
"""

import numpy as np
import pytest
import torch

import block_quantized_matmul_q4_amd as qmm
import kv_reference as ref
from test_gpu_kv import Setup, device, gpu  # noqa: F401  (device: a fixture)

pytestmark = pytest.mark.gpu

SLOTS = 512                                             # requests x KV heads from which on tiles are pairs
DIMS = [64, 96, 128]

SHAPES = [
    # lens, new rows, kv heads, group, dim, page; rows (new x group) past a multiple of 32:
    ([200], [133], 2, 4, 128, 16),                      # 20
    ([257, 31, 64], [40, 31, 5], 2, 7, 96, 32),         # 24, 25, 3
    ([70], [70], 4, 1, 64, 32),                         # 6
    ([50, 3], [150, 9], 1, 2, 128, 16),                 # 12, 18; more new rows than tokens
    ([700, 1300], [130, 400], 2, 3, 64, 256),           # 6, 16
    ([513], [17], 1, 16, 128, 64),                      # 16
    ([1030], [17], 1, 1, 96, 16),                       # 17: one row in the second tile
    ([129, 1, 33], [129, 1, 33], 1, 1, 64, 64),         # 1
    ([300, 0, 90], [12, 0, 1], 8, 8, 128, 128),         # 0, 8
]
PARTS = [2048, 2049, 4097, 9000]                        # tokens, around the ends of parts of 2048
LONG = 40001                                            # the hint that makes 17 parts of 512 requests


class Pairs(Setup):
    """Requests as in Setup, and empty ones behind them up to the number of workgroup slots."""

    def __init__(self, lens, news, kv_heads, *args, **kwargs):
        more = [0] * (-(-SLOTS // kv_heads) - len(lens))
        super().__init__(list(lens) + more, list(news) + more, kv_heads, *args, **kwargs)

    def floor(self):
        at = ref.places(self.page, self.dim).vs.reshape(-1)
        d = np.stack([self.cache[..., at], self.cache[..., at + 1]], -1).view(np.float16)
        keys = int(min(max(self.lens.max(), 0), self.table.shape[1] * self.page))
        return keys * 2.0 ** -19 if (np.abs(d) >= 512).any() else super().floor()


def sizes(s, max_q=None, max_len=None, window=0):
    """T, B, KV heads, group, dim, max_q, max_len and window of a call on `s`."""
    tokens, heads, dim = s.q.shape
    kv_heads = s.cache.shape[1]
    return (tokens, len(s.lens), kv_heads, heads // kv_heads, dim, max_q or max(tokens, 1),
            max_len or s.table.shape[1] * s.page, window)


@pytest.mark.parametrize("lens,news,kv_heads,group,dim,page", SHAPES)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 5), (True, 200), (False, 40)])
def test_masks(lens, news, kv_heads, group, dim, page, causal, window):
    Pairs(lens, news, kv_heads, group, dim, page).check(causal=causal, window=window)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("max_len", [9000, LONG])       # five parts, and more than 16
def test_parts(dim, max_len):
    for n in PARTS:
        Pairs([n, 200, 1], [20, 1, 1], 1, 1, dim, 64).check(max_q=20, max_len=max_len)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("k_size,v_size,q_size,mean", [
    (1, 8, 1, 0), (1, 3000, 1, 0), (1, 1e-4, 1, 0), (1e-3, 1, 1e3, 0), (100, 1, 1e-2, 0),
    (1, 1, 0, 0), (1, 1, 1e-30, 0), (3, 1, 3, 0), (1, 1, 1, 0.2), (1, 30000, 1, 1),
    (30000, 1, 1e-5, 1), (30000, 30000, 3e-6, 0),
])
def test_magnitudes(dim, k_size, v_size, q_size, mean):
    Pairs([300, 1000], [50, 50], 2, 4, dim, 16, k_size=k_size, v_size=v_size, q_size=q_size, mean=mean).check()


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("which", ["k", "v"])
def test_scales_on_both_sides_of_the_limit(dim, which):
    """Every 37th token: other scales in each block, some of 512 and far more."""
    s = Pairs([700], [150], 2, 4, dim, 32)
    if which == "k":
        s.q *= 1e-4
    for t in range(0, 700, 37):
        s.scales(which, 0, t, t % 2, np.exp(s.rng.uniform(0, np.log(60000), dim // 32)))
    s.check()


@pytest.mark.parametrize("scale", [0.0, -0.07, 3.0])
def test_scales_of_scores(scale):
    Pairs([300], [20], 2, 2, 64, 64).check(scale=scale)


def test_q_of_unequal_rows():
    s = Pairs([300], [20], 1, 4, 128, 16)
    s.q *= np.exp(s.rng.uniform(-12, 1, (20, 4, 1))).astype(np.float32)
    s.q[3, 1] = 0
    s.q[5, 2, 1:] = 0
    s.check()


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("new", [20, 200])
def test_hidden_tokens_hold_nan_and_inf(dim, new):
    s = Pairs([330, 45], [new, min(new, 45)], 2, 4, dim, 64)
    clean = s.run(window=100)
    for b, n in ((0, 330), (1, 45)):
        for t in range(n, -(-n // 64) * 64):            # the tail of the last page
            for which in "kv":
                s.scales(which, b, t, t % 2, (np.nan, np.inf, -np.inf, 60000)[t % 4])
    spare = np.setdiff1d(np.arange(len(s.cache)), s.table)
    s.cache[spare] = 0xFF                               # pages of nobody: NaN scales
    for t in range(0, 330 - new - 99):                  # out of every row's window
        s.scales("kv"[t % 2], 0, t, t // 2 % 2, np.nan)
    o, lse = s.check(window=100)
    assert np.array_equal(o, clean[0]) and np.array_equal(lse, clean[1])


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_visible_nan_reaches_its_rows_only(dim, which, value):
    """The rows that see it start inside a tile."""
    s = Pairs([400], [100], 2, 2, dim, 32)
    clean = s.run()
    bad = np.full(dim // 32, 0.1, np.float16)
    bad[1] = value
    s.scales(which, 0, 350, 1, bad)                     # rows from 50 on, heads 2 and 3
    s.scales(which, 0, 399, 0, bad)                     # the last row, heads 0 and 1
    o, lse = s.run()
    hit = np.isnan(o)
    assert hit[50:, 2:].any() and not hit[:50].any() and not hit[:99, :2].any()
    assert np.array_equal(o[:50], clean[0][:50]) and np.array_equal(o[:99, :2], clean[0][:99, :2])
    if which == "v":                                    # only the block's own columns
        assert hit[50:, 2:, 32:64].all() and not hit[..., :32].any() and not hit[..., 64:].any()
        assert hit[99, :2, 32:64].all()


def test_nan_in_q_stays_in_its_row():
    s = Pairs([200], [40], 2, 4, 128, 32)
    clean = s.run()
    s.q[7, 3, 11] = np.nan
    s.q[9, 6, 100] = np.inf
    o, lse = s.run()
    bad = np.zeros(lse.shape, bool)
    bad[7, 3] = bad[9, 6] = True
    assert np.isnan(lse[bad]).all() and np.isnan(o[bad]).all()
    assert np.array_equal(o[~bad], clean[0][~bad]) and np.array_equal(lse[~bad], clean[1][~bad])


def test_all_visible_keys_nan():
    s = Pairs([70], [70], 1, 2, 96, 16)
    for t in range(70):
        s.scales("k", 0, t, 0, np.nan)
    o, lse = s.run()
    assert np.isnan(o).all() and np.isnan(lse).all()


def test_pages_that_the_cache_does_not_have():
    s = Pairs([300, 200], [130, 130], 2, 1, 128, 16)
    for i, bad in ((0, -1), (3, len(s.cache)), (7, 2**31 - 1), (18, -2**31)):
        s.table[0, i] = bad
    s.table[1] = -5                                     # no page at all: empty rows
    o, lse = s.check()
    assert (o[130:] == 0).all() and (lse[130:] == -np.inf).all()


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("max_q", [17, 33, 100])
def test_hints_and_determinism(dim, max_q):
    """Fewer tiles than the rows need (the workgroups walk on), the same bits each time."""
    s = Pairs([3000, 300], [100, 60], 2, 4, dim, 32)
    first = s.check(max_q=max_q, max_len=3000)
    for _ in range(2):
        again = s.run(max_q=max_q, max_len=3000)
        assert all(np.array_equal(a, b) for a, b in zip(first, again))


def test_graph_replays():
    s = Pairs([3000, 700], [60, 33], 2, 4, 128, 64)
    q, args = gpu(s.q), [gpu(x) for x in (s.cache, s.table, s.lens, s.cu)]
    hints = {"max_q": 60, "max_len": 3000, "return_lse": True}
    qmm.attend_q4_0(q, *args, **hints)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = qmm.attend_q4_0(q, *args, **hints)
    for i in range(3):
        q.mul_(-0.7 - 0.1 * i)
        graph.replay()
        torch.cuda.synchronize()
        want, want_lse = qmm.attend_q4_0(q, *args, **hints)
        assert torch.equal(out, want) and torch.equal(lse, want_lse), i
