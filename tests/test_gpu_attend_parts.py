"""Attention whose keys are shared out over parts: what a row gets may not depend on how
many parts there are. Tolerances are those of test_gpu_kv.py."""

import numpy as np
import pytest
import torch

import block_quantized_matmul_q4_amd as qmm
import kv_reference as ref
from test_gpu_kv import Setup, device, gpu  # noqa: F401  (device: a fixture)

pytestmark = pytest.mark.gpu

# tokens of a request whose keys make one part, a few, and more than 16 (256 keys each)
PARTS = [1000, 3000, 6000]


@pytest.mark.parametrize("keys", PARTS)
@pytest.mark.parametrize("new", [1, 40])
def test_visible_nan_far_below_the_maximum(keys, new):
    """A value that is NaN reaches its rows although another part's scores are so much higher
    that its own weight underflows to 0 (0 times NaN)."""
    s = Setup([keys], [new], 1, 1, 64, 16)
    s.q[:] = s.q[0]
    scale = 64 ** -0.5
    # token 100's score lies 400 above a bound of all others' (8 |q| 8 d, d up to 4 x 0.22 nearly
    # always), where exp2 of the difference is 0
    others = 8 * 0.88 * np.abs(s.q[0, 0]).sum() * scale
    s.scales("k", 0, 100, 0, 1.0)
    page, place = s.tokens(0, 100)
    k, _ = ref.get(s.cache[page, 0], 16, 64)
    s.scales("k", 0, 100, 0, (others + 400) / (scale * (k[place] @ s.q[0, 0])))
    s.scales("v", 0, keys - 80, 0, [0.1, np.nan])
    o, lse = s.check(max_q=new)
    assert np.isnan(o[..., 32:]).all() and np.isfinite(o[..., :32]).all() and np.isfinite(lse).all()
    assert (lse > others + 350).all()


@pytest.mark.parametrize("keys", PARTS)
@pytest.mark.parametrize("new", [2, 40])
def test_rows_of_no_request_are_left(keys, new):
    """Before cu[0] and from cu[B] on, whatever the workspace held."""
    s = Setup([keys, 30], [new, 3], 1, 2, 64, 16)
    n = new + 3
    q = torch.randn(n + 7, 2, 64, device="cuda")
    q[4:n + 4] = gpu(s.q)
    out, lse = torch.full_like(q, 7.0), torch.full((n + 7, 2), 7.0, device="cuda")
    qmm.attend_q4_0(q, gpu(s.cache), gpu(s.table), gpu(s.lens), gpu(s.cu + 4), out=out, lse=lse, max_q=new,
                    workspace=torch.full((1 << 24,), 63, dtype=torch.uint8, device="cuda"))
    for x in (out, lse):
        assert (x[:4] == 7).all() and (x[n + 4:] == 7).all()
    s.run = lambda **_: [x[4:n + 4].cpu().numpy().astype(np.float64) for x in (out, lse)]
    s.check()


@pytest.mark.parametrize("dim,keys", [(128, 700), (64, 6000)])
def test_a_batch_in_two_calls(dim, keys):
    """Decoding requests first, prompt chunks after them: each call writes its requests' rows of the
    same out, by slices of the table, the lengths and cu."""
    s = Setup([keys, 300, 40, 400, 90], [1, 1, 1, 50, 33], 2, 4, dim, 16)
    q, cache, table, lens, cu = (gpu(x) for x in (s.q, s.cache, s.table, s.lens, s.cu))
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    qmm.attend_q4_0(q, cache, table[:3], lens[:3], cu[:4], max_q=1, out=out, lse=lse)
    assert (out[3:] == 7).all() and (lse[3:] == 7).all()
    qmm.attend_q4_0(q, cache, table[3:], lens[3:], cu[3:], max_q=50, out=out, lse=lse)
    s.run = lambda **_: [x.cpu().numpy().astype(np.float64) for x in (out, lse)]
    s.check()
