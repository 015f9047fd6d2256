"""Plans whose sums over the batch pass 32 bits: what cannot be granted gets its status, and
nothing outside the arrays is written."""

import numpy as np
import pytest
import torch

import block_quantized_matmul_q4_amd as qmm
from test_gpu_kv import device, gpu, pool_state  # noqa: F401  (device: a fixture)

pytestmark = pytest.mark.gpu

GUARD = 1 << 16


def guarded(n, dtype):
    """A tensor of n values inside a longer one, whose other values are -5."""
    whole = torch.full((n + 2 * GUARD,), -5, dtype=dtype, device="cuda")
    return whole, whole[GUARD:GUARD + n]


def untouched(whole):
    return bool((whole[:GUARD] == -5).all()) and bool((whole[-GUARD:] == -5).all())


@pytest.mark.parametrize("tokens", [10, 4096])
@pytest.mark.parametrize("each", [4194303, 3000000, 4194304, 2097152])    # of at most 4194304
@pytest.mark.parametrize("batch", [1025, 2100])
def test_rows_asked_for_pass_32_bits(tokens, each, batch):
    """The first 1024 requests ask for 2^31 rows and more in all (2^32 exactly, too)."""
    page, width = 256, 16384
    lens = np.zeros(batch, np.int32)
    want = np.full(batch, each, np.int32)
    want[0], want[-1] = 7, 3                            # only the first has its rows in the batch
    if each == 2097152:
        want[1] += each - 7
    table, ring, pool = pool_state(np.random.default_rng(batch), lens, width, page, 40)
    slots_all, slots = guarded(tokens, torch.int64)
    positions_all, positions = guarded(tokens, torch.int32)
    cu_all, cu = guarded(batch + 1, torch.int32)
    t = [gpu(x) for x in (want, lens, table, ring, pool)]
    out = qmm.KvPlan(torch.empty_like(t[1]), torch.empty_like(t[4]), cu, slots, positions,
                     torch.empty_like(t[1]))
    qmm.kv_plan(*t, tokens, page, out=out)
    assert all(map(untouched, (slots_all, positions_all, cu_all)))
    assert out.lens.tolist() == [7] + [0] * (batch - 1)
    assert out.status.tolist() == [qmm.KV_OK] + [qmm.KV_NO_ROWS] * (batch - 1)
    first = int(ring[pool[0]])
    assert slots.tolist() == [first * page + i for i in range(7)] + [-1] * (tokens - 7)
    assert positions.tolist() == [*range(7)] + [-1] * (tokens - 7)
    rows = np.concatenate([[0], np.cumsum(want.astype(np.int64))])
    assert np.array_equal(cu.cpu().numpy(), np.minimum(rows, 2**31 - 1))
    assert out.pool.tolist() == [(pool[0] + 1) % len(ring), pool[1] - 1]
    table[0, 0] = first
    assert np.array_equal(t[2].cpu().numpy(), table) and np.array_equal(t[3].cpu().numpy(), ring)


def test_pages_given_back_pass_32_bits():
    """2^20 requests give back 2^32 pages in all, to a ring with room for five (a table of 16 GiB)."""
    batch, width, page, size = 1 << 20, 1 << 12, 16, 20
    table = torch.zeros(batch, width, dtype=torch.int32, device="cuda")
    table[0] = torch.arange(width, dtype=torch.int32, device="cuda") + 100
    lens = torch.full((batch,), width * page, dtype=torch.int32, device="cuda")
    want = torch.zeros_like(lens)
    ring_all, ring = guarded(size, torch.int32)
    ring.copy_(torch.arange(size, device="cuda"))
    pool = torch.tensor([12, 15], device="cuda")
    step = qmm.kv_plan(want, lens, table, ring, pool, 4, page)
    assert untouched(ring_all)
    # the free places are 7 .. 11
    assert ring.tolist() == [*range(7), *range(100, 105), *range(12, 20)]
    assert step.pool.tolist() == [12, 20] and not step.status.any() and not step.lens.any()
    assert not step.cu.any() and (step.slots == -1).all()


def test_ring_of_more_than_2_to_the_30():
    """Head and count add up to more than 2^31 (a ring of 6 GiB)."""
    size, page = 3 << 29, 16
    ring_all, ring = guarded(size, torch.int32)
    head, count = size - 2, size - 3
    ring.fill_(9)
    ring[-2:] = torch.tensor([50, 51], device="cuda")
    ring[:2] = torch.tensor([52, 53], device="cuda")
    table = torch.tensor([[0, 0, 0], [3, 4, 5]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    want = torch.tensor([48, 10], dtype=torch.int32, device="cuda")
    step = qmm.kv_plan(want, lens, table, ring, torch.tensor([head, count], device="cuda"), 48, page)
    assert table.tolist() == [[50, 51, 52], [3, 4, 5]] and step.pool.tolist() == [1, count - 1]
    end = (head + count) % size
    assert ring[end:end + 2].tolist() == [4, 5] and int((ring[2:end] != 9).sum()) == 0
    assert int((ring[end + 2:-2] != 9).sum()) == 0 and untouched(ring_all)


@pytest.mark.parametrize("tokens", [2**31 - 1, 2**31 - 256])
def test_the_largest_number_of_rows(tokens):
    """The rows' workgroups are counted past 2^31 (24 GiB of slots and positions)."""
    lens = torch.tensor([20, 0], dtype=torch.int32, device="cuda")
    want = torch.tensor([25, 1], dtype=torch.int32, device="cuda")
    table = torch.tensor([[7, 3], [0, 0]], dtype=torch.int32, device="cuda")
    ring = torch.tensor([8], dtype=torch.int32, device="cuda")
    step = qmm.kv_plan(want, lens, table, ring, torch.tensor([0, 1], device="cuda"), tokens, 16)
    assert step.slots[:6].tolist() == [3 * 16 + 4 + i for i in range(5)] + [8 * 16]
    assert step.positions[:6].tolist() == [20, 21, 22, 23, 24, 0]
    for x in (step.slots, step.positions):
        assert len(x) == tokens and all((part == -1).all() for part in x[6:].split(1 << 28))


def test_in_place_where_nothing_changes():
    """want, lens and the new lens in one array."""
    lens = torch.tensor([20, 0, 33], dtype=torch.int32, device="cuda")
    table = torch.tensor([[7, 3, 0], [0, 0, 0], [1, 2, 4]], dtype=torch.int32, device="cuda")
    ring, pool = torch.tensor([8, 9], dtype=torch.int32, device="cuda"), torch.tensor([1, 1], device="cuda")
    before = table.clone()
    out = qmm.KvPlan(lens, pool, torch.empty(4, dtype=torch.int32, device="cuda"),
                     torch.empty(2, dtype=torch.int64, device="cuda"), None, torch.empty_like(lens))
    qmm.kv_plan(lens, lens, table, ring, pool, 2, 16, out=out)
    assert lens.tolist() == [20, 0, 33] and pool.tolist() == [1, 1] and torch.equal(table, before)
    assert out.cu.tolist() == [0] * 4 and out.slots.tolist() == [-1, -1] and not out.status.any()
