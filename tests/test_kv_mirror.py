"""The address-level calls of the paged KV cache that the package mirrors by name: refusals
with their status and message (CPU: nothing is launched), and on the GPU the same results as
the tensor front ends."""

import pytest
import torch

import block_quantized_matmul_q4_amd as qmm

PAGE, HEADS, DIM = 16, 2, 64


def geometry(pages, **other):
    return qmm.KvCache(*{**dict(pages=pages, num_pages=9, page_size=PAGE, kv_heads=HEADS, head_dim=DIM),
                         **other}.values())


def test_refusals():
    far = [(i + 1) << 40 for i in range(12)]            # addresses that are never followed
    assert qmm.qmm_kv_plan(0, *far[1:11], 1, 1, 1, 1, PAGE) == qmm.QMM_EINVAL
    assert "null pointer" in qmm.qmm_last_error()
    assert qmm.qmm_kv_plan(*far[:11], 1, 1, 1, 1, 24) == qmm.QMM_EUNSUPPORTED
    assert "page_size" in qmm.qmm_last_error()
    assert qmm.qmm_kv_append_q4_0(far[0], 64, far[1], 128, geometry(far[2]), far[3], 5) == qmm.QMM_EINVAL
    assert "k_stride" in qmm.qmm_last_error()
    assert qmm.qmm_kv_append_q4_0(far[0], 128, far[1], 128, geometry(far[2]), far[3], 0) == qmm.QMM_OK
    assert qmm.qmm_kv_read_q4_0(geometry(far[0], head_dim=80), far[1], far[2], far[3], 5) == qmm.QMM_EUNSUPPORTED
    assert "head_dim" in qmm.qmm_last_error()
    assert qmm.qmm_kv_read_q4_0(geometry(far[0]), far[1], far[2] + 8, far[3], 5) == qmm.QMM_EALIGN
    sizes = dict(T=3, B=2, q_heads=4, max_q=2, max_len=100)
    assert qmm.qmm_attend_q4_0_workspace(geometry(None), *sizes.values(), 0) == 0
    assert qmm.qmm_attend_q4_0_workspace(geometry(None), *sizes.values(), -1) == -qmm.QMM_EINVAL
    ends = far[2], 4, far[3], far[4], far[5], far[6], 0, 0
    assert qmm.qmm_attend_q4_0(far[0], 256, geometry(far[1]), *ends, *sizes.values(), 0.1, 2, 0) == qmm.QMM_EINVAL
    assert "causal" in qmm.qmm_last_error()
    assert qmm.qmm_attend_q4_0(far[0] + 4, 256, geometry(far[1]), *ends, *sizes.values(), 0.1, 1,
                               0) == qmm.QMM_EALIGN


@pytest.mark.parametrize("name", ["status", "cu", "positions", "slots", "table", "ring"])
@pytest.mark.parametrize("twin", ["lens", "pool"])
def test_a_plan_in_place_lets_no_other_output_share_the_array(name, twin):
    names = ("want", "lens", "table", "ring", "pool", "new_lens", "new_pool", "cu", "slots", "positions", "status")
    at = {n: (i + 1) << 40 for i, n in enumerate(names)}
    at["new_" + twin] = at[name] = at[twin]
    assert qmm.qmm_kv_plan(*at.values(), 3, 5, 4, 50, PAGE) == qmm.QMM_EINVAL
    assert "overlaps" in qmm.qmm_last_error()


@pytest.mark.gpu
def test_the_same_as_the_front_ends():
    g = torch.Generator().manual_seed(3)
    want = torch.tensor([20, 3], dtype=torch.int32, device="cuda")
    lens = torch.zeros_like(want)
    tokens, batch, width = 23, 2, 4
    k, v, q = (torch.randn(tokens, heads, DIM, generator=g).cuda() for heads in (HEADS, HEADS, 6))
    results = []
    for mirrored in (False, True):
        cache = qmm.kv_cache_q4_0(9, PAGE, HEADS, DIM)
        table = torch.zeros(batch, width, dtype=torch.int32, device="cuda")
        ring = torch.arange(9, dtype=torch.int32, device="cuda")
        pool = torch.tensor([2, 9], device="cuda")
        if not mirrored:
            step = qmm.kv_plan(want, lens, table, ring, pool, tokens, PAGE)
            qmm.kv_append_q4_0(k, v, cache, step.slots)
            back = qmm.kv_read_q4_0(cache, step.slots, DIM)
            out, lse = qmm.attend_q4_0(q, cache, table, step.lens, step.cu, return_lse=True)
        else:
            stream = torch.cuda.current_stream().cuda_stream
            at = [x.data_ptr() for x in (want, lens, table, ring, pool)]
            step = qmm.KvPlan(*(torch.empty(n, dtype=t, device="cuda") for n, t in (
                (batch, torch.int32), (2, torch.int64), (batch + 1, torch.int32), (tokens, torch.int64),
                (tokens, torch.int32), (batch, torch.int32))))
            qmm.check(qmm.qmm_kv_plan(*at, *(x.data_ptr() for x in step), batch, tokens, width, 9, PAGE, stream))
            c = geometry(cache.data_ptr())
            row = HEADS * DIM
            qmm.check(qmm.qmm_kv_append_q4_0(k.data_ptr(), row, v.data_ptr(), row, c, step.slots.data_ptr(),
                                             tokens, stream))
            back = torch.empty_like(k), torch.empty_like(v)
            qmm.check(qmm.qmm_kv_read_q4_0(c, step.slots.data_ptr(), *(x.data_ptr() for x in back), tokens, stream))
            out, lse = torch.empty_like(q), torch.empty(tokens, 6, device="cuda")
            sizes = tokens, batch, 6, tokens, width * PAGE
            need = qmm.qmm_attend_q4_0_workspace(c, *sizes, 0)
            assert need >= 0
            room = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
            qmm.check(qmm.qmm_attend_q4_0(q.data_ptr(), 6 * DIM, c, table.data_ptr(), width, step.lens.data_ptr(),
                                          step.cu.data_ptr(), out.data_ptr(), lse.data_ptr(), room.data_ptr(),
                                          need, *sizes, DIM ** -0.5, 1, 0, stream))
        results.append([*step, cache, table, ring, *back, out, lse])
    assert all(torch.equal(a, b) for a, b in zip(*results))
