"""Attention of one decoder layer over a paged Q4_0 KV cache, prompt and decoding.

A few requests of unlike lengths bring their prompts and then decode one token
a step, through one layer's projections (Q4_0 matrices, 2048 -> 2048 for q and o
with 8 heads of 256, 2048 -> 512 for k and v with 2 heads; synthetic weights) and
its cache:

    step = kv_plan(want, lens, table, ring, pool, tokens, page_size)
    q, k, v = x @ Wq, x @ Wk, x @ Wv
    kv_append_q4_0(k, v, cache, step.slots)
    y = attend_q4_0(q, cache, table, step.lens, step.cu, max_q=1) @ Wo     # decoding

Each step's attention is compared with plain attention in 64 bits over the
values that the cache holds (kv_read_q4_0). Requests end on the way and give
their pages back. Run from the repository's root on a machine with a GPU:

    python examples/paged_attention.py
"""

import pathlib
import sys

import torch

sys.path.insert(0, str(pathlib.Path(__file__).resolve().parent.parent))

import block_quantized_matmul_q4_amd as qmm
import synth

HIDDEN, Q_HEADS, KV_HEADS, HEAD_DIM = 2048, 8, 2, 256
PAGE, PAGES, WIDTH = 64, 48, 16


def weights(n, seed):
    return torch.from_numpy(synth.q4_0_weights(n, HIDDEN, seed=seed).reshape(-1)).cuda()


def project(x, w, n):
    """x W^T: the GEMV's f32 arithmetic for a few rows, the matrix cores for many."""
    return (qmm.gemv_q4_0 if x.shape[0] <= qmm.GEMV_MAX_M else qmm.gemm_q4_0)(x, w, n, HIDDEN)


class Layer:
    """One layer's projections and cache, and the block table that a server's layers share."""

    def __init__(self, requests):
        self.wq, self.wk = weights(Q_HEADS * HEAD_DIM, 1), weights(KV_HEADS * HEAD_DIM, 2)
        self.wv, self.wo = weights(KV_HEADS * HEAD_DIM, 3), weights(HIDDEN, 4)
        self.cache = qmm.kv_cache_q4_0(PAGES, PAGE, KV_HEADS, HEAD_DIM)
        self.table = torch.full((requests, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.ring = torch.arange(PAGES, dtype=torch.int32, device="cuda")
        self.pool = torch.tensor([0, PAGES], device="cuda")
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")

    def step(self, x, want, max_q, max_len):
        """x [rows, HIDDEN]: the new tokens, request after request; want: their lengths after the step."""
        rows = x.shape[0]
        step = qmm.kv_plan(want, self.lens, self.table, self.ring, self.pool, rows, PAGE)
        self.lens, self.pool = step.lens, step.pool
        q = project(x, self.wq, Q_HEADS * HEAD_DIM).view(rows, Q_HEADS, HEAD_DIM)
        k = project(x, self.wk, KV_HEADS * HEAD_DIM).view(rows, KV_HEADS, HEAD_DIM)
        v = project(x, self.wv, KV_HEADS * HEAD_DIM).view(rows, KV_HEADS, HEAD_DIM)
        qmm.kv_append_q4_0(k, v, self.cache, step.slots)
        o = qmm.attend_q4_0(q, self.cache, self.table, step.lens, step.cu, max_q=max_q, max_len=max_len)
        y = project(o.view(rows, -1), self.wo, HIDDEN)
        return q, o, y, step

    def plain(self, q, step):
        """The same attention in 64 bits, over the values that the cache holds."""
        out = torch.zeros_like(q, dtype=torch.float64)
        cu = step.cu.tolist()
        for b, n in enumerate(step.lens.tolist()):
            first, end = cu[b], cu[b + 1]
            if first == end:
                continue
            t = torch.arange(n, device="cuda")
            slots = self.table[b, t // PAGE].long() * PAGE + t % PAGE
            k, v = (x.double().repeat_interleave(Q_HEADS // KV_HEADS, 1).transpose(0, 1).contiguous()
                    for x in qmm.kv_read_q4_0(self.cache, slots, HEAD_DIM))     # [heads, n, D]
            rows = q[first:end].double().transpose(0, 1).contiguous()
            score = (rows[:, :, None] * k[:, None]).sum(-1) * HEAD_DIM ** -0.5
            at = torch.arange(n - (end - first), n, device="cuda")
            score.masked_fill_(t > at[:, None], float("-inf"))
            p = torch.softmax(score, -1)
            out[first:end] = (p[..., None] * v[:, None]).sum(2).transpose(0, 1)
        return out


def main(prompts=(70, 33, 5, 128), steps=12, ends={4: 1, 9: 0}):
    """Returns the largest error of a step's attention, relative to its largest value."""
    torch.manual_seed(0)
    layer = Layer(len(prompts))
    lens = list(prompts)
    x = torch.randn(sum(prompts), HIDDEN, device="cuda")
    worst = 0.0
    for i in range(steps + 1):
        want = torch.tensor(lens, dtype=torch.int32, device="cuda")
        q, o, y, step = layer.step(x, want, max_q=max(prompts) if i == 0 else 1, max_len=max(lens))
        if int(step.status.abs().sum()):
            raise RuntimeError(f"step {i} was refused: {step.status.tolist()}")
        exact = layer.plain(q, step)
        error = float((o - exact).abs().max() / exact.abs().max())
        worst = max(worst, error)
        print(f"step {i}: {x.shape[0]} rows, lengths {step.lens.tolist()}, "
              f"{int(layer.pool[1])} pages free, error {error:.1e}", flush=True)
        # the next step: a token more for each request that has not ended
        last = step.cu[1:].long() - 1
        ended = ends.get(i + 1)
        running = [b for b, n in enumerate(lens) if n and b != ended]
        x = torch.nn.functional.normalize(y[last[running]]) * HIDDEN ** 0.5
        lens = [n + 1 if b in running else 0 for b, n in enumerate(lens)]
    return worst


if __name__ == "__main__":
    print(f"largest error {main():.1e}")
