"""An attention layer out of this library's operators: 4-bit projections, normalised and
rotated heads, a paged 4-bit key/value cache and the attention that reads it.

    python examples/attention_layer.py

takes the prompts of several sequences in one packed call, then one token of each
sequence at a time from a CUDA graph, and at the end asks for the same tokens again in one
call over the cache as it stands: the outputs are the same up to rounding.  The weights
and the inputs are random.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import affine_bit_matmul_gb300 as mxq  # noqa: E402


class Cache:
    """Pages for `seqs` sequences of up to `most` tokens, given out in a random order."""

    def __init__(self, seqs, most, kv_heads, head_dim, page_size, device, seed=0):
        each = -(-most // page_size)
        gen = torch.Generator().manual_seed(seed)
        self.page_size = page_size
        self.pages = torch.zeros((seqs * each, kv_heads, mxq.kv_block_bytes(head_dim, page_size)),
                                 dtype=torch.uint8, device=device)
        self.table = torch.randperm(seqs * each, generator=gen).view(seqs, each).int().to(device)

    def slots(self, seq, position):
        """int32 [T]: where tokens `position` of sequences `seq` go."""
        page = self.table[seq.long(), (position // self.page_size).long()]
        return page * self.page_size + position % self.page_size


class AttentionLayer:
    def __init__(self, hidden, heads, kv_heads, head_dim, device, seed=0):
        gen = torch.Generator().manual_seed(seed)

        def weights(n, k):
            w = torch.randn((n, k), generator=gen) * k ** -0.5
            return mxq.quantize(w.to(device), bits=4)

        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.qkv = weights((heads + 2 * kv_heads) * head_dim, hidden)
        self.out = weights(hidden, heads * head_dim)
        self.q_norm = torch.ones(head_dim, dtype=torch.bfloat16, device=device)
        self.k_norm = torch.ones(head_dim, dtype=torch.bfloat16, device=device)
        self.inv_freq, self.rope_scale = mxq.rope_inv_freq(head_dim, device=device)

    def __call__(self, x, positions, slots, cache, ctx_lens, q_starts=None, max_q_len=1):
        """x bf16 [T, hidden] -> bf16 [T, hidden]: rows q_starts[i]:q_starts[i+1] (None: row i)
        are the last tokens of sequence i, whose ctx_lens[i] tokens are in the cache after
        this call has written its own to `slots`."""
        T, H, K, D = x.shape[0], self.heads, self.kv_heads, self.head_dim
        rows = mxq.qmm(x, *self.qkv, bits=4).view(T, H + 2 * K, D)
        q, k, v = rows[:, :H], rows[:, H:H + K], rows[:, H + K:]
        mxq.qk_norm_rope(q, k, positions, self.inv_freq, self.q_norm, self.k_norm,
                         rope_scale=self.rope_scale, q_out=q, k_out=k)
        mxq.kv_append(k, v, cache.pages, slots)
        o = mxq.kv_attention(q, cache.pages, cache.table, ctx_lens, q_starts, max_q_len)
        return mxq.qmm(o.view(T, H * D), *self.out, bits=4)


def run(hidden=1024, heads=8, kv_heads=2, head_dim=128, page_size=64, prompts=(300, 17, 1, 129),
        steps=24, device="cuda", seed=0):
    """Returns (outputs of the steps, the same asked for at once, microseconds a step)."""
    gen = torch.Generator().manual_seed(seed + 1)
    seqs = len(prompts)
    cache = Cache(seqs, max(prompts) + steps, kv_heads, head_dim, page_size, device, seed)
    layer = AttentionLayer(hidden, heads, kv_heads, head_dim, device, seed)
    new = torch.randn((steps, seqs, hidden), generator=gen).bfloat16().to(device)

    # the prompts, packed
    lens = torch.tensor(prompts, dtype=torch.int32, device=device)
    starts = torch.zeros(seqs + 1, dtype=torch.int32, device=device)
    starts[1:] = lens.cumsum(0)
    seq = torch.repeat_interleave(torch.arange(seqs, device=device), lens)
    positions = torch.cat([torch.arange(n, device=device) for n in prompts]).int()
    x = torch.randn((sum(prompts), hidden), generator=gen).bfloat16().to(device)
    layer(x, positions, cache.slots(seq, positions), cache, lens, starts, max(prompts))

    # one token of each sequence at a time: the step reads and moves its own state
    all_seqs = torch.arange(seqs, device=device)
    x, at, ctx = new[0].clone(), lens.clone(), lens + 1

    def step():
        y = layer(x, at, cache.slots(all_seqs, at), cache, ctx)
        at.add_(1)
        ctx.add_(1)
        return y

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # loads the kernels; the graph's first step writes the same tokens again
    torch.cuda.current_stream().wait_stream(side)
    at.copy_(lens)
    ctx.copy_(lens + 1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    outs = torch.empty((steps, seqs, hidden), dtype=torch.bfloat16, device=device)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    begin.record()
    for i in range(steps):
        x.copy_(new[i])
        graph.replay()
        outs[i] = y
    end.record()
    torch.cuda.synchronize()

    # the same tokens in one call over what the cache holds (negative slots: nothing is written)
    positions = (lens[:, None] + torch.arange(steps, device=device)).int().flatten()
    again = layer(new.transpose(0, 1).reshape(seqs * steps, hidden), positions,
                  torch.full_like(positions, -1), cache, lens + steps,
                  torch.arange(0, seqs * steps + 1, steps, device=device).int(), steps)
    return outs, again.view(seqs, steps, hidden).transpose(0, 1), begin.elapsed_time(end) * 1e3 / steps


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--hidden", type=int, default=5120)
    a.add_argument("--heads", type=int, default=40)
    a.add_argument("--kv-heads", type=int, default=8)
    a.add_argument("--head-dim", type=int, default=128, choices=(64, 128, 256))
    a.add_argument("--page-size", type=int, default=64, choices=(16, 32, 64, 128))
    a.add_argument("--prompts", type=int, nargs="+", default=[4000, 573, 1, 1500])
    a.add_argument("--steps", type=int, default=64)
    o = a.parse_args()
    outs, again, us = run(o.hidden, o.heads, o.kv_heads, o.head_dim, o.page_size, tuple(o.prompts), o.steps)
    off = (outs.double() - again.double()).norm() / again.double().norm()
    print("%d sequences, %.1f us a step; steps against one call over the cache: %.2e of the norm" % (
        len(o.prompts), us, off.item()))


if __name__ == "__main__":
    main()
