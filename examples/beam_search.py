"""Beam search over a 4-bit cache: the prompts' pages shared by their beams, one layer of attention,
4-bit projections.

    python examples/beam_search.py

takes the prompts in one packed call, then goes on with several beams of each: every step selects
the best continuations, reorders the cache and attends over the prompt, once for all of its beams, and each
beam's own tokens.  At the end the beams found are asked for in one call, each a sequence of its own: their
scores are the same up to rounding.  The weights and the prompts are random.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import affine_bit_matmul_gb300 as mxq  # noqa: E402
from attention_layer import AttentionLayer, Cache  # noqa: E402


class Model(AttentionLayer):
    """Embeddings, one attention layer beside them, and the logits of the next token."""

    def __init__(self, vocab, hidden, heads, kv_heads, head_dim, device, seed=0):
        super().__init__(hidden, heads, kv_heads, head_dim, device, seed)
        gen = torch.Generator().manual_seed(seed + 2)
        self.embed = torch.randn((vocab, hidden), generator=gen).bfloat16().to(device)
        head = torch.randn((vocab, hidden), generator=gen) * 2.0 * hidden ** -0.5
        self.head = mxq.quantize(head.to(device), bits=4)

    def logits(self, x, y):
        return mxq.qmm(x + y, *self.head, bits=4)

    def beams(self, x, positions, slots, pages, prefix, table, lens):
        """One row of each beam after its group's prefix (page table, lengths)."""
        T, H, K, D = x.shape[0], self.heads, self.kv_heads, self.head_dim
        rows = mxq.qmm(x, *self.qkv, bits=4).view(T, H + 2 * K, D)
        q, k, v = rows[:, :H], rows[:, H:H + K], rows[:, H + K:]
        mxq.qk_norm_rope(q, k, positions, self.inv_freq, self.q_norm, self.k_norm, rope_scale=self.rope_scale, q_out=q, k_out=k)
        mxq.kv_append(k, v, pages, slots)
        o = mxq.kv_attention_shared(q, pages, *prefix, table, lens)
        return self.logits(x, mxq.qmm(o.view(T, H * D), *self.out, bits=4))


def run(vocab=512, hidden=512, heads=8, kv_heads=2, head_dim=128, page_size=16, prompts=(70, 5, 33), beams=4, steps=20,
        device="cuda", seed=0):
    """Returns (tokens [prompts, beams, steps], which of them count, their scores, the same scores asked for
    at once, the largest logit)."""
    gen = torch.Generator().manual_seed(seed + 1)
    n, end = len(prompts), 0
    model = Model(vocab, hidden, heads, kv_heads, head_dim, device, seed)
    each = -(-steps // page_size)
    cache = Cache(n, max(prompts), kv_heads, head_dim, page_size, device, seed)
    pages = torch.cat((cache.pages, torch.zeros((n * beams * each,) + cache.pages.shape[1:], dtype=torch.uint8, device=device)))
    cache.pages = pages

    # the prompts, packed; the last row of each gives the first logits of its beams
    text = [torch.randint(1, vocab, (p,), generator=gen).to(device) for p in prompts]
    lens = torch.tensor(prompts, dtype=torch.int32, device=device)
    starts = torch.zeros(n + 1, dtype=torch.int32, device=device)
    starts[1:] = lens.cumsum(0)
    seq = torch.repeat_interleave(torch.arange(n, device=device), lens)
    positions = torch.cat([torch.arange(p, device=device) for p in prompts]).int()
    x = model.embed[torch.cat(text)]
    y = model(x, positions, cache.slots(seq, positions), cache, lens, starts, max(prompts))
    last = (starts[1:] - 1).long()
    logits = model.logits(x[last], y[last]).repeat_interleave(beams, 0)

    # pages for the beams' own tokens
    home = (cache.table.numel() + torch.arange(n * beams * each, dtype=torch.int32, device=device)).view(n * beams, each)
    table, own = home.clone(), torch.zeros(n * beams, dtype=torch.int32, device=device)
    scores = torch.full((n, beams), float("-inf"), device=device)
    scores[:, 0] = 0.0  # all beams are the same yet
    done = torch.zeros((n, beams), dtype=torch.bool, device=device)
    all_beams, prompt_of = torch.arange(n * beams, device=device), torch.arange(n, device=device).repeat_interleave(beams)
    history = []
    for _ in range(steps):
        scores, parents, tokens, done = mxq.beam_select(logits, scores, done=done, end_token=end)
        history.append((parents, tokens, done))
        mxq.kv_reorder(pages, table, home, own, parents, head_dim, table_out=table, lens_out=own)
        slots = table[all_beams, (own // page_size).long()] * page_size + own % page_size
        at = lens[prompt_of] + own
        own += 1
        logits = model.beams(model.embed[tokens.flatten().long()], at, slots, pages, (cache.table, lens), table, own)

    # the beams' tokens, from the last step back
    out, counts = torch.empty((n, beams, steps), dtype=torch.long, device=device), torch.empty((n, beams, steps), dtype=torch.bool, device=device)
    beam = torch.arange(beams, device=device).expand(n, beams)
    for i in reversed(range(steps)):
        parents, tokens, _ = history[i]
        out[..., i] = tokens.gather(1, beam)
        beam = parents.gather(1, beam).long()
        before = history[i - 1][2].gather(1, beam) if i else torch.zeros_like(beam, dtype=torch.bool)
        counts[..., i] = ~before  # (a beam that has ended goes on with end tokens that count nothing)

    # all of them again, each prompt and its continuation a sequence of its own
    rows = [torch.cat((text[g], out[g, b])) for g in range(n) for b in range(beams)]
    whole = torch.tensor([len(r) for r in rows], dtype=torch.int32, device=device)
    again = Cache(n * beams, max(prompts) + steps, kv_heads, head_dim, page_size, device, seed)
    starts = torch.zeros(n * beams + 1, dtype=torch.int32, device=device)
    starts[1:] = whole.cumsum(0)
    seq = torch.repeat_interleave(torch.arange(n * beams, device=device), whole)
    positions = torch.cat([torch.arange(len(r), device=device) for r in rows]).int()
    x = model.embed[torch.cat(rows)]
    y = model(x, positions, again.slots(seq, positions), again, whole, starts, max(prompts) + steps)
    want = (starts[1:].long()[:, None] - steps - 1) + torch.arange(steps, device=device)  # rows before each token
    z = model.logits(x[want.flatten()], y[want.flatten()]).double()
    top = z[z.isfinite()].abs().max().item()
    each = z.log_softmax(-1).gather(1, out.view(-1, 1)).view(n, beams, steps)
    return out, counts, scores, torch.where(counts, each, 0.0).sum(-1), top


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--vocab", type=int, default=32768)
    a.add_argument("--hidden", type=int, default=2048)
    a.add_argument("--heads", type=int, default=16)
    a.add_argument("--kv-heads", type=int, default=4)
    a.add_argument("--head-dim", type=int, default=128, choices=(64, 128, 256))
    a.add_argument("--page-size", type=int, default=64, choices=(16, 32, 64, 128))
    a.add_argument("--prompts", type=int, nargs="+", default=[1000, 573, 60])
    a.add_argument("--beams", type=int, default=8)
    a.add_argument("--steps", type=int, default=100)
    o = a.parse_args()
    tokens, counts, scores, again, _ = run(o.vocab, o.hidden, o.heads, o.kv_heads, o.head_dim, o.page_size, tuple(o.prompts), o.beams, o.steps)
    for g in range(len(o.prompts)):
        print("prompt of %d tokens: best score %.3f (at once: %.3f)" % (o.prompts[g], scores[g, 0].item(), again[g, 0].item()))


if __name__ == "__main__":
    main()
