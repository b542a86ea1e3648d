"""The example's search: selection, reordering and shared attention together, as they are used."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "beam_search.py")
    spec = importlib.util.spec_from_file_location("beam_search", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("heads,kv_heads,head_dim,page,prompts,beams,steps", [
    (8, 2, 128, 16, (70, 5, 33), 4, 20), (4, 4, 64, 32, (200,), 3, 40), (8, 1, 256, 64, (40, 41, 42, 43), 9, 12), (8, 2, 128, 16, (9, 300), 33, 18)])
def test_beams_have_their_scores(heads, kv_heads, head_dim, page, prompts, beams, steps):
    """Every beam's score is that of its tokens after its prompt.  A logit in bf16 is off by 2^-8 of itself where
    the values before it differ by roundings; those of the layer's output and of the sum with the embedding
    move it as much again each (2^-8 of numbers of its size): 3 * 2^-8 of the largest logit for a token's and 3 *
    2^-8 for the logarithm of its row's sum, in each step of both ways."""
    tokens, counts, scores, again, top = example().run(heads=heads, kv_heads=kv_heads, head_dim=head_dim, page_size=page,
                                                       prompts=prompts, beams=beams, steps=steps)
    assert scores.isfinite().all() and (scores[:, :-1] >= scores[:, 1:]).all()
    assert counts[..., 0].all()
    assert ((scores.double() - again).abs() <= 6 * 2.0 ** -8 * top * counts.sum(-1)).all()
    # no two beams of a prompt are the same
    for g in range(len(prompts)):
        kept = {tuple(t for t, c in zip(tokens[g, b].tolist(), counts[g, b].tolist()) if c) for b in range(beams)}
        assert len(kept) == beams
