"""The example's layer: projections, norm and rotation, cache and attention together."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("heads,kv_heads,head_dim,page,prompts", [
    (8, 2, 128, 64, (300, 17, 1, 129)), (6, 6, 64, 16, (40,)), (8, 1, 256, 128, (5, 200))])
def test_steps_are_the_prompt(heads, kv_heads, head_dim, page, prompts):
    """The two ways differ by roundings alone: of the attention's result, 5e-3 of the norm for each
    at most, of the queries to bf16 (2^-8 of scores of about one, in each), and of the layer's
    output (2^-8 for each): below 1e-2 + 8e-3 + 8e-3."""
    outs, again, _ = example().run(hidden=512, heads=heads, kv_heads=kv_heads, head_dim=head_dim, page_size=page,
                                   prompts=prompts, steps=12)
    a, b = outs.double(), again.double()
    assert a.isfinite().all() and b.norm() > 0
    assert (a - b).norm() / b.norm() < 2.6e-2
