"""The projections, the cache and the attention together, as a decoder layer uses them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("hidden,heads,kv_heads,dim,prompts", [
    (512, 4, 2, 128, [70, 1, 129, 17]), (400, 8, 1, 64, [3]), (1040, 5, 5, 64, [200, 64]), (512, 2, 1, 256, [40, 90])])
def test_prompt_then_tokens(hidden, heads, kv_heads, dim, prompts):
    """An e4m3 rounding is at most 2^-4 of its value, 2^-4 / sqrt(3) in the mean square at the very
    most.  Input, weight, cached value, attention's output and weight again lie on the way of a value
    (sqrt(5) of them: 0.081), input, weight and cached key on the way of a score, whose softmax passes on
    less than its own size of the error for scores of unit variance (sqrt(3): 0.063 more): under 0.15."""
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    err, same, _, _ = example.run(hidden, heads, kv_heads, dim, prompts, 6)
    assert err < 0.15 and same
