"""Normalising append, attention of drafted trees, compaction and forks together, as a server uses them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("hidden,heads,kv_heads,dim,prompts,samples", [
    (512, 4, 2, 128, [70, 1, 129, 17], 2), (400, 8, 1, 64, [3], 1), (1040, 5, 5, 64, [200, 64], 3), (512, 2, 1, 256, [40, 90], 2)])
def test_prompts_samples_drafts(hidden, heads, kv_heads, dim, prompts, samples):
    """An e4m3 rounding is at most 2^-4 of its value, 2^-4 / sqrt(3) in the mean square at the very
    most.  Each layer is compared on the inputs that it had: input, weight, cached value, attention's output
    and weight again lie on the way of a value (sqrt(5) of them: 0.081), input, weight and cached key on the
    way of a score, whose softmax passes on less than its own size of the error for scores of unit variance
    (sqrt(3): 0.063 more; a norm only takes the part of an error along the head away).  Codes that are moved,
    or scaled for a larger exponent, change by a power of two, which is exact but where a code becomes
    subnormal (off by 2^-10, in a page whose largest is 224 or more): under 0.15."""
    spec = importlib.util.spec_from_file_location("drafted_tokens", os.path.join(ROOT, "examples", "drafted_tokens.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    err, same, right, kept, _ = example.run(hidden, heads, kv_heads, dim, prompts, samples, 6)
    assert err < 0.15 and same and right and kept >= 1
