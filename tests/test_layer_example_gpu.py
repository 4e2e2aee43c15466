"""Norm, 8-bit products and rotary positions together with the cache, as examples/hybrid_decoder.py uses them."""
import pytest

from test_hybrid_example_gpu import example  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,tail", [((70, 1, 133), 3), ((5, 0, 200, 16), 2)])
def test_prompts_then_tokens_agree_with_8_bit_projections(example, lens, tail):  # noqa: F811
    """One layer of four has its two projections in 8 bits.  An activation whose bf16 value differs by a step between the two
    runs may be rounded to the next e4m3 value, 2^-3 of itself off at most: with a few such per row of 512, a row's sums are off by
    some 2^-3 sqrt(5 / 512) = 0.012 of its RMS, less than what the bf16 steps and the cache's scales give (0.03 typically).
    The bound is the one for bf16 projections."""
    assert example.compare(lens, tail, eight_bit=True) <= 0.3
