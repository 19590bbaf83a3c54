"""The example block: prompts in chunks and then single tokens, against whole sequences at once."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_prompts_then_single_tokens():
    import __graft_entry__

    __graft_entry__.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "linear_attention_block.py")
    spec = importlib.util.spec_from_file_location("linear_attention_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # two blocks of about ten bf16 roundings each (2^-9 of a value in the mean, twice that at most),
    # those of the two orders independent of one another
    assert example.main() <= 2 * 20 ** 0.5 * 2.0 ** -8
