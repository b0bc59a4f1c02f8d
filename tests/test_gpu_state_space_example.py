"""The example block: a prompt and then single tokens give what one long prompt gives."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tokens_continue_a_prompt():
    """Both paths round the block's five intermediate rows to bf16 (and the prompt's projections their weights): ten
    roundings of at most 2^-8 of their values each."""
    spec = importlib.util.spec_from_file_location("state_space_block", os.path.join(ROOT, "examples", "state_space_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    worst, drift = module.main(["--model", "256", "--prompt", "150", "--tokens", "12", "--batch", "3"])
    assert worst < 10 * 2.0 ** -8
    assert max(drift) < 10 * 2.0 ** -8
