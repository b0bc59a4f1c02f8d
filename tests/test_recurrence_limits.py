"""What the recurrence's entry points ask for and refuse at the ends of their ranges, without a GPU (CPU only)."""
import pytest

import test_recurrence_abi as abi


@pytest.mark.parametrize("tokens", [0, 100, 1 << 30])
@pytest.mark.parametrize("bias", [0, 11 * abi.G])
def test_gradient_of_no_sequences_needs_nothing(tokens, bias):
    """Packed rows without a sequence: no chunk, and so no workgroup that would look for its offsets."""
    assert abi._back(nseq=0, tokens=tokens, offsets=20 * abi.G, grad_forget_bias=bias) == 0
