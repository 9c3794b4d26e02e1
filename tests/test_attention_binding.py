"""Arguments of the attention layer's Python calls that need no GPU."""
import pytest
import torch

import delta_rule_sequence_amd as prism
from delta_rule_sequence_amd import attention, layer


@pytest.mark.parametrize("window", [-2 ** 32 + 5, -2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5])
def test_windows_that_a_c_int_would_cut_off(window):
    """-2^32 + 5 would arrive as 5."""
    m = (torch.Size((1, 2, 8, 64)), (1024, 512, 64, 1), torch.float32)
    with pytest.raises(prism.PrismError):
        layer._sizes(8, window)
    with pytest.raises(prism.PrismError):
        attention._prompt(m, m, m, None, True, window, 0)
