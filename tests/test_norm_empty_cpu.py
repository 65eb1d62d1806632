"""A batch of no images: modulations without rows for no rows (no GPU needed)."""

import pytest
import torch

from rotation_quantized_int8_amd import norms


def test_empty_batch_has_an_empty_modulation():
    x, mod = torch.zeros((0, 8), dtype=torch.float16), torch.zeros((0, 8), dtype=torch.float16)
    assert norms._modulation(x, 0, 8, mod, mod, mod, None)[0] is None
    index = torch.zeros((0,), dtype=torch.int32)
    assert norms._modulation(x, 0, 8, mod, mod, mod, index)[0] is None
    with pytest.raises(ValueError, match="split"):
        norms._modulation(torch.zeros((2, 8), dtype=torch.float16), 2, 8, mod, mod, None, None)
    with pytest.raises(ValueError):
        norms._modulation(x, 0, 8, mod, torch.zeros((1, 8), dtype=torch.float16), None, None)
