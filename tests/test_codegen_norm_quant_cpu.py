"""Registers of the quantising norms' kernels (no GPU needed): compiled for gfx950,
none of them may spill to memory."""

import pytest

import test_codegen_mx_cpu as base


@pytest.mark.skipif(base._hipcc() is None, reason="hipcc not available")
def test_no_quantising_norm_spills_to_memory(tmp_path):
    base.test_no_kernel_spills_to_memory("norm_quant.hip", tmp_path)
