"""What the compiler gave the attention layer's kernels, from the metadata of the built library's code objects."""
import os

import pytest

import delta_rule_sequence_amd as prism
from tests.test_layer_resources import kernels


def test_no_register_goes_to_scratch():
    if not os.path.exists(prism.LIB_PATH):
        pytest.fail("libprism.so is not built (run __graft_entry__.build())")
    layer = {n: f for n, f in kernels(prism.LIB_PATH).items() if "5prism4attn" in n or "5prism4rope" in n}
    assert len(layer) > 60
    spilled = {n: (f[".private_segment_fixed_size"], f[".vgpr_spill_count"]) for n, f in layer.items()
               if f[".private_segment_fixed_size"] or f[".vgpr_spill_count"]}
    assert not spilled, spilled


def test_two_waves_per_simd_where_the_design_counts_on_them():
    """Kernels of bfloat16 whose blocks share a CU (or have eight waves) stay within 256 registers."""
    for n, f in kernels(prism.LIB_PATH).items():
        if "5prism4attn10fwd_kernelIDF16b" in n or ("5prism4attn9dq_kernelIDF16b" in n and "ELi1ELi64ELb1E" in n):
            assert f[".vgpr_count"] <= 256, (n, f[".vgpr_count"])
