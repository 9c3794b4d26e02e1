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


# what the kernels' names say (type, width, form), how many there are, and the registers that leave a SIMD its waves
WAVES = {"forwards over prompts, rows of up to 128 bytes: four waves": ("fwd_kernel", ("IDF16bLi32E", "IDF16bLi64E", "IfLi32E"), "KeysE0E", 4, 128),
         "forwards of bfloat16: two waves": ("fwd_kernel", ("IDF16b",), "", 13, 256),
         "few rows of up to 256 bytes: two waves": ("few_kernel", ("IDF16b", "IfLi32E", "IfLi64E"), "", 13, 256),
         "dq of many bfloat16 rows: two waves": ("dq_kernel", ("IDF16b",), "ELb1E", 3, 256),
         "dk and dv of many bfloat16 rows in eight waves: two": ("dkv_kernel", ("IDF16b",), "ELb1E", 2, 256)}


@pytest.mark.parametrize("name", WAVES)
def test_registers_of_each_form(name):
    kernel, types, form, count, most = WAVES[name]
    found = {n: f[".vgpr_count"] for n, f in kernels(prism.LIB_PATH).items()
             if "5prism4attn" in n and kernel in n and form in n and any(kernel + t in n for t in types)}
    assert len(found) == count, found
    assert max(found.values()) <= most, found
