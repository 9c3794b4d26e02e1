"""What the compiler gave the state space layer's kernels, from the metadata of the built library's code objects."""
import os
import struct

import pytest

import delta_rule_sequence_amd as prism

msgpack = pytest.importorskip("msgpack")


def kernels(path):
    """The metadata of every gfx950 kernel in the library: name -> fields."""
    data, found, at = open(path, "rb").read(), {}, 0
    while (at := data.find(b"\x7fELF\x02\x01\x01", at + 1)) > 0:              # embedded 64-bit objects (the library itself is at 0)
        if struct.unpack_from("<H", data, at + 18)[0] != 0xe0:                # EM_AMDGPU
            continue
        table, = struct.unpack_from("<Q", data, at + 0x28)
        width, count = struct.unpack_from("<HH", data, at + 0x3a)
        for k in range(count):
            kind, _, _, offset, size = struct.unpack_from("<IQQQQ", data, at + table + k * width + 4)
            if kind != 7:                                                     # SHT_NOTE
                continue
            names, length, note = struct.unpack_from("<III", data, at + offset)
            if note == 32:                                                    # the code object's metadata
                start = at + offset + 12 + (names + 3) // 4 * 4
                for f in msgpack.unpackb(data[start:start + length], strict_map_key=False)["amdhsa.kernels"]:
                    found[f[".name"]] = f
    return found


def test_no_register_goes_to_scratch():
    if not os.path.exists(prism.LIB_PATH):
        pytest.fail("libprism.so is not built (run __graft_entry__.build())")
    layer = {n: f for n, f in kernels(prism.LIB_PATH).items() if any(s in n for s in ("5prism3ssm", "5prism4conv", "5prism4norm"))}
    assert len(layer) > 100
    spilled = {n: (f[".private_segment_fixed_size"], f[".vgpr_spill_count"]) for n, f in layer.items()
               if f[".private_segment_fixed_size"] or f[".vgpr_spill_count"]}
    assert not spilled, spilled
