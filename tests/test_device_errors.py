"""The bits of the sticky device error word: one cause each, in one place."""
import os
import re

from selective_state_space_fwd_gb300.build import CSRC


def test_every_bit_has_one_meaning():
    bits, places = [], set()
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            found = re.findall(r"constexpr\s+unsigned(?:\s+int)?\s+kErr\w+\s*=\s*(\w+)u", f.read())
        bits += [int(v, 0) for v in found]
        places |= {name} if found else set()
    assert len(bits) >= 6
    assert len(set(bits)) == len(bits), bits
    assert all(v and v & (v - 1) == 0 and v < 1 << 32 for v in bits), bits
    assert len(places) == 1, places
