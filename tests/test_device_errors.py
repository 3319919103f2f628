"""The bits of the sticky device error word: one cause each."""
import os
import re

from selective_state_space_fwd_gb300.build import CSRC


def test_every_bit_has_one_meaning():
    bits = {}
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            for which, v in re.findall(r"constexpr\s+unsigned(?:\s+int)?\s+(kErr\w+)\s*=\s*(\w+)u;", f.read()):
                assert which not in bits, which
                bits[which] = int(v, 0)
    assert len(bits) >= 6
    assert len(set(bits.values())) == len(bits), bits
    assert all(v and v & (v - 1) == 0 and v < 1 << 32 for v in bits.values()), bits
