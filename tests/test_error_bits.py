"""Host check that the device error word's bits are the same, and distinct, in the three places that name
them: the kernels' one list, the public header and the Python binding."""
import os
import re

from deepseek_v4_engram_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def read(*path):
    with open(os.path.join(ROOT, *path)) as f:
        return f.read()


def test_error_bits_agree():
    header = dict(re.findall(r"#define ENGRAM_DEVERR_(\w+) (\d+)u", read("include", "engram.h")))
    header = {name: int(bit) for name, bit in header.items()}
    assert len(set(header.values())) == len(header) >= 5
    assert all(bit & (bit - 1) == 0 and bit > 0 for bit in header.values())
    assert {n[len("DEVERR_"):]: b for n, b in vars(_lib).items() if n.startswith("DEVERR_")} == header
    csrc = os.path.join("deepseek_v4_engram_gb300", "csrc")
    enum = re.search(r"enum : uint32_t \{(.*?)\};", read(csrc, "device.cuh"), re.S).group(1)
    kernels = {int(bit) for bit in re.findall(r"kErr\w+ = (\d+)u", enum)}
    assert kernels == set(header.values())
    # and no bit is defined anywhere else
    for name in os.listdir(os.path.join(ROOT, csrc)):
        if name != "device.cuh":
            assert not re.search(r"\bkErr\w+ = ", read(csrc, name)), name
