"""A frequency as a fraction of a turn (lbx_qk_norm_rope), checked on the host against
integers of 2000 bits (no GPU needed)."""
import os
import random
import struct
import subprocess
from fractions import Fraction

from tree_verify_linear_gb300 import build


def _pi(bits):
    """pi 2^bits, within 64 of it: 16 atan(1/5) - 4 atan(1/239)."""
    def atan(n):
        term, total, k = (1 << bits) // n, 0, 0
        while term:
            total += -(term // (2 * k + 1)) if k % 2 else term // (2 * k + 1)
            term, k = term // (n * n), k + 1
        return total
    return 16 * atan(5) - 4 * atan(239)


def test_turns_of(tmp_path):
    here, exe = os.path.dirname(os.path.abspath(__file__)), str(tmp_path / "check")
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC,
                    "-o", exe, os.path.join(here, "page_turn_check.cu")], check=True, capture_output=True)
    random.seed(1)
    bits = [s << 31 | e << 23 | m for s in (0, 1) for e in range(255) for m in (0, 1, 0x400000, 0x7fffff)]
    bits += [random.randrange(0x30000000, 0x4c000000) for _ in range(2000)]
    r = subprocess.run([exe], input="\n".join(map(str, bits)), capture_output=True, text=True, timeout=60)
    got = [int(x) for x in r.stdout.split()]
    assert len(got) == len(bits)
    at, one = 2000, 1 << 64
    pi = _pi(at)
    for f, g in zip(bits, got):
        x = Fraction(struct.unpack("f", struct.pack("I", f))[0])
        # x / (2 pi) in units of 2^-64, to 2^-64 of one
        exact = Fraction(x.numerator * (1 << (at + 127)) // (x.denominator * pi), one)
        off = abs(exact - g) % one
        off = min(off, one - off)
        # half a unit, and 1 / (2 pi) off by 2^-129
        assert off <= Fraction(1, 2) + abs(x) / (1 << 65) + Fraction(1, 1 << 60), hex(f)
