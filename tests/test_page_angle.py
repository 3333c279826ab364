"""A position's angle as halves of a turn (lbx_qk_norm_rope), checked on the host against
fractions (no GPU needed).

The frequency's fraction of a turn is off by half a unit of 2^-64 and |f| 2^-129 turns
(test_page_turn), so that of the position by |pos| times that; the conversion to fp32 takes
2^-24 of the value. In halves of a turn, from -1 to 1 (which are the same angle)."""
import os
import random
import struct
import subprocess
from fractions import Fraction

from test_page_turn import _pi
from tree_verify_linear_gb300 import build


def _bits(x):
    return struct.unpack("I", struct.pack("f", x))[0]


def test_half_turns(tmp_path):
    here, exe = os.path.dirname(os.path.abspath(__file__)), str(tmp_path / "check")
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC,
                    "-o", exe, os.path.join(here, "page_angle_check.cu")], check=True, capture_output=True)
    random.seed(2)
    positions = [0, 1, -1, 2, -3, 1000, 4097, 131072, 2 ** 31 - 1, -2 ** 31]
    freqs = [10.0 ** -e for e in range(13)] + [1e7 ** (-i / 64) for i in range(64)] + [-1e-6, 3.0, 40.5, 0.0]
    pairs = [(_bits(f), p) for f in freqs for p in positions]
    pairs += [(_bits(10.0 ** random.uniform(-10, 1)), random.randrange(-2 ** 31, 2 ** 31)) for _ in range(1000)]
    pairs += [(_bits(10.0 ** random.uniform(-10, 0)), random.randrange(5000)) for _ in range(1000)]
    r = subprocess.run([exe], input="\n".join("%u %d" % x for x in pairs), capture_output=True, text=True, timeout=60)
    got = [Fraction(float.fromhex(x)) for x in r.stdout.split()]
    assert len(got) == len(pairs)
    at = 400
    pi = Fraction(_pi(at), 1 << at)
    for (bits, p), g in zip(pairs, got):
        f = Fraction(struct.unpack("f", struct.pack("I", bits))[0])
        exact = f * p / pi  # halves of a turn
        exact -= 2 * ((exact + 1) // 2)
        off = abs(exact - g)
        off = min(off, abs(2 - off))
        assert -1 <= g <= 1
        assert off <= abs(exact) / (1 << 24) + Fraction(2 * abs(p), 1 << 64) * (1 + abs(f)), (bits, p)
