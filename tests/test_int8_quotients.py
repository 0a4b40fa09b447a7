"""The codes of the quantisation to 8-bit integers (a correctly rounded reciprocal,
a product and two fma) are those of the division: all 2^23 scales of one binade
with two values on either side of each of the 127 borders between two codes, and
every seventh scale of binades up to the ends of the range that the kernel takes
that way (scales from 2^-92).  On the CPU; the kernel itself is compared with the
division at sampled scales in test_gpu_int8."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.slow
def test_all_scales_and_borders(tmp_path):
    cc = shutil.which("g++")
    if cc is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "int8_quotients")
    # (an fma of the processor where there is one, else the library's: the same result)
    subprocess.run([cc, "-O3", "-march=native", "-ffp-contract=off", "-pthread", "-o", exe, os.path.join(HERE, "int8_quotients.cpp")],
                   check=True, timeout=120)
    binades = {0: 1, -92: 7, -91: 7, -45: 7, 60: 7, 120: 7}
    out = subprocess.run([exe] + [str(v) for b in binades.items() for v in b], check=True, timeout=600, stdout=subprocess.PIPE)
    lines = [[int(v) for v in line.split()] for line in out.stdout.decode().splitlines()]
    assert [v[0] for v in lines] == list(binades)
    for exponent, n, bad, plain in lines:
        # (the last scales of a thread's part may be one less or more)
        assert n >= (1 << 23) // binades[exponent] * 127 * 5 and bad == 0, (exponent, bad)
        assert 0.05 < plain / n < 0.06, "a product with the reciprocal alone: 5 % other codes"
