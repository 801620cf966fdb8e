"""The rule that says in how many segments a dense FP32 prompt goes (gdelta_rec_segments), on the CPU: it is a function of the sizes and the
number of SMs alone."""
import ctypes
import subprocess
import sys

import pytest

from recurrent_state_02_gb300 import build

RULE = "_ZN2la19gdelta_rec_segmentsEiiiiii"     # la::gdelta_rec_segments(B, H, T, r, dv, sms)


def rule():
    fn = getattr(ctypes.CDLL(build.build()), RULE)
    fn.argtypes, fn.restype = [ctypes.c_int] * 6, ctypes.c_int
    return fn


def test_no_tokens():
    """No tokens are one segment (a segment of no tokens would be divided by: in a process of its own, since that ends it)."""
    build.build()
    code = ("import ctypes; from recurrent_state_02_gb300 import build; "
            f"fn = getattr(ctypes.CDLL(build.build()), '{RULE}'); "
            "assert all(fn(B, H, 0, r, dv, sms) == 1 for B, H, r, dv, sms in "
            "((1, 1, 128, 128, 152), (2, 4, 64, 96, 152), (1, 1, 1, 1, 1), (1, 1, 256, 256, 148)))")
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, (done.returncode, done.stderr)


@pytest.mark.parametrize("r,dv", [(1, 1), (64, 96), (128, 128), (256, 256)])
@pytest.mark.parametrize("sms", [0, 1, 20, 152])
def test_segments_cover_the_tokens(r, dv, sms):
    """Segments are whole blocks of 16 tokens, none is empty, and the first pass's CTAs find an SM each."""
    fn = rule()
    for B, H in ((1, 1), (2, 4), (5, 7), (64, 16)):
        for T in (0, 1, 15, 16, 17, 31, 33, 100, 257, 1001, 8192, 100000, 1 << 30):
            n = fn(B, H, T, r, dv, sms)
            assert 1 <= n <= 16
            if n > 1:
                length = -(-(-(-T // n)) // 16) * 16
                assert (n - 1) * length < T <= n * length
                assert n * B * H * (-(-dv // 32) + -(-r // 32)) <= sms + sms // 8
