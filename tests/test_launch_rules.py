"""Sizes and choices behind the launches (csrc/launch_rules.h), compiled for the host: what a kernel
reads stays in its arrays, and what is chosen is what the device can run."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "recurrent_state_02_gb300", "csrc")


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    src, lib = d / "rules.cpp", d / "rules.so"
    src.write_text('#include "launch_rules.h"\n'
                   'extern "C" int whole_granules(int V, int ge) { return la::whole_granules(V, ge); }\n'
                   'extern "C" int rec_columns(int rows, long long ctas, int brief, int sms)\n'
                   '{ return la::rec_columns(rows, ctas, brief != 0, sms); }\n'
                   'extern "C" int rec_segments(long long units, int rows, int T, const int *one, const int *two)\n'
                   '{ return la::rec_segments(units, rows, T, one, two); }\n')
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    lib = ctypes.CDLL(str(lib))
    lib.rec_columns.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    lib.rec_segments.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    return lib


@pytest.mark.parametrize("ge", [4, 8])
def test_granules_end_inside_the_row(rules, ge):
    """The 16-byte loads of an aligned row cover no element past its end, and leave less than a granule."""
    for V in [*range(1, 70), 1501, 32003, 131071, 131072, (1 << 30) - 1, 1 << 30]:
        n = rules.whole_granules(V, ge)
        assert n * ge <= V < (n + 1) * ge, V


@pytest.mark.parametrize("sms", [152, 132, 20])
def test_columns_of_the_recurrence(rules, sms):
    """Packed sequences of up to 64 rows keep few columns per lane (four take a third longer on long prompts); the
    border between few CTAs and many is the device's SM count."""
    for brief in (0, 1):
        for rows in (1, 32, 33, 64):
            assert rules.rec_columns(rows, sms, brief, sms) == 1
            assert all(rules.rec_columns(rows, n, brief, sms) == 2 for n in (sms + 1, 4096, 1 << 40))
        for rows in (65, 128, 129, 256):
            assert rules.rec_columns(rows, sms, brief, sms) == 2
            assert rules.rec_columns(rows, sms + 1, brief, sms) == (4 if brief else 2)


# clusters of 2 .. 16 CTAs with one, two CTAs per SM: a whole device, one without clusters of more than 8, a partition of
# few SMs, and one that places none
ROOM = {
    "whole": ([76, 46, 36, 28, 23, 15, 15, 15, 13, 8, 8, 7, 7, 7, 7], [152, 97, 74, 58, 46, 38, 36, 30, 28, 23, 23, 19, 14, 14, 14]),
    "portable": ([76, 46, 36, 28, 23, 15, 15] + [0] * 8, [152, 97, 74, 58, 46, 38, 36] + [0] * 8),
    "partition": ([8, 5, 4, 2, 2, 2, 1] + [0] * 8, [16, 10, 8, 5, 4, 4, 3] + [0] * 8),
    "none": ([0] * 15, [0] * 15),
}


@pytest.mark.parametrize("device", ROOM)
def test_segments_find_room(rules, device):
    """The recurrence is cut only into clusters that the device places, all of them at once, and never when it places
    none; a short sequence stays whole."""
    one, two = ROOM[device]
    arrays = [(ctypes.c_int * 17)(0, 0, *x) for x in (one, two)]
    seen = set()
    for units in [*range(1, 160), 65536, 1 << 32]:
        for rows in (1, 32, 64, 100, 128, 129, 256):
            for T in (1, 127, 128, 300, 512, 1001, 16384, 1 << 30):
                n = rules.rec_segments(units, rows, T, *arrays)
                seen.add(n)
                assert 1 <= n <= 16 and (T >= 128 or n == 1)
                assert n == 1 or units <= one[n - 2] or (rows <= 128 and units <= two[n - 2]), (units, rows, T, n)
    assert max(seen) == {"whole": 16, "portable": 8, "partition": 8, "none": 1}[device]
