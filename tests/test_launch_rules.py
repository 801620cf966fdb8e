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
                   '{ return la::rec_columns(rows, ctas, brief != 0, sms); }\n')
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    lib = ctypes.CDLL(str(lib))
    lib.rec_columns.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
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
