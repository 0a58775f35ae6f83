"""Several status words read as one, with copies that fail (fakes on the host)."""
import ctypes
import os
import subprocess

import pytest

from combine_quant_gb300 import build as cqbuild

SOURCE = r"""
#include "cq_status.h"
// calls 0..n-1 read, n waits, n + 1 + i clears word i; call `bad` (-1: none) fails with -7
extern "C" int run(int n, uint32_t* words, int bad, uint32_t* status) {
  static uint32_t copies[8];
  return cq::collect_status(
      n, copies, [&](int i, uint32_t* read) { if (i == bad) return -7; *read = words[i]; return 0; },
      [&] { return bad == n ? -7 : 0; },
      [&](int i) { if (n + 1 + i == bad) return -7; words[i] = 0; return 0; }, status);
}
"""
UNTOUCHED = 0xdead


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    d = tmp_path_factory.mktemp("status")
    src, lib = d / "status.cpp", d / "libstatus.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(cqbuild.CSRC), str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).run

    def call(words, bad=-1):
        w, st = (ctypes.c_uint32 * len(words))(*words), ctypes.c_uint32(UNTOUCHED)
        return f(len(words), w, bad, ctypes.byref(st)), st.value, list(w)
    return call


def test_all_words_in_one_and_cleared(run):
    assert run([1, 0, 4, 8, 1]) == (0, 13, [0] * 5)
    assert run([0] * 5) == (0, 0, [0] * 5)


@pytest.mark.parametrize("bad", range(6))
def test_a_failing_read_or_wait_loses_nothing(run, bad):
    words = [1, 0, 4, 8, 1]
    assert run(words, bad) == (-7, UNTOUCHED, words)


@pytest.mark.parametrize("bad", [0, 2, 3, 4])
def test_a_failing_clear_loses_nothing(run, bad):
    words = [1, 0, 4, 8, 1]
    rc, status, left = run(words, 6 + bad)
    assert (rc, status) == (-7, 13)
    assert left == [v if i == bad else 0 for i, v in enumerate(words)]
