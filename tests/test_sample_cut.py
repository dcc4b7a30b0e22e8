"""CPU test of how the sampler cuts rows into clusters (bl_sample_cut.h, compiled
here for the host), with a stand-in for the device's answer whether a cluster of
more than eight CTAs can run."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIXED = 40000
SMEM_MAX = 225 * 1024

SOURCE = """
#include "bl_sample_cut.h"
extern "C" void cut(int64_t B, int64_t V, int sms, size_t fixed, int large_fit, int64_t* out) {
  int asked = 0;
  const bl::SampleCut c = bl::sample_cut(B, V, sms, fixed, [&](const bl::SampleCut& s) {
    ++asked;
    out[6] = s.cluster;
    return large_fit != 0;
  });
  out[0] = c.cluster;
  out[1] = c.per;
  out[2] = c.resident;
  out[3] = c.wide;
  out[4] = (int64_t)c.smem;
  out[5] = asked;
}
"""


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    d = tmp_path_factory.mktemp("cut")
    (d / "c.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "bit_ternary_b200", "csrc"), "-o", str(d / "c.so"), str(d / "c.cpp")],
                   check=True)
    fn = ctypes.CDLL(str(d / "c.so")).cut
    fn.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p]

    def call(B, V, large_fit=True, sms=148):
        out = (ctypes.c_int64 * 7)()
        fn(B, V, sms, FIXED, int(large_fit), out)
        return dict(zip(("cluster", "per", "resident", "wide", "smem", "asked", "asked_for"), out))

    return call


SIZES = [(B, V) for B in (1, 2, 9, 10, 64, 256, 100003, (1 << 31) - 1)
         for V in (1, 7, 2048, 4096, 32000, 50021, 128000, 131075, 262128, 262129, 500009, 1000003, 1 << 22)]


@pytest.mark.parametrize("B,V", SIZES)
def test_every_row_is_covered(cut, B, V):
    for large in (True, False):
        c = cut(B, V, large)
        assert c["cluster"] in (1, 2, 4, 8, 16)
        assert c["per"] * c["cluster"] >= V
        assert c["smem"] <= SMEM_MAX
        assert c["resident"] == (FIXED + 4 * (c["per"] + 16) <= SMEM_MAX)
        assert c["smem"] == FIXED + (4 * (c["per"] + 16) if c["resident"] else 0)
        assert not c["wide"] or (c["resident"] and B * c["cluster"] <= 148)


@pytest.mark.parametrize("B,V", SIZES)
def test_where_sixteen_cannot_run_eight_take_the_row(cut, B, V):
    with_large, without = cut(B, V, True), cut(B, V, False)
    assert without["cluster"] == min(with_large["cluster"], 8)
    if with_large["cluster"] <= 8:
        assert with_large["asked"] == 0 and without == with_large  # nothing to ask
    else:
        assert with_large["asked"] == without["asked"] == 1 and without["asked_for"] == 16


def test_a_row_with_sms_to_itself_takes_sixteen(cut):
    assert cut(1, 128000)["cluster"] == 16 and cut(1, 128000)["wide"] == 1
    assert cut(256, 128000)["cluster"] == 8 and cut(256, 128000)["wide"] == 0
    assert cut(1, 1 << 22)["cluster"] == 16 and cut(1, 1 << 22)["resident"] == 0
