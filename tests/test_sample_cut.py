"""CPU test of how the sampler cuts rows into clusters (bl_sample_cut.h, compiled
here for the host), with stand-ins for the device's answers how many clusters of a
form it runs at a time."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FIXED = 40000
SMEM_MAX = 225 * 1024
PACK_MAX = 16383
SMS = 148

SOURCE = """
#include "bl_sample_cut.h"
typedef int (*AtOnce)(int cluster, int wide, size_t smem);
extern "C" void cut(int64_t B, int64_t V, int sms, size_t fixed, AtOnce at_once, int64_t* out) {
  const bl::SampleCut c = bl::sample_cut(B, V, sms, fixed, [&](const bl::SampleCut& s) {
    return at_once(s.cluster, s.wide, s.smem);
  });
  out[0] = c.cluster;
  out[1] = c.per;
  out[2] = c.resident;
  out[3] = c.wide;
  out[4] = (int64_t)c.smem;
}
"""
AT_ONCE = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_size_t)


def per_sm(wide, smem):
    return 1 if wide or 2 * (smem + 1024) > 228 * 1024 else 2


def b200(cluster, wide, smem):
    """The counts of one B200."""
    wide_counts = {16: 7, 8: 15, 4: 34, 2: 74, 1: 148}
    narrow_counts = {16: 14, 8: 33, 4: 70, 2: 148, 1: 296}
    return (wide_counts if per_sm(wide, smem) == 1 else narrow_counts)[cluster]


def no_large(cluster, wide, smem):
    return 0 if cluster > 8 else b200(cluster, wide, smem)


def no_answer(cluster, wide, smem):
    return 0


@pytest.fixture(scope="module")
def cut(tmp_path_factory):
    d = tmp_path_factory.mktemp("cut")
    (d / "c.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "bit_ternary_b200", "csrc"), "-o", str(d / "c.so"), str(d / "c.cpp")],
                   check=True)
    fn = ctypes.CDLL(str(d / "c.so")).cut
    fn.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, AT_ONCE, ctypes.c_void_p]

    def call(B, V, at_once=b200):
        out = (ctypes.c_int64 * 5)()
        fn(B, V, SMS, FIXED, AT_ONCE(at_once), out)
        return dict(zip(("cluster", "per", "resident", "wide", "smem"), out))

    return call


ROWS = [1, 2, 7, 8, 9, 10, 15, 16, 18, 19, 20, 33, 34, 36, 64, 256, 100003, (1 << 31) - 1]
VOCABULARIES = [1, 7, 2048, 4096, 32000, 50021, 128000, 131075, 262128, 262129, 500009, 1000003, 1 << 22]


@pytest.mark.parametrize("at_once", [b200, no_large, no_answer])
@pytest.mark.parametrize("V", VOCABULARIES)
def test_every_row_is_covered(cut, V, at_once):
    for B in ROWS:
        covered(B, V, at_once, cut(B, V, at_once))


def covered(B, V, at_once, c):
    assert c["cluster"] in (1, 2, 4, 8, 16)
    assert c["per"] * c["cluster"] >= V > c["per"] * (c["cluster"] - 1)
    assert c["resident"] == (FIXED + 4 * (c["per"] + 16) <= SMEM_MAX)
    assert c["smem"] == FIXED + (4 * (c["per"] + 16) if c["resident"] else 0)
    assert not c["wide"] or (c["resident"] and B * c["cluster"] <= SMS)
    # Stretches that some cut packs are packed.
    assert c["per"] <= PACK_MAX or V > PACK_MAX * (16 if at_once is b200 else 8)


@pytest.mark.parametrize("V", VOCABULARIES)
def test_a_cluster_that_the_device_cannot_run_is_not_asked_of_it(cut, V):
    for B in ROWS:
        for at_once in (no_large, no_answer):
            assert cut(B, V, at_once)["cluster"] <= 8
        c = cut(B, V)
        assert b200(c["cluster"], c["wide"], c["smem"]) > 0


@pytest.mark.parametrize("V", VOCABULARIES)
def test_all_rows_run_at_once_where_a_packed_cut_of_theirs_can(cut, V):
    for B in ROWS:
        at_once_where_they_can(B, V, cut(B, V))


def at_once_where_they_can(B, V, c):
    most = 1
    while most < 16 and ((V + most - 1) // most > PACK_MAX or (B * most * 2 <= 2 * SMS and V // (2 * most) >= 2048)):
        most *= 2
    can = False
    for C in (16, 8, 4, 2, 1):
        if C <= most and (C == most or -(-V // C) <= PACK_MAX):
            smem = FIXED + 4 * (-(-V // C) + 16)
            smem = smem if smem <= SMEM_MAX else FIXED
            can = can or b200(C, False, smem) >= B
    assert (b200(c["cluster"], c["wide"], c["smem"]) >= B) == can, (B, V, c)


def test_known_cuts(cut):
    def form(B, V, at_once=b200):
        c = cut(B, V, at_once)
        return c["cluster"], "wide" if c["wide"] else "narrow"

    assert form(1, 128000) == form(7, 128000) == (16, "wide")
    assert form(8, 128000) == form(14, 128000) == (16, "narrow")  # seven wide ones run at a time
    assert form(15, 128000) == (8, "wide")
    assert form(16, 128000) == form(33, 128000) == (8, "narrow")
    assert form(34, 128000) == form(256, 128000) == (8, "narrow")  # four CTAs would not pack
    assert form(36, 50021) == (4, "narrow")
    assert form(8, 128000, no_large) == (8, "wide")
    assert cut(1, 1 << 22)["cluster"] == 16 and cut(1, 1 << 22)["resident"] == 0
