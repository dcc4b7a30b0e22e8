"""CPU test of the bounds by which the sampler places the border of top-p
(bl_sample_bounds.h, compiled here for the host): every bin's exact weight lies
between them.

The bins are filled as the kernel fills them (fp32 positions, rounded to 64ths,
counts and sums of places in 13 + 19 or 14 + 18 bits, or counts alone). The
bounds are computed in fp32: eight roundings of 2^-24 relative on either side,
the position's two (of up to 2047 bins, within the 0.002 bins that the bounds
allow) and the weight's slack of 2^-40 per token are what the comparison leaves room for.
"""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BINS = 2048
ROUNDING = 8 * 2.0 ** -24

SOURCE = """
#include "bl_sample_bounds.h"
extern "C" void bounds(float e, float delta, int packed, uint32_t count, uint32_t off, float* out) {
  const bl::WeightBounds w = bl::bin_weight(e, delta, bl::bin_places(packed), count, off);
  out[0] = w.lo;
  out[1] = w.hi;
}
"""


@pytest.fixture(scope="module")
def bounds(tmp_path_factory):
    d = tmp_path_factory.mktemp("bounds")
    (d / "b.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "bit_ternary_b200", "csrc"), "-o", str(d / "b.so"), str(d / "b.cpp")],
                   check=True)
    fn = ctypes.CDLL(str(d / "b.so")).bounds
    fn.argtypes = [ctypes.c_float, ctypes.c_float, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint32, ctypes.c_void_p]

    def call(e, delta, packed, count, off):
        out = (ctypes.c_float * 2)()
        fn(e, delta, packed, count, off, out)
        return out[0], out[1]

    return call


def place_sum(v, packed):
    """The sum that the histogram keeps of places v (64ths of a bin)."""
    return int((v // 4).sum()) if packed == 18 else (int(v.sum()) if packed == 19 else len(v))


def inside(bounds, e, delta, packed, places, exact):
    lo, hi = bounds(e, delta, packed, len(places), place_sum(places, packed))
    slack = len(places) * 2.0 ** -40
    assert lo * (1 - ROUNDING) - slack <= exact, (delta, packed, lo / exact - 1)
    assert exact <= hi * (1 + ROUNDING) + slack, (delta, packed, exact / hi - 1)


@pytest.mark.parametrize("packed", [19, 18, 0])
@pytest.mark.parametrize("delta", [2.0 ** -k for k in range(6, 21)] + [29 / 2047, 0.004, 0.0039, 0.01])
def test_tokens_at_either_end_of_their_places(bounds, delta, packed):
    """A place is a rounded 64th: its tokens lie up to 1/128 of a bin to either side,
    those of place 0 before the bin's start."""
    edge = 1 / 128
    d = float(np.float32(delta))
    for v in (0, 1, 3, 4, 31, 32, 60, 63):
        for count in (1, 2, 1000):
            places = np.full(count, v)
            for f in (v / 64 - edge, v / 64, v / 64 + edge):
                inside(bounds, 1.0, d, packed, places, count * np.exp(-d * f))
    both = np.array([0, 63] * 500)  # half at the start's far side, half at the end's
    for f0, f1 in ((-edge, 63 / 64 - edge), (edge, 63 / 64 + edge), (-edge, 63 / 64 + edge)):
        inside(bounds, 1.0, d, packed, both, 500 * (np.exp(-d * f0) + np.exp(-d * f1)))


@pytest.mark.parametrize("packed", [19, 18, 0])
@pytest.mark.parametrize("T", [0.1, 1.0, 3.0, 30.0])
@pytest.mark.parametrize("shape", ["body", "ties", "narrow"])
def test_bins_of_whole_rows(bounds, shape, T, packed):
    g = np.random.default_rng([packed, int(10 * T)])
    x = (g.standard_normal(8000) * 2.2).astype(np.float32)
    if shape == "ties":
        x = np.round(x * 8).astype(np.float32) / np.float32(8)
    elif shape == "narrow":  # all within half a place of the largest
        x = np.float32(4) - (np.abs(x) * np.float32(29 * T / 2047 / 600)).astype(np.float32)
    top = x.max()
    f32 = np.float32
    reach = min(f32(29) * f32(T), top - x.min())
    scale = f32(BINS - 1) / f32(reach)
    delta = f32(f32(1 / float(f32(T))) / scale)
    pos = np.minimum((top - x) * scale, f32(BINS - 1))
    place = np.rint(pos.astype(np.float64) * 64).astype(np.int64)
    weight = np.exp((x.astype(np.float64) - float(top)) / float(f32(T)))
    for b in np.unique(place >> 6):
        if b == BINS - 1:
            continue  # the last bin is open: it has no lower bound
        mine = (place >> 6) == b
        # The weight at the bin's start from the bins' own scale, in 64 bits: the roundings of
        # the exponent (1 / T, delta, up to 29 in all) are the kernel's margin, not the bounds'.
        e = float(f32(np.exp(-b / (float(f32(T)) * float(scale)))))
        inside(bounds, e, float(delta), packed, place[mine] & 63, weight[mine].sum())
