"""CPU pins of the 4-bit group-scale oracle and the sampler's oracle, and the
argument checks of their entry points (no GPU needed)."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from bit_ternary_b200 import _lib, build
from oracle import sample_oracle as SO
from oracle import w4_oracle as WO

FAKE = 0x10000  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    build.build_library()
    return _lib.lib()


# ------------------------------------------------------------------ oracles
def test_quantise_by_hand():
    W = np.zeros((1, 48), np.float32)
    W[0, :4] = [7.0, -3.5, 0.5, 1.5]     # S = 1: ties go to even
    W[0, 32:34] = [-14.0, 3.0]           # second, short group: S = 2, 3/2 = 1.5 -> 2
    codes, S = WO.w4_quantise(W, 32)
    assert S.tolist() == [[1.0, 2.0]]
    assert codes[0, :4].tolist() == [7, -4, 0, 2] and codes[0, 32:34].tolist() == [-7, 2]
    assert WO.w4_nibbles(codes)[0, 0] == (15 | (4 << 4))


def test_quantise_zero_group_and_bf16_scale():
    W = np.zeros((2, 32), np.float32)
    W[1, 0] = 1.0
    codes, S = WO.w4_quantise(W, 32, bf16_scales=True)
    assert S[0, 0] == 0 and not codes[0].any()
    assert S[1, 0] == np.float32(0.142578125)  # 1/7 to 8 significand bits
    assert codes[1, 0] == 7


def test_forward_against_rationals():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 48)).astype(np.float32)
    codes = rng.integers(-8, 8, (3, 48)).astype(np.int8)
    S = rng.random((3, 2)).astype(np.float32)
    y = WO.w4_forward(x, codes, S, 32)
    for m in range(2):
        for n in range(3):
            t = sum(Fraction(float(S[n, k // 32])) * int(codes[n, k]) * Fraction(float(x[m, k])) for k in range(48))
            assert abs(y[m, n] - float(t)) <= 1e-12


def test_sample_by_hand():
    row = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    assert SO.sample_kept(row)[0].tolist() == [0, 1, 2, 3]
    assert SO.sample_kept(row, k=2)[0].tolist() == [1, 3]
    assert SO.sample_kept(row, p=0.75)[0].tolist() == [1, 2, 3]  # .4, .7, .9
    assert SO.sample_kept(row, p=0.65)[0].tolist() == [1, 3]
    assert SO.sample_kept(row, p=0.0)[0].tolist() == [1]
    assert SO.sample_kept(row, m=0.6)[0].tolist() == [1, 3]      # .24 of .4 at least
    assert SO.sample_kept(row, k=2, p=0.6)[0].tolist() == [1, 3]  # .4 of .7 is short of .42
    assert SO.sample_kept(row, k=2, p=0.5)[0].tolist() == [1]
    assert [SO.sample_row(row, u)[0] for u in (0.0, 0.05, 0.15, 0.49, 0.55, 0.95)] == [0, 0, 1, 1, 2, 3]
    assert SO.sample_row(row, 0.9, T=0.0) == (1, 0.0)
    t, lp = SO.sample_row(row, 0.99, k=2)
    assert t == 3 and abs(lp - math.log(0.3 / 0.7)) < 1e-9


def test_sample_ties_and_empty_rows():
    assert SO.sample_kept([1.0, 2.0, 2.0, 2.0], k=2)[0].tolist() == [1, 2]
    assert SO.sample_kept([2.0, 2.0, 2.0, 2.0], p=0.5)[0].tolist() == [0, 1]
    assert SO.sample_row([-math.inf, math.nan], 0.3) == (-1, -math.inf)
    assert SO.sample_row([math.nan, 1.0, -math.inf], 0.999) == (1, 0.0)
    assert SO.sample_kept([math.inf, 1.0, math.inf])[1].tolist() == [SO.ONE, 0, SO.ONE]


# ---------------------------------------------------------- entry points
def test_w4_sizes(L):
    assert L.bitlinear_w4_groups(2560, 128) == 20 and L.bitlinear_w4_groups(144, 64) == 3
    for K, g in ((0, 32), (24, 32), (64, 16), (64, 256), (131072 + 16, 32)):
        assert L.bitlinear_w4_groups(K, g) == 0
    # 2 row tiles x 2 blocks x (1024 bytes of codes + 16 rows x 4 groups x 4 or 2 bytes)
    assert L.bitlinear_w4_packed_bytes(17, 144, 32, 0) == 4 * (1024 + 256)
    assert L.bitlinear_w4_packed_bytes(17, 144, 32, 1) == 4 * (1024 + 128)
    assert L.bitlinear_w4_packed_bytes(17, 144, 128, 1) == 4 * (1024 + 32)
    assert L.bitlinear_w4_packed_bytes(17, 144, 32, 2) == 0
    assert L.bitlinear_w4_packed_bytes(-1, 144, 32, 0) == 0
    assert L.bitlinear_w4_workspace_size(3, 5, 24) == 0 and L.bitlinear_w4_workspace_size(-1, 5, 32) == 0
    assert L.bitlinear_w4_workspace_size(3, 5, 32) % 256 == 0
    assert L.bitlinear_w4_sample_workspace_size(3, 1000, 32) >= L.bitlinear_w4_workspace_size(3, 1000, 32) + 12000


def test_w4_entry_points_validate_before_cuda(L):
    big = 1 << 24
    f, fb = L.bitlinear_forward_w4, L.bitlinear_forward_w4_bf16
    for fn in (f, fb):
        assert fn(None, 0, 5, 16, 32, 0, None, None, None, 0, None) == 0
        assert fn(None, 5, 0, 16, 32, 0, None, None, None, 0, None) == 0
        assert fn(FAKE, 1, 1, 24, 32, 0, FAKE, FAKE, FAKE, big, None) == 2
        assert fn(FAKE, 1, 1, 32, 48, 0, FAKE, FAKE, FAKE, big, None) == 2
        assert fn(FAKE, 1, 1, 32, 32, 7, FAKE, FAKE, FAKE, big, None) == 2
        assert fn(FAKE, -1, 1, 32, 32, 0, FAKE, FAKE, FAKE, big, None) == 2
        assert fn(FAKE, 1, 1 << 31, 32, 32, 0, FAKE, FAKE, FAKE, big, None) == 2
        for hole in (0, 6, 7, 8):
            a = [FAKE, 1, 1, 32, 32, 0, FAKE, FAKE, FAKE, big, None]
            a[hole] = None
            assert fn(*a) == 1
            a[hole] = FAKE + 8
            assert fn(*a) == 3
        assert fn(FAKE, 4, 1, 32, 32, 0, FAKE, FAKE, FAKE, 256, None) == 4
    for fn in (L.bitlinear_pack_weights_w4, L.bitlinear_pack_weights_w4_bf16):
        assert fn(FAKE, 0, 32, 32, 0, FAKE, FAKE, big, None) == 2
        assert fn(FAKE, 1, 32, 33, 0, FAKE, FAKE, big, None) == 2
        assert fn(None, 1, 32, 32, 0, FAKE, FAKE, big, None) == 1
        assert fn(FAKE + 4, 1, 32, 32, 0, FAKE, FAKE, big, None) == 3
        assert fn(FAKE, 1, 32, 32, 0, FAKE, FAKE, 16, None) == 4
    assert L.bitlinear_w4_import(FAKE, FAKE, 1, 8, 32, 0, FAKE, None) == 2
    assert L.bitlinear_w4_import(FAKE, None, 1, 16, 32, 0, FAKE, None) == 1
    assert L.bitlinear_w4_import(FAKE, FAKE + 4, 1, 16, 32, 0, FAKE, None) == 3
    assert L.bitlinear_w4_import(None, None, 0, 16, 32, 0, None, None) == 0
    assert L.bitlinear_w4_export(FAKE, 1, 16, 0, 0, FAKE, FAKE, None) == 2
    assert L.bitlinear_w4_export(FAKE, 1, 16, 32, 0, None, FAKE, None) == 1
    assert L.bitlinear_w4_export(FAKE, 1, 16, 32, 0, FAKE + 4, FAKE, None) == 3


def test_sample_entry_points_validate_before_cuda(L):
    how = _lib.Sampling(None, None, None, None, 1.0, 0, 1.0, 0.0)
    h = ctypes.byref(how)
    for fn, odd in ((L.bitlinear_sample, 2), (L.bitlinear_sample_bf16, 1)):
        assert fn(None, 0, 8, 8, None, None, None, None, None) == 0
        assert fn(FAKE, 1, 0, 8, h, FAKE, FAKE, FAKE, None) == 2
        assert fn(FAKE, -1, 8, 8, h, FAKE, FAKE, FAKE, None) == 2
        assert fn(FAKE, 1, 8, 7, h, FAKE, FAKE, FAKE, None) == 2
        assert fn(FAKE, 1, (1 << 22) + 1, 1 << 23, h, FAKE, FAKE, FAKE, None) == 2
        assert fn(None, 1, 8, 8, h, FAKE, FAKE, FAKE, None) == 1
        assert fn(FAKE, 1, 8, 8, None, FAKE, FAKE, FAKE, None) == 1
        assert fn(FAKE, 1, 8, 8, h, None, FAKE, FAKE, None) == 1
        assert fn(FAKE, 1, 8, 8, h, FAKE, None, FAKE, None) == 1
        assert fn(FAKE + odd, 1, 8, 8, h, FAKE, FAKE, FAKE, None) == 3
        assert fn(FAKE, 1, 8, 8, h, FAKE, FAKE + 4, FAKE, None) == 3
        assert fn(FAKE, 1, 8, 8, h, FAKE + 2, FAKE, FAKE, None) == 3
    bad = _lib.Sampling(FAKE + 2, None, None, None, 1.0, 0, 1.0, 0.0)
    assert L.bitlinear_sample(FAKE, 1, 8, 8, ctypes.byref(bad), FAKE, FAKE, FAKE, None) == 3
    for fn in (L.bitlinear_forward_w4_sample, L.bitlinear_forward_w4_sample_bf16):
        need = L.bitlinear_w4_sample_workspace_size(2, 8, 32)
        assert fn(FAKE, 2, 8, 32, 32, 0, FAKE, h, FAKE, FAKE, FAKE, FAKE, need - 1, None) == 4
        assert fn(FAKE, 2, 8, 32, 32, 0, FAKE, h, FAKE, FAKE, FAKE, None, need, None) == 1
        assert fn(FAKE, 2, 8, 32, 32, 0, FAKE, None, FAKE, FAKE, FAKE, FAKE, need, None) == 1
        assert fn(FAKE, 2, 8, 40, 32, 0, FAKE, h, FAKE, FAKE, FAKE, FAKE, need, None) == 2
        assert fn(FAKE, 2, 8, 32, 40, 0, FAKE, h, FAKE, FAKE, FAKE, FAKE, need, None) == 2
        assert fn(FAKE, 2, 0, 32, 32, 0, FAKE, h, FAKE, FAKE, FAKE, FAKE, need, None) == 2
        assert fn(None, 0, 8, 32, 32, 0, None, None, None, None, None, None, 0, None) == 0


def test_python_refusals_on_cpu_tensors():
    torch = pytest.importorskip("torch")
    from bit_ternary_b200 import bitlinear as B

    with pytest.raises(ValueError):
        B.sample(torch.zeros(1, 4), torch.zeros(1))
    with pytest.raises(ValueError):
        B.import_w4(torch.zeros((1, 16), dtype=torch.uint8), torch.zeros(1, 1), 32)
    with pytest.raises(ValueError):
        B.pack_weights_w4(torch.zeros(1, 16))
