"""GPU tests of the 4-bit group-scale linear at both sides of its grid rule and over
the range of fp32 activations.

Tolerance of a sum: as for its other tests, (group + 2 G + 10) * 2^-23 * sum |S c x|.
Where values are tiny an absolute part comes to it, derived below.
"""
import numpy as np
import pytest

from oracle import w4_oracle as WO

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_ternary_b200 import _lib, bitlinear, build

    build.build_library()
    assert _lib.lib().bitlinear_device_check() == 0, "device is not sm_100"
    return bitlinear


def make(N, K, group, seed):
    rng = np.random.default_rng([seed, N, K, group])
    codes = rng.integers(-8, 8, (N, K)).astype(np.int8)
    S = (0.02 * (0.5 + rng.random((N, -(-K // group))))).astype(np.float32)
    return codes, S


def put(B, codes, S, group):
    return B.import_w4(torch.from_numpy(WO.w4_nibbles(codes)).cuda(), torch.from_numpy(S).cuda(), group)


def check(y, x, codes, S, group, absolute=0.0):
    ref = WO.w4_forward(x, codes, S, group)
    K, G = codes.shape[1], S.shape[1]
    tol = (min(group, K) + 2 * G + 10) * 2.0 ** -23 * WO.w4_sum_abs(x, codes, S, group) + absolute
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= tol).all(), f"worst {np.nanmax(err / np.maximum(tol, 1e-300))} of the bound"


# Row tiles of 16 below, at and above one, two and four for each of 148 SMs.
@pytest.mark.parametrize("bf16,M", [(True, 8), (True, 9), (True, 16), (False, 2), (False, 3), (False, 5)])
@pytest.mark.parametrize("tiles", [148, 149, 160, 296, 297, 592, 593, 700])
def test_row_tiles_around_the_sms(B, tiles, M, bf16):
    for N, K in ((16 * tiles, 256), (16 * tiles - 5, 1040)):
        codes, S = make(N, K, 64, 1)
        x = np.random.default_rng([2, M, K]).standard_normal((M, K)).astype(np.float32)
        x = WO.bf16_rn(x) if bf16 else x
        xd = torch.from_numpy(x).cuda()
        check(B.forward_w4(xd.bfloat16() if bf16 else xd, put(B, codes, S, 64)), x, codes, S, 64)


# ------------------------------------------------------------- the range of fp32 x
#
# An fp32 x takes part as three bf16 pieces. A piece is a multiple of 2^-133, so up to
# 2^-133 of an |x| < 2^-110 is left out: sum |S c| * 2^-133. Products of pieces with c * 2^-6
# are multiples of 2^-139 and exact. A group's sum times its scale, in units of 2^-6 too, is
# rounded to a multiple of 2^-149 where it is subnormal, half of that 64 times over after
# the last multiplication: 2^-144 for each of the G groups (and for the last rounding).

def tiny_tolerance(codes, S, group):
    G = S.shape[1]
    per_row = np.abs(WO._dequant(codes, S, group)).sum(axis=1)
    return per_row[None, :] * 2.0 ** -133 + (G + 1) * 2.0 ** -144


def tiny_x(kind, M, K, seed):
    rng = np.random.default_rng([seed, M, K])
    sign = rng.choice([-1.0, 1.0], (M, K))
    if kind == "full significands":  # (1 + 2^-23) 2^-k and random ones, down into the dropped bits
        e = -rng.integers(105, 127, (M, K)).astype(np.float64)
        sig = np.where(rng.random((M, K)) < 0.5, 1 + 2.0 ** -23, 1 + rng.integers(0, 1 << 23, (M, K)) * 2.0 ** -23)
        x = sign * sig * 2.0 ** e
    elif kind == "subnormal":
        x = sign * rng.integers(0, 1 << 23, (M, K)) * 2.0 ** -149
    else:  # "mixed": ordinary values beside tiny ones
        x = rng.standard_normal((M, K)) * 10.0 ** rng.integers(-44, 3, (M, K))
    return x.astype(np.float32)


@pytest.mark.parametrize("M", [1, 5, 6, 40, 130])
@pytest.mark.parametrize("K,group", [(128, 128), (1040, 32)])
@pytest.mark.parametrize("kind", ["full significands", "subnormal", "mixed"])
def test_tiny_fp32_x(B, kind, K, group, M):
    N = 100
    codes, S = make(N, K, group, 3)
    S *= np.float32(50)
    x = tiny_x(kind, M, K, 4)
    check(B.forward_w4(torch.from_numpy(x).cuda(), put(B, codes, S, group)), x, codes, S, group,
          tiny_tolerance(codes, S, group))


@pytest.mark.parametrize("M", [1, 2, 16, 40])
def test_tiny_bf16_x(B, M):
    """A subnormal bf16 is a multiple of 2^-133: nothing of it is left out."""
    N, K, group = 100, 272, 64
    codes, S = make(N, K, group, 5)
    S *= np.float32(50)
    rng = np.random.default_rng([6, M])
    x = (rng.choice([-1.0, 1.0], (M, K)) * rng.integers(0, 1 << 9, (M, K)) * 2.0 ** -133)
    x = WO.bf16_rn(x.astype(np.float32))
    y = B.forward_w4(torch.from_numpy(x).cuda().bfloat16(), put(B, codes, S, group))
    check(y, x, codes, S, group, (S.shape[1] + 1) * 2.0 ** -144)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M", [1, 5, 16, 40, 130])
def test_largest_x(B, M, bf16):
    """The largest finite values, under scales that keep y finite; next to them, a token of ordinary size."""
    N, K, group = 70, 272, 64
    codes, S = make(N, K, group, 7)
    S *= np.float32(2.0 ** -6)
    rng = np.random.default_rng([8, M])
    x = np.zeros((M, K), np.float32)
    top = np.float32(3.3895314e38) if bf16 else np.finfo(np.float32).max  # of bf16: 255 * 2^120
    x[:, 5] = top * rng.choice(np.array([-1, 1], np.float32), M)
    x[:, 200] = top
    if M > 1:
        x[1] = WO.bf16_rn(rng.standard_normal(K).astype(np.float32))
    xd = torch.from_numpy(x).cuda()
    if bf16:
        xd = xd.bfloat16()
        assert np.array_equal(xd.float().cpu().numpy(), x)
    y = B.forward_w4(xd, put(B, codes, S, group))
    assert torch.isfinite(y).all()
    check(y, x, codes, S, group)
