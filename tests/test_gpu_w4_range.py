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
