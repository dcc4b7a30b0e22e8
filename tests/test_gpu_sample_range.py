"""GPU tests of the sampler where its bins stop describing the row: vocabularies of
more tokens than a histogram word packs, and settings at which the logits' span
has no fp32 value. Tokens equal the integer oracle's.

Log-probabilities: rounded to fp32 once (2^-24 relative); a weight of the kernel's
may be one unit of 2^-40 of the largest beside the oracle's, V * 2^-40 of the sum
at most, which is at least 1.
"""
import math

import numpy as np
import pytest

from oracle import sample_oracle as SO

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


def close(lp, l, V):
    return lp == l if math.isinf(l) else abs(lp - l) <= 2.0 ** -24 * abs(l) + 2.0 ** -40 * V


HUGE = [dict(T=T, p=p, k=k) for T in (1.2e37, 2e37, 1e38, 3e38) for p in (0.2, 0.4, 0.9, 1.0) for k in (0, 40)]


@pytest.mark.parametrize("V", [2, 100, 700, 5000])
def test_spans_past_the_largest_fp32_value(B, V):
    """The largest logit less the least is more than fp32 holds, and so is the bins' range."""
    g = np.random.default_rng([1, V])
    x = np.empty((4, V), np.float32)
    x[0], x[0, V // 2] = -3e38, 3e38
    x[1] = g.uniform(-3.4, 3.4, V) * 1e38
    x[2] = g.choice([-3.3e38, -1e38, 1e38, 3.3e38], V)
    x[3], x[3, 0] = g.uniform(-3.4, -3.3, V) * 1e38, 3.4e38
    u = np.array([0.9, 0.3, 0.6, 0.97], np.float32)
    xd, ud = torch.from_numpy(x).cuda(), torch.from_numpy(u).cuda()
    for how in HUGE:
        tok, lp = B.sample(xd, ud, how["T"], how["k"], how["p"])
        for r in range(4):
            t, l = SO.sample_row(x[r], float(u[r]), float(np.float32(how["T"])), how["k"], float(np.float32(how["p"])))
            assert int(tok[r]) == t, (how, r, int(tok[r]), t)
            assert close(float(lp[r]), l, V), (how, r)
