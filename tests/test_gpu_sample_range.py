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


# ------------------------------------------------------------- large vocabularies

def sample_row_int64(row, u, T, k, p, m):
    """SO.sample_row for long rows: the same integers, in int64 (sums below 2^62)."""
    row = np.asarray(row, np.float64)
    idx = np.flatnonzero(~np.isnan(row) & (row != -np.inf))
    idx = idx[np.argsort(-row[idx], kind="stable")]
    best = row[idx[0]]
    w = np.rint(np.exp((row[idx] - best) / T) * 2.0 ** 40).astype(np.int64)
    if k > 0:
        idx, w = idx[:k], w[:k]
    if p < 1:
        run = np.cumsum(w)
        need = max(p, 0.0) * float(run[-1])
        n = 1 + int(np.searchsorted(run.astype(np.float64), need, side="left"))
        idx, w = idx[:n], w[:n]
    keep = w >= min(m, 1.0) * 2.0 ** 40
    idx, w = idx[keep], w[keep]
    order = np.argsort(idx)
    idx, w = idx[order], w[order]
    run = np.cumsum(w)
    total = int(run[-1])
    target = min(int(u * float(total)), total - 1)
    i = int(np.searchsorted(run, target, side="right"))
    return int(idx[i]), (row[idx[i]] - best) / T - math.log(total / 2.0 ** 40)


def test_the_oracle_for_long_rows_is_the_oracle():
    g = np.random.default_rng(2)
    for V in (1, 50, 1500):
        for how in ((1.0, 0, 1.0, 0.0), (0.75, 40, 0.9, 0.0), (1.5, 0, 0.5, 0.03125), (1.0, 7, 1.0, 0.5)):
            x = np.round(g.standard_normal(V) * 4).astype(np.float32) / 2
            u = float(np.float32(g.random()))
            t, l = sample_row_int64(x, u, *how)
            t2, l2 = SO.sample_row(x, u, *how)
            assert t == t2 and abs(l - l2) < 1e-12


def long_row(V, kind, seed):
    g = np.random.default_rng([seed, V])
    x = (g.standard_normal(V) * 2.2).astype(np.float32)
    if kind == "ties":
        x = np.round(x * 4).astype(np.float32) / np.float32(4)
    elif kind == "flat":
        x = (g.random(V) * 0.001).astype(np.float32)
    elif kind == "masked":
        x[g.random(V) < 0.7] = -np.inf
        x[g.random(V) < 0.1] = np.finfo(np.float32).min
    return x


# 16 CTAs take a row. 262128 tokens are the last that pack counts above sums of places
# in a word; past them a bin has a count alone. 1000003 tokens stay in global memory.
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [131075, 262128, 262129, 262144, 500009, 1000003])
def test_vocabularies_past_a_packed_histogram(B, V, bf16):
    rows = [long_row(V, kind, 3) for kind in ("body", "ties", "flat", "masked")]
    xd = torch.from_numpy(np.stack(rows)).cuda()
    if bf16:
        xd = xd.bfloat16()
        rows = list(xd.float().cpu().numpy())
    u = np.array([0.3, 0.62, 0.97, 0.5], np.float32)
    ud = torch.from_numpy(u).cuda()
    settings = [(1.0, 0, p, 0.0) for p in (0.5, 0.9, 0.99, 0.9999)]
    settings += [(0.75, 5000, 0.9, 0.0), (1.0, 60000, 0.99, 0.0), (1.0, 60000, 1.0, 0.0), (2.0, 0, 0.8, 0.0625),
                 (1.0, 0, 1.0, 0.0)]
    for T, k, p, m in settings:
        tok, lp = B.sample(xd, ud, T, k, p, m)
        for r, x in enumerate(rows):
            t, l = sample_row_int64(x, float(u[r]), T, k, float(np.float32(p)), m)
            assert int(tok[r]) == t, (T, k, p, m, r, int(tok[r]), t)
            assert close(float(lp[r]), l, V), (T, k, p, m, r)


def test_one_row_and_many_of_a_large_vocabulary(B):
    """One row (1024 threads a CTA) and 40 of them (two CTAs an SM) of the same logits."""
    V = 262144
    x = long_row(V, "body", 4)
    u = ((np.arange(40) + 0.5) / 40).astype(np.float32)
    one = torch.from_numpy(x[None]).cuda()
    ud = torch.from_numpy(u).cuda()
    for p in (0.9, 0.99):
        tok, lp = B.sample(one.expand(40, V).contiguous(), ud, 1.0, 0, p)
        for i in range(40):
            t, l = sample_row_int64(x, float(u[i]), 1.0, 0, float(np.float32(p)), 0.0)
            assert int(tok[i]) == t and close(float(lp[i]), l, V)
            if i % 8 == 0:
                a, b = B.sample(one, ud[i:i + 1], 1.0, 0, p)
                assert int(a) == t and float(b) == float(lp[i])


# Row counts at which the cut changes: the most that run at once as clusters of 16 wide and
# narrow CTAs, of 8 and of 4, and one more.
@pytest.mark.parametrize("rows", [7, 8, 14, 15, 16, 33, 36])
@pytest.mark.parametrize("V", [20000, 50021])
def test_row_counts_at_which_the_cut_changes(B, V, rows):
    x = np.stack([long_row(V, ("body", "ties", "flat", "masked")[r % 4], 5 + r) for r in range(rows)])
    u = ((np.arange(rows) + 0.5) / rows).astype(np.float32)
    xd, ud = torch.from_numpy(x).cuda(), torch.from_numpy(u).cuda()
    for T, k, p, m in ((1.0, 0, 0.9, 0.0), (0.75, 50, 0.9, 0.0), (1.0, 0, 1.0, 0.0)):
        tok, lp = B.sample(xd, ud, T, k, p, m)
        for r in range(rows):
            t, l = sample_row_int64(x[r], float(u[r]), T, k, float(np.float32(p)), m)
            assert int(tok[r]) == t and close(float(lp[r]), l, V), (T, k, p, r)
