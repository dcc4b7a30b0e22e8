"""GPU tests of the sampler against its integer oracle: tokens equal, and
log-probabilities to the rounding of their fp32 result.

Tolerance of a log-probability: it is rounded to fp32 once (2^-24 relative); the
64-bit value behind it differs from the oracle's by the weights' rounding to
2^-40 of the largest, V * 2^-41 relative to the sum at most, far below.
"""
import math

import numpy as np
import pytest

from oracle import sample_oracle as SO
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


def check(B, logits, u, T=1.0, k=0, p=1.0, m=0.0, settings=None):
    """logits: fp32 or bf16 CUDA [rows, V]; scalars, or lists with one setting per row."""
    rows = logits.shape[0]

    def per_row(v):
        return list(v) if isinstance(v, (list, tuple, np.ndarray)) else [v] * rows

    Ts, ks, ps, ms = per_row(T), per_row(k), per_row(p), per_row(m)
    f = dict(dtype=torch.float32, device="cuda")
    ut = torch.tensor(u, **f)
    tok, lp = B.sample(logits, ut, torch.tensor(Ts, **f), torch.tensor(ks, dtype=torch.int32, device="cuda"),
                       torch.tensor(ps, **f), torch.tensor(ms, **f))
    tok, lp, x = tok.cpu().numpy(), lp.cpu().numpy(), logits.float().cpu().numpy()
    f32 = lambda v: float(np.float32(v))  # noqa: E731  (settings reach the kernel in fp32)
    for r in range(rows):
        t, l = SO.sample_row(x[r], f32(u[r]), f32(Ts[r]), ks[r], f32(ps[r]), f32(ms[r]))
        assert tok[r] == t, f"row {r}: token {tok[r]} instead of {t}"
        if math.isinf(l):
            assert lp[r] == l
        else:
            assert abs(lp[r] - l) <= 2.0 ** -24 * abs(l) + 2.0 ** -41 * x.shape[1] + 1e-12
    return tok, lp


def body(rows, V, seed, sigma=2.0):
    g = np.random.default_rng([seed, rows, V])
    x = (g.standard_normal((rows, V)) * sigma).astype(np.float32)
    x[:, g.integers(0, V, 5)] += 6
    return x, g.random(rows).astype(np.float32)


def put(x, bf16=False):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.bfloat16() if bf16 else t


MODES = [dict(), dict(T=0.7), dict(T=0.0), dict(k=1), dict(k=50), dict(k=1000), dict(p=0.9), dict(p=0.0),
         dict(p=0.9999), dict(m=0.05), dict(m=1.0), dict(k=40, p=0.95), dict(T=1.3, k=100, p=0.8, m=0.02),
         dict(p=0.5, m=0.3), dict(k=3, p=0.999), dict(T=30.0, p=0.97)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("mode", MODES, ids=[str(m) for m in MODES])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4099])
def test_modes(B, V, mode, bf16):
    x, u = body(4, V, 1)
    check(B, put(x, bf16), u, **mode)


@pytest.mark.parametrize("mode", [dict(), dict(k=50, p=0.95), dict(p=0.9), dict(k=5000), dict(k=20000, p=0.99)],
                         ids=str)
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [32000, 50021, 131075])
def test_large_vocabularies(B, V, bf16, mode):
    x, u = body(2, V, 2, 1.0)
    check(B, put(x, bf16), u, **mode)


def test_settings_per_row(B):
    x, u = body(64, 3001, 3)
    g = np.random.default_rng(4)
    check(B, put(x), u, T=g.choice([0.0, 0.5, 1.0, 2.0], 64), k=[int(v) for v in g.choice([0, 1, 5, 100, 9999], 64)],
          p=g.choice([0.0, 0.3, 0.9, 1.0], 64), m=g.choice([0.0, 0.01, 0.5], 64))


@pytest.mark.parametrize("V", [7, 5000, 70001])
def test_masked_rows(B, V):
    """Nothing left, one token left, -inf, the type's lowest value, NaN, +inf."""
    x, _ = body(9, V, 5)
    x[0] = -np.inf
    x[1] = np.nan
    x[2] = -np.inf
    x[2, V - 1] = -3.0
    x[3, ::2] = np.finfo(np.float32).min
    x[4] = np.finfo(np.float32).min
    x[5, 1::2] = np.nan
    x[6, [1, V - 2]] = np.inf
    x[7, : V - 1] = -np.inf
    x[8] = np.finfo(np.float32).max
    u = np.full(9, 0.6, np.float32)
    for mode in (dict(), dict(k=2), dict(p=0.7), dict(T=0.0), dict(m=0.5), dict(k=3, p=0.5, T=0.01)):
        check(B, put(x), u, **mode)


@pytest.mark.parametrize("V", [9, 4097, 66000])
def test_ties(B, V):
    """All equal, two levels, and runs of equal values across the threshold."""
    g = np.random.default_rng(6)
    x = np.zeros((4, V), np.float32)
    x[1, ::3] = 1.0
    x[2] = np.round(g.standard_normal(V) * 2)
    x[3] = np.where(g.random(V) < 0.5, 0.0, -0.0)
    u = np.array([0.25, 0.999, 0.5, 0.75], np.float32)
    for mode in (dict(), dict(k=3), dict(k=V // 2), dict(p=0.5), dict(p=0.31, k=V - 2), dict(T=0.0), dict(m=0.9)):
        check(B, put(x), u, **mode)


def test_u_at_the_ends(B):
    x, _ = body(6, 513, 7)
    u = np.array([0.0, -1.0, np.nan, np.nextafter(np.float32(1), np.float32(0)), 1.0, 2.0], np.float32)
    for mode in (dict(), dict(k=10), dict(p=0.9), dict(T=0.0)):
        check(B, put(x), u, **mode)


def test_extreme_settings(B):
    x, u = body(8, 1025, 8)
    nan, inf = math.nan, math.inf
    check(B, put(x), u, T=[1e-45, 1e-30, 1e30, inf, -1.0, nan, 1e-3, 1.0], k=[0] * 7 + [-5])
    check(B, put(x), u, p=[nan, -1.0, inf, 1e-45, 2.0, 0.5, 1.0, 0.0])
    check(B, put(x), u, m=[nan, -1.0, inf, 1e-45, 2.0, 0.5, 1.0, 0.0], k=[2 ** 31 - 1] * 8)


def test_wide_range_of_logits(B):
    """Values over the whole fp32 range: subnormals, huge gaps."""
    g = np.random.default_rng(9)
    x = (g.standard_normal((4, 3000)) * 10.0 ** g.integers(-44, 38, (4, 3000))).astype(np.float32)
    x[1] *= np.float32(1e-30)
    x[2] = np.float32(1e-40) * g.standard_normal(3000).astype(np.float32)
    u = g.random(4).astype(np.float32)
    for mode in (dict(), dict(k=500), dict(p=0.6), dict(k=2999, p=0.99), dict(T=1e-38, p=0.9)):
        check(B, put(x), u, **mode)


def test_scalars_are_the_same_as_tensors(B):
    x, u = body(5, 2000, 10)
    tok, lp = check(B, put(x), u, T=0.75, k=30, p=0.5, m=0.125)
    t2, l2 = B.sample(put(x), torch.from_numpy(u).cuda(), 0.75, 30, 0.5, 0.125)
    assert np.array_equal(t2.cpu().numpy(), tok) and np.array_equal(l2.cpu().numpy(), lp)


@pytest.mark.parametrize("bf16", [False, True])
def test_rows_apart_and_unaligned(B, bf16):
    x, u = body(6, 1003, 11)
    wide = put(np.pad(x, ((0, 0), (3, 9)), constant_values=100.0), bf16)  # neighbours must not be read as tokens
    view = wide[:, 3:1006]
    assert not view.is_contiguous()
    for mode in (dict(), dict(k=20), dict(p=0.9)):
        check(B, view, u, **mode)


def test_draws_follow_the_distribution(B):
    """100000 draws of one row, stratified u: every token's count is within one of its share."""
    p = np.array([0.05, 0.2, 0.1, 0.4, 0.25])
    x = np.log(p).astype(np.float32)
    n = 100000
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    tok, _ = B.sample(put(np.tile(x, (n, 1))), torch.from_numpy(u).cuda())
    share = np.bincount(tok.cpu().numpy(), minlength=5) / n
    # u is rounded to fp32 (2^-25) and log p too (2^-24 * |log p| * p): under 1e-6 per border
    assert np.abs(share - p).max() <= 2 / n + 2e-6


def test_streams_and_graphs(B):
    x, u = body(3, 40001, 12)
    ref, _ = check(B, put(x), u, k=50, p=0.9)
    xd, ud = put(x), torch.from_numpy(u).cuda()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for i in range(6):  # two calls at once
        with torch.cuda.stream(s1 if i % 2 else s2):
            outs.append(B.sample(xd, ud, 1.0, 50, 0.9)[0])
    torch.cuda.synchronize()
    assert all(np.array_equal(o.cpu().numpy(), ref) for o in outs)
    xin, uin = torch.zeros_like(xd), torch.zeros_like(ud)
    g = torch.cuda.CUDAGraph()
    B.sample(xin, uin, 1.0, 50, 0.9)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        tok, lp = B.sample(xin, uin, 1.0, 50, 0.9)
    for seed in (12, 13):
        x, u = body(3, 40001, seed)
        xin.copy_(put(x))
        uin.copy_(torch.from_numpy(u).cuda())
        g.replay()
        torch.cuda.synchronize()
        t, _ = check(B, put(x), u, k=50, p=0.9)
        assert np.array_equal(tok.cpu().numpy(), t)


def test_largest_vocabulary(B):
    V = 1 << 22
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((2, V), generator=g, device="cuda")
    x[:, 4000000] = 9.0
    for mode in (dict(k=20), dict(k=20, p=0.5), dict(T=0.0)):
        # The oracle on the kept candidates only: everything below the top 64 is out in these modes.
        tok, lp = B.sample(x, torch.tensor([0.3, 0.8], device="cuda"), mode.get("T", 1.0), mode.get("k", 0),
                           mode.get("p", 1.0))
        for r, u in enumerate((0.3, 0.8)):
            idx = torch.topk(x[r], 64).indices.sort().values.cpu().numpy()
            t, l = SO.sample_row(x[r].cpu().numpy()[idx], np.float32(u), **mode)
            assert int(tok[r]) == int(idx[t]) and abs(float(lp[r]) - l) < 1e-5
    # Everything kept: compare the running sum at the drawn token in 64 bits.
    tok, lp = B.sample(x, torch.tensor([0.3, 0.8], device="cuda"))
    for r, u in enumerate((0.3, 0.8)):
        w = torch.exp(x[r].double() - x[r].max().double())
        run = torch.cumsum(w, 0) / w.sum()
        t, u = int(tok[r]), float(np.float32(u))  # 64 bits on both sides of the comparison
        assert float(run[t]) > u - 1e-9 and (t == 0 or float(run[t - 1]) <= u + 1e-9)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M", [1, 5, 40])
def test_decode_step_end_to_end(B, M, bf16):
    """As used: a ternary layer, the 4-bit output matrix, the token. Its two halves
    give the same token, which the oracle draws from the logits."""
    K, N = 512, 5003
    g = np.random.default_rng([14, M])
    packed, D = B.pack_weights(put((g.standard_normal((K, 256)) * 0.02).astype(np.float32)))
    hidden = B.forward(put(g.standard_normal((M, 256)).astype(np.float32)), packed, D)
    w = B.pack_weights_w4(put((g.standard_normal((N, K)) * 0.2).astype(np.float32)), 64, torch.bfloat16)
    x = hidden.bfloat16() if bf16 else hidden
    u = torch.from_numpy(g.random(M).astype(np.float32)).cuda()
    logits = B.forward_w4(x, w)
    codes, S = B.unpack_w4(w)
    ref = WO.w4_forward(x.float().cpu().numpy(), codes.cpu().numpy(), S.float().cpu().numpy(), 64)
    assert np.abs(logits.cpu().numpy() - ref).max() < 1e-3 * np.abs(ref).max()
    check(B, logits, u.cpu().numpy(), T=0.8, k=40, p=0.9, m=0.01)
    tok, lp = B.sample(logits, u, 0.8, 40, 0.9, 0.01)
    ws = torch.full((B.w4_sample_workspace_size(M, N, K),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        t2, l2 = B.forward_w4_sample(x, w, u, 0.8, 40, 0.9, 0.01, ws=ws)
        assert torch.equal(t2, tok) and torch.equal(l2, lp)
    greedy, _ = B.forward_w4_sample(x, w, u, 0.0)
    assert torch.equal(greedy, logits.argmax(1))


def test_a_batch_of_many_short_rows(B):
    rows, V = 100003, 3
    x, u = body(rows, V, 16)
    tok, _ = B.sample(put(x), torch.from_numpy(u).cuda(), 0.9, 2)
    tok = tok.cpu().numpy()
    for r in list(range(0, rows, 997)) + [rows - 1]:
        assert tok[r] == SO.sample_row(x[r], float(u[r]), float(np.float32(0.9)), 2, 1.0, 0.0)[0]


def test_settings_past_their_types(B):
    """A top_k that no int32 holds filters nothing, and a negative one neither."""
    x, u = body(2, 5000, 17)
    xd, ud = put(x), torch.from_numpy(u).cuda()
    ref = B.sample(xd, ud)[0]
    for k in (1 << 31, (1 << 32) + 1, -(1 << 31), 1 - (1 << 32), 5000, 4999 + (1 << 33)):
        assert torch.equal(B.sample(xd, ud, top_k=k)[0], ref), k
    with pytest.raises(TypeError):
        B.sample(xd, ud, top_k=1.5)
    # A temperature that fp32 rounds to zero or to infinity.
    assert torch.equal(B.sample(xd, ud, 1e-60)[0], xd.argmax(1))
    check(B, xd, u, T=float("inf"))


@pytest.mark.parametrize("M", [1, 24])
def test_decode_loop_in_a_graph(B, M):
    """Steps that feed one another, captured as one graph: launches that begin while
    the one before them runs read what it writes. Equal to steps taken one by one."""
    K, N, steps = 256, 2003, 6
    g = np.random.default_rng([18, M])
    w = B.pack_weights_w4(put((g.standard_normal((N, K)) * 0.3).astype(np.float32)), 32)
    embedding = put(g.standard_normal((N, K)).astype(np.float32))
    start, u = torch.zeros(M, dtype=torch.int64, device="cuda"), torch.zeros(steps, M, device="cuda")
    ws = torch.empty(B.w4_sample_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")

    def loop(sync):
        tok, out = start, []
        for i in range(steps):
            x = embedding[tok]
            tok, lp = B.forward_w4_sample(x, w, u[i], 0.9, 100, 0.95, ws=ws)
            logits = B.forward_w4(x, w, ws=ws)  # into the same workspace
            tok, lp = B.sample(logits, u[i], 0.9, 100, 0.95)
            out += [tok, lp]
            if sync:
                torch.cuda.synchronize()
        return torch.stack([t.double() for t in out])

    loop(True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = loop(False)
    for seed in (1, 2):
        r = np.random.default_rng([19, M, seed])
        start.copy_(torch.from_numpy(r.integers(0, N, M)))
        u.copy_(torch.from_numpy(r.random((steps, M)).astype(np.float32)))
        ref = loop(True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, ref)
        assert torch.equal(loop(False), ref)


def test_refusals(B):
    x, u = put(np.zeros((2, 8), np.float32)), torch.zeros(2, device="cuda")
    with pytest.raises(ValueError):
        B.sample(x, torch.zeros(3, device="cuda"))
    with pytest.raises(TypeError):
        B.sample(x.half(), u)
    with pytest.raises(TypeError):
        B.sample(x, u.double())
    with pytest.raises(ValueError):
        B.sample(x.t(), torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError):
        B.sample(x[0], u)
    with pytest.raises(ValueError):
        B.sample(x[:1].expand(2, 8), u)
    with pytest.raises(TypeError):
        B.sample(x, u, top_k=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        B.sample(x, u, top_p=torch.ones(1, device="cuda"))
    with pytest.raises(RuntimeError):
        B.sample(x[:, :0], u)
    assert B.sample(x[:0], u[:0])[0].shape == (0,)
