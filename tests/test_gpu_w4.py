"""GPU tests of the 4-bit group-scale linear against its 64-bit oracle.

Tolerance of y: codes and their products with x are exact, so what rounds is
the 32-bit sum. A group's products pass through at most `group` additions and
the groups' terms through one product and one addition each; three pieces of an
fp32 x add two more additions, a split of K over warps or tiles a few (8 cover
them). Each is off by at most one step of 2^-23 relative to the partial sums
(half a step where it rounds to nearest, one where the tensor cores cut off),
and no partial sum exceeds sum |S c x|: |y - exact| <= (group + 2 G + 10) *
2^-23 * sum |S c x|.
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


def make(N, K, group, bf16_scales, seed):
    rng = np.random.default_rng([seed, N, K, group])
    codes = rng.integers(-8, 8, (N, K)).astype(np.int8)
    S = (0.02 * (0.5 + rng.random((N, -(-K // group))))).astype(np.float32)
    if bf16_scales:
        S = WO.bf16_rn(S)
    return codes, S


def put(B, codes, S, group, bf16_scales):
    St = torch.from_numpy(S).cuda()
    return B.import_w4(torch.from_numpy(WO.w4_nibbles(codes)).cuda(), St.bfloat16() if bf16_scales else St, group)


def make_x(M, K, bf16, seed):
    rng = np.random.default_rng([seed, M, K])
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.random(K) < 0.02] *= 20
    return WO.bf16_rn(x) if bf16 else x


def put_x(x, bf16):
    t = torch.from_numpy(x).cuda()
    return t.bfloat16() if bf16 else t


def check(y, x, codes, S, group, cols=None):
    ref = WO.w4_forward(x, codes, S, group)
    K, G = codes.shape[1], S.shape[1]
    tol = (min(group, K) + 2 * G + 10) * 2.0 ** -23 * WO.w4_sum_abs(x, codes, S, group)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= tol).all(), f"worst {np.nanmax(err / np.maximum(tol, 1e-300))} of the bound"


SHAPES = [(1, 16), (15, 48), (17, 128), (33, 144), (128, 256), (130, 272), (257, 1152), (100, 2560), (64, 6912)]


@pytest.mark.parametrize("bf16_scales", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", SHAPES)
def test_layout_round_trip(B, N, K, group, bf16_scales):
    codes, S = make(N, K, group, bf16_scales, 1)
    w = put(B, codes, S, group, bf16_scales)
    c, s = B.unpack_w4(w)
    assert np.array_equal(c.cpu().numpy(), codes)
    assert np.array_equal(s.float().cpu().numpy(), S)


@pytest.mark.parametrize("bf16_w", [False, True])
@pytest.mark.parametrize("bf16_scales", [False, True])
@pytest.mark.parametrize("N,K,group", [(1, 16, 32), (15, 48, 32), (17, 144, 64), (33, 272, 128), (100, 1152, 32)])
def test_pack_is_the_oracles(B, N, K, group, bf16_scales, bf16_w):
    W = (np.random.default_rng([N, K]).standard_normal((N, K)) * 0.02).astype(np.float32)
    if bf16_w:
        W = WO.bf16_rn(W)
    W[0, : min(16, K)] = 0
    if N > 2:
        W[2] = 0
        W[3, :16] = 1e-44  # a / 7 rounds to the smallest subnormals or to zero
    c_ref, S_ref = WO.w4_quantise(W, group, bf16_scales)
    c, s = B.unpack_w4(B.pack_weights_w4(put_x(W, bf16_w), group, torch.bfloat16 if bf16_scales else torch.float32))
    assert np.array_equal(s.float().cpu().numpy(), S_ref)
    assert np.array_equal(c.cpu().numpy(), c_ref)


@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_pack_reports_nonfinite(B, bad):
    from bit_ternary_b200 import _lib

    W = torch.randn(20, 64, device="cuda")
    W[7, 33] = bad
    with pytest.raises(_lib.BitLinearError) as e:
        B.pack_weights_w4(W, 32)
    assert e.value.status == 5


MS = [1, 2, 3, 5, 6, 8, 9, 16, 17, 31, 48, 64, 65, 127, 128, 129, 300]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M", MS)
@pytest.mark.parametrize("N,K,group,bf16_scales", [(1, 16, 32, False), (17, 144, 64, True), (130, 272, 32, True),
                                                    (257, 1152, 128, False), (100, 2560, 128, True)])
def test_forward(B, M, N, K, group, bf16_scales, bf16):
    codes, S = make(N, K, group, bf16_scales, 2)
    x = make_x(M, K, bf16, 3)
    y = B.forward_w4(put_x(x, bf16), put(B, codes, S, group, bf16_scales))
    check(y, x, codes, S, group)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("group,bf16_scales", [(32, False), (32, True), (64, False), (64, True), (128, False),
                                               (128, True)])
@pytest.mark.parametrize("M", [1, 4, 12, 40, 200])
def test_forward_every_format(B, M, group, bf16_scales, bf16):
    N, K = 1000, 1040
    codes, S = make(N, K, group, bf16_scales, 4)
    x = make_x(M, K, bf16, 5)
    check(B.forward_w4(put_x(x, bf16), put(B, codes, S, group, bf16_scales)), x, codes, S, group)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 33, 131072), (3, 20, 40000), (16, 40, 16400), (40, 140, 20000), (1, 20011, 256),
                                   (2, 3001, 512), (150, 5003, 144), (7, 9000, 1040)])
def test_forward_long_rows_and_many(B, M, N, K, bf16):
    codes, S = make(N, K, 64, False, 6)
    x = make_x(M, K, bf16, 7)
    check(B.forward_w4(put_x(x, bf16), put(B, codes, S, 64, False)), x, codes, S, 64)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M", [1, 9, 70])
def test_forward_writes_only_y(B, M, bf16):
    N, K = 129, 272
    codes, S = make(N, K, 32, False, 8)
    x = make_x(M, K, bf16, 9)
    big = torch.full((M * N + 64,), 7.0, device="cuda")
    y = big[32:32 + M * N].view(M, N)
    B.forward_w4(put_x(x, bf16), put(B, codes, S, 32, False), out=y)
    check(y, x, codes, S, 32)
    assert (big[:32] == 7).all() and (big[32 + M * N:] == 7).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M", [1, 4, 16, 70])
def test_nonfinite_tokens_stay_in_their_rows(B, M, bf16):
    N, K = 150, 272
    codes, S = make(N, K, 32, False, 10)
    codes[codes == 0] = 1  # inf * 0 is NaN in the formula too
    codes[5, 17] = 0
    x = make_x(M, K, bf16, 11)
    x[0, 17] = np.inf
    if M > 2:
        x[2, 40] = np.nan
    y = B.forward_w4(put_x(x, bf16), put(B, codes, S, 32, False)).cpu().numpy()
    assert np.isnan(y[0, 5])
    rest = np.delete(np.arange(N), 5)
    assert np.array_equal(np.sign(y[0, rest]), np.sign(codes[rest, 17])) and np.isinf(y[0, rest]).all()
    if M > 2:
        assert np.isnan(y[2]).all()
    ok = [m for m in range(M) if m not in (0, 2)]
    if ok:
        check(torch.from_numpy(y[ok]), x[ok], codes, S, 32)


@pytest.mark.parametrize("M", [1, 5, 16, 40, 130])
def test_fp32_x_over_its_range(B, M):
    """Every bit of an fp32 x takes part: tokens of one large and one tiny scale, the
    largest finite value, subnormals, and x = 1 + 2^-23 against codes that cancel the 1."""
    N, K = 40, 128
    codes, S = make(N, K, 128, False, 12)
    S[:] = 1.0
    x = make_x(M, K, False, 13)
    x[0] = 0
    x[0, 0], x[0, 1] = 1 + 2.0 ** -23, 1.0
    # 4 (1 + 2^-23) has 24 significant bits, so every 32-bit sum holds it (3 (1 + 2^-23) has 25).
    codes[:, 0], codes[:, 1] = 4, -4
    if M > 4:
        x[1] *= np.float32(1e-30)
        x[2] *= np.float32(1e30)
        x[3] = 0
        x[3, 0] = np.finfo(np.float32).max / 8
        x[4] = 0
        x[4, 0] = np.float32(2.0 ** -120)
    y = B.forward_w4(torch.from_numpy(x).cuda(), put(B, codes, S, 128, False))
    check(y, x, codes, S, 128)
    assert (y[0].cpu().numpy() == 4 * 2.0 ** -23).all()


@pytest.mark.parametrize("M", [1, 8, 33, 200])
def test_same_inputs_same_bits(B, M):
    N, K = 1030, 2576
    codes, S = make(N, K, 64, True, 14)
    w = put(B, codes, S, 64, True)
    x = put_x(make_x(M, K, False, 15), False)
    y = B.forward_w4(x, w)
    for _ in range(5):
        assert torch.equal(B.forward_w4(x, w), y)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M", [1, 20, 140])
def test_streams_graphs_and_reused_workspace(B, M, bf16):
    N, K = 700, 1152
    codes, S = make(N, K, 32, False, 16)
    w = put(B, codes, S, 32, False)
    xs = [make_x(M, K, bf16, 20 + i) for i in range(3)]
    ws = torch.full((B.w4_workspace_size(M, N, K),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ys = [B.forward_w4(put_x(x, bf16), w, ws=ws) for x in xs]  # stream order guards ws
    xin = put_x(xs[0], bf16)
    out = torch.zeros(M, N, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.forward_w4(xin, w, out=out, ws=ws)
    for i, x in enumerate(xs):
        check(ys[i], x, codes, S, 32)
        xin.copy_(put_x(x, bf16))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ys[i])
    assert B.workspace_error(ws) == 0


def test_offsets_past_32_bits(B):
    """A packed weight of more than 4 GiB: its last rows."""
    N, K, group = 262153, 32768, 128
    M = 3
    gen = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    for n in range(0, N, 16384):
        codes[n:n + 16384] = torch.randint(0, 256, codes[n:n + 16384].shape, dtype=torch.uint8, device="cuda",
                                           generator=gen)
    S = 0.01 + 0.01 * torch.rand((N, K // group), device="cuda", generator=gen)
    w = B.import_w4(codes, S, group)
    assert w.data.numel() > 1 << 32
    for M in (2, 40):
        x = make_x(M, K, True, 21)
        y = B.forward_w4(put_x(x, True), w)
        for rows in (slice(0, 5), slice(131070, 131080), slice(N - 20, N)):
            b = codes[rows].cpu().numpy()
            c = np.empty((b.shape[0], K), np.int8)
            c[:, 0::2] = (b & 15).astype(np.int8) - 8
            c[:, 1::2] = (b >> 4).astype(np.int8) - 8
            check(y[:, rows], x, c, S[rows].cpu().numpy(), group)


@pytest.mark.parametrize("M", [2, 90, 300])
def test_two_calls_at_once(B, M):
    """Calls of one weight on two streams, a workspace each."""
    N, K = 900, 640
    codes, S = make(N, K, 64, True, 31)
    w = put(B, codes, S, 64, True)
    xs = [make_x(M, K, False, 32 + i) for i in range(2)]
    xd = [put_x(x, False) for x in xs]
    ws = [torch.empty(B.w4_workspace_size(M, N, K), dtype=torch.uint8, device="cuda") for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    ys = [[], []]
    torch.cuda.synchronize()
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                ys[i].append(B.forward_w4(xd[i], w, ws=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        check(ys[i][0], xs[i], codes, S, 64)
        assert all(torch.equal(y, ys[i][0]) for y in ys[i])


def test_packed_bytes_stay_with_their_weight(B):
    codes, S = make(32, 64, 32, False, 33)
    w = put(B, codes, S, 32, False)
    with pytest.raises(AttributeError):
        w.data = torch.zeros(16, dtype=torch.uint8, device="cuda")
    v = B.W4Weights(w.data.clone(), 32, 64, 32, torch.float32)
    x = put_x(make_x(3, 64, False, 34), False)
    assert torch.equal(B.forward_w4(x, v), B.forward_w4(x, w))


def test_refusals(B):
    codes, S = make(32, 64, 32, False, 30)
    w = put(B, codes, S, 32, False)
    x = torch.zeros(2, 64, device="cuda")
    with pytest.raises(ValueError):
        B.forward_w4(torch.zeros(2, 48, device="cuda"), w)
    with pytest.raises(TypeError):
        B.forward_w4(x.half(), w)
    with pytest.raises(ValueError):
        B.forward_w4(torch.zeros(64, 2, device="cuda").t(), w)
    with pytest.raises(ValueError):
        B.forward_w4(x, w, out=torch.zeros(2, 31, device="cuda"))
    with pytest.raises(ValueError):
        B.forward_w4(x.cpu(), w)
    with pytest.raises(ValueError):
        B.import_w4(torch.zeros(4, 32, dtype=torch.uint8, device="cuda"), torch.zeros(4, 3, device="cuda"), 32)
    with pytest.raises(ValueError):
        B.import_w4(torch.zeros(4, 20, dtype=torch.uint8, device="cuda"), torch.zeros(4, 2, device="cuda"), 32)
    with pytest.raises(TypeError):
        B.import_w4(torch.zeros(4, 32, dtype=torch.uint8, device="cuda"), torch.zeros(4, 2, device="cuda").half(), 32)
    with pytest.raises(ValueError):
        B.pack_weights_w4(x, 48)
    with pytest.raises(RuntimeError):
        B.forward_w4(x, w, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        B.W4Weights(w.data[:-16], 32, 64, 32, torch.float32)
    assert B.forward_w4(torch.zeros(0, 64, device="cuda"), w).shape == (0, 32)
