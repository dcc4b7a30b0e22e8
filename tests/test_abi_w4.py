"""CPU-side checks of the C entry points of 4-bit weights and the sampler: every
refusal that their header names comes before any CUDA work (no GPU needed)."""
import ctypes

import pytest

from bit_ternary_b200 import _lib, build

NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 4
FAKE = 0x10000  # never dereferenced: validation fails first
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    build.build_library()
    return _lib.lib()


@pytest.mark.parametrize("bad", [dict(K=0), dict(K=-16), dict(K=24), dict(K=131088), dict(group=0), dict(group=48),
                                 dict(group=256), dict(group=-32), dict(scale=2), dict(scale=-1), dict(N=-1),
                                 dict(N=1 << 31)], ids=str)
def test_sizes_are_refused(L, bad):
    a = dict(N=8, K=64, group=32, scale=0)
    a.update(bad)
    N, K, g, s = a["N"], a["K"], a["group"], a["scale"]
    assert L.bitlinear_w4_packed_bytes(N, K, g, s) == 0
    for sfx in ("", "_bf16"):
        assert getattr(L, "bitlinear_pack_weights_w4" + sfx)(FAKE, N, K, g, s, FAKE, FAKE, BIG, None) == SHAPE
        assert getattr(L, "bitlinear_forward_w4" + sfx)(FAKE, 1, N, K, g, s, FAKE, FAKE, FAKE, BIG, None) == SHAPE
        how = _lib.Sampling()
        assert getattr(L, "bitlinear_forward_w4_sample" + sfx)(FAKE, 1, N, K, g, s, FAKE, how, FAKE, FAKE, FAKE, FAKE,
                                                               BIG, None) == SHAPE
    assert L.bitlinear_w4_import(FAKE, FAKE, N, K, g, s, FAKE, None) == SHAPE
    assert L.bitlinear_w4_export(FAKE, N, K, g, s, FAKE, FAKE, None) == SHAPE


def test_sizes_of_buffers(L):
    assert [L.bitlinear_w4_groups(272, g) for g in (32, 64, 128, 16)] == [9, 5, 3, 0]
    assert L.bitlinear_w4_packed_bytes(17, 272, 64, 1) == 2 * 3 * (1024 + 16 * 2 * 2)
    assert L.bitlinear_w4_packed_bytes(0, 272, 64, 1) == 0
    assert L.bitlinear_w4_workspace_size(-1, 8, 64) == L.bitlinear_w4_workspace_size(1, 8, 24) == 0
    for M, N, K in ((1, 1, 16), (33, 1003, 272), (4096, 13824, 2560)):
        ws = L.bitlinear_w4_workspace_size(M, N, K)
        assert ws % 256 == 0 and ws >= 256 + 6 * M * K
        assert L.bitlinear_w4_sample_workspace_size(M, N, K) >= ws + 4 * M * N


@pytest.mark.parametrize("sfx", ["", "_bf16"])
def test_forward(L, sfx):
    f = getattr(L, "bitlinear_forward_w4" + sfx)
    ws = L.bitlinear_w4_workspace_size(3, 8, 64)
    assert f(None, 0, 8, 64, 32, 0, None, None, None, 0, None) == 0
    assert f(None, 3, 0, 64, 32, 0, None, None, None, 0, None) == 0
    assert f(FAKE, -1, 8, 64, 32, 0, FAKE, FAKE, FAKE, BIG, None) == SHAPE
    assert f(FAKE, 1 << 31, 8, 64, 32, 0, FAKE, FAKE, FAKE, BIG, None) == SHAPE
    for i in range(4):
        p = [FAKE] * 4
        p[i] = None
        assert f(p[0], 3, 8, 64, 32, 0, p[1], p[2], p[3], BIG, None) == NULL
        p[i] = FAKE + 8
        assert f(p[0], 3, 8, 64, 32, 0, p[1], p[2], p[3], BIG, None) == ALIGN
    assert f(FAKE, 3, 8, 64, 32, 0, FAKE, FAKE, FAKE + 16, BIG, None) == ALIGN  # ws: 256 bytes
    assert f(FAKE, 3, 8, 64, 32, 0, FAKE, FAKE, FAKE, ws - 1, None) == WORKSPACE


@pytest.mark.parametrize("sfx", ["", "_bf16"])
def test_pack(L, sfx):
    f = getattr(L, "bitlinear_pack_weights_w4" + sfx)
    assert f(FAKE, 0, 64, 32, 0, FAKE, FAKE, BIG, None) == SHAPE
    for i in range(3):
        p = [FAKE] * 3
        p[i] = None
        assert f(p[0], 8, 64, 32, 0, p[1], p[2], BIG, None) == NULL
        p[i] = FAKE + 8
        assert f(p[0], 8, 64, 32, 0, p[1], p[2], BIG, None) == ALIGN
    assert f(FAKE, 8, 64, 32, 0, FAKE, FAKE, L.bitlinear_pack_workspace_size(8, 64) - 1, None) == WORKSPACE


def test_import_and_export(L):
    for f, at in ((L.bitlinear_w4_import, (0, 1, 6)), (L.bitlinear_w4_export, (0, 5, 6))):
        sizes = (8, 64, 32, 0)

        def call(p):
            a = [None] * 7
            for i, v in zip(at, p):
                a[i] = v
            rest = iter(sizes)
            return f(*[v if i in at else next(rest) for i, v in enumerate(a)], None)

        for i in range(3):
            p = [FAKE] * 3
            p[i] = None
            assert call(p) == NULL
            p[i] = FAKE + 4
            assert call(p) == ALIGN
        sizes = (0, 64, 32, 0)
        assert call([None] * 3) == 0


SETTINGS = ("temperature", "top_k", "top_p", "min_p")


@pytest.mark.parametrize("sfx", ["", "_bf16"])
def test_sample(L, sfx):
    f = getattr(L, "bitlinear_sample" + sfx)
    how = _lib.Sampling()
    assert f(None, 0, 8, 8, None, None, None, None, None) == 0
    for B, V, ld in ((-1, 8, 8), (1 << 31, 8, 8), (2, 0, 8), (2, -5, 8), (2, (1 << 22) + 1, 1 << 23), (2, 8, 7)):
        assert f(FAKE, B, V, ld, how, FAKE, FAKE, FAKE, None) == SHAPE, (B, V, ld)
    assert f(None, 2, 8, 8, how, FAKE, FAKE, FAKE, None) == NULL
    assert f(FAKE, 2, 8, 8, None, FAKE, FAKE, FAKE, None) == NULL
    assert f(FAKE, 2, 8, 8, how, None, FAKE, FAKE, None) == NULL
    assert f(FAKE, 2, 8, 8, how, FAKE, None, FAKE, None) == NULL
    assert f(FAKE + 1, 2, 8, 8, how, FAKE, FAKE, FAKE, None) == ALIGN
    assert f(FAKE, 2, 8, 8, how, FAKE + 2, FAKE, FAKE, None) == ALIGN
    assert f(FAKE, 2, 8, 8, how, FAKE, FAKE + 4, FAKE, None) == ALIGN
    assert f(FAKE, 2, 8, 8, how, FAKE, FAKE, FAKE + 1, None) == ALIGN
    for name in SETTINGS:
        how = _lib.Sampling()
        setattr(how, name, FAKE + 2)
        assert f(FAKE, 2, 8, 8, how, FAKE, FAKE, FAKE, None) == ALIGN


@pytest.mark.parametrize("sfx", ["", "_bf16"])
def test_forward_and_sample(L, sfx):
    f = getattr(L, "bitlinear_forward_w4_sample" + sfx)
    how = _lib.Sampling()
    ws = L.bitlinear_w4_sample_workspace_size(3, 8, 64)

    def call(x=FAKE, M=3, N=8, packed=FAKE, how=how, u=FAKE, tokens=FAKE, logprobs=FAKE, w=FAKE, ws_bytes=ws):
        return f(x, M, N, 64, 32, 0, packed, how, u, tokens, logprobs, w, ws_bytes, None)

    assert call(M=0) == 0
    for bad in (dict(M=-1), dict(N=0), dict(N=(1 << 22) + 1)):
        assert call(**bad) == SHAPE
    for bad in (dict(x=None), dict(packed=None), dict(how=None), dict(u=None), dict(tokens=None), dict(w=None)):
        assert call(**bad) == NULL, bad
    for bad in (dict(x=FAKE + 8), dict(packed=FAKE + 8), dict(u=FAKE + 2), dict(tokens=FAKE + 4),
                dict(logprobs=FAKE + 2), dict(w=FAKE + 16)):
        assert call(**bad) == ALIGN, bad
    assert call(ws_bytes=ws - 1) == WORKSPACE
    assert call(ws_bytes=L.bitlinear_w4_workspace_size(3, 8, 64)) == WORKSPACE  # the forward's alone has no room for the logits


def test_the_mirror_of_the_settings_has_the_headers_layout():
    offsets = [getattr(_lib.Sampling, n).offset for n, _ in _lib.Sampling._fields_]
    assert offsets == [0, 8, 16, 24, 32, 36, 40, 44] and ctypes.sizeof(_lib.Sampling) == 48
