"""CPU tests of the binding's checks of 4-bit weights: sizes that a C type would
take modulo 2^32 or 2^64 (the kernels would then index with another layout than
the tensors have) are refused before any launch."""
import pytest

from bit_ternary_b200 import build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def B():
    from bit_ternary_b200 import bitlinear

    build.build_library()
    return bitlinear


@pytest.mark.parametrize("group", [0, -32, 31, 48, 256, (1 << 32) + 32, (1 << 32) + 128, 64 - (1 << 32), 1 << 64])
def test_groups_other_than_the_three_are_refused(B, group):
    with pytest.raises(ValueError):
        B._w4_packed_bytes(4, 256, group, torch.float32)


@pytest.mark.parametrize("N,K", [(4, 0), (4, -16), (4, 24), (4, 131088), (4, (1 << 64) + 256), (4, 256 - (1 << 64)),
                                 (-1, 256), (1 << 31, 256), ((1 << 64) + 4, 256)])
def test_sizes_out_of_range_are_refused(B, N, K):
    with pytest.raises(ValueError):
        B._w4_packed_bytes(N, K, 32, torch.float32)


@pytest.mark.parametrize("dtype,scale_bytes", [(torch.float32, 4), (torch.bfloat16, 2)])
def test_packed_bytes(B, dtype, scale_bytes):
    for N, K, group in ((1, 16, 32), (16, 128, 32), (17, 144, 64), (33, 131072, 128)):
        tiles, blocks = -(-N // 16), -(-K // 128)
        assert B._w4_packed_bytes(N, K, group, dtype) == tiles * blocks * (1024 + 16 * (128 // group) * scale_bytes)
    assert B._w4_packed_bytes(0, 128, 32, dtype) == 0
