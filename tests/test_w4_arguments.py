"""The binding's checks of 4-bit weights: sizes that a C type would
take modulo 2^32 or 2^64 (the kernels would then index with another layout than
the tensors have) and workspaces with fewer bytes than elements are refused
before any launch."""
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


def test_a_workspace_is_as_large_as_it_says(B):
    """One byte expanded to a size, or every second byte, is not that many bytes."""
    cpu = torch.device("cpu")
    assert B._workspace(torch.zeros(512, dtype=torch.uint8), cpu) == 512
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(512), torch.zeros(1024, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            B._workspace(ws, cpu)
    with pytest.raises(ValueError):
        B._workspace(torch.zeros(512, dtype=torch.uint8), torch.device("cuda:0"))


@pytest.mark.gpu
def test_calls_refuse_a_workspace_that_is_smaller_than_it_says(B):
    W, x, u = torch.randn(32, 64, device="cuda"), torch.randn(2, 64, device="cuda"), torch.rand(2, device="cuda")
    w = B.pack_weights_w4(W, 32)
    ws = torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 20)
    for call in (lambda: B.pack_weights_w4(W, 32, ws=ws), lambda: B.forward_w4(x, w, ws=ws),
                 lambda: B.forward_w4_sample(x, w, u, ws=ws)):
        with pytest.raises(ValueError):
            call()


def test_a_weight_keeps_the_sizes_it_was_laid_out_for(B):
    """Sizes that do not belong to the packed bytes would be read past their end."""
    w = B.W4Weights.__new__(B.W4Weights)
    names = ("out_features", "in_features", "group", "scale_dtype", "scale_type")
    for name in names:
        setattr(w, name, 1)
    for name in names:
        with pytest.raises(AttributeError):
            setattr(w, name, 2)
        assert getattr(w, name) == 1
    with pytest.raises(AttributeError):
        w.data = torch.zeros(16, dtype=torch.uint8)
