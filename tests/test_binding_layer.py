"""What only the binding can see of the operators between 4-bit layers (CPU
only: shapes and types, no call)."""
import pytest
import torch

ns = pytest.importorskip("newton_schulz_amd")


def nv(N, K):
    return torch.zeros(N, K // 2, dtype=torch.uint8), torch.zeros(N, K // 16, dtype=torch.uint8)


def test_nvfp4_weights_of_the_other_orientation():
    """[K][N / 2] in place of [N][K / 2] has the same number of elements."""
    for N, K in ((32, 64), (33, 48), (1, 16)):
        codes, scales = nv(N, K)
        ns._need_nv_rows(codes, scales, N, K)
        ns._need_nv_rows(codes.view(-1), scales.view(-1), N, K)
    codes, scales = nv(64, 32)
    for c, s in ((codes, scales), (nv(32, 64)[0], scales), (codes, nv(32, 64)[1])):
        with pytest.raises(ValueError):
            ns._need_nv_rows(c, s, 32, 64)


def test_nvfp4_weights_of_another_size():
    codes, scales = nv(32, 64)
    for N, K in ((31, 64), (33, 64), (32, 48), (32, 80), (16, 64)):
        with pytest.raises(ValueError):
            ns._need_nv_rows(codes, scales, N, K)
        with pytest.raises(ValueError):
            ns._need_nv_rows(codes.view(-1), scales.view(-1), N, K)
    with pytest.raises(TypeError):
        ns._need_nv_rows(codes.to(torch.int32), scales, 32, 64)
    with pytest.raises(TypeError):
        ns._need_nv_rows(codes, scales.view(torch.int8), 32, 64)
