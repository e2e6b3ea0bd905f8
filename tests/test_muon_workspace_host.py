"""Muon's workspace against what the header says of it; no GPU."""

import pytest

pytest.importorskip("torch")

import delayed_scaling_gemm_amd as dsg  # noqa: E402


def padded(v):
    """The most that a side may be rounded up to: a tile of 64, 128 or 256, not twice itself."""
    return max(64, min((v + 255) // 256 * 256, 2 * v))


@pytest.mark.parametrize("R,C", [(1, 1), (8, 128256), (1, 1 << 19), (64, 32513), (64, 16257), (33, 20000), (65, 128256),
                                 (130, 128256), (333, 130), (512, 512), (4096, 14336), (4096, 4096),
                                 (1000, 1600), (128256, 4096), (1 << 17, 1 << 17), (1 << 15, 1 << 19)])
def test_workspace_is_what_the_header_says(R, C):
    m, n = min(R, C), max(R, C)
    m_, n_ = padded(m), padded(n)
    most = 12 * m_ * n_ + 20 * m_ * m_ + (4 << 20) + (20 << 10)
    least = 12 * m * n + 8 * m * m
    for shape in ((R, C), (C, R)):
        assert least <= dsg.fp8ds_muon_workspace(*shape) <= most
    if n < 1.2 * m and n >= 2048:  # no groups of steps
        assert dsg.fp8ds_muon_workspace(R, C) <= 12 * m_ * n_ + 8 * m_ * m_ + (4 << 20) + (20 << 10)


def test_long_thin_matrices_are_not_padded_to_large_tiles():
    # 64 rows at least: 12 bytes of each of 64 x 128256, 20 of 64 x 64, partial sums
    assert dsg.fp8ds_muon_workspace(8, 128256) <= 12 * 64 * 128256 + (5 << 20)
    assert dsg.fp8ds_muon_workspace(64, 1 << 19) <= 12 * 64 * (1 << 19) + (5 << 20)
