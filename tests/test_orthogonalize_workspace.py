"""The workspace of moe_orthogonalize against what the header states (no GPU)."""

import pytest

from moe_layer_router_amd import lib


def _up(v, to):
    return (v + to - 1) // to * to


@pytest.mark.parametrize("batch", [1, 3, 100])
@pytest.mark.parametrize("M,N", [(65, 65), (80, 80), (100, 130), (130, 100), (256, 7168), (7168, 2048), (2048, 7168),
                                 (300, 20000), (16384, 32768)])
def test_wide(batch, M, N):
    m, n = sorted((_up(M, 64), _up(N, 64)))
    one = 6 * m * n + 4 * m * m + 512
    size = lib.moe_orthogonalize_workspace_size(batch, M, N)
    held = min(batch, max(1, (8 << 30) // one))
    assert size <= held * one + (128 << 20) + 8 * 256
    # as many as 8 GiB hold, but for the partial sums and the norms' 512 bytes each
    held = min(batch, max(1, ((8 << 30) - (128 << 20)) // one))
    assert size >= held * one
    assert size <= max(one, 8 << 30) + (128 << 20) + 8 * 256


@pytest.mark.parametrize("batch", [1, 7, 65535])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 300), (17, 33), (40, 64), (64, 64), (64, 7168), (20000, 16), (33, 32768)])
def test_narrow(batch, M, N):
    m, n = sorted((M, N))
    s = 16 if m <= 16 else 32 if m <= 32 else 64
    p = min(16, _up(n, 64) // 64)
    size = lib.moe_orthogonalize_workspace_size(batch, M, N)
    assert 8 * (p + 1) * s * s * batch <= size <= 8 * (p + 1) * s * s * batch + 2 * 256


@pytest.mark.parametrize("M,N", [(512, 1000), (2048, 7168), (65, 65)])
def test_a_large_batch_is_bounded(M, N):
    a, b = (lib.moe_orthogonalize_workspace_size(k, M, N) for k in (60000, 65535))
    assert a == b <= (8 << 30) + (32 << 20)            # (norms' 512 bytes for each of up to 60000 matrices)
