"""Which kernel the block-128 grouped GEMM runs, on the CPU (256 compute units are
assumed there, as an MI355X has): one size for each kernel, what the hint changes,
and the sizes that run nothing."""
import pytest

import fp4_grouped_gemm_quantize_amd as mxg


@pytest.mark.parametrize("G,T,N,K,hint,rows", [
    (128, 65536, 1536, 4096, 0, 256),
    (1, 16400, 520, 1184, 0, 256),
    (1, 16400, 1000, 1184, 0, 256),
    (5, 16400, 1000, 1184, 0, 128),   # 132 either way: the smaller tile
    (64, 1024, 2048, 7168, 0, 128),
    (24, 5003, 1000, 2080, 0, 128),
    (2, 200, 4096, 4096, 0, 32),
    (1, 3, 520, 1184, 0, 16),
    (256, 1000, 264, 512, 0, 16),
    (256, 1000, 264, 512, 128, 16),
    (256, 1000, 264, 512, 129, 32),
    (256, 1000, 264, 512, 1 << 62, 32),
    (256, 1000, 264, 512, -5, 16),
])
def test_choice(G, T, N, K, hint, rows):
    assert mxg.block128_tile(G, T, N, K, hint) == rows


@pytest.mark.parametrize("G,T,N,K", [(0, 1, 8, 32), (1, 0, 8, 32), (1, 1, 0, 32), (1, 1, 8, 0), (1, 1, 8, 48),
                                     (1025, 1, 8, 32), (1, 1, 8, mxg.MAX_K + 32), (1, 1, 2 ** 30, 32),
                                     (1, 2 ** 31, 8, 32), (-1, 4, 8, 32)])
def test_nothing_to_run(G, T, N, K):
    assert mxg.block128_tile(G, T, N, K) == 0
