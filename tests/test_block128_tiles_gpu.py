"""Every kernel of the block-128 grouped GEMM, each test asserting by
mxg_block128_tile which one its sizes run: the 256-row tile at several stages,
scale chunks, tails of K, partial column tiles, split last rounds and a ring that
runs across tiles; the kernels against each other; weights past 2^32 bytes under
every tile.

Between kernels.  A block's product is the same instruction on the same pieces in
every kernel, so results differ by the fp32 sum over the nb blocks alone.  A sum in
any order is off by at most (nb + 3) 2^-24 of the sum of magnitudes (nb fused
additions, the two scales' product, joining four partial sums adds three more), so
two are apart by (2 nb + 9) 2^-24 of it, and each is rounded to bf16 by half a step,
2^-8 of the value."""
import numpy as np
import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg
import oracle
from common import offsets_gpu, to_gpu
from test_block128_gpu import B, check_gemm, nblk, operands

pytestmark = pytest.mark.gpu


def cut(T, groups, seed):
    """Offsets of `groups` groups of T rows: an empty one, one of one row, the others uneven."""
    if groups == 1:
        return [0, T]
    inner = np.sort(np.random.default_rng(seed).integers(2, T, groups - 3)) if groups > 3 else np.array([], int)
    return [0, 0, 1] + inner.tolist() + [T] if groups > 2 else [0, 1, T]


@pytest.mark.parametrize("T,groups,N,K", [
    (16400, 1, 520, 1184),   # a second chunk of scales, a short last block
    (16400, 4, 513, 2080),   # columns that are no multiple of 8: element stores
    (16390, 5, 520, 288),    # the ring across tiles, three stages each
    (16400, 4, 513, 96),     # one stage, shorter than a block
    (16400, 3, 768, 4096),   # whole column tiles, rows of whole pages
    (33000, 9, 768, 2080),
    (40000, 6, 1000, 1184),  # several rounds
    (30000, 7, 1030, 160),
    (60000, 1, 1, 160), (60000, 2, 130, 416), (60000, 3, 255, 64), (60000, 1, 264, 1056),
    (16640, 1, 512, 128),    # whole tiles alone
])
def test_256_row_tile(T, groups, N, K):
    assert mxg.block128_tile(groups, T, N, K) == 256
    off = cut(T, groups, T + N)
    assert len(off) == groups + 1
    check_gemm(T, 3, N, K, off, [(2 * g + 1) % 3 for g in range(groups)], seed=N + K)


@pytest.mark.parametrize("K", [160, 1056, 2080])
def test_256_row_tile_split_rounds(K):
    """A last round of few tiles, each in two halves by columns, the second half of the last column tile empty
    (N = 600: 88 columns in it)."""
    T, N = 45000, 600  # 43 and 133 row tiles of 3 column tiles: 528, on 256 compute units 16 of them split
    assert mxg.block128_tile(2, T, N, K) == 256
    check_gemm(T, 2, N, K, [0, 11000, T], [1, 0], seed=K)


def tile_of(T, N, K, rows_of_kernel):
    assert mxg.block128_tile(1, T, N, K) == rows_of_kernel
    return T


def spread_of(a, sa, b, sb, rows, c1, c2):
    """Tolerance of the difference of two kernels' results c1 and c2 for `rows`."""
    K, N = a.shape[1], b.shape[0]
    val = torch.from_numpy(oracle.e4m3_value_array(np.arange(256, dtype=np.uint8))).cuda()
    kb, nb = torch.arange(K, device="cuda") // B, torch.arange(N, device="cuda") // B
    mag = (val[a[rows].long()] * sa[rows].double()[:, kb]).abs() @ (val[b.long()] * sb.double()[nb][:, kb]).abs().t()
    return (2 * nblk(K) + 9) * 2.0 ** -24 * mag + (c1.abs() + c2.abs()) * 2.0 ** -8 + 2.0 ** -133


@pytest.mark.parametrize("N,K", [(520, 1184), (513, 160)])
def test_kernels_agree(N, K):
    """One group's rows through every kernel: the tiles add a row's blocks in the same order, bit for bit; the
    kernel of few rows joins four waves' sums."""
    a, sa, b, sb = (to_gpu(v) for v in operands(16400, 2, N, K, 21))
    ids = to_gpu(np.array([1], np.int32))

    def first3(rows_of_kernel, T):
        tile_of(T, N, K, rows_of_kernel)
        return mxg.grouped_matmul_block128(a[:T].contiguous(), sa[:T].contiguous(), b, sb,
                                           offsets_gpu(np.array([0, T], np.uint32)), ids)[:3]

    c256, c128, c32, c16 = first3(256, 16400), first3(128, 5000), first3(32, 40), first3(16, 3)
    assert torch.equal(c256.view(torch.int16), c128.view(torch.int16))
    assert torch.equal(c256.view(torch.int16), c32.view(torch.int16))
    got, ref = c16.double(), c256.double()
    assert bool(((got - ref).abs() <= spread_of(a, sa, b[1], sb[1], slice(0, 3), got, ref)).all())


@pytest.mark.parametrize("K", [4096, 8192])
def test_rows_of_whole_pages(K):
    """K a multiple of 4096: the 128-row tile begins an expert's sum at a block of K that goes by the expert's id,
    so the same rows under the same weights of another expert, or through another kernel, differ by the order of
    the sum and no more; the other kernels' sums do not depend on the id."""
    N, E = 520, 6
    a, sa, b, sb = operands(16400, E, N, K, 5)
    b[5], sb[5] = b[0], sb[0]  # the same weights under two ids
    a, sa, b, sb = (to_gpu(v) for v in (a, sa, b, sb))

    def first3(rows_of_kernel, T, e):
        tile_of(T, N, K, rows_of_kernel)
        return mxg.grouped_matmul_block128(a[:T].contiguous(), sa[:T].contiguous(), b, sb,
                                           offsets_gpu(np.array([0, T], np.uint32)), to_gpu(np.array([e], np.int32)))[:3]

    sizes = {256: 16400, 128: 5000, 32: 40, 16: 3}
    ref = first3(256, 16400, 0)
    for rows_of_kernel, T in sizes.items():
        c0, c5 = first3(rows_of_kernel, T, 0), first3(rows_of_kernel, T, 5)
        if rows_of_kernel != 128:
            assert torch.equal(c0.view(torch.int16), c5.view(torch.int16))
        assert torch.equal(c5.view(torch.int16), first3(rows_of_kernel, T, 5).view(torch.int16))  # the same call twice
        for c in (c0.double(), c5.double()):
            assert bool(((c - ref.double()).abs() <= spread_of(a, sa, b[0], sb[0], slice(0, 3), c, ref.double())).all())


@pytest.mark.parametrize("T,G,N,K", [(1000, 256, 264, 512), (40, 4, 130, 1184), (300, 100, 33, 96)])
def test_hint_changes_the_kernel(T, G, N, K):
    assert mxg.block128_tile(G, T, N, K, 0) == 16 and mxg.block128_tile(G, T, N, K, 1 << 62) != 16
    sizes = np.random.default_rng(T).multinomial(T, np.full(G, 1 / G))
    off = np.concatenate([[0], np.cumsum(sizes)])
    for hint in (0, int(sizes.max()), 1 << 62):
        check_gemm(T, 3, N, K, off, [g % 3 for g in range(G)], seed=K, hint=hint)


@pytest.mark.parametrize("T,rows_of_kernel", [(3, 16), (200, 32), (1000, 128), (3000, 256)])
def test_weights_past_32_bits(T, rows_of_kernel):
    """The first and the last of weights of more than 2^32 bytes, under every kernel."""
    E, N, K = 300, 4096, 4096  # 5 GB
    assert mxg.block128_tile(2, T, N, K) == rows_of_kernel
    b = torch.full((E, N, K), 0x38, dtype=torch.uint8, device="cuda")  # ones
    b[E - 1] = 0x40                                                     # twos
    bs = torch.ones((E, 32, 32), device="cuda")
    bs[E - 1] = 4.0
    a = torch.full((T, K), 0x38, dtype=torch.uint8, device="cuda")
    half = T // 2
    c = mxg.grouped_matmul_block128(a, torch.ones((T, 32), device="cuda"), b, bs,
                                    offsets_gpu(np.array([0, half, T], np.uint32)),
                                    to_gpu(np.array([0, E - 1], np.int32)))
    assert torch.all(c[:half] == K) and torch.all(c[half:] == 8 * K)
