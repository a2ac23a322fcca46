"""Every kernel of the BF16 products and their gradients, each test asserting by mxg_bf16_tile which one its
sizes run: several stages and one, tails of the depth, partial rows and columns, columns that are no
vectors, several rounds of tiles and split last rounds, expert ranges, weights, rows and gradients past
2^32 bytes.  Bounds as in test_matmul_bf16_gpu.py."""
import math

import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg
from test_matmul_bf16_gpu import BF, F32, Routing, forward_case, rand, rows_case, weights_case

pytestmark = pytest.mark.gpu

FWD, BWD, WTS = mxg.BF16_FORWARD, mxg.BF16_BACKWARD, mxg.BF16_BACKWARD_WEIGHTS


def routing(T, E):
    """An expert without rows, one with a single one, the others uneven; a row behind the last group."""
    if E == 1:
        return Routing(T, 1)
    cuts = [0, 0, 1] + [1 + (T - 2) * i * i // ((E - 2) * (E - 2)) for i in range(1, E - 1)]
    return Routing(T, E, cuts, list(range(E)))


@pytest.mark.parametrize("T,E,N,K,tile", [
    (16640, 1, 520, 320, (256, 256)),    # three column tiles, the last of 8 columns; five stages
    (16400, 1, 517, 1096, (256, 256)),   # columns that are no vectors, a tail of 8
    (33000, 9, 776, 72, (256, 256)),     # two stages, the second of 8; several rounds
    (40000, 4, 1032, 64, (256, 256)),    # one stage a tile
    (45000, 3, 600, 136, (256, 256)),    # a split last round
    (4000, 5, 1000, 2080, (256, 128)), (2500, 1, 2049, 1000, (256, 128)), (33000, 24, 264, 72, (256, 128)),
    (2048, 6, 1544, 520, (128, 128)), (2048, 1, 2048, 200, (128, 128)), (16640, 80, 71, 1032, (128, 128)),
    (16640, 6, 64, 8, (128, 128)),
    (2048, 24, 520, 264, (64, 128)), (1500, 6, 775, 264, (64, 128)), (700, 6, 1544, 4104, (64, 128)),
    (900, 80, 262, 1000, (32, 128)), (700, 80, 1030, 136, (32, 128)),
    (1000, 1, 1024, 264, (64, 64)), (900, 1, 999, 520, (64, 64)), (120, 1, 4096, 1040, (64, 64)), (8192, 1, 60, 4104, (64, 64)),
    (17, 1, 4100, 2056, (32, 32)), (60, 1, 1030, 1000, (32, 32)),
    (1, 1, 100, 7168, (16, 32)), (33, 1, 65, 4360, (16, 32)), (5, 1, 31, 8, (32, 32)),
])
def test_product(T, E, N, K, tile):
    assert mxg.bf16_tile(FWD, E, E, T, N, K) == tile
    act = mxg.ACT_SWIGLU if N % 2 == 0 else mxg.ACT_GELU
    forward_case(routing(T, E), K, N, act, bias=True, residual=True, c_type=BF if K % 16 else F32, keep=True, seed=T)
    forward_case(routing(T, E), K, N, mxg.ACT_NONE, bias=False, residual=False, c_type=F32 if K % 16 else BF,
                 keep=False, seed=T + 10)


@pytest.mark.parametrize("T,E,K,N,tile", [
    (16640, 1, 520, 320, (256, 256)), (33000, 9, 776, 72, (256, 256)), (40000, 4, 1032, 64, (256, 256)),
    (45000, 3, 600, 136, (256, 256)), (8192, 1, 7168, 64, (256, 256)),
    (4000, 5, 1000, 2080, (256, 128)), (2500, 1, 2056, 1000, (256, 128)), (8192, 24, 520, 8, (256, 128)),
    (1000, 6, 2056, 72, (128, 128)), (8192, 6, 264, 2080, (128, 128)), (16640, 6, 8, 1024, (128, 128)),
    (2048, 24, 520, 264, (64, 128)), (4100, 24, 264, 264, (64, 128)), (900, 80, 264, 1000, (32, 128)),
    (1000, 1, 1024, 264, (64, 64)), (120, 1, 4096, 1040, (64, 64)), (8192, 1, 64, 4104, (64, 64)),
    (17, 1, 4104, 2056, (32, 32)),
    (1, 1, 104, 7168, (16, 32)), (33, 1, 72, 4360, (16, 32)),
])
def test_rows_gradient(T, E, K, N, tile):
    assert mxg.bf16_tile(BWD, E, E, T, N, K) == tile
    rows_case(routing(T, E), K, N, mxg.ACT_SWIGLU if T % 2 else mxg.ACT_SILU, seed=T)
    rows_case(routing(T, E), K, N, mxg.ACT_NONE, seed=T + 10)


@pytest.mark.parametrize("T,E,K,N,tile", [
    (9000, 1, 4096, 1544, (256, 256)), (5000, 33, 1288, 1032, (256, 256)), (700, 80, 1024, 776, (256, 256)),
    (16000, 8, 2056, 264, (128, 128)), (8000, 20, 520, 264, (128, 128)),
    (1500, 1, 4104, 72, (64, 64)), (300, 6, 264, 264, (64, 64)), (4100, 1, 1032, 512, (64, 64)),
    (6000, 1, 1544, 200, (64, 32)), (300, 6, 520, 72, (64, 32)), (8192, 1, 7168, 64, (64, 32)), (8192, 1, 4096, 8, (64, 32)), (3, 1, 64, 8, (64, 32)),
])
def test_weights_gradient(T, E, K, N, tile):
    assert mxg.bf16_tile(WTS, E, E, T, N, K) == tile
    weights_case(routing(T, E), K, N, F32, True, False, seed=T)
    weights_case(routing(T, E), K, N, BF, True, True, seed=T + 10)


def test_weights_gradient_of_more_experts_than_groups():
    """2000 experts, three of them named (one twice): the others' gradients are zeros."""
    r = Routing(90, 2000, [0, 20, 50, 70, 90], [1999, 3, 1999, 1024])
    weights_case(r, 72, 40, F32, True, False)
    weights_case(r, 72, 40, BF, False, True)


@pytest.mark.parametrize("T,hint", [(64, 0), (700, 0), (8000, 0), (3, 3)])
def test_experts_past_4_gib(T, hint):
    """Weights of which the last expert lies past 2^32 bytes."""
    E, N, K = 34, 8192, 8192
    b = torch.zeros((E, N, K), dtype=BF, device="cuda")
    b[E - 1] = rand(1, N, K, scale=1 / math.sqrt(K))
    a = rand(2, T, K)
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    ids = torch.tensor([E - 1], dtype=torch.int32, device="cuda")
    c = mxg.grouped_matmul_bf16(a, b, off, ids, max_rows_per_group_hint=hint)
    one = mxg.grouped_matmul_bf16(a, b[E - 1:].clone(), max_rows_per_group_hint=hint)
    assert torch.equal(c, one) and bool((c != 0).any())
    da, da1 = torch.empty_like(a), torch.empty_like(a)
    mxg.mx_grouped_matmul_bf16_backward(c, b, da, off, ids)
    mxg.mx_grouped_matmul_bf16_backward(c, b[E - 1:].clone(), da1)
    assert torch.equal(da, da1)


def test_rows_past_4_gib():
    """The last rows of a, c, dc and z lie past 2^32 bytes."""
    T, K, N = 600000, 4096, 64
    a = torch.zeros((T, K), dtype=BF, device="cuda")
    tail = rand(1, 500, K)
    a[-500:] = tail
    b = rand(2, 1, N, K, scale=1 / 64)
    c = mxg.grouped_matmul_bf16(a, b, dtype=F32)
    want = tail.double() @ b[0].double().t().contiguous()
    bound = (K + 8) * 2.0 ** -23 * (tail.double().abs() @ b[0].double().abs().t().contiguous())
    assert bool(((c[-500:].double() - want).abs() <= bound + 2.0 ** -24 * want.abs()).all())
    assert torch.count_nonzero(c[:-500]) == 0
    dc = torch.zeros((T, N), dtype=BF, device="cuda")
    dc[-500:] = rand(3, 500, N)
    da = torch.ones((T, K), dtype=BF, device="cuda")
    mxg.mx_grouped_matmul_bf16_backward(dc, b, da)
    want = dc[-500:].double() @ b[0].double()
    bound = (N + 8) * 2.0 ** -23 * (dc[-500:].double().abs() @ b[0].double().abs())
    assert bool(((da[-500:].double() - want).abs() <= bound * 1.01 + 2.0 ** -8 * want.abs()).all())
    assert torch.count_nonzero(da[:-500]) == 0
    dw = torch.empty((1, N, K), device="cuda")
    mxg.mx_grouped_matmul_bf16_backward_weights(dc, a, dw)
    want = dc[-500:].double().t().contiguous() @ tail.double()
    bound = 524 * 2.0 ** -23 * (dc[-500:].double().abs().t().contiguous() @ tail.double().abs())
    assert bool(((dw[0].double() - want).abs() <= bound + 2.0 ** -24 * want.abs()).all())


def test_weights_gradient_past_4_gib():
    E, N, K, T = 40, 4096, 8192, 300
    dc, a = rand(1, T, N), rand(2, T, K)
    off = torch.tensor([0, 100, 200, T], dtype=torch.int32, device="cuda")
    ids = torch.tensor([E - 1, 0, E - 1], dtype=torch.int32, device="cuda")
    dw = torch.ones((E, N, K), device="cuda")
    mxg.mx_grouped_matmul_bf16_backward_weights(dc, a, dw, off, ids)
    for e, rows in ((0, slice(100, 200)), (E - 1, [*range(100), *range(200, T)])):
        d, x = dc[rows].double().t().contiguous(), a[rows].double()
        far = (dw[e].double() - d @ x).abs() - 324 * 2.0 ** -23 * (d.abs() @ x.abs())
        assert bool((far <= 2.0 ** -24 * dw[e].double().abs()).all())
    assert torch.count_nonzero(dw[1:E - 1]) == 0


def test_many_groups():
    """1024 groups, most of them empty, in every product."""
    G, T, K, N = 1024, 3000, 72, 136
    g = torch.Generator().manual_seed(1)
    cuts = torch.sort(torch.randint(0, T + 1, (G + 1,), generator=g)).values.tolist()
    ids = torch.randint(-2, 22, (G,), generator=g).tolist()
    r = Routing(T, 20, cuts, ids)
    forward_case(r, K, N, mxg.ACT_SWIGLU, bias=True, residual=True, c_type=BF, keep=True)
    rows_case(r, K, N, mxg.ACT_GELU)
    weights_case(r, K, N, F32, True, False)


@pytest.mark.parametrize("N,K,hint,tile", [(40, 64, 0, (32, 32)), (40, 4104, 0, (16, 32)), (2080, 264, 200, (64, 64)),
                                           (2080, 264, 0, (32, 128))])
def test_rows_beside_an_overlap(N, K, hint, tile):
    """Offsets that go back: more tiles than the rows have.  The row that one group alone owns is right."""
    T, E, G = 201, 2, 61
    off = torch.tensor([0, 200] * 30 + [200, 201], dtype=torch.int32, device="cuda")
    assert off.numel() == G + 1
    ids = torch.tensor([0] * (G - 1) + [1], dtype=torch.int32, device="cuda")
    assert mxg.bf16_tile(FWD, G, E, T, N, K, hint) == tile
    a, b = rand(1, T, K), rand(2, E, N, K, scale=1 / math.sqrt(K))
    c = mxg.grouped_matmul_bf16(a, b, off, ids, dtype=F32, max_rows_per_group_hint=hint)
    want, size = a[200].double() @ b[1].double().t(), a[200].double().abs() @ b[1].double().t().abs()
    assert bool(((c[200].double() - want).abs() <= (K + 8) * 2.0 ** -23 * size + 2.0 ** -24 * want.abs()).all())


@pytest.mark.parametrize("T,N", [(260, 264), (20, 40)])
def test_longest_depth(T, N):
    """K (in the rows' gradient N) of 2^22, a tile's rows 8 MiB apart; what counts stands in its last 72."""
    D, last = 1 << 22, 72
    a, b = torch.zeros((T, D), dtype=BF, device="cuda"), torch.zeros((1, N, D), dtype=BF, device="cuda")
    a[:, -last:], b[0, :, -last:] = rand(1, T, last), rand(2, N, last)
    c = mxg.grouped_matmul_bf16(a, b, dtype=F32)
    x, y = a[:, -last:].double(), b[0, :, -last:].double().t().contiguous()
    want, size = x @ y, x.abs() @ y.abs()
    assert bool(((c.double() - want).abs() <= (last + 8) * 2.0 ** -23 * size + 2.0 ** -24 * want.abs()).all())
    del b
    w = torch.zeros((1, D, N), dtype=BF, device="cuda")
    w[0, -last:] = rand(2, N, last).t()
    da = torch.empty((T, N), dtype=BF, device="cuda")
    mxg.mx_grouped_matmul_bf16_backward(a, w, da)
    bound = (last + 8) * 2.0 ** -23 * size * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    assert bool(((da.double() - want).abs() <= bound).all())
    # the weights' gradient with rows of 2^22 of one operand, then of the other: 40 rows
    del w, da
    d, g = a[:min(T, 40)], rand(3, min(T, 40), 72)
    for rows, dc in ((d, g), (g, d)):
        dw = torch.empty((1, dc.shape[1], rows.shape[1]), device="cuda")
        mxg.mx_grouped_matmul_bf16_backward_weights(dc, rows, dw)
        u, v = (t[:, -last:].double() for t in (dc, rows))
        got = dw[0, -last:, -last:].double()
        want, size = u.t().contiguous() @ v, u.abs().t().contiguous() @ v.abs()
        assert bool(((got - want).abs() <= 64 * 2.0 ** -23 * size + 2.0 ** -24 * want.abs()).all())
        assert not dw[0, :-last].any() if dc is d else not dw[0, :, :-last].any()


def test_very_many_rows():
    T = (1 << 27) + 1000
    a, b = torch.zeros((T, 8), dtype=BF, device="cuda"), torch.eye(8, dtype=BF, device="cuda")[None]
    a[-1500:] = rand(1, 1500, 8)
    assert torch.equal(mxg.grouped_matmul_bf16(a, b), a)
    da = torch.ones_like(a)
    mxg.mx_grouped_matmul_bf16_backward(a, b, da)
    assert torch.equal(da, a)


@pytest.mark.parametrize("accumulate", [False, True])
def test_weights_gradient_of_more_tiles_than_a_launch_has_workgroups(accumulate):
    E, T = (1 << 22) + 300, 6
    assert mxg.bf16_tile(WTS, 3, E, T, 8, 8) == (64, 32)
    dc, a = rand(1, T, 8), rand(2, T, 8)
    off = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, E - 1, E - 250], dtype=torch.int32, device="cuda")
    dw, db = torch.ones((E, 8, 8), device="cuda"), torch.ones((E, 8), device="cuda")
    mxg.mx_grouped_matmul_bf16_backward_weights(dc, a, dw, off, ids, dbias=db, accumulate=accumulate)
    old = float(accumulate)
    for g, e in enumerate(ids.tolist()):
        d, x = dc[2 * g:2 * g + 2].double().t().contiguous(), a[2 * g:2 * g + 2].double()
        want, size = d @ x + old, d.abs() @ x.abs() + old
        assert bool(((dw[e].double() - want).abs() <= 26 * 2.0 ** -23 * size).all())
        assert bool(((db[e].double() - d.sum(1) - old).abs() <= 26 * 2.0 ** -23 * (d.abs().sum(1) + old)).all())
        dw[e], db[e] = old, old
    assert bool((dw == old).all()) and bool((db == old).all())
