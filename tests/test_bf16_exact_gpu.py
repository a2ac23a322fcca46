"""The BF16 products and their gradients on small whole numbers: every product and every partial sum, in whatever
order, is a whole number below 2^24, which fp32 holds exactly, so the results have to equal those of 64-bit
arithmetic, rounded once where they are bf16.  A row, a stage or a term of the depth that is lost or taken twice shows
at any length, where a bound of rounding errors grows with it."""
import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg
from test_matmul_bf16_gpu import BF, F32, Routing

pytestmark = pytest.mark.gpu

FWD, BWD, WTS = mxg.BF16_FORWARD, mxg.BF16_BACKWARD, mxg.BF16_BACKWARD_WEIGHTS
MOST = 3  # the inputs' magnitude; never 0, so that each term counts


def whole(seed, *shape, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    v = torch.randint(1, MOST + 1, shape, generator=g, device="cuda")
    return (v * (2 * torch.randint(0, 2, shape, generator=g, device="cuda") - 1)).to(dtype)


def uneven(T, E):
    """An expert without rows, one with a single row, the others uneven; the last row behind the last group."""
    if E == 1:
        return Routing(T, 1)
    cuts = [0, 0, 1] + [1 + (T - 2) * i * i // ((E - 2) * (E - 2)) for i in range(1, E - 1)]
    return Routing(T, E, cuts, list(range(E)))


def split_experts(T, E):
    """Each expert's rows in two groups of odd lengths, the experts in turn."""
    cuts = [T * i * (i + 1) // (2 * E * (2 * E + 1)) for i in range(2 * E + 1)]
    return Routing(T, E, cuts, [i % E for i in range(2 * E)])


def rounded(x, dtype):
    return x.to(F32).to(dtype)  # both steps exact or, the second, the one rounding


def check_weights(r, N, K, dw_type, accumulate, seed):
    dc, a = whole(seed, r.T, N), whole(seed + 1, r.T, K)
    dw = whole(seed + 2, r.E, N, K, dtype=dw_type)
    db = whole(seed + 3, r.E, N, dtype=F32)
    want, want_b = torch.zeros((r.E, N, K), dtype=F32, device="cuda"), torch.zeros((r.E, N), dtype=F32, device="cuda")
    for lo, hi, e in r.ranges:
        d = dc[lo:hi].double().t().contiguous()
        want[e] += (d @ a[lo:hi].double()).float()
        want_b[e] += d.sum(1).float()
    if accumulate:
        want += dw.float()
        want_b += db
    assert float(want.abs().max()) < 2 ** 24
    mxg.mx_grouped_matmul_bf16_backward_weights(dc, a, dw, r.off, r.ids, dbias=db, accumulate=accumulate)
    assert torch.equal(dw, want.to(dw_type))
    assert torch.equal(db, want_b)
    plain = torch.empty_like(dw)  # the kernel without the bias
    if not accumulate:
        mxg.mx_grouped_matmul_bf16_backward_weights(dc, a, plain, r.off, r.ids)
        assert torch.equal(plain, dw)


@pytest.mark.parametrize("T,E,N,K,tile", [
    (20001, 1, 64, 520, (64, 32)), (8192, 1, 64, 7168, (64, 32)), (9000, 3, 1032, 64, (64, 32)),
    (100001, 3, 8, 96, (64, 32)), (4100, 7, 520, 200, (64, 64)), (20001, 1, 512, 1032, (64, 64)),
    (8192, 1, 2048, 2048, (128, 128)), (16384, 8, 256, 2048, (128, 128)), (100003, 1, 1544, 2056, (128, 128)),
    (33000, 5, 1544, 1024, (256, 256)), (2000, 40, 768, 512, (256, 256)), (9000, 1, 4104, 4096, (256, 256)),
    (65537, 3, 2056, 2048, (256, 256)),
])
@pytest.mark.parametrize("groups", [uneven, split_experts])
def test_weights_gradient(T, E, N, K, tile, groups):
    assert mxg.bf16_tile(WTS, E if groups is uneven else 2 * E, E, T, N, K) == tile
    check_weights(groups(T, E), N, K, F32, False, T)
    check_weights(groups(T, E), N, K, BF, True, T + 1)


@pytest.mark.parametrize("T,E,N,K", [
    (16640, 1, 520, 4104), (33000, 9, 776, 2056), (4000, 5, 1000, 2080), (2048, 6, 1544, 7176), (16640, 80, 71, 1032),
    (1500, 6, 775, 2056), (900, 80, 262, 4104), (120, 1, 4096, 7176), (17, 1, 4100, 16392), (1, 1, 100, 65544),
    (33, 1, 65, 20008), (45000, 3, 600, 136),
])
def test_products(T, E, N, K):
    r = uneven(T, E)
    a, b, bias = whole(T, T, K), whole(T + 1, E, N, K), whole(T + 2, E, N, dtype=F32)
    res = whole(T + 3, T, N, dtype=F32)
    c, z = torch.full((T, N), 7.0, device="cuda"), torch.full((T, N), 7.0, dtype=BF, device="cuda")
    want, want_z = c.clone(), z.clone()
    for lo, hi, e in r.ranges:
        sums = (a[lo:hi].double() @ b[e].double().t().contiguous()).float() + bias[e]
        want[lo:hi], want_z[lo:hi] = sums + res[lo:hi], sums.to(BF)
    mxg.mx_grouped_matmul_bf16(a, b, c, r.off, r.ids, bias=bias, residual=res, z=z)
    assert torch.equal(c, want) and torch.equal(z, want_z)


@pytest.mark.parametrize("T,E,K,N", [
    (16640, 1, 520, 4104), (33000, 9, 776, 2056), (4000, 5, 1000, 2080), (2048, 24, 520, 7176), (900, 80, 264, 4104),
    (1000, 6, 2056, 72), (120, 1, 4096, 7176), (17, 1, 4104, 16392), (1, 1, 104, 65544), (33, 1, 72, 20008),
])
def test_rows_gradient(T, E, K, N):
    r = uneven(T, E)
    dc, b, da = whole(T, T, N), whole(T + 1, E, N, K), torch.full((T, K), 7.0, dtype=BF, device="cuda")
    want = da.clone()
    for lo, hi, e in r.ranges:
        want[lo:hi] = rounded(dc[lo:hi].double() @ b[e].double(), BF)
    mxg.mx_grouped_matmul_bf16_backward(dc, b, da, r.off, r.ids)
    assert torch.equal(da, want)
