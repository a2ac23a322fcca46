"""The BF16 products with their epilogue and the gradients of both, against 64-bit
arithmetic.

Bounds.  A product of two bf16 numbers is exact in fp32, so a sum of K of them is off by the
additions alone: at most one unit (2^-23) of the magnitudes' sum each, (K + 8) 2^-23 of
it with the joining of partial sums.  The activations and their derivatives: slopes of at
most 1.2 (silu 1.1, gelu 1.13; their derivatives' 0.8 at most), and fp32 arithmetic of 2^-18
of the values they are made of.  Rounding to bf16: 2^-8, to fp32: 2^-24."""
import math

import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ACTS = [mxg.ACT_NONE, mxg.ACT_RELU, mxg.ACT_GELU, mxg.ACT_SILU, mxg.ACT_SWIGLU]
ARITH = 2.0 ** -18


def rand(seed, *shape, scale=1.0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


class Routing:
    """Row ranges [lo, hi) of expert e, in group order; rows outside them are not covered."""

    def __init__(self, T, E, offsets=None, ids=None):
        self.T, self.E = T, E
        if offsets is None:
            self.off = self.ids = None
            self.ranges = [(0, T, 0)]
            return
        self.off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        self.ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
        self.ranges = []
        for g, e in enumerate(ids):
            lo, hi = min(offsets[g], T), min(offsets[g + 1], T)
            if lo < hi and 0 <= e < E:
                self.ranges.append((lo, hi, e))

    def covered(self):
        m = torch.zeros(self.T, dtype=torch.bool, device="cuda")
        for lo, hi, _ in self.ranges:
            m[lo:hi] = True
        return m


ROUTINGS = {
    "dense_1": lambda: Routing(1, 1),
    "dense_17": lambda: Routing(17, 1),
    "dense_300": lambda: Routing(300, 1),
    "one_row_each": lambda: Routing(5, 5, [0, 1, 2, 3, 4, 5], [4, 2, 0, 1, 3]),
    "ragged": lambda: Routing(700, 6, [0, 3, 3, 260, 261, 517, 700], [0, 1, 2, 3, 4, 5]),
    # a gap before the first row and behind the last, an id twice, two out of range, a descending
    # offset (behind a group that is not taken, so that no row has two owners), an offset past the rows
    "odd_ids": lambda: Routing(200, 4, [7, 40, 41, 100, 90, 150, 900], [2, 2, 9, 0, 3, -1]),
    "tail": lambda: Routing(150, 3, [5, 60, 61, 139], [1, 0, 1]),
    "many": lambda: Routing(900, 64, list(range(0, 65 * 14, 14)), list(range(63, -1, -1))),
}


def exact_act(z, act):
    if act == mxg.ACT_RELU:
        return z * (z > 0)
    if act == mxg.ACT_GELU:
        return z * torch.special.ndtr(z)
    if act == mxg.ACT_SILU:
        return z / (1 + torch.exp(-z))
    if act == mxg.ACT_SWIGLU:
        return z[:, 0::2] / (1 + torch.exp(-z[:, 0::2])) * z[:, 1::2]
    return z


def check_rows(c, want, limit, covered, before):
    assert torch.equal(c[~covered], before[~covered])
    far = (c.double() - want).abs()[covered] - limit[covered]
    assert bool((far <= 0).all()), float(far.max())


def forward_case(r, K, N, act, bias, residual, c_type, keep, seed=1, hint=0):
    a, b = rand(seed, r.T, K), rand(seed + 1, r.E, N, K, scale=1 / math.sqrt(K))
    bias = rand(seed + 2, r.E, N, dtype=F32) if bias else None
    wide = N // 2 if act == mxg.ACT_SWIGLU else N
    c = torch.full((r.T, wide), 7.0, dtype=c_type, device="cuda")
    res = rand(seed + 3, r.T, wide, dtype=c_type) if residual else None
    z = torch.full((r.T, N), 7.0, dtype=BF, device="cuda") if keep else None
    before = c.clone()
    mxg.mx_grouped_matmul_bf16(a, b, c, r.off, r.ids, bias=bias, act=act, residual=res, z=z,
                               max_rows_per_group_hint=hint)
    want, limit = (torch.zeros((r.T, wide), dtype=torch.float64, device="cuda") for _ in range(2))
    zs, zlim = (torch.zeros((r.T, N), dtype=torch.float64, device="cuda") for _ in range(2))
    for lo, hi, e in r.ranges:
        aa, bb = a[lo:hi].double(), b[e].double().t().contiguous()
        zs[lo:hi] = aa @ bb
        zlim[lo:hi] = aa.abs() @ bb.abs()
        if bias is not None:
            zs[lo:hi] += bias[e].double()
            zlim[lo:hi] += bias[e].double().abs()
    zlim *= (K + 8) * 2.0 ** -23
    want = exact_act(zs, act)
    if act == mxg.ACT_SWIGLU:
        limit = (1.2 * zlim[:, 0::2] * zs[:, 1::2].abs() + zs[:, 0::2].abs() * zlim[:, 1::2] +
                 ARITH * (zs[:, 0::2] * zs[:, 1::2]).abs() + zlim[:, 0::2] * zlim[:, 1::2])
    else:
        limit = 1.2 * zlim + (0 if act in (mxg.ACT_NONE, mxg.ACT_RELU) else ARITH * zs.abs())
    if residual:
        want = want + res.double()
        limit = limit + 2.0 ** -24 * want.abs()
    half = torch.finfo(c_type).eps / 2
    cov = r.covered()
    check_rows(c, want, limit * (1 + half) + half * want.abs() + 1e-38, cov, before)
    if keep:
        check_rows(z, zs, zlim * (1 + 2.0 ** -8) + 2.0 ** -8 * zs.abs() + 1e-38, cov, torch.full_like(z, 7.0))
    return a, b, c, z


@pytest.mark.parametrize("name", list(ROUTINGS))
@pytest.mark.parametrize("K,N", [(8, 1), (64, 64), (72, 34), (136, 130), (520, 97), (32, 300), (1024, 520)])
def test_product(name, K, N):
    forward_case(ROUTINGS[name](), K, N, mxg.ACT_NONE, bias=K % 16 == 8, residual=False, c_type=BF, keep=False)


@pytest.mark.parametrize("c_type", [BF, F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("name,K,N", [("ragged", 104, 72), ("odd_ids", 64, 70), ("dense_17", 192, 256),
                                      ("dense_300", 64, 38), ("tail", 648, 264), ("many", 64, 200)])
def test_epilogue(name, K, N, act, c_type):
    forward_case(ROUTINGS[name](), K, N, act, bias=True, residual=True, c_type=c_type, keep=True)


@pytest.mark.parametrize("name,K,N,act,c_type,hint", [
    ("dense_300", 2048, 1040, mxg.ACT_SWIGLU, BF, 0), ("ragged", 4104, 264, mxg.ACT_GELU, F32, 257),
    ("dense_17", 7168, 64, mxg.ACT_NONE, F32, 17), ("dense_1", 7168, 2064, mxg.ACT_SILU, BF, 1),
    ("one_row_each", 2080, 1000, mxg.ACT_NONE, BF, 1)])
def test_longer_sums(name, K, N, act, c_type, hint):
    forward_case(ROUTINGS[name](), K, N, act, bias=True, residual=False, c_type=c_type, keep=False, hint=hint)


@pytest.mark.parametrize("T,E,K,N", [(2600, 1, 320, 776), (4100, 7, 200, 520), (40000, 3, 64, 264)])
def test_many_rows(T, E, K, N):
    cuts = [T * i * i // (E * E) for i in range(E + 1)]
    r = Routing(T, E, cuts, list(range(E))) if E > 1 else Routing(T, 1)
    a, b, c, _ = forward_case(r, K, N, mxg.ACT_SWIGLU, bias=True, residual=True, c_type=BF, keep=True)
    again = torch.empty_like(c)
    d = rand(9, T, N // 2)
    mxg.mx_grouped_matmul_bf16(a, b, again, r.off, r.ids, act=mxg.ACT_SWIGLU, residual=d)
    same = d.clone()
    mxg.mx_grouped_matmul_bf16(a, b, same, r.off, r.ids, act=mxg.ACT_SWIGLU, residual=same)  # in place
    cov = r.covered()
    assert torch.equal(same[cov], again[cov])


def test_non_finite_values_stay_in_their_rows():
    """An infinity or NaN in a row, or in rows and weights no result depends on, changes no other result."""
    r = Routing(100, 2, [10, 50, 90], [0, 1])
    K, N = 72, 40
    a, b = rand(1, 100, K), rand(2, 2, N, K)
    clean = mxg.grouped_matmul_bf16(a, b, r.off, r.ids)
    a2, b2 = a.clone(), b.clone()
    a2[:10], a2[90:], a2[49] = float("nan"), float("inf"), float("inf")
    b2[1, 7, 3] = float("nan")
    c = mxg.grouped_matmul_bf16(a2, b2, r.off, r.ids)
    keep = torch.ones_like(c, dtype=torch.bool)
    keep[49] = False
    keep[50:90, 7] = False
    assert torch.equal(c[keep], clean[keep])
    assert not torch.isfinite(c[49]).any() and torch.isnan(c[50:90, 7]).all()
    # infinities go through the activations as their formulas have it; relu keeps a NaN
    z = mxg.grouped_matmul_bf16(a2, b2, r.off, r.ids, act=mxg.ACT_RELU)
    assert torch.isnan(z[50:90, 7]).all() and bool((z[10:49] >= 0).all())


def exact_grad(z, d, act):
    """d times the activation's derivative at z, and a bound of the terms it is made of."""
    if act == mxg.ACT_NONE:
        return d, d.abs()
    if act == mxg.ACT_RELU:
        return d * (z > 0), d.abs()
    if act == mxg.ACT_GELU:
        return d * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)), 1.2 * d.abs()
    g, u = (z, None) if act == mxg.ACT_SILU else (z[:, 0::2], z[:, 1::2])
    s = 1 / (1 + torch.exp(-g))
    slope = s + g * s * (1 - s)
    if act == mxg.ACT_SILU:
        return d * slope, d.abs() * (s + g.abs() * s)
    out, size = torch.empty_like(z), torch.empty_like(z)
    out[:, 0::2], out[:, 1::2] = d * u * slope, d * g * s
    size[:, 0::2], size[:, 1::2] = (d * u).abs() * (s + g.abs() * s), (d * g).abs()
    return out, size


def rows_case(r, K, N, act, seed=1, hint=0, in_place=False):
    dc, b = rand(seed, r.T, N), rand(seed + 1, r.E, N, K, scale=1 / math.sqrt(N))
    wide = 2 * K if act == mxg.ACT_SWIGLU else K
    z = None if act == mxg.ACT_NONE else rand(seed + 2, r.T, wide)
    da = torch.full((r.T, wide), 7.0, dtype=BF, device="cuda")
    zd = None if z is None else z.double()
    if in_place and z is not None:
        da = z
    before = da.clone()
    mxg.mx_grouped_matmul_bf16_backward(dc, b, da, r.off, r.ids, act=act, z=z, max_rows_per_group_hint=hint)
    d, dlim = (torch.zeros((r.T, K), dtype=torch.float64, device="cuda") for _ in range(2))
    for lo, hi, e in r.ranges:
        d[lo:hi] = dc[lo:hi].double() @ b[e].double()
        dlim[lo:hi] = (dc[lo:hi].double().abs() @ b[e].double().abs()) * ((N + 8) * 2.0 ** -23)
    want, size = exact_grad(zd, d, act)
    lim = exact_grad(zd, dlim, act)[1] if act != mxg.ACT_NONE else dlim
    check_rows(da, want, (1.2 * lim + ARITH * size) * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 1e-38, r.covered(),
               before)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("name", list(ROUTINGS))
@pytest.mark.parametrize("K,N", [(8, 8), (72, 40), (136, 256), (520, 1048)])
def test_rows_gradient(name, K, N, act):
    rows_case(ROUTINGS[name](), K, N, act, in_place=K == 72)


@pytest.mark.parametrize("T,E,K,N,act", [(2600, 1, 776, 320, mxg.ACT_SWIGLU), (4100, 7, 200, 520, mxg.ACT_GELU),
                                         (40000, 3, 264, 64, mxg.ACT_NONE), (300, 1, 2048, 4096, mxg.ACT_SILU)])
def test_rows_gradient_many_rows(T, E, K, N, act):
    cuts = [T * i * i // (E * E) for i in range(E + 1)]
    rows_case(Routing(T, E, cuts, list(range(E))) if E > 1 else Routing(T, 1), K, N, act, hint=cuts[-1] // 2)


def weights_case(r, K, N, dw_type, bias, accumulate, seed=1):
    dc, a = rand(seed, r.T, N), rand(seed + 1, r.T, K)
    dw = rand(seed + 2, r.E, N, K, dtype=dw_type)
    db = rand(seed + 3, r.E, N, dtype=F32) if bias else None
    old_w, old_b = dw.double(), None if db is None else db.double()
    mxg.mx_grouped_matmul_bf16_backward_weights(dc, a, dw, r.off, r.ids, dbias=db, accumulate=accumulate)
    want, size = torch.zeros_like(old_w), torch.zeros_like(old_w)
    want_b, size_b = (torch.zeros((r.E, N), dtype=torch.float64, device="cuda") for _ in range(2))
    rows = torch.zeros(r.E, dtype=torch.float64, device="cuda")
    for lo, hi, e in r.ranges:
        d = dc[lo:hi].double().t().contiguous()
        want[e] += d @ a[lo:hi].double()
        size[e] += d.abs() @ a[lo:hi].double().abs()
        want_b[e] += d.sum(1)
        size_b[e] += d.abs().sum(1)
        rows[e] += hi - lo
    half = torch.finfo(dw_type).eps / 2
    additions = ((rows + 24) * 2.0 ** -23)[:, None, None]
    limit = additions * size
    if accumulate:
        want, limit = want + old_w, limit + 2.0 ** -23 * (size + old_w.abs())
    far = (dw.double() - want).abs() - (limit + half * want.abs() + 1e-38)
    assert bool((far <= 0).all()), float(far.max())
    if bias:
        lim_b = additions[:, :, 0] * size_b
        if accumulate:
            want_b, lim_b = want_b + old_b, lim_b + 2.0 ** -23 * (size_b + old_b.abs())
        assert bool(((db.double() - want_b).abs() <= lim_b + 2.0 ** -24 * want_b.abs()).all())


@pytest.mark.parametrize("dw_type,bias,accumulate", [(F32, True, False), (BF, False, False), (F32, True, True),
                                                     (BF, True, True), (F32, False, False)])
@pytest.mark.parametrize("name", list(ROUTINGS))
@pytest.mark.parametrize("K,N", [(8, 8), (72, 40), (136, 264), (520, 64)])
def test_weights_gradient(name, K, N, dw_type, bias, accumulate):
    weights_case(ROUTINGS[name](), K, N, dw_type, bias, accumulate)


@pytest.mark.parametrize("T,E,K,N", [(3000, 1, 776, 320), (4100, 7, 200, 520), (20001, 1, 520, 64), (9000, 3, 64, 1032),
                                     (2000, 40, 512, 768)])
def test_weights_gradient_many_rows(T, E, K, N):
    cuts = [T * i * i // (E * E) for i in range(E + 1)]
    weights_case(Routing(T, E, cuts, list(range(E))) if E > 1 else Routing(T, 1), K, N, F32, True, False)


def test_weights_gradient_non_finite_rows():
    """Rows of other experts, and rows no group covers, take no part, whatever they hold."""
    r = Routing(130, 3, [10, 55, 56, 120], [0, 1, 2])
    dc, a = rand(1, 130, 72), rand(2, 130, 136)
    clean, dw = (torch.empty((3, 72, 136), device="cuda") for _ in range(2))
    mxg.mx_grouped_matmul_bf16_backward_weights(dc, a, clean, r.off, r.ids)
    for t in (dc, a):
        t[:10], t[120:], t[55] = float("nan"), float("inf"), float("inf")
    db = torch.empty((3, 72), device="cuda")
    mxg.mx_grouped_matmul_bf16_backward_weights(dc, a, dw, r.off, r.ids, dbias=db)
    assert torch.equal(dw[0], clean[0]) and torch.equal(dw[2], clean[2]) and not torch.isfinite(dw[1]).any()
    assert torch.isfinite(db[[0, 2]]).all() and torch.isinf(db[1]).all()


def test_no_rows():
    a, b = rand(1, 0, 64), rand(2, 2, 16, 64)
    off, ids = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.arange(2, dtype=torch.int32, device="cuda")
    assert mxg.grouped_matmul_bf16(a, b, off, ids).shape == (0, 16)
    for acc in (False, True):
        dw, db = torch.full((2, 16, 64), 3.0, device="cuda"), torch.full((2, 16), 3.0, device="cuda")
        mxg.mx_grouped_matmul_bf16_backward_weights(rand(3, 0, 16), a, dw, off, ids, dbias=db, accumulate=acc)
        assert bool((dw == (3.0 if acc else 0.0)).all()) and bool((db == (3.0 if acc else 0.0)).all())
    # rows, but no group
    dw = torch.full((2, 16, 64), 3.0, dtype=BF, device="cuda")
    mxg.mx_grouped_matmul_bf16_backward_weights(rand(3, 5, 16), rand(4, 5, 64), dw, off[:1], ids[:0])
    assert torch.count_nonzero(dw) == 0


@pytest.mark.parametrize("act", ACTS[1:])
def test_activation_gradient(act):
    T, N = 37, 136
    wide = 2 * N if act == mxg.ACT_SWIGLU else N
    dc, z = rand(1, T, N), rand(2, T, wide, scale=3.0)
    z[0, :8] = torch.tensor([0.0, -0.0, 80.0, -80.0, 1e30, -1e30, 1e-30, 12.0], device="cuda")
    dz = torch.empty_like(z)
    mxg.mx_activation_backward(act, dc, z, dz)
    want, size = exact_grad(z.double(), dc.double(), act)
    assert bool(((dz.double() - want).abs() <= ARITH * size + 2.0 ** -8 * want.abs() + 1e-38).all())
    zp = z.clone()
    mxg.mx_activation_backward(act, dc, zp, zp)
    assert torch.equal(zp, dz)
    if act != mxg.ACT_SWIGLU:
        dp = dc.clone()
        mxg.mx_activation_backward(act, dp, z, dp)
        assert torch.equal(dp, dz)


def test_gradients_against_differences():
    """A loss <dc, act(a W1^T + b1) W2^T + b2> along random directions of its inputs: central differences in 64 bits
    (step 1e-4: their own error is below 1e-6 of the terms) against the gradients as the calls give them.  The chain
    rounds z, dz and da to bf16, each 2^-8 of its value: the derivative along a direction is off by at most
    3 * 2^-8 of the sum of magnitudes."""
    r = ROUTINGS["ragged"]()
    K, I, N, act = 40, 24, 48, mxg.ACT_SWIGLU
    a, w1, b1 = rand(1, r.T, K), rand(2, r.E, 2 * I, K, scale=0.3), rand(3, r.E, 2 * I, scale=0.3, dtype=F32)
    w2, b2, dc = rand(4, r.E, N, I, scale=0.3), rand(5, r.E, N, dtype=F32), rand(6, r.T, N)
    e = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    z, y, c = e(r.T, 2 * I), e(r.T, I), e(r.T, N)
    mxg.mx_grouped_matmul_bf16(a, w1, y, r.off, r.ids, bias=b1, act=act, z=z)
    mxg.mx_grouped_matmul_bf16(y, w2, c, r.off, r.ids, bias=b2)
    dz, da, dw1, db1 = e(r.T, 2 * I), e(r.T, K), e(r.E, 2 * I, K, dt=F32), e(r.E, 2 * I, dt=F32)
    mxg.mx_grouped_matmul_bf16_backward(dc, w2, dz, r.off, r.ids, act=act, z=z)
    mxg.mx_grouped_matmul_bf16_backward(dz, w1, da, r.off, r.ids)
    mxg.mx_grouped_matmul_bf16_backward_weights(dz, a, dw1, r.off, r.ids, dbias=db1)

    def loss(a, w1, b1):
        total = 0.0
        for lo, hi, x in r.ranges:
            h = exact_act(a[lo:hi] @ w1[x].t().contiguous() + b1[x], act)
            total = total + (dc[lo:hi].double() * (h @ w2[x].double().t().contiguous())).sum()
        return total

    at = [a.double(), w1.double(), b1.double()]
    terms = None
    for i, got in enumerate((da, dw1, db1)):
        v = rand(10 + i, *at[i].shape, dtype=torch.float64)
        lo, hi = list(at), list(at)
        lo[i], hi[i] = at[i] - 1e-4 * v, at[i] + 1e-4 * v
        along = float(loss(*hi) - loss(*lo)) / 2e-4
        terms = float((got.double() * v).abs().sum())
        assert abs(along - float((got.double() * v).sum())) <= 3 * 2.0 ** -8 * terms


def test_refusals():
    a, b, c = rand(1, 8, 64), rand(2, 2, 16, 64), torch.empty((8, 16), dtype=BF, device="cuda")
    off, ids = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda"), torch.arange(2, dtype=torch.int32, device="cuda")
    f = mxg.mx_grouped_matmul_bf16
    bad = (ValueError, TypeError, mxg.MxgError)
    for args, kw in [((a, b, c), {}), ((a, b, c, off), {}), ((a, b, c, off, ids), dict(act=9)),
                     ((a, b, c, off, ids), dict(bias=rand(3, 2, 16))), ((a, b, c, off, ids), dict(z=c)),
                     ((a, b, c, off, ids), dict(residual=c.float())), ((a, b, c, off, ids), dict(act=mxg.ACT_SWIGLU)),
                     ((a[:, :60], b, c, off, ids), {}), ((a, b[0], c, off, ids), {}), ((a.float(), b, c, off, ids), {}),
                     ((a, b, c.cpu(), off, ids), {}), ((a, b, c, off[:2], ids), {})]:
        with pytest.raises(bad):
            f(*args, **kw)
    with pytest.raises(mxg.MxgError):
        f(rand(1, 4, 20), rand(2, 1, 16, 20), torch.empty((4, 16), dtype=BF, device="cuda"))  # K = 20
    g = mxg.mx_grouped_matmul_bf16_backward
    dc, da = rand(4, 8, 16), torch.empty((8, 64), dtype=BF, device="cuda")
    for args, kw in [((dc, b, da, off, ids), dict(z=a)), ((dc, b, da, off, ids), dict(act=mxg.ACT_RELU)),
                     ((dc, b, da, off, ids), dict(act=mxg.ACT_SWIGLU, z=a)), ((dc, b, dc, off, ids), {})]:
        with pytest.raises(bad):
            g(*args, **kw)
    with pytest.raises(mxg.MxgError):  # N = 12
        g(rand(4, 8, 12), rand(5, 1, 12, 64), da)
    w = mxg.mx_grouped_matmul_bf16_backward_weights
    dw = torch.empty((2, 16, 64), device="cuda")
    for args, kw in [((dc, a, dw), {}), ((dc, a, dw[:, :8], off, ids), {}), ((dc, a[:7], dw, off, ids), {}),
                     ((dc, a, dw.half(), off, ids), {}), ((dc, a, dw, off, ids), dict(dbias=rand(1, 2, 16)))]:
        with pytest.raises(bad):
            w(*args, **kw)
    for args in [(mxg.ACT_NONE, dc, dc.clone(), dc.clone()), (mxg.ACT_SWIGLU, dc, rand(1, 8, 32), dc)]:
        with pytest.raises(bad):
            mxg.mx_activation_backward(*args)
    f(a, b, c, off, ids)


def test_graph_and_streams():
    """A step forward and backward captured and replayed, with other inputs and eager work between; and on another
    stream: the eager step's bits."""
    r = ROUTINGS["ragged"]()
    K, I, N, act = 136, 64, 72, mxg.ACT_SWIGLU
    ins = dict(a=rand(1, r.T, K), w1=rand(2, r.E, 2 * I, K), b1=rand(3, r.E, 2 * I, dtype=F32), w2=rand(4, r.E, N, I),
               res=rand(5, r.T, N, dtype=F32), dc=rand(6, r.T, N))

    def fresh():
        e = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
        return dict(z=e(r.T, 2 * I), y=e(r.T, I), c=e(r.T, N, dt=F32), dz=e(r.T, 2 * I), da=e(r.T, K),
                    dw1=e(r.E, 2 * I, K, dt=F32), db1=e(r.E, 2 * I, dt=F32), dw2=e(r.E, N, I))

    def step(o):
        m = mxg
        m.mx_grouped_matmul_bf16(ins["a"], ins["w1"], o["y"], r.off, r.ids, bias=ins["b1"], act=act, z=o["z"])
        m.mx_grouped_matmul_bf16(o["y"], ins["w2"], o["c"], r.off, r.ids, residual=ins["res"])
        m.mx_grouped_matmul_bf16_backward(ins["dc"], ins["w2"], o["dz"], r.off, r.ids, act=act, z=o["z"])
        m.mx_grouped_matmul_bf16_backward(o["dz"], ins["w1"], o["da"], r.off, r.ids)
        m.mx_grouped_matmul_bf16_backward_weights(o["dz"], ins["a"], o["dw1"], r.off, r.ids, dbias=o["db1"])
        m.mx_grouped_matmul_bf16_backward_weights(ins["dc"], o["y"], o["dw2"], r.off, r.ids)

    cap, eager, side = fresh(), fresh(), fresh()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(cap)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cap)
    for i in range(3):
        ins["a"].copy_(rand(20 + i, r.T, K))
        ins["dc"].copy_(rand(30 + i, r.T, N))
        graph.replay()
        step(eager)
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step(side)
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(cap[k], eager[k]) and torch.equal(side[k], eager[k]), k
