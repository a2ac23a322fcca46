"""Calls with more rows than a launch holds workgroups for: the kernels loop over what is left.

The inputs repeat every P rows (P prime), so that every row of the large call has to have the bits of its row
of a small call, whose P rows are one a workgroup and are compared with 64-bit arithmetic."""
import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg

pytestmark = pytest.mark.gpu

BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
P = 1021


def rand(seed, *shape, scale=1.0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def repeated(rows, S):
    """[S, ...] of the P rows over and over."""
    out = torch.empty((S, *rows.shape[1:]), dtype=rows.dtype, device="cuda")
    whole = S // P * P
    out[:whole].view(S // P, P, *rows.shape[1:]).copy_(rows.expand(S // P, *rows.shape))
    out[whole:].copy_(rows[:S - whole])
    return out


def check_repeats(out, rows):
    """Every row of out has the bits of its row of rows."""
    bits = {2: torch.int16, 4: torch.int32, 1: U8}[rows.element_size()]
    out, rows = out.view(bits), rows.view(bits)
    S, step = out.shape[0], max(1, (1 << 28) // max(rows.numel(), 1)) * P
    for lo in range(0, S, step):
        part = out[lo:lo + step]
        n = part.shape[0] // P
        assert bool((part[:n * P].view(n, P, *rows.shape[1:]) == rows).all()), lo
        assert torch.equal(part[n * P:], rows[:part.shape[0] - n * P]), lo


def norm_outputs(S, H, form, residual):
    e = lambda shape, dtype: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    out = dict(h=None if residual is None else e((S, H), residual.dtype),
               y=e((S, H), BF) if form == mxg.NORM_PLAIN else None)
    if form != mxg.NORM_PLAIN:
        out["q"] = e((S, H), U8)
        out["scales"] = {mxg.NORM_FP8_ROWWISE: lambda: e((S,), F32), mxg.NORM_MXFP8: lambda: e((S, H // 32), U8),
                         mxg.NORM_FP8_BLOCK128: lambda: e((S, -(-H // 128)), F32)}[form]()
    return out


# workgroups of 64, 256 and 1024 threads: 2^22, 2^20 and 2^18 of them a launch
@pytest.mark.parametrize("S,H,form,residual", [
    ((1 << 26) + 37, 8, mxg.NORM_PLAIN, None),          # 2^32 threads at a workgroup a row
    ((1 << 23) + 5, 32, mxg.NORM_FP8_BLOCK128, F32),
    ((1 << 22) + 1, 520, mxg.NORM_PLAIN, BF),
    ((1 << 20) + 19, 2080, mxg.NORM_FP8_ROWWISE, None),
    ((1 << 20) + 3, 4128, mxg.NORM_MXFP8, None),
    ((1 << 18) + 7, 8224, mxg.NORM_FP8_ROWWISE, BF),
    ((1 << 18) + 7, 32800, mxg.NORM_FP8_BLOCK128, BF)])
def test_norm(S, H, form, residual):
    x, w = rand(1, P, H), rand(2, H, dtype=F32)
    res = None if residual is None else rand(3, P, H, dtype=residual)
    small = norm_outputs(P, H, form, res)
    mxg.mx_rmsnorm(x, w, residual=res, form=form, eps=1e-5, **small)
    # the small call itself: fp32 arithmetic is off by less than 2^-16 of y, bf16 by 2^-8, e4m3 by 2^-4 of y or
    # 2^-10 of the scale, which here is at most the row's maximum / 448
    h = x.double() if res is None else (small["h"] if residual == BF else x.float() + res).double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-5) * w.double()
    if form == mxg.NORM_PLAIN:
        assert bool(((small["y"].double() - y).abs() <= (2.0 ** -8 + 2.0 ** -15) * y.abs() + 1e-38).all())
    else:
        block = {mxg.NORM_FP8_ROWWISE: H, mxg.NORM_MXFP8: 32, mxg.NORM_FP8_BLOCK128: 128}[form]
        sc = small["scales"].view(P, -1)
        sc = torch.exp2(sc.double() - 127) if form == mxg.NORM_MXFP8 else sc.double()
        sc = sc.repeat_interleave(block, dim=1)[:, :H]
        got = small["q"].view(torch.float8_e4m3fn).double() * sc
        half = (2.0 ** -4 + 2.0 ** -14) * y.abs() + 2.0 ** -10 * sc
        if form == mxg.NORM_MXFP8:  # values from 448 of the scale on, up to 2^9 of it, become 448
            top = y.abs() > 448 * sc
            half = torch.where(top, 2.0 ** -3 * y.abs(), half)
        assert bool(((got - y).abs() <= half).all())
    large = norm_outputs(S, H, form, res)
    xs, rs = repeated(x, S), None if res is None else repeated(res, S)
    if rs is not None:  # h in the residual's place
        large["h"] = rs
    mxg.mx_rmsnorm(xs, w, residual=rs, form=form, eps=1e-5, **large)
    del xs
    for name in ("h", "y", "q", "scales"):
        if large.get(name) is not None:
            check_repeats(large[name], small[name])


@pytest.mark.parametrize("H", [1 << 24, (1 << 24) + 72, (1 << 25) + 8])
def test_norm_gradient_of_long_rows(H):
    """dweight of more columns than a launch takes in one round (2^24).  A thread adds up H / 1024 squares and as many
    products, the lanes and waves 22 more terms: a row's sums, of squares and of products' magnitudes, are off by less than
    (H / 1024 + 22) 2^-24 of themselves, r by half of that."""
    T = 3
    h, dy, w = rand(1, T, H), rand(2, T, H), rand(3, H, dtype=F32)
    dx, dw = torch.zeros_like(h), torch.full((H,), 7.0, device="cuda")
    mxg.mx_rmsnorm_backward(dy, h, w, dx, dweight=dw, eps=1e-5)
    sums = (H / 1024 + 22 + 16) * 2.0 ** -24
    hd, d, g = h.double(), dy.double(), dy.double() * w.double()
    r = 1 / torch.sqrt((hd * hd).mean(1, keepdim=True) + 1e-5)
    terms = d * hd * r
    assert bool(((dw.double() - terms.sum(0)).abs() <= (sums + 2.0 ** -20) * terms.abs().sum(0)).all())
    back = hd * r ** 3 * (g * hd).mean(1, keepdim=True)
    size = (g * r).abs() + hd.abs() * r ** 3 * (g * hd).abs().mean(1, keepdim=True)
    want = r * g - back
    assert bool(((dx.double() - want).abs() <= (3 * sums + 2.0 ** -20) * size + 2.0 ** -8 * want.abs() + 1e-38).all())


def test_norm_gradient_of_no_rows():
    """Zeros, for rows of 2^30 - 8 elements (2^34 threads at 64 columns a workgroup of 1024)."""
    H = (1 << 30) - 8
    e = lambda *s: torch.empty(s, dtype=BF, device="cuda")  # noqa: E731
    dw = torch.full((H,), 7.0, device="cuda")
    mxg.mx_rmsnorm_backward(e(0, H), e(0, H), e(H), dweight=dw)
    assert torch.count_nonzero(dw) == 0


@pytest.mark.parametrize("act,S,N", [(mxg.ACT_SWIGLU, (1 << 24) + 3, 1024), (mxg.ACT_SILU, (1 << 22) + 5, 520),
                                     (mxg.ACT_RELU, (1 << 28) + 1, 8)])
def test_activation_gradient(act, S, N):
    """More vectors than a launch has threads (2^28): 2^32 of them with the first, z and dz 64 GiB in one place."""
    wide = 2 * N if act == mxg.ACT_SWIGLU else N
    dc, z = rand(1, P, N), rand(2, P, wide, scale=3.0)
    small = torch.zeros_like(z)
    mxg.mx_activation_backward(act, dc, z, small)
    g, d = z.double(), dc.double()
    if act == mxg.ACT_RELU:
        want = d * (g > 0)
        size = want.abs()
    else:
        if act == mxg.ACT_SWIGLU:
            g, u = g[:, 0::2], g[:, 1::2]
        s = 1 / (1 + torch.exp(-g))
        slope, terms = s + g * s * (1 - s), s + g.abs() * s
        if act == mxg.ACT_SILU:
            want, size = d * slope, d.abs() * terms
        else:
            want = torch.stack((d * u * slope, d * g * s), 2).flatten(1)
            size = torch.stack(((d * u).abs() * terms, (d * g).abs()), 2).flatten(1)
    # fp32 arithmetic of 2^-18 of the terms, rounded once
    assert bool(((small.double() - want).abs() <= 2.0 ** -18 * size + 2.0 ** -8 * want.abs() + 1e-38).all())
    dcs, zs = repeated(dc, S), repeated(z, S)
    mxg.mx_activation_backward(act, dcs, zs, zs)
    check_repeats(zs, small)


@pytest.mark.parametrize("S,H,k", [((1 << 26) + 9, 8, 1), ((1 << 22) + 5, 40, 3)])
def test_combine(S, H, k):
    """More tokens than a launch has waves for (2^22): 2^32 threads with the first.  Every P tokens share their rows'
    numbers and weights; the last token's last slot is dropped."""
    y = rand(1, 4096, H)
    rows = torch.arange(P * k, dtype=torch.int32, device="cuda").view(P, k) * 7 % 4096
    w = rand(2, P, k, dtype=F32)
    small = torch.zeros((P, H), dtype=BF, device="cuda")
    mxg.mx_moe_combine(y, rows.flatten(), w.flatten(), small)
    terms = y[rows.long()].double() * w.double().unsqueeze(2)
    want = terms.sum(1)
    assert bool(((small.double() - want).abs() <= k * 2.0 ** -24 * terms.abs().sum(1) * (1 + 2.0 ** -8) +
                 2.0 ** -8 * want.abs() + 1e-38).all())
    many = repeated(rows, S)
    many[-1, -1] = -1
    out = torch.full((S, H), 7.0, dtype=BF, device="cuda")
    mxg.mx_moe_combine(y, many.flatten(), repeated(w, S).flatten(), out)
    check_repeats(out[:-1], small)
    last = terms[(S - 1) % P, :k - 1].sum(0)
    assert bool(((out[-1].double() - last).abs() <= 2.0 ** -7 * terms[(S - 1) % P].abs().sum(0)).all())
