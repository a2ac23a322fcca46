"""The norm with the residual's addition and its 8-bit outputs, and its gradient, against
64-bit arithmetic.

Bounds.  fp32 arithmetic: a thread adds up at most 64 squares, the lanes and waves 22 more
terms, so a row's sum is off by less than 2^-17 of itself (every square is positive; rows
past 32768 elements: H / 1024 terms a thread, here below 64 too), r by half of that and
the root's, quotient's and products' roundings, 8 of 2^-24; y by less than 2^-16 of
itself before it is rounded.  bf16 rounding: 2^-8.  e4m3: half a step, 2^-4 of the value or
2^-10 of the scale."""
import math

import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ARITH = 2.0 ** -16
FORMS = [mxg.NORM_PLAIN, mxg.NORM_FP8_ROWWISE, mxg.NORM_MXFP8, mxg.NORM_FP8_BLOCK128]


def rand(seed, *shape, scale=1.0, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def outputs(S, H, form):
    q = None if form == mxg.NORM_PLAIN else torch.full((S, H), 0x5C, dtype=torch.uint8, device="cuda")
    scales = {mxg.NORM_PLAIN: None,
              mxg.NORM_FP8_ROWWISE: torch.full((S,), -1.0, device="cuda"),
              mxg.NORM_MXFP8: torch.full((S, H // 32), 7, dtype=torch.uint8, device="cuda"),
              mxg.NORM_FP8_BLOCK128: torch.full((S, -(-H // 128)), -1.0, device="cuda")}[form]
    return torch.full((S, H), -3.0, dtype=BF, device="cuda"), q, scales


def exact_y(h, w, offset, eps):
    h = h.double()
    return h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * (w.double() + offset)


def check_codes(y, q, scales, form):
    """Codes and scales of y (fp64), block by block."""
    S, H = y.shape
    size = {mxg.NORM_FP8_ROWWISE: H, mxg.NORM_MXFP8: 32, mxg.NORM_FP8_BLOCK128: 128}[form]
    got = q.view(torch.float8_e4m3fn).double()
    scales = scales.reshape(S, -1)
    for i, lo in enumerate(range(0, H, size)):
        part, code = y[:, lo:lo + size], got[:, lo:lo + size]
        top = part.abs().amax(1)
        if form == mxg.NORM_MXFP8:
            s = torch.exp2(scales[:, i].double() - 127)
            zero = scales[:, i] == 0
            # the largest magnitude lies in the scale's binade, but for its own error
            m = top / s / 256
            assert bool((((m >= 1 - 2 * ARITH) & (m < 2 * (1 + 2 * ARITH))) | zero).all())
        else:
            s = scales[:, i].double()
            assert bool(((s - top / 448).abs() <= 2 * ARITH * top / 448 + 2.0 ** -149).all())
        s = s[:, None]
        limit = part.abs() * (2.0 ** -4 + 2 * ARITH) + s * 2.0 ** -10
        # past the largest code the value saturates (MX: up to 511 of its scale)
        want = torch.minimum(torch.maximum(part, -448 * s), 448 * s)
        assert bool(((code * s - want).abs() <= limit + 2.0 ** -149).all())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("S,H,stream,residual,wtype,offset", [
    (1, 32, BF, True, BF, 0.0), (3, 128, BF, True, F32, 1.0), (5, 160, F32, True, BF, 0.0),
    (67, 512, BF, False, BF, 0.0), (33, 544, BF, True, BF, 1.0), (4, 2048, F32, False, F32, 0.0),
    (9, 2080, F32, True, BF, 1.0), (1, 7168, BF, True, BF, 0.0), (513, 4096, BF, True, BF, 0.0),
    (6, 4128, BF, False, BF, 0.0), (5, 8192, F32, True, BF, 0.0), (3, 8224, BF, True, BF, 0.0),
    (2, 32768, BF, True, BF, 0.0), (2, 32800, BF, True, BF, 0.0), (3, 33024, F32, False, F32, 1.0),
    (1100, 96, F32, True, BF, 0.0)])
def test_forward(S, H, stream, residual, wtype, offset, form):
    res = rand(1, S, H, scale=3.0, dtype=stream) if residual else None
    x = rand(2, S, H, dtype=BF if residual else stream)
    w = rand(3, H, scale=0.2, dtype=wtype)
    y, q, scales = outputs(S, H, form)
    h = torch.empty_like(res) if residual else None
    mxg.mx_rmsnorm(x, w, residual=res, h=h, y=y, form=form, q=q, scales=scales, eps=1e-5, weight_offset=offset)
    if residual:
        assert torch.equal(h, (x.float() + res.float()).to(stream))
    want = exact_y(h if residual else x, w, offset, 1e-5)
    assert bool(((y.double() - want).abs() <= want.abs() * (2.0 ** -8 + ARITH)).all())
    if q is not None:
        check_codes(want, q, scales, form)
        # without y the same codes
        q2, s2 = torch.empty_like(q), torch.empty_like(scales)
        mxg.mx_rmsnorm(x, w, residual=res, h=h, form=form, q=q2, scales=s2, eps=1e-5, weight_offset=offset)
        assert torch.equal(q, q2) and torch.equal(scales, s2)


@pytest.mark.parametrize("H", [8, 40, 8200, 32776])
def test_rows_of_eights(H):
    """Rows that are no multiple of 32 have the plain form."""
    x, w = rand(5, 7, H, dtype=BF), rand(6, H, dtype=BF)
    y = mxg.rmsnorm(x, w)[0]
    want = exact_y(x, w, 0.0, 1e-6)
    assert bool(((y.double() - want).abs() <= want.abs() * (2.0 ** -8 + ARITH)).all())


def test_in_place_and_allocating():
    S, H = 21, 320
    x, w, res = rand(1, S, H, dtype=BF), rand(2, H, dtype=BF), rand(3, S, H, dtype=BF)
    y, h, q, s = mxg.rmsnorm(x, w, res, mxg.NORM_FP8_BLOCK128)
    for target in ("residual", "x"):
        x2, res2, y2 = x.clone(), res.clone(), torch.empty_like(y)
        mxg.mx_rmsnorm(x2, w, residual=res2, h=res2 if target == "residual" else x2, y=y2)
        assert torch.equal(res2 if target == "residual" else x2, h) and torch.equal(y2, y)
        assert torch.equal(x2 if target == "residual" else res2, x if target == "residual" else res)
    res32 = res.float()
    y32, h32, _, _ = mxg.rmsnorm(x, w, res32)
    again, y3 = res32.clone(), torch.empty_like(y)
    mxg.mx_rmsnorm(x, w, residual=again, h=again, y=y3)
    assert torch.equal(again, h32) and torch.equal(y3, y32)


@pytest.mark.parametrize("form", FORMS)
def test_zero_and_non_finite_rows(form):
    H = 256
    x, w = rand(1, 6, H, dtype=BF), torch.ones(H, dtype=BF, device="cuda")
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, 200] = float("inf")
    x[3] = torch.finfo(BF).min          # squares pass fp32: r is 0
    x[4] = 1e-30                        # squares vanish: eps alone
    y, q, scales = outputs(6, H, form)
    mxg.mx_rmsnorm(x, w, y=y, form=form, q=q, scales=scales, eps=1e-6)
    assert torch.equal(y[0], torch.zeros_like(y[0])) and torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 200]) and torch.count_nonzero(y[2].nan_to_num(0.0)) == 0
    assert torch.count_nonzero(y[3]) == 0
    assert bool(((y[4].double() - x[4].double() * 1e3).abs() <= x[4].double().abs() * 1e3 * (2.0 ** -8 + ARITH)).all())
    if form == mxg.NORM_PLAIN:
        return
    v = q.view(torch.float8_e4m3fn).float()
    assert torch.count_nonzero(v[0]) == 0 and torch.isnan(v[1]).all()
    assert torch.isnan(v[2, 200]) and torch.count_nonzero(v[3]) == 0
    if form == mxg.NORM_MXFP8:
        assert bool((scales[1] == 255).all()) and scales[2].tolist() == [0] * 6 + [255] + [0]
        assert bool((scales[0] == 0).all())
    else:
        s = scales.reshape(6, -1)
        assert torch.isnan(s[1]).all() and torch.isnan(s[2, -1]) and bool((s[0] == 0).all())
    check_codes(exact_y(x[5:], w, 0.0, 1e-6), q[5:], scales[5:], form)


def test_eps_zero():
    x, w = rand(1, 2, 64, scale=1e-3, dtype=BF), torch.ones(64, dtype=BF, device="cuda")
    want = exact_y(x, w, 0.0, 0.0)
    y = mxg.rmsnorm(x, w, eps=0.0)[0]
    assert bool(((y.double() - want).abs() <= want.abs() * (2.0 ** -8 + ARITH)).all())


def exact_grad(dy, h, w, offset, eps, dh):
    h, dy = h.double(), dy.double()
    r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    g = dy * (w.double() + offset)
    dot, mags = (g * h).mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
    dx = r * g - h * r ** 3 * dot
    size = (r * g).abs() + h.abs() * r ** 3 * mags  # of the terms that dx is made of
    if dh is not None:
        dx, size = dx + dh.double(), size + dh.double().abs()
    return dx, size, (dy * h * r).sum(0), (dy * h * r).abs().sum(0)


@pytest.mark.parametrize("S,H,stream,wtype,offset,past", [
    (1, 8, BF, BF, 0.0, True), (3, 128, BF, F32, 1.0, False), (700, 160, F32, BF, 0.0, True),
    (67, 512, BF, BF, 0.0, True), (33, 1544, BF, BF, 1.0, True), (4, 2048, F32, F32, 0.0, False),
    (9, 2080, F32, BF, 1.0, True), (1, 7168, BF, BF, 0.0, True), (600, 4096, BF, BF, 0.0, True),
    (5, 8192, F32, BF, 0.0, True), (3, 8200, BF, BF, 0.0, True), (2, 16384, F32, BF, 0.0, True),
    (520, 16392, BF, BF, 0.0, True), (3, 32776, F32, F32, 1.0, False)])
def test_backward(S, H, stream, wtype, offset, past):
    h, dy, w = rand(1, S, H, scale=2.0, dtype=stream), rand(2, S, H, dtype=BF), rand(3, H, scale=0.3, dtype=wtype)
    dh = rand(4, S, H, dtype=stream) if past else None
    dx = torch.full((S, H), 9.0, dtype=stream, device="cuda")
    dx16 = torch.full((S, H), 9.0, dtype=BF, device="cuda")
    dw = torch.full((H,), 9.0, device="cuda")
    ws = torch.full((mxg.rmsnorm_workspace_bytes(S, H) // 4,), float("nan"), device="cuda")
    mxg.mx_rmsnorm_backward(dy, h, w, dx, dh=dh, dx_bf16=dx16, dweight=dw, workspace=ws, eps=1e-5,
                            weight_offset=offset)
    want, size, want_w, size_w = exact_grad(dy, h, w, offset, 1e-5, dh)
    half = torch.finfo(stream).eps / 2
    assert bool(((dx.double() - want).abs() <= want.abs() * half + size * 4 * ARITH).all())
    assert bool(((dx16.double() - want).abs() <= want.abs() * 2.0 ** -8 + size * 4 * ARITH).all())
    assert bool(((dw.double() - want_w).abs() <= size_w * (ARITH + (S + 32) * 2.0 ** -24)).all())
    # each output by itself, dx in place of dh, a workspace of torch's: the same bits
    only = torch.empty_like(dw)
    mxg.mx_rmsnorm_backward(dy, h, w, dweight=only, eps=1e-5, weight_offset=offset)
    assert torch.equal(only, dw)
    place = dh.clone() if past else torch.empty_like(dx)
    mxg.mx_rmsnorm_backward(dy, h, w, place, dh=place if past else None, eps=1e-5, weight_offset=offset)
    assert torch.equal(place, dx)
    only16 = torch.empty_like(dx16)
    mxg.mx_rmsnorm_backward(dy, h, w, dh=dh, dx_bf16=only16, eps=1e-5, weight_offset=offset)
    assert torch.equal(only16, dx16)


def test_gradient_against_differences():
    """Central differences of the forward's formula in 64 bits along random directions: their own error, of second
    order, stays below 1e-6 of the derivative's terms at a step of 1e-4 on values near 1."""
    S, H, step = 4, 96, 1e-4
    h, dy, w = rand(1, S, H), rand(2, S, H, dtype=BF), rand(3, H, scale=0.5) + 1.0
    dx, dw = torch.empty_like(h), torch.empty_like(w)
    mxg.mx_rmsnorm_backward(dy, h, w, dx, dweight=dw, eps=1e-3)

    def loss(hh, ww):
        return (dy.double() * (hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + 1e-3) * ww)).sum(1)

    vh, vw = rand(4, S, H).double(), rand(5, H).double()
    hd, wd = h.double(), w.double()
    along = (loss(hd + step * vh, wd) - loss(hd - step * vh, wd)) / (2 * step)
    size = (dx.double() * vh).abs().sum(1)
    assert bool(((along - (dx.double() * vh).sum(1)).abs() <= size * 2.0 ** -13 + 1e-4).all())
    along = ((loss(hd, wd + step * vw) - loss(hd, wd - step * vw)) / (2 * step)).sum()
    assert abs(float(along - (dw.double() * vw).sum())) <= float((dw.double() * vw).abs().sum()) * 2.0 ** -13


def test_no_tokens():
    w = torch.ones(64, dtype=BF, device="cuda")
    x, dw = torch.empty((0, 64), dtype=BF, device="cuda"), torch.full((64,), 5.0, device="cuda")
    assert mxg.rmsnorm(x, w)[0].shape == (0, 64)
    mxg.mx_rmsnorm_backward(x, x, w, torch.empty_like(x), dweight=dw)
    assert torch.count_nonzero(dw) == 0


def test_refusals():
    x, w = rand(1, 4, 64, dtype=BF), rand(2, 64, dtype=BF)
    y, q, s = outputs(4, 64, mxg.NORM_MXFP8)
    ok = dict(y=y)
    bad = [dict(y=y, q=q, scales=s), dict(y=y, form=mxg.NORM_MXFP8), dict(y=y, form=mxg.NORM_MXFP8, q=q), dict(),
           dict(y=x), dict(y=y, residual=x), dict(y=y, residual=x, h=y), dict(y=y, h=y),
           dict(y=y.float()), dict(y=y[:, :32])]
    for args in bad:
        with pytest.raises((ValueError, TypeError, mxg.MxgError)):
            mxg.mx_rmsnorm(x, w, **args)
    for args in (dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(mxg.MxgError):
            mxg.mx_rmsnorm(x, w, **ok, **args)
    with pytest.raises((ValueError, TypeError)):
        mxg.mx_rmsnorm(x.float(), w, y=y, residual=x, h=torch.empty_like(x))
    with pytest.raises(mxg.MxgError):  # rows of 40: no 8-bit form
        x2 = rand(1, 2, 40, dtype=BF)
        mxg.mx_rmsnorm(x2, w[:40].clone(), form=mxg.NORM_FP8_BLOCK128,
                       q=torch.empty((2, 40), dtype=torch.uint8, device="cuda"), scales=torch.empty((2, 1), device="cuda"))
    for args in (dict(), dict(dx=x), dict(dx=y, dh=y.float()), dict(dweight=torch.empty(64, device="cuda"),
                                                                     workspace=torch.empty(63, device="cuda"))):
        with pytest.raises((ValueError, TypeError, mxg.MxgError)):
            mxg.mx_rmsnorm_backward(y, x, w, **args)
    mxg.mx_rmsnorm(x, w, **ok)
    assert math.isfinite(float(y.float().sum()))


def test_graph_and_streams():
    """Captured and replayed with other inputs and eager work between, on a stream of its own."""
    S, H = 40, 1056
    bufs = dict(x=rand(1, S, H, dtype=BF), res=rand(2, S, H), w=rand(3, H, dtype=BF), dy=rand(4, S, H, dtype=BF))

    def step(o):
        mxg.mx_rmsnorm(bufs["x"], bufs["w"], residual=bufs["res"], h=o["h"], y=o["y"], form=mxg.NORM_FP8_BLOCK128,
                       q=o["q"], scales=o["s"])
        mxg.mx_rmsnorm_backward(bufs["dy"], o["h"], bufs["w"], o["dx"], dx_bf16=o["dx16"], dweight=o["dw"],
                                workspace=o["ws"])

    def fresh():
        y, q, s = outputs(S, H, mxg.NORM_FP8_BLOCK128)
        return dict(h=rand(9, S, H), y=y, q=q, s=s, dx=rand(8, S, H), dx16=torch.empty_like(y), dw=rand(7, H),
                    ws=torch.empty(mxg.rmsnorm_workspace_bytes(S, H) // 4, device="cuda"))

    cap, eager = fresh(), fresh()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(cap)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cap)
    for i in range(3):
        bufs["x"].copy_(rand(20 + i, S, H, dtype=BF))
        bufs["dy"].copy_(rand(30 + i, S, H, dtype=BF))
        graph.replay()
        step(eager)
        torch.cuda.synchronize()
        for k in eager:
            if k != "ws":
                assert torch.equal(cap[k], eager[k]), k


def test_rows_past_4_gib():
    """The last rows of every operand of two bytes an element lie past 2^32 bytes; each row is its own."""
    S, H, n = 600100, 4096, 100
    x, res = (torch.zeros((S, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x[-n:], res[-n:] = rand(1, n, H), rand(2, n, H)
    w = rand(3, H)
    h, y = torch.ones_like(x), torch.ones_like(x)
    q = torch.ones((S, H), dtype=torch.uint8, device="cuda")
    sc = torch.ones((S, H // 128), dtype=torch.float32, device="cuda")
    mxg.mx_rmsnorm(x, w, residual=res, h=h, y=y, form=mxg.NORM_FP8_BLOCK128, q=q, scales=sc, eps=1e-5)
    part = [torch.empty_like(t[:n]) for t in (h, y, q, sc)]
    mxg.mx_rmsnorm(x[-n:].clone(), w, residual=res[-n:].clone(), h=part[0], y=part[1], form=mxg.NORM_FP8_BLOCK128,
                   q=part[2], scales=part[3], eps=1e-5)
    for whole, tail in zip((h, y, q, sc), part):
        assert torch.equal(whole[-n:], tail)
        rest = whole[:-n]
        if whole is q:  # 0 under a negative weight is -0, whose code keeps the sign
            assert bool((rest == ((w < 0).to(torch.uint8) << 7)).all())
        else:
            assert torch.count_nonzero(rest) == 0
    del y, q, sc, res
    dw, dx = torch.empty(H, device="cuda"), torch.ones_like(x)
    mxg.mx_rmsnorm_backward(x, h, w, dx, dweight=dw, eps=1e-5)
    dw_tail, dx_tail = torch.empty(H, device="cuda"), torch.empty_like(x[:n])
    mxg.mx_rmsnorm_backward(x[-n:].clone(), h[-n:].clone(), w, dx_tail, dweight=dw_tail, eps=1e-5)
    assert torch.equal(dx[-n:], dx_tail) and torch.count_nonzero(dx[:-n]) == 0
    hh = h[-n:].double()
    terms = x[-n:].double() * hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + 1e-5)
    # n terms of four fp32 roundings and r's, added by workgroup and then by at most 512 partial sums
    bound = (n + 512 + 40) * 2.0 ** -23 * terms.abs().sum(0)
    assert bool(((dw.double() - terms.sum(0)).abs() <= bound).all())
    assert bool(((dw_tail.double() - terms.sum(0)).abs() <= bound).all())
