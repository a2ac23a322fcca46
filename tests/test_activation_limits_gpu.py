"""The activations and their derivatives where they run out of range: far below zero and at infinities.  Bounds: fp32
arithmetic of 2^-18 of a value; silu and its derivative below 2^-121 may be 0."""
import math

import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg

pytestmark = pytest.mark.gpu

INF = math.inf
Z = [0.0, -1.0, -40.0, -86.5, -88.5, -89.0, -91.0, -104.0, -1000.0, -3e38, 40.0, 89.0, 1000.0, 3e38, INF, -INF]


def forward(act, z):
    """act of z in fp32: the product of nothing and a bias of z."""
    zero = torch.zeros((1, 8), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros((1, z.numel(), 8), dtype=torch.bfloat16, device="cuda")
    return mxg.grouped_matmul_bf16(zero, b, bias=z[None], act=act, dtype=torch.float32)[0].double()


def test_forward():
    z = torch.tensor(Z, device="cuda")
    e = z.double()
    finite = torch.isfinite(z)
    silu, gelu = forward(mxg.ACT_SILU, z), forward(mxg.ACT_GELU, z)
    want = e / (1 + torch.exp(-e))
    assert bool(((silu - want).abs() <= 2.0 ** -18 * want.abs() + (e < -88.7) * 2.0 ** -121 + 1e-38)[finite].all())
    want = e * torch.special.ndtr(e)
    assert bool(((gelu - want).abs() <= 2.0 ** -18 * want.abs() + 1e-38)[finite].all())
    for got in (silu, gelu):
        assert got[-2] == INF and torch.isnan(got[-1])
    pairs = torch.stack((z, torch.full_like(z, 2.0)), 1).flatten()
    got = forward(mxg.ACT_SWIGLU, pairs)
    twice = (2 * silu[:-1]).float().double()  # exact, but for 6e38, which is past fp32's range: infinity
    assert torch.equal(got[:-1], twice) and torch.isnan(got[-1])


def test_derivatives():
    z = torch.tensor(Z, device="cuda").to(torch.bfloat16).view(1, -1)
    d = torch.ones_like(z)
    e = z.double()
    finite = torch.isfinite(z)
    s = 1 / (1 + torch.exp(-e))
    for act, want, size in ((mxg.ACT_SILU, s * (1 + e * (1 - s)), s + e.abs() * s),
                            (mxg.ACT_GELU, torch.special.ndtr(e) + e * torch.exp(-e * e / 2) / math.sqrt(2 * math.pi),
                             torch.ones_like(e))):
        got = torch.empty_like(z)
        mxg.mx_activation_backward(act, d, z, got)
        off = (got.double() - want).abs()
        assert bool((off <= 2.0 ** -18 * size + 2.0 ** -8 * want.abs() + 2.0 ** -121)[finite].all())
        assert torch.isnan(got[0, -2:]).all()
