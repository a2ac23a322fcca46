"""The norm's gradient where its arithmetic is exact: a stream of ones and minus ones without eps has r = 1, and with
small whole numbers in dy and the weight every sum is a whole number below 2^24, whatever its order.  A row that is lost
or taken twice shows at any number of rows, where a bound of rounding errors grows with it."""
import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg

pytestmark = pytest.mark.gpu


def signs(seed, *shape, most=1, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    v = torch.randint(1, most + 1, shape, generator=g, device="cuda")
    return (v * (2 * torch.randint(0, 2, shape, generator=g, device="cuda") - 1)).to(dtype)


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S,H", [(1, 8), (511, 128), (512, 512), (513, 1024), (100003, 256), (20001, 2048), (8191, 8192),
                                 (3001, 16384), (2049, 32768), (1025, 65536)])
def test_weight_and_rows(S, H, stream):
    h, dy, w = signs(1, S, H, dtype=stream), signs(2, S, H, most=3), signs(3, H, most=3)
    dx, dw = torch.empty_like(h), torch.empty(H, device="cuda")
    mxg.mx_rmsnorm_backward(dy, h, w, dx, dweight=dw, eps=0.0)
    want = torch.zeros(H, dtype=torch.float64, device="cuda")
    for lo in range(0, S, 4096):
        want += (dy[lo:lo + 4096].double() * h[lo:lo + 4096].double()).sum(0)
    assert torch.equal(dw.double(), want)
    # H is a power of two, so the row's sum over H is exact too, and one rounding at most is left in fp32, one in bf16
    half = torch.finfo(stream).eps / 2
    for lo in range(0, S, 4096):
        g, hh = dy[lo:lo + 4096].double() * w.double(), h[lo:lo + 4096].double()
        rows = g - hh * (g * hh).mean(1, keepdim=True)
        off = (dx[lo:lo + 4096].double() - rows).abs()
        assert bool((off <= (half + 2.0 ** -24) * rows.abs() * (1 + half)).all())
