"""The workspace of the norm's gradient on 4 bytes: the results have the bits of those with one on 16, and nothing
beside it is written."""
import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg

pytestmark = pytest.mark.gpu


def rand(seed, *shape, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S,H", [(1, 8), (700, 160), (3, 1544), (530, 4096), (5, 8200), (600, 16392)])
def test_workspace_on_4_bytes(S, H, stream):
    dy, h, w = rand(1, S, H, dtype=torch.bfloat16), rand(2, S, H, dtype=stream), rand(3, H, dtype=torch.bfloat16)
    dx, dw = torch.empty_like(h), torch.empty(H, device="cuda")
    mxg.mx_rmsnorm_backward(dy, h, w, dx, dweight=dw)
    n = mxg.rmsnorm_workspace_bytes(S, H) // 4
    for shift in (1, 2, 3):
        ws = torch.full((n + 8,), -7.0, device="cuda")
        assert ws.data_ptr() % 16 == 0
        dx2, dw2 = torch.empty_like(h), torch.empty(H, device="cuda")
        mxg.mx_rmsnorm_backward(dy, h, w, dx2, dweight=dw2, workspace=ws[shift:shift + n])
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
        assert bool((ws[:shift] == -7.0).all()) and bool((ws[shift + n:] == -7.0).all())
