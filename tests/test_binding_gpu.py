"""The binding's two ways to the current device and stream: torch's raw handles, and the
public calls that stand in where a torch build lacks them."""
import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("public", [False, True])
def test_calls_go_to_the_current_stream(monkeypatch, public):
    if public:
        monkeypatch.setattr(mxg, "_raw_stream", mxg._current_stream)
        monkeypatch.setattr(mxg, "_current_device", torch.cuda.current_device)
    index = torch.cuda.current_device()
    side = torch.cuda.Stream()
    assert mxg._current_device() == index
    assert mxg._raw_stream(index) == torch.cuda.current_stream().cuda_stream
    ids = torch.randint(0, 50, (20000, 4), dtype=torch.int32, device="cuda")
    want = mxg.moe_sort(ids, 50)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert mxg._raw_stream(index) == side.cuda_stream
        shuffled = ids.flip(0).contiguous()  # written on this stream just before the call reads it
        back = mxg.moe_sort(shuffled.flip(0).contiguous(), 50)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, back):
        assert torch.equal(a, b)
