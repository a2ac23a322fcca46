"""The operators together, as a layer uses them: the router's choice, the routing
plan, the token-major quantise, the gate/up product, SwiGLU with its requant, the
down product and the combine; then the gradient of the whole layer back to the
tokens and to the router's logits, through the quantised experts.

Against fp64 on the library's own quantised operands the only errors are the
bf16 and e4m3 roundings between the steps, which differ from one step's operand
to the next; each step is therefore compared on its own inputs as it ran, and
the layer's gradient against the same chain of exact steps.  Captured in a graph
the layer gives the eager step's bits at every replay."""
import numpy as np
import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg

pytestmark = pytest.mark.gpu

S, E, K_TOP, H, I = 200, 12, 4, 416, 288   # neither width a multiple of 128


def blocks(n):
    return -(-n // 128)


class Layer:
    """Quantised experts and every buffer of one step, forward and backward."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.w13 = mxg.quantize_weights_block128(
            (torch.randn((E, 2 * I, H), generator=g, device="cuda") * 0.05).to(torch.bfloat16), True)
        self.w2 = mxg.quantize_weights_block128(
            (torch.randn((E, H, I), generator=g, device="cuda") * 0.05).to(torch.bfloat16), True)
        self.bias = torch.randn(E, generator=g, device="cuda") * 0.1
        self.expert_ids = torch.arange(E, dtype=torch.int32, device="cuda")
        self.x, self.logits, self.dout = self.inputs(seed + 1)
        T = S * K_TOP
        e = lambda shape, dt: torch.zeros(shape, dtype=dt, device="cuda")  # noqa: E731
        i32, f32, u8, bf = torch.int32, torch.float32, torch.uint8, torch.bfloat16
        self.ids, self.wt = e((S, K_TOP), i32), e((S, K_TOP), f32)
        self.off, self.ros, self.sor = e(E + 1, i32), e(T, i32), e(T, i32)
        self.xq, self.xs = e((T, H), u8), e((T, blocks(H)), f32)
        self.h, self.yq, self.ys = e((T, 2 * I), bf), e((T, I), u8), e((T, blocks(I)), f32)
        self.y, self.out = e((T, H), bf), e((S, H), bf)
        self.dy, self.dwt = e((T, H), bf), e((S, K_TOP), f32)
        self.dyq, self.dys = e((T, H), u8), e((T, blocks(H)), f32)
        self.da, self.dhq, self.dhs = e((T, I), bf), e((T, 2 * I), u8), e((T, blocks(2 * I)), f32)
        self.drows, self.dx, self.dlogits = e((T, H), bf), e((S, H), bf), e((S, E), f32)

    @staticmethod
    def inputs(seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        x = torch.randn((S, H), generator=g, device="cuda").to(torch.bfloat16)
        logits = torch.randn((S, E), generator=g, device="cuda")
        logits[:, 3] = -float("inf")     # an expert nobody may take
        logits[5] = -float("inf")        # a token that no expert takes
        logits[6, 2:] = -float("inf")    # one with fewer experts than slots
        return x, logits, (torch.randn((S, H), generator=g, device="cuda") * 0.1).to(torch.bfloat16)

    def step(self):
        m = mxg
        m.mx_moe_topk(m.SCORE_SIGMOID, self.logits, self.ids, self.wt, self.bias, True, 1.5)
        m.mx_moe_sort(self.ids, self.off, self.ros, self.sor)
        m.mx_grouped_quantize_block128_scatter(self.x, self.ros, self.xq, self.xs, self.off)
        m.mx_grouped_matmul_block128(self.xq, self.xs, self.w13[0], self.w13[1], self.h, self.off, self.expert_ids)
        m.mx_silu_quantize_block128(self.h, self.yq, self.ys, self.off)
        m.mx_grouped_matmul_block128(self.yq, self.ys, self.w2[0], self.w2[1], self.y, self.off, self.expert_ids)
        m.mx_moe_combine(self.y, self.ros, self.wt.view(-1), self.out)
        # the gradient
        m.mx_moe_combine_backward(self.dout, self.y, self.ros, self.wt.view(-1), self.dy, self.dwt.view(-1))
        m.mx_moe_topk_backward(m.SCORE_SIGMOID, self.logits, self.ids, self.dwt, self.dlogits, True, 1.5)
        m.mx_grouped_quantize_block128(self.dy, self.dyq, self.dys, self.off)
        m.mx_grouped_matmul_block128(self.dyq, self.dys, self.w2[2], self.w2[3], self.da, self.off, self.expert_ids)
        m.mx_silu_backward_block128(self.h, self.da, self.off, dh_q=self.dhq, dh_scales=self.dhs)
        m.mx_grouped_matmul_block128(self.dhq, self.dhs, self.w13[2], self.w13[3], self.drows, self.off,
                                     self.expert_ids)
        m.mx_moe_permute_backward(self.drows, self.ros, self.dx)

    def outputs(self):
        return [self.ids, self.wt, self.off, self.ros, self.sor, self.out, self.dx, self.dlogits]


def value(q, s, transposed_tile=False):
    """fp64 values of block-scaled codes (activations, or weights where s has their tiles)."""
    v = q.view(torch.float8_e4m3fn).double()
    wide = s.double().repeat_interleave(128, -1)[..., :q.shape[-1]]
    if transposed_tile:
        wide = wide.repeat_interleave(128, -2)[..., :q.shape[-2], :]
    return v * wide


def grouped(a, w, off):
    out = torch.zeros((a.shape[0], w.shape[1]), dtype=torch.float64, device="cuda")
    for e in range(E):
        out[off[e]:off[e + 1]] = a[off[e]:off[e + 1]] @ w[e].t()
    return out


def near(got, want, rel, rows=None):
    """Within rel of the row's largest magnitude (the sums run over a whole row)."""
    got, want = got.double(), want.double()
    if rows is not None:
        got, want = got[:rows], want[:rows]
    top = want.abs().amax(1, keepdim=True)
    assert bool(((got - want).abs() <= rel * top + 1e-30).all()), float(((got - want).abs() / (top + 1e-30)).max())


def test_layer_forward_and_gradient():
    L = Layer(1)
    L.step()
    torch.cuda.synchronize()
    off = L.off.tolist()
    n = off[E]
    assert n == S * K_TOP - K_TOP - (K_TOP - 2)  # a token without experts, one with two
    assert L.ids[5].tolist() == [-1] * 4 and L.wt[5].tolist() == [0.0] * 4 and (L.ids != 3).all()
    assert torch.count_nonzero(L.out[5]) == 0 and torch.count_nonzero(L.dx[5]) == 0
    assert torch.count_nonzero(L.dlogits[5]) == 0 and torch.count_nonzero(L.dlogits[:, 3]) == 0
    w13, w2 = value(L.w13[0], L.w13[1], True), value(L.w2[0], L.w2[1], True)
    # each step on the inputs it had: bf16 half steps, or for the products that and
    # the matrix core's cuts (2^-9 of the eights' largest products, under the row's largest)
    tok = (L.sor[:n] // K_TOP).long()
    near(value(L.xq, L.xs)[:n], L.x[tok], 2.0 ** -4)
    near(L.h, grouped(value(L.xq, L.xs), w13, off), 2.0 ** -7, n)
    h = L.h.double()
    g, u = h[:, 0::2], h[:, 1::2]
    sg = torch.sigmoid(g)
    near(value(L.yq, L.ys), g * sg * u, 2.0 ** -4, n)
    near(L.y, grouped(value(L.yq, L.ys), w2, off), 2.0 ** -7, n)
    near(L.da, grouped(value(L.dyq, L.dys), w2.transpose(1, 2), off), 2.0 ** -7, n)
    da = L.da.double()
    dh = torch.stack((da * u * sg * (1 + g * (1 - sg)), da * g * sg), 2).reshape(h.shape)
    near(value(L.dhq, L.dhs), dh, 2.0 ** -4, n)
    near(L.drows, grouped(value(L.dhq, L.dhs), w13.transpose(1, 2), off), 2.0 ** -7, n)
    # rows behind the last routed one stay as they were
    for t in (L.xq, L.xs, L.h, L.yq, L.y, L.dy, L.dyq, L.da, L.dhq, L.drows):
        assert torch.count_nonzero(t[n:].float()) == 0


def test_layer_gradient_against_differences():
    """The layer's gradient along random directions of the router's logits, by
    differences of the layer itself in 64 bits on the same choice and the same
    quantised rows (the path logits -> weights -> combine is exact there); what
    the library rounds on it is y (shared by both sides) and fp32 sums."""
    L = Layer(2)
    L.step()
    torch.cuda.synchronize()
    y, ros, ids = L.y.double(), L.ros.view(S, K_TOP).long(), L.ids.long()
    live = ids >= 0

    def loss(x):
        ls = torch.where(live, torch.nn.functional.logsigmoid(x).gather(1, ids.clamp_min(0)), -torch.inf)
        w = torch.where(live.any(1, keepdim=True), torch.softmax(ls, 1), 0.0) * 1.5
        rows = torch.where(live[..., None], y[ros.clamp_min(0)], 0.0)
        return ((rows * w.nan_to_num()[..., None]).sum(1) * L.dout.double()).sum(1)

    x = torch.where(torch.isinf(L.logits), -1e3, L.logits.double())
    v = torch.randn(S, E, dtype=torch.float64, device="cuda")
    num = (loss(x + 1e-4 * v) - loss(x - 1e-4 * v)) / 2e-4
    got = (L.dlogits.double() * v).sum(1)
    scale = (L.dlogits.double().abs() * v.abs()).sum(1)
    assert bool(((got - num).abs() <= 1e-4 * scale + 1e-6).all())


def test_layer_in_a_graph():
    L = Layer(3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        L.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.step()
    eager = Layer(3)
    for rep in range(4):
        x, logits, dout = Layer.inputs(100 + rep)
        for lay in (L, eager):
            lay.x.copy_(x), lay.logits.copy_(logits), lay.dout.copy_(dout)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in L.outputs()]
        eager.step()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, eager.outputs())):
            assert torch.equal(a, b), (rep, i)


def test_two_layers_on_two_streams():
    """Two steps at once on two streams, against each alone: no state is shared."""
    alone = []
    for seed in (4, 5):
        L = Layer(seed)
        L.step()
        torch.cuda.synchronize()
        alone.append([t.clone() for t in L.outputs()])
    layers = [Layer(4), Layer(5)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for L, st in zip(layers, streams):
            with torch.cuda.stream(st):
                L.step()
    torch.cuda.synchronize()
    for L, want in zip(layers, alone):
        for a, b in zip(L.outputs(), want):
            assert torch.equal(a, b)
