"""The operators together, as a layer trained in BF16 uses them: the norm with the residual's addition, the
router's logits, choice and plan, the routed experts' gate/up and down products, the combine, a shared
expert whose down product adds it all up; then the gradient of the layer back to the stream, the norm's
weight, the router and every expert's weights and biases.

Against the same layer in 64 bits (autograd) on the choice that was made.  Between a leaf and a gradient lie
at most twelve roundings to bf16, each off by 2^-8 at most and by 2^-8 / sqrt 3 in the root mean square, of
values of which each enters the gradient once or, through a norm or a softmax, twice: the root mean square
of their sum is below sqrt(24) 2^-8 / sqrt 3 = 1.2 %, and 3 % of a gradient's norm is the bound.  Captured
in a graph the layer gives the eager step's bits at every replay."""
import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg

pytestmark = pytest.mark.gpu

S, E, K_TOP, H, I, SHARED = 160, 8, 2, 256, 136, 200
T = S * K_TOP
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
EPS = 1e-5


def rand(seed, *shape, scale=1.0, dtype=BF):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


class Layer:
    def __init__(self, seed):
        self.norm = (1 + rand(seed, H, scale=0.1, dtype=F32)).to(BF)
        self.wr, self.br = rand(seed + 1, 1, E, H, scale=0.06), rand(seed + 2, 1, E, scale=0.1, dtype=F32)
        self.w13, self.b13 = rand(seed + 3, E, 2 * I, H, scale=0.06), rand(seed + 4, E, 2 * I, scale=0.1, dtype=F32)
        self.w2 = rand(seed + 5, E, H, I, scale=0.08)
        self.s13, self.s2 = rand(seed + 6, 1, 2 * SHARED, H, scale=0.06), rand(seed + 7, 1, H, SHARED, scale=0.07)
        self.x, self.res, self.dout = rand(seed + 8, S, H), rand(seed + 9, S, H, scale=2.0, dtype=F32), rand(seed + 10, S, H)
        self.expert_ids = torch.arange(E, dtype=I32, device="cuda")
        e = lambda shape, dt=BF: torch.zeros(shape, dtype=dt, device="cuda")  # noqa: E731
        self.h, self.y, self.q, self.qs = e((S, H), F32), e((S, H)), e((S, H), torch.uint8), e((S, H // 128), F32)
        self.logits, self.ids, self.wt = e((S, E)), e((S, K_TOP), I32), e((S, K_TOP), F32)
        self.off, self.ros, self.sor = e(E + 1, I32), e(T, I32), e(T, I32)
        self.rows, self.z, self.a, self.down = e((T, H)), e((T, 2 * I)), e((T, I)), e((T, H))
        self.out, self.zs, self.sa = e((S, H)), e((S, 2 * SHARED)), e((S, SHARED))
        self.dz, self.ds, self.ddown, self.drows = e((T, 2 * I)), e((S, 2 * SHARED)), e((T, H)), e((T, H))
        self.dwt, self.dlogits = e((S, K_TOP), F32), e((S, E))
        self.dy1, self.dy2, self.dy3 = e((S, H)), e((S, H)), e((S, H))
        self.dres, self.dx, self.dnorm = e((S, H), F32), e((S, H)), e(H, F32)
        self.dwr, self.dbr = e((1, E, H), F32), e((1, E), F32)
        self.dw13, self.db13, self.dw2 = e((E, 2 * I, H), F32), e((E, 2 * I), F32), e((E, H, I), F32)
        self.ds13, self.ds2 = e((1, 2 * SHARED, H), F32), e((1, H, SHARED), F32)
        self.ws = e(mxg.rmsnorm_workspace_bytes(S, H) // 4, F32)

    def step(self):
        m = mxg
        m.mx_rmsnorm(self.x, self.norm, residual=self.res, h=self.h, y=self.y, form=m.NORM_FP8_BLOCK128, q=self.q,
                     scales=self.qs, eps=EPS)
        m.mx_grouped_matmul_bf16(self.y, self.wr, self.logits, bias=self.br)
        m.mx_moe_topk(m.SCORE_SOFTMAX, self.logits, self.ids, self.wt)
        m.mx_moe_sort(self.ids, self.off, self.ros, self.sor)
        m.mx_moe_permute(self.y, self.ros, self.rows)
        m.mx_grouped_matmul_bf16(self.rows, self.w13, self.a, self.off, self.expert_ids, bias=self.b13,
                                 act=m.ACT_SWIGLU, z=self.z)
        m.mx_grouped_matmul_bf16(self.a, self.w2, self.down, self.off, self.expert_ids)
        m.mx_moe_combine(self.down, self.ros, self.wt.view(-1), self.out)
        m.mx_grouped_matmul_bf16(self.y, self.s13, self.sa, act=m.ACT_SWIGLU, z=self.zs)
        m.mx_grouped_matmul_bf16(self.sa, self.s2, self.out, residual=self.out)
        # the gradient
        m.mx_grouped_matmul_bf16_backward(self.dout, self.s2, self.ds, act=m.ACT_SWIGLU, z=self.zs)
        m.mx_grouped_matmul_bf16_backward_weights(self.dout, self.sa, self.ds2)
        m.mx_grouped_matmul_bf16_backward(self.ds, self.s13, self.dy1)
        m.mx_grouped_matmul_bf16_backward_weights(self.ds, self.y, self.ds13)
        m.mx_moe_combine_backward(self.dout, self.down, self.ros, self.wt.view(-1), self.ddown, self.dwt.view(-1))
        m.mx_grouped_matmul_bf16_backward(self.ddown, self.w2, self.dz, self.off, self.expert_ids, act=m.ACT_SWIGLU,
                                          z=self.z)
        m.mx_grouped_matmul_bf16_backward_weights(self.ddown, self.a, self.dw2, self.off, self.expert_ids)
        m.mx_grouped_matmul_bf16_backward(self.dz, self.w13, self.drows, self.off, self.expert_ids)
        m.mx_grouped_matmul_bf16_backward_weights(self.dz, self.rows, self.dw13, self.off, self.expert_ids,
                                                  dbias=self.db13)
        m.mx_moe_permute_backward(self.drows, self.ros, self.dy2)
        m.mx_moe_topk_backward(m.SCORE_SOFTMAX, self.logits, self.ids, self.dwt, self.dlogits)
        m.mx_grouped_matmul_bf16_backward(self.dlogits, self.wr, self.dy3)
        m.mx_grouped_matmul_bf16_backward_weights(self.dlogits, self.y, self.dwr, dbias=self.dbr)
        dy = (self.dy1.float() + self.dy2.float() + self.dy3.float()).to(BF)
        m.mx_rmsnorm_backward(dy, self.h, self.norm, self.dres, dx_bf16=self.dx, dweight=self.dnorm, workspace=self.ws,
                              eps=EPS)

    def outputs(self):
        return dict(out=self.out, logits=self.logits, ids=self.ids, q=self.q, dres=self.dres, dx=self.dx,
                    dnorm=self.dnorm, dwr=self.dwr, dbr=self.dbr, dw13=self.dw13, db13=self.db13, dw2=self.dw2,
                    ds13=self.ds13, ds2=self.ds2)


def exact(L):
    """The layer's output and gradients in 64 bits."""
    leaves = {k: getattr(L, k).double().cpu().requires_grad_() for k in
              ("x", "res", "norm", "wr", "br", "w13", "b13", "w2", "s13", "s2")}
    v = leaves
    h = v["x"] + v["res"]
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * v["norm"]
    logits = y @ v["wr"][0].T + v["br"][0]
    ids = L.ids.cpu().long()
    p = torch.softmax(logits, 1).gather(1, ids)
    w = p / p.sum(1, keepdim=True)

    def swiglu(z):
        return torch.nn.functional.silu(z[:, 0::2]) * z[:, 1::2]

    rows = []
    for k in range(K_TOP):
        parts = torch.zeros((S, H), dtype=torch.float64)
        for e in range(E):
            t = (ids[:, k] == e).nonzero()[:, 0]
            d = swiglu(y[t] @ v["w13"][e].T + v["b13"][e]) @ v["w2"][e].T
            parts = parts.index_add(0, t, d)
        rows.append(w[:, k:k + 1] * parts)
    out = sum(rows) + swiglu(y @ v["s13"][0].T) @ v["s2"][0].T
    (out * L.dout.double().cpu()).sum().backward()
    return out.detach(), {k: t.grad for k, t in leaves.items()}


def near(got, want):
    got = got.double().cpu()
    assert float((got - want).norm()) <= 0.03 * float(want.norm()), float((got - want).norm() / want.norm())


def test_layer_forward_and_gradient():
    L = Layer(1)
    L.step()
    torch.cuda.synchronize()
    out, grad = exact(L)
    near(L.out, out)
    for name, got in (("x", L.dx), ("res", L.dres), ("norm", L.dnorm), ("wr", L.dwr), ("br", L.dbr), ("w13", L.dw13),
                      ("b13", L.db13), ("w2", L.dw2), ("s13", L.ds13), ("s2", L.ds2)):
        near(got, grad[name])
    # the norm's codes are those of its output
    v = L.q.view(torch.float8_e4m3fn).double() * L.qs.double().repeat_interleave(128, 1)
    assert bool(((v - L.y.double()).abs() <= 2.0 ** -4 * 1.1 * L.y.double().abs() +
                 L.qs.double().repeat_interleave(128, 1) * 2.0 ** -9).all())


def test_layer_in_a_graph():
    cap, eager = Layer(1), Layer(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cap.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap.step()
    for i in range(3):
        for L in (cap, eager):
            L.x.copy_(rand(50 + i, S, H))
            L.dout.copy_(rand(60 + i, S, H))
        graph.replay()
        eager.step()
        torch.cuda.synchronize()
        a, b = cap.outputs(), eager.outputs()
        for k in a:
            assert torch.equal(a[k], b[k]), k
