"""Measured cases of the dense steps around the experts: the norm that makes their input, products kept in
BF16, and the gradients of both.

Each case is one call as a program that serves or trains a mixture of experts makes it.  ``run`` computes it
in elementary torch operations, or, with ``own`` true, through the library's entry points; ``exact`` computes
it from the definition in 64 bits.  The operators:

  norm          root-mean-square norm of a residual stream, the layer's output added on the way, into BF16 and
                into one of the 8-bit formats of the experts' products
  norm_grad     its gradient: of the stream, with the gradient that goes past the norm added, and of the weight
  product       ragged grouped BF16 product (one group: a dense one) with bias, activation and residual in its
                epilogue
  rows_grad     the gradient of a product's rows, multiplied by the derivative of the activation before it
  weights_grad  the gradient of the experts' weights and biases
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
FP8_MAX = 448.0
EPS = 1e-6
ACTS = ("none", "relu", "gelu", "silu", "swiglu")
FORMS = ("plain", "rowwise", "mxfp8", "block128")


def _mxg():
    import fp4_grouped_gemm_quantize_amd as mxg
    return mxg


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a serving step's norm before the experts: few tokens, where latency counts
        dict(name="norm_decode", op="norm", tokens=64, width=7168, stream="bf16", residual=True, form="rowwise",
             offset=0.0),
        # a prompt's norm, kept for the router and quantised for the experts
        dict(name="norm_prefill", op="norm", tokens=8192, width=4096, stream="bf16", residual=True, form="block128",
             offset=0.0),
        # a stream kept in fp32, an odd number of tokens, rows that fill no block of 512
        dict(name="norm_odd", op="norm", tokens=1021, width=2080, stream="fp32", residual=True, form="mxfp8",
             offset=1.0),
        # a training step's gradient of the norm
        dict(name="norm_grad", op="norm_grad", tokens=8192, width=7168, stream="bf16", offset=0.0),
        # a serving step's router logits: a long sum, few columns, fp32 out
        dict(name="router_logits", op="product", rows=64, experts=1, width=7168, out=64, act="none", bias=True,
             residual=False, keep=False, wide=True, spread=0.0, empty=0),
        # a serving step through a shared expert's gate and up: bound by the weights
        dict(name="shared_decode", op="product", rows=128, experts=1, width=7168, out=4096, act="swiglu", bias=False,
             residual=False, keep=False, wide=False, spread=0.0, empty=0),
        # a prompt's projection added to the residual stream
        dict(name="project_residual", op="product", rows=8192, experts=1, width=4096, out=7168, act="none",
             bias=False, residual=True, keep=False, wide=False, spread=0.0, empty=0),
        # a training step's gate and up product over unevenly used experts, pre-activations kept
        dict(name="experts_forward", op="product", rows=65536, experts=128, width=4096, out=1536, act="swiglu",
             bias=True, residual=False, keep=True, wide=False, spread=1.1, empty=0),
        # odd sizes: rows, columns and a last stage that fill no tile, some experts without rows
        dict(name="experts_odd", op="product", rows=5003, experts=24, width=2080, out=1000, act="gelu", bias=True,
             residual=False, keep=False, wide=False, spread=1.0, empty=2),
        # the gradient of the down product's rows through SwiGLU
        dict(name="experts_rows_grad", op="rows_grad", rows=32768, experts=64, width=1536, out=4096, act="swiglu",
             spread=0.8, empty=1),
        # the gradient of the experts' weights and biases, some experts without rows
        dict(name="experts_weights_grad", op="weights_grad", rows=32768, experts=64, width=4096, out=1536, bias=True,
             spread=0.8, empty=2),
        # the gradient of the router's weights: few rows of output, a long sum over tokens
        dict(name="router_weights_grad", op="weights_grad", rows=8192, experts=1, width=7168, out=64, bias=True,
             spread=0.0, empty=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "product", "product", "product", "rows_grad", "weights_grad"])
    if op in ("norm", "norm_grad"):
        case = dict(op=op, tokens=_log_int(rng, 1, 8192), width=32 * _log_int(rng, 4, 256),
                    stream=rng.choice(["bf16", "fp32"]), offset=rng.choice([0.0, 1.0]))
        if op == "norm":
            case.update(residual=rng.random() < 0.7, form=rng.choice(FORMS))
        return case
    experts = rng.choice([1, _log_int(rng, 2, 64)])
    case = dict(op=op, rows=_log_int(rng, 1, 16384), experts=experts, width=8 * _log_int(rng, 8, 512),
                spread=rng.choice([0.0, 0.5, 1.1]), empty=rng.randint(0, experts // 4))
    if op == "product":
        act = rng.choice(ACTS)
        case.update(out=2 * _log_int(rng, 16, 1024) + (act != "swiglu") * rng.randint(0, 1), act=act,
                    bias=rng.random() < 0.5, residual=rng.random() < 0.4, keep=rng.random() < 0.4,
                    wide=rng.random() < 0.3)
        return case
    case["out"] = 8 * _log_int(rng, 8, 256)
    if op == "rows_grad":
        case["act"] = rng.choice(ACTS)
    else:
        case["bias"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs
def _row_counts(case, seed):
    """Rows of each expert: popularity falling as rank^-spread, some experts with none."""
    r = np.random.default_rng(seed)
    p = (1.0 + np.arange(case["experts"])) ** -float(case["spread"])
    p[r.permutation(case["experts"])[: case["empty"]]] = 0.0
    return r.multinomial(case["rows"], r.permutation(p) / p.sum())


def _activations(g, rows, width, scale=1.0):
    """N(0, 1) rows with a few large channels."""
    x = torch.randn((rows, width), generator=g, device="cuda")
    return x * torch.where(torch.rand(width, generator=g, device="cuda") < 0.01, 20.0 * scale, scale)


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _blocks(n, size=BLOCK):
    return (n + size - 1) // size


BF16, F32 = torch.bfloat16, torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("norm", "norm_grad"):
        T, H = case["tokens"], case["width"]
        kind = BF16 if case["stream"] == "bf16" else F32
        s["weight"] = (1.0 - case["offset"] + 0.1 * torch.randn(H, generator=g, device="cuda")).to(BF16)
        stream = _activations(g, T, H, 2.0).to(kind)
        if op == "norm":
            s["residual"], s["h"] = (stream, _empty((T, H), kind)) if case["residual"] else (None, None)
            s["x"] = _activations(g, T, H).to(BF16) if case["residual"] else stream
            s["y"] = _empty((T, H), BF16)
            if case["form"] != "plain":
                s["q"] = _empty((T, H), torch.uint8)
                s["scales"] = (_empty(T, F32) if case["form"] == "rowwise" else
                               _empty((T, H // 32), torch.uint8) if case["form"] == "mxfp8" else
                               _empty((T, _blocks(H)), F32))
            return s
        s["h"] = stream
        s["dy"] = _activations(g, T, H, 0.1).to(BF16)
        s["dh"] = (0.1 * torch.randn((T, H), generator=g, device="cuda")).to(kind)
        s["dx"], s["dweight"] = _empty((T, H), kind), _empty(H, F32)
        s["dx_bf16"] = None if kind == BF16 else _empty((T, H), BF16)
        return s
    T, E, K, N = case["rows"], case["experts"], case["width"], case["out"]
    counts = _row_counts(case, seed)
    offsets = np.zeros(E + 1, np.int32)
    offsets[1:] = np.cumsum(counts)
    s["offsets_host"], s["most"] = offsets.tolist(), int(counts.max())
    if E > 1:
        s["offsets"] = torch.from_numpy(offsets).cuda()
        s["expert_ids"] = torch.arange(E, dtype=torch.int32, device="cuda")
    else:  # a dense product has no routing
        s["offsets"] = s["expert_ids"] = None
    if op == "weights_grad":
        s["a"] = _activations(g, T, K).to(BF16)
        s["dc"] = (0.1 * torch.randn((T, N), generator=g, device="cuda")).to(BF16)
        s["dw"] = _empty((E, N, K), F32)
        s["dbias"] = _empty((E, N), F32) if case["bias"] else None
        return s
    s["b"] = _empty((E, N, K), BF16)
    for e in range(E):
        s["b"][e] = (torch.randn((N, K), generator=g, device="cuda") / math.sqrt(K)).to(BF16)
    swiglu = case["act"] == "swiglu"
    if op == "product":
        s["a"] = _activations(g, T, K).to(BF16)
        s["bias"] = 0.1 * torch.randn((E, N), generator=g, device="cuda") if case["bias"] else None
        kind, wide = F32 if case["wide"] else BF16, N // 2 if swiglu else N
        s["residual"] = torch.randn((T, wide), generator=g, device="cuda").to(kind) if case["residual"] else None
        s["c"] = _empty((T, wide), kind)
        s["z"] = _empty((T, N), BF16) if case["keep"] else None
        return s
    s["dc"] = (0.1 * torch.randn((T, N), generator=g, device="cuda")).to(BF16)
    wide = 2 * K if swiglu else K
    s["z"] = None if case["act"] == "none" else torch.randn((T, wide), generator=g, device="cuda").to(BF16)
    s["da"] = _empty((T, wide), BF16)
    return s


# ------------------------------------------------------------------ plain forms
def _fp8(v):
    """Nearest e4m3 value (as torch.float8_e4m3fn), saturating at 448."""
    return v.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def _blocked(x, size):
    """Rows of x [T, H] in blocks of `size`, the last one filled up with zeros: [T, blocks, size]."""
    T, H = x.shape
    n = _blocks(H, size)
    if H % size:
        x = torch.nn.functional.pad(x, (0, n * size - H))
    return x.reshape(T, n, size)


def _quantize(x, form):
    """(codes as e4m3 values, scales) of fp32 x [T, H] in one of the 8-bit formats."""
    T, H = x.shape
    size = H if form == "rowwise" else 32 if form == "mxfp8" else BLOCK
    x = _blocked(x, size)
    top = x.abs().amax(2)
    if form == "mxfp8":  # a power of two: the largest magnitude's, eight binades down
        power = torch.where(top > 0, torch.frexp(top).exponent - 1 - 8, -127).clamp(-127, 127)
        codes = _fp8(torch.ldexp(x, -power[..., None]))
        scales = (power + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        scales = top / FP8_MAX
        codes = _fp8(torch.where(scales[..., None] > 0, x / scales[..., None], x * 0))
    if form == "rowwise":
        scales = scales[:, 0]
    return codes.reshape(T, -1)[:, :H].contiguous(), scales


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "swiglu":
        gate, up = z[:, 0::2], z[:, 1::2]
        return gate * torch.sigmoid(gate) * up
    return z


def _act_grad(z, d, act):
    """d times the derivative of act at z."""
    if act == "relu":
        return torch.where(z > 0, d, 0.0)
    if act == "gelu":
        return d * (0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "silu":
        sig = torch.sigmoid(z)
        return d * sig * (1 + z * (1 - sig))
    if act == "swiglu":
        gate, up = z[:, 0::2], z[:, 1::2]
        sig = torch.sigmoid(gate)
        return torch.stack((d * up * sig * (1 + gate * (1 - sig)), d * gate * sig), 2).reshape(z.shape)
    return d


def _norm_plain(s):
    c = s["case"]
    h = s["x"]
    out = dict()
    if c["residual"]:
        out["h"] = h = (h.float() + s["residual"].float()).to(s["residual"].dtype)
    h = h.float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * (s["weight"].float() + c["offset"])
    out["y"] = y.to(BF16)
    if c["form"] != "plain":
        out["q"], out["scales"] = _quantize(y, c["form"])
    return out


def _norm_grad_plain(s):
    c = s["case"]
    h, dy = s["h"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    n = h * r
    g = dy * (s["weight"].float() + c["offset"])
    dx = s["dh"].float() + r * (g - n * (g * n).mean(1, keepdim=True))
    out = dict(dx=dx.to(s["h"].dtype), dweight=(dy * n).sum(0))
    if s["dx_bf16"] is not None:
        out["dx_bf16"] = dx.to(BF16)
    return out


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        return _norm_plain(s)
    if op == "norm_grad":
        return _norm_grad_plain(s)
    off = s["offsets_host"]
    for e in range(c["experts"]):  # one product for each expert that has rows
        lo, hi = off[e], off[e + 1]
        if op == "weights_grad":
            d = s["dc"][lo:hi].float()
            torch.mm(d.t(), s["a"][lo:hi].float(), out=s["dw"][e])
            if c["bias"]:
                s["dbias"][e] = d.sum(0)
            continue
        if lo == hi:
            continue
        if op == "rows_grad":
            d = s["dc"][lo:hi].float() @ s["b"][e].float()
            z = None if s["z"] is None else s["z"][lo:hi].float()
            s["da"][lo:hi] = _act_grad(z, d, c["act"]).to(BF16)
            continue
        z = s["a"][lo:hi].float() @ s["b"][e].float().t()
        if c["bias"]:
            z += s["bias"][e]
        if c["keep"]:
            s["z"][lo:hi] = z.to(BF16)
        y = _act(z, c["act"])
        s["c"][lo:hi] = (y + s["residual"][lo:hi].float() if c["residual"] else y).to(s["c"].dtype)
    if op == "weights_grad":
        return dict(dw=s["dw"], dbias=s["dbias"]) if c["bias"] else dict(dw=s["dw"])
    if op == "rows_grad":
        return dict(da=s["da"])
    return dict(c=s["c"], z=s["z"]) if c["keep"] else dict(c=s["c"])


# ------------------------------------------------------------------ the library's calls
def _calls(s):
    mxg = _mxg()
    c = s["case"]
    op = c["op"]
    if op == "norm":
        form = (mxg.NORM_PLAIN, mxg.NORM_FP8_ROWWISE, mxg.NORM_MXFP8, mxg.NORM_FP8_BLOCK128)[FORMS.index(c["form"])]
        mxg.mx_rmsnorm(s["x"], s["weight"], residual=s["residual"], h=s["h"], y=s["y"], form=form, q=s.get("q"),
                       scales=s.get("scales"), eps=EPS, weight_offset=c["offset"])
        out = dict(h=s["h"]) if c["residual"] else dict()
        out["y"] = s["y"]
        if c["form"] != "plain":
            out["q"] = s["q"].view(torch.float8_e4m3fn)
            out["scales"] = s["scales"].view(torch.float8_e8m0fnu) if c["form"] == "mxfp8" else s["scales"]
        return out
    if op == "norm_grad":
        mxg.mx_rmsnorm_backward(s["dy"], s["h"], s["weight"], s["dx"], dh=s["dh"], dx_bf16=s["dx_bf16"],
                                dweight=s["dweight"], eps=EPS, weight_offset=c["offset"])
        out = dict(dx=s["dx"], dweight=s["dweight"])
        if s["dx_bf16"] is not None:
            out["dx_bf16"] = s["dx_bf16"]
        return out
    if op == "weights_grad":
        mxg.mx_grouped_matmul_bf16_backward_weights(s["dc"], s["a"], s["dw"], s["offsets"], s["expert_ids"],
                                                    dbias=s["dbias"])
        return dict(dw=s["dw"], dbias=s["dbias"]) if c["bias"] else dict(dw=s["dw"])
    act = (mxg.ACT_NONE, mxg.ACT_RELU, mxg.ACT_GELU, mxg.ACT_SILU, mxg.ACT_SWIGLU)[ACTS.index(c["act"])]
    if op == "rows_grad":
        mxg.mx_grouped_matmul_bf16_backward(s["dc"], s["b"], s["da"], s["offsets"], s["expert_ids"], act=act,
                                            z=s["z"], max_rows_per_group_hint=s["most"])
        return dict(da=s["da"])
    mxg.mx_grouped_matmul_bf16(s["a"], s["b"], s["c"], s["offsets"], s["expert_ids"], bias=s["bias"], act=act,
                               residual=s["residual"], z=s["z"], max_rows_per_group_hint=s["most"])
    return dict(c=s["c"], z=s["z"]) if c["keep"] else dict(c=s["c"])


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n = case["tokens"] * case["width"]
        size = 2 if case["stream"] == "bf16" else 4
        if op == "norm_grad":  # dy, h and dh in, dx out
            return dict(bytes=n * (2 + 3 * size + (2 if size == 4 else 0)) + 6 * case["width"], flops=12 * n)
        total = n * (2 + (2 + 2 * size if case["residual"] else size)) + 2 * case["width"]
        if case["form"] != "plain":
            total += n + case["tokens"] * (4 if case["form"] == "rowwise" else case["width"] // 32
                                           if case["form"] == "mxfp8" else 4 * _blocks(case["width"]))
        return dict(bytes=total, flops=8 * n)
    T, E, K, N = case["rows"], case["experts"], case["width"], case["out"]
    used = min(T, E - case["empty"])  # an expert without rows is not read
    if op == "weights_grad":
        return dict(bytes=2 * T * (K + N) + 4 * E * N * (K + (1 if case["bias"] else 0)), flops=2 * T * N * K)
    swiglu = case["act"] == "swiglu"
    if op == "rows_grad":
        wide = 2 * K if swiglu else K
        return dict(bytes=2 * T * N + 2 * used * N * K + 2 * T * wide * (1 if case["act"] == "none" else 2),
                    flops=2 * T * N * K)
    wide, size = N // 2 if swiglu else N, 4 if case["wide"] else 2
    return dict(bytes=2 * T * K + used * N * (2 * K + (4 if case["bias"] else 0)) + (2 * T * N if case["keep"] else 0)
                + size * T * wide * (2 if case["residual"] else 1), flops=2 * T * N * K)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_e4m3(v):
    """Nearest e4m3 value, ties to even: a step of 2^(exponent - 3), 2^-9 at the least."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448).float()


def _exact_codes(y, form):
    """The 8-bit values and scales of fp64 y, block by block."""
    T, H = y.shape
    size = {"rowwise": H, "mxfp8": 32, "block128": BLOCK}[form]
    values, scales = torch.empty_like(y, dtype=torch.float32), []
    for lo in range(0, H, size):
        part = y[:, lo:lo + size]
        top = part.abs().max(1).values
        if form == "mxfp8":
            scale = torch.exp2((torch.floor(torch.log2(top)) - 8).clamp(-127, 127))
            scale = torch.where(top > 0, scale, 2.0 ** -127)
        else:
            scale = top / 448
        inverse = torch.where(scale > 0, 1 / scale, 0.0)
        values[:, lo:lo + size] = _exact_e4m3(part * inverse[:, None])
        scales.append(scale)
    return values, scales[0] if form == "rowwise" else torch.stack(scales, 1)


def _exact_phi(z):
    return torch.special.ndtr(z)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        out = dict()
        h = s["x"].double()
        if case["residual"]:
            out["h"] = s["x"].double() + s["residual"].double()
            h = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype).double()  # as it is stored
        norm = torch.sqrt(h.square().sum(1) / case["width"] + EPS)
        y = h / norm[:, None] * (s["weight"].double() + case["offset"])
        out["y"] = y
        if case["form"] != "plain":
            out["q"], out["scales"] = _exact_codes(y, case["form"])
        return out
    if op == "norm_grad":
        h, dy = s["h"].double(), s["dy"].double()
        norm = torch.sqrt(h.square().sum(1, keepdim=True) / case["width"] + EPS)
        g = dy * (s["weight"].double() + case["offset"])
        dot = (g * h).sum(1, keepdim=True) / case["width"]
        dx = s["dh"].double() + g / norm - h * dot / norm ** 3
        out = dict(dx=dx, dweight=(dy * h / norm).sum(0))
        if s["dx_bf16"] is not None:
            out["dx_bf16"] = dx
        return out
    off = s["offsets_host"]
    T, E, K, N = case["rows"], case["experts"], case["width"], case["out"]

    def zeros(*shape):
        return torch.zeros(shape, dtype=torch.float64, device="cuda")

    if op == "weights_grad":
        if 8 * E * N * K > 2 ** 34:
            return None
        dw, dbias = zeros(E, N, K), zeros(E, N)
        for e in range(E):
            d = s["dc"][off[e]:off[e + 1]].double().t().contiguous()
            dw[e] = torch.mm(d, s["a"][off[e]:off[e + 1]].double())
            dbias[e] = d.sum(1)
        return dict(dw=dw, dbias=dbias) if case["bias"] else dict(dw=dw)
    act = case["act"]
    if op == "rows_grad":
        da = zeros(*s["da"].shape)
        for e in range(E):
            rows = slice(off[e], off[e + 1])
            d = torch.mm(s["dc"][rows].double(), s["b"][e].double())
            if act == "none":
                da[rows] = d
                continue
            z = s["z"][rows].double()
            if act == "relu":
                da[rows] = d * (z > 0)
            elif act == "gelu":
                da[rows] = d * (_exact_phi(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
            elif act == "silu":
                sig = 1 / (1 + torch.exp(-z))
                da[rows] = d * (sig + z * sig * (1 - sig))
            else:
                gate, up = z[:, 0::2], z[:, 1::2]
                sig = 1 / (1 + torch.exp(-gate))
                da[rows, 0::2] = d * up * (sig + gate * sig * (1 - sig))
                da[rows, 1::2] = d * gate * sig
        return dict(da=da)
    c, kept = zeros(*s["c"].shape), zeros(T, N)
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        z = torch.mm(s["a"][rows].double(), s["b"][e].double().t().contiguous())
        if case["bias"]:
            z = z + s["bias"][e].double()
        kept[rows] = z
        if act == "relu":
            y = z * (z > 0)
        elif act == "gelu":
            y = z * _exact_phi(z)
        elif act == "silu":
            y = z / (1 + torch.exp(-z))
        elif act == "swiglu":
            y = z[:, 0::2] / (1 + torch.exp(-z[:, 0::2])) * z[:, 1::2]
        else:
            y = z
        c[rows] = y + s["residual"][rows].double() if case["residual"] else y
    return dict(c=c, z=kept) if case["keep"] else dict(c=c)
