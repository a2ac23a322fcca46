"""Measured cases of the expert path's routing, block-scaled FP8 and gradient operators.

Each case is one call (or the two calls of one step) as a program that serves
or trains a mixture of experts makes it.  ``run`` computes it in elementary
torch operations, or, with ``own`` true, through the library's entry points;
``exact`` computes it from the definition in 64 bits.  The operators:

  router    top-k expert choice from router logits (softmax or sigmoid scores,
            a selection bias, renormalised weights), and its gradient
  sort      tokens sorted by expert (row offsets, both slot maps), the rows
            copied into that order, and the gradients of the way there and back
  gemm      ragged grouped product of FP8 operands with one fp32 scale for each
            1 x 128 block of activations and 128 x 128 block of weights, and the
            two quantisers that make its operands
  swiglu    gated activation with a 1 x 128 block FP8 requant, and its gradient
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
FP8_MAX = 448.0


def _mxg():
    import fp4_grouped_gemm_quantize_amd as mxg
    return mxg


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a serving step of few tokens: sigmoid scores chosen under a balancing bias, bf16 logits
        dict(name="router_decode", op="router", tokens=64, experts=64, top_k=8, score="sigmoid", bias=True,
             renorm=True, half=True, grad=False),
        # a training step's router: softmax over fp32 logits, renormalised, forward and gradient
        dict(name="router_train", op="router", tokens=8192, experts=128, top_k=8, score="softmax", bias=False,
             renorm=True, half=False, grad=True),
        # the routing plan of a serving step, where only latency counts
        dict(name="sort_decode", op="sort", tokens=128, experts=64, top_k=8, width=0, dropped=0.0),
        # a prompt's tokens sorted and copied into expert order
        dict(name="dispatch_prefill", op="sort", tokens=8192, experts=128, top_k=8, width=4096, dropped=0.0),
        # the gradient of the way back and of the way there, some slots dropped by a capacity limit
        dict(name="combine_grad", op="unsort", tokens=4096, experts=128, top_k=8, width=7168, dropped=0.02),
        # a prompt's activations quantised on their way into expert order
        dict(name="quantize_rows", op="quantize", tokens=8192, experts=128, top_k=8, width=4096),
        # a training step's weights quantised for the product and, transposed, for its gradient
        dict(name="quantize_weights", op="weights", experts=8, rows=4096, width=7168),
        # a serving step: few rows an expert, bound by the weights
        dict(name="gemm_decode", op="gemm", rows=1024, experts=64, width=7168, out=2048, spread=0.2, empty=4),
        # the gradient of the activations at odd sizes: rows, columns and a last block that fill no tile
        dict(name="gemm_grad_odd", op="gemm", rows=5003, experts=24, width=2080, out=1000, spread=1.0, empty=2),
        # a prompt over many unevenly used experts
        dict(name="gemm_prefill", op="gemm", rows=65536, experts=128, width=4096, out=1536, spread=1.1, empty=0),
        # a small batch's gated activation, quantised for the down product
        dict(name="swiglu_rows", op="swiglu", rows=1021, experts=32, width=2048, grad=False),
        # a training step's gradient of the gated activation, kept and quantised
        dict(name="swiglu_grad", op="swiglu", rows=32768, experts=64, width=2048, grad=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "sort", "unsort", "quantize", "weights", "gemm", "gemm", "gemm", "swiglu"])
    if op in ("router", "sort", "unsort", "quantize"):
        experts = rng.choice([rng.randint(2, 32), rng.randint(33, 256)])
        top_k = rng.randint(1, min(8, experts))
        tokens = _log_int(rng, 1, 8192)
    if op == "router":
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, renorm=rng.random() < 0.7, half=rng.random() < 0.5,
                    grad=rng.random() < 0.5)
    if op == "sort":
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k,
                    width=0 if rng.random() < 0.3 else 8 * _log_int(rng, 8, 512),
                    dropped=rng.choice([0.0, 0.05]))
    if op == "unsort":
        return dict(op=op, tokens=_log_int(rng, 1, 4096), experts=experts, top_k=top_k, width=8 * _log_int(rng, 8, 896),
                    dropped=rng.choice([0.0, 0.05]))
    if op == "quantize":
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, width=32 * _log_int(rng, 4, 128))
    if op == "weights":
        return dict(op=op, experts=rng.randint(1, 8), rows=32 * _log_int(rng, 4, 128), width=32 * _log_int(rng, 4, 224))
    if op == "swiglu":
        return dict(op=op, rows=_log_int(rng, 1, 32768), experts=rng.randint(1, 64), width=32 * _log_int(rng, 4, 64),
                    grad=rng.random() < 0.5)
    experts = _log_int(rng, 1, 64)
    return dict(op=op, rows=_log_int(rng, 1, 16384), experts=experts, width=32 * _log_int(rng, 4, 128),
                out=_log_int(rng, 64, 2048), spread=rng.choice([0.0, 0.5, 1.1]), empty=rng.randint(0, experts // 4))


# ------------------------------------------------------------------ inputs
def _ids(g, tokens, experts, top_k, dropped=0.0):
    """int32 [tokens, top_k]: distinct experts a token, unevenly popular; a share of the slots dropped (-1)."""
    popular = torch.randn(experts, generator=g, device="cuda")
    noise = torch.rand((tokens, experts), generator=g, device="cuda").clamp_min_(1e-20)
    ids = torch.topk(popular - torch.log(-torch.log(noise)), top_k, dim=1).indices.to(torch.int32)
    if dropped:
        ids[torch.rand((tokens, top_k), generator=g, device="cuda") < dropped] = -1
    return ids.contiguous()


def _sorted(ids, experts):
    """(row_offsets [E + 1], row_of_slot, slot_of_row), int32: slots in the order (expert, slot), dropped ones last."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    ordered, slot = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ordered, torch.arange(experts + 1, device=key.device))
    live = ordered < experts
    place = torch.arange(flat.numel(), device=key.device)
    row_of_slot = torch.empty_like(flat)
    row_of_slot[slot] = torch.where(live, place, -1)
    slot_of_row = torch.where(live, slot, -1)
    return offsets.to(torch.int32), row_of_slot.to(torch.int32), slot_of_row.to(torch.int32)


def _row_counts(case, seed):
    """Rows of each expert: popularity falling as rank^-spread, some experts with none."""
    r = np.random.default_rng(seed)
    p = (1.0 + np.arange(case["experts"])) ** -float(case.get("spread", 0.5))
    p[r.permutation(case["experts"])[: case.get("empty", 0)]] = 0.0
    return r.multinomial(case["rows"], r.permutation(p) / p.sum())


def _offsets(counts):
    off = np.zeros(len(counts) + 1, np.int32)
    off[1:] = np.cumsum(counts)
    return off


def _activations(g, rows, width):
    """N(0, 1) rows with a few large channels, bf16."""
    x = torch.randn((rows, width), generator=g, device="cuda")
    x = x * torch.where(torch.rand(width, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(torch.bfloat16)


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "router":
        S, E, k = case["tokens"], case["experts"], case["top_k"]
        kind = torch.bfloat16 if case["half"] else torch.float32
        logits = torch.randn((S, E), generator=g, device="cuda") * 1.5 + torch.randn(E, generator=g, device="cuda")
        s["logits"] = logits.to(kind)
        s["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        s["ids"], s["weights"] = _empty((S, k), torch.int32), _empty((S, k), torch.float32)
        if case["grad"]:
            s["dweights"] = torch.randn((S, k), generator=g, device="cuda")
            s["dlogits"] = _empty((S, E), kind)
        return s
    if op in ("sort", "unsort", "quantize"):
        S, E, k, W = case["tokens"], case["experts"], case["top_k"], case["width"]
        s["ids"] = _ids(g, S, E, k, case.get("dropped", 0.0))
        if op == "sort":
            s["plan"] = (_empty(E + 1, torch.int32), _empty(S * k, torch.int32), _empty(S * k, torch.int32))
            if W:
                s["x"] = _activations(g, S, W)
                s["out"] = torch.zeros((S * k, W), dtype=torch.bfloat16, device="cuda")
            return s
        s["plan"] = _sorted(s["ids"], E)
        if op == "quantize":
            s["x"] = _activations(g, S, W)
            s["q"] = _empty((S * k, W), torch.uint8)
            s["scales"] = _empty((S * k, _blocks(W)), torch.float32)
            return s
        s["y"] = _activations(g, S * k, W)
        s["dout"] = (0.1 * torch.randn((S, W), generator=g, device="cuda")).to(torch.bfloat16)
        s["drows"] = (0.1 * torch.randn((S * k, W), generator=g, device="cuda")).to(torch.bfloat16)
        s["weights"] = torch.softmax(torch.randn((S, k), generator=g, device="cuda"), 1).reshape(-1)
        s["dy"] = torch.zeros((S * k, W), dtype=torch.bfloat16, device="cuda")
        s["dweights"], s["dx"] = _empty(S * k, torch.float32), _empty((S, W), torch.bfloat16)
        return s
    if op == "weights":
        E, N, K = case["experts"], case["rows"], case["width"]
        s["w"] = _empty((E, N, K), torch.bfloat16)
        for e in range(E):
            s["w"][e] = (0.02 * torch.randn((N, K), generator=g, device="cuda")).to(torch.bfloat16)
        s["q"], s["q_t"] = _empty((E, N, K), torch.uint8), _empty((E, K, N), torch.uint8)
        s["scales"] = _empty((E, _blocks(N), _blocks(K)), torch.float32)
        s["scales_t"] = _empty((E, _blocks(K), _blocks(N)), torch.float32)
        return s
    counts = _row_counts(case, seed)
    off = _offsets(counts)
    s["offsets_host"] = off.tolist()
    s["offsets"] = torch.from_numpy(off).cuda()
    s["expert_ids"] = torch.arange(case["experts"], dtype=torch.int32, device="cuda")
    s["most"] = int(counts.max())
    T, W = case["rows"], case["width"]
    if op == "gemm":
        E, N = case["experts"], case["out"]
        codes, scales = _quantize_rows(_activations(g, T, W).float())
        s["a"], s["a_scales"] = codes.view(torch.uint8), scales
        s["b"], s["b_scales"] = _empty((E, N, W), torch.uint8), _empty((E, _blocks(N), _blocks(W)), torch.float32)
        for e in range(E):
            codes, s["b_scales"][e] = _quantize_tiles(0.02 * torch.randn((N, W), generator=g, device="cuda"))
            s["b"][e] = codes.view(torch.uint8)
        s["c"] = _empty((T, N), torch.bfloat16)
        return s
    s["h"] = _activations(g, T, 2 * W)
    s["q"] = _empty((T, 2 * W if case["grad"] else W), torch.uint8)
    s["scales"] = _empty((T, _blocks(2 * W if case["grad"] else W)), torch.float32)
    if case["grad"]:
        s["dy"] = (0.1 * torch.randn((T, W), generator=g, device="cuda")).to(torch.bfloat16)
        s["dh"] = _empty((T, 2 * W), torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms
def _fp8(v):
    """Nearest e4m3 value (as torch.float8_e4m3fn), saturating at 448."""
    return v.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)


def _quantize_rows(x):
    """(codes, scales) of fp32 x [T, K], a scale for each 1 x 128 block: scale = amax / 448, code = e4m3(x / scale)."""
    T, K = x.shape
    nb = _blocks(K)
    if K % BLOCK:
        x = torch.nn.functional.pad(x, (0, nb * BLOCK - K))
    x = x.reshape(T, nb, BLOCK)
    scale = x.abs().amax(2) / FP8_MAX
    codes = _fp8(torch.where(scale[..., None] > 0, x / scale[..., None], x * 0))
    return codes.reshape(T, nb * BLOCK)[:, :K].contiguous(), scale


def _quantize_tiles(w):
    """(codes, scales) of fp32 w [N, K], a scale for each 128 x 128 tile."""
    N, K = w.shape
    nn, nk = _blocks(N), _blocks(K)
    if N % BLOCK or K % BLOCK:
        w = torch.nn.functional.pad(w, (0, nk * BLOCK - K, 0, nn * BLOCK - N))
    t = w.reshape(nn, BLOCK, nk, BLOCK)
    scale = t.abs().amax((1, 3)) / FP8_MAX
    wide = scale[:, None, :, None]
    codes = _fp8(torch.where(wide > 0, t / wide, t * 0))
    return codes.reshape(nn * BLOCK, nk * BLOCK)[:N, :K].contiguous(), scale


def _router_keys(logits, bias, score):
    """What experts are chosen by: the logits (both scores rise with them), or, under a bias, score + bias in 64
    bits, since two sums can lie closer together than 32 bits resolve."""
    if bias is None:
        return logits.float()
    x = logits.double()
    return (torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)) + bias.double()


def _router_plain(s):
    c = s["case"]
    x = s["logits"].float()
    keys = _router_keys(s["logits"], s["bias"], c["score"])
    # ties go to the lowest index: a stable sort, falling
    ids = torch.sort(keys, dim=1, descending=True, stable=True).indices[:, : c["top_k"]]
    # log of the scores, so that their ratios survive where the scores themselves underflow
    logs = torch.log_softmax(x, 1) if c["score"] == "softmax" else torch.nn.functional.logsigmoid(x)
    chosen = logs.gather(1, ids)
    w = torch.softmax(chosen, 1) if c["renorm"] else torch.exp(chosen)
    out = dict(ids=ids.to(torch.int32), weights=w * SCALE)
    if c["grad"]:
        d = s["dweights"] * SCALE
        dlog = w * (d - (w * d).sum(1, keepdim=True)) if c["renorm"] else w * d  # of the chosen scores' logs
        if c["score"] == "sigmoid":
            dx = torch.zeros_like(x).scatter_(1, ids, dlog * torch.sigmoid(-x.gather(1, ids)))
        else:
            dx = torch.zeros_like(x).scatter_(1, ids, dlog)
            if not c["renorm"]:  # a renormalised softmax leaves the others out of it
                dx = dx - torch.softmax(x, 1) * dlog.sum(1, keepdim=True)
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


SCALE = 2.5  # what the chosen weights are multiplied by


def _combine_grad_plain(s):
    c = s["case"]
    S, k, W = c["tokens"], c["top_k"], c["width"]
    _, row_of_slot, slot_of_row = s["plan"]
    live_row = slot_of_row >= 0
    slot = slot_of_row.long().clamp_min(0)
    dout, y = s["dout"].float(), s["y"].float()
    dy = dout[slot // k] * s["weights"][slot][:, None]
    s["dy"].copy_(torch.where(live_row[:, None], dy, s["dy"].float()))  # dropped rows stay as they were
    live, row = row_of_slot >= 0, row_of_slot.long().clamp_min(0)
    dots = (y[row].reshape(S, k, W) * dout[:, None, :]).sum(2).reshape(-1)
    rows = torch.where(live[:, None], s["drows"].float()[row], 0.0)
    return dict(dy=s["dy"], dweights=torch.where(live, dots, 0.0), dx=rows.reshape(S, k, W).sum(1).to(torch.bfloat16))


def _gemm_plain(s):
    c = s["case"]
    K, N, off = c["width"], c["out"], s["offsets_host"]
    a = s["a"].view(torch.float8_e4m3fn).float() * s["a_scales"].repeat_interleave(BLOCK, 1)[:, :K]
    for e in range(c["experts"]):  # one product for each expert that has rows
        if off[e + 1] > off[e]:
            scale = s["b_scales"][e].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
            b = s["b"][e].view(torch.float8_e4m3fn).float() * scale
            s["c"][off[e]:off[e + 1]] = (a[off[e]:off[e + 1]] @ b.t()).to(torch.bfloat16)
    return s["c"]


def _swiglu_plain(s):
    h = s["h"].float()
    gate, up = h[:, 0::2], h[:, 1::2]
    sig = torch.sigmoid(gate)
    if not s["case"]["grad"]:
        codes, scales = _quantize_rows(gate * sig * up)
        return dict(q=codes, scales=scales)
    dy = s["dy"].float()
    dh = torch.stack((dy * up * sig * (1 + gate * (1 - sig)), dy * gate * sig), 2).reshape(h.shape)
    codes, scales = _quantize_rows(dh)
    return dict(dh=dh.to(torch.bfloat16), q=codes, scales=scales)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "router":
        return _router_plain(s)
    if op == "sort":
        offsets, row_of_slot, slot_of_row = _sorted(s["ids"], c["experts"])
        out = dict(offsets=offsets, row_of_slot=row_of_slot, slot_of_row=slot_of_row)
        if c["width"]:
            live = (slot_of_row >= 0)[:, None]
            rows = s["x"].float()[slot_of_row.long().clamp_min(0) // c["top_k"]]
            s["out"].copy_(torch.where(live, rows, s["out"].float()))
            out["rows"] = s["out"]
        return out
    if op == "unsort":
        return _combine_grad_plain(s)
    if op == "quantize":
        codes, scales = _quantize_rows(s["x"].float()[s["plan"][2].long() // c["top_k"]])
        return dict(q=codes, scales=scales)
    if op == "weights":
        E, N, K = s["w"].shape
        nn, nk = _blocks(N), _blocks(K)
        w = torch.nn.functional.pad(s["w"].float(), (0, nk * BLOCK - K, 0, nn * BLOCK - N))
        w = w.reshape(E * nn * BLOCK, nk * BLOCK)
        codes, scales = _quantize_tiles(w)
        codes = codes.view(torch.uint8).reshape(E, nn * BLOCK, nk * BLOCK)[:, :N, :K].contiguous()
        scales = scales.reshape(E, nn, nk)
        return dict(q=codes.view(torch.float8_e4m3fn), scales=scales,
                    q_t=codes.transpose(1, 2).contiguous().view(torch.float8_e4m3fn),
                    scales_t=scales.transpose(1, 2).contiguous())
    return _gemm_plain(s) if op == "gemm" else _swiglu_plain(s)


# ------------------------------------------------------------------ the library's calls
def _calls(s):
    mxg = _mxg()
    c = s["case"]
    op = c["op"]
    if op == "router":
        score = mxg.SCORE_SOFTMAX if c["score"] == "softmax" else mxg.SCORE_SIGMOID
        mxg.mx_moe_topk(score, s["logits"], s["ids"], s["weights"], bias=s["bias"], renormalize=c["renorm"],
                        scale=SCALE)
        out = dict(ids=s["ids"], weights=s["weights"])
        if c["grad"]:
            mxg.mx_moe_topk_backward(score, s["logits"], s["ids"], s["dweights"], s["dlogits"],
                                     renormalize=c["renorm"], scale=SCALE)
            out["dlogits"] = s["dlogits"]
        return out
    if op == "sort":
        offsets, row_of_slot, slot_of_row = s["plan"]
        mxg.mx_moe_sort(s["ids"], offsets, row_of_slot, slot_of_row)
        out = dict(offsets=offsets, row_of_slot=row_of_slot, slot_of_row=slot_of_row)
        if c["width"]:
            mxg.mx_moe_permute(s["x"], row_of_slot, s["out"])
            out["rows"] = s["out"]
        return out
    if op == "unsort":
        row_of_slot = s["plan"][1]
        mxg.mx_moe_combine_backward(s["dout"], s["y"], row_of_slot, s["weights"], s["dy"], s["dweights"])
        mxg.mx_moe_permute_backward(s["drows"], row_of_slot, s["dx"])
        return dict(dy=s["dy"], dweights=s["dweights"], dx=s["dx"])
    if op == "quantize":
        mxg.mx_grouped_quantize_block128_scatter(s["x"], s["plan"][1], s["q"], s["scales"], s["plan"][0])
        return dict(q=s["q"].view(torch.float8_e4m3fn), scales=s["scales"])
    if op == "weights":
        mxg.mx_quantize_weights_block128(s["w"], s["q"], s["scales"], s["q_t"], s["scales_t"])
        return dict(q=s["q"].view(torch.float8_e4m3fn), scales=s["scales"], q_t=s["q_t"].view(torch.float8_e4m3fn),
                    scales_t=s["scales_t"])
    if op == "gemm":
        mxg.mx_grouped_matmul_block128(s["a"], s["a_scales"], s["b"], s["b_scales"], s["c"], s["offsets"],
                                       s["expert_ids"], max_rows_per_group_hint=s["most"])
        return s["c"]
    if c["grad"]:
        mxg.mx_silu_backward_block128(s["h"], s["dy"], s["offsets"], dh=s["dh"], dh_q=s["q"], dh_scales=s["scales"])
        return dict(dh=s["dh"], q=s["q"].view(torch.float8_e4m3fn), scales=s["scales"])
    mxg.mx_silu_quantize_block128(s["h"], s["q"], s["scales"], s["offsets"])
    return dict(q=s["q"].view(torch.float8_e4m3fn), scales=s["scales"])


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "router":
        S, E, k = case["tokens"], case["experts"], case["top_k"]
        size = 2 if case["half"] else 4
        n = S * E * size + 8 * S * k + (4 * E if case["bias"] else 0)
        flops = S * E * 4
        if case["grad"]:
            n += 2 * S * E * size + 8 * S * k
            flops += S * E * 6
        return dict(bytes=n, flops=flops)
    if op in ("sort", "unsort", "quantize"):
        S, k, W = case["tokens"], case["top_k"], case["width"]
        slots = S * k
        if op == "sort":
            return dict(bytes=12 * slots + 4 * (case["experts"] + 1) + (2 * W * (S + slots) if W else 0), flops=slots)
        if op == "unsort":
            # dout, y and the rows' gradients in; the rows' gradients and the tokens' out
            return dict(bytes=2 * W * (2 * S + 3 * slots) + 12 * slots, flops=4 * slots * W)
        return dict(bytes=2 * S * W + slots * (W + 4 * _blocks(W)) + 4 * slots, flops=2 * slots * W)
    if op == "weights":
        n = case["experts"] * case["rows"] * case["width"]
        return dict(bytes=2 * n + 2 * n + 8 * case["experts"] * _blocks(case["rows"]) * _blocks(case["width"]),
                    flops=2 * n)
    T, W = case["rows"], case["width"]
    if op == "gemm":
        N = case["out"]
        used = min(T, case["experts"] - case["empty"])  # an expert without rows is not read
        return dict(bytes=T * (W + 4 * _blocks(W)) + used * (N * W + 4 * _blocks(N) * _blocks(W)) + 2 * T * N,
                    flops=2 * T * N * W)
    if case["grad"]:
        return dict(bytes=4 * T * W + 2 * T * W + 4 * T * W + T * (2 * W + 4 * _blocks(2 * W)), flops=12 * T * W)
    return dict(bytes=4 * T * W + T * (W + 4 * _blocks(W)), flops=6 * T * W)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rows(x):
    """Block-scaled values of fp64 x [T, K]: the scales amax / 448 and the nearest e4m3 values of x / scale."""
    T, K = x.shape
    edges = list(range(0, K, BLOCK))
    scales = torch.stack([x[:, b:b + BLOCK].abs().amax(1) / 448 for b in edges], 1)
    inverse = torch.where(scales > 0, 1 / scales, 0.0)
    return _exact_e4m3(x * inverse.repeat_interleave(BLOCK, 1)[:, :K]), scales


def _exact_e4m3(v):
    """Nearest e4m3 value, ties to even: a step of 2^(exponent - 3), 2^-9 at the least."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448).float()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "router":
        x = s["logits"].double()
        score = x.softmax(1) if case["score"] == "softmax" else 1 / (1 + torch.exp(-x))
        key = x if s["bias"] is None else score + s["bias"].double()
        ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, : case["top_k"]]
        p = score.gather(1, ids)
        total = p.sum(1, keepdim=True) if case["renorm"] else torch.ones_like(p[:, :1])
        out = dict(ids=None, weights=SCALE * p / total)
        if case["grad"]:
            d = SCALE * s["dweights"].double()
            dp = (d - (d * p / total).sum(1, keepdim=True)) / total if case["renorm"] else d
            ds = torch.zeros_like(x)
            ds.scatter_(1, ids, dp)
            if case["score"] == "softmax":
                out["dlogits"] = score * (ds - (ds * score).sum(1, keepdim=True))
            else:
                out["dlogits"] = ds * score * (1 - score)
        return out
    if op == "sort":
        return None  # whole numbers and copies
    if op == "unsort":
        k = case["top_k"]
        dy, dx = s["dy"].double(), torch.zeros_like(s["dx"], dtype=torch.float64)
        dw = torch.zeros(s["weights"].numel(), dtype=torch.float64, device="cuda")
        rows = s["plan"][1].long().reshape(-1, k)
        for j in range(k):
            live = torch.nonzero(rows[:, j] >= 0)[:, 0]
            at = rows[live, j]
            d = s["dout"][live].double()
            dw[live * k + j] = (d * s["y"][at].double()).sum(1)
            dy[at] = d * s["weights"].double()[live * k + j][:, None]
            dx[live] += s["drows"][at].double()
        return dict(dy=dy, dweights=dw, dx=dx)
    if op == "quantize":
        token = torch.div(s["plan"][2].long(), case["top_k"], rounding_mode="floor")
        values, scales = _exact_rows(s["x"].double())
        return dict(q=values[token], scales=scales[token])
    if op == "weights":
        E, N, K = s["w"].shape
        q, scales = _empty((E, N, K), torch.float32), _empty(s["scales"].shape, torch.float64)
        for e in range(E):
            w = s["w"][e].double()
            for i, lo in enumerate(range(0, N, BLOCK)):
                band = w[lo:lo + BLOCK]
                tops = torch.stack([band[:, b:b + BLOCK].abs().max() for b in range(0, K, BLOCK)]) / 448
                scales[e, i] = tops
                inverse = torch.where(tops > 0, 1 / tops, 0.0)
                q[e, lo:lo + BLOCK] = _exact_e4m3(band * inverse.repeat_interleave(BLOCK)[:K])
        return dict(q=q, scales=scales, q_t=q.transpose(1, 2).contiguous(),
                    scales_t=scales.transpose(1, 2).contiguous())
    off = s["offsets_host"]
    if op == "gemm":
        K, N = case["width"], case["out"]
        out = torch.zeros((case["rows"], N), dtype=torch.float64, device="cuda")
        wide_k = torch.arange(K, device="cuda") // BLOCK
        wide_n = torch.arange(N, device="cuda") // BLOCK
        for e in range(case["experts"]):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            a = s["a"][lo:hi].view(torch.float8_e4m3fn).double() * s["a_scales"][lo:hi].double()[:, wide_k]
            b = s["b"][e].view(torch.float8_e4m3fn).double() * s["b_scales"][e].double()[wide_n][:, wide_k]
            out[lo:hi] = torch.mm(a, b.t())
        return out
    gate, up = s["h"][:, 0::2].double(), s["h"][:, 1::2].double()
    sig = 1 / (1 + torch.exp(-gate))
    if not case["grad"]:
        values, scales = _exact_rows(gate * sig * up)
        return dict(q=values, scales=scales)
    dy = s["dy"].double()
    dh = torch.empty(s["h"].shape, dtype=torch.float64, device="cuda")
    dh[:, 0::2] = dy * up * (sig + gate * sig * (1 - sig))
    dh[:, 1::2] = dy * gate * sig
    values, scales = _exact_rows(dh)
    return dict(dh=dh, q=values, scales=scales)
