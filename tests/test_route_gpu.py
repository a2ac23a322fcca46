"""The router, the routing plan, the permutation and their gradients against
plain numpy in 64 bits.

Tolerances.  A score is formed from fp32 exponentials of differences: with R the
largest |log score| or |logit - maximum| that enters it, an exponential is off by
(R + 2) 2^-23 relative (its argument's rounding and two ulps), a sum of n
positive terms by n 2^-24, a quotient or product by 2^-24 each; weights are held
to w (4 R + n + 16) 2^-23.  bf16 results add half a step, 2^-8 of the value
(2^-134 at zero).  Integers and copies are exact."""
import numpy as np
import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg
from common import Guarded, to_gpu

pytestmark = pytest.mark.gpu

SOFTMAX, SIGMOID = mxg.SCORE_SOFTMAX, mxg.SCORE_SIGMOID


def bf16(a):
    """numpy fp64 -> torch bf16 on the GPU and its exact fp64 values."""
    t = torch.from_numpy(np.ascontiguousarray(a, np.float64)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def half_step_bf16(v):
    return np.abs(v) * 2.0 ** -8 + 2.0 ** -134


# ------------------------------------------------------------------ router
def scores(x, score):
    if score == SIGMOID:
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    m = np.max(x, axis=1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    p = np.exp(x - m)
    with np.errstate(invalid="ignore", divide="ignore"):
        return p / p.sum(1, keepdims=True)


def log_scores(x, score):
    if score == SIGMOID:
        return np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))
    m = np.max(x, axis=1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(divide="ignore", invalid="ignore"):
        return x - m - np.log(np.exp(x - m).sum(1, keepdims=True))


def ref_topk(x, k, score, bias, renorm, scale):
    key = x if bias is None else np.where(x > -np.inf, scores(x, score) + bias, -np.inf)
    key = np.where(np.isnan(key), -np.inf, key)
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    live = np.take_along_axis(key, order, 1) > -np.inf
    ids = np.where(live, order, -1)
    ls = np.where(live, np.take_along_axis(log_scores(x, score), order, 1), -np.inf)
    if renorm:
        m = np.max(ls, 1, keepdims=True)
        w = np.exp(ls - np.where(np.isfinite(m), m, 0))
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    else:
        w = np.exp(ls)
    return ids.astype(np.int32), scale * w


def spread(x, score):
    """R of the tolerance: what the exponentials' arguments reach."""
    f = np.where(np.isfinite(x), x, 0.0)
    return float(np.max(np.abs(f)) + (np.max(f) - np.min(f))) if f.size else 0.0


def ref_topk_backward(x, ids, dw, score, renorm, scale):
    S, E = x.shape
    out, mag = np.zeros((S, E)), np.zeros((S, E))
    s, ls = scores(x, score), log_scores(x, score)
    for t in range(S):
        slots = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E and x[t, ids[t, j]] > -np.inf]
        if not slots:
            continue
        i = ids[t, slots]
        d = scale * dw[t, slots]
        if renorm:
            r = np.exp(ls[t, i] - ls[t, i].max())
            r /= r.sum()
            g, gm = r * (d - (r * d).sum()), r * (np.abs(d) + (r * np.abs(d)).sum())
        else:
            g, gm = s[t, i] * d, s[t, i] * np.abs(d)
        if score == SIGMOID:
            q = scores(-x[t:t + 1, i], SIGMOID)[0]  # 1 - s, without its cancellation
            g, gm = g * q, gm * q
        np.add.at(out[t], i, g)
        np.add.at(mag[t], i, gm)
        if score == SOFTMAX and not renorm:
            out[t] -= s[t] * g.sum()
            mag[t] += s[t] * gm.sum()
    return out, mag


def logits_of(kind, S, E, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 2, (S, E))
    if kind == "ties":
        x = np.round(x)            # many equal logits, zeros of both signs
        x[x == 0] = rng.choice([0.0, -0.0], (x == 0).sum())
    if kind == "masked":
        x[rng.random((S, E)) < 0.5] = -np.inf
        x[0] = -np.inf             # nothing left
        if S > 1:
            x[1] = -np.inf
            x[1, E // 2] = 0.3     # one left
    if kind == "lowest":
        x[rng.random((S, E)) < 0.5] = float(torch.finfo(torch.bfloat16).min)
        x[0] = float(torch.finfo(torch.bfloat16).min)
    if kind == "far":
        x *= 40.0                  # scores that underflow
    return x


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("S,E,k", [(1, 1, 1), (5, 8, 8), (33, 64, 8), (17, 65, 3), (9, 128, 16), (7, 256, 6),
                                   (6, 100, 17), (3, 300, 8), (2, 1024, 64)])
def test_topk_shapes(S, E, k, half):
    for n, (score, biased, renorm) in enumerate([(SOFTMAX, False, True), (SOFTMAX, False, False),
                                                 (SIGMOID, False, True), (SIGMOID, True, True),
                                                 (SOFTMAX, True, False), (SIGMOID, False, False)]):
        check_topk("ties" if n % 2 else "plain", S, E, k, half, score, biased, renorm, seed=S * 1000 + E + n)


@pytest.mark.parametrize("S,E,k", [(4, 257, 8), (3, 512, 64), (5, 400, 20), (2, 513, 9), (70, 16, 16), (65, 48, 5)])
@pytest.mark.parametrize("biased", [False, True])
def test_topk_ties_at_every_width(S, E, k, biased):
    """Logits of five values and -infinity (and equal biases): the choice is the first of equals."""
    rng = np.random.default_rng(E + k)
    x = rng.choice(np.array([-np.inf, -3.0, -0.0, 0.0, 1.5, 2.0], np.float32), (S, E))
    bias = torch.full((E,), 0.25, device="cuda") if biased else None
    ids, _ = mxg.moe_topk(SIGMOID, to_gpu(x), k, bias)
    for row, got in zip(x, ids.cpu().numpy()):
        order = np.argsort(-row, kind="stable")
        order = order[row[order] > -np.inf][:k]
        assert got.tolist() == order.tolist() + [-1] * (k - len(order))


@pytest.mark.parametrize("kind", ["plain", "ties", "masked", "lowest", "far"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_topk_values(kind, score, biased, renorm):
    check_topk(kind, 40, 96, 8, False, score, biased, renorm, seed=3)
    check_topk(kind, 40, 96, 8, True, score, biased, renorm, seed=4)


def check_topk(kind, S, E, k, half, score, biased, renorm, seed):
    rng = np.random.default_rng(seed + 77)
    x64 = logits_of(kind, S, E, seed)
    if half:
        xg, x = bf16(x64)
    else:
        xg = torch.from_numpy(x64.astype(np.float32)).cuda()
        x = x64.astype(np.float32).astype(np.float64)
    bias = (rng.normal(0, 0.2, E)).astype(np.float32) if biased else None
    scale = 1.75
    ids_g, w_g = Guarded(np.full((S, k), 77, np.int32)), Guarded(np.full((S, k), 7.0, np.float32))
    mxg.mx_moe_topk(score, xg, ids_g.view(), w_g.view(), None if bias is None else to_gpu(bias), renorm, scale)
    torch.cuda.synchronize()
    ids_g.check(), w_g.check()
    ids, w = ref_topk(x, k, score, bias, renorm, scale)
    assert np.array_equal(ids_g.numpy(), ids)
    R = min(spread(x, score), 200.0)  # past e^-104 an fp32 score is 0: the absolute term
    tol = np.abs(w) * (4 * R + E + 16) * 2.0 ** -23 + scale * 2.0 ** -120
    assert np.all(np.abs(w_g.numpy() - w) <= tol)

    dw = rng.normal(0, 1, (S, k)).astype(np.float32)
    d_g = Guarded(np.full((S, E), 7, np.int16 if half else np.float32))
    dl = d_g.view(torch.bfloat16) if half else d_g.view()
    mxg.mx_moe_topk_backward(score, xg, ids_g.view(), to_gpu(dw), dl, renorm, scale)
    torch.cuda.synchronize()
    d_g.check()
    ref, mag = ref_topk_backward(x, ids, dw.astype(np.float64), score, renorm, scale)
    tol = mag * (8 * R + E + 4 * k + 32) * 2.0 ** -23 + 2.0 ** -115
    if half:
        tol = tol + half_step_bf16(ref)
    assert np.all(np.abs(dl.double().cpu().numpy() - ref) <= tol)


def test_topk_gradient_against_differences():
    """The derivative of sum(weights * dw) along a random direction by central
    differences in 64 bits of the same choice: step h leaves h^2 times the third
    derivative, under 1e-6 of the values here at h = 1e-3."""
    rng = np.random.default_rng(5)
    S, E, k, h = 12, 48, 6, 1e-3
    x = rng.normal(0, 1.5, (S, E))
    v = rng.normal(0, 1, (S, E))
    dw = rng.normal(0, 1, (S, k)).astype(np.float32)
    for score in (SOFTMAX, SIGMOID):
        for renorm in (False, True):
            xg = torch.from_numpy(x.astype(np.float32)).cuda()
            ids, _ = mxg.moe_topk(score, xg, k, None, renorm, 1.5)
            dl = torch.empty((S, E), device="cuda")
            mxg.mx_moe_topk_backward(score, xg, ids, to_gpu(dw), dl, renorm, 1.5)
            at = ids.cpu().numpy()

            def loss(y):
                ls = np.take_along_axis(log_scores(y, score), at, 1)
                w = np.exp(ls - (np.log(np.exp(ls).sum(1, keepdims=True)) if renorm else 0.0))
                return (1.5 * w * dw).sum(1)

            num = (loss(x + h * v) - loss(x - h * v)) / (2 * h)
            got = (dl.double().cpu().numpy() * v).sum(1)
            assert np.all(np.abs(got - num) <= 1e-4 * (1 + np.abs(num))), (score, renorm)


def test_topk_nan_and_infinity():
    """A NaN or -infinity is never chosen; a NaN reaches the weights only where they depend on it."""
    x = torch.tensor([[1.0, float("nan"), 3.0, -float("inf")], [float("nan")] * 4, [2.0, float("inf"), 1.0, 0.0]],
                     device="cuda")
    ids, w = mxg.moe_topk(SOFTMAX, x, 3, None, True)
    assert ids.tolist() == [[2, 0, -1], [-1, -1, -1], [1, 0, 2]]
    assert torch.isfinite(w[:2]).all() and w[1].tolist() == [0, 0, 0] and w[0, 2] == 0
    ids, w = mxg.moe_topk(SOFTMAX, x, 3, None, False)
    assert torch.isnan(w[0, :2]).all() and w[0, 2] == 0 and w[1].tolist() == [0, 0, 0]
    ids, w = mxg.moe_topk(SIGMOID, x, 2, None, False)
    assert ids.tolist() == [[2, 0], [-1, -1], [1, 0]] and w[2, 0] == 1.0 and torch.isfinite(w).all()
    bias = torch.tensor([0.0, 0.0, -float("inf"), 0.0], device="cuda")
    ids, _ = mxg.moe_topk(SIGMOID, x, 2, bias, True)
    assert ids.tolist() == [[0, -1], [-1, -1], [1, 0]]


def test_topk_backward_repeated_and_invalid_ids():
    rng = np.random.default_rng(2)
    x = rng.normal(0, 1, (4, 10))
    ids = np.array([[3, 3, 3], [1, -1, 1], [99, -7, 10], [0, 9, 0]], np.int32)
    dw = rng.normal(0, 1, (4, 3)).astype(np.float32)
    x32 = x.astype(np.float32)
    for score in (SOFTMAX, SIGMOID):
        for renorm in (False, True):
            dl = torch.full((4, 10), 9.0, device="cuda")
            mxg.mx_moe_topk_backward(score, to_gpu(x32), to_gpu(ids), to_gpu(dw), dl, renorm, 2.0)
            ref, mag = ref_topk_backward(x32.astype(np.float64), ids, dw.astype(np.float64), score, renorm, 2.0)
            assert np.all(np.abs(dl.cpu().numpy() - ref) <= mag * 100 * 2.0 ** -23 + 1e-30)


# ------------------------------------------------------------------ sort
def ref_sort(ids, E):
    flat = ids.reshape(-1)
    live = (flat >= 0) & (flat < E)
    order = np.flatnonzero(live)[np.argsort(flat[live], kind="stable")]
    off = np.zeros(E + 1, np.int64)
    off[1:] = np.cumsum(np.bincount(flat[live], minlength=E))
    ros = np.full(flat.size, -1, np.int32)
    ros[order] = np.arange(order.size, dtype=np.int32)
    sor = np.full(flat.size, -1, np.int32)
    sor[:order.size] = order
    return off, ros, sor


@pytest.mark.parametrize("S,k,E", [(1, 1, 1), (1, 8, 64), (7, 3, 5), (128, 8, 64), (512, 8, 128), (513, 8, 1024),
                                   (8191, 8, 100), (8192, 8, 128), (16411, 5, 17), (100003, 3, 9)])
@pytest.mark.parametrize("law", ["even", "one", "dropped", "none"])
def test_sort(S, k, E, law):
    rng = np.random.default_rng(S + E)
    ids = rng.integers(0, E, (S, k)).astype(np.int32)
    if law == "one":
        ids[:] = E - 1
    if law == "dropped":
        ids[rng.random((S, k)) < 0.3] = -1
        ids[rng.random((S, k)) < 0.1] = E
        ids[0, 0] = -2 ** 31
        ids[-1, -1] = 2 ** 31 - 1
    if law == "none":
        ids[:] = -1
    off_g, ros_g, sor_g = (Guarded(np.full(n, 123456, np.int32)) for n in (E + 1, S * k, S * k))
    mxg.mx_moe_sort(to_gpu(ids), off_g.view(), ros_g.view(), sor_g.view())
    torch.cuda.synchronize()
    off, ros, sor = ref_sort(ids, E)
    for g, want in ((off_g, off), (ros_g, ros), (sor_g, sor)):
        g.check()
        assert np.array_equal(g.numpy(), want)


@pytest.mark.parametrize("S,k,E", [(8193, 8, 256), (16411, 8, 128), (2063, 8, 1024), (70001, 1, 1), (70001, 1, 3),
                                   (140000, 1, 1000), (17000, 64, 64)])
@pytest.mark.parametrize("law", ["even", "one", "dropped", "none"])
def test_sort_of_many(S, k, E, law):
    """Lists that are cut into chunks: a last chunk longer than the others, counts of up to
    1024 experts, one expert or none with (nearly) all slots."""
    rng = np.random.default_rng(S + E)
    ids = rng.integers(0, E, (S, k)).astype(np.int32)
    if law == "one":
        ids[rng.random((S, k)) < 0.97] = E // 2
    elif law == "dropped":
        ids[rng.random((S, k)) < 0.3] = -1
        ids[rng.random((S, k)) < 0.1] = E
    elif law == "none":
        ids[:] = -5
    g = [Guarded(np.full(n, 7, np.int32)) for n in (E + 1, S * k, S * k)]
    mxg.mx_moe_sort(to_gpu(ids), *(x.view() for x in g))
    torch.cuda.synchronize()
    for got, want in zip(g, ref_sort(ids, E)):
        got.check()
        assert np.array_equal(got.numpy(), want)


def test_sort_of_many_in_a_graph_and_on_two_streams():
    """Replays with other ids, and two such sorts at once, give what the calls alone give."""
    S, k, E = 16411, 8, 200
    rng = np.random.default_rng(0)
    lists = [rng.integers(-1, E + 1, (S, k)).astype(np.int32) for _ in range(3)]
    want = [ref_sort(v, E) for v in lists]
    ids = to_gpu(lists[0])
    out = mxg.moe_sort(ids, E)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxg.mx_moe_sort(ids, *out)
    for i in (1, 2, 0, 1):
        ids.copy_(to_gpu(lists[i]))
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(out, want[i]):
            assert np.array_equal(got.cpu().numpy(), w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    gpu = [to_gpu(v) for v in lists]
    torch.cuda.synchronize()
    res = []
    for rep in range(4):
        for s, v in zip(streams, gpu):
            with torch.cuda.stream(s):
                res.append(mxg.moe_sort(v, E))
    torch.cuda.synchronize()
    for i, r in enumerate(res):
        for got, w in zip(r, want[i % 2]):
            assert np.array_equal(got.cpu().numpy(), w)


def test_sort_without_tokens():
    off = torch.full((6,), 9, dtype=torch.int32, device="cuda")
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    mxg.mx_moe_sort(torch.empty((0, 4), dtype=torch.int32, device="cuda"), off, none, none)
    assert off.tolist() == [0] * 6


# ------------------------------------------------------------------ permute and the gradients
def plan(S, k, E, dropped, seed):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (S, k)).astype(np.int32)
    ids[rng.random((S, k)) < dropped] = -1
    return ref_sort(ids, E)


SHAPES = [(1, 1, 8), (1, 8, 7168), (3, 2, 24), (50, 8, 2056), (37, 5, 4096), (200, 70, 520), (129, 4, 8192)]


@pytest.mark.parametrize("S,k,H", SHAPES)
@pytest.mark.parametrize("extra", [0, 3])
def test_permute(S, k, H, extra):
    off, ros, sor = plan(S, k, 9, 0.2, S + H)
    T = max(int(off[-1]) + extra, 1)
    rng = np.random.default_rng(H)
    x = rng.integers(-2 ** 15, 2 ** 15, (S, H)).astype(np.int16)  # every bit pattern, NaN among them
    before = np.full((T, H), 0x5A5A, np.int16)
    g = Guarded(before)
    mxg.mx_moe_permute(to_gpu(x).view(torch.bfloat16), to_gpu(ros), g.view(torch.bfloat16))
    torch.cuda.synchronize()
    g.check()
    want = before.copy()
    n = int(off[-1])
    want[:n] = x[sor[:n] // k]
    assert np.array_equal(g.numpy(), want)


@pytest.mark.parametrize("S,k,H", SHAPES)
def test_permute_backward(S, k, H):
    off, ros, _ = plan(S, k, 9, 0.2, S + H)
    T = max(int(off[-1]), 1)
    rng = np.random.default_rng(H + 1)
    d_t, d = bf16(rng.normal(0, 1, (T, H)) * np.exp(rng.uniform(-3, 3, (T, 1))))
    g = Guarded(np.full((S, H), 0x5A5A, np.int16))
    mxg.mx_moe_permute_backward(d_t, to_gpu(ros), g.view(torch.bfloat16))
    torch.cuda.synchronize()
    g.check()
    want, mag = np.zeros((S, H)), np.zeros((S, H))
    for j, r in enumerate(ros):
        if r >= 0:
            want[j // k] += d[r]
            mag[j // k] += np.abs(d[r])
    got = g.view(torch.bfloat16).double().cpu().numpy()
    assert np.all(np.abs(got - want) <= half_step_bf16(want) + (k + 1) * 2.0 ** -24 * mag)


@pytest.mark.parametrize("S,k,H", SHAPES)
def test_combine_backward(S, k, H):
    off, ros, _ = plan(S, k, 9, 0.2, S + H)
    ros = ros.copy()
    T = max(int(off[-1]), 1)
    if ros.size > 4 and off[-1] > 2:
        ros[np.flatnonzero(ros == off[-1] - 1)] = T + 5  # a slot past the rows: dropped, its row left as it was
    rng = np.random.default_rng(H + 2)
    do_t, do = bf16(rng.normal(0, 1, (S, H)))
    y_t, y = bf16(rng.normal(0, 1, (T, H)))
    w = rng.normal(0, 1, S * k).astype(np.float32)
    before = np.full((T, H), 0x5A5A, np.int16)
    dy_g, dw_g = Guarded(before), Guarded(np.full(S * k, 7.0, np.float32))
    mxg.mx_moe_combine_backward(do_t, y_t, to_gpu(ros), to_gpu(w), dy_g.view(torch.bfloat16), dw_g.view())
    torch.cuda.synchronize()
    dy_g.check(), dw_g.check()
    got_dy, got_dw = dy_g.view(torch.bfloat16).double().cpu().numpy(), dw_g.numpy()
    named = np.zeros(T, bool)
    terms = 8 * -(-H // 2048) + 12  # fp32 additions on the longest path
    for j, r in enumerate(ros):
        if 0 <= r < T:
            named[r] = True
            want = float(w[j]) * do[j // k]
            assert np.all(np.abs(got_dy[r] - want) <= half_step_bf16(want) * (1 + 2.0 ** -14))
            prod = do[j // k] * y[r]
            assert abs(got_dw[j] - prod.sum()) <= terms * 2.0 ** -24 * np.abs(prod).sum()
        else:
            assert got_dw[j] == 0.0
    assert np.all(dy_g.numpy()[~named] == 0x5A5A)


def test_combine_gradient_against_differences():
    """sum(combine(y, w) * dout) is linear in y and in w: a difference along a direction is the gradient's product."""
    S, k, H = 16, 4, 256
    off, ros, _ = plan(S, k, 8, 0.1, 4)
    T = int(off[-1])
    rng = np.random.default_rng(9)
    do_t, do = bf16(rng.normal(0, 1, (S, H)))
    y_t, y = bf16(rng.normal(0, 1, (T, H)))
    w = rng.uniform(0.1, 1, S * k).astype(np.float32)
    dy, dw = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda"), torch.empty(S * k, device="cuda")
    mxg.mx_moe_combine_backward(do_t, y_t, to_gpu(ros), to_gpu(w), dy, dw)

    def loss(yy, ww):
        return sum(float(ww[j]) * (yy[r] * do[j // k]).sum() for j, r in enumerate(ros) if r >= 0)

    vy, vw = rng.normal(0, 1, (T, H)), rng.normal(0, 1, S * k)
    num_y, num_w = loss(y + vy, w) - loss(y, w), loss(y, w + vw) - loss(y, w.astype(np.float64))
    dy64, dw64 = dy.double().cpu().numpy(), dw.double().cpu().numpy()
    assert abs((dy64 * vy).sum() - num_y) <= (np.abs(dy64 * vy) * 2.0 ** -8).sum() + 1e-9
    assert abs((dw64 * vw).sum() - num_w) <= (np.abs(dw64 * vw)).sum() * 40 * 2.0 ** -24 + 1e-3


def test_outputs_over_inputs_are_refused():
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    a, b = torch.zeros((2, 8), dtype=torch.int32, device="cuda")
    x = torch.zeros((4, 2), device="cuda")
    y, d = torch.zeros((2, 4, 8), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(8, device="cuda")
    for call in (lambda: mxg.mx_moe_sort(ids, off, ids.view(-1), b), lambda: mxg.mx_moe_sort(ids, off, a, ids.view(-1)),
                 lambda: mxg.mx_moe_sort(ids, off, a, a),
                 lambda: mxg.mx_moe_topk_backward(SOFTMAX, x, ids, w.view(4, 2), x),
                 lambda: mxg.mx_moe_topk_backward(SOFTMAX, x, ids, w.view(4, 2), w.view(4, 2)),
                 lambda: mxg.mx_moe_permute(y, a, y), lambda: mxg.mx_moe_permute_backward(y, a, y),
                 lambda: mxg.mx_moe_combine_backward(y, d, a, w, d, w.clone()),
                 lambda: mxg.mx_moe_combine_backward(y, d, a, w, torch.empty_like(d), w)):
        with pytest.raises(ValueError, match="overlap"):
            call()


def test_repeated_rows_are_refused_under_validation(monkeypatch):
    x = torch.zeros((2, 8), dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")
    dy, f = torch.zeros_like(rows), torch.zeros(4, device="cuda")
    twice = torch.tensor([0, 1, 1, -1], dtype=torch.int32, device="cuda")
    once = torch.tensor([0, 1, 2, -1], dtype=torch.int32, device="cuda")
    monkeypatch.setenv("MXG_VALIDATE", "1")
    mxg.mx_moe_permute(x, once, rows)
    mxg.mx_moe_combine_backward(x, rows, once, f, dy, f.clone())
    assert mxg.validation_message() == ""
    for call in (lambda: mxg.mx_moe_permute(x, twice, rows),
                 lambda: mxg.mx_moe_combine_backward(x, rows, twice, f, dy, f.clone())):
        with pytest.raises(mxg.MxgError) as e:
            call()
        assert e.value.status == mxg.ERROR_INVALID_VALUE and "again" in mxg.validation_message()


def test_row_offsets_past_32_bits():
    """Rows whose elements lie past 2^32 bytes: the copies and sums reach them."""
    H, T = 8192, 280_000  # 4.6 GB
    rows = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((3, H), device="cuda").to(torch.bfloat16)
    ros = torch.tensor([T - 1, 5, T - 2], dtype=torch.int32, device="cuda")
    mxg.mx_moe_permute(x, ros, rows)
    assert torch.equal(rows[[T - 1, 5, T - 2]], x)
    dx = torch.empty_like(x)
    mxg.mx_moe_permute_backward(rows, ros, dx)
    assert torch.equal(dx, x)
    dy, dw = torch.zeros_like(rows), torch.empty(3, device="cuda")
    mxg.mx_moe_combine_backward(x, rows, ros, torch.ones(3, device="cuda"), dy, dw)
    assert torch.equal(dy[[T - 1, 5, T - 2]], x)
