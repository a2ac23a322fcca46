"""FP8 with a scale per block of 128: the quantisers bit for bit against numpy and
the oracle's e4m3 encoder, the grouped GEMM and SwiGLU against 64 bits.

GEMM tolerance.  The FP8 matrix core adds eight consecutive products at a time,
aligned to the largest of them: measured with a large product, its negative and
a small one of 2^-j times it in each place, the small one survives exactly at j <=
12 and is lost from j = 14 on among those eight, while across eights the sum
keeps fp32's 24 bits.  A product is therefore cut by less than 2^-12 of the
largest of its eight, eight of them by less than 2^-9 of it; the largest is at
most the product of the two operands' largest magnitudes there.  The 16 eights
of a block, the blocks' additions, the two scales' product and its product with
the block round to fp32: 16 + nb + 3 times 2^-24 of the sum of magnitudes.  The
result is rounded to bf16 by half a step, 2^-8 of the value (2^-134 at zero).

SwiGLU: the sigmoid is off by (|g| + 4) 2^-23 relative (its argument's two
roundings, exp2, the sum, the reciprocal), see each check."""
import numpy as np
import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg
import oracle
from common import Guarded, bits, offsets_gpu, to_gpu

pytestmark = pytest.mark.gpu

B = 128


def nblk(n):
    return -(-n // B)


def bf16_values(bits16):
    return oracle.bf16_value_array(bits16)


def e4m3(v):
    return oracle.e4m3_encode_array(np.asarray(v, np.float64))


def ref_rows(x):
    """x fp32 [T, K] -> (codes u8, scales fp32) by IEEE fp32 divisions."""
    T, K = x.shape
    q, s = np.zeros((T, K), np.uint8), np.zeros((T, nblk(K)), np.float32)
    for b in range(nblk(K)):
        v = x[:, b * B:(b + 1) * B].astype(np.float32)
        s[:, b] = np.abs(v).max(1) / np.float32(448)
        with np.errstate(divide="ignore", invalid="ignore"):
            quo = np.where(s[:, b:b + 1] > 0, v / s[:, b:b + 1], v * np.float32(0))
        q[:, b * B:(b + 1) * B] = e4m3(quo).reshape(v.shape)
    return q, s


def activations(T, K, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (T, K)) * np.exp(rng.uniform(-6, 6, (T, 1)))
    x[:, rng.integers(0, K, max(1, K // 50))] *= 30
    x[rng.random((T, K)) < 0.02] = 0.0
    if T > 2:
        x[1] = 0.0                                   # a row of zeros
        x[2, :min(K, B)] = -0.0                      # a block of negative zeros
    if T > 4:
        x[3, :min(K, B)] = 2.0 ** -133               # bf16's smallest subnormal
        x[4, 0] = 3.3e38                             # the largest binade
    t = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)
    return t, t.float().numpy()


KS = [32, 96, 128, 160, 1024, 2048 + 32, 4096, 7168]


@pytest.mark.parametrize("T,K", [(1, 32), (5, 96), (7, 128), (6, 160), (33, 1024), (9, 2080), (5, 4096), (3, 7168)])
def test_quantize_rows(T, K):
    x_t, x = activations(T, K, K)
    off = np.array([0, T // 3, T // 3, T], np.uint32)
    q_g, s_g = Guarded(np.full((T, K), 0xA5, np.uint8)), Guarded(np.full((T, nblk(K)), 7.0, np.float32))
    mxg.mx_grouped_quantize_block128(x_t.cuda(), q_g.view(), s_g.view(), offsets_gpu(off))
    torch.cuda.synchronize()
    q_g.check(), s_g.check()
    q, s = ref_rows(x)
    assert np.array_equal(s_g.numpy().view(np.uint32), s.view(np.uint32))
    assert np.array_equal(q_g.numpy(), q)


@pytest.mark.parametrize("exponent", [1, 20, 66, 67, 100, 127, 200, 254])
def test_quantize_every_quotient(exponent):
    """Every bf16 magnitude of the ten binades below a block's maximum (below that
    the codes are 0), under maxima of every mantissa, in binades from the smallest
    normals to the largest: the codes of IEEE division, bit for bit."""
    rows = []
    for m in range(128):
        amax = (exponent << 7) | m
        vals = np.arange(max(0, amax - 1280), amax + 1)
        vals = np.concatenate([vals, np.full(-len(vals) % 127, amax)]).reshape(-1, 127)
        rows.append(np.concatenate([vals, np.full((len(vals), 1), amax)], 1))
    xb = np.concatenate(rows).astype(np.uint16)
    xb[1::2] |= 0x8000  # both signs
    x = bf16_values(xb).astype(np.float32).reshape(xb.shape)
    q, s = ref_rows(x)
    got_q, got_s = mxg.quantize_block128(to_gpu(xb.view(np.int16)).view(torch.bfloat16),
                                         offsets_gpu(np.array([0, len(xb)], np.uint32)))
    assert np.array_equal(got_s.cpu().numpy(), s) and np.array_equal(got_q.cpu().numpy(), q)


def test_quantize_uncovered_rows_stay():
    T, K = 12, 256
    x_t, x = activations(T, K, 1)
    off = np.array([2, 5, 4, 9], np.uint32)  # [2, 5) taken, [5, 4) inverted, [4, 9) taken
    q_t = torch.full((T, K), 0xA5, dtype=torch.uint8, device="cuda")
    s_t = torch.full((T, 2), 7.0, device="cuda")
    mxg.mx_grouped_quantize_block128(x_t.cuda(), q_t, s_t, offsets_gpu(off))
    q, s = ref_rows(x)
    cov = np.zeros(T, bool)
    cov[2:9] = True
    assert np.array_equal(q_t.cpu().numpy()[cov], q[cov]) and np.array_equal(s_t.cpu().numpy()[cov], s[cov])
    assert torch.all(q_t[torch.from_numpy(~cov).cuda()] == 0xA5) and torch.all(s_t[torch.from_numpy(~cov).cuda()] == 7)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_non_finite_block(bad):
    x = torch.ones((2, 384), dtype=torch.bfloat16, device="cuda")
    x[0, 200] = bad
    q, s = mxg.quantize_block128(x, offsets_gpu(np.array([0, 2], np.uint32)))
    fin = torch.isfinite(s).cpu().numpy()
    assert np.array_equal(fin, [[True, False, True], [True, True, True]])
    w = torch.ones((1, 128, 384), dtype=torch.bfloat16, device="cuda")
    bq, bs = mxg.quantize_weights_block128(w)
    c = mxg.grouped_matmul_block128(q, s, bq, bs, offsets_gpu(np.array([0, 2], np.uint32)),
                                    torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert not torch.isfinite(c[0]).any() and torch.isfinite(c[1]).all()


@pytest.mark.parametrize("S,k,K", [(1, 8, 2080), (9, 3, 128), (40, 8, 4096), (5, 64, 96)])
def test_quantize_scatter(S, k, K):
    rng = np.random.default_rng(S)
    x_t, x = activations(S, K, K + S)
    T = S * k
    ros = rng.permutation(T).astype(np.int32)
    ros[rng.random(T) < 0.2] = -1
    ros[0] = T + 3
    hi = max(1, T - 2)
    off = np.array([0, hi], np.uint32)  # the last rows are covered by no group
    q_g, s_g = Guarded(np.full((T, K), 0xA5, np.uint8)), Guarded(np.full((T, nblk(K)), 7.0, np.float32))
    mxg.mx_grouped_quantize_block128_scatter(x_t.cuda(), to_gpu(ros), q_g.view(), s_g.view(), offsets_gpu(off))
    torch.cuda.synchronize()
    q_g.check(), s_g.check()
    q, s = ref_rows(x)
    want_q, want_s = np.full((T, K), 0xA5, np.uint8), np.full((T, nblk(K)), 7.0, np.float32)
    for j, r in enumerate(ros):
        if 0 <= r < hi:
            want_q[r], want_s[r] = q[j // k], s[j // k]
    assert np.array_equal(q_g.numpy(), want_q) and np.array_equal(s_g.numpy(), want_s)


@pytest.mark.parametrize("E,N,K", [(1, 32, 32), (2, 128, 256), (3, 160, 416), (1, 1, 64), (2, 100, 160), (1, 512, 1056)])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_weights(E, N, K, transposed):
    if transposed and N % 32:
        with pytest.raises(mxg.MxgError):
            mxg.quantize_weights_block128(torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda"), True)
        return
    rng = np.random.default_rng(N + K)
    w_t = torch.from_numpy((0.02 * rng.normal(0, 1, (E, N, K))).astype(np.float32)).to(torch.bfloat16)
    w_t[0, :min(N, 128), :min(K, 128)] = 0.0
    w = w_t.float().numpy()
    q = np.zeros((E, N, K), np.uint8)
    s = np.zeros((E, nblk(N), nblk(K)), np.float32)
    for e in range(E):
        for i in range(nblk(N)):
            for j in range(nblk(K)):
                blk = w[e, i * B:(i + 1) * B, j * B:(j + 1) * B]
                s[e, i, j] = np.abs(blk).max() / np.float32(448)
                quo = blk / s[e, i, j] if s[e, i, j] > 0 else blk * np.float32(0)
                q[e, i * B:(i + 1) * B, j * B:(j + 1) * B] = e4m3(quo).reshape(blk.shape)
    gq, gs = Guarded(np.full(q.shape, 0xA5, np.uint8)), Guarded(np.full(s.shape, 7.0, np.float32))
    if transposed:
        gt, gst = Guarded(np.full((E, K, N), 0xA5, np.uint8)), Guarded(np.full((E, nblk(K), nblk(N)), 7.0, np.float32))
        mxg.mx_quantize_weights_block128(w_t.cuda(), gq.view(), gs.view(), gt.view(), gst.view())
        torch.cuda.synchronize()
        gt.check(), gst.check()
        assert np.array_equal(gt.numpy(), q.transpose(0, 2, 1)) and np.array_equal(gst.numpy(), s.transpose(0, 2, 1))
    else:
        mxg.mx_quantize_weights_block128(w_t.cuda(), gq.view(), gs.view())
        torch.cuda.synchronize()
    gq.check(), gs.check()
    assert np.array_equal(gs.numpy(), s) and np.array_equal(gq.numpy(), q)


# ------------------------------------------------------------------ GEMM
def operands(T, E, N, K, seed):
    """Codes of every finite e4m3 value, scales over a few binades (some zero)."""
    rng = np.random.default_rng(seed)

    def codes(shape):
        c = rng.integers(0, 127, shape, dtype=np.uint8)
        return c | (rng.integers(0, 2, shape, dtype=np.uint8) << 7)

    def scl(shape):
        s = np.exp(rng.uniform(-4, 1, shape)).astype(np.float32)
        s[rng.random(shape) < 0.03] = 0.0
        return s

    return codes((T, K)), scl((T, nblk(K))), codes((E, N, K)), scl((E, nblk(N), nblk(K)))


def check_gemm(T, E, N, K, off, ids, seed=0, hint=0):
    a, sa, b, sb = operands(T, E, N, K, seed)
    before = np.full((T, N), 0x5A5A, np.int16)
    g = Guarded(before)
    mxg.mx_grouped_matmul_block128(to_gpu(a), to_gpu(sa), to_gpu(b), to_gpu(sb), g.view(torch.bfloat16),
                                   offsets_gpu(np.asarray(off, np.uint32)), to_gpu(np.asarray(ids, np.int32)), hint)
    torch.cuda.synchronize()
    g.check()
    got = g.view(torch.bfloat16).double()
    val = torch.from_numpy(oracle.e4m3_value_array(np.arange(256, dtype=np.uint8))).cuda()
    kb = torch.arange(K, device="cuda") // B
    nb = torch.arange(N, device="cuda") // B
    cov = np.zeros(T, bool)
    for g_i, e in enumerate(ids):
        lo, hi = min(int(off[g_i]), T), min(int(off[g_i + 1]), T)
        if hi <= lo or e < 0 or e >= E:
            continue
        cov[lo:hi] = True
        av = val[to_gpu(a[lo:hi]).long()] * to_gpu(sa[lo:hi]).double()[:, kb]
        bv = val[to_gpu(b[e]).long()] * to_gpu(sb[e]).double()[nb][:, kb]
        want, mag = av @ bv.t(), av.abs() @ bv.abs().t()
        eights = av.abs().reshape(hi - lo, K // 8, 8).amax(2) @ bv.abs().reshape(N, K // 8, 8).amax(2).t()
        tol = (want.abs() * 2.0 ** -8 + 2.0 ** -134 + eights * 2.0 ** -9 + mag * (16 + nblk(K) + 3) * 2.0 ** -24)
        err = (got[lo:hi] - want).abs()
        assert bool(torch.all(err <= tol)), (g_i, float((err / tol).max()))
    assert np.array_equal(g.numpy()[~cov], before[~cov])
    return g


@pytest.mark.parametrize("K", KS)
@pytest.mark.parametrize("T,N", [(1, 256), (3, 8), (20, 130), (70, 1000), (300, 513), (700, 384)])
def test_gemm_sizes(T, N, K):
    check_gemm(T, 2, N, K, [0, T // 3, T], [1, 0], seed=T + N + K)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 256, 257])
def test_gemm_rows_of_one_group(T):
    check_gemm(T, 1, 264, 384, [0, T], [0], seed=T)


@pytest.mark.parametrize("N", [1, 2, 7, 15, 17, 64, 100, 127, 129, 255, 257, 300, 511])
def test_gemm_columns(N):
    check_gemm(40, 2, N, 288, [0, 11, 40], [0, 1], seed=N)
    check_gemm(300, 1, N, 288, [0, 300], [0], seed=N)


def test_gemm_ragged():
    """Empty groups, repeated, permuted and out-of-range experts, gaps, inverted and past-the-end offsets."""
    T = 900
    check_gemm(T, 6, 520, 640, [0, 0, 300, 301, 301, 640, 900, 900], [5, 3, 3, 0, 1, 2, 4])
    check_gemm(T, 6, 520, 640, [5, 200, 150, 400, 2000], [5, 2, -1, 6])
    check_gemm(T, 6, 520, 640, [100, 100, 100], [5, 2])
    check_gemm(T, 3, 264, 256, [0, 100, 400, 100], [0, 1, 2])
    check_gemm(T, 3, 264, 256, [0, 100, 1 << 31], [0, 1])


@pytest.mark.parametrize("T,E", [(4100, 3), (16500, 5)])
@pytest.mark.parametrize("N,K", [(1000, 32), (1030, 288), (1001, 160), (776, 1152), (256, 2080)])
def test_gemm_larger_tiles(T, E, N, K):
    """Enough rows for the 128- and 256-row tiles (the sizes above run the row
    kernel and the 32-row tiles): partial tiles, a group of one row, an empty one,
    split last rounds, columns that fill no tile, one stage and many."""
    cuts = sorted(np.random.default_rng(T + N).integers(0, T, E - 2).tolist())
    off = [0, 1] + cuts + [cuts[-1] if cuts else 1, T]
    ids = [i % E for i in range(len(off) - 1)]
    check_gemm(T, E, N, K, off, ids, seed=N)


def test_gemm_kernels_agree():
    """One group's rows through every kernel the sizes around it select: each kernel
    keeps a row's sum to itself, so more rows beside it change at most the last bit
    (the row kernel joins its waves' sums in another order)."""
    N, K, E = 520, 1184, 2
    a, sa, b, sb = (to_gpu(v) for v in operands(16400, E, N, K, 21))
    ids = to_gpu(np.array([1], np.int32))
    ref = None
    for T in (3, 40, 5000, 16400):
        c = mxg.grouped_matmul_block128(a[:T].contiguous(), sa[:T].contiguous(), b, sb,
                                        offsets_gpu(np.array([0, T], np.uint32)), ids)[:3].double()
        if ref is None:
            ref = c
        # a neighbour in bf16 where the fp32 sums straddle a rounding border
        assert bool(((c - ref).abs() <= ref.abs() * 2.0 ** -7 + 1e-3 * ref.abs().amax()).all())


def test_gemm_many_groups():
    rng = np.random.default_rng(3)
    G = 1024
    off = np.concatenate([[0], np.cumsum(rng.integers(0, 4, G))])
    check_gemm(int(off[-1]), 7, 136, 160, off, rng.integers(0, 7, G))


@pytest.mark.parametrize("K", [4096, 8192, 4128])
@pytest.mark.parametrize("T,E,N", [(1500, 40, 520), (4100, 3, 1000), (40, 2, 264)])
def test_gemm_rows_of_whole_pages(K, T, E, N):
    """Rows a multiple of 4096 bytes apart, where tiles begin each at another block of K."""
    rng = np.random.default_rng(K + T)
    off = np.concatenate([[0], np.sort(rng.integers(0, T + 1, E - 1)), [T]])
    check_gemm(T, E, N, K, off, rng.permutation(E), seed=T)


@pytest.mark.parametrize("law", ["one", "two", "falling", "edges"])
@pytest.mark.parametrize("T,G,N,K", [(256, 64, 520, 416), (900, 256, 1024, 128), (4096, 1024, 1000, 96), (17, 5, 33, 64),
                                     (60, 16, 64, 1184)])
def test_gemm_few_rows_unevenly(T, G, N, K, law):
    """Few rows a group on average, many in some: what lies past 16 rows of a group, past the
    groups the grid holds at once, and a last block of one row."""
    rng = np.random.default_rng(T + G)
    sizes = np.zeros(G, np.int64)
    if law == "one":
        sizes[G // 2] = T
    elif law == "two":
        sizes[[0, G - 1]] = T // 2, T - T // 2
    elif law == "falling":
        p = (1.0 + np.arange(G)) ** -1.3
        sizes = rng.multinomial(T, p / p.sum())
    else:
        left = T
        for i, n in enumerate((16, 17, 15, 32, 33, 1, 0, 48, 49)):
            if i < G and n <= left:
                sizes[i] = n
                left -= n
    off = np.concatenate([[0], np.cumsum(sizes)])
    check_gemm(T, 5, N, K, off, rng.integers(-1, 6, G), seed=K)


@pytest.mark.parametrize("most,N,K", [(128, 256, 160), (391, 512, 32)])
def test_gemm_many_groups_of_larger_tiles(most, N, K):
    """As many groups as there may be, of 0 to `most` rows: the 128- and the 256-row tiles."""
    rng = np.random.default_rng(most)
    G = 1024
    sizes = rng.integers(0, most + 1, G)
    sizes[[0, 1, G - 1]] = 0, 1, 0
    off = np.concatenate([[0], np.cumsum(sizes)])
    check_gemm(int(off[-1]) + 5, 7, N, K, off, rng.integers(0, 7, G))


@pytest.mark.parametrize("hint", [0, 1, 64, 1 << 20, 1 << 62])
def test_gemm_hint(hint):
    check_gemm(150, 5, 264, 512, [0, 10, 20, 140, 150], [0, 1, 2, 3], hint=hint)


def test_gemm_weights_past_32_bits():
    """The last of weights of more than 2^32 bytes."""
    E, N, K = 300, 4096, 4096  # 5 GB
    b = torch.full((E, N, K), 0x38, dtype=torch.uint8, device="cuda")  # ones
    b[E - 1] = 0x40                                                      # twos
    bs = torch.ones((E, 32, 32), device="cuda")
    a = torch.full((3, K), 0x38, dtype=torch.uint8, device="cuda")
    sa = torch.ones((3, 32), device="cuda")
    off = offsets_gpu(np.array([0, 1, 3], np.uint32))
    for hint in (0, 1 << 20):
        c = mxg.grouped_matmul_block128(a, sa, b, bs, off, to_gpu(np.array([0, E - 1], np.int32)), hint)
        assert torch.all(c[0] == K) and torch.all(c[1:] == 2 * K)


def test_gemm_is_deterministic_and_streams():
    """The same bits on a side stream, on the default stream and twice over, with other work between."""
    T, E, N, K = 333, 4, 392, 1120
    a, sa, b, sb = (to_gpu(v) for v in operands(T, E, N, K, 8))
    off, ids = offsets_gpu(np.array([0, 100, 101, 333], np.uint32)), to_gpu(np.array([2, 0, 3], np.int32))
    first = mxg.grouped_matmul_block128(a, sa, b, sb, off, ids)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = mxg.grouped_matmul_block128(a, sa, b, sb, off, ids)
        third = mxg.grouped_matmul_block128(a, sa, b, sb, off, ids)
    fourth = mxg.grouped_matmul_block128(a, sa, b, sb, off, ids)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for other in (second, third, fourth):
        assert torch.equal(first.view(torch.int16), other.view(torch.int16))


# ------------------------------------------------------------------ SwiGLU
def gate_up(T, I, seed):
    rng = np.random.default_rng(seed)
    h = rng.normal(0, 2, (T, 2 * I))
    h[0, 0::2] = rng.uniform(-100, 100, I)  # gates whose sigmoid saturates
    if T > 1:
        h[1] = 0.0
    t = torch.from_numpy(h.astype(np.float32)).to(torch.bfloat16)
    return t, t.double().numpy()


def sig(g):
    return 1.0 / (1.0 + np.exp(-g))


def check_requant(q, s, v, err):
    """Codes q u8 and scales s fp32 of exact values v, each formed to within err: the
    scale is one formed maximum / 448 (one more rounding), each code the nearest to
    its formed quotient (half a step: 2^-4 of it, 2^-10 below 2^-6)."""
    T, K = v.shape
    for b in range(nblk(K)):
        sl = slice(b * B, (b + 1) * B)
        top, slack = np.abs(v[:, sl]).max(1), err[:, sl].max(1)
        sb = s[:, b].astype(np.float64)
        assert np.all(np.abs(sb * 448 - top) <= slack + top * 2.0 ** -23 + 448 * 2.0 ** -149)
        val = oracle.e4m3_value_array(q[:, sl]).reshape(T, -1)
        quo = np.where(sb[:, None] > 0, v[:, sl] / np.where(sb > 0, sb, 1)[:, None], 0)
        slack_q = np.where(sb[:, None] > 0, err[:, sl] / np.where(sb > 0, sb, 1)[:, None], 0)
        half = np.maximum(np.abs(quo) * 2.0 ** -4, 2.0 ** -10)
        assert np.all(np.abs(val - quo) <= half * (1 + 2.0 ** -10) + 2 * slack_q)


@pytest.mark.parametrize("T,I", [(1, 32), (3, 96), (5, 128), (7, 544), (40, 2048), (300, 160)])
def test_silu_quantize(T, I):
    h_t, h = gate_up(T, I, I)
    off = np.array([0, T // 2, T], np.uint32)
    q_g, s_g = Guarded(np.full((T, I), 0xA5, np.uint8)), Guarded(np.full((T, nblk(I)), 7.0, np.float32))
    mxg.mx_silu_quantize_block128(h_t.cuda(), q_g.view(), s_g.view(), offsets_gpu(off))
    torch.cuda.synchronize()
    q_g.check(), s_g.check()
    g, u = h[:, 0::2], h[:, 1::2]
    y = g * sig(g) * u
    err = np.abs(y) * (np.abs(g) + 6) * 2.0 ** -23 + np.abs(g * u) * 2.0 ** -125
    check_requant(q_g.numpy(), s_g.numpy(), y, err)


@pytest.mark.parametrize("T,I", [(1, 32), (3, 96), (5, 128), (7, 544), (40, 2048), (300, 160)])
@pytest.mark.parametrize("keep,quant,inplace", [(True, True, False), (True, False, True), (False, True, False)])
def test_silu_backward(T, I, keep, quant, inplace):
    h_t, h = gate_up(T, I, I + 1)
    rng = np.random.default_rng(I + 2)
    dy_t = torch.from_numpy(rng.normal(0, 0.3, (T, I)).astype(np.float32)).to(torch.bfloat16)
    dy = dy_t.double().numpy()
    off = np.array([0, T // 2, T], np.uint32)
    hg = Guarded(bits(h_t).view(np.int16))
    dh_g = hg if inplace else Guarded(np.full((T, 2 * I), 0x5A5A, np.int16))
    q_g, s_g = Guarded(np.full((T, 2 * I), 0xA5, np.uint8)), Guarded(np.full((T, nblk(2 * I)), 7.0, np.float32))
    mxg.mx_silu_backward_block128(hg.view(torch.bfloat16), dy_t.cuda(), offsets_gpu(off),
                                  dh=dh_g.view(torch.bfloat16) if keep else None,
                                  dh_q=q_g.view() if quant else None, dh_scales=s_g.view() if quant else None)
    torch.cuda.synchronize()
    hg.check(), dh_g.check(), q_g.check(), s_g.check()
    g, u = h[:, 0::2], h[:, 1::2]
    s = sig(g)
    want, err = np.empty_like(h), np.empty_like(h)
    want[:, 0::2], want[:, 1::2] = dy * u * s * (1 + g * (1 - s)), dy * g * s
    # s off by (|g| + 4) 2^-23 relative; 1 - s by that of s and a rounding, times |g|; four products
    err[:, 0::2] = np.abs(dy * u) * (s * (1 + np.abs(g)) * (np.abs(g) + 8) * 2.0 ** -22 + (1 + np.abs(g)) * 2.0 ** -125)
    err[:, 1::2] = np.abs(dy * g) * (s * (np.abs(g) + 6) * 2.0 ** -23 + 2.0 ** -125)
    if keep:
        got = dh_g.view(torch.bfloat16).double().cpu().numpy()
        assert np.all(np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + 2.0 ** -134 + err * (1 + 2.0 ** -7))
    if quant:
        check_requant(q_g.numpy(), s_g.numpy(), want, err)


def test_silu_gradient_against_differences():
    """d/dt sum(swiglu(h + t v) dy) by central differences in 64 bits, step 1e-4; the kept
    gradient is rounded to bf16, 2^-8 of each term."""
    T, I, st = 8, 256, 1e-4
    h_t, _ = gate_up(T, I, 3)
    rng = np.random.default_rng(4)
    h_t[0] = h_t[2]
    h = h_t.double().numpy()
    dy_t = torch.from_numpy(rng.normal(0, 1, (T, I)).astype(np.float32)).to(torch.bfloat16)
    dy, v = dy_t.double().numpy(), rng.normal(0, 1, (T, 2 * I))
    dh = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda")
    mxg.mx_silu_backward_block128(h_t.cuda(), dy_t.cuda(), offsets_gpu(np.array([0, T], np.uint32)), dh=dh)

    def loss(x):
        return (x[:, 0::2] * sig(x[:, 0::2]) * x[:, 1::2] * dy).sum(1)

    num = (loss(h + st * v) - loss(h - st * v)) / (2 * st)
    d = dh.double().cpu().numpy()
    assert np.all(np.abs((d * v).sum(1) - num) <= (np.abs(d * v) * 2.0 ** -8).sum(1) + 1e-5)


def test_silu_uncovered_rows_stay():
    T, I = 9, 64
    h_t, _ = gate_up(T, I, 5)
    off = offsets_gpu(np.array([2, 4, 3, 6], np.uint32))
    q, s = torch.full((T, I), 0xA5, dtype=torch.uint8, device="cuda"), torch.full((T, 1), 7.0, device="cuda")
    mxg.mx_silu_quantize_block128(h_t.cuda(), q, s, off)
    out = torch.tensor([0, 1, 6, 7, 8], device="cuda")
    assert torch.all(q[out] == 0xA5) and torch.all(s[out] == 7) and not torch.any(s[2:6] == 7)
    dh = torch.full((T, 2 * I), 5.0, dtype=torch.bfloat16, device="cuda")
    mxg.mx_silu_backward_block128(h_t.cuda(), torch.ones((T, I), dtype=torch.bfloat16, device="cuda"), off, dh=dh)
    assert torch.all(dh[out] == 5.0)
