"""Codes of a 128-block that holds an infinity or a NaN, from every quantiser of
the block-128 format.  The definition gives them: the scale is amax / 448, not
finite here, and a code is e4m3 of the IEEE quotient x / scale, so under an
infinite scale a finite value has the zero of its sign and an infinity a NaN;
under a NaN all are NaN.  Nothing is rounded: codes are compared bit for bit (a
NaN without its sign)."""
import numpy as np
import pytest
import torch

import fp4_grouped_gemm_quantize_amd as mxg
import oracle
from common import offsets_gpu, to_gpu

pytestmark = pytest.mark.gpu

B = 128
BAD = {"inf": [np.inf], "-inf": [-np.inf], "both": [np.inf, -np.inf], "nan": [np.nan], "nan and inf": [np.nan, np.inf]}


def quotients(x, scales):
    """IEEE fp32 x / scale, scale repeated over its block."""
    with np.errstate(divide="ignore", invalid="ignore"):
        return np.where(scales == 0, x * np.float32(0), x / scales).astype(np.float32)


def check_codes(codes, quo):
    nan = np.isnan(quo)
    assert np.all((codes[nan] & 0x7F) == 0x7F)
    assert np.array_equal(codes[~nan], oracle.e4m3_encode_array(quo[~nan].astype(np.float64)).reshape(-1))


def rows_with(bad, T, K, seed):
    """bf16 rows, as fp32, whose second block (and the last row's last one) holds the values `bad`."""
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(0, 1, (T, K)).astype(np.float32)).to(torch.bfloat16).float().numpy()
    x[0, 3] = 0.0
    x[0, 200], x[1, 200] = 3e38, -0.0
    for j, v in enumerate(bad):
        x[:T - 1, 130 + 5 * j] = v
        x[T - 1, K - 1 - j] = v
    return x


def row_scales(x):
    K = x.shape[1]
    return np.stack([np.abs(x[:, b:b + B]).max(1) for b in range(0, K, B)], 1) / np.float32(448)


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("K", [256, 416])
def test_rows(bad, K):
    x = rows_with(BAD[bad], 5, K, K)
    q, s = mxg.quantize_block128(to_gpu(x).to(torch.bfloat16), offsets_gpu(np.array([0, 5], np.uint32)))
    want = row_scales(x)
    assert np.array_equal(s.cpu().numpy(), want, equal_nan=True)
    check_codes(q.cpu().numpy(), quotients(x, np.repeat(want, B, 1)[:, :K]))


@pytest.mark.parametrize("bad", BAD)
def test_scatter(bad):
    S, k, K = 3, 2, 288
    x = rows_with(BAD[bad], S, K, 1)
    ros = np.array([4, 0, 3, 5, 1, 2], np.int32)
    q = torch.empty((S * k, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((S * k, 3), device="cuda")
    mxg.mx_grouped_quantize_block128_scatter(to_gpu(x).to(torch.bfloat16), to_gpu(ros), q, s,
                                             offsets_gpu(np.array([0, S * k], np.uint32)))
    token = np.empty(S * k, np.int64)
    token[ros] = np.arange(S * k) // k
    want = row_scales(x)
    assert np.array_equal(s.cpu().numpy(), want[token], equal_nan=True)
    check_codes(q.cpu().numpy(), quotients(x, np.repeat(want, B, 1)[:, :K])[token])


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("transposed", [False, True])
def test_weights(bad, transposed):
    N, K = 160, 256
    x = rows_with([], N, K, 2)
    for j, v in enumerate(BAD[bad]):
        x[100, 130 + j] = x[150, j] = v
    want = np.stack([[np.abs(x[n:n + B, b:b + B]).max() for b in range(0, K, B)] for n in range(0, N, B)]) / np.float32(448)
    quo = quotients(x, np.repeat(np.repeat(want, B, 0)[:N], B, 1))
    got = mxg.quantize_weights_block128(to_gpu(x[None]).to(torch.bfloat16), transposed)
    assert np.array_equal(got[1].cpu().numpy()[0], want, equal_nan=True)
    check_codes(got[0].cpu().numpy()[0], quo)
    if transposed:
        assert np.array_equal(got[3].cpu().numpy()[0], want.T, equal_nan=True)
        check_codes(got[2].cpu().numpy()[0], quo.T)


def gates(T, I, seed):
    """Gates and values of magnitudes from 1 to 2, so that no product below vanishes."""
    rng = np.random.default_rng(seed)
    h = rng.uniform(1, 2, (T, 2 * I)) * rng.choice([-1, 1], (T, 2 * I))
    return torch.from_numpy(h.astype(np.float32)).to(torch.bfloat16)


def check_overflowed(codes, scales, values):
    """values: fp64, of blocks that each overflow fp32 somewhere; the others keep the zero of their sign."""
    over = np.abs(values) > 3.5e38
    assert np.all(np.isinf(scales)) and over.any()
    assert np.all((codes[over] & 0x7F) == 0x7F)
    assert np.array_equal(codes[~over], np.where(values[~over] < 0, 0x80, 0).astype(np.uint8))


def test_silu_quantize():
    """A product of finite factors that overflows."""
    T, I = 3, 256
    h = gates(T, I, 3)
    h[:, [60, 300]], h[:, [61, 301]] = 1e38, -1e3
    q, s = mxg.silu_quantize_block128(h.cuda(), offsets_gpu(np.array([0, T], np.uint32)))
    g, u = h.double().numpy()[:, 0::2], h.double().numpy()[:, 1::2]
    check_overflowed(q.cpu().numpy(), s.cpu().numpy(), g / (1 + np.exp(-g)) * u)


@pytest.mark.parametrize("keep", [False, True])
def test_silu_backward(keep):
    T, I = 3, 128
    h = gates(T, I, 4)
    rng = np.random.default_rng(5)
    dy = torch.from_numpy(rng.uniform(1, 2, (T, I)).astype(np.float32)).to(torch.bfloat16)
    h[:, [40, 180]], h[:, [41, 181]], dy[:, [20, 90]] = 1e3, 1.0, 3e38  # there dg = dy u, du = dy g: past the range
    q = torch.empty((T, 2 * I), dtype=torch.uint8, device="cuda")
    s = torch.empty((T, 2), device="cuda")
    dh = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda") if keep else None
    mxg.mx_silu_backward_block128(h.cuda(), dy.cuda(), offsets_gpu(np.array([0, T], np.uint32)), dh=dh, dh_q=q,
                                  dh_scales=s)
    h64, d = h.double().numpy(), dy.double().numpy()
    g, u = h64[:, 0::2], h64[:, 1::2]
    sig = 1 / (1 + np.exp(-g))
    want = np.empty_like(h64)
    want[:, 0::2], want[:, 1::2] = d * u * sig * (1 + g * (1 - sig)), d * g * sig
    check_overflowed(q.cpu().numpy(), s.cpu().numpy(), want)
