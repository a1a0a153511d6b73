"""Codes and scales of 8-bit integers against max |row| / 127 in 64 bits.

The scale is max |row| times fp32(1 / 127): two roundings of 2^-24 (half a
step) each, so it is within 2^-23 of the quotient, relatively.  A code is the
integer nearest to fp32(x / s): x / s is within |127 x / max| (2^-23 + 2^-24),
below 2^-15, of 127 x / max, and wherever that lies further than 2^-15 from
halfway between two integers the code is the integer nearest to it."""
import numpy as np
import pytest
import torch

import bf16_gemm_vla_amd as vla
import synthetic
from tests.gpu_util import Guarded, bf16_f64, dev

pytestmark = pytest.mark.gpu

MORE = 1 + 2.0 ** -20                              # products of the bounds above


def check(x, codes, scales):
    most = np.abs(x).max(1)
    ratio = scales.astype(np.float64) * 127.0 / most
    assert (np.abs(ratio - 1) <= 2.0 ** -23 * MORE).all()
    exact = 127.0 * x / most[:, None]
    clear = np.abs(np.abs(exact - np.floor(exact)) - 0.5) > 2.0 ** -15
    assert clear.mean() > 0.99
    assert np.array_equal(codes[clear], np.rint(exact[clear]).astype(np.int8))
    assert (np.abs(codes - exact) <= 0.5 + 2.0 ** -15).all()
    assert (np.abs(codes).max(1) == 127).all()


@pytest.mark.parametrize("M,K", [(1, 32), (50, 1024), (700, 96), (513, 2080), (9, 16384), (3, 20000), (2100, 4096)])
def test_tokens(M, K):
    r = synthetic.rng(69000 + M + K)
    x = synthetic.fp32_to_bf16_bits((r.standard_normal((M, K)) * np.exp(3 * r.standard_normal((M, 1)))).astype(np.float32))
    q, s = Guarded(M * K), Guarded(M * 4)
    vla.vla_quantize_tokens_int8(dev(x), q.t, s.t, M, K)
    q.check()
    s.check()
    check(bf16_f64(x), q.numpy(np.int8).reshape(M, K), s.numpy(np.float32))


@pytest.mark.parametrize("N,K", [(16, 32), (64, 1024), (4096, 1024), (48, 16384)])
def test_weights(N, K):
    r = synthetic.rng(69100 + N + K)
    W = (r.standard_normal((N, K)) * 0.02 * np.exp(r.standard_normal((N, 1)))).astype(np.float32)
    q, s = Guarded(N * K), Guarded(N * 4)
    vla.vla_quantize_pack(dev(W), q.t, s.t, N, K, vla.VLA_WFMT_INT8, vla.VLA_LAYOUT_ROWMAJOR)
    q.check()
    s.check()
    check(W.astype(np.float64), q.numpy(np.int8).reshape(N, K), s.numpy(np.float32))


def test_every_ratio_of_two_bf16_values():
    """x / max over every fraction of x and several of max: a row per maximum, its own values below it."""
    tops = [0x3F80 + f for f in range(0, 128, 3)] + [0x4300, 0x42FE, 0x3C24]
    rows = np.stack([np.arange(t + 1 - 15 * 128, t + 1, dtype=np.uint16) for t in tops])
    M, K = rows.shape
    rows[:, ::2] |= 0x8000
    q, s = torch.empty(M * K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    vla.vla_quantize_tokens_int8(dev(rows), q, s, M, K)
    x = bf16_f64(rows)
    exact = 127.0 * x / np.abs(x).max(1)[:, None]
    codes = q.cpu().numpy().reshape(M, K)
    clear = np.abs(np.abs(exact - np.floor(exact)) - 0.5) > 2.0 ** -15
    assert np.array_equal(codes[clear], np.rint(exact[clear]).astype(np.int8))
    assert (np.abs(codes - exact) <= 0.5 + 2.0 ** -15).all()
    assert (np.abs(s.cpu().numpy() * 127.0 / np.abs(x).max(1) - 1) <= 2.0 ** -23 * MORE).all()
