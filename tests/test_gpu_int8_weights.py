"""Weights in 8-bit integers whose rows are not finite: zeros and a NaN scale,
as tokens have them, so that their channel of the product is NaN and no other."""
import numpy as np
import pytest
import torch

import bf16_gemm_vla_amd as vla
import oracle
import synthetic
from tests.eight_bit_ref import product, quantize_tokens
from tests.gpu_util import Guarded, bf16_f64, dev, zeros_ws

pytestmark = pytest.mark.gpu


def weights(N, K):
    W = (synthetic.rng(59000 + N + K).standard_normal((N, K)) * 0.02).astype(np.float32)
    W[1, K - 1] = np.nan
    W[2, 0] = np.inf
    W[N // 2, K // 2] = -np.inf
    W[N - 1, [3, K - 2]] = np.nan, np.inf
    W[0, 1] = np.float32(3.4e38)                  # finite: as large as fp32 goes
    W[5] = np.float32(1e-42)                      # subnormal
    W[6] = 0
    W[7] = -np.float32(np.nan)
    return W, [1, 2, 7, N // 2, N - 1]


@pytest.mark.parametrize("N,K", [(16, 32), (48, 96), (64, 1024), (32, 4128), (16, 131040)])
@pytest.mark.parametrize("layout", [vla.VLA_LAYOUT_ROWMAJOR, vla.VLA_LAYOUT_MFMA])
def test_rows_that_are_not_finite(N, K, layout):
    W, bad = weights(N, K)
    with np.errstate(invalid="ignore"):
        want, s = quantize_tokens(W)
    assert np.isnan(s[bad]).all() and np.isnan(s).sum() == len(bad)
    g, gs = Guarded(vla.vla_packed_bytes(N, K, vla.VLA_WFMT_INT8)), Guarded(N * 4)
    vla.vla_quantize_pack(dev(W), g.t, gs.t, N, K, vla.VLA_WFMT_INT8, layout)
    g.check()
    gs.check()
    expected = want.view(np.uint8) if layout == vla.VLA_LAYOUT_ROWMAJOR else oracle.pack(want.view(np.uint8), 8)
    assert np.array_equal(gs.numpy(np.float32), s, equal_nan=True)
    assert np.array_equal(g.numpy(np.uint8), expected.ravel())


@pytest.mark.parametrize("M", [1, 10, 50, 70, 200])
def test_their_channels_are_nan(M):
    N, K = 64, 96
    W, bad = weights(N, K)
    q, s = (torch.empty(n, dtype=t, device="cuda") for n, t in ((N * K, torch.int8), (N, torch.float32)))
    vla.vla_quantize_pack(dev(W), q, s, N, K, vla.VLA_WFMT_INT8, vla.VLA_LAYOUT_MFMA)
    r = synthetic.rng(59100 + M)
    a, s_a = r.integers(-127, 128, (M, K)).astype(np.int8), np.float32(r.uniform(0.01, 0.1, M))
    n = vla.vla_gemm_workspace_bytes(M, N, K, vla.VLA_WFMT_INT8)
    y, ws = Guarded(M * N * 2), zeros_ws(n)
    vla.vla_gemm_int8(dev(a), dev(s_a), q, s, None, None, y.t, ws, ws.numel(), M, N, K)
    y.check()
    got = bf16_f64(y.numpy(np.uint16).reshape(M, N))
    good = np.setdiff1d(np.arange(N), bad)
    assert np.isnan(got[:, bad]).all()
    codes, scales = quantize_tokens(W[good])
    want, _ = product(a, s_a, codes, scales)
    # the sum and the two scalings round by 2^-24 each, the output by 2^-8 (row 5: by half the smallest bf16 step); row 0's
    # largest results pass bf16's last value, 2^128 - 2^120, by more than half a step (2^119): those round to infinity
    past = np.abs(want) > 2.0 ** 128 - 2.0 ** 119
    assert past.any() == (M > 1) and np.array_equal(got[:, good][past], np.sign(want[past]) * np.inf)
    error = np.abs(got[:, good] - want)[~past]
    assert (error <= (2.0 ** -8 + 2.0 ** -21) * np.abs(want[~past]) + 2.0 ** -133).all()
