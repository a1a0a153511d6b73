"""GPU parity of the 8-bit integer operators against their 64-bit forms.

Codes and scales of tokens and weights are equal (one IEEE division each).
The product's sums are exact integers; they become fp32 (2^-24), are scaled
(two roundings of 2^-24), meet the bias (one) and are rounded to bf16 once:
|error| <= (2^-8 + 2^-22) |y| + 2^-22 |sum s_a s_w|, and one step of the
smallest bf16.  With a residual the result is the nearest bf16 of
residual + that bf16."""
import numpy as np
import pytest
import torch

import bf16_gemm_vla_amd as vla
import oracle
import synthetic
from tests.eight_bit_ref import product, quantize_tokens
from tests.gpu_util import Guarded, bf16_f64, dev, host, zeros_ws

pytestmark = pytest.mark.gpu


def rng(seed):
    return synthetic.rng(29000 + seed)


def bits(x):
    return synthetic.fp32_to_bf16_bits(np.asarray(x, np.float32))


# ---------------------------------------------------------------- tokens

def run_tokens(a_bits):
    M, K = a_bits.shape
    q, s = Guarded(M * K, fill=0x55), Guarded(M * 4, fill=0x55)
    vla.vla_quantize_tokens_int8(dev(a_bits), q.t, s.t, M, K)
    q.check()
    s.check()
    got_q, got_s = q.numpy(np.int8).reshape(M, K), s.numpy(np.float32)
    with np.errstate(invalid="ignore"):
        want_q, want_s = quantize_tokens(bf16_f64(a_bits))
    assert np.array_equal(got_q, want_q), np.argwhere(got_q != want_q)[:3]
    assert np.array_equal(got_s, want_s, equal_nan=True)
    return got_q, got_s


@pytest.mark.parametrize("M,K", [(1, 32), (50, 1024), (3, 64), (5, 544), (7, 512), (2, 2048), (9, 2080), (129, 4096), (4, 4128),
                                 (3, 8192), (2, 16384), (2, 16416), (1, 131040), (3, 65536), (1000, 96)])
def test_tokens_equal_the_division(M, K):
    r = rng(M + K)
    run_tokens(bits(r.standard_normal((M, K)) * np.exp(2 * r.standard_normal((M, 1)))))


@pytest.mark.parametrize("M,K", [(513, 2080), (512, 2080), (515, 4096), (520, 4128), (513, 8224), (513, 16384), (512, 16384), (2049, 544),
                                 (2050, 1024), (2048, 1024), (4097, 2048), (9001, 32)])
def test_tokens_many_rows(M, K):
    """On either side of the numbers of rows from which fewer waves take a row; rows of zeros and with NaN among them."""
    x = bits(rng(M + K).standard_normal((M, K)).astype(np.float32))
    x[M // 2] = 0
    x[M - 1, K - 1], x[3, 0] = 0x7FC0, 0xFF80
    run_tokens(x)


def test_tokens_ties_extremes_and_rows_that_are_not_finite():
    K = 96
    r = rng(1)
    a = r.standard_normal((14, K)).astype(np.float32)
    a[0] = 0
    a[1] = np.float32(1e-40)                     # subnormal rows: their scale is, too
    a[2, :] = np.linspace(-3e38, 3e38, K)
    a[3] = np.arange(K) - 40                     # scale 55 / 127
    a[4] = (np.arange(K) % 64) * 2 + 1           # halves of the step where the maximum is 254
    a[4, 5] = 254
    a[5] = -(np.arange(K) % 64) - 0.5
    a[5, 9] = 127
    a[6, 3] = np.inf
    a[7, 4] = np.nan
    a[8, 5] = -np.inf
    a[8, 6] = np.nan
    a[9] = 2.0 ** -126
    a[10, 0] = 9.2e-41
    a[10, 1:] = 0
    q, s = run_tokens(bits(a))
    assert (q[6:9] == 0).all() and np.isnan(s[6:9]).all() and np.isfinite(np.delete(s, [6, 7, 8])).all()
    assert s[0] == 1 and (q[0] == 0).all()
    big = bits(r.standard_normal((4, 20000 // 32 * 32)))          # the long form
    big[1, 777] = 0x7F80
    big[2] = 0
    q, s = run_tokens(big)
    assert np.isnan(s[1]) and s[2] == 1


def test_tokens_every_bf16_value():
    """Every finite magnitude under several maxima, each row with its own."""
    every = np.arange(0x7F80, dtype=np.uint16)
    for top in (0x7F7F, 0x4300, 0x3F80, 0x0100, 0x007F, 0x42FE):
        row = every[every <= top][-4064 + 32:]
        row = np.concatenate([row, row[:1] * 0 + np.uint16(top)])
        row = row[len(row) % 32:]
        run_tokens(np.stack([row, row | 0x8000]))


# --------------------------------------------------------------- weights

@pytest.mark.parametrize("N,K", [(16, 32), (48, 96), (64, 1024), (32, 4128)])
def test_weights_pack_both_layouts(N, K):
    W = (rng(N + K).standard_normal((N, K)) * 0.02).astype(np.float32)
    W[3] = 0
    W[5, 7] = 1e30
    want, s = quantize_tokens(W)
    for layout in (vla.VLA_LAYOUT_ROWMAJOR, vla.VLA_LAYOUT_MFMA):
        g, gs = Guarded(vla.vla_packed_bytes(N, K, vla.VLA_WFMT_INT8)), Guarded(N * 4)
        vla.vla_quantize_pack(dev(W), g.t, gs.t, N, K, vla.VLA_WFMT_INT8, layout)
        g.check()
        gs.check()
        expected = want.view(np.uint8) if layout == vla.VLA_LAYOUT_ROWMAJOR else oracle.pack(want.view(np.uint8), 8)
        assert np.array_equal(g.numpy(np.uint8), expected.ravel())
        assert np.array_equal(gs.numpy(np.float32), s)


# --------------------------------------------------------------- product

def pack(w):
    d = dev(w.view(np.uint8))
    p = torch.empty(w.size, dtype=torch.uint8, device="cuda")
    vla.vla_pack_fp8(d, p, *w.shape)
    return p


def run_product(a, s_a, w, s_w, bias=None, resid=None, in_place=False, packed=None, ws=None, stream=None, check=True):
    (M, K), N = a.shape, w.shape[0]
    n = vla.vla_gemm_workspace_bytes(M, N, K, vla.VLA_WFMT_INT8)
    ws = zeros_ws(n) if ws is None else ws
    y = Guarded(M * N * 2, fill=0x3A)
    r = None if resid is None else dev(resid)
    if in_place:
        y.t.copy_(r.flatten().view(torch.uint8))
        r = y.t
    vla.vla_gemm_int8(dev(a), dev(s_a), pack(w) if packed is None else packed, dev(s_w), None if bias is None else dev(bias), r, y.t,
                      ws, ws.numel(), M, N, K, stream=stream)
    y.check()
    vla.vla_workspace_status(ws)
    assert not ws[:61440].any()                                   # counters as they were
    got = y.numpy(np.uint16).reshape(M, N)
    if check:
        check_product(got, a, s_a, w, s_w, bias, resid)
    return got


def check_product(got, a, s_a, w, s_w, bias=None, resid=None):
    with np.errstate(over="ignore"):
        ref, sums = product(a, s_a, w, s_w, None if bias is None else bf16_f64(bias))
    scaled = np.abs(sums) * s_a.astype(np.float64)[:, None] * s_w.astype(np.float64)
    tol = (2.0 ** -8 + 2.0 ** -22) * np.abs(ref) + 2.0 ** -22 * scaled + 2.0 ** -133
    y = bf16_f64(got)
    if resid is not None:
        # the nearest bf16 of residual + y for some bf16 y within its tolerance
        r = bf16_f64(resid)
        tol = tol + 2.0 ** -8 * (np.abs(r + ref) + tol)
        ref = r + ref
    # past half a step over bf16's largest value, (2 - 2^-8) 2^127, the nearest bf16 is an infinity
    past = np.abs(ref) > (2 - 2.0 ** -8) * 2.0 ** 127 * (1 + 2.0 ** -22)
    assert np.array_equal(y[past], np.sign(ref[past]) * np.inf)
    y, ref, tol = y[~past], ref[~past], tol[~past]
    bad = ~(np.abs(y - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[0]}: {y[bad][0]} for {ref[bad][0]}"


def draw(M, N, K, seed):
    r = rng(seed)
    a, w = r.integers(-127, 128, (M, K)).astype(np.int8), r.integers(-127, 128, (N, K)).astype(np.int8)
    s_a = np.exp(r.standard_normal(M)).astype(np.float32) * 0.01
    s_w = np.exp(r.standard_normal(N)).astype(np.float32) * 0.01
    return a, s_a, w, s_w


@pytest.mark.parametrize("M,N,K", [
    (1, 16, 32), (4, 64, 128), (10, 1024, 4096), (16, 48, 96), (17, 4096, 1024), (33, 1040, 544), (50, 4096, 1024), (50, 1024, 4096),
    (64, 16, 8192), (64, 2048, 64), (7, 16384, 2048), (65, 16, 32), (65, 128, 4096), (191, 272, 160), (192, 256, 64), (193, 4096, 1056),
    (571, 2048, 16384), (768, 2048, 2048), (300, 16384, 96), (1000, 8208, 512), (50, 16, 131040), (70, 32, 131040)])
def test_product_matches_the_exact_sums(M, N, K):
    print(M, N, K, vla.vla_gemm_plan(M, N, K, vla.VLA_WFMT_INT8), flush=True)
    run_product(*draw(M, N, K, M + N + K))


@pytest.mark.parametrize("M,N,K", [
    (10, 8208, 2080), (16, 16384, 2048), (1, 8192, 1056), (10, 8192, 4096), (9, 4112, 8192), (3, 1024, 16384), (16, 48, 8224),
    (16, 4096, 4096), (17, 4112, 4096), (32, 8208, 1056), (30, 4096, 1024), (33, 2064, 16416), (64, 16384, 2048), (40, 32768, 1024),
    (20, 8192, 16384), (17, 131072, 1024), (50, 1048576, 32),
    (50, 2048, 4096), (33, 2064, 2080), (30, 4112, 2048), (17, 4096, 4096), (64, 8208, 1056), (30, 2048, 4096), (24, 4096, 8192)])
def test_few_rows_of_every_tiling(M, N, K):
    """Tilings of few rows by rows, columns and K, partial column groups, and those that the wide kernel takes."""
    print(M, N, K, vla.vla_gemm_plan(M, N, K, vla.VLA_WFMT_INT8), flush=True)
    run_product(*draw(M, N, K, M + N + K))


@pytest.mark.parametrize("M,N,K", [(50, 1024, 4096), (33, 96, 640), (768, 2048, 4096), (100, 144, 96), (700, 4096, 1024)])
def test_product_bias_and_residual(M, N, K):
    a, s_a, w, s_w = draw(M, N, K, M + K)
    r = rng(M)
    bias, resid = bits(r.standard_normal(N) * 20), bits(r.standard_normal((M, N)) * 50)
    plain = run_product(a, s_a, w, s_w, bias)
    want = oracle.bf16_round(bf16_f64(resid) + bf16_f64(plain))
    got = run_product(a, s_a, w, s_w, bias, resid)
    assert np.array_equal(got, want.reshape(M, N))
    assert np.array_equal(run_product(a, s_a, w, s_w, bias, resid, in_place=True), got)


@pytest.mark.parametrize("M", [3, 50, 200])
def test_product_of_the_extreme_codes(M):
    """-128 times -128 over the longest K stays inside 32 bits, exactly."""
    N, K = 32, 131040
    a, w = np.full((M, K), -128, np.int8), np.full((N, K), -128, np.int8)
    w[1] = 127
    one = np.ones(M, np.float32), np.ones(N, np.float32)
    got = bf16_f64(run_product(a, one[0], w, one[1]))
    assert (got[:, 0] == 2.0 ** 31).all() and (got[:, 1] < -2.0 ** 30).all()       # 2146959360 rounds to 2^31


@pytest.mark.parametrize("M", [20, 130])
def test_product_scales_beyond_fp32(M):
    """Scales whose product leaves fp32's normal range, while sum times both does not; zero, infinite and NaN ones."""
    N, K = 64, 256
    a, _, w, _ = draw(M, N, K, 5)
    s_a = np.full(M, 1.0, np.float32)
    s_w = np.full(N, 1.0, np.float32)
    s_a[0], s_w[0] = 1e-20, 1e-21
    s_a[1], s_w[1] = 1e30, 1e-38
    s_a[2], s_w[2] = 1e-42, 1e38
    s_a[3], s_w[3] = 0.0, 3.0
    before = run_product(a, s_a, w, s_w)
    s_a[5] = np.nan
    s_w[7] = np.nan
    s_a[6] = np.inf
    after = run_product(a, s_a, w, s_w, check=False)
    got = bf16_f64(after)
    assert np.isnan(got[5]).all() and np.isnan(got[:, 7]).all()
    others = [np.delete(np.delete(x, [5, 6], 0), 7, 1) for x in (before, after)]
    assert np.array_equal(*others)                                # the other rows and columns as they were


def test_product_places_every_channel_and_k():
    """One-hot rows: every code of the weights comes out at its place."""
    for M, N, K in ((64, 48, 64), (256, 272, 256)):
        w = rng(9).integers(-128, 128, (N, K)).astype(np.int8)
        a = np.zeros((M, K), np.int8)
        a[np.arange(M), np.arange(M) % K] = 1
        got = run_product(a, np.ones(M, np.float32), w, np.ones(N, np.float32))
        assert np.array_equal(bf16_f64(got), w.T[np.arange(M) % K].astype(np.float64))


def test_product_rows_do_not_depend_on_their_neighbours():
    a, s_a, w, s_w = draw(300, 1024, 2048, 21)
    whole = run_product(a, s_a, w, s_w)
    for rows in (slice(0, 1), slice(3, 40), slice(100, 220)):
        assert np.array_equal(run_product(a[rows], s_a[rows], w, s_w, check=False), whole[rows])


def test_product_captured_shared_workspace_and_streams():
    shapes = [(50, 1024, 4096), (768, 2048, 4096)]
    ws = zeros_ws(max(vla.vla_gemm_workspace_bytes(*s, vla.VLA_WFMT_INT8) for s in shapes))
    calls = []
    for M, N, K in shapes:
        a, s_a, w, s_w = draw(M, N, K, M)
        calls.append((dev(a), dev(s_a), pack(w), dev(s_w), torch.empty(M * N, dtype=torch.int16, device="cuda"), M, N, K,
                      run_product(a, s_a, w, s_w, ws=ws)))
    torch.cuda.synchronize()
    def go():
        for a, s_a, w, s_w, y, M, N, K, _ in calls:
            vla.vla_gemm_int8(a, s_a, w, s_w, None, None, y, ws, ws.numel(), M, N, K)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        for c in calls:
            c[4].zero_()
        graph.replay()
        go()                                                      # eager work between the replays
        torch.cuda.synchronize()
        for c in calls:
            c[4].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for c in calls:
            assert np.array_equal(host(c[4], np.uint16).reshape(c[5], c[6]), c[8])
    vla.vla_workspace_status(ws)


def test_product_wait_that_gives_up_leaves_nan():
    """The K split's bounded wait, forced from the host: owner slices NaN, cause in the status word."""
    M, N, K = 768, 2048, 16384
    rc, info = vla.vla_gemm_plan(M, N, K, vla.VLA_WFMT_INT8)
    assert rc == 0 and info[5] > 1
    a, s_a, w, s_w = draw(M, N, K, 31)
    ws = zeros_ws(vla.vla_gemm_workspace_bytes(M, N, K, vla.VLA_WFMT_INT8))
    p = pack(w)
    y = torch.zeros(M * N, dtype=torch.int16, device="cuda")
    d = dev(a), dev(s_a), dev(s_w)
    gave_up = False
    try:
        vla.vla_set_wait_limit(1)
        for _ in range(20):
            vla.vla_gemm_int8(d[0], d[1], p, d[2], None, None, y, ws, ws.numel(), M, N, K)
            torch.cuda.synchronize()
            try:
                vla.vla_workspace_status(ws)
            except RuntimeError as e:
                assert "split-K" in str(e)
                gave_up = True
                break
    finally:
        vla.vla_set_wait_limit(0)
    got = bf16_f64(host(y, np.uint16).reshape(M, N))
    assert gave_up and np.isnan(got).any()
    assert not ws[:61440].any()
    vla.vla_gemm_int8(d[0], d[1], p, d[2], None, None, y, ws, ws.numel(), M, N, K)
    check_product(host(y, np.uint16).reshape(M, N), a, s_a, w, s_w)


def test_tokens_then_product():
    """Quantized tokens times quantized weights against the fp64 product of what both stand for, and near the unquantized one."""
    M, N, K = 50, 4096, 1024
    x = bits(rng(41).standard_normal((M, K)))
    W = (rng(42).standard_normal((N, K)) * 0.02).astype(np.float32)
    x[7, 5] = 0x7FC0
    q, s = torch.empty(M * K, dtype=torch.int8, device="cuda"), torch.empty(M, dtype=torch.float32, device="cuda")
    p, sw = torch.empty(N * K, dtype=torch.int8, device="cuda"), torch.empty(N, dtype=torch.float32, device="cuda")
    vla.vla_quantize_tokens_int8(dev(x), q, s, M, K)
    vla.vla_quantize_pack(dev(W), p, sw, N, K, vla.VLA_WFMT_INT8, vla.VLA_LAYOUT_MFMA)
    ws = zeros_ws(vla.vla_gemm_workspace_bytes(M, N, K, vla.VLA_WFMT_INT8))
    y = torch.empty(M * N, dtype=torch.int16, device="cuda")
    vla.vla_gemm_int8(q, s, p, sw, None, None, y, ws, ws.numel(), M, N, K)
    got = bf16_f64(host(y, np.uint16).reshape(M, N))
    assert np.isnan(got[7]).all()
    keep = np.arange(M) != 7
    wq, ws_ = quantize_tokens(W)
    check_product(host(y, np.uint16).reshape(M, N)[keep], host(q).reshape(M, K)[keep], host(s)[keep], wq, ws_)
    # half a step per value on either side: K (|a| s_w + |w| s_a) / 2 at most
    exact = bf16_f64(x[keep]) @ W.astype(np.float64).T
    bound = 0.5 * (np.abs(bf16_f64(x[keep])).sum(1)[:, None] * ws_ + host(s)[keep][:, None] * (np.abs(W).sum(1) + 0.5 * K * ws_))
    assert (np.abs(got[keep] - exact) <= bound + 2.0 ** -7 * np.abs(exact)).all()


def test_tokens_past_one_launch():
    """More rows than a launch takes, the first, the last and those on either side of the seam."""
    M, K = (1 << 20) + 3, 32
    x = bits(rng(77).standard_normal((64, K)))
    rows = dev(x).repeat(M // 64 + 1, 1)[:M].contiguous()
    q, s = torch.zeros(M, K, dtype=torch.int8, device="cuda"), torch.zeros(M, device="cuda")
    vla.vla_quantize_tokens_int8(rows, q, s, M, K)
    want_q, want_s = quantize_tokens(bf16_f64(x))
    want_q, want_s = torch.from_numpy(want_q).cuda(), torch.from_numpy(want_s).cuda()
    at = torch.arange(M, device="cuda") % 64
    assert torch.equal(q, want_q[at]) and torch.equal(s, want_s[at])


@pytest.mark.parametrize("M,K", [(50, 1024), (700, 4096), (2100, 544)])
def test_tokens_equal_an_array_programs(M, K):
    """The codes and scales of the definition in array operations, bit for bit."""
    x = torch.randn(M, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(M)).bfloat16()
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    vla.vla_quantize_tokens_int8(x, q, s, M, K)
    scale = x.float().abs().amax(1) / 127.0
    assert torch.equal(s, scale)
    assert torch.equal(q, torch.round(x.float() / scale[:, None]).to(torch.int8))
