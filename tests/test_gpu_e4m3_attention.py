"""GPU parity of attention over an E4M3 cache against the fp64 oracle.

A cached value is its code's value times a power of two, a bf16 number, and
enters the products exactly; tolerances are those of attention over a bf16
cache (tests/test_gpu_attention.py), on the values that the codes stand for."""
import math

import numpy as np
import pytest
import torch

import bf16_gemm_vla_amd as vla
import synthetic
from tests.eight_bit_ref import E4M3, e4m3_code, e8m0_value, scale_byte
from tests.gpu_util import Guarded, bf16_f64, dev, host, zeros_ws
from tests.test_gpu_attention import HEADS, assert_attention, attention_bound, rand

pytestmark = pytest.mark.gpu


class Cache:
    """Pages of codes in shuffled order; every sequence's keys are the prefix's slots, then its own."""

    def __init__(self, B, hkv, D, page, block, prefix, lens, seed, n_prefix_pages=None, pages_per_seq=None):
        r = synthetic.rng(49000 + seed)
        self.npp = -(-prefix // page) if n_prefix_pages is None else n_prefix_pages
        self.pps = -(-max(lens, default=0) // page) if pages_per_seq is None else pages_per_seq
        self.page, self.block, self.hkv, self.D = page, block, hkv, D
        self.pages = self.npp + B * self.pps + max(2, -(-block // page))
        order = r.permutation(self.pages).astype(np.int32)
        self.prefix_pages, self.table = order[:self.npp].copy(), order[self.npp:self.npp + B * self.pps].reshape(B, self.pps).copy()
        rows = self.pages * page
        self.codes, self.bytes = [], []
        for _ in range(2):
            x = r.standard_normal((rows // block, block, hkv, D)) * np.exp(r.standard_normal((rows // block, 1, hkv, 1)))
            byte = scale_byte(np.abs(x).max((1, 3)))
            self.bytes.append(byte)
            self.codes.append(e4m3_code(x * np.exp2(127.0 - byte)[:, None, :, None]).reshape(rows, hkv, D))
        self.keys = []
        for b in range(B):
            pre, own = np.arange(prefix), np.arange(lens[b])
            self.keys.append(np.concatenate([self.prefix_pages[pre // page].astype(np.int64) * page + pre % page if prefix else pre,
                                             self.table[b][own // page].astype(np.int64) * page + own % page if lens[b] else own]))

    def values(self, i, slots):
        """bf16 bits of the cached rows: what codes and scales stand for."""
        v = E4M3[self.codes[i][slots]] * e8m0_value(self.bytes[i][slots // self.block])[..., None]
        with np.errstate(over="ignore"):
            return synthetic.fp32_to_bf16_bits(v.astype(np.float32))

    def call(self, q, prefix, lens, L, hq, causal, scale, ws=None, stream=None, check=True):
        B = len(lens)
        n = vla.vla_attn_shared_prefix_e4m3_workspace_bytes(B, L, hq, self.hkv, self.D, self.npp * self.page, self.pps * self.page)
        o = Guarded(B * L * hq * self.D * 2, fill=0x5A)
        w = Guarded(n, fill=0xFF) if ws is None else ws
        vla.vla_attn_shared_prefix_e4m3(
            dev(q), dev(self.codes[0]), dev(self.codes[1]), dev(self.bytes[0]), dev(self.bytes[1]),
            dev(self.prefix_pages) if self.npp else None, dev(np.array([prefix], np.int32)) if self.npp else None,
            dev(self.table) if self.pps else None, dev(np.array(lens, np.int32)) if self.pps else None, o.t, w.t, n, B, L, hq,
            self.hkv, self.D, self.pages, self.page, self.block, self.npp, self.pps, hq * self.D, hq * self.D, causal, scale,
            stream=stream)
        o.check()
        if ws is None:
            w.check()
        return o.numpy(np.uint16).reshape(B, L, hq, self.D)


def limits(L, prefix, n, causal):
    if not causal:
        return np.full(L, prefix + n, np.int64)
    return prefix + np.clip(np.arange(L) + 1 + n - L, 0, n)


def run(B, L, hq, hkv, D, page, block, prefix, lens, causal, scale=None, seed=0, lens_given=None, change=None, check=True, **sizes):
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    c = Cache(B, hkv, D, page, block, prefix, lens, seed, **sizes)
    q = rand(20000 + seed, B * L, hq, D, scale=2.0)
    if change:
        change(c)
    got = c.call(q, prefix, lens if lens_given is None else lens_given, L, hq, causal, scale)
    if check:
        for b in range(B):
            at = c.keys[b]
            assert_attention(got[b], q.reshape(B, L, hq, D)[b], c.values(0, at), c.values(1, at), limits(L, prefix, lens[b], causal),
                             float(np.float32(scale)), f"sequence {b}")
    return got, c, q


@pytest.mark.parametrize("hq,hkv,D", HEADS)
@pytest.mark.parametrize("B,L,page,block,prefix,lens,causal", [
    (1, 1, 16, 16, 0, [1], True), (1, 1, 8, 2, 0, [777], True), (1, 10, 16, 16, 768, [10], False), (2, 1, 1, 1, 5, [3, 0], True),
    (3, 7, 32, 8, 0, [7, 200, 64], True), (5, 1, 64, 64, 1000, [1, 65, 128, 0, 300], False), (2, 3, 128, 128, 131, [3, 129], True)])
def test_matches_oracle(hq, hkv, D, B, L, page, block, prefix, lens, causal):
    run(B, L, hq, hkv, D, page, block, prefix, lens, causal, seed=D + L + page)


@pytest.mark.parametrize("hq,hkv,D", [(8, 1, 256), (8, 2, 128), (6, 1, 64), (12, 2, 72)])
def test_many_rows(hq, hkv, D):
    """128-row tiles for the prefix, for the suffix, and for both."""
    run(20, 1, hq, hkv, D, 16, 16, 333, [1 + 13 * b for b in range(20)], True, seed=500 + D)
    run(3, 50, hq, hkv, D, 16, 4, 200, [50, 170, 64], True, seed=520 + D)
    run(1, 50, hq, hkv, D, 16, 16, 100, [90], False, seed=540 + D)
    run(2, 3, hq, hkv, D, 32, 32, 70, [3, 9], True, seed=560 + D)


@pytest.mark.parametrize("hq,hkv,D,B,L", [(8, 1, 256, 20, 64), (8, 1, 256, 40, 64), (16, 4, 128, 20, 64), (32, 8, 128, 20, 64),
                                         (16, 4, 64, 20, 65), (32, 8, 72, 20, 65)])
def test_tall_suffix_tiles(hq, hkv, D, B, L):
    run(B, L, hq, hkv, D, 16, 8, 70, [(L + 3 * b) if b else 0 for b in range(B)], True, seed=700 + D + B)


@pytest.mark.parametrize("hq,hkv,D", [(8, 1, 256), (8, 1, 64), (16, 2, 128), (24, 3, 72)])
def test_tall_prefix_tiles(hq, hkv, D):
    run(41, 1, hq, hkv, D, 16, 16, 333, [1 + 3 * b for b in range(41)], True, seed=580 + D)
    run(41, 1, hq, hkv, D, 16, 16, 50, [0] * 41, False, pages_per_seq=0, seed=590 + D)


@pytest.mark.parametrize("hq,hkv,D,B", [(64, 8, 128, 300), (8, 1, 256, 1100)])
def test_many_single_tokens(hq, hkv, D, B):
    run(B, 1, hq, hkv, D, 16, 16, 75, [b % 4 for b in range(B)], True, seed=720 + D)


@pytest.mark.parametrize("hq,hkv,D", [(8, 8, 64), (4, 1, 128), (8, 1, 256), (5, 5, 72)])
def test_long_split_keys(hq, hkv, D):
    run(1, 1, hq, hkv, D, 64, 32, 0, [9001], True, seed=800 + D)
    run(3, 2, hq, hkv, D, 16, 16, 1111, [2000, 0, 31], True, seed=810 + D)


def test_edges():
    got, _, _ = run(2, 2, 4, 2, 64, 16, 16, 0, [0, 40], True, pages_per_seq=3, seed=601)
    assert not got[0].any()
    got, _, _ = run(2, 5, 4, 2, 64, 16, 16, 0, [3, 5], True, seed=602)
    assert not got[0, :2].any() and got[0, 2:].any()
    run(3, 1, 4, 2, 64, 16, 16, 100, [2, 9, 1], True, pages_per_seq=40, n_prefix_pages=300, seed=603)
    run(2, 1, 4, 2, 64, 16, 16, 48, [32, 32], False, lens_given=[1 << 30, 33], seed=604)
    run(3, 1, 4, 2, 64, 16, 16, 320, [0, 0, 0], False, pages_per_seq=0, seed=605)
    run(2, 1, 4, 2, 64, 16, 16, 0, [5, 6], False, n_prefix_pages=4, seed=607)
    got, _, _ = run(2, 1, 4, 2, 64, 16, 16, 0, [5, 6], False, lens_given=[-3, 6], check=False, seed=609)
    assert not got[0].any() and got[1].any()


def test_missing_pages_hold_no_keys():
    for b0, prefix, lens in ((2, 100, [50, 90]), (1, 100, [50])):
        c = Cache(b0, 2, 64, 16, 16, prefix, lens, seed=620)
        q = rand(621, b0 * 3, 4, 64)
        keys = [c.keys[b].copy() for b in range(b0)]
        c.prefix_pages[3], c.prefix_pages[6] = -1, c.pages
        c.table[0, 2] = 1 << 30
        got = c.call(q, prefix, lens, 3, 4, False, 0.125)
        for b in range(b0):
            j, i = np.arange(prefix), np.arange(lens[b])
            keep = np.concatenate([(j // 16 != 3) & (j // 16 != 6), (i // 16 != 2) if b == 0 else i >= 0])
            at = keys[b][keep]
            assert_attention(got[b], q.reshape(b0, 3, 4, 64)[b], c.values(0, at), c.values(1, at), np.full(3, len(at)), 0.125)


@pytest.mark.parametrize("hq,hkv,D,B,L,prefix", [(4, 2, 128, 2, 4, 0), (4, 2, 128, 2, 4, 40), (8, 1, 256, 20, 64, 70), (8, 1, 256, 40, 64, 0),
                                                (32, 8, 128, 20, 64, 70), (16, 4, 64, 20, 64, 33), (64, 1, 64, 2, 1, 9)])
def test_unseen_values_have_no_part(hq, hkv, D, B, L, prefix):
    """NaN codes in the last key and value of every sequence, and NaN scales and codes behind them, stay out of the other rows."""
    lens = [L + 5 * b for b in range(B)]
    c = Cache(B, hkv, D, 16, 1, prefix, lens, seed=650 + D + B, pages_per_seq=-(-max(lens) // 16) + 1)
    q = rand(651, B * L, hq, D)
    for b in range(B):
        at = c.keys[b][-1]
        for i in range(2):
            c.codes[i][at] = 0x7F if b % 2 else 0xFF
            n = lens[b]
            behind = c.table[b][n // 16].astype(np.int64) * 16 + n % 16
            c.codes[i][behind] = 0x7F
            c.bytes[i][behind] = 255
    got = c.call(q, prefix, lens, L, hq, True, 0.1)
    for b in range(B):
        s, total = c.keys[b], len(c.keys[b])
        lim = np.arange(L - 1) + 1 + total - L
        if L > 1:
            assert_attention(got[b, :L - 1], q.reshape(B, L, hq, D)[b, :L - 1], c.values(0, s[:-1]), c.values(1, s[:-1]), lim, float(np.float32(0.1)))
        assert np.isnan(bf16_f64(got[b, L - 1])).all()


def test_visible_nan_reaches_its_rows_and_channel_alone():
    def change(c):
        c.codes[1][c.keys[0][70], 0, 5] = 0x7F
    got, c, q = run(1, 30, 2, 1, 64, 16, 16, 60, [40], True, seed=660, change=change, check=False)
    g, lim = bf16_f64(got[0]), limits(30, 60, 40, True)
    sees = lim > 70
    assert np.isnan(g[sees][:, :, 5]).all() and np.isfinite(g[~sees]).all() and np.isfinite(np.delete(g, 5, 2)).all()
    c.codes[1][c.keys[0][70], 0, 5] = 0
    keep = np.arange(64) != 5
    ref, tol = attention_bound(q.reshape(30, 2, 64), c.values(0, c.keys[0]), c.values(1, c.keys[0]), lim, float(np.float32(0.125)))
    assert (np.abs(g - ref)[..., keep] <= tol[..., keep]).all()


@pytest.mark.parametrize("L", [1, 40])
def test_scales_of_the_whole_range(L):
    """The smallest and the largest scales, keys and values; a scale byte of 255 is NaN to the rows that see it."""
    for i, byte in ((1, 0), (1, 1), (1, 9), (1, 200), (0, 0), (0, 100)):
        def change(c, i=i, byte=byte):
            c.bytes[i][:] = byte
        got, _, _ = run(1, L, 4, 2, 64, 16, 16, 40, [100], True, seed=670, change=change)
        assert got.any() or byte == 0
    for i in range(2):
        def change(c, i=i):
            c.bytes[i][c.keys[0][139] // 16] = 255
        got, _, _ = run(1, L, 4, 2, 64, 16, 16, 40, [100], True, seed=671, change=change, check=False)
        assert np.isnan(bf16_f64(got[0, -1])).all()


@pytest.mark.parametrize("hq,hkv,D", [(4, 2, 128), (8, 1, 256), (2, 2, 64)])
@pytest.mark.parametrize("rows", [1, 300])
def test_cache_past_4_gib(hq, hkv, D, rows):
    """A prefix and suffixes spread over codes of 5 GiB, for few rows and for tall tiles."""
    page, block, L = 16, 8, rows
    pages = (5 << 30) // (hkv * D) // page
    small = Cache(2, hkv, D, page, block, 60, [33, 48], seed=680 + D)
    spread = np.sort(synthetic.rng(681).choice(pages, small.pages, replace=False))
    spread[-1] = pages - 1
    codes = [torch.zeros(pages * page, hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(pages * page // block, hkv, dtype=torch.uint8, device="cuda") for _ in range(2)]
    rows_at = torch.from_numpy((spread[:, None] * page + np.arange(page)).ravel()).cuda()
    blocks_at = torch.from_numpy((spread[:, None] * (page // block) + np.arange(page // block)).ravel()).cuda()
    for i in range(2):
        codes[i][rows_at] = dev(small.codes[i])
        scales[i][blocks_at] = dev(small.bytes[i])
    pre, table = (dev(spread[x].astype(np.int32)) for x in (small.prefix_pages, small.table))
    q = rand(682, 2 * L, hq, D, scale=2.0)
    n = vla.vla_attn_shared_prefix_e4m3_workspace_bytes(2, L, hq, hkv, D, small.npp * page, small.pps * page)
    o, w = Guarded(2 * L * hq * D * 2), zeros_ws(n)
    vla.vla_attn_shared_prefix_e4m3(dev(q), *codes, *scales, pre, dev(np.array([60], np.int32)), table,
                                    dev(np.array([33, 48], np.int32)), o.t, w, n, 2, L, hq, hkv, D, pages, page, block, small.npp,
                                    small.pps, hq * D, hq * D, False, 0.1)
    o.check()
    got = o.numpy(np.uint16).reshape(2, L, hq, D)
    for b in range(2):
        at = small.keys[b]
        assert_attention(got[b], q.reshape(2, L, hq, D)[b], small.values(0, at), small.values(1, at), np.full(L, len(at)), float(np.float32(0.1)))
    # appended at the far end through the cache's own writer
    x = rand(683, 1, hkv, D)
    vla.vla_kv_append_e4m3(dev(x), dev(x), None, dev(np.array([[pages - 1]], np.int32)), dev(np.array([16], np.int32)), *codes, *scales,
                           1, 1, 1, hkv, D, pages, page, block, 1, hkv * D, hkv * D)
    last = host(codes[0][-1]).reshape(hkv, D)
    s = e8m0_value(host(scales[0][-1]))[:, None]
    assert (np.abs(E4M3[last] * s - bf16_f64(x[0])) <= np.maximum(2.0 ** -4 * np.abs(bf16_f64(x[0])), 2.0 ** -10 * s)).all()


def test_workspace_needs_no_clearing_and_results_repeat():
    c = Cache(3, 2, 128, 16, 16, 300, [0, 600, 3], seed=690, pages_per_seq=38)
    q = rand(691, 3 * 2, 8, 128)
    n = vla.vla_attn_shared_prefix_e4m3_workspace_bytes(3, 2, 8, 2, 128, c.npp * 16, c.pps * 16)
    got = [c.call(q, 300, [0, 600, 3], 2, 8, True, 0.1, ws=Guarded(n, fill=f)) for f in (0, 0xFF, 0x7F)]
    assert np.array_equal(got[0], got[1]) and np.array_equal(got[0], got[2])


def test_captured_calls_follow_device_lengths_and_streams():
    """Append and attention in one graph, replayed while lengths grow, against the same calls run at once; two graphs share a
    workspace one after the other; the same on another stream."""
    hq, hkv, D, page, block, B, pps = 8, 2, 64, 16, 16, 3, 6
    pages = B * pps + 4
    kc, vc = (torch.zeros(pages * page, hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages * page // block, hkv, dtype=torch.uint8, device="cuda") for _ in range(2))
    pp, table = dev(np.arange(4, dtype=np.int32)), dev(np.arange(4, pages, dtype=np.int32).reshape(B, pps))
    plen, lens = dev(np.array([50], np.int32)), dev(np.array([1, 20, 47], np.int32))
    k, v, q = (torch.zeros(B, n * D, dtype=torch.int16, device="cuda") for n in (hkv, hkv, hq))
    first = dev(rand(900, 50, 2 * hkv * D))
    vla.vla_kv_append_e4m3(first, first[:, hkv * D:], None, pp.reshape(1, 4), plen, kc, vc, ks, vs, 1, 50, 50, hkv, D, pages, page,
                           block, 4, 2 * hkv * D, 2 * hkv * D)
    n = vla.vla_attn_shared_prefix_e4m3_workspace_bytes(B, 1, hq, hkv, D, 64, pps * page)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(B, hq * D, dtype=torch.int16, device="cuda") for _ in range(2)]

    def call(out, stream=None):
        vla.vla_kv_append_e4m3(k, v, None, table, lens, kc, vc, ks, vs, B, 1, B, hkv, D, pages, page, block, pps, hkv * D, hkv * D,
                               stream=stream)
        vla.vla_attn_shared_prefix_e4m3(q, kc, vc, ks, vs, pp, plen, table, lens, out, ws, n, B, 1, hq, hkv, D, pages, page, block, 4,
                                        pps, hq * D, hq * D, True, 0.125, stream=stream)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call(outs[0])
    side.synchronize()
    graphs = []
    for out in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out)
        graphs.append(g)
    for step in range(4):
        lens.add_(1)
        for t, width in ((k, hkv), (v, hkv), (q, hq)):
            t.copy_(dev(rand(910 + 3 * step + width, B, width * D, scale=1.0 + step)))
        call(outs[0])
        torch.cuda.synchronize()
        want = outs[0].clone()
        assert want.any()
        for g, out in zip(graphs, outs):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        outs[1].zero_()
        call(outs[1], side)
        side.synchronize()
        assert torch.equal(outs[1], want)
