"""Attention over an E4M3 cache in every tile that its planner takes, against the
fp64 oracle: each case states the query rows of a tile and the parts of the
keys that it is there for, and asks the planner for them.  Tolerances are
those of tests/test_gpu_attention.py."""
import math

import numpy as np
import pytest
import torch

import bf16_gemm_vla_amd as vla
import synthetic
from tests.gpu_util import Guarded, bf16_f64, dev, zeros_ws
from tests.test_gpu_attention import assert_attention, attention_bound, rand
from tests.test_gpu_e4m3_attention import Cache, limits, run

pytestmark = pytest.mark.gpu


def planned(c, B, L, hq, prefix_rows, suffix_rows, split=None):
    """The cache's calls take tiles of so many rows; split: whether either range of keys is cut into parts."""
    rc, info = vla.vla_attn_shared_prefix_plan(B, L, hq, c.hkv, c.D, c.npp * c.page, c.pps * c.page, True)
    assert rc == 0 and info[:2] == [prefix_rows, suffix_rows], info
    assert split is None or (max(info[2:4]) > 1) == split, info


def checked(B, L, hq, hkv, D, page, block, prefix, lens, causal, prefix_rows, suffix_rows, split=None, seed=0, **sizes):
    run(B, L, hq, hkv, D, page, block, prefix, lens, causal, seed=seed,
        change=lambda c: planned(c, B, L, hq, prefix_rows, suffix_rows, split), **sizes)


# ------------------------------------------- 32 rows: few rows in two groups

@pytest.mark.parametrize("D", [64, 72, 128, 104])
def test_32_rows_of_each_sequence(D):
    checked(100, 5, 20, 4, D, 16, 8, 0, [b % 37 for b in range(100)], True, 0, 32, split=False, seed=1000 + D)
    checked(100, 20, 4, 4, D, 16, 16, 60, [b % 17 for b in range(100)], D == 72, 32, 32, split=False, seed=1010 + D)


@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("G", [5, 6])
def test_32_rows_behind_a_long_prefix(D, G):
    """Parts of the prefix, with and without parts of the suffixes; 25 and 30 rows."""
    checked(5, 1, 2 * G, 2, D, 16, 16, 4100, [1, 0, 9, 16, 5], True, 32, 32, split=True, seed=1100 + D + G)
    checked(5, 1, G, 1, D, 64, 32, 4097, [1000, 0, 900, 33, 1024], False, 32, 32, split=True, seed=1110 + D + G)
    checked(5, 1, G, 1, D, 16, 4, 4111, [0] * 5, False, 32, 0, split=True, seed=1120 + D + G, pages_per_seq=0)


@pytest.mark.parametrize("hq,hkv,D,L", [(8, 8, 64, 1603), (8, 8, 72, 1603), (16, 8, 128, 801)])
def test_32_rows_of_one_long_chunk(hq, hkv, D, L):
    """A prefill chunk over its cache: causal limits run through the sub-tiles."""
    checked(1, L, hq, hkv, D, 16, 16, 70, [L + 40], True, 0, 32, seed=1200 + D)


@pytest.mark.parametrize("D", [64, 104])
def test_32_rows_of_each_sequence_over_parts(D):
    checked(200, 50, 1, 1, D, 64, 64, 1970, [0] * 200, False, 0, 32, split=True, seed=1300 + D, pages_per_seq=0)


# --------------------------------------------------- tall tiles, 64 and 128

TALL = [  # sequences, rows, heads, key/value heads, rows of a prefix tile, of a suffix tile
    (300, 10, 4, 1, 0, 64), (300, 20, 4, 1, 0, 128), (1100, 2, 8, 2, 64, 64), (65, 20, 32, 8, 128, 128), (1100, 1, 32, 8, 128, 16),
    (2000, 20, 1, 1, 128, 32), (1100, 10, 4, 1, 128, 64), (300, 10, 4, 1, 16, 64), (41, 10, 32, 8, 32, 64)]


@pytest.mark.parametrize("B,L,hq,hkv,prefix_rows,suffix_rows", TALL)
@pytest.mark.parametrize("D", [64, 128, 72])
def test_tall_tiles(B, L, hq, hkv, prefix_rows, suffix_rows, D):
    prefix = 60 if prefix_rows else 0
    checked(B, L, hq, hkv, D, 16, 8, prefix, [b % 17 for b in range(B)], L > 1, prefix_rows, suffix_rows, seed=2000 + D + B)


@pytest.mark.parametrize("B,L,hq,hkv,prefix_rows,suffix_rows", [
    (65, 10, 8, 2, 0, 64), (65, 20, 8, 2, 0, 128), (65, 10, 8, 2, 16, 64), (1100, 2, 4, 1, 64, 64), (1100, 2, 8, 2, 128, 16),
    (65, 10, 32, 8, 128, 64), (300, 20, 4, 1, 128, 128)])
@pytest.mark.parametrize("D", [256, 136])
def test_tall_tiles_of_wide_heads(B, L, hq, hkv, prefix_rows, suffix_rows, D):
    prefix = 60 if prefix_rows else 0
    checked(B, L, hq, hkv, D, 16, 16, prefix, [b % 17 for b in range(B)], True, prefix_rows, suffix_rows, seed=2100 + D + B)


@pytest.mark.parametrize("hq,hkv,D,L,rows", [(8, 8, 64, 2100, 64), (32, 8, 128, 1100, 128), (8, 1, 256, 1100, 64), (8, 1, 256, 2100, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_tall_tiles_of_one_long_chunk(hq, hkv, D, L, rows, causal):
    """Several stages of keys, the causal limit among them, behind a prefix that each row sees whole."""
    checked(1, L, hq, hkv, D, 16, 16, 70, [L + 133], causal, 0, rows, seed=2200 + D + L)


@pytest.mark.parametrize("hq,hkv,D", [(32, 8, 64), (32, 8, 128), (16, 4, 256)])
def test_tall_prefix_of_several_stages(hq, hkv, D):
    checked(1100, 1, hq, hkv, D, 16, 16, 141, [0] * 1100, False, 128, 0, seed=2300 + D, pages_per_seq=0)


# ------------------------------------- what is not finite, and what is not there

FORMS = [  # sequences, rows, heads, key/value heads, size, rows of a tile
    (5, 9, 4, 2, 64, 16), (5, 9, 4, 2, 256, 16), (100, 5, 20, 4, 64, 32), (100, 5, 20, 4, 72, 32), (100, 5, 20, 4, 128, 32),
    (300, 10, 4, 1, 64, 64), (300, 10, 4, 1, 128, 64), (65, 10, 8, 2, 256, 64), (300, 20, 4, 1, 64, 128), (300, 20, 4, 1, 128, 128),
    (65, 20, 8, 2, 256, 128)]


@pytest.mark.parametrize("B,L,hq,hkv,D,rows", FORMS)
@pytest.mark.parametrize("what", ["value code", "value scale", "key code", "key scale"])
def test_nan_reaches_the_rows_that_see_it(B, L, hq, hkv, D, rows, what):
    """A NaN in the middle of every second sequence's new rows: the rows before it are as without it, the others NaN, in that
    channel alone where it is a value's code."""
    lens = [L + b % 23 for b in range(B)]
    at = [n - L // 2 - 1 for n in lens]                       # the key that row L - 1 - L // 2 is the first to see
    i, seed = int(what.startswith("value")), 3000 + D + rows

    def change(c):
        planned(c, B, L, hq, 0, rows)
        for b in range(0, B, 2):
            slot = c.keys[b][at[b]]
            if what.endswith("code"):
                c.codes[i][slot, hkv - 1, 5] = 0xFF if b % 4 else 0x7F
            else:
                c.bytes[i][slot, hkv - 1] = 255               # blocks of one row
    got, c, q = run(B, L, hq, hkv, D, 16, 1, 0, lens, True, seed=seed, change=change, check=False)
    first = L - 1 - L // 2
    for b in range(B):
        lim = limits(L, 0, lens[b], True)
        k, v = c.values(0, c.keys[b]), c.values(1, c.keys[b])
        if b % 2:
            assert_attention(got[b], q.reshape(B, L, hq, D)[b], k, v, lim, float(np.float32(1 / math.sqrt(D))), f"sequence {b}")
            continue
        g = bf16_f64(got[b]).reshape(L, hkv, hq // hkv, D)
        bad = np.zeros(g.shape, bool)
        bad[first:, -1, :, 5 if what == "value code" else slice(None)] = True
        assert np.isnan(g[bad]).all() and np.isfinite(g[~bad]).all(), b
        k[at[b], -1], v[at[b], -1] = 0, 0                     # rows that do not see it need no value of it
        ref, tol = attention_bound(q.reshape(B, L, hq, D)[b, :first], k, v, lim[:first], float(np.float32(1 / math.sqrt(D))))
        assert (np.abs(g.reshape(L, hq, D)[:first] - ref) <= tol).all(), b


@pytest.mark.parametrize("B,L,hq,hkv,D,rows", FORMS)
def test_nan_value_of_a_key_whose_score_is_minus_infinity(B, L, hq, hkv, D, rows):
    """The weight is 0, and 0 times NaN is NaN; with a finite value there the row is as without the key."""
    lens = [L + b % 23 for b in range(B)]
    q = rand(3900, B * L, hq, D, scale=2.0)
    q[:, :, 0] = 0x7F7F                                       # bf16's largest: times -2 the score leaves fp32
    for nan in (None, "code", "scale"):
        c = Cache(B, hkv, D, 16, 1, 0, lens, 3901)
        planned(c, B, L, hq, 0, rows)
        c.codes[0][:, :, 0] = 0
        for b in range(B):
            slot = c.keys[b][0]                               # every row sees it
            c.codes[0][slot, :, 0] = 0xC0                     # -2
            c.bytes[0][slot] = 127
            if nan == "code":
                c.codes[1][slot] = 0x7F
            elif nan == "scale":
                c.bytes[1][slot] = 255
        got = c.call(q, 0, lens, L, hq, True, 1.0)
        for b in range(B):
            g, lim = bf16_f64(got[b]), limits(L, 0, lens[b], True)
            sees_more = lim > 1                               # a row whose only score is -inf gives 0, whatever the value
            if nan:
                assert np.isnan(g[sees_more]).all(), (b, nan)
            else:
                k, v = c.values(0, c.keys[b][1:]), c.values(1, c.keys[b][1:])
                ref, tol = attention_bound(q.reshape(B, L, hq, D)[b][sees_more], k, v, lim[sees_more] - 1, 1.0)
                # scores differ by hundreds here: exponentials below 2^-126 are 0 beside the largest one's, which is at least 1
                tol += 2.0 ** -126 * np.repeat(np.abs(bf16_f64(v)).sum(0), hq // hkv, 0)
                assert (np.abs(g[sees_more] - ref) <= tol).all(), b


@pytest.mark.parametrize("B,L,hq,hkv,D,rows", FORMS)
def test_pages_that_are_not_there(B, L, hq, hkv, D, rows):
    lens = [L + 20 + b % 23 for b in range(B)]
    c = Cache(B, hkv, D, 16, 16, 0, lens, 3950)
    planned(c, B, L, hq, 0, rows)
    keys = [x.copy() for x in c.keys]
    for b in range(B):
        c.table[b, b % 2] = (-1, c.pages, 1 << 30)[b % 3]
    q = rand(3951, B * L, hq, D)
    got = c.call(q, 0, lens, L, hq, False, 0.1)
    for b in range(B):
        j = np.arange(lens[b])
        at = keys[b][j // 16 != b % 2]
        assert_attention(got[b], q.reshape(B, L, hq, D)[b], c.values(0, at), c.values(1, at), np.full(L, len(at)), float(np.float32(0.1)))


@pytest.mark.parametrize("B,L,hq,hkv,D,prefix,prefix_rows,suffix_rows", [
    (5, 1, 12, 2, 64, 4100, 32, 32), (5, 1, 12, 2, 72, 4100, 32, 32), (5, 1, 12, 2, 128, 4100, 32, 32), (20, 64, 16, 4, 64, 0, 0, 64),
    (20, 64, 16, 4, 128, 0, 0, 64), (20, 64, 16, 4, 120, 0, 0, 64), (20, 64, 8, 1, 256, 70, 0, 64), (20, 64, 32, 8, 64, 0, 0, 128),
    (20, 64, 32, 8, 128, 70, 0, 128), (40, 64, 8, 1, 256, 0, 0, 128), (1100, 1, 32, 8, 128, 60, 128, 16)])
def test_cache_past_4_gib_in_each_tile(B, L, hq, hkv, D, prefix, prefix_rows, suffix_rows):
    page, block = 16, 8
    lens = [L + b % 5 for b in range(B)]
    small = Cache(B, hkv, D, page, block, prefix, lens, 4000 + D)
    planned(small, B, L, hq, prefix_rows, suffix_rows)
    pages = (5 << 30) // (hkv * D) // page
    spread = np.sort(synthetic.rng(4001).choice(pages, small.pages, replace=False))
    spread[-1] = pages - 1
    codes = [torch.zeros(pages * page, hkv, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(pages * page // block, hkv, dtype=torch.uint8, device="cuda") for _ in range(2)]
    rows_at = torch.from_numpy((spread[:, None] * page + np.arange(page)).ravel()).cuda()
    blocks_at = torch.from_numpy((spread[:, None] * (page // block) + np.arange(page // block)).ravel()).cuda()
    for i in range(2):
        codes[i][rows_at] = dev(small.codes[i])
        scales[i][blocks_at] = dev(small.bytes[i])
    q = rand(4002, B * L, hq, D, scale=2.0)
    n = vla.vla_attn_shared_prefix_e4m3_workspace_bytes(B, L, hq, hkv, D, small.npp * page, small.pps * page)
    o, w = Guarded(B * L * hq * D * 2), zeros_ws(n)
    vla.vla_attn_shared_prefix_e4m3(
        dev(q), *codes, *scales, dev(spread[small.prefix_pages].astype(np.int32)) if prefix else None,
        dev(np.array([prefix], np.int32)) if prefix else None, dev(spread[small.table].astype(np.int32)),
        dev(np.array(lens, np.int32)), o.t, w, n, B, L, hq, hkv, D, pages, page, block, small.npp, small.pps, hq * D, hq * D, True, 0.1)
    o.check()
    got = o.numpy(np.uint16).reshape(B, L, hq, D)
    for b in range(B):
        at = small.keys[b]
        assert_attention(got[b], q.reshape(B, L, hq, D)[b], small.values(0, at), small.values(1, at), limits(L, prefix, lens[b], True),
                         float(np.float32(0.1)), f"sequence {b}")
