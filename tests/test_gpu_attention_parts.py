"""Keys split into parts, or a prefix and a suffix walked apart: a part whose
only keys have a score of -inf.  The row sees them, so a NaN value among them
is NaN in the result (0 times NaN), as it is where the keys are one range, and
a finite one has no part."""
import numpy as np
import pytest

import bf16_gemm_vla_amd as vla
import synthetic
from tests.gpu_util import Guarded, bf16_f64, dev, zeros_ws
from tests.test_gpu_attention import attention_bound, rand
from tests.test_gpu_e4m3_attention import Cache

pytestmark = pytest.mark.gpu

# sequences, rows, heads, key/value heads, size, prefix, a sequence's own keys (the last one is alone in its part); causal
# never, so that every row sees every key
CASES = [(1, 1, 4, 2, 64, 0, 129), (1, 2, 8, 1, 256, 0, 65), (1, 1, 8, 1, 256, 0, 129), (1, 9, 4, 2, 128, 0, 257), (3, 1, 4, 2, 72, 40, 1),
         (20, 5, 4, 2, 128, 70, 1), (1100, 2, 8, 2, 64, 60, 1), (1100, 1, 32, 8, 128, 60, 1), (1100, 2, 4, 1, 256, 60, 1)]


def check(got, q, k, v, keys, nan, B, L, hq, hkv, D):
    """k, v: the values of all keys of sequence b, keys[b] of them."""
    for b in range(B):
        g = bf16_f64(got[b])
        if nan == "channel":
            assert np.isnan(g[..., 5]).all() and np.isfinite(np.delete(g, 5, 2)).all(), b
        elif nan:
            assert np.isnan(g).all(), b
        else:
            kb, vb = k(b)[:-1], v(b)[:-1]
            ref, tol = attention_bound(q.reshape(B, L, hq, D)[b], kb, vb, np.full(L, keys - 1), 1.0)
            # exponentials below 2^-126 are 0 beside the largest one's, which is at least 1
            tol += 2.0 ** -126 * np.repeat(np.abs(bf16_f64(vb)).sum(0), hq // hkv, 0)
            assert (np.abs(g - ref) <= tol).all(), b


def queries(B, L, hq, D):
    q = rand(7001, B * L, hq, D, scale=2.0)
    q[:, :, 0] = 0x7F7F                            # bf16's largest: times -2 the score leaves fp32
    return q


@pytest.mark.parametrize("B,L,hq,hkv,D,prefix,own", CASES)
@pytest.mark.parametrize("nan", [None, "channel", "all"])
def test_e4m3_cache(B, L, hq, hkv, D, prefix, own, nan):
    c = Cache(B, hkv, D, 16, 1, prefix, [own] * B, 7000)
    q = queries(B, L, hq, D)
    c.codes[0][:, :, 0] = 0
    for b in range(B):
        slot = c.keys[b][-1]
        c.codes[0][slot, :, 0], c.bytes[0][slot] = 0xC0, 127
        if nan == "channel":
            c.codes[1][slot, :, 5] = 0x7F
        elif nan:
            c.bytes[1][slot] = 255
    got = c.call(q, prefix, [own] * B, L, hq, False, 1.0)
    check(got, q, lambda b: c.values(0, c.keys[b]), lambda b: c.values(1, c.keys[b]), prefix + own, nan, B, L, hq, hkv, D)


@pytest.mark.parametrize("B,L,hq,hkv,D,prefix,own", CASES)
@pytest.mark.parametrize("nan", [None, "channel", "all"])
def test_bf16_cache(B, L, hq, hkv, D, prefix, own, nan):
    page = 16
    npp, pps = -(-prefix // page), -(-own // page)
    pages = npp + B * pps
    order = synthetic.rng(7002).permutation(pages).astype(np.int32)
    pre, table = order[:npp], order[npp:].reshape(B, pps)
    k, v = rand(7003, pages * page, hkv, D), rand(7004, pages * page, hkv, D)
    k[:, :, 0] = 0
    keys = []
    for b in range(B):
        i, j = np.arange(prefix), np.arange(own)
        keys.append(np.concatenate([pre[i // page].astype(np.int64) * page + i % page if prefix else i,
                                    table[b][j // page].astype(np.int64) * page + j % page]))
        k[keys[b][-1], :, 0] = 0xC000
        if nan:
            v[keys[b][-1], :, 5 if nan == "channel" else slice(None)] = 0x7FC0
    q = queries(B, L, hq, D)
    n = vla.vla_attn_shared_prefix_workspace_bytes(B, L, hq, hkv, D, npp * page, pps * page)
    o = Guarded(B * L * hq * D * 2, fill=0x5A)
    vla.vla_attn_shared_prefix(dev(q), dev(k), dev(v), dev(pre) if npp else None, dev(np.array([prefix], np.int32)) if npp else None,
                               dev(table), dev(np.full(B, own, np.int32)), o.t, zeros_ws(n), n, B, L, hq, hkv, D, pages, page, npp, pps,
                               hq * D, hq * D, False, 1.0)
    o.check()
    check(o.numpy(np.uint16).reshape(B, L, hq, D), q, lambda b: k[keys[b]], lambda b: v[keys[b]], prefix + own, nan, B, L, hq, hkv, D)


def test_rows_that_see_nothing_stay_0_beside_them():
    """Causal rows without keys, and keys on pages that are not there, among parts whose scores are -inf."""
    B, L, hq, hkv, D = 3, 4, 4, 2, 64
    for missing in (False, True):
        c = Cache(B, hkv, D, 16, 1, 0, [1, 2, 130], 7010)
        q = queries(B, L, hq, D)
        c.codes[0][:, :, 0], c.bytes[0][:] = 0xC0, 127            # every score
        if missing:
            c.table[:] = -1
        got = c.call(q, 0, [1, 2, 130], L, hq, True, 1.0)
        assert not got.any()


@pytest.mark.parametrize("B,L,hq,hkv,D", [(5, 9, 4, 2, 64), (100, 5, 20, 4, 128), (300, 10, 4, 1, 64), (65, 20, 8, 2, 256)])
def test_first_rows_whose_only_score_is_minus_infinity(B, L, hq, hkv, D):
    """Causal rows over their own keys: the first sees one key, whose value is NaN in one channel.  That channel is NaN, the
    others are 0, over codes (16, 32, 64 and 128 rows a tile) and for packed prompts."""
    c = Cache(B, hkv, D, 16, 1, 0, [L] * B, 7020)
    q = queries(B, L, hq, D)
    c.codes[0][:, :, 0] = 0
    for b in range(B):
        slot = c.keys[b][0]
        c.codes[0][slot, :, 0], c.bytes[0][slot], c.codes[1][slot, :, 5] = 0xC0, 127, 0x7F
    rows = [c.call(q, 0, [L] * B, L, hq, True, 1.0)[:, 0]]
    k, v = (np.concatenate([c.values(i, c.keys[b]) for b in range(B)]) for i in range(2))
    cu = np.arange(B + 1, dtype=np.int32) * L
    o = Guarded(B * L * hq * D * 2, fill=0x5A)
    vla.vla_attn_prompt(dev(q), dev(k), dev(v), dev(cu), None, o.t, B, B * L, B * L, hq, hkv, D, hq * D, hkv * D, hkv * D, hq * D, True, 1.0)
    o.check()
    rows.append(o.numpy(np.uint16).reshape(B, L, hq, D)[:, 0])
    for g in rows:
        g = bf16_f64(g)
        assert np.isnan(g[..., 5]).all() and not np.delete(g, 5, 2).any()
