"""Calls on an E4M3 cache that the documentation allows beside the usual ones:
rows that are columns of a wider matrix, pages named more than once, the
largest pages, scale bytes that other programs may leave."""
import numpy as np
import pytest
import torch

import bf16_gemm_vla_amd as vla
import synthetic
from tests.eight_bit_ref import append
from tests.gpu_util import Guarded, bf16_f64, dev, zeros_ws
from tests.test_gpu_attention import assert_attention, rand
from tests.test_gpu_e4m3_append import Cache as AppendCache
from tests.test_gpu_e4m3_append import rows
from tests.test_gpu_e4m3_attention import Cache, limits

pytestmark = pytest.mark.gpu

FORMS = [(5, 9, 4, 2, 64), (3, 1, 4, 2, 72), (100, 5, 20, 4, 128), (300, 10, 4, 1, 64), (65, 20, 8, 2, 256)]   # 16, 16, 32, 64, 128 rows


@pytest.mark.parametrize("B,L,hq,hkv,D", FORMS)
@pytest.mark.parametrize("prefix", [0, 37])
def test_rows_in_wider_matrices(B, L, hq, hkv, D, prefix):
    """q's and the results' rows are column blocks of one matrix each: what lies between them stays."""
    lens = [L + b % 11 for b in range(B)]
    c = Cache(B, hkv, D, 16, 4, prefix, lens, 5000 + D)
    q = rand(5001, B * L, hq, D, scale=2.0)
    width = hq * D + 24
    wide = synthetic.rng(5002).integers(0, 1 << 16, (B * L, width)).astype(np.uint16)
    wide[:, 8:8 + hq * D] = q.reshape(B * L, -1)
    d = dev(wide)
    o = Guarded(B * L * width * 2, fill=0x5A)
    out = o.t.view(torch.int16).reshape(B * L, width)[:, 16:]
    n = vla.vla_attn_shared_prefix_e4m3_workspace_bytes(B, L, hq, hkv, D, c.npp * 16, c.pps * 16)
    vla.vla_attn_shared_prefix_e4m3(
        d[:, 8:], dev(c.codes[0]), dev(c.codes[1]), dev(c.bytes[0]), dev(c.bytes[1]), dev(c.prefix_pages) if prefix else None,
        dev(np.array([prefix], np.int32)) if prefix else None, dev(c.table), dev(np.array(lens, np.int32)), out, zeros_ws(n), n, B, L,
        hq, hkv, D, c.pages, 16, 4, c.npp, c.pps, width, width, True, 0.1)
    o.check()
    got = o.numpy(np.uint16).reshape(B * L, width)
    assert (got[:, :16] == 0x5A5A).all() and (got[:, 16 + hq * D:] == 0x5A5A).all()
    got = got[:, 16:16 + hq * D].reshape(B, L, hq, D)
    for b in range(B):
        at = c.keys[b]
        assert_attention(got[b], q.reshape(B, L, hq, D)[b], c.values(0, at), c.values(1, at), limits(L, prefix, lens[b], True),
                         float(np.float32(0.1)), f"sequence {b}")


@pytest.mark.parametrize("B,L,hq,hkv,D", FORMS)
def test_pages_named_more_than_once(B, L, hq, hkv, D):
    """By the prefix, within a sequence and by several sequences: each place counts."""
    page, prefix, lens = 16, 40, [L + 30 + b % 7 for b in range(B)]
    c = Cache(B, hkv, D, page, 16, prefix, lens, 5100 + D)
    c.prefix_pages[2] = c.prefix_pages[0]
    c.table[:, 1] = c.table[:, 0]
    c.table[1:, 2] = c.table[0, 2]
    c.table[:, 0] = c.prefix_pages[1]
    q = rand(5101, B * L, hq, D, scale=2.0)
    got = c.call(q, prefix, lens, L, hq, True, 0.1)
    for b in range(B):
        pre, own = np.arange(prefix), np.arange(lens[b])
        at = np.concatenate([c.prefix_pages[pre // page].astype(np.int64) * page + pre % page,
                             c.table[b][own // page].astype(np.int64) * page + own % page])
        assert_attention(got[b], q.reshape(B, L, hq, D)[b], c.values(0, at), c.values(1, at), limits(L, prefix, lens[b], True),
                         float(np.float32(0.1)), f"sequence {b}")


def test_pages_of_65536_rows():
    """Filled by the append (a chunk within the page, one over the border of two, one row at the end) and read again."""
    page, block, hkv, D, hq = 65536, 128, 1, 16, 4
    c = AppendCache(3, page, block, hkv, D, 5200)
    table = np.array([[2, 0]])
    for first, count, seed in ((0, 1000, 0), (65000, 1200, 1), (2 * page - 1, 1, 2)):
        k, v = rows(5201 + seed, count, hkv, D)
        d = dev(np.concatenate([k, v], 1).reshape(count, -1))
        vla.vla_kv_append_e4m3(d, d[:, D:], None, dev(table.astype(np.int32)), dev(np.array([first + count], np.int32)), c.gpu[0].t,
                               c.gpu[2].t, c.gpu[1].t, c.gpu[3].t, 1, count, count, hkv, D, 3, page, block, 2, 2 * D, 2 * D)
        for x, codes, scales in ((k, 0, 1), (v, 2, 3)):
            append(bf16_f64(x), np.array([0, count]), table, [first + count], c.host[codes], c.host[scales], page, block, count)
    c.check()
    lens = 66111
    q = rand(5210, 1, hq, D, scale=2.0)
    n = vla.vla_attn_shared_prefix_e4m3_workspace_bytes(1, 1, hq, hkv, D, 0, 2 * page)
    o = Guarded(hq * D * 2)
    vla.vla_attn_shared_prefix_e4m3(dev(q), c.gpu[0].t, c.gpu[2].t, c.gpu[1].t, c.gpu[3].t, None, None, dev(table.astype(np.int32)),
                                    dev(np.array([lens], np.int32)), o.t, zeros_ws(n), n, 1, 1, hq, hkv, D, 3, page, block, 0, 2, hq * D,
                                    hq * D, True, 0.25)
    o.check()
    at = np.arange(lens)
    at = table[0][at // page] * page + at % page
    values = Cache.__new__(Cache)
    values.codes, values.bytes, values.block = (c.host[0], c.host[2]), (c.host[1], c.host[3]), block
    assert_attention(o.numpy(np.uint16).reshape(1, hq, D), q, values.values(0, at), values.values(1, at), np.array([lens]), 0.25)


@pytest.mark.parametrize("block,D", [(16, 64), (128, 256)])
def test_append_behind_any_scale_byte(block, D):
    """A block of earlier rows keeps a larger scale, up to 254; 255 counts as 254, and a block that starts afresh forgets it."""
    c = AppendCache(6, 128, block, 1, D, 5300)
    for g, h in ((c.gpu[1], c.host[1]), (c.gpu[3], c.host[3])):
        h[:, 0] = np.array([255, 254, 253, 1, 0], np.uint8)[np.arange(len(h)) % 5]
        g.t.copy_(dev(h).flatten())
    table, first = np.arange(6).reshape(6, 1), np.arange(6) * (128 // block)
    for h in c.host[1::2]:
        h[first] = np.minimum(h[first], 254)                      # the blocks that the calls reach, in the 64-bit form
    for n in (4, 5, 1):                                           # behind three rows, behind four, from the first row again
        k, v = rows(5301 + n, 6, 1, D)
        c.append(k, v, None, table, [n] * 6, 1)
        assert (max(h[first].max() for h in c.host[1::2]) == 254) == (n > 1)


def test_append_offsets_that_fall_leave_rows_out_at_most():
    """Offsets are to rise; where they do not, so that sequences share rows, a block is appended as the definition has it or
    not at all."""
    B, n, page, block, hkv, D = 12, 300, 16, 16, 2, 64
    each = n // page + 1
    c = AppendCache(B * each, page, block, hkv, D, 5400)
    table = np.arange(B * each).reshape(B, each)
    k, v = rows(5401, n, hkv, D)
    cu, lens = np.array([0, n] * (B // 2) + [0]), np.full(B, n)
    before = [h.copy() for h in c.host]
    dk, dv = dev(k.reshape(n, -1)), dev(v.reshape(n, -1))
    vla.vla_kv_append_e4m3(dk, dv, dev(cu.astype(np.int32)), dev(table.astype(np.int32)), dev(lens.astype(np.int32)), c.gpu[0].t,
                           c.gpu[2].t, c.gpu[1].t, c.gpu[3].t, B, n, n, hkv, D, B * each, page, block, each, hkv * D, hkv * D)
    for x, codes, scales in ((k, 0, 1), (v, 2, 3)):
        for b in range(0, B, 2):                                  # the even sequences have all of the rows, the odd ones none
            append(bf16_f64(x), np.array([0, n]), table[b:b + 1], [n], c.host[codes], c.host[scales], page, block, n)
        got = [c.gpu[i].numpy(np.uint8).reshape(c.host[i].shape) for i in (codes, scales)]
        blocks = [y.reshape(B * each, -1, hkv, D) for y in (got[0], c.host[codes], before[codes])]
        done = (got[1] == c.host[scales]) & (blocks[0] == blocks[1]).all((1, 3))
        kept = (got[1] == before[scales]) & (blocks[0] == blocks[2]).all((1, 3))
        assert (done | kept).all() and done.any()
    for g in c.gpu:
        g.check()
