"""GPU parity of the append to an E4M3 cache: codes and scale bytes are equal
to the 64-bit form's, every step being exact or one rounding to nearest."""
import numpy as np
import pytest
import torch

import bf16_gemm_vla_amd as vla
import synthetic
from tests.eight_bit_ref import E4M3, append, e8m0_value
from tests.gpu_util import Guarded, bf16_f64, dev, host

pytestmark = pytest.mark.gpu


def rng(seed):
    return synthetic.rng(39000 + seed)


def bits(x):
    return synthetic.fp32_to_bf16_bits(np.asarray(x, np.float32))


class Cache:
    """A filled cache on the host and, guarded, on the GPU."""

    def __init__(self, pages, page, block, hkv, D, seed):
        r = rng(seed)
        self.pages, self.page, self.block, self.hkv, self.D = pages, page, block, hkv, D
        rows = pages * page
        self.host = []
        for i in range(2):
            codes = r.integers(0, 256, (rows, hkv, D)).astype(np.uint8)
            codes[(codes & 0x7F) == 0x7F] = 0x40
            self.host += [codes, r.integers(110, 130, (rows // block, hkv)).astype(np.uint8)]
        self.gpu = [Guarded(x.size) for x in self.host]
        for g, x in zip(self.gpu, self.host):
            g.t.copy_(dev(x).flatten())

    def append(self, k, v, cu, table, lens, longest, strides=None, stream=None):
        """One call and its 64-bit form; both caches are then equal."""
        total = k.shape[0]
        merged = np.concatenate([k.reshape(total, -1), v.reshape(total, -1), np.zeros((total, 8), np.uint16)], 1)
        d = dev(merged)
        width = merged.shape[1]
        vla.vla_kv_append_e4m3(d, d[:, self.hkv * self.D:], None if cu is None else dev(np.asarray(cu, np.int32)),
                               dev(np.asarray(table, np.int32)), dev(np.asarray(lens, np.int32)), self.gpu[0].t, self.gpu[2].t,
                               self.gpu[1].t, self.gpu[3].t, len(lens), longest, total, self.hkv, self.D, self.pages, self.page,
                               self.block, np.asarray(table).shape[1], width, width, stream=stream)
        ref_cu = np.arange(len(lens) + 1) * longest if cu is None else np.asarray(cu)
        for x, codes, scales in ((k, 0, 1), (v, 2, 3)):
            append(bf16_f64(x), ref_cu, np.asarray(table), lens, self.host[codes], self.host[scales], self.page, self.block, longest)
        self.check()

    def check(self):
        for name, g, x in zip(("k codes", "k scales", "v codes", "v scales"), self.gpu, self.host):
            g.check()
            got = g.numpy(np.uint8).reshape(x.shape)
            assert np.array_equal(got, x), (name, np.argwhere(got != x)[:3], got[got != x][:3], x[got != x][:3])


def rows(seed, total, hkv, D, spread=1.5):
    r = rng(seed)
    return tuple(bits(r.standard_normal((total, hkv, D)) * np.exp(spread * r.standard_normal((total, hkv, 1)))) for _ in range(2))


@pytest.mark.parametrize("hkv,D,page,block", [(8, 128, 16, 16), (1, 256, 64, 32), (2, 64, 128, 128), (16, 72, 32, 8), (1, 8, 16, 16),
                                              (3, 200, 64, 64), (4, 80, 16, 1), (2, 256, 128, 128), (5, 16, 1, 1), (1, 248, 8, 4)])
@pytest.mark.parametrize("lengths", [[(1, 0)], [(1, 5), (1, 16), (1, 31), (1, 300)], [(37, 0), (200, 13), (0, 40), (1, 64), (130, 127)]])
def test_append_equals_the_definition(hkv, D, page, block, lengths):
    new, before = [n for n, _ in lengths], [b for _, b in lengths]
    lens = [n + b for n, b in lengths]
    each = max(-(-n // page) for n in lens) + 1
    c = Cache(each * len(lens) + 2, page, block, hkv, D, D + page)
    table = rng(D).permutation(c.pages)[:each * len(lens)].reshape(len(lens), each)
    k, v = rows(D + block, sum(new) + 3, hkv, D)
    cu = np.concatenate([[0], np.cumsum(new)])
    c.append(k, v, cu, table, lens, max(new))
    # again behind those rows, blocks now partly filled, with larger values: scales grow
    k, v = rows(D + block + 1, sum(new) + 3, hkv, D, 3.0)
    lens = [n + m for n, m in zip(lens, new)]
    if max(-(-n // page) for n in lens) <= each:
        c.append(k, v, cu, table, lens, max(new))


def test_append_uniform_rows_and_many_sequences():
    for B, L in ((130, 1), (70, 3), (3, 50)):
        c = Cache(B * 8 + 1, 16, 16, 2, 64, B)
        table = rng(B).permutation(c.pages)[:B * 8].reshape(B, 8)
        lens = rng(B + 1).integers(L, 100, B)
        c.append(*rows(B, B * L, 2, 64), None, table, lens, L)
        for step in range(3):
            lens = np.minimum(lens + L, 128)
            c.append(*rows(B + step, B * L, 2, 64, 1.0 + step), None, table, lens, L)


@pytest.mark.parametrize("B", [63, 64, 65, 200])
def test_append_ragged_batches_find_every_block(B):
    """Sequences of no rows among them, longest far above the others: the scan over the batch."""
    r = rng(B)
    new = r.integers(0, 5, B)
    new[B // 3] = 90
    new[::7] = 0
    before = r.integers(0, 40, B)
    lens = new + before
    c = Cache(9 * B + 3, 16, 8, 1, 32, B)
    table = r.permutation(c.pages)[:9 * B].reshape(B, 9)
    c.append(*rows(B, int(new.sum()) + 2, 1, 32), np.concatenate([[0], np.cumsum(new)]), table, lens, int(new.max()))


def test_append_bad_pages_lengths_and_offsets():
    """Nothing in device arrays leads outside: missing pages, lengths past the table and below the new rows, offsets outside."""
    c = Cache(6, 16, 16, 2, 64, 5)
    table = np.array([[0, -1, 2, 7], [1 << 30, 3, -(1 << 31), 4], [5, 5, 5, 5]])
    k, v = rows(5, 90, 2, 64)
    c.append(k, v, [0, 40, 80, 80], table, [50, 40, 7], 40)
    c.append(k, v, [0, 3, 30, 30], table, [1 << 30, 20, 0], 40)         # past the table: bounded; row 0 of 20 is the 8th new one
    c.append(k, v, [0, 40, 70, 70], table, [10, -5, 3], 40)             # more new rows than the length: the last 10
    g = [x.t.clone() for x in c.gpu]
    d = dev(k.reshape(90, -1))
    for cu in ([-5, -1, -1, -9], [95, 1 << 30, 1 << 30, (1 << 31) - 1], [-(1 << 31), -(1 << 31), -1, 0]):
        vla.vla_kv_append_e4m3(d, d, dev(np.array(cu, np.int32)), dev(table.astype(np.int32)), dev(np.array([50, 40, 7], np.int32)),
                               c.gpu[0].t, c.gpu[2].t, c.gpu[1].t, c.gpu[3].t, 3, 40, 90, 2, 64, 6, 16, 16, 4, 128, 128)
    c.check()
    assert all(torch.equal(a, b.t) for a, b in zip(g, c.gpu))


def test_append_extreme_values():
    hkv, D, page = 1, 64, 16
    c = Cache(8, page, 16, hkv, D, 7)
    x = np.zeros((16, 1, D), np.float32)
    x[0] = 0                                      # a block that starts with zeros: scale byte 0
    x[1] = 1e-40                                  # subnormal bf16
    x[2, 0, :3] = 9.2e-41, -9.2e-41, 1e-38
    x[3] = 1.0
    x[4, 0, 5] = np.inf
    x[4, 0, 6] = np.nan
    x[4, 0, 7] = -np.inf
    x[5] = 3.3e38
    x[6] = -0.0
    x[7] = 2.0 ** -9 * np.arange(D)
    b = bits(x)
    b[8:, 0, :] = rng(8).integers(0, 0x7F80, (8, D))          # every exponent in one block
    c.append(b, b[::-1].copy(), None, [[3, 4]], [16], 16)     # at once
    for i in range(16):                                       # and row by row: the scale grows over the whole range
        c.append(b[i:i + 1], b[15 - i:16 - i], None, [[5, 6]], [i + 1], 1)
    at_once, by_rows = (host(c.gpu[1].t)[p] for p in (3, 5))
    assert at_once == by_rows
    # nan codes stay, and the finite rows around them keep their values
    codes = c.gpu[0].numpy(np.uint8).reshape(-1, D)[5 * page + 4]
    assert (codes[5:8] == 0x7F).all() and (codes[:5] == 0).all()
    for most in (448.0, 449.0, 450.0, 224.0, 2.0 ** -118, 1.75 * 2.0 ** -119, 1.7578125 * 2.0 ** -119):
        c.append(bits(np.full((1, 1, D), most)), bits(np.full((1, 1, D), -most)), None, [[1, 2]], [1], 1)


def test_append_every_bf16_under_every_code():
    """Each bf16 magnitude from 2^-18 to 511 under the scale 1 (or 2), ties among them, against nearest-even."""
    D = 256
    every = np.arange(0x3F80 - 18 * 128, 0x3F80 + 9 * 128, dtype=np.uint16)
    every = np.concatenate([every, np.full(-len(every) % D, 0x43E0, np.uint16)]).reshape(-1, 1, D)
    n = len(every)
    c = Cache(n + 1, 1, 1, 1, D, 9)
    every[:, 0, 0] = 0x43E0                       # 448: the scale is 1, but of the last row, which goes up to 511
    c.append(every, every | 0x8000, None, np.arange(n)[None], [n], n)
    assert (c.gpu[1].numpy(np.uint8)[:n] == [127] * (n - 1) + [128]).all()


def test_append_prefix_then_suffix_values():
    """What the cache stands for is within half an E4M3 step of the rows, or of the subnormal step."""
    hkv, D, page, block, T = 4, 128, 64, 16, 300
    c = Cache(20, page, block, hkv, D, 11)
    k, v = rows(12, T, hkv, D)
    pages = rng(13).permutation(20)[:6]
    c.append(k, v, None, pages[None], [T], T)
    slot = pages[np.arange(T) // page] * page + np.arange(T) % page
    for x, codes, scales in ((k, 0, 1), (v, 2, 3)):
        s = e8m0_value(c.host[scales][slot // block])[..., None]
        got, want = E4M3[c.host[codes][slot]] * s, bf16_f64(x)
        assert (np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * s)).all()


def test_append_captured_and_on_another_stream():
    c = Cache(40, 16, 16, 2, 64, 15)
    table, lens = dev(rng(16).permutation(40)[:32].reshape(4, 8).astype(np.int32)), dev(np.array([3, 17, 60, 100], np.int32))
    k, v = (dev(x.reshape(4, -1)) for x in rows(17, 4, 2, 64))
    start = [g.t.clone() for g in c.gpu]

    def call():
        vla.vla_kv_append_e4m3(k, v, None, table, lens, c.gpu[0].t, c.gpu[2].t, c.gpu[1].t, c.gpu[3].t, 4, 1, 4, 2, 64, 40, 16, 16,
                               8, 128, 128)
    def fresh():
        for g, x in zip(c.gpu, start):
            g.t.copy_(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(3):
        lens.add_(1)
        k.copy_(dev(rows(18 + step, 4, 2, 64)[0].reshape(4, -1)))
        fresh()
        call()
        torch.cuda.synchronize()
        eager = [g.t.clone() for g in c.gpu]
        fresh()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g.t, x) for g, x in zip(c.gpu, eager))
        for g in c.gpu:
            g.check()
