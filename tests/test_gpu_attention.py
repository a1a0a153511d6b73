"""GPU parity of the attention operators against the fp64 oracle.

Tolerances, from the arithmetic alone:
  * append: an output is one bf16 rounding (half a step, 2^-8 relative) of an
    fp32 result.  The angle is rounded once as a fraction of a revolution
    (pi * 2^-24 radians at most) and its sine and cosine are within 2^-23, the
    norm and the two products of a pair add at most 6 roundings of 2^-24: in
    all below 2^-20 of |a| + |b| for the pair (a, b), times rot_scale.
  * attention: scores are exact products summed in fp32, so a score is off by
    at most (D + 8) 2^-24 of scale * sum|q k|; the weights take that error as
    a relative one (twice: in the sum too), 2^-8 from their rounding to bf16,
    2^-20 from exp2 and its argument's rounding per unit of score below 2^4
    (larger arguments belong to weights below 2^-16), and the sums over m keys
    m 2^-24 each; the output is rounded once (2^-8)."""
import math

import numpy as np
import pytest
import torch

import bf16_gemm_vla_amd as vla
import oracle
import synthetic
from tests.gpu_util import Guarded, bf16_f64, dev, host, zeros_ws

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -8          # half a bf16 step, relative
TINY = 2.0 ** -133       # half the smallest bf16 step


def rand(seed, *shape, scale=1.0):
    x = synthetic.rng(9000 + seed).standard_normal(shape, dtype=np.float32) * np.float32(scale)
    return synthetic.fp32_to_bf16_bits(x)


def out_bits(t, *shape):
    return host(t, np.uint16).reshape(shape)


# ---------------------------------------------------------------- append

def freqs(rot, base=10000.0):
    return (base ** (-2.0 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)


def check_rotated(got, x, w, freq, pos, rot, inter, rot_scale, eps, what):
    ref = oracle.norm_rope(x, w, freq, pos, rot, inter, rot_scale, eps)
    size = np.abs(oracle.norm_rope(x, w, None, None, 0, False, 1.0, eps))
    pair = size.copy()
    if rot:
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
        pair[..., a] = pair[..., b] = abs(rot_scale) * (size[..., a] + size[..., b])
    err = np.abs(bf16_f64(got) - ref)
    bad = err > EPS * np.abs(ref) + 2.0 ** -20 * pair * (1 + EPS) + TINY
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[0]}"


def run_append(T, hq, hkv, D, rot, inter=False, norm=(True, True), append=True, k_out=True, pos=None, rot_scale=1.0,
               eps=1e-6, slots=None, merged=True, in_place=False, q=None, seed=0, extra=0):
    q = rand(seed, T, hq, D) if q is None else q
    k, v = rand(seed + 1, T, hkv, D), rand(seed + 2, T, hkv, D)
    qw, kw = (rand(seed + 3 + i, D, scale=0.5) if norm[i] else None for i in range(2))
    pos = np.arange(T, dtype=np.int32) * 3 + 5 if pos is None else np.asarray(pos, np.int32)
    freq = freqs(rot)
    n_slots = T + 7
    slots = synthetic.rng(9100 + seed).permutation(n_slots)[:T].astype(np.int64) if slots is None else np.asarray(slots, np.int64)
    kc, vc = rand(seed + 5, n_slots, hkv, D), rand(seed + 6, n_slots, hkv, D)
    if merged:
        width = (hq + 2 * hkv) * D + 8 * extra
        rows = np.zeros((T, width), np.uint16)
        rows[:, :(hq + 2 * hkv) * D] = np.concatenate([x.reshape(T, -1) for x in (q, k, v)], 1)
        d = dev(rows)
        dq, dk, dv = d[:, :hq * D], d[:, hq * D:(hq + hkv) * D], d[:, (hq + hkv) * D:]
        sq = sk = sv = width
    else:
        dq, dk, dv, sq, sk, sv = dev(q), dev(k), dev(v), hq * D, hkv * D, hkv * D
    go, gk = Guarded(T * hq * D * 2), Guarded(T * hkv * D * 2)
    gkc, gvc = Guarded(kc.nbytes), Guarded(vc.nbytes)
    gkc.t.copy_(dev(kc).flatten().view(torch.uint8))
    gvc.t.copy_(dev(vc).flatten().view(torch.uint8))
    qo, qs = (dq, sq) if in_place else (go.t, hq * D)
    ko, ks = (None, 0) if not k_out else ((dk, sk) if in_place else (gk.t, hkv * D))
    vla.vla_qk_norm_rope_append(dq, dk, dv if append else None, None if qw is None else dev(qw),
                                None if kw is None else dev(kw), dev(freq) if rot else None, dev(pos) if rot else None,
                                dev(slots) if append else None, qo, ko, gkc.t if append else None,
                                gvc.t if append else None, T, hq, hkv, D, rot, sq, sk, sv if append else 0, qs, ks,
                                n_slots if append else 0, vla.VLA_ROPE_INTERLEAVED if inter else vla.VLA_ROPE_HALF,
                                rot_scale, eps)
    for g in (go, gk, gkc, gvc):
        g.check()
    def strided(t, stride, n):
        if stride == n:
            return out_bits(t.contiguous() if t.dtype == torch.int16 else t, T, n)
        return host(t).view(np.uint16)[:, :n]
    got_q = strided(qo, qs, hq * D).reshape(T, hq, D)
    check_rotated(got_q, q, qw, freq, pos, rot, inter, rot_scale, eps, "q")
    if k_out:
        got_k = strided(ko, ks, hkv * D).reshape(T, hkv, D)
        check_rotated(got_k, k, kw, freq, pos, rot, inter, rot_scale, eps, "k")
    got_kc, got_vc = gkc.numpy(np.uint16).reshape(kc.shape), gvc.numpy(np.uint16).reshape(vc.shape)
    if append:
        kept = (slots >= 0) & (slots < n_slots)
        check_rotated(got_kc[slots[kept]], k[kept], kw, freq, pos[kept], rot, inter, rot_scale, eps, "k_cache")
        if k_out:
            assert np.array_equal(got_kc[slots[kept]], got_k[kept])
        vc[slots[kept]] = v[kept]
        kc[slots[kept]] = got_kc[slots[kept]]
    assert np.array_equal(got_kc, kc) and np.array_equal(got_vc, vc)          # other slots as they were
    if in_place:
        assert np.array_equal(host(d).view(np.uint16)[:, (hq + hkv) * D:], rows[:, (hq + hkv) * D:])
    return got_q


@pytest.mark.parametrize("T,hq,hkv,D,rot,inter,norm", [
    (1, 8, 1, 256, 256, False, (False, False)), (50, 8, 1, 256, 256, False, (False, False)),
    (3, 4, 2, 8, 8, True, (True, True)), (17, 16, 16, 72, 72, False, (True, True)), (5, 12, 12, 80, 32, True, (True, False)),
    (129, 28, 4, 128, 64, True, (True, True)), (33, 5, 5, 104, 0, False, (True, True)), (700, 8, 8, 64, 16, False, (False, True)),
    (9000, 2, 1, 64, 64, False, (True, True)), (2, 40, 8, 128, 128, True, (True, True)), (7, 3, 1, 16, 8, False, (True, False)),
    (4, 6, 2, 40, 40, True, (False, False)), (1, 1, 1, 248, 240, False, (True, True))])
def test_append_matches_oracle(T, hq, hkv, D, rot, inter, norm):
    run_append(T, hq, hkv, D, rot, inter, norm, rot_scale=1.1, seed=10 * T + D)


def test_append_slots_outside_the_cache_append_nothing():
    slots = [3, -1, 18, 1 << 40, 0, -(1 << 50), 17, 18 + (1 << 32), 5, -1, -1]
    run_append(11, 4, 2, 64, 64, slots=slots, seed=31)


def test_append_forms():
    run_append(9, 8, 2, 64, 64, merged=True, in_place=True, extra=3, seed=41)
    run_append(9, 8, 2, 72, 64, merged=True, in_place=True, k_out=False, seed=42)
    run_append(9, 8, 2, 64, 64, append=False, seed=43)
    run_append(9, 8, 2, 64, 64, k_out=False, merged=False, seed=44)
    run_append(9, 8, 2, 64, 64, merged=True, in_place=True, append=False, inter=True, seed=45)


def test_append_far_positions_and_extreme_rows():
    pos = [0, -1, 1 << 20, (1 << 31) - 1, -(1 << 31), 1000003, 7, 8]
    run_append(8, 4, 1, 128, 128, pos=pos, rot_scale=-1.5, seed=51)
    q = rand(52, 8, 4, 64)
    q[0] = 0                                   # zero rows: eps alone
    q[1] = 0x7F00                              # 2^127: its square is past fp32
    q[2] = 0x0001                              # the smallest bf16
    q[3, 0] = synthetic.fp32_to_bf16_bits(np.full(64, 1e-20, np.float32))
    run_append(8, 4, 1, 64, 0, q=q, norm=(True, True), eps=1e-6, seed=53)
    q[0] = 0x3F80
    run_append(8, 4, 1, 64, 0, q=q, norm=(True, True), eps=0.0, seed=53)


# ------------------------------------------------------------- attention

def attention_bound(q, k, v, limits, scale):
    ref, wabs = oracle.attention(q, k, v, limits, scale)
    n, hq, D = q.shape
    m, hkv = k.shape[0], k.shape[1]
    size = np.zeros((n, hq, 1))
    if m:
        kabs = np.abs(bf16_f64(k))
        kabs[~np.isfinite(kabs)] = 0
        for h in range(hq):
            size[:, h, 0] = (np.abs(bf16_f64(q[:, h])) @ kabs[:, h * hkv // hq].T).max(1) * scale
    score = (D + 8) * 2.0 ** -24 * size
    tol = EPS * np.abs(ref) + (EPS + 2 * score + 2 * m * 2.0 ** -24 + 2.0 ** -20) * (1 + EPS) * wabs + TINY
    return ref, tol


def assert_attention(got, q, k, v, limits, scale, what=""):
    ref, tol = attention_bound(q, k, v, limits, scale)
    g = bf16_f64(got)
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[0]}: {g[bad][0]} for {ref[bad][0]}"


def offsets(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


def run_prompt(nq, nk, hq, hkv, D, causal, scale=None, pad=(0, 0), seed=0, qkv=None, same_cu=False, merged=False,
               check=True, poison=None):
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    cq, ck = offsets(nq), offsets(nk)
    Tq, Tk = max(1, int(cq[-1]) + pad[0]), max(1, int(ck[-1]) + pad[1])
    q, k, v = rand(seed, Tq, hq, D, scale=2.0), rand(seed + 1, Tk, hkv, D), rand(seed + 2, Tk, hkv, D)
    if poison:
        poison(q, k, v)
    if merged:
        rows = np.concatenate([x.reshape(Tq, -1) for x in (q, k, v)] + [np.zeros((Tq, 16), np.uint16)], 1)
        d = dev(rows)
        dq, dk, dv = d, d[:, hq * D:], d[:, (hq + hkv) * D:]
        sq = sk = sv = rows.shape[1]
    else:
        dq, dk, dv, sq, sk, sv = dev(q), dev(k), dev(v), hq * D, hkv * D, hkv * D
    o = Guarded(Tq * hq * D * 2, fill=0x5A)
    vla.vla_attn_prompt(dq, dk, dv, dev(cq), None if same_cu else dev(ck), o.t, len(nq), Tq, Tk, hq, hkv, D, sq, sk, sv,
                        hq * D, causal, scale)
    o.check()
    got = o.numpy(np.uint16).reshape(Tq, hq, D)
    if check:
        for b in range(len(nq)):
            a, e, s, t = cq[b], cq[b + 1], ck[b], ck[b + 1]
            lim = np.full(e - a, t - s, np.int64)
            if causal:
                lim = np.clip(np.arange(e - a) + 1 + (t - s) - (e - a), 0, t - s)
            assert_attention(got[a:e], q[a:e], k[s:t], v[s:t], lim, float(np.float32(scale)), f"sequence {b}")
        assert (got[cq[-1]:] == 0x5A5A).all()                     # rows behind the last sequence
    return got, (q, k, v)


HEADS = [(8, 1, 256), (8, 2, 128), (4, 4, 64), (3, 1, 72), (5, 5, 8), (16, 8, 80), (2, 1, 200)]


@pytest.mark.parametrize("hq,hkv,D", HEADS)
@pytest.mark.parametrize("causal", [False, True])
def test_prompt_ragged(hq, hkv, D, causal):
    run_prompt([1, 0, 65, 128, 33, 7], [1, 3, 65, 200, 0, 64], hq, hkv, D, causal, pad=(3, 2), seed=100 + D)


@pytest.mark.parametrize("hq,hkv,D", [(32, 8, 64), (40, 8, 128), (64, 4, 256), (48, 4, 72)])
def test_prompt_wide_tiles(hq, hkv, D):
    """Enough rows for the 128-row tiles, at sizes that end inside a tile."""
    n = {64: 1300, 128: 900, 256: 560, 72: 700}[D]
    run_prompt([n, 129], [n, 300], hq, hkv, D, True, seed=200 + D)


def test_prompt_rows_without_keys():
    """Causal with fewer keys than rows: the first rows see nothing and are 0."""
    got, _ = run_prompt([100, 70], [40, 1], 4, 2, 64, True, seed=301)
    assert not got[:60].any() and not got[100:169].any() and got[169].any()
    got, _ = run_prompt([5], [0], 4, 2, 64, False, pad=(0, 4), seed=302)
    assert not got.any()


def test_prompt_single_tokens_and_many_sequences():
    run_prompt([1] * 150, list(range(150)), 4, 1, 64, True, seed=303)


def test_prompt_reads_column_blocks_of_one_matrix():
    run_prompt([50, 31], [50, 31], 8, 1, 256, False, seed=304, same_cu=True, merged=True)
    run_prompt([130], [130], 6, 2, 72, True, seed=305, same_cu=True, merged=True)


@pytest.mark.parametrize("hq,hkv,D,n", [(4, 2, 64, 150), (8, 1, 256, 90), (40, 8, 128, 900)])
def test_prompt_unseen_values_have_no_part(hq, hkv, D, n):
    """Infinities and NaN in keys and values a row does not see leave it as it
    is: in later positions, in other sequences and behind the last one."""
    def poison(q, k, v):
        for x in (k, v):
            x[n // 2, :, 1::3] = 0x7FC0          # NaN
            x[n // 2 + 1] = 0x7F80               # +inf
            x[n - 1, :, ::2] = 0xFF80            # -inf
            x[n + 20:] = 0x7FC0                  # behind the sequences
        q[n + 20:] = 0x7FC0
    clean, (q, k, v) = run_prompt([n, 20], [n, 20], hq, hkv, D, True, seed=310 + D, pad=(4, 4))
    got, _ = run_prompt([n, 20], [n, 20], hq, hkv, D, True, seed=310 + D, pad=(4, 4), poison=poison, check=False)
    assert np.isfinite(bf16_f64(got[:n // 2])).all()
    for x, y in ((got[:n // 2], clean[:n // 2]), (got[n:n + 20], clean[n:n + 20])):
        a, b = bf16_f64(x), bf16_f64(y)
        assert np.abs(a - b).max() <= 2 * EPS * np.abs(b).max()
    lim = np.arange(n // 2) + 1
    assert_attention(got[:n // 2], q[:n // 2], k[:n // 2], v[:n // 2], lim, float(np.float32(1 / math.sqrt(D))))
    assert np.isnan(bf16_f64(got[n // 2])).all()                  # the row that sees the NaN key


def test_prompt_seen_infinities():
    """A visible infinite value reaches the rows that see it, and only its channel."""
    def poison(q, k, v):
        v[70, 0, 5] = 0x7F80
    got, (q, k, v) = run_prompt([100], [100], 2, 1, 64, True, seed=330, poison=poison, check=False)
    g = bf16_f64(got)
    assert np.isposinf(g[70:, :, 5]).all() and np.isfinite(g[:70]).all()
    assert np.isfinite(np.delete(g[70:], 5, axis=2)).all()
    v = v.copy()
    v[70, 0, 5] = 0
    ref, tol = attention_bound(q, k, v, np.arange(100) + 1, 0.125)
    keep = np.ones(64, bool)
    keep[5] = False
    assert (np.abs(g - ref)[..., keep] <= tol[..., keep]).all()


def test_prompt_large_scores():
    """Scores of hundreds: the running maximum keeps every weight in range."""
    run_prompt([200], [200], 4, 2, 64, True, scale=4.0, seed=340)
    run_prompt([64], [300], 4, 4, 128, False, scale=1e-30, seed=341)


def test_prompt_offsets_are_bounded():
    """Offsets outside the tensors are cut to them."""
    q, k, v = rand(350, 64, 2, 64), rand(351, 64, 2, 64), rand(352, 64, 2, 64)
    o = Guarded(64 * 2 * 64 * 2, fill=0)
    cu = dev(np.array([-5, 30, 1 << 30], np.int32))
    vla.vla_attn_prompt(dev(q), dev(k), dev(v), cu, None, o.t, 2, 64, 64, 2, 2, 64, 128, 128, 128, 128, False, 0.125)
    o.check()
    got = o.numpy(np.uint16).reshape(64, 2, 64)
    for a, e in ((0, 30), (30, 64)):
        assert_attention(got[a:e], q[a:e], k[a:e], v[a:e], np.full(e - a, e - a), 0.125)


@pytest.mark.parametrize("hq,hkv,D,n,causal", [
    (32, 8, 64, 1300, False), (40, 8, 128, 900, False), (48, 4, 72, 700, False), (64, 4, 256, 560, False),
    (64, 8, 64, 1150, True), (64, 8, 128, 1100, True), (64, 4, 256, 200, False), (64, 4, 256, 300, True)])
def test_prompt_tile_heights(hq, hkv, D, n, causal):
    """Both tile heights above the smallest, with and without a causal mask,
    ending inside a tile and behind keys of an earlier chunk."""
    run_prompt([n, 75], [n, 203], hq, hkv, D, causal, seed=210 + D + n)


@pytest.mark.parametrize("hq,hkv,D,n", [(64, 8, 64, 1150), (64, 8, 128, 1100), (64, 4, 256, 560), (64, 4, 200, 300)])
def test_prompt_unseen_values_in_tall_tiles(hq, hkv, D, n):
    """NaN in one late key and value stays out of every row before it."""
    at = n - 40
    def poison(q, k, v):
        k[at, :, 3] = v[at, :, 5] = 0x7FC0
        v[at - 90, :, 0] = 0x7F80
    got, (q, k, v) = run_prompt([n], [n], hq, hkv, D, True, seed=330 + D, poison=poison, check=False)
    lim = np.arange(at - 90) + 1
    assert_attention(got[:at - 90], q[:at - 90], k[:at - 90], v[:at - 90], lim, float(np.float32(1 / math.sqrt(D))))
    f = bf16_f64(got)
    assert np.isfinite(f[:at, :, 1:]).all() and np.isnan(f[at:]).all()


@pytest.mark.parametrize("B", [2, 63, 64, 65, 130])
@pytest.mark.parametrize("causal", [False, True])
def test_prompt_batches(B, causal):
    """Every tile of every sequence is found once, with sequences of no rows
    or no keys among them, more rows than keys and more keys than rows."""
    r = synthetic.rng(9300 + B)
    nq, nk = r.integers(0, 70, B), r.integers(0, 300, B)
    nq[::7] = 0
    nk[3::11] = 0
    nq[1] = 333
    run_prompt([int(x) for x in nq], [int(x) for x in nk], 6, 2, 64, causal, pad=(2, 2), seed=340 + B)


# --------------------------------------------------------- shared prefix

class Cache:
    """A paged cache with its pages in random order and NaN in every row no
    sequence uses."""

    def __init__(self, B, hkv, D, page, prefix, lens, pages_per_seq=None, n_prefix_pages=None, seed=0, spare=3):
        self.page, self.prefix, self.lens = page, prefix, list(lens)
        self.npp = -(-prefix // page) if n_prefix_pages is None else n_prefix_pages
        self.pps = max([-(-n // page) for n in lens] + [0]) if pages_per_seq is None else pages_per_seq
        self.pages = self.npp + B * self.pps + spare
        order = synthetic.rng(9200 + seed).permutation(self.pages).astype(np.int32)
        self.prefix_pages = order[:self.npp]
        self.table = order[self.npp:self.npp + B * self.pps].reshape(B, self.pps)
        self.k = np.full((self.pages * page, hkv, D), 0x7FC0, np.uint16)
        self.v = np.full((self.pages * page, hkv, D), 0xFFC0, np.uint16)
        self.keys = []
        pre = self.slots(self.prefix_pages, prefix)
        self.k[pre], self.v[pre] = rand(seed + 1, prefix, hkv, D), rand(seed + 2, prefix, hkv, D)
        for b in range(B):
            s = self.slots(self.table[b], self.lens[b])
            self.k[s], self.v[s] = rand(seed + 10 + b, len(s), hkv, D), rand(seed + 510 + b, len(s), hkv, D)
            self.keys.append(np.concatenate([pre, s]))

    def slots(self, pages, n):
        j = np.arange(n)
        return pages[j // self.page].astype(np.int64) * self.page + j % self.page if n else np.zeros(0, np.int64)


def run_shared(B, L, hq, hkv, D, page, prefix, lens, causal, seed=0, check=True, lens_given=None, q_extra=0, ws=None, **kw):
    c = Cache(B, hkv, D, page, prefix, lens, seed=seed, **kw)
    scale = 1.0 / math.sqrt(D)
    q = rand(seed, B * L, hq, D, scale=2.0)
    qs = hq * D + 8 * q_extra
    qrows = np.zeros((B * L, qs), np.uint16)
    qrows[:, :hq * D] = q.reshape(B * L, -1)
    n = vla.vla_attn_shared_prefix_workspace_bytes(B, L, hq, hkv, D, c.npp * page, c.pps * page)
    w = Guarded(n, fill=0) if ws is None else ws
    o = Guarded(B * L * hq * D * 2, fill=0x5A)
    def call():
        vla.vla_attn_shared_prefix(
            dev(qrows), dev(c.k), dev(c.v), dev(c.prefix_pages) if c.npp else None,
            dev(np.array([prefix], np.int32)) if c.npp else None, dev(c.table) if c.pps else None,
            dev(np.array(lens if lens_given is None else lens_given, np.int32)) if c.pps else None, o.t, w.t, n,
            B, L, hq, hkv, D, c.pages, page, c.npp, c.pps, qs, hq * D, causal, scale)
        o.check()
        w.check()
        return o.numpy(np.uint16).reshape(B, L, hq, D).copy()
    got = call()
    if check:
        for b in range(B):
            lim = np.full(L, prefix + lens[b], np.int64)
            if causal:
                lim = prefix + np.clip(np.arange(L) + 1 + lens[b] - L, 0, lens[b])
            s = c.keys[b]
            assert_attention(got[b], q.reshape(B, L, hq, D)[b], c.k[s], c.v[s], lim, float(np.float32(scale)), f"sequence {b}")
    assert np.array_equal(call(), got)                            # the workspace is left ready, results repeat
    return got, q.reshape(B, L, hq, D), c


@pytest.mark.parametrize("hq,hkv,D", HEADS)
@pytest.mark.parametrize("B,L,page,prefix,lens,causal", [
    (1, 1, 16, 0, [1], True), (1, 1, 8, 0, [777], True), (1, 10, 16, 768, [10], False), (2, 1, 1, 5, [3, 0], True),
    (3, 7, 32, 0, [7, 200, 64], True), (5, 1, 64, 1000, [1, 65, 128, 0, 300], False)])
def test_shared_matches_oracle(hq, hkv, D, B, L, page, prefix, lens, causal):
    run_shared(B, L, hq, hkv, D, page, prefix, lens, causal, seed=400 + D + L)


@pytest.mark.parametrize("hq,hkv,D", [(8, 1, 256), (8, 2, 128), (6, 1, 64), (12, 2, 72)])
def test_shared_many_rows(hq, hkv, D):
    """128-row tiles for the prefix, for the suffix, and for both."""
    run_shared(20, 1, hq, hkv, D, 16, 333, [1 + 13 * b for b in range(20)], True, seed=500 + D)
    run_shared(3, 50, hq, hkv, D, 16, 200, [50, 170, 64], True, seed=520 + D)
    run_shared(1, 50, hq, hkv, D, 16, 100, [90], False, seed=540 + D)
    run_shared(2, 3, hq, hkv, D, 16, 70, [3, 9], True, seed=560 + D)


def test_shared_workspace_needs_no_clearing():
    """What the workspace held before has no part in the result, not even in rows without keys."""
    for causal, lens in ((True, [0, 600, 3]), (False, [1, 40, 0])):
        n = vla.vla_attn_shared_prefix_workspace_bytes(3, 2, 8, 2, 128, 304, 608)
        kw = dict(pages_per_seq=38, n_prefix_pages=19, seed=615)
        clean, _, _ = run_shared(3, 2, 8, 2, 128, 16, 300, lens, causal, ws=Guarded(n, fill=0), **kw)
        dirty, _, _ = run_shared(3, 2, 8, 2, 128, 16, 300, lens, causal, ws=Guarded(n, fill=0xFF), **kw)
        assert np.array_equal(clean, dirty)
    n = vla.vla_attn_shared_prefix_workspace_bytes(2, 1, 4, 2, 64, 0, 640)
    got, _, _ = run_shared(2, 1, 4, 2, 64, 16, 0, [0, 640], True, pages_per_seq=40, seed=618, ws=Guarded(n, fill=0xFF))
    assert not got[0].any()


def test_shared_edges():
    # no key at all, rows before the first suffix key, lengths past the capacity, capacity past the lengths
    got, _, _ = run_shared(2, 2, 4, 2, 64, 16, 0, [0, 40], True, pages_per_seq=3, seed=601)
    assert not got[0].any()
    got, _, _ = run_shared(2, 5, 4, 2, 64, 16, 0, [3, 5], True, seed=602)
    assert not got[0, :2].any() and got[0, 2:].any()
    run_shared(3, 1, 4, 2, 64, 16, 100, [2, 9, 1], True, pages_per_seq=40, n_prefix_pages=300, seed=603)
    run_shared(2, 1, 4, 2, 64, 16, 48, [32, 32], False, lens_given=[1 << 30, 33], seed=604)
    run_shared(3, 1, 4, 2, 64, 16, 320, [0, 0, 0], False, pages_per_seq=0, seed=605)       # prefix alone
    run_shared(1, 2, 4, 2, 64, 16, 320, [0], False, pages_per_seq=0, seed=606)
    run_shared(2, 1, 4, 2, 64, 16, 0, [5, 6], False, n_prefix_pages=4, seed=607)           # an empty prefix
    run_shared(2, 2, 4, 2, 64, 16, 20, [5, 6], False, q_extra=5, seed=608)
    got, _, _ = run_shared(2, 1, 4, 2, 64, 16, 0, [5, 6], False, lens_given=[-3, 6], check=False, seed=609)
    assert not got[0].any() and got[1].any()


def test_shared_missing_pages_hold_no_keys():
    B, L, hq, hkv, D, page, prefix, lens = 2, 3, 4, 2, 64, 16, 100, [50, 90]
    for merged in (False, True):
        b0 = 1 if merged else 2
        c = Cache(b0, hkv, D, page, prefix, lens[:b0], seed=620)
        q = rand(621, b0 * L, hq, D)
        keys = []
        gone = {0: [2], 1: [0, 5]}
        pp = c.prefix_pages.copy()
        pp[3] = -1
        pp[6] = c.pages                                            # the last, partly filled page
        table = c.table.copy()
        for b in range(b0):
            table[b, gone[b]] = [1 << 30, -(1 << 31)][:len(gone[b])]
            j, i = np.arange(prefix), np.arange(lens[b])
            keep = np.concatenate([(j // page != 3) & (j // page != 6), ~np.isin(i // page, gone[b])])
            keys.append(c.keys[b][keep])
        n = vla.vla_attn_shared_prefix_workspace_bytes(b0, L, hq, hkv, D, c.npp * page, c.pps * page)
        o, w = Guarded(b0 * L * hq * D * 2), zeros_ws(n)
        vla.vla_attn_shared_prefix(dev(q), dev(c.k), dev(c.v), dev(pp), dev(np.array([prefix], np.int32)), dev(table),
                                   dev(np.array(lens[:b0], np.int32)), o.t, w, n, b0, L, hq, hkv, D, c.pages, page, c.npp,
                                   c.pps, hq * D, hq * D, False, 0.125)
        o.check()
        got = o.numpy(np.uint16).reshape(b0, L, hq, D)
        for b in range(b0):
            assert_attention(got[b], q.reshape(b0, L, hq, D)[b], c.k[keys[b]], c.v[keys[b]], np.full(L, len(keys[b])), 0.125)


def test_shared_unseen_values_have_no_part():
    """Causal rows of one sequence: the last row's NaN key and value stay its own."""
    B, L, hq, hkv, D = 2, 4, 4, 2, 128
    for prefix in (0, 40):
        c = Cache(B, hkv, D, 16, prefix, [20, 30], seed=640)
        q = rand(641, B * L, hq, D)
        for b in range(B):
            c.k[c.keys[b][-1]] = c.v[c.keys[b][-1]] = 0x7FC0
        n = vla.vla_attn_shared_prefix_workspace_bytes(B, L, hq, hkv, D, c.npp * 16, c.pps * 16)
        o, w = Guarded(B * L * hq * D * 2), zeros_ws(n)
        vla.vla_attn_shared_prefix(dev(q), dev(c.k), dev(c.v), dev(c.prefix_pages) if prefix else None,
                                   dev(np.array([prefix], np.int32)) if prefix else None, dev(c.table),
                                   dev(np.array([20, 30], np.int32)), o.t, w, n, B, L, hq, hkv, D, c.pages, 16, c.npp,
                                   c.pps, hq * D, hq * D, True, 0.1)
        got = o.numpy(np.uint16).reshape(B, L, hq, D)
        for b in range(B):
            s, total = c.keys[b], len(c.keys[b])
            lim = np.arange(L - 1) + 1 + total - L
            assert_attention(got[b, :L - 1], q.reshape(B, L, hq, D)[b, :L - 1], c.k[s[:-1]], c.v[s[:-1]], lim, float(np.float32(0.1)))
            assert np.isnan(bf16_f64(got[b, L - 1])).all()


def test_shared_cache_past_4_gib():
    """Keys in pages whose byte offsets need more than 32 bits."""
    hq, hkv, D, page, n = 4, 2, 64, 16, 100
    rows = (5 << 30) // (hkv * D * 2)
    pages = rows // page
    k = torch.zeros(pages * page, hkv, D, dtype=torch.int16, device="cuda")
    v = torch.zeros_like(k)
    table = np.array([[pages - 1, 3, pages // 2 + 7, pages - 2, 0, pages // 4 * 3, 1]], np.int32)
    j = np.arange(n)
    slots = table[0][j // page].astype(np.int64) * page + j % page
    kb, vb, q = rand(650, n, hkv, D), rand(651, n, hkv, D), rand(652, 1, hq, D)
    freq = freqs(D)
    # appended through the cache's own operator at position 0: unrotated
    kd, vd = dev(kb), dev(vb)
    junk = torch.empty(n * hkv * D, dtype=torch.int16, device="cuda")
    vla.vla_qk_norm_rope_append(kd, kd, vd, None, None, dev(freq), dev(np.zeros(n, np.int32)), dev(slots), junk, None, k, v,
                                n, hkv, hkv, D, D, hkv * D, hkv * D, hkv * D, hkv * D, 0, pages * page, 0, 1.0, 0.0)
    s = torch.from_numpy(slots).cuda()
    assert np.array_equal(host(k[s], np.uint16), kb) and np.array_equal(host(v[s], np.uint16), vb)
    nb = vla.vla_attn_shared_prefix_workspace_bytes(1, 1, hq, hkv, D, 0, 7 * page)
    o, w = Guarded(hq * D * 2), zeros_ws(nb)
    vla.vla_attn_shared_prefix(dev(q), k, v, None, None, dev(table), dev(np.array([n], np.int32)), o.t, w, nb, 1, 1, hq, hkv,
                               D, pages, page, 0, 7, hq * D, hq * D, True, 0.125)
    o.check()
    assert_attention(o.numpy(np.uint16).reshape(1, hq, D), q, kb, vb, [n], 0.125)


@pytest.mark.parametrize("hq,hkv,D", [(4, 2, 128), (8, 1, 256), (2, 2, 64)])
@pytest.mark.parametrize("rows", [1, 300])
def test_shared_cache_past_4_gib_in_every_tile(hq, hkv, D, rows):
    """A prefix and suffixes spread over a cache of 5 GiB, for few rows and for tall tiles."""
    page, L = 16, rows
    pages = (5 << 30) // (hkv * D * 2) // page
    k = torch.zeros(pages * page, hkv, D, dtype=torch.int16, device="cuda")
    v = torch.zeros_like(k)
    pre = np.array([pages - 1, 5, pages // 2 + 1, pages // 4 * 3], np.int32)
    table = np.array([[pages - 3, 7, pages // 5 * 4], [2, pages - 9, pages // 3 * 2]], np.int32)
    lens, n_pre = [33, 48], 60
    def slots(p, n):
        return p[np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page
    keys = []
    for b in range(2):
        at = np.concatenate([slots(pre, n_pre), slots(table[b], lens[b])])
        keys.append((at, rand(660 + b, len(at), hkv, D), rand(662 + b, len(at), hkv, D)))
        if b:
            for x in (1, 2):
                keys[1][x][:n_pre] = keys[0][x][:n_pre]
        t = torch.from_numpy(at).cuda()
        k[t], v[t] = torch.from_numpy(keys[b][1].view(np.int16)).cuda(), torch.from_numpy(keys[b][2].view(np.int16)).cuda()
    q = rand(664, 2 * L, hq, D, scale=2.0)
    n = vla.vla_attn_shared_prefix_workspace_bytes(2, L, hq, hkv, D, 4 * page, 3 * page)
    o, w = Guarded(2 * L * hq * D * 2), zeros_ws(n)
    vla.vla_attn_shared_prefix(dev(q), k, v, dev(pre), dev(np.array([n_pre], np.int32)), dev(table),
                               dev(np.array(lens, np.int32)), o.t, w, n, 2, L, hq, hkv, D, pages, page, 4, 3, hq * D, hq * D,
                               False, 0.1)
    o.check()
    got = o.numpy(np.uint16).reshape(2, L, hq, D)
    for b in range(2):
        assert_attention(got[b], q.reshape(2, L, hq, D)[b], keys[b][1], keys[b][2], np.full(L, len(keys[b][0])), float(np.float32(0.1)))


@pytest.mark.parametrize("hq,hkv,D", [(8, 1, 256), (8, 1, 64), (16, 2, 128), (24, 3, 72)])
def test_shared_tall_prefix_tiles(hq, hkv, D):
    """Tall tiles for the prefix beside short ones for the suffixes, and the
    prefix ahead of every sequence's own keys."""
    run_shared(41, 1, hq, hkv, D, 16, 333, [1 + 3 * b for b in range(41)], True, seed=580 + D)
    run_shared(41, 1, hq, hkv, D, 16, 50, [0] * 41, False, pages_per_seq=0, seed=590 + D)
    run_shared(3, 40, hq, hkv, D, 16, 150, [40, 77, 0], True, seed=595 + D)


@pytest.mark.parametrize("hq,hkv,D,B,L", [(8, 1, 256, 20, 64), (8, 1, 256, 40, 64), (16, 4, 128, 20, 64), (32, 8, 128, 20, 64),
                                         (16, 4, 64, 20, 65), (32, 8, 72, 20, 65)])
def test_shared_tall_suffix_tiles(hq, hkv, D, B, L):
    """64-row and 128-row tiles for every sequence's rows, the prefix ahead of their own keys."""
    run_shared(B, L, hq, hkv, D, 16, 70, [(L + 3 * b) if b else 0 for b in range(B)], True, seed=700 + D + B)


def test_shared_long_chunk():
    """A chunk of a prompt over the cache: many rows of few sequences, one of them without keys of its own."""
    run_shared(2, 600, 32, 8, 72, 16, 45, [0, 650], True, seed=790)


@pytest.mark.parametrize("hq,hkv,D,B,prefix", [(8, 1, 256, 20, 70), (8, 1, 256, 40, 0), (32, 8, 128, 20, 70), (16, 4, 64, 20, 33)])
def test_shared_unseen_values_in_tall_tiles(hq, hkv, D, B, prefix):
    """NaN in the second to last key and value of every sequence is seen by its last two rows alone."""
    L, lens = 64, [64 + 5 * b for b in range(B)]
    c = Cache(B, hkv, D, 16, prefix, lens, seed=650 + D)
    q = rand(651, B * L, hq, D)
    for b in range(B):
        c.k[c.keys[b][-2]] = c.v[c.keys[b][-2]] = 0x7FC0
    n = vla.vla_attn_shared_prefix_workspace_bytes(B, L, hq, hkv, D, c.npp * 16, c.pps * 16)
    o, w = Guarded(B * L * hq * D * 2), zeros_ws(n)
    vla.vla_attn_shared_prefix(dev(q), dev(c.k), dev(c.v), dev(c.prefix_pages) if prefix else None,
                               dev(np.array([prefix], np.int32)) if prefix else None, dev(c.table),
                               dev(np.array(lens, np.int32)), o.t, w, n, B, L, hq, hkv, D, c.pages, 16, c.npp,
                               c.pps, hq * D, hq * D, True, 0.1)
    o.check()
    got = o.numpy(np.uint16).reshape(B, L, hq, D)
    for b in range(B):
        s, total = c.keys[b], len(c.keys[b])
        lim = np.arange(L - 2) + 1 + total - L
        assert_attention(got[b, :L - 2], q.reshape(B, L, hq, D)[b, :L - 2], c.k[s[:-2]], c.v[s[:-2]], lim, float(np.float32(0.1)))
        assert np.isnan(bf16_f64(got[b, L - 2:])).all()


@pytest.mark.parametrize("hq,hkv,D,B", [(64, 8, 64, 600), (64, 8, 128, 300), (8, 1, 256, 1100), (8, 1, 256, 2100)])
def test_shared_many_single_tokens(hq, hkv, D, B):
    """64-row and 128-row tiles for the prefix, 32-row tiles for the suffixes."""
    run_shared(B, 1, hq, hkv, D, 16, 75, [b % 4 for b in range(B)], True, seed=720 + D + B)


# ------------------------------------------------------- graphs, streams

def capture(call):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call(s)
    return g


def test_captured_calls_follow_device_values():
    """One graph of an append and both attentions, replayed with new lengths,
    slots and inputs between eager calls; two graphs share one workspace."""
    hq, hkv, D, page, L, B = 8, 2, 64, 16, 2, 3
    prefix_cap, pps = 64, 4
    pages = prefix_cap // page + B * pps
    pp, table = dev(np.arange(4, dtype=np.int32)), dev(np.arange(4, pages, dtype=np.int32).reshape(B, pps))
    kc = torch.zeros(pages * page * hkv * D, dtype=torch.int16, device="cuda")
    vc = torch.zeros_like(kc)
    T, width = B * L, (hq + 2 * hkv) * D
    qkv = torch.zeros(T, width, dtype=torch.int16, device="cuda")
    plen, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    pos, slots = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int64, device="cuda")
    freq, cu = dev(freqs(D)), dev(np.array([0, 2, 4, 6], np.int32))
    n = vla.vla_attn_shared_prefix_workspace_bytes(B, L, hq, hkv, D, prefix_cap, pps * page)
    ws = zeros_ws(n)
    outs = [torch.zeros(T * hq * D, dtype=torch.int16, device="cuda") for _ in range(2)]
    ko = torch.zeros(T * hkv * D, dtype=torch.int16, device="cuda")
    qo = torch.zeros(T * hq * D, dtype=torch.int16, device="cuda")

    def call(s=None, which=(0, 1)):
        vla.vla_qk_norm_rope_append(qkv, qkv[:, hq * D:], qkv[:, (hq + hkv) * D:], None, None, freq, pos, slots, qo, ko, kc, vc,
                                    T, hq, hkv, D, D, width, width, width, hq * D, hkv * D, pages * page, 0, 1.0, 0.0, stream=s)
        if 0 in which:
            vla.vla_attn_shared_prefix(qo, kc, vc, pp, plen, table, lens, outs[0], ws, n, B, L, hq, hkv, D, pages, page, 4, pps,
                                       hq * D, hq * D, True, 0.125, stream=s)
        if 1 in which:
            vla.vla_attn_prompt(qo, ko, qkv[:, (hq + hkv) * D:], cu, None, outs[1], B, T, T, hq, hkv, D, hq * D, hkv * D,
                                width, hq * D, True, 0.125, stream=s)

    def set_step(i):
        kc.copy_(dev(rand(700 + i, pages * page * hkv * D)))
        vc.copy_(dev(rand(710 + i, pages * page * hkv * D)))
        qkv.copy_(dev(rand(720 + i, T, width)))
        ln = np.array([2 + i, 10 + 17 * i, 30], np.int32)
        lens.copy_(dev(ln))
        plen.fill_(13 * i + 1)
        tab = np.arange(4, pages).reshape(B, pps)
        at = np.array([[ln[b] - L + r for r in range(L)] for b in range(B)])
        slots.copy_(dev(np.array([tab[b][at[b, r] // page] * page + at[b, r] % page for b in range(B) for r in range(L)], np.int64)))
        pos.copy_(dev(at.reshape(-1).astype(np.int32)))
        torch.cuda.synchronize()

    set_step(0)
    g1, g2 = capture(call), capture(lambda s: call(s, which=(0,)))
    for i in (1, 2, 0, 3):
        set_step(i)
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs + [kc, vc, qo, ko]]
        assert all(bool(t.any()) for t in want)
        for g in (g1, g2, g1):
            for t in outs + [qo, ko]:
                t.zero_() if g is g1 or t is not outs[1] else None
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for t, x in zip(outs + [kc, vc, qo, ko], want):
                assert torch.equal(t, x)


def test_another_stream_and_repeats():
    q, k, v = rand(800, 300, 8, 128), rand(801, 300, 2, 128), rand(802, 300, 2, 128)
    d = [dev(x) for x in (q, k, v, offsets([300]))]
    outs = [torch.zeros(300 * 8 * 128, dtype=torch.int16, device="cuda") for _ in range(4)]
    streams = [torch.cuda.Stream() for _ in range(3)] + [torch.cuda.current_stream()]
    torch.cuda.synchronize()
    for s, o in zip(streams, outs):
        vla.vla_attn_prompt(*d, None, o, 1, 300, 300, 8, 2, 128, 1024, 256, 256, 1024, True, 0.1, stream=s)
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


# ----------------------------------------------------------- used together

def test_layer_from_qkv_gemm_to_attention():
    """A prompt and then two decoding steps of one layer: QKV GEMM with FP8
    weights, append, attention, each checked on its own inputs, and the
    decoded rows against attention over the whole sequence."""
    H, hq, hkv, D, page, B = 256, 8, 2, 64, 16, 3
    width = (hq + 2 * hkv) * D
    W = synthetic.weights(width, H, 850)
    Wq = torch.empty(width * H, dtype=torch.uint8, device="cuda")
    sw = torch.empty(width, dtype=torch.float32, device="cuda")
    vla.vla_quantize_pack(dev(W), Wq, sw, width, H, vla.VLA_WFMT_E4M3_OCP, vla.VLA_LAYOUT_MFMA)
    ws = zeros_ws(vla.vla_gemm_workspace_bytes(64, width, H, vla.VLA_WFMT_E4M3_OCP))
    qw, kw, freq = rand(851, D), rand(852, D), freqs(D)
    lens = [33, 5, 16]
    pps = 4
    pages = B * pps
    table = synthetic.rng(853).permutation(pages).astype(np.int32).reshape(B, pps)
    kc = torch.zeros(pages * page, hkv, D, dtype=torch.int16, device="cuda")
    vc = torch.zeros_like(kc)
    n = vla.vla_attn_shared_prefix_workspace_bytes(B, 1, hq, hkv, D, 0, pps * page)
    aws = zeros_ws(n)
    seen_k, seen_v = [[] for _ in range(B)], [[] for _ in range(B)]

    def project_and_append(x, where):
        T = len(where)
        qkv = torch.empty(T, width, dtype=torch.int16, device="cuda")
        vla.vla_gemm_fp8w(dev(x), None, Wq, sw, None, None, qkv, ws, ws.numel(), T, width, H)
        raw = host(qkv, np.uint16).reshape(T, -1)
        slots = np.array([table[b][j // page] * page + j % page for b, j in where], np.int64)
        pos = np.array([j for _, j in where], np.int32)
        vla.vla_qk_norm_rope_append(qkv, qkv[:, hq * D:], qkv[:, (hq + hkv) * D:], dev(qw), dev(kw), dev(freq), dev(pos),
                                    dev(slots), qkv, qkv[:, hq * D:], kc, vc, T, hq, hkv, D, D, width, width, width, width, width,
                                    pages * page, vla.VLA_ROPE_HALF, 1.0, 1e-6)
        now = host(qkv, np.uint16).reshape(T, -1)
        check_rotated(now[:, :hq * D].reshape(T, hq, D), raw[:, :hq * D].reshape(T, hq, D), qw, freq, pos, D, False, 1.0, 1e-6, "q")
        check_rotated(now[:, hq * D:(hq + hkv) * D].reshape(T, hkv, D), raw[:, hq * D:(hq + hkv) * D].reshape(T, hkv, D), kw,
                      freq, pos, D, False, 1.0, 1e-6, "k")
        for t, (b, _) in enumerate(where):
            seen_k[b].append(now[t, hq * D:(hq + hkv) * D].reshape(hkv, D))
            seen_v[b].append(raw[t, (hq + hkv) * D:].reshape(hkv, D))
        return qkv, now[:, :hq * D].reshape(T, hq, D)

    where = [(b, j) for b in range(B) for j in range(lens[b])]
    qkv, q = project_and_append(synthetic.activations(len(where), H, 854), where)
    out = torch.empty(len(where), hq * D, dtype=torch.int16, device="cuda")
    cu = offsets(lens)
    vla.vla_attn_prompt(qkv, qkv[:, hq * D:], qkv[:, (hq + hkv) * D:], dev(cu), None, out, B, len(where), len(where), hq, hkv, D,
                        width, width, width, hq * D, True, 0.125)
    got = out_bits(out, len(where), hq, D)
    for b in range(B):
        assert_attention(got[cu[b]:cu[b + 1]], q[cu[b]:cu[b + 1]], np.array(seen_k[b]), np.array(seen_v[b]),
                         np.arange(lens[b]) + 1, 0.125, "prompt")
    for step in range(2):
        where = [(b, lens[b]) for b in range(B)]
        qkv, q = project_and_append(synthetic.activations(B, H, 860 + step), where)
        lens = [x + 1 for x in lens]
        out = torch.empty(B, hq * D, dtype=torch.int16, device="cuda")
        vla.vla_attn_shared_prefix(qkv, kc, vc, None, None, dev(table), dev(np.array(lens, np.int32)), out, aws, n, B, 1, hq, hkv,
                                   D, pages, page, 0, pps, width, hq * D, True, 0.125)
        got = out_bits(out, B, hq, D)
        for b in range(B):
            assert_attention(got[b:b + 1], q[b:b + 1], np.array(seen_k[b]), np.array(seen_v[b]), [lens[b]], 0.125, f"step {step}")


# ------------------------------------------- infinities and NaN among the keys

KINDS = (0x7FC0, 0x7F80, 0xFF80)          # NaN, +inf, -inf


def poison_values(v, at):
    """Value row at[j] is not finite in channel j; returns the clean copy."""
    clean = v.copy()
    assert len(set(int(x) for x in at)) == len(at) <= v.shape[2]
    for j, key in enumerate(at):
        v[key, :, j] = KINDS[j % 3]
    return clean


def assert_poisoned(got, q, k, clean, limits, scale, at, what=""):
    """A row that sees key at[j] has that key's infinity or NaN in channel j;
    everything else is as if the values were finite."""
    limits = np.asarray(limits)
    ref, tol = attention_bound(q, k, clean, limits, scale)
    g = bf16_f64(got)
    seen = np.zeros((len(limits), 1, k.shape[2]), bool)
    for j, key in enumerate(at):
        seen[:, 0, j] = limits > key
        x = g[limits > key, :, j]
        assert (np.isnan(x) if j % 3 == 0 else x == (np.inf if j % 3 == 1 else -np.inf)).all(), f"{what}: seen key {key}"
    bad = ~(np.abs(g - ref) <= tol) & ~seen
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[0]}: {g[bad][0]} for {ref[bad][0]}"


def poisoned_prompt(n, m, hq, hkv, D, causal, at, every=1, behind=0, seed=0):
    """One sequence of n rows and m keys, `behind` rows of NaN after its keys."""
    q, k, v = rand(seed, n, hq, D, scale=2.0), rand(seed + 1, m + behind, hkv, D), rand(seed + 2, m + behind, hkv, D)
    clean = poison_values(v, at)
    k[m:] = v[m:] = 0x7FC0
    scale = float(np.float32(1 / math.sqrt(D)))
    o = Guarded(n * hq * D * 2, fill=0x5A)
    vla.vla_attn_prompt(dev(q), dev(k), dev(v), dev(offsets([n])), dev(offsets([m])), o.t, 1, n, m + behind, hq, hkv, D, hq * D,
                        hkv * D, hkv * D, hq * D, causal, scale)
    o.check()
    lim = np.clip(np.arange(n) + 1 + m - n, 0, m) if causal else np.full(n, m)
    s = slice(None, None, every)
    assert_poisoned(o.numpy(np.uint16).reshape(n, hq, D)[s], q[s], k[:m], clean[:m], lim[s], scale, at)


def poisoned_shared(L, hq, hkv, D, prefix, lens, at, every=1, page=16, seed=0):
    """Causal rows over the cache; at counts a sequence's own keys, from its end if negative."""
    B = len(lens)
    c = Cache(B, hkv, D, page, prefix, lens, seed=seed)
    q = rand(seed + 5, B * L, hq, D, scale=2.0)
    clean, where = c.v.copy(), []
    for b in range(B):
        where.append([prefix + (a if a >= 0 else lens[b] + a) for a in at if -lens[b] <= a < lens[b]])
        for j, key in enumerate(where[b]):
            c.v[c.keys[b][key], :, j] = KINDS[j % 3]
    scale = float(np.float32(1 / math.sqrt(D)))
    n = vla.vla_attn_shared_prefix_workspace_bytes(B, L, hq, hkv, D, c.npp * page, c.pps * page)
    o, w = Guarded(B * L * hq * D * 2, fill=0x5A), zeros_ws(n)
    vla.vla_attn_shared_prefix(dev(q), dev(c.k), dev(c.v), dev(c.prefix_pages) if prefix else None,
                               dev(np.array([prefix], np.int32)) if prefix else None, dev(c.table),
                               dev(np.array(lens, np.int32)), o.t, w, n, B, L, hq, hkv, D, c.pages, page, c.npp, c.pps,
                               hq * D, hq * D, True, scale)
    o.check()
    got, q = o.numpy(np.uint16).reshape(B, L, hq, D), q.reshape(B, L, hq, D)
    s = slice(None, None, every)
    for b in range(B):
        lim = prefix + np.clip(np.arange(L) + 1 + lens[b] - L, 0, lens[b])
        assert_poisoned(got[b, s], q[b, s], c.k[c.keys[b]], clean[c.keys[b]], lim[s], scale, where[b], f"sequence {b}")


@pytest.mark.parametrize("hq,hkv,D,L,prefix", [
    (8, 8, 64, 1200, 0), (2, 2, 64, 1200, 0), (40, 40, 64, 1200, 0), (4, 4, 256, 1200, 0), (8, 8, 200, 1200, 30),
    (16, 2, 128, 1200, 0), (2, 2, 72, 2300, 0), (3, 3, 64, 1500, 37)])
def test_shared_values_far_past_a_row(hq, hkv, D, L, prefix):
    """NaN and infinities hundreds of keys after what a row sees, in every
    tile height, with the keys in one part and in several."""
    poisoned_shared(L, hq, hkv, D, prefix, [L], [100, 511, 700, 1000, 1100, -1], every=3, seed=670)


def test_shared_values_far_past_a_row_of_a_batch():
    poisoned_shared(1100, 4, 4, 64, 20, [1100, 1300, 0, 640], [5, 600, 1090, -3], every=5, seed=675)


@pytest.mark.parametrize("hq,hkv,D,n", [
    (32, 1, 128, 300), (32, 1, 128, 1000), (48, 1, 64, 800), (71, 1, 64, 500), (128, 1, 64, 600), (64, 1, 256, 150),
    (64, 1, 256, 300), (64, 1, 256, 560), (96, 2, 72, 700), (2048, 1, 8, 70)])
def test_prompt_unseen_values_beside_one_token_of_many_heads(hq, hkv, D, n):
    """A wave whose rows all belong to one token, in a tile that walks on for later tokens."""
    at = sorted({min(x, n - 1) for x in (0, 1, 17, 31, 32, n // 2, n - 34)})
    poisoned_prompt(n, n, hq, hkv, D, True, at, every=max(1, n * hq // 12000), seed=680)


@pytest.mark.parametrize("hq,hkv,D,n,m", [
    (4, 4, 64, 300, 100), (64, 64, 64, 600, 200), (64, 64, 64, 1300, 70), (40, 40, 128, 700, 1), (64, 64, 256, 300, 90),
    (32, 1, 64, 800, 40)])
def test_prompt_rows_without_keys_beside_unseen_values(hq, hkv, D, n, m):
    """Rows that see nothing are 0 in tiles whose later rows see infinities and NaN."""
    at = sorted({0, m // 2, m - 1})
    poisoned_prompt(n, m, hq, hkv, D, True, at, every=max(1, n * hq // 12000), seed=690)


@pytest.mark.parametrize("hq,hkv,D,L,prefix,lens", [
    (32, 1, 64, 2, 0, [64]), (32, 1, 128, 2, 0, [2]), (48, 1, 64, 7, 20, [7, 40, 300]), (71, 1, 64, 3, 50, [3, 90]),
    (32, 1, 256, 40, 0, [40, 3]), (64, 2, 128, 33, 16, [20, 60, 33]), (4, 4, 64, 200, 0, [50, 0, 230]),
    (64, 64, 64, 300, 10, [60, 300])])
def test_shared_unseen_values_beside_rows_of_one_limit(hq, hkv, D, L, prefix, lens):
    """Waves whose rows all see the same keys, or none, over the cache."""
    poisoned_shared(L, hq, hkv, D, prefix, lens, [0, 1, -1, -2], every=max(1, L * hq // 6000), seed=700)


@pytest.mark.parametrize("hq,hkv,D,n,m", [
    (2, 2, 64, 40, 1), (2, 2, 64, 40, 33), (8, 1, 128, 70, 97), (3, 1, 72, 10, 63), (8, 1, 256, 300, 129), (2, 1, 200, 9, 2),
    (64, 64, 64, 1300, 65), (40, 40, 128, 700, 45), (64, 64, 256, 300, 66)])
def test_prompt_nothing_is_read_behind_the_keys(hq, hkv, D, n, m):
    """All rows see all keys; the rows behind them in the tensors are NaN."""
    poisoned_prompt(n, m, hq, hkv, D, False, [], every=max(1, n * hq // 6000), behind=128, seed=710)


@pytest.mark.parametrize("B", [1, 3, 70])
@pytest.mark.parametrize("causal", [False, True])
def test_prompt_offsets_of_any_value(B, causal):
    """Offsets at the ends of 32 bits: every sequence is its rows and keys cut
    to the tensors, and only rows of a sequence are written."""
    total, low, high = 64, -(1 << 31), (1 << 31) - 1
    q, k, v = rand(730, total, 4, 64), rand(731, total, 2, 64), rand(732, total, 2, 64)
    some = {1: [10, low], 3: [low, 20, low, high], 70: [20, low] + [low, 5, high, low] * 17 + [low]}[B]
    for cu_q, cu_k in ((some, some), (some, [0] * (B + 1)), ([0] * B + [total], some)):
        o = Guarded(total * 4 * 64 * 2, fill=0x5A)
        vla.vla_attn_prompt(dev(q), dev(k), dev(v), dev(np.array(cu_q, np.int32)), dev(np.array(cu_k, np.int32)), o.t, B,
                            total, total, 4, 2, 64, 256, 128, 128, 256, causal, 0.125)
        o.check()
        written = np.zeros(total, bool)
        for b in range(B):
            a = min(max(cu_q[b], 0), total)
            written[a:max(min(cu_q[b + 1], total), a)] = True
        got = o.numpy(np.uint16).reshape(total, -1)
        assert (got[~written] == 0x5A5A).all() and np.isfinite(bf16_f64(got[written])).all()
        if not all(x <= y for x, y in zip(cu_q, cu_q[1:])):
            continue                                             # sequences that share rows have no one result
        s, e = (min(max(x, 0), total) for x in cu_k[-2:])
        e = max(e, s)
        lim = np.clip(np.arange(total) + 1 + (e - s) - total, 0, e - s) if causal else np.full(total, e - s)
        assert_attention(got.reshape(total, 4, 64), q, k[s:e], v[s:e], lim, 0.125)


@pytest.mark.parametrize("D", [8, 24, 64, 72, 80, 96, 120, 248])
def test_append_norm_of_the_largest_and_smallest_values(D):
    """Rows whose mean square leaves fp32: one value at bf16's largest beside
    small ones that a large weight brings back, and rows of the smallest."""
    rows = np.zeros((6, 2, D), np.uint16)
    rows[0, :, 0] = 0x7F7F                       # the largest bf16
    rows[1, :, D - 1] = 0xFF7F
    rows[2] = 0x7F7F
    rows[3, :, :] = 0x3580                       # 2^-20
    rows[3, :, 3] = 0x7F00                       # beside 2^127
    rows[4] = 0x0001                             # the smallest
    rows[5, :, 1] = 0x0001
    w = np.full(D, 0x3F80, np.uint16)
    for weight in (w, np.full(D, 0x7180, np.uint16)):            # 1, 2^100
        for rot in (0, 8):
            pos, freq = np.arange(6, dtype=np.int32), freqs(rot)
            go, gk = Guarded(rows.nbytes), Guarded(rows.nbytes)
            vla.vla_qk_norm_rope_append(dev(rows), dev(rows), None, dev(weight), dev(w), dev(freq) if rot else None,
                                        dev(pos) if rot else None, None, go.t, gk.t, None, None, 6, 2, 2, D, rot, 2 * D,
                                        2 * D, 0, 2 * D, 2 * D, 0, vla.VLA_ROPE_HALF, 1.0, 0.0)
            for g, x in ((go, weight), (gk, w)):
                g.check()
                check_rotated(g.numpy(np.uint16).reshape(6, 2, D), rows, x, freq, pos, rot, False, 1.0, 0.0, f"rot {rot}")


@pytest.mark.parametrize("hq,hkv,D,n", [(4, 1, 64, 3000), (8, 1, 256, 1500), (8, 2, 128, 40000)])
def test_shared_seen_values_of_weights_that_vanish(hq, hkv, D, n):
    """A visible NaN has its part in the result also where its key's weight, and
    that of every key in its part of the cache, is 0 in fp32."""
    c = Cache(1, hkv, D, 16, 0, [n], seed=720)
    q = np.full((1, hq, D), 0x3F80, np.uint16)                   # ones
    for lo, hi, x in ((0, n // 2, 0x4180), (n // 2, n, 0xC180)):  # scores +-16 D
        c.k[c.keys[0][lo:hi]] = x
    at = [n - 1, n // 2 + 40]
    for j, key in enumerate(at):
        c.v[c.keys[0][key], :, 3 * j] = 0x7FC0
    size = vla.vla_attn_shared_prefix_workspace_bytes(1, 1, hq, hkv, D, 0, c.pps * 16)
    assert size > 256                                            # the keys are split
    o, w = Guarded(hq * D * 2), zeros_ws(size)
    vla.vla_attn_shared_prefix(dev(q), dev(c.k), dev(c.v), None, None, dev(c.table), dev(np.array([n], np.int32)), o.t, w,
                               size, 1, 1, hq, hkv, D, c.pages, 16, 0, c.pps, hq * D, hq * D, True, 1.0)
    o.check()
    g = bf16_f64(o.numpy(np.uint16).reshape(hq, D))
    assert np.isnan(g[:, [0, 3]]).all() and np.isfinite(np.delete(g, [0, 3], axis=1)).all()


def test_scores_of_minus_infinity():
    """Keys of score -inf weigh nothing; rows that see no others are 0."""
    n, gone, hq, hkv, D = 100, 60, 4, 2, 64
    q, k, v = rand(740, n, hq, D), rand(741, n, hkv, D), rand(742, n, hkv, D)
    q[..., 0], k[:gone, :, 0] = 0x3F80, 0xFF80
    o = Guarded(n * hq * D * 2)
    vla.vla_attn_prompt(dev(q), dev(k), dev(v), dev(offsets([n])), None, o.t, 1, n, n, hq, hkv, D, hq * D, hkv * D, hkv * D,
                        hq * D, True, 0.125)
    o.check()
    got = o.numpy(np.uint16).reshape(n, hq, D)
    assert not (got[:gone] & 0x7FFF).any()
    assert_attention(got[gone:], q[gone:], k, v, np.arange(gone, n) + 1, 0.125)
    table = dev(np.arange(1000, dtype=np.int32))
    for m in (40, 1000):                                         # keys in one part and in several
        kc, vc = rand(743, m, hkv, D), rand(744, m, hkv, D)
        kc[:, :, 0] = 0xFF80
        for keep in (0, 3):
            kc[m - keep:, :, 0] = 0
            size = vla.vla_attn_shared_prefix_workspace_bytes(1, 1, hq, hkv, D, 0, m)
            o, w = Guarded(hq * D * 2, fill=0x5A), zeros_ws(size)
            vla.vla_attn_shared_prefix(dev(q[:1]), dev(kc), dev(vc), None, None, table, dev(np.array([m], np.int32)), o.t, w,
                                       size, 1, 1, hq, hkv, D, m, 1, 0, m, hq * D, hq * D, True, 0.125)
            o.check()
            got = o.numpy(np.uint16).reshape(1, hq, D)
            if keep:
                assert_attention(got, q[:1], kc, vc, [m], 0.125)
            else:
                assert not (got & 0x7FFF).any()


def test_calls_run_on_the_current_stream():
    """Without a stream a call takes torch's current one, also under capture."""
    from bf16_gemm_vla_amd._lib import _stream

    side = torch.cuda.Stream()
    assert _stream(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert _stream(None) == side.cuda_stream == torch.cuda.current_stream().cuda_stream
    q, k, v = (rand(750 + i, 70, n, 64) for i, n in enumerate((4, 2, 2)))
    d = [dev(x) for x in (q, k, v, offsets([70]))]
    out = torch.zeros(70 * 4 * 64, dtype=torch.int16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert _stream(None) == torch.cuda.current_stream().cuda_stream
        vla.vla_attn_prompt(*d, None, out, 1, 70, 70, 4, 2, 64, 256, 128, 128, 256, True, 0.125)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert_attention(out_bits(out, 70, 4, 64), q, k, v, np.arange(70) + 1, 0.125)


def test_outputs_with_gaps_between_rows():
    """Rows of out further apart than their heads: what lies between stays."""
    n, hq, hkv, D, gap = 75, 6, 2, 72, 24
    q, k, v = rand(760, n, hq, D), rand(761, n, hkv, D), rand(762, n, hkv, D)
    stride, d = hq * D + gap, [dev(x) for x in (q, k, v)]
    def check(o, limits):
        o.check()
        rows = np.append(o.numpy(np.uint16), np.full(gap, 0x5A5A, np.uint16)).reshape(n, stride)
        assert (rows[:, hq * D:] == 0x5A5A).all()
        assert_attention(rows[:, :hq * D].reshape(n, hq, D), q, k, v, limits, 0.125)
    o = Guarded((n * stride - gap) * 2, fill=0x5A)
    vla.vla_attn_prompt(*d, dev(offsets([n])), None, o.t, 1, n, n, hq, hkv, D, hq * D, hkv * D, hkv * D, stride, True, 0.125)
    check(o, np.arange(n) + 1)
    size = vla.vla_attn_shared_prefix_workspace_bytes(1, n, hq, hkv, D, 0, n)
    o, w = Guarded((n * stride - gap) * 2, fill=0x5A), zeros_ws(size)
    vla.vla_attn_shared_prefix(*d, None, None, dev(np.arange(n, dtype=np.int32)), dev(np.array([n], np.int32)), o.t, w, size, 1, n,
                               hq, hkv, D, n, 1, 0, n, hq * D, stride, False, 0.125)
    check(o, np.full(n, n))


@pytest.mark.parametrize("D", [8, 128])
def test_pages_named_more_than_once_and_large_pages(D):
    """Sequences that name the same pages, the prefix's among them, and pages of
    65536 rows, two calls at once on streams and workspaces of their own."""
    hq, hkv, page = 4, 2, 65536
    k, v = rand(770, 2 * page, hkv, D), rand(771, 2 * page, hkv, D)
    q = rand(772, 3, hq, D)
    dk, dv, dq = dev(k), dev(v), dev(q)
    pre, n_pre = dev(np.array([1], np.int32)), 70
    table, lens = np.array([[1, 0], [1, 0], [0, 0]], np.int32), [30, page + 5, 90]
    dt, dl, dn = dev(table), dev(np.array(lens, np.int32)), dev(np.array([n_pre], np.int32))
    size = vla.vla_attn_shared_prefix_workspace_bytes(3, 1, hq, hkv, D, page, 2 * page)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, ws = [Guarded(3 * hq * D * 2, fill=0x5A) for _ in streams], [zeros_ws(size) for _ in streams]
    torch.cuda.synchronize()
    for s, o, w in zip(streams, outs, ws):
        for _ in range(3):
            vla.vla_attn_shared_prefix(dq, dk, dv, pre, dn, dt, dl, o.t, w, size, 3, 1, hq, hkv, D, 2, page, 1, 2, hq * D, hq * D,
                                       True, 0.125, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        o.check()
        got = o.numpy(np.uint16).reshape(3, hq, D)
        for b in range(3):
            j = np.arange(lens[b])
            at = np.concatenate([page + np.arange(n_pre), table[b][j // page].astype(np.int64) * page + j % page])
            assert_attention(got[b:b + 1], q[b:b + 1], k[at], v[at], [len(at)], 0.125, f"sequence {b}")
