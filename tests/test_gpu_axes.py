"""GPU parity of the append with positions on several axes against its 64-bit
form.  Tolerance: that of the one-axis append (tests/test_gpu_attention.py) -
one bf16 rounding, and angle, sine, cosine, norm and products together below
2^-20 of |a| + |b| for the pair (a, b), times rot_scale."""
import numpy as np
import pytest
import torch

import bf16_gemm_vla_amd as vla
import synthetic
from tests.eight_bit_ref import turn_axes
from tests.gpu_util import Guarded, bf16_f64, dev, host

pytestmark = pytest.mark.gpu

EPS, TINY = 2.0 ** -8, 2.0 ** -133


def rand(seed, *shape, scale=1.0):
    x = synthetic.rng(19000 + seed).standard_normal(shape, dtype=np.float32) * np.float32(scale)
    return synthetic.fp32_to_bf16_bits(x)


def check(got, x, w, freq, axis_of, pos, rot, inter, rot_scale, eps, what):
    x, w = bf16_f64(x), None if w is None else bf16_f64(w)
    ref = turn_axes(x, w, freq, axis_of, pos, rot, inter, rot_scale, eps)
    size = np.abs(turn_axes(x, w, None, None, None, 0, False, 1.0, eps))
    pair = size.copy()
    if rot:
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
        pair[..., a] = pair[..., b] = abs(rot_scale) * (size[..., a] + size[..., b])
    bad = np.abs(bf16_f64(got) - ref) > EPS * np.abs(ref) + 2.0 ** -20 * pair * (1 + EPS) + TINY
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[0]}"


def run(T, hq, hkv, D, rot, axes, inter=False, norm=True, append=True, pos=None, axis_of=None, rot_scale=1.1, seed=0,
        in_place=False, single=False, stream=None):
    r = synthetic.rng(19500 + seed)
    q, k, v = rand(seed, T, hq, D), rand(seed + 1, T, hkv, D), rand(seed + 2, T, hkv, D)
    qw, kw = (rand(seed + 3 + i, D, scale=0.5) if norm else None for i in range(2))
    pos = r.integers(0, 3000, (axes, T)).astype(np.int32) if pos is None else np.asarray(pos, np.int32)
    axis_of = r.integers(0, axes, max(rot // 2, 1)).astype(np.uint8) if axis_of is None else np.asarray(axis_of, np.uint8)
    freq = (10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)
    n_slots = T + 5
    slots = r.permutation(n_slots)[:T].astype(np.int64)
    slots[T // 2::7] = -1
    kc, vc = rand(seed + 5, n_slots, hkv, D), rand(seed + 6, n_slots, hkv, D)
    dq, dk = dev(q), dev(k)
    go, gk, gkc, gvc = Guarded(q.nbytes), Guarded(k.nbytes), Guarded(kc.nbytes), Guarded(vc.nbytes)
    gkc.t.copy_(dev(kc).flatten().view(torch.uint8))
    gvc.t.copy_(dev(vc).flatten().view(torch.uint8))
    qo, ko = (dq, dk) if in_place else (go.t, gk.t)
    head = (dq, dk, dev(v) if append else None, None if qw is None else dev(qw), None if kw is None else dev(kw),
            dev(freq) if rot else None)
    where = (dev(slots) if append else None, qo, ko, gkc.t if append else None, gvc.t if append else None, T, hq, hkv, D, rot)
    rest = (hq * D, hkv * D, hkv * D if append else 0, hq * D, hkv * D, n_slots if append else 0, int(inter), rot_scale, 1e-6)
    if single:
        vla.vla_qk_norm_rope_append(*head, dev(pos[0]) if rot else None, *where, *rest)
    else:
        vla.vla_qk_norm_rope_axes_append(*head, dev(axis_of) if rot else None, dev(pos) if rot else None, *where, axes, *rest,
                                         stream=stream)
    torch.cuda.synchronize()
    for g in (go, gk, gkc, gvc):
        g.check()
    got_q, got_k = (host(t).view(np.uint16).reshape(x.shape) for t, x in ((qo, q), (ko, k)))
    check(got_q, q, qw, freq, axis_of, pos, rot, inter, rot_scale, 1e-6, "q")
    check(got_k, k, kw, freq, axis_of, pos, rot, inter, rot_scale, 1e-6, "k")
    if append:
        kept = slots >= 0
        kc[slots[kept]], vc[slots[kept]] = got_k[kept], v[kept]
        assert np.array_equal(gkc.numpy(np.uint16).reshape(kc.shape), kc)     # other slots as they were
        assert np.array_equal(gvc.numpy(np.uint16).reshape(vc.shape), vc)
    return got_q, got_k


@pytest.mark.parametrize("T,hq,hkv,D,rot,axes,inter,norm,append", [
    (1, 8, 1, 256, 256, 3, False, False, True), (50, 8, 1, 256, 128, 2, True, True, True),
    (256, 16, 16, 72, 72, 2, False, False, False), (17, 12, 12, 80, 40, 3, True, True, True),
    (129, 28, 4, 128, 64, 4, True, True, True), (3, 4, 2, 8, 8, 2, False, True, True),
    (9000, 2, 1, 64, 64, 3, False, True, True), (33, 5, 5, 104, 0, 3, False, True, True), (7, 3, 1, 16, 8, 1, True, False, False),
    (1, 1, 1, 248, 240, 4, False, True, True), (700, 8, 8, 64, 16, 3, False, False, True), (2, 40, 8, 128, 128, 3, True, True, False)])
def test_axes_match_the_64_bit_form(T, hq, hkv, D, rot, axes, inter, norm, append):
    run(T, hq, hkv, D, rot, axes, inter, norm, append, seed=T + D)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (72, 40)])
def test_equal_positions_give_the_one_axis_bits(D, rot, inter):
    row = synthetic.rng(19900).integers(-5000, 5000, 77).astype(np.int32)
    one = run(77, 4, 2, D, rot, 1, inter, seed=5, pos=row[None], single=True, axis_of=np.zeros(rot // 2))
    for axes in (1, 3):
        got = run(77, 4, 2, D, rot, axes, inter, seed=5, pos=np.repeat(row[None], axes, 0))
        assert all(np.array_equal(x, y) for x, y in zip(one, got))


def test_axes_far_positions_in_place_and_unknown_axes():
    pos = [[0, -1, 1 << 20, (1 << 31) - 1, -(1 << 31), 1000003, 7, 8], [5, 1 << 30, 0, -7, 3, (1 << 31) - 1, 9, -1]]
    run(8, 4, 1, 128, 128, 2, pos=pos, rot_scale=-1.5, in_place=True, seed=7)
    # axes that the tokens do not have, 255 among them: turned as at position 0
    run(8, 4, 1, 128, 128, 2, pos=pos, axis_of=[0, 1, 2, 3, 4, 7, 128, 255] * 8, seed=8)
    run(8, 4, 1, 72, 40, 2, pos=pos, axis_of=[255, 1, 2, 0, 3] * 4, inter=True, seed=9)


def test_axes_on_another_stream_and_captured():
    want = run(60, 8, 2, 64, 64, 3, seed=11)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(60, 8, 2, 64, 64, 3, seed=11, stream=side)
    assert all(np.array_equal(x, y) for x, y in zip(want, got))
    T, hq, D = 40, 4, 64
    q = dev(rand(12, T, 2 * hq * D))
    axis_of, freq = dev(np.arange(32, dtype=np.uint8) % 3), dev(np.full(32, 0.01, np.float32))
    pos = dev(np.zeros((3, T), np.int32))
    qo, ko = (torch.empty(T * hq * D, dtype=torch.int16, device="cuda") for _ in range(2))
    def call():
        vla.vla_qk_norm_rope_axes_append(q, q[:, hq * D:], None, None, None, freq, axis_of, pos, None, qo, ko, None, None, T, hq,
                                         hq, D, 64, 3, 2 * hq * D, 2 * hq * D, 0, hq * D, hq * D, 0, 0, 1.0, 0.0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(3):                                        # a captured call follows device positions
        pos.copy_(dev(synthetic.rng(19800 + step).integers(0, 500, (3, T)).astype(np.int32)))
        call()
        torch.cuda.synchronize()
        eager = qo.clone(), ko.clone()
        qo.zero_(), ko.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, eager[0]) and torch.equal(ko, eager[1])
