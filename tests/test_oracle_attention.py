"""Pins of the oracle's attention operators against definitions that share
nothing with its code: torch's fp64 complex product, rms_norm and softmax,
and properties of rotary positions (CPU only)."""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

import oracle
import synthetic


def values(bits):
    return torch.from_numpy((bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64))


def bits(rng, *shape, scale=1.0):
    return synthetic.fp32_to_bf16_bits((rng.standard_normal(shape) * scale).astype(np.float32))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,norm", [(64, 64, False), (72, 72, True), (128, 32, True), (8, 0, True), (80, 16, False)])
def test_norm_rope_against_complex_product(D, rot, norm, interleaved):
    rng = np.random.default_rng(11)
    T, heads = 5, 3
    x = bits(rng, T, heads, D)
    w = bits(rng, D) if norm else None
    freq = (10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)
    pos = np.array([0, 1, -7, 4099, 1 << 20], np.int32)
    got = oracle.norm_rope(x, w, freq, pos, rot, interleaved, 1.25, 1e-5)
    ref = values(x)
    if norm:
        ref = F.rms_norm(ref, (D,), eps=float(np.float32(1e-5))) * values(w)
    turn = 1.25 * torch.exp(1j * torch.from_numpy(pos.astype(np.float64))[:, None] * torch.from_numpy(freq.astype(np.float64)))
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(ref[..., a], ref[..., b]) * turn[:, None, :]
    ref = ref.clone()
    ref[..., a], ref[..., b] = z.real, z.imag
    assert np.allclose(got, ref.numpy(), rtol=0, atol=1e-9)


def test_norm_rope_properties():
    rng = np.random.default_rng(12)
    D = 32
    freq = (100.0 ** (-2.0 * np.arange(D // 2) / D)).astype(np.float32)
    x = bits(rng, 1, 2, D)
    same = oracle.norm_rope(x, None, freq, [0], D, False)
    assert np.array_equal(same, values(x).numpy())                   # position 0 turns nothing
    far = [oracle.norm_rope(x, None, freq, [p], D, False)[0] for p in (3, 10, 103, 110)]
    assert np.allclose((far[0][0] * far[1][1]).sum(), (far[2][0] * far[3][1]).sum())   # a product depends on the distance
    assert np.allclose((far[0] ** 2).sum(-1), (values(x)[0].numpy() ** 2).sum(-1))     # lengths are kept


@pytest.mark.parametrize("n,m,hq,hkv,D", [(3, 7, 4, 2, 16), (1, 1, 2, 2, 8), (5, 33, 6, 1, 72)])
def test_attention_against_torch_softmax(n, m, hq, hkv, D):
    rng = np.random.default_rng(13)
    q, k, v = bits(rng, n, hq, D, scale=3.0), bits(rng, m, hkv, D), bits(rng, m, hkv, D)
    limits = rng.integers(0, m + 1, n)
    limits[0] = 0 if n > 1 else m
    out, wabs = oracle.attention(q, k, v, limits, 0.3)
    scale = float(np.float32(0.3))
    for h in range(hq):
        g = h * hkv // hq
        s = values(q)[:, h] @ values(k)[:, g].T * scale
        for i in range(n):
            if limits[i] == 0:
                assert not out[i, h].any()
                continue
            p = torch.softmax(s[i, :limits[i]], 0)
            assert np.allclose(out[i, h], (p @ values(v)[:limits[i], g]).numpy(), rtol=1e-12, atol=1e-12)
            assert np.allclose(wabs[i, h], (p @ values(v)[:limits[i], g].abs()).numpy(), rtol=1e-12, atol=1e-12)


def test_attention_of_equal_keys_is_the_mean():
    rng = np.random.default_rng(14)
    k = np.repeat(bits(rng, 1, 1, 8), 6, 0)
    v = bits(rng, 6, 1, 8)
    out, _ = oracle.attention(bits(rng, 1, 1, 8), k, v, [4], 1.0)
    assert np.allclose(out[0, 0], values(v)[:4, 0].mean(0).numpy())


def test_pins_under_asan_and_ubsan():
    """The pins above against a build of the oracle with sanitizers."""
    import os
    import subprocess
    import sys

    if os.environ.get("ORACLE_SANITIZE") == "1":
        pytest.skip("already inside the instrumented run")
    path = subprocess.run(["gcc", "-print-file-name=libasan.so"], capture_output=True, text=True).stdout.strip()
    if not (os.path.isabs(path) and os.path.exists(path)):
        pytest.skip("gcc's AddressSanitizer runtime is not installed")
    oracle.build(force=True, sanitize=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, ORACLE_SANITIZE="1", LD_PRELOAD=path, OMP_NUM_THREADS="4",
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-m", "not gpu",
                        "tests/test_oracle_attention.py"], cwd=root, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
