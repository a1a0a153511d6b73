"""Refusals of the eight-bit layer's operators, before any device work: every
bad argument gets its status code.  Addresses are fake and never dereferenced."""
import pytest

import bf16_gemm_vla_amd as vla

A = 1 << 40          # fake device addresses, 1 GiB apart
GB = 1 << 30
EINVAL, ESHAPE, EALIGN, EWS = vla.VLA_EINVAL, vla.VLA_ESHAPE, vla.VLA_EALIGN, vla.VLA_EWORKSPACE


def refused(name, args, code, word=None):
    rc = getattr(vla.load(), name)(*args.values(), None)
    assert rc == code, (rc, vla.last_error())
    assert name in vla.last_error()
    if word:
        assert word in vla.last_error()


def axes_args(**change):
    names = ["q", "k", "v", "q_weight", "k_weight", "inv_freq", "axis_of", "positions", "slots", "q_out", "k_out", "k_cache",
             "v_cache"]
    a = {n: A + i * GB for i, n in enumerate(names)}
    a |= dict(T=4, Hq=8, Hkv=2, D=64, rot=32, axes=3, q_stride=512, k_stride=128, v_stride=128, q_out_stride=512,
              k_out_stride=128, num_slots=64, layout=0, rot_scale=1.0, eps=1e-6)
    return a | change


@pytest.mark.parametrize("change,code", [
    (dict(q=None), EINVAL), (dict(q_out=None), EINVAL), (dict(axis_of=None), EINVAL), (dict(positions=None), EINVAL),
    (dict(inv_freq=None), EINVAL), (dict(rot=0), EINVAL), (dict(rot=0, inv_freq=None, positions=None), EINVAL),
    (dict(axis_of=A + 6 * GB + 8), EALIGN), (dict(positions=A + 4), EALIGN), (dict(axes=0), EINVAL), (dict(axes=-1), EINVAL),
    (dict(axes=5), ESHAPE), (dict(T=0), EINVAL), (dict(T=(1 << 24) + 1), ESHAPE), (dict(D=60), ESHAPE), (dict(rot=20), ESHAPE),
    (dict(layout=2), EINVAL), (dict(rot_scale=float("nan")), EINVAL), (dict(eps=-1.0), EINVAL), (dict(v=None), EINVAL),
    (dict(num_slots=0), EINVAL), (dict(q_stride=504), ESHAPE), (dict(k_out_stride=64), ESHAPE)])
def test_axes_refuses(change, code):
    refused("vla_qk_norm_rope_axes_append", axes_args(**change), code)


def test_axes_refuses_overlaps():
    base = axes_args()
    # the second and third axis's positions count, and every pair's axis
    for change in (dict(q_out=base["positions"] + 32), dict(k_out=base["axis_of"]), dict(k_cache=base["v"]),
                   dict(q_out=base["q"] + 16)):
        refused("vla_qk_norm_rope_axes_append", axes_args(**change), EINVAL, "overlap")
