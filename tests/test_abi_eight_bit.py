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


def tokens_args(**change):
    return dict(A=A, qa=A + GB, s_a=A + 2 * GB, M=4, K=64) | change


@pytest.mark.parametrize("change,code", [
    (dict(A=None), EINVAL), (dict(qa=None), EINVAL), (dict(s_a=None), EINVAL), (dict(A=A + 8), EALIGN), (dict(s_a=A + 4), EALIGN),
    (dict(M=0), EINVAL), (dict(K=0), EINVAL), (dict(K=48), ESHAPE), (dict(M=(1 << 24) + 1), ESHAPE), (dict(qa=A), EINVAL),
    (dict(s_a=A + 16), EINVAL), (dict(s_a=A + GB + 64), EINVAL), (dict(qa=A + 496), EINVAL)])
def test_tokens_refuses(change, code):
    refused("vla_quantize_tokens_int8", tokens_args(**change), code)


def product_args(**change):
    names = ["A", "s_a", "Wq", "s_w", "bias", "residual", "Y", "ws"]
    a = {n: A + i * GB for i, n in enumerate(names)}
    return a | dict(ws_bytes=1 << 28, M=50, N=64, K=128) | change


@pytest.mark.parametrize("change,code", [
    (dict(A=None), EINVAL), (dict(s_a=None), EINVAL), (dict(Wq=None), EINVAL), (dict(s_w=None), EINVAL), (dict(Y=None), EINVAL),
    (dict(ws=None), EINVAL), (dict(bias=A + 2), EALIGN), (dict(residual=A + 8), EALIGN), (dict(M=0), EINVAL), (dict(N=24), ESHAPE),
    (dict(K=48), ESHAPE), (dict(K=131072), ESHAPE), (dict(ws_bytes=100), EWS), (dict(Y=A), EINVAL), (dict(Y=A + 2 * GB), EINVAL),
    (dict(Y=A + GB + 64), EINVAL), (dict(Y=A + 4 * GB), EINVAL), (dict(Y=A + 5 * GB + 16), EINVAL),
    (dict(M=1 << 24, K=1024, residual=None, Y=A + 64 * GB), ESHAPE),
    (dict(M=100, N=1 << 25, K=128, residual=None, Y=A + 64 * GB), ESHAPE)])
def test_product_refuses(change, code):
    refused("vla_gemm_int8", product_args(**change), code)


def test_int8_plans():
    n = vla.VLA_WFMT_INT8
    assert vla.vla_packed_bytes(64, 128, n) == 64 * 128
    for M in (1, 10, 50, 64, 65, 571, 768, 8191, 16384):
        for N, K in ((4096, 1024), (1024, 4096), (16384, 2048), (2048, 16384), (16, 32), (1040, 96)):
            rc, info = vla.vla_gemm_plan(M, N, K, n)
            assert rc == 0 and info[6] == vla.vla_gemm_workspace_bytes(M, N, K, n), (M, N, K)
            assert info[5] == 1 or info[9] <= 15360
    assert vla.vla_gemm_supported(50, 64, 131040, n) == 0 and vla.vla_gemm_supported(50, 64, 131072, n) == ESHAPE
    assert vla.vla_gemm_supported(50, 64, 64, n, fp8_act=True) == EINVAL
    assert vla.vla_gemm_supported(50, 64, 64, n, gelu_mul=True) == EINVAL


def append_args(**change):
    names = ["k", "v", "cu_rows", "block_table", "seq_lens", "k_cache", "v_cache", "k_scales", "v_scales"]
    a = {n: A + i * GB for i, n in enumerate(names)}
    a |= dict(B=3, L=2, total=6, Hkv=2, D=64, num_pages=100, page_size=16, block_size=16, pages_per_seq=4, k_stride=128,
              v_stride=128)
    return a | change


@pytest.mark.parametrize("change,code", [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(block_table=None), EINVAL), (dict(seq_lens=None), EINVAL),
    (dict(k_cache=None), EINVAL), (dict(v_scales=None), EINVAL), (dict(k_scales=A + 8), EALIGN), (dict(cu_rows=A + 4), EALIGN),
    (dict(B=0), EINVAL), (dict(L=0), EINVAL), (dict(total=0), EINVAL), (dict(pages_per_seq=0), EINVAL), (dict(B=(1 << 20) + 1), ESHAPE),
    (dict(total=(1 << 30) + 1), ESHAPE), (dict(cu_rows=None, total=7), ESHAPE), (dict(Hkv=0), EINVAL), (dict(Hkv=4097, k_stride=1 << 20), ESHAPE),
    (dict(D=60), ESHAPE), (dict(D=264), ESHAPE), (dict(num_pages=0), EINVAL), (dict(page_size=24), ESHAPE), (dict(page_size=1 << 17), ESHAPE),
    (dict(num_pages=1 << 28), ESHAPE), (dict(block_size=0), EINVAL), (dict(block_size=-16), EINVAL), (dict(block_size=12), ESHAPE),
    (dict(block_size=32), ESHAPE), (dict(page_size=256, block_size=256), ESHAPE), (dict(k_stride=120), ESHAPE), (dict(v_stride=132), ESHAPE),
    (dict(pages_per_seq=1 << 27), ESHAPE), (dict(k_cache=A), EINVAL), (dict(v_cache=A + 5 * GB), EINVAL), (dict(v_scales=A + 7 * GB), EINVAL),
    (dict(k_scales=A + 6 * GB + 64), EINVAL), (dict(v_cache=A + 4 * GB), EINVAL),
    (dict(B=1 << 20, total=1 << 26, L=1 << 20, block_size=1), ESHAPE)])
def test_kv_append_refuses(change, code):
    refused("vla_kv_append_e4m3", append_args(**change), code)


def attention_args(**change):
    names = ["q", "k_cache", "v_cache", "k_scales", "v_scales", "prefix_pages", "prefix_len", "block_table", "seq_lens", "out", "ws"]
    a = {n: A + i * GB for i, n in enumerate(names)}
    a |= dict(ws_bytes=1 << 28, B=3, L=2, Hq=4, Hkv=2, D=64, num_pages=100, page_size=16, block_size=16, n_prefix_pages=20,
              pages_per_seq=4, q_stride=256, out_stride=256, causal=0, scale=0.125)
    return a | change


@pytest.mark.parametrize("change,code", [
    (dict(q=None), EINVAL), (dict(k_cache=None), EINVAL), (dict(v_cache=None), EINVAL), (dict(k_scales=None), EINVAL),
    (dict(v_scales=None), EINVAL), (dict(out=None), EINVAL), (dict(ws=None), EINVAL), (dict(k_scales=A + 4), EALIGN),
    (dict(prefix_pages=A + 4), EALIGN), (dict(B=0), EINVAL), (dict(L=0), EINVAL), (dict(num_pages=0), EINVAL), (dict(page_size=24), ESHAPE),
    (dict(num_pages=1 << 28), ESHAPE), (dict(block_size=0), EINVAL), (dict(block_size=-1), EINVAL), (dict(block_size=24), ESHAPE),
    (dict(block_size=32), ESHAPE), (dict(page_size=256, block_size=256), ESHAPE), (dict(prefix_pages=None), EINVAL),
    (dict(seq_lens=None), EINVAL), (dict(pages_per_seq=0), EINVAL), (dict(Hq=5), ESHAPE), (dict(D=20), ESHAPE), (dict(q_stride=200), ESHAPE),
    (dict(out_stride=128), ESHAPE), (dict(causal=-1), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=3e38), EINVAL), (dict(ws_bytes=0), EWS),
    (dict(n_prefix_pages=1 << 26), ESHAPE), (dict(out=A), EINVAL), (dict(out=A + 2 * GB), EINVAL), (dict(ws=A + 4 * GB + 64), EINVAL),
    (dict(out=A + 3 * GB), EINVAL), (dict(out=A + 10 * GB), EINVAL)])
def test_attention_refuses(change, code):
    refused("vla_attn_shared_prefix_e4m3", attention_args(**change), code)


def test_attention_workspace_query():
    n = vla.vla_attn_shared_prefix_e4m3_workspace_bytes
    assert n(0, 1, 4, 2, 64, 16, 16) == 0 and n(1, 1, 4, 2, 64, 0, 0) == 0 and n(1, 1, 5, 2, 64, 16, 16) == 0
    assert n(1, 1, 32, 8, 128, 0, 131072) > 0
    assert n(1 << 20, 1 << 10, 2, 1, 8, 16, 16) == 0


def test_product_grids_past_a_launch_are_refused():
    supported = lambda M, N, K: vla.vla_gemm_supported(M, N, K, vla.VLA_WFMT_INT8)   # noqa: E731
    assert supported(192 * 65535, 16, 32) == 0 and supported(192 * 65535 + 1, 16, 32) == ESHAPE      # blocks of rows
    assert supported(1, 1 << 26, 32) == 0 and supported(1, 1 << 30, 32) == ESHAPE                    # threads
    assert supported(1 << 23, 1 << 23, 32) == ESHAPE
    for M in (1, 16, 17, 32, 33, 64):                                                                # weights past 2 GiB
        assert supported(M, 1 << 17, 1 << 14) == 0 and supported(M, (1 << 17) - 16, 1 << 14) == 0
    assert supported(65, 1 << 17, 1 << 14) == ESHAPE
    for M in (1, 10, 16, 17, 30, 33, 50, 64):
        for K in (32, 1024, 1056, 4096, 4128, 8192, 8704):
            assert supported(M, 245760, K) == 0, (M, K)


def test_extreme_sizes_are_planned_or_refused():
    """Every size at both ends of its range and past it: a status code or a plan, never an overflow on the way."""
    big = (1, 31, 1 << 20, (1 << 31) - 1, 1 << 31, 1 << 40, (1 << 62) + 16, (1 << 63) - 1, -1, -(1 << 63))
    lib = vla.load()
    for m in big:
        for n in (16, (1 << 31) - 16, 1 << 40, (1 << 63) - 16):
            for k in (32, 131040, 131072, 1 << 40, (1 << 63) - 32):
                vla.vla_gemm_plan(m, n, k, vla.VLA_WFMT_INT8)
                vla.vla_gemm_workspace_bytes(m, n, k, vla.VLA_WFMT_INT8)
                vla.vla_packed_bytes(n, k, vla.VLA_WFMT_INT8)
    for x in big:
        for y in big:
            for D in (8, 64, 200, 256):
                vla.vla_attn_shared_prefix_e4m3_workspace_bytes(x, 1, 32, 8, D, 0, y)
                vla.vla_attn_shared_prefix_e4m3_workspace_bytes(1, x, 8, 1, D, y, 16)
                vla.vla_attn_shared_prefix_e4m3_workspace_bytes(4, x, y, 1, D, 4096, 4096)
    for name, make, keys in (("vla_kv_append_e4m3", append_args, ("B", "L", "total", "Hkv", "D", "num_pages", "page_size", "block_size",
                                                                  "pages_per_seq", "k_stride", "v_stride")),
                             ("vla_attn_shared_prefix_e4m3", attention_args, ("B", "L", "Hq", "Hkv", "D", "num_pages", "page_size",
                                                                              "block_size", "pages_per_seq", "q_stride", "out_stride")),
                             ("vla_quantize_tokens_int8", tokens_args, ("M", "K")), ("vla_gemm_int8", product_args, ("M", "N", "K")),
                             ("vla_qk_norm_rope_axes_append", axes_args, ("T", "Hq", "Hkv", "D", "rot", "axes", "num_slots"))):
        for key in keys:
            for x in (0, -1, -(1 << 63), 1 << 62, (1 << 63) - 1):
                if name == "vla_qk_norm_rope_axes_append" and key == "rot" and x == 0:
                    continue
                assert getattr(lib, name)(*make(**{key: x}).values(), None) in (EINVAL, ESHAPE, EALIGN, EWS), (name, key, x)


def test_refusals_under_asan_and_ubsan():
    """The tests above against a build whose host code is instrumented."""
    import glob
    import os
    import subprocess
    import sys

    from bf16_gemm_vla_amd import build as vla_build

    runtime = sorted(glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))
    if not runtime:
        pytest.skip("clang's AddressSanitizer runtime is not installed")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lib = vla_build.build(sanitize=True)
    runner = ("import sys; sys.path.insert(0, %r)\n"
              "import bf16_gemm_vla_amd._lib as L; L.LIB_PATH = %r\n"
              "import pytest; sys.exit(pytest.main(['-q', '-x', '-p', 'no:cacheprovider', '-k', 'not asan', "
              "'tests/test_abi_eight_bit.py']))\n") % (root, lib)
    env = dict(os.environ, LD_PRELOAD=runtime[-1], ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-c", runner], cwd=root, env=env, capture_output=True, text=True, timeout=900)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert "passed" in r.stdout and "ERROR: AddressSanitizer" not in tail and "runtime error" not in tail, tail
