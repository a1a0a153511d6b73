"""Refusals of the attention operators, before any device work: every bad
argument gets its status code.  Addresses are fake and never dereferenced."""
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


def append_args(**change):
    names = ["q", "k", "v", "q_weight", "k_weight", "inv_freq", "positions", "slots", "q_out", "k_out", "k_cache", "v_cache"]
    a = {n: A + i * GB for i, n in enumerate(names)}
    a |= dict(T=4, Hq=8, Hkv=2, D=64, rot=32, q_stride=512, k_stride=128, v_stride=128, q_out_stride=512,
              k_out_stride=128, num_slots=64, layout=0, rot_scale=1.0, eps=1e-6)
    return a | change


@pytest.mark.parametrize("change,code", [
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(q_out=None), EINVAL), (dict(q=A + 8), EALIGN),
    (dict(slots=A + 8), EALIGN), (dict(T=0), EINVAL), (dict(T=(1 << 24) + 1), ESHAPE), (dict(Hq=0), EINVAL),
    (dict(Hq=9, q_stride=576, q_out_stride=576), ESHAPE), (dict(D=60), ESHAPE), (dict(D=264), ESHAPE), (dict(D=0), EINVAL),
    (dict(rot=72), ESHAPE), (dict(rot=-8), ESHAPE), (dict(rot=20), ESHAPE), (dict(layout=2), EINVAL),
    (dict(rot_scale=float("inf")), EINVAL), (dict(eps=-1e-6), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(inv_freq=None), EINVAL), (dict(positions=None), EINVAL), (dict(rot=0), EINVAL),
    (dict(v=None), EINVAL), (dict(slots=None), EINVAL), (dict(v_cache=None), EINVAL), (dict(num_slots=0), EINVAL),
    (dict(num_slots=-1), EINVAL), (dict(num_slots=1 << 31), ESHAPE),
    (dict(v=None, slots=None, k_cache=None, v_cache=None, num_slots=0, k_out=None), EINVAL),
    (dict(q_stride=504), ESHAPE), (dict(q_stride=516), ESHAPE), (dict(k_stride=120), ESHAPE), (dict(v_stride=0), ESHAPE),
    (dict(q_out_stride=256), ESHAPE), (dict(k_out_stride=64), ESHAPE)])
def test_append_refuses(change, code):
    refused("vla_qk_norm_rope_append", append_args(**change), code)


def test_append_refuses_overlaps():
    base = append_args()
    merged = dict(q=A, k=A + 1024, v=A + 1280, q_stride=768, k_stride=768, v_stride=768)
    for change in (dict(q_out=A + 16), dict(q_out=A, q_out_stride=1024), dict(k_out=base["k"] + 16),
                   dict(k_cache=base["v"]), dict(v_cache=base["k_cache"]), dict(k_out=base["q_out"]),
                   # in place over the wrong column block, or one column too wide
                   merged | dict(q_out=A + 16, q_out_stride=768), merged | dict(k_out=A + 1280, k_out_stride=768),
                   merged | dict(k_out=A + 1008, k_out_stride=768)):
        refused("vla_qk_norm_rope_append", append_args(**change), EINVAL, "overlap")


def prompt_args(**change):
    names = ["q", "k", "v", "cu_q", "cu_k", "out"]
    a = {n: A + i * GB for i, n in enumerate(names)}
    a |= dict(B=2, total_q=10, total_k=12, Hq=4, Hkv=2, D=64, q_stride=256, k_stride=128, v_stride=128, out_stride=256,
              causal=1, scale=0.125)
    return a | change


@pytest.mark.parametrize("change,code", [
    (dict(q=None), EINVAL), (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(cu_q=None), EINVAL), (dict(out=None), EINVAL),
    (dict(k=A + 2), EALIGN), (dict(cu_k=A + 4), EALIGN), (dict(B=0), EINVAL), (dict(total_q=0), EINVAL), (dict(total_k=-1), EINVAL),
    (dict(B=(1 << 20) + 1), ESHAPE), (dict(total_q=(1 << 30) + 1), ESHAPE), (dict(Hkv=3), ESHAPE), (dict(D=12), ESHAPE),
    (dict(D=512), ESHAPE), (dict(q_stride=248), ESHAPE), (dict(out_stride=260), ESHAPE), (dict(k_stride=64), ESHAPE),
    (dict(v_stride=64), ESHAPE), (dict(causal=2), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(scale=-1.0), EINVAL), (dict(total_q=1 << 30, Hq=4096, Hkv=64, q_stride=4096 * 64, out_stride=4096 * 64, k_stride=4096, v_stride=4096), ESHAPE),
    (dict(out=A), EINVAL), (dict(out=A + GB), EINVAL), (dict(out=A + 3 * GB), EINVAL)])
def test_prompt_refuses(change, code):
    refused("vla_attn_prompt", prompt_args(**change), code)


def test_prompt_refuses_rows_past_31_bits():
    """A key/value head's rows (tokens times query heads per key/value head) are numbered in 31 bits."""
    few = dict(total_q=(1 << 22), total_k=12, Hq=512, Hkv=1, D=8, q_stride=4096, k_stride=8, v_stride=8, out_stride=4096)
    refused("vla_attn_prompt", prompt_args(**few), ESHAPE, "too many")


def shared_args(**change):
    names = ["q", "k_cache", "v_cache", "prefix_pages", "prefix_len", "block_table", "seq_lens", "out", "ws"]
    a = {n: A + i * GB for i, n in enumerate(names)}
    a |= dict(ws_bytes=1 << 28, B=3, L=2, Hq=4, Hkv=2, D=64, num_pages=100, page_size=16, n_prefix_pages=20,
              pages_per_seq=4, q_stride=256, out_stride=256, causal=0, scale=0.125)
    return a | change


@pytest.mark.parametrize("change,code", [
    (dict(q=None), EINVAL), (dict(k_cache=None), EINVAL), (dict(v_cache=None), EINVAL), (dict(out=None), EINVAL), (dict(ws=None), EINVAL),
    (dict(prefix_pages=A + 4), EALIGN), (dict(seq_lens=A + 4), EALIGN), (dict(B=0), EINVAL), (dict(L=0), EINVAL),
    (dict(num_pages=0), EINVAL), (dict(page_size=0), EINVAL), (dict(page_size=24), ESHAPE), (dict(page_size=1 << 17), ESHAPE),
    (dict(num_pages=1 << 28), ESHAPE), (dict(n_prefix_pages=-1), EINVAL), (dict(pages_per_seq=-1), EINVAL),
    (dict(prefix_pages=None), EINVAL), (dict(prefix_len=None), EINVAL), (dict(block_table=None), EINVAL), (dict(seq_lens=None), EINVAL),
    (dict(n_prefix_pages=0), EINVAL), (dict(pages_per_seq=0), EINVAL),
    (dict(prefix_pages=None, prefix_len=None, n_prefix_pages=0, block_table=None, seq_lens=None, pages_per_seq=0), EINVAL),
    (dict(Hq=5), ESHAPE), (dict(D=20), ESHAPE), (dict(q_stride=200), ESHAPE), (dict(out_stride=128), ESHAPE),
    (dict(causal=-1), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(ws_bytes=0), EWS),
    (dict(n_prefix_pages=1 << 26), ESHAPE), (dict(B=1 << 20, L=1 << 20), ESHAPE),
    (dict(out=A), EINVAL), (dict(out=A + 2 * GB), EINVAL), (dict(ws=A), EINVAL), (dict(out=A + 8 * GB), EINVAL)])
def test_shared_refuses(change, code):
    refused("vla_attn_shared_prefix", shared_args(**change), code)


def test_shared_refuses_numbers_past_31_bits():
    """Rows of a key/value head and keys of a sequence are numbered in 31 bits, steps past the last one included."""
    half = (1 << 30) - 1
    refused("vla_attn_shared_prefix", shared_args(page_size=1, n_prefix_pages=half, pages_per_seq=half), ESHAPE, "too large")
    n = vla.vla_attn_shared_prefix_workspace_bytes
    assert n(1, 1, 4, 2, 64, half, half) == 0 and n(1, 1, 4, 2, 64, half, 1 << 29) > 0
    assert n(1 << 10, 1 << 9, 4095, 1, 8, 16, 16) > 0 and n((1 << 20) - 1, 1 << 10, 2, 1, 8, 16, 16) > 0
    assert n(1 << 20, 1 << 10, 2, 1, 8, 16, 16) == 0


@pytest.mark.parametrize("scale", [3e38, float("-inf"), -0.0])
def test_scales_refused(scale):
    refused("vla_attn_prompt", prompt_args(scale=scale), EINVAL, "scale")
    refused("vla_attn_shared_prefix", shared_args(scale=scale), EINVAL, "scale")


def test_shared_workspace_query():
    n = vla.vla_attn_shared_prefix_workspace_bytes
    assert n(3, 2, 4, 2, 64, 320, 64) > 0
    refused("vla_attn_shared_prefix", shared_args(ws_bytes=n(3, 2, 4, 2, 64, 320, 64) - 1), EWS)
    assert n(0, 2, 4, 2, 64, 320, 64) == 0 and n(3, 2, 4, 3, 64, 320, 64) == 0 and n(3, 2, 4, 2, 64, 0, 0) == 0
    for B in (1, 2, 64, 4096):
        for L in (1, 10, 50, 1000):
            for hq, hkv, D in ((8, 1, 256), (32, 8, 128), (16, 16, 72), (1, 1, 8)):
                for pre in (0, 1, 768, 100000):
                    for suf in (0, 16, 131072):
                        if pre + suf:
                            assert n(B, L, hq, hkv, D, pre, suf) > 0


def test_binding_raises():
    with pytest.raises(RuntimeError, match="vla_attn_prompt: .*scale"):
        vla.vla_attn_prompt(*[A + i * GB for i in range(6)], 1, 1, 1, 1, 1, 8, 8, 8, 8, 8, True, 0.0, stream=0)


def test_refusals_under_asan_and_ubsan():
    """The tests above against a build whose host code is instrumented: the
    checks and the launch plans neither overflow nor read out of bounds."""
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
              "'tests/test_abi_attention.py']))\n") % (root, lib)
    env = dict(os.environ, LD_PRELOAD=runtime[-1], ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-c", runner], cwd=root, env=env, capture_output=True, text=True, timeout=900)
    tail = (r.stdout + r.stderr)[-4000:]
    assert r.returncode == 0, tail
    assert "passed" in r.stdout and "ERROR: AddressSanitizer" not in tail and "runtime error" not in tail, tail


def test_row_offsets_of_any_value_stay_in_the_tensor(tmp_path):
    """The bounds that the prompt kernel puts on its offsets, compiled for the
    host with UndefinedBehaviorSanitizer: no difference passes 32 bits, and no
    pair of offsets leads outside."""
    import os
    import shutil
    import subprocess

    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "rows.cpp"
    src.write_text('''#include <cstdio>
#include <algorithm>
#include "bounded.h"
int main() {
    const int32_t values[] = {INT32_MIN, INT32_MIN + 1, -65, -1, 0, 1, 30, 63, 64, 65, 1 << 30, INT32_MAX};
    for (int32_t total : {1, 64, 1 << 30})
        for (int32_t begin : values)
            for (int32_t end : values) {
                int32_t first, n;
                vla::bounded_rows(begin, end, total, first, n);
                const int64_t b = std::min<int64_t>(std::max<int64_t>(begin, 0), total);
                const int64_t e = std::min<int64_t>(std::max<int64_t>(end, b), total);
                if (first != b || n != e - b) { printf("%d %d of %d: %d %d\\n", begin, end, total, first, n); return 1; }
            }
    return 0;
}
''')
    exe = str(tmp_path / "rows")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=undefined", "-I",
                    os.path.join(root, "bf16_gemm_vla_amd", "csrc"), str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr


def test_sizes_past_one_launch_are_refused():
    """A launch holds fewer than 2^24 workgroups of 256 threads: row tiles of a
    prompt, work items and joined rows over the cache."""
    one = dict(B=1 << 20, total_q=1 << 20, total_k=1 << 20, D=8)
    for heads in (16, 64):
        strides = {f"{x}_stride": heads * 8 for x in ("q", "k", "v", "out")}
        refused("vla_attn_prompt", prompt_args(Hq=heads, Hkv=heads, **one, **strides), ESHAPE, "too many")
    n = vla.vla_attn_shared_prefix_workspace_bytes
    most = 1 << 20
    for heads, kv, prefix, suffix in ((16, 16, 0, 16), (64, 4, 16, 16)):       # items, joined rows
        assert n(most, 1, heads, kv, 64, prefix, suffix) == 0 and "too many" in vla.last_error()
        assert n(most - 1, 1, heads, kv, 64, prefix, suffix) > 0
        refused("vla_attn_shared_prefix", shared_args(
            B=most, L=1, Hq=heads, Hkv=kv, n_prefix_pages=prefix // 16, prefix_pages=A + 3 * GB if prefix else None,
            prefix_len=A + 4 * GB if prefix else None, pages_per_seq=1, q_stride=heads * 64, out_stride=heads * 64,
            ws_bytes=1 << 50), ESHAPE, "too many")
