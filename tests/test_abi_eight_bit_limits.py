"""Limits of the eight-bit layer's operators that their documentation states,
before any device work.  Addresses are fake and never dereferenced."""
import os
import subprocess
import sys

import pytest

import bf16_gemm_vla_amd as vla
from tests.test_abi_eight_bit import A, EINVAL, ESHAPE, GB, product_args, refused

INT8 = vla.VLA_WFMT_INT8


def supported(M, N, K):
    return vla.vla_gemm_supported(M, N, K, INT8)


# ------------------------------------------------ workspace of the product

@pytest.mark.parametrize("M,N,K", [(50, 64, 128), (50, 1024, 4096), (768, 2048, 16384), (8191, 1024, 1024)])
def test_product_refuses_a_workspace_that_overlaps(M, N, K):
    """Counters that a later call needs at zero, partial sums that other workgroups still read."""
    need = vla.vla_gemm_workspace_bytes(M, N, K, INT8)
    ws = A + 7 * GB
    for at in (ws, ws + 16, ws + 61440, ws + (need - 1) // 16 * 16):
        refused("vla_gemm_int8", product_args(M=M, N=N, K=K, residual=None, Y=at), EINVAL, "Y overlaps ws")
        for name in ("A", "s_a", "Wq", "s_w", "bias", "residual"):
            refused("vla_gemm_int8", product_args(M=M, N=N, K=K, **{name: at}), EINVAL, "ws overlaps input")
    # the workspace's end inside Y, and a residual that is Y
    refused("vla_gemm_int8", product_args(M=M, N=N, K=K, residual=None, Y=ws - 16), EINVAL, "Y overlaps ws")
    refused("vla_gemm_int8", product_args(M=M, N=N, K=K, residual=ws, Y=ws), EINVAL, "overlaps")


def test_product_counts_the_bytes_it_uses():
    """What lies behind the bytes that a shape needs is another tensor's, however large the workspace is said to be."""
    need = vla.vla_gemm_workspace_bytes(50, 64, 128, INT8)
    assert need % 16 == 0
    args = product_args(residual=None, Y=A + 7 * GB + need, ws_bytes=need - 1)
    refused("vla_gemm_int8", args, vla.VLA_EWORKSPACE)               # no overlap is seen, the size is


# --------------------------------------------------------- channels that fit

def test_channels_that_always_fit():
    """N up to 32768 with every number of rows and every K that the product takes."""
    rows = [1, 2, 5, 10, 15, 16, 17, 31, 32, 33, 47, 48, 49, 50, 63, 64, 65, 128, 191, 192, 193, 384, 385, 768, 1000, 8191, 65536, 1 << 20,
            (1 << 23) + 1, 12582720]
    depths = [32, 64, 160, 512, 544, 1024, 1056, 2048, 2080, 4096, 4128, 8192, 8704, 16384, 32768, 65536, 65568, 98304, 131008, 131040]
    for N in (16, 1024, 16384, 16400, 32752, 32768):
        for M in rows:
            for K in depths:
                fits = M <= 64 or (M * K < 1 << 31 and N * K < 1 << 31)
                assert supported(M, N, K) == (0 if fits else ESHAPE), (M, N, K)


def test_more_channels_fit_where_the_documentation_says():
    for M, N, K, code in ((50, 245760, 131040, ESHAPE), (2000000, 245760, 32, ESHAPE), (12582720, 245760, 32, ESHAPE),
                          (12582720, 32784, 32, ESHAPE), (12582720, 32768, 32, 0), (64, 245760, 65536, 0), (64, 32768, 131040, 0),
                          (8191, 245760, 8704, 0)):
        assert supported(M, N, K) == code, (M, N, K)


# ------------------------------------------------------------- the planner

def test_attention_plan_query():
    plan = vla.vla_attn_shared_prefix_plan
    for e4m3, query in ((False, vla.vla_attn_shared_prefix_workspace_bytes), (True, vla.vla_attn_shared_prefix_e4m3_workspace_bytes)):
        for args in ((1, 1, 32, 8, 128, 0, 131072), (64, 1, 32, 8, 128, 2064, 3008), (1, 10, 8, 1, 256, 768, 16), (1, 2048, 32, 8, 128, 0, 8192),
                     (41, 1, 8, 1, 64, 64, 0)):
            rc, info = plan(*args, e4m3)
            assert rc == 0 and info[5] == query(*args)
            assert info[0] in (0, 16, 32, 64, 128) and info[1] in (0, 16, 32, 64, 128) and (e4m3 or 16 not in info[:2])
            assert (info[0] > 0) == (info[2] > 0) and (info[1] > 0) == (info[3] > 0) and info[0] + info[1] > 0
            assert not (info[4] and info[0])
        assert plan(0, 1, 4, 2, 64, 16, 16, e4m3)[0] == EINVAL and plan(1, 1, 5, 2, 64, 16, 16, e4m3)[0] == ESHAPE
        assert plan(1, 1, 4, 2, 64, 0, 0, e4m3)[0] == EINVAL
    lib = vla.load()
    assert lib.vla_attn_shared_prefix_plan(1, 1, 4, 2, 64, 16, 16, 2, None, 0) == EINVAL
    assert lib.vla_attn_shared_prefix_plan(1, 1, 4, 2, 64, 16, 16, 1, None, 1) == EINVAL
    assert lib.vla_attn_shared_prefix_plan(1, 1, 4, 2, 64, 16, 16, 1, None, -1) == EINVAL
    assert lib.vla_attn_shared_prefix_plan(1, 1, 4, 2, 64, 16, 16, 1, None, 0) == 0
    assert "vla_attn_shared_prefix_plan" in vla.last_error()


# -------------------------------------------------------- a forked process

def test_a_forked_process_asks_torch_again():
    """The GPU's runtime does not outlive a fork: torch refuses its first call in the child, and so does a call that takes
    the stream from torch, whatever the parent had looked up."""
    script = ("import os, sys\n"
              "import bf16_gemm_vla_amd._lib as L\n"
              "L._current = (lambda device: 7), (lambda: 0)\n"
              "assert L._stream(None) == 7\n"
              "pid = os.fork()\n"
              "if pid == 0:\n"
              "    import torch\n"
              "    def refuse(): raise RuntimeError('forked')\n"
              "    torch.cuda.current_device = refuse\n"
              "    try:\n"
              "        L._stream(None)\n"
              "    except RuntimeError as e:\n"
              "        os._exit(0 if 'forked' in str(e) else 2)\n"
              "    os._exit(1)\n"
              "sys.exit(os.waitstatus_to_exitcode(os.waitpid(pid, 0)[1]) or (L._stream(None) != 7))\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", script], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
