"""Limits of the eight-bit layer's operators that their documentation states,
before any device work.  Addresses are fake and never dereferenced."""
import bf16_gemm_vla_amd as vla
from tests.test_abi_eight_bit import EINVAL, ESHAPE


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
