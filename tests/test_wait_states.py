"""No reader of a matrix or dot product instruction's result comes too early,
in the listings of every source that uses one (compiled as the build does)."""
import importlib.util
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

import wait_states

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_spec = importlib.util.spec_from_file_location(
    "moe_build", os.path.join(ROOT, "mixture_experts_ffn_moe_amd", "build.py"))
build = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(build)


def _listing(src):
    r = subprocess.run([build.HIPCC, *build.FLAGS, "-S", "--offload-device-only", src, "-o", "-"],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    return r.stdout


LISTING = """
f:
	v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], 0
	s_cbranch_scc1 .LBB0_2
	s_nop {n}
	v_add_f32_e32 v5, v2, v4
.LBB0_2:
	s_nop 7
	v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]
	s_endpgm
"""


@pytest.mark.parametrize("n", [0, 6])
def test_a_reader_behind_a_branch_is_seen(n):
    assert wait_states.distances(LISTING.format(n=n))["v_mfma_f32_16x16x32_bf16"][0] == n + 2


def test_readers_keep_the_wait_states():
    srcs = build.sources()
    with ThreadPoolExecutor(4) as ex:
        found = {os.path.basename(s): wait_states.distances(t) for s, t in zip(srcs, ex.map(_listing, srcs))}
    assert "v_mfma_f32_16x16x32_bf16" in found["q4_decode.hip"] and "v_dot2c_f32_bf16" in found["q4_w13.hip"]
    early = [(f, op, d) for f, ds in found.items() for op, d in ds.items() if d[0] < wait_states.NEEDED[op]]
    assert not early, early
