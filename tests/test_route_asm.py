"""Static checks on the compiled scored routing (CPU only: hipcc
cross-compiles gfx950 assembly).

The row selection branches where lanes are switched off and on again; a
register that the compiler saves to scratch memory inside such a region, or
around a call in it, is lost to the lanes that were off.  The kernels are
bounded so that nothing is saved: no scratch access and no call."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def compile_asm(src, out):
    if not (os.path.exists(HIPCC) or shutil.which("hipcc")):
        pytest.skip("hipcc not available")
    cmd = [HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature",
           "-Xclang", "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "--cuda-device-only", "-S",
           os.path.join(ROOT, "fp4_expert_ffn_amd", "csrc", src), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return out.read_text()


def test_scored_routing_neither_spills_nor_calls(tmp_path):
    asm = compile_asm("route_scored.hip", tmp_path / "route.s")
    kernels = re.findall(r"^\s*\.amdhsa_kernel (\S+)", asm, re.M)
    assert len([k for k in kernels if "k_route_one" in k]) == 7
    code = [ln.split(";")[0].strip() for ln in asm.split("\n")]
    bad = [ln for ln in code if ln.startswith(("scratch_", "s_swappc", "buffer_store_dword off", "s_call"))]
    assert not bad, bad[:5]


def test_linear_tile_waits_and_m0(tmp_path):
    """The tile kernel of the linear product: M0 belongs to its direct-to-LDS loads, nothing spills,
    and every counted wait of its loop precedes a barrier."""
    asm = compile_asm("linear_tile.hip", tmp_path / "tile.s")
    code = [ln.split(";")[0].strip() for ln in asm.split("\n")]
    assert not [ln for ln in code if ln.startswith(("scratch_", "s_swappc"))]
    for n, ln in enumerate(code):
        if re.search(r"\bm0\b", ln):
            assert ln.startswith("s_mov_b32 m0,"), ln
            nxt = [t for t in code[n + 1:n + 8] if t and not t.startswith((".", "#"))][:2]
            assert nxt[0] == "s_nop 0" and nxt[1].startswith("global_load_lds_"), (ln, nxt)
    assert sum(ln.startswith("global_load_lds_dwordx4") for ln in code) > 100
