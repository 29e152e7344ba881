"""The block-scaled tile kernels' direct-to-LDS loads take their destination
from M0, which each sets right before itself (CPU only: hipcc cross-compiles
gfx950 assembly).  Inline assembly and the compiler share the register: a use of
it by the compiler in between would send a load elsewhere."""
import re

import pytest

from tests.test_route_asm import compile_asm


def strays(code):
    """Uses of M0 that are not a direct-to-LDS load's own, and loads that do not set it."""
    bad = []
    for n, ln in enumerate(code):
        if re.search(r"\bm0\b", ln):
            nxt = [t for t in code[n + 1:n + 8] if t and not t.startswith((".", "#"))][:2]
            if not (ln.startswith("s_mov_b32 m0,") and nxt[:1] == ["s_nop 0"] and nxt[1].startswith("global_load_lds_")):
                bad.append(ln)
        elif ln.startswith("global_load_lds_"):
            back = [t for t in code[max(0, n - 7):n] if t and not t.startswith((".", "#"))][-2:]
            if not (len(back) == 2 and back[0].startswith("s_mov_b32 m0,") and back[1] == "s_nop 0"):
                bad.append(ln)
    return bad


@pytest.mark.parametrize("name,kernels,least", [("linear_block_tile", 20, 200), ("linear_block_big", 2, 32),
                                                ("linear_block_stream", 4, 60)])
def test_m0_belongs_to_the_loads_into_lds(name, kernels, least, tmp_path):
    asm = compile_asm(name + ".hip", tmp_path / "tile.s")
    code = [ln.split(";")[0].strip() for ln in asm.split("\n")]
    assert len(re.findall(r"^\s*\.amdhsa_kernel \S+", asm, re.M)) >= kernels
    assert not strays(code)
    assert sum(ln.startswith("global_load_lds_dwordx4") for ln in code) > least
    assert sum(ln.startswith("global_load_lds_dword ") for ln in code) > least // 10


def test_the_check_sees_a_use_between():
    own = ["s_mov_b32 m0, s4", "s_nop 0", "global_load_lds_dwordx4 v1, s[2:3]"]
    assert not strays(own + ["v_add_u32 v1, v2, v3"] + own)
    assert strays(["s_mov_b32 m0, -1"] + own[1:2] + ["ds_read_b32 v1, v2"])
    assert strays(own[:1] + ["s_mov_b32 m0, s9"] + own[1:])
    assert strays(own + [own[2]])
