"""Static checks on the compiled tile kernels of the linear product (CPU only:
hipcc cross-compiles gfx950 assembly).

The kernels read what direct-to-LDS loads leave in the ring.  Those loads are
ordered by counted waits of the kernels' own, each behind a barrier that makes
the other waves' loads visible too: a wait that counts too many, or a read
ahead of the barrier, would race."""
import re

import pytest

from tests.test_route_asm import compile_asm


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """name -> instructions of every tile kernel."""
    asm = compile_asm("linear_tile.hip", tmp_path_factory.mktemp("asm") / "tile.s")
    out, name = {}, None
    for ln in asm.split("\n"):
        m = re.match(r"(_ZN3moe13k_linear_tile\S+):", ln)
        if m:
            name = m.group(1)
            out[name] = []
        elif name and ln.startswith("\t.section"):
            name = None
        elif name:
            t = ln.split(";")[0].strip()
            if t and not t.startswith("#"):
                out[name].append(t)
    return out


def shape_of(name):
    p = re.match(r"_ZN3moe13k_linear_tileILi(\d)ELb(\d)ELb(\d)ELi(\d)ELi(\d)ELi(\d)ELi(\d)ELi(\d)E", name)
    return tuple(int(v) for v in p.groups())


def main_loop(code):
    """First and last line of the loop around the matrix instructions: the backward branch with the most of them inside."""
    at = {ln[:-1]: n for n, ln in enumerate(code) if ln.endswith(":")}
    best, span = 0, None
    for n, ln in enumerate(code):
        m = re.match(r"s_c?branch\S* (\.LBB\S+)", ln)
        if m and at.get(m.group(1), n) < n:
            k = sum(t.startswith("v_mfma") for t in code[at[m.group(1)]:n])
            if k > best:
                best, span = k, (at[m.group(1)], n)
    return span


def test_every_tile_kernel_is_there(kernels):
    assert len(kernels) == 46 and len({shape_of(k) for k in kernels}) == len(kernels)


def test_counted_waits_are_the_rings_and_precede_a_barrier(kernels):
    for name, code in kernels.items():
        qm, _, _, wm, wn, tm, tn, stages = shape_of(name)
        waves = wm * wn
        loads = wm * tm * 2 // waves + wn * tn * 2 // waves + (1 if qm == 2 else 0)  # a wave's of one step
        full = (stages - 1) * loads                                                  # in flight behind a step's
        inner = full if stages == 2 else full - full // (stages - 1)
        last = main_loop(code)[1]
        seen = []
        for n, ln in enumerate(code[:last]):
            m = re.fullmatch(r"s_waitcnt vmcnt\((\d+)\)", ln)
            if not m or int(m.group(1)) < 2:
                continue  # the compiler's own, of the scales and biases
            seen.append(int(m.group(1)))
            ahead = next(t for t in code[n + 1:] if t.startswith(("s_barrier", "ds_read", "v_mfma")))
            assert ahead == "s_barrier", (name, ln, ahead)
        assert full in seen and inner in seen and max(seen) == full, (name, seen, full, inner)
        assert set(seen) <= {full, inner}, (name, seen, full, inner)


def test_a_loop_pass_loads_one_step(kernels):
    for name, code in kernels.items():
        qm, _, _, wm, wn, tm, tn, _ = shape_of(name)
        a, b = main_loop(code)
        body = code[a:b]
        waves = wm * wn
        assert sum(t.startswith("global_load_lds_dwordx4") for t in body) == (wm * tm * 2 + wn * tn * 2) // waves, name
        assert sum(t.startswith("global_load_lds_dword ") for t in body) == (1 if qm == 2 else 0), name
