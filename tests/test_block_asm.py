"""Static checks on the compiled kernels of the block-scaled product and of the
token log probabilities (CPU only: hipcc cross-compiles gfx950 assembly): the
counted waits of the rings, each ahead of a barrier, the loads of a step that
they count, and no spills to scratch memory."""
import re

import pytest

from tests.test_linear_asm import main_loop
from tests.test_route_asm import compile_asm


def kernels_of(asm, prefix):
    out, name = {}, None
    for ln in asm.split("\n"):
        m = re.match(r"(_ZN\S*" + prefix + r"\S*):", ln)
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


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    made = {}

    def of(name):
        if name not in made:
            made[name] = compile_asm(name + ".hip", tmp_path_factory.mktemp("asm") / (name + ".s"))
        return made[name]
    return of


def inner_loop(code, least):
    """The shortest loop with at least that many matrix instructions."""
    at = {ln[:-1]: n for n, ln in enumerate(code) if ln.endswith(":")}
    spans = []
    for n, ln in enumerate(code):
        m = re.match(r"s_c?branch\S* (\.LBB\S+)", ln)
        if m and at.get(m.group(1), n) < n and sum(t.startswith("v_mfma") for t in code[at[m.group(1)]:n]) >= least:
            spans.append((n - at[m.group(1)], at[m.group(1)], n))
    return min(spans)[1:]


def waits(code):
    """(count, the next barrier, LDS read or matrix instruction) of every counted wait."""
    for n, ln in enumerate(code):
        m = re.fullmatch(r"s_waitcnt vmcnt\((\d+)\)", ln)
        if m:
            yield int(m.group(1)), next((t for t in code[n + 1:] if t.startswith(("s_barrier", "ds_read", "v_mfma"))), None)


def loads(code):
    return (sum(t.startswith("global_load_lds_dwordx4") for t in code), sum(t.startswith("global_load_lds_dword ") for t in code))


def test_tiles(asm):
    code = kernels_of(asm("linear_block_tile"), "k_block_tile")
    assert len(code) == 20
    for name, c in code.items():
        wm, wn, tm, tn, stages = (int(v) for v in re.search(r"ELi(\d)ELi(\d)ELi(\d)ELi(\d)ELi(\d)E", name).groups())
        x4 = (wm * tm + wn * tn) * 2 // (wm * wn)
        full = (stages - 1) * (x4 + 1)
        inner = full if stages == 2 else full - (x4 + 1)
        a, b = main_loop(c)
        assert loads(c[a:b]) == (x4, 1), name
        seen = [(n, t) for n, t in waits(c[:b]) if n >= 2]
        assert {n for n, _ in seen} == {full, inner} and all(t == "s_barrier" for _, t in seen), (name, seen)
        assert [n for n, _ in waits(c[a:b])] == [inner] * (2 if stages == 2 else 1), name


def test_big_tiles(asm):
    code = kernels_of(asm("linear_block_big"), "k_block_big")
    assert len(code) == 2
    for name, c in code.items():
        a, b = main_loop(c)
        assert loads(c[a:b]) == (8, 1) and sum(t.startswith("v_mfma") for t in c[a:b]) == 32, name
        assert list(waits(c[a:b])) == [(4, "s_barrier")], name
        assert sum(t == "s_barrier" for t in c[a:b]) == 2, name


def test_walked_tiles(asm):
    code = kernels_of(asm("linear_block_stream"), "k_block_stream")
    assert len(code) == 4
    for name, c in code.items():
        a, b = inner_loop(c, 16)
        assert loads(c[a:b]) == (8, 1) and sum(t.startswith("v_mfma") for t in c[a:b]) == 16, name
        assert list(waits(c[a:b])) == [(9, "s_barrier"), (6, "s_barrier")], name
        a, b = main_loop(c)
        ends = [t for t in waits(c[a:b]) if t[1] == "s_barrier" and t[0] > 0]  # 0: the compiler's, of a residual's loads
        assert ends == [(9, "s_barrier"), (6, "s_barrier")] * 3, (name, ends)  # the loop's step and the two behind it


@pytest.mark.parametrize("name,prefix,n", [("linear_block", "k_block_small", 26), ("linear_block_tile", "k_block_tile", 20),
                                           ("linear_block_big", "k_block_big", 2), ("linear_block_stream", "k_block_stream", 4),
                                           ("logprob", "k_logprob", 12)])
def test_no_scratch_and_no_flat_accesses(asm, name, prefix, n):
    code = kernels_of(asm(name), prefix)
    assert len(code) == n, sorted(code)
    for k, c in code.items():
        assert not [t for t in c if t.startswith(("scratch_", "flat_"))], k
