"""Every kernel form of the linear product: each tile shape with one K-step, two,
three and more, with a partial last step, with K split where the shape splits
it, gated and not, bf16 and fp32 outputs, whole 16-byte rows and ragged ones;
the few-token kernel with 16 gated columns a workgroup; and the calls whose
strides do not fit the tiles.

Which case takes which shape is the host's choice (linear_plan.h); a CPU test
compiles that choice and fails where a shape, or a form of it, has no case
here.  Tolerances as in test_gpu_linear."""
import ctypes
import os
import subprocess

import pytest

from tests.conftest import ROOT
from tests.gpu_util import DEV, need_gpu, say, torch
from tests.test_gpu_linear import U, encode, reference


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


# tokens, weight rows, bytes of a row: 256 x 256, 128 x 256, 128 x 128, 64 x 128 and 64 x 64 tiles of one to six
# K-steps, then K split (never with 256 x 256)
TILES = ([(1009, 8200, kb) for kb in (128, 208, 304, 656)] + [(413, 8200, kb) for kb in (128, 208, 304, 656)] +
         [(203, 8200, kb) for kb in (128, 208, 304, 656)] + [(131, 6008, kb) for kb in (128, 208, 304, 656)] +
         [(70, 200, kb) for kb in (128, 208, 304, 656)] +
         [(4100, 134, 14352), (4100, 136, 14336), (3001, 136, 8208), (1025, 520, 8208), (17, 72, 3024)])
# what a case is run with: gated, output, activation, odd width, strided rows
FORMS = [(False, "bf16", "none", False, True), (True, "f32", "silu", True, False), (True, "bf16", "gelu_tanh", False, False),
         (False, "f32", "gelu_erf", False, False), (False, "bf16", "relu", True, True)]
FMTS = ["bf16", "fp8", "mxfp8"]
# gated, 2049 to 4096 columns: tokens, columns, bytes of a row
FEW = [(1, 2100, 1040), (5, 3001, 2320), (16, 4096, 5008), (16, 2049, 3088), (2, 2056, 144)]


def columns(R, gated, odd):
    return (R // 2 if gated else R) - (1 if odd else 0)


def row_of(kb, fmt):
    """K of a row of about kb bytes in whole units of the type."""
    return {"bf16": kb // 16 * 8, "fp8": kb // 16 * 16, "mxfp8": (kb + 127) // 128 * 128}[fmt]


def row_bytes(K, fmt):
    return 2 * K if fmt == "bf16" else K


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """(shape, splits, steps a run) and the few-token choices, compiled from the library's own source."""
    d = tmp_path_factory.mktemp("plan")
    src = d / "plan.cpp"
    src.write_text('#include "%s"\n' % os.path.join(ROOT, "fp4_expert_ffn_amd", "csrc", "linear_plan.h") + """
extern "C" int tiles(int T, int R, int kb, int exact, int* splits) {
  const moe::TilePlan p = moe::plan_tiles(T, R, kb, exact != 0);
  *splits = p.splits;
  return p.shape;
}
extern "C" int few(int T, int R, int gated, int kb, int exact) { return moe::small_wins(T, R, gated != 0, kb, exact != 0); }
extern "C" int eight(int T, int N, int kb) { return moe::eight_columns(T, N, kb); }
""")
    out = str(d / "plan.so")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", str(src), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(out)


@pytest.mark.parametrize("fmt", FMTS)
def test_every_tile_form_has_a_case(plan, fmt):
    seen = set()
    for T, R, kb in TILES:
        K = row_of(kb, fmt)
        b = row_bytes(K, fmt)
        for gated, out, _, odd, _ in FORMS:
            N = columns(R, gated, odd)
            n = ctypes.c_int()
            exact = fmt != "bf16" and out == "f32"
            rows = 2 * N if gated else N
            assert not plan.few(T, rows, gated, b, exact)
            shape = plan.tiles(T, rows, b, exact, ctypes.byref(n))
            steps = min((b + 127) // 128, 4) if n.value == 1 else 0  # 4: more than the ring holds; 0: split
            seen.add((shape, exact, gated, steps))
    for shape in range(5):
        for exact in ((False, True) if fmt != "bf16" else (False,)):
            if shape == 0 and exact:
                continue  # fp32 outputs of 8-bit operands do not take it
            for gated in (False, True):
                for steps in ((1, 2, 3, 4) if shape == 0 else (0, 1, 2, 3, 4)):
                    assert (shape, exact, gated, steps) in seen, (shape, exact, gated, steps)


@pytest.mark.parametrize("fmt", FMTS)
def test_gated_few_token_cases_take_sixteen_columns(plan, fmt):
    waves = set()
    for T, N, kb in FEW:
        b = row_bytes(row_of(kb, fmt), fmt)
        assert plan.few(T, 2 * N, 1, b, 0) and not plan.eight(T, N, b)
        steps = (b + 127) // 128
        waves.add(16 if steps > 32 else (8 if steps > 16 else 4))
    assert waves == {4, 8, 16}


def rand(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g)


def wide(t, extra):
    """t as the left columns of wider rows whose other bytes are 0xFF (NaN in bf16 and E4M3)."""
    es = t.element_size()
    w = torch.full((t.shape[0], (t.shape[1] + extra) * es), 0xFF, dtype=torch.uint8, device=DEV)
    w[:, :t.shape[1] * es] = t.contiguous().view(torch.uint8)
    return w.view(t.dtype)[:, :t.shape[1]]


def run(m, T, N, K, fmt, gated, out, fn, strided, in_place=False):
    R = 2 * N if gated else N
    xq, xs, xv = encode(rand(T + K, T, K), fmt)
    wq, ws, wv = encode(rand(N + K + 1, R, K) / K ** 0.5, fmt)
    bias = rand(5, R) if strided or fn == "gelu_erf" else None
    res = None if out == "f32" and gated else rand(6, T, N).to(torch.bfloat16)
    pad = 64 if strided else 0  # whole 16-byte pieces
    kind = torch.bfloat16 if out == "bf16" else torch.float32
    big = torch.full((T + 2, N + pad // 8), 7.0, dtype=kind, device=DEV)
    o = big[:T, :N]
    rd = res
    if in_place:
        o.copy_(res)
        rd = o
    elif res is not None and strided:
        rd = wide(res, 8)
    a = m.linear_args(x=wide(xq, pad), w=wide(wq, pad), fmt=fmt, x_scale=xs, w_scale=ws, bias=bias, act=fn, gated=gated,
                      residual=rd, out=o)
    n = m.moe_linear_workspace_size(a)
    wsp = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device=DEV)
    a.workspace, a.workspace_bytes = wsp.data_ptr(), n
    say(f"linear T={T} N={N} K={K} {fmt} {fn} gated={gated} out={out} strided={strided} in_place={in_place} ws={n}")
    m.moe_linear(a)
    torch.cuda.synchronize()
    want, tol = reference(xv, wv, bias, fn, gated, res, N, K, fmt != "bf16" and out == "bf16")
    tol = tol + want.abs() * (2.0 ** -8 if out == "bf16" else U) + 1e-30
    bad = ~((o.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[:4], (o.double() - want).abs()[bad].max())
    assert torch.all(big[T:] == 7.0) and torch.all(big[:, N:] == 7.0)
    assert torch.all(wsp[n:] == 0xFF)
    return o


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,R,kb", TILES)
def test_linear_tile_forms(m, T, R, kb, fmt):
    need_gpu()
    for i, (gated, out, fn, odd, strided) in enumerate(FORMS):
        run(m, T, columns(R, gated, odd), row_of(kb, fmt), fmt, gated, out, fn, strided, in_place=i == 2)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,N,kb", FEW)
def test_linear_few_tokens_sixteen_gated_columns(m, T, N, kb, fmt):
    need_gpu()
    K = row_of(kb, fmt)
    run(m, T, N, K, fmt, True, "bf16", "silu", True)
    run(m, T, N, K, fmt, True, "f32", "gelu_tanh", False)
    run(m, T, N, K, fmt, True, "bf16", "none", False, in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["x", "w", "residual", "out"])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_strides_beyond_the_tiles(m, gated, which):
    """Rows 2^24 bytes (x, w) or 2^24 elements (residual, out) apart and more than 16 tokens: the few-token kernel,
    16 tokens a workgroup."""
    need_gpu()
    T, N, K = 20, 11, 136
    R = 2 * N if gated else N
    xq, _, xv = encode(rand(1, T, K), "bf16")
    wq, _, wv = encode(rand(2, R, K) / K ** 0.5, "bf16")
    res = rand(3, T, N).to(torch.bfloat16)

    def far(t, ld):
        w = torch.zeros((len(t) - 1) * ld + t.shape[1], dtype=t.dtype, device=DEV).as_strided(t.shape, (ld, 1))
        w.copy_(t)
        return w

    t = {"x": xq, "w": wq, "residual": res, "out": torch.zeros_like(res)}
    t[which] = far(t[which], 1 << (23 if which in "xw" else 24))
    a = m.linear_args(x=t["x"], w=t["w"], residual=t["residual"], act="silu", gated=gated, out=t["out"])
    say("linear, far rows of", which, gated)
    m.moe_linear(a)  # without a workspace: nothing here splits
    torch.cuda.synchronize()
    want, tol = reference(xv, wv, None, "silu", gated, res, N, K)
    assert torch.all((t["out"].double() - want).abs() <= tol + want.abs() * 2.0 ** -8 + 1e-30)
