"""Every kernel form of the block-scaled product, dense and over routed experts:
each tile shape with one K-step, two, three and more, with K split where the
shape splits it, gated and not, bf16 and fp32 outputs; tiles walked one after
the other, several a workgroup; the few-row kernel with every number of waves;
and calls whose strides do not fit the tiles.

Which case takes which shape is the host's choice (linear_block_plan.h); a CPU
test compiles that choice and fails where a shape, or a form of it, has no
case here.  Tolerances as in test_gpu_fp8_block."""
import ctypes
import os
import subprocess

import pytest

from tests.conftest import ROOT
from tests.gpu_util import DEV, need_gpu, say, torch
from tests.test_gpu_fp8_block import FEW, _rand, block_rows, block_weights, run_linear
from tests.test_gpu_grouped import expert_weights, run_grouped
from tests.test_gpu_linear import reference


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


BIG, STREAM = 0, 5
STEPS = (128, 256, 384, 640)
# tokens, columns, K: the shape and the K-steps that each is here for (steps 0: K split)
DENSE = ([(513, 8200, K, True) for K in STEPS] + [(3001, 4104, K, False) for K in STEPS] +       # 256 x 256
         [(413, 8200, K, True) for K in STEPS[1:]] + [(2050, 4100, K, False) for K in STEPS[1:]] +  # walked
         [(2050, 1000, K, False) for K in STEPS] + [(4100, 200, K, True) for K in STEPS] +       # 128 x 128
         [(3001, 136, 8192, False), (3001, 72, 8192, True)] +
         [(4100, 200, K, False) for K in STEPS] + [(4100, 100, K, True) for K in STEPS] +        # 64 x 128
         [(17, 4104, 4096, False), (19, 2056, 4096, True)] +
         [(70, 200, K, False) for K in STEPS] + [(70, 99, K, True) for K in STEPS] +             # 64 x 64
         [(17, 72, 4096, False), (33, 40, 4096, True)])


def counts_of(kind):
    """Rows of the experts of a grouped case."""
    return {"few": [1, 0, 2, 1, 1, 0, 1, 1], "some": [5, 0, 9, 1, 3, 0, 4, 2], "many": [100, 3, 129, 0, 1, 260, 128, 31],
            "long": [400 - 17 * (e % 5) - (e == 3) * 300 for e in range(24)]}[kind]


# rows, columns, K, gated: the few-row kernel with 4 and 8 waves, 64 x 128 tiles, 128 x 128 a workgroup, walked
GROUPED = ([("few", 200, K, g) for K in (128, 640, 4096, 4224) for g in (False, True)] +
           [("some", 136, K, g) for K in STEPS for g in (False, True)] +
           [("many", 200, K, g) for K in STEPS for g in (False, True)] + [("long", 4100, 256, False), ("long", 2049, 384, True)])


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src = d / "plan.cpp"
    src.write_text('#include "%s"\n' % os.path.join(ROOT, "fp4_expert_ffn_amd", "csrc", "linear_block_plan.h") + """
extern "C" int small(int T, int R, int gated, int K, int exact) { return moe::block_small_wins(T, R, gated != 0, K, exact != 0); }
extern "C" int eight(int T, int N, int K) { return moe::eight_columns(T, N, K); }
extern "C" int dense(int T, int N, int gated, int K, int exact, int* splits) {
  const moe::TilePlan p = moe::plan_block_tiles(T, N, gated != 0, K, exact != 0);
  *splits = p.splits;
  return p.shape;
}
extern "C" int grouped_small(int T, int E) { return moe::grouped_small_wins(T, E); }
extern "C" int grouped(int T, int E, int N, int gated, int K, int exact, long long most) {
  return moe::plan_grouped_tiles(T, E, N, gated != 0, K, exact != 0, most).shape;
}
""")
    out = str(d / "plan.so")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", str(src), "-o", out], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(out)


def test_every_dense_form_has_a_case(plan):
    seen = set()
    for T, N, K, gated in DENSE:
        for exact in (False, True):
            assert not plan.small(T, 2 * N if gated else N, gated, K, exact)
            n = ctypes.c_int()
            shape = plan.dense(T, N, gated, K, exact, ctypes.byref(n))
            seen.add((shape, exact, gated, min(K // 128, 4) if n.value == 1 else 0))
    for gated in (False, True):
        want = [(BIG, False, s) for s in (1, 2, 3, 4)] + [(STREAM, False, s) for s in (2, 3, 4)]
        want += [(shape, exact, s) for shape in (2, 3, 4) for exact in (False, True) for s in range(5)]
        for shape, exact, s in want:
            assert (shape, exact, gated, s) in seen, (shape, exact, gated, s)


def test_every_few_token_form_has_a_case(plan):
    """4, 8 and 16 waves, with 8 and with 16 gated columns a workgroup."""
    seen = set()
    for T, N, K in FEW + FEW_WIDE:
        steps = K // 128
        assert plan.small(T, 2 * N, 1, K, 0) or plan.small(T, N, 0, K, 0)
        seen.add((16 if steps > 32 else (8 if steps > 16 else 4), bool(plan.eight(T, N, K))))
    assert seen == {(w, e) for w in (4, 8, 16) for e in (False, True)}


def test_every_grouped_form_has_a_case(plan):
    seen, tiles = set(), 0
    for kind, N, K, gated in GROUPED:
        counts = counts_of(kind)
        T, E = sum(counts), len(counts)
        most = min(T, E) + (T - min(T, E)) // 128
        for exact in (False, True):
            if plan.grouped_small(T, E):
                seen.add(("small", exact, gated, 8 if K // 128 >= 32 else 4))
                continue
            shape = plan.grouped(T, E, N, gated, K, exact, ctypes.c_longlong(most))
            seen.add((shape, exact, gated, min(K // 128, 4)))
            if shape == STREAM:
                tiles = max(tiles, sum((c + 127) // 128 for c in counts) * ((N + 63) // 64 if gated else (N + 127) // 128))
    for gated in (False, True):
        want = [("small", e, w) for e in (False, True) for w in (4, 8)] + [(3, e, s) for e in (False, True) for s in (1, 2, 3, 4)]
        want += [(2, False, 1)] + [(2, True, s) for s in (1, 2, 3, 4)] + [(STREAM, False, s) for s in (2, 3, 4)]
        for shape, exact, s in want:
            assert (shape, exact, gated, s) in seen, (shape, exact, gated, s)
    assert tiles > 4 * 512  # more tiles a workgroup than it holds row numbers of


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K,gated", DENSE)
def test_dense_forms(m, T, N, K, gated):
    need_gpu()
    run_linear(m, T, N, K, "silu" if gated else "none", gated=gated, bias=True, strided=N % 2 == 0)
    run_linear(m, T, N, K, "relu", gated=gated, res=K == 256, out="f32")
    if K == 256:
        run_linear(m, T, N, K, "gelu_tanh", gated=gated, res=True, in_place=True)


# gated: 16 columns a workgroup
FEW_WIDE = [(1, 2100, 1024), (16, 2064, 2304), (5, 2100, 4224), (2, 4097, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", FEW_WIDE)
def test_few_tokens_wide(m, T, N, K):
    need_gpu()
    run_linear(m, T, N, K, "silu", gated=True, bias=True)
    run_linear(m, T, N, K, "gelu_erf", gated=True, out="f32", strided=True)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,N,K,gated", GROUPED)
def test_grouped_forms(m, kind, N, K, gated):
    need_gpu()
    counts = counts_of(kind)
    E = len(counts)
    run_grouped(m, counts, N, K, gated=gated, k=4, gather=True, extra=3, slots=[(e * 3) % E for e in range(E)], bias=True)
    if kind != "long":
        run_grouped(m, counts, N, K, gated=gated, out="f32", k=2, gather=K % 256 == 0)
    if kind == "many":
        run_grouped(m, counts, N, K, gated=gated, strided=True)


@pytest.mark.gpu
def test_strides_beyond_the_tiles(m):
    """Rows 2^24 bytes apart: more than the tiles' offsets hold, so the few-row kernel takes the batch."""
    need_gpu()
    T, N, K, far = 70, 40, 256, 1 << 24
    xq, xs, xv = block_rows(_rand(1, T, K))
    wq, ws, wv = block_weights(_rand(2, N, K) / 16)
    x = torch.empty(T * far, dtype=torch.uint8, device=DEV).view(T, far)[:, :K].view(torch.float8_e4m3fn)
    x.copy_(xq)
    w = torch.empty(N * far, dtype=torch.uint8, device=DEV).view(N, far)[:, :K].view(torch.float8_e4m3fn)
    w.copy_(wq)
    xs, ws = xs.to(DEV), ws.to(DEV)
    want, tol = reference(xv.to(DEV), wv.to(DEV), None, "none", False, None, N, K, True)
    near = lambda got: bool(((got.double() - want).abs() <= tol + want.abs() * 2.0 ** -8 + 1e-30).all())  # noqa: E731
    for xx, ww in ((x, wq.to(DEV)), (xq.to(DEV), w)):
        out = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
        a = m.linear_args(x=xx, w=ww, fmt="fp8_block", x_scale=xs, w_scale=ws, out=out)
        n = m.moe_linear_workspace_size(a)
        wsp = torch.empty(n + 16, dtype=torch.uint8, device=DEV)
        a.workspace, a.workspace_bytes = wsp.data_ptr(), n
        say("linear, block scales, far rows")
        m.moe_linear(a)
        torch.cuda.synchronize()
        assert near(out)
    out = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 50, T], dtype=torch.int32, device=DEV)
    say("grouped, far rows")
    m.moe_linear_grouped(m.grouped_args(x=x, x_scale=xs, w=wq.to(DEV)[None], w_scale=ws[None],
                                        offsets=off, slot_of_expert=torch.zeros(2, dtype=torch.int32, device=DEV), out=out))
    torch.cuda.synchronize()
    assert near(out)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,N,K", [(6, 8, 136, 512), (40, 8, 200, 384), (1500, 8, 264, 512)])
def test_grouped_captured_with_other_routes(m, T, E, N, K):
    """One captured call, replayed with other offsets, rows and x each time (the experts' shares are known on the
    device alone), with eager calls and a side stream's between the replays: each equals the formula, and the rows
    behind the last expert's are left as they were."""
    need_gpu()
    wq, ws, wv = expert_weights(E, 2 * N, K, 2)
    xq, xs, xv = block_rows(_rand(T, T, K))
    x, s, w, wsd = (torch.empty_like(xq, device=DEV), torch.empty_like(xs, device=DEV), wq.to(DEV), ws.to(DEV))
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    rows = torch.zeros(T, dtype=torch.int32, device=DEV)
    out = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    a = m.grouped_args(x=x, x_scale=s, w=w, w_scale=wsd, offsets=off, rows=rows, rows_div=1, act="silu", gated=True, out=out)
    say("grouped, captured", T, E, N, K)

    def load(seed):
        g = torch.Generator().manual_seed(seed)
        n = T - seed % 3  # routed rows
        which = torch.sort(torch.randint(E, (n,), generator=g) if seed % 2 else torch.full((n,), seed % E))[0]
        o = torch.searchsorted(which, torch.arange(E + 1))
        p = torch.randperm(T, generator=g)
        x.copy_(xq)
        s.copy_(xs)
        off.copy_(o.int())
        rows.copy_(p.int())
        out.fill_(7.0)
        want, tol = torch.full((T, N), 7.0, dtype=torch.double), torch.zeros((T, N), dtype=torch.double)
        for e in range(E):
            lo, hi = int(o[e]), int(o[e + 1])
            if lo < hi:
                v, t = reference(xv[p[lo:hi]], wv[e], None, "silu", True, None, N, K, True)
                want[lo:hi], tol[lo:hi] = v, t + v.abs() * 2.0 ** -8 + 1e-30
        return want, tol

    def check(want, tol):
        torch.cuda.synchronize()
        assert torch.all((out.cpu().double() - want).abs() <= tol)

    want = load(1)
    m.moe_linear_grouped(a)
    check(*want)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        m.moe_linear_grouped(a, torch.cuda.current_stream())
    for seed in (2, 3, 4, 5):
        want = load(seed)
        torch.cuda.synchronize()
        g.replay()
        check(*want)
        want = load(seed + 10)
        side.wait_stream(torch.cuda.current_stream())
        m.moe_linear_grouped(a, side)
        check(*want)
