"""The linear product with its epilogue, on the GPU through the C ABI, against
the formula in 64 bits.

Tolerances (u = 2^-24).  The products of bf16 or E4M3 operands are exact in
fp32; K of them are summed in fp32 in some order, so a sum is off by at most
(K + 16) u times the sum of their magnitudes S (the 16: joining partial sums,
scales and bias).  Every activation has a slope of at most 1.13 and is
evaluated within 2^-20 of its value; a gate multiplies.  The output adds half
a step of its type.

With bf16 outputs the products of E4M3 rows may run on the FP8 matrix
instructions, which add groups of 8 neighbouring products after cutting each
below 2^-13 of the exponent of the largest (checked by
test_fp8_instruction_cuts_small_products): at most 7 * 2^-13 times the
group's largest product a group."""
import math

import pytest

from tests.gpu_util import DEV, need_gpu, say, torch

U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float32)


def encode(v, fmt):
    """fp32 rows -> (codes, scales, the values they stand for in 64 bits)."""
    R, K = v.shape
    if fmt == "bf16":
        q = v.to(torch.bfloat16)
        return q, None, q.double()
    if fmt == "fp8":
        s = v.abs().amax(1) / 448.0
        q = (v / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        return q, s, q.double() * s.double()[:, None]
    b = v.view(R, K // 32, 32)
    e = torch.frexp(b.abs().amax(2))[1] - 9
    q = torch.ldexp(b, -e[:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    val = torch.ldexp(q.double(), e[:, :, None]).view(R, K)
    codes = (e + 127).to(torch.uint8).view(R, K // 128, 4).permute(1, 0, 2).contiguous()
    return q.view(R, K), codes, val


def act64(z, fn):
    if fn == "silu":
        return z * torch.sigmoid(z)
    if fn == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if fn == "gelu_erf":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    return z.clamp(min=0) if fn == "relu" else z


def reference(xv, wv, bias, fn, gated, res, N, K, fp8_sums=False):
    """(exact output, bound of the fp32 result's error) in 64 bits."""
    z, S = xv @ wv.t(), xv.abs() @ wv.abs().t()
    if bias is not None:
        z, S = z + bias.double(), S + bias.double().abs()
    dz = (K + 16) * U * S
    if fp8_sums:
        top = lambda v: v.abs().view(v.shape[0], K // 8, 8).amax(2)  # noqa: E731
        dz = dz + 7 * 2.0 ** -13 * (top(xv) @ top(wv).t())
    a = act64(z[:, :N], fn)
    da = 1.13 * dz[:, :N] + 2.0 ** -20 * a.abs()
    if gated:
        up, du = z[:, N:], dz[:, N:]
        a, da = a * up, da * up.abs() + a.abs() * du + da * du
    if res is not None:
        a = a + res.double()
    return a, da + 4 * U * a.abs()


def _wide(t, extra, fill):
    """t as the left columns of a wider device tensor whose other bytes are `fill`."""
    es = t.element_size()
    w = torch.full((t.shape[0], (t.shape[1] + extra) * es), fill, dtype=torch.uint8, device=DEV)
    w[:, :t.shape[1] * es] = t.contiguous().view(torch.uint8).to(DEV)
    return w.view(t.dtype)[:, :t.shape[1]]


def run_case(m, T, N, K, fmt, fn="none", gated=False, bias=False, res=False, out="bf16", strided=False, ws_fill=0xFF):
    R = 2 * N if gated else N
    xq, xs, xv = encode(_rand(T * 7 + K, T, K), fmt)
    wq, ws, wv = encode(_rand(N * 3 + K + 1, R, K) / math.sqrt(K), fmt)
    b = _rand(5, R) if bias else None
    r = _rand(6, T, N).to(torch.bfloat16) if res else None
    pad = 128 if strided else 0
    xd = _wide(xq, pad, 0xFF)  # 0xFF: NaN in bf16 and E4M3
    wd = _wide(wq, pad, 0xFF)
    od = torch.full((T + 3, N + (5 if strided else 0)), 7.0, device=DEV,
                    dtype=torch.bfloat16 if out == "bf16" else torch.float32)
    rd = None
    if r is not None:
        rd = torch.full((T, N + (3 if strided else 0)), 9.0, device=DEV, dtype=torch.bfloat16)[:, :N]
        rd.copy_(r)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    a = m.linear_args(x=xd, w=wd, fmt=fmt, x_scale=dev(xs), w_scale=dev(ws), bias=dev(b), act=fn, gated=gated,
                      residual=rd, out=od[:T, :N])
    n = m.moe_linear_workspace_size(a)
    wsp = torch.full((n + 256,), ws_fill, dtype=torch.uint8, device=DEV)
    a.workspace, a.workspace_bytes = wsp.data_ptr(), n
    say(f"linear T={T} N={N} K={K} {fmt} {fn} gated={gated} bias={bias} res={res} out={out} strided={strided} ws={n}")
    m.moe_linear(a)
    torch.cuda.synchronize()
    got = od[:T, :N].cpu().double()
    want, tol = reference(xv, wv, b, fn, gated, r, N, K, fmt != "bf16" and out == "bf16")
    tol = tol + want.abs() * (2.0 ** -8 if out == "bf16" else U) + 1e-30
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), (got - want).abs()[bad].max(), torch.nonzero(bad)[:4])
    assert torch.all(od[T:] == 7.0) and torch.all(od[:, N:] == 7.0)
    assert torch.all(wsp[n:] == ws_fill)  # nothing behind the workspace's stated size is written


SMALL = [(1, 16, 128), (1, 1, 128), (2, 17, 256), (16, 64, 384), (15, 33, 1024), (17, 48, 128), (5, 130, 2048),
         (1, 256, 7168)]


# few tokens whose rows are too long for one CU to stream: the tiles, K split
@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K,fmt,gated", [
    (1, 40, 8192, "bf16", True), (1, 33, 15000, "bf16", False), (16, 70, 7168, "bf16", False),
    (2, 64, 14336, "fp8", True), (16, 100, 16000, "fp8", False), (13, 72, 8192, "mxfp8", True),
    (16, 4112, 7168, "bf16", False)])
def test_linear_few_tokens_long_rows(m, T, N, K, fmt, gated):
    need_gpu()
    n = m.moe_linear_workspace_size(_ok(m, T=T, N=N, K=K, fmt=fmt, gated=gated))
    assert n > 0  # split
    for strided in (False, True):
        run_case(m, T, N, K, fmt, fn="silu" if gated else "none", gated=gated, bias=True, res=strided, strided=strided)
    # fp32 outputs of 8-bit operands: the few-token form at any length
    run_case(m, T, N, K, fmt, gated=gated, out="f32")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8"])
@pytest.mark.parametrize("T,N,K", SMALL)
def test_linear_small(m, T, N, K, fmt):
    need_gpu()
    run_case(m, T, N, K, fmt, bias=T % 2 == 1, res=N % 2 == 0, strided=T % 3 != 0)
    run_case(m, T, N, K, fmt, fn="silu", gated=True, bias=N % 2 == 0, out="f32", strided=T % 2 == 0)


LARGE = [(33, 256, 128), (64, 512, 512), (65, 100, 256), (128, 128, 128), (129, 257, 384), (200, 2048, 2048),
         (257, 640, 1152), (513, 1000, 640), (1024, 768, 2048), (300, 16, 7168)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8"])
@pytest.mark.parametrize("T,N,K", LARGE)
def test_linear_large(m, T, N, K, fmt):
    need_gpu()
    run_case(m, T, N, K, fmt, bias=T % 2 == 0, res=T % 2 == 1, strided=N % 3 == 1)
    run_case(m, T, N, K, fmt, fn="silu", gated=True, res=T % 2 == 0, out="f32" if N % 3 else "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 40, 300])
@pytest.mark.parametrize("K,fmt", [(8, "bf16"), (72, "bf16"), (136, "bf16"), (776, "bf16"), (1000, "bf16"), (16, "fp8"),
                                   (48, "fp8"), (144, "fp8"), (1008, "fp8")])
def test_linear_partial_steps(m, T, K, fmt):
    """Rows that end inside a K-step; NaN bytes follow them."""
    need_gpu()
    run_case(m, T, 77, K, fmt, fn="gelu_tanh", bias=True, strided=True)
    run_case(m, T, 40, K, fmt, fn="relu", gated=True, strided=True)


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["none", "silu", "gelu_tanh", "gelu_erf", "relu"])
@pytest.mark.parametrize("T", [4, 260])
def test_linear_activations(m, fn, T):
    need_gpu()
    run_case(m, T, 96, 256, "bf16", fn=fn, bias=True, res=True, out="f32")
    run_case(m, T, 96, 256, "fp8", fn=fn, gated=True, bias=True, res=True)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8"])
@pytest.mark.parametrize("T", [3, 270])
def test_linear_residual_in_place_and_special_values(m, fmt, T):
    """out is the residual; NaN and infinity stay in their row and column."""
    need_gpu()
    N, K = 130, 384
    xq, xs, xv = encode(_rand(1, T, K), fmt)
    wq, ws, wv = encode(_rand(2, N, K), fmt)
    nan = float("nan")
    if fmt == "bf16":
        xq[1, K - 1] = float("inf")
    else:
        xq.view(torch.uint8)[1, K - 1] = 0x7F
    wq.view(torch.uint8)[7, 3 * wq.element_size():4 * wq.element_size()] = 0xFF
    r = _rand(3, T, N).to(torch.bfloat16)
    out = r.to(DEV)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    a = m.linear_args(x=dev(xq), w=dev(wq), fmt=fmt, x_scale=dev(xs), w_scale=dev(ws), residual=out, out=out)
    n = m.moe_linear_workspace_size(a)
    wsp = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    a.workspace, a.workspace_bytes = wsp.data_ptr(), n
    say("linear in place, special values", fmt, T)
    m.moe_linear(a)
    torch.cuda.synchronize()
    got = out.cpu().double()
    want, tol = reference(xv, wv, None, "none", False, r, N, K, fmt != "bf16")
    ok = torch.ones(T, N, dtype=torch.bool)
    ok[1], ok[:, 7] = False, False
    assert torch.all(((got - want).abs() <= tol + want.abs() * 2.0 ** -8)[ok])
    assert torch.isnan(got[:, 7]).all()
    if fmt == "bf16":
        up = wq.float()[:, K - 1] > 0
        up[7] = False  # its sum holds a NaN
        assert torch.isinf(got[1, up]).all()
    else:
        assert torch.isnan(got[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 300])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_mxfp8_far_scales(m, T, out):
    """Block scales of x and w far from 1 and from each other; their products are ordinary."""
    need_gpu()
    N, K = 64, 512
    xq, xs, xv = encode(_rand(21, T, K), "mxfp8")
    wq, ws, wv = encode(_rand(22, N, K), "mxfp8")
    for kt, e in ((0, 90), (1, -90), (2, 110), (3, -112)):  # K-tile kt: x scaled by 2^e, w by 2^-e
        xs[kt], ws[kt] = (xs[kt].int() + e).to(torch.uint8), (ws[kt].int() - e).to(torch.uint8)
    o = torch.empty((T, N), dtype=torch.bfloat16 if out == "bf16" else torch.float32, device=DEV)
    a = m.linear_args(x=xq.to(DEV), w=wq.to(DEV), fmt="mxfp8", x_scale=xs.to(DEV), w_scale=ws.to(DEV), out=o)
    n = m.moe_linear_workspace_size(a)
    wsp = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    a.workspace, a.workspace_bytes = wsp.data_ptr(), n
    say("linear mxfp8, far scales", T, out)
    m.moe_linear(a)
    torch.cuda.synchronize()
    want, tol = reference(xv, wv, None, "none", False, None, N, K, out == "bf16")
    assert torch.all((o.cpu().double() - want).abs() <= tol + want.abs() * (2.0 ** -8 if out == "bf16" else U))


@pytest.mark.gpu
def test_fp8_instruction_cuts_small_products(m):
    """The rule behind the tolerance of bf16 outputs: of 8 neighbouring products, two of 2^16 that cancel
    and a small one, what is left is the small one within 2^-13 of 2^16; in a group of its own it is whole."""
    need_gpu()
    T, N, K = 64, 64, 128
    small = torch.tensor([2.0 ** (i % 10 - 4) for i in range(T)])
    for at, off in ((2, 2.0 ** 3), (7, 2.0 ** 3), (8, 0.0), (100, 0.0)):
        x, w = torch.zeros(T, K), torch.zeros(N, K)
        x[:, :2], w[:, 0], w[:, 1] = 256.0, 256.0, -256.0
        x[:, at], w[:, at] = small, 2.0
        ones = torch.ones(64, device=DEV)
        o = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
        a = m.linear_args(x=x.to(torch.float8_e4m3fn).to(DEV), w=w.to(torch.float8_e4m3fn).to(DEV), fmt="fp8",
                          x_scale=ones, w_scale=ones, out=o)
        n = m.moe_linear_workspace_size(a)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        a.workspace, a.workspace_bytes = ws.data_ptr(), n
        say("fp8 products, small one at", at)
        m.moe_linear(a)
        torch.cuda.synchronize()
        assert torch.all((o.cpu().float() - 2 * small[:, None]).abs() <= off)


@pytest.mark.gpu
def test_linear_few_tokens_captured(m):
    """A split product of few tokens, replayed with new inputs and a workspace filled in between."""
    need_gpu()
    T, N, K = 3, 80, 8192
    x, w = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV), _rand(1, N, K).to(torch.bfloat16).to(DEV)
    outs = [torch.empty((T, N), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    args = []
    for o in outs:
        a = m.linear_args(x=x, w=w, out=o)
        n = m.moe_linear_workspace_size(a)
        assert n > 0
        a.buf = torch.empty(n, dtype=torch.uint8, device=DEV)
        a.workspace, a.workspace_bytes = a.buf.data_ptr(), n
        args.append(a)
    say("captured split product of few tokens")
    m.moe_linear(args[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_linear(args[0])
    for seed in range(3):
        x.copy_(_rand(20 + seed, T, K).to(torch.bfloat16))
        m.moe_linear(args[1])
        for fill in (0xFF, 0x00):
            args[0].buf.fill_(fill)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[0], outs[1])


def _ok(L, **kw):
    a = dict(T=4, N=32, K=128, x=0x10000, w=0x20000, out=0x30000)
    a.update(kw)
    return L.linear_args(**a)


@pytest.mark.parametrize("kw,msg", [
    (dict(T=-1), "bad sizes"), (dict(N=0), "bad sizes"), (dict(K=0), "bad sizes"), (dict(T=1 << 24), "bad sizes"),
    (dict(K=132), "multiple of 8"), (dict(K=136, fmt="fp8"), "multiple of 16"), (dict(K=192, fmt="mxfp8"), "multiple of 128"),
    (dict(fmt="fp8"), "null"), (dict(fmt="mxfp8", x_scale=0x40000), "null"), (dict(act=9), "fn"), (dict(fmt=5), "qmode"),
    (dict(x=0x10008), "16-byte"), (dict(w=0x20004), "16-byte"), (dict(out=0x30001), "misaligned"),
    (dict(out=0x30002, out_f32=True), "misaligned"), (dict(bias=0x50002), "misaligned"),
])
def test_linear_refusals(m, kw, msg):
    with pytest.raises(m.MoeError) as e:
        m.moe_linear(_ok(m, **kw), stream=0)
    assert e.value.status == 1 and msg in str(e.value)


def test_linear_refuses_bad_strides_and_nulls(m):
    for field, ld in (("ldx", 120), ("ldx", 132), ("ldw", 64), ("ldw", 129), ("ldr", 31), ("ldo", 8)):
        a = _ok(m)
        setattr(a, field, ld)
        with pytest.raises(m.MoeError) as e:
            m.moe_linear(a, stream=0)
        assert "stride" in str(e.value)
    for field in ("x", "w", "out"):
        a = _ok(m)
        setattr(a, field, None)
        with pytest.raises(m.MoeError) as e:
            m.moe_linear(a, stream=0)
        assert "null" in str(e.value)
    assert m.moe_linear(_ok(m, T=0), stream=0) is None


def test_linear_workspace(m):
    """A call that splits K says so in its workspace size, and refuses a smaller or misaligned one."""
    assert m.moe_linear_workspace_size(_ok(m, T=1, N=4096, K=8192)) == 0
    a = _ok(m, T=64, N=64, K=8192)
    n = m.moe_linear_workspace_size(a)
    assert n >= 2 * 64 * 64 * 4
    for p, size, status, msg in ((None, n, 4, "workspace"), (0x40000, n - 1, 4, "workspace"), (0x40008, n, 1, "16-byte")):
        a.workspace, a.workspace_bytes = p, size
        with pytest.raises(m.MoeError) as e:
            m.moe_linear(a, stream=0)
        assert e.value.status == status and msg in str(e.value)
    assert m.moe_linear_workspace_size(_ok(m, T=64, N=64, K=8192, out_f32=True, fmt="fp8")) > 0


def test_linear_args_refuse_tensors(m):
    x, w = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(32, 128, dtype=torch.bfloat16)
    o = torch.zeros(4, 32, dtype=torch.bfloat16)
    for kw, msg in ((dict(x=x, w=w[:, :64], out=o), "not on a GPU"), (dict(x=x[0], w=w, out=o), "two dimensions"),
                    (dict(x=x.float(), w=w, out=o), "float32")):
        with pytest.raises(m.MoeError) as e:
            m.linear_args(**kw)
        assert msg in str(e.value)
