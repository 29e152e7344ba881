"""8-bit rows with one scale per 128 columns, and their product with weights
that have one scale per 128 x 128 block, on the GPU through the C ABI, against
the formulas in 64 bits.

Rows: the scale is fp32(amax / 448), the code the fp32 quotient rounded to
E4M3, bit for bit where the encoding reads bf16 values; behind the norm the
values themselves are within 2^-19 (see test_gpu_norm).

Product (u = 2^-24): the sum over a block of 128 columns is off by at most
128 u times the sum of magnitudes, the scales' product and the addition to the
running sum add 2 u each, K / 128 blocks and up to 16 waves or runs are added:
below (K + 16) u of the sum of magnitudes, with the cut of the FP8 instruction
where the output is bf16 (see test_gpu_linear)."""
import math

import pytest

from tests.gpu_util import DEV, need_gpu, say, torch
from tests.test_gpu_linear import U, _wide, reference
from tests.test_gpu_norm import F32, _padded, _reference


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float32)


def block_rows(v):
    """fp32 rows -> (codes, scales [K/128, rows], the values they stand for in 64 bits)."""
    T, K = v.shape
    b = v.view(T, K // 128, 128)
    s = torch.clamp(b.abs().amax(2) / 448.0, min=2.0 ** -126)
    q = (b / s[:, :, None]).to(torch.float8_e4m3fn)
    val = (q.double() * s.double()[:, :, None]).view(T, K)
    return q.view(T, K), s.t().contiguous(), val


def block_weights(v, parts=1):
    """fp32 [parts * N, K] -> (codes, scales [parts * ceil(N/128), K/128], values in 64 bits); a part's row blocks
    are counted from its own first row."""
    R, K = v.shape
    N = R // parts
    codes, scales, vals = [], [], []
    for p in range(parts):
        for n0 in range(0, N, 128):
            b = v[p * N + n0: p * N + min(n0 + 128, N)]
            b = b.view(len(b), K // 128, 128)
            s = torch.clamp(b.abs().amax(dim=(0, 2)) / 448.0, min=2.0 ** -126)
            q = (b / s[None, :, None]).to(torch.float8_e4m3fn)
            codes.append(q.view(-1, K))
            scales.append(s)
            vals.append((q.double() * s.double()[None, :, None]).view(-1, K))
    return torch.cat([c.view(torch.uint8) for c in codes]).view(torch.float8_e4m3fn), torch.stack(scales), torch.cat(vals)


# ------------------------------------------------------------------ rows

def check_block_codes(y, q, scale, rel):
    """q, scale (device) against exact rows y (64 bits, CPU) that the kernel knows within `rel`."""
    T, H = y.shape
    s = scale.cpu().double().t()
    want = torch.clamp(y.view(T, H // 128, 128).abs().amax(2) / 448.0, min=2.0 ** -126)
    assert torch.all((s - want).abs() <= want * (rel + 2.0 ** -23))
    sw = s.repeat_interleave(128, 1)
    ref = torch.clamp(y / sw, -448.0, 448.0)
    off = (q.cpu().view(torch.float8_e4m3fn).double() - ref).abs()
    assert torch.all(off <= torch.clamp(ref.abs() * 2.0 ** -4, min=2.0 ** -10) + ref.abs() * (rel + 2.0 ** -23)), off.max()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,res,weight,out", [
    (1, 128, "none", "bf16", False), (3, 256, "bf16", "f32", True), (5, 384, "f32", "bf16", True),
    (9, 1024, "none", "none", True), (130, 2048, "bf16", "bf16", True), (4, 2176, "f32", "f32", False),
    (1, 7168, "bf16", "bf16", True), (33, 7168, "none", "f32", True), (2, 8320, "bf16", "bf16", True),
    (2, 16512, "f32", "bf16", True), (2, 32768, "bf16", "f32", False)])
def test_norm_block_rows(m, T, H, res, weight, out):
    need_gpu()
    x = _rand(T + H, T, H).to(torch.bfloat16)
    x[:, H // 3] *= 50.0
    kinds = {"bf16": torch.bfloat16, "f32": torch.float32}
    r = None if res == "none" else (_rand(7, T, H) * 3.0).to(kinds[res])
    w = None if weight == "none" else (1 + 0.3 * _rand(9, H)).to(kinds[weight])
    xd = _padded(x, 8, float("nan"))
    rd = None if r is None else _padded(r, 24, float("nan"))
    ro = None if r is None else torch.full_like(rd, 7.0)
    yd = torch.full((T, H + 16), 7.0, dtype=torch.bfloat16, device=DEV) if out else None
    qd = torch.full((T + 1, H + 8), 0x55, dtype=torch.uint8, device=DEV)
    sd = torch.full((H // 128 * T + 8,), 7.0, device=DEV)
    cut = lambda t: None if t is None else t[:T, :H]  # noqa: E731
    say(f"norm, block rows T={T} H={H} residual={res} weight={weight} out={out}")
    m.moe_rmsnorm(m.norm_args(x=cut(xd), weight=None if w is None else w.to(DEV), eps=1e-5, residual=cut(rd),
                              residual_out=cut(ro), out=cut(yd), q=cut(qd), q_scale=sd[:H // 128 * T].view(H // 128, T),
                              qmode="fp8_block"))
    torch.cuda.synchronize()
    er, ey = _reference(x, r, w, 1e-5)
    if r is not None:
        assert torch.all((cut(ro).cpu().double() - er).abs() <= er.abs() * (2.0 ** -8 + F32 if res == "bf16" else F32))
    if out:
        assert torch.all((cut(yd).cpu().double() - ey).abs() <= ey.abs() * (2.0 ** -8 + F32))
    check_block_codes(ey, cut(qd).contiguous(), sd[:H // 128 * T].view(H // 128, T), F32)
    assert torch.all(qd[:T, H:] == 0x55) and torch.all(qd[T:] == 0x55) and torch.all(sd[H // 128 * T:] == 7.0)


def rows_of_every_kind(T, K):
    """bf16 rows with blocks of very different sizes, one of zeros and one of subnormals."""
    x = _rand(T * 3 + K, T, K)
    b = x.view(T, K // 128, 128)
    b *= torch.exp2(((torch.arange(T)[:, None] * 7 + torch.arange(K // 128)[None] * 5) % 61 - 30).float())[:, :, None]
    if T > 1:
        b[1, 0] = 0.0
        b[T - 1, K // 128 - 1] = _rand(1, 128) * 2.0 ** -130
    return x.to(torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,pad", [(1, 128, 0), (3, 256, 8), (17, 640, 16), (300, 768, 0), (1000, 2048, 0), (5, 7168, 8),
                                     (2, 32768, 0)])
def test_quantize_block_rows_exactly(m, T, K, pad):
    need_gpu()
    x = rows_of_every_kind(T, K)
    xd = _padded(x, pad, float("nan"))[:, :K]
    q = torch.full((T, K), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((K // 128, T), 7.0, device=DEV)
    say("quantize, block rows", T, K, pad)
    m.moe_quantize_fp8(xd, T, K, "fp8_block", q, s)
    torch.cuda.synchronize()
    want, ws, _ = block_rows(x.float())
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(q.cpu(), want.view(torch.uint8))


@pytest.mark.gpu
def test_quantize_block_rows_not_finite(m):
    """NaN stays NaN and counts for no maximum; with an infinite value its block's scale is infinite, that value's
    code NaN and the others 0; other blocks are not touched by it."""
    need_gpu()
    x = _rand(3, 2, 384).to(torch.bfloat16)
    x[0, 5], x[0, 130], x[1, 260] = float("nan"), float("inf"), -float("inf")
    q, s = torch.empty((2, 384), dtype=torch.uint8, device=DEV), torch.empty((3, 2), device=DEV)
    say("quantize, block rows, not finite")
    m.moe_quantize_fp8(x.to(DEV), 2, 384, "fp8_block", q, s)
    torch.cuda.synchronize()
    clean = x.clone()
    clean[0, 5] = 0.0
    want, ws, _ = block_rows(clean.float())
    got, gs, want = q.cpu(), s.cpu(), want.view(torch.uint8)
    assert gs[1, 0] == float("inf") and gs[2, 1] == float("inf")
    fine = torch.ones(2, 384, dtype=torch.bool)
    fine[0, 128:256] = fine[1, 256:] = fine[0, 5] = False
    assert torch.equal(got[fine], want[fine]) and gs[0, 0] == ws[0, 0] and gs[1, 1] == ws[1, 1]
    assert (got[0, 5] & 0x7F) == 0x7F and (got[0, 130] & 0x7F) == 0x7F and (got[1, 260] & 0x7F) == 0x7F
    zero = (got & 0x7F) == 0
    assert zero[0, 128:256].sum() == 127 and zero[1, 256:].sum() == 127


# ------------------------------------------------------------------ the dense product

def run_linear(m, T, N, K, fn="none", gated=False, bias=False, res=False, out="bf16", strided=False, in_place=False,
               ws_fill=0xFF):
    R = 2 * N if gated else N
    xq, xs, xv = block_rows(_rand(T * 7 + K, T, K) * torch.exp2(_rand(2, K // 128).repeat_interleave(128)))
    wq, ws, wv = block_weights(_rand(N * 3 + K + 1, R, K) * torch.exp2(_rand(3, R)).clamp(0.1, 8)[:, None] / math.sqrt(K),
                               2 if gated else 1)
    b = _rand(5, R) if bias else None
    r = _rand(6, T, N).to(torch.bfloat16) if res else None
    pad = 64 if strided else 0
    kind = torch.bfloat16 if out == "bf16" else torch.float32
    od = torch.full((T + 3, N + (5 if strided else 0)), 7.0, device=DEV, dtype=kind)
    o, rd = od[:T, :N], None
    if r is not None:
        if in_place:
            o.copy_(r)
            rd = o
        else:
            rd = torch.full((T, N + (3 if strided else 0)), 9.0, device=DEV, dtype=torch.bfloat16)[:, :N]
            rd.copy_(r)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    a = m.linear_args(x=_wide(xq, pad, 0xFF), w=_wide(wq, pad, 0xFF), fmt="fp8_block", x_scale=dev(xs), w_scale=dev(ws),
                      bias=dev(b), act=fn, gated=gated, residual=rd, out=o)
    n = m.moe_linear_workspace_size(a)
    wsp = torch.full((n + 256,), ws_fill, dtype=torch.uint8, device=DEV)
    a.workspace, a.workspace_bytes = wsp.data_ptr(), n
    say(f"linear, block scales T={T} N={N} K={K} {fn} gated={gated} bias={bias} res={res} out={out} strided={strided} ws={n}")
    m.moe_linear(a)
    torch.cuda.synchronize()
    want, tol = reference(xv.to(DEV), wv.to(DEV), dev(b), fn, gated, dev(r), N, K, out == "bf16")
    tol = tol + want.abs() * (2.0 ** -8 if out == "bf16" else U) + 1e-30
    bad = ~((o.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[:4], (o.double() - want).abs()[bad].max())
    assert torch.all(od[T:] == 7.0) and torch.all(od[:, N:] == 7.0)
    assert torch.all(wsp[n:] == ws_fill)
    return o.clone()


FEW = [(1, 16, 128), (1, 1, 128), (2, 17, 256), (16, 64, 384), (15, 33, 1024), (5, 130, 2048), (1, 256, 7168),
       (16, 129, 4096), (3, 127, 640)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", FEW)
def test_linear_block_few_tokens(m, T, N, K):
    need_gpu()
    run_linear(m, T, N, K)
    run_linear(m, T, N, K, "silu", gated=True, bias=True, strided=True)
    run_linear(m, T, N, K, "gelu_tanh", bias=True, res=True, out="f32")
    run_linear(m, T, N, K, "relu", gated=True, out="f32", strided=True)
    run_linear(m, T, N, K, "gelu_erf", res=True, in_place=True)


BATCH = [(17, 48, 128), (33, 300, 256), (100, 128, 384), (129, 640, 1152), (333, 2056, 896), (1000, 257, 512),
         (300, 1000, 2048), (4100, 136, 2048), (257, 4104, 640)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", BATCH)
def test_linear_block_batches(m, T, N, K):
    need_gpu()
    run_linear(m, T, N, K, bias=True)
    run_linear(m, T, N, K, "silu", gated=True, strided=True)
    run_linear(m, T, N, K, "gelu_tanh", res=True, out="f32", strided=True)
    run_linear(m, T, N, K, "silu", gated=True, res=True, in_place=True)


@pytest.mark.gpu
def test_linear_block_scales_of_every_size(m):
    """Scales whose product leaves fp32's range as a product of codes would not: each block's sum is scaled once."""
    need_gpu()
    for T, N in ((2, 40), (70, 200)):
        K = 384
        g = torch.Generator().manual_seed(T)
        xq = torch.randint(-8, 9, (T, K), generator=g).float().to(torch.float8_e4m3fn)
        wq = torch.randint(-8, 9, (N, K), generator=g).float().to(torch.float8_e4m3fn)
        xs = torch.exp2(torch.tensor([-60.0, 0.0, 60.0]))[:, None].repeat(1, T) * (1 + torch.arange(T) / 64)
        ws = torch.exp2(torch.tensor([50.0, 0.0, -70.0]))[None].repeat((N + 127) // 128, 1) * 1.5
        out = torch.empty((T, N), dtype=torch.float32, device=DEV)
        say("linear, block scales of every size", T)
        a = m.linear_args(x=xq.to(DEV), w=wq.to(DEV), fmt="fp8_block", x_scale=xs.to(DEV), w_scale=ws.to(DEV), out=out)
        n = m.moe_linear_workspace_size(a)
        wsp = torch.empty(n + 16, dtype=torch.uint8, device=DEV)
        a.workspace, a.workspace_bytes = wsp.data_ptr(), n
        m.moe_linear(a)
        torch.cuda.synchronize()
        xv = xq.double() * xs.double().t().repeat_interleave(128, 1)
        wv = wq.double() * ws.double().repeat_interleave(128, 1).repeat_interleave(128, 0)[:N]
        tol = (K + 16) * U * (xv.abs() @ wv.abs().t())
        assert torch.all((out.cpu().double() - xv @ wv.t()).abs() <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 300])
def test_linear_block_rows_apart(m, T):
    """A row's result does not depend on the batch: a NaN in one token's scales stays in its row."""
    need_gpu()
    N, K = 200, 512
    xq, xs, _ = block_rows(_rand(1, T, K))
    wq, ws, _ = block_weights(_rand(2, N, K))
    bad = xs.clone()
    bad[1, T // 2] = float("nan")
    o = [torch.empty((T, N), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for s, out in zip((xs, bad), o):
        a = m.linear_args(x=xq.to(DEV), w=wq.to(DEV), fmt="fp8_block", x_scale=s.to(DEV), w_scale=ws.to(DEV), out=out)
        n = m.moe_linear_workspace_size(a)
        wsp = torch.empty(n + 16, dtype=torch.uint8, device=DEV)
        a.workspace, a.workspace_bytes = wsp.data_ptr(), n
        say("linear, block scales, rows apart", T)
        m.moe_linear(a)
        torch.cuda.synchronize()
    keep = torch.arange(T, device=DEV) != T // 2
    assert torch.equal(o[0][keep], o[1][keep]) and torch.isnan(o[1][T // 2]).all()


# ------------------------------------------------------------------ refusals (CPU)

def _ok(m, **kw):
    a = dict(T=4, N=32, K=128, x=0x10000, w=0x20000, out=0x30000, x_scale=0x40000, w_scale=0x50000, fmt="fp8_block")
    a.update(kw)
    return m.linear_args(**a)


@pytest.mark.parametrize("kw,msg", [
    (dict(K=192), "multiple of 128"), (dict(K=64), "multiple of 128"), (dict(x_scale=None), "null"),
    (dict(w_scale=None), "null"), (dict(x_scale=0x40002), "misaligned"), (dict(w_scale=0x50001), "misaligned"),
    (dict(x=0x10008), "16-byte"), (dict(w=0x20004), "16-byte"), (dict(T=-1), "bad sizes"), (dict(N=0), "bad sizes"),
    (dict(act=9), "fn")])
def test_linear_block_refusals(m, kw, msg):
    with pytest.raises(m.MoeError) as e:
        m.moe_linear(_ok(m, **kw), stream=0)
    assert e.value.status == 1 and msg in str(e.value)


def test_linear_block_no_tokens(m):
    assert m.moe_linear(_ok(m, T=0), stream=0) is None


@pytest.mark.parametrize("args,msg", [
    ((0x10000, 0, 4, 192, 3, 0x20000, 0x30000), "128"), ((0x10000, 0, 4, 256, 3, 0x20000, 0x30004), "misaligned"),
    ((0x10000, 0, 4, 256, 3, 0x20000, None), "null"), ((0x10000, 200, 4, 256, 3, 0x20000, 0x30000), "stride"),
    ((0x10000, 0, 4, 256, 4, 0x20000, 0x30000), "qmode")])
def test_quantize_block_refusals(m, args, msg):
    x, ldx, rows, cols, qm, q, s = args
    with pytest.raises(m.MoeError) as e:
        m.moe_quantize_fp8(x, rows, cols, qm, q, s, stream=0, ldx=ldx)
    assert e.value.status == 1 and msg in str(e.value)


def test_norm_block_refusals(m):
    for kw, msg in ((dict(H=200), "128"), (dict(q_scale=0x50004), "misaligned"), (dict(q_scale=None), "null"),
                    (dict(qmode=4), "qmode")):
        a = dict(x=0x10000, T=4, H=256, q=0x40000, q_scale=0x50000, qmode="fp8_block")
        a.update(kw)
        with pytest.raises(m.MoeError) as e:
            m.moe_rmsnorm(m.norm_args(**a), stream=0)
        assert e.value.status == 1 and msg in str(e.value)


def test_block_scales_of_another_shape(m):
    for name, shape in (("x_scale", (4, 2)), ("w_scale", (2, 2))):
        kw = dict(x=0x10000, w=0x20000, T=4, K=256, N=300, out=0x30000, fmt="fp8_block", x_scale=0x40000, w_scale=0x50000)
        kw[name] = torch.zeros(shape)
        with pytest.raises(m.MoeError) as e:
            m.linear_args(**kw)
        assert name in str(e.value) and "shape" in str(e.value)
