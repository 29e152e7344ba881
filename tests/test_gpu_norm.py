"""RMS norm with the residual's addition and the 8-bit row encodings, on the
GPU through the C ABI, against the formulas in 64 bits.

Tolerances (u = 2^-24).  r = x + residual is one fp32 rounding.  The sum of
squares adds positive terms in chains of at most 32 and a tree of at most 16
more: relative error at most 50 u, half of it after the square root; with r,
the weight's product, rstd's and the last product y is within 32 u < 2^-19 of
its exact value.  A bf16 output adds half a step, 2^-8 of the value; an E4M3
code half a step, 2^-4 of the value, or 2^-10 of the scale below 2^-6."""
import numpy as np
import pytest

from tests.gpu_util import DEV, need_gpu, say, torch

F32 = 2.0 ** -19
BF16 = 2.0 ** -8 + F32


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float32)


def _padded(t, extra, fill):
    """t as the left columns of a wider device tensor whose other columns hold `fill`."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=DEV)
    wide[:, :t.shape[1]] = t.to(DEV)
    return wide


def _reference(x, res, w, eps):
    r = x.double() + (res.double() if res is not None else 0.0)
    y = r / torch.sqrt((r * r).mean(1, keepdim=True) + eps)
    return r, y * w.double() if w is not None else y


def _block_exponent(amax):
    return torch.where(amax > 0, torch.frexp(amax)[1] - 9, torch.zeros_like(amax, dtype=torch.int32))


def check_codes(y, q, scale, qmode):
    """q, scale (device) against exact rows y (double, CPU)."""
    T, H = y.shape
    v = q.cpu().view(torch.float8_e4m3fn).float().double()
    if qmode == "fp8":
        s = scale.cpu().double()
        want = torch.clamp(y.abs().amax(1) / 448.0, min=2.0 ** -126)
        assert torch.all((s - want).abs() <= want * F32)
        s = s[:, None].expand(T, H)
    else:
        amax = y.view(T, H // 32, 32).abs().amax(2)
        e = scale.cpu().view(torch.uint8).permute(1, 0, 2).reshape(T, H // 32).int() - 127
        lo, hi = _block_exponent(amax * (1 - F32)), _block_exponent(amax * (1 + F32))
        assert torch.all((e == lo) | (e == hi))
        s = torch.ldexp(torch.ones(T, H // 32, dtype=torch.float64), e).repeat_interleave(32, 1)
    ref = torch.clamp(y / s, -448.0, 448.0)
    off = (v - ref).abs()
    assert torch.all(off <= torch.clamp(ref.abs() * 2.0 ** -4, min=2.0 ** -10) + ref.abs() * F32), off.max()


CASES = [  # T, H, residual, weight, out, q
    (1, 8, "none", "bf16", True, "none"), (3, 24, "bf16", "f32", True, "fp8"), (5, 128, "f32", "bf16", True, "mxfp8"),
    (7, 200, "f32", "none", False, "fp8"), (9, 512, "bf16", "bf16", True, "none"), (4, 520, "bf16", "f32", True, "fp8"),
    (33, 1024, "none", "bf16", True, "mxfp8"), (130, 2048, "bf16", "bf16", True, "mxfp8"),
    (65, 2048, "f32", "f32", True, "fp8"), (6, 2056, "bf16", "bf16", True, "fp8"),
    (2, 4096, "f32", "bf16", True, "mxfp8"), (1, 7168, "bf16", "bf16", True, "none"),
    (300, 7168, "bf16", "f32", False, "mxfp8"), (3, 8192, "none", "f32", True, "fp8"),
    (2, 8200, "bf16", "bf16", True, "fp8"), (2, 32768, "f32", "bf16", True, "mxfp8"),
    (1, 2048, "bf16", "bf16", True, "fp8"), (16, 7168, "bf16", "bf16", True, "mxfp8"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,res,weight,out,q", CASES)
def test_norm_matches_the_formula(m, T, H, res, weight, out, q):
    need_gpu()
    x = _rand(T + H, T, H).to(torch.bfloat16)
    x[:, H // 3] *= 50.0
    r = None if res == "none" else (_rand(7, T, H) * 3.0).to({"bf16": torch.bfloat16, "f32": torch.float32}[res])
    w = None if weight == "none" else (1 + 0.3 * _rand(9, H)).to({"bf16": torch.bfloat16, "f32": torch.float32}[weight])
    eps = 1e-5
    # rows of wider tensors: what lies beside them is neither read (NaN) nor written
    xd = _padded(x, 8, float("nan"))
    rd = None if r is None else _padded(r, 24, float("nan"))
    ro = None if r is None else torch.full_like(rd, 7.0)
    yd = torch.full((T, H + 16), 7.0, dtype=torch.bfloat16, device=DEV) if out else None
    qd = torch.full((T, H + 8), 0x55, dtype=torch.uint8, device=DEV) if q != "none" else None
    sd = {"none": lambda: None, "fp8": lambda: torch.zeros(T, device=DEV),
          "mxfp8": lambda: torch.zeros((H // 128, T, 4), dtype=torch.uint8, device=DEV)}[q]()
    cut = lambda t: None if t is None else t[:, :H]  # noqa: E731
    a = m.norm_args(x=cut(xd), weight=None if w is None else w.to(DEV), eps=eps, residual=cut(rd), residual_out=cut(ro),
                    out=cut(yd), q=cut(qd), q_scale=sd, qmode=q)
    say(f"norm T={T} H={H} residual={res} weight={weight} out={out} q={q}")
    m.moe_rmsnorm(a)
    torch.cuda.synchronize()
    er, ey = _reference(x, r, w, eps)
    if r is not None:
        step = BF16 if res == "bf16" else F32
        assert torch.all((cut(ro).cpu().double() - er).abs() <= er.abs() * step)
        assert torch.all(ro[:, H:] == 7.0)
    if out:
        assert torch.all((cut(yd).cpu().double() - ey).abs() <= ey.abs() * BF16)
        assert torch.all(yd[:, H:] == 7.0)
    if q != "none":
        check_codes(ey, cut(qd).contiguous(), sd, q)
        assert torch.all(qd[:, H:] == 0x55)


# Widths on both sides of where a row takes more threads.
@pytest.mark.gpu
@pytest.mark.parametrize("T,H,q", [(9, 1032, "fp8"), (9, 1152, "mxfp8"), (5, 2048, "none"), (5, 2176, "mxfp8"),
                                   (5, 4104, "fp8"), (3, 4224, "mxfp8"), (3, 8192, "mxfp8"), (3, 8320, "mxfp8"),
                                   (2, 16384, "mxfp8"), (2, 16384, "fp8"), (2, 16392, "fp8"), (2, 16512, "mxfp8")])
def test_norm_row_widths(m, T, H, q):
    test_norm_matches_the_formula(m, T, H, "bf16", "f32", True, q)
    test_norm_matches_the_formula(m, T, H, "f32", "bf16", True, q)


@pytest.mark.gpu
@pytest.mark.parametrize("res", ["bf16", "f32"])
def test_norm_in_place(m, res):
    """residual_out is residual, out is x."""
    need_gpu()
    T, H = 37, 2048
    kind = {"bf16": torch.bfloat16, "f32": torch.float32}[res]
    x, r = _rand(1, T, H).to(torch.bfloat16), _rand(2, T, H).to(kind)
    xd, rd = x.to(DEV), r.to(DEV)
    say(f"norm in place, residual {res}")
    m.moe_rmsnorm(m.norm_args(x=xd, residual=rd, residual_out=rd, out=xd, eps=0.0))
    torch.cuda.synchronize()
    er, ey = _reference(x, r, None, 0.0)
    assert torch.all((rd.cpu().double() - er).abs() <= er.abs() * (BF16 if res == "bf16" else F32))
    assert torch.all((xd.cpu().double() - ey).abs() <= ey.abs() * BF16)


@pytest.mark.gpu
def test_norm_special_rows(m):
    """Zero rows, NaN and infinite values stay in their rows."""
    need_gpu()
    T, H = 6, 256
    x = _rand(3, T, H).to(torch.bfloat16)
    x[1] = 0.0
    x[2, 17] = float("nan")
    x[3, 18] = float("inf")
    x[4] *= 1e-30
    for q in ("fp8", "mxfp8"):
        y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        codes = torch.empty((T, H), dtype=torch.uint8, device=DEV)
        s = torch.empty(T, device=DEV) if q == "fp8" else torch.empty((2, T, 4), dtype=torch.uint8, device=DEV)
        say("norm special rows", q)
        m.moe_rmsnorm(m.norm_args(x=x.to(DEV), out=y, eps=1e-6, q=codes, q_scale=s, qmode=q))
        torch.cuda.synchronize()
        yc, v = y.cpu().float(), codes.cpu().view(torch.float8_e4m3fn).float()
        _, ey = _reference(x, None, None, 1e-6)
        for t in (0, 4, 5):
            assert torch.all((yc[t].double() - ey[t]).abs() <= ey[t].abs() * BF16)
            assert not torch.isnan(v[t]).any()
        assert torch.all(yc[1] == 0) and torch.all(v[1] == 0)
        assert torch.isnan(yc[2]).all() and torch.isnan(v[2]).all()
        keep = torch.arange(H) != 18
        assert torch.isnan(yc[3, 18]) and torch.all(yc[3, keep] == 0)
        if q == "fp8":
            assert s[1].item() == 2.0 ** -126
        else:
            assert torch.all(s.view(torch.uint8)[:, 1] == 127)


@pytest.mark.gpu
def test_quantize_fp8_bitexact(m):
    """Scales that are powers of two divide exactly: the codes are the nearest E4M3 value of
    x / scale, ties to even, saturating; every tie and the bottom of the exponent range."""
    need_gpu()
    rows, cols = 70, 384
    x = _rand(5, rows, cols).to(torch.bfloat16)
    ties = torch.arange(0, 256, dtype=torch.float32)
    x[0, :256] = (ties / 16.0).to(torch.bfloat16)            # every E4M3 step of a block, and the values between
    x[1] = (x[1].float() * 2.0 ** -130).to(torch.bfloat16)   # subnormal bf16 values
    x[2] = (x[2].float() * 2.0 ** 120).to(torch.bfloat16)
    x[3] = 0.0
    x[4, 5] = float("nan")
    x[5, 40] = float("-inf")
    q = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty((cols // 128, rows, 4), dtype=torch.float8_e8m0fnu, device=DEV)
    wide = _padded(x, 8, float("nan"))
    say("quantize mxfp8", rows, cols)
    m.moe_quantize_fp8(wide[:, :cols], rows, cols, "mxfp8", q, s)
    torch.cuda.synchronize()
    b = x.double().view(rows, cols // 32, 32)
    amax = torch.where(torch.isnan(b), 0.0, b.abs()).amax(2)
    e = torch.where(torch.isinf(amax), 120, torch.clamp(_block_exponent(amax), min=-127))
    got_e = s.cpu().view(torch.uint8).permute(1, 0, 2).reshape(rows, cols // 32).int() - 127
    assert torch.equal(got_e, e.int())
    v = torch.ldexp(b, -e[:, :, None])
    want = torch.where(torch.isnan(v), v, v.clamp(-448, 448)).float().to(torch.float8_e4m3fn).view(rows, cols)
    got = q.cpu()
    nan = torch.isnan(want.float())
    assert torch.equal(torch.isnan(got.float()), nan)
    assert torch.equal(got.view(torch.uint8)[~nan], want.view(torch.uint8)[~nan])
    # one scale a row: amax 448 * 2^k
    x = _rand(6, 9, 136).to(torch.bfloat16)
    x[:, 3] = torch.tensor([448.0 * 2.0 ** k for k in (-20, -3, -1, 0, 1, 2, 5, 9, 30)], dtype=torch.bfloat16)
    q = torch.empty((9, 136), dtype=torch.uint8, device=DEV)
    s = torch.empty(9, dtype=torch.float32, device=DEV)
    x *= torch.where(x.abs() <= x[:, 3:4], 1.0, 0.0).to(torch.bfloat16)
    say("quantize fp8", 9, 136)
    m.moe_quantize_fp8(x.to(DEV), 9, 136, "fp8", q, s)
    torch.cuda.synchronize()
    assert torch.equal(s.cpu(), x[:, 3].float() / 448.0)
    want = (x.double() / s.cpu().double()[:, None]).float().to(torch.float8_e4m3fn)
    assert torch.equal(q.cpu(), want.view(torch.uint8))


def _ok(L, **kw):
    a = dict(T=4, H=256, x=0x10000, out=0x20000)
    a.update(kw)
    return L.norm_args(**a)


@pytest.mark.parametrize("kw,msg", [
    (dict(H=12), "multiple of 8"), (dict(H=0), "bad sizes"), (dict(H=32776), "32768"), (dict(T=-1), "bad sizes"),
    (dict(eps=-1.0), "eps"), (dict(out=None), "no output"), (dict(x=None, T=4, H=256), "null"),
    (dict(x=0x10008), "misaligned"), (dict(out=0x20004), "misaligned"), (dict(residual_out=0x30000), "without residual"),
    (dict(qmode="fp8", q=0x40000), "null"), (dict(qmode=7), "qmode"),
    (dict(H=200, qmode="mxfp8", q=0x40000, q_scale=0x50000), "128"),
    (dict(qmode="fp8", q=0x40004, q_scale=0x50000), "misaligned"),
])
def test_norm_refusals(m, kw, msg):
    if "x" in kw and kw["x"] is None:
        a = _ok(m)
        a.x = None
    else:
        a = _ok(m, **kw)
    with pytest.raises(m.MoeError) as e:
        m.moe_rmsnorm(a, stream=0)
    assert e.value.status == 1 and msg in str(e.value)


def test_norm_refuses_bad_strides(m):
    for field in ("ldx", "ldr", "ldo", "ldq"):
        for ld in (248, 260):
            a = _ok(m)
            setattr(a, field, ld)
            with pytest.raises(m.MoeError) as e:
                m.moe_rmsnorm(a, stream=0)
            assert "stride" in str(e.value)
    assert m.moe_rmsnorm(_ok(m, T=0), stream=0) is None  # no tokens: nothing to do


def test_norm_args_refuse_tensors(m):
    """Types, shapes, strides and devices of tensors are checked before any address is taken."""
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    for kw, msg in ((dict(x=x.float(), out=x), "float32"), (dict(x=x[0], out=x), "shape"), (dict(x=x, out=x), "not on a GPU")):
        with pytest.raises(m.MoeError) as e:
            m.norm_args(**kw)
        assert msg in str(e.value)
    with pytest.raises(m.MoeError) as e:
        m.moe_quantize_fp8(x, 4, 128, "fp8", x, x)
    assert "shape" in str(e.value)


@pytest.mark.parametrize("args,msg", [
    ((0x10000, 0, 4, 12, 1, 0x20000, 0x30000), "multiple of 8"), ((0x10000, 0, 4, 256, 0, 0x20000, 0x30000), "qmode"),
    ((0x10000, 0, 4, 200, 2, 0x20000, 0x30000), "128"), ((0x10000, 128, 4, 256, 1, 0x20000, 0x30000), "stride"),
    ((None, 0, 4, 256, 1, 0x20000, 0x30000), "null"), ((0x10002, 0, 4, 256, 1, 0x20000, 0x30000), "misaligned"),
])
def test_quantize_fp8_refusals(m, args, msg):
    x, ldx, rows, cols, qm, q, s = args
    with pytest.raises(m.MoeError) as e:
        m.moe_quantize_fp8(x, rows, cols, qm, q, s, stream=0, ldx=ldx)
    assert e.value.status == 1 and msg in str(e.value)


def test_norm_refuses_more_rows_than_a_grid_holds(m):
    for n in (1 << 22, (1 << 31) - 1):
        with pytest.raises(m.MoeError) as e:
            m.moe_rmsnorm(m.norm_args(x=0x10000, T=n, H=64, out=0x20000), stream=0)
        assert e.value.status == 1 and "bad sizes" in str(e.value)
        with pytest.raises(m.MoeError) as e:
            m.moe_quantize_fp8(0x10000, n, 64, "fp8", 0x20000, 0x30000, stream=0)
        assert e.value.status == 1 and "bad sizes" in str(e.value)
