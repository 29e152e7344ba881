"""8-bit rows whose fp32 scale is no power of two: a code is the fp32 quotient
value / scale, rounded once more to E4M3 (to nearest even), bit for bit."""
import pytest

from tests.gpu_util import DEV, need_gpu, say, torch


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


def rows_near_ties():
    """Every bf16 significand as a row's largest magnitude, with every significand of 12 binades below it:
    quotients on and beside the ties between two codes."""
    mant = (torch.arange(128, dtype=torch.float32) + 128) / 128
    v = torch.cat([mant * 2.0 ** e for e in range(-8, 4)])
    x = v.repeat(128, 1)
    amax = mant[:, None] * 8.0
    x = torch.where(x <= amax, x, 0.0)
    x[:, 0] = amax[:, 0]
    return (x * torch.where(torch.arange(x.shape[1]) % 3 == 1, -1.0, 1.0)).to(torch.bfloat16)


def codes_of(x):
    s = torch.clamp(x.float().abs().amax(1) / 448.0, min=2.0 ** -126)
    return (x.float() / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def test_a_rounded_reciprocal_would_differ():
    """The rows tell the quotient from a product with the scale's rounded reciprocal."""
    x = rows_near_ties()
    want, s = codes_of(x)
    other = (x.float() * (1.0 / s)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert (want != other).sum() > 50


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, -120, 100])
def test_quantize_fp8_quotients(m, shift):
    need_gpu()
    x = (rows_near_ties().float() * 2.0 ** shift).to(torch.bfloat16)
    rows, cols = x.shape
    q = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
    s = torch.empty(rows, dtype=torch.float32, device=DEV)
    say("quantize fp8, quotients", rows, cols, shift)
    m.moe_quantize_fp8(x.to(DEV), rows, cols, "fp8", q, s)
    torch.cuda.synchronize()
    want, ws = codes_of(x)
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(q.cpu(), want)
