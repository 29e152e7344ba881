"""The linear product's activations over their whole range, on every path that
evaluates them: the few-token kernel, the tiles and the join of a split K.

The operands are zero, so that a pre-activation is its bias.  Tolerances (u =
2^-24), relative to the value: 2^-20 for the exponential, the reciprocal and
the products; GELU-tanh's exponent 2 t is off by at most 6 u of itself (its
two constants, their products and the fused sum), and so is its exponential by
6 u |2 t|; the argument of GELU-erf's erfc is off by 2 u of itself, which moves
erfc(y) by 2 y^2 2 u at most, 2 u z^2, and erfc is within 16 units of its last
place, 2^-19.  (For z > 0 both are 6 u and 2 u at most: t exp(-t) < 1.)  A reciprocal or exponential below 2^-126 may be flushed: 2^-125
|z|.  The output adds u of itself (fp32) or 2^-8 (bf16)."""
import math

import pytest

from tests.gpu_util import DEV, need_gpu, say, torch
from tests.test_gpu_linear import act64

U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


def exact(z, fn):
    if fn == "gelu_tanh":  # 1 + tanh(t) cancels in 64 bits too: 2 sigmoid(2 t)
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return act64(z, fn)


def bound(z, fn):
    """The error of fn(z) in fp32."""
    a = exact(z, fn).abs()
    rel = torch.full_like(z, 2.0 ** -20)
    if fn == "gelu_tanh":
        rel = rel + 6 * U * torch.where(z < 0, (2 * math.sqrt(2 / math.pi) * (0.044715 * z ** 3 + z)).abs(), 1.0)
    if fn == "gelu_erf":
        rel = rel + 2.0 ** -19 + 2 * U * torch.where(z < 0, z * z, 1.0)
    return a * rel + 2.0 ** -125 * z.abs() + 1e-37


# few tokens, tiles, K split
@pytest.mark.gpu
@pytest.mark.parametrize("T,K", [(3, 64), (300, 64), (64, 8192)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fn", ["none", "silu", "gelu_tanh", "gelu_erf", "relu"])
def test_activation_over_its_range(m, fn, gated, T, K):
    need_gpu()
    z = torch.cat([torch.linspace(-200, 200, 2001), torch.linspace(-16, 16, 1001), torch.linspace(-139, -88, 511),
                   torch.tensor([0.0, -0.0, 1e30, -1e30, 3e38, 1e-30, -1e-30])]).float()
    N = z.numel()
    R = 2 * N if gated else N
    bias = torch.cat([z, torch.ones(N)]) if gated else z
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((R, K), dtype=torch.bfloat16, device=DEV)
    for out, step in ((torch.float32, U), (torch.bfloat16, 2.0 ** -8)):
        o = torch.full((T, N), 7.0, dtype=out, device=DEV)
        a = m.linear_args(x=x, w=w, bias=bias.to(DEV), act=fn, gated=gated, out=o)
        n = m.moe_linear_workspace_size(a)
        assert (n > 0) == (K > 64)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        a.workspace, a.workspace_bytes = ws.data_ptr(), n
        say(f"activation {fn} gated={gated} T={T} K={K} {out}")
        m.moe_linear(a)
        torch.cuda.synchronize()
        want = exact(z.double(), fn)
        got = o.cpu().double()
        off = (got - want).abs()
        tol = bound(z.double(), fn) + want.abs() * step
        if out == torch.bfloat16:
            tol = torch.where(want.abs() > 3e38, math.inf, tol)  # rounds to infinity
        bad = ~(off <= tol)
        assert not bad.any(), (int(bad.sum()), z[bad[0]][:5], got[0][bad[0]][:5])


@pytest.mark.gpu
@pytest.mark.parametrize("T,K", [(3, 64), (300, 64), (64, 8192)])
def test_activation_of_infinity_and_nan(m, T, K):
    need_gpu()
    N = 70
    bias = torch.zeros(N)
    bias[3], bias[40] = math.inf, math.nan
    x = torch.zeros((T, K), dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((N, K), dtype=torch.bfloat16, device=DEV)
    for fn in ("none", "silu", "gelu_tanh", "gelu_erf", "relu"):
        o = torch.empty((T, N), device=DEV)
        a = m.linear_args(x=x, w=w, bias=bias.to(DEV), act=fn, out=o)
        n = m.moe_linear_workspace_size(a)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        a.workspace, a.workspace_bytes = ws.data_ptr(), n
        say(f"activation {fn} of infinity and NaN, T={T} K={K}")
        m.moe_linear(a)
        torch.cuda.synchronize()
        assert torch.all(o[:, 3] == math.inf) and torch.isnan(o[:, 40]).all()
        rest = [i for i in range(N) if i not in (3, 40)]
        assert torch.all(o[:, rest] == 0)
