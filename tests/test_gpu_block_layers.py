"""The layers of the block-scaled products: DenseLayer with "fp8_block" rows,
BlockMoELayer with slots and inputs of its own, and TokenHead with every kind
of weights, each stage against its formula in 64 bits on what the stage before
it wrote.  Tolerances as in test_gpu_fp8_block and test_gpu_logprobs."""
import math

import pytest

from tests.gpu_util import DEV, need_gpu, say, torch
from tests.test_gpu_fp8_block import _rand, block_weights, check_block_codes
from tests.test_gpu_grouped import layer_of, values
from tests.test_gpu_linear import encode, reference
from tests.test_gpu_norm import F32, _reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    need_gpu()
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


def near(got, want, tol):
    return bool(((got.cpu().double() - want).abs() <= tol + want.abs() * 2.0 ** -8 + 1e-30).all())


def norm_rows(m, x, res, w, T, H):
    """The norm's rows, from a call of its own."""
    q, s = torch.empty((T, H), dtype=torch.uint8, device=DEV), torch.empty((H // 128, T), device=DEV)
    m.moe_rmsnorm(m.norm_args(x=x, residual=res, weight=w, q=q, q_scale=s, qmode="fp8_block"))
    return q, s


@pytest.mark.parametrize("T,with_residual", [(1, True), (16, False), (17, True), (100, False), (300, True)])
def test_dense_layer_stage_by_stage(m, T, with_residual):
    from fp4_expert_ffn_amd.layer import DenseLayer
    H, I = 256, 384
    gq, gs, gv = block_weights(_rand(11, 2 * I, H) / math.sqrt(H), 2)
    dq, ds, dv = block_weights(_rand(12, H, I) / math.sqrt(I))
    nw = (1 + 0.2 * _rand(13, H)).to(torch.bfloat16).to(DEV)
    layer = DenseLayer(H=H, I=I, fmt="fp8_block", max_tokens=300, norm_weight=nw, gate_up=gq.to(DEV), down=dq.to(DEV),
                       gate_up_scale=gs.to(DEV), down_scale=ds.to(DEV), device=DEV)
    x = _rand(T, T, H).to(torch.bfloat16)
    res = _rand(T + 1, T, H).to(torch.bfloat16) if with_residual else None
    xd, rd = x.to(DEV), None if res is None else res.to(DEV)
    say("dense layer, block rows", T, with_residual)
    out = layer.forward(xd, rd)
    torch.cuda.synchronize()
    q, s = norm_rows(m, xd, rd, nw, T, H)
    kept = xd if res is None else layer.residual[:T]
    er, ey = _reference(x, res, nw.cpu(), 1e-6)
    if res is not None:
        assert torch.all((kept.cpu().double() - er).abs() <= er.abs() * (2.0 ** -8 + F32))
    check_block_codes(ey, q, s, F32)
    assert near(layer.h[:T], *reference(values(q, s), gv, None, "silu", True, None, I, H, True))
    hq, hs = layer._rows(T, I)
    check_block_codes(layer.h[:T].cpu().double(), hq, hs, 0.0)
    assert near(out, *reference(values(hq, hs), dv, None, "none", False, kept.cpu(), H, I, True))


def test_dense_layer_needs_whole_blocks(m):
    from fp4_expert_ffn_amd.layer import DenseLayer
    with pytest.raises(m.MoeError) as e:
        DenseLayer(H=256, I=200, fmt="fp8_block", max_tokens=4, norm_weight=None, gate_up=None, down=None, device=DEV)
    assert "128" in str(e.value)


def test_block_layer_in_slots_and_on_its_own_output(m):
    """Experts in another order of slots give what the same experts in order give; the last output as the next input
    gives what a copy of it does."""
    from fp4_expert_ffn_amd.layer import BlockMoELayer
    layer, gv, dv, sv = layer_of(m, shared=False)
    T, E = 60, layer.E
    x, logits = _rand(1, T, layer.H).to(torch.bfloat16).to(DEV), _rand(2, T, E).to(DEV)
    say("block layer, slots")
    want = layer.forward(x, logits=logits).clone()
    slots = torch.tensor([(5 * e + 3) % E for e in range(E)])
    order = torch.argsort(slots)  # slot -> expert
    moved = BlockMoELayer(E=E, k=layer.k, H=layer.H, I=layer.I, max_tokens=T, gate_up=layer.gate_up.view(torch.uint8)[order],
                          gate_up_scale=layer.gate_up_scale[order], down=layer.down.view(torch.uint8)[order],
                          down_scale=layer.down_scale[order], slot_of_expert=slots.int().to(DEV), device=DEV)
    assert torch.equal(moved.forward(x, logits=logits), want)
    again = layer.forward(want.clone(), logits=logits).clone()
    out = layer.forward(x, logits=logits)
    assert torch.equal(layer.forward(out, logits=logits), again)


def test_block_layer_forward_refuses(m):
    layer, _, _, _ = layer_of(m, shared=False)
    x, logits = _rand(1, 5, layer.H).to(torch.bfloat16).to(DEV), _rand(2, 5, layer.E).to(DEV)
    q, s = norm_rows(m, x, None, None, 5, layer.H)
    for kw, msg in ((dict(), "neither"), (dict(logits=logits[:4]), "shape"), (dict(logits=logits.half()), "float16"),
                    (dict(logits=logits.cpu()), "not on a GPU"), (dict(logits=logits.t().contiguous().t()), "contiguous"),
                    (dict(w_router=logits), "shape"), (dict(logits=logits, rows=(q[:4], s)), "shape"),
                    (dict(logits=logits, rows=(q, s[:1])), "shape")):
        with pytest.raises(m.MoeError) as e:
            layer.forward(x, **kw)
        assert e.value.status == 1 and msg in str(e.value), (msg, str(e.value))
    assert layer.forward(x[:0], logits=logits[:0]).shape == (0, layer.H)


def vocabulary(fmt, V, H):
    """(weights, scales or None, values in 64 bits)."""
    v = _rand(31, V, H) / math.sqrt(H)
    return block_weights(v) if fmt == "fp8_block" else encode(v, fmt)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8", "fp8_block"])
@pytest.mark.parametrize("T,k,f32", [(1, 0, True), (3, 20, False), (40, 5, True)])
def test_token_head(m, fmt, T, k, f32):
    """The log probabilities of the head's own logits, those the product of its own rows."""
    from fp4_expert_ffn_amd.layer import TokenHead
    H, V, scale = 256, 1003, 1.25
    wq, ws, wv = vocabulary(fmt, V, H)
    nw = (1 + 0.2 * _rand(32, H)).to(torch.bfloat16).to(DEV)
    head = TokenHead(H=H, V=V, fmt=fmt, max_tokens=64, norm_weight=nw, w=wq.to(DEV), w_scale=None if ws is None else ws.to(DEV),
                     k=k, logits_f32=f32, device=DEV)
    x, res = (_rand(s, T, H).to(torch.bfloat16).to(DEV) for s in (1, 2))
    ids = torch.randint(V, (T,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(DEV)
    say("token head", fmt, T, k, f32)
    got = {n: v.clone() for n, v in head.forward(x, res, ids=ids, scale=scale).items()}
    assert set(got) == {"logits", "lse", "entropy", "logprob", "rank"} | ({"top_ids", "top_logprob"} if k else set())
    if fmt in ("bf16", "fp8_block"):
        xv = head.n[:T].cpu().double() if fmt == "bf16" else values(head.q[:T * H].view(T, H),
                                                                    head.q_scale[:T * H // 32].view(torch.float32).view(H // 128, T))
        want, tol = reference(xv, wv.cpu().double(), None, "none", False, None, V, H, fmt != "bf16" and not f32)
        assert torch.all((got["logits"].cpu().double() - want).abs()
                         <= tol + want.abs() * (2.0 ** -24 if f32 else 2.0 ** -8) + 1e-30)
    l = got["logits"].cpu().double() * scale
    z = torch.log_softmax(l, 1)
    at = z.gather(1, ids.cpu().long()[:, None])[:, 0]
    close = lambda a, b: torch.allclose(a.cpu().double(), b, rtol=1e-6, atol=2e-6)  # noqa: E731
    assert close(got["logprob"], at) and close(got["lse"], torch.logsumexp(l, 1)) and close(got["entropy"], -(z.exp() * z).sum(1))
    order = got["logits"].cpu().float().sort(dim=1, descending=True, stable=True)[1]
    if k:
        assert torch.equal(got["top_ids"].cpu().long(), order[:, :k]) and close(got["top_logprob"], z.gather(1, order[:, :k]))
    again = head.forward(x, res, scale=scale)  # without ids: neither logprob nor rank
    assert set(again) == set(got) - {"logprob", "rank"}
    for n in again:
        assert torch.equal(again[n], got[n]), n


def test_token_head_refuses(m):
    from fp4_expert_ffn_amd.layer import TokenHead
    H, V = 256, 300
    wq, ws, _ = vocabulary("fp8_block", V, H)
    make = lambda **kw: TokenHead(**{**dict(H=H, V=V, fmt="fp8_block", max_tokens=8, norm_weight=None, w=wq.to(DEV),  # noqa: E731
                                            w_scale=ws.to(DEV), device=DEV), **kw})
    with pytest.raises(m.MoeError) as e:
        make(H=200)
    assert "128" in str(e.value)
    with pytest.raises(m.MoeError) as e:
        make(V=310)
    assert "shape" in str(e.value)
    head = make()
    x = _rand(1, 5, H).to(torch.bfloat16)
    for a, kw, msg in ((x, {}, "cpu"), (x.to(DEV).float(), {}, "float32"), (x.to(DEV)[:, :128], {}, "shape"),
                       (x.to(DEV), dict(ids=torch.zeros(4, dtype=torch.int32, device=DEV)), "shape"),
                       (x.to(DEV), dict(ids=torch.zeros(5, dtype=torch.int64, device=DEV)), "int64"),
                       (x.to(DEV), dict(scale=0.0), "scale")):
        with pytest.raises(m.MoeError) as e:
            head.forward(a, **kw)
        assert e.value.status == 1 and msg in str(e.value), (msg, str(e.value))
    assert head.forward(x[:0].to(DEV))["logits"].shape == (0, V)
