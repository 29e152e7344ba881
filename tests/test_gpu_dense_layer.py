"""DenseLayer when its weights are replaced between calls, and what it keeps."""
import math

import pytest

from tests.gpu_util import DEV, need_gpu, say, torch
from tests.test_gpu_block import dense
from tests.test_gpu_linear import encode

pytestmark = pytest.mark.gpu


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float32)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8"])
def test_replaced_weights_are_used(fmt):
    """After a weight, its scales or the norm's weight are replaced, a batch size seen before gives what a layer
    made of the new ones gives."""
    need_gpu()
    layer, nw, _, _ = dense(fmt)
    H, I = layer.H, layer.I
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    x, res = _rand(1, 5, H).to(torch.bfloat16).to(DEV), _rand(2, 5, H).to(torch.bfloat16).to(DEV)
    say("dense layer, replaced weights", fmt)
    old = layer.forward(x, res).clone()
    gq, gs, _ = encode(_rand(21, 2 * I, H) / math.sqrt(H), fmt)
    dq, ds, _ = encode(_rand(22, H, I) / math.sqrt(I), fmt)
    from fp4_expert_ffn_amd.layer import DenseLayer
    w = dict(gate_up=dev(gq), down=dev(dq), gate_up_scale=dev(gs), down_scale=dev(ds))
    want = DenseLayer(H=H, I=I, fmt=fmt, max_tokens=5, norm_weight=dev(nw), device=DEV, **w).forward(x, res)
    for name, t in w.items():
        setattr(layer, name, t)
    got = layer.forward(x, res)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and not torch.equal(got, old)
    layer.norm_weight = dev(nw) * 2
    assert not torch.equal(layer.forward(x, res), want)


def test_replaced_weights_of_another_shape_are_refused():
    need_gpu()
    import fp4_expert_ffn_amd as m
    layer, _, _, _ = dense("bf16")
    x = _rand(1, 5, layer.H).to(torch.bfloat16).to(DEV)
    layer.forward(x)
    layer.down = layer.down[:-16].contiguous()
    with pytest.raises(m.MoeError) as e:
        layer.forward(x)
    assert "shape" in str(e.value)


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_inputs_in_the_layers_own_buffers(fmt):
    """The last output's first rows as the next input: as from a copy.  Other rows of it, or every second one,
    which the second product would overwrite while it adds them, are refused."""
    need_gpu()
    import fp4_expert_ffn_amd as m
    layer, _, _, _ = dense(fmt)
    x = _rand(1, 200, layer.H).to(torch.bfloat16).to(DEV)
    say("dense layer, inputs in its own buffers", fmt)
    y = layer.forward(x)
    want = layer.forward(y.clone()).clone()
    y = layer.forward(x)
    assert torch.equal(layer.forward(y), want)
    y = layer.forward(x)
    part = y[3:90].clone()
    for rows in (y[3:90], y[::2]):
        with pytest.raises(m.MoeError) as e:
            layer.forward(rows)
        assert e.value.status == 1 and "copy" in str(e.value)
    want = layer.forward(part).clone()
    y = layer.forward(x)
    assert torch.equal(layer.forward(y[110:197].copy_(part)), want)  # behind the rows written: no overlap
    # a residual stream of its own buffer's rows
    res = _rand(2, 200, layer.H).to(torch.bfloat16).to(DEV)
    layer.forward(x, res)
    kept = layer.residual[:200].clone()
    want = layer.forward(x, kept).clone()
    layer.residual[:200].copy_(kept)
    assert torch.equal(layer.forward(x, layer.residual[:200]), want)
    for a, b in ((x[:50], layer.residual[1:51]), (layer.residual[1:51], res[:50])):
        with pytest.raises(m.MoeError):
            layer.forward(a, b)


def test_scale_buffer_holds_the_scales_alone():
    """One byte per 32 columns of the wider of the two operands (MXFP8), four a row (FP8)."""
    need_gpu()
    for fmt, size in (("mxfp8", 300 * 384 // 32), ("fp8", 300 * 4)):
        assert dense(fmt)[0].q_scale.numel() == size


def test_refusals():
    need_gpu()
    import fp4_expert_ffn_amd as m
    from fp4_expert_ffn_amd.layer import DenseLayer
    layer, _, _, _ = dense("mxfp8")
    x = _rand(1, 5, layer.H).to(torch.bfloat16)
    for bad, msg in ((x, "cpu"), (x.to(DEV).float(), "float32"), (x.to(DEV)[:, :128], "shape"),
                     (x.to(DEV)[:, None], "shape")):
        with pytest.raises(m.MoeError) as e:
            layer.forward(bad)
        assert e.value.status == 1 and msg in str(e.value)
    with pytest.raises(m.MoeError) as e:
        DenseLayer(H=256, I=200, fmt="mxfp8", max_tokens=4, norm_weight=None, gate_up=None, down=None, device=DEV)
    assert "128" in str(e.value)
