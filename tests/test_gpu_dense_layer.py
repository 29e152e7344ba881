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
