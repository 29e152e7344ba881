"""What BlockMoELayer cannot serve is refused before any of its calls is made
(no kernel runs here), at its construction where no batch could be served."""
import pytest

from tests.gpu_util import DEV, need_gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


def layer(**kw):
    from fp4_expert_ffn_amd.layer import BlockMoELayer
    a = dict(E=4, k=1, H=128, I=128, max_tokens=4, gate_up=None, gate_up_scale=None, down=None, down_scale=None, device="cpu")
    return BlockMoELayer(**{**a, **kw})


@pytest.mark.parametrize("kw", [dict(k=17, E=32), dict(k=0), dict(k=5), dict(E=1025), dict(E=0), dict(I=32896),
                                dict(H=0), dict(I=-128)])
def test_sizes_that_no_call_serves(m, kw):
    with pytest.raises(m.MoeError) as e:
        layer(**kw)
    assert e.value.status == 1 and "bad sizes" in str(e.value)


@pytest.fixture
def made(monkeypatch):
    """The names of the calls that are made."""
    from fp4_expert_ffn_amd import _lib as L
    made = []
    for n in ("moe_router_logits", "moe_route_permute", "moe_route_scored_permute", "moe_quantize_fp8", "moe_linear_grouped",
              "moe_combine_bf16"):
        monkeypatch.setattr(L, n, lambda *a, n=n, **kw: made.append(n))
    return made


@pytest.mark.parametrize("T,k,I", [(65536, 1, 128), (65536, 2, 128), (43691, 3, 128), (8193, 16, 128), (8192, 16, 32768)])
def test_batches_past_the_calls_limits(m, made, T, k, I):
    """Nothing is routed, encoded or multiplied for a batch that the last call, or one between, would refuse."""
    lay = layer(E=16, k=k, I=I, max_tokens=4)
    lay.max_tokens = T  # without the buffers of such a batch
    x = torch.empty((T, 128), dtype=torch.bfloat16)
    with pytest.raises(m.MoeError) as e:
        lay.forward(x, logits=torch.empty(0))
    assert e.value.status == 1 and f"T={T}" in str(e.value) and not made


def test_rows_too_long_for_the_encoder(m, made):
    """Refused where the layer would encode x; its encoding as an argument goes on to the next check."""
    lay = layer(H=32896)
    x = torch.empty((2, 32896), dtype=torch.bfloat16)
    for rows, msg in ((None, "H=32896"), ((x, x), "not on a GPU")):
        with pytest.raises(m.MoeError) as e:
            lay.forward(x, logits=torch.empty(0), rows=rows)
        assert e.value.status == 1 and msg in str(e.value) and not made


def test_largest_sizes_are_taken(m):
    assert layer(E=1024, k=16, H=32768, I=32768, max_tokens=1).k == 16


@pytest.mark.gpu
@pytest.mark.parametrize("own_logits", [False, True])
def test_another_device_than_the_current_one(m, made, monkeypatch, own_logits):
    """The router's calls take addresses: the layer itself sees that its tensors lie where the stream runs."""
    need_gpu()
    lay = layer(device=DEV)
    x, w = torch.zeros((2, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((4, 128), device=DEV)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(m.MoeError) as e:
        lay.forward(x, stream=0, **(dict(logits=w[:2, :4].contiguous()) if own_logits else dict(w_router=w)))
    assert e.value.status == 1 and "current device cuda:1" in str(e.value) and not made, made
