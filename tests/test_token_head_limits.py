"""TokenHead refuses what one of its calls would refuse before any of them is
enqueued, and at its construction where no batch could be answered."""
import pytest

from tests.gpu_util import DEV, need_gpu, torch


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


@pytest.mark.parametrize("kw", [dict(k=65), dict(k=-1), dict(V=20, k=21), dict(V=1 << 24), dict(V=0)])
def test_sizes_that_no_call_serves(m, kw):
    from fp4_expert_ffn_amd.layer import TokenHead
    a = dict(H=128, V=100, fmt="bf16", max_tokens=1, norm_weight=None, w=None, device="cpu")
    with pytest.raises(m.MoeError) as e:
        TokenHead(**{**a, **kw})
    assert e.value.status == 1 and "bad sizes" in str(e.value)


@pytest.mark.gpu
def test_a_refused_call_leaves_the_last_answer(m):
    """Given tokens of another type or shape, and scales that are no temperature's, are refused with nothing enqueued:
    the head's buffers still hold the last call's results."""
    need_gpu()
    from fp4_expert_ffn_amd.layer import TokenHead
    H, V, T = 128, 300, 5
    g = torch.Generator().manual_seed(1)
    w, x, y = (torch.randn(n, H, generator=g).to(torch.bfloat16).to(DEV) for n in (V, T, T))
    ids = torch.arange(T, dtype=torch.int32, device=DEV)
    head = TokenHead(H=H, V=V, fmt="bf16", max_tokens=8, norm_weight=None, w=w, k=3, device=DEV)
    got = head.forward(x, ids=ids)
    want = {n: v.clone() for n, v in got.items()}
    for kw, msg in ((dict(ids=ids.long()), "int64"), (dict(ids=ids[:4]), "shape"), (dict(ids=ids.cpu()), "not on a GPU"),
                    (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"), (dict(scale=1e-50), "scale"),
                    (dict(scale=float("inf")), "scale"), (dict(scale=float("nan")), "scale")):
        with pytest.raises(m.MoeError) as e:
            head.forward(y, **kw)
        assert e.value.status == 1 and msg in str(e.value), (msg, str(e.value))
        torch.cuda.synchronize()
        for n, v in want.items():
            assert torch.equal(got[n], v), (kw, n)
    head.forward(y, ids=ids)
    assert not torch.equal(got["logits"], want["logits"])
