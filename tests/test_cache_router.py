"""A cache's scored routers: what moe_cache_use_router refuses."""
import gc
import weakref

import pytest

from tests.gpu_util import DEV, need_gpu, torch


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


class Bias:
    """What the library asks of a bias tensor; its address is never read here."""
    dtype, is_cuda = "torch.float32", True

    def __init__(self, n, index=0):
        self.n, self.shape = n, (n,)
        self.device = type("Device", (), {"index": index, "__str__": lambda s: f"cuda:{s.index}"})()

    def numel(self):
        return self.n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


class Pool:
    """A slot pool on device `index`; its address is never used here."""
    is_cuda = True

    def __init__(self, index):
        self.device = type("Device", (), {"index": index})()

    def data_ptr(self):
        return 0x100000


def test_router_bias_has_the_caches_experts_and_device(m):
    c = m.moe_cache_create(4, 1 << 20, Pool(0), 2, 16)
    for bias, msg in ((Bias(15), "15"), (Bias(17), "17"), (Bias(1), "bias"), (Bias(16, 1), "cuda:1")):
        with pytest.raises(m.MoeError) as e:
            m.moe_cache_use_router(c, 0, m.router(score="sigmoid", bias=bias))
        assert e.value.status == 1 and msg in str(e.value)
    m.moe_cache_use_router(c, -1, m.router(score="sigmoid", bias=Bias(16)))
    c.close()


def test_a_refused_router_leaves_the_one_in_use_alive(m):
    c = m.moe_cache_create(4, 1 << 20, 0, 2, 16)
    bias = Bias(16)
    m.moe_cache_use_router(c, 0, m.router(bias=bias))
    alive = weakref.ref(bias)
    del bias
    with pytest.raises(m.MoeError):
        m.moe_cache_use_router(c, 0, m.router(n_group=3))
    gc.collect()
    assert alive() is not None
    m.moe_cache_use_router(c, -1, None)  # no layer reads it any more
    gc.collect()
    assert alive() is None
    c.close()


@pytest.mark.gpu
def test_short_router_biases_are_refused(m):
    need_gpu()
    from fp4_expert_ffn_amd.layer import CachedDecoder
    with pytest.raises(m.MoeError) as e:
        CachedDecoder(num_layers=1, num_experts=16, k=2, H=256, I=128, fmt="nvfp4", num_slots=4,
                      host_blob=lambda l, e: None, device=DEV, router=m.router(bias=torch.zeros(8, device=DEV)))
    assert "bias" in str(e.value)
