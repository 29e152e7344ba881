"""A cache's scored routers: what moe_cache_use_router and the steps refuse (host
only), and the hybrid miss policy behind a router (GPU)."""
import gc
import weakref

import numpy as np
import pytest

import oracle
import synth
from tests.gpu_util import DEV, need_gpu, say, torch


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

    def get_device(self):
        return self.device.index

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


def prefill_step(m, E, T, k):
    """A prefill step whose addresses are never read: the call is refused before."""
    st = m.CachePrefill()
    st.layer, st.logits, st.topk_ids, st.dev_map = 0, 0x1000, 0x2000, 0x10000
    st.ffn = m.ffn_args(T=T, k=k, E=E, H=256, I=128, wfmt="bf16", out=0x3000, topk_w=0x4000, inv=0x5000, counts=0x6000,
                        offsets=0x7000, perm=0x8000)
    return st


def decode_step(m, E, T, k):
    st = m.CacheStep()
    st.layer, st.logits, st.topk_ids, st.dev_map = 0, 0x1000, 0x2000, 0x10000
    st.host_counts, st.host_map, st.host_blobs = 0x11000, 0x12000, 0x13000
    st.ffn = m.ffn_args(T=T, k=k, E=E, H=256, I=128, wfmt="bf16", y=0x9000, out=0x3000, topk_w=0x4000, inv=0x5000,
                        counts=0x6000, offsets=0x7000, perm=0x8000)
    return st


@pytest.mark.parametrize("T,k,msg", [(3, 5, "k=5"), (3, 17, "k=17"), (40000, 4, "131072")])
@pytest.mark.parametrize("kind", ["prefill", "decode"])
def test_a_router_that_cannot_serve_the_step_is_refused_first(m, kind, T, k, msg):
    """Too few experts in the open groups for the step's k, or a batch too long for the permutation: refused before
    the lookup, the waits and the routing."""
    E = 64
    c = m.moe_cache_create(E, 1 << 20, 0x100000, 1, E)
    m.cache_lookup(c, 0, np.arange(E))
    before = m.moe_cache_stats(c)
    kw = dict(n_group=16, topk_group=1) if k == 5 else {}
    m.moe_cache_use_router(c, -1, m.router(score="sigmoid", **kw))
    with pytest.raises(m.MoeError) as e:
        if kind == "prefill":
            m.moe_cache_prefill_step(c, prefill_step(m, E, T, k), compute_stream=0)
        else:
            m.moe_cache_decode_step(c, decode_step(m, E, T, k), copy_stream=0, compute_stream=0)
    assert e.value.status == 1 and msg in str(e.value)
    assert m.moe_cache_stats(c) == before
    if kind == "decode":  # an empty step has nothing to route
        m.moe_cache_decode_step(c, decode_step(m, E, 0, k), copy_stream=0, compute_stream=0)
    c.close()


@pytest.mark.gpu
@pytest.mark.parametrize("copy_ratio", [0.0, 0.5, 1.0])
def test_hybrid_decode_with_a_router(m, copy_ratio):
    """Misses split between copies and the host FFN, the step's experts chosen by a scored router."""
    need_gpu()
    from fp4_expert_ffn_amd.layer import CachedDecoder, to_numpy_bf16
    from tests.test_gpu_cache import _pinned_blob
    from tests.test_gpu_route_scored import rule
    E, k, H, I, T = 16, 4, 256, 128, 2
    stride = (m.moe_blob_bytes("nvfp4", H, I) + 255) // 256 * 256
    experts = [synth.expert("nvfp4", H, I, config=80, expert_id=e) for e in range(E)]
    bank = [_pinned_blob(ex, stride) for ex in experts]
    kw = dict(score="sigmoid", n_group=4, topk_group=2, group_rank="top2", scale=2.5)
    bias = (np.random.default_rng(1).standard_normal(E) * 0.1).astype(np.float32)
    dec = CachedDecoder(num_layers=1, num_experts=E, k=k, H=H, I=I, fmt="nvfp4", num_slots=8, max_tokens=T,
                        host_blob=lambda l, e: bank[e], device=DEV, copy_ratio=copy_ratio, host_threads=2,
                        router=m.router(bias=torch.from_numpy(bias).to(DEV), **kw))
    rng = np.random.default_rng(9)
    say(f"hybrid decode with a router, copy_ratio={copy_ratio}")
    for t in range(6):
        logits = rng.standard_normal((T, E)).astype(np.float32)
        x = synth.f32_to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
        out, _ = dec.step(0, torch.from_numpy(x.view(np.int16)).to(DEV), torch.from_numpy(logits).to(DEV))
        torch.cuda.synchronize()
        ids, _ = rule(logits, k, bias=bias, **kw)
        assert np.array_equal(dec.ids[:T].cpu().numpy(), ids)
        ref = oracle.moe.layer_outputs(x, ids, dec.w[:T].cpu().numpy(), E,
                                       lambda e: oracle.moe.dequant_expert(experts[e]))
        assert oracle.moe.relative_error(synth.bf16_bits_to_f32(to_numpy_bf16(out)), ref) <= 1e-2
    dec.close()


@pytest.mark.gpu
def test_short_router_biases_are_refused(m):
    need_gpu()
    from fp4_expert_ffn_amd.layer import CachedDecoder
    with pytest.raises(m.MoeError) as e:
        CachedDecoder(num_layers=1, num_experts=16, k=2, H=256, I=128, fmt="nvfp4", num_slots=4,
                      host_blob=lambda l, e: None, device=DEV, router=m.router(bias=torch.zeros(8, device=DEV)))
    assert "bias" in str(e.value)
