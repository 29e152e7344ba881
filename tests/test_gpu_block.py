"""The operators around the expert layer, run together as a model would: norm
and residual in front of a scored-routed sparse layer, a dense layer on
moe_linear, captured and replayed, and on streams of their own."""
import math

import numpy as np
import pytest

import oracle
import synth
from tests.gpu_util import DEV, need_gpu, out_f32, say, torch
from tests.test_gpu_linear import U, act64, encode
from tests.test_gpu_norm import BF16, check_codes
from tests.test_gpu_route_scored import rule

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    need_gpu()
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float32)


def dense(fmt, H=256, I=384, max_tokens=300):
    """A DenseLayer and its weights in 64 bits."""
    from fp4_expert_ffn_amd.layer import DenseLayer
    gq, gs, gv = encode(_rand(11, 2 * I, H) / math.sqrt(H), fmt)
    dq, ds, dv = encode(_rand(12, H, I) / math.sqrt(I), fmt)
    nw = (1 + 0.2 * _rand(13, H)).to(torch.bfloat16)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    layer = DenseLayer(H=H, I=I, fmt=fmt, max_tokens=max_tokens, norm_weight=dev(nw), gate_up=dev(gq), down=dev(dq),
                       gate_up_scale=dev(gs), down_scale=dev(ds), device=DEV)
    return layer, nw, gv, dv


def decoded(q, s, fmt):
    v = q.cpu().view(torch.float8_e4m3fn).float().double()
    if fmt == "fp8":
        return v * s.cpu().double()[:, None]
    e = s.cpu().view(torch.uint8).permute(1, 0, 2).reshape(v.shape[0], -1).int() - 127
    return torch.ldexp(v.view(v.shape[0], -1, 32), e[:, :, None]).view(v.shape)


def product_tol(xv, wv, fmt):
    K = xv.shape[1]
    tol = (K + 16) * U * (xv.abs() @ wv.abs().t())
    if fmt != "bf16":  # the FP8 instructions' cut sums (see test_gpu_linear)
        top = lambda v: v.abs().view(v.shape[0], K // 8, 8).amax(2)  # noqa: E731
        tol = tol + 7 * 2.0 ** -13 * (top(xv) @ top(wv).t())
    return tol


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8"])
@pytest.mark.parametrize("T,with_residual", [(1, True), (16, True), (17, False), (100, True), (300, False)])
def test_dense_layer_stage_by_stage(m, fmt, T, with_residual):
    """Every stage's output against its formula on what the stage before it wrote."""
    layer, nw, gv, dv = dense(fmt)
    H, I = layer.H, layer.I
    x, res = _rand(T, T, H).to(torch.bfloat16), (_rand(T + 1, T, H) * 2).to(torch.bfloat16)
    xd, rd = x.to(DEV), res.to(DEV)
    say(f"dense layer {fmt} T={T} residual={with_residual}")
    out = layer.forward(xd, rd if with_residual else None).cpu().double()
    torch.cuda.synchronize()
    r = x.double() + (res.double() if with_residual else 0.0)
    n = r / torch.sqrt((r * r).mean(1, keepdim=True) + layer.eps) * nw.double()
    kept = x.double()
    if with_residual:
        kept = layer.residual[:T].cpu().double()
        assert torch.all((kept - r).abs() <= r.abs() * BF16)
    # the first product's operand: the norm again by itself
    if fmt == "bf16":
        nv = layer.n[:T].cpu().double()
        assert torch.all((nv - n).abs() <= n.abs() * BF16)
    else:
        q = torch.empty((T, H), dtype=torch.uint8, device=DEV)
        s = torch.empty(T, device=DEV) if fmt == "fp8" else torch.empty((H // 128, T, 4), dtype=torch.uint8, device=DEV)
        m.moe_rmsnorm(m.norm_args(x=xd, weight=layer.norm_weight, eps=layer.eps, residual=rd if with_residual else None,
                                  q=q, q_scale=s, qmode=fmt))
        torch.cuda.synchronize()
        check_codes(n, q, s, fmt)
        nv = decoded(q, s, fmt)
    z, dz = nv @ gv.t(), product_tol(nv, gv, fmt)
    a, da = act64(z[:, :I], "silu"), 1.13 * dz[:, :I]
    h, dh = a * z[:, I:], da * z[:, I:].abs() + a.abs() * dz[:, I:] + da * dz[:, I:]
    got = layer.h[:T].cpu().double()
    assert torch.all((got - h).abs() <= dh + h.abs() * (2.0 ** -8 + 2.0 ** -19) + 1e-30)
    hv = got
    if fmt != "bf16":
        hq, hs = layer._rows(T, I)
        check_codes(got, hq, hs, fmt)
        hv = decoded(hq, hs, fmt)
    want = kept + hv @ dv.t()
    assert torch.all((out - want).abs() <= product_tol(hv, dv, fmt) + want.abs() * (2.0 ** -8 + 4 * U))


def sparse(m, T, router_kw, H=256, I=128, E=16, k=4):
    from fp4_expert_ffn_amd.layer import MoELayer, blob_of
    bias = torch.from_numpy((np.random.default_rng(3).standard_normal(E) * 0.1).astype(np.float32)).to(DEV)
    experts = [synth.expert("mxfp4", H, I, config=77, expert_id=e) for e in range(E)]
    layer = MoELayer(E=E, k=k, H=H, I=I, fmt="mxfp4", max_tokens=T, device=DEV, router=m.router(bias=bias, **router_kw))
    for e, ex in enumerate(experts):
        layer.load_expert(e, blob_of(ex))
    w_r = torch.from_numpy((np.random.default_rng(4).standard_normal((E, H)) * 0.1).astype(np.float32)).to(DEV)
    return layer, experts, w_r, bias


ROUTER = dict(score="sigmoid", n_group=4, topk_group=2, group_rank="top2", scale=2.5)


@pytest.mark.parametrize("T", [1, 5, 70, 300])
def test_sparse_layer_behind_the_norm(m, T):
    """norm -> router logits -> scored routing -> experts -> combine."""
    layer, experts, w_r, bias = sparse(m, T, ROUTER)
    H, k, E = layer.H, layer.k, layer.E
    x, res = _rand(T + 5, T, H).to(torch.bfloat16).to(DEV), (_rand(T + 6, T, H) * 2).to(torch.bfloat16).to(DEV)
    n = torch.empty_like(x)
    say(f"sparse layer behind the norm, T={T}")
    m.moe_rmsnorm(m.norm_args(x=x, residual=res, residual_out=res, out=n))
    layer.forward(n, w_router=w_r)
    torch.cuda.synchronize()
    logits = layer.logits[:T].cpu().numpy()
    ids, w = rule(logits, k, bias=bias.cpu().numpy(), **ROUTER)
    assert np.array_equal(layer.ids[:T].cpu().numpy(), ids)
    gw = layer.w[:T].cpu().numpy()
    assert np.all(np.abs(gw - w) <= w * (2.0 ** -24 + 2.0 ** -40))
    x_bits = n.view(torch.int16).cpu().numpy().view(np.uint16)
    dq = [oracle.moe.dequant_expert(e) for e in experts]
    ref = oracle.moe.layer_outputs(x_bits, ids, gw, E, lambda e: dq[e])
    ref = ref["out"] if isinstance(ref, dict) else ref
    assert oracle.moe.relative_error(out_f32(layer, T), ref) <= 1e-2


@pytest.mark.parametrize("T", [1, 16, 70, 300])
def test_captured_block_replays(m, T):
    """Norm, scored routing, experts and a dense layer in one graph: replays on new inputs, with
    eager calls of the same layers between them, give the eager results."""
    layer, _, w_r, _ = sparse(m, T, ROUTER)
    other, _, _, _ = sparse(m, T, ROUTER)
    fmt = "mxfp8" if T % 2 == 0 else "fp8"
    d, _, _, _ = dense(fmt)
    d2, _, _, _ = dense(fmt)
    H = layer.H
    inputs = [((_rand(30 + i, T, H)).to(torch.bfloat16).to(DEV), _rand(40 + i, T, H).to(torch.bfloat16).to(DEV))
              for i in range(4)]
    x, res = torch.empty_like(inputs[0][0]), torch.empty_like(inputs[0][1])

    def block(lay, dl, x, res):
        n, r = torch.empty_like(x), torch.empty_like(x)
        m.moe_rmsnorm(m.norm_args(x=x, residual=res, residual_out=r, out=n))
        lay.forward(n, w_router=w_r)
        y = lay.out[:T].view(torch.bfloat16)
        return y, dl.forward(y, r)

    x.copy_(inputs[0][0])
    res.copy_(inputs[0][1])
    say(f"captured block T={T} {fmt}")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(layer, d, x, res)  # warm up
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, z = block(layer, d, x, res)
    for a, b in inputs:
        want_y, want_z = (t.clone() for t in block(other, d2, a, b))
        x.copy_(a)
        res.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(z, want_z)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(z, want_z)


def test_two_streams_at_once(m):
    """The same calls on two streams with buffers of their own."""
    T, N, K = 200, 512, 2048
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls, outs, wants = [], [], []
    for i in range(2):
        x, w = _rand(50 + i, T, K).to(torch.bfloat16).to(DEV), _rand(52 + i, N, K).to(torch.bfloat16).to(DEV)
        o = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
        a = m.linear_args(x=x, w=w, out=o)
        ws = torch.empty(max(m.moe_linear_workspace_size(a), 16), dtype=torch.uint8, device=DEV)
        a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
        m.moe_linear(a)
        torch.cuda.synchronize()
        wants.append(o.clone())
        calls.append((a, ws))
        outs.append(o)
    say("two streams")
    for _ in range(20):
        for i in range(2):
            outs[i].zero_()
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for i in range(2):
            m.moe_linear(calls[i][0], stream=streams[i])
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        assert all(torch.equal(outs[i], wants[i]) for i in range(2))


@pytest.mark.parametrize("copy_engine", [False, True])
@pytest.mark.parametrize("T", [1, 3])
def test_cached_decode_with_routers(m, T, copy_engine):
    """The cached decode stream with a scored router a layer: the step's experts are the rule's, the
    outputs the oracle's."""
    from fp4_expert_ffn_amd.layer import CachedDecoder, to_numpy_bf16
    from tests.test_gpu_cache import _pinned_blob
    layers, E, k, H, I, tokens = 2, 16, 4, 256, 128, 10
    stride = (m.moe_blob_bytes("nvfp4", H, I) + 255) // 256 * 256
    experts = {(l, e): synth.expert("nvfp4", H, I, config=78, layer=l, expert_id=e) for l in range(layers) for e in range(E)}
    bank = {key: _pinned_blob(ex, stride) for key, ex in experts.items()}
    bias = (np.random.default_rng(1).standard_normal(E) * 0.1).astype(np.float32)
    kws = [dict(ROUTER), dict(score="softmax", n_group=2, topk_group=1, group_rank="max", renormalize=False)]
    routers = [m.router(bias=torch.from_numpy(bias).to(DEV), **kw) for kw in kws]
    dec = CachedDecoder(num_layers=layers, num_experts=E, k=k, H=H, I=I, fmt="nvfp4", num_slots=20, max_tokens=T,
                        host_blob=lambda l, e: bank[l, e], device=DEV, copy_engine=copy_engine, router=routers)
    rng = np.random.default_rng(9)
    say(f"cached decode with routers T={T} copy_engine={copy_engine}")
    for t in range(tokens):
        for l in range(layers):
            logits = rng.standard_normal((T, E)).astype(np.float32)
            x = synth.f32_to_bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
            out, trace = dec.step(l, torch.from_numpy(x.view(np.int16)).to(DEV), torch.from_numpy(logits).to(DEV))
            torch.cuda.synchronize()
            ids, w = rule(logits, k, bias=bias, **kws[l])
            assert np.array_equal(dec.ids[:T].cpu().numpy(), ids)
            assert trace[0].tolist() == sorted(set(ids.reshape(-1).tolist()))
            ref = oracle.moe.layer_outputs(x, ids, dec.w[:T].cpu().numpy(), E,
                                           lambda e: oracle.moe.dequant_expert(experts[l, e]))
            assert oracle.moe.relative_error(synth.bf16_bits_to_f32(to_numpy_bf16(out)), ref) <= 1e-2
    # back to the softmax routing
    m.moe_cache_use_router(dec.cache, -1, None)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    dec.step(0, torch.from_numpy(x.view(np.int16)).to(DEV), torch.from_numpy(logits).to(DEV))
    torch.cuda.synchronize()
    assert np.array_equal(dec.ids[:T].cpu().numpy(), oracle.moe.route(logits, k)[0])
    dec.close()


def test_cached_prefill_with_a_router(m):
    from fp4_expert_ffn_amd.layer import CachedPrefill, to_numpy_bf16
    from tests.test_gpu_cache import _pinned_blob
    layers, E, k, H, I, T = 2, 8, 2, 256, 128, 90
    stride = (m.moe_blob_bytes("nvfp4", H, I) + 255) // 256 * 256
    experts = {(l, e): synth.expert("nvfp4", H, I, config=79, layer=l, expert_id=e) for l in range(layers) for e in range(E)}
    bank = {key: _pinned_blob(ex, stride) for key, ex in experts.items()}
    kw = dict(score="sigmoid", scale=1.5)
    pf = CachedPrefill(num_layers=layers, num_experts=E, k=k, H=H, I=I, fmt="nvfp4", max_tokens=T,
                       host_blob=lambda l, e: bank[l, e], device=DEV, router=m.router(**kw))
    rng = np.random.default_rng(10)
    logits = rng.standard_normal((layers, T, E)).astype(np.float32)
    x = synth.f32_to_bf16_bits(rng.standard_normal((layers, T, H)).astype(np.float32))
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    outs = [torch.empty((T, H), dtype=torch.int16, device=DEV) for _ in range(layers)]
    say("cached prefill with a router")
    pf.run([dev(x[l].view(np.int16)) for l in range(layers)], [dev(logits[l]) for l in range(layers)], outs)
    torch.cuda.synchronize()
    for l in range(layers):
        ids, w = rule(logits[l], k, **kw)
        ref = oracle.moe.layer_outputs(x[l], ids, w, E, lambda e: oracle.moe.dequant_expert(experts[l, e]))
        assert oracle.moe.relative_error(synth.bf16_bits_to_f32(to_numpy_bf16(outs[l])), ref) <= 1e-2
    pf.close()
