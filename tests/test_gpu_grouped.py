"""The block-scaled product over the rows of routed experts, on the GPU
through the C ABI, against the formula in 64 bits (tolerances as in
test_gpu_fp8_block), and the layer made of it."""
import math

import pytest

from tests.gpu_util import DEV, need_gpu, say, torch
from tests.test_gpu_fp8_block import _rand, block_rows, block_weights, check_block_codes
from tests.test_gpu_linear import U, reference


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


def expert_weights(S, R, K, parts, seed=1):
    q, s, v = zip(*(block_weights(_rand(seed * 1000 + e, R, K) / math.sqrt(K), parts) for e in range(S)))
    return torch.stack([t.view(torch.uint8) for t in q]).view(torch.float8_e4m3fn), torch.stack(s), v


def run_grouped(m, counts, N, K, *, gated=False, k=1, gather=False, slots=None, bias=False, out="bf16", fn=None, extra=0,
                strided=False):
    """counts: rows of each expert; slots: slot of each expert; extra: rows of out behind the last expert's."""
    E, T = len(counts), sum(counts)
    parts = 2 if gated else 1
    fn = fn or ("silu" if gated else "none")
    S = E if slots is None else max(slots) + 1
    wq, ws, wv = expert_weights(S, parts * N, K, parts)
    X = max(T + extra, 1) if not gather else max((T + k - 1) // k, 1)
    xq, xs, xv = block_rows(_rand(T + K, X, K))
    perm = torch.randperm(T, generator=torch.Generator().manual_seed(T)) if gather else None
    b = _rand(9, S, parts * N) if bias else None
    off = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)
    kind = torch.bfloat16 if out == "bf16" else torch.float32
    od = torch.full((T + extra + 1, N + (5 if strided else 0)), 7.0, dtype=kind, device=DEV)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    rows = None
    if gather:  # rows behind the last expert's: addresses that must not be read
        rows = torch.cat([perm, torch.full((extra,), 2 ** 30)]).int()
    a = m.grouped_args(x=dev(xq), x_scale=dev(xs), w=dev(wq), w_scale=dev(ws), offsets=dev(off), rows=dev(rows),
                       rows_div=k, slot_of_expert=None if slots is None else torch.tensor(slots, dtype=torch.int32, device=DEV),
                       bias=dev(b), act=fn, gated=gated, out=od[:T + extra, :N])
    say(f"grouped E={E} T={T} max={max(counts)} N={N} K={K} gated={gated} k={k} gather={gather} slots={slots is not None} "
        f"bias={bias} out={out} extra={extra}")
    m.moe_linear_grouped(a)
    torch.cuda.synchronize()
    at = 0
    for e, n in enumerate(counts):
        if n:
            src = perm[at:at + n] // k if gather else torch.arange(at, at + n)
            s = e if slots is None else slots[e]
            want, tol = reference(xv[src].to(DEV), wv[s].to(DEV), None if b is None else b[s].to(DEV), fn, gated, None, N, K,
                                  out == "bf16")
            tol = tol + want.abs() * (2.0 ** -8 if out == "bf16" else U) + 1e-30
            got = od[at:at + n, :N].double()
            bad = ~((got - want).abs() <= tol)
            assert not bad.any(), (e, int(bad.sum()), torch.nonzero(bad)[:4], (got - want).abs()[bad].max())
        at += n
    assert torch.all(od[T:] == 7.0) and torch.all(od[:, N:] == 7.0)
    return od[:T, :N].clone()


CASES = [  # rows of the experts, N, K
    ([1], 16, 128), ([0, 1, 0], 130, 256), ([1, 1, 1, 1, 1, 1, 1, 1], 256, 1024), ([3, 0, 17, 1, 0, 16], 48, 384),
    ([0, 0, 40, 0], 200, 640), ([33, 1, 0, 64, 15, 90], 384, 256), ([200, 3, 129, 0, 1, 128], 264, 512),
    ([700, 20, 300, 5], 136, 1152)]


@pytest.mark.gpu
@pytest.mark.parametrize("counts,N,K", CASES)
def test_grouped_matches_the_formula(m, counts, N, K):
    need_gpu()
    run_grouped(m, counts, N, K)
    run_grouped(m, counts, N, K, gated=True, k=3, gather=True, extra=2)
    run_grouped(m, counts, N, K, gated=True, bias=True, out="f32", strided=True)
    run_grouped(m, counts, N, K, gather=True, k=2, bias=True, fn="gelu_tanh", extra=5,
                slots=[len(counts) - 1 - e for e in range(len(counts))])
    run_grouped(m, counts, N, K, gather=True, k=1, out="f32")


@pytest.mark.gpu
def test_grouped_experts_without_rows(m):
    """No rows at all: nothing is written; rows in one of 1024 experts; the last expert of 65 and of 130."""
    need_gpu()
    run_grouped(m, [0, 0, 0], 40, 128, extra=20)
    for E, e in ((1024, 1023), (1024, 512), (65, 64), (130, 129), (64, 63)):
        counts = [0] * E
        counts[e] = 5
        run_grouped(m, counts, 20, 128, slots=[0] * E, gather=True, k=2)
    counts = [1 if e % 3 == 0 else 0 for e in range(257)]
    counts[256] = 40
    run_grouped(m, counts, 20, 128, slots=[e % 4 for e in range(257)])


@pytest.mark.gpu
def test_grouped_shared_slots_and_rows(m):
    """Two experts in one slot, and one row of x read by many."""
    need_gpu()
    run_grouped(m, [20, 7, 33], 72, 256, slots=[1, 0, 1], gather=True, k=60)


# ------------------------------------------------------------------ refusals (CPU)

def _args(m, **kw):
    g = m.GroupedArgs()
    a = g.lin
    a.T, a.N, a.K, a.qmode, a.x, a.w, a.out, a.x_scale, a.w_scale = 8, 32, 128, 3, 0x10000, 0x20000, 0x30000, 0x40000, 0x50000
    g.x_rows, g.E, g.offsets, g.rows_div = 8, 4, 0x60000, 1
    for name, v in kw.items():
        setattr(a if hasattr(a, name) else g, name, v)
    return g


@pytest.mark.parametrize("kw,msg", [
    (dict(qmode=1), "qmode"), (dict(K=192), "128"), (dict(E=0), "E=0"), (dict(E=1025), "E=1025"), (dict(fn=7), "fn"),
    (dict(residual=0x70000), "residual"), (dict(rows=0x70000, rows_div=0), "rows_div"), (dict(x_rows=7), "x_rows"),
    (dict(rows=0x70000, x_rows=0), "x_rows"), (dict(ldx=120), "stride"), (dict(ldw=136), "stride"), (dict(ldo=31), "stride"),
    (dict(offsets=None), "null"), (dict(x=None), "null"), (dict(x_scale=None), "null"), (dict(w=0x20008), "16-byte"),
    (dict(offsets=0x60002), "misaligned"), (dict(rows=0x70001), "misaligned"), (dict(slot_of_expert=0x70002), "misaligned"),
    (dict(w_stride=8), "stride"), (dict(w_scale_stride=6), "stride"), (dict(T=-1), "bad sizes"), (dict(N=0), "bad sizes"),
    (dict(x_rows=1 << 20, ldx=4096), "2^32"), (dict(T=1 << 23, x_rows=1 << 23, N=100000), "grid")])
def test_grouped_refusals(m, kw, msg):
    with pytest.raises(m.MoeError) as e:
        m.moe_linear_grouped(_args(m, **kw), stream=0)
    assert e.value.status == 1 and msg in str(e.value)


def test_grouped_no_rows(m):
    assert m.moe_linear_grouped(_args(m, T=0, x_rows=0), stream=0) is None


def test_grouped_args_refuse_tensors(m):
    e4 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    ok = dict(x=e4(4, 128), x_scale=torch.zeros(1, 4), w=e4(2, 32, 128), w_scale=torch.zeros(2, 1, 1),
              offsets=torch.zeros(3, dtype=torch.int32), out=torch.zeros(4, 32, dtype=torch.bfloat16))
    for kw, msg in ((dict(w=e4(32, 128)), "dimensions"), (dict(w=e4(2, 30, 128)), "rows a slot"),
                    (dict(w=e4(1, 32, 128)), "slots"), (dict(gated=True), "rows a slot"), (dict(), "not on a GPU"),
                    (dict(x=torch.zeros(4, 128)), "float32")):
        with pytest.raises(m.MoeError) as e:
            m.grouped_args(**{**ok, **kw})
        assert msg in str(e.value)


def test_combine_bf16_refusals(m):
    for kw, msg in ((dict(k=17), "sizes"), (dict(T=65536), "sizes"), (dict(H=100), "sizes"), (dict(y=None), "null"),
                    (dict(y=0x10008), "aligned"), (dict(ysh=0x20008), "aligned")):
        a = dict(y=0x10000, inv=0x30000, w=0x40000, ysh=None, T=4, k=2, H=128, out=0x50000)
        a.update(kw)
        with pytest.raises(m.MoeError) as e:
            m.moe_combine_bf16(a["y"], a["inv"], a["w"], a["ysh"], a["T"], a["k"], a["H"], a["out"], stream=0)
        assert e.value.status == 1 and msg in str(e.value)


# ------------------------------------------------------------------ the layer

def layer_of(m, E=12, k=3, H=256, I=384, max_tokens=200, shared=True, router=None):
    from fp4_expert_ffn_amd.layer import BlockMoELayer
    gq, gs, gv = expert_weights(E, 2 * I, H, 2, seed=2)
    dq, ds, dv = expert_weights(E, H, I, 1, seed=3)
    sh = sv = None
    if shared:
        a, b, c = block_weights(_rand(4, 2 * I, H) / math.sqrt(H), 2)
        d, e, f = block_weights(_rand(5, H, I) / math.sqrt(I))
        sh, sv = tuple(t.to(DEV) for t in (a, b, d, e)), (c, f)
    layer = BlockMoELayer(E=E, k=k, H=H, I=I, max_tokens=max_tokens, gate_up=gq.to(DEV), gate_up_scale=gs.to(DEV),
                          down=dq.to(DEV), down_scale=ds.to(DEV), shared=sh, router=router, device=DEV)
    return layer, gv, dv, sv


def values(q, s):
    return q.cpu().view(torch.float8_e4m3fn).double() * s.cpu().double().t().repeat_interleave(128, 1)


def check_stages(layer, gv, dv, sv, x, T):
    """Every stage's output against its formula on what the stage before it wrote."""
    H, I, k, E = layer.H, layer.I, layer.k, layer.E
    xq, xs = layer._rows(layer.xq, layer.xs, T, H)
    check_block_codes(x.double(), xq, xs, 0.0)
    xv = values(xq, xs)
    off, perm = layer.offsets.cpu().tolist(), layer.perm[:T * k].cpu().long()
    hq, hs = layer._rows(layer.hq, layer.hs, T * k, I)
    check_block_codes(layer.h[:T * k].cpu().double(), hq, hs, 0.0)
    hv = values(hq, hs)
    near = lambda got, want, tol: torch.all((got.cpu().double() - want).abs() <= tol + want.abs() * 2.0 ** -8 + 1e-30)  # noqa: E731
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            assert near(layer.h[lo:hi], *reference(xv[perm[lo:hi] // k], gv[e], None, "silu", True, None, I, H, True))
            assert near(layer.y[lo:hi], *reference(hv[lo:hi], dv[e], None, "none", False, None, H, I, True))
    y = layer.y[:T * k].cpu().double()[layer.inv[:T * k].cpu().long()].view(T, k, H)
    w = layer.w[:T].cpu().double()
    want, mag = (w[:, :, None] * y).sum(1), (w[:, :, None] * y).abs().sum(1)
    if sv is not None:
        sv_h = values(*layer._rows(layer.sq, layer.ss, T, I))
        assert near(layer.shared_h[:T], *reference(xv, sv[0], None, "silu", True, None, I, H, True))
        assert near(layer.shared_y[:T], *reference(sv_h, sv[1], None, "none", False, None, H, I, True))
        ysh = layer.shared_y[:T].cpu().double()
        want, mag = want + ysh, mag + ysh.abs()
    assert near(layer.out[:T], want, 20 * U * mag)


@pytest.mark.gpu
@pytest.mark.parametrize("T,shared", [(1, True), (2, False), (16, True), (70, False), (200, True)])
def test_block_layer_stage_by_stage(m, T, shared):
    need_gpu()
    layer, gv, dv, sv = layer_of(m, shared=shared)
    x, logits = _rand(T, T, layer.H).to(torch.bfloat16), _rand(T + 1, T, layer.E)
    say("block layer", T, shared)
    layer.forward(x.to(DEV), logits=logits.to(DEV))
    torch.cuda.synchronize()
    check_stages(layer, gv, dv, sv, x, T)


@pytest.mark.gpu
def test_block_layer_behind_the_norm_and_in_front_of_the_head(m):
    """norm (bf16 and block rows) -> router -> experts -> norm -> vocabulary -> log probabilities, captured; the
    replays equal the eager call, with eager work on the same buffers between them."""
    need_gpu()
    from fp4_expert_ffn_amd.layer import TokenHead
    router = m.router(score="sigmoid", n_group=4, topk_group=2, group_rank="top2", scale=2.5)
    layer, gv, dv, sv = layer_of(m, router=router)
    T, H, V = 40, layer.H, 1000
    vq, vs, vv = block_weights(_rand(31, V, H) / math.sqrt(H))
    nw = (1 + 0.2 * _rand(32, H)).to(torch.bfloat16).to(DEV)
    head = TokenHead(H=H, V=V, fmt="fp8_block", max_tokens=T, norm_weight=nw, w=vq.to(DEV), w_scale=vs.to(DEV), k=5,
                     logits_f32=True, device=DEV)
    w_r = (_rand(33, layer.E, H) * 0.1).to(DEV)
    ids = torch.randint(V, (T,), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(DEV)
    x, res = torch.empty((T, H), dtype=torch.bfloat16, device=DEV), torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    n = torch.empty_like(x)
    q, s = torch.empty((T, H), dtype=torch.uint8, device=DEV), torch.empty((H // 128, T), device=DEV)

    def step(stream=None):
        m.moe_rmsnorm(m.norm_args(x=x, residual=res, weight=nw, residual_out=res, out=n, q=q, q_scale=s, qmode="fp8_block"), stream)
        y = layer.forward(n, w_router=w_r, rows=(q, s), stream=stream)
        return head.forward(y, res, ids=ids, scale=0.8, stream=stream)

    def load(seed):
        x.copy_(_rand(seed, T, H))
        res.copy_(_rand(seed + 1, T, H) * 2)

    say("block layer between norm and head")
    want = []
    for seed in (1, 11, 21):
        load(seed)
        want.append({k: v.clone() for k, v in step().items()})
    torch.cuda.synchronize()
    layer.xq[:T * H], layer.xs[:T * H // 128] = q.view(-1), s.view(-1)  # the norm's rows where check_stages looks
    check_stages(layer, gv, dv, sv, values(q, s), T)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    load(1)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        got = step(torch.cuda.current_stream())
    for i, seed in enumerate((1, 11, 21)):
        load(seed)
        g.replay()
        torch.cuda.synchronize()
        for k, v in want[i].items():
            assert torch.equal(got[k], v), (seed, k)
        load(5)
        step()  # eager work on the same buffers
        torch.cuda.synchronize()
    out = head.forward(layer.out[:T], res, ids=ids, scale=0.8)
    torch.cuda.synchronize()
    z = torch.log_softmax(out["logits"].cpu().double() * 0.8, 1)
    assert torch.allclose(out["logprob"].cpu().double(), z.gather(1, ids.cpu().long()[:, None])[:, 0], rtol=1e-6, atol=1e-6)
    assert torch.equal(out["top_ids"].cpu().long(), out["logits"].cpu().sort(dim=1, descending=True, stable=True)[1][:, :5])


@pytest.mark.gpu
def test_block_layer_refusals(m):
    need_gpu()
    from fp4_expert_ffn_amd.layer import BlockMoELayer
    layer, _, _, _ = layer_of(m, shared=False)
    x = _rand(1, 5, layer.H).to(torch.bfloat16)
    logits = _rand(2, 5, layer.E).to(DEV)
    for bad, msg in ((x, "cpu"), (x.to(DEV).float(), "float32"), (x.to(DEV)[:, :128], "shape"), (x.to(DEV)[:, ::2], "dense")):
        with pytest.raises(m.MoeError) as e:
            layer.forward(bad, logits=logits)
        assert e.value.status == 1 and msg in str(e.value)
    with pytest.raises(m.MoeError):
        BlockMoELayer(E=2, k=1, H=256, I=200, max_tokens=4, gate_up=None, gate_up_scale=None, down=None, down_scale=None, device=DEV)
