"""Log probabilities, ranks, entropies and alternatives, on the GPU through
the C ABI, against the definitions in 64 bits.

Tolerances (u = 2^-24).  d = scale (l - m) log2(e) takes three roundings, each
of at most u |d|, and exp2 1 ulp: a term e is off by (3 |d| + 2) u of itself
(the base-2 |d| times ln 2 is the base-e one, so 3 |d_e| u too).  A thread adds
at most a = V / 256 + 8 terms in fp32: a u of the sum.  So s0 is off by at most
u (3 E|d| + a + 2) of itself, E|d| the mean distance from the maximum, which is
entropy-like: E|d| = log s0 - entropy.  log s0 moves by as much, absolutely; s1
/ s0 by u (3 E d^2 + (a + 5) E|d|) more.  Outputs add their own rounding, u of
the value; d of a single token is exact to 64 bits."""
import math

import pytest

from tests.gpu_util import DEV, need_gpu, say, torch

U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


def definition(l, scale, ids, k):
    """64 bits, CPU; l [T,V] in its own type."""
    T, V = l.shape
    scale = torch.tensor(scale, dtype=torch.float32).item()  # as the call takes it
    v = l.double()
    key = torch.where(torch.isnan(v), -math.inf, v)
    # NaN behind -inf: two stable sorts
    order = key.sort(dim=1, descending=True, stable=True)[1]
    last = torch.isnan(v.gather(1, order)).int().sort(dim=1, stable=True)[1]
    order = order.gather(1, last)
    mx = key.amax(1, keepdim=True)
    d = torch.where(v == mx, 0.0, (v - mx) * scale)  # inf - inf: 0
    d = torch.where(torch.isnan(v), math.nan, d)
    e = torch.exp(d)
    s0 = e.sum(1)
    dz = torch.where(d == -math.inf, 0.0, d)
    s1 = (dz * e).sum(1)
    s2 = (dz * dz * e).sum(1)
    logs = torch.log(s0)
    lp = d - logs[:, None]
    out = {"lse": scale * mx[:, 0] + logs, "entropy": logs - s1 / s0, "lp": lp, "order": order,
           "mean": -s1 / s0, "square": s2 / s0, "max": mx[:, 0]}
    if ids is not None:
        i = ids.long().clamp(0, V - 1)[:, None]
        out["logprob"] = lp.gather(1, i)[:, 0]
        out["rank"] = (order == i).int().argmax(1)
        nan = torch.isnan(v.gather(1, i)[:, 0])
        out["rank"][nan] = -1
        out["logprob"][ids >= V], out["rank"][ids >= V] = math.nan, -1
        out["logprob"][ids < 0], out["rank"][ids < 0] = 0.0, -1
    return out


def near(got, want, tol):
    got = got.cpu().double()
    want = torch.where(want.abs() > torch.finfo(torch.float32).max, torch.sign(want) * math.inf, want)  # fp32 outputs
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    return same | ((got - want).abs() <= tol + want.abs() * U)


def run(m, l, scale=1.0, ids=None, k=0, pad=0, shift=0, ws_fill=0xFF):
    """l [T,V] (CPU): placed `shift` elements into its memory, rows `pad` elements longer, NaN around them."""
    T, V = l.shape
    buf = torch.full((T * (V + pad) + shift + 8,), float("nan"), dtype=l.dtype, device=DEV)
    ld = buf[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
    ld.copy_(l)
    f = lambda *n, t=torch.float32: torch.full(n, 7, dtype=t, device=DEV)  # noqa: E731
    lp, rank, ent, lse = f(T + 1), f(T + 1, t=torch.int32), f(T + 1), f(T + 1)
    ti, tl = (f(T + 1, k, t=torch.int32), f(T + 1, k)) if k else (None, None)
    given = dict(ids=ids.to(DEV), logprob=lp[:T], rank=rank[:T]) if ids is not None else {}
    a = m.logprob_args(logits=ld, scale=scale, entropy=ent[:T], lse=lse[:T], top_ids=ti[:T] if k else None,
                       top_logprob=tl[:T] if k else None, **given)
    n = m.moe_logprobs_workspace_size(a)
    ws = torch.full((n + 256,), ws_fill, dtype=torch.uint8, device=DEV)
    a.workspace, a.workspace_bytes = ws.data_ptr(), n
    say(f"logprobs T={T} V={V} {l.dtype} scale={scale} k={k} pad={pad} shift={shift} ws={n}")
    m.moe_logprobs(a)
    torch.cuda.synchronize()
    w = definition(l, scale, ids, k)
    a = V / 256 + 8
    tol0 = U * (3 * w["mean"] + a + 2)
    tol0 = torch.where(torch.isfinite(tol0), tol0, 0.0)
    tol1 = tol0 + U * (3 * torch.nan_to_num(w["square"]) + (a + 5) * torch.nan_to_num(w["mean"]))
    assert near(lse[:T], w["lse"], tol0).all(), (lse[:T].cpu().double() - w["lse"]).abs().max()
    assert near(ent[:T], w["entropy"], tol1).all(), (ent[:T].cpu().double() - w["entropy"]).abs().max()
    if ids is not None:
        assert near(lp[:T], w["logprob"], tol0).all(), (lp[:T].cpu().double() - w["logprob"]).abs().max()
        assert torch.equal(rank[:T].cpu().long(), w["rank"].long())
    if k:
        best = w["order"][:, :k]
        assert torch.equal(ti[:T].cpu().long(), best), torch.nonzero(ti[:T].cpu().long() != best)[:5]
        assert near(tl[:T], w["lp"].gather(1, best), tol0[:, None]).all()
        assert torch.all(ti[T] == 7) and torch.all(tl[T] == 7)
    for t in (lp, rank, ent, lse):
        assert torch.all(t[T:] == 7)
    assert torch.all(ws[n:] == ws_fill)
    return {"lse": lse[:T], "entropy": ent[:T], "logprob": lp[:T], "rank": rank[:T]}


def logits(T, V, dtype="bf16", seed=0, std=3.0):
    g = torch.Generator().manual_seed(seed + T * 31 + V)
    return (torch.randn(T, V, generator=g) * std).to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def tokens(T, V, seed=1):
    return torch.randint(V, (T,), generator=torch.Generator().manual_seed(seed + T), dtype=torch.int32)


SHAPES = [(1, 1), (1, 2), (3, 7), (2, 64), (5, 100), (1, 2047), (1, 2048), (1, 2049), (7, 5000), (600, 999), (1, 50021),
          (16, 32768), (33, 4097), (513, 2100), (1, 131072), (2, 200003)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", SHAPES)
def test_logprobs_match_the_definition(m, T, V, dtype):
    """bf16 logits have many equal values: the order among them is by id."""
    need_gpu()
    l, ids = logits(T, V, dtype), tokens(T, V)
    run(m, l, 1.0, ids, min(V, 20))
    run(m, l, 0.7, ids, 0, pad=3, shift=1)
    run(m, l, 1.3, None, min(V, 64), pad=1, shift=3)
    run(m, l, 2.0, ids, 1, pad=8)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [300, 40000])
@pytest.mark.parametrize("order", ["up", "down", "equal", "steps"])
def test_logprobs_of_ordered_rows(m, V, order):
    """Rows in ascending, descending and no order: every logit passes the list, or none does; equal ones by id."""
    need_gpu()
    at = torch.arange(V, dtype=torch.float32)
    v = {"up": at / V * 20, "down": -at / V * 20, "equal": at * 0 + 1.5, "steps": torch.floor(at / 70) % 5}[order]
    for T in (1, 3, 600):
        run(m, v.repeat(T, 1), 1.0, tokens(T, V), 64)
        run(m, v.repeat(T, 1).to(torch.bfloat16), 1.0, tokens(T, V), 33)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [37, 5000, 40000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_masked_rows(m, V, dtype):
    """-inf and the type's lowest value as masks; rows of nothing else, of one token, of fewer tokens than k; infinite
    and NaN logits."""
    need_gpu()
    inf, nan = math.inf, math.nan
    low = torch.finfo(torch.bfloat16 if dtype == "bf16" else torch.float32).min
    l = logits(12, V, dtype)
    l[0] = -inf
    l[1] = low
    l[2], l[2, V // 2] = -inf, 3.0
    l[3], l[3, V - 1] = low, -2.0
    l[4, ::2] = -inf
    l[5, :V - 3] = -inf
    l[6, 5] = inf
    l[7, 3], l[7, V - 2] = inf, inf
    l[8, V // 3] = nan
    l[9] = nan
    l[10, 1], l[10, 2], l[10, 3] = inf, nan, -inf
    l[11] = -inf
    l[11, 7] = nan
    ids = torch.tensor([3, 4, V // 2, 0, 1, V - 1, 5, 0, 2, 3, 1, 8], dtype=torch.int32)
    run(m, l, 1.0, ids, min(V, 20))
    run(m, l, 1.0, ids, min(V, 64), shift=1, pad=1)
    ids = torch.tensor([-1, V, 2 ** 31 - 1, -2 ** 31, V - 1, 0, 7, V - 2, V // 3, -5, 3, 7], dtype=torch.int32)
    run(m, l, 0.5, ids, 1)
    run(m, l[8:9], 1.0, ids[8:9], min(V, 40))


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 300, 8192, 8193, 40000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_best_alone(m, V, dtype):
    """k = 1: the first of equal largest logits, +0 and -0 among them, wherever they stand; rows cut and whole, and
    pieces of a row that are masked throughout."""
    need_gpu()
    kind = torch.bfloat16 if dtype == "bf16" else torch.float32
    for T in (1, 3, 700):
        l = torch.full((T, V), -1.0)
        l[0] = 0.0
        l[0, ::2] = -0.0
        for t in range(1, min(T, 50)):
            l[t, t * 37 % V:] = 2.5
        if T > 60:
            l[50:60] = -math.inf
            for t in range(51, 60):
                l[t, t * 797 % V] = -3.0 * t
        for shift, pad in ((0, 0), (1, 3)):
            run(m, l.to(kind), 1.0, tokens(T, V), 1, pad=pad, shift=shift)


@pytest.mark.gpu
def test_logprobs_huge_and_tiny(m):
    """Logits over the whole range of their type; a nearly certain row; scales from 1e-3 to 1e3."""
    need_gpu()
    V = 3000
    l = logits(4, V, "f32")
    l[0] *= 1e37
    l[1] *= 1e-38
    l[2, 17] = 60.0
    for scale in (1e-3, 1.0, 1e3):
        run(m, l, scale, tokens(4, V), 20)


@pytest.mark.gpu
def test_logprobs_pieces_do_not_matter(m):
    """The order, ranks and top tokens of a row are those of the same row in a longer batch, where it is not cut."""
    need_gpu()
    V = 20000
    l, ids = logits(1, V), tokens(1, V)
    one = run(m, l, 1.0, ids, 20)
    many = run(m, l.repeat(600, 1), 1.0, ids.repeat(600), 20)
    assert torch.all(many["rank"] == one["rank"][0])


@pytest.mark.gpu
def test_logprobs_captured_and_on_streams(m):
    """Two captured calls with workspaces of their own, replayed in turn with eager work between; a side stream."""
    need_gpu()
    T, V, k = 2, 60000, 10
    ls = [logits(T, V, "bf16", seed=s).to(DEV) for s in (1, 2, 3)]
    ids = tokens(T, V).to(DEV)

    def call(buf, stream=None):
        o = {"logprob": torch.empty(T, device=DEV), "lse": torch.empty(T, device=DEV), "entropy": torch.empty(T, device=DEV),
             "rank": torch.empty(T, dtype=torch.int32, device=DEV), "top_logprob": torch.empty((T, k), device=DEV),
             "top_ids": torch.empty((T, k), dtype=torch.int32, device=DEV)}
        a = m.logprob_args(logits=buf, ids=ids, **o)
        ws = torch.empty(m.moe_logprobs_workspace_size(a), dtype=torch.uint8, device=DEV)
        a.workspace, a.workspace_bytes = ws.data_ptr(), ws.numel()
        o["_keep"] = (a, ws)
        return o, lambda s=stream: m.moe_logprobs(a, s)

    say("logprobs, captured")
    want = []
    for l in ls:
        o, go = call(l)
        go()
        want.append(o)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        buf = torch.empty_like(ls[0])
        o, go = call(buf)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            go(torch.cuda.current_stream())
        graphs.append((g, buf, o))
    for i in range(6):
        g, buf, o = graphs[i % 2]
        buf.copy_(ls[i % 3])
        g.replay()
        torch.cuda.synchronize()
        for n in ("logprob", "lse", "entropy", "rank", "top_ids", "top_logprob"):
            assert torch.equal(o[n], want[i % 3][n]), (i, n)
        call(ls[(i + 1) % 3])[1]()
    with torch.cuda.stream(side):
        o, go = call(ls[0])
        go()
    side.synchronize()
    assert torch.equal(o["top_ids"], want[0]["top_ids"]) and torch.equal(o["lse"], want[0]["lse"])


# ------------------------------------------------------------------ refusals (CPU)

def _ok(m, **kw):
    a = dict(logits=0x10000, T=4, V=100, entropy=0x20000)
    a.update(kw)
    return m.logprob_args(**a)


@pytest.mark.parametrize("kw,msg", [
    (dict(T=-1), "bad sizes"), (dict(T=1 << 22), "bad sizes"), (dict(V=0), "bad sizes"), (dict(V=1 << 30), "bad sizes"),
    (dict(k=65, top_ids=0x30000), "bad sizes"), (dict(V=10, k=11, top_ids=0x30000), "bad sizes"),
    (dict(k=3), "without top_ids"), (dict(top_ids=0x30000), "with top_ids"), (dict(scale=0.0), "scale"),
    (dict(scale=-1.0), "scale"), (dict(scale=float("inf")), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(entropy=None), "no output"), (dict(logprob=0x30000), "need ids"), (dict(rank=0x30000), "need ids"),
    (dict(ld=99), "stride"), (dict(logits=0x10001), "misaligned"), (dict(logits=0x10002, logits_f32=True), "misaligned"),
    (dict(entropy=0x20002), "misaligned"), (dict(ids=0x30001), "misaligned")])
def test_logprobs_refusals(m, kw, msg):
    with pytest.raises(m.MoeError) as e:
        m.moe_logprobs(_ok(m, **kw), stream=0)
    assert e.value.status == 1 and msg in str(e.value)


def test_logprobs_null_and_empty(m):
    a = _ok(m)
    a.logits = None
    with pytest.raises(m.MoeError) as e:
        m.moe_logprobs(a, stream=0)
    assert "null" in str(e.value)
    assert m.moe_logprobs(_ok(m, T=0), stream=0) is None


def test_logprobs_workspace(m):
    assert m.moe_logprobs_workspace_size(_ok(m, T=4096, V=50000)) == 0
    a = _ok(m, T=1, V=100000, k=20, top_ids=0x30000)
    n = m.moe_logprobs_workspace_size(a)
    assert n > 20 * 8
    for p, size, status, msg in ((None, n, 4, "workspace"), (0x40000, n - 1, 4, "workspace"), (0x40008, n, 1, "16-byte")):
        a.workspace, a.workspace_bytes = p, size
        with pytest.raises(m.MoeError) as e:
            m.moe_logprobs(a, stream=0)
        assert e.value.status == status and msg in str(e.value)


def test_logprob_args_refuse_tensors(m):
    l = torch.zeros(4, 100)
    for kw, msg in ((dict(logits=l[0]), "[T, V]"), (dict(logits=l, entropy=torch.zeros(4)), "not on a GPU"),
                    (dict(logits=l.half()), "float16"), (dict(logits=0x10000, T=4, V=100, ids=torch.zeros(4)), "float32"),
                    (dict(logits=0x10000, T=4, V=100, entropy=torch.zeros(5)), "shape")):
        with pytest.raises(m.MoeError) as e:
            m.logprob_args(**kw)
        assert msg in str(e.value)
