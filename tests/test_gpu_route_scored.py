"""Scored routing on the GPU through the C ABI against the rule in 64 bits.

The expert ids and the permutation have to be equal; a weight is one fp32
rounding (2^-24) of a value computed in 64 bits, with 2^-40 for the 64-bit
steps."""
import math

import numpy as np
import pytest

from tests.gpu_util import DEV, need_gpu, say, torch

TOL = 2.0 ** -24 + 2.0 ** -40


@pytest.fixture(scope="module")
def m():
    import fp4_expert_ffn_amd as m  # fails loudly if libmoe.so is missing
    return m


def _rank(v, i):
    """Sort key: larger first, NaN last, the lower index first among equals."""
    return (1, 0.0, i) if math.isnan(v) else (0, -v, i)


def rule(logits, k, *, score="softmax", n_group=1, topk_group=1, group_rank="max", renormalize=True, scale=1.0,
         bias=None):
    """The rule of include/moe.h, row by row in Python floats."""
    T, E = logits.shape
    gs = E // n_group
    ids, w = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        l = [float(v) for v in logits[t]]
        if score == "sigmoid":
            s = [v if math.isnan(v) else (1 / (1 + math.exp(-v)) if v > -700 else 0.0) for v in l]
            num, den = s, 1.0
        else:
            real = [v for v in l if not math.isnan(v)]
            top = max(real) if real else 0.0
            num = [v if math.isnan(v) else (1.0 if v == top else math.exp(v - top)) for v in l]
            den = sum(v for v in num if not math.isnan(v))
            s = [v / den if den > 0 else v for v in num]
        key = l if bias is None else [a + float(b) for a, b in zip(s, bias)]
        by = s if bias is None and group_rank == "top2" else key
        ranks = []
        for g in range(n_group):
            part = by[g * gs:(g + 1) * gs]
            real = sorted((-math.inf if math.isnan(v) else v for v in part), reverse=True)
            if group_rank == "top2" and gs > 1:
                ranks.append(real[0] + real[1])
            else:
                ranks.append(math.nan if all(math.isnan(v) for v in part) else real[0])
        live = set(sorted(range(n_group), key=lambda g: _rank(ranks[g], g))[:topk_group])
        order = sorted((e for e in range(E) if e // gs in live), key=lambda e: _rank(key[e], e))[:k]
        ids[t] = order
        sel = [0.0 if math.isnan(num[e]) else num[e] for e in order]
        d = sum(sel) if renormalize else den
        w[t] = [(v / d if d > 0 else 1.0 / k) * scale for v in sel]
    return ids, w


def _router(m, **kw):
    kw = dict(kw)
    b = kw.pop("bias", None)
    return m.router(bias=None if b is None else torch.from_numpy(np.asarray(b, np.float32)).to(DEV), **kw)


def run(m, logits, k, permute=True, **kw):
    T, E = logits.shape
    i32 = lambda *n: torch.full(n, -7, dtype=torch.int32, device=DEV)  # noqa: E731
    lg = torch.from_numpy(np.ascontiguousarray(logits, np.float32)).to(DEV)
    ids, w = i32(T + 1, k), torch.full((T + 1, k), -7.0, device=DEV)
    counts, offsets, perm, inv = i32(E), i32(E + 1), i32(T * k + 1), i32(T * k + 1)
    r = _router(m, **kw)
    say(f"route T={T} E={E} k={k} permute={permute}", {n: v for n, v in kw.items() if n != "bias"}, "bias" in kw)
    if permute:
        m.moe_route_scored_permute(r, lg, T, E, k, ids, w, counts, offsets, perm, inv)
    else:
        m.moe_route_scored(r, lg, T, E, k, ids, w)
    torch.cuda.synchronize()
    assert torch.all(ids[T] == -7) and torch.all(w[T] == -7.0)
    assert perm[T * k].item() == -7 and inv[T * k].item() == -7
    cpu = lambda t, n: t.cpu().numpy()[:n]  # noqa: E731
    return cpu(ids, T), cpu(w, T), cpu(counts, E), cpu(offsets, E + 1), cpu(perm, T * k), cpu(inv, T * k)


def check(m, logits, k, **kw):
    T, E = logits.shape
    ids, w = rule(logits, k, **kw)
    order = np.argsort(ids.reshape(-1), kind="stable")
    for permute in (True, False):
        gi, gw, gc, go, gp, gv = run(m, logits, k, permute, **kw)
        assert np.array_equal(gi, ids), np.argwhere(gi != ids)[:4]
        assert np.all(np.abs(gw - w) <= np.abs(w) * TOL + 1e-44), np.abs(gw / w - 1).max()
        if permute:
            assert np.array_equal(gc, np.bincount(ids.reshape(-1), minlength=E))
            assert np.array_equal(go, np.concatenate([[0], np.cumsum(gc)]))
            assert np.array_equal(gp, order) and np.array_equal(gv[gp], np.arange(T * k))


CASES = [  # T, E, k, router
    (1, 256, 8, dict(score="sigmoid", n_group=8, topk_group=4, group_rank="top2", scale=2.5)),
    (40, 256, 8, dict(score="sigmoid", n_group=8, topk_group=4, group_rank="top2", scale=2.5)),
    (200, 256, 8, dict(score="sigmoid", n_group=8, topk_group=4, group_rank="top2", renormalize=False)),
    (65, 128, 8, dict(score="softmax")), (64, 128, 6, dict(score="softmax", renormalize=False, scale=0.5)),
    (33, 60, 4, dict(score="softmax", n_group=4, topk_group=2, group_rank="max")),
    (33, 60, 6, dict(score="sigmoid", n_group=4, topk_group=3, group_rank="top2")),
    (17, 64, 1, dict(score="sigmoid", n_group=64, topk_group=16, group_rank="top2")),
    (9, 8, 2, dict(score="softmax", n_group=2, topk_group=1, group_rank="top2")),
    (5, 1024, 16, dict(score="sigmoid", n_group=16, topk_group=5, group_rank="top2")),
    (70, 1000, 16, dict(score="softmax", n_group=8, topk_group=8, group_rank="max")),
    (130, 512, 8, dict(score="sigmoid", n_group=8, topk_group=3, group_rank="max")),
    (3, 1, 1, dict(score="sigmoid")), (2, 2, 2, dict(score="softmax")), (70, 300, 5, dict(score="sigmoid")),
    (1500, 96, 8, dict(score="sigmoid", n_group=3, topk_group=2, group_rank="top2", scale=1.5)),
    (300, 160, 6, dict(score="softmax", n_group=5, topk_group=2, group_rank="top2")),
]


@pytest.mark.gpu
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T,E,k,kw", CASES)
def test_route_matches_the_rule(m, T, E, k, kw, biased):
    need_gpu()
    rng = np.random.default_rng(T * 1000 + E + biased)
    logits = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if biased else None
    check(m, logits, k, **kw, **({"bias": bias} if biased else {}))


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(score="softmax"), dict(score="sigmoid"),
                                dict(score="sigmoid", n_group=4, topk_group=2, group_rank="top2"),
                                dict(score="softmax", n_group=4, topk_group=2, group_rank="top2"),
                                dict(score="sigmoid", n_group=4, topk_group=2, group_rank="max", renormalize=False)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_special_rows(m, kw, biased):
    """Ties, masked experts, infinities, NaN, rows without a finite logit, tiny scores."""
    need_gpu()
    E, k = 64, 6
    rng = np.random.default_rng(5)
    inf, nan = np.inf, np.nan
    rows = [np.zeros(E), np.full(E, -inf), np.full(E, nan), np.full(E, -1e4), np.full(E, -100.0), np.full(E, 90.0)]
    r = rng.integers(-2, 3, (12, E)) / 2.0                # ties
    rows += list(r)
    a = rng.standard_normal(E)
    for mask in (-inf, -1e4, np.finfo(np.float32).min, nan):
        for keep in (0, 1, 3, 5, 7, 30):                  # experts left by the mask, among them fewer than k
            b = np.full(E, mask)
            pick = rng.permutation(E)[:keep]
            b[pick] = a[pick]
            rows.append(b)
    b = a.copy()
    b[3] = inf
    rows.append(b)
    b = a.copy()
    b[[5, 9, 60]] = inf
    rows.append(b)
    rows.append(rng.standard_normal(E) - 80.0)            # sigmoid scores near 1e-35
    rows.append(rng.standard_normal(E) * 30.0)
    logits = np.asarray(rows, np.float32)
    bias = None
    if biased:
        bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
        bias[[2, 40]] = -inf
        bias[7] = nan
        bias[11] = 5.0
    check(m, logits, k, **kw, **({"bias": bias} if biased else {}))


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [1, 8])
def test_route_near_ties(m, score, groups):
    """Keys that differ by less than an fp32 step of themselves, across ids and groups."""
    need_gpu()
    E, k, T = 256, 8, 96
    rng = np.random.default_rng(8)
    base = rng.standard_normal(T).astype(np.float32)
    steps = rng.integers(-3, 4, (T, E)).astype(np.float32)
    logits = (base[:, None] + steps * np.spacing(np.abs(base))[:, None]).astype(np.float32)
    bias = np.where(rng.random(E) < 0.5, 0.25, 0.25 + 2.0 ** -24).astype(np.float32)
    check(m, logits, k, score=score, n_group=groups, topk_group=min(groups, 3), group_rank="top2", bias=bias)
    check(m, logits, k, score=score, n_group=groups, topk_group=min(groups, 3), group_rank="top2")
    # saturated scores: exactly equal keys, the lower ids win
    check(m, np.full((70, E), 50.0, np.float32), k, score="sigmoid", n_group=groups, topk_group=min(groups, 3),
          group_rank="top2", bias=np.full(E, 0.5, np.float32))


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k", [(16384, 256, 8), (8193, 128, 8), (5000, 512, 16), (4097, 1024, 3), (4099, 24, 1)])
def test_route_long_batches(m, T, E, k):
    """Long batches against sorted 64-bit keys."""
    need_gpu()
    rng = np.random.default_rng(T)
    logits = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    logits[::3, : E // 2] -= 3.0  # uneven experts
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    gi, gw, gc, go, gp, gv = run(m, logits, k, True, score="sigmoid", bias=bias, scale=2.0)
    s = 1.0 / (1.0 + np.exp(-logits.astype(np.float64)))
    ids = np.argsort(-(s + bias.astype(np.float64)), axis=1, kind="stable")[:, :k]
    assert np.array_equal(gi, ids)
    w = np.take_along_axis(s, ids, 1)
    w = 2.0 * w / w.sum(1, keepdims=True)
    assert np.all(np.abs(gw - w) <= w * TOL)
    assert np.array_equal(gc, np.bincount(ids.reshape(-1), minlength=E))
    assert np.array_equal(go, np.concatenate([[0], np.cumsum(gc)]))
    assert np.array_equal(gp, np.argsort(ids.reshape(-1), kind="stable"))
    assert np.array_equal(gv[gp], np.arange(T * k))


# Both sides of where a batch is routed by a launch of its own: rows a workgroup takes at once, 1024 tokens a pass.
@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,G", [(8, 480, 8, 3), (9, 480, 8, 3), (16, 320, 8, 1), (17, 320, 8, 1), (32, 200, 8, 1),
                                     (33, 200, 8, 1), (64, 512, 8, 1), (65, 512, 8, 1), (2048, 210, 8, 3),
                                     (2049, 210, 8, 3), (4096, 320, 8, 1), (4097, 320, 8, 1), (8192, 480, 8, 3),
                                     (8193, 480, 8, 3), (2049, 200, 3, 1), (5, 1000, 16, 8), (4, 1000, 16, 8)])
def test_route_split_batches(m, T, E, k, G):
    need_gpu()
    rng = np.random.default_rng(T + E)
    logits = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    check(m, logits, k, score="sigmoid", n_group=G, topk_group=max(1, G - 1), group_rank="top2" if G > 1 else "max",
          bias=bias)


@pytest.mark.gpu
def test_route_no_tokens(m):
    need_gpu()
    c, o = torch.full((16,), -7, dtype=torch.int32, device=DEV), torch.full((17,), -7, dtype=torch.int32, device=DEV)
    m.moe_route_scored_permute(m.router(score="sigmoid"), None, 0, 16, 2, None, None, c, o, None, None)
    torch.cuda.synchronize()
    assert torch.all(c == 0) and torch.all(o == 0)


@pytest.mark.gpu
def test_softmax_router_equals_the_plain_routing(m):
    """Without bias and groups the choice is moe_route's."""
    need_gpu()
    rng = np.random.default_rng(2)
    logits = torch.from_numpy((rng.standard_normal((50, 128)) * 3).astype(np.float32)).to(DEV)
    a = [torch.empty((50, 8), dtype=d, device=DEV) for d in (torch.int32, torch.float32) * 2]
    for renorm in (True, False):
        m.moe_route(logits, 50, 128, 8, renorm, a[0], a[1])
        m.moe_route_scored(m.router(renormalize=renorm), logits, 50, 128, 8, a[2], a[3])
        torch.cuda.synchronize()
        assert torch.equal(a[0], a[2])
        assert torch.all((a[1] - a[3]).abs() <= a[3] * 2.0 ** -20)


@pytest.mark.parametrize("T,E,k,kw,msg", [
    (4, 64, 65, {}, "k=65"), (4, 64, 17, {}, "k=17"), (4, 64, 0, {}, "k=0"), (-1, 64, 2, {}, "bad sizes"),
    (4, 1025, 2, {}, "bad sizes"), (4, 0, 1, {}, "bad sizes"), (4, 64, 2, dict(n_group=3), "n_group"),
    (4, 1024, 2, dict(n_group=128), "n_group"), (4, 64, 2, dict(n_group=0), "n_group"),
    (4, 64, 2, dict(n_group=4, topk_group=5), "topk_group"), (4, 64, 2, dict(n_group=4, topk_group=0), "topk_group"),
    (4, 64, 9, dict(n_group=8, topk_group=1), "k=9"), (4, 64, 2, dict(score=5), "score"),
    (4, 64, 2, dict(group_rank=3), "group_rank"), (70000, 64, 2, {}, "131072"),
])
def test_route_refusals(m, T, E, k, kw, msg):
    r = m.router(**kw)
    with pytest.raises(m.MoeError) as e:
        m.moe_route_scored_permute(r, 0x1000, T, E, k, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 0x7000, stream=0)
    assert e.value.status == 1 and msg in str(e.value)
    if "131072" not in msg:
        with pytest.raises(m.MoeError) as e:
            m.moe_route_scored(r, 0x1000, T, E, k, 0x2000, 0x3000, stream=0)
        assert msg in str(e.value)


def test_route_refuses_nulls_and_bad_biases(m):
    for i in range(7):
        p = [0x1000 * (j + 1) for j in range(7)]
        p[i] = None
        with pytest.raises(m.MoeError) as e:
            m.moe_route_scored_permute(m.router(), p[0], 4, 64, 2, *p[1:], stream=0)
        assert "null" in str(e.value)
    for bias in (torch.zeros(64), torch.zeros(64, dtype=torch.float64)):
        with pytest.raises(m.MoeError):
            m.router(bias=bias)


def test_route_refuses_more_rows_than_a_grid_holds(m):
    for T in (1 << 25, (1 << 31) - 1):
        with pytest.raises(m.MoeError) as e:
            m.moe_route_scored(m.router(), 0x10000, T, 8, 2, 0x20000, 0x30000, stream=0)
        assert e.value.status == 1 and "bad sizes" in str(e.value)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,G", [(64, 512, 1), (1, 210, 3), (300, 480, 8), (300, 128, 1)])
def test_route_captured(m, T, E, G):
    """Replays with new logits give the eager results, whatever launches the batch takes."""
    need_gpu()
    k = 8
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    new = lambda: (i32(T, k), torch.empty((T, k), device=DEV), i32(E), i32(E + 1), i32(T * k), i32(T * k))  # noqa: E731
    r = m.router(score="softmax", n_group=G, topk_group=max(1, G // 2), group_rank="top2")
    lg = torch.zeros((T, E), device=DEV)
    a, b = new(), new()
    say(f"captured route T={T} E={E} G={G}")
    m.moe_route_scored_permute(r, lg, T, E, k, *a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_route_scored_permute(r, lg, T, E, k, *a)
    for seed in range(3):
        lg.copy_(torch.from_numpy(np.random.default_rng(seed).standard_normal((T, E)).astype(np.float32)))
        m.moe_route_scored_permute(r, lg, T, E, k, *b)
        for _ in range(2):
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_route_refuses_tensors(m):
    """Strided, short or mistyped tensors and tensors outside the GPU never reach the kernels."""
    lg = torch.zeros(4, 64)
    i, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for bad in ((lg.double(), i, w), (lg.t().contiguous().t(), i, w), (lg[:3], i, w), (lg, i.long(), w), (lg, i, w[:1]),
                (lg, i, w)):
        with pytest.raises(m.MoeError) as e:
            m.moe_route_scored(m.router(), bad[0], 4, 64, 2, bad[1], bad[2], stream=0)
        assert e.value.status == 1 and "dense" in str(e.value)


def test_cache_router_refusals(m):
    c = m.moe_cache_create(4, 1 << 20, 0, 2, 16)
    for layer, kw, msg in ((2, {}, "layer 2"), (-2, {}, "layer -2"), (0, dict(n_group=3), "n_group"),
                           (0, dict(score=9), "score")):
        with pytest.raises(m.MoeError) as e:
            m.moe_cache_use_router(c, layer, m.router(**kw))
        assert e.value.status == 1 and msg in str(e.value)
    m.moe_cache_use_router(c, -1, m.router(score="sigmoid", n_group=4, topk_group=2))
    m.moe_cache_use_router(c, 1, None)
    c.close()
