"""Timed cases of the dense operators around the expert layer: scored expert
routing, RMS norm with the residual's addition and 8-bit outputs, and the
linear product with its fused epilogue.

`run` computes one pass of a case: with `own` false in elementary torch
operations, with `own` true through this package's entry points.  `exact`
gives the same results in 64 bits, written apart from both.

Sizes are those of this repository's two layers (hidden 2048, 128 experts,
top-8, intermediate 768; hidden 7168, 256 experts, intermediate 2048), its
batches (1, 16, 2048 to 4096 tokens), the longest batch the permutation takes
(T * k = 131072), and odd ones in between.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the least row scale of an 8-bit row


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of the large layer: a sigmoid router whose bias balances the
        # load, 4 of 8 groups by their two best experts; latency counts
        dict(name="route one token", op="route", T=1, E=256, k=8, score="sigmoid", n_group=8, topk_group=4,
             rank="top2", renorm=True, scale=2.5, bias=True, masked=0),
        # a ragged prefill batch of the small layer: softmax scores with a bias, no groups, 8 experts masked out
        dict(name="route ragged prefill", op="route", T=4099, E=128, k=8, score="softmax", n_group=1, topk_group=1,
             rank="max", renorm=False, scale=1.0, bias=True, masked=8),
        # the longest batch the permutation takes, the large layer's router
        dict(name="route longest batch", op="route", T=16384, E=256, k=8, score="sigmoid", n_group=8, topk_group=4,
             rank="top2", renorm=True, scale=2.5, bias=True, masked=0),
        # one decode token in front of the large layer, bf16 out for the router and the experts
        dict(name="norm one token", op="norm", T=1, H=7168, residual="bf16", weight="bf16", out=True, q="none"),
        # a ragged prefill batch, fp32 residual stream, bf16 out and 8-bit rows with one scale each
        dict(name="norm ragged prefill fp8", op="norm", T=1027, H=2048, residual="f32", weight="f32", out=True,
             q="fp8"),
        # a long prefill batch of the large layer, 8-bit blocks of 32 for the linear product alone
        dict(name="norm long prefill mxfp8", op="norm", T=16384, H=7168, residual="bf16", weight="bf16", out=False,
             q="mxfp8"),
        # one decode token: the shared expert's (or a dense layer's) gate and up projections with SwiGLU
        dict(name="linear one token fp8", op="linear", T=1, N=2048, K=7168, fmt="fp8", act="silu", gated=True,
             bias=False, residual=False, out="bf16"),
        # a decode batch: a down projection added to the residual
        dict(name="linear 16 tokens mxfp8", op="linear", T=16, N=7168, K=2048, fmt="mxfp8", act="none", gated=False,
             bias=False, residual=True, out="bf16"),
        # a ragged batch between decode and prefill: a projection with a bias and GELU
        dict(name="linear ragged batch bf16", op="linear", T=333, N=2056, K=776, fmt="bf16", act="gelu_tanh",
             gated=False, bias=True, residual=False, out="bf16"),
        # prefill of the small layer's width, added to the residual
        dict(name="linear prefill bf16", op="linear", T=4096, N=2048, K=2048, fmt="bf16", act="none", gated=False,
             bias=True, residual=True, out="bf16"),
        # prefill of the large layer: down projection of 8-bit rows, added to the residual
        dict(name="linear prefill fp8", op="linear", T=4096, N=7168, K=2048, fmt="fp8", act="none", gated=False,
             bias=False, residual=True, out="bf16"),
        # prefill of the large layer: gate and up projections with SwiGLU, 8-bit blocks
        dict(name="linear prefill mxfp8", op="linear", T=4096, N=2048, K=7168, fmt="mxfp8", act="silu", gated=True,
             bias=False, residual=False, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "linear"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 3, 4, 8])
        per = max(4, _log(rng, 16, 512) // groups)
        E = groups * per
        taken = rng.randint(1, groups)
        T = _log(rng, 1, 16384)
        k = rng.randint(1, min(8, taken * per))
        return dict(op=op, T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), n_group=groups, topk_group=taken,
                    rank=rng.choice(["max", "top2"]), renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                    bias=rng.random() < 0.7, masked=rng.choice([0, 0, 2]))
    if op == "norm":
        q = rng.choice(["none", "fp8", "mxfp8"])
        H = _log(rng, 64, 8192)
        H = max(128, H // 128 * 128) if q == "mxfp8" else max(64, H // 8 * 8)
        T = min(_log(rng, 1, 16384), (16384 * 7168) // H)
        return dict(op=op, T=T, H=H, residual=rng.choice(["none", "bf16", "f32"]), weight=rng.choice(["bf16", "f32"]),
                    out=q == "none" or rng.random() < 0.5, q=q)
    fmt = rng.choice(["bf16", "fp8", "mxfp8"])
    step = {"bf16": 8, "fp8": 16, "mxfp8": 128}[fmt]
    T, N, K = _log(rng, 1, 4096), _log(rng, 16, 7168), max(step, _log(rng, 64, 7168) // step * step)
    gated = rng.random() < 0.3
    if gated:
        N = max(8, N // 2)
    return dict(op=op, T=T, N=N, K=K, fmt=fmt, act=rng.choice(["none", "silu", "gelu_tanh", "gelu_erf", "relu"]),
                gated=gated, bias=rng.random() < 0.5, residual=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))


def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 4 * (T * E + (E if c["bias"] else 0) + 4 * T * k + 2 * E + 1), "flops": 8 * T * E}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        r = {"none": 0, "bf16": 2, "f32": 4}[c["residual"]]
        n = T * H * (2 + 2 * r + (2 if c["out"] else 0) + (1 if c["q"] != "none" else 0))
        n += H * (2 if c["weight"] == "bf16" else 4)
        n += {"none": 0, "fp8": 4 * T, "mxfp8": T * H // 32}[c["q"]]
        return {"bytes": n, "flops": 6 * T * H}
    T, N, K = c["T"], c["N"], c["K"]
    R = 2 * N if c["gated"] else N
    b = 2 if c["fmt"] == "bf16" else 1
    n = (T + R) * K * b + T * N * ((2 if c["out"] == "bf16" else 4) + (2 if c["residual"] else 0))
    n += 4 * R if c["bias"] else 0
    n += {"bf16": 0, "fp8": 4 * (T + R), "mxfp8": (T + R) * K // 32}[c["fmt"]]
    return {"bytes": n, "flops": 2 * T * R * K}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rows_fp8(v):
    """fp32 rows as E4M3 codes with one fp32 scale a row."""
    s = (v.abs().amax(1) / E4M3_MAX).clamp_min(TINY)
    return (v / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def _rows_mxfp8(v):
    """fp32 rows as E4M3 codes with one power-of-two scale per 32 values; the
    scale codes K-tile-major: [K / 128, rows, 4]."""
    R, K = v.shape
    b = v.view(R, K // 32, 32)
    e = torch.frexp(b.abs().amax(2))[1] - 9
    q = torch.ldexp(b, -e[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(R, K).to(torch.float8_e4m3fn)
    codes = (e + 127).clamp(0, 254).to(torch.uint8)
    return q, codes.view(R, K // 128, 4).permute(1, 0, 2).contiguous()


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    randn = lambda *n: torch.randn(*n, device=DEV, generator=g)  # noqa: E731
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        c["logits"] = randn(T, E) * 1.5 + randn(E)  # popular and unpopular experts
        if c["masked"]:
            c["logits"][:, torch.randperm(E, device=DEV, generator=g)[: c["masked"]]] = -1e4
        c["bias_t"] = randn(E) * 0.1 if c["bias"] else None
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
        c["ids"], c["w"] = i32((T, k)), torch.empty((T, k), dtype=torch.float32, device=DEV)
        c["counts"], c["offsets"], c["perm"], c["inv"] = i32(E), i32(E + 1), i32(T * k), i32(T * k)
        if own:
            import fp4_expert_ffn_amd as m
            c["router"] = m.router(score=c["score"], n_group=c["n_group"], topk_group=c["topk_group"],
                                   group_rank=c["rank"], renormalize=c["renorm"], scale=c["scale"], bias=c["bias_t"])
        return c
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        loud = 1.0 + 15.0 * (torch.rand(H, device=DEV, generator=g) < 0.01)  # a few loud channels
        c["x"] = (randn(T, H) * loud).to(torch.bfloat16)
        kind = {"bf16": torch.bfloat16, "f32": torch.float32}
        c["eps"] = 1e-6
        c["w"] = (1.0 + 0.2 * randn(H)).to(kind[c["weight"]])
        c["res"] = (randn(T, H) * 2.0 * loud).to(kind[c["residual"]]) if c["residual"] != "none" else None
        c["res_out"] = torch.empty_like(c["res"]) if c["res"] is not None else None
        c["y"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV) if c["out"] else None
        c["codes"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV) if c["q"] != "none" else None
        c["scale"] = {"none": lambda: None, "fp8": lambda: torch.empty(T, dtype=torch.float32, device=DEV),
                      "mxfp8": lambda: torch.empty((H // 128, T, 4), dtype=torch.float8_e8m0fnu, device=DEV)}[c["q"]]()
        if own:
            import fp4_expert_ffn_amd as m
            c["args"] = m.norm_args(x=c["x"], weight=c["w"], eps=c["eps"], residual=c["res"], residual_out=c["res_out"],
                                    out=c["y"], q=c["codes"], q_scale=c["scale"], qmode=c["q"])
        return c
    T, N, K = c["T"], c["N"], c["K"]
    R = 2 * N if c["gated"] else N
    x, w = randn(T, K), randn(R, K) * (1.0 / math.sqrt(K))
    c["xs"] = c["ws"] = None
    if c["fmt"] == "bf16":
        c["x"], c["w"] = x.to(torch.bfloat16), w.to(torch.bfloat16)
    else:
        enc = _rows_fp8 if c["fmt"] == "fp8" else _rows_mxfp8
        (c["x"], c["xs"]), (c["w"], c["ws"]) = enc(x), enc(w)
    c["bias_t"] = randn(R) * 0.5 if c["bias"] else None
    c["res"] = randn(T, N).to(torch.bfloat16) if c["residual"] else None
    c["y"] = torch.empty((T, N), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV)
    if own:
        import fp4_expert_ffn_amd as m
        a = m.linear_args(x=c["x"], w=c["w"], fmt=c["fmt"], x_scale=c["xs"], w_scale=c["ws"], bias=c["bias_t"],
                          act=c["act"], gated=c["gated"], residual=c["res"], out=c["y"])
        n = m.moe_linear_workspace_size(a)
        c["ws_buf"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        a.workspace, a.workspace_bytes = c["ws_buf"].data_ptr(), n
        c["args"] = a
    return c


# ------------------------------------------------------------------ one pass

def _route_plain(c):
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    l = c["logits"].double()  # the choice between neighbouring experts: 64 bits
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        p = torch.exp(l - l.amax(1, keepdim=True))
        s = p / p.sum(1, keepdim=True)
    key = l if c["bias_t"] is None else s + c["bias_t"].double()
    if G > 1:
        # without a bias the experts are ordered by their logits; a group's
        # two best are summed as scores
        by = (s if c["bias_t"] is None and c["rank"] == "top2" else key).view(T, G, E // G)
        best = by.sort(dim=2, descending=True)[0][:, :, : 2 if c["rank"] == "top2" else 1].sum(2)
        take = best.sort(dim=1, descending=True, stable=True)[1][:, : c["topk_group"]]
        live = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, take, True)
        key = torch.where(live.repeat_interleave(E // G, 1), key, -math.inf)
    ids = key.sort(dim=1, descending=True, stable=True)[1][:, :k]
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (w * c["scale"]).float()
    flat = ids.reshape(-1)
    perm = flat.sort(stable=True)[1]
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k, device=l.device)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return {"ids": ids.int(), "w": w, "counts": counts.int(), "offsets": offsets.int(), "perm": perm.int(),
            "inv": inv.int()}


def _norm_plain(c):
    s = c["x"].float()
    out = {}
    if c["res"] is not None:
        s = s + c["res"].float()
        out["residual"] = s.to(c["res"].dtype)
    y = s * torch.rsqrt((s * s).mean(1, keepdim=True) + c["eps"]) * c["w"].float()
    if c["out"]:
        out["y"] = y.to(torch.bfloat16)
    if c["q"] == "fp8":
        out["q"], out["scale"] = _rows_fp8(y)
    elif c["q"] == "mxfp8":
        out["q"], codes = _rows_mxfp8(y)
        out["scale"] = codes.view(torch.float8_e8m0fnu)
    return out


def _widen(v, s, fmt):
    """Codes and scales as the fp32 values they stand for."""
    v = v.float()
    if fmt == "fp8":
        return v * s[:, None]
    if fmt == "mxfp8":
        R, K = v.shape
        e = s.permute(1, 0, 2).reshape(R, K // 32).int() - 127
        return torch.ldexp(v.view(R, K // 32, 32), e[:, :, None]).view(R, K)
    return v


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "gelu_erf":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return torch.where(z < 0, 0.0, z) if act == "relu" else z


def _linear_plain(c):
    z = _widen(c["x"], c["xs"], c["fmt"]) @ _widen(c["w"], c["ws"], c["fmt"]).t()
    if c["bias_t"] is not None:
        z = z + c["bias_t"]
    N = c["N"]
    y = _act(z[:, :N], c["act"]) * z[:, N:] if c["gated"] else _act(z, c["act"])
    if c["res"] is not None:
        y = y + c["res"].float()
    return {"y": y.to(c["y"].dtype)}


def _own(c):
    import fp4_expert_ffn_amd as m
    if c["op"] == "route":
        m.moe_route_scored_permute(c["router"], c["logits"], c["T"], c["E"], c["k"], c["ids"], c["w"], c["counts"],
                                   c["offsets"], c["perm"], c["inv"])
        return {n: c[n] for n in ("ids", "w", "counts", "offsets", "perm", "inv")}
    if c["op"] == "norm":
        m.moe_rmsnorm(c["args"])
        out = {"residual": c["res_out"], "y": c["y"], "q": c["codes"], "scale": c["scale"]}
        return {n: v for n, v in out.items() if v is not None}
    m.moe_linear(c["args"])
    return {"y": c["y"]}


def run(state):
    if own:
        return _own(state)
    return {"route": _route_plain, "norm": _norm_plain, "linear": _linear_plain}[state["op"]](state)


# ------------------------------------------------------------------ in 64 bits

def _exact_route(c):
    """numpy: scores, a lexicographic sort per row (key down, index up), and the permutation."""
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    l = c["logits"].cpu().numpy().astype(np.float64)
    b = None if c["bias_t"] is None else c["bias_t"].cpu().numpy().astype(np.float64)
    if c["score"] == "sigmoid":
        with np.errstate(over="ignore"):
            s = np.reciprocal(1.0 + np.exp(-l))
    else:
        s = np.exp(l - l.max(axis=1)[:, None])
        s /= s.sum(axis=1)[:, None]
    key = l.copy() if b is None else s + b[None]
    if G > 1:
        per = (s if b is None and c["rank"] == "top2" else key).reshape(T, G, E // G)
        if c["rank"] == "top2" and E // G > 1:
            best = np.partition(per, E // G - 2, axis=2)[:, :, -2:].sum(axis=2)
        else:
            best = per.max(axis=2)
        order = np.lexsort((np.broadcast_to(np.arange(G), (T, G)), -best), axis=1)
        dead = np.ones((T, G), bool)
        np.put_along_axis(dead, order[:, : c["topk_group"]], False, axis=1)
        key[np.repeat(dead, E // G, axis=1)] = -np.inf
    ids = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -key), axis=1)[:, :k]
    w = np.take_along_axis(s, ids, axis=1)
    if c["renorm"]:
        w = w / w.sum(axis=1)[:, None]
    f = ids.reshape(-1)
    perm = np.lexsort((np.arange(T * k), f))
    inv = np.argsort(perm)
    counts = np.array([np.count_nonzero(f == e) for e in range(E)])
    return {"ids": ids, "w": w * c["scale"], "counts": counts, "offsets": np.concatenate([[0], np.cumsum(counts)]),
            "perm": perm, "inv": inv}


def _exact_norm(c):
    s = c["x"].double()
    out = {}
    if c["res"] is not None:
        s = s + c["res"].double()
        out["residual"] = s
    y = s * c["w"].double() / torch.sqrt(s.square().sum(1, keepdim=True) / c["H"] + c["eps"])
    if c["out"]:
        out["y"] = y
    if c["q"] == "fp8":
        out["scale"] = torch.clamp(y.abs().max(1)[0] / E4M3_MAX, min=TINY)
        out["q"] = y / out["scale"].unsqueeze(1)
    elif c["q"] == "mxfp8":
        b = y.unflatten(1, (-1, 32))
        sc = torch.exp2(torch.floor(torch.log2(b.abs().max(2)[0])) - 8.0)
        out["q"] = torch.clamp(b / sc.unsqueeze(2), -E4M3_MAX, E4M3_MAX).flatten(1)
        out["scale"] = sc.unflatten(1, (-1, 4)).transpose(0, 1)
    return out


def _exact_linear(c):
    def wide(v, s):
        v = v.double()
        if c["fmt"] == "fp8":
            return v * s.double().unsqueeze(1)
        if c["fmt"] == "mxfp8":
            f = torch.exp2(s.double() - 127.0).transpose(0, 1).flatten(1)  # [rows, K / 32]
            return v * f.repeat_interleave(32, 1)
        return v
    z = torch.mm(wide(c["x"], c["xs"]), wide(c["w"], c["ws"]).t().contiguous())
    if c["bias_t"] is not None:
        z += c["bias_t"].double()
    a = z[:, : c["N"]]
    if c["act"] == "silu":
        a = a / (1.0 + torch.exp(-a))
    elif c["act"] == "gelu_tanh":
        a = a * 0.5 * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (a + 0.044715 * a ** 3)))
    elif c["act"] == "gelu_erf":
        a = a * 0.5 * (1.0 + torch.erf(a / 2.0 ** 0.5))
    elif c["act"] == "relu":
        a = torch.maximum(a, torch.zeros_like(a))
    if c["gated"]:
        a = a * z[:, c["N"]:]
    return {"y": a if c["res"] is None else a + c["res"].double()}


def exact(case, seed):
    c = prepare(case, seed)
    return {"route": _exact_route, "norm": _exact_norm, "linear": _exact_linear}[c["op"]](c)
