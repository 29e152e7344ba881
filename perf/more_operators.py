"""Timed cases of the 8-bit products with a scale for each block of 128 and of
the log probabilities of tokens:

  rows      E4M3 rows with one fp32 scale per 128 columns, from the RMS norm
            with the residual's addition or from bf16 rows alone
  linear    the dense product of such rows with weights that have one fp32
            scale per 128 x 128 block, and its fused epilogue
  experts   the same product over the rows of routed experts, each expert's
            rows by its own weights, which lie in slots of a pool
  logprobs  log probability and rank of one given token a row, the row's
            entropy and log sum, and its k best alternatives

`run` computes one pass of a case: with `own` false in elementary torch
operations, with `own` true through this package's entry points.  `exact`
gives the same results in 64 bits, written apart from both.

Sizes are those of this repository's two layers (hidden 2048, 128 experts,
top-8, intermediate 768; hidden 7168, 256 experts, intermediate 2048), its
batches (1, 16, 4096 tokens), generic vocabularies, and odd ones in between.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the least scale of a block
BLOCK = 128


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode token in front of the large layer: the norm writes the experts' operand; latency counts
        dict(name="rows one token norm", op="rows", T=1, H=7168, norm=True, residual=True),
        # SwiGLU outputs of a long routed batch, the down product's operand
        dict(name="rows long routed batch", op="rows", T=32768, H=2048, norm=False, residual=False),
        # one decode token: the large layer's shared expert, gate and up with SwiGLU
        dict(name="linear one token", op="linear", T=1, N=2048, K=7168, act="silu", gated=True, bias=False,
             residual=False, out="bf16"),
        # a decode batch: a down projection added to the residual
        dict(name="linear 16 tokens", op="linear", T=16, N=7168, K=2048, act="none", gated=False, bias=False,
             residual=True, out="bf16"),
        # a ragged batch, columns that end inside a block, fp32 logits of a head with a bias
        dict(name="linear ragged batch f32", op="linear", T=333, N=2056, K=896, act="none", gated=False, bias=True,
             residual=False, out="f32"),
        # prefill of the large layer's shared expert
        dict(name="linear prefill", op="linear", T=4096, N=2048, K=7168, act="silu", gated=True, bias=False,
             residual=False, out="bf16"),
        # one decode token of the large layer: 8 of 256 experts, their weights in a pool of 16 slots
        dict(name="experts one token", op="experts", T=1, k=8, E=256, slots=16, N=2048, K=7168, gated=True,
             gather=True),
        # a decode batch of the small layer: the down products of 128 routed rows
        dict(name="experts 16 tokens down", op="experts", T=16, k=8, E=128, slots=128, N=2048, K=768, gated=False,
             gather=False),
        # prefill of the small layer: gate and up with SwiGLU, rows gathered by the permutation
        dict(name="experts prefill", op="experts", T=4096, k=8, E=128, slots=128, N=768, K=2048, gated=True,
             gather=True),
        # one sampled token with the 20 alternatives that a client may ask for
        dict(name="logprobs one token", op="logprobs", T=1, V=131072, dtype="bf16", scale=1.25, top=20, masked=False),
        # a ragged batch under a grammar's mask: most of an odd vocabulary at -inf, fp32 logits
        dict(name="logprobs ragged masked", op="logprobs", T=333, V=50021, dtype="f32", scale=1.0, top=5,
             masked=True),
        # the scores of a long prompt's tokens
        dict(name="logprobs long prompt", op="logprobs", T=4096, V=131072, dtype="bf16", scale=1.0, top=1,
             masked=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "linear", "experts", "logprobs"])
    if op == "rows":
        H = max(1, _log(rng, 128, 8192) // BLOCK) * BLOCK
        T = min(_log(rng, 1, 32768), (32768 * 2048) // H)
        norm = rng.random() < 0.5
        return dict(op=op, T=T, H=H, norm=norm, residual=norm and rng.random() < 0.5)
    if op == "linear":
        T, N, K = _log(rng, 1, 4096), _log(rng, 16, 7168), max(1, _log(rng, 128, 7168) // BLOCK) * BLOCK
        gated = rng.random() < 0.4
        if gated:
            N = max(8, N // 4)
        T = min(T, 4096 * 4096 * 7168 // ((2 * N if gated else N) * K))
        return dict(op=op, T=T, N=N, K=K, act=rng.choice(["none", "silu", "gelu_tanh", "relu"]), gated=gated,
                    bias=rng.random() < 0.3, residual=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "experts":
        E = _log(rng, 4, 128)
        k = rng.randint(1, min(8, E))
        K = max(1, _log(rng, 256, 2048) // BLOCK) * BLOCK
        gated = rng.random() < 0.5
        N = _log(rng, 128, 768) if gated else _log(rng, 128, 1536)
        return dict(op=op, T=_log(rng, 1, 4096), k=k, E=E, slots=E, N=N, K=K, gated=gated, gather=rng.random() < 0.5)
    V = _log(rng, 1000, 131072)
    return dict(op=op, T=_log(rng, 1, 4096), V=V, dtype=rng.choice(["bf16", "f32"]) if V < 65536 else "bf16",
                scale=rng.choice([1.0, 1.25, 0.5]), top=rng.choice([0, 1, 5, 20]), masked=rng.random() < 0.3)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    c = case
    if c["op"] == "rows":
        n = c["T"] * c["H"]
        b = 3 * n + n // 32 + (4 * n if c["residual"] else 0) + (2 * c["H"] if c["norm"] else 0)
        return {"bytes": b, "flops": (8 if c["norm"] else 3) * n}
    if c["op"] == "logprobs":
        n = c["T"] * c["V"]
        return {"bytes": n * (2 if c["dtype"] == "bf16" else 4) + 4 * c["T"] * (5 + 2 * c["top"]), "flops": 5 * n}
    T, N, K = c["T"], c["N"], c["K"]
    R = 2 * N if c["gated"] else N
    wb = R * K + 4 * _blocks(N) * (R // N) * (K // BLOCK)
    if c["op"] == "linear":
        b = T * K + T * K // 32 + wb + T * N * ((2 if c["out"] == "bf16" else 4) + (2 if c["residual"] else 0))
        return {"bytes": b + (4 * R if c["bias"] else 0), "flops": 2 * T * R * K}
    rows = T * c["k"]
    # experts with rows: all of them once a batch is long (the routing is skewed, so a few stay idle)
    touched = min(c["E"], c["slots"], rows) if c["T"] > 1 else c["k"]
    x = T if c["gather"] else rows
    return {"bytes": touched * wb + x * K + x * K // 32 + rows * N * 2, "flops": 2 * rows * R * K}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _rows(v):
    """fp32 rows as E4M3 codes with one fp32 scale per 128 columns, the scales column block by column block."""
    T, K = v.shape
    b = v.view(T, K // BLOCK, BLOCK)
    s = (b.abs().amax(2) / E4M3_MAX).clamp_min(TINY)
    q = (b / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(T, K).to(torch.float8_e4m3fn)
    return q, s.t().contiguous()


def _weights(v, parts):
    """fp32 [parts * N, K] as E4M3 codes with one scale per 128 x 128 block of each part: [parts * blocks, K / 128]."""
    R, K = v.shape
    N, nb = R // parts, _blocks(R // parts)
    a = v.abs().view(parts, N, K // BLOCK, BLOCK).amax(3)
    pad = torch.zeros((parts, nb * BLOCK, K // BLOCK), device=v.device)
    pad[:, :N] = a
    s = (pad.view(parts, nb, BLOCK, K // BLOCK).amax(2) / E4M3_MAX).clamp_min(TINY)
    per_row = s.repeat_interleave(BLOCK, 1)[:, :N]
    q = (v.view(parts, N, K // BLOCK, BLOCK) / per_row[:, :, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.view(R, K).to(torch.float8_e4m3fn), s.view(parts * nb, K // BLOCK)


def _routing(T, k, E, g):
    """ids [T, k] by Zipf(1.1) popularity over a random order of the experts, and the stable permutation by expert."""
    rank = torch.randperm(E, device=DEV, generator=g).float() + 1.0
    u = torch.rand((T, E), device=DEV, generator=g).clamp_min(1e-20)
    ids = torch.topk(-1.1 * torch.log(rank) - torch.log(-torch.log(u)), k, dim=1)[1]
    flat = ids.reshape(-1)
    perm = flat.sort(stable=True)[1]
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return ids, perm.int(), offsets.int(), counts.tolist()


def _prepare_experts(c, g, randn):
    T, k, E, S, N, K = c["T"], c["k"], c["E"], c["slots"], c["N"], c["K"]
    parts = 2 if c["gated"] else 1
    R, rows = parts * N, T * k
    _, c["perm"], c["offsets"], c["counts"] = _routing(T, k, E, g)
    used = [e for e in range(E) if c["counts"][e]] if S < E else list(range(E))
    slot = torch.zeros(E, dtype=torch.int32, device=DEV)
    slot[torch.tensor(used, device=DEV)] = torch.randperm(S, device=DEV, generator=g)[: len(used)].int()
    c["slot"], c["slot_list"] = slot, slot.tolist()
    c["w"] = torch.empty((S, R, K), dtype=torch.float8_e4m3fn, device=DEV)
    c["ws"] = torch.empty((S, parts * _blocks(N), K // BLOCK), device=DEV)
    for s in range(S):
        c["w"][s], c["ws"][s] = _weights(randn(R, K) * (1.0 / math.sqrt(K)), parts)
    c["x"], c["xs"] = _rows(randn(T if c["gather"] else rows, K))
    c["y"] = torch.empty((rows, N), dtype=torch.bfloat16, device=DEV)
    c["act"] = "silu" if c["gated"] else "none"
    if own:
        import fp4_expert_ffn_amd as m
        c["args"] = m.grouped_args(x=c["x"], x_scale=c["xs"], w=c["w"], w_scale=c["ws"], offsets=c["offsets"],
                                   rows=c["perm"] if c["gather"] else None, rows_div=k, slot_of_expert=c["slot"],
                                   act=c["act"], gated=c["gated"], out=c["y"])
    return c


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    randn = lambda *n: torch.randn(*n, device=DEV, generator=g)  # noqa: E731
    if c["op"] == "experts":
        return _prepare_experts(c, g, randn)
    T = c["T"]
    if c["op"] == "rows":
        H = c["H"]
        loud = 1.0 + 15.0 * (torch.rand(H, device=DEV, generator=g) < 0.01)  # a few loud channels
        c["x"] = (randn(T, H) * loud).to(torch.bfloat16)
        c["eps"] = 1e-6
        c["w"] = (1.0 + 0.2 * randn(H)).to(torch.bfloat16) if c["norm"] else None
        c["res"] = (randn(T, H) * 2.0 * loud).to(torch.bfloat16) if c["residual"] else None
        c["res_out"] = torch.empty_like(c["res"]) if c["residual"] else None
        c["q"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
        c["qs"] = torch.empty((H // BLOCK, T), dtype=torch.float32, device=DEV)
        if own and c["norm"]:
            import fp4_expert_ffn_amd as m
            c["args"] = m.norm_args(x=c["x"], weight=c["w"], eps=c["eps"], residual=c["res"],
                                    residual_out=c["res_out"], q=c["q"], q_scale=c["qs"], qmode="fp8_block")
        return c
    if c["op"] == "linear":
        N, K = c["N"], c["K"]
        parts = 2 if c["gated"] else 1
        c["x"], c["xs"] = _rows(randn(T, K))
        c["w"], c["ws"] = _weights(randn(parts * N, K) * (1.0 / math.sqrt(K)), parts)
        c["bias_t"] = randn(parts * N) * 0.5 if c["bias"] else None
        c["res"] = randn(T, N).to(torch.bfloat16) if c["residual"] else None
        c["y"] = torch.empty((T, N), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV)
        if own:
            import fp4_expert_ffn_amd as m
            a = m.linear_args(x=c["x"], w=c["w"], fmt="fp8_block", x_scale=c["xs"], w_scale=c["ws"], bias=c["bias_t"],
                              act=c["act"], gated=c["gated"], residual=c["res"], out=c["y"])
            n = m.moe_linear_workspace_size(a)
            c["ws_buf"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
            a.workspace, a.workspace_bytes = c["ws_buf"].data_ptr(), n
            c["args"] = a
        return c
    V, k = c["V"], c["top"]
    c["logits"] = (randn(T, V) * 2.0 + 2.0 * randn(V)).to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
    ids = torch.randint(V, (T,), device=DEV, generator=g)
    if c["masked"]:  # nine tokens in ten are not allowed at a position; the given one is
        cut = torch.rand((T, V), device=DEV, generator=g) < 0.9
        cut[torch.arange(T, device=DEV), ids] = False
        c["logits"].masked_fill_(cut, -math.inf)
    c["ids"] = ids.int()
    f32 = lambda *n: torch.empty(n, dtype=torch.float32, device=DEV)  # noqa: E731
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    c["lp"], c["lse"], c["ent"], c["rank"] = f32(T), f32(T), f32(T), i32(T)
    c["top_lp"], c["top_ids"] = (f32(T, k), i32(T, k)) if k else (None, None)
    if own:
        import fp4_expert_ffn_amd as m
        a = m.logprob_args(logits=c["logits"], scale=c["scale"], ids=c["ids"], logprob=c["lp"], rank=c["rank"],
                           entropy=c["ent"], lse=c["lse"], top_ids=c["top_ids"], top_logprob=c["top_lp"])
        n = m.moe_logprobs_workspace_size(a)
        c["ws_buf"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        a.workspace, a.workspace_bytes = c["ws_buf"].data_ptr(), n
        c["args"] = a
    return c


# ------------------------------------------------------------------ one pass

def _rows_plain(c):
    v = c["x"].float()
    out = {}
    if c["norm"]:
        if c["residual"]:
            v = v + c["res"].float()
            out["residual"] = v.to(torch.bfloat16)
        v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + c["eps"]) * c["w"].float()
    out["q"], out["scale"] = _rows(v)
    return out


def _wide_rows(q, s):
    T, K = q.shape
    return (q.float().view(T, K // BLOCK, BLOCK) * s.t()[:, :, None]).view(T, K)


def _wide_weights(q, s, parts):
    R, K = q.shape
    per_row = s.view(parts, -1, K // BLOCK).repeat_interleave(BLOCK, 1)[:, : R // parts].reshape(R, K // BLOCK)
    return (q.float().view(R, K // BLOCK, BLOCK) * per_row[:, :, None]).view(R, K)


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return torch.where(z < 0, 0.0, z) if act == "relu" else z


def _linear_plain(c):
    z = _wide_rows(c["x"], c["xs"]) @ _wide_weights(c["w"], c["ws"], 2 if c["gated"] else 1).t()
    if c["bias_t"] is not None:
        z = z + c["bias_t"]
    N = c["N"]
    y = _act(z[:, :N], c["act"]) * z[:, N:] if c["gated"] else _act(z, c["act"])
    if c["res"] is not None:
        y = y + c["res"].float()
    return {"y": y.to(c["y"].dtype)}


def _experts_plain(c):
    x = _wide_rows(c["x"], c["xs"])
    if c["gather"]:
        x = x[torch.div(c["perm"], c["k"], rounding_mode="floor").long()]
    N, at = c["N"], 0
    for e, n in enumerate(c["counts"]):  # one product an expert
        if n:
            s = c["slot_list"][e]
            z = x[at: at + n] @ _wide_weights(c["w"][s], c["ws"][s], 2 if c["gated"] else 1).t()
            c["y"][at: at + n] = _act(z[:, :N], "silu") * z[:, N:] if c["gated"] else z
            at += n
    return {"y": c["y"]}


def _logprobs_plain(c):
    T, V = c["T"], c["V"]
    raw = c["logits"].float()
    l = raw * c["scale"]
    m = l.amax(1, keepdim=True)
    d = l - m
    e = torch.exp(d)
    s0 = e.sum(1, dtype=torch.float64)
    s1 = torch.where(e > 0, d * e, 0.0).sum(1, dtype=torch.float64)
    log_s = torch.log(s0)
    ids = c["ids"].long()[:, None]
    given = raw.gather(1, ids)
    at = torch.arange(V, device=raw.device)[None]
    out = {"logprob": (d.gather(1, ids)[:, 0] - log_s).float(), "lse": (m[:, 0] + log_s).float(),
           "entropy": (log_s - s1 / s0).float(),
           "rank": ((raw > given) | ((raw == given) & (at < ids))).sum(1).int()}
    if c["top"]:
        bits = (raw + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) - at  # value up, then index down
        best = torch.topk(key, c["top"], dim=1)[1]
        out["top_ids"], out["top_logprob"] = best.int(), (d.gather(1, best) - log_s[:, None]).float()
    return out


def _own(c):
    import fp4_expert_ffn_amd as m
    if c["op"] == "rows":
        if not c["norm"]:
            m.moe_quantize_fp8(c["x"], c["T"], c["H"], "fp8_block", c["q"], c["qs"])
            return {"q": c["q"], "scale": c["qs"]}
        m.moe_rmsnorm(c["args"])
        return {**({"residual": c["res_out"]} if c["residual"] else {}), "q": c["q"], "scale": c["qs"]}
    if c["op"] == "logprobs":
        m.moe_logprobs(c["args"])
        out = {"logprob": c["lp"], "lse": c["lse"], "entropy": c["ent"], "rank": c["rank"]}
        return {**out, "top_ids": c["top_ids"], "top_logprob": c["top_lp"]} if c["top"] else out
    if c["op"] == "linear":
        m.moe_linear(c["args"])
    else:
        m.moe_linear_grouped(c["args"])
    return {"y": c["y"]}


def run(state):
    if own:
        return _own(state)
    return {"rows": _rows_plain, "linear": _linear_plain, "experts": _experts_plain,
            "logprobs": _logprobs_plain}[state["op"]](state)


# ------------------------------------------------------------------ in 64 bits

def _exact_rows(c):
    v = c["x"].double()
    out = {}
    if c["norm"]:
        if c["res"] is not None:
            v = v + c["res"].double()
            out["residual"] = v
        v = v * c["w"].double() / torch.sqrt(v.square().sum(1, keepdim=True) / c["H"] + c["eps"])
    b = v.unflatten(1, (-1, BLOCK))
    s = torch.clamp(b.abs().max(2)[0] / E4M3_MAX, min=TINY)
    out["q"], out["scale"] = (b / s.unsqueeze(2)).flatten(1), s.transpose(0, 1)
    return out


def _exact_product(x, xs, w, ws, gated):
    """Block by block of K: the codes' sums, times the scales of their rows and column blocks."""
    R, K = w.shape
    N = R // 2 if gated else R
    col = torch.arange(R, device=w.device)
    block = torch.div(col % N, BLOCK, rounding_mode="floor") + torch.div(col, N, rounding_mode="floor") * _blocks(N)
    z = torch.zeros((x.shape[0], R), dtype=torch.float64, device=w.device)
    for b in range(K // BLOCK):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        p = torch.mm(x[:, at].double(), w[:, at].double().t().contiguous())
        z += p * xs[b].double().unsqueeze(1) * ws[block, b].double().unsqueeze(0)
    return z


def _exact_linear(c):
    z = _exact_product(c["x"], c["xs"], c["w"], c["ws"], c["gated"])
    if c["bias_t"] is not None:
        z += c["bias_t"].double()
    a = z[:, : c["N"]]
    if c["act"] == "silu":
        a = a / (1.0 + torch.exp(-a))
    elif c["act"] == "gelu_tanh":
        a = a * 0.5 * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (a + 0.044715 * a ** 3)))
    elif c["act"] == "relu":
        a = torch.maximum(a, torch.zeros_like(a))
    if c["gated"]:
        a = a * z[:, c["N"]:]
    return {"y": a if c["res"] is None else a + c["res"].double()}


def _exact_experts(c):
    src = torch.arange(c["T"] * c["k"], device=DEV)
    if c["gather"]:
        src = c["perm"].long() // c["k"]
    y = torch.zeros((c["T"] * c["k"], c["N"]), dtype=torch.float64, device=DEV)
    bounds = c["offsets"].tolist()
    for e in range(c["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo < hi:
            s, r = c["slot_list"][e], src[lo:hi]
            z = _exact_product(c["x"].view(torch.uint8)[r].view(torch.float8_e4m3fn), c["xs"][:, r], c["w"][s],
                               c["ws"][s], c["gated"])
            y[lo:hi] = z[:, c["N"]:] * (z[:, : c["N"]] * torch.sigmoid(z[:, : c["N"]])) if c["gated"] else z
    return {"y": y}


def _exact_logprobs(c):
    """Row by row: probabilities by a softmax in 64 bits, the order by a stable sort."""
    T, k, ids = c["T"], c["top"], c["ids"].tolist()
    f64 = lambda *n: torch.empty(n, dtype=torch.float64, device=DEV)  # noqa: E731
    out = {"logprob": f64(T), "lse": f64(T), "entropy": f64(T), "rank": torch.empty(T, dtype=torch.int64, device=DEV)}
    if k:
        out["top_ids"] = torch.empty((T, k), dtype=torch.int64, device=DEV)
        out["top_logprob"] = f64(T, k)
    for t in range(T):
        l = c["logits"][t].double() * c["scale"]
        z = torch.logsumexp(l, 0)
        lp = l - z
        p = torch.exp(lp)
        live = p > 0
        order = torch.sort(c["logits"][t].double(), descending=True, stable=True)[1]
        out["logprob"][t], out["lse"][t] = lp[ids[t]], z
        out["entropy"][t] = -(p[live] * lp[live]).sum()
        out["rank"][t] = torch.nonzero(order == ids[t])[0, 0]
        if k:
            out["top_ids"][t], out["top_logprob"][t] = order[:k], lp[order[:k]]
    return out


def exact(case, seed):
    c = prepare(case, seed)
    return {"rows": _exact_rows, "linear": _exact_linear, "experts": _exact_experts,
            "logprobs": _exact_logprobs}[c["op"]](c)
