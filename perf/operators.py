"""The operators around and inside a sparse expert layer, as measured cases.

Five operators, each reached through the package's public functions:

* ``route``       logits -> top-K experts and weights (softmax or sigmoid
                  scores, correction bias, routing groups, renormalisation),
                  and the gradient of the weights in the logits;
* ``block_norm``  h' = a h + g RMSNorm(y), x = RMSNorm(h'): the norm after one
                  block and the norm before the next, with the gate and the
                  residual scale, and all their gradients;
* ``quantize``    values -> 8-bit floating point (e4m3) with a scale for each
                  128 values of a row;
* ``matmul``      the product of two such matrices (weights: a scale for each
                  128 x 128 block);
* ``experts``     the same product grouped by expert.

``run`` computes a case in its plain form (elementary torch operations) or,
with ``own`` set, by the package's kernels; ``exact`` computes it in 64 bits.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -126
BLOCK = 128

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "bf16": 2}


# ---- cases -------------------------------------------------------------------


def _route(name, tokens, experts, top_k, score="sigmoid", bias=True, groups=1, kept=1, best=2,
           renorm=True, scale=5.0, dtype="f32", train=False):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top_k": top_k,
            "score": score, "bias": bias, "groups": groups, "kept": kept, "best": best,
            "renorm": renorm, "scale": scale, "dtype": dtype, "train": train}


def _norm(name, tokens, width, stream="bf16", dtype="bf16", gate="channel", train=False):
    return {"name": name, "op": "norm", "tokens": tokens, "width": width, "stream": stream,
            "dtype": dtype, "gate": gate, "train": train}


def _quant(name, rows, cols, dtype="bf16"):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "dtype": dtype}


def _mm(name, rows, n, k, out="bf16"):
    return {"name": name, "op": "matmul", "rows": rows, "n": n, "k": k, "out": out}


def _experts(name, tokens, top_k, experts, n, k, gather, out="bf16"):
    return {"name": name, "op": "experts", "tokens": tokens, "top_k": top_k, "experts": experts,
            "n": n, "k": k, "gather": gather, "out": out}


def listed():
    return [
        # the router of one decode step of 32 sequences
        _route("route_decode", 32, 512, 22),
        # a prompt's tokens through group-limited routing (8 groups, 4 kept)
        _route("route_prompt_grouped", 8192, 512, 22, groups=8, kept=4),
        # a training step with a softmax router on a ragged batch and an odd expert count
        _route("route_train", 8111, 509, 8, score="softmax", bias=False, renorm=True, scale=1.0,
               dtype="bf16", train=True),
        # between two blocks of a decode step
        _norm("norm_decode", 32, 8192),
        # between two blocks of a training step on a ragged batch, gated per token and channel,
        # with an fp32 residual stream
        _norm("norm_train", 4099, 8192, stream="f32", gate="full", train=True),
        # a prompt's activations ahead of a product
        _quant("quantize_prompt", 8192, 8192),
        # the shared expert's hidden rows of a speculative-verify batch
        _quant("quantize_verify", 192, 10240),
        # one token through the shared expert's up projection
        _mm("matmul_token", 1, 10240, 8192),
        # a speculative-verify batch (192 tokens, ragged) through the latent projection
        _mm("matmul_verify", 187, 2048, 8192),
        # a prompt through the shared expert's up projection
        _mm("matmul_prompt", 8192, 10240, 8192),
        # a decode batch through the experts' up projection (rows gathered from the latent)
        _experts("experts_decode", 32, 22, 512, 5120, 2048, True),
        # a prompt through the experts' down projection
        _experts("experts_prompt", 8192, 22, 512, 2048, 5120, False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "norm", "quantize", "matmul", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log_int(rng, 8, 1024 // groups)
        kept = rng.randint(1, groups)
        top_k = rng.randint(1, min(32, kept * (experts // groups)))
        return _route("", _log_int(rng, 1, 8192), experts, top_k,
                      score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.5,
                      groups=groups, kept=kept, best=rng.choice([1, 2]),
                      renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5, 5.0]),
                      dtype=rng.choice(["f32", "bf16"]), train=rng.random() < 0.5)
    if op == "norm":
        width = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            width = max(64, width // 64 * 64)
        return _norm("", _log_int(rng, 1, 8192), width, stream=rng.choice(["bf16", "f32"]),
                     dtype=rng.choice(["bf16", "bf16", "f32"]),
                     gate=rng.choice(["channel", "token", "full", "none"]),
                     train=rng.random() < 0.5)
    if op == "quantize":
        return _quant("", _log_int(rng, 1, 16384), 16 * _log_int(rng, 8, 640),
                      dtype=rng.choice(["bf16", "f32"]))
    if op == "matmul":
        return _mm("", _log_int(rng, 1, 8192), 16 * _log_int(rng, 16, 640),
                   BLOCK * _log_int(rng, 2, 80), out=rng.choice(["bf16", "f32"]))
    experts = _log_int(rng, 8, 256)
    return _experts("", _log_int(rng, 1, 4096), rng.randint(1, min(8, experts)), experts,
                    16 * _log_int(rng, 16, 160), BLOCK * _log_int(rng, 2, 20),
                    rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))


# ---- inputs ------------------------------------------------------------------


def _fp8_values(q):
    return q.to(torch.float32)


def _plain_quantize(x):
    """(codes, scales): each 128 consecutive values of a row scaled by their
    largest magnitude / 448 and rounded to the nearest e4m3 value."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = x.to(torch.float32)
    if nb * BLOCK != cols:
        v = torch.cat([v, v.new_zeros(rows, nb * BLOCK - cols)], 1)
    v = v.view(rows, nb, BLOCK)
    top = torch.full((), E4M3_MAX, device=x.device)
    s = (v.abs().amax(2) / top).clamp_min(MIN_SCALE)
    q = (v / s[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(rows, nb * BLOCK)[:, :cols].contiguous(), s


def _quantize_weight(w):
    """(codes, scales) of w [N, K] with one scale for each 128 x 128 block."""
    n, k = w.shape
    nb, kb = -(-n // BLOCK), k // BLOCK
    v = w.to(torch.float32)
    if nb * BLOCK != n:
        v = torch.cat([v, v.new_zeros(nb * BLOCK - n, k)], 0)
    v = v.view(nb, BLOCK, kb, BLOCK)
    top = torch.full((), E4M3_MAX, device=w.device)
    s = (v.abs().amax((1, 3)) / top).clamp_min(MIN_SCALE)
    q = (v / s[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(nb * BLOCK, k)[:n].contiguous(), s


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    st = dict(case)
    op = case["op"]
    if op == "route":
        t, e = case["tokens"], case["experts"]
        st["logits"] = randn(t, e, dtype=_DTYPES[case["dtype"]])
        st["beta"] = randn(e, std=0.1) if case["bias"] else None
        st["dw"] = randn(t, case["top_k"]) if case["train"] else None
        if own:
            import sparse_moe_layer_latentmoe_amd as lmoe
            st["router"] = lmoe.make_router(
                e, case["top_k"], score=(lmoe.SCORE_SOFTMAX if case["score"] == "softmax"
                                         else lmoe.SCORE_SIGMOID),
                n_group=case["groups"], topk_group=case["kept"], group_score=case["best"],
                renormalise=case["renorm"], scale=case["scale"])
    elif op == "norm":
        t, d = case["tokens"], case["width"]
        hs, ys = _DTYPES[case["stream"]], _DTYPES[case["dtype"]]
        st["h"] = randn(t, d, std=3.0, dtype=hs)
        st["y"] = randn(t, d, dtype=ys)
        bf = torch.bfloat16
        st["pre"] = (1.0 + randn(d, std=0.1)).to(bf)
        st["post"] = (1.0 + randn(d, std=0.1)).to(bf)
        st["alpha"] = (1.0 + randn(d, std=0.05)).to(bf)
        gate = case["gate"]
        st["gate_t"] = {"channel": lambda: randn(d, std=0.3, dtype=bf),
                        "token": lambda: randn(t, 1, std=0.3, dtype=bf),
                        "full": lambda: randn(t, d, std=0.3, dtype=bf),
                        "none": lambda: None}[gate]()
        if case["train"]:
            st["dh_out"] = randn(t, d, dtype=hs)
            st["dx"] = randn(t, d, dtype=ys)
    elif op == "quantize":
        v = randn(case["rows"], case["cols"])
        # rows of different size, as activations are
        v *= torch.exp(randn(case["rows"], 1))
        st["x"] = v.to(_DTYPES[case["dtype"]])
    elif op == "matmul":
        st["xc"], st["xs"] = _plain_quantize(randn(case["rows"], case["k"], dtype=torch.bfloat16))
        st["wc"], st["ws"] = _quantize_weight(randn(case["n"], case["k"], std=0.02))
    else:
        t, k_, e, n, k = (case[i] for i in ("tokens", "top_k", "experts", "n", "k"))
        rows = t * k_
        pick = torch.rand((t, e), generator=g, device=dev).topk(k_, 1).indices.sort(1).values
        order = torch.sort(pick.reshape(-1), stable=True).indices
        counts = torch.bincount(pick.reshape(-1), minlength=e)
        ends = torch.cumsum(counts, 0)
        st["offsets"] = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
        st["bounds"] = st["offsets"].tolist()
        # gathered: sorted row i reads token order[i] // top_k; else rows are in expert order
        st["index"] = (order // k_).to(torch.int32) if case["gather"] else None
        xrows = t if case["gather"] else rows
        xc = torch.empty(xrows, k, dtype=torch.float8_e4m3fn, device=dev)
        xs = torch.empty(xrows, k // BLOCK, device=dev)
        for r in range(0, xrows, 16384):
            m = min(16384, xrows - r)
            x = randn(m, k)
            # hidden rows hold squares of rectified values; the latent is signed
            x = x if case["gather"] else torch.relu(x) ** 2
            xc[r:r + m], xs[r:r + m] = _plain_quantize(x.to(torch.bfloat16))
        st["xc"], st["xs"] = xc, xs
        st["wc"] = torch.empty(e, n, k, dtype=torch.float8_e4m3fn, device=dev)
        st["ws"] = torch.empty(e, -(-n // BLOCK), k // BLOCK, device=dev)
        for i in range(e):
            st["wc"][i], st["ws"][i] = _quantize_weight(randn(n, k, std=0.02))
    return st


# ---- plain forms -------------------------------------------------------------


def _plain_scores(logits, score):
    """Scores in 64 bits (selection compares values next to each other)."""
    v = logits.to(torch.float64)
    if score == "softmax":
        ex = torch.exp(v - v.amax(1, keepdim=True))
        return ex / ex.sum(1, keepdim=True)
    return 1.0 / (1.0 + torch.exp(-v))


def _plain_route(st):
    t, e, k = st["tokens"], st["experts"], st["top_k"]
    s = _plain_scores(st["logits"], st["score"])
    if st["beta"] is not None:
        key = s + st["beta"].to(torch.float64)
        biased = key
    else:
        key = st["logits"].to(torch.float64)
        biased = s
    if st["groups"] > 1:
        per = biased.view(t, st["groups"], e // st["groups"])
        best = torch.sort(per, dim=2, descending=True).values[:, :, :st["best"]].sum(2)
        first = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :st["kept"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, first, True)
        keep = keep[:, :, None].expand_as(per).reshape(t, e)
        key = torch.where(keep, key, torch.full_like(key, -math.inf))
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    idx = torch.sort(idx, dim=1).values
    sel = torch.gather(s, 1, idx)
    w = sel / (sel.sum(1, keepdim=True) + 1e-20) if st["renorm"] else sel
    out = [idx.to(torch.int32), (w * st["scale"]).to(torch.float32)]
    if st["train"]:
        dsel = st["dw"].to(torch.float64) * st["scale"]
        if st["renorm"]:
            tot = sel.sum(1, keepdim=True) + 1e-20
            dsel = (dsel - (dsel * sel).sum(1, keepdim=True) / tot) / tot
        ds = torch.zeros_like(s).scatter_(1, idx, dsel)
        if st["score"] == "softmax":
            dl = s * (ds - (ds * s).sum(1, keepdim=True))
        else:
            dl = ds * s * (1.0 - s)
        out.append(dl.to(st["logits"].dtype))
    return out


def _plain_norm(st):
    f = torch.float32
    d = st["width"]
    eps = 1e-5
    h, y = st["h"].to(f), st["y"].to(f)
    pre, post, alpha = st["pre"].to(f), st["post"].to(f), st["alpha"].to(f)
    gate = 1.0 if st["gate_t"] is None else st["gate_t"].to(f)
    ry = 1.0 / torch.sqrt((y * y).sum(1, keepdim=True) / d + eps)
    n = post * (y * ry)
    h2 = alpha * h + gate * n
    rh = 1.0 / torch.sqrt((h2 * h2).sum(1, keepdim=True) / d + eps)
    x = pre * (h2 * rh)
    out = {"h": h2.to(st["h"].dtype), "x": x.to(st["y"].dtype)}
    if st["train"]:
        dho, dx = st["dh_out"].to(f), st["dx"].to(f)
        hn = h2 * rh
        a = pre * dx
        big = dho + rh * (a - hn * ((a * hn).sum(1, keepdim=True) / d))
        yn = y * ry
        b = big * gate * post
        out["dh"] = (alpha * big).to(st["h"].dtype)
        out["dy"] = (ry * (b - yn * ((b * yn).sum(1, keepdim=True) / d))).to(st["y"].dtype)
        out["dpre"] = (dx * hn).sum(0).to(st["pre"].dtype)
        out["dpost"] = (big * gate * yn).sum(0).to(st["post"].dtype)
        out["dalpha"] = (big * h).sum(0).to(st["alpha"].dtype)
        if st["gate_t"] is not None:
            dg = big * n
            if st["gate"] == "channel":
                dg = dg.sum(0)
            elif st["gate"] == "token":
                dg = dg.sum(1, keepdim=True)
            out["dgate"] = dg.to(st["gate_t"].dtype)
    return out


def _plain_values(q, s, rows_per_scale):
    """The fp32 values that codes [R, K] with block scales stand for."""
    r, k = q.shape
    s = s.repeat_interleave(rows_per_scale, 0)[:r] if rows_per_scale > 1 else s
    return (_fp8_values(q).view(r, -1, BLOCK) * s[:, :, None]).view(r, k)


def _plain_matmul(st):
    x = _plain_values(st["xc"], st["xs"], 1)
    w = _plain_values(st["wc"], st["ws"], BLOCK)
    return torch.matmul(x, w.t()).to(_DTYPES[st["out"]])


def _plain_experts(st):
    rows = st["tokens"] * st["top_k"]
    y = torch.empty(rows, st["n"], dtype=_DTYPES[st["out"]], device=st["xc"].device)
    b = st["bounds"]
    for i in range(st["experts"]):
        if b[i] == b[i + 1]:
            continue
        if st["index"] is None:
            q, s = st["xc"][b[i]:b[i + 1]], st["xs"][b[i]:b[i + 1]]
        else:
            at = st["index"][b[i]:b[i + 1]].to(torch.int64)
            q, s = st["xc"].view(torch.uint8)[at].view(torch.float8_e4m3fn), st["xs"][at]
        x = _plain_values(q, s, 1)
        w = _plain_values(st["wc"][i], st["ws"][i], BLOCK)
        y[b[i]:b[i + 1]] = torch.matmul(x, w.t()).to(y.dtype)
    return y


def _run_plain(st):
    op = st["op"]
    if op == "route":
        return _plain_route(st)
    if op == "norm":
        return _plain_norm(st)
    if op == "quantize":
        q, s = _plain_quantize(st["x"])
        return {"values": q, "scales": s}
    if op == "matmul":
        return _plain_matmul(st)
    return _plain_experts(st)


# ---- the package's kernels -----------------------------------------------------


def _run_own(st):
    import sparse_moe_layer_latentmoe_amd as lmoe
    op = st["op"]
    if op == "route":
        idx, w = lmoe.route_logits(st["router"], st["logits"], bias=st["beta"])
        if not st["train"]:
            return [idx, w]
        return [idx, w, lmoe.route_logits_backward(st["router"], st["logits"], idx, st["dw"])]
    if op == "norm":
        par = dict(pre_weight=st["pre"], post_weight=st["post"], gate=st["gate_t"],
                   res_scale=st["alpha"], eps=1e-5)
        if not st["train"]:
            h2, x, _ = lmoe.block_norm(st["h"], st["y"], **par)
            return {"h": h2, "x": x}
        h2, x, stats = lmoe.block_norm(st["h"], st["y"], want_stats=True, **par)
        g = lmoe.block_norm_backward(st["h"], st["y"], stats, dh_out=st["dh_out"], dx=st["dx"],
                                     **par)
        out = {"h": h2, "x": x, "dh": g.dh, "dy": g.dy, "dpre": g.dpre_weight,
               "dpost": g.dpost_weight, "dalpha": g.dres_scale}
        if st["gate_t"] is not None:
            out["dgate"] = g.dgate
        return out
    if op == "quantize":
        q, s = lmoe.quantize_fp8(st["x"])
        return {"values": q, "scales": s}
    out = _DTYPES[st["out"]]
    if op == "matmul":
        return lmoe.fp8_matmul(st["xc"], st["xs"], st["wc"], st["ws"], out_dtype=out)
    return lmoe.fp8_matmul(st["xc"], st["xs"], st["wc"], st["ws"], offsets=st["offsets"],
                           rows=st["index"], out_dtype=out)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without --------------------------------------------


def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        el = _BYTES[case["dtype"]]
        b = t * e * el + (4 * e if case["bias"] else 0) + t * k * 8
        # a score is about ten operations, the selection one comparison an expert
        f = 11 * t * e
        if case["train"]:
            b += t * k * 4 + t * e * el
            f += 4 * t * e
        return {"bytes": b, "flops": f}
    if op == "norm":
        t, d = case["tokens"], case["width"]
        hb, yb = _BYTES[case["stream"]], _BYTES[case["dtype"]]
        gb = {"channel": 2 * d, "token": 2 * t, "full": 2 * t * d, "none": 0}[case["gate"]]
        b = t * d * 2 * (hb + yb) + 6 * d + gb
        f = 10 * t * d
        if case["train"]:
            b += t * d * 2 * (hb + yb) + 6 * d + gb
            f += 25 * t * d
        return {"bytes": b, "flops": f}
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (_BYTES[case["dtype"]] + 1) + n // BLOCK * 4, "flops": 3 * n}
    n, k = case["n"], case["k"]
    if op == "matmul":
        rows, xrows, used = case["rows"], case["rows"], 1.0
    else:
        rows = case["tokens"] * case["top_k"]
        xrows = case["tokens"] if case["gather"] else rows
        # experts that a token at random picks at least once
        e = case["experts"]
        used = e * (1.0 - (1.0 - case["top_k"] / e) ** case["tokens"])
    b = xrows * (k + 4 * (k // BLOCK)) + used * (n * k + 4 * (-(-n // BLOCK)) * (k // BLOCK))
    b += rows * n * _BYTES[case["out"]]
    return {"bytes": int(b), "flops": 2 * rows * n * k}


# ---- definitions in 64 bits ----------------------------------------------------


def _exact_route(case, st):
    z = st["logits"].double()
    t, e = z.shape
    k, rho = case["top_k"], case["scale"]
    if case["score"] == "softmax":
        lse = torch.logsumexp(z, 1, keepdim=True)
        s = torch.exp(z - lse)
    else:
        s = torch.sigmoid(z)
    b = s if st["beta"] is None else s + st["beta"].double()
    order = z if st["beta"] is None else b
    allowed = torch.ones_like(z, dtype=torch.bool)
    if case["groups"] > 1:
        gs = b.reshape(t, case["groups"], -1).topk(case["best"], 2).values.sum(2)
        better = (gs[:, None, :] > gs[:, :, None]).sum(2)
        lower = torch.ones(case["groups"], case["groups"], device=z.device).tril(-1).bool()
        better = better + ((gs[:, None, :] == gs[:, :, None]) & lower).sum(2)
        allowed = (better < case["kept"]).repeat_interleave(e // case["groups"], 1)
    # an expert is taken when fewer than k allowed experts come before it
    chosen = torch.zeros_like(allowed)
    lower = torch.ones(e, e, device=z.device).tril(-1).bool()
    step = max(1, (1 << 28) // (e * e))
    for r in range(0, t, step):
        o, al = order[r:r + step], allowed[r:r + step]
        before = (o[:, None, :] > o[:, :, None]) | ((o[:, None, :] == o[:, :, None]) & lower)
        chosen[r:r + step] = al & ((before & al[:, None, :]).sum(2) < k)
    idx = chosen.nonzero()[:, 1].reshape(t, k)
    p = s[chosen].reshape(t, k)
    total = p.sum(1, keepdim=True) + 1e-20 if case["renorm"] else torch.ones_like(p[:, :1])
    out = [idx.to(torch.int32), rho * p / total]
    if case["train"]:
        dw = st["dw"].double()
        dp = rho / total * dw
        if case["renorm"]:
            dp = dp - rho * (dw * p).sum(1, keepdim=True) / total ** 2
        if case["score"] == "softmax":
            # d p_j / d z_i = p_j ([i = j] - p_i)
            mean = (dp * p).sum(1, keepdim=True)
            dz = -s * mean
            dz.scatter_add_(1, idx, dp * p)
        else:
            dz = torch.zeros_like(s).scatter_(1, idx, dp * p * torch.sigmoid(-z).gather(1, idx))
        out.append(dz)
    return out


def _exact_norm(case, st):
    t, d = case["tokens"], case["width"]
    names = ["h", "y", "pre", "post", "alpha"] + (["gate_t"] if st["gate_t"] is not None else [])
    v = {n: st[n].double() for n in names}
    parts = []
    step = max(1, (1 << 26) // d)
    sums = {}
    for r in range(0, t, step):
        sl = slice(r, min(t, r + step))
        h, y = v["h"][sl], v["y"][sl]
        g = v.get("gate_t")
        if g is None:
            g = torch.ones((), dtype=torch.float64, device=h.device)
        elif case["gate"] != "channel":
            g = g[sl]
        iy = (y.square().mean(1, keepdim=True) + 1e-5).rsqrt()
        out = v["alpha"] * h + g * v["post"] * y * iy
        ih = (out.square().mean(1, keepdim=True) + 1e-5).rsqrt()
        o = {"h": out, "x": v["pre"] * out * ih}
        if case["train"]:
            dx, dho = st["dx"][sl].double(), st["dh_out"][sl].double()
            c = (v["pre"] * dx * out).sum(1, keepdim=True)
            dout = dho + v["pre"] * dx * ih - out * ih ** 3 * c / d
            dn = dout * g
            c2 = (v["post"] * dn * y).sum(1, keepdim=True)
            o["dh"] = v["alpha"] * dout
            o["dy"] = v["post"] * dn * iy - y * iy ** 3 * c2 / d
            cols = {"dpre": dx * out * ih, "dpost": dn * y * iy, "dalpha": dout * h}
            if case["gate"] != "none":
                dg = dout * v["post"] * y * iy
                if case["gate"] == "channel":
                    cols["dgate"] = dg
                else:
                    o["dgate"] = dg if case["gate"] == "full" else dg.sum(1, keepdim=True)
            for n, c in cols.items():
                sums[n] = sums.get(n, 0) + c.sum(0)
        parts.append(o)
    res = {n: torch.cat([p[n] for p in parts]) for n in ("h", "x")}
    if case["train"]:
        for n in ("dh", "dy"):
            res[n] = torch.cat([p[n] for p in parts])
        for n in ("dpre", "dpost", "dalpha"):
            res[n] = sums[n]
        if case["gate"] == "channel":
            res["dgate"] = sums["dgate"]
        elif case["gate"] != "none":
            res["dgate"] = torch.cat([p["dgate"] for p in parts])
    return res


def _exact_product(xc, xs, wc, ws):
    x = xc.to(torch.float32).double() * xs.double().repeat_interleave(BLOCK, 1)
    w = wc.to(torch.float32).double()
    w *= ws.double().repeat_interleave(BLOCK, 0)[:w.shape[0]].repeat_interleave(BLOCK, 1)
    return x @ w.t()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op == "norm":
        return _exact_norm(case, st)
    if op == "quantize":
        # the codes are defined by fp32 steps; only the scales have a 64-bit value
        x = st["x"].double().abs()
        pad = -x.shape[1] % BLOCK
        x = torch.nn.functional.pad(x, (0, pad)).unflatten(1, (-1, BLOCK))
        return {"values": None, "scales": (x.amax(2) / E4M3_MAX).clamp_min(MIN_SCALE)}
    if op == "matmul":
        return _exact_product(st["xc"], st["xs"], st["wc"], st["ws"])
    y = torch.empty(case["tokens"] * case["top_k"], case["n"], dtype=torch.float64,
                    device=st["xc"].device)
    for i in range(case["experts"]):
        a, b = st["bounds"][i], st["bounds"][i + 1]
        if b > a:
            at = slice(a, b) if st["index"] is None else st["index"][a:b].long()
            xc = st["xc"].view(torch.uint8)[at].view(torch.float8_e4m3fn)
            y[a:b] = _exact_product(xc, st["xs"][at], st["wc"][i], st["ws"][i])
    return y
