"""Operators in 4-bit floating point and the sparse layer of a few tokens, as
measured cases.

Three operators, each reached through the package's public functions:

* ``quantize``  values -> microscaled 4-bit floating point (E2M1 elements, a
                power-of-two scale for each 32 values of a row), and back;
* ``matmul``    the product of two such matrices: dense, grouped by expert,
                with gathered rows;
* ``tokens``    a whole sparse layer for a few tokens: router, top-K, the
                selected experts' two projections with the activation between
                them, the weighted sum, and a shared expert; weights in bf16,
                in 8-bit floating point or in 4-bit.

``run`` computes a case in its plain form (elementary torch operations) or,
with ``own`` set, by the package's kernels; ``exact`` computes it in 64 bits.
"""

import math

import torch

own = False

MX = 32          # values that share a scale in 4-bit floating point
BLOCK = 128      # rows and columns that share one in 8-bit
E4M3_MAX = 448.0

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "bf16": 2}


# ---- cases -------------------------------------------------------------------


def _quant(name, rows, cols, dtype="bf16"):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "dtype": dtype}


def _mm(name, rows, n, k, out="bf16"):
    return {"name": name, "op": "matmul", "rows": rows, "n": n, "k": k, "out": out, "experts": 0,
            "top_k": 1, "gather": False}


def _grouped(name, tokens, top_k, experts, n, k, gather, out="bf16"):
    return {"name": name, "op": "matmul", "rows": tokens, "n": n, "k": k, "out": out,
            "experts": experts, "top_k": top_k, "gather": gather}


def _tokens(name, tokens, experts, top_k, width, hidden, fmt="bf16", act="relu2", shared=0,
            score="sigmoid", bias=True, renorm=True, scale=5.0, dtype="bf16", out="bf16"):
    return {"name": name, "op": "tokens", "tokens": tokens, "experts": experts, "top_k": top_k,
            "width": width, "hidden": hidden, "fmt": fmt, "act": act, "shared": shared,
            "score": score, "bias": bias, "renorm": renorm, "scale": scale, "dtype": dtype,
            "out": out}


def listed():
    return [
        # a prompt's activations, kept in 4 bits and read back
        _quant("quantize_prompt", 8192, 8192),
        # the latent of one decode step of 32 sequences
        _quant("quantize_decode", 32, 2048, "f32"),
        # one token through the shared expert's up projection
        _mm("matmul_token", 1, 10240, 8192),
        # a speculative-verify batch (187 tokens, ragged) through the latent projection
        _mm("matmul_verify", 187, 2048, 8192, "f32"),
        # a prompt through the shared expert's up projection
        _mm("matmul_prompt", 8192, 10240, 8192),
        # a decode batch through the experts' up projection (rows gathered from the latent)
        _grouped("experts_decode", 32, 22, 512, 5120, 2048, True),
        # a prompt through the experts' down projection
        _grouped("experts_prompt", 8192, 22, 512, 2048, 5120, False),
        # one token of a single sequence through the latent sparse layer, bf16 and 4-bit experts
        _tokens("tokens_one", 1, 512, 22, 2048, 5120, dtype="f32"),
        _tokens("tokens_one_mxfp4", 1, 512, 22, 2048, 5120, fmt="mxfp4", dtype="f32"),
        # a token and its five speculated successors, 8-bit experts
        _tokens("tokens_verify_fp8", 6, 512, 22, 2048, 5120, fmt="fp8", dtype="f32", out="f32"),
        # a small layer with gated experts, a softmax router and a shared expert: latency counts
        _tokens("tokens_small_gated", 1, 60, 6, 1024, 704, act="swiglu", shared=1408,
                score="softmax", bias=False, renorm=False, scale=1.0),
        # thirteen sequences through a layer with gated 4-bit experts
        _tokens("tokens_gated_mxfp4", 13, 128, 8, 2048, 768, fmt="mxfp4", act="swiglu",
                score="softmax", bias=False, scale=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "grouped", "tokens", "tokens"])
    if op == "quantize":
        return _quant("", _log_int(rng, 1, 8192), _log_int(rng, 32, 8192),
                      rng.choice(["bf16", "f32"]))
    if op == "matmul":
        return _mm("", _log_int(rng, 1, 8192), 16 * _log_int(rng, 16, 640),
                   BLOCK * _log_int(rng, 2, 64), rng.choice(["bf16", "f32"]))
    if op == "grouped":
        experts = _log_int(rng, 8, 256)
        return _grouped("", _log_int(rng, 1, 4096), rng.randint(1, min(8, experts)), experts,
                        16 * _log_int(rng, 16, 160), BLOCK * _log_int(rng, 2, 20),
                        rng.random() < 0.5, rng.choice(["bf16", "f32"]))
    experts = _log_int(rng, 8, 256)
    fmt = rng.choice(["bf16", "fp8", "mxfp4"])
    step = 64 if fmt == "bf16" else BLOCK
    return _tokens("", rng.randint(1, 16), experts, rng.randint(1, min(8, experts)),
                   step * _log_int(rng, 2, 2048 // step), step * _log_int(rng, 2, 2048 // step),
                   fmt=fmt, act=rng.choice(["relu2", "swiglu"]),
                   shared=rng.choice([0, step * _log_int(rng, 2, 2048 // step)]),
                   score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.5,
                   renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5, 5.0]),
                   dtype=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))


# ---- 4-bit and 8-bit values ----------------------------------------------------


def _tables(dev):
    """What the plain forms look up: the 16 codes' values, and 2^(i - 127)."""
    mag = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    val = torch.tensor(mag + [-m for m in mag], device=dev)
    power = torch.tensor([math.ldexp(1.0, i - 127) for i in range(255)], device=dev)
    return val, power


def _plain_mx_quantize(x, power):
    """(codes [.., ceil(K / 32) * 16], scales [.., ceil(K / 32)]) of x [.., K]:
    scale 2^(floor(log2 max) - 2) a block of 32, elements to the nearest of 0,
    0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), larger ones to 6."""
    k = x.shape[-1]
    nb = -(-k // MX)
    v = x.to(torch.float32)
    if nb * MX != k:
        v = torch.cat([v, v.new_zeros(*v.shape[:-1], nb * MX - k)], -1)
    v = v.reshape(*v.shape[:-1], nb, MX)
    top = v.abs().amax(-1)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 127)
    e = torch.where(top > 0, e, torch.full_like(e, -127))
    a = v.abs() * power[127 - e.long()][..., None]
    c = (a > 0.25).to(torch.uint8)
    for t, strict in ((0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False),
                      (5.0, True)):
        c += (a > t) if strict else (a >= t)
    c += 8 * ((v < 0) & (c > 0)).to(torch.uint8)
    c = c.reshape(*x.shape[:-1], nb * MX // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), (e + 127).to(torch.uint8)


def _plain_mx_values(codes, scales, tables):
    """The fp32 values of codes [.., K / 2] and scales [.., K / 32]."""
    val, power = tables
    v = torch.stack([val[(codes & 15).long()], val[(codes >> 4).long()]], -1)
    v = v.reshape(*scales.shape, MX) * power[scales.long()][..., None]
    return v.reshape(*scales.shape[:-1], scales.shape[-1] * MX)


def _plain_fp8_values(codes, scales):
    """The fp32 values of codes [.., N, K] with a scale for each 128 x 128 block."""
    n, k = codes.shape[-2:]
    s = scales.repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]
    return codes.to(torch.float32) * s


def _fp8_quantize(w):
    n, k = w.shape
    nb = -(-n // BLOCK)
    v = w
    if nb * BLOCK != n:
        v = torch.cat([v, v.new_zeros(nb * BLOCK - n, k)], 0)
    v = v.view(nb, BLOCK, k // BLOCK, BLOCK)
    s = (v.abs().amax((1, 3)) / E4M3_MAX).clamp_min(2.0 ** -126)
    q = (v / s[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(nb * BLOCK, k)[:n], s


# ---- inputs ------------------------------------------------------------------


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev) * std

    st = dict(case)
    st["tables"] = _tables(dev)
    power = st["tables"][1]
    op = case["op"]
    if op == "quantize":
        v = randn(case["rows"], case["cols"])
        # rows of different size, as activations are
        v *= torch.exp(randn(case["rows"], 1))
        st["x"] = v.to(_DTYPES[case["dtype"]])
        return st

    def weights(fmt, *shape):
        """Codes and scales (scales None in bf16) of weights [N, K] or [E, N, K]."""
        lead, (n, k) = shape[:-2], shape[-2:]
        c = torch.empty(*lead, n, k // 2 if fmt == "mxfp4" else k, device=dev,
                        dtype={"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn,
                               "mxfp4": torch.uint8}[fmt])
        s = None
        if fmt == "fp8":
            s = torch.empty(*lead, -(-n // BLOCK), k // BLOCK, device=dev)
        elif fmt == "mxfp4":
            s = torch.empty(*lead, n, k // MX, dtype=torch.uint8, device=dev)
        for i in range(lead[0] if lead else 1):
            w = randn(n, k, std=0.02)
            at = i if lead else slice(None)
            if fmt == "bf16":
                c[at] = w
            elif fmt == "fp8":
                c[at], s[at] = _fp8_quantize(w)
            else:
                c[at], s[at] = _plain_mx_quantize(w, power)
        return c, s

    if op == "matmul":
        t, k_, e, n, k = (case[i] for i in ("rows", "top_k", "experts", "n", "k"))
        rows = t * k_
        st["offsets"] = st["index"] = None
        if e:
            pick = torch.rand((t, e), generator=g, device=dev).topk(k_, 1).indices.sort(1).values
            order = torch.sort(pick.reshape(-1), stable=True).indices
            ends = torch.cumsum(torch.bincount(pick.reshape(-1), minlength=e), 0)
            st["offsets"] = torch.cat([ends.new_zeros(1), ends]).to(torch.int32)
            st["bounds"] = st["offsets"].tolist()
            # gathered: sorted row i reads token order[i] // top_k; else rows are in expert order
            st["index"] = (order // k_).to(torch.int32) if case["gather"] else None
        xrows = t if case["gather"] else rows
        st["xc"] = torch.empty(xrows, k // 2, dtype=torch.uint8, device=dev)
        st["xs"] = torch.empty(xrows, k // MX, dtype=torch.uint8, device=dev)
        for r in range(0, xrows, 16384):
            x = randn(min(16384, xrows - r), k)
            # hidden rows hold squares of rectified values; the others are signed
            x = torch.relu(x) ** 2 if e and not case["gather"] else x
            st["xc"][r:r + 16384], st["xs"][r:r + 16384] = _plain_mx_quantize(x, power)
        st["wc"], st["ws"] = weights("mxfp4", *((e, n, k) if e else (n, k)))
        return st

    t, e, d, f, s = (case[i] for i in ("tokens", "experts", "width", "hidden", "shared"))
    two = 2 if case["act"] == "swiglu" else 1
    st["x"] = randn(t, d).to(_DTYPES[case["dtype"]])
    st["gate"] = randn(e, d, std=1.0 / math.sqrt(d))
    st["beta"] = randn(e, std=0.1) if case["bias"] else None
    fmt = case["fmt"]
    st["up"], st["up_s"] = weights(fmt, e, two * f, d)
    st["down"], st["down_s"] = weights(fmt, e, d, f)
    if s:
        st["shared_up"], st["shared_up_s"] = weights(fmt, two * s, d)
        st["shared_down"], st["shared_down_s"] = weights(fmt, d, s)
    else:
        st["shared_up"] = st["shared_up_s"] = st["shared_down"] = st["shared_down_s"] = None
    if own:
        import sparse_moe_layer_latentmoe_amd as lmoe
        st["router"] = lmoe.make_router(
            e, case["top_k"], score=(lmoe.SCORE_SOFTMAX if case["score"] == "softmax"
                                     else lmoe.SCORE_SIGMOID),
            renormalise=case["renorm"], scale=case["scale"])
    return st


# ---- plain forms -------------------------------------------------------------


def _plain_matmul(st):
    tb, dt = st["tables"], _DTYPES[st["out"]]
    if not st["experts"]:
        x = _plain_mx_values(st["xc"], st["xs"], tb)
        return torch.matmul(x, _plain_mx_values(st["wc"], st["ws"], tb).t()).to(dt)
    y = torch.empty(st["rows"] * st["top_k"], st["n"], dtype=dt, device=st["xc"].device)
    b = st["bounds"]
    for i in range(st["experts"]):
        if b[i] == b[i + 1]:
            continue
        at = slice(b[i], b[i + 1])
        if st["index"] is not None:
            at = st["index"][at].long()
        x = _plain_mx_values(st["xc"][at], st["xs"][at], tb)
        w = _plain_mx_values(st["wc"][i], st["ws"][i], tb)
        y[b[i]:b[i + 1]] = torch.matmul(x, w.t()).to(dt)
    return y


def _plain_expert_values(st, name, at=None):
    """fp32 values of the experts' matrices `at`, or of the shared expert's."""
    c, s = st[name], st[name + "_s"]
    if at is not None:
        c = c.view(torch.uint8)[at].view(torch.float8_e4m3fn) if st["fmt"] == "fp8" else c[at]
        s = None if s is None else s[at]
    if st["fmt"] == "bf16":
        return c.to(torch.float32)
    if st["fmt"] == "fp8":
        return _plain_fp8_values(c, s)
    return _plain_mx_values(c, s, st["tables"])


def _plain_act(u, act):
    if act == "relu2":
        return torch.clamp_min(u, 0.0) ** 2
    a, b = u.chunk(2, -1)
    return a / (1.0 + torch.exp(-a)) * b


def _plain_tokens(st):
    f = torch.float32
    x = st["x"].to(f)
    # the router in 64 bits: it compares values next to each other
    logits = torch.matmul(x.double(), st["gate"].double().t())
    if st["score"] == "softmax":
        ex = torch.exp(logits - logits.amax(1, keepdim=True))
        s = ex / ex.sum(1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-logits))
    key = logits if st["beta"] is None else s + st["beta"].double()
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :st["top_k"]]
    idx = torch.sort(idx, dim=1).values
    w = torch.gather(s, 1, idx)
    if st["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    w = (w * st["scale"]).to(f)
    y = torch.empty_like(x)
    for t in range(st["tokens"]):
        u = torch.matmul(_plain_expert_values(st, "up", idx[t]), x[t])
        h = _plain_act(u, st["act"])
        o = torch.matmul(_plain_expert_values(st, "down", idx[t]), h[:, :, None])[:, :, 0]
        y[t] = (o * w[t][:, None]).sum(0)
    if st["shared_up"] is not None:
        h = _plain_act(torch.matmul(x, _plain_expert_values(st, "shared_up").t()), st["act"])
        y = y + torch.matmul(h, _plain_expert_values(st, "shared_down").t())
    return {"y": y.to(_DTYPES[st["out"]]), "experts": idx.to(torch.int32), "weights": w}


def _run_plain(st):
    if st["op"] == "quantize":
        c, s = _plain_mx_quantize(st["x"], st["tables"][1])
        return _plain_mx_values(c, s, st["tables"])[:, :st["cols"]].to(torch.bfloat16)
    return _plain_matmul(st) if st["op"] == "matmul" else _plain_tokens(st)


# ---- the package's kernels -----------------------------------------------------


def _run_own(st):
    import sparse_moe_layer_latentmoe_amd as lmoe
    if st["op"] == "quantize":
        codes, scales = lmoe.quantize_mxfp4_rows(st["x"])
        return lmoe.dequantize_mxfp4(codes, scales, cols=st["cols"])
    out = _DTYPES[st["out"]]
    if st["op"] == "matmul":
        return lmoe.mxfp4_matmul(st["xc"], st["xs"], st["wc"], st["ws"], offsets=st["offsets"],
                                 rows=st["index"], out_dtype=out)
    y, idx, w = lmoe.moe_tokens(
        st["router"], st["x"], st["gate"], st["up"], st["down"], bias=st["beta"],
        up_scales=st["up_s"], down_scales=st["down_s"], shared_up=st["shared_up"],
        shared_down=st["shared_down"], shared_up_scales=st["shared_up_s"],
        shared_down_scales=st["shared_down_s"],
        activation=lmoe.ACT_SWIGLU if st["act"] == "swiglu" else lmoe.ACT_RELU2, out_dtype=out)
    return {"y": y, "experts": idx, "weights": w}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without --------------------------------------------


def _used(tokens, top_k, experts):
    """Experts that tokens with top_k experts at random pick at least once."""
    return experts * (1.0 - (1.0 - top_k / experts) ** tokens)


def work(case):
    op = case["op"]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        nb = -(-c // MX)
        # read, write codes and scales, read them, write bf16
        return {"bytes": r * c * _BYTES[case["dtype"]] + 2 * r * nb * 17 + 2 * r * c,
                "flops": 4 * r * c}
    if op == "matmul":
        n, k, e = case["n"], case["k"], case["experts"]
        rows = case["rows"] * case["top_k"]
        xrows = case["rows"] if case["gather"] else rows
        used = _used(case["rows"], case["top_k"], e) if e else 1.0
        b = (xrows + used * n) * (k // 2 + k // MX) + rows * n * _BYTES[case["out"]]
        return {"bytes": int(b), "flops": 2 * rows * n * k}
    t, e, k, d, f, s = (case[i] for i in ("tokens", "experts", "top_k", "width", "hidden",
                                          "shared"))
    per = {"bf16": 2.0, "fp8": 1.0 + 4.0 / BLOCK ** 2, "mxfp4": 0.5 + 1.0 / MX}[case["fmt"]]
    m = 3 if case["act"] == "swiglu" else 2
    b = 4 * e * d + m * d * per * (_used(t, k, e) * f + s)
    b += t * d * (_BYTES[case["dtype"]] + _BYTES[case["out"]]) + 8 * t * k
    return {"bytes": int(b), "flops": 2 * t * d * (e + m * (k * f + s))}


# ---- definitions in 64 bits ----------------------------------------------------


_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_power(e):
    """2^e in 64 bits, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_mx(codes, scales):
    """64-bit values, from the bits of a code: sign, two exponent bits, one of
    the mantissa."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int64)
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e > 0, (1.0 + 0.5 * m) * _exact_power(e - 1), 0.5 * m)
    v = torch.where(c >= 8, -v, v)
    return v * _exact_power(scales.long() - 127).repeat_interleave(MX, -1)


def _exact_quantize(st):
    x = st["x"].double()
    pad = -x.shape[1] % MX
    b = torch.nn.functional.pad(x, (0, pad)).unflatten(1, (-1, MX))
    _, ex = torch.frexp(b.abs().amax(2, keepdim=True))
    step = _exact_power((ex - 3).clamp(-127, 127))
    a = b.abs() / step
    # neighbours are 0.5, 1 or 2 apart; half way goes to the even one
    q = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    r = (torch.round(a / q) * q).clamp_max(_GRID[-1])
    return (torch.sign(b) * r * step).flatten(1)[:, :st["cols"]]


def _exact_matrix(st, name, i=None):
    c, s = st[name], st[name + "_s"]
    if i is not None:
        c, s = c[i], None if s is None else s[i]
    if st["fmt"] == "bf16":
        return c.double()
    if st["fmt"] == "mxfp4":
        return _exact_mx(c, s)
    n, k = c.shape
    w = c.to(torch.float32).double()
    for r in range(0, n, BLOCK):
        w[r:r + BLOCK] *= s[r // BLOCK].double().repeat_interleave(BLOCK)[:k]
    return w


def _exact_tokens(case, st):
    x = st["x"].double()
    z = x @ st["gate"].double().t()
    s = torch.softmax(z, 1) if case["score"] == "softmax" else torch.sigmoid(z)
    o = z if st["beta"] is None else s + st["beta"].double()
    e, k = case["experts"], case["top_k"]
    lower = torch.ones(e, e, device=z.device).tril(-1).bool()
    before = (o[:, None, :] > o[:, :, None]) | ((o[:, None, :] == o[:, :, None]) & lower)
    chosen = before.sum(2) < k
    idx = chosen.nonzero()[:, 1].reshape(-1, k)
    p = s[chosen].reshape(-1, k)
    w = case["scale"] * (p / (p.sum(1, keepdim=True) + 1e-20) if case["renorm"] else p)

    def expert(i, rows, sh=""):
        u = rows @ _exact_matrix(st, sh + "up", i).t()
        if case["act"] == "relu2":
            h = torch.relu(u).square()
        else:
            n = u.shape[1] // 2
            h = torch.nn.functional.silu(u[:, :n]) * u[:, n:]
        return h @ _exact_matrix(st, sh + "down", i).t()

    y = expert(None, x, "shared_") if st["shared_up"] is not None else torch.zeros_like(x)
    for i in torch.unique(idx).tolist():
        t, j = (idx == i).nonzero(as_tuple=True)
        y[t] += w[t, j][:, None] * expert(i, x[t])
    return {"y": y, "experts": idx.to(torch.int32), "weights": w}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_quantize(st)
    if case["op"] == "tokens":
        return _exact_tokens(case, st)
    if not case["experts"]:
        return _exact_mx(st["xc"], st["xs"]) @ _exact_mx(st["wc"], st["ws"]).t()
    y = torch.empty(case["rows"] * case["top_k"], case["n"], dtype=torch.float64,
                    device=st["xc"].device)
    for i in range(case["experts"]):
        a, b = st["bounds"][i], st["bounds"][i + 1]
        if b > a:
            at = slice(a, b) if st["index"] is None else st["index"][a:b].long()
            y[a:b] = _exact_mx(st["xc"][at], st["xs"][at]) @ _exact_mx(st["wc"][i],
                                                                      st["ws"][i]).t()
    return y
