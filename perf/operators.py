"""The operators around the routed experts of a mixture-of-experts block, as cases that can be timed and checked.

Three operators: `block_norm` (norms after and before a block with gate and residual scale), `dense_linear`
(matrix product with bias, activation, gating and residual in its epilogue) and `moe_route_grouped_topk` (grouped
expert routing).  With `own` false, run() computes them from elementary torch operations in 32 bits; with `own`
true it calls the library.  exact() computes them once more in 64 bits from their definitions.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# --- cases ---------------------------------------------------------------------------------------------------

def _norm(T, H, dtype="bf16", rdtype="bf16", post="rms", pre="rms", gate="none", branch=1.0, resid=1.0, bias=False):
    return dict(op="norm", T=T, H=H, dtype=dtype, rdtype=rdtype, post=post, pre=pre, gate=gate, branch=branch,
                resid=resid, bias=bias)


def _linear(M, N, K, dtype="bf16", out="bf16", act="none", gated=False, bias=False, residual=False):
    return dict(op="linear", M=M, N=N, K=K, dtype=dtype, out=out, act=act, gated=gated, bias=bias, residual=residual)


def _route(T, E, k, score="sigmoid", dtype="f32", bias=True, groups=1, keep=1, top=1, renorm=True, scale=1.0,
           masked=False):
    return dict(op="route", T=T, E=E, k=k, score=score, dtype=dtype, bias=bias, groups=groups, keep=keep, top=top,
                renorm=renorm, scale=scale, masked=masked)


def listed():
    return [
        # a decode step of 64 tokens: norm of the attention output into the residual stream, next norm
        dict(_norm(64, 7168), name="norm decode 64"),
        # a prefill step, with a learned gate per channel (layer scale)
        dict(_norm(8192, 7168, gate="channel", branch=0.5), name="norm prefill 8192"),
        # LayerNorm with biases over a 32-bit residual stream, a gate per token, sizes that divide nothing
        dict(_norm(3001, 5119, dtype="f16", rdtype="f32", post="layer", pre="layer", gate="token", resid=0.7,
                   bias=True), name="norm odd 3001x5119"),
        # the router gate for a single token, 32-bit logits
        dict(_linear(1, 256, 7168, out="f32"), name="gate 1"),
        # the router gate of a prefill step
        dict(_linear(8192, 256, 7168, out="f32"), name="gate prefill 8192"),
        # the shared expert's gate and up products of a decode step, SiLU(gate) * up
        dict(_linear(64, 4096, 7168, act="silu", gated=True), name="shared up decode 64"),
        # the same in prefill
        dict(_linear(8192, 4096, 7168, act="silu", gated=True), name="shared up prefill 8192"),
        # the shared expert's down product, added to the routed experts' output
        dict(_linear(8192, 7168, 2048, residual=True), name="shared down prefill 8192"),
        # an ordinary layer with bias, GELU and residual at sizes without any alignment
        dict(_linear(777, 1001, 1537, dtype="f16", out="f16", act="gelu", bias=True, residual=True),
             name="linear odd 777x1001x1537"),
        # grouped sigmoid routing with a balance bias, a decode step
        dict(_route(64, 256, 8, groups=8, keep=4, top=2, scale=2.5), name="route decode 64"),
        # the same in prefill
        dict(_route(8192, 256, 8, groups=8, keep=4, top=2, scale=2.5), name="route prefill 8192"),
        # grouped softmax routing of a large batch with experts taken out by -inf and tokens without any
        dict(_route(65531, 160, 6, score="softmax", bias=False, groups=8, keep=3, top=1, renorm=False, scale=16.0,
                    masked=True), name="route softmax 65531x160"),
    ]


def _log_int(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_norm(rng):
    while True:
        T, H = _log_int(rng, 1, 16384), _log_int(rng, 64, 16384)
        if rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        if T * H <= 5000 * 7168:
            break
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    kinds = rng.choice([("rms", "rms"), ("none", "rms"), ("rms", "none"), ("layer", "layer"), ("none", "layer")])
    return _norm(T, H, dtype=dtype, rdtype=rng.choice([dtype, "f32"]), post=kinds[0], pre=kinds[1],
                 gate=rng.choice(["none", "channel", "token", "full"]), branch=rng.choice([1.0, 0.5, 0.22]),
                 resid=rng.choice([1.0, 1.4, 0.7]), bias=rng.random() < 0.4)


def _draw_linear(rng):
    while True:
        M, N, K = _log_int(rng, 1, 8192), _log_int(rng, 16, 8192), _log_int(rng, 64, 8192)
        if M * N * K <= 8192 * 4096 * 4096 and N * K >= 65536:
            break
    if rng.random() < 0.7:  # most models' widths are round; the number of tokens is not
        N, K = max(64, N // 64 * 64), max(64, K // 64 * 64)
    gated = rng.random() < 0.3
    dtype = rng.choice(["bf16", "bf16", "f16"])
    return _linear(M, N // 2 * 2 if gated else N, K, dtype=dtype, out=rng.choice([dtype, dtype, "f32"]),
                   act=rng.choice(["silu", "gelu_tanh"]) if gated else rng.choice(["none", "none", "relu", "silu",
                                                                                  "gelu", "gelu_tanh"]),
                   gated=gated, bias=rng.random() < 0.5, residual=rng.random() < 0.5)


def _draw_route(rng):
    T = _log_int(rng, 1, 65536)
    groups = rng.choice([1, 1, 2, 4, 8, 16, 5])
    per = _log_int(rng, 4, min(64, 512 // groups)) if groups > 1 else _log_int(rng, 8, 512)
    keep = rng.randint(1, groups)
    k = rng.randint(1, min(8, keep * per))
    score = rng.choice(["sigmoid", "softmax"])
    bias = score == "sigmoid" and rng.random() < 0.7  # a softmax with a bias ranks by sums whose last bit depends on order
    top = rng.choice([1, 2]) if score == "sigmoid" else 1
    return _route(T, groups * per, k, score=score, dtype=rng.choice(["f32", "f32", "bf16"]), bias=bias, groups=groups,
                  keep=keep, top=top, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5, 16.0]),
                  masked=rng.random() < 0.3)


def draw(rng):
    return rng.choice([_draw_norm, _draw_linear, _draw_route])(rng)


def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        g = {"none": 0, "channel": H, "token": T, "full": T * H}[case["gate"]]
        w = H * ((case["post"] != "none") + (case["pre"] != "none")) * (2 if case["bias"] else 1)
        return {"bytes": T * H * 2 * (_SIZE[case["dtype"]] + _SIZE[case["rdtype"]]) + g * _SIZE[case["dtype"]] + 4 * w,
                "flops": 12 * T * H}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        n_out = N // 2 if case["gated"] else N
        s = _SIZE[case["out"]]
        return {"bytes": (M + N) * K * 2 + M * n_out * s * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    return {"bytes": T * E * _SIZE[case["dtype"]] + T * k * 8 + (4 * E if case["bias"] else 0), "flops": 6 * T * E}


# --- inputs --------------------------------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    st = {"case": case}
    if case["op"] == "norm":
        T, H, dt = case["T"], case["H"], _DT[case["dtype"]]
        spread = 1.0 + 4.0 * torch.rand(H, generator=g, device=dev) ** 8  # a few channels are much larger than the rest
        st["f"] = (randn(T, H) * spread + 0.1).to(dt)
        st["r"] = (3.0 * randn(T, H)).to(_DT[case["rdtype"]])
        for name in ("post", "pre"):
            st["w_" + name] = 1.0 + 0.2 * randn(H) if case[name] != "none" else None
            st["b_" + name] = 0.1 * randn(H) if case["bias"] and case[name] == "layer" else None
        shape = {"none": None, "channel": (1, H), "token": (T, 1), "full": (T, H)}[case["gate"]]
        st["gate"] = None if shape is None else (0.5 + 0.3 * randn(*shape)).to(dt)
    elif case["op"] == "linear":
        M, N, K, dt = case["M"], case["N"], case["K"], _DT[case["dtype"]]
        n_out = N // 2 if case["gated"] else N
        st["x"] = randn(M, K).to(dt)
        st["w"] = (randn(N, K) * (1.5 / math.sqrt(K))).to(dt)
        st["bias"] = 0.3 * randn(N) if case["bias"] else None
        st["residual"] = randn(M, n_out).to(_DT[case["out"]]) if case["residual"] else None
    else:
        T, E = case["T"], case["E"]
        logits = randn(T, E) + 0.5 * randn(E)
        if case["masked"]:  # one expert in eight is away, and one token in sixteen is padding
            logits.masked_fill_(torch.rand(E, generator=g, device=dev) < 0.125, -math.inf)
            logits.masked_fill_(torch.rand(T, 1, generator=g, device=dev) < 0.0625, -math.inf)
        st["logits"] = logits.to(_DT[case["dtype"]])
        st["bias"] = 0.05 * randn(E) if case["bias"] else None
    return st


# --- one pass ------------------------------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "route": _own_route}[op](st)
    return {"norm": _plain_norm, "linear": _plain_linear, "route": _plain_route}[op](st)


def _own_norm(st):
    import w4afp8_mixture_experts_gb300 as lib
    c = st["case"]
    return lib.block_norm(st["f"], st["r"], post=c["post"], w_post=st["w_post"], b_post=st["b_post"], gate=st["gate"],
                          branch_scale=c["branch"], residual_scale=c["resid"], pre=c["pre"], w_pre=st["w_pre"],
                          b_pre=st["b_pre"], eps=1e-6)


def _own_linear(st):
    import w4afp8_mixture_experts_gb300 as lib
    c = st["case"]
    return lib.dense_linear(st["x"], st["w"], bias=st["bias"], act=c["act"], gated=c["gated"], residual=st["residual"],
                            out_dtype=_DT[c["out"]])


def _own_route(st):
    import w4afp8_mixture_experts_gb300 as lib
    c = st["case"]
    return lib.moe_route_grouped_topk(st["logits"], c["k"], bias=st["bias"], score=c["score"], n_group=c["groups"],
                                      topk_group=c["keep"], group_top=c["top"], renormalize=c["renorm"],
                                      scale=c["scale"])


def _plain_norm_of(v, kind, w, b):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6)
    v = v * w
    return v if b is None else v + b


def _plain_norm(st):
    c = st["case"]
    u = _plain_norm_of(st["f"].float(), c["post"], st["w_post"], st["b_post"])
    if st["gate"] is not None:
        u = u * st["gate"].float()
    h = c["resid"] * st["r"].float() + c["branch"] * u
    y = _plain_norm_of(h, c["pre"], st["w_pre"], st["b_pre"])
    return h.to(st["r"].dtype), y.to(st["f"].dtype)


def _plain_act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_linear(st):
    c = st["case"]
    z = st["x"].float() @ st["w"].float().t()
    if st["bias"] is not None:
        z = z + st["bias"]
    if c["gated"]:
        half = c["N"] // 2
        v = _plain_act(z[:, :half], c["act"]) * z[:, half:]
    else:
        v = _plain_act(z, c["act"])
    if st["residual"] is not None:
        v = v + st["residual"].float()
    return v.to(_DT[c["out"]])


def _plain_route(st):
    c = st["case"]
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    logits = st["logits"].float()
    here = logits > -math.inf
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-logits))
        choice = s
    else:
        top = logits.amax(1, keepdim=True)
        e = torch.exp(logits - torch.where(top > -math.inf, top, torch.zeros_like(top)))
        total = e.sum(1, keepdim=True)
        s = torch.where(total > 0, e / total, torch.zeros_like(e))
        choice = logits  # the softmax keeps the logits' order
    if st["bias"] is not None:
        choice = choice + st["bias"]
    choice = torch.where(here, choice, torch.full_like(choice, -math.inf))
    if G > 1:
        per = choice.view(T, G, E // G)
        group = per.topk(c["top"], dim=2).values.sum(2)
        order = group.sort(dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=logits.device).scatter_(1, order, True)
        choice = torch.where(kept[:, :, None], per, torch.full_like(per, -math.inf)).view(T, E)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    # an expert that is away, or whose group was left out, only fills a place: it weighs nothing
    w = torch.where(choice.gather(1, ids) > -math.inf, s.gather(1, ids), torch.zeros_like(choice[:, :k]))
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return ids.to(torch.int32), w * c["scale"]


# --- the definitions in 64 bits --------------------------------------------------------------------------------

def _exact_norm(st):
    c = st["case"]

    def normed(v, kind, w, b):
        if kind == "none":
            return v
        mu = torch.sum(v, 1) / v.shape[1] if kind == "layer" else torch.zeros_like(v[:, 0])
        d = v - mu[:, None]
        q = torch.sum(d * d, 1) / v.shape[1] + 1e-6
        out = d / torch.sqrt(q)[:, None] * w.double()[None, :]
        return out if b is None else out + b.double()[None, :]

    u = normed(st["f"].double(), c["post"], st["w_post"], st["b_post"])
    g = torch.ones(1, 1, dtype=torch.float64, device=u.device) if st["gate"] is None else st["gate"].double()
    h = st["r"].double() * c["resid"] + g * u * c["branch"]
    return h, normed(h, c["pre"], st["w_pre"], st["b_pre"])


def _exact_linear(st):
    c = st["case"]
    z = torch.einsum("mk,nk->mn", st["x"].double(), st["w"].double())
    if c["bias"]:
        z += st["bias"].double()
    g, u = (z[:, : c["N"] // 2], z[:, c["N"] // 2:]) if c["gated"] else (z, None)
    if c["act"] == "relu":
        g = torch.maximum(g, torch.zeros_like(g))
    elif c["act"] == "silu":
        g = g * torch.special.expit(g)
    elif c["act"] == "gelu":
        g = g * torch.special.ndtr(g)
    elif c["act"] == "gelu_tanh":
        g = g * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))
    v = g if u is None else g * u
    return v + st["residual"].double() if c["residual"] else v


def _exact_route(st):
    c = st["case"]
    l = st["logits"].double()
    away = torch.isneginf(l)
    if c["score"] == "sigmoid":
        s = torch.special.expit(l)
        choice = s + st["bias"].double() if c["bias"] else s.clone()
    else:
        s = torch.nan_to_num(torch.softmax(l, 1), nan=0.0)
        choice = l.clone()
    choice[away] = -math.inf
    per = c["E"] // c["groups"]
    best = torch.sort(choice.view(-1, c["groups"], per), dim=2, descending=True).values[:, :, : c["top"]].sum(2)
    rank = torch.argsort(torch.argsort(best, dim=1, descending=True, stable=True), dim=1)
    choice[(rank >= c["keep"]).repeat_interleave(per, dim=1)] = -math.inf
    value, ids = torch.sort(choice, dim=1, descending=True, stable=True)
    w = s.gather(1, ids[:, : c["k"]])
    w[torch.isneginf(value[:, : c["k"]])] = 0.0
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return None, w * c["scale"]


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "route": _exact_route}[case["op"]](st)
