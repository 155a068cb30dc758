"""The attention half of a block around the routed experts, as cases that can be timed and checked.

Four operators: `rotary_embedding` (rotation of heads by position), `paged_kv_append` (new keys and values into a paged
cache, rotated on the way), `paged_attention_decode` (attention of one new token per sequence over such a cache) and
`fp8_block_linear` (E4M3 matrix product with a scale per token and 128 columns, and per 128 x 128 weights: the
projections).  With `own` false, run() computes them from elementary torch operations in 32 bits (angles in 64); with
`own` true it calls the library.  exact() computes them once more in 64 bits from their definitions.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4, "fp8": 1}


# --- cases ---------------------------------------------------------------------------------------------------

def _rotary(T, H, D, R, dtype="bf16", pairs="half", start=0, far=4096, factor=1.0, inverse=False):
    return dict(op="rotary", T=T, H=H, D=D, R=R, dtype=dtype, pairs=pairs, start=start, far=far, factor=factor,
                inverse=inverse)


def _append(B, new, past, Hkv, D, R, page, dtype="bf16", Hq=0, pairs="half", start=0, factor=1.0, padding=0):
    """B sequences with up to `new` new and up to `past` earlier tokens each; new = 0: exactly one new token each."""
    return dict(op="append", B=B, new=new, past=past, Hkv=Hkv, D=D, R=R, page=page, dtype=dtype, Hq=Hq, pairs=pairs,
                start=start, factor=factor, padding=padding)


def _attend(B, longest, Hq, Hkv, D, page, dtype="bf16", cache="bf16", ragged=True, window=0, empty=0):
    return dict(op="attend", B=B, longest=longest, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype, cache=cache,
                ragged=ragged, window=window, empty=empty)


def _linear(M, N, K, out="bf16"):
    return dict(op="linear", M=M, N=N, K=K, out=out)


def listed():
    return [
        # queries and keys of a prefill step, 64 + 8 heads in one tensor, positions of a context that was extended 40 times
        dict(_rotary(8192, 72, 128, 128, far=163840, factor=40.0), name="rotary prefill 8192"),
        # the rotation's gradient (its transpose) for 64 dimensions behind 128 others, neighbouring pairs, 32 bits
        dict(_rotary(1999, 17, 192, 64, dtype="f32", pairs="neighbours", start=128, inverse=True),
             name="rotary gradient odd 1999"),
        # a decode step of 64 sequences: one new token each, its queries rotated in the same call
        dict(_append(64, 0, 1024, 8, 128, 128, 16, Hq=64, factor=40.0), name="append decode 64"),
        # a prefill step of four prompts of up to 4096 tokens into pages of 64
        dict(_append(4, 4096, 0, 8, 128, 128, 64, Hq=64, factor=40.0), name="append prefill 4 x 4096"),
        # prompts behind earlier tokens, pages that end inside everything, half of each head rotated, padded rows
        dict(_append(19, 211, 700, 5, 96, 48, 7, dtype="f16", pairs="neighbours", start=48, padding=133),
             name="append odd 19 x 211"),
        # a single short sequence: latency
        dict(_attend(1, 333, 32, 8, 128, 16, ragged=False), name="attend 1 x 333"),
        # a decode step of 64 sequences of up to 8192 tokens
        dict(_attend(64, 8192, 64, 8, 128, 64), name="attend 64 x 8192"),
        # one long context
        dict(_attend(1, 131072, 64, 8, 128, 16, ragged=False), name="attend 1 x 131072"),
        # a large padded batch over a cache in 8 bits, 16 query heads to each of its heads
        dict(_attend(192, 8192, 128, 8, 128, 32, cache="fp8", empty=17), name="attend fp8 192 x 8192"),
        # a projection of a decode step
        dict(_linear(64, 7168, 16384), name="fp8 linear decode 64"),
        # a projection of a prefill step
        dict(_linear(8192, 18432, 7168), name="fp8 linear prefill 8192"),
        # sizes that fill no tile, 32-bit outputs
        dict(_linear(777, 1001, 1536, out="f32"), name="fp8 linear odd 777x1001x1536"),
    ]


def _log_int(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rotary(rng):
    while True:
        T, H = _log_int(rng, 1, 16384), _log_int(rng, 1, 128)
        D = rng.choice([64, 80, 96, 128, 128, 192, 256, rng.randint(8, 256)])
        if T * H * D <= 8192 * 72 * 128:
            break
    R = rng.choice([D // 2 * 2, max(2, D // 4 * 2), max(2, D // 8 * 2)])
    return _rotary(T, H, D, R, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                   pairs=rng.choice(["half", "neighbours"]), start=rng.choice([0, D - R]),
                   far=_log_int(rng, 64, 1 << 20), factor=rng.choice([1.0, 4.0, 40.0]), inverse=rng.random() < 0.3)


def _draw_append(rng):
    while True:
        B, new, past = _log_int(rng, 1, 512), rng.choice([0, 0, _log_int(rng, 1, 4096)]), _log_int(rng, 1, 8192)
        Hkv, D = _log_int(rng, 1, 32), rng.choice([64, 128, 128, 256, 8 * rng.randint(2, 32)])
        Hq = rng.choice([0, Hkv, 4 * Hkv, 8 * Hkv])
        if B * max(1, new) * (Hq + 2 * Hkv) * D <= 4 * 4096 * 80 * 128 and B * (new + past) * Hkv * D <= 1 << 28:
            break
    R = rng.choice([D, D // 2])
    return _append(B, new, past, Hkv, D, R, rng.choice([1, 16, 32, 64, 128, rng.randint(2, 100)]),
                   dtype=rng.choice(["bf16", "bf16", "f16"]), Hq=Hq, pairs=rng.choice(["half", "neighbours"]),
                   start=rng.choice([0, D - R]), factor=rng.choice([1.0, 8.0]),
                   padding=rng.choice([0, 0, rng.randint(1, 200)]) if Hq == 0 else 0)


def _draw_attend(rng):
    while True:
        B, longest = _log_int(rng, 1, 512), _log_int(rng, 1, 131072)
        Hkv, G = _log_int(rng, 1, 32), rng.choice([1, 2, 4, 7, 8, 8, 12, 16, 32, 64])
        cache = rng.choice(["same", "same", "fp8"])
        D = rng.choice([64, 128, 128, 128, 256, 16 * rng.randint(2, 16)])
        if B * longest * Hkv * D <= 192 * 8192 * 8 * 128 // (1 if cache == "fp8" else 2) and Hkv * G <= 256:
            break
    dtype = rng.choice(["bf16", "bf16", "f16"])
    return _attend(B, longest, Hkv * G, Hkv, D, rng.choice([1, 16, 32, 64, 128, rng.randint(2, 100)]), dtype=dtype,
                   cache=dtype if cache == "same" else cache, ragged=rng.random() < 0.7,
                   window=rng.choice([0, 0, 0, _log_int(rng, 1, 4096)]), empty=rng.choice([0, 0, min(B - 1, 3)]))


def _draw_linear(rng):
    while True:
        M, N, K = _log_int(rng, 1, 8192), _log_int(rng, 1, 24576), 128 * _log_int(rng, 1, 144)
        if M * N * K <= 8192 * 18432 * 7168 and N * K >= 65536:
            break
    if rng.random() < 0.7:  # most models' widths are round; the number of tokens is not
        N = max(64, N // 64 * 64)
    return _linear(M, N, K, out=rng.choice(["bf16", "bf16", "f16", "f32"]))


def draw(rng):
    return rng.choice([_draw_rotary, _draw_append, _draw_attend, _draw_linear])(rng)


def _lengths(case):
    """Tokens of each sequence before and in the call: from the case alone, so that the work is known without inputs."""
    B = case["B"]
    if case["op"] == "attend":
        n = case["longest"]
        lens = [n - (n * ((37 * b + 11) % 97) // 97 if case["ragged"] and b else 0) for b in range(B)]
        for j in range(case["empty"]):
            lens[(B - 1) - j * (B // max(1, case["empty"]))] = 0
        return lens, [0] * B
    new = [case["new"] - case["new"] * ((53 * b) % 71) // 90 for b in range(B)] if case["new"] else [1] * B
    past = [case["past"] * ((29 * b + 90) % 101) // 101 for b in range(B)]
    return past, new


def work(case):
    s = _SIZE[case.get("dtype", "bf16")]
    if case["op"] == "rotary":
        n = case["T"] * case["H"]
        return {"bytes": 2 * n * case["D"] * s + 8 * case["T"], "flops": 3 * n * case["R"]}
    if case["op"] == "append":
        new = sum(_lengths(case)[1])
        heads = 2 * case["Hkv"] + case["Hq"]
        return {"bytes": 2 * new * heads * case["D"] * s + 4 * new, "flops": 3 * new * (heads - case["Hkv"]) * case["R"]}
    if case["op"] == "attend":
        w = case["window"]
        tokens = sum(min(n, w) if w else n for n in _lengths(case)[0])
        kv = 2 * tokens * case["Hkv"] * case["D"] * _SIZE[case["cache"]]
        return {"bytes": kv + 2 * case["B"] * case["Hq"] * case["D"] * s, "flops": 4 * tokens * case["Hq"] * case["D"]}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": (M + N) * K + 4 * M * (K // 128) + 4 * -(-N // 128) * (K // 128) + M * N * _SIZE[case["out"]],
            "flops": 2 * M * N * K}


# --- inputs --------------------------------------------------------------------------------------------------

def _inv_freq(R, factor):
    """Radians per position of each pair: base 10000, and where the context was extended `factor` times beyond 4096,
    frequencies of less than one turn over it divided by factor, those of more than 32 kept, in between a ramp (YaRN)."""
    at = [10000.0 ** (-2.0 * i / R) for i in range(R // 2)]
    if factor == 1.0:
        return at

    def pair_of(turns):
        return R * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))
    lo, hi = max(math.floor(pair_of(32)), 0), min(math.ceil(pair_of(1)), R - 1)
    keep = [1.0 - min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(R // 2)]
    return [f / factor * (1.0 - k) + f * k for f, k in zip(at, keep)]


def _frequencies(st, R, factor, dev):
    """The same twice: radians in 64 bits, and turns per position in units of 2^-64."""
    f = _inv_freq(R, factor)
    st["inv_freq"] = torch.tensor(f, dtype=torch.float64, device=dev)
    st["freqs"] = torch.tensor([int(v / (2 * math.pi) * 2.0 ** 64) for v in f], dtype=torch.int64, device=dev)
    st["scale"] = 1.0 if factor == 1.0 else 0.1 * math.log(factor) + 1.0


def _pages(lens, page, g, dev):
    """A page table for sequences of these lengths, its pages in random order among a few that nobody has; -1 behind."""
    need = torch.tensor([-(-n // page) for n in lens], dtype=torch.int64)
    first = torch.cumsum(need, 0) - need
    total = int(need.sum())
    order = torch.randperm(total + 3, generator=g, device=dev).to(torch.int32)
    at = torch.arange(max(1, int(need.max())))[None, :]
    use = (at < need[:, None]).to(dev)
    table = torch.where(use, order[torch.where(use, (first[:, None] + at).to(dev), 0)], -1)
    return table.to(torch.int32).contiguous(), total + 3


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    st = {"case": case}
    dt = _DT[case.get("dtype", "bf16")]
    if case["op"] == "rotary":
        T, H, D = case["T"], case["H"], case["D"]
        st["x"] = randn(T, H, D).to(dt)
        st["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=dev, dtype=torch.int32)
        _frequencies(st, case["R"], case["factor"], dev)
    elif case["op"] == "append":
        past, new = _lengths(case)
        Hkv, D, page = case["Hkv"], case["D"], case["page"]
        rows = sum(new) + case["padding"]
        st["table"], count = _pages([a + b for a, b in zip(past, new)], page, g, dev)
        st["k"], st["v"] = randn(rows, Hkv, D).to(dt), randn(rows, Hkv, D).to(dt)
        st["q"] = randn(rows, case["Hq"], D).to(dt) if case["Hq"] else None
        st["k_cache"] = randn(count, page, Hkv, D).to(dt)
        st["v_cache"] = randn(count, page, Hkv, D).to(dt)
        st["lens"] = torch.tensor([a + b for a, b in zip(past, new)], dtype=torch.int32, device=dev)
        ends = torch.cumsum(torch.tensor([0] + new), 0)
        st["indptr"] = ends.to(torch.int32).to(dev) if case["new"] else None  # one new token each needs none
        _frequencies(st, case["R"], case["factor"], dev)
    elif case["op"] == "attend":
        lens, _ = _lengths(case)
        Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
        st["table"], count = _pages(lens, page, g, dev)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        st["q"] = (1.5 * randn(case["B"], Hq, D)).to(dt)
        caches = []
        for _ in range(2):
            c = torch.empty((count, page, Hkv, D), dtype=dt, device=dev).normal_(generator=g)
            c[table_free(st["table"], count)] = math.nan  # what nobody wrote
            if case["cache"] == "fp8":
                c = (c * 32.0).to(torch.float8_e4m3fn)
            caches.append(c)
        st["k_cache"], st["v_cache"] = caches
        scale = 1.0 / 32.0 if case["cache"] == "fp8" else 1.0
        st["k_scale"] = scale * (1.0 + 0.2 * torch.rand(Hkv, generator=g, device=dev)) if scale != 1.0 else None
        st["v_scale"] = scale * (1.0 + 0.2 * torch.rand(Hkv, generator=g, device=dev)) if scale != 1.0 else None
    else:
        M, N, K = case["M"], case["N"], case["K"]
        x = randn(M, K // 128, 128) * (1.0 + 3.0 * torch.rand(M, 1, 1, generator=g, device=dev))
        s = x.abs().amax(2).clamp_min(1e-12) / 448.0
        st["a"] = (x / s[:, :, None]).to(torch.float8_e4m3fn).view(M, K).view(torch.uint8)
        ld = max(4, (M + 3) // 4 * 4)
        st["a_scales"] = torch.zeros((K // 128, ld), device=dev)
        st["a_scales"][:, :M] = s.t()
        st["b"] = randn(N, K).mul_(96.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        st["b_scales"] = (0.5 + torch.rand((-(-N // 128), K // 128), generator=g, device=dev)) / (96.0 * math.sqrt(K))
    return st


def table_free(table, count):
    """The pages that no sequence has."""
    free = torch.ones(count + 1, dtype=torch.bool, device=table.device)
    free[table.flatten().long()] = False  # -1 is the place behind the last page
    return free[:count]


# --- one pass ------------------------------------------------------------------------------------------------

def run(st):
    op = st["case"]["op"]
    if own:
        return {"rotary": _own_rotary, "append": _own_append, "attend": _own_attend, "linear": _own_linear}[op](st)
    return {"rotary": _plain_rotary, "append": _plain_append, "attend": _plain_attend, "linear": _plain_linear}[op](st)


def _own_rotary(st):
    import w4afp8_mixture_experts_gb300 as lib
    c = st["case"]
    return lib.rotary_embedding(st["x"], st["positions"], st["freqs"], interleaved=c["pairs"] == "neighbours",
                                start=c["start"], scale=st["scale"], inverse=c["inverse"])


def _own_append(st):
    import w4afp8_mixture_experts_gb300 as lib
    c = st["case"]
    q = lib.paged_kv_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["lens"], st["indptr"],
                            freqs=st["freqs"], interleaved=c["pairs"] == "neighbours", start=c["start"],
                            scale=st["scale"], q=st["q"])
    return st["k_cache"], st["v_cache"], q


def _own_attend(st):
    import w4afp8_mixture_experts_gb300 as lib
    return lib.paged_attention_decode(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                                      window=st["case"]["window"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                                      return_lse=True)


def _own_linear(st):
    import w4afp8_mixture_experts_gb300 as lib
    return lib.fp8_block_linear(st["a"], st["a_scales"], st["b"], st["b_scales"], out_dtype=_DT[st["case"]["out"]])


def _plain_rotate(x, positions, st, inverse=False):
    """x [T, H, D] in 32 bits, rotated; the angles in 64 bits."""
    c = st["case"]
    R, s = c["R"], c["start"]
    angle = positions.double()[:, None] * st["inv_freq"][None, :]
    cos = (angle.cos() * st["scale"]).float()[:, None, :]
    sin = (angle.sin() * (-st["scale"] if inverse else st["scale"])).float()[:, None, :]
    part = x[:, :, s:s + R]
    first, second = ((part[:, :, : R // 2], part[:, :, R // 2:]) if c["pairs"] == "half"
                     else (part[:, :, 0::2], part[:, :, 1::2]))
    a, b = first * cos - second * sin, second * cos + first * sin
    turned = torch.cat([a, b], 2) if c["pairs"] == "half" else torch.stack([a, b], 3).flatten(2)
    return torch.cat([x[:, :, :s], turned, x[:, :, s + R:]], 2)


def _plain_rotary(st):
    x = st["x"]
    return _plain_rotate(x.float(), st["positions"], st, st["case"]["inverse"]).to(x.dtype)


def _plain_append(st):
    c = st["case"]
    lens = st["lens"].long()
    if st["indptr"] is None:
        seq, at = torch.arange(c["B"], device=lens.device), lens - 1
    else:
        ends = st["indptr"].long()
        row = torch.arange(sum(_lengths(c)[1]), device=lens.device)
        seq = torch.searchsorted(ends[1:].contiguous(), row, right=True)
        at = lens[seq] - (ends[seq + 1] - row)
    n = seq.numel()
    place = (st["table"][seq, at // c["page"]].long(), at % c["page"])
    st["k_cache"][place] = _plain_rotate(st["k"][:n].float(), at, st).to(st["k"].dtype)
    st["v_cache"][place] = st["v"][:n]
    q = None if st["q"] is None else _plain_rotate(st["q"][:n].float(), at, st).to(st["q"].dtype)
    return st["k_cache"], st["v_cache"], q


def _plain_attend(st):
    c = st["case"]
    q, table, lens = st["q"], st["table"], st["lens"].long()
    B, Hq, D = q.shape
    Hkv, G, page = c["Hkv"], c["Hq"] // c["Hkv"], c["page"]
    L = table.shape[1] * page
    at = torch.arange(L, device=q.device)[None, :]
    seen = at < lens[:, None]
    if c["window"]:
        seen = seen & (at >= lens[:, None] - c["window"])
    away = ~seen[:, :, None, None]
    pages = table.long().clamp_min(0)
    k = st["k_cache"][pages].view(B, L, Hkv, D).float().masked_fill_(away, 0.0)
    s = torch.matmul(q.float().view(B, Hkv, G, D), k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(D))
    if st["k_scale"] is not None:
        s = s * st["k_scale"][None, :, None, None]
    del k
    s = s.masked_fill_(~seen[:, None, None, :], -math.inf)
    top = s.amax(3, keepdim=True)
    top = torch.where(top > -math.inf, top, torch.zeros_like(top))
    p = torch.exp(s - top)
    total = p.sum(3, keepdim=True)
    v = st["v_cache"][pages].view(B, L, Hkv, D).float().masked_fill_(away, 0.0)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, torch.ones_like(total))
    if st["v_scale"] is not None:
        o = o * st["v_scale"][None, :, None, None]
    return o.reshape(B, Hq, D).to(q.dtype), (torch.log(total) + top).view(B, Hq)


def _plain_linear(st):
    c = st["case"]
    M, N, K = c["M"], c["N"], c["K"]
    a = st["a"].view(torch.float8_e4m3fn).float().view(M, K // 128, 128) * st["a_scales"][:, :M].t()[:, :, None]
    w = st["b"].view(torch.float8_e4m3fn).float().view(N, K // 128, 128)
    w = w * st["b_scales"].repeat_interleave(128, dim=0)[:N, :, None]
    return (a.view(M, K) @ w.view(N, K).t()).to(_DT[c["out"]])


# --- the definitions in 64 bits --------------------------------------------------------------------------------

def _exact_rotate(x, positions, st, inverse=False):
    """The rotated part as complex numbers times scale * e^(i angle)."""
    c = st["case"]
    R, s = c["R"], c["start"]
    out = x.double().clone()
    part = out[..., s:s + R].unflatten(-1, (2, R // 2) if c["pairs"] == "half" else (R // 2, 2))
    axis = -2 if c["pairs"] == "half" else -1
    z = torch.complex(part.select(axis, 0).contiguous(), part.select(axis, 1).contiguous())
    f = torch.tensor(_inv_freq(R, c["factor"]), dtype=torch.float64, device=x.device)
    angle = torch.outer(positions.double(), f)
    z = z * torch.polar(torch.full_like(angle, st["scale"]), -angle if inverse else angle)[:, None, :]
    out[..., s:s + R] = torch.stack([z.real, z.imag], axis).flatten(-2)
    return out


def _exact_append(st):
    c = st["case"]
    past, new = _lengths(c)
    seq = torch.tensor([b for b, n in enumerate(new) for _ in range(n)])
    at = torch.tensor([a + i for a, n in zip(past, new) for i in range(n)])
    slot = (st["table"].cpu().long()[seq, at // c["page"]] * c["page"] + at % c["page"]).cuda()
    n, at = len(seq), at.cuda()
    k, v = (st[name].double().flatten(0, 1) for name in ("k_cache", "v_cache"))
    k[slot] = _exact_rotate(st["k"][:n], at, st)
    v[slot] = st["v"][:n].double()
    q = None if st["q"] is None else _exact_rotate(st["q"][:n], at, st)
    return k.view(st["k_cache"].shape), v.view(st["v_cache"].shape), q


def _exact_attend(st):
    c = st["case"]
    Hkv, D = c["Hkv"], c["D"]
    q = st["q"].double() / math.sqrt(D)
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for b, n in enumerate(_lengths(c)[0]):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            continue
        at = torch.arange(lo, n, device=q.device)
        slot = st["table"][b].long()[at // c["page"]] * c["page"] + at % c["page"]
        k, v = (st[name].flatten(0, 1)[slot].double() for name in ("k_cache", "v_cache"))
        if st["k_scale"] is not None:
            k, v = k * st["k_scale"].double()[None, :, None], v * st["v_scale"].double()[None, :, None]
        s = torch.einsum("hgd,nhd->hgn", q[b].view(Hkv, -1, D), k)
        lse[b] = torch.logsumexp(s, 2).flatten()
        out[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(s, 2), v).flatten(0, 1)
    return out, lse


def _exact_linear(st):
    c = st["case"]
    M, N, K = c["M"], c["N"], c["K"]
    z = torch.zeros((M, N), dtype=torch.float64, device=st["a"].device)
    for j in range(0, K // 128, 8):  # eight blocks of K at a time, each operand scaled before the product
        cols = slice(128 * j, min(K, 128 * (j + 8)))
        a = st["a"][:, cols].contiguous().view(torch.float8_e4m3fn).double()
        w = st["b"][:, cols].contiguous().view(torch.float8_e4m3fn).double()
        a = a * st["a_scales"][j:j + 8, :M].double().t().repeat_interleave(128, 1)
        w = w * st["b_scales"][:, j:j + 8].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
        z.addmm_(a, w.t())
    return z


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotate(st["x"], st["positions"], st, case["inverse"])
    return {"append": _exact_append, "attend": _exact_attend, "linear": _exact_linear}[case["op"]](st)
