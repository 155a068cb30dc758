"""Grouped routing on the GPU against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

F32_MIN = float(np.finfo(np.float32).min)


def _run(lib, logits, k, **kw):
    bias = kw.pop("bias", None)
    t = logits if isinstance(logits, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(logits)).cuda()
    b = None if bias is None else torch.from_numpy(np.asarray(bias, np.float32)).cuda()
    ids, w = lib.moe_route_grouped_topk(t, k, bias=b, **kw)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def _logits(rng, T, E, bias, kw, dtype=torch.float32):
    """Logits of the type whose compared values all differ by more than fp32 scores can be off (rows are redrawn)."""
    out = np.zeros((T, E), np.float32)
    todo = np.arange(T)
    for _ in range(2000):
        if not todo.size:
            return out
        l = torch.from_numpy(rng.standard_normal((todo.size, E)).astype(np.float32) * 2).to(dtype).float().numpy()
        _, _, gap = ref.route(l, 1, kw["score"], bias, kw.get("n_group", 1), kw.get("topk_group", 1),
                              kw.get("group_top", 1))
        ok = gap > 2e-6  # scores and sums of two: at most four roundings of 2^-24 below 4
        out[todo[ok]] = l[ok]
        todo = todo[~ok]
    raise AssertionError("no rows without near ties")


CASES = [
    # E, k, keywords, bias
    (256, 8, dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5), True),
    (256, 8, dict(score="sigmoid", n_group=8, topk_group=8, group_top=2), True),
    (160, 6, dict(score="softmax", n_group=8, topk_group=3, renormalize=False, scale=16.0), False),
    (64, 6, dict(score="softmax", renormalize=False), False),
    (60, 4, dict(score="softmax", n_group=4, topk_group=2, group_top=2), True),
    (61, 7, dict(score="sigmoid"), False),
    (128, 1, dict(score="sigmoid", n_group=16, topk_group=1), True),
    (33, 3, dict(score="sigmoid", n_group=11, topk_group=1, group_top=2), False),
    (1, 1, dict(score="softmax"), False),
    (5, 5, dict(score="sigmoid"), True),
    (1, 1, dict(score="sigmoid", renormalize=False), True),
    (96, 32, dict(score="sigmoid", n_group=3, topk_group=2, group_top=2), True),
    (510, 8, dict(score="sigmoid", n_group=17, topk_group=5, group_top=2), False),
    (300, 9, dict(score="sigmoid", n_group=1), False),
    (320, 16, dict(score="sigmoid", n_group=32, topk_group=7, group_top=2), True),
    (384, 6, dict(score="sigmoid", n_group=16, topk_group=4), False),
    (384, 8, dict(score="sigmoid"), True),
    (454, 6, dict(score="softmax"), False),
    (900, 12, dict(score="sigmoid", n_group=2, topk_group=1), False),
    (160, 16, dict(score="softmax", n_group=2, topk_group=1, renormalize=False), False),
    (24, 3, dict(score="sigmoid", n_group=8, topk_group=3), True),
    (40, 8, dict(score="softmax", n_group=5, topk_group=4, group_top=2), True),
    (96, 12, dict(score="sigmoid", n_group=4, topk_group=3, group_top=2), False),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("T", [1, 37])
def test_against_definition(lib, case, T):
    E, k, kw, with_bias = CASES[case]
    rng = np.random.default_rng(100 + case)
    bias = rng.standard_normal(E).astype(np.float32) * 0.1 if with_bias else None
    logits = _logits(rng, T, E, bias, kw)
    ids, w = _run(lib, logits, k, bias=bias, **kw)
    rid, rw, _ = ref.route(logits, k, bias=bias, **kw)
    assert np.array_equal(ids, rid)
    assert np.all(np.abs(w - rw) <= 64 * 2.0 ** -24 * rw + 1e-37)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_16_bit_logits_and_row_stride(lib, dtype):
    kw = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2)
    rng = np.random.default_rng(5)
    bias = rng.standard_normal(48).astype(np.float32) * 0.2  # separates logits that are equal in 16 bits
    logits = _logits(rng, 9, 48, bias, kw, dtype)
    wide = torch.full((9, 53), float("nan"), dtype=dtype, device="cuda")
    wide[:, 2:50] = torch.from_numpy(logits).to(dtype)
    ids, w = _run(lib, wide[:, 2:50], 6, bias=bias, **kw)
    rid, rw, _ = ref.route(logits, 6, bias=bias, **kw)
    assert np.array_equal(ids, rid)
    assert np.all(np.abs(w - rw) <= 64 * 2.0 ** -24 * rw)


def test_ties_go_to_the_lowest_id_and_group(lib):
    logits = np.zeros((3, 64), np.float32)
    logits[1, 40:48] = 1.0
    logits[2] = -0.0
    logits[2, ::2] = 0.0
    ids, w = _run(lib, logits, 6, score="sigmoid", n_group=8, topk_group=2, group_top=2)
    assert ids.tolist() == [[0, 1, 2, 3, 4, 5], [40, 41, 42, 43, 44, 45], [0, 1, 2, 3, 4, 5]]
    assert np.all(np.abs(w - 1 / 6) <= 2.0 ** -22)
    ids, _ = _run(lib, logits, 3, score="softmax")
    assert ids.tolist() == [[0, 1, 2], [40, 41, 42], [0, 1, 2]]
    # sigmoid saturates: scores that round to the same fp32 value are equal
    ids, _ = _run(lib, np.array([[20.0, 30.0, 1.0, 40.0]], np.float32), 3, score="sigmoid")
    assert ids.tolist() == [[0, 1, 3]]


@pytest.mark.parametrize("away", [-np.inf, F32_MIN, np.nan])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_masked_experts(lib, away, score):
    rng = np.random.default_rng(8)
    logits = rng.standard_normal((6, 24)).astype(np.float32)
    bias = np.full(24, 3.0, np.float32) if score == "sigmoid" else None  # a bias does not bring a masked expert back
    logits[0] = away                 # nothing left: the lowest ids with weight 0
    logits[1, 1:] = away             # one expert left
    logits[2, :6] = away             # a whole group out
    logits[3, [0, 7, 13, 23]] = away
    logits[4, 3:] = away             # three left, all in the first group
    for kw in (dict(n_group=4, topk_group=2, group_top=2), dict(n_group=4, topk_group=1, group_top=1), dict()):
        ids, w = _run(lib, logits, 5, bias=bias, score=score, **kw)
        rid, rw, _ = ref.route(logits, 5, score, bias, **kw)
        assert np.array_equal(ids, rid), (kw, ids, rid)
        assert np.all(np.abs(w - rw) <= 64 * 2.0 ** -24 * rw)
        assert np.all(w[0] == 0) and np.all(np.sort(ids, axis=1)[:, 1:] != np.sort(ids, axis=1)[:, :-1])


def test_infinite_and_huge_logits(lib):
    logits = np.array([[np.inf, 0, np.inf, 1], [3e38, 0, -3e38, 1], [-100.0, -101.0, -200.0, -3e38]], np.float32)
    ids, w = _run(lib, logits, 3, score="softmax")
    assert ids.tolist() == [[0, 2, 3], [0, 3, 1], [0, 1, 2]]
    e = np.exp(-1.0)
    assert np.allclose(w, [[0.5, 0.5, 0], [1, 0, 0], [1 / (1 + e), e / (1 + e), 0]], rtol=1e-6, atol=1e-30)
    ids, w = _run(lib, logits[:2], 3, score="sigmoid", renormalize=False)
    assert ids.tolist() == [[0, 2, 3], [0, 3, 1]]
    assert np.allclose(w, [[1, 1, 1 / (1 + e)], [1, 1 / (1 + e), 0.5]], rtol=1e-6)


def test_same_choice_as_the_plain_router(lib):
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.standard_normal((500, 256)).astype(np.float32)).cuda()
    for renorm in (True, False):
        a, aw = lib.moe_route_topk(x, 8, renorm)
        b, bw = lib.moe_route_grouped_topk(x, 8, score="softmax", renormalize=renorm)
        assert torch.equal(a, b)
        assert torch.all((aw - bw).abs() <= 32 * 2.0 ** -24 * aw)


def test_many_tokens_and_no_tokens(lib):
    kw = dict(score="sigmoid", n_group=8, topk_group=4, group_top=2)
    x = torch.randn((20011, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    ids, w = lib.moe_route_grouped_topk(x, 4, **kw)
    for part in (slice(0, 3), slice(9000, 9004), slice(20008, 20011)):  # a token's result does not depend on its place
        i, v = lib.moe_route_grouped_topk(x[part].contiguous(), 4, **kw)
        assert torch.equal(i, ids[part]) and torch.equal(v, w[part])
    ids, w = lib.moe_route_grouped_topk(x[:0], 4, **kw)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def test_refusals(lib):
    x = torch.zeros((4, 16), device="cuda")
    for kw, what in [(dict(k=0), "k=0"), (dict(k=17), "k=17"), (dict(k=2, n_group=3), "n_group=3"),
                     (dict(k=2, n_group=4, topk_group=5), "topk_group=5"), (dict(k=2, group_top=3), "group_top=3"),
                     (dict(k=5, n_group=4, topk_group=1), "k=5"), (dict(k=2, n_group=16, group_top=2), "group_top=2")]:
        with pytest.raises(lib.W4A8Error, match=what):
            lib.moe_route_grouped_topk(x, **kw)
    with pytest.raises(ValueError, match="score"):
        lib.moe_route_grouped_topk(x, 2, score="tanh")
    with pytest.raises(ValueError, match="bias"):
        lib.moe_route_grouped_topk(x, 2, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(TypeError, match="logits"):
        lib.moe_route_grouped_topk(x.double(), 2)
    with pytest.raises(TypeError, match="logits"):
        lib.moe_route_grouped_topk(x.cpu(), 2)
    with pytest.raises(ValueError, match="contiguous rows"):
        lib.moe_route_grouped_topk(torch.zeros((16, 4), device="cuda").t(), 2)


def _pairs_of_softmax(l, k, n_group, topk_group, away):
    """(ids, distance of the logarithms of the group scores that decide): groups by the sum of their two largest softmax
    scores, in 64 bits."""
    ids, gap = [], []
    for row, out in zip(np.asarray(l, np.float64), away):
        e = np.where(out, 0.0, np.exp(np.where(out, 0.0, row - np.max(row[~out], initial=-1e300))))
        with np.errstate(divide="ignore"):
            c = np.where(out, -np.inf, e / e.sum() if e.sum() else e).reshape(n_group, -1)
            two = np.log(np.maximum(np.sort(c, axis=1)[:, -2:].sum(axis=1), 0.0))
        order = np.argsort(-two, kind="stable")
        best = two[order]
        gap.append(best[topk_group - 1] - best[topk_group] if topk_group < n_group and np.isfinite(best[topk_group - 1])
                   else np.inf)
        kept = np.isin(np.arange(n_group), order[:topk_group])
        live = np.where(out | ~np.repeat(kept, c.shape[1]), -np.inf, row)
        ids.append(np.argsort(-live, kind="stable")[:k])
    return np.array(ids), np.array(gap)


@pytest.mark.parametrize("E,k,G,keep", [(64, 6, 8, 3), (256, 8, 8, 4), (40, 8, 5, 4), (96, 3, 4, 1), (512, 8, 16, 5)])
@pytest.mark.parametrize("spread,offset", [(2.0, 0.0), (0.3, 1000.0), (60.0, -50.0)])
@pytest.mark.parametrize("masked", [False, True])
def test_groups_by_the_sum_of_two_softmax_scores(lib, E, k, G, keep, spread, offset, masked):
    rng = np.random.default_rng(E + k)
    l = (rng.standard_normal((300, E)) * spread + offset).astype(np.float32)
    away = rng.random((300, E)) < (0.3 if masked else 0.0)
    l[away] = -np.inf
    ids, _ = _run(lib, l, k, score="softmax", n_group=G, topk_group=keep, group_top=2)
    rid, gap = _pairs_of_softmax(l, k, G, keep, away)
    # the logarithm is off by at most its subtraction, sum and 4 units of exp and log1p, all below 2^9 * 2^-24 = 4e-5
    far = gap > 1e-4
    assert far.mean() > 0.9
    assert np.array_equal(ids[far], rid[far])
    if offset == 0.0 and not masked:  # a bias of zeros changes no sum
        with_bias, _ = _run(lib, l, k, bias=np.zeros(E, np.float32), score="softmax", n_group=G, topk_group=keep, group_top=2)
        assert np.array_equal(np.sort(ids[far], 1), np.sort(with_bias[far], 1))


def test_groups_of_two_with_infinite_logits(lib):
    l = np.zeros((3, 12), np.float32)
    l[0, [4, 9]] = np.inf          # one infinite logit in each of two groups: equal sums, lower group first
    l[1, [8, 9, 4]] = np.inf       # two in the last group
    l[1, 0:4] = 5.0                # finite scores are 0 beside an infinite one
    l[2, :] = [3e38, -3e38, 0, 0, 3e38, 3e38, 0, 0, 1, 1, 1, 1]
    ids, _ = _run(lib, l, 2, score="softmax", n_group=3, topk_group=1, group_top=2)
    assert ids.tolist() == [[4, 5], [8, 9], [4, 5]]


@pytest.mark.parametrize("T,E,k,kw,with_bias", [
    (20011, 64, 4, dict(score="sigmoid", n_group=8, topk_group=4, group_top=2), True),        # 8 lanes to a token
    (10003, 160, 6, dict(score="softmax", n_group=8, topk_group=3, renormalize=False), False),  # 16
    (10003, 96, 12, dict(score="sigmoid", n_group=4, topk_group=3, group_top=2), False),
    (5107, 256, 8, dict(score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5), True),  # 32
    (5107, 454, 6, dict(score="softmax"), False),
    (5107, 384, 8, dict(score="sigmoid"), True),
])
def test_more_tokens_than_the_device_holds(lib, T, E, k, kw, with_bias):
    # every warp walks through several tokens: the first, some in between and the last against the definition, all of them
    # against calls that are too short for that
    rng = np.random.default_rng(E)
    x = torch.randn((T, E), device="cuda", generator=torch.Generator("cuda").manual_seed(E)) * 2
    bias = rng.standard_normal(E).astype(np.float32) * 0.1 if with_bias else None
    dev_bias = None if bias is None else torch.from_numpy(bias).cuda()
    ids, w = lib.moe_route_grouped_topk(x, k, bias=dev_bias, **kw)
    for at in range(0, T, 2000):
        i, v = lib.moe_route_grouped_topk(x[at:at + 2000], k, bias=dev_bias, **kw)
        assert torch.equal(i, ids[at:at + 2000]) and torch.equal(v, w[at:at + 2000])
    rows = np.r_[0:100, T // 2:T // 2 + 50, T - 250:T]
    rid, rw, gap = ref.route(x.cpu().numpy()[rows], k, bias=bias, **kw)
    far = gap > 2e-6  # as above
    assert far.mean() > 0.4
    assert np.array_equal(ids.cpu().numpy()[rows][far], rid[far])
    assert np.all(np.abs(w.cpu().double().numpy()[rows][far] - rw[far]) <= 64 * 2.0 ** -24 * rw[far] + 1e-37)


@pytest.mark.parametrize("T", [1, 40, 6000])
def test_other_stream_and_graph(lib, T):
    x = torch.randn((T, 256), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    kw = dict(n_group=8, topk_group=4, group_top=2)
    want = lib.moe_route_grouped_topk(x, 8, **kw)
    given = torch.zeros_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.moe_route_grouped_topk(given, 8, **kw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = lib.moe_route_grouped_topk(given, 8, **kw)
        given.copy_(x)
        graph.replay()
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
