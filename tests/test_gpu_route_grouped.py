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
