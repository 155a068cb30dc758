"""The example block on the GPU: its operators run together, against a plain 64-bit block on the CPU."""
import os
import sys

import numpy as np
import pytest
import torch

import block_reference as ref
import oracle
from gpu_util import decode_prepacked, rel_fro

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


def _rms(v, w, eps=1e-6):
    return v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps) * w


@pytest.mark.parametrize("T", [1, 37, 300])
@pytest.mark.parametrize("post", [True, False])
def test_block_against_plain(lib, T, post):
    import moe_block
    H, I, E, k = 256, 128, 16, 4
    block = moe_block.random_block(H, I, E, k, shared=192, n_group=4, topk_group=2, seed=3)
    if not post:
        block.norm_out = None
    g = torch.Generator("cuda").manual_seed(T)
    attn, residual = (torch.randn((T, H), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    keep = residual.clone()
    out_res, out_y = block(attn, residual)
    torch.cuda.synchronize()
    assert lib.device_error() == 0 and torch.equal(residual, keep)  # inputs are not touched

    r = _np(attn) + _np(residual)
    x = oracle.round_bf16(_rms(r, _np(block.norm_in)))
    r = oracle.round_bf16(r)
    logits = x @ _np(block.gate).T
    # the routing that the block computed itself, so that a near tie does not decide the comparison
    x_dev = torch.from_numpy(np.asarray(x, np.float32)).cuda().to(torch.bfloat16)
    ids, w = (t.cpu().numpy() for t in block.route(x_dev))
    rid, rw, gap = ref.route(logits, k, "sigmoid", _np(block.gate_bias), 4, 2, 2, True, 2.5)
    far = gap > 1e-5  # logits differ by the rounding of x here and there
    assert far.mean() > 0.9 or T == 1
    assert np.array_equal(ids[far], rid[far]) and np.allclose(w[far], rw[far], rtol=1e-4)
    w13, w13_s, w2, w2_s = block.experts
    W13 = decode_prepacked(w13.cpu().numpy()).astype(np.float64) * np.repeat(_np(w13_s), 128, axis=1).transpose(0, 2, 1)
    W2 = decode_prepacked(w2.cpu().numpy()).astype(np.float64) * np.repeat(_np(w2_s), 128, axis=1).transpose(0, 2, 1)
    routed = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            z = W13[ids[t, j]] @ x[t]
            routed[t] += w[t, j] * (W2[ids[t, j]] @ (z[:I] / (1 + np.exp(-z[:I])) * z[I:]))
    z = x @ _np(block.shared_up).T
    f = (z[:, :192] / (1 + np.exp(-z[:, :192])) * z[:, 192:]) @ _np(block.shared_down).T + routed
    u = _rms(f, _np(block.norm_out)) if post else f
    h = r + u
    y = _rms(h, _np(block.norm_next))
    # E4M3 activations have relative steps of 2^-4: rounding errors of at most 2^-4 and rms 2^-4 / sqrt(12) = 1.8 %, twice
    # in the routed half; everything else is rounded to bf16 (0.2 %)
    assert rel_fro(_np(out_res), h) <= 0.04
    assert rel_fro(_np(out_y), y) <= 0.04


def test_given_routing_equals_the_layers_own(lib):
    import moe_block
    block = moe_block.random_block(256, 128, 16, 4, shared=64, n_group=1, topk_group=1, seed=5)
    g = torch.Generator("cuda").manual_seed(9)
    x = torch.randn((150, 256), device="cuda", generator=g).to(torch.bfloat16)
    logits = torch.randn((150, 16), device="cuda", generator=g)
    want = lib.w4a8_moe_forward(x, logits, 4, *block.experts)
    ids, w = lib.moe_route_topk(logits, 4)
    assert torch.equal(lib.w4a8_moe_forward_routed(x, ids, w, *block.experts), want)
    ids, w = lib.moe_route_grouped_topk(logits, 4, score="softmax")
    assert rel_fro(_np(lib.w4a8_moe_forward_routed(x, ids, w, *block.experts)), _np(want)) <= 2.0 ** -8


def test_routed_refusals(lib):
    import moe_block
    block = moe_block.random_block(256, 128, 8, 2, shared=64, n_group=1, topk_group=1)
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    ids, w = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda")
    with pytest.raises(ValueError, match="rows"):
        lib.w4a8_moe_forward_routed(x, ids, w[:3], *block.experts)
    with pytest.raises(lib.W4A8Error, match="k=9"):
        lib.w4a8_moe_forward_routed(x, ids.new_zeros((4, 9)), w.new_zeros((4, 9)), *block.experts)
    with pytest.raises(lib.W4A8Error, match="workspace"):
        lib.w4a8_moe_forward_routed(x, ids, w, *block.experts, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    out = lib.w4a8_moe_forward_routed(x[:0], ids[:0], w[:0], *block.experts)
    assert out.shape == (0, 256)


def test_routed_refuses_what_does_not_fit_the_layer(lib):
    # every one of these would be read or written out of range
    import moe_block
    block = moe_block.random_block(256, 128, 8, 2, shared=64, n_group=1, topk_group=1)
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    ids, w = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda")
    w13, w13_s, w2, w2_s = block.experts
    need = lib.moe_workspace_layout(4, 256, 128, 8, 2).total
    args = dict(x=x, topk_ids=ids, topk_w=w, w13=w13, w13_s=w13_s, w2=w2, w2_s=w2_s, ws=None, out=None)
    ws, out = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty_like(x)
    for name, bad in [("w13", w13[:, :, :64].contiguous()), ("w13", w13[:, :255].contiguous()), ("w2", w2[:7]),
                      ("w2", w2[:, :128].contiguous()), ("w2", w2[:, :, :32].contiguous()), ("w13_s", w13_s[:7]),
                      ("w13_s", w13_s[:, :1].contiguous()), ("w2_s", w2_s[:7]), ("w2_s", w2_s[:, :, :128].contiguous()),
                      ("out", out[:3]), ("out", torch.empty((4, 512), dtype=torch.bfloat16, device="cuda")[:, :256]),
                      ("ws", torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2]), ("topk_ids", ids[:, :1]),
                      ("x", torch.zeros((4, 512), dtype=torch.bfloat16, device="cuda")[:, ::2])]:
        with pytest.raises(ValueError, match=name):
            lib.w4a8_moe_forward_routed(**{**args, name: bad})
    for name, bad in [("out", out.half()), ("out", out.cpu()), ("ws", ws.int()), ("ws", ws.cpu()), ("w2", w2.int()),
                      ("w2_s", w2_s.half()), ("topk_ids", ids.long()), ("topk_w", w.half()), ("topk_w", w.cpu())]:
        with pytest.raises(TypeError, match=name):
            lib.w4a8_moe_forward_routed(**{**args, name: bad})
    assert lib.w4a8_moe_forward_routed(**{**args, "ws": ws, "out": out}) is out


@pytest.mark.parametrize("T", [1, 8, 16, 64, 600])
def test_calls_that_follow_their_producer_at_once(lib, T):
    # each call reads what the one before it writes into the same memory, with nothing in between; the inputs change from
    # turn to turn, so that a value read too early is another one
    g = torch.Generator("cuda").manual_seed(T)
    H, E, turns = 4096, 64, 40
    w = (torch.randn((E, H), device="cuda", generator=g) * H ** -0.5).to(torch.bfloat16)
    up = (torch.randn((H, E), device="cuda", generator=g) * E ** -0.5).to(torch.bfloat16)
    attn = torch.randn((turns, T, H), device="cuda", generator=g).to(torch.bfloat16)
    res = torch.randn((T, H), device="cuda", generator=g).to(torch.bfloat16)
    h, x, f = torch.empty_like(res), torch.empty_like(res), torch.empty_like(res)
    logits = torch.empty((T, E), device="cuda")
    small = torch.empty((T, E), dtype=torch.bfloat16, device="cuda")

    def turn(a, wait):
        outs = []
        for call in (lambda: lib.block_norm(a, res, post="rms", pre="rms", h=h, y=x),
                     lambda: lib.dense_linear(x, w, out_dtype=torch.float32, out=logits),
                     lambda: outs.extend(lib.moe_route_grouped_topk(logits, 4, n_group=8, topk_group=4, group_top=2)),
                     lambda: lib.dense_linear(x, w, act="silu", out=small),
                     lambda: lib.dense_linear(small, up, residual=h, out=f)):
            call()
            if wait:
                torch.cuda.synchronize()
        return outs + [f.clone()]

    at_once = [turn(a, False) for a in attn]
    for a, got in zip(attn, at_once):
        assert all(torch.equal(p, q) for p, q in zip(got, turn(a, True)))
    assert lib.device_error() == 0


@pytest.mark.parametrize("T", [1, 64, 3000])
def test_outputs_are_tensors_of_their_own(lib, T):
    # each output has its own memory, as large as itself: keeping, saving or resizing one does not concern the other
    import io
    f, r = torch.randn((T, 128), device="cuda").to(torch.bfloat16), torch.randn((T, 128), device="cuda")
    for pair in (lib.block_norm(f, r), lib.moe_route_grouped_topk(r, 8)):
        a, b = pair
        assert a.untyped_storage().data_ptr() != b.untyped_storage().data_ptr()
        for t in pair:
            assert t.is_contiguous() and t.storage_offset() == 0
            assert t.untyped_storage().nbytes() == t.numel() * t.element_size()
        file = io.BytesIO()
        torch.save(list(pair), file)
        file.seek(0)
        assert all(torch.equal(p, q) for p, q in zip(torch.load(file), pair))
        keep = b.clone()
        a.resize_(2 * T, a.shape[1]).zero_()
        assert torch.equal(b, keep)
