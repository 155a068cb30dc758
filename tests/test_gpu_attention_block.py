"""The example block's attention half on the GPU: its operators run together, against a plain 64-bit half on the CPU."""
import os
import sys

import numpy as np
import pytest
import torch

import attention_reference as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

VALUES = ref.e4m3_values()


def _np(t):
    return t.double().cpu().numpy()


def _weights(w, s):
    v = VALUES[w.view(torch.uint8).cpu().numpy()]
    return v * np.repeat(np.repeat(_np(s), 128, 0)[:v.shape[0]], 128, 1)


def _rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


class Plain:
    """The same half in 64 bits; the projections' inputs are quantised as the half's, nothing else is rounded."""

    def __init__(self, lib, half, f, scale):
        self.lib, self.half, self.f, self.scale = lib, half, f, scale
        self.wqkv, self.wo = _weights(half.wqkv, half.wqkv_s), _weights(half.wo, half.wo_s)
        self.k, self.v = {}, {}

    def quantised(self, x):
        codes, s, _ = self.lib.fp8_quant_per_token_group(x.to(torch.bfloat16).contiguous())
        return VALUES[codes.cpu().numpy()] * np.repeat(_np(s)[:, :x.shape[0]].T, 128, 1)

    def take(self, x, seq, at):
        x = self.quantised(x)
        Hq, Hkv = self.half.heads, self.half.kv_heads
        qkv = (x @ self.wqkv.T).reshape(x.shape[0], Hq + 2 * Hkv, -1)
        q, _ = ref.rotate(qkv[:, :Hq], at, self.f, scale=self.scale)
        k, _ = ref.rotate(qkv[:, Hq:Hq + Hkv], at, self.f, scale=self.scale)
        for i, b in enumerate(seq):
            self.k.setdefault(b, []).append(k[i])
            self.v.setdefault(b, []).append(qkv[i, Hq + Hkv:])
        return q

    def decode(self, x, seq, at):
        q = self.take(x, seq, at)
        D = q.shape[2]
        o = np.stack([ref.attend(q[i], np.stack(self.k[b]), np.stack(self.v[b]), D ** -0.5, "f32", 0.0)[0]
                      for i, b in enumerate(seq)])
        return self.quantised(torch.from_numpy(o.reshape(len(seq), -1)).cuda()) @ self.wo.T


@pytest.mark.parametrize("cache_type", ["bf16", "fp8"])
def test_prompts_then_single_tokens(lib, cache_type):
    import moe_block
    H, heads, kv, D, page, B = 256, 8, 2, 64, 16, 4
    half = moe_block.random_half(H, heads, kv, D, seed=4)
    scale = half.rotary["scale"]
    f = 2 * np.pi * half.rotary["freqs"].double().cpu().numpy() * 2.0 ** -64
    plain = Plain(lib, half, f, scale)
    fp8 = cache_type == "fp8"
    s = torch.full((kv,), 0.02, device="cuda") if fp8 else None
    cache = moe_block.PagedCache(40, page, kv, D, B, 10, torch.float8_e4m3fn if fp8 else torch.bfloat16, s, s)
    g = torch.Generator("cuda").manual_seed(6)
    cache.page_table.copy_(torch.randperm(40, generator=torch.Generator().manual_seed(7)).view(B, 10))
    lens = [37, 0, 5, 100]  # the second is a place that no sequence has
    cache.seq_lens.copy_(torch.tensor(lens))
    rows = sum(lens)
    x = torch.randn((rows + 6, H), device="cuda", generator=g).to(torch.bfloat16)  # six rows of padding
    indptr = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    q = half.prefill(x, cache, indptr)
    seq = np.repeat(np.arange(B), lens)
    at = np.concatenate([np.arange(n) for n in lens])
    want = plain.take(x[:rows], seq, at)
    assert _rel(_np(q)[:rows], want) <= 2 * 2.0 ** -8  # rounded to bf16 twice

    live = [0, 2, 3]
    out = torch.empty((B, H), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((B, H), device="cuda", generator=g).to(torch.bfloat16)
    keep = cache.seq_lens.clone()
    step = torch.tensor([1, 0, 1, 1], dtype=torch.int32, device="cuda")
    cache.seq_lens.add_(step)
    half(x, cache)  # warm, before the capture: the slots of the next tokens, which are written again below
    cache.seq_lens.copy_(keep)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.seq_lens.add_(step)
        out.copy_(half(x, cache))
    for i in range(30):
        x.copy_(torch.randn((B, H), device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert lib.device_error() == 0
        lens = [n + int(b in live) for b, n in enumerate(lens)]
        assert cache.seq_lens.tolist() == lens
        want = plain.decode(x[live], live, np.array([lens[b] - 1 for b in live]))
        # A rounding to bf16 is off by 2^-8 / sqrt(3) = 0.23 % rms at most, one to E4M3 by 2^-4 / sqrt(3) = 3.6 %.  Scores
        # have a spread of 1.9 (rotary scale 1.37 squared), so errors d of keys and queries move the weights by 1.9 d:
        # bf16 caches: two roundings each of q and k, 1.9 * 2 * 0.23 % = 0.9 %, with those of v and o 1 %.  The output's
        # own E4M3 codes then differ where a value lies within 1 % of a border, steps being 2^-3 at most: sqrt(0.01 *
        # 0.125) = 3.5 % rms.  E4M3 caches: 1.9 * 3.6 % = 6.9 %, with v's 7.8 %; codes that have nothing to do with one
        # another, sqrt(2) * 3.6 % = 5.1 %; together 9.3 %.
        assert _rel(_np(out)[live], want) <= (0.12 if fp8 else 0.045), i
        assert torch.all(out[1] == 0)  # an empty sequence attends to nothing


def test_whole_block_of_a_decode_step(lib):
    # the attention half into the expert half, twice, on a stream of its own: the same bits as call by call with a wait
    import moe_block
    H, heads, kv, D, page, B = 256, 8, 2, 64, 16, 5
    half = moe_block.random_half(H, heads, kv, D, seed=1)
    block = moe_block.random_block(H, 128, 16, 4, shared=192, n_group=4, topk_group=2, seed=3)
    g = torch.Generator("cuda").manual_seed(2)
    x, res = (torch.randn((B, H), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))

    def run(wait):
        cache = moe_block.PagedCache(20, page, kv, D, B, 4)
        cache.page_table.copy_(torch.arange(20).view(B, 4))
        y, r = x, res
        for _ in range(40):
            cache.seq_lens.add_(1)
            a = half(y, cache)
            if wait:
                torch.cuda.synchronize()
            r, y = block(a, r)
            if wait:
                torch.cuda.synchronize()
        return y, r, cache.k, cache.v

    want = run(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(False)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and lib.device_error() == 0
