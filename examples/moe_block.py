"""One mixture-of-experts block of a transformer: its attention half for single new tokens, and from the attention's
output to the next block's input.

    q, k, v     = x Wqkv^T                        FP8 (E4M3, scales per token and 128, per 128 x 128 weights)
    cache, q    = k and v into the paged cache, k and q rotated by position
    attn        = attention of each new token over its sequence's pages, then Wo^T in FP8

    residual, x = norm before the block (fused with the residual of the attention's output)
    logits      = x gate^T                        fp32
    ids, w      = grouped sigmoid routing with a balance bias
    routed      = W4AFP8 experts of the chosen ids, weighted
    shared      = SiLU(x up_gate^T) * (x up^T)    shared expert, bf16
    f           = shared down^T + routed
    residual, y = norm after the block, into the residual stream, and the next block's norm

python examples/moe_block.py [tokens [context]]  runs a block with random weights and prints its time per call, and its
attention half's where the tokens are up to 512 new ones.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import w4afp8_mixture_experts_gb300 as m  # noqa: E402


class PagedCache:
    """Keys and values of B sequences in pages; `seq_lens` counts the tokens of each (0: no sequence)."""

    def __init__(self, pages, page_size, heads, D, B, table_pages, dtype=torch.bfloat16, k_scale=None, v_scale=None,
                 device="cuda"):
        self.k, self.v = (torch.zeros((pages, page_size, heads, D), device=device).to(dtype) for _ in range(2))
        self.page_table = torch.full((B, table_pages), -1, dtype=torch.int32, device=device)
        self.seq_lens = torch.zeros(B, dtype=torch.int32, device=device)
        self.scales = dict(k_scale=k_scale, v_scale=v_scale)


class AttentionHalf:
    """The attention half of a block.  wqkv, wo: E4M3 codes [N, K] and their scales [ceil(N/128), K/128]; freqs from
    rotary_frequencies for the first 2 len(freqs) elements of a head."""

    def __init__(self, wqkv, wqkv_s, wo, wo_s, heads, kv_heads, freqs, rotary_scale=1.0, interleaved=False):
        self.wqkv, self.wqkv_s, self.wo, self.wo_s = wqkv, wqkv_s, wo, wo_s
        self.heads, self.kv_heads = heads, kv_heads
        self.rotary = dict(freqs=freqs, scale=rotary_scale, interleaved=interleaved)

    @staticmethod
    def project(x, w, w_s):
        codes, scales, _ = m.fp8_quant_per_token_group(x)
        return m.fp8_block_linear(codes, scales, w, w_s)

    def project_qkv(self, x):
        """x bf16 [T, H] -> q [T, heads, D], k, v [T, kv_heads, D], parts of one tensor."""
        qkv = self.project(x, self.wqkv, self.wqkv_s).view(x.shape[0], self.heads + 2 * self.kv_heads, -1)
        return qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)

    def prefill(self, x, cache, indptr):
        """Keys and values of the prompts x bf16 [T, H], rows indptr[b] ... indptr[b + 1] the last tokens of sequence b, into
        the cache; returns the rotated queries (attention of prompts is not among the operators; rows of padding come back as
        they are)."""
        q, k, v = self.project_qkv(x)
        return m.paged_kv_append(k, v, cache.k, cache.v, cache.page_table, cache.seq_lens, indptr, q=q, q_out=q,
                                 **self.rotary, **cache.scales)

    def __call__(self, x, cache):
        """x bf16 [B, H], one new token of each sequence, counted in cache.seq_lens -> bf16 [B, H]."""
        q, k, v = self.project_qkv(x)
        q = m.paged_kv_append(k, v, cache.k, cache.v, cache.page_table, cache.seq_lens, q=q, **self.rotary, **cache.scales)
        o = m.paged_attention_decode(q, cache.k, cache.v, cache.page_table, cache.seq_lens, **cache.scales)
        return self.project(o.flatten(1), self.wo, self.wo_s)


class MoeBlock:
    """Weights and buffers of one block.  `norms`: the fp32 weights of the norm before the block, the norm behind it
    and the next block's norm (None for the middle one: the block's output joins the residual as it is)."""

    def __init__(self, gate, gate_bias, w13, w13_s, w2, w2_s, shared_up, shared_down, norms, k, n_group=1, topk_group=1,
                 scale=1.0, eps=1e-6):
        self.gate, self.gate_bias = gate, gate_bias
        self.experts = (w13, w13_s, w2, w2_s)
        self.shared_up, self.shared_down = shared_up, shared_down
        self.norm_in, self.norm_out, self.norm_next = norms
        self.k, self.n_group, self.topk_group, self.scale, self.eps = k, n_group, topk_group, scale, eps
        self.ws = None

    def route(self, x):
        logits = m.dense_linear(x, self.gate, out_dtype=torch.float32)
        return m.moe_route_grouped_topk(logits, self.k, bias=self.gate_bias, score="sigmoid", n_group=self.n_group,
                                        topk_group=self.topk_group, group_top=2 if self.n_group > 1 else 1,
                                        scale=self.scale)

    def __call__(self, attn, residual):
        """attn, residual bf16 [T, H] -> (residual behind the block, input of the next block)."""
        T, H = attn.shape
        w13 = self.experts[0]
        need = m.moe_workspace_layout(T, H, w13.shape[1] // 2, w13.shape[0], self.k).total
        if self.ws is None or self.ws.numel() < need:
            self.ws = torch.empty(need, dtype=torch.uint8, device=attn.device)
        residual, x = m.block_norm(attn, residual, post="none", pre="rms", w_pre=self.norm_in, eps=self.eps)
        ids, w = self.route(x)
        routed = m.w4a8_moe_forward_routed(x, ids, w, *self.experts, ws=self.ws)
        shared = m.dense_linear(x, self.shared_up, act="silu", gated=True)
        f = m.dense_linear(shared, self.shared_down, residual=routed, out=routed)
        return m.block_norm(f, residual, post="none" if self.norm_out is None else "rms", w_post=self.norm_out,
                            pre="rms", w_pre=self.norm_next, eps=self.eps, h=residual)


def random_block(H, I, E, k, shared, n_group, topk_group, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=device) * scale

    def int4(*shape):
        return torch.randint(0, 256, shape, dtype=torch.uint8, generator=g, device=device)

    w13 = m.w4a8_prepack_weights(int4(E, 2 * I, H // 2))
    w2 = m.w4a8_prepack_weights(int4(E, H, I // 2))
    w13_s = torch.rand((E, H // 128, 2 * I), generator=g, device=device) * (0.4 / H ** 0.5)
    w2_s = torch.rand((E, I // 128, H), generator=g, device=device) * (0.4 / I ** 0.5)
    bf = torch.bfloat16
    return MoeBlock(randn(E, H, scale=H ** -0.5).to(bf), randn(E, scale=0.05), w13, w13_s, w2, w2_s,
                    randn(2 * shared, H, scale=H ** -0.5).to(bf), randn(H, shared, scale=shared ** -0.5).to(bf),
                    [1 + 0.1 * randn(H) for _ in range(3)], k, n_group, topk_group, scale=2.5)


def random_half(H, heads, kv_heads, D, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)

    def weights(N, K):  # about K^-0.5 in size
        codes = (torch.randn((N, K), generator=g, device=device) * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
        return codes, (0.75 + 0.5 * torch.rand((-(-N // 128), K // 128), generator=g, device=device)) / (64 * K ** 0.5)

    return AttentionHalf(*weights((heads + 2 * kv_heads) * D, H), *weights(H, heads * D), heads, kv_heads,
                         m.rotary_frequencies(D, scaling="yarn", factor=40.0, device=device), m.rotary_yarn_scale(40.0))


def timed(call, turns=20):
    for _ in range(3):
        call()
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    for _ in range(turns):
        got = call()
    stop.record()
    torch.cuda.synchronize()
    if m.device_error() or not all(torch.isfinite(t.float()).all() for t in (got if isinstance(got, tuple) else (got,))):
        raise SystemExit("the block failed")
    return start.elapsed_time(stop) / turns * 1e3


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 64
    context = int(sys.argv[2]) if len(sys.argv) > 2 else 4096
    H, I, E, k, heads, kv_heads, D = 7168, 2048, 256, 8, 64, 8, 128
    block = random_block(H, I, E, k, shared=I, n_group=8, topk_group=4)
    attn, residual = (torch.randn((tokens, H), device="cuda").to(torch.bfloat16) for _ in range(2))
    us = timed(lambda: block(attn, residual))
    print(f"one block, {tokens} tokens, H={H} I={I} E={E} k={k}: {us:.1f} us a call")
    if tokens > 512:
        return
    half = random_half(H, heads, kv_heads, D)
    pages = -(-context // 64)
    cache = PagedCache(tokens * pages, 64, kv_heads, D, tokens, pages)
    cache.page_table.copy_(torch.randperm(tokens * pages, device="cuda").view(tokens, pages))
    cache.seq_lens.fill_(context)
    us = timed(lambda: half(attn, cache))
    print(f"its attention half, {tokens} new tokens over {context} each, {heads} heads of {D} over {kv_heads}: {us:.1f} us a call")


if __name__ == "__main__":
    main()
