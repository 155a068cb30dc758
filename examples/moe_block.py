"""One mixture-of-experts block of a transformer, from the attention's output to the next block's input.

    residual, x = norm before the block (fused with the residual of the attention's output)
    logits      = x gate^T                        fp32
    ids, w      = grouped sigmoid routing with a balance bias
    routed      = W4AFP8 experts of the chosen ids, weighted
    shared      = SiLU(x up_gate^T) * (x up^T)    shared expert, bf16
    f           = shared down^T + routed
    residual, y = norm after the block, into the residual stream, and the next block's norm

python examples/moe_block.py [tokens]  runs a block with random weights and prints its time per call.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import w4afp8_mixture_experts_gb300 as m  # noqa: E402


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


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 64
    H, I, E, k = 7168, 2048, 256, 8
    block = random_block(H, I, E, k, shared=I, n_group=8, topk_group=4)
    attn, residual = (torch.randn((tokens, H), device="cuda").to(torch.bfloat16) for _ in range(2))
    for _ in range(3):
        block(attn, residual)
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    torch.cuda.synchronize()
    start.record()
    for _ in range(20):
        res, y = block(attn, residual)
    stop.record()
    torch.cuda.synchronize()
    if m.device_error() or not torch.isfinite(y.float()).all():
        raise SystemExit("the block failed")
    print(f"one block, {tokens} tokens, H={H} I={I} E={E} k={k}: {start.elapsed_time(stop) / 20 * 1e3:.1f} us a call")


if __name__ == "__main__":
    main()
