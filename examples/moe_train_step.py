"""Training steps of one mixture-of-experts layer and a vocabulary projection,
from the router to the clipped update, on synthetic data:

    python examples/moe_train_step.py [--tokens 2048] [--steps 8] [--adamw]

Forward: router logits -> moe_topk -> moe_sort -> moe_dispatch_mx (token rows
to their experts, MX E4M3) -> the expert up-projection with SwiGLU and MX
quantization in its epilogue -> the down-projection -> moe_combine -> residual
-> linear_cross_entropy against the vocabulary.
Backward: linear_cross_entropy_backward -> moe_combine_backward ->
moe_topk_backward, then GradientSet.clip and a plain gradient step, or
GradientSet.norm and AdamW with 8-bit moments, which clips on the way.  The
experts are frozen MX E4M3 weights; the router and the projection learn.
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import mxfp4_precision_numerics_amd as mxq  # noqa: E402


class Layer:
    """The layer's weights, and every buffer of a step of `tokens` tokens."""

    def __init__(self, tokens, hidden, inter, experts, topk, vocab, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device=device)
        empty = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=device)
        bf16, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
        T, C, I, E, k, V = tokens, hidden, inter, experts, topk, vocab
        self.shape = T, C, I, E, k, V
        # experts: gate and up rows, then the down-projection, as MX E4M3 codes and scales
        self.up = self._quantized(rn(E * 2 * I, C) * C ** -0.5)
        self.down = self._quantized(rn(E * C, I) * I ** -0.5)
        self.router = rn(E, C) * C ** -0.5
        self.proj = (rn(V, C) * C ** -0.5).to(bf16)
        self.router_master, self.proj_master = self.router.clone(), self.proj.float()
        # the step's buffers
        R = T * k
        self.ids, self.pos, self.src = empty(T, k, dtype=i32), empty(T, k, dtype=i32), empty(R, dtype=i32)
        self.weights, self.off = empty(T, k), empty(E + 1, dtype=torch.int64)
        self.sort_ws = empty(max(16, mxq.moe_sort_workspace(T, k, E)), dtype=u8)
        self.q, self.s = empty(R, C, dtype=u8), empty(R, C // 32, dtype=u8)
        self.hq, self.hs = empty(R, I, dtype=u8), empty(R, I // 32, dtype=u8)
        self.rows, self.y = empty(R, C, dtype=bf16), empty(T, C, dtype=bf16)
        self.loss, self.lse, self.dloss = empty(T), empty(T), empty(T)
        self.loss_ws = empty(mxq.linear_cross_entropy_workspace(T, C, V, backward=True), dtype=u8)
        self.dx, self.dproj = empty(T, C, dtype=bf16), empty(V, C, dtype=bf16)
        self.dweights, self.dlogits, self.drouter = empty(T, k), empty(T, E), empty(E, C)
        self.norm = empty(1)
        self.grads = mxq.GradientSet([self.drouter, self.dproj])  # clipped in place
        masters = [self.router_master, self.proj_master]
        codes = lambda: [torch.zeros(p.numel(), dtype=u8, device=device) for p in masters]
        scales = lambda: [torch.zeros(-(-p.numel() // mxq.AdamW.BLOCK), device=device) for p in masters]
        self.adamw = mxq.AdamW(masters, [self.drouter, self.dproj], codes(), codes(), scales(), scales(),
                               copies=[None, self.proj], decay=[False, True])

    @staticmethod
    def _quantized(w):
        q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
        s = torch.empty(w.shape[0], w.shape[1] // 32, dtype=torch.uint8, device=w.device)
        mxq.quantize_mx(w.to(torch.bfloat16), mxq.E4M3, q, s)
        return q, s

    def forward(self, h, targets):
        """Per-token losses of hidden states `h` [tokens, hidden] (bfloat16);
        a target of -100 is ignored."""
        T, C, I, E, k, V = self.shape
        R, blk = T * k, mxq.SCALE_BLK32
        self.logits = torch.mm(h.float(), self.router.t())
        mxq.moe_topk(self.logits, self.ids, self.weights, renormalize=True)
        mxq.moe_sort(self.ids, E, self.off, self.src, self.pos, self.sort_ws)
        mxq.moe_dispatch_mx(h, self.pos, mxq.E4M3, self.q, self.s)
        mxq.grouped_gemm_swiglu_quantize_mx(self.q, mxq.E4M3, self.s, blk, self.up[0], mxq.E4M3, self.up[1], blk,
                                            self.off, E, R, I, C, mxq.E4M3, self.hq, self.hs)
        mxq.grouped_scaled_gemm(self.hq, mxq.E4M3, self.hs, blk, self.down[0], mxq.E4M3, self.down[1], blk, self.off, E,
                                R, C, I, self.rows, out=mxq.OUT_BF16)
        mxq.moe_combine(self.rows, self.pos, self.y, weights=self.weights)
        self.x = h + self.y
        mxq.linear_cross_entropy(self.x, self.proj, targets, self.loss, self.lse, self.loss_ws)
        return self.loss

    def backward(self, h, targets):
        """Gradients of the mean loss over the tokens that count, for the
        router (`drouter`) and the projection (`dproj`)."""
        valid = (targets >= 0).float()
        torch.div(valid, valid.sum().clamp(min=1), out=self.dloss)
        mxq.linear_cross_entropy_backward(self.x, self.proj, targets, self.lse, self.dloss, self.dx, self.dproj,
                                          self.loss_ws)
        mxq.moe_combine_backward(self.dx, self.pos, rows=self.rows, dweights=self.dweights)
        mxq.moe_topk_backward(self.logits, self.ids, self.dweights, self.dlogits, renormalize=True)
        torch.mm(self.dlogits.t(), h.float(), out=self.drouter)

    def update(self, rate, max_norm):
        """Clip by the global norm, then one plain gradient step."""
        self.grads.clip(max_norm, self.norm)
        self.router_master.sub_(self.drouter, alpha=rate)
        self.proj_master.sub_(self.dproj.float(), alpha=rate)
        self.router.copy_(self.router_master)
        self.proj.copy_(self.proj_master)

    def update_adamw(self, step, rate, max_norm):
        """Step number `step` of AdamW, its gradients clipped by the global norm."""
        self.grads.norm(self.norm)
        self.adamw.step(step, rate, betas=(0.9, 0.95), norm=self.norm, max_norm=max_norm, seed=1)
        self.router.copy_(self.router_master)


def train(tokens=2048, hidden=1024, inter=512, experts=16, topk=4, vocab=32000, steps=8, rate=4.0, max_norm=1.0,
          seed=0, adamw=False):
    """Mean losses of `steps` steps on one synthetic batch."""
    layer = Layer(tokens, hidden, inter, experts, topk, vocab, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    h = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    targets = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    targets[torch.rand(tokens, generator=g, device="cuda") < 0.1] = -100
    count = (targets >= 0).sum()
    losses = []
    for n in range(steps):
        losses.append(layer.forward(h, targets).sum() / count)
        layer.backward(h, targets)
        if adamw:
            layer.update_adamw(n + 1, rate, max_norm)
        else:
            layer.update(rate, max_norm)
    return [float(x) for x in losses], layer


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    a.add_argument("--tokens", type=int, default=2048)
    a.add_argument("--steps", type=int, default=8)
    a.add_argument("--adamw", action="store_true")
    args = a.parse_args()
    for n, x in enumerate(train(tokens=args.tokens, steps=args.steps, rate=3e-3 if args.adamw else 4.0, adamw=args.adamw)[0]):
        print(f"step {n}: loss {x:.4f}", flush=True)
