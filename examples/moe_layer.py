"""One mixture-of-experts layer with LoRA adapters, from router logits to the layer's output.

    python examples/moe_layer.py [--tokens 256] [--experts 256] [--local 32] [--topk 8] [--hidden 7168]
                                 [--inter 2048] [--loras 4] [--rank 64] [--weights bf16|mx4]

Every step of the layer is a call of the library, in stream order:

    moe_route          topk experts of every token, their weights, the pairs' product slots
    TokenMeta.prepare  the pairs grouped by expert (products) ...
    moe_pair_slots     ... and, through their (adapter, expert) slots, TokenMeta.prepare again (LoRA)
    moe_product        w13 of the local experts: token rows -> [gate | up] rows of the pairs
    apply              the adapters' w13 delta, added to those rows
    moe_act            silu(gate) * up
    moe_product        w2
    apply              the adapters' w2 delta
    moe_combine        the weighted sum over each token's choices

With ``--weights mx4`` the experts' weights and the products' inputs are in the microscaled 4-bit format
(mx4_quantize); the adapters work on the bf16 rows either way. Random weights and inputs; prints the time of a
step replayed from a CUDA graph.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import rank_adapter_gb300 as ra  # noqa: E402


class MoELayer:
    """Weights, adapters, metadata and row buffers of one layer for up to ``max_tokens`` tokens."""

    def __init__(self, w13, w2, num_experts, topk, max_tokens, expert_map=None, num_loras=0, rank=16, mx4=False):
        local, two_inter, hidden = w13.shape
        self.E, self.L, self.topk, self.hidden, self.inter = num_experts, local, topk, hidden, two_inter // 2
        self.expert_map, self.num_loras, self.mx4 = expert_map, num_loras, mx4
        self.e13, self.e2 = self._experts(w13, topk), self._experts(w2, 1)
        P = max_tokens * topk
        self.meta = ra.TokenMeta(P, local + 1)
        bf16 = dict(dtype=torch.bfloat16, device="cuda")
        self.ids = torch.empty(max_tokens, topk, dtype=torch.int32, device="cuda")
        self.w = torch.empty(max_tokens, topk, dtype=torch.float32, device="cuda")
        self.y13, self.h = torch.empty(P, two_inter, **bf16), torch.empty(P, self.inter, **bf16)
        self.y2 = torch.empty(P, hidden, **bf16)
        if mx4:
            self.xq, self.hq = ra.mx4_buffers(max_tokens, hidden), ra.mx4_buffers(P, self.inter)
        if num_loras:
            slots = 1 + num_loras * local
            self.lmeta = ra.TokenMeta(P, slots)
            self.t13 = ra.SlotTable(hidden, [self.inter, self.inter], slots, rank, x_row_div=topk)
            self.t2 = ra.SlotTable(self.inter, [hidden], slots, rank)
            tables = (self.t13, self.t2)
            self.ws = ra.workspace(max(tables, key=lambda t: ra.lora_workspace_bytes(t.desc, P)), P)

    def _experts(self, w, x_row_div):
        if not self.mx4:
            return ra.ExpertWeights(w, x_row_div=x_row_div)
        codes, scales = ra.mx4_quantize(w.reshape(-1, w.shape[2]))
        return ra.ExpertWeights(codes.view(*w.shape[:2], -1), scales.view(*w.shape[:2], -1), x_row_div=x_row_div)

    def set_adapter(self, adapter, expert, rank, scale, a13, b13, a2, b2):
        """Adapter 1.. of local expert 0..: a13 [hidden, rank] twice (gate, up), b13 [rank, inter] twice, a2, b2."""
        slot = 1 + (adapter - 1) * self.L + expert
        self.t13.set_slot(slot, rank, scale, a13, b13)
        self.t2.set_slot(slot, rank, scale, [a2], [b2])

    def __call__(self, x, logits, out, token_slot=None):
        """out [T, hidden] = the layer's output for x [T, hidden] and router logits [T, E]; ``token_slot``: the
        tokens' adapters (0: none)."""
        T, K = x.shape[0], self.topk
        P, pair = T * K, self.meta.token_slot[:T * K]
        ids, w = self.ids[:T], self.w[:T]
        y13, h, y2 = self.y13[:P], self.h[:P], self.y2[:P]
        ra.moe_route(logits, K, expert_map=self.expert_map, local_experts=self.L, topk_ids=ids, topk_w=w, pair_slot=pair)
        self.meta.set_num_tokens(P)
        self.meta.prepare()
        lora = self.num_loras and token_slot is not None
        if lora:
            self.lmeta.set_num_tokens(P)
            ra.moe_pair_slots(token_slot, ids, self.num_loras, self.E, self.L, self.expert_map,
                              pair_slot=self.lmeta.token_slot[:P])
            self.lmeta.prepare()
        if self.mx4:
            ra.mx4_quantize(x, *self.xq)
            ra.moe_product(self.e13, self.meta, self.xq[0], y13, x_scale=self.xq[1])
        else:
            ra.moe_product(self.e13, self.meta, x, y13)
        if lora:
            ra.apply(self.t13, self.lmeta, x, y13, ws=self.ws)
        if self.mx4 and not lora:
            ra.moe_act_mx4(y13, *self.hq, pair_slot=pair)
        else:
            ra.moe_act(y13, h, pair_slot=pair)
        if self.mx4:
            if lora:
                ra.mx4_quantize(h, *self.hq)
            ra.moe_product(self.e2, self.meta, self.hq[0], y2, x_scale=self.hq[1])
        else:
            ra.moe_product(self.e2, self.meta, h, y2)
        if lora:
            ra.apply(self.t2, self.lmeta, h, y2, ws=self.ws)
        return ra.moe_combine(y2, w, out, pair_slot=pair)


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in dict(tokens=256, experts=256, local=32, topk=8, hidden=7168, inter=2048, loras=4, rank=64).items():
        p.add_argument(f"--{name}", type=int, default=value)
    p.add_argument("--weights", choices=["bf16", "mx4"], default="bf16")
    a = p.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    emap = None
    if a.local < a.experts:
        emap = torch.full((a.experts,), -1, dtype=torch.int32, device="cuda")
        emap[:a.local] = torch.arange(a.local, dtype=torch.int32, device="cuda")
    layer = MoELayer(randn(a.local, 2 * a.inter, a.hidden) * a.hidden ** -0.5, randn(a.local, a.hidden, a.inter) * a.inter ** -0.5,
                     a.experts, a.topk, a.tokens, emap, a.loras, a.rank, a.weights == "mx4")
    for s in range(1, a.loras + 1):
        for e in range(a.local):
            layer.set_adapter(s, e, a.rank, 1.0, [randn(a.hidden, a.rank) / 64 for _ in "gu"],
                              [randn(a.rank, a.inter) / 16 for _ in "gu"], randn(a.inter, a.rank) / 64, randn(a.rank, a.hidden) / 16)
    x, logits = randn(a.tokens, a.hidden), torch.randn(a.tokens, a.experts, device="cuda", generator=g)
    slot = torch.randint(0, a.loras + 1, (a.tokens,), dtype=torch.int32, device="cuda", generator=g)
    out = torch.empty_like(x)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(3):
            layer(x, logits, out, slot)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        layer(x, logits, out, slot)
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    t0.record()
    for _ in range(20):
        graph.replay()
    t1.record()
    torch.cuda.synchronize()
    ra.check(ra.lora_query_status(layer.meta.c)[0], "moe layer")
    print(f"{a.tokens} tokens, {a.local} of {a.experts} experts, top {a.topk}, {a.hidden} x {a.inter}, {a.weights} weights, "
          f"{a.loras} adapters: {t0.elapsed_time(t1) / 20 * 1e3:.1f} us a step, |out| {out.float().norm():.1f}")


if __name__ == "__main__":
    main()
