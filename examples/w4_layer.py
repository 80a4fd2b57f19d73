"""A 4-bit MoE layer served from a slot cache, its router balanced, and a 4-bit output head on top.

    python examples/w4_layer.py [--tokens 16] [--steps 40]

1. The experts and the output head are quantised to 4-bit codes with group scales (once, on the device).
2. The router is tuned for balance over packed sequences with padding: the balance loss and its gradient.
3. Tokens are decoded greedily: the layer keeps half of its experts in slots (missing ones are gathered from pinned
   host memory, packed as they are), and the head turns its output into the next token.

Weights are random, so the text means nothing; the loads, the losses and the rates are real.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import expert_slot_cache_gb300 as M  # noqa: E402

H, I, E, K, GROUP, VOCAB = 512, 256, 32, 4, 64, 4000


def imbalance(counts):
    load = counts.sum(0).float()
    return float(load.max() / load.mean())


def balance_router(wr, tokens, seq_start, mask, steps, rate=1e-3):
    """Gradient steps on the balance loss alone; returns the router and (loss, max / mean load) before and after."""
    wr = wr.clone().requires_grad_()
    seen = []
    for step in range(steps + 1):
        logits = tokens.float() @ wr
        ids = logits.topk(K, dim=1).indices.to(torch.int32)
        loss, counts = M.BalanceLoss.apply(logits, ids, 1.0, seq_start, mask)
        seen.append((loss.item(), imbalance(counts)))
        if step < steps:
            (g,) = torch.autograd.grad(loss, wr)
            with torch.no_grad():
                wr -= rate * g
    return wr.detach(), seen[0], seen[-1]


def main(argv=None):
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=16)
    p.add_argument("--steps", type=int, default=40)
    a = p.parse_args(argv)
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    slabs = (normal(E, 3 * H * I) * H ** -0.5).to(torch.bfloat16)
    head = (normal(H, VOCAB) * H ** -0.5).to(torch.bfloat16)
    embed = normal(VOCAB, H).to(torch.bfloat16)
    wr = normal(H, E) * H ** -0.5

    packed = M.w4_quantize_slabs(slabs, H, I, GROUP)
    op_head = M.W4Linear(M.w4_quantize(head, GROUP), H, VOCAB, GROUP, out_dtype=torch.float32)
    print(f"experts {slabs.nbytes / 2**20:.1f} -> {packed.nbytes / 2**20:.1f} MiB")

    # four packed sequences, the last tokens of each are padding; tokens that share a direction overload experts
    seq_start = torch.tensor([0, 700, 1000, 1900, 2048], dtype=torch.int32, device=dev)
    mask = torch.ones(2048, dtype=torch.bool, device=dev)
    for end in seq_start[1:].tolist():
        mask[end - 20:end] = False
    tokens = (normal(2048, H) + 2 * normal(1, H)).to(torch.bfloat16)
    wr, before, after = balance_router(wr, tokens, seq_start, mask, a.steps)
    print(f"balance loss {before[0]:.3f} -> {after[0]:.3f}, largest / mean load {before[1]:.2f} -> {after[1]:.2f}")

    slots = E // 2
    resident = torch.arange(slots, dtype=torch.int32).numpy()
    host = torch.empty(packed.shape, dtype=torch.uint8, pin_memory=True)
    host.copy_(packed)
    router = wr.to(torch.bfloat16).contiguous()  # the layer's router is bf16
    layer = M.SlotCachedMoELayer(router, packed[:slots].clone(), K, I, M.MODE_GATHER, M.POLICY_LRU,
                                 host_slabs=host, state=M.CacheState.from_slots(resident, E), max_tokens=1, quant=2,
                                 quant_group=GROUP)
    token, text = torch.zeros(1, dtype=torch.int64, device=dev), []
    op_head.forward(embed[token] + layer.forward(embed[token])["out"]).argmax(dim=1)  # the first call sets the kernels up
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(a.tokens):
        x = embed[token]
        y = layer.forward(x)["out"]
        token = op_head.forward(x + y).argmax(dim=1)
        text.append(token)
    text = torch.cat(text).tolist()
    misses = int(layer.stats[0])
    print(f"{a.tokens} tokens in {(time.perf_counter() - t0) * 1e3:.2f} ms; {misses} of {(a.tokens + 1) * K} experts gathered")
    assert int(layer.dev_status.item()) == 0 and int(op_head.dev_status.item()) == 0
    return dict(before=before, after=after, text=text, packed=packed, slabs=slabs, head=head, op_head=op_head, layer=layer,
                router=router, embed=embed)


if __name__ == "__main__":
    main()
