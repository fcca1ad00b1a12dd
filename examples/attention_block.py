"""An attention block of POET-X projections: a few training steps on packed
documents, then one of the documents again token by token over a cache.

    python examples/attention_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from orthogonal_reparameterized_02_amd.attention import AttentionPlan, KVCache, POETXAttention  # noqa: E402


def main(n=512, heads=8, kv_heads=4, b=64, lengths=(100, 37, 119), steps=4, say=print):
    torch.manual_seed(0)
    block = POETXAttention(n, heads, kv_heads, b, k=4, cap=30.0, dropout=0.1, positions=1024,
                           scaling=("ramp", 4.0, 256, 1, 32))
    T = sum(lengths)
    x = torch.randn(T, n, device="cuda").bfloat16()
    target = torch.randn(T, n, device="cuda")
    cu = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(m, dtype=torch.int32) for m in lengths]).cuda()
    plan = AttentionPlan(cu, T)

    opt = torch.optim.SGD(block.parameters(), lr=2.0)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        loss = (block(x, plan, pos).float() - target).square().mean()
        loss.backward()
        opt.step()
        losses.append(loss.item())
        say(f"loss {losses[-1]:.5f}")

    block.eval()
    with torch.no_grad():
        packed = block(x, plan, pos)
        cache = KVCache(1, 256, kv_heads, block.D)
        half = lengths[0] // 2
        out = [block.prefill(x[:half], cache)]
        for t in range(half, lengths[0]):
            out.append(block.decode(x[t:t + 1], cache))
        served = torch.cat(out)
    far = ((served - packed[:lengths[0]]).float().norm() / packed[:lengths[0]].float().norm()).item()
    say(f"token by token against packed: relative difference {far:.2e}")
    return losses, far


if __name__ == "__main__":
    main()
