"""One adapted attention layer serving three requests, each with its own adapter: their prompts in one step, then a token of
each at a time, over a paged e4m3 (or bf16) cache. The layer's outputs of the stepwise run are compared with those of the
whole sequences taken in one step.

    python examples/attention_serving.py [bf16|e4m3]
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from rank_adapter_gemm_token_gb300 import layer  # noqa: E402

HIDDEN, HQ, HKV, HD, PAGE = 1024, 8, 2, 128, 16
QKV = (HQ + 2 * HKV) * HD
PROMPTS, NEW = (75, 130, 9), 12


def main(kind: str = "e4m3") -> float:
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *shape, std=1.0: (std * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    W_qkv, W_o = rand(QKV, HIDDEN, std=0.02), rand(HIDDEN, HQ * HD, std=0.02)
    q_norm, k_norm = 1 + rand(HD, std=0.1), 1 + rand(HD, std=0.1)
    pools = layer.AdapterPool(4, 16, HIDDEN, QKV), layer.AdapterPool(4, 16, HQ * HD, HIDDEN)
    for slot in range(3):
        for pool in pools:
            pool.load(slot, rand(16, pool.K, std=0.02), rand(pool.D, 16, std=0.02), 16, 32.0)
    rope = layer.Rope(HD, theta=500000.0)
    dtype = torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16
    lens = [p + NEW for p in PROMPTS]
    x = [rand(n, HIDDEN) for n in lens]                     # the layer's inputs of each request

    # pages as an allocator would hand them out: any free page, the three requests' mixed
    n_pages = sum(-(-n // PAGE) for n in lens)
    free = np.random.default_rng(0).permutation(n_pages).tolist()
    table = torch.full((3, max(-(-n // PAGE) for n in lens)), -1, dtype=torch.int32)
    for s, n in enumerate(lens):
        for i in range(-(-n // PAGE)):
            table[s, i] = free.pop()
    table = table.cuda()
    meta = layer.StepMeta(sum(lens), 1, 16)
    seq = layer.SeqMeta(3, sum(lens), table.shape[1], HQ, HKV, HD)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def step(cache, rows, lengths):
        """The layer on the next rows of each request; lengths: with them."""
        starts = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).tolist()
        slots = ints([s for s, r in enumerate(rows) for _ in range(len(r))])
        meta.build(slots, None, pools[0])
        seq.build(ints(starts), ints(lengths), table, starts[-1], cache, max_new=max(len(r) for r in rows))
        y = layer.attention_block(meta, seq, cache, torch.cat(rows), pools[0], W_qkv, pools[1], W_o, q_norm=q_norm,
                                  k_norm=k_norm, rope=rope)
        meta.status()
        seq.status()
        return y.split([len(r) for r in rows])

    cache = layer.KVCache(n_pages, PAGE, HKV, HD, dtype)
    parts = [[y] for y in step(cache, [r[:p] for r, p in zip(x, PROMPTS)], list(PROMPTS))]
    for i in range(NEW):
        for s, y in enumerate(step(cache, [r[p + i:p + i + 1] for r, p in zip(x, PROMPTS)], [p + i + 1 for p in PROMPTS])):
            parts[s].append(y)
    whole = step(layer.KVCache(n_pages, PAGE, HKV, HD, dtype), x, lens)
    worst = max(float((torch.cat(a) - b).norm() / b.norm()) for a, b in zip(parts, whole))
    print(f"{kind}: prompts {PROMPTS} and {NEW} tokens each, one at a time; largest relative difference from one step: {worst:.1e}")
    for pool in pools:
        pool.close()
    return worst


if __name__ == "__main__":
    main(*sys.argv[1:2])
