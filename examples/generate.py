"""Tokens from a small decoder with random NVFP4 weights: prompts of different
lengths are prefilled together, then every sequence decodes a token a step.

A layer is one attention block and one gated projection.  Its products run on
the quantized planes (``qmm``, ``qmm_glu``), keys and values go into a paged
8-bit cache (``kv_append``), ``paged_attention`` reads it and ``sample`` draws
the next token from given random numbers.

    python examples/generate.py [steps]
"""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import nvfp4_quantized_matmul_amd as nv  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, FEED, VOCAB, LAYERS, PAGE = 512, 8, 2, 64, 1024, 4096, 2, 64


class Decoder:
    def __init__(self, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def plane(rows, cols):
            w = torch.randn(rows, cols, generator=g) * cols ** -0.5
            return nv.quantize(w.to(torch.bfloat16).to(device))

        self.embedding = torch.randn(VOCAB, HIDDEN, generator=g).to(torch.bfloat16).to(device)
        self.layers = [{"qkv": plane((HEADS + 2 * KV_HEADS) * DIM, HIDDEN), "out": plane(HIDDEN, HEADS * DIM),
                        "gate": plane(FEED, HIDDEN), "up": plane(FEED, HIDDEN), "down": plane(HIDDEN, FEED)}
                       for _ in range(LAYERS)]
        self.head = plane(VOCAB, HIDDEN)
        self.inv_freq = (10000.0 ** (-torch.arange(0, DIM, 2).float() / DIM)).to(device)

    @staticmethod
    def norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def __call__(self, tokens, caches, table, lens, cu_q=None, max_q=None):
        """Hidden states of the new tokens, whose keys and values join the caches."""
        x = self.embedding[tokens.long()]
        for p, cache in zip(self.layers, caches):
            qkv = nv.qmm(self.norm(x), *p["qkv"])
            q, k, v = qkv.split([HEADS * DIM, KV_HEADS * DIM, KV_HEADS * DIM], 1)
            q = nv.kv_append(k.unflatten(1, (KV_HEADS, DIM)), v.unflatten(1, (KV_HEADS, DIM)), cache, table, lens,
                             q=q.unflatten(1, (HEADS, DIM)), cu_q=cu_q, max_q=max_q, inv_freq=self.inv_freq)
            o = nv.paged_attention(q, cache, table, lens, cu_q=cu_q, max_q=max_q)
            x = x + nv.qmm(o.flatten(1), *p["out"])
            h = nv.qmm_glu(self.norm(x), *p["gate"], *p["up"], act="silu")
            x = x + nv.qmm(h, *p["down"])
        return self.norm(x)


def generate(prompts, steps, temperature=0.8, top_k=50, top_p=0.95, seed=1, device="cuda"):
    """int32 [sequences, steps]: what follows each prompt (a list of token lists)."""
    model = Decoder(device)
    n = len(prompts)
    counts = [len(p) for p in prompts]
    width = -(-(max(counts) + steps) // PAGE)
    table = torch.randperm(n * width, generator=torch.Generator().manual_seed(seed)).int().view(n, width).to(device)
    caches = [nv.KVCache.empty(n * width, KV_HEADS, PAGE, DIM, device) for _ in range(LAYERS)]
    u = torch.rand(steps, n, generator=torch.Generator().manual_seed(seed)).to(device)
    row = lambda value, dtype: torch.full((n,), value, dtype=dtype, device=device)  # noqa: E731
    settings = {"temperature": row(temperature, torch.float32), "top_k": row(top_k, torch.int32),
                "top_p": row(top_p, torch.float32)}
    ends = torch.tensor(counts).cumsum(0)
    cu = torch.cat((torch.zeros(1, dtype=torch.int64), ends)).int().to(device)
    lens = torch.tensor(counts, dtype=torch.int32, device=device)
    x = model(torch.tensor(sum(prompts, []), device=device), caches, table, lens, cu_q=cu, max_q=max(counts))
    x = x[(ends - 1).to(device)]
    out = []
    for i in range(steps):
        out.append(nv.sample(nv.qmm(x, *model.head), u[i], **settings))
        if i + 1 < steps:
            lens = lens + 1
            x = model(out[-1], caches, table, lens)
    return torch.stack(out, 1)


if __name__ == "__main__":
    prompts = [[1, 2, 3], list(range(100)), [7] * 65]
    for tokens in generate(prompts, int(sys.argv[1]) if len(sys.argv) > 1 else 16).tolist():
        print(tokens)
