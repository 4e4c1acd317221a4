"""Tokens from a small decoder with random NVFP4 weights: prompts of different
lengths are prefilled together, then every sequence decodes a token a step.

A layer is one attention block and one gated projection.  Its products run on
the quantized planes (``qmm``, ``qmm_glu``), keys and values go into a paged
8-bit cache (``kv_append``, with norms of the heads if wanted),
``paged_attention`` reads it and ``sample`` draws the next token from given
random numbers.

The layers' caches share a pool of pages: ``kv_reserve`` finds pages for new
tokens, ``kv_fork`` makes several samples of each prompt that share its pages,
and with a window and sinks ``kv_free`` gives back what no token sees any more,
so that a sequence never holds more than these.

    python examples/generate.py [steps]
"""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import nvfp4_quantized_matmul_amd as nv  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, FEED, VOCAB, LAYERS, PAGE = 512, 8, 2, 64, 1024, 4096, 2, 64


class Decoder:
    def __init__(self, device="cuda", seed=0, norm=False, window=0, sinks=0):
        g = torch.Generator().manual_seed(seed)
        self.window, self.sinks = window, sinks

        def plane(rows, cols):
            w = torch.randn(rows, cols, generator=g) * cols ** -0.5
            return nv.quantize(w.to(torch.bfloat16).to(device))

        self.embedding = torch.randn(VOCAB, HIDDEN, generator=g).to(torch.bfloat16).to(device)
        self.layers = [{"qkv": plane((HEADS + 2 * KV_HEADS) * DIM, HIDDEN), "out": plane(HIDDEN, HEADS * DIM),
                        "gate": plane(FEED, HIDDEN), "up": plane(FEED, HIDDEN), "down": plane(HIDDEN, FEED)}
                       for _ in range(LAYERS)]
        self.head = plane(VOCAB, HIDDEN)
        self.norms = {}
        if norm:
            self.norms = {side: (1.0 + 0.2 * torch.randn(DIM, generator=g)).to(device) for side in ("q_norm", "k_norm")}
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
                             q=q.unflatten(1, (HEADS, DIM)), cu_q=cu_q, max_q=max_q, inv_freq=self.inv_freq,
                             **self.norms)
            o = nv.paged_attention(q, cache, table, lens, cu_q=cu_q, max_q=max_q, window=self.window, sinks=self.sinks)
            x = x + nv.qmm(o.flatten(1), *p["out"])
            h = nv.qmm_glu(self.norm(x), *p["gate"], *p["up"], act="silu")
            x = x + nv.qmm(h, *p["down"])
        return self.norm(x)


def generate(prompts, steps, temperature=0.8, top_k=50, top_p=0.95, seed=1, device="cuda", samples=1, window=0, sinks=0,
             norm=False, pages=None):
    """int32 [sequences, steps]: what follows each prompt (a list of token lists), `samples` times one after the other.

    pages: of the pool, by default as many as the whole sequences would fill."""
    model = Decoder(device, norm=norm, window=window, sinks=sinks)
    counts = [len(p) for p in prompts]
    n = len(prompts) * samples
    width = -(-(max(counts) + steps) // PAGE)
    pages = pages or n * width
    caches = [nv.KVCache.empty(pages, KV_HEADS, PAGE, DIM, device) for _ in range(LAYERS)]
    table = torch.full((len(prompts), width), -1, dtype=torch.int32, device=device)
    refs = torch.zeros(pages, dtype=torch.int32, device=device)
    u = torch.rand(steps, n, generator=torch.Generator().manual_seed(seed)).to(device)
    row = lambda value, dtype: torch.full((n,), value, dtype=dtype, device=device)  # noqa: E731
    settings = {"temperature": row(temperature, torch.float32), "top_k": row(top_k, torch.int32),
                "top_p": row(top_p, torch.float32)}
    ends = torch.tensor(counts).cumsum(0)
    cu = torch.cat((torch.zeros(1, dtype=torch.int64), ends)).int().to(device)
    lens = torch.tensor(counts, dtype=torch.int32, device=device)
    small = f"the pool of {pages} pages was too small"
    if nv.kv_reserve(caches, table, lens, refs, cu_q=cu, tokens=sum(counts)).any():
        raise RuntimeError(small)
    x = model(torch.tensor(sum(prompts, []), device=device), caches, table, lens, cu_q=cu, max_q=max(counts))
    x = x[(ends - 1).to(device)]
    if samples > 1:
        parent = torch.arange(len(prompts), dtype=torch.int32, device=device).repeat_interleave(samples)
        table, lens = nv.kv_fork(table, lens, refs, parent)
        x = x[parent.long()]
    out, waited = [], torch.zeros(n, dtype=torch.bool, device=device)
    for i in range(steps):
        out.append(nv.sample(nv.qmm(x, *model.head), u[i], **settings))
        if i + 1 < steps:
            lens = lens + 1
            if window > 0:
                nv.kv_free(table, lens, refs, PAGE, keep=window, sinks=sinks)
            # who got no pages waits: with length 0 its token goes nowhere, and the step comes again
            waits = nv.kv_reserve(caches, table, lens, refs) > 0
            x = torch.where(waits[:, None], x, model(out[-1], caches, table, torch.where(waits, 0, lens)))
            lens, waited = lens - waits.int(), waited | waits
    # read once, at the end: who waited has fewer tokens than steps
    if waited.any():
        raise RuntimeError(small)
    return torch.stack(out, 1)


if __name__ == "__main__":
    prompts = [[1, 2, 3], list(range(100)), [7] * 65]
    for tokens in generate(prompts, int(sys.argv[1]) if len(sys.argv) > 1 else 16).tolist():
        print(tokens)
    print("two samples each, 64 tokens and 4 first ones seen, normed heads:")
    for tokens in generate(prompts, 16, samples=2, window=64, sinks=4, norm=True).tolist():
        print(tokens)
