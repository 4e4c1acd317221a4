"""The rotation's roundings: to 32 bits, then once to the queries' type."""

import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV
from test_serving_gpu import BF16, F16, rotate

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,off", [(600, 0), (2400, 0), (600, 1)])
def test_rotated_queries_are_rounded_twice(dtype, interleaved, tokens, off):
    """Bit for bit.  One rounding instead of the two differs in 1 of 2^17 (bf16)
    or 2^14 (f16) of these 0.6 to 2.5 million values; sines and cosines that are
    off by 4e-13 in fewer than 1 of 2^32, as they have to move a 32-bit value on
    or off the middle between two 2-byte ones."""
    g = torch.Generator().manual_seed(tokens + off)
    heads, dim = 8, 128
    base = torch.randn(tokens, heads * dim + off, generator=g).to(dtype)
    q = base[:, off:].unflatten(1, (heads, dim))
    dq = base.to(DEV)[:, off:].unflatten(1, (heads, dim))
    inv = 10000.0 ** (-torch.arange(0, dim, 2).float() / dim)
    lens = torch.tensor([tokens + 31], dtype=torch.int32, device=DEV)
    pages = (tokens + 31) // 64 + 1
    cache = nv.KVCache.empty(pages, 1, 64, dim)
    table = torch.arange(pages, dtype=torch.int32, device=DEV)[None]
    k = torch.zeros(tokens, 1, dim, dtype=dtype, device=DEV)
    got = nv.kv_append(k, k, cache, table, lens, q=dq, cu_q=torch.tensor([0, tokens], dtype=torch.int32, device=DEV),
                       inv_freq=inv.to(DEV), interleaved=interleaved)
    want = rotate(q, torch.arange(31, tokens + 31), inv, interleaved).to(dtype)
    assert (got.cpu() != want).sum() == 0
