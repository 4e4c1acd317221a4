"""Keys of the append with norms at the end of a page, whose angles have been
turned on from round to round: values are good to 1e-12.

Codes hold 4 bits, so what shows an error of 1e-12 is a value beside a border:
one whose rounding to 32 bits decides between two codes.  A pair's two weights
are searched for values at 2e-12 to 4e-12 of themselves on either side of one.
The first angles are off by 4e-13 at most, each turn adds some 2^-52 (1.4e-14
in 63 turns); with |p cos| + |q sin| at most twice the value and both parts off
by as much, values are off by less than 1e-12, half of the distance.
"""

import numpy as np
import pytest
import torch

import nvfp4_quantized_matmul_amd as nv
from gpu_util import DEV

pytestmark = pytest.mark.gpu

DIM = PAGE = 256
HALF = DIM // 2
LD = np.longdouble


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def border_beside(u):
    """The value at which the rounding to 32 bits, and then to a code, turns over, nearest to u > 0."""
    e = np.floor(np.log2(float(u)))
    k = np.round((float(u) / 2.0 ** e - 1) * 8 - 0.5)          # the tie 1 + (2k + 1) / 16 between two codes
    k = min(max(k, 0), 7)
    tie = LD((1 + (2 * k + 1) / 16) * 2.0 ** e)
    half = LD(2.0 ** (e - 24))                                 # half a step of 32 bits
    return tie + half if k % 2 == 0 else tie - half            # the tie itself goes to the even code


def weights_beside(p, q, side):
    """float32 (w, v) with p w + q v at 2e-12 to 4e-12 beside a border, on that side of it."""
    want = border_beside(abs(p + q)) * np.sign(p + q) * (1 + side * LD(3e-12))
    v = (1 + np.arange(1 << 19, dtype=np.float64) * 2.0 ** -23).astype(np.float32)
    w = ((want - q * v.astype(LD)) / p).astype(np.float32)
    off = np.abs((p * w.astype(LD) + q * v.astype(LD)) / want - 1)
    at = int(np.argmin(off))
    assert off[at] <= 1e-12, "no such weights"
    return w[at], v[at]


@pytest.mark.parametrize("aligned,each", [(True, 8), (False, 4)])     # tokens of a round: 31 and 63 turns to the last one
def test_values_beside_a_border(aligned, each):
    rng = np.random.default_rng(7)
    x = rng.uniform(-1, 1, (PAGE, DIM)).astype(np.float32)
    inv = np.zeros(HALF, np.float32)
    weight = np.ones(DIM, np.float32)
    factor = 1 / np.sqrt((x.astype(LD) ** 2).mean(1) + LD(1e-6))
    targets, i = [], 0
    while len(targets) < 24:
        # a round's angle just below pi / 4 (mod pi / 2), where a cosine's sum is the least exact
        inv[i] = (np.pi / 4 - rng.uniform(0.002, 0.03) + np.pi / 2 * rng.integers(0, 3)) / each
        t = PAGE - each + i % each
        angle = LD(t) * LD(inv[i])
        p, q = factor[t] * x[t, i] * np.cos(angle), -factor[t] * x[t, i + HALF] * np.sin(angle)
        if abs(p + q) > 0.05 and abs(p) + abs(q) < 1.8 * abs(p + q) and abs(p) > 0.3 * abs(q):
            side = 1 if len(targets) % 2 else -1
            weight[i], weight[i + HALF] = weights_beside(p, q, side)
            u = p * LD(weight[i]) + q * LD(weight[i + HALF])
            targets.append((t, i, np.float32(u)))
        i += 1
    base = torch.zeros(PAGE, DIM + (0 if aligned else 1))
    base[:, base.shape[1] - DIM:] = torch.from_numpy(x)
    k = base.to(DEV)[:, base.shape[1] - DIM:].unflatten(1, (1, DIM))
    cache = nv.KVCache.empty(1, 1, PAGE, DIM, DEV)
    nv.kv_append(k, torch.zeros(PAGE, 1, DIM, device=DEV), cache, i32([[0]]), i32([PAGE]), cu_q=i32([0, PAGE]), max_q=PAGE,
                 inv_freq=torch.from_numpy(inv).to(DEV), k_norm=torch.from_numpy(weight).to(DEV))
    up = 127 - int(cache.k_scales[0, 0])
    codes = cache.k[0, 0].cpu()
    want = torch.tensor([float(u) for _, _, u in targets]).mul(2.0 ** up).to(torch.float8_e4m3fn).view(torch.uint8)
    got = torch.stack([codes[t, i] for t, i, _ in targets])
    assert torch.equal(got, want), (got != want).nonzero().flatten().tolist()
