"""jt_chunk_attn_paged on batches whose work slots hold runs of pieces of one key
tile beside longer ones (the softmax warps are then furthest ahead of the epilogue):
against the 64-bit form, with identical bits from repeated calls."""
import random

import pytest
import torch

from kv_util import batch
from test_gpu_chunk_attn import check, run, workspace

pytestmark = pytest.mark.gpu


def alternating(n, seed):
    """Contexts of 129 to 256 keys beside contexts of 1 to 128, one new token each."""
    r = random.Random(seed)
    return [r.randint(128, 255) if i % 2 == 0 else r.randint(0, 127) for i in range(n)], [1] * n


def prompts(n, seed):
    """Prompts of 129 to 256 tokens on an empty cache (G = 8: units of 1, 1, 1, 1, 2, 2, 2, 2 tiles)."""
    r = random.Random(seed)
    return [0] * n, [r.randint(129, 256) for _ in range(n)]


def mixed(n, seed, most):
    """Contexts of 1 to 128 or of 129 to 384 keys, the last 1 to `most` of them new."""
    r = random.Random(seed)
    keys = [r.randint(1, 128) if r.random() < 0.6 else r.randint(129, 384) for _ in range(n)]
    new = [min(k, r.choice([1, r.randint(1, most)])) for k in keys]
    return [k - b for k, b in zip(keys, new)], new


BATCHES = [("tokens64", alternating(64, 1), 8), ("tokens96", alternating(96, 2), 8), ("prompts16", prompts(16, 3), 64),
           ("prompts32", prompts(32, 4), 64), ("mixed64", mixed(64, 5, 64), 8), ("mixed128", mixed(128, 6, 64), 32),
           ("mixed256", mixed(256, 7, 16), 32)]


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("name,lens,Hq", BATCHES, ids=[b[0] for b in BATCHES])
def test_runs_of_one_tile_pieces(name, lens, Hq, D):
    s = batch(40, lens[0], lens[1], Hq, 8, D)
    ws = workspace(s)
    first = tuple(t.clone() for t in run(s, ws))
    check(s, *first)
    for _ in range(30):
        out, lse = run(s, ws)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
