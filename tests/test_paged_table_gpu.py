"""Table entries that belong to no row (needs a B200)."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_run import check_lse, check_norm, pages, queries
from test_paged_gpu import attend

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)


@pytest.mark.parametrize("first", [0, 17, 1023])
@pytest.mark.parametrize("junk", [-1, 2 ** 31 - 1, -2 ** 31, 10 ** 6])
@pytest.mark.parametrize("prefix", [True, False])
def test_entries_past_the_rows_do_not_matter(cuda_dev, first, junk, prefix):
    """The first sequence (whose entries are the first to be looked at) is empty, short, or a row short of
    the prefix: whatever its other entries, and everybody's past their rows, hold, the result is
    the same and nothing is flagged."""
    B, Hq, Hkv, P = 14, 16, 8, 1024
    lens = [first, 5] + [P + 30 * i for i in range(B - 2)]
    K, V, table = pages(lens, Hkv, 16, torch.bfloat16, seed=first, shared=P, dev=cuda_dev)
    Q = queries(B, Hq, torch.bfloat16, dev=cuda_dev)
    table = table.clone()
    for b, n in enumerate(lens):
        table[b, -(-n // 16):] = junk
    O, lse = attend(K, V, table, Q, lens, prefix=P if prefix else None)
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE)
    check_norm(O, want, lens, torch.bfloat16, prefix)
    check_lse(lse, wl)
