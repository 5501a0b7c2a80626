"""The paged attention over thousands of sequences (needs a B200)."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_run import check_attn, check_lse, pages, queries, random_rows
from top_sparse_attention_02_b200 import binding as tsa

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (3, 1)])
@pytest.mark.parametrize("kind", ["rows", "list", "prefix"])
def test_thousands_of_sequences(cuda_dev, Hq, Hkv, kind):
    """More rows of output than the joining kernel has warps; lengths of none, few and (so that units
    lie in several CTAs) a thousand rows; lists; a prefix that most sequences hold."""
    B = 4900 if Hq == 3 else 2500
    rng = np.random.default_rng(B)
    P = 40 if kind == "prefix" else 0
    assert B * Hq > 1184 * 8 and (not P or (B - 1) * P * Hkv >= 81920)
    lens = [int(x) for x in rng.integers(0, 30, B) + P * (rng.random(B) < 0.9)]
    for b in range(7, B, 601):
        lens[b] = 1000 + b % 13
    K, V, table = pages(lens, Hkv, 16, torch.bfloat16, seed=B, shared=P, dev=cuda_dev)
    Q = queries(B, Hq, torch.bfloat16, dev=cuda_dev)
    idx = random_rows(lens, Hkv, 50, seed=1) if kind == "list" else None
    ln = torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    cache = tsa.paged_cache(K, V, table)
    ws = tsa.new_paged_workspace(cache, Hq, P)
    O, lse = torch.full_like(Q, float("nan")), torch.full((B, Hq), float("nan"), device=cuda_dev)
    a = tsa.paged_attn_args(cache, Q, ln, O, ws, scale=SCALE, prefix_len=P, lse=lse,
                            idx=None if idx is None else torch.from_numpy(idx).to(cuda_dev))
    (tsa.prefix_attn if P else tsa.paged_attn)(a)
    tsa.check_device_status(ws)
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE, idx)
    check_attn(O, want, torch.bfloat16, 8 if P else 16, float(torch.nan_to_num(V.float()).abs().max()))
    check_lse(lse, wl)


def test_work_grows_with_the_batch_not_with_its_square(cuda_dev):
    """Sixteen times as many one-page sequences take less than 32 times as long (16 is even; a joining
    CTA for every 8 rows, each adding up all lengths, made it 57)."""
    def took(B):
        table = torch.arange(B, dtype=torch.int32, device=cuda_dev).view(B, 1)
        K, V = (torch.zeros(B, 1, 16, 128, dtype=torch.bfloat16, device=cuda_dev) for _ in range(2))
        Q = torch.zeros(B, 8, 128, dtype=torch.bfloat16, device=cuda_dev)
        cache = tsa.paged_cache(K, V, table)
        ws = tsa.new_paged_workspace(cache, 8)
        a = tsa.paged_attn_args(cache, Q, torch.full((B,), 16, dtype=torch.int32, device=cuda_dev), torch.empty_like(Q), ws,
                                scale=SCALE)
        times = []
        for _ in range(7):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            for _ in range(8):
                tsa.paged_attn(a)
            e[1].record()
            torch.cuda.synchronize()
            times.append(e[0].elapsed_time(e[1]))
        tsa.check_device_status(ws)
        return min(times)

    assert took(65536) < 32 * took(4096)
