"""The values that come out of the paged attention, by the norm of their error (needs a B200).  The
largest error of an element says little over thousands of rows, where the outputs are as small."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_run import DT, check_attn, check_lse, check_norm, pages, queries, random_rows
from test_paged_gpu import PREFIX, attend, check_rounded, freqs, vmax
from top_sparse_attention_02_b200 import binding as tsa

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv,page,order,prefix,lens", [c for c in PREFIX if max(c[5]) >= 300])
def test_shared_prefix_and_own_rows(cuda_dev, dt, Hq, Hkv, page, order, prefix, lens):
    """Over a prefix with a pass of its own the weights are rounded to the element type, once; without
    one, and through tsa_paged_attn, they keep 16 bits and more."""
    K, V, table = pages(lens, Hkv, page, DT[dt], order, seed=prefix, shared=prefix, dev=cuda_dev)
    Q = queries(len(lens), Hq, DT[dt], dev=cuda_dev)
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE)
    own_pass = (len(lens) - 1) * prefix * Hkv >= 81920
    O, lse = attend(K, V, table, Q, lens, prefix=prefix)
    check_norm(O, want, lens, DT[dt], own_pass, "prefix")
    check_lse(lse, wl)
    O, lse = attend(K, V, table, Q, lens)
    check_norm(O, want, lens, DT[dt], False, "every row")
    check_lse(lse, wl)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv,page,order,lens,k", [
    (5, 1, 48, "row", [700], 0), (14, 2, 64, "head", [333, 1, 128, 2000], 0), (9, 1, 16, "head", [5000], 0),
    (8, 1, 16, "head", [21000], 0), (12, 1, 48, "row", [900, 901], 333), (64, 8, 128, "row", [9000], 700)])
def test_rows_of_each_sequence(cuda_dev, dt, Hq, Hkv, page, order, lens, k):
    K, V, table = pages(lens, Hkv, page, DT[dt], order, seed=sum(lens), dev=cuda_dev)
    Q = queries(len(lens), Hq, DT[dt], dev=cuda_dev)
    idx = random_rows(lens, Hkv, k, seed=k) if k else None
    O, lse = attend(K, V, table, Q, lens, idx=idx)
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE, idx)
    check_norm(O, want, lens, DT[dt], False)
    check_lse(lse, wl)


def test_bad_page_in_a_shared_prefix_leaves_out_its_rows_only(cuda_dev):
    B, Hq, Hkv, P = 33, 16, 8, 400
    lens = [P + i for i in range(B)]
    K, V, table = pages(lens, Hkv, 16, torch.bfloat16, seed=8, shared=P, dev=cuda_dev)
    Q = queries(B, Hq, torch.bfloat16, dev=cuda_dev)
    t = table.clone()
    t[0, 2] = -7  # of the sequence whose table serves the prefix: rows 32..47 of everybody's
    ws = tsa.new_paged_workspace(tsa.paged_cache(K, V, t), Hq, P)
    O, lse = attend(K, V, t, Q, lens, prefix=P, ws=ws, check=False)
    with pytest.raises(tsa.TsaError) as e:
        tsa.check_device_status(ws)
    assert e.value.status == tsa.TSA_ERR_DEVICE_BOUNDS
    rows = np.array([r for r in range(max(lens)) if not 32 <= r < 48])
    idx = np.full((B, Hkv, max(lens)), -1, np.int32)
    for b, n in enumerate(lens):
        idx[b, :, :(rows < n).sum()] = rows[rows < n]
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE, idx)
    check_norm(O, want, lens, torch.bfloat16, True)
    check_lse(lse, wl)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("shared", [True, False])
def test_replayed_steps_attend_to_the_row_they_append(cuda_dev, dt, shared):
    """A captured step (norm and rotation, append, attention) replayed while lengths, rows and inputs
    change: a length that stays behind by one row, or a new row that is not attended, shows."""
    B, Hq, Hkv, page, P = 12, 16, 8, 32, 1024
    start = [P + 5 * b for b in range(B)]
    K, V, table = pages([n + 8 for n in start], Hkv, page, DT[dt], seed=22, shared=P, dev=cuda_dev)
    cache = tsa.paged_cache(K, V, table)
    ws = tsa.new_paged_workspace(cache, Hq, P)
    f = freqs(128, cuda_dev)
    w = 1 + 0.1 * torch.randn(128, device=cuda_dev)
    qkv = torch.zeros(B, Hq + 2 * Hkv, 128, dtype=DT[dt], device=cuda_dev)
    row, lens = (torch.tensor(start, dtype=torch.int32, device=cuda_dev) for _ in range(2))
    Q, k = (torch.empty(B, h, 128, dtype=DT[dt], device=cuda_dev) for h in (Hq, Hkv))
    O, lse = torch.empty_like(Q), torch.empty(B, Hq, device=cuda_dev)
    norm = tsa.qk_norm_rope_args(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], Q, k, q_weight=w, k_weight=w, positions=row, inv_freq=f)
    app = tsa.paged_append_args(cache, k, qkv[:, Hq + Hkv:], row, ws)
    att = tsa.paged_attn_args(cache, Q, lens, O, ws, scale=SCALE, prefix_len=P if shared else 0, lse=lse)

    def step():
        tsa.qk_norm_rope(norm)
        tsa.paged_append(app)
        (tsa.prefix_attn if shared else tsa.paged_attn)(att)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # the kernels are loaded
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    gen = torch.Generator().manual_seed(1)
    for n in range(5):
        at = [s + n for s in start]
        x = torch.randn(qkv.shape, generator=gen)
        x[:, Hq:Hq + Hkv] = x[:, :Hq].view(B, Hkv, -1, 128).mean(2) * 2  # the new key is one that its queries attend to
        qkv.copy_(x)
        row.copy_(torch.tensor(at, dtype=torch.int32))
        lens.copy_(torch.tensor([r + 1 for r in at], dtype=torch.int32))
        graph.replay()
        tsa.check_device_status(ws)
        for b in range(B):
            pg, off = int(table[b, at[b] // page]), at[b] % page
            assert torch.equal(K[pg, :, off], k[b]) and torch.equal(V[pg, :, off], qkv[b, Hq + Hkv:])
        want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), [r + 1 for r in at], SCALE)
        check_norm(O, want, at, DT[dt], shared, f"step {n}")
        check_lse(lse, wl, f"step {n}")
    del graph


@pytest.mark.parametrize("dt,size", [("bf16", 1.5e18), ("bf16", 1e-16), ("fp16", 6e4), ("fp16", 6e-8)])
def test_norm_over_the_range_of_elements(cuda_dev, dt, size):
    """The largest elements whose squares' sum fp32 holds, and the smallest ones, without an eps."""
    g = torch.Generator().manual_seed(3)
    x = ((torch.rand(33, 6, 128, generator=g, dtype=torch.float64) * 2 - 1) * size).to(DT[dt]).to(cuda_dev)
    x[:, :, 0] = size
    w, f = 1 + 0.2 * torch.randn(128, generator=g), freqs(64, cuda_dev)
    pos = torch.arange(33, dtype=torch.int32, device=cuda_dev) * 77
    o = torch.empty_like(x)
    tsa.qk_norm_rope(tsa.qk_norm_rope_args(x, None, o, None, q_weight=w.to(cuda_dev), eps=0.0, positions=pos, inv_freq=f))
    check_rounded(o, oracle.norm_rope(x, w, 0.0, pos.cpu(), f, False), DT[dt], f"{size}")
