"""Caches, inputs and lists laid out in other ways than a pool of whole pages (needs a B200)."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_run import DT, check_attn, check_lse, check_norm, pages, queries, random_rows
from test_paged_gpu import WEIGHT_BITS, attend, check_rounded, freqs, vmax
from top_sparse_attention_02_b200 import binding as tsa

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)


def laid_out(t, how):
    """The pages t [P, Hkv, page, 128] as a view of a buffer in another order or with gaps (of NaN)."""
    P, H, R, _ = t.shape
    nan = lambda *shape: torch.full(shape, float("nan"), dtype=t.dtype, device=t.device)
    if how == "heads outermost":
        v = nan(H, P, R, 128).permute(1, 0, 2, 3)
    elif how == "rows outermost":
        v = nan(R, H, P, 128).permute(2, 1, 0, 3)
    elif how == "heads, rows, pages":
        v = nan(H, R, P, 128).permute(2, 0, 1, 3)
    elif how == "padded rows":
        v = nan(P, H, R, 136)[..., :128]
    elif how == "padded rows before heads":
        v = nan(P, R, H, 152).permute(0, 2, 1, 3)[..., :128]
    elif how == "padded heads and pages":
        v = torch.as_strided(nan(P * (H * (R * 128 + 8) + 24)), (P, H, R, 128), (H * (R * 128 + 8) + 24, R * 128 + 8, 128, 1))
    else:
        raise KeyError(how)
    v.copy_(t)
    return v


ORDERS = ["heads outermost", "rows outermost", "heads, rows, pages", "padded rows", "padded rows before heads",
          "padded heads and pages"]


@pytest.mark.parametrize("how", ORDERS)
@pytest.mark.parametrize("page,Hkv", [(16, 3), (80, 8), (128, 1)])
def test_orders_and_gaps(cuda_dev, how, page, Hkv):
    """Every order of pages, heads and rows, and strides that are no multiple of one another: attention over
    every row, lists and a shared prefix, and appending, touch the cache's rows and nothing else."""
    dt, P, B = torch.float16, 1000, 13 if Hkv == 8 else 100
    prefix = P if (B - 1) * P * Hkv >= 81920 else 0
    lens = [P + 7 * b % 90 for b in range(B)]
    K, V, table = pages(lens, Hkv, page, dt, seed=page, shared=P, dev=cuda_dev)
    Q = queries(B, 2 * Hkv, dt, dev=cuda_dev)
    Ks, Vs = laid_out(K, how), laid_out(V, how)
    few = lens[:3]
    idx = random_rows(few, Hkv, 70, seed=2)
    for kw in (dict(), dict(prefix=prefix)) if prefix else (dict(),):
        a, la = attend(K, V, table, Q, lens, **kw)
        b, lb = attend(Ks, Vs, table, Q, lens, **kw)
        assert torch.equal(a, b) and torch.equal(la, lb)
    a, la = attend(K, V, table[:3], Q[:3].contiguous(), few, idx=idx)
    b, lb = attend(Ks, Vs, table[:3], Q[:3].contiguous(), few, idx=idx)
    assert torch.equal(a, b) and torch.equal(la, lb)
    want, wl = oracle.paged_attn(Q[:3], K.cpu(), V.cpu(), table[:3].cpu(), few, SCALE, idx)
    check_attn(b, want, dt, WEIGHT_BITS["fp16"], vmax(V))
    # one more token each, out of a fused and padded projection
    kv = torch.randn(B, 2 * Hkv, 136, device=cuda_dev).to(dt)
    k, v = kv[:, :Hkv, :128], kv[:, Hkv:, :128]
    row = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device=cuda_dev)
    for t in ((K, V), (Ks, Vs)):
        cache = tsa.paged_cache(*t, table)
        ws = tsa.new_paged_workspace(cache)
        before = [x.clone() for x in t]
        tsa.paged_append(tsa.paged_append_args(cache, k, v, row, ws, inv_freq=freqs(96, cuda_dev), interleaved=True))
        tsa.check_device_status(ws)
        for x, old in zip(t, before):
            changed = (x.contiguous().view(torch.int16) != old.contiguous().view(torch.int16)).any(-1).sum()
            assert changed <= B * Hkv
    for x, y in ((K, Ks), (V, Vs)):
        assert torch.equal(x.view(torch.int16), y.contiguous().view(torch.int16))
        base = y._base if y._base is not None else y
        gaps = base.numel() - y.numel()
        assert torch.isnan(base).sum() == torch.isnan(y).sum() + gaps


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_lists_of_no_entry(cuda_dev, dt):
    """k_per_seq of 0 next to others; entries past k are not read."""
    lens = [500, 300, 0, 90]
    K, V, table = pages(lens, 2, 16, DT[dt], seed=3, dev=cuda_dev)
    Q = queries(4, 12, DT[dt], dev=cuda_dev)
    idx = random_rows(lens, 2, 64, seed=3)
    kreq = [0, 10, 5, 64]
    idx[0] = 10 ** 6
    idx[1, :, 10:] = 10 ** 6
    O, lse = attend(K, V, table, Q, lens, idx=idx, kreq=kreq)
    assert (O[0] == 0).all() and (O[2] == 0).all() and torch.isneginf(lse[[0, 2]]).all()
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE, idx, kreq)
    check_attn(O, want, DT[dt], WEIGHT_BITS[dt], vmax(V))
    check_lse(lse, wl)


def test_the_same_row_over_and_over(cuda_dev):
    """A row listed many times counts as often."""
    lens = [700]
    K, V, table = pages(lens, 2, 32, torch.bfloat16, seed=4, dev=cuda_dev)
    Q = queries(1, 4, torch.bfloat16, dev=cuda_dev)
    idx = np.concatenate([np.full((1, 2, 200), 123), np.full((1, 2, 100), 5), np.arange(300)[None, None].repeat(2, 1)], 2).astype(np.int32)
    O, lse = attend(K, V, table, Q, lens, idx=idx)
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE, idx)
    check_attn(O, want, torch.bfloat16, 16, vmax(V))
    check_lse(lse, wl)


def test_broadcast_inputs(cuda_dev):
    """Queries that are one token's for all, and a head's for all heads."""
    x = torch.randn(1, 1, 128, device=cuda_dev).to(torch.bfloat16).expand(9, 5, 128)
    pos = torch.arange(9, dtype=torch.int32, device=cuda_dev) * 1000
    f, w = freqs(128, cuda_dev), torch.ones(128, device=cuda_dev)
    o = torch.empty(9, 5, 128, dtype=torch.bfloat16, device=cuda_dev)
    tsa.qk_norm_rope(tsa.qk_norm_rope_args(x, None, o, None, q_weight=w, positions=pos, inv_freq=f))
    check_rounded(o, oracle.norm_rope(x, w, 1e-6, pos.cpu(), f, False), torch.bfloat16, "broadcast")
    with pytest.raises(tsa.TsaError, match="overlap"):
        tsa.qk_norm_rope(tsa.qk_norm_rope_args(x, None, x, None, q_weight=w, positions=pos, inv_freq=f))


@pytest.mark.parametrize("order", ["head", "row"])
def test_one_page_for_everybody(cuda_dev, order):
    """Several sequences whose tables name the same pages (reading), the largest group, pages of one tile."""
    lens = [48, 31, 1, 47]
    K, V, table = pages([48], 1, 16, torch.bfloat16, order, seed=5, dev=cuda_dev)
    K, V = torch.nan_to_num(K), torch.nan_to_num(V)
    table = table.expand(4, -1).contiguous()
    Q = queries(4, 16, torch.bfloat16, dev=cuda_dev)
    O, lse = attend(K, V, table, Q, lens)
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE)
    check_attn(O, want, torch.bfloat16, 16, vmax(V))
    check_lse(lse, wl)
