"""The paged decode path against its definition in 64 bits (needs a B200)."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_run import DT, check_attn, check_lse, half_step, pages, queries, random_rows
from top_sparse_attention_02_b200 import binding as tsa

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)
WEIGHT_BITS = {"bf16": 16, "fp16": 20}  # p as a number and the rest of it, both of the element type


def freqs(rot, dev):
    return None if rot == 0 else (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).to(dev)


# ------------------------------------------------------------------ norm and rotation

def check_rounded(got, want, dtype, what):
    """One rounding of a value computed in fp32: half a step of it, plus 16 fp32 roundings of
    the larger of a pair's products (|pair| <= sqrt(2) * the head's largest element)."""
    err = np.abs(got.detach().cpu().double().numpy() - want)
    big = np.abs(want).max(-1, keepdims=True) * math.sqrt(2.0)
    tol = half_step(dtype) * np.abs(want) + 16 * 2.0 ** -24 * big + torch.finfo(dtype).tiny
    assert (err <= tol).all(), f"{what}: off by {(err / tol).max():.2f} of the tolerance"


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,Hq,Hkv,rot,interleaved,norm", [
    (1, 8, 2, 128, False, True), (1, 1, 1, 16, True, True), (5, 28, 4, 64, False, True), (3, 5, 1, 96, True, True),
    (130, 3, 3, 48, False, False), (1187, 16, 2, 128, True, True), (1300, 5, 2, 32, False, True), (7, 2, 1, 0, False, True),
    (33, 32, 8, 128, False, False)])
def test_norm_rope(cuda_dev, dt, T, Hq, Hkv, rot, interleaved, norm):
    dtype = DT[dt]
    g = torch.Generator().manual_seed(T + rot)
    qkv = (torch.randn(T, Hq + 2 * Hkv, 128, generator=g) * 3).to(dtype)
    qkv[T // 2, 0] = 0  # a head of zeros
    pos = torch.randint(0, 1 << 20, (T,), generator=g).to(torch.int32)
    wq, wk = 1 + 0.3 * torch.randn(128, generator=g), 1 + 0.3 * torch.randn(128, generator=g)
    f = freqs(rot, cuda_dev)
    x = qkv.to(cuda_dev)
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    qo, ko = torch.full_like(x[:, :Hq].contiguous(), float("nan")), torch.full_like(x[:, :Hkv].contiguous(), float("nan"))
    a = tsa.qk_norm_rope_args(q, k, qo, ko, q_weight=wq.to(cuda_dev) if norm else None, eps=1e-5,
                              k_weight=wk.to(cuda_dev) if norm else None, positions=pos.to(cuda_dev), inv_freq=f,
                              interleaved=interleaved)
    tsa.qk_norm_rope(a)
    assert torch.equal(x.cpu(), qkv)
    wants = [oracle.norm_rope(qkv[:, s], w if norm else None, 1e-5, pos, f, interleaved)
             for s, w in ((slice(0, Hq), wq), (slice(Hq, Hq + Hkv), wk))]
    check_rounded(qo, wants[0], dtype, "queries")
    check_rounded(ko, wants[1], dtype, "keys")
    # in place, out of the same fused buffer: the same bits, and the values untouched
    b = tsa.qk_norm_rope_args(q, k, q, k, q_weight=a._tensors[4], k_weight=a._tensors[5], eps=1e-5,
                              positions=pos.to(cuda_dev), inv_freq=f, interleaved=interleaved)
    tsa.qk_norm_rope(b)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(x[:, Hq + Hkv:].cpu(), qkv[:, Hq + Hkv:])


def test_norm_rope_one_side_and_no_token(cuda_dev):
    x = torch.randn(6, 4, 128, device=cuda_dev).to(torch.bfloat16)
    w, f = torch.ones(128, device=cuda_dev), freqs(128, cuda_dev)
    pos = torch.arange(6, dtype=torch.int32, device=cuda_dev)
    for q, k in ((x, None), (None, x)):
        o = torch.empty_like(x)
        tsa.qk_norm_rope(tsa.qk_norm_rope_args(q, k, o if q is not None else None, o if k is not None else None,
                                               q_weight=w if q is not None else None,
                                               k_weight=w if k is not None else None, positions=pos, inv_freq=f))
        check_rounded(o, oracle.norm_rope(x, w, 1e-6, pos.cpu(), f, False), torch.bfloat16, "one side")
    n = tsa.launch_count()
    tsa.qk_norm_rope(tsa.qk_norm_rope_args(x[:0], None, x[:0], None, positions=pos[:0], inv_freq=f))
    assert tsa.launch_count() == n


def test_far_positions_keep_their_angle(cuda_dev):
    """At the end of int32's range a 32-bit angle has no fraction left."""
    x = torch.randn(4, 2, 128, device=cuda_dev).to(torch.float16)
    f = freqs(128, cuda_dev)
    pos = torch.tensor([2 ** 31 - 1, 10 ** 9 + 7, 2 ** 24 + 1, -5], dtype=torch.int32, device=cuda_dev)
    o = torch.empty_like(x)
    tsa.qk_norm_rope(tsa.qk_norm_rope_args(x, None, o, None, positions=pos, inv_freq=f))
    # 2^31 radians in 64 bits: 2^-22 of a radian, in the oracle as here
    want = oracle.norm_rope(x, None, 0.0, pos.cpu(), f, False)
    err = np.abs(o.cpu().double().numpy() - want)
    big = np.abs(want).max(-1, keepdims=True) * 1.5
    assert (err <= half_step(torch.float16) * np.abs(want) + (2.0 ** -20 + 2.0 ** -21) * big).all()


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("order", ["head", "row"])
@pytest.mark.parametrize("page,Hkv,before,counts,rot,interleaved", [
    (16, 2, [0, 15, 31, 100], [1, 1, 1, 1], 128, False), (48, 3, [0, 47, 200], [130, 1, 17], 64, True),
    (128, 8, [5, 0], [700, 613], 128, False), (32, 1, [3], [9], 0, False)])
def test_append(cuda_dev, dt, order, page, Hkv, before, counts, rot, interleaved):
    dtype = DT[dt]
    after = [a + c for a, c in zip(before, counts)]
    K, V, table = pages(after, Hkv, page, dtype, order, seed=page, dev=cuda_dev)
    K0, V0 = K.clone(), V.clone()
    seq = np.repeat(np.arange(len(before)), counts)
    row = np.concatenate([np.arange(a, a + c) for a, c in zip(before, counts)])
    perm = np.random.default_rng(1).permutation(seq.size)  # any order of tokens, padding among them
    seq, row = np.append(seq[perm], -1).astype(np.int32), np.append(row[perm], 10 ** 9).astype(np.int32)
    T = seq.size
    kv = torch.randn(T, 2 * Hkv, 128, generator=torch.Generator().manual_seed(7)).to(dtype).to(cuda_dev)
    k, v = kv[:, :Hkv], kv[:, Hkv:]
    f = freqs(rot, cuda_dev)
    cache = tsa.paged_cache(K, V, table)
    ws = tsa.new_paged_workspace(cache)
    tsa.paged_append(tsa.paged_append_args(cache, k, v, torch.from_numpy(row).to(cuda_dev), ws,
                                           seq=torch.from_numpy(seq).to(cuda_dev), inv_freq=f, interleaved=interleaved))
    tsa.check_device_status(ws)
    want = oracle.norm_rope(k, None, 0.0, np.minimum(row, 10 ** 6), f, interleaved)
    tab = table.cpu()
    touched = torch.zeros(K.shape[0], page, dtype=torch.bool)
    for t in range(T - 1):
        pg, off = int(tab[seq[t], row[t] // page]), row[t] % page
        touched[pg, off] = True
        check_rounded(K[pg, :, off], want[t], dtype, f"key of token {t}")
        assert torch.equal(V[pg, :, off], v[t])
    for new, old in ((K, K0), (V, V0)):  # every other row as it was, bit by bit
        same = new.cpu().view(torch.int16) == old.cpu().view(torch.int16)
        assert same.permute(0, 2, 1, 3)[~touched].all()


def test_append_positions_apart_from_rows_and_default_sequences(cuda_dev):
    K, V, table = pages([40, 40], 2, 16, torch.bfloat16, dev=cuda_dev)
    k = torch.randn(2, 2, 128, device=cuda_dev).to(torch.bfloat16)
    row = torch.tensor([3, 33], dtype=torch.int32, device=cuda_dev)
    pos = torch.tensor([1000, 7], dtype=torch.int32, device=cuda_dev)
    f = freqs(128, cuda_dev)
    cache = tsa.paged_cache(K, V, table)
    ws = tsa.new_paged_workspace(cache)
    tsa.paged_append(tsa.paged_append_args(cache, k, k, row, ws, positions=pos, inv_freq=f))
    tsa.check_device_status(ws)
    want = oracle.norm_rope(k, None, 0.0, pos.cpu(), f, False)
    for t in range(2):
        pg, off = int(table[t, int(row[t]) // 16]), int(row[t]) % 16
        check_rounded(K[pg, :, off], want[t], torch.bfloat16, "key")
        assert torch.equal(V[pg, :, off], k[t])


def test_append_out_of_range_is_skipped_and_flagged(cuda_dev):
    K, V, table = pages([32, 32], 1, 16, torch.bfloat16, dev=cuda_dev)  # table: 2 pages and an entry of -1
    cache = tsa.paged_cache(K, V, table)
    ws = tsa.new_paged_workspace(cache)
    k = torch.ones(1, 1, 128, device=cuda_dev).to(torch.bfloat16)
    K0 = K.clone()
    bad_table = table.clone()
    bad_table[0, 0] = K.shape[0]
    for seq, row, tab in ((2, 0, table), (0, -1, table), (0, 48, table), (0, 40, table), (0, 0, bad_table)):
        c = tsa.paged_cache(K, V, tab)
        i32 = [torch.tensor([x], dtype=torch.int32, device=cuda_dev) for x in (row, seq)]
        tsa.paged_append(tsa.paged_append_args(c, k, k, i32[0], ws, seq=i32[1]))
        with pytest.raises(tsa.TsaError) as e:
            tsa.check_device_status(ws)
        assert e.value.status == tsa.TSA_ERR_DEVICE_BOUNDS
        assert torch.equal(K.view(torch.int16), K0.view(torch.int16))
    tsa.check_device_status(ws)


# ------------------------------------------------------------------ attention

def attend(K, V, table, Q, lens, *, prefix=None, idx=None, kreq=None, ws=None, check=True, lse=True):
    dev = Q.device
    cache = tsa.paged_cache(K, V, table)
    ws = tsa.new_paged_workspace(cache, Q.shape[1], prefix or 0) if ws is None else ws
    O = torch.full_like(Q, float("nan"))
    out = torch.full(Q.shape[:2], float("nan"), device=dev) if lse else None
    i32 = lambda x: None if x is None else torch.as_tensor(np.asarray(x), dtype=torch.int32).to(dev)
    a = tsa.paged_attn_args(cache, Q, i32(lens), O, ws, scale=SCALE, idx=i32(idx), k_per_seq=i32(kreq),
                            prefix_len=prefix or 0, lse=out)
    (tsa.paged_attn if prefix is None else tsa.prefix_attn)(a)
    if check:
        tsa.check_device_status(ws)
    return O, out


def vmax(V):
    return float(torch.nan_to_num(V.float()).abs().max())


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv,page,order,lens", [
    (8, 2, 16, "head", [1]), (8, 2, 16, "row", [0]), (4, 4, 32, "head", [15, 16, 17, 63, 64, 65, 0, 1]),
    (5, 1, 48, "row", [700]), (14, 2, 64, "head", [333, 1, 128, 2000]), (32, 2, 128, "row", [513, 0, 77]),
    (9, 1, 16, "head", [5000]), (16, 8, 256, "head", [0, 0, 0, 300]), (8, 1, 16, "head", [21000])])
def test_paged_attn_every_row(cuda_dev, dt, Hq, Hkv, page, order, lens):
    K, V, table = pages(lens, Hkv, page, DT[dt], order, seed=sum(lens), dev=cuda_dev)
    Q = queries(len(lens), Hq, DT[dt], dev=cuda_dev)
    O, lse = attend(K, V, table, Q, lens)
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE)
    check_attn(O, want, DT[dt], WEIGHT_BITS[dt], vmax(V))
    check_lse(lse, wl)
    for b, n in enumerate(lens):
        if n == 0:
            assert (O[b] == 0).all()


def test_paged_attn_many_ragged_units(cuda_dev):
    """Units that begin and end inside a CTA's share, and more sequences than threads."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 90, 300)]
    K, V, table = pages(lens, 3, 16, torch.bfloat16, seed=9, dev=cuda_dev)
    Q = queries(300, 6, torch.bfloat16, dev=cuda_dev)
    ws = None
    O, lse = attend(K, V, table, Q, lens)
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE)
    check_attn(O, want, torch.bfloat16, 16, vmax(V))
    check_lse(lse, wl)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv,page,order,lens,k", [
    (8, 2, 16, "head", [1000], 1), (32, 8, 64, "head", [5000, 0, 30], 100), (12, 1, 48, "row", [900, 901], 333),
    (6, 3, 32, "head", [2000, 17, 3], 64), (64, 8, 128, "row", [9000], 700)])
def test_paged_attn_selected_rows(cuda_dev, dt, Hq, Hkv, page, order, lens, k):
    K, V, table = pages(lens, Hkv, page, DT[dt], order, seed=k, dev=cuda_dev)
    Q = queries(len(lens), Hq, DT[dt], dev=cuda_dev)
    idx = random_rows(lens, Hkv, k, seed=k)
    idx[0, 0, 0] = -1  # a hole in the list
    kreq = [max(1, k - 3 * b) for b in range(len(lens))]
    for kr in (None, kreq):
        O, lse = attend(K, V, table, Q, lens, idx=idx, kreq=kr)
        want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE, idx, kr)
        check_attn(O, want, DT[dt], WEIGHT_BITS[dt], vmax(V))
        check_lse(lse, wl)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv,page,order,prefix,lens", [
    (8, 2, 16, "head", 64, [64, 65, 100, 0, 63]), (4, 1, 32, "row", 1, [1, 2, 40]), (28, 4, 48, "head", 1007, [1007, 1300, 900]),
    (64, 8, 128, "row", 384, [400, 384, 512, 385, 1000, 383]), (16, 1, 16, "head", 130, [131 + 7 * i for i in range(20)]),
    (8, 8, 64, "head", 500, [0, 0, 3]), (2, 1, 16, "head", 0, [5, 0]), (9, 1, 64, "head", 3000, [3001] * 40)])
def test_prefix_attn(cuda_dev, dt, Hq, Hkv, page, order, prefix, lens):
    K, V, table = pages(lens, Hkv, page, DT[dt], order, seed=prefix, shared=prefix, dev=cuda_dev)
    Q = queries(len(lens), Hq, DT[dt], dev=cuda_dev)
    O, lse = attend(K, V, table, Q, lens, prefix=prefix)
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE)
    check_attn(O, want, DT[dt], {"bf16": 8, "fp16": 11}[dt], vmax(V))
    check_lse(lse, wl)


def test_attention_flags_bad_pages_and_lengths(cuda_dev):
    lens = [100, 100]
    K, V, table = pages(lens, 2, 16, torch.bfloat16, dev=cuda_dev)
    Q = queries(2, 8, torch.bfloat16, dev=cuda_dev)
    idx = random_rows(lens, 2, 20)
    good, _ = attend(K, V, table, Q, lens)
    for bad in (K.shape[0], -1, 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        cache = tsa.paged_cache(K, V, t)
        ws = tsa.new_paged_workspace(cache, 8, 64)
        full_list = np.tile(np.arange(100, dtype=np.int32), (2, 2, 1))
        for kw in (dict(), dict(idx=full_list), dict(prefix=64)):
            O, _ = attend(K, V, t, Q, lens, ws=ws, check=False, **kw)
            with pytest.raises(tsa.TsaError) as e:
                tsa.check_device_status(ws)
            assert e.value.status == tsa.TSA_ERR_DEVICE_BOUNDS
            # the rows of that page are left out
            rows = np.array([r for r in range(100) if not 32 <= r < 48], dtype=np.int32)
            sub = np.full((2, 2, 100), -1, np.int32)
            sub[:, :, :rows.size] = rows
            if "prefix" not in kw:
                want, _ = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE, sub)
                check_attn(O[:1], want[:1], torch.bfloat16, 8, vmax(V))
                check_attn(O[1:], good[1:].double().cpu().numpy(), torch.bfloat16, 7, vmax(V))
            assert torch.isfinite(O).all()
    cache = tsa.paged_cache(K, V, table)
    ws = tsa.new_paged_workspace(cache, 8)
    over = table.shape[1] * 16 + 1
    for kw, ln in ((dict(), [-1, 100]), (dict(), [over, 100]), (dict(idx=np.full((2, 2, 3), 100, np.int32)), lens),
                   (dict(idx=idx, kreq=[21, 1]), lens), (dict(idx=idx, kreq=[-1, 1]), lens)):
        O, _ = attend(K, V, table, Q, ln, ws=ws, check=False, **kw)
        with pytest.raises(tsa.TsaError) as e:
            tsa.check_device_status(ws)
        assert e.value.status == tsa.TSA_ERR_DEVICE_BOUNDS
    O, _ = attend(K, V, table, Q, lens, ws=ws)  # the workspace still works
    assert torch.equal(O, good)
