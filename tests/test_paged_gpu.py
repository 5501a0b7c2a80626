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


# (B - 1) * prefix * Hkv >= 81920 rows: the prefix gets its own pass; the first row of
# cases is below that (each sequence reads its own table)
PREFIX = [
    (8, 2, 16, "head", 64, [64, 65, 100, 0, 63]), (4, 1, 32, "row", 1, [1, 2, 40]), (8, 8, 64, "head", 500, [0, 0, 3]),
    (2, 1, 16, "head", 0, [5, 0]),
    # a group of 7, two row tiles (196 rows), the prefix ends inside a tile, a page and a box
    (28, 4, 48, "row", 1007, [1007 + 13 * i % 300 for i in range(28)]),
    # one row tile (30 rows of one head each), pages of a whole tile, whole tiles
    (8, 8, 128, "head", 512, [512 + i % 3 for i in range(30)]),
    # 144 rows; the first sequences are empty, short, one row short
    (32, 2, 256, "head", 5200, [0, 17, 5199] + [5200 + 40 * i for i in range(9)]),
    # 320 rows: a group of 256 and one of 64; many splits; pages of one box
    (8, 1, 16, "row", 2200, [2200 + i for i in range(40)]),
    # 300 sequences (more than a warp's and a CTA's worth), 5 row groups of one head
    (4, 1, 32, "head", 290, [290 + i % 5 for i in range(299)] + [3]),
    # a single split's worth of tiles less one row
    (64, 8, 64, "head", 383, [383 + i for i in range(33)]),
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv,page,order,prefix,lens", PREFIX)
def test_prefix_attn(cuda_dev, dt, Hq, Hkv, page, order, prefix, lens):
    K, V, table = pages(lens, Hkv, page, DT[dt], order, seed=prefix, shared=prefix, dev=cuda_dev)
    Q = queries(len(lens), Hq, DT[dt], dev=cuda_dev)
    O, lse = attend(K, V, table, Q, lens, prefix=prefix)
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE)
    check_attn(O, want, DT[dt], {"bf16": 8, "fp16": 11}[dt], vmax(V))
    check_lse(lse, wl)
    for b, n in enumerate(lens):
        if n == 0:
            assert (O[b] == 0).all()


def test_prefix_that_grows_and_large_scores(cuda_dev):
    """Maxima that climb along the prefix (the sums are rescaled again and again), scores of
    several hundred, and prefix rows that only some sequences attend holding infinities."""
    B, Hq, Hkv, page, P = 33, 16, 8, 64, 640
    lens = [P + 1 + i for i in range(B - 1)] + [300]
    K, V, table = pages(lens, Hkv, page, torch.bfloat16, seed=5, shared=P, dev=cuda_dev)
    Q = queries(B, Hq, torch.bfloat16, dev=cuda_dev)
    row = torch.arange(P, device=cuda_dev)
    pg = table[0][row // page].long()
    K[pg, :, row % page] = (K[pg, :, row % page].float() * (1 + row.float() / 16)[:, None, None]).to(K.dtype)
    O, lse = attend(K, V, table, Q, lens, prefix=P)
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE)
    # logits up to 40 times as large as check_attn's: so are their errors (2^-16 * 40 = 2^-10.7)
    check_attn(O, want, torch.bfloat16, 7.8, vmax(V))
    assert np.abs(lse.cpu().double().numpy() - wl).max() <= 40 * 2e-4
    # the last sequence is shorter than the prefix and has its own pages: nothing of the others' reaches it
    clean = O[-1].clone()
    V[table[0, 1].long()] = float("inf")
    O, _ = attend(K, V, table, Q, lens, prefix=P)
    assert torch.equal(O[-1], clean) and not torch.isfinite(O[:-1]).all()


def test_a_prefix_that_no_sequence_holds(cuda_dev):
    B, Hq, Hkv, P = 30, 16, 8, 400
    lens = [P - 1 - 3 * i for i in range(B)]
    K, V, table = pages(lens, Hkv, 16, torch.bfloat16, seed=12, dev=cuda_dev)
    Q = queries(B, Hq, torch.bfloat16, dev=cuda_dev)
    # (the table is as wide as the prefix: (B - 1) * P * Hkv = 92,800 rows would be shared)
    wide = torch.full((B, 26), -1, dtype=torch.int32, device=cuda_dev)
    wide[:, :table.shape[1]] = table
    assert torch.equal(attend(K, V, wide, Q, lens, prefix=P)[0], attend(K, V, wide, Q, lens)[0])


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("gap", [17.0, 19.0, 23.0])
def test_a_long_flat_tail_below_a_spike(cuda_dev, dt, gap):
    """One row far above tens of thousands that are worth exp(-gap) of it each, below fp16's smallest
    number, with values that do not cancel: together they are worth more than an output's rounding."""
    n, B, Hq, Hkv = 40000, 4, 16, 2
    one = torch.ones(128) / math.sqrt(128.0)
    K = torch.zeros(n // 64, Hkv, 64, 128, dtype=DT[dt])
    K[0, :, 5] = (one * 16).to(DT[dt])
    V = torch.full((n // 64, Hkv, 64, 128), 1.0, dtype=DT[dt])
    V[0, :, 5] = 0
    K, V = K.to(cuda_dev), V.to(cuda_dev)
    table = torch.arange(n // 64, dtype=torch.int32, device=cuda_dev).repeat(B, 1).contiguous()
    # q . k = gap / SCALE for the spike
    Q = (one * gap / SCALE / 16).to(DT[dt]).expand(B, Hq, 128).contiguous().to(cuda_dev)
    lens = [n] * B
    want, wl = oracle.paged_attn(Q[:1], K.cpu(), V.cpu(), table[:1].cpu(), lens[:1], SCALE)
    for P in (None, n - 100):
        O, lse = attend(K, V, table, Q, lens, prefix=P)
        # every output is the tail's share of the weight: its relative error is the tail weights'
        # (one value of all of them: their rounding to 8 or 11 bits does not average out over a prefix)
        bits = WEIGHT_BITS[dt] if P is None else {"bf16": 9, "fp16": 11}[dt]
        tol = (half_step(DT[dt]) + 2.0 ** -bits + 2.0 ** -14) * want + torch.finfo(DT[dt]).eps * torch.finfo(DT[dt]).tiny
        assert (np.abs(O.double().cpu().numpy() - want) <= tol).all(), (P, O[0, 0, 0].item(), want[0, 0, 0])
        check_lse(lse, np.broadcast_to(wl, (B, Hq)))


def test_not_a_number_stays_in_its_row(cuda_dev):
    B, Hq, Hkv, P = 33, 16, 8, 384
    lens = [P + 20 + i for i in range(B)]
    K, V, table = pages(lens, Hkv, 64, torch.float16, seed=6, shared=P, dev=cuda_dev)
    Q = queries(B, Hq, torch.float16, dev=cuda_dev)
    good = [attend(K, V, table, Q, lens, **kw)[0] for kw in (dict(prefix=P), dict())]
    Q[7, 3] = float("nan")
    Q[9, 5, 0] = float("inf")
    for kw, ref in zip((dict(prefix=P), dict()), good):
        O, lse = attend(K, V, table, Q, lens, **kw)
        assert torch.isnan(O[7, 3]).all() and torch.isnan(O[9, 5]).all() and torch.isnan(lse[7, 3])
        keep = torch.ones(B, Hq, dtype=torch.bool)
        keep[7, 3] = keep[9, 5] = False
        assert torch.equal(O[keep.to(cuda_dev)], ref[keep.to(cuda_dev)])


def test_bad_page_in_a_shared_prefix(cuda_dev):
    B, Hq, Hkv, P = 33, 16, 8, 400
    lens = [P + i for i in range(B)]
    K, V, table = pages(lens, Hkv, 16, torch.bfloat16, seed=8, shared=P, dev=cuda_dev)
    Q = queries(B, Hq, torch.bfloat16, dev=cuda_dev)
    t = table.clone()
    t[0, 2] = K.shape[0]  # of the sequence whose table serves the prefix: rows 32..47 of everybody's
    ws = tsa.new_paged_workspace(tsa.paged_cache(K, V, t), Hq, P)
    O, _ = attend(K, V, t, Q, lens, prefix=P, ws=ws, check=False)
    with pytest.raises(tsa.TsaError) as e:
        tsa.check_device_status(ws)
    assert e.value.status == tsa.TSA_ERR_DEVICE_BOUNDS
    keep = np.array([r for r in range(max(lens)) if not 32 <= r < 48])
    idx = np.full((B, Hkv, max(lens)), -1, np.int32)
    for b, n in enumerate(lens):
        rows = keep[keep < n]
        idx[b, :, :rows.size] = rows
    want, _ = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE, idx)
    check_attn(O, want, torch.bfloat16, 8, vmax(V))


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


# ------------------------------------------------------------------ as they are used

def test_same_bits_on_every_call_and_on_a_shared_workspace(cuda_dev):
    """The work is divided by the lengths alone: a second call, a call after others of other shapes on
    the same workspace, and a call on another stream give the same bits."""
    lens = [700, 0, 33, 5000, 64]
    K, V, table = pages(lens, 2, 16, torch.bfloat16, seed=1, dev=cuda_dev)
    Q = queries(5, 16, torch.bfloat16, dev=cuda_dev)
    P = 2300
    plens = [P + 50 * i for i in range(20)]
    Kp, Vp, tp = pages(plens, 2, 32, torch.bfloat16, seed=2, shared=P, dev=cuda_dev)
    Qp = queries(20, 16, torch.bfloat16, seed=3, dev=cuda_dev)
    ws = tsa.new_paged_workspace(tsa.paged_cache(Kp, Vp, tp), 16, P)
    idx = random_rows(lens, 2, 50)
    first = [attend(K, V, table, Q, lens, ws=ws), attend(Kp, Vp, tp, Qp, plens, prefix=P, ws=ws),
             attend(K, V, table, Q, lens, idx=idx, ws=ws)]
    ws.random_(0, 256)  # nothing but the flag has to be zero
    tsa.workspace_init(ws[:256])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [attend(K, V, table, Q, lens, idx=idx, ws=ws), attend(K, V, table, Q, lens, ws=ws),
                 attend(Kp, Vp, tp, Qp, plens, prefix=P, ws=ws)]
    torch.cuda.synchronize()
    for (o, l), (o2, l2) in zip(first, (again[1], again[2], again[0])):
        assert torch.equal(o, o2) and torch.equal(l, l2)


def test_two_calls_at_once(cuda_dev):
    """Two streams, a workspace each."""
    lens = [3000 + 7 * i for i in range(12)]
    K, V, table = pages(lens, 4, 64, torch.float16, seed=11, dev=cuda_dev)
    Qs = [queries(12, 16, torch.float16, seed=i, dev=cuda_dev) for i in range(2)]
    want = [attend(K, V, table, q, lens)[0] for q in Qs]
    cache = tsa.paged_cache(K, V, table)
    ln = torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    Os = [torch.empty_like(q) for q in Qs]
    wss = [tsa.new_paged_workspace(cache, 16) for _ in Qs]
    args = [tsa.paged_attn_args(cache, q, ln, o, w, scale=SCALE) for q, o, w in zip(Qs, Os, wss)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Qs]
    for _ in range(20):
        for a, s in zip(args, streams):
            tsa.paged_attn(a, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(Os, want):
        assert torch.equal(o, w)
    for w in wss:
        tsa.check_device_status(w)


def test_captured_steps_follow_their_inputs(cuda_dev):
    """A captured decode step (norm and rotation, append, attention over a shared prefix) replayed
    while the lengths, rows and projections change under it, two graphs on one workspace."""
    B, Hq, Hkv, page, P = 12, 16, 8, 32, 1024
    start = [P + 5 * b for b in range(B)]
    K, V, table = pages([n + 8 for n in start], Hkv, page, torch.bfloat16, seed=21, shared=P, dev=cuda_dev)
    Kr, Vr = K.clone(), V.clone()  # what the pages should hold
    cache = tsa.paged_cache(K, V, table)
    ws = tsa.new_paged_workspace(cache, Hq, P)
    f = freqs(128, cuda_dev)
    w = 1 + 0.1 * torch.randn(128, device=cuda_dev)
    qkv = torch.zeros(B, Hq + 2 * Hkv, 128, dtype=torch.bfloat16, device=cuda_dev)
    row, lens = (torch.zeros(B, dtype=torch.int32, device=cuda_dev) for _ in range(2))
    Q, k = torch.empty(B, Hq, 128, dtype=torch.bfloat16, device=cuda_dev), torch.empty(B, Hkv, 128, dtype=torch.bfloat16, device=cuda_dev)
    O = torch.empty_like(Q)
    norm = tsa.qk_norm_rope_args(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], Q, k, q_weight=w, k_weight=w, positions=row, inv_freq=f)
    app = tsa.paged_append_args(cache, k, qkv[:, Hq + Hkv:], row, ws)
    att = tsa.paged_attn_args(cache, Q, lens, O, ws, scale=SCALE, prefix_len=P)
    plain = tsa.paged_attn_args(cache, Q, lens, O, ws, scale=SCALE)

    def step(a, fn):
        tsa.qk_norm_rope(norm)
        tsa.paged_append(app)
        fn(a)

    graphs = []
    side = torch.cuda.Stream()
    lens.copy_(torch.tensor(start))
    row.copy_(torch.tensor(start))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(att, tsa.prefix_attn)  # the kernels are loaded
        tsa.paged_attn(plain)
        for a, fn in ((att, tsa.prefix_attn), (plain, tsa.paged_attn)):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step(a, fn)
            graphs.append(g)
    torch.cuda.synchronize()
    gen = torch.Generator().manual_seed(0)
    tab = table.cpu()
    for n in range(6):
        x = torch.randn(qkv.shape, generator=gen).to(torch.bfloat16)
        at = [s + n for s in start]
        qkv.copy_(x)
        row.copy_(torch.tensor(at, dtype=torch.int32))
        lens.copy_(torch.tensor([r + 1 for r in at], dtype=torch.int32))
        graphs[n % 2].replay()
        tsa.check_device_status(ws)
        # the step itself, from its parts' definitions
        Qw = oracle.norm_rope(x[:, :Hq], w.cpu(), 1e-6, at, f, False)
        kw = oracle.norm_rope(x[:, Hq:Hq + Hkv], w.cpu(), 1e-6, at, f, False)
        check_rounded(Q, Qw, torch.bfloat16, "queries")
        for b in range(B):
            pg, off = int(tab[b, at[b] // page]), at[b] % page
            check_rounded(K[pg, :, off], kw[b], torch.bfloat16, "key")
            Kr[pg, :, off], Vr[pg, :, off] = K[pg, :, off], qkv[b, Hq + Hkv:]
        assert torch.equal(K.view(torch.int16), Kr.view(torch.int16)) and torch.equal(V.view(torch.int16), Vr.view(torch.int16))
        want, _ = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), [r + 1 for r in at], SCALE)
        check_attn(O, want, torch.bfloat16, 8, vmax(V))
    del graphs


def test_a_contiguous_cache_is_a_paged_cache(cuda_dev):
    """tsa_paged_append feeds tsa_decode_step, and tsa_paged_attn over the rows that a SELECT step
    chose is that step's attention."""
    B, Hq, Hkv, N, k = 3, 32, 8, 2048, 100
    lens = [2000, 777, 1500]
    g = torch.Generator().manual_seed(3)
    K, V = (torch.randn(B, Hkv, N, 128, generator=g).to(torch.bfloat16).to(cuda_dev) for _ in range(2))
    Q = queries(B, Hq, torch.bfloat16, dev=cuda_dev)
    table = torch.arange(B, dtype=torch.int32, device=cuda_dev)[:, None].contiguous()
    cache = tsa.paged_cache(K, V, table)
    new = torch.randn(B, 2 * Hkv, 128, generator=g).to(torch.bfloat16).to(cuda_dev)
    ws = tsa.new_paged_workspace(cache, Hq)
    row = torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    tsa.paged_append(tsa.paged_append_args(cache, new[:, :Hkv], new[:, Hkv:], row, ws, inv_freq=freqs(128, cuda_dev)))
    tsa.check_device_status(ws)
    for b in range(B):
        assert torch.equal(V[b, :, lens[b]], new[b, Hkv:])
    ln = row + 1
    shape = tsa.shape_of(Q, K)
    for mode in (tsa.SELECT, tsa.FULL):
        sws = tsa.new_workspace(shape, k, 1, mode, cuda_dev)
        O32 = torch.empty(B, Hq, 128, device=cuda_dev)
        idx = torch.empty(B, Hkv, k, dtype=torch.int32, device=cuda_dev) if mode == tsa.SELECT else None
        tsa.decode_step(tsa.step_args(Q, K, V, ln, O32, sws, mode=mode, scale=SCALE, k_max=k if idx is not None else 0, idx_out=idx))
        tsa.check_device_status(sws)
        O = torch.empty_like(Q)
        tsa.paged_attn(tsa.paged_attn_args(cache, Q, ln, O, ws, scale=SCALE, idx=idx))
        tsa.check_device_status(ws)
        # two roundings of P to 16 bits and more (2^-16 each), one of the output
        err = (O.float() - O32).abs()
        assert (err <= half_step(torch.bfloat16) * O32.abs() + 4 * 2.0 ** -16 * vmax(V)).all()


def test_parts_of_two_caches_combine_through_their_lse(cuda_dev):
    """tsa_paged_attn's lse is what tsa_shard_combine takes: a sequence's rows in two halves."""
    lens = [900, 64]
    K, V, table = pages(lens, 2, 16, torch.float16, seed=2, dev=cuda_dev)
    Q = queries(2, 8, torch.float16, dev=cuda_dev)
    whole, _ = attend(K, V, table, Q, lens)
    halves = [attend(K, V, table, Q, [400, 32]),
              attend(K, V, torch.cat([table[:1, 25:], table[:1, 25:]]).contiguous(), Q, [500, 0])]
    tail = attend(K, V, torch.cat([table[1:, 2:], table[1:, 2:]]).contiguous(), Q, [0, 32])
    O_parts = torch.stack([halves[0][0], halves[1][0] + tail[0]]).float().contiguous()
    lse = torch.stack([halves[0][1], torch.maximum(halves[1][1], tail[1])]).contiguous()
    O = torch.empty(2, 8, 128, device=cuda_dev)
    tsa.shard_combine(O_parts, lse, tsa.tsa_shape(2, 8, 2, 16, 128), O)
    # both parts and the whole were rounded to fp16
    assert (O - whole.float()).abs().max() <= 2 * half_step(torch.float16) * vmax(V) + 2.0 ** -12


def test_pages_beyond_32_bit_offsets(cuda_dev):
    """Pages whose elements lie past 2^32 (a pool of 8.6 GB each of K and V)."""
    Hkv, page = 8, 256
    P = 2 ** 32 // (Hkv * page * 128) + 6
    K, V = (torch.empty(P, Hkv, page, 128, dtype=torch.bfloat16, device=cuda_dev) for _ in range(2))
    last = torch.tensor([[P - 1, 0, P - 3], [P - 2, P - 4, 1]], dtype=torch.int32)
    used = last.flatten().long().to(cuda_dev)
    for t in (K, V):
        t[used] = torch.randn(6, Hkv, page, 128, device=cuda_dev).to(torch.bfloat16)
    table = last.to(cuda_dev)
    lens = [700, 600]
    Q = queries(2, 16, torch.bfloat16, dev=cuda_dev)
    cache = tsa.paged_cache(K, V, table)
    ws = tsa.new_paged_workspace(cache, 16)
    new = torch.randn(2, Hkv, 128, device=cuda_dev).to(torch.bfloat16)
    row = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device=cuda_dev)
    tsa.paged_append(tsa.paged_append_args(cache, new, new, row, ws))
    tsa.check_device_status(ws)
    small = [t[used].cpu() for t in (K, V)]
    assert torch.equal(small[0][2, :, (lens[0] - 1) % page], new[0].cpu())
    assert torch.equal(small[1][5, :, (lens[1] - 1) % page], new[1].cpu())
    tab = torch.arange(6, dtype=torch.int32).view(2, 3)
    idx = random_rows(lens, Hkv, 64)
    for ix in (None, idx):
        O, lse = attend(K, V, table, Q, lens, idx=ix)
        want, wl = oracle.paged_attn(Q, *small, tab, lens, SCALE, ix)
        check_attn(O, want, torch.bfloat16, 16, 6.0)
        check_lse(lse, wl)


def test_interleaved_halves_of_one_buffer(cuda_dev):
    """K and V pages as the two halves of one [num_pages, 2, ...] buffer."""
    lens = [100, 333]
    K, V, table = pages(lens, 4, 32, torch.float16, seed=4, dev=cuda_dev)
    kv = torch.stack([K, V], 1).contiguous()
    Q = queries(2, 8, torch.float16, dev=cuda_dev)
    a, _ = attend(K, V, table, Q, lens)
    b, _ = attend(kv[:, 0], kv[:, 1], table, Q, lens)
    assert torch.equal(a, b)


def test_many_sequences(cuda_dev):
    """More sequences than one pass over the lengths takes, most of them short."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 40, 1500)]
    K, V, table = pages(lens, 1, 16, torch.float16, seed=10, dev=cuda_dev)
    Q = queries(1500, 3, torch.float16, dev=cuda_dev)
    O, lse = attend(K, V, table, Q, lens)
    want, wl = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE)
    check_attn(O, want, torch.float16, 20, vmax(V))
    check_lse(lse, wl)


def test_no_sequence_and_no_row(cuda_dev):
    K, V, table = pages([20], 2, 16, torch.bfloat16, dev=cuda_dev)
    empty = tsa.paged_cache(K, V, table[:0])
    ws = tsa.new_paged_workspace(empty, 8)
    Q = torch.empty(0, 8, 128, dtype=torch.bfloat16, device=cuda_dev)
    tsa.paged_attn(tsa.paged_attn_args(empty, Q, torch.empty(0, dtype=torch.int32, device=cuda_dev), Q, ws, scale=SCALE))
    O, lse = attend(K, V, table, queries(1, 8, torch.bfloat16, dev=cuda_dev), [0])
    assert (O == 0).all() and torch.isneginf(lse).all()
    O, lse = attend(K, V, table, queries(1, 8, torch.bfloat16, dev=cuda_dev), [20], idx=np.full((1, 2, 7), -1))
    assert (O == 0).all() and torch.isneginf(lse).all()
