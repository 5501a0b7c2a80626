"""The paged entry points without a GPU: what they refuse before anything is
enqueued, what their workspaces need, and the oracle of their tests pinned to
facts other than itself."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from paged_run import pages, queries, random_rows


@pytest.fixture(scope="module")
def tsa():
    from top_sparse_attention_02_b200 import build

    build.build()
    from top_sparse_attention_02_b200 import binding

    return binding


def cache(tsa, **kw):
    # fake but aligned addresses: every call here must fail its checks
    c = tsa.tsa_paged_cache()
    v = dict(K=0x10000, V=0x20000, page_table=0x30000, page_stride=2 * 16 * 128, head_stride=16 * 128, row_stride=128,
             num_pages=9, page_size=16, max_pages=4, B=3, Hkv=2, d=128, dtype=0)
    v.update(kw)
    for k, x in v.items():
        setattr(c, k, x)
    return c


BAD_CACHE = [
    (dict(dtype=2), 2, "dtype"), (dict(d=64), 2, "head dimension"), (dict(B=-1), 1, "B >= 0"), (dict(Hkv=0), 1, "Hkv"),
    (dict(num_pages=0), 1, "num_pages"), (dict(max_pages=0), 1, "max_pages"), (dict(page_size=0), 2, "page_size"),
    (dict(page_size=24), 2, "page_size"), (dict(row_stride=132), 1, "multiples of 8"), (dict(row_stride=64), 1, "at least d"),
    (dict(head_stride=-2048), 1, "strides"), (dict(page_stride=1 << 40), 1, "strides"),
    (dict(head_stride=16 * 128 - 8), 1, "overlap"), (dict(page_stride=16 * 128), 1, "overlap"),
    (dict(row_stride=2 * 128, head_stride=128, page_stride=16 * 2 * 128 - 8), 1, "overlap"),
    (dict(B=1 << 20, Hkv=8, head_stride=16 * 128, page_stride=8 * 16 * 128), 2, "B*Hkv"),
]


def attn_args(tsa, c, **kw):
    a = tsa.tsa_paged_attn_args()
    a.cache = c
    v = dict(Q=0x40000, seq_lens=0x50000, O=0x60000, Hq=8, scale=0.1, ws=0x100000, ws_bytes=1 << 40)
    v.update(kw)
    for k, x in v.items():
        setattr(a, k, x)
    return a


def append_args(tsa, c, **kw):
    a = tsa.tsa_append_args()
    a.cache = c
    rot = tsa.tsa_rotation(kw.pop("inv_freq", 0x90000), kw.pop("rot_dim", 128), 0)
    v = dict(K=0x40000, V=0x50000, k_stride_t=256, k_stride_h=128, v_stride_t=256, v_stride_h=128, seq=0x60000, row=0x70000,
             rot=rot, T=5, ws=0x100000, ws_bytes=256)
    v.update(kw)
    for k, x in v.items():
        setattr(a, k, x)
    return a


def qk_args(tsa, **kw):
    a = tsa.tsa_qk_args()
    rot = tsa.tsa_rotation(kw.pop("inv_freq", 0x90000), kw.pop("rot_dim", 128), 0)
    v = dict(q=0x10000, k=0x20000, q_out=0x30000, k_out=0x40000, q_stride_t=1024, q_stride_h=128, k_stride_t=256,
             k_stride_h=128, q_out_stride_t=1024, q_out_stride_h=128, k_out_stride_t=256, k_out_stride_h=128,
             q_weight=0x50000, k_weight=0x60000, positions=0x70000, rot=rot, T=4, Hq=8, Hkv=2, d=128, dtype=0, eps=1e-6)
    v.update(kw)
    for k, x in v.items():
        setattr(a, k, x)
    return a


def refused(tsa, name, a, status, msg):
    assert getattr(tsa.lib(), name)(ctypes.byref(a), None) == status, tsa.last_error()
    assert msg in tsa.last_error(), tsa.last_error()


@pytest.mark.parametrize("kw,status,msg", BAD_CACHE)
def test_a_bad_cache_is_refused_everywhere(tsa, kw, status, msg):
    c = cache(tsa, **kw)
    refused(tsa, "tsa_paged_attn", attn_args(tsa, c), status, msg)
    refused(tsa, "tsa_prefix_attn", attn_args(tsa, c), status, msg)
    refused(tsa, "tsa_paged_append", append_args(tsa, c), status, msg)
    assert tsa.lib().tsa_paged_workspace_size(ctypes.byref(c), 8, 0) == 0 and msg in tsa.last_error()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(Q=None), 1, "NULL"), (dict(O=None), 1, "NULL"), (dict(seq_lens=None), 1, "NULL"), (dict(Q=0x40008), 1, "aligned"),
    (dict(O=0x60004), 1, "aligned"), (dict(O=0x40000), 1, "must not be Q"), (dict(Hq=7), 1, "multiple"),
    (dict(Hq=0), 1, "multiple"), (dict(Hq=34), 2, "group"), (dict(scale=0.0), 1, "scale"), (dict(scale=float("inf")), 1, "scale"),
    (dict(scale=float("nan")), 1, "scale"), (dict(ws=None), 3, "NULL"), (dict(ws=0x100080), 3, "256-byte"),
    (dict(ws_bytes=256), 3, "needs")])
def test_attention_refusals(tsa, kw, status, msg):
    for name in ("tsa_paged_attn", "tsa_prefix_attn"):
        refused(tsa, name, attn_args(tsa, cache(tsa), **kw), status, msg)


def test_attention_refusals_of_one_call(tsa):
    c = cache(tsa)
    refused(tsa, "tsa_paged_attn", attn_args(tsa, c, prefix_len=16), 1, "prefix_len must be 0")
    refused(tsa, "tsa_prefix_attn", attn_args(tsa, c, prefix_len=-1), 1, "prefix_len must be >= 0")
    refused(tsa, "tsa_prefix_attn", attn_args(tsa, c, prefix_len=(1 << 30) + 1), 2, "2^30")
    refused(tsa, "tsa_prefix_attn", attn_args(tsa, c, idx=0x70000, k_max=4), 1, "NULL")
    refused(tsa, "tsa_prefix_attn", attn_args(tsa, c, k_per_seq=0x70000), 1, "NULL")
    refused(tsa, "tsa_paged_attn", attn_args(tsa, c, idx=0x70000, k_max=0), 1, "k_max")
    refused(tsa, "tsa_paged_attn", attn_args(tsa, c, idx=0x70000, k_max=-4), 1, "k_max")
    refused(tsa, "tsa_paged_attn", attn_args(tsa, c, k_max=4), 1, "index list")
    refused(tsa, "tsa_paged_attn", attn_args(tsa, c, k_per_seq=0x70000), 1, "index list")
    for name in ("K", "V", "page_table"):
        refused(tsa, "tsa_paged_attn", attn_args(tsa, cache(tsa, **{name: None})), 1, "cache: NULL")
    refused(tsa, "tsa_paged_attn", attn_args(tsa, cache(tsa, V=0x20008)), 1, "aligned")
    # more rows named than 32-bit granule numbers reach
    refused(tsa, "tsa_paged_attn", attn_args(tsa, cache(tsa, B=65536, max_pages=1 << 20)), 2, "2^37")
    for name in ("tsa_paged_attn", "tsa_prefix_attn", "tsa_paged_append", "tsa_qk_norm_rope"):
        assert getattr(tsa.lib(), name)(None, None) == 1 and "NULL args" in tsa.last_error()


@pytest.mark.parametrize("kw,status,msg", [
    (dict(K=None), 1, "NULL"), (dict(V=None), 1, "NULL"), (dict(row=None), 1, "row"), (dict(T=-1), 1, "T must"),
    (dict(seq=None), 1, "without seq"), (dict(K=0x40002), 1, "aligned"), (dict(k_stride_t=252), 1, "multiples of 8"),
    (dict(v_stride_h=-128), 1, "not negative"), (dict(rot_dim=24), 1, "rot_dim"), (dict(rot_dim=144), 1, "rot_dim"),
    (dict(rot_dim=-16), 1, "rot_dim"), (dict(inv_freq=None), 1, "inv_freq"), (dict(inv_freq=0x90004), 1, "inv_freq"),
    (dict(ws=None), 3, "NULL"), (dict(ws_bytes=255), 3, "needs")])
def test_append_refusals(tsa, kw, status, msg):
    refused(tsa, "tsa_paged_append", append_args(tsa, cache(tsa), **kw), status, msg)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(q=None), 1, "NULL"), (dict(k_out=None), 1, "NULL"), (dict(positions=None), 1, "positions"), (dict(T=-1), 1, "T"),
    (dict(Hq=-1), 1, "Hq"), (dict(d=96), 2, "head dimension"), (dict(dtype=7), 2, "dtype"), (dict(eps=-1.0), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"), (dict(q=0x10008), 1, "aligned"), (dict(k_weight=0x60004), 1, "aligned"),
    (dict(q_stride_h=130), 1, "multiples of 8"), (dict(q_out_stride_h=64), 1, "overlap"),
    (dict(k_out_stride_t=128), 1, "overlap"), (dict(q_out_stride_t=0), 1, "overlap"), (dict(rot_dim=8), 1, "rot_dim"),
    (dict(q_out=0x10000, q_out_stride_t=2048), 1, "its strides")])
def test_norm_rope_refusals(tsa, kw, status, msg):
    refused(tsa, "tsa_qk_norm_rope", qk_args(tsa, **kw), status, msg)


def test_workspace_sizes(tsa):
    size = lambda c, *a: tsa.lib().tsa_paged_workspace_size(ctypes.byref(c), *a)
    c = cache(tsa, B=64, Hkv=8, page_stride=8 * 16 * 128, max_pages=4096)
    assert size(c, 0, 0) == 256
    plain = size(c, 64, 0)
    assert plain % 256 == 0 and plain >= 256 + 2 * 296 * 8 * 528
    last = plain
    for n in (1, 64, 700, 5000, 32768, 65536):
        assert size(c, 64, n) >= last
        last = size(c, 64, n)
    assert last >= plain + 64 * 64 * 528  # a long prefix has partials of its own
    assert size(c, 64, -1) == 0 and size(c, 63, 0) == 0 and size(c, 8 * 17, 0) == 0
    assert tsa.lib().tsa_paged_workspace_size(None, 8, 0) == 0


def test_binding_refusals(tsa):
    K = torch.zeros(5, 2, 16, 128, dtype=torch.bfloat16)
    tab = torch.zeros(3, 4, dtype=torch.int32)
    Q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    lens = torch.zeros(3, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)

    def bad(fn, *a, **kw):
        with pytest.raises(tsa.TsaError) as e:
            fn(*a, **kw)
        assert e.value.status == tsa.TSA_ERR_INVALID_ARG

    bad(tsa.paged_cache, K.float(), K.float(), tab)
    bad(tsa.paged_cache, K, K.half(), tab)
    bad(tsa.paged_cache, K, K[:, :1], tab)
    bad(tsa.paged_cache, K, K.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3), tab)
    bad(tsa.paged_cache, K.transpose(2, 3), K.transpose(2, 3), tab)
    bad(tsa.paged_cache, K, K, tab.long())
    bad(tsa.paged_cache, K, K, tab[:, ::2])
    bad(tsa.paged_cache, K[0], K[0], tab)
    c = tsa.paged_cache(K, K, tab)
    ok = dict(scale=0.1)
    bad(tsa.paged_attn_args, c, Q.half(), lens, Q, ws, **ok)
    bad(tsa.paged_attn_args, c, Q[:2], lens, Q[:2], ws, **ok)
    bad(tsa.paged_attn_args, c, Q, lens.long(), Q, ws, **ok)
    bad(tsa.paged_attn_args, c, Q, lens, Q.float(), ws, **ok)
    bad(tsa.paged_attn_args, c, Q.transpose(0, 1).contiguous().transpose(0, 1), lens, Q, ws, **ok)
    bad(tsa.paged_attn_args, c, Q, lens, Q, ws, idx=torch.zeros(3, 1, 4, dtype=torch.int32), **ok)
    bad(tsa.paged_attn_args, c, Q, lens, Q, ws, lse=torch.zeros(3, 8, dtype=torch.float64), **ok)
    bad(tsa.paged_attn_args, c, Q, lens, Q, ws, lse=torch.zeros(3, 2), **ok)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    f = torch.zeros(64, dtype=torch.float64)
    bad(tsa.paged_append_args, c, k, k[:2], lens, ws)
    bad(tsa.paged_append_args, c, k, k, lens[:2], ws)
    bad(tsa.paged_append_args, c, k, k, None, ws)
    bad(tsa.paged_append_args, c, k, k, lens, ws, inv_freq=f.float())
    bad(tsa.qk_norm_rope_args, None, None, None, None)
    bad(tsa.qk_norm_rope_args, Q, None, Q, Q)
    bad(tsa.qk_norm_rope_args, Q, k.half(), Q, k)
    bad(tsa.qk_norm_rope_args, Q, k[:2], Q, k[:2])
    bad(tsa.qk_norm_rope_args, Q, None, Q, None, q_weight=torch.ones(128, dtype=torch.bfloat16))
    bad(tsa.qk_norm_rope_args, Q, None, Q, None, positions=lens.long(), inv_freq=f)
    # host tensors make arguments, but no call
    a = tsa.qk_norm_rope_args(Q, None, Q, None, positions=lens, inv_freq=f)
    bad(tsa.qk_norm_rope, a)
    bad(tsa.qk_norm_rope, a, stream=0)
    bad(tsa.paged_append, tsa.paged_append_args(c, k, k, lens, ws))
    bad(tsa.paged_attn, tsa.paged_attn_args(c, Q, lens, Q.clone(), ws, **ok))
    # the C side's refusals come through as they are: an inv_freq of 12 would rotate 24 elements
    a = tsa.qk_norm_rope_args(Q, None, Q, None, positions=lens, inv_freq=f[:12])
    assert tsa.lib().tsa_qk_norm_rope(ctypes.byref(a), None) == 1 and "rot_dim" in tsa.last_error()


# ------------------------------------------------------------------ the oracle's pins

def test_oracle_rotation_is_a_rotation_by_position():
    f = np.array([1.0, 0.25])
    x = np.arange(2 * 1 * 6, dtype=np.float64).reshape(2, 1, 6)
    y = oracle.rotate(x, [0, 3], f, False)
    np.testing.assert_array_equal(y[0], x[0])  # position 0: nothing
    np.testing.assert_array_equal(y[:, :, 4:], x[:, :, 4:])  # the elements past the pairs
    a, b = x[1, 0, 0], x[1, 0, 2]  # pair 0 is (0, 2): by 3 radians
    np.testing.assert_allclose(y[1, 0, [0, 2]], [a * math.cos(3) - b * math.sin(3), b * math.cos(3) + a * math.sin(3)])
    z = oracle.rotate(x, [0, 3], f, True)  # interleaved: pair 1 is (2, 3), by 3/4 of a radian
    a, b = x[1, 0, 2], x[1, 0, 3]
    np.testing.assert_allclose(z[1, 0, 2:4], [a * math.cos(.75) - b * math.sin(.75), b * math.cos(.75) + a * math.sin(.75)])
    # scores depend on the distance alone
    q, k = np.random.default_rng(0).standard_normal((2, 1, 1, 6))
    dot = lambda p, r: (oracle.rotate(q, [p], f, False) * oracle.rotate(k, [r], f, False)).sum()
    np.testing.assert_allclose(dot(7, 5), dot(107, 105), rtol=1e-12)


def test_oracle_norm():
    x = torch.tensor([[[3.0, 4.0] + [0.0] * 126]], dtype=torch.float16)
    w = torch.full((128,), 2.0)
    y = oracle.norm_rope(x, w, 0.0, None, None, False)  # rms = 5 / sqrt(128)
    np.testing.assert_allclose(y[0, 0, :2], [2 * 3 / 5 * math.sqrt(128), 2 * 4 / 5 * math.sqrt(128)])
    np.testing.assert_array_equal(oracle.norm_rope(x, None, 0.0, None, None, False), x.double().numpy())


@pytest.mark.parametrize("order", ["head", "row"])
def test_oracle_paged_attention_is_attention_over_the_rows(order):
    lens = [37, 0, 80]
    K, V, table = pages(lens, 2, 16, torch.bfloat16, order)
    Q = queries(3, 6, torch.bfloat16)
    O, lse = oracle.paged_attn(Q, K, V, table, lens, 0.3)
    for b, n in enumerate(lens):
        if n == 0:
            assert (O[b] == 0).all() and np.isneginf(lse[b]).all()
            continue
        at = torch.arange(n)
        k, v = (t[table[b][at // 16].long(), :, at % 16].double() for t in (K, V))  # [n, Hkv, d]
        k, v = (x.transpose(0, 1).repeat_interleave(3, 0) for x in (k, v))
        want = torch.nn.functional.scaled_dot_product_attention(Q[b].double()[:, None], k, v, scale=0.3)[:, 0]
        np.testing.assert_allclose(O[b], want.numpy(), rtol=1e-9, atol=1e-12)
        logits = (Q[b].double()[:, None] * k).sum(-1) * 0.3
        np.testing.assert_allclose(lse[b], torch.logsumexp(logits, -1).numpy() / math.log(2), rtol=1e-12)
    idx = random_rows(lens, 2, 9, seed=4)
    Oi, _ = oracle.paged_attn(Q, K, V, table, lens, 0.3, idx, [9, 9, 4])
    Ok = Q[2].double()[3:] @ torch.stack([K[int(table[2][r // 16]), 1, r % 16].double() for r in idx[2, 1, :4]]).T * 0.3
    Vk = torch.stack([V[int(table[2][r // 16]), 1, r % 16].double() for r in idx[2, 1, :4]])
    np.testing.assert_allclose(Oi[2, 3:], (torch.softmax(Ok, -1) @ Vk).numpy(), rtol=1e-9)
