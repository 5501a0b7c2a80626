"""What include/tsa.h says about the paged calls, held against the library."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def tsa():
    from top_sparse_attention_02_b200 import build

    build.build()
    from top_sparse_attention_02_b200 import binding

    return binding


@pytest.fixture(scope="module")
def header():
    return re.sub(r"\s*\n \*\s*", " ", open(os.path.join(ROOT, "include", "tsa.h")).read())


def shape(tsa, B, Hkv, rows, page=16):
    c = tsa.tsa_paged_cache()
    for k, x in dict(page_stride=Hkv * page * 128, head_stride=page * 128, row_stride=128, num_pages=9, page_size=page,
                     max_pages=-(-rows // page), B=B, Hkv=Hkv, d=128, dtype=0).items():
        setattr(c, k, x)
    return c


@pytest.mark.parametrize("B,Hkv", [(2, 1), (2, 8), (9, 8), (33, 4), (641, 8), (1, 8)])
def test_header_says_where_the_weights_are_coarser(tsa, header, B, Hkv):
    """The pass with weights of the element type is the one that needs room for a prefix's partials:
    from the product on that the header names, and not past the table's rows."""
    at = re.search(r"\(B - 1\) \* prefix_len \* Hkv >= (\d+)", header)
    assert at, "the header does not say from where on the prefix has its own pass"
    first = -(-int(at.group(1)) // max(1, (B - 1) * Hkv))
    c = shape(tsa, B, Hkv, 2 * first)
    size = lambda n: tsa.lib().tsa_paged_workspace_size(ctypes.byref(c), 4 * Hkv, n)
    assert size(first - 1) == size(0) > 0
    assert (size(first) > size(0)) == (B > 1)
    assert size(2 * first + 16) == size(0)  # no sequence can hold it


def test_header_says_that_prefix_attention_may_round_its_weights(header):
    text = header[header.index("for a batch whose sequences begin with the same prefix_len rows"):]
    text = text[:text.index("tsa_status tsa_prefix_attn")]
    assert "weight to the cache's type" in text and "tsa_paged_attn over the same tables" in text


def test_a_scale_without_a_finite_base_2_logarithm_is_refused(tsa):
    """Scores are scale * log2(e) * <q, k>: with an infinite factor a product of 0 would be NaN."""
    c = shape(tsa, 3, 2, 64)
    c.K, c.V, c.page_table = 0x10000, 0x20000, 0x30000
    a = tsa.tsa_paged_attn_args()
    a.cache = c
    for k, x in dict(Q=0x40000, seq_lens=0x50000, O=0x60000, Hq=8, ws=0x100000, ws_bytes=0).items():
        setattr(a, k, x)
    for name in ("tsa_paged_attn", "tsa_prefix_attn"):
        for scale, status, msg in ((3e38, 1, "scale"), (2.4e38, 1, "scale"), (2.35e38, 3, "needs"), (1e-45, 3, "needs")):
            a.scale = scale
            assert getattr(tsa.lib(), name)(ctypes.byref(a), None) == status and msg in tsa.last_error(), (name, scale)


def test_the_stride_of_a_dimension_of_one_does_not_matter(tsa):
    """One page, or one head: what torch reports as its stride depends on where the tensor came from."""
    import torch

    table = torch.zeros(2, 1, dtype=torch.int32)
    pool = torch.zeros(4, 2, 2, 16, 128, dtype=torch.bfloat16)
    K, V = pool[1:2, 0], torch.zeros(1, 2, 16, 128, dtype=torch.bfloat16)  # one page: strides 8192 and 4096
    assert K.stride(0) != V.stride(0)
    c = tsa.paged_cache(K, V, table)
    assert (c.head_stride, c.row_stride) == (2048, 128)
    K, V = pool[:, 0, :1], torch.zeros(4, 2, 1, 16, 128, dtype=torch.bfloat16)[:, 0]  # one head
    with pytest.raises(tsa.TsaError, match="same strides"):
        tsa.paged_cache(K, V, table)  # (the pages' strides differ: 8192 and 4096)
    size = lambda c: tsa.lib().tsa_paged_workspace_size(ctypes.byref(c), 0, 0)
    c = tsa.paged_cache(pool[:, 0, :1], pool[:, 1, 1:], table)
    assert size(c) == 256


def test_a_prefix_length_past_32_bits_is_refused(tsa):
    """It is not cut to its low 32 bits."""
    import torch

    K, table = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32)
    Q, lens, ws = torch.zeros(2, 4, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32), torch.zeros(1 << 16, dtype=torch.uint8)
    c = tsa.paged_cache(K, K, table)
    for n in (2 ** 32 + 16, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(tsa.TsaError, match="prefix_len"):
            tsa.paged_attn_args(c, Q, lens, Q.clone(), ws, scale=0.1, prefix_len=n)
        with pytest.raises(tsa.TsaError, match="prefix_len"):
            tsa.paged_workspace_size(c, 4, n)
