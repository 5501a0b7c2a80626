"""Scores so large that a 32-bit number has no fraction left for them (needs a B200)."""
import math

import numpy as np
import pytest
import torch

from paged_run import DT, check_attn
from top_sparse_attention_02_b200 import binding as tsa

pytestmark = pytest.mark.gpu


def in_64_bits(Q, K, V, lens, scale):
    """Attention and its log-sum-exp over pages in their order, the same for every sequence."""
    Hkv, n = K.shape[1], K.shape[0] * K.shape[2]
    k, v = (t.transpose(0, 1).reshape(Hkv, n, 128).double() for t in (K, V))
    s = torch.einsum("bhgd,hnd->bhgn", Q.double().view(Q.shape[0], Hkv, -1, 128), k) * scale
    s = s.masked_fill(torch.arange(n, device=s.device) >= lens[:, None, None, None], -math.inf)
    O = torch.einsum("bhgn,hnd->bhgd", torch.softmax(s, -1), v).reshape(Q.shape)
    return O.cpu().numpy(), (torch.logsumexp(s, -1) / math.log(2.0)).reshape(Q.shape[:2]).cpu().numpy()


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("climb", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_finite_scores_of_any_size(cuda_dev, dt, prefix, climb, sign):
    """Logits of 2^e in base 2: whole steps of fp32 apart, and lowered maxima (fp16 weights are formed
    relative to one) that a step of the maximum may round by more than the lowering.  Rows tie with
    the largest or are below it by 2^e / 128 at least, which is 2^13 or more: the result is the
    mean of the tied rows' values, however the logits are rounded."""
    B, Hq, Hkv, page, n = 12, 16, 2, 64, 4160
    g = torch.Generator().manual_seed(sign + 2 * climb)
    K = torch.zeros(n // page, Hkv, page, 128)
    if climb:  # the largest grows (or, for negative queries, falls) in steps of 1/128 along the rows
        K[..., 0] = (1 + (torch.arange(n) // 64) / 128).view(-1, 1, page)
    else:
        K[..., 0] = torch.where(torch.rand(n // page, Hkv, page, generator=g) < 0.3, 1.0, 1.0 - sign / 2)
    V = torch.randn(n // page, Hkv, page, 128, generator=g)
    Q = torch.zeros(B, Hq, 128)
    Q[..., 0] = sign * (1 + 2.0 ** -7)  # a product that has to be rounded
    K, V, Q = (x.to(DT[dt]).to(cuda_dev) for x in (K, V, Q))
    table = torch.arange(n // page, dtype=torch.int32, device=cuda_dev).repeat(B, 1).contiguous()
    lens = [n - 3 * b for b in range(B)]
    P = n - 64 if prefix else 0
    assert not prefix or (B - 1) * P * Hkv >= 81920
    ln = torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    cache = tsa.paged_cache(K, V, table)
    ws = tsa.new_paged_workspace(cache, Hq, P)
    O, lse = torch.empty_like(Q), torch.empty(B, Hq, device=cuda_dev)
    for e in (20, 21, 22, 23, 24, 25, 26, 27, 28, 29, 30, 31, 32, 34, 40, 60, 100):
        scale = float(np.float32(2.0 ** e * 1.00001 / math.log2(math.e)))
        tsa_call = tsa.prefix_attn if prefix else tsa.paged_attn
        tsa_call(tsa.paged_attn_args(cache, Q, ln, O, ws, scale=scale, prefix_len=P, lse=lse))
        tsa.check_device_status(ws)
        want, wl = in_64_bits(Q, K, V, ln, scale)
        # (equal weights of the tied rows: 1 exactly in both types, or 2^12, or one value for all of a pass)
        check_attn(O, want, DT[dt], {"bf16": 8, "fp16": 11}[dt] if prefix else 16, float(V.float().abs().max()), f"2^{e}")
        # the logit's three roundings (scale * log2(e), the sum of products, the product with it) and lse's own
        assert (np.abs(lse.cpu().double().numpy() - wl) <= 5 * 2.0 ** -24 * np.abs(wl) + 2e-4).all(), f"2^{e}"
