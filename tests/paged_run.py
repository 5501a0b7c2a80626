"""Builds paged caches for the tests, and holds the tolerances of what comes out of them."""
from __future__ import annotations

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dtype) -> float:
    """A rounding to dtype is off by at most this much of the value."""
    return torch.finfo(dtype).eps / 2


def pages(lens, Hkv, page, dtype, order="head", seed=0, shared=0, spare=2, fill=float("nan"), width=None, dev="cpu"):
    """K and V pages with the rows of len(lens) sequences drawn N(0, 1), everything else (rows
    past the sequences, pages nobody holds) set to `fill`; pages in a random order; the
    rows [0, shared) the same for each sequence that has them.  Returns K, V
    [P, Hkv, page, 128] and the table [B, width] with -1 in the entries nobody reads."""
    g = torch.Generator()
    g.manual_seed(seed)
    npg = [-(-n // page) for n in lens]
    full = shared // page
    own = [n - full if lens[b] >= shared else n for b, n in enumerate(npg)]
    P = full + sum(own) + spare
    width = width or max(1, max(npg, default=0)) + 1
    perm = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    pool = []
    for _ in range(2):
        shape = (P, Hkv, page, 128) if order == "head" else (P, page, Hkv, 128)
        t = torch.full(shape, fill, dtype=dtype)
        pool.append(t if order == "head" else t.permute(0, 2, 1, 3))
    at = full
    for b, n in enumerate(npg):
        c = full if lens[b] >= shared else 0
        table[b, :c] = perm[:c]
        table[b, c:n] = perm[at:at + n - c]
        at += n - c
    common = [torch.randn(shared, Hkv, 128, generator=g).to(dtype) for _ in range(2)]
    for b, n in enumerate(lens):
        rows = torch.arange(n)
        pg, off = table[b][rows // page].long(), rows % page
        for t, c in zip(pool, common):
            x = torch.randn(n, Hkv, 128, generator=g).to(dtype)
            if shared and n >= shared:
                x[:shared] = c
            t[pg, :, off] = x
    # (a permuted pool keeps its strides on the device)
    out = [t.to(dev) if order == "head" else t.permute(0, 2, 1, 3).contiguous().to(dev).permute(0, 2, 1, 3) for t in pool]
    return out[0], out[1], table.to(dev)


def queries(B, Hq, dtype, seed=0, dev="cpu"):
    g = torch.Generator()
    g.manual_seed(1000 + seed)
    return torch.randn(B, Hq, 128, generator=g).to(dtype).to(dev)


def random_rows(lens, Hkv, k, seed=0):
    """Index lists as a selecting layer writes them: ascending distinct rows, then -1."""
    rng = np.random.default_rng(seed)
    idx = np.full((len(lens), Hkv, k), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            m = min(k, n)
            idx[b, h, :m] = np.sort(rng.choice(n, m, replace=False)) if m else []
    return idx


def check_attn(O, want, dtype, weight_bits, vmax, what=""):
    """|O - want| <= half a step of the output's rounding of want, plus the weights' error.

    Each weight p_j / sum(p) is off by a relative e at most: its rounding to
    `weight_bits` bits (2^-weight_bits), the 2^-21 of exp2 and the 2^-16 that an error of
    1e-5 in a logit makes (a sum of 128 exact products in fp32: |logit| < 16, so
    128 * 2^-24 * 16 = 1.2e-4 at worst, sqrt(128) of that as a random walk).  The output is
    a mean of values of magnitude vmax, so it is off by 2 e vmax at most (the weights
    in the numerator, and their sum below it)."""
    got, want = O.detach().cpu().double().numpy(), np.asarray(want)
    assert got.shape == want.shape and np.isfinite(got).all(), f"{what}: shape or non-finite output"
    e = 2.0 ** -weight_bits + 2.0 ** -21 + 2.0 ** -16
    tol = half_step(dtype) * np.abs(want) + 2 * e * vmax + torch.finfo(dtype).tiny
    err = np.abs(got - want)
    assert (err <= tol).all(), f"{what}: off by {(err / tol).max():.2f} of the tolerance, {err.max():.3e} at most"


def check_lse(lse, want, what=""):
    """Logits are within 1.2e-4 * log2(e) at worst (see check_attn); a sum of weights within 2^-20."""
    got = lse.detach().cpu().double().numpy()
    empty = np.isneginf(want)
    assert np.isneginf(got[empty]).all(), f"{what}: a sequence without a row has lse -inf"
    assert np.abs(got[~empty] - want[~empty]).max(initial=0.0) <= 2e-4, what


def norm_tolerance(dtype, coarse_weights: bool) -> float:
    """What the error of a row of O may be, relative to the row, both as norms over its 128 elements.

    The output's rounding is off by half a step h of a value at most, h / sqrt(3) as a root mean square
    (evenly spread over the step).  A weight's rounding, e_j <= h where a pass keeps the weights in
    the element type, makes the error sum_j p_j e_j (v_j - O): with independent e_j and values of one
    size its norm is the root mean square of e_j times |O|, h / sqrt(3) again; with 16 bits and more
    it does not count.  The squares add up.  1.3: such a norm over 128 elements, or over the 100
    rows and more that carry the weight, strays by 8 to 10% of its square, 4 times that at most
    (over all rows of all tests); sums and logits in 32 bits (1e-5) lie in it too."""
    return 1.3 * half_step(dtype) / np.sqrt(3.0) * np.sqrt(2.0 if coarse_weights else 1.0)


def check_norm(O, want, lens, dtype, coarse_weights: bool, what=""):
    """Each row of O [B, Hq, d] is within norm_tolerance of `want`, for sequences of 300 rows and more
    (shorter ones: check_attn).  A bound by the largest value, as check_attn's, is as large as the
    outputs themselves over thousands of rows."""
    got, want = O.detach().cpu().double().numpy(), np.asarray(want)
    long = np.asarray(lens) >= 300
    assert long.any() and np.isfinite(got).all(), f"{what}: nothing to check, or non-finite output"
    err = np.linalg.norm((got - want)[long], axis=-1) / np.linalg.norm(want[long], axis=-1)
    tol = norm_tolerance(dtype, coarse_weights)
    assert (err <= tol).all(), f"{what}: a row is off by {err.max():.2e} of its norm, allowed {tol:.2e}"
