"""The check of the paged attention's values finds what it is there to find: mistakes planted in the oracle."""
import math

import numpy as np
import pytest
import torch

import oracle
from paged_run import DT, check_norm, half_step, norm_tolerance, pages, queries

SCALE = 1 / math.sqrt(128)


def rounded(x, dt):
    return torch.from_numpy(np.asarray(x)).to(DT[dt])


def coarse(Q, K, V, table, lens, dt):
    """The oracle with each weight rounded to the element type, as a pass over a shared prefix has them."""
    B, Hq, d = Q.shape
    Hkv = K.shape[1]
    O = np.zeros((B, Hq, d))
    for b, n in enumerate(lens):
        k, v = (oracle.paged_rows(t, table, b, range(n)) for t in (K, V))
        for h in range(Hq):
            s = (Q[b, h].double().numpy() @ k[h * Hkv // Hq].T) * SCALE
            p = np.exp(s - s.max())
            O[b, h] = torch.from_numpy(p).to(DT[dt]).double().numpy() @ v[h * Hkv // Hq] / p.sum()
    return O


# the long cases of the shared prefix's GPU tests, two sequences of each
CASES = [(32, 2, 256, 5200, [5200, 5240]), (8, 1, 16, 2200, [2200, 2239]), (28, 4, 48, 1007, [1007, 1020]), (4, 1, 32, 290, [300, 301])]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("Hq,Hkv,page,prefix,lens", CASES)
def test_lost_values_are_found(dt, Hq, Hkv, page, prefix, lens):
    K, V, table = pages(lens, Hkv, page, DT[dt], seed=prefix, shared=min(prefix, min(lens)))
    K, V = torch.nan_to_num(K), torch.nan_to_num(V)
    Q = queries(len(lens), Hq, DT[dt])
    want, _ = oracle.paged_attn(Q, K, V, table, lens, SCALE)
    check_norm(rounded(want, dt), want, lens, DT[dt], False)
    check_norm(rounded(coarse(Q, K, V, table, lens, dt), dt), want, lens, DT[dt], True)

    def with_v(change):
        v = V.clone()
        for b in range(len(lens)):
            change(v, b)
        return oracle.paged_attn(Q, K, v, table, lens, SCALE)[0]

    def lose(first, last):
        def change(v, b):
            for r in range(first, min(last, lens[b])):
                v[int(table[b, r // page]), :, r % page] = 0
        return change

    at = min(256, prefix - 160)
    faults = {"a tile of V": with_v(lose(at, at + 128)), "a box of V": with_v(lose(at, at + 16)),
              "one row of V": with_v(lose(at, at + 1)),
              "the last five rows": oracle.paged_attn(Q, K, V, table, [n - 5 for n in lens], SCALE)[0],
              "a hundredth too much": want * 1.01}
    for name, got in faults.items():
        with pytest.raises(AssertionError):
            check_norm(rounded(got, dt), want, lens, DT[dt], True)
            pytest.fail(f"{name}: not found")


def test_tolerance_is_a_few_thousandths_in_bf16():
    assert norm_tolerance(torch.bfloat16, True) < 4.3e-3 and norm_tolerance(torch.bfloat16, False) < 3e-3
    assert norm_tolerance(torch.float16, True) == norm_tolerance(torch.bfloat16, True) / 8
    assert half_step(torch.bfloat16) == 2.0 ** -8


def test_check_wants_something_to_check():
    with pytest.raises(AssertionError, match="nothing"):
        check_norm(torch.zeros(1, 1, 128), np.zeros((1, 1, 128)), [20], torch.bfloat16, False)
