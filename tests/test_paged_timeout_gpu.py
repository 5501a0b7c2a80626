"""The paged kernels' bounded waits: a load that never comes is reported as
TSA_ERR_DEVICE_TIMEOUT and the next call works (the test-only build of the
library, whose waits are short and which can leave one load out)."""
import ctypes
import math
import os

import pytest
import torch

import oracle
from paged_run import check_attn, pages, queries
from top_sparse_attention_02_b200 import binding as tsa

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(128)


@pytest.fixture(scope="module")
def dbg():
    path = os.path.join(os.path.dirname(tsa._LIB_PATH), "libtsa_debug.so")
    if not os.path.exists(path):
        from top_sparse_attention_02_b200 import build

        build.build(debug=True)
    lib = ctypes.CDLL(path)  # its own copy of every symbol, separate from libtsa.so
    for name in ("tsa_paged_attn", "tsa_prefix_attn"):
        getattr(lib, name).argtypes = [ctypes.POINTER(tsa.tsa_paged_attn_args), ctypes.c_void_p]
    lib.tsa_check_device_status.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.tsa_debug_paged_skip_tile.argtypes = [ctypes.c_int, ctypes.c_int]
    yield lib
    for which in (0, 1):
        lib.tsa_debug_paged_skip_tile(which, -1)


# few and many rows of one kv-head: the prefix's pass with one row tile and with two
# (P = 4000: 32 tiles in 8 splits, so that CTA 0 has four)
@pytest.mark.parametrize("which,B,Hq,P,tile", [(0, 3, 16, 0, 0), (0, 3, 16, 0, 3), (1, 33, 8, 400, 0), (1, 33, 64, 400, 0),
                                               (1, 33, 64, 4000, 1)])
def test_a_wait_runs_out_then_recovers(dbg, cuda_dev, which, B, Hq, P, tile):
    # (3 x 8 units of 51 granules over 296 CTAs: five of them, 0 to 4, are CTA 0's)
    lens = [P + 300 + i for i in range(B)] if which else [3210 + i for i in range(B)]
    K, V, table = pages(lens, 8, 64, torch.bfloat16, seed=1, shared=P, dev=cuda_dev)
    Q = queries(B, Hq, torch.bfloat16, dev=cuda_dev)
    cache = tsa.paged_cache(K, V, table)
    ws = tsa.new_paged_workspace(cache, Hq, P)
    O = torch.zeros_like(Q)
    ln = torch.tensor(lens, dtype=torch.int32, device=cuda_dev)
    a = tsa.paged_attn_args(cache, Q, ln, O, ws, scale=SCALE, prefix_len=P)
    name = "tsa_prefix_attn" if which else "tsa_paged_attn"
    call = lambda lib: getattr(lib, name)(ctypes.byref(a), torch.cuda.current_stream().cuda_stream)
    assert dbg.tsa_debug_paged_skip_tile(which, tile) == 0
    assert call(dbg) == 0
    assert dbg.tsa_check_device_status(ws.data_ptr(), None) == tsa.TSA_ERR_DEVICE_TIMEOUT
    assert dbg.tsa_debug_paged_skip_tile(which, -1) == 0
    (tsa.prefix_attn if which else tsa.paged_attn)(a)  # the product library, the same workspace
    tsa.check_device_status(ws)
    want, _ = oracle.paged_attn(Q, K.cpu(), V.cpu(), table.cpu(), lens, SCALE)
    check_attn(O, want, torch.bfloat16, 8 if which else 16, float(torch.nan_to_num(V.float()).abs().max()))
