"""Calls of the paged path one behind the other, each started while the one before still runs (needs a B200)."""
import pytest
import torch

from top_sparse_attention_02_b200 import binding as tsa

pytestmark = pytest.mark.gpu


def test_positions_and_rows_that_the_kernel_before_writes(cuda_dev):
    """A top-k writes the positions (and rows) that the norm and the append behind it read, forty
    times in a row: the same bits as with every call on its own."""
    n, k, H, page, steps = 4096, 300, 4, 32, 40
    g = torch.Generator().manual_seed(0)
    scores = torch.randn(steps, 1, 1, n, generator=g).to(cuda_dev)
    shape = tsa.tsa_shape(1, H, 1, n, 128)
    lens = torch.tensor([n], dtype=torch.int32, device=cuda_dev)
    sws = tsa.new_workspace(shape, k, 1, tsa.SELECT, cuda_dev)
    idx = torch.zeros(1, 1, k, dtype=torch.int32, device=cuda_dev)  # written again by every step
    flat = idx.view(k)
    x = torch.randn(k, H, 128, generator=g).to(torch.bfloat16).to(cuda_dev)
    f = (10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).to(cuda_dev)
    seq = torch.zeros(k, dtype=torch.int32, device=cuda_dev)
    table = torch.randperm(n // page, generator=g).to(torch.int32).view(1, -1).to(cuda_dev)

    def buffers():
        out = [torch.zeros_like(x) for _ in range(steps)]
        pools = [torch.zeros(2, n // page, H, page, 128, dtype=torch.bfloat16, device=cuda_dev) for _ in range(steps)]
        calls, ws = [], None
        for o, (K, V) in zip(out, pools):
            cache = tsa.paged_cache(K, V, table)
            ws = tsa.new_paged_workspace(cache) if ws is None else ws
            calls.append((tsa.qk_norm_rope_args(x, None, o, None, positions=flat, inv_freq=f),
                          tsa.paged_append_args(cache, x, x, flat, ws, seq=seq, inv_freq=f)))
        return out, pools, calls, ws

    got, want = buffers(), buffers()
    torch.cuda.synchronize()
    for s, (norm, app) in zip(scores, got[2]):
        tsa.topk_select(s, lens, None, k, shape, 1, idx, sws)
        tsa.qk_norm_rope(norm)
        tsa.topk_select(s, lens, None, k, shape, 1, idx, sws)
        tsa.paged_append(app)
    for s, (norm, app) in zip(scores, want[2]):
        for call in (lambda: tsa.qk_norm_rope(norm), lambda: tsa.paged_append(app)):
            tsa.topk_select(s, lens, None, k, shape, 1, idx, sws)
            torch.cuda.synchronize()
            call()
            torch.cuda.synchronize()
    for ws in (sws, got[3], want[3]):
        tsa.check_device_status(ws)
    for a, b in zip(got[0] + got[1], want[0] + want[1]):
        assert torch.equal(a, b)
    assert len({o.sum().item() for o in got[0]}) > steps // 2  # (the steps differ)


def test_prefix_calls_and_decode_steps_at_once(cuda_dev):
    """Two shared-prefix calls and a SELECT step (all of them use tensor memory) on a stream each, over
    and over: the bits of each on its own."""
    from paged_run import pages, queries

    P, calls = 1024, []
    for i, (B, Hq) in enumerate(((14, 32), (40, 16))):
        lens = [P + 11 * b for b in range(B)]
        K, V, table = pages(lens, 8, 64, torch.bfloat16, seed=i, shared=P, dev=cuda_dev)
        cache = tsa.paged_cache(K, V, table)
        Q = queries(B, Hq, torch.bfloat16, seed=i, dev=cuda_dev)
        ws = tsa.new_paged_workspace(cache, Hq, P)
        a = tsa.paged_attn_args(cache, Q, torch.tensor(lens, dtype=torch.int32, device=cuda_dev), torch.empty_like(Q), ws,
                                scale=128 ** -0.5, prefix_len=P)
        calls.append((lambda s, a=a: tsa.prefix_attn(a, stream=s), a._tensors[3], ws))
    g = torch.Generator().manual_seed(5)
    K, V = (torch.randn(2, 8, 8192, 128, generator=g).to(torch.bfloat16).to(cuda_dev) for _ in range(2))
    Q = queries(2, 32, torch.bfloat16, dev=cuda_dev)
    ws = tsa.new_workspace(tsa.shape_of(Q, K), 200, 1, tsa.SELECT, cuda_dev)
    O = torch.empty(2, 32, 128, device=cuda_dev)
    idx = torch.empty(2, 8, 200, dtype=torch.int32, device=cuda_dev)
    rows = torch.tensor([8192, 5000], dtype=torch.int32, device=cuda_dev)  # (step_args keeps no tensor alive)
    step = tsa.step_args(Q, K, V, rows, O, ws, mode=tsa.SELECT, scale=128 ** -0.5, k_max=200, idx_out=idx)
    calls.append((lambda s: tsa.decode_step(step, stream=s), O, ws))
    want = []
    for call, out, _ in calls:
        call(None)
        torch.cuda.synchronize()
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(30):
        for (call, _, _), s in zip(calls, streams):
            call(s)
    torch.cuda.synchronize()
    for (_, out, ws), w in zip(calls, want):
        tsa.check_device_status(ws)
        assert torch.equal(out, w)
