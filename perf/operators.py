"""The paged decode path's operators as a user's program calls them, on real shapes.

Four operators around a paged key-value cache:

``norm_rope``    the RMS norm of each query and key head, then the position rotation
``append``       new keys (rotated on the way) and values into the pages
``paged_attn``   one decode token per sequence over its pages: every row, or selected rows
``prefix_attn``  the same for a batch whose sequences share a long prefix, read once for all

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, angles in 64, one rounding at the end) or, where ``own`` is true, makes
the framework's call.  ``exact`` computes it from the definition in 64 bits.

Definitions.  Head dimension d = 128.
  norm       y = x / sqrt(mean(x^2) + eps) * w                         (a head at a time)
  rotation   the first ``rot`` elements in pairs (i, i + rot/2), or (2i, 2i + 1) when
             interleaved: (a, b) -> (a cos t - b sin t, b cos t + a sin t), t = position * inv_freq[i]
  attention  O = sum_j p_j v_j,  p = softmax_j(scale * q . k_j), 0 for a sequence with no row;
             lse = log2(sum_j exp(scale * q . k_j))
The pages are [num_pages, Hkv, page_size, d]; row j of sequence b lies in page
table[b, j // page_size] at j % page_size.
"""
from __future__ import annotations

import math

import torch

own = False

D = 128
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one stream: a call's latency is all there is
        dict(name="norm_rope_one_token", op="norm_rope", T=1, Hq=8, Hkv=2, rot=128, interleaved=False, fused=True,
             norm=True, far=131072, dtype="bf16"),
        # a prompt's chunk out of a fused projection
        dict(name="norm_rope_prompt", op="norm_rope", T=8192, Hq=32, Hkv=8, rot=128, interleaved=False, fused=True,
             norm=True, far=131072, dtype="bf16"),
        # an odd number of tokens, half of each head rotated, neighbours paired
        dict(name="norm_rope_ragged_interleaved", op="norm_rope", T=4099, Hq=64, Hkv=8, rot=64, interleaved=True,
             fused=False, norm=True, far=1 << 20, dtype="fp16"),
        # a decode step of a large batch: one token a sequence
        dict(name="append_decode", op="append", B=64, new=1, lo=0, hi=1024, Hkv=8, page=16, order="head",
             rot=128, interleaved=False, dtype="bf16"),
        # prompts' chunks of odd lengths, pages token by token, half of each head rotated
        dict(name="append_prompts", op="append", B=8, new=2047, lo=0, hi=4096, Hkv=8, page=128, order="row", rot=64,
             interleaved=True, dtype="fp16"),
        # the smallest decode step
        dict(name="paged_attn_one_stream", op="paged_attn", B=1, Hq=8, Hkv=2, lo=4096, hi=4096, page=16,
             order="head", k=0, lse=False, dtype="bf16"),
        # a layer that reuses an earlier layer's selected rows at a long context
        dict(name="paged_attn_selected_rows", op="paged_attn", B=1, Hq=32, Hkv=8, lo=131072, hi=131072, page=64,
             order="head", k=2621, lse=False, dtype="bf16"),
        # ordinary serving: ragged lengths, a group of 5, pages token by token
        dict(name="paged_attn_ragged", op="paged_attn", B=17, Hq=40, Hkv=8, lo=1, hi=6001, page=48, order="row",
             k=0, lse=True, dtype="fp16"),
        # the largest: every row of a large batch
        dict(name="paged_attn_large_batch", op="paged_attn", B=64, Hq=64, Hkv=8, lo=8192, hi=32768, page=64,
             order="head", k=0, lse=False, dtype="bf16"),
        # a few streams over one system prompt
        dict(name="prefix_attn_few_streams", op="prefix_attn", B=8, Hq=32, Hkv=8, prefix=4096, tail_lo=1, tail_hi=512, short=0,
             page=16, order="head", lse=False, dtype="bf16"),
        # an odd prefix that ends inside a page, a group of 7, some sequences without the whole prefix
        dict(name="prefix_attn_ragged", op="prefix_attn", B=33, Hq=28, Hkv=4, prefix=10007, tail_lo=1, tail_hi=1500, short=2,
             page=32, order="row", lse=False, dtype="fp16"),
        # a large batch over a long document
        dict(name="prefix_attn_large_batch", op="prefix_attn", B=64, Hq=64, Hkv=8, prefix=32768, tail_lo=1, tail_hi=2048,
             short=0, page=128, order="head", lse=True, dtype="bf16"),
    ]


HEADS = [(8, 2), (32, 8), (64, 8), (8, 8), (28, 4), (40, 8), (5, 1), (16, 1), (24, 8), (12, 6)]
PAGES = [16, 32, 48, 64, 128, 256]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "paged_attn", "paged_attn", "prefix_attn", "prefix_attn"])
    Hq, Hkv = rng.choice(HEADS)
    case = dict(op=op, Hkv=Hkv, dtype=rng.choice(["bf16", "fp16"]))
    if op in ("norm_rope", "append"):
        case.update(rot=rng.choice([128, 128, 64, 32, 96]), interleaved=rng.random() < 0.4)
    if op == "norm_rope":
        case.update(Hq=Hq, T=_log_uniform(rng, 1, 8192), fused=rng.random() < 0.5, norm=rng.random() < 0.8,
                    far=_log_uniform(rng, 1024, 1 << 20))
        return case
    case.update(page=rng.choice(PAGES), order=rng.choice(["head", "head", "row"]))
    if op == "append":
        B = _log_uniform(rng, 1, 128)
        case.update(B=B, new=_log_uniform(rng, 1, max(1, 16384 // B)), lo=0,
                    hi=_log_uniform(rng, 1, min(8192, 500000 // (B * Hkv))))
        return case
    case.update(Hq=Hq, B=_log_uniform(rng, 1, 64))
    if op == "paged_attn":
        top = _log_uniform(rng, 1, min(131072, 10000000 // (case["B"] * Hkv)))
        case.update(lo=rng.choice([0, 1, top // 2, top]), hi=top)
        case.update(k=_log_uniform(rng, 1, max(1, top // 4)) if rng.random() < 0.4 else 0,
                    lse=case["lo"] > 0 and rng.random() < 0.5)
        return case
    case.update(prefix=_log_uniform(rng, 64, 32768), tail_lo=rng.choice([0, 1]), tail_hi=_log_uniform(rng, 1, 2048),
                short=rng.choice([0, 0, 1]), lse=False)
    return case


# ------------------------------------------------------------------ inputs

def _inv_freq(rot, device):
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=device)
    return 500000.0 ** (-i / rot)


def _pool(P, case, g, dev):
    """K and V pages, [P, Hkv, page, D], laid out head by head or token by token in each page."""
    dt = DTYPES[case["dtype"]]
    shape = (P, case["Hkv"], case["page"], D) if case["order"] == "head" else (P, case["page"], case["Hkv"], D)
    out = [torch.empty(shape, dtype=dt, device=dev).normal_(generator=g) for _ in range(2)]
    return [t if case["order"] == "head" else t.permute(0, 2, 1, 3) for t in out]


def _lens(case):
    """Ragged lengths, a property of the case: its inputs have the same shapes whatever the seed."""
    lo, hi = case["lo"], case["hi"]
    gl = torch.Generator()
    gl.manual_seed(case["B"] + hi)
    lens = torch.randint(lo, hi + 1, (case["B"],), generator=gl)
    if case["B"] > 2 and lo < hi:
        lens[0], lens[-1] = hi, lo
    return lens.tolist()


def _table(lens, page, gc, shared=0, slack=3):
    """Pages in a random order; sequences of at least ``shared`` rows share the pages that hold only those."""
    npg = [-(-n // page) for n in lens]
    width = max(1, max(npg)) + 1
    common = shared // page
    own_pages = [n - common if lens[b] >= shared else n for b, n in enumerate(npg)]
    P = common + sum(own_pages) + slack
    perm = torch.randperm(P, generator=gc)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = common
    for b, n in enumerate(npg):
        c = common if lens[b] >= shared else 0
        table[b, :c] = perm[:c].to(torch.int32)
        table[b, c:n] = perm[at:at + n - c].to(torch.int32)
        at += n - c
    return table, P


def _plant(Kp, Q, lens, table, case, g, gc):
    """One row in a hundred is drawn towards one of its group's queries: real attention has heavy keys."""
    Hkv, page = case["Hkv"], case["page"]
    grp = Q.shape[1] // Hkv
    for b, n in enumerate(lens):
        c = n // 100
        if c == 0:
            continue
        rows = torch.randperm(n, generator=gc)[:c].to(Kp.device)
        pages = table[b].to(Kp.device)[rows // page].long()
        pick = torch.randint(0, grp, (Hkv, c), generator=gc).to(Kp.device) + \
            torch.arange(Hkv, device=Kp.device)[:, None] * grp
        q = Q[b].float()[pick.t()]  # [c, Hkv, D]
        new = 3.0 * q / q.norm(dim=-1, keepdim=True) + torch.randn(q.shape, generator=g, device=Kp.device)
        Kp[pages, :, rows % page] = new.to(Kp.dtype)


def _inputs(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    gc = torch.Generator()
    gc.manual_seed(seed + 1)
    dt = DTYPES[case["dtype"]]
    Hkv = case["Hkv"]

    def normal(*shape):
        return torch.empty(shape, dtype=dt, device=dev).normal_(generator=g)

    s = dict(case=case)
    if case["op"] == "norm_rope":
        T, Hq = case["T"], case["Hq"]
        if case["fused"]:  # one projection's output: queries, keys and values side by side
            qkv = normal(T, Hq + 2 * Hkv, D) * 2.0
            s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        else:
            s["q"], s["k"] = normal(T, Hq, D), normal(T, Hkv, D)
        s["positions"] = torch.randint(0, case["far"], (T,), generator=gc).to(torch.int32).to(dev)
        s["inv_freq"] = _inv_freq(case["rot"], dev)
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=dev)
            s["k_weight"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=dev)
        return s
    if case["op"] == "append":
        B, new, page = case["B"], case["new"], case["page"]
        before = _lens(case)
        count = [new - b % (new // 2 + 1) for b in range(B)]  # ragged, half of the longest at least
        table, P = _table([n + c for n, c in zip(before, count)], page, gc)
        s["Kp"], s["Vp"] = _pool(P, case, g, dev)
        seq = torch.repeat_interleave(torch.arange(B), torch.tensor(count))
        row = torch.cat([torch.arange(n, n + c) for n, c in zip(before, count)])
        T = row.numel()
        kv = normal(T, 2 * Hkv, D)
        s["k"], s["v"] = kv[:, :Hkv], kv[:, Hkv:]
        s["seq"], s["row"] = seq.to(torch.int32).to(dev), row.to(torch.int32).to(dev)
        s["inv_freq"] = _inv_freq(case["rot"], dev)
        s["table"] = table.to(dev)
        return s
    B, Hq = case["B"], case["Hq"]
    shared = 0
    if case["op"] == "prefix_attn":
        shared = case["prefix"]
        lens = [n + shared for n in _lens(dict(B=B, lo=case["tail_lo"], hi=case["tail_hi"]))]
        for i in range(min(case["short"], B - 1)):  # sequences that stop inside the prefix, the first one empty
            lens[i] = 0 if i == 0 else shared // 2
    else:
        lens = _lens(case)
    table, P = _table(lens, case["page"], gc, shared)
    s["Kp"], s["Vp"] = _pool(P, case, g, dev)
    s["Q"] = normal(B, Hq, D)
    _plant(s["Kp"], s["Q"], lens, table, case, g, gc)
    whole = [b for b, n in enumerate(lens) if n >= shared]
    if shared % case["page"] and whole:  # the page in which the prefix ends: a copy for each sequence
        first, part = int(table[whole[0], shared // case["page"]]), shared % case["page"]
        for b in whole[1:]:
            for t in (s["Kp"], s["Vp"]):
                t[int(table[b, shared // case["page"]]), :, :part] = t[first, :, :part]
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["lens_host"] = lens
    s["table"] = table.to(dev)
    s["idx"] = None
    if case.get("k", 0) > 0:  # ascending distinct rows, then -1, as a selecting layer writes them
        k = case["k"]
        idx = torch.full((B, Hkv, k), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            for h in range(Hkv):
                m = min(k, n)
                idx[b, h, :m] = torch.randperm(n, generator=gc)[:m].sort().values.to(torch.int32)
        s["idx"] = idx.to(dev)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    from top_sparse_attention_02_b200 import binding as tsa

    if case["op"] == "norm_rope":
        s["q_out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=s["q"].device)
        s["k_out"] = torch.empty(s["k"].shape, dtype=s["k"].dtype, device=s["k"].device)
        s["args"] = tsa.qk_norm_rope_args(s["q"], s["k"], s["q_out"], s["k_out"], q_weight=s["q_weight"],
                                          k_weight=s["k_weight"], eps=EPS, positions=s["positions"],
                                          inv_freq=s["inv_freq"], interleaved=case["interleaved"])
        return s
    cache = tsa.paged_cache(s["Kp"], s["Vp"], s["table"])
    if case["op"] == "append":
        s["ws"] = tsa.new_paged_workspace(cache)
        s["args"] = tsa.paged_append_args(cache, s["k"], s["v"], s["row"], s["ws"], seq=s["seq"],
                                          inv_freq=s["inv_freq"], interleaved=case["interleaved"])
        return s
    prefix = case.get("prefix", 0)
    s["ws"] = tsa.new_paged_workspace(cache, case["Hq"], prefix_len=prefix)
    s["O"] = torch.empty_like(s["Q"])
    s["lse"] = torch.empty(s["Q"].shape[:2], dtype=torch.float32, device=s["Q"].device) if case["lse"] else None
    s["args"] = tsa.paged_attn_args(cache, s["Q"], s["lens"], s["O"], s["ws"], scale=D ** -0.5, idx=s["idx"],
                                    prefix_len=prefix, lse=s["lse"])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    if op == "norm_rope":
        return _plain_norm_rope(state)
    if op == "append":
        return _plain_append(state)
    if op == "paged_attn":
        return _plain_paged(state)
    return _plain_prefix(state)


def _run_own(s, op):
    from top_sparse_attention_02_b200 import binding as tsa

    if op == "norm_rope":
        tsa.qk_norm_rope(s["args"])
        return s["q_out"], s["k_out"]
    if op == "append":
        tsa.paged_append(s["args"])
        return s["Kp"], s["Vp"]
    (tsa.paged_attn if op == "paged_attn" else tsa.prefix_attn)(s["args"])
    return (s["O"], s["lse"]) if s["lse"] is not None else s["O"]


def _rotate(x, positions, inv_freq, interleaved):
    """x [T, H, D] in 32 bits: its first 2 * len(inv_freq) elements rotated."""
    half = inv_freq.numel()
    ang = positions.double()[:, None] * inv_freq[None, :]
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2] = a * cos - b * sin
        y[..., 1:2 * half:2] = b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half] = a * cos - b * sin
        y[..., half:2 * half] = b * cos + a * sin
    return y


def _plain_norm_rope(s):
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        f = x.float()
        if w is not None:
            f = f / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS) * w
        out.append(_rotate(f, s["positions"], s["inv_freq"], s["case"]["interleaved"]).to(x.dtype))
    return tuple(out)


def _plain_append(s):
    page = s["case"]["page"]
    k = _rotate(s["k"].float(), s["row"], s["inv_freq"], s["case"]["interleaved"]).to(s["k"].dtype)
    row = s["row"].long()
    pages = s["table"][s["seq"].long(), row // page].long()
    s["Kp"][pages, :, row % page] = k
    s["Vp"][pages, :, row % page] = s["v"]
    return s["Kp"], s["Vp"]


def _gather(s, b, h, rows):
    """Rows of sequence b out of the pages, in 32 bits: K, V [n, D] of kv-head h (every head if None)."""
    page = s["case"]["page"]
    rows = rows.long()
    pages, off = s["table"][b, rows // page].long(), rows % page
    if h is not None:
        return s["Kp"][pages, h, off].float(), s["Vp"][pages, h, off].float()
    return s["Kp"][pages, :, off].float().transpose(0, 1), s["Vp"][pages, :, off].float().transpose(0, 1)


def _softmax_parts(q, K, V):
    """q [.., g, D], K, V [.., n, D] -> the row maximum, the sum of exp(s - max) and its product with V."""
    sc = torch.matmul(q, K.transpose(-1, -2)) * D ** -0.5
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m)
    return m, p.sum(-1, keepdim=True), torch.matmul(p, V)


def _log2e(x):
    return x * 1.4426950408889634


def _plain_paged(s):
    case, Q = s["case"], s["Q"]
    Hkv = case["Hkv"]
    O = torch.zeros(Q.shape, dtype=torch.float32, device=Q.device)
    lse = torch.full(Q.shape[:2], float("-inf"), dtype=torch.float32, device=Q.device)
    for b, n in enumerate(s["lens_host"]):
        if n == 0:
            continue
        q = Q[b].float().view(Hkv, -1, D)
        if s["idx"] is None:
            K, V = _gather(s, b, None, torch.arange(n, device=Q.device))
        else:
            rows = s["idx"][b, :, :min(n, case["k"])]
            kv = [_gather(s, b, h, rows[h]) for h in range(Hkv)]
            K, V = torch.stack([x[0] for x in kv]), torch.stack([x[1] for x in kv])
        m, l, o = _softmax_parts(q, K, V)
        O[b] = (o / l).reshape(-1, D)
        lse[b] = _log2e(m + torch.log(l)).reshape(-1)
    return (O.to(Q.dtype), lse) if case["lse"] else O.to(Q.dtype)


def _plain_prefix(s):
    case, Q = s["case"], s["Q"]
    B, Hkv, pre = Q.shape[0], case["Hkv"], case["prefix"]
    g = Q.shape[1] // Hkv
    O = torch.zeros(Q.shape, dtype=torch.float32, device=Q.device)
    lse = torch.full(Q.shape[:2], float("-inf"), dtype=torch.float32, device=Q.device)
    whole = [b for b, n in enumerate(s["lens_host"]) if n >= pre]
    if whole:  # the prefix, read once for every sequence that has it
        K, V = _gather(s, whole[0], None, torch.arange(pre, device=Q.device))
        q = Q.float().view(B, Hkv, g, D).transpose(0, 1).reshape(Hkv, B * g, D)
        pm, pl, po = (x.view(Hkv, B, g, -1) for x in _softmax_parts(q, K, V))
    for b, n in enumerate(s["lens_host"]):
        if n == 0:
            continue
        start = pre if n >= pre else 0
        q = Q[b].float().view(Hkv, g, D)
        parts = [(pm[:, b], pl[:, b], po[:, b])] if start else []
        if n > start:
            parts.append(_softmax_parts(q, *_gather(s, b, None, torch.arange(start, n, device=Q.device))))
        m = torch.stack([p[0] for p in parts]).amax(0)
        l = sum(torch.exp(p[0] - m) * p[1] for p in parts)
        o = sum(torch.exp(p[0] - m) * p[2] for p in parts)
        O[b] = (o / l).reshape(-1, D)
        lse[b] = _log2e(m + torch.log(l)).reshape(-1)
    return (O.to(Q.dtype), lse) if case["lse"] else O.to(Q.dtype)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    elem = 2
    if case["op"] == "norm_rope":
        heads = case["T"] * (case["Hq"] + case["Hkv"])
        return dict(bytes=heads * D * elem * 2 + case["T"] * 4, flops=heads * (6 * D if case["norm"] else 3 * D))
    if case["op"] == "append":
        tokens = sum(case["new"] - b % (case["new"] // 2 + 1) for b in range(case["B"]))
        return dict(bytes=tokens * (case["Hkv"] * D * elem * 4 + 8), flops=tokens * case["Hkv"] * 3 * case["rot"])
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    qo = 2 * B * Hq * D * elem
    if case["op"] == "paged_attn":
        rows = B * (case["lo"] + case["hi"]) / 2
        if case["k"]:
            rows = min(rows, B * case["k"])
            return dict(bytes=int(rows * Hkv * (2 * D * elem + 4) + qo), flops=int(4 * D * Hq * rows))
        return dict(bytes=int(rows * (Hkv * 2 * D * elem + 4 / case["page"]) + qo), flops=int(4 * D * Hq * rows))
    tails = B * (case["tail_lo"] + case["tail_hi"]) / 2
    rows = case["prefix"] + tails
    return dict(bytes=int(rows * Hkv * 2 * D * elem + qo), flops=int(4 * D * Hq * (B * case["prefix"] + tails)))


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_rotation(x, positions, inv_freq, interleaved):
    """x [T, H, D] float64, through complex numbers: the pair (a, b) times e^{i t}."""
    half = inv_freq.numel()
    turn = torch.polar(torch.ones(positions.numel(), half, dtype=torch.float64, device=x.device),
                       positions.to(torch.float64)[:, None] * inv_freq)[:, None]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    pairs = head.unflatten(-1, (half, 2)) if interleaved else head.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, rest], -1)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "norm_rope":
        out = []
        for name in ("q", "k"):
            x, w = s[name].to(torch.float64), s[name + "_weight"]
            if w is not None:
                x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.to(torch.float64)
            out.append(_exact_rotation(x, s["positions"], s["inv_freq"], case["interleaved"]))
        return tuple(out)
    page = case["page"]
    if case["op"] == "append":
        k = _exact_rotation(s["k"].to(torch.float64), s["row"], s["inv_freq"], case["interleaved"])
        Kp, Vp = s["Kp"].to(torch.float64), s["Vp"].to(torch.float64)
        row, seq = s["row"].long(), s["seq"].long()
        flat = s["table"].flatten()[seq * s["table"].shape[1] + torch.div(row, page, rounding_mode="floor")].long()
        Kp.transpose(1, 2)[flat, row.remainder(page)] = k
        Vp.transpose(1, 2)[flat, row.remainder(page)] = s["v"].to(torch.float64)
        return Kp, Vp
    Q = s["Q"].to(torch.float64)
    B, Hq = Q.shape[:2]
    Hkv = case["Hkv"]
    O, lse = torch.zeros_like(Q), torch.full((B, Hq), -math.inf, dtype=torch.float64, device=Q.device)
    for b in range(B):
        n = s["lens_host"][b]
        if n == 0:
            continue
        np_ = -(-n // page)
        pages = s["table"][b, :np_].long()
        for h in range(Hkv):
            K = s["Kp"][pages, h].reshape(np_ * page, D)[:n].to(torch.float64)
            V = s["Vp"][pages, h].reshape(np_ * page, D)[:n].to(torch.float64)
            if s["idx"] is not None:
                keep = s["idx"][b, h]
                keep = keep[keep >= 0].long()
                K, V = K[keep], V[keep]
            q = Q[b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)]
            logits = (q @ K.T) / math.sqrt(D)
            O[b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] = torch.softmax(logits, -1) @ V
            lse[b, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] = torch.logsumexp(logits, -1) / math.log(2.0)
    return (O, lse) if case["lse"] else O
