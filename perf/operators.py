"""The operators of a served request around the quantised projections, in plain torch form, and the calls of the
library that compute the same: writing new keys and values into a paged cache, attention over packed prompts, attention
of one new token per sequence, and scoring tokens against their logits.

A case is a dict of plain values; ``op`` says which operator it is:

* ``append``: RoPE of q and k, then k and v into the cache pages and q into the cache's type (``q4_kv_append``);
* ``prefill``: causal attention of packed prompt rows over the pages of their sequences (``q4_attn_prefill``);
* ``decode``: RoPE, append and attention of one new token per sequence (``q4_attn_paged``);
* ``score``: log probabilities of given tokens, entropy and the top alternatives of logit rows (``q4_logprobs``).

A cache page holds ``page`` positions of every kv head, ``[kv_heads][page][dim]``; ``table[b][i]`` is the page of
positions ``i * page ..`` of sequence b.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
THETA = 10000.0


def listed():
    return [
        # one decode step's new rows for a batch of 16 sequences (the widest batch of the matrix-vector calls)
        {"name": "append 16 rows f16", "op": "append", "dtype": "f16", "heads": 32, "kv_heads": 8, "dim": 64,
         "page": 16, "seqs": 16, "rows": 16, "prefix": 1000},
        # the rows of eight packed prompts after the prefill projections
        {"name": "append 8191 rows bf16", "op": "append", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "seqs": 8, "rows": 8191, "prefix": 0},
        # a short question: one prompt of 33 tokens
        {"name": "prefill 33 f16", "op": "prefill", "dtype": "f16", "heads": 32, "kv_heads": 8, "dim": 64,
         "page": 16, "seqs": 1, "rows": 33, "prefix": 0, "window": 0},
        # a serving step's mix: prompts of one to a few thousand tokens, some continuing a cached prefix
        {"name": "prefill 9 ragged bf16", "op": "prefill", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "seqs": 9, "rows": 5001, "prefix": 2000, "window": 0},
        # one long document
        {"name": "prefill 8192 f16", "op": "prefill", "dtype": "f16", "heads": 32, "kv_heads": 8, "dim": 64,
         "page": 128, "seqs": 1, "rows": 8192, "prefix": 0, "window": 0},
        # a prompt for the fp32 caches of the decode step (heads and caches of the real 16-layer step)
        {"name": "prefill 2048 f32", "op": "prefill", "dtype": "f32", "heads": 32, "kv_heads": 8, "dim": 64,
         "page": 4096, "seqs": 1, "rows": 2048, "prefix": 0, "window": 0},
        # one chat turn on the fp32 cache: latency
        {"name": "decode 1 x 512 f32", "op": "decode", "dtype": "f32", "heads": 32, "kv_heads": 8, "dim": 64,
         "page": 64, "seqs": 1, "context": 512, "window": 0},
        # the widest batch of the matrix-vector calls, contexts of all lengths up to 4096
        {"name": "decode 16 ragged f16", "op": "decode", "dtype": "f16", "heads": 32, "kv_heads": 8, "dim": 64,
         "page": 16, "seqs": 16, "context": 4096, "window": 0},
        # one long context
        {"name": "decode 1 x 32768 bf16", "op": "decode", "dtype": "bf16", "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "seqs": 1, "context": 32768, "window": 0},
        # a full server: 64 sequences of up to 8192
        {"name": "decode 64 ragged bf16", "op": "decode", "dtype": "bf16", "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "seqs": 64, "context": 8192, "window": 0},
        # the logits of one decoded token (the 65536-row projection), with the alternatives an API returns
        {"name": "score 1 row", "op": "score", "rows": 1, "vocab": 65536, "top": 20},
        # a prompt scored at once
        {"name": "score 512 rows", "op": "score", "rows": 512, "vocab": 65536, "top": 20},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "prefill", "prefill", "decode", "decode", "score"])
    if op == "score":
        vocab = _log_int(rng, 100, 140000)
        return {"op": op, "rows": _log_int(rng, 1, max(1, 30_000_000 // vocab) if vocab > 60000 else 512),
                "vocab": vocab, "top": rng.randint(0, 32)}
    dtype = rng.choice(["f16", "bf16", "f32"])
    dim, kv_heads, group = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8])
    case = {"op": op, "dtype": dtype, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim,
            "page": rng.choice([16, 32, 48, 64, 128, 256])}
    if op == "append":
        case["rows"] = _log_int(rng, 1, 6000)
        case["seqs"] = rng.randint(1, min(case["rows"], 12))
        case["prefix"] = rng.choice([0, rng.randint(1, 3000)])
    elif op == "prefill":
        case["rows"] = _log_int(rng, 1, 4000)
        case["seqs"] = rng.randint(1, min(case["rows"], 8))
        case["prefix"] = rng.choice([0, rng.randint(1, 2000)])
        case["window"] = rng.choice([0, 0, rng.randint(1, 2000)])
    else:
        case["context"] = _log_int(rng, 1, 8000)
        case["seqs"] = _log_int(rng, 1, 40)
        case["window"] = rng.choice([0, 0, rng.randint(1, 4000)])
    return case


def _lengths(case):
    """Host: (rows of each sequence, cached positions before them), the same for every seed of a case."""
    n = case["seqs"]
    gen = torch.Generator().manual_seed(1000 + n)
    if case["op"] == "decode":
        # contexts from one token to the longest, the new token included; the longest is always there
        u = torch.rand(n, generator=gen, dtype=torch.float64)
        u[0] = 1.0
        lens = [max(1, int(round(case["context"] * float(x)))) for x in u]
        return [1] * n, [x - 1 for x in lens]
    w = torch.rand(n, generator=gen, dtype=torch.float64) ** 2 + 0.01
    if case["rows"] == n:
        rows = [1] * n
    else:
        extra = (w / w.sum() * (case["rows"] - n)).floor().long().tolist()
        rows = [1 + x for x in extra]
        rows[0] += case["rows"] - sum(rows)
    u = torch.rand(n, generator=gen, dtype=torch.float64)
    prefix = [int(case["prefix"] * float(x)) for x in u]
    return rows, prefix


def _rope(positions, dim, device):
    """Tables [positions][dim / 2] of cos and sin, rounded once from 64 bits."""
    j = torch.arange(dim // 2, device=device, dtype=torch.float64)
    angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * THETA ** (-2.0 * j / dim)
    return angle.cos().float(), angle.sin().float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=gen, device=dev)  # noqa: E731
    if case["op"] == "score":
        rows, n = case["rows"], case["vocab"]
        logits = randn(rows, n) * 3.0
        # a tenth of the vocabulary is forbidden, as constrained decoding forbids it
        logits.masked_fill_(torch.rand(rows, n, generator=gen, device=dev) < 0.1, -math.inf)
        tokens = torch.randint(0, n, (rows,), generator=gen, device=dev, dtype=torch.int32)
        logits[torch.arange(rows, device=dev), tokens.long()] = randn(rows)  # a scored token is allowed
        return {"case": case, "logits": logits, "tokens": tokens}
    dt, hkv, dim, page, n = DTYPES[case["dtype"]], case["kv_heads"], case["dim"], case["page"], case["seqs"]
    rows, prefix = _lengths(case)
    need = [-(-(r + p) // page) for r, p in zip(rows, prefix)]
    width, used = max(need), sum(need)
    total = used + max(1, used // 8)  # a pool with some pages left
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b in range(n):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    k_pages = torch.empty((total, hkv, page, dim), dtype=dt, device=dev)
    v_pages = torch.empty_like(k_pages)
    for t in (k_pages, v_pages):  # in parts: a pool in fp32 would need twice its room
        for part in t.split(max(1, (1 << 26) // (hkv * page * dim))):
            part.copy_(randn(*part.shape))
    T = sum(rows)
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    s = {"case": case, "k_pages": k_pages, "v_pages": v_pages, "table": table, "cu": ints(cu), "start": ints(prefix),
         "longest_rows": max(rows), "longest": max(r + p for r, p in zip(rows, prefix)),
         "rope": _rope(width * page, dim, dev)}
    if case["op"] == "prefill":
        s["q"] = (randn(T, case["heads"], dim) * 1.5).to(dt)
        s["out"] = torch.empty_like(s["q"])
    else:
        s["q"] = randn(T, case["heads"], dim) * 1.5
        s["k"], s["v"] = randn(T, hkv, dim), randn(T, hkv, dim)
        s["out"] = torch.empty(T, case["heads"], dim, dtype=dt if case["op"] == "append" else torch.float32, device=dev)
    if own:
        import bit_weight_quantized_q4_gb300 as q4
        s["pages"] = q4.KVPages(k_pages, v_pages, table)
        if case["op"] == "prefill":
            s["ws"] = q4.q4_attn_prefill_workspace(s["pages"], T, case["heads"])
        elif case["op"] == "decode":
            s["ws"] = q4.q4_attn_paged_workspace(s["pages"], case["heads"])
    return s


def _rotate(x, cos, sin):
    """Element j pairs with j + dim / 2: (a, b) -> (a c - b s, b c + a s); x [T][heads][dim], tables [T][dim / 2]."""
    half = x.shape[-1] // 2
    a, b, c, s = x[..., :half], x[..., half:], cos[:, None], sin[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _of_row(s):
    """Each row's sequence and absolute position."""
    T = s["q"].shape[0]
    row = torch.arange(T, device=s["q"].device)
    seq = torch.searchsorted(s["cu"][1:].long().contiguous(), row, right=True)
    return seq, s["start"].long()[seq] + row - s["cu"].long()[seq]


def _plain_append(s):
    seq, pos = _of_row(s)
    page = s["case"]["page"]
    cos, sin = (t[pos] for t in s["rope"])
    where = (s["table"].long()[seq, pos // page], slice(None), pos % page)
    s["k_pages"][where] = _rotate(s["k"], cos, sin).to(s["k_pages"].dtype)
    s["v_pages"][where] = s["v"].to(s["v_pages"].dtype)
    return _rotate(s["q"], cos, sin)


def _plain_attention(s, q):
    """q [T][heads][dim] fp32 in its packed rows, over the pages; fp32 out."""
    case = s["case"]
    page, hkv, dim, n = case["page"], case["kv_heads"], case["dim"], case["seqs"]
    dev, G, Q, L = q.device, case["heads"] // hkv, s["longest_rows"], s["longest"]
    seq, pos = _of_row(s)
    at = pos - s["start"].long()[seq]
    key = torch.arange(L, device=dev)
    pg = s["table"].long()[:, key // page].clamp_min(0)                              # [n][L]
    K = s["k_pages"][pg, :, key % page].float().permute(0, 2, 3, 1)                  # [n][hkv][dim][L]
    qp = torch.zeros(n, hkv, Q, G, dim, device=dev)
    qp[seq, :, at] = q.view(-1, hkv, G, dim) / math.sqrt(dim)
    S = torch.matmul(qp.view(n, hkv, Q * G, dim), K).view(n, hkv, Q, G, L)
    del K
    p = s["start"].long()[:, None] + torch.arange(Q, device=dev)                    # [n][Q]
    hide = key > p[..., None]
    if case["window"]:
        hide |= key <= p[..., None] - case["window"]
    S.masked_fill_(hide[:, None, :, None, :], -math.inf)
    S -= S.amax(-1, keepdim=True).nan_to_num_(neginf=0.0)
    S.exp_()
    total = S.sum(-1, keepdim=True)
    V = s["v_pages"][pg, :, key % page].float().permute(0, 2, 1, 3)                  # [n][hkv][L][dim]
    V.masked_fill_(key[:, None] > p[:, -1, None, None, None], 0.0)
    out = torch.matmul(S.view(n, hkv, Q * G, L), V).view(n, hkv, Q, G, dim) / total
    return out[seq, :, at].reshape(q.shape)


def _plain_score(s):
    x, tokens, k = s["logits"], s["tokens"].long(), s["case"]["top"]
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    lse = m[:, 0] + e.sum(-1).log()
    p = e / e.sum(-1, keepdim=True)
    entropy = lse - (p * x.masked_fill(x == -math.inf, 0.0)).sum(-1)
    val, idx = torch.sort(x, dim=-1, descending=True, stable=True)
    k = min(k, x.shape[1])
    return (x.gather(1, tokens[:, None])[:, 0] - lse, entropy, val[:, :k] - lse[:, None],
            idx[:, :k].to(torch.int32).contiguous())


def _answer(op, s, got):
    if op == "score":
        return dict(zip(("logprob", "entropy", "top_logprob", "top_index"), got))
    if op == "prefill":
        return {"out": got}
    return {"q" if op == "append" else "out": got, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import bit_weight_quantized_q4_gb300 as q4
        if op == "append":
            got = q4.q4_kv_append(s["k"], s["v"], s["pages"], s["cu"], s["start"], q=s["q"], rope=s["rope"],
                                  q_out=s["out"])
        elif op == "prefill":
            got = q4.q4_attn_prefill(s["q"], s["pages"], s["cu"], s["start"], window=s["case"]["window"],
                                     out=s["out"], workspace=s["ws"])
        elif op == "decode":
            got = q4.q4_attn_paged(s["q"], s["k"], s["v"], s["pages"], s["start"], window=s["case"]["window"],
                                   rope=s["rope"], out=s["out"], workspace=s["ws"])
        else:
            got = q4.q4_logprobs(s["logits"], s["tokens"], top=s["case"]["top"])
        return _answer(op, s, got)
    if op == "append":
        return _answer(op, s, _plain_append(s).to(s["k_pages"].dtype))
    if op == "prefill":
        return _answer(op, s, _plain_attention(s, s["q"].float()).to(s["q"].dtype))
    if op == "decode":
        return _answer(op, s, _plain_attention(s, _plain_append(s)))
    return _answer(op, s, _plain_score(s))


def work(case):
    if case["op"] == "score":
        rows, n, k = case["rows"], case["vocab"], min(case["top"], case["vocab"])
        return {"bytes": 4 * rows * n + rows * (4 + 8 + 8 * k), "flops": 4 * rows * n}
    rows, prefix = _lengths(case)
    T, B, H, hkv, dim = sum(rows), BYTES[case["dtype"]], case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        return {"bytes": T * dim * ((H + 2 * hkv) * (4 + B) + 4), "flops": 3 * T * dim * (H + hkv)}
    pairs, keys = 0, 0
    for r, p in zip(rows, prefix):
        w = case["window"] or r + p
        pairs += sum(min(w, p + i + 1) for i in range(r))
        keys += r + p - max(0, p + 1 - w)
    moved = 2 * keys * hkv * dim * B
    if case["op"] == "decode":
        return {"bytes": moved + T * dim * 4 * (2 * H + 2 * hkv + 1), "flops": 4 * dim * H * pairs}
    return {"bytes": moved + 2 * T * H * dim * B, "flops": 4 * dim * H * pairs}


def exact(case, seed):
    """The definitions in 64 bits, one sequence and kv head at a time."""
    s = prepare(case, seed)
    if case["op"] == "score":
        x = s["logits"].double()
        lp = torch.log_softmax(x, -1)
        k = min(case["top"], case["vocab"])
        top = torch.sort(lp, dim=-1, descending=True).values[:, :k]
        ent = -torch.where(lp == -math.inf, torch.zeros_like(lp), lp.exp() * lp).sum(-1)
        return {"logprob": lp.gather(1, s["tokens"].long()[:, None])[:, 0], "entropy": ent, "top_logprob": top,
                "top_index": None}
    cu, start, page, hkv = s["cu"].tolist(), s["start"].tolist(), case["page"], case["kv_heads"]
    G, dim, op = case["heads"] // hkv, case["dim"], case["op"]
    q = s["q"].double()
    pools = [s["k_pages"], s["v_pages"]]
    if op == "append":  # unrounded rows beside the ones that were there
        pools = [t.double() for t in pools]
    for b in range(case["seqs"]):
        if op == "prefill":
            break
        at = torch.arange(start[b], start[b] + cu[b + 1] - cu[b], device=q.device)
        c, sn = (t.double()[at][:, None, :] for t in s["rope"])
        turn = lambda x: torch.complex(x[..., :dim // 2], x[..., dim // 2:]) * torch.complex(c, sn)  # noqa: E731
        rows = slice(cu[b], cu[b + 1])
        zq, zk = turn(q[rows]), turn(s["k"][rows].double())
        q[rows] = torch.cat([zq.real, zq.imag], -1)
        for pool, new in zip(pools, (torch.cat([zk.real, zk.imag], -1), s["v"][rows].double())):
            pool[s["table"][b].long()[at // page], :, at % page] = new.to(pool.dtype)
    if op == "append":
        return {"q": q, "k_pages": pools[0], "v_pages": pools[1]}
    out = torch.empty_like(q)
    for b in range(case["seqs"]):
        end = start[b] + cu[b + 1] - cu[b]
        lo = max(0, start[b] + 1 - case["window"]) if case["window"] else 0
        j = torch.arange(lo, end, device=q.device)
        i = torch.arange(start[b], end, device=q.device)
        seen = j[None] <= i[:, None]
        if case["window"]:
            seen &= j[None] > i[:, None] - case["window"]
        where = s["table"][b].long()[j // page]
        for h in range(hkv):
            K, V = (t[where, h, j % page].double() for t in pools)
            for g in range(G):
                score = q[cu[b]:cu[b + 1], h * G + g] @ K.T / math.sqrt(dim)
                w = torch.softmax(torch.where(seen, score, torch.full_like(score, -math.inf)), -1)
                out[cu[b]:cu[b + 1], h * G + g] = w @ V
    if op == "prefill":
        return {"out": out}
    return {"out": out, "k_pages": None, "v_pages": None}
