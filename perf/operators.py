"""Timed cases of the prompt operators: causal attention over packed prompts
(``prompt_attention``), the attention weight each prompt token gathers from the
last queries (``prompt_weights``), and the eviction that keeps a prompt's
heaviest tokens before it is quantized (``evict``).

``own`` False runs each operator in its plain form (torch products, sums,
exponentials, sorts and gathers, in fp32); ``own`` True calls the library.
Inputs follow the repository's synthetic workloads: Keys with one log-uniform
scale per channel and outlier channels ten times larger, Values with a scale
per token, normal queries.
"""

import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases ---------------------------------------------------------------------

def _case(op, lens, heads_q, heads_kv, dim, dtype, **more):
    return {"op": op, "lens": " ".join(str(n) for n in lens), "heads_q": heads_q, "heads_kv": heads_kv, "dim": dim,
            "dtype": dtype, **more}


def _lens(case):
    return [int(n) for n in case["lens"].split()]


def listed():
    return [
        # the smallest prompt of the repository's tiny fp32 configuration: launch latency
        {"name": "attention tiny fp32", **_case("attention", [40], 2, 2, 16, "fp32")},
        # a serving batch of short, ragged chat turns in one packed call
        {"name": "attention short turns", **_case("attention", [17, 300, 1, 129, 64, 255, 33, 402, 128, 90, 211, 5],
                                                  32, 8, 128, "bf16")},
        # one 4096-token prompt of the single-layer decode configuration
        {"name": "attention 4096", **_case("attention", [4096], 32, 8, 128, "bf16")},
        # the longest prompt: a document
        {"name": "attention 16384", **_case("attention", [16384], 32, 8, 128, "bf16")},
        # ragged prompts of a model without shared heads and with a narrow head
        {"name": "attention ragged d64", **_case("attention", [2048, 777, 1500, 64], 16, 16, 64, "bf16")},
        # an fp32 cache's prompt, odd length
        {"name": "attention fp32 1999", **_case("attention", [1999], 8, 2, 128, "fp32")},
        # which tokens of long prompts the last 64 queries look at (before an eviction)
        {"name": "weights last 64", **_case("weights", [8192, 5003, 6500, 1024], 32, 8, 128, "bf16", last=64)},
        # the same over every query of one prompt
        {"name": "weights whole 4096", **_case("weights", [4096], 32, 8, 128, "bf16", last=4096)},
        # a short fp32 prompt
        {"name": "weights fp32 300", **_case("weights", [300], 8, 2, 64, "fp32", last=32)},
        # one short prompt cut to a 128-token budget: latency
        {"name": "evict 300 to 128", **_case("evict", [300], 8, 8, 128, "bf16", budget=128, first=4, recent=32)},
        # a batch of ragged prompts cut to 1024 tokens a head
        {"name": "evict batch to 1024", **_case("evict", [8192, 5003, 6500, 1024, 900, 3001, 8000, 2222], 32, 8, 128,
                                                "bf16", budget=1024, first=4, recent=64)},
        # the long-video context (30 frames of 14400 tokens) cut to one frame's tokens
        {"name": "evict 432000 to 14400", **_case("evict", [432000], 32, 8, 128, "bf16", budget=14400, first=0,
                                                  recent=256)},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "weights", "evict"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    heads_kv = rng.choice([1, 2, 4, 8])
    heads_q = heads_kv * rng.choice([1, 2, 4, 4, 7, 8])
    dim = rng.choice([128, 128, 64, 64, 16, 80, 256])
    n = _log_int(rng, 1, 12)
    if op == "evict":
        top = _log_int(rng, 64, 200000)
        lens = [_log_int(rng, 1, top) for _ in range(n)]
        while sum(lens) * heads_kv * dim * (2 if dtype == "bf16" else 4) > 1 << 30:
            lens = [(m + 1) // 2 for m in lens]
        budget = _log_int(rng, 48, max(64, top // 2))
        return _case(op, lens, heads_q, heads_kv, dim, dtype, budget=budget, first=rng.choice([0, 1, 4]),
                     recent=rng.choice([0, 16, 32]))
    # the padded plain form holds n * heads_q * longest^2 scores
    most = 2.0e9 if dtype == "bf16" and dim in (64, 128) else 2.0e8
    top = min(12000, max(2, int(math.sqrt(most / (n * heads_q)))))
    top = _log_int(rng, min(16, top), top)
    lens = [_log_int(rng, 1, top) for _ in range(n)]
    if op == "weights":
        return _case(op, lens, heads_q, heads_kv, dim, dtype, last=_log_int(rng, 1, max(lens)))
    return _case(op, lens, heads_q, heads_kv, dim, dtype)


# ---- inputs --------------------------------------------------------------------

def _inputs(case, seed):
    """q [tokens, heads_q, dim], k and v [tokens, heads_kv, dim], packed."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    tokens, hq, hkv, d = sum(_lens(case)), case["heads_q"], case["heads_kv"], case["dim"]
    dt = _DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def log_uniform(lo, hi, *shape):
        u = torch.rand(*shape, generator=gen, device="cuda")
        return torch.exp(u * (math.log(hi) - math.log(lo)) + math.log(lo))

    q = normal(tokens, hq, d).to(dt)
    sigma = log_uniform(0.05, 5.0, hkv, d)
    sigma[:, 5::16] *= 10.0
    k = (normal(tokens, hkv, d) * sigma).to(dt)
    v = (normal(tokens, hkv, d) * log_uniform(0.5, 2.0, tokens, hkv, 1)).to(dt)
    return q, k, v, gen


def _starts(lens):
    return [sum(lens[:i]) for i in range(len(lens))]


def _grid(lens):
    """Padded positions of packed sequences: rows [n, longest] of the packed
    tensor (clamped to each sequence), and the flat places of the real rows."""
    n = torch.tensor(lens, device="cuda")
    start = torch.tensor(_starts(lens), device="cuda")
    pos = torch.arange(max(lens), device="cuda")
    rows = start[:, None] + torch.minimum(pos[None, :], n[:, None] - 1)
    real = (pos[None, :] < n[:, None]).reshape(-1).nonzero().reshape(-1)
    return n, rows, real


def prepare(case, seed):
    lens = _lens(case)
    q, k, v, gen = _inputs(case, seed)
    s = {"case": case, "lens": lens, "k": k}
    s["n"], s["rows"], s["real"] = _grid(lens)
    if case["op"] == "attention":
        s["q"], s["v"] = q, v
        return s
    if case["op"] == "weights":
        # the log-sum-exp that the prompt's attention returned, for the queries that count
        s["q"] = q
        s["lse"] = torch.zeros(case["heads_q"], sum(lens), device="cuda")
        g, d = case["heads_q"] // case["heads_kv"], case["dim"]
        for a, n in zip(_starts(lens), lens):
            first = max(0, n - case["last"])
            pos = torch.arange(first, n, device="cuda")
            hidden = torch.arange(n, device="cuda")[None, :] > pos[:, None]
            for h in range(case["heads_q"]):
                x = (q[a + first:a + n, h].double() @ k[a:a + n, h // g].double().T) / math.sqrt(d) \
                    if n * len(pos) < 1 << 20 else (q[a + first:a + n, h].float() @ k[a:a + n, h // g].float().T) / math.sqrt(d)
                s["lse"][h, a + first:a + n] = torch.logsumexp(x.masked_fill_(hidden, -math.inf), 1).float()
        return s
    # evict: gathered attention weights, heavy-tailed, in few enough bits that some are equal
    s["v"] = v
    w = torch.exp(2.0 * torch.randn(case["heads_kv"], sum(lens), generator=gen, device="cuda")) * 0.01
    s["weights"] = w.bfloat16().float()
    s["keep"] = [min(n, max(case["budget"], case["first"] + case["recent"])) for n in lens]
    keep = torch.tensor(s["keep"], device="cuda")
    most = max(s["keep"])
    live = torch.arange(most, device="cuda")[None, :] < keep[:, None]
    s["kept"] = live[:, None, :].expand(-1, case["heads_kv"], -1).reshape(-1).nonzero().reshape(-1)
    return s


# ---- one pass --------------------------------------------------------------------

def _padded_scores(s, q, k):
    """Scaled scores [n, heads_kv, g, longest, longest] of the padded prompts in fp32."""
    case, rows = s["case"], s["rows"]
    g = case["heads_q"] // case["heads_kv"]
    n, top = rows.shape
    qp = q.float()[rows].view(n, top, case["heads_kv"], g, case["dim"]).permute(0, 2, 3, 1, 4)
    kp = k.float()[rows].permute(0, 2, 3, 1)[:, :, None]
    return torch.matmul(qp, kp).mul_(1.0 / math.sqrt(case["dim"]))


def _plain_attention(s):
    case, rows = s["case"], s["rows"]
    n, top = rows.shape
    x = _padded_scores(s, s["q"], s["k"])
    pos = torch.arange(top, device="cuda")
    x.masked_fill_(pos[None, :] > pos[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    vp = s["v"].float()[rows].permute(0, 2, 1, 3)[:, :, None]
    o = torch.matmul(p, vp) / l
    o = o.permute(0, 3, 1, 2, 4).reshape(n * top, case["heads_q"], case["dim"])
    lse = (m + torch.log(l)).permute(1, 2, 0, 3, 4).reshape(case["heads_q"], n * top)
    return {"out": o[s["real"]].to(s["q"].dtype), "lse": lse[:, s["real"]].contiguous()}


def _plain_weights(s):
    case, rows = s["case"], s["rows"]
    n, top = rows.shape
    last = min(case["last"], top)
    # the last queries of each sequence, and the keys that come after each of them or after the sequence
    at = s["n"][:, None] - last + torch.arange(last, device="cuda")[None, :]
    start = rows[:, :1]
    qrows = start + at.clamp(min=0)
    g = case["heads_q"] // case["heads_kv"]
    qp = s["q"].float()[qrows].view(n, last, case["heads_kv"], g, case["dim"]).permute(0, 2, 3, 1, 4)
    kp = s["k"].float()[rows].permute(0, 2, 3, 1)[:, :, None]
    x = torch.matmul(qp, kp).mul_(1.0 / math.sqrt(case["dim"]))
    lse = s["lse"][:, qrows].view(case["heads_kv"], g, n, last).permute(2, 0, 1, 3)
    x.sub_(lse[..., None])
    pos = torch.arange(top, device="cuda")
    hidden = (pos[None, None, :] > at[:, :, None]) | (at[:, :, None] < 0)
    p = x.masked_fill_(hidden[:, None, None], -math.inf).exp_()
    w = p.sum((2, 3)).permute(1, 0, 2).reshape(case["heads_kv"], n * top)
    return {"weights": w[:, s["real"]].contiguous()}


def _plain_evict(s):
    case, rows = s["case"], s["rows"]
    n, top = rows.shape
    hkv, d = case["heads_kv"], case["dim"]
    pos = torch.arange(top, device="cuda")[None, :]
    w = s["weights"][:, rows].permute(1, 0, 2)
    always = (pos < case["first"]) | (pos >= s["n"][:, None] - case["recent"])
    w = w.masked_fill(always[:, None], math.inf).masked_fill((pos >= s["n"][:, None])[:, None], -math.inf)
    most = max(s["keep"])
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :most]
    keep = torch.minimum(s["n"], torch.full_like(s["n"], max(case["budget"], case["first"] + case["recent"])))
    late = torch.arange(most, device="cuda")[None, None, :] >= keep[:, None, None]
    index = torch.sort(order.masked_fill(late, top), dim=-1).values
    row = rows[:, :1, None] + index
    head = torch.arange(hkv, device="cuda")[None, :, None].expand_as(row)
    row, head, index = (t.reshape(-1)[s["kept"]] for t in (row, head, index))
    return {"k": s["k"][row, head], "v": s["v"][row, head], "index": index.to(torch.int32)}


def run(s):
    case = s["case"]
    if own:
        import quantized_kv_cache_02_gb300 as kvq
        if case["op"] == "attention":
            out, lse = kvq.prompt_attention(s["q"], s["k"], s["v"], s["lens"])
            return {"out": out, "lse": lse}
        if case["op"] == "weights":
            return {"weights": kvq.prompt_weights(s["q"], s["k"], s["lse"], s["lens"], last=case["last"])}
        kept = kvq.evict(s["k"], s["v"], s["weights"], s["lens"], s["keep"], first=case["first"],
                         recent=case["recent"])
        return {"k": kept.k, "v": kept.v, "index": kept.index}
    return {"attention": _plain_attention, "weights": _plain_weights, "evict": _plain_evict}[case["op"]](s)


def work(case):
    lens, hq, hkv, d = _lens(case), case["heads_q"], case["heads_kv"], case["dim"]
    size = 2 if case["dtype"] == "bf16" else 4
    tokens = sum(lens)
    if case["op"] == "attention":
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": tokens * d * size * (2 * hq + 2 * hkv) + 4 * tokens * hq, "flops": 4.0 * pairs * hq * d}
    if case["op"] == "weights":
        seen = [min(n, case["last"]) for n in lens]
        pairs = sum(m * n - m * (m - 1) // 2 for n, m in zip(lens, seen))
        return {"bytes": tokens * hkv * (d * size + 4) + sum(seen) * hq * (d * size + 4), "flops": 2.0 * pairs * hq * d}
    keep = sum(min(n, max(case["budget"], case["first"] + case["recent"])) for n in lens)
    return {"bytes": 4 * tokens * hkv + keep * hkv * (4 * d * size + 4), "flops": 0}


# ---- in 64 bits, from the definitions ------------------------------------------------

def exact(case, seed):
    lens, hq, hkv, d = _lens(case), case["heads_q"], case["heads_kv"], case["dim"]
    g = hq // hkv
    begin = np.concatenate([[0], np.cumsum(lens)])
    if case["op"] == "evict":
        s = prepare(case, seed)
        w = s["weights"].cpu().numpy().astype(np.float64)
        ks, vs, at = [], [], []
        for b, n in enumerate(lens):
            free = np.arange(min(case["first"], n), max(min(case["first"], n), n - case["recent"]))
            left = s["keep"][b] - (n - len(free))
            for h in range(hkv):
                x = w[h, begin[b]:begin[b + 1]]
                best = free[np.lexsort((free, -x[free]))[:left]]
                gone = np.ones(n, bool)
                gone[best] = False
                gone[:case["first"]] = False
                gone[n - min(n, case["recent"]):] = False
                t = torch.from_numpy(np.flatnonzero(~gone))
                at.append(t)
                ks.append(s["k"][begin[b]:begin[b + 1], h][t.cuda()].double())
                vs.append(s["v"][begin[b]:begin[b + 1], h][t.cuda()].double())
        return {"k": torch.cat(ks), "v": torch.cat(vs), "index": torch.cat(at).to(torch.int32)}
    if case["op"] == "attention":
        q, k, v, _ = _inputs(case, seed)
        out = torch.empty(sum(lens), hq, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(hq, sum(lens), dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            for h in range(hq):
                keys, values = k[begin[b]:begin[b + 1], h // g].double(), v[begin[b]:begin[b + 1], h // g].double()
                for i in range(0, n, 4096):
                    j = min(n, i + 4096)  # queries i .. j - 1 see keys 0 .. their own
                    z = q[begin[b] + i:begin[b] + j, h].double() @ keys[:j].T / d ** 0.5
                    z += torch.full((j - i, j), -math.inf, dtype=torch.float64, device="cuda").triu(i + 1)
                    e = torch.logsumexp(z, 1)
                    lse[h, begin[b] + i:begin[b] + j] = e
                    out[begin[b] + i:begin[b] + j, h] = torch.exp(z - e[:, None]) @ values[:j]
        return {"out": out, "lse": lse}
    s = prepare(case, seed)
    w = torch.zeros(hkv, sum(lens), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        first = max(0, n - case["last"])
        for h in range(hq):
            z = s["q"][begin[b] + first:begin[b] + n, h].double() @ s["k"][begin[b]:begin[b + 1], h // g].double().T
            z = torch.exp(z / d ** 0.5 - s["lse"][h, begin[b] + first:begin[b] + n, None].double())
            w[h // g, begin[b]:begin[b + 1]] += z.tril(first).sum(0)
    return {"weights": w}
