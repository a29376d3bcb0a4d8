"""Timed cases of the operators around a decoder's cache: rotary positions with
several axes (``rotary``), attention over an encoder's states
(``cross_attention``), and the copy of whole cached sequences
(``KVQCache.fork``, read back through ``KVQCache.restore``).

``own`` False runs each operator in its plain form (torch products, sums,
exponentials, indexing, in fp32; angles in 64 bits); ``own`` True calls the
library.  Inputs follow the repository's synthetic workloads.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---- cases ---------------------------------------------------------------------

def _text(values):
    return " ".join(str(v) for v in values)


def _ints(text):
    return [int(v) for v in text.split()]


def _rotary(tokens, heads_q, heads_kv, dim, dtype, sections, **more):
    """``restart``: every axis has its own falling frequencies (else one series
    runs over all pairs); ``adjacent``: pairs of neighbouring channels (else of
    the two halves); ``reach``: positions per axis are below these."""
    return {"op": "rotary", "tokens": tokens, "heads_q": heads_q, "heads_kv": heads_kv, "dim": dim, "dtype": dtype,
            "sections": _text(sections), "restart": False, "adjacent": False, "theta": 10000.0, **more}


def _cross(q_lens, kv_lens, heads_q, heads_kv, dim, dtype):
    return {"op": "cross", "q_lens": _text(q_lens), "kv_lens": _text(kv_lens), "heads_q": heads_q,
            "heads_kv": heads_kv, "dim": dim, "dtype": dtype}


def _fork(lens, src, heads_kv, dim, dtype, residual, group, qmax, paged):
    """The first len(lens) sequences are held; sequence len(lens) + i becomes a copy of src[i]."""
    return {"op": "fork", "lens": _text(lens), "src": _text(src), "heads_kv": heads_kv, "dim": dim, "dtype": dtype,
            "residual": residual, "group": group, "qmax": qmax, "paged": paged}


def listed():
    return [
        # the new tokens of a batch-32 decode step of the benchmark layer: latency
        {"name": "rotary decode 32", **_rotary(32, 32, 8, 128, "bf16", [64], reach="8192")},
        # one frame of the long-video context, positions in time, height and width
        {"name": "rotary frame", **_rotary(14400, 32, 8, 128, "bf16", [16, 24, 24], reach="30 90 160")},
        # eight of its frames in one prompt, every axis with its own frequencies, far along the video
        {"name": "rotary 8 frames", **_rotary(115200, 32, 8, 128, "bf16", [22, 21, 21], reach="432000 90 160",
                                              restart=True, adjacent=True)},
        # an fp32 cache's prompt of odd length, a quarter of each head left as it is
        {"name": "rotary fp32 1999", **_rotary(1999, 8, 2, 128, "fp32", [48], reach="1999")},
        # one new token each of 32 sequences over their encoder's states
        {"name": "cross decode 32", **_cross([1] * 32, [1500] * 32, 16, 16, 64, "bf16")},
        # one new token over a long document's states
        {"name": "cross decode long", **_cross([1], [16384], 32, 8, 128, "bf16")},
        # a video frame's tokens over a text prompt's states
        {"name": "cross frame to text", **_cross([14400], [512], 32, 8, 128, "bf16")},
        # ragged prompts over ragged states, without shared heads and with a narrow head
        {"name": "cross ragged d64", **_cross([2048, 777, 1, 1500, 64], [1500, 333, 1024, 77, 2999], 16, 16, 64,
                                              "bf16")},
        # a short fp32 prompt over fp32 states
        {"name": "cross fp32 300", **_cross([300], [777], 8, 2, 128, "fp32")},
        # a short prompt of the tiny fp32 configuration sampled twice: latency
        {"name": "fork tiny", **_fork([40], [0, 0], 2, 16, "fp32", 16, 8, 7, False)},
        # a prompt of the benchmark's length sampled seven times more from a paged cache
        {"name": "fork samples paged", **_fork([8192], [0] * 7, 8, 128, "bf16", 128, 32, 7, True)},
        # a beam search's four kept beams over its four dropped ones
        {"name": "fork beams", **_fork([2100, 2100, 2100, 2100], [0, 0, 1, 3], 8, 128, "bf16", 128, 32, 7, False)},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cut(rng, n, parts):
    """n cut into ``parts`` positive parts."""
    at = sorted(rng.sample(range(1, n), parts - 1))
    return [b - a for a, b in zip([0] + at, at + [n])]


def draw(rng):
    op = rng.choice(["rotary", "cross", "cross", "fork"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    size = 2 if dtype == "bf16" else 4
    heads_kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([128, 128, 64, 64, 16, 80, 256])
    if op == "fork":
        n, copies = rng.randint(1, 4), rng.randint(1, 8)
        top = _log_int(rng, 8, 12000)
        while copies * heads_kv * top * dim * size > 1 << 28:
            top = (top + 1) // 2
        lens = [_log_int(rng, 1, top) for _ in range(n)]
        group = rng.choice([8, 32, 64])
        return _fork(lens, [rng.randrange(n) for _ in range(copies)], heads_kv, dim, dtype, rng.choice([16, 100, 128]),
                     group, rng.choice([1, 7, 7, 127]), rng.random() < 0.5)
    heads_q = heads_kv * rng.choice([1, 2, 4, 4, 7, 8])
    if op == "rotary":
        axes = rng.choice([1, 2, 3, 3, 4])
        pairs = dim // 2 if rng.random() < 0.7 else rng.randint(axes, dim // 2)
        tokens = _log_int(rng, 1, min(120000, (1 << 30) // ((heads_q + heads_kv) * dim * size)))
        return _rotary(tokens, heads_q, heads_kv, dim, dtype, _cut(rng, pairs, axes) if axes > 1 else [pairs],
                       reach=_text(_log_int(rng, 1, 1000000) for _ in range(axes)), restart=rng.random() < 0.4,
                       adjacent=rng.random() < 0.4, theta=rng.choice([10000.0, 500000.0, 1000000.0]))
    n = _log_int(rng, 1, 40)
    # the padded plain form holds n * heads_q * (longest prompt) * (most states) scores
    most = 2.0e8 if dtype == "bf16" and dim in (64, 128) else 2.0e7
    top_kv = _log_int(rng, 1, 20000)
    while n * top_kv * heads_kv * dim * size > 1 << 28:
        top_kv = (top_kv + 1) // 2
    top_q = max(1, min(20000, int(most / (n * heads_q * top_kv))))
    top_q = 1 if rng.random() < 0.3 else _log_int(rng, 1, top_q)
    return _cross([_log_int(rng, 1, top_q) for _ in range(n)], [_log_int(rng, 1, top_kv) for _ in range(n)], heads_q,
                  heads_kv, dim, dtype)


# ---- inputs --------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _log_uniform(gen, lo, hi, *shape):
    u = torch.rand(*shape, generator=gen, device="cuda")
    return torch.exp(u * (math.log(hi) - math.log(lo)) + math.log(lo))


def _frequencies(case):
    """Radians per step of every pair, and the axis of its position."""
    sections = _ints(case["sections"])
    axes = [a for a, n in enumerate(sections) for _ in range(n)]
    if case["restart"]:
        freq = [case["theta"] ** (-i / n) for n in sections for i in range(n)]
    else:
        freq = [case["theta"] ** (-i / len(axes)) for i in range(len(axes))]
    return freq, axes


def _rotary_inputs(case, seed):
    gen, dt = _generator(seed), _DTYPES[case["dtype"]]
    q, k = (torch.randn(case["tokens"], h, case["dim"], generator=gen, device="cuda", dtype=torch.float32).to(dt)
            for h in (case["heads_q"], case["heads_kv"]))
    # positions in order along the last axis, then the one before it, behind a random start of the first
    reach = _ints(case["reach"])
    at = torch.arange(case["tokens"], device="cuda")
    columns = []
    for size in reversed(reach[1:]):
        columns.append(at % size)
        at = at // size
    start = int(torch.randint(reach[0], (1,), generator=gen, device="cuda").item())
    columns.append((at + start) % reach[0])
    return q, k, torch.stack(columns[::-1], 1).contiguous()


def _cross_inputs(case, seed):
    gen, dt = _generator(seed), _DTYPES[case["dtype"]]
    nq, nkv = sum(_ints(case["q_lens"])), sum(_ints(case["kv_lens"]))
    hkv, d = case["heads_kv"], case["dim"]
    q = torch.randn(nq, case["heads_q"], d, generator=gen, device="cuda").to(dt)
    k = (torch.randn(nkv, hkv, d, generator=gen, device="cuda") * _log_uniform(gen, 0.25, 2.0, hkv, d)).to(dt)
    v = (torch.randn(nkv, hkv, d, generator=gen, device="cuda") * _log_uniform(gen, 0.5, 2.0, nkv, hkv, 1)).to(dt)
    return q, k, v


def _fork_inputs(case, seed):
    """Keys and Values [heads_kv, tokens, dim] of every held sequence."""
    gen, dt = _generator(seed), _DTYPES[case["dtype"]]
    h, d, out = case["heads_kv"], case["dim"], []
    for n in _ints(case["lens"]):
        sigma = _log_uniform(gen, 0.05, 5.0, h, 1, d)
        sigma[..., 5::16] *= 10.0
        k = (torch.randn(h, n, d, generator=gen, device="cuda") * sigma).to(dt)
        v = (torch.randn(h, n, d, generator=gen, device="cuda") * _log_uniform(gen, 0.5, 2.0, h, n, 1)).to(dt)
        out.append((k, v))
    return out


def _quantized(n, residual, group):
    """Tokens of a sequence of n that are held as codes; the rest is the window."""
    return (n - residual) // group * group if n >= residual + group else 0


def _quantize(x, qmax, dims):
    """The cache's codes and scales (one scale over ``dims``)."""
    x = x.float()
    scale = torch.full((), float(qmax), device="cuda") / x.abs().amax(dims, keepdim=True).clamp_min(1e-8)
    return (x * scale).round().clamp(-qmax, qmax).to(torch.int8), scale


def _grid(q_lens, kv_lens):
    """Rows [n, longest] of the packed tensors, and the flat places of the real query rows."""
    out = []
    for lens in (q_lens, kv_lens):
        n = torch.tensor(lens, device="cuda")
        start = torch.tensor([sum(lens[:i]) for i in range(len(lens))], device="cuda")
        pos = torch.arange(max(lens), device="cuda")
        out.append((n, pos, start[:, None] + torch.minimum(pos[None, :], n[:, None] - 1)))
    (nq, pq, rows_q), (nkv, pkv, rows_kv) = out
    real = (pq[None, :] < nq[:, None]).reshape(-1).nonzero().reshape(-1)
    return rows_q, rows_kv, real, pkv[None, :] >= nkv[:, None]


def prepare(case, seed):
    s = {"case": case}
    if case["op"] == "rotary":
        s["q"], s["k"], s["positions"] = _rotary_inputs(case, seed)
        freq, axes = _frequencies(case)
        if own:
            import quantized_kv_cache_02_gb300 as kvq
            s["plan"] = kvq.Rotary(case["dim"], freq, axes, interleaved=case["adjacent"])
        else:
            s["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
            s["axes"] = torch.tensor(axes, device="cuda")
        return s
    if case["op"] == "cross":
        s["q"], s["k"], s["v"] = _cross_inputs(case, seed)
        s["q_lens"], s["kv_lens"] = _ints(case["q_lens"]), _ints(case["kv_lens"])
        if not own:
            s["rows_q"], s["rows_kv"], s["real"], s["past"] = _grid(s["q_lens"], s["kv_lens"])
        return s
    held = _fork_inputs(case, seed)
    lens, src = _ints(case["lens"]), _ints(case["src"])
    n, copies, h, d = len(lens), len(src), case["heads_kv"], case["dim"]
    s["top"] = max(lens[i] for i in src)
    dt = _DTYPES[case["dtype"]]
    if own:
        import quantized_kv_cache_02_gb300 as kvq
        blocks = sum(_quantized(m, case["residual"], case["group"]) // case["group"] for m in lens)
        cache = kvq.KVQCache(n + copies, h, h, d, case["residual"], case["group"], case["qmax"], max(lens) + 64,
                             dtype=case["dtype"], pool_blocks=blocks + 4 * (n + copies) if case["paged"] else 0)
        for i, (k, v) in enumerate(held):
            cache.append(k[None].contiguous(), v[None].contiguous(), i)
        s.update(cache=cache, src=src, dst=list(range(n, n + copies)), first=n, copies=copies)
        s["k"], s["v"] = (torch.zeros(copies, h, s["top"], d, dtype=dt, device="cuda") for _ in range(2))
        return s
    # every slot's codes, scales and window, padded to the longest
    g, top = case["group"], max(lens)
    q = [_quantized(m, case["residual"], g) for m in lens]
    most, window = max(q), max(m - a for m, a in zip(lens, q))
    kc, vc = (torch.zeros(n + copies, h, most, d, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(n + copies, h, a, b, device="cuda") for a, b in ((most // g, d), (most, 1)))
    wk, wv = (torch.zeros(n + copies, h, window, d, dtype=dt, device="cuda") for _ in range(2))
    for i, (k, v) in enumerate(held):
        if q[i]:
            c, scale = _quantize(k[:, :q[i]].view(h, q[i] // g, g, d), case["qmax"], 2)
            kc[i, :, :q[i]], ks[i, :, :q[i] // g] = c.reshape(h, q[i], d), scale[:, :, 0]
            vc[i, :, :q[i]], vs[i, :, :q[i]] = _quantize(v[:, :q[i]], case["qmax"], 2)
        wk[i, :, :lens[i] - q[i]], wv[i, :, :lens[i] - q[i]] = k[:, q[i]:], v[:, q[i]:]
    s["slots"] = [kc, vc, ks, vs, wk, wv]
    s["src"], s["dst"] = torch.tensor(src, device="cuda"), torch.arange(n, n + copies, device="cuda")
    total, old = (torch.tensor([x[i] for i in src], device="cuda")[:, None] for x in (lens, q))
    pos = torch.arange(s["top"], device="cuda")[None, :]
    s["in_window"] = ((pos >= old) & (pos < total))[:, None, :, None]
    s["past"] = (pos >= total)[:, None, :, None]
    s["at"] = pos.clamp(max=max(most - 1, 0)).reshape(-1)
    s["window_at"] = (pos - old).clamp(min=0, max=window - 1)
    return s


# ---- one pass --------------------------------------------------------------------

def _plain_rotary(s):
    angle = s["positions"][:, s["axes"]].double() * s["freq"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    pairs, out = len(s["axes"]), []
    for x in (s["q"], s["k"]):
        y = x.float()
        if s["case"]["adjacent"]:
            a, b = y[..., 0:2 * pairs:2], y[..., 1:2 * pairs:2]
            turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = y[..., :pairs], y[..., pairs:2 * pairs]
            turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        out.append(torch.cat((turned, y[..., 2 * pairs:]), -1).to(x.dtype))
    return {"q": out[0], "k": out[1]}


def _plain_cross(s):
    case = s["case"]
    hkv, d = case["heads_kv"], case["dim"]
    g = case["heads_q"] // hkv
    n, top = s["rows_q"].shape
    qp = s["q"].float()[s["rows_q"]].view(n, top, hkv, g, d).permute(0, 2, 3, 1, 4)
    kp = s["k"].float()[s["rows_kv"]].permute(0, 2, 3, 1)[:, :, None]
    x = torch.matmul(qp, kp).mul_(1.0 / math.sqrt(d))
    x.masked_fill_(s["past"][:, None, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, s["v"].float()[s["rows_kv"]].permute(0, 2, 1, 3)[:, :, None]) / l
    o = o.permute(0, 3, 1, 2, 4).reshape(n * top, case["heads_q"], d)
    lse = (m + torch.log(l)).permute(1, 2, 0, 3, 4).reshape(case["heads_q"], n * top)
    return {"out": o[s["real"]].to(s["q"].dtype), "lse": lse[:, s["real"]].contiguous()}


def _plain_fork(s):
    for slot in s["slots"]:
        slot[s["dst"]] = slot[s["src"]]
    kc, vc, ks, vs, wk, wv = (slot[s["dst"]] for slot in s["slots"])
    copies, h, _, d = wk.shape
    index = s["window_at"][:, None, :, None].expand(copies, h, s["top"], d)
    out = []
    for codes, scales, window in ((kc, ks, wk), (vc, vs, wv)):
        x = torch.gather(window, 2, index).float()
        if codes.shape[2]:
            group = codes.shape[2] // scales.shape[2]
            restored = codes[:, :, s["at"]].float() / scales[:, :, s["at"] // group].clamp_min(1e-8)
            x = torch.where(s["in_window"], x, restored)
        out.append(x.masked_fill(s["past"], 0.0).to(wk.dtype))
    return {"k": out[0], "v": out[1]}


def run(s):
    case = s["case"]
    if own:
        import quantized_kv_cache_02_gb300 as kvq
        if case["op"] == "rotary":
            q, k = kvq.rotary(s["q"], s["k"], s["positions"], s["plan"])
            return {"q": q, "k": k}
        if case["op"] == "cross":
            out, lse = kvq.cross_attention(s["q"], s["k"], s["v"], s["q_lens"], s["kv_lens"])
            return {"out": out, "lse": lse}
        s["cache"].fork(s["src"], s["dst"])
        k, v = s["cache"].restore(s["first"], s["copies"], s["top"], case["dtype"], s["k"], s["v"])
        return {"k": k, "v": v}
    return {"rotary": _plain_rotary, "cross": _plain_cross, "fork": _plain_fork}[case["op"]](s)


def work(case):
    size, d, hkv = 2 if case["dtype"] == "bf16" else 4, case["dim"], case["heads_kv"]
    if case["op"] == "rotary":
        rows = case["tokens"] * (case["heads_q"] + hkv)
        sections = _ints(case["sections"])
        return {"bytes": 2 * rows * d * size + 8 * case["tokens"] * len(sections), "flops": 6 * rows * sum(sections)}
    if case["op"] == "cross":
        q, kv, hq = _ints(case["q_lens"]), _ints(case["kv_lens"]), case["heads_q"]
        return {"bytes": sum(q) * hq * (2 * d * size + 4) + 2 * sum(kv) * hkv * d * size,
                "flops": 4.0 * sum(a * b for a, b in zip(q, kv)) * hq * d}
    # what the copied sequences hold is read, the copies' windows are written (pages too where they are not
    # shared), and the copies' contents are written out
    lens, src, g = _ints(case["lens"]), _ints(case["src"]), case["group"]
    bits = 2 if case["qmax"] <= 1 else 4 if case["qmax"] <= 7 else 8
    q = [_quantized(n, case["residual"], g) for n in lens]
    pages = [hkv * (2 * a * d * bits // 8 + 4 * (a // g) * d + 4 * a) for a in q]
    window = [2 * hkv * (n - a) * d * size for n, a in zip(lens, q)]
    read = sum(pages[i] + window[i] for i in set(src))
    copied = sum(window[i] + (0 if case["paged"] else pages[i]) for i in src)
    return {"bytes": read + copied + sum(2 * hkv * lens[i] * d * size for i in src),
            "flops": sum(2 * hkv * q[i] * d for i in src)}


# ---- in 64 bits, from the definitions ------------------------------------------------

def exact(case, seed):
    d, hkv = case["dim"], case["heads_kv"]
    if case["op"] == "rotary":
        q, k, positions = _rotary_inputs(case, seed)
        freq, axes = _frequencies(case)
        first, step = (0, 2) if case["adjacent"] else (len(freq), 1)
        out = []
        for x in (q, k):
            y = x.double()
            for i, (f, a) in enumerate(zip(freq, axes)):
                one, two = (2 * i, 2 * i + 1) if step == 2 else (i, first + i)
                z = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), positions[:, a, None].double() * f)
                z = z * torch.complex(y[..., one], y[..., two])
                y[..., one], y[..., two] = z.real, z.imag
            out.append(y)
        return {"q": out[0], "k": out[1]}
    if case["op"] == "cross":
        q, k, v = _cross_inputs(case, seed)
        hq = case["heads_q"]
        out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(hq, len(q), dtype=torch.float64, device="cuda")
        i = j = 0
        for n, m in zip(_ints(case["q_lens"]), _ints(case["kv_lens"])):
            for h in range(hq):
                z = q[i:i + n, h].double() @ k[j:j + m, h * hkv // hq].double().T / d ** 0.5
                lse[h, i:i + n] = torch.logsumexp(z, 1)
                out[i:i + n, h] = torch.softmax(z, 1) @ v[j:j + m, h * hkv // hq].double()
            i, j = i + n, j + m
        return {"out": out, "lse": lse}
    lens, src, g, qmax = _ints(case["lens"]), _ints(case["src"]), case["group"], case["qmax"]
    held = _fork_inputs(case, seed)
    result = [torch.zeros(len(src), hkv, max(lens[i] for i in src), d, dtype=torch.float64, device="cuda")
              for _ in range(2)]
    for at, i in enumerate(src):
        n = lens[i]
        old = max(0, (n - case["residual"]) // g) * g
        for x, to, per_token in ((held[i][0], result[0], False), (held[i][1], result[1], True)):
            y = x.double()
            for t in range(0, old, g):
                part = y[:, t:t + g]
                top = part.abs().amax(2 if per_token else 1, keepdim=True).clamp_min(float(torch.tensor(1e-8)))
                scale = (qmax / top).float().double()  # scales are held in fp32, and so is the product that is rounded
                code = torch.round((part * scale).float().double()).clamp(-qmax, qmax)
                y[:, t:t + g] = code / scale.clamp_min(float(torch.tensor(1e-8)))
            to[at, :, :n] = y
    return {"k": result[0], "v": result[1]}
