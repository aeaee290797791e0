"""What a serving step with a paged KV cache does around its layers, and what scoring text takes, as cases to measure.

Three operators, each in its plain form (elementary torch operations) and, where `own` is true, through
`quantized_transformer_decode_gb300.qw3`:

  append     raw q/k/v projections of a ragged batch -> per-head Q/K RMSNorm, RoPE, K and V written as f16 into the pages
             of each sequence (the rotated queries come out, and the cache)
  attention  grouped-query causal attention of a ragged batch over the pages: whole prompts, chunks of new tokens behind a
             cached context, single tokens, and all of them mixed; whole, or through a sliding window with a few first
             tokens that stay visible
  logprobs   log probabilities of given tokens, the entropy of each row and its most likely alternatives

The cache: f16 [page][K|V][kv head][page_size][head_dim]. A batch: rows starts[b] .. starts[b + 1] - 1 of the activations
are the newest tokens of sequence b, which holds lens[b] positions with them; position p lies in page
table[b][p / page_size].
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 1e6
#: (query heads, kv heads, head_dim): this repository's 0.6B and 8B geometries and its tiny one, and groups of 1 and 8.
HEADS = ((16, 8, 128), (32, 8, 128), (4, 2, 64), (8, 8, 128), (16, 2, 64))
TYPES = {"f32": torch.float32, "f16": torch.float16}


def listed():
    small = {"nh": 16, "nkv": 8, "hd": 128}      # 0.6B heads
    large = {"nh": 32, "nkv": 8, "hd": 128}      # 8B heads
    return [
        # one token of one conversation: the smallest call, where latency counts
        {"name": "append_1_token", "op": "append", "batch": 1, "rows": 1, "long_rows": 0, "max_len": 517, "ragged": False, "page": 16, "dtype": "f32", **small},
        # one step of 64 conversations at scattered lengths
        {"name": "append_64_tokens", "op": "append", "batch": 64, "rows": 1, "long_rows": 0, "max_len": 4101, "ragged": True, "page": 64, "dtype": "f16", **large},
        # a 4096-token chunk of a prompt
        {"name": "append_chunk_4096", "op": "append", "batch": 1, "rows": 4096, "long_rows": 0, "max_len": 8190, "ragged": False, "page": 16, "dtype": "f32", **large},
        # one token of one short conversation
        {"name": "attn_1x517", "op": "attention", "batch": 1, "rows": 1, "long_rows": 0, "max_len": 517, "ragged": False, "page": 16, "dtype": "f32", "window": 0, "sinks": 0, **small},
        # one token of one conversation at this model family's native context
        {"name": "attn_1x32768", "op": "attention", "batch": 1, "rows": 1, "long_rows": 0, "max_len": 32768, "ragged": False, "page": 64, "dtype": "f16", "window": 0, "sinks": 0, **large},
        # one step of 64 conversations of lengths from 1 to 4101
        {"name": "attn_64_ragged", "op": "attention", "batch": 64, "rows": 1, "long_rows": 0, "max_len": 4101, "ragged": True, "page": 16, "dtype": "f32", "window": 0, "sinks": 0, **small},
        # a 4096-token prompt at once
        {"name": "attn_prompt_4096", "op": "attention", "batch": 1, "rows": 4096, "long_rows": 0, "max_len": 4096, "ragged": False, "page": 64, "dtype": "f16", "window": 0, "sinks": 0, **large},
        # the last 509-token chunk of a prompt of 8189, f32 activations
        {"name": "attn_chunk_509_of_8189", "op": "attention", "batch": 1, "rows": 509, "long_rows": 0, "max_len": 8189, "ragged": False, "page": 16, "dtype": "f32", "window": 0, "sinks": 0, **large},
        # 32 conversations that decode and one whose prompt goes on by 300 tokens, through a window of 1024 with 4 first tokens
        {"name": "attn_33_mixed_window", "op": "attention", "batch": 33, "rows": 1, "long_rows": 300, "max_len": 6001, "ragged": True, "page": 32, "dtype": "f16", "window": 1024, "sinks": 4, **small},
        # the next token of one conversation, with five alternatives
        {"name": "logprobs_1", "op": "logprobs", "batch": 1, "vocab": 151936, "given": 1, "top": 5},
        # a scored chunk of 512 tokens, with 20 alternatives each
        {"name": "logprobs_512_top20", "op": "logprobs", "batch": 512, "vocab": 151936, "given": 1, "top": 20},
        # seven questions with four answers each, a small odd vocabulary
        {"name": "logprobs_7_small", "op": "logprobs", "batch": 7, "vocab": 4099, "given": 4, "top": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "attention", "attention", "attention", "logprobs"))
    if op == "logprobs":
        vocab = _log_int(rng, 1000, 152064)
        return {"op": op, "batch": _log_int(rng, 1, 512), "vocab": vocab, "given": rng.choice((1, 1, 2, 5)), "top": rng.choice((0, 1, 5, 20, 37))}
    nh, nkv, hd = rng.choice(HEADS)
    c = {"op": op, "page": rng.choice((16, 32, 64, 128, 256)), "dtype": rng.choice(("f32", "f16")), "nh": nh, "nkv": nkv, "hd": hd}
    kind = rng.choice(("tokens", "tokens", "chunk", "chunk", "mixed"))
    if kind == "tokens":
        batch = _log_int(rng, 1, 64)
        c.update(batch=batch, rows=rng.choice((1, 1, 1, 2, 5)), long_rows=0, max_len=_log_int(rng, 6, min(32768, 262144 // batch)))
    elif kind == "chunk":
        batch = rng.choice((1, 1, 1, 2, 3))
        rows = _log_int(rng, 17, 4096 // batch)
        c.update(batch=batch, rows=rows, long_rows=0, max_len=rows + rng.randint(0, 4096 - rows))
    else:
        c.update(batch=rng.randint(2, 40), rows=1, long_rows=_log_int(rng, 8, 300), max_len=_log_int(rng, 400, 6000))
    c["ragged"] = rng.random() < 0.5 or kind == "mixed"
    if op == "attention":
        window = 0 if rng.random() < 0.6 else _log_int(rng, 16, 2048)
        c.update(window=window, sinks=rng.choice((0, 1, 4, 70)) if window else 0)
    return c


def _counts(case):
    """(rows, length) of each sequence: `rows` new tokens each, or `long_rows` for the last one where it is given; lengths all max_len,
    or in equal steps from the shortest possible to it."""
    b, n = case["batch"], case["max_len"]
    rows = [case["rows"]] * b
    if case["long_rows"]:
        rows[-1] = case["long_rows"]
    if not case["ragged"] or b == 1:
        return rows, [n] * b
    return rows, [r + (n - r) * i // (b - 1) for i, r in enumerate(rows)]


def _visible(case):
    """(pairs of a row and a position that it attends to, positions that some row attends to) of the whole batch."""
    pairs = held = 0
    w, s = case["window"], case["sinks"]
    for r, n in zip(*_counts(case)):
        p = np.arange(n - r, n)
        first = np.maximum(p - w + 1, 0) if w else np.zeros_like(p)
        sunk = np.minimum(s, first) if w else np.zeros_like(p)
        pairs += int((p + 1 - first + sunk).sum())
        held += int(n - first[0] + min(s if w else 0, first[0]))
    return pairs, held


def work(case):
    if case["op"] == "logprobs":
        b, v = case["batch"], case["vocab"]
        return {"bytes": b * (v * 4 + 8 * case["given"] + 4 + 8 * case["top"]), "flops": b * v * 4}
    nh, nkv, hd = case["nh"], case["nkv"], case["hd"]
    m, size = sum(_counts(case)[0]), 4 if case["dtype"] == "f32" else 2
    if case["op"] == "append":
        return {"bytes": m * ((2 * nh + 2 * nkv) * hd * size + 2 * nkv * hd * 2 + hd * 4), "flops": m * (nh + nkv) * hd * 7}
    pairs, held = _visible(case)
    return {"bytes": 2 * m * nh * hd * size + held * 2 * nkv * hd * 2, "flops": 4 * pairs * nh * hd}


# ---------------------------------------------------------------- states

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    rnd = np.random.default_rng(int(seed))
    ints = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] == "logprobs":
        b, v = case["batch"], case["vocab"]
        # a spread-out vocabulary with a few hundred candidates well above it, as a language model's logits have
        x = torch.randn(b, v, generator=g, device="cuda") * 2.2
        k = min(400, v)
        top = torch.arange(k, device="cuda") * (v // k) + torch.randint(0, v // k, (b, k), generator=g, device="cuda")
        top = top.gather(1, torch.rand(b, k, generator=g, device="cuda").argsort(1))
        x.scatter_add_(1, top, -2.5 * torch.log(torch.rand(top.shape, generator=g, device="cuda").clamp_min(1e-6)))
        s["logits"] = x
        # given tokens: mostly likely ones, as in real text
        t = torch.randint(0, v, (b, case["given"]), generator=g, device="cuda")
        t = torch.where(torch.rand(t.shape, generator=g, device="cuda") < 0.8, top[:, :case["given"]], t)
        s["tokens"] = t.int()
        return s
    nh, nkv, hd, page = (case[k] for k in ("nh", "nkv", "hd", "page"))
    rows, lens = _counts(case)
    if not case["long_rows"]:
        lens = rnd.permutation(lens)
    b, m = case["batch"], sum(rows)
    dtype = TYPES[case["dtype"]]
    s["starts"] = ints(np.concatenate(([0], np.cumsum(rows))))
    s["lens"] = ints(lens)
    used = -(-np.asarray(lens) // page)
    s["pages"] = int(used.sum()) + 3
    # pages as an allocator hands them out: in no order, none twice; -1 behind a sequence's last one
    table = np.full((b, int(used.max())), -1, np.int64)
    table[np.arange(table.shape[1]) < used[:, None]] = rnd.permutation(s["pages"])[:int(used.sum())]
    s["table"] = ints(table)
    # keys after their norm (unit size, a few channels larger), values around 0.4
    gain = 1 + 0.3 * torch.randn(2, nkv, 1, hd, generator=g, device="cuda").abs()
    gain[1] *= 0.4
    s["data"] = (torch.randn(s["pages"], 2, nkv, page, hd, generator=g, device="cuda") * gain).half()
    if case["op"] == "append":
        s["qkv"] = (torch.randn(m, (nh + 2 * nkv) * hd, generator=g, device="cuda") * 0.7).to(dtype)
        s["q_norm"] = 1 + 0.1 * torch.randn(hd, generator=g, device="cuda")
        s["k_norm"] = 1 + 0.1 * torch.randn(hd, generator=g, device="cuda")
        i = torch.arange(hd // 2, dtype=torch.float64, device="cuda")
        a = torch.arange(case["max_len"], dtype=torch.float64, device="cuda")[:, None] * THETA ** (-2 * i / hd)
        s["rope"] = torch.stack((a.cos(), a.sin()), -1).float()
    else:
        s["q"] = (torch.randn(m, nh, hd, generator=g, device="cuda") * 1.2).to(dtype)
        s["max_rows"] = max(rows)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    return {"append": _append, "attention": _attention, "logprobs": _logprobs}[s["op"]](s)


def _own(s):
    from quantized_transformer_decode_gb300 import qw3
    if s["op"] == "logprobs":
        return qw3.logprobs(s["logits"], s["tokens"], top=s["top"])
    cache = qw3.KVCachePaged(s["pages"], s["page"], s["nkv"], s["hd"], data=s["data"])
    if s["op"] == "append":
        q = cache.append(s["qkv"], s["starts"], s["lens"], s["table"], s["rope"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return q, s["data"]
    return cache.attention(s["q"], s["starts"], s["lens"], s["table"], max_rows=s["max_rows"], max_len=s["max_len"],
                           window=s["window"], sinks=s["sinks"])


def _append(s):
    nh, nkv, hd, page = s["nh"], s["nkv"], s["hd"], s["page"]
    starts, lens, table = s["starts"].long(), s["lens"].long(), s["table"].long()
    x = s["qkv"].float().unflatten(-1, (nh + 2 * nkv, hd))
    row = torch.arange(len(x), device="cuda")
    seq = torch.searchsorted(starts, row, right=True) - 1
    pos = lens[seq] - (starts[seq + 1] - row)
    cs = s["rope"][pos][:, None]

    def turned(h, w):
        h = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * w
        a, b = h.chunk(2, -1)
        return torch.cat((a * cs[..., 0] - b * cs[..., 1], b * cs[..., 0] + a * cs[..., 1]), -1)

    at, off = table[seq, pos // page], pos % page
    s["data"][at, 0, :, off] = turned(x[:, nh:nh + nkv], s["k_norm"]).half()
    s["data"][at, 1, :, off] = x[:, nh + nkv:].half()
    return turned(x[:, :nh], s["q_norm"]).to(s["qkv"].dtype), s["data"]


def _attention(s):
    nh, nkv, hd, page, r, n = s["nh"], s["nkv"], s["hd"], s["page"], s["max_rows"], s["max_len"]
    starts, lens, table = s["starts"].long(), s["lens"].long(), s["table"].long()
    b, m = len(lens), len(s["q"])
    j = torch.arange(n, device="cuda")
    at = table[:, j // page].clamp_min(0)                                               # [b][position]
    k = s["data"][at, 0, :, j % page].float()                                           # [b][position][kv head][hd]
    v = s["data"][at, 1, :, j % page].float()
    held = (j < lens[:, None])[..., None, None]
    v = torch.where(held, v, torch.zeros_like(v))
    t = torch.arange(r, device="cuda")
    q = s["q"][(starts[:-1, None] + t).clamp_max(m - 1)].float().unflatten(2, (nkv, nh // nkv))   # [b][row][kv head][group][hd]
    p = (lens - (starts[1:] - starts[:-1]))[:, None] + t                                # [b][row]: its position
    seen = (j <= p[..., None]) & held[:, None, :, 0, 0]
    if s["window"]:
        seen &= (j > p[..., None] - s["window"]) | (j < s["sinks"])
    sc = torch.einsum("brgtd,bjgd->bgrtj", q, k) * (1 / math.sqrt(hd))
    sc = torch.where(seen[:, None, :, None], sc, torch.full((), -torch.inf, device="cuda"))
    top = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(top == -torch.inf, torch.zeros_like(top), top))
    total = e.sum(-1)
    o = torch.einsum("bgrtj,bjgd->bgrtd", e, v) / torch.where(total == 0, torch.ones_like(total), total)[..., None]
    row = torch.arange(m, device="cuda")
    seq = torch.searchsorted(starts, row, right=True) - 1
    return o[seq, :, row - starts[seq]].reshape(m, nh, hd).to(s["q"].dtype)


def _logprobs(s):
    x, n = s["logits"], s["top"]
    d = (x - x.amax(-1, keepdim=True)).double()
    e = torch.exp(d)
    total = e.sum(-1, keepdim=True)
    log = torch.log(total)
    entropy = log[:, 0] - (e * d).sum(-1) / total[:, 0]
    given = d.gather(1, s["tokens"].long()) - log
    best = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :n]            # equal logits: the lowest index first
    return given.float(), entropy.float(), best.int(), (d.gather(1, best) - log).float()


# ---------------------------------------------------------------- from the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        given, entropy, ids, alts = [], [], [], []
        for x, t in zip(s["logits"].cpu().numpy(), s["tokens"].cpu().numpy()):
            y = x.astype(np.float64) - float(x.max())
            rest = np.exp(y)
            rest[int(x.argmax())] = 0
            lp = y - np.log1p(rest.sum())
            given.append(lp[t])
            entropy.append(-(np.exp(lp) * lp).sum())
            near = np.argpartition(-x, min(len(x) - 1, 2 * s["top"] + 64))[:2 * s["top"] + 65] if s["top"] else np.zeros(0, int)
            near = near[np.lexsort((near, -x[near]))][:s["top"]]
            ids.append(near.astype(np.int32))
            alts.append(lp[near])
        return np.array(given), np.array(entropy), np.array(ids), np.array(alts)
    nh, nkv, hd, page = (case[k] for k in ("nh", "nkv", "hd", "page"))
    starts, lens, table = (s[k].cpu().numpy() for k in ("starts", "lens", "table"))
    if case["op"] == "append":
        x = s["qkv"].double().cpu().numpy().reshape(-1, nh + 2 * nkv, hd)
        rope = s["rope"].double().cpu().numpy()
        data = s["data"].double().cpu().numpy()
        q = np.empty((len(x), nh, hd))
        wq, wk = s["q_norm"].double().cpu().numpy(), s["k_norm"].double().cpu().numpy()

        def turn(h, w, cs):
            h = h * (1 / np.sqrt(np.square(h).sum(-1, keepdims=True) / hd + EPS)) * w
            z = (h[..., :hd // 2] + 1j * h[..., hd // 2:]) * (cs[:, 0] + 1j * cs[:, 1])
            return np.concatenate((z.real, z.imag), -1)

        for i in range(case["batch"]):
            for row in range(starts[i], starts[i + 1]):
                p = int(lens[i]) - int(starts[i + 1]) + row
                q[row] = turn(x[row, :nh], wq, rope[p])
                data[table[i, p // page], 0, :, p % page] = turn(x[row, nh:nh + nkv], wk, rope[p])
                data[table[i, p // page], 1, :, p % page] = x[row, nh + nkv:]
        return q, data
    out = torch.zeros(len(s["q"]), nh, hd, dtype=torch.float64, device="cuda")
    for i in range(case["batch"]):
        a, z, n = int(starts[i]), int(starts[i + 1]), int(lens[i])
        pages = s["data"][s["table"][i, :-(-n // page)].long()].transpose(0, 1)            # [K|V][page][kv head][place][hd]
        k, v = pages.transpose(1, 2).reshape(2, nkv, -1, hd)[:, :, :n].double()
        for h in range(nh):
            sc = s["q"][a:z, h].double() @ k[h // (nh // nkv)].T * hd ** -0.5
            p = torch.arange(n - (z - a), n, device="cuda")[:, None]
            back = p - torch.arange(n, device="cuda")
            hidden = back < 0
            if case["window"]:
                hidden |= (back >= case["window"]) & (p - back >= case["sinks"])
            out[a:z, h] = torch.softmax(sc.masked_fill(hidden, -torch.inf), -1) @ v[h // (nh // nkv)]
    return out
