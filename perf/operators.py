"""What a decode step does around the 4-bit KV cache and the logits, as cases to measure.

Four operators, each in its plain form (elementary torch operations) and, where `own` is true, through
`quantized_transformer_decode_gb300.qw3`:

  append     raw q/k/v projections -> per-head Q/K RMSNorm, RoPE, K and V written to the 4-bit cache (the rotated queries
             come out); the rows written are then read back, so that what the cache holds is part of the outputs
  read       cached rows back as f32
  attention  grouped-query attention of 1 to 16 query rows per sequence over the 4-bit cache
  sample     temperature, top-k, top-p and min-p sampling from given uniform numbers

The cache (bytes): [slot][K|V][kv head]{codes [capacity][hd/2], scales [capacity][hd/32] f16}. A row of hd values is hd/32
blocks of 32 values, value = scale * (code - 8). A block's 16 code bytes hold its values in order, the even value in the low
nibble; a K row interleaves the blocks' 4-byte words, a V row their 2-byte halfwords.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
THETA = 1e6
#: (query heads, kv heads, head_dim): this repository's 0.6B and 8B geometries and its tiny one, and groups of 1 and 8.
HEADS = ((16, 8, 128), (32, 8, 128), (4, 2, 64), (8, 8, 128), (16, 2, 64))


def listed():
    return [
        # one token of one conversation, 0.6B heads: the smallest call, where latency counts
        {"name": "append_1_row", "op": "append", "rows": 1, "prefill": False, "slots": 1, "capacity": 1024, "nh": 16, "nkv": 8, "hd": 128},
        # one step of a batch of 64 conversations at scattered positions, 8B heads
        {"name": "append_64_slots", "op": "append", "rows": 64, "prefill": False, "slots": 64, "capacity": 2176, "nh": 32, "nkv": 8, "hd": 128},
        # a 4096-token prompt chunk into one slot, 8B heads
        {"name": "append_prompt_4096", "op": "append", "rows": 4096, "prefill": True, "slots": 2, "capacity": 8320, "nh": 32, "nkv": 8, "hd": 128},
        # an inspection of a short odd run of rows, tiny heads
        {"name": "read_77_rows", "op": "read", "rows": 77, "slots": 3, "capacity": 320, "nkv": 2, "hd": 64},
        # a whole 8192-token conversation back as f32 (a prompt's continuation attends over it)
        {"name": "read_8192_rows", "op": "read", "rows": 8192, "slots": 2, "capacity": 8320, "nkv": 8, "hd": 128},
        # batch-1 decode in a short conversation, 0.6B heads
        {"name": "attn_1x517", "op": "attention", "batch": 1, "rows": 1, "max_len": 517, "ragged": False, "nh": 16, "nkv": 8, "hd": 128},
        # batch-1 decode at a long context, 8B heads
        {"name": "attn_1x8317", "op": "attention", "batch": 1, "rows": 1, "max_len": 8317, "ragged": False, "nh": 32, "nkv": 8, "hd": 128},
        # a batch of 64 conversations of lengths from 1 to 4101, 0.6B heads
        {"name": "attn_64_ragged", "op": "attention", "batch": 64, "rows": 1, "max_len": 4101, "ragged": True, "nh": 16, "nkv": 8, "hd": 128},
        # verifying 5 drafted tokens of 24 conversations of 8192 tokens, 8B heads
        {"name": "attn_24x8192_verify5", "op": "attention", "batch": 24, "rows": 5, "max_len": 8192, "ragged": False, "nh": 32, "nkv": 8, "hd": 128},
        # one token of one conversation from the whole vocabulary, the usual settings
        {"name": "sample_1", "op": "sample", "batch": 1, "vocab": 151936, "settings": "usual"},
        # a batch of 64 conversations, each with its own settings
        {"name": "sample_64_mixed", "op": "sample", "batch": 64, "vocab": 151936, "settings": "mixed"},
        # a small odd vocabulary without any cut
        {"name": "sample_7_small", "op": "sample", "batch": 7, "vocab": 4099, "settings": "open"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "read", "attention", "attention", "sample"))
    nh, nkv, hd = rng.choice(HEADS)
    if op == "append":
        prefill = rng.random() < 0.5
        rows = _log_int(rng, 1, 4096 if prefill else 64)
        slots = rng.randint(1, 4) if prefill else rng.randint(rows, 64)
        capacity = 32 * _log_int(rng, max(1, -(-rows // 32)) if prefill else 2, 260)
        return {"op": op, "rows": rows, "prefill": prefill, "slots": slots, "capacity": capacity, "nh": nh, "nkv": nkv, "hd": hd}
    if op == "read":
        rows = _log_int(rng, 1, 8192)
        return {"op": op, "rows": rows, "slots": rng.randint(1, 3), "capacity": 32 * rng.randint(-(-rows // 32), 260), "nkv": nkv, "hd": hd}
    if op == "attention":
        batch = _log_int(rng, 1, 64)
        max_len = _log_int(rng, 1, min(8400, 24 * 8192 // batch))
        return {"op": op, "batch": batch, "rows": rng.choice((1, 1, 1, 2, 3, 5, 8, 16)) if batch <= 8 else rng.choice((1, 1, 4)),
                "max_len": max_len, "ragged": rng.random() < 0.5, "nh": nh, "nkv": nkv, "hd": hd}
    return {"op": op, "batch": _log_int(rng, 1, 64), "vocab": _log_int(rng, 1000, 152064), "settings": rng.choice(("usual", "mixed", "open"))}


def _lens(case):
    """The batch's lengths (before they are shuffled): from 1 to max_len in equal steps, or max_len everywhere."""
    b, n = case["batch"], case["max_len"]
    if not case["ragged"] or b == 1:
        return [n] * b
    return [1 + (n - 1) * i // (b - 1) for i in range(b)]


def work(case):
    if case["op"] == "append":
        m, nh, nkv, hd = case["rows"], case["nh"], case["nkv"], case["hd"]
        held = 2 * nkv * hd * 9 / 16
        return {"bytes": m * ((nh + 2 * nkv) * hd * 4 + hd * 4 + 8 + nh * hd * 4 + 2 * held + 2 * nkv * hd * 4),
                "flops": m * ((nh + nkv) * hd * 7 + 2 * nkv * hd * 4)}
    if case["op"] == "read":
        m, nkv, hd = case["rows"], case["nkv"], case["hd"]
        return {"bytes": m * (2 * nkv * hd * (9 / 16 + 4) + 8), "flops": m * 2 * nkv * hd}
    if case["op"] == "attention":
        total, t, nh, nkv, hd = sum(_lens(case)), case["rows"], case["nh"], case["nkv"], case["hd"]
        return {"bytes": total * 2 * nkv * hd * 9 / 16 + 2 * case["batch"] * t * nh * hd * 4 + 8 * case["batch"],
                "flops": 4 * total * t * nh * hd}
    return {"bytes": case["batch"] * (case["vocab"] * 4 + 28), "flops": case["batch"] * case["vocab"] * 4}


# ---------------------------------------------------------------- the cache in its plain form

def _head_bytes(capacity, hd):
    return capacity * (hd // 2 + hd // 16)


def _planes(cache, slots, capacity, nkv, hd):
    """Views of the cache: codes [slot][K|V][head][capacity][hd/2] and scales [slot][K|V][head][capacity][hd/32]."""
    c = cache.view(slots, 2, nkv, _head_bytes(capacity, hd))
    codes = c[..., :capacity * hd // 2].unflatten(-1, (capacity, hd // 2))
    scales = c[..., capacity * hd // 2:].view(torch.float16).unflatten(-1, (capacity, hd // 32))
    return codes, scales


def _half(d):
    """d rounded once to f16, nearest even: through f32 with the bits below it kept as an odd last bit."""
    f, d = d.float(), d.double()
    f = torch.where(f.double().abs() > d.abs(), torch.nextafter(f, torch.zeros_like(f)), f)
    return (f.view(torch.int32) | (f.double() != d).int()).view(torch.float32).half()


def _encode(x):
    """Blocks of x [..., hd] (float64): scales [..., hd/32] f16 and codes [..., hd/32, 32] as whole float64."""
    b = x.unflatten(-1, (-1, 32))
    p, n = b.amax(-1), (-b).amax(-1)
    m = torch.where(p >= n, p, -n)
    y = b * -8 / torch.where(m == 0, torch.ones_like(m), m)[..., None]
    code = torch.floor(y + 8.5).clamp(0, 15)
    return _half(m / -8), torch.where((m == 0)[..., None], torch.full_like(code, 8), code)


def _pack(code, word):
    """Codes [..., nb, 32] -> row bytes [..., 16 nb], the blocks interleaved in words of `word` bytes."""
    c = code.to(torch.uint8).unflatten(-1, (16, 2))
    byte = c[..., 0] | (c[..., 1] << 4)
    return byte.unflatten(-1, (16 // word, word)).transpose(-3, -2).flatten(-3)


def _unpack(rows, scales, word):
    """Row bytes [..., 16 nb] and scales [..., nb] -> values [..., 32 nb], f32."""
    nb = scales.shape[-1]
    byte = rows.unflatten(-1, (16 // word, nb, word)).transpose(-3, -2).flatten(-2)
    code = torch.stack((byte & 15, byte >> 4), -1).flatten(-2)
    return ((code.float() - 8) * scales.float()[..., None]).flatten(-2)


def _rope_table(capacity, hd):
    i = torch.arange(hd // 2, dtype=torch.float64, device="cuda")
    a = torch.arange(capacity, dtype=torch.float64, device="cuda")[:, None] * THETA ** (-2 * i / hd)
    return torch.stack((a.cos(), a.sin()), -1).float()


def _normed(x, w, cs, dtype):
    """Per-head RMSNorm and rotation of x [M][heads][hd] in `dtype`."""
    x, w, cs = x.to(dtype), w.to(dtype), cs.to(dtype)
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    a, b = x.chunk(2, -1)
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _random_cache(g, slots, capacity, nkv, hd):
    """A cache full of encoded rows: keys after their norm (unit size, a few channels larger), values around 0.4."""
    cache = torch.empty(slots * 2 * nkv * _head_bytes(capacity, hd), dtype=torch.uint8, device="cuda")
    codes, scales = _planes(cache, slots, capacity, nkv, hd)
    gain = 1 + 0.3 * torch.randn(2, nkv, 1, hd, generator=g, device="cuda").abs()
    gain[1] *= 0.4
    for s in range(slots):
        x = torch.randn(2, nkv, capacity, hd, generator=g, device="cuda") * gain
        sc, code = _encode(x)
        scales[s] = sc
        codes[s, 0] = _pack(code[0], 4)
        codes[s, 1] = _pack(code[1], 2)
    return cache


# ---------------------------------------------------------------- states

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    ints = lambda v: torch.tensor([int(x) for x in v], dtype=torch.int32, device="cuda")  # noqa: E731
    rnd = np.random.default_rng(int(seed))
    s = dict(case)
    if case["op"] == "append":
        m, nh, nkv, hd, cap = (case[k] for k in ("rows", "nh", "nkv", "hd", "capacity"))
        s["qkv"] = torch.randn(m, (nh + 2 * nkv) * hd, generator=g, device="cuda") * 0.7
        s["q_norm"] = 1 + 0.1 * torch.randn(hd, generator=g, device="cuda")
        s["k_norm"] = 1 + 0.1 * torch.randn(hd, generator=g, device="cuda")
        s["rope"] = _rope_table(cap, hd)
        s["cache"] = torch.randint(0, 256, (case["slots"] * 2 * nkv * _head_bytes(cap, hd),), generator=g, device="cuda", dtype=torch.uint8)
        if case["prefill"]:
            first = int(rnd.integers(0, cap - m + 1))
            s["slot"], s["pos"] = ints([rnd.integers(0, case["slots"])] * m), ints(range(first, first + m))
        else:
            s["slot"], s["pos"] = ints(rnd.permutation(case["slots"])[:m]), ints(rnd.integers(0, cap, m))
    elif case["op"] == "read":
        m, cap = case["rows"], case["capacity"]
        s["cache"] = _random_cache(g, case["slots"], cap, case["nkv"], case["hd"])
        first = int(rnd.integers(0, cap - m + 1))
        s["slot"], s["pos"] = ints([rnd.integers(0, case["slots"])] * m), ints(range(first, first + m))
    elif case["op"] == "attention":
        b, t, nh, nkv, hd = (case[k] for k in ("batch", "rows", "nh", "nkv", "hd"))
        s["capacity"] = -(-case["max_len"] // 32) * 32
        s["slots"] = b
        s["cache"] = _random_cache(g, b, s["capacity"], nkv, hd)
        s["q"] = torch.randn(b * t, nh, hd, generator=g, device="cuda") * 1.2
        s["lens"] = ints(rnd.permutation(_lens(case)))
        s["slot"] = ints(rnd.permutation(b))
    else:
        b, v = case["batch"], case["vocab"]
        # a spread-out vocabulary with a few hundred candidates well above it, as a language model's logits have
        x = torch.randn(b, v, generator=g, device="cuda") * 2.2
        top = torch.randint(0, v, (b, min(400, v)), generator=g, device="cuda")
        x.scatter_add_(1, top, -2.5 * torch.log(torch.rand(top.shape, generator=g, device="cuda").clamp_min(1e-6)))
        s["logits"] = x
        s["u"] = torch.rand(b, generator=g, device="cuda")
        kind = [case["settings"]] * b if case["settings"] != "mixed" else [("usual", "open", "top_p", "top_k", "greedy")[i % 5] for i in range(b)]
        table = {"usual": (0.7, 20, 0.95, 0.02), "open": (1.0, 0, 1.0, 0.0), "top_p": (1.1, 0, 0.92, 0.0), "top_k": (0.9, 200, 1.0, 0.0), "greedy": (0.0, 0, 1.0, 0.0)}
        cols = list(zip(*(table[k] for k in kind)))
        f32 = lambda v: torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = f32(cols[0]), ints(cols[1]), f32(cols[2]), f32(cols[3])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    return {"append": _append, "read": _read, "attention": _attention, "sample": _sample}[s["op"]](s)


def _own(s):
    from quantized_transformer_decode_gb300 import qw3
    if s["op"] == "sample":
        return qw3.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    cache = qw3.KVCacheQ4(s["slots"], s["capacity"], s["nkv"], s["hd"], data=s["cache"])
    if s["op"] == "append":
        q = cache.append(s["qkv"], s["q_norm"], s["k_norm"], EPS, s["rope"], slots=s["slot"], pos=s["pos"])
        return (q, *cache.read(slots=s["slot"], pos=s["pos"]))
    if s["op"] == "read":
        return cache.read(slots=s["slot"], pos=s["pos"])
    return cache.attention(s["q"], s["lens"], rows=s["rows"], slots=s["slot"], max_len=s["max_len"])


def _append(s):
    nh, nkv, hd = s["nh"], s["nkv"], s["hd"]
    x = s["qkv"].unflatten(-1, (nh + 2 * nkv, hd))
    slot, pos = s["slot"].long(), s["pos"].long()
    cs = s["rope"][pos]
    q = _normed(x[:, :nh], s["q_norm"], cs, torch.float32)
    # a code is decided at a border between two: 64 bits up to there
    ks, kc = _encode(_normed(x[:, nh:nh + nkv], s["k_norm"], cs, torch.float64))
    vs, vc = _encode(x[:, nh + nkv:].double())
    codes, scales = _planes(s["cache"], s["slots"], s["capacity"], nkv, hd)
    codes[slot, 0, :, pos] = _pack(kc, 4)
    codes[slot, 1, :, pos] = _pack(vc, 2)
    scales[slot, 0, :, pos] = ks
    scales[slot, 1, :, pos] = vs
    return (q, *_read(s))


def _read(s):
    codes, scales = _planes(s["cache"], s["slots"], s["capacity"], s["nkv"], s["hd"])
    slot, pos = s["slot"].long(), s["pos"].long()
    return _unpack(codes[slot, 0, :, pos], scales[slot, 0, :, pos], 4), _unpack(codes[slot, 1, :, pos], scales[slot, 1, :, pos], 2)


def _attention(s):
    b, t, nh, nkv, hd, n = s["batch"], s["rows"], s["nh"], s["nkv"], s["hd"], s["max_len"]
    codes, scales = _planes(s["cache"], s["slots"], s["capacity"], nkv, hd)
    slot = s["slot"].long()
    k = _unpack(codes[slot, 0, :, :n], scales[slot, 0, :, :n], 4)
    v = _unpack(codes[slot, 1, :, :n], scales[slot, 1, :, :n], 2)
    q = s["q"].view(b, t, nkv, nh // nkv, hd).transpose(1, 2)                       # [b][kv head][row][group][hd]
    sc = torch.einsum("bgthd,bgjd->bgthj", q, k) / math.sqrt(hd)
    last = s["lens"].long()[:, None] - t + torch.arange(t, device="cuda")             # [b][row]: the row's own position
    seen = (torch.arange(n, device="cuda") <= last[..., None])[:, None, :, None]
    sc = torch.where(seen, sc, torch.full_like(sc, -torch.inf))
    top = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - torch.where(top == -torch.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("bgthj,bgjd->bgthd", e, v) / torch.where(total == 0, torch.ones_like(total), total)
    return o.transpose(1, 2).reshape(b * t, nh, hd)


def _sample(s):
    x, v = s["logits"], s["vocab"]
    temp, k, p, mp = s["temperature"].double(), s["top_k"].long(), s["top_p"].double(), s["min_p"].double()
    greedy = temp <= 0
    sx, order = torch.sort(x, dim=-1, descending=True, stable=True)                  # equal logits: the lowest index first
    w = torch.exp((sx.double() - sx[:, :1].double()) / torch.where(greedy, torch.ones_like(temp), temp)[:, None])
    rank = torch.arange(v, device="cuda")
    k = torch.where(greedy, torch.ones_like(k), torch.where(k <= 0, torch.full_like(k, v), k))
    w = torch.where(rank < k[:, None], w, torch.zeros_like(w))
    before = torch.cumsum(w, -1) - w
    keep = (before < (p * w.sum(-1))[:, None]) | (p >= 1)[:, None]
    keep = (keep & (w >= mp[:, None])) | (rank == 0)
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, torch.zeros_like(w)))
    c = torch.cumsum(w, -1)
    token = (c <= (s["u"].double() * c[:, -1])[:, None]).sum(-1, keepdim=True)
    return token.squeeze(1).int(), (w.gather(1, token) / c[:, -1:]).squeeze(1).float()


# ---------------------------------------------------------------- from the definition, in 64 bits

def _values(s, which):
    """Every cached value [slots][head][capacity][hd] of K (0) or V (1) in f64, by the place of each value."""
    nkv, hd, cap = s["nkv"], s["hd"], s["capacity"]
    nb = hd // 32
    d = np.arange(hd)
    block, byte = d // 32, d % 32 // 2
    u = 4 if which == 0 else 2
    at = torch.from_numpy((byte // u * nb + block) * u + byte % u).cuda()
    shift = torch.from_numpy(d % 2 * 4).cuda()
    raw = s["cache"].view(s["slots"], 2 * nkv, -1)[:, which * nkv:(which + 1) * nkv]
    for b in range(s["slots"]):
        row = raw[b, :, :cap * hd // 2].reshape(nkv, cap, hd // 2)[..., at].int()
        sc = raw[b, :, cap * hd // 2:].contiguous().view(torch.float16).view(nkv, cap, nb).double()
        yield (((row >> shift) & 15) - 8).double() * sc[..., torch.from_numpy(block).cuda()]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        nh, nkv, hd = s["nh"], s["nkv"], s["hd"]
        x = s["qkv"].double().cpu().numpy().reshape(s["rows"], nh + 2 * nkv, hd)
        cs = s["rope"].double().cpu().numpy()[s["pos"].cpu().numpy()][:, None]

        def turn(h, w):
            h = h * (1 / np.sqrt(np.square(h).sum(-1, keepdims=True) / hd + EPS)) * w.double().cpu().numpy()
            z = (h[..., :hd // 2] + 1j * h[..., hd // 2:]) * (cs[..., 0] + 1j * cs[..., 1])
            return np.concatenate((z.real, z.imag), -1)

        def held(h):
            h = h.reshape(*h.shape[:-1], hd // 32, 32)
            hi, lo = h.max(-1, keepdims=True), h.min(-1, keepdims=True)
            m = np.where(hi >= -lo, hi, lo)
            with np.errstate(divide="ignore", invalid="ignore"):
                code = np.where(m == 0, 0, np.minimum(np.floor(-8 * h / m + 0.5), 7))
            return (code * (m / -8).astype(np.float16).astype(np.float64)).reshape(s["rows"], nkv, hd)

        return turn(x[:, :nh], s["q_norm"]), held(turn(x[:, nh:nh + nkv], s["k_norm"])), held(x[:, nh + nkv:])
    if case["op"] == "read":
        slot, pos = s["slot"].long(), s["pos"].long()
        got = []
        for which in (0, 1):
            rows = torch.stack([v[:, pos].transpose(0, 1) for v in _values(s, which)])
            got.append(rows[slot, torch.arange(len(pos), device="cuda")])
        return tuple(got)
    if case["op"] == "attention":
        b, t, nh, nkv, hd = (case[k] for k in ("batch", "rows", "nh", "nkv", "hd"))
        place = {int(x): i for i, x in enumerate(s["slot"].tolist())}
        lens = s["lens"].tolist()
        out = torch.zeros(b, t, nh, hd, dtype=torch.float64, device="cuda")
        for slot, (k, v) in enumerate(zip(_values(s, 0), _values(s, 1))):
            i = place[slot]
            for r in range(t):
                n = lens[i] - t + r + 1
                if n > 0:
                    q = s["q"].view(b, t, nkv, nh // nkv, hd)[i, r].double()
                    a = torch.softmax(q @ k[:, :n].transpose(1, 2) * hd ** -0.5, -1)
                    out[i, r] = (a @ v[:, :n]).reshape(nh, hd)
        return out.reshape(b * t, nh, hd)
    tokens, probs = [], []
    for i in range(case["batch"]):
        x = s["logits"][i].double().cpu().numpy()
        temp, k, p, mp, u = (float(s[n][i]) for n in ("temperature", "top_k", "top_p", "min_p", "u"))
        if temp <= 0:
            tokens.append(int(np.argmax(x)))
            probs.append(1.0)
            continue
        by = np.argsort(-x, kind="stable")
        if k > 0:
            by = by[:int(k)]
        w = np.exp((x[by] - x[by[0]]) / temp)
        if p < 1:
            n = int(np.searchsorted(np.cumsum(w), p * w.sum(), side="left")) + 1
            by, w = by[:n], w[:n]
        some = (w >= mp) | (np.arange(len(w)) == 0)
        by, w = by[some], w[some]
        at = np.argsort(by)
        c = np.cumsum(w[at])
        j = min(int(np.searchsorted(c, u * c[-1], side="right")), len(c) - 1)
        tokens.append(int(by[at[j]]))
        probs.append(float(w[at[j]] / c[-1]))
    return np.array(tokens, np.int32), np.array(probs)
