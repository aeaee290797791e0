"""The 4-bit KV cache entries against plain 64-bit arithmetic: rows written
(codes, scales and bytes exactly), read back, attended over, and a run of the
three together.

Tolerances. A rotated query is within 20 f32 roundings (2^-24 each) of its
row's largest normalised value: 9 for the sum of squares and its root, 3
products, one sum, times sqrt 2. Codes and scales are those of the exact values:
no tolerance. Attention: a score is a sum of head_dim products of a query kept
to 22 bits (2^-22 relative at most) in f32, head_dim / 16 + 4 partial sums each
rounded or truncated once (2^-23): within ds = scale * sum|q k| * (2^-22 +
(head_dim / 16 + 4) * 2^-23); an output moves by at most 2 ds times sum p |v|,
plus the P V products (p kept to 22 bits, exp within 2^-22 of its value for an
argument rounded at 2^-24 of up to 128, chains of 2^-23 roundings: 64 of them
in all), so |error| <= (2 ds + 64 * 2^-23) sum p |v|. To that comes a floor: p
times a V scale enters the tensor core as two f16 parts, cut at 2^-24 where the
largest such product may be anything from 2^12 to 2^15 (the unit follows the
largest scale s in steps that leave up to 3 bits free); times a code of at most
8 that is 2^-36 * 8 s for each of n positions, and 8 s is the largest |v|:
n * 2^-36 * max |v|.
"""
import numpy as np
import pytest

from oracle import qw3_oracle as orc

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_transformer_decode_gb300 import build
    build.build()
    return t


def rope_table(capacity, hd, theta=1e6):
    a = np.arange(capacity)[:, None] * theta ** (-2.0 * np.arange(hd // 2) / hd)
    return np.stack((np.cos(a), np.sin(a)), -1).astype(np.float32)


def norm_rope(x, w, cs):
    """x [M, heads, hd] f32 -> (normalised, rotated) in f64."""
    x, w, cs = (np.asarray(v, np.float64) for v in (x, w, cs))
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + np.float64(np.float32(EPS))) * w
    h = x.shape[-1] // 2
    a, b, c, s = n[..., :h], n[..., h:], cs[:, None, :, 0], cs[:, None, :, 1]
    return n, np.concatenate((a * c - b * s, b * c + a * s), -1)


def planes(cache):
    """(codes uint8 [slot][2][head][cap][hd/2], scales f16) of a cache's bytes."""
    raw = cache.data.cpu().numpy()
    cap, hd = cache.capacity, cache.head_dim
    raw = raw[:cache.slots * 2 * cache.n_kv_heads * cap * hd * 9 // 16].reshape(cache.slots, 2, cache.n_kv_heads, -1)
    codes = raw[..., :cap * hd // 2].reshape(*raw.shape[:3], cap, hd // 2)
    scales = np.ascontiguousarray(raw[..., cap * hd // 2:]).view(np.float16).reshape(*raw.shape[:3], cap, hd // 32)
    return codes, scales


def put_rows(cache, torch, k, v):
    """Fill a cache [slots, cap] with encoded rows k, v [slots, cap, nkv, hd] through its bytes; the values that it then
    stands for."""
    out, raw = [], []
    for x, value_row in ((k, False), (v, True)):
        c, s = orc.kv_q4_encode(x)
        out.append(orc.kv_q4_decode(c, s))
        b = orc.kv_q4_row_bytes(c, value_row)
        tr = lambda z: np.ascontiguousarray(np.swapaxes(z, 1, 2))  # noqa: E731  -> [slots, nkv, cap, ...]
        raw.append(np.concatenate([tr(b).reshape(*tr(b).shape[:2], -1),
                                   tr(s).view(np.uint8).reshape(*tr(s).shape[:2], -1)], -1))
    cache.data.copy_(torch.from_numpy(np.stack(raw, 1).reshape(-1)).cuda())
    return out


def new_cache(torch, slots, cap, nkv, hd, fill=0xFF):
    """A cache whose unwritten bytes are NaN scales."""
    from quantized_transformer_decode_gb300.qw3 import KVCacheQ4, qw3_kv_q4_bytes
    return KVCacheQ4(slots, cap, nkv, hd,
                     data=torch.full((qw3_kv_q4_bytes(slots, cap, nkv, hd),), fill, dtype=torch.uint8, device="cuda"))


def cu(torch, x, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(x if dtype is None else np.asarray(x, dtype))).cuda()


# ---------------------------------------------------------------- append and read

@pytest.mark.parametrize("nh,nkv,hd,M,cap", [(16, 8, 128, 1, 64), (32, 8, 128, 37, 96), (4, 2, 64, 19, 32),
                                             (2, 2, 64, 700, 704), (8, 1, 128, 300, 320), (48, 3, 128, 5, 32)])
def test_append_writes_the_exact_codes(torch, nh, nkv, hd, M, cap):
    rng = np.random.default_rng([nh, hd, M])
    slots = 3
    x = rng.standard_normal((M, nh + 2 * nkv, hd)).astype(np.float32) * np.exp(rng.standard_normal((M, 1, 1)) * 2).astype(np.float32)
    qw, kw = (1 + 0.2 * rng.standard_normal((2, hd))).astype(np.float32)
    places = rng.permutation(slots * cap)[:M]
    slot, pos = places // cap, places % cap
    rope = rope_table(cap, hd)
    cache = new_cache(torch, slots, cap, nkv, hd)
    before = cache.data.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = cache.append(cu(torch, x.reshape(M, -1)), cu(torch, qw), cu(torch, kw), EPS, cu(torch, rope),
                     slots=cu(torch, slot, np.int32), pos=cu(torch, pos, np.int32), status=status)
    k, v = cache.read(slots=cu(torch, slot, np.int32), pos=cu(torch, pos, np.int32))
    torch.cuda.synchronize()
    assert int(status) == 0
    qn, want_q = norm_rope(x[:, :nh], qw, rope[pos])
    bound = 20 * 2.0 ** -24 * np.abs(qn).max(-1, keepdims=True)
    assert np.all(np.abs(q.cpu().numpy() - want_q) <= bound)
    _, want_k = norm_rope(x[:, nh:nh + nkv], kw, rope[pos])
    codes, scales = planes(cache)
    for sel, rows, got in ((0, want_k, k), (1, x[:, nh + nkv:].astype(np.float64), v)):
        c, s = orc.kv_q4_encode(rows)
        assert np.array_equal(got.cpu().numpy(), orc.kv_q4_decode(c, s))
        assert np.array_equal(codes[slot, sel, :, pos], orc.kv_q4_row_bytes(c, bool(sel)))
        assert np.array_equal(scales[slot, sel, :, pos], s)
    # everything else in the cache is as it was
    old = new_cache(torch, slots, cap, nkv, hd)
    old.data.copy_(before)
    oc, os_ = planes(old)
    rest = np.ones((slots, cap), bool)
    rest[slot, pos] = False
    for got, was in ((codes, oc), (scales.view(np.uint16), os_.view(np.uint16))):
        assert np.array_equal(np.moveaxis(got, 3, 1)[rest], np.moveaxis(was, 3, 1)[rest])


def test_append_ties_and_borders(torch):
    """Values on the borders between two codes, opposite equals, zero blocks,
    tiny and huge blocks: V rows, whose values are exact."""
    hd, nkv = 128, 1
    rows = []
    for m in (1.0, -1.0, 3.7, -2.0 ** -40, 1e-38, -1e-42, 524000.0, 7.0):
        m = np.float32(m)
        y = np.concatenate([np.arange(-7.5, 8.0, 0.5), [8.0]])             # x / d at halves: exactly on a border
        r = np.zeros(hd, np.float32)
        r[:32] = (np.float64(m) / -8 * y).astype(np.float32)
        r[31] = m
        r[32:64] = np.where(np.arange(32) % 2, m, -m)                      # opposite equals
        r[64:96] = np.nextafter(r[:32], np.float32(0))
        rows.append(r)
    rng = np.random.default_rng(1)
    rows += [np.zeros(hd, np.float32)] + list(np.round(rng.standard_normal((40, hd)) * 4).astype(np.float32))
    V = np.stack(rows)
    M = len(V)
    x = np.zeros((M, 3, hd), np.float32)
    x[:, 1] = rng.standard_normal((M, hd))
    x[:, 2] = V
    one = np.ones(hd, np.float32)
    cache = new_cache(torch, 1, 64, nkv, hd)
    cache.append(cu(torch, x.reshape(M, -1)), cu(torch, one), cu(torch, one), EPS, cu(torch, rope_table(64, hd)))
    _, v = cache.read(n=M)
    c, s = orc.kv_q4_encode(V)
    assert np.array_equal(v.cpu().numpy()[:, 0], orc.kv_q4_decode(c, s))


@pytest.mark.parametrize("hd", [64, 128])
def test_append_decides_near_borders_by_the_exact_value(torch, hd):
    """Many keys: some lie so near a border that f32 cannot decide them."""
    M, nkv = 4096, 4
    rng = np.random.default_rng(hd)
    x = rng.standard_normal((M, 3 * nkv, hd)).astype(np.float32)
    w = (1 + 0.1 * rng.standard_normal(hd)).astype(np.float32)
    rope = rope_table(M, hd)
    cache = new_cache(torch, 1, M, nkv, hd)
    cache.append(cu(torch, x.reshape(M, -1)), cu(torch, w), cu(torch, w), EPS, cu(torch, rope))
    k, _ = cache.read(n=M)
    _, want = norm_rope(x[:, nkv:2 * nkv], w, rope)
    assert np.array_equal(k.cpu().numpy(), orc.kv_q4_decode(*orc.kv_q4_encode(want)))


def test_append_zero_key_rows(torch):
    """A zero head stays zero under the norm; a head whose weight is zero in a
    block gives a zero block only where its partner is zero too."""
    hd = 64
    x = np.zeros((3, 3, hd), np.float32)
    x[1, 1] = 1.0
    x[2, 1, 5] = 1e-30
    w = np.ones(hd, np.float32)
    w[:32] = 0
    rope = rope_table(32, hd)
    cache = new_cache(torch, 1, 32, 1, hd)
    cache.append(cu(torch, x.reshape(3, -1)), cu(torch, w), cu(torch, w), EPS, cu(torch, rope))
    k, v = cache.read(n=3)
    _, want = norm_rope(x[:, 1:2], w, rope[:3])
    assert np.array_equal(k.cpu().numpy(), orc.kv_q4_decode(*orc.kv_q4_encode(want)))
    assert not v.cpu().numpy().any()


def test_append_non_finite_blocks(torch):
    hd, M = 128, 4
    rng = np.random.default_rng(2)
    x = rng.standard_normal((M, 4, hd)).astype(np.float32)       # 2 query heads, 1 key, 1 value
    x[0, 2, 7] = np.nan                                            # a key: its norm is NaN, all blocks go
    x[1, 3, 40] = np.inf                                           # a value: its own block goes
    x[2, 3, 100] = 524160.0
    x[3, 3, 3] = 524159.0                                          # still an f16 scale
    one = np.ones(hd, np.float32)
    rope = rope_table(32, hd)
    cache = new_cache(torch, 1, 32, 1, hd)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.append(cu(torch, x.reshape(M, -1)), cu(torch, one), cu(torch, one), EPS, cu(torch, rope), status=status)
    k, v = (t.cpu().numpy()[:, 0] for t in cache.read(n=M))
    assert int(status) == 5
    assert not k[0].any()
    want = orc.kv_q4_decode(*orc.kv_q4_encode(np.nan_to_num(x[:, 3].astype(np.float64), posinf=0)))
    want[1, 32:64] = 0
    want[2, 96:] = 0
    assert np.array_equal(v, want)
    _, wk = norm_rope(x[1:, 2:3], one, rope[1:4])
    assert np.array_equal(k[1:], orc.kv_q4_decode(*orc.kv_q4_encode(wk))[:, 0])


def test_rows_outside_the_cache_are_left_out(torch):
    hd, cap = 64, 32
    rng = np.random.default_rng(8)
    x = rng.standard_normal((6, 4, hd)).astype(np.float32)
    one = np.ones(hd, np.float32)
    slot = np.array([0, -1, 2, 1, 1, 0], np.int32)
    pos = np.array([3, 3, 3, -1, 32, 31], np.int32)
    cache = new_cache(torch, 2, cap, 1, hd)
    args = (cu(torch, one), cu(torch, one), EPS, cu(torch, rope_table(cap, hd)))
    q = cache.append(cu(torch, x.reshape(6, -1)), *args, slots=cu(torch, slot), pos=cu(torch, pos))
    k, v = cache.read(slots=cu(torch, slot), pos=cu(torch, pos))
    codes, _ = planes(cache)
    written = (codes != 0xFF).any(axis=(1, 2, 4))
    assert np.argwhere(written).tolist() == [[0, 3], [0, 31]]
    for t in (q, k, v):
        t = t.cpu().numpy()
        assert not t[1:5].any() and t[0].any() and t[5].any()


def test_append_in_place_and_strided(torch):
    """The queries may replace themselves in qkv; rows may be strided and start
    at any float."""
    from quantized_transformer_decode_gb300 import qw3
    nh, nkv, hd, M = 4, 2, 128, 9
    rng = np.random.default_rng(4)
    w = (nh + 2 * nkv) * hd
    buf = cu(torch, rng.standard_normal((M, w + 3)).astype(np.float32))
    view = buf[:, 1:1 + w]
    one = cu(torch, np.ones(hd, np.float32))
    rope = cu(torch, rope_table(32, hd))
    a, b = new_cache(torch, 1, 32, nkv, hd), new_cache(torch, 1, 32, nkv, hd)
    want = a.append(view, one, one, EPS, rope, first=7)
    s = torch.cuda.current_stream().cuda_stream
    qw3.qw3_kv_q4_append(b.c, view.data_ptr(), M, w + 3, nh, one.data_ptr(), one.data_ptr(), EPS, rope.data_ptr(), 0, 0,
                         0, 7, view.data_ptr(), w + 3, 0, s)
    assert torch.equal(view[:, :nh * hd].reshape(M, nh, hd), want)
    assert torch.equal(a.data, b.data)


@pytest.mark.parametrize("hd", [64, 128])
def test_append_many_unaligned_rows_and_unaligned_outputs(torch, hd):
    """Several heads to a warp without wide accesses: rows at odd strides and
    starts in, queries and read-back values at odd starts out."""
    from quantized_transformer_decode_gb300 import qw3
    nh, nkv, M = 12, 2, 2500
    rng = np.random.default_rng([hd, 4])
    w = (nh + 2 * nkv) * hd
    x = rng.standard_normal((M, w)).astype(np.float32)
    buf = cu(torch, np.pad(x, ((0, 0), (1, 2))))
    qw, kw = (1 + 0.1 * rng.standard_normal((2, hd))).astype(np.float32)
    rope = rope_table(2528, hd)
    cache = new_cache(torch, 1, 2528, nkv, hd)
    q = torch.full((M * nh * hd + 1,), 5.0, device="cuda")
    kv = torch.full((2, M * nkv * hd + 1), 5.0, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    dq, dk, dr = cu(torch, qw), cu(torch, kw), cu(torch, rope)
    qw3.qw3_kv_q4_append(cache.c, buf[:, 1:].data_ptr(), M, w + 3, nh, dq.data_ptr(), dk.data_ptr(), EPS, dr.data_ptr(), 0,
                         0, 0, 28, q[1:].data_ptr(), nh * hd, 0, s)
    qw3.qw3_kv_q4_read(cache.c, M, 0, 0, 0, 28, kv[0, 1:].data_ptr(), kv[1, 1:].data_ptr(), s)
    x = x.reshape(M, nh + 2 * nkv, hd)
    qn, want_q = norm_rope(x[:, :nh], qw, rope[28:])
    got = q.cpu().numpy()
    assert got[0] == 5 and np.all(np.abs(got[1:].reshape(M, nh, hd) - want_q) <= 20 * 2.0 ** -24 * np.abs(qn).max(-1, keepdims=True))
    _, want_k = norm_rope(x[:, nh:nh + nkv], kw, rope[28:])
    for got, rows in zip(kv.cpu().numpy(), (want_k, x[:, nh + nkv:])):
        assert got[0] == 5
        assert np.array_equal(got[1:].reshape(M, nkv, hd), orc.kv_q4_decode(*orc.kv_q4_encode(rows)))


@pytest.mark.parametrize("scale", [1e-25, 1e-12, 1e12, 1e17])
def test_append_extreme_sizes(torch, scale):
    """Inputs whose squares or products leave two floats' range."""
    hd, M, nkv = 128, 600, 2
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((M, 3 * nkv, hd)) * scale).astype(np.float32)
    x[:, 2 * nkv:] = np.clip(x[:, 2 * nkv:], -5e5, 5e5)
    w = (1 + 0.1 * rng.standard_normal(hd)).astype(np.float32)
    w[5] = 1e-20
    rope = rope_table(608, hd)
    cache = new_cache(torch, 1, 608, nkv, hd)
    cache.append(cu(torch, x.reshape(M, -1)), cu(torch, w), cu(torch, w), EPS, cu(torch, rope))
    k, v = cache.read(n=M)
    _, want = norm_rope(x[:, nkv:2 * nkv], w, rope[:M])
    assert np.array_equal(k.cpu().numpy(), orc.kv_q4_decode(*orc.kv_q4_encode(want)))
    assert np.array_equal(v.cpu().numpy(), orc.kv_q4_decode(*orc.kv_q4_encode(x[:, 2 * nkv:])))


# ---------------------------------------------------------------- attention

def plain_attention(q, k, v, lens, rows, scale):
    """q [B * rows, nh, hd], k and v [B, L, nkv, hd] (values of the sequences in
    order) in f64: (out, error bound)."""
    B, nh, hd = len(lens), q.shape[1], q.shape[2]
    G = nh // k.shape[2]
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        for t in range(rows):
            n = lens[b] - rows + t + 1
            if n <= 0:
                continue
            for h in range(nh):
                kk, vv = k[b, :n, h // G].astype(np.float64), v[b, :n, h // G].astype(np.float64)
                qq = q[b * rows + t, h].astype(np.float64)
                s = kk @ qq * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[b * rows + t, h] = p @ vv
                ds = abs(scale) * (np.abs(kk) @ np.abs(qq)).max() * (2.0 ** -22 + (hd / 16 + 4) * 2.0 ** -23)
                tol[b * rows + t, h] = (2 * ds + 64 * 2.0 ** -23) * (p @ np.abs(vv)) + n * 2.0 ** -36 * np.abs(vv).max() + 1e-30
    return out, tol


def check_attention(torch, nh, nkv, hd, lens, rows=1, slots=None, cap=None, max_len=None, scale=None, seed=0, spread=1.0,
                    vgain=1.0, qgain=1.0):
    rng = np.random.default_rng([nh, nkv, hd, rows, seed, *lens])
    B = len(lens)
    n_slots = B if slots is None else max(max(slots) + 1, B)
    cap = cap or max(32, (max(lens) + 31) // 32 * 32)
    k = rng.standard_normal((n_slots, cap, nkv, hd)) * spread
    v = rng.standard_normal((n_slots, cap, nkv, hd)) * vgain
    cache = new_cache(torch, n_slots, cap, nkv, hd)
    k, v = put_rows(cache, torch, k, v)
    # what lies past each sequence is NaN: it must not be used
    codes, scales = planes(cache)
    order = list(range(B)) if slots is None else list(slots)
    raw = cache.data.view(n_slots, 2, nkv, -1)
    for b, s in enumerate(order):
        raw[s, :, :, cap * hd // 2 + lens[b] * hd // 16:] = 0xFF
        raw[s, :, :, lens[b] * hd // 2:cap * hd // 2] = 0xFF
    q = (rng.standard_normal((B * rows, nh, hd)) * qgain).astype(np.float32)
    got = cache.attention(cu(torch, q), cu(torch, lens, np.int32), rows=rows,
                          slots=None if slots is None else cu(torch, slots, np.int32), max_len=max_len, scale=scale)
    want, tol = plain_attention(q, k[order], v[order], lens, rows, hd ** -0.5 if scale is None else scale)
    got = got.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), float((np.abs(got - want) / np.maximum(tol, 1e-300)).max()))
    norm = np.linalg.norm(want)
    assert norm == 0 or np.linalg.norm(got - want) / norm < 1e-5
    return got


@pytest.mark.parametrize("nh,nkv,hd", [(16, 8, 128), (32, 8, 128), (4, 2, 64), (8, 8, 128), (16, 2, 64), (16, 1, 128),
                                       (6, 2, 64), (10, 2, 128), (64, 64, 64), (5, 1, 64), (14, 2, 128)])
@pytest.mark.parametrize("rows", [1, 3])
def test_attention_heads_and_groups(torch, nh, nkv, hd, rows):
    check_attention(torch, nh, nkv, hd, [1, 67, 200], rows=rows)


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513, 1000, 1025])
def test_attention_lengths(torch, n):
    check_attention(torch, 4, 2, 128, [n])
    check_attention(torch, 4, 2, 64, [n, 3], cap=1056)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 7, 8, 11, 16])
@pytest.mark.parametrize("G", [1, 2, 4, 7, 16])
def test_attention_rows(torch, rows, G):
    """Sequences shorter than the rows leave rows without any position: zeros."""
    got = check_attention(torch, 2 * G, 2, 64, [0, 1, 2, rows, rows + 1, 40, 150], rows=rows)
    assert not got[:rows].any()


@pytest.mark.parametrize("rows", [1, 4])
def test_attention_long_split(torch, rows):
    check_attention(torch, 8, 2, 128, [5001], rows=rows)
    check_attention(torch, 2, 1, 64, [9000, 17, 4096], rows=rows)


@pytest.mark.parametrize("nh,nkv,hd,lens,rows", [(8, 1, 128, [40000], 1), (4, 1, 64, [36001], 3), (2, 2, 64, [33333, 0, 1], 1),
                                                 (4, 1, 128, [34000, 20000], 8)])
def test_attention_results_of_many_ctas(torch, nh, nkv, hd, lens, rows):
    """A few long sequences, whose units more CTAs work on than join in one go."""
    check_attention(torch, nh, nkv, hd, lens, rows=rows)
    if rows == 1:
        check_attention(torch, nh, nkv, hd, lens, rows=rows, spread=6.0)


def test_attention_batch_of_many_lengths(torch):
    rng = np.random.default_rng(5)
    lens = [int(n) for n in rng.integers(0, 400, 40)]
    check_attention(torch, 4, 2, 64, lens, slots=[int(s) for s in rng.permutation(45)[:40]], cap=448)


def test_attention_max_len_is_a_bound(torch):
    """A bound far above the lengths gives the same answers; lengths above it
    are cut to it."""
    a = check_attention(torch, 4, 2, 128, [70, 33], cap=4096, max_len=4096)
    b = check_attention(torch, 4, 2, 128, [70, 33], cap=4096, max_len=70)
    assert np.abs(a - b).max() < 1e-5
    cache = new_cache(torch, 1, 64, 1, 64)
    rng = np.random.default_rng(0)
    put_rows(cache, torch, rng.standard_normal((1, 64, 1, 64)), rng.standard_normal((1, 64, 1, 64)))
    q = cu(torch, rng.standard_normal((1, 2, 64)).astype(np.float32))
    ask = lambda n, m: cache.attention(q, cu(torch, [n], np.int32), max_len=m)  # noqa: E731
    assert torch.equal(ask(64, 40), ask(40, 40)) and torch.equal(ask(2147483647, 64), ask(64, 64))
    assert not ask(-5, 64).any() and not ask(64, 0).any()


@pytest.mark.parametrize("B", [1, 150])
def test_attention_nan_query_stays_in_its_head(torch, B):
    """A NaN query gives a NaN output, and no other head or sequence one."""
    rng = np.random.default_rng(8)
    cache = new_cache(torch, B, 64, 2, 64)
    put_rows(cache, torch, rng.standard_normal((B, 64, 2, 64)), rng.standard_normal((B, 64, 2, 64)))
    q = rng.standard_normal((B, 8, 64)).astype(np.float32)
    lens = cu(torch, np.full(B, 50), np.int32)
    want = cache.attention(cu(torch, q), lens)
    q[0, 5, 3] = np.nan
    got = cache.attention(cu(torch, q), lens)
    bad = torch.isnan(got)
    assert bool(bad[0, 5].all()) and int(bad.sum()) == 64
    assert torch.equal(got[~bad], want[~bad])


def test_attention_slots_outside_and_named_twice(torch):
    rng = np.random.default_rng(6)
    cache = new_cache(torch, 3, 64, 2, 64)
    put_rows(cache, torch, rng.standard_normal((3, 64, 2, 64)), rng.standard_normal((3, 64, 2, 64)))
    q = cu(torch, rng.standard_normal((1, 4, 64)).astype(np.float32).repeat(5, 0))
    got = cache.attention(q, cu(torch, [50, 50, 50, 50, 20], np.int32), slots=cu(torch, [1, -1, 1, 3, 1], np.int32))
    assert torch.equal(got[0], got[2]) and not got[1].any() and not got[3].any() and got[4].any()


@pytest.mark.parametrize("kw", [dict(spread=30.0), dict(vgain=1e-4), dict(vgain=3e4), dict(scale=0.0), dict(scale=-0.3),
                                dict(qgain=1e-20), dict(qgain=1e15, spread=1e-4, scale=1e-12), dict(spread=0.0),
                                dict(vgain=0.0), dict(spread=1e-4, vgain=1e-4)])
def test_attention_ranges(torch, kw):
    """Peaked, flat and reversed scores; tiny and large keys, values, queries."""
    for hd, nh in ((128, 4), (64, 2)):
        check_attention(torch, nh, 2, hd, [300, 45], rows=2, **kw)


@pytest.mark.parametrize("hd,rows,n", [(128, 1, 700), (64, 5, 700), (128, 8, 6000)])
@pytest.mark.parametrize("way", ["up", "down", "late", "steps"])
def test_attention_scores_that_drift(torch, hd, rows, n, way):
    """Scores that rise or fall along the sequence by a fraction of a bit a
    position, that jump in the last tile, or rise in steps; V grows with them."""
    rng = np.random.default_rng([hd, rows, n])
    at = np.arange(n)
    ramp = {"up": at * 0.06, "down": -at * 0.06, "late": np.where(at >= n - 3, 30.0, 0.0),
            "steps": at // 100 * 3.0}[way]
    q = rng.standard_normal((rows, 4, hd)).astype(np.float32)
    k, v = rng.standard_normal((1, n, 2, hd)), rng.standard_normal((1, n, 2, hd)) * 2.0 ** (np.clip(ramp, -20, 20) / 4)[:, None, None]
    for g in range(2):
        # along the first query of the group, in units of its scores
        k[0, :, g] += np.outer(ramp, q[0, 2 * g]) * hd ** 0.5 / (q[0, 2 * g] @ q[0, 2 * g])
    cap = (n + 31) // 32 * 32
    cache = new_cache(torch, 1, cap, 2, hd)
    pad = ((0, 0), (0, cap - n), (0, 0), (0, 0))
    k, v = put_rows(cache, torch, np.pad(k, pad), np.pad(v, pad))
    got = cache.attention(cu(torch, q), cu(torch, [n], np.int32), rows=rows).cpu().numpy()
    want, tol = plain_attention(q, k, v, [n], rows, hd ** -0.5)
    assert np.all(np.abs(got - want) <= tol)


def test_attention_values_of_very_different_sizes(torch):
    """A token with values 10^4 times the others' and a small weight must not
    cost the others their precision."""
    rng = np.random.default_rng(11)
    for big in (0, 100, 290):
        cache = new_cache(torch, 1, 320, 1, 128)
        k, v = rng.standard_normal((1, 320, 1, 128)), rng.standard_normal((1, 320, 1, 128))
        v[0, big] *= 1e4
        q = rng.standard_normal((2, 1, 128)).astype(np.float32) * 3
        k[0, big] = -6 * q[0, 0]
        k, v = put_rows(cache, torch, k, v)
        got = cache.attention(cu(torch, q), cu(torch, [300], np.int32), rows=2).cpu().numpy()
        want, tol = plain_attention(q, k, v, [300], 2, 128 ** -0.5)
        assert np.all(np.abs(got - want) <= tol)


def test_attention_strides_output_and_repeat(torch):
    """Strided rows through the C names; the same call twice gives the same bits;
    what lies between the output rows is left alone."""
    from quantized_transformer_decode_gb300 import qw3
    rng = np.random.default_rng(9)
    nh, nkv, hd, B, rows, cap = 4, 2, 128, 3, 2, 1024
    cache = new_cache(torch, B, cap, nkv, hd)
    put_rows(cache, torch, rng.standard_normal((B, cap, nkv, hd)), rng.standard_normal((B, cap, nkv, hd)))
    q = cu(torch, rng.standard_normal((B * rows, nh * hd + 5)).astype(np.float32))
    lens = cu(torch, [1000, 3, 700], np.int32)
    want = cache.attention(q[:, 1:1 + nh * hd].reshape(B * rows, nh, hd).contiguous(), lens, rows=rows, max_len=1000)
    out = torch.full((B * rows, nh * hd + 7), 77.0, device="cuda")
    n = qw3.qw3_kv_q4_attn_workspace_bytes(B, rows, nh, nkv, hd, 1000)
    ws = torch.full((n + 16,), 0xAB, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        qw3.qw3_kv_q4_attn(cache.c, q[:, 1:].data_ptr(), nh * hd + 5, nh, 0, lens.data_ptr(), B, rows, 1000, hd ** -0.5,
                           out[:, 3:].data_ptr(), nh * hd + 7, ws.data_ptr(), n, 0,
                           torch.cuda.current_stream().cuda_stream)
        assert torch.equal(out[:, 3:3 + nh * hd].reshape(B * rows, nh, hd), want)
    assert bool((out[:, :3] == 77).all()) and bool((out[:, 3 + nh * hd:] == 77).all())
    assert bool((ws[n:] == 0xAB).all())


def test_long_cache_offsets_past_32_bits(torch):
    """A cache of 4.9 GB: the last slot's rows lie past 2^32 bytes."""
    slots, cap, nkv, hd = 33, 65536, 16, 128
    from quantized_transformer_decode_gb300.qw3 import KVCacheQ4
    cache = KVCacheQ4(slots, cap, nkv, hd)
    rng = np.random.default_rng(3)
    n = 130
    x = rng.standard_normal((n, 3 * nkv, hd)).astype(np.float32)
    one = cu(torch, np.ones(hd, np.float32))
    rope = cu(torch, rope_table(cap, hd))
    slot = cu(torch, np.full(n, slots - 1, np.int32))
    last = cap - n
    cache.append(cu(torch, x.reshape(n, -1)), one, one, EPS, rope, slots=slot,
                 pos=cu(torch, np.arange(last, cap, dtype=np.int32)))
    k, v = cache.read(slot=slots - 1, first=last, n=n)
    _, wk = norm_rope(x[:, nkv:2 * nkv], np.ones(hd), rope_table(cap, hd)[last:])
    assert np.array_equal(k.cpu().numpy(), orc.kv_q4_decode(*orc.kv_q4_encode(wk)))
    assert np.array_equal(v.cpu().numpy(), orc.kv_q4_decode(*orc.kv_q4_encode(x[:, 2 * nkv:])))


# ---------------------------------------------------------------- together

def test_a_decode_loop_of_the_operators(torch):
    """Prompt, steps of a ragged batch and a verify block through append and
    attention, each step against f64 over the rows read back."""
    nh, nkv, hd, cap, B = 8, 2, 128, 320, 3
    rng = np.random.default_rng(21)
    w = (nh + 2 * nkv) * hd
    qn, kn = (1 + 0.1 * rng.standard_normal((2, hd))).astype(np.float32)
    rope = cu(torch, rope_table(cap, hd))
    cache = new_cache(torch, B + 1, cap, nkv, hd)
    slots, lens = [2, 0, 3], [100, 31, 257]
    args = (cu(torch, qn), cu(torch, kn), EPS, rope)
    for s, n in zip(slots, lens):
        cache.append(cu(torch, rng.standard_normal((n, w)).astype(np.float32)), *args, slot=s)
    for rows in (1, 1, 4, 1):
        x = cu(torch, rng.standard_normal((B * rows, w)).astype(np.float32))
        at = np.concatenate([np.arange(n, n + rows) for n in lens])
        q = cache.append(x, *args, slots=cu(torch, np.repeat(slots, rows), np.int32), pos=cu(torch, at, np.int32))
        lens = [n + rows for n in lens]
        got = cache.attention(q, cu(torch, lens, np.int32), rows=rows, slots=cu(torch, slots, np.int32)).cpu().numpy()
        k, v = (np.zeros((B, cap, nkv, hd), np.float32) for _ in range(2))
        for b in range(B):
            kk, vv = cache.read(slot=slots[b], n=lens[b])
            k[b, :lens[b]], v[b, :lens[b]] = kk.cpu().numpy(), vv.cpu().numpy()
        want, tol = plain_attention(q.cpu().numpy(), k, v, lens, rows, hd ** -0.5)
        assert np.all(np.abs(got - want) <= tol)


def test_captured_and_replayed(torch):
    """A captured step replays on new contents of the same buffers; two captured
    attentions with workspaces of their own may run at once."""
    nh, nkv, hd, cap = 4, 2, 128, 2048
    rng = np.random.default_rng(31)
    one = cu(torch, np.ones(hd, np.float32))
    rope = cu(torch, rope_table(cap, hd))
    cache = new_cache(torch, 1, cap, nkv, hd)
    cache.append(cu(torch, rng.standard_normal((1500, (nh + 2 * nkv) * hd)).astype(np.float32)), one, one, EPS, rope)
    x = cu(torch, rng.standard_normal((1, (nh + 2 * nkv) * hd)).astype(np.float32))
    slot, pos, lens = cu(torch, [0], np.int32), cu(torch, [1500], np.int32), cu(torch, [1501], np.int32)

    def step():
        q = cache.append(x, one, one, EPS, rope, slots=slot, pos=pos)
        return cache.attention(q, lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(step())
    for n in (1501, 700, 1502):
        x.copy_(cu(torch, rng.standard_normal(x.shape).astype(np.float32)))
        pos.fill_(n - 1)
        lens.fill_(n)
        want = step().clone()
        torch.cuda.synchronize()
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        with torch.cuda.stream(a):
            graphs[0].replay()
        with torch.cuda.stream(b):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_calls_while_another_device_is_current(torch, monkeypatch):
    """The calls go through a switch to the cache's device with all they were
    given (the switch stands in for a second device)."""
    from quantized_transformer_decode_gb300 import qw3
    rng = np.random.default_rng(41)
    nh, nkv, hd, cap = 4, 2, 64, 96
    w = [cu(torch, (1 + 0.1 * rng.standard_normal(hd)).astype(np.float32)) for _ in range(2)]
    rope = cu(torch, rope_table(cap, hd))
    x = cu(torch, rng.standard_normal((5, (nh + 2 * nkv) * hd)).astype(np.float32))
    lens, slots = cu(torch, [7], np.int32), cu(torch, [1], np.int32)
    logits = cu(torch, rng.standard_normal((3, 500)).astype(np.float32))
    one = lambda v, d=np.float32: cu(torch, np.full(3, v), d)  # noqa: E731

    def calls():
        status = cu(torch, [0], np.int32)
        cache = new_cache(torch, 2, cap, nkv, hd)
        q = cache.append(x, *w, EPS, rope, slot=1, first=2, status=status)
        cache.append(x[:2], *w, EPS, rope, slots=cu(torch, [1, 1], np.int32), pos=cu(torch, [0, 1], np.int32))
        rows = cache.read(slot=1, first=3, n=4) + cache.read(cu(torch, [1, 0], np.int32), cu(torch, [2, 95], np.int32))
        out = torch.empty_like(q[:2])
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        got = cache.attention(q[3:], lens, 2, slots, 64, 0.3, out, ws, status)
        token, prob = qw3.sample(logits, one(0.7), one(0.8), one(50, np.int32), one(0.9), one(0.01), status)
        assert got is out and int(status) == 0
        return (q, *rows, out, token, prob)

    want = calls()
    seen = []

    def elsewhere(torch, index):
        seen.append(index)
        return len(seen) % 2 == 1   # asked again after the switch

    monkeypatch.setattr(qw3, "_elsewhere", elsewhere)
    for a, b in zip(want, calls()):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))   # the unwritten row read is NaN
    assert seen == [0] * 12


def test_wrapper_refusals(torch):
    from quantized_transformer_decode_gb300.qw3 import KVCacheQ4, Qw3Error
    cache = KVCacheQ4(2, 64, 2, 64)
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    good = (f(64), f(64), EPS, f(64, 32, 2))
    for bad in (lambda: cache.append(f(3, 500), *good), lambda: cache.append(f(3, 256), *good),
                lambda: cache.append(f(3, 512).half(), *good), lambda: cache.append(f(512, 3).t(), *good),
                lambda: cache.append(f(3, 512), f(63), *good[1:]), lambda: cache.append(f(3, 512), *good[:3], f(63, 32, 2)),
                lambda: cache.append(f(3, 512), *good, slots=i(0, 1)), lambda: cache.append(f(3, 512), *good, slots=i(0, 1, 1).long()),
                lambda: cache.append(f(3, 512), *good, slot=2), lambda: cache.append(f(3, 512), *good, first=62),
                lambda: cache.append(f(3, 512).cpu(), *good),
                lambda: cache.read(), lambda: cache.read(n=-1), lambda: cache.read(n=65), lambda: cache.read(slots=i(0), n=2),
                lambda: cache.attention(f(2, 4, 64), i(1)), lambda: cache.attention(f(1, 4, 32), i(1)),
                lambda: cache.attention(f(1, 4, 64), i(1).long()), lambda: cache.attention(f(1, 4, 64), i(1), max_len=65),
                lambda: cache.attention(f(17, 4, 64), i(1), rows=17), lambda: cache.attention(f(1, 3, 64), i(1)),
                lambda: cache.attention(f(1, 4, 64), i(1), out=f(1, 64, 4)), lambda: cache.attention(f(3, 4, 64), i(1, 1, 1)),
                lambda: cache.attention(f(1, 4, 64).cpu(), i(1)), lambda: KVCacheQ4(2, 64, 2, 64, data=cache.data[:-1])):
        with pytest.raises(Qw3Error):
            bad()
    assert cache.read(n=0)[0].shape == (0, 2, 64) and cache.attention(f(0, 4, 64), i()).shape == (0, 4, 64)
    assert cache.append(f(0, 512), *good).shape == (0, 4, 64)
