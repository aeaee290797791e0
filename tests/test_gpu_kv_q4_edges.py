"""The 4-bit KV cache entries at the ends of f32. Tolerances as in test_gpu_kv_q4.py,
and as derived beside each test."""
import numpy as np
import pytest

from oracle import qw3_oracle as orc
from test_gpu_kv_q4 import EPS, check_attention, cu, new_cache, planes, put_rows, rope_table, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def normed(x, w, cs, eps):
    """norm_rope for any eps."""
    x, w, cs = (np.asarray(v, np.float64) for v in (x, w, cs))
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + np.float64(np.float32(eps))) * w
    h = x.shape[-1] // 2
    a, b, c, s = n[..., :h], n[..., h:], cs[:, None, :, 0], cs[:, None, :, 1]
    return n, np.concatenate((a * c - b * s, b * c + a * s), -1)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("M", [5, 2600])
@pytest.mark.parametrize("scale,eps", [(3e17, EPS), (2e18, EPS), (1e19, EPS), (1e30, EPS), (1e38, EPS), (1e-12, 0.0), (1e-20, 0.0),
                                       (1e-25, 0.0), (1e-38, 0.0), (1e-43, 0.0), (1e-19, 1e-38)])
def test_append_norms_whose_squares_leave_f32(torch, hd, M, scale, eps):  # noqa: F811
    """Finite heads of any size have finite norms: queries within their bound, exact
    codes, no status. (M: one head to a warp, and four.)"""
    nh, nkv = 6, 2
    rng = np.random.default_rng([hd, M])
    x = (np.clip(rng.standard_normal((M, nh + 2 * nkv, hd)), -3.3, 3.3) * scale).astype(np.float32)
    x[:, nh + nkv:] = rng.standard_normal((M, nkv, hd))
    if eps == 0:
        x[:, :, 0] = scale                                    # no head of zeros
    qw, kw = (1 + 0.2 * rng.standard_normal((2, hd))).astype(np.float32)
    cap = (M + 31) // 32 * 32
    rope = rope_table(cap, hd)
    cache = new_cache(torch, 1, cap, nkv, hd)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = cache.append(cu(torch, x.reshape(M, -1)), cu(torch, qw), cu(torch, kw), eps, cu(torch, rope), status=status)
    k, v = cache.read(n=M)
    assert int(status) == 0
    qn, want_q = normed(x[:, :nh], qw, rope[:M], eps)
    assert np.all(np.abs(q.cpu().numpy() - want_q) <= 20 * 2.0 ** -24 * np.abs(qn).max(-1, keepdims=True))
    _, want_k = normed(x[:, nh:nh + nkv], kw, rope[:M], eps)
    assert np.array_equal(k.cpu().numpy(), orc.kv_q4_decode(*orc.kv_q4_encode(want_k)))
    assert np.array_equal(v.cpu().numpy(), orc.kv_q4_decode(*orc.kv_q4_encode(x[:, nh + nkv:])))


@pytest.mark.parametrize("big,fits", [(524159.96875, True), (524160.0, None), (524160.03125, False)])
def test_append_keys_at_the_largest_scale(torch, big, fits):  # noqa: F811
    """Heads of one value c have norm 1 exactly whatever c: a key value just under
    524160 is held, one above is not, and no scale is ever infinite."""
    hd, M = 128, 512
    rng = np.random.default_rng(1)
    x = np.repeat(rng.uniform(0.5, 2, (M, 3, 1)).astype(np.float32), hd, 2)
    w = np.ones(hd, np.float32)
    w[7] = big
    rope = np.zeros((M, hd // 2, 2), np.float32)
    rope[..., 0] = 1
    cache = new_cache(torch, 1, M, 1, hd)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    one = cu(torch, np.ones(hd, np.float32))
    cache.append(cu(torch, x.reshape(M, -1)), one, cu(torch, w), 0.0, cu(torch, rope), status=status)
    k = cache.read(n=M)[0].cpu().numpy()[:, 0]
    assert np.isfinite(k).all()
    want = orc.kv_q4_decode(*orc.kv_q4_encode(np.broadcast_to(np.where(np.arange(hd) == 7, 0.0 if fits is False else big, 1.0), (M, hd))))
    if fits is False:
        want[:, :32] = 0                                      # the whole block goes
    assert np.array_equal(k[:, 32:], want[:, 32:])
    if fits is not None:
        assert np.array_equal(k, want) and int(status) == (0 if fits else 5)


def test_append_subnormal_scales(torch):  # noqa: F811
    """Scales among f16's subnormals, and at the border to zero, to nearest even."""
    hd, M = 64, 256
    rng = np.random.default_rng(2)
    x = np.zeros((M, 3, hd), np.float32)
    step = 8 * 2.0 ** -24
    x[:, 2] = rng.uniform(-1, 1, (M, hd)) * step
    x[:, 2, 3] = -(np.arange(M) / 8) * step                  # scales in eighths of the smallest subnormal, halves among them
    x[:, 2, 40] = np.exp(rng.uniform(np.log(1e-8), np.log(1e-4), M)) * 8
    one = cu(torch, np.ones(hd, np.float32))
    cache = new_cache(torch, 1, M, 1, hd)
    cache.append(cu(torch, x.reshape(M, -1)), one, one, EPS, cu(torch, rope_table(M, hd)))
    assert np.array_equal(cache.read(n=M)[1].cpu().numpy()[:, 0], orc.kv_q4_decode(*orc.kv_q4_encode(x[:, 2])))
    assert np.array_equal(planes(cache)[1][0, 1, 0].view(np.uint16) & 0x7fff, orc.kv_q4_encode(x[:, 2])[1].view(np.uint16) & 0x7fff)


# ---------------------------------------------------------------- attention

SHAPES = [(2, 2, 64, 1, 1), (2, 1, 128, 1, 45), (8, 2, 128, 1, 700), (4, 1, 64, 8, 300), (8, 1, 128, 5, 2000), (8, 1, 128, 1, 40000),
          (4, 2, 64, 3, 36001)]


@pytest.mark.parametrize("nh,nkv,hd,rows,n", SHAPES)
@pytest.mark.parametrize("gain", [1.0, -1e6, 3e7, 1e8, -1e9, 1e12, 1e30])
def test_attention_equal_scores_of_any_size(torch, nh, nkv, hd, rows, n, gain):  # noqa: F811
    """One key throughout: every score of a row is the same number, so the output is
    the mean of V however large that number is (the score's own error drops out of
    the tolerance), V of sizes that differ from tile to tile."""
    rng = np.random.default_rng([nh, hd, rows, n])
    cap = (n + 31) // 32 * 32
    cache = new_cache(torch, 1, cap, nkv, hd)
    k = np.broadcast_to(rng.standard_normal((1, 1, nkv, hd)), (1, cap, nkv, hd))
    v = rng.standard_normal((1, cap, nkv, hd)) * 2.0 ** np.array([3.0, -10.0, 0.0, 4.0, -4.0])[np.arange(cap) // 96 % 5][:, None, None]
    k, v = put_rows(cache, torch, k, v)
    q = rng.standard_normal((rows, nh, hd)).astype(np.float32)
    kk = np.repeat(k[0, 0], nh // nkv, 0)                     # [nh, hd]
    q *= (gain / np.einsum("thd,hd->th", q, kk))[..., None]   # q . k = gain
    got = cache.attention(cu(torch, q.astype(np.float32)), cu(torch, [n], np.int32), rows=rows, scale=1.0).cpu().numpy()
    for t in range(rows):
        m = max(0, n - rows + t + 1)
        vv = np.repeat(v[0, :m], nh // nkv, 1).astype(np.float64)
        want = vv.mean(0) if m else np.zeros((nh, hd))
        tol = 64 * 2.0 ** -23 * np.abs(vv).mean(0) + m * 2.0 ** -36 * np.abs(vv).max() if m else 0.0
        assert np.all(np.abs(got[t] - want) <= tol), (t, float(np.abs(got[t] - want).max()))


@pytest.mark.parametrize("nh,nkv,hd,rows,n", SHAPES[1:])
@pytest.mark.parametrize("gain", [1e7, 1e9, 1e20])
def test_attention_a_winner_by_far(torch, nh, nkv, hd, rows, n, gain):  # noqa: F811
    """Scores so large that only the highest counts: its V, wherever the score's error
    cannot have made another the highest."""
    rng = np.random.default_rng([nh, hd, rows, n, 1])
    cap = (n + 31) // 32 * 32
    cache = new_cache(torch, 1, cap, nkv, hd)
    k, v = put_rows(cache, torch, rng.standard_normal((1, cap, nkv, hd)), rng.standard_normal((1, cap, nkv, hd)) * 0.003)
    q = (rng.standard_normal((rows, nh, hd)) * gain).astype(np.float32)
    got = cache.attention(cu(torch, q), cu(torch, [n], np.int32), rows=rows).cpu().numpy()
    clear = 0
    for t in range(rows):
        for h in range(nh):
            m = n - rows + t + 1
            kk, vv = (x[0, :m, h // (nh // nkv)].astype(np.float64) for x in (k, v))
            s = kk @ q[t, h].astype(np.float64) * hd ** -0.5
            ds = hd ** -0.5 * (np.abs(kk) @ np.abs(q[t, h].astype(np.float64))).max() * (2.0 ** -22 + (hd / 16 + 4) * 2.0 ** -23)
            a, b = np.sort(s)[-2:]
            if b - a > 2 * ds + 40:
                clear += 1
                want = vv[int(np.argmax(s))]
                assert np.all(np.abs(got[t, h] - want) <= 64 * 2.0 ** -23 * np.abs(want) + m * 2.0 ** -36 * np.abs(vv).max())
    assert clear >= 0.7 * rows * nh


@pytest.mark.parametrize("qgain,scale", [(1e36, 1e-36), (6e37, 2e-38), (1e-34, 1e34), (1e-37, 1e37), (3e-39, 1e38)])
def test_attention_the_largest_and_smallest_queries(torch, qgain, scale):  # noqa: F811
    for nh, nkv, hd, rows, lens in ((4, 2, 128, 2, [300, 45]), (2, 2, 64, 1, [77]), (8, 1, 128, 5, [6000, 1])):
        check_attention(torch, nh, nkv, hd, lens, rows=rows, qgain=qgain, scale=scale)


def test_attention_past_32_bits(torch):  # noqa: F811
    """A cache of 4.9 GB: the last slot's rows lie past 2^32 bytes, its last ones past
    2^31 from its start."""
    slots, cap, nkv, hd, nh, n = 2, 2097152, 8, 128, 16, 300
    from quantized_transformer_decode_gb300.qw3 import KVCacheQ4
    cache = KVCacheQ4(slots, cap, nkv, hd)
    cache.data.zero_()                                        # scores 0, V 0 up to the last rows
    rng = np.random.default_rng(3)
    x = rng.standard_normal((n, nh + 2 * nkv, hd)).astype(np.float32)
    one = cu(torch, np.ones(hd, np.float32))
    rope = torch.zeros(cap, hd // 2, 2, device="cuda")
    rope[..., 0] = 1
    q = cache.append(cu(torch, x.reshape(n, -1)), one, one, EPS, rope, slots=cu(torch, np.full(n, slots - 1, np.int32)),
                     pos=cu(torch, np.arange(cap - n, cap, dtype=np.int32)))[-1:] * 4
    got = cache.attention(q, cu(torch, [cap], np.int32), slots=cu(torch, [slots - 1], np.int32)).cpu().numpy()
    k, v = (t.cpu().numpy().astype(np.float64) for t in cache.read(slot=slots - 1, first=cap - n, n=n))
    for h in range(nh):
        s = k[:, h // 2] @ q[0, h].cpu().numpy().astype(np.float64) * hd ** -0.5
        top = max(s.max(), 0.0)
        p, rest = np.exp(s - top), (cap - n) * np.exp(-top)
        p /= p.sum() + rest
        ds = hd ** -0.5 * (np.abs(k[:, h // 2]) @ np.abs(q[0, h].cpu().numpy())).max() * (2.0 ** -22 + (hd / 16 + 4) * 2.0 ** -23)
        # the sum of 2^21 weights: 65536 tiles of 8 heads over 456 CTAs of 4 warps, 4 roundings of 2^-24 to a
        # thread in each: some 1150 of 2^-24
        tol = (2 * ds + (64 + 600) * 2.0 ** -23) * (p @ np.abs(v[:, h // 2])) + n * 2.0 ** -36 * np.abs(v).max()
        assert np.all(np.abs(got[0, h] - p @ v[:, h // 2]) <= tol)


@pytest.mark.parametrize("nh,nkv,hd,rows,lens", [(4, 2, 128, 1, [70]), (4, 2, 64, 3, [5, 0, 2100]), (8, 1, 128, 5, [30000, 400]),
                                                 (2, 1, 64, 1, [130] * 400)])
def test_attention_in_place_of_its_queries(torch, nh, nkv, hd, rows, lens):  # noqa: F811
    rng = np.random.default_rng(4)
    B, cap = len(lens), (max(lens) + 31) // 32 * 32
    cache = new_cache(torch, B, cap, nkv, hd)
    put_rows(cache, torch, rng.standard_normal((B, cap, nkv, hd)), rng.standard_normal((B, cap, nkv, hd)))
    q = cu(torch, rng.standard_normal((B * rows, nh, hd)).astype(np.float32))
    n = cu(torch, lens, np.int32)
    want = cache.attention(q, n, rows=rows)
    assert cache.attention(q, n, rows=rows, out=q) is q and torch.equal(q, want)


def test_places_past_31_bits_are_refused(torch):  # noqa: F811
    """A slot, position or length is not taken modulo 2^32."""
    from quantized_transformer_decode_gb300.qw3 import KVCacheQ4, Qw3Error
    cache = KVCacheQ4(2, 64, 1, 64)
    cache.data.zero_()
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    good = (f(64), f(64), EPS, f(64, 32, 2))
    lens = torch.ones(1, dtype=torch.int32, device="cuda")
    for bad in (lambda: cache.append(f(1, 192), *good, first=2 ** 32), lambda: cache.append(f(1, 192), *good, slot=2 ** 32),
                lambda: cache.read(n=1, first=2 ** 32), lambda: cache.read(n=1, slot=2 ** 32 + 1),
                lambda: cache.attention(f(1, 1, 64), lens, max_len=2 ** 32 + 32),
                lambda: cache.attention(f(1, 1, 64), lens, max_len=-2 ** 32),
                lambda: cache.append(f(1, 192), *good, first=-2 ** 32)):
        with pytest.raises(Qw3Error):
            bad()
    assert not cache.data.any()


def test_every_entry_on_another_device(torch):  # noqa: F811
    """The kernels' limits are set on each device that a call runs on."""
    if torch.cuda.device_count() < 2:
        pytest.skip("one device")
    from quantized_transformer_decode_gb300 import qw3
    rng = np.random.default_rng(7)
    got = []
    for d in ("cuda:0", "cuda:1"):
        dev = lambda x, t=np.float32: torch.from_numpy(np.asarray(x, t)).to(d)  # noqa: B023, E731
        cache = qw3.KVCacheQ4(1, 1024, 2, 128, device=d)
        rng = np.random.default_rng(7)
        one = dev(np.ones(128))
        q = cache.append(dev(rng.standard_normal((900, 8 * 128))), one, one, EPS, dev(rope_table(1024, 128)))
        out = cache.attention(q[-1:].contiguous(), dev([900], np.int32))
        token, prob = qw3.sample(dev(rng.standard_normal((2, 151936))), dev([0.3, 0.6]))
        got.append([t.cpu() for t in (q, out, token, prob)])
    for a, b in zip(*got):
        assert torch.equal(a, b)
