"""Log probabilities, entropies and alternatives against 64-bit arithmetic.

Tolerances. In R, the sum of the other terms over the largest one, a term e^d is
within 2^-22 of its value (the exponential) and |d| 2^-23 (its argument d log2 e,
rounded twice at 2^-24 of at most 1.45 |d|), or within 2^-149 where it is
subnormal (half a step, or flushed to zero: then below 2^-126, see below); a sum
of up to 2^22 terms runs over 2^9 of a thread's and 20 joins (2^-24 each, random
in sign: 2^-19 with room):
    dR = sum e^d (2^-22 + |d| 2^-23) + 2^-19 R + V 2^-149.
(A flushed term loses up to 2^-126; where that is not nothing beside R, R is
itself below V 2^-100, and the kernel's exponential keeps subnormal values.)
log1p(R) then moves by at most dR / (1 + R) and has two roundings of 2^-23 of its
own, l - max one. So
    |dp| <= dR / (1 + R) + 2^-22 (|l - max| + log1p R),
and 2^-149 for a result that is subnormal. The entropy's second term W / (1 + R)
moves by the same relative amounts, twice over. A log probability below the
least f32 is -inf in f32.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.skip("no CUDA device")
    from quantized_transformer_decode_gb300 import build
    build.build()
    return t


def expect(x, tokens, top):
    """(log p of all, entropy, best ids, tolerances) of one row, in f64."""
    y = x.astype(np.float64)
    best = int(np.argmax(y))
    d = y - y[best]
    e = np.exp(d)
    rest = e.sum() - 1 if e.sum() > 2 else np.delete(e, best).sum()
    log = np.log1p(rest)
    w = -(e[e > 0] * d[e > 0]).sum() / (1 + rest)
    with np.errstate(invalid="ignore", over="ignore"):
        lp = d - log
        far = np.where(e > 0, np.abs(d), 0)
        dr = (e * (2.0 ** -22 + far * 2.0 ** -23)).sum() + 2.0 ** -19 * rest + len(x) * 2.0 ** -149
        tol = dr / (1 + rest) + 2.0 ** -22 * (np.abs(d) + log) + 2.0 ** -149
    dw = (e * far * (2.0 ** -22 + far * 2.0 ** -23)).sum() + 2.0 ** -19 * w * (1 + rest) + len(x) * 200 * 2.0 ** -149
    etol = (1 + w) * dr / (1 + rest) + dw / (1 + rest) + 2.0 ** -22 * (log + w)
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf][:top]
    return lp, log + w, order, tol, etol


def near(got, want, tol):
    return np.where(want < -3.4028235e38, got == -np.inf, np.abs(got - want) <= tol).all()


def check(torch, x, tokens=None, top=0, dev=None):
    from quantized_transformer_decode_gb300 import qw3
    x = np.asarray(x, np.float32)
    B, V = x.shape
    if tokens is None:
        tokens = np.random.default_rng(1).integers(0, V, (B, 2)).astype(np.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = qw3.logprobs(torch.from_numpy(x).cuda() if dev is None else dev, torch.from_numpy(tokens).cuda(), top=top, status=status)
    lp, h, ids, alts = (t.cpu().numpy() for t in got)
    assert int(status) == 0 and lp.shape == tokens.shape and ids.shape == alts.shape == (B, top)
    for i in range(B):
        want, entropy, order, tol, etol = expect(x[i], tokens[i], top)
        for t, v in zip(np.atleast_1d(tokens[i]), np.atleast_1d(lp[i])):
            if not 0 <= t < V or want[t] < -3.4028235e38:
                assert v == -np.inf
            else:
                assert abs(v - want[t]) <= tol[t], (i, t, v, want[t], tol[t])
        assert abs(h[i] - entropy) <= etol, (i, h[i], entropy, etol)
        assert np.array_equal(ids[i, :len(order)], order) and (ids[i, len(order):] == -1).all()
        assert near(alts[i, :len(order)], want[order], tol[order]) and (alts[i, len(order):] == -np.inf).all()
    return got


def rows(B, V, seed=0, spread=2.2):
    g = np.random.default_rng(seed)
    x = g.standard_normal((B, V)) * spread
    k = min(V, 300)
    for r in x:
        r[g.permutation(V)[:k]] += g.exponential(2.5, k)
    return x.astype(np.float32)


@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 64, 1000, 4099, 8192, 8193, 32768, 50257, 151936])
@pytest.mark.parametrize("top", [0, 1, 5, 20, 64])
def test_vocabularies(torch, V, top):
    check(torch, rows(3, V, V), top=top)


@pytest.mark.parametrize("B,V", [(1, 151936), (7, 20011), (80, 20011), (300, 9001), (700, 9001), (1300, 4099)])
def test_row_counts(torch, B, V):
    """Every cluster size, one CTA to a row among them."""
    check(torch, rows(B, V, B), top=5)


def test_the_largest_vocabulary(torch):
    x = np.random.default_rng(0).standard_normal((1, 1 << 22)).astype(np.float32)
    check(torch, x, top=64)


@pytest.mark.parametrize("kind", ["ascending", "descending", "flat", "two", "blocks", "masked", "late", "lowest"])
@pytest.mark.parametrize("B,V", [(1, 151936), (2, 8200), (700, 30011)])
def test_orders_ties_and_masks(torch, kind, B, V):
    """Lists that overflow, plateaus, masks of -inf and of the type's lowest value."""
    i = np.arange(V)
    lowest = np.finfo(np.float32).min
    x = {"ascending": i * 1e-3, "descending": -i * 1e-3, "flat": np.zeros(V), "two": i % 2, "blocks": i // 1000 % 7 * 1.0,
         "masked": np.where(i % 3 == 0, i % 101 * 0.1, -np.inf), "late": np.where(i > V - 30, i * 1.0, -np.inf),
         "lowest": np.where(i % 5000 == 77, 1.0, lowest)}[kind].astype(np.float32)
    from quantized_transformer_decode_gb300 import qw3
    if B < 100:
        check(torch, np.tile(x, (B, 1)), top=64)
        check(torch, np.tile(x, (B, 1)), top=3)
        return
    # many rows of one: the first is checked, the others equal it
    dev = torch.from_numpy(x).cuda().expand(B, V).contiguous()
    got = qw3.logprobs(dev, torch.zeros(B, dtype=torch.int32, device="cuda"), top=20)
    for t in got:       # (rows that begin at the same place of a 16-byte word, as every fourth does, add in the same order)
        for k in range(4):
            assert torch.equal(t[k::4], t[k:k + 1].expand_as(t[k::4]))
    lp, h, order, tol, etol = expect(x, [0], 20)
    assert np.array_equal(got[2][0].cpu().numpy()[:len(order)], order) and abs(float(got[1][0]) - h) <= etol


def test_certain_rows(torch):
    """A token of almost all the probability keeps its digits."""
    x = np.full((4, 3001), -20.0, np.float32)
    x[0, 7] = 10.0          # 1 - p = 3000 e^-30
    x[1, 3000] = 80.0
    x[2, :] = -np.inf
    x[2, 5] = 3.0           # the only one
    x[3, 1:3] = 15.0
    lp, h, ids, _ = check(torch, x, tokens=np.array([[7], [3000], [5], [2]], np.int32), top=4)
    assert abs(float(lp[0, 0]) + 3000 * np.exp(-30.0)) < 1e-5 * 3000 * np.exp(-30.0)
    assert float(lp[2, 0]) == 0 and float(h[2]) == 0 and ids[2].tolist() == [5, -1, -1, -1]


def test_large_logits(torch):
    g = np.random.default_rng(3)
    for size in (1e4, 1e30, 3e38, 1e-30):
        check(torch, (g.uniform(-1, 1, (3, 5000)) * size).astype(np.float32), top=7)
    x = np.full((1, 100), -3.4028234663852886e38, np.float32)
    check(torch, x, top=3)              # all at the type's lowest: a flat row
    x[0, 50] = 3.4028234663852886e38
    check(torch, x, top=3)


def test_rows_without_an_answer(torch):
    from quantized_transformer_decode_gb300 import qw3
    for V in (100, 50000):
        for B in (8, 700):
            x = rows(B, V)
            x[1, V // 2] = np.nan
            x[3, V - 1] = np.inf
            x[4, :] = -np.inf
            x[6, [0, V - 1]] = np.inf, np.nan
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            lp, h, ids, alts = qw3.logprobs(torch.from_numpy(x).cuda(), torch.zeros(B, dtype=torch.int32, device="cuda"), top=3,
                                            status=status)
            assert int(status) == 5
            dead = [1, 3, 4, 6]
            assert torch.isnan(lp[dead]).all() and torch.isnan(h[dead]).all() and (ids[dead] == -1).all() and torch.isnan(alts[dead]).all()
            live = [i for i in range(B) if i not in dead]
            assert torch.isfinite(lp[live]).all() and torch.isfinite(h[live]).all() and (ids[live] >= 0).all()


def test_tokens_outside_the_vocabulary_and_none(torch):
    from quantized_transformer_decode_gb300 import qw3
    check(torch, rows(3, 501), tokens=np.array([[-1, 0, 501], [500, 2 ** 31 - 1, -2 ** 31], [3, 3, 3]], np.int32))
    lp, h, ids, alts = qw3.logprobs(torch.zeros((4, 9), device="cuda"), torch.zeros((4, 0), dtype=torch.int32, device="cuda"))
    assert lp.shape == (4, 0) and ids.shape == (4, 0) and torch.allclose(h, torch.full_like(h, np.log(9)))
    lp, _, _, _ = qw3.logprobs(torch.zeros((0, 9), device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert lp.shape == (0,)
    check(torch, rows(5, 77), tokens=np.arange(5, dtype=np.int32))


@pytest.mark.parametrize("V,stride,first", [(1001, 1001, 0), (1001, 1003, 1), (20002, 20005, 3), (9, 10, 2), (3, 7, 1), (40000, 40001, 0)])
def test_strides_and_odd_alignments(torch, V, stride, first):
    """Rows that begin at any 4-byte boundary; what lies around them is not read into them."""
    wide = torch.full((6, stride + 4), float("nan"), device="cuda")
    x = rows(6, V, 5)
    flat = wide.flatten()
    view = flat[first:first + 5 * stride + V].as_strided((6, V), (stride, 1))
    view.copy_(torch.from_numpy(x))
    check(torch, x, top=8, dev=view)


def test_equal_calls_streams_and_graphs(torch):
    from quantized_transformer_decode_gb300 import qw3
    x = torch.from_numpy(rows(40, 33333)).cuda()
    t = torch.arange(40, dtype=torch.int32, device="cuda")
    first = qw3.logprobs(x, t, top=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [qw3.logprobs(x, t, top=9) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = qw3.logprobs(x, t, top=9)
    g.replay()
    for other in again + [held]:
        for a, b in zip(first, other):
            assert torch.equal(a, b)
    x.copy_(torch.from_numpy(rows(40, 33333, 8)))
    g.replay()
    for a, b in zip(qw3.logprobs(x, t, top=9), held):
        assert torch.equal(a, b)


def test_refusals(torch):
    from quantized_transformer_decode_gb300 import qw3
    x, t = torch.zeros((3, 10), device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    for call in (lambda: qw3.logprobs(x.double(), t), lambda: qw3.logprobs(x.cpu(), t), lambda: qw3.logprobs(x, t.long()),
                 lambda: qw3.logprobs(x, t[:2]), lambda: qw3.logprobs(x, t.cpu()), lambda: qw3.logprobs(x, t, top=65),
                 lambda: qw3.logprobs(x, t, top=-1), lambda: qw3.logprobs(x[0], t), lambda: qw3.logprobs(x.t(), t),
                 lambda: qw3.logprobs(x[:, :0], t), lambda: qw3.logprobs(x, t.view(3, 1, 1))):
        with pytest.raises(qw3.Qw3Error):
            call()


@pytest.mark.parametrize("top", [1, 5, 64])
@pytest.mark.parametrize("first", [0, 1, 2, 3])
@pytest.mark.parametrize("B,V", [(1, 50257), (2, 50258), (3, 50259), (300, 9001), (301, 9002), (302, 9003)])
def test_equal_logits_at_a_rows_end(torch, B, V, first, top):
    """The last of the alternatives is one of several equal logits, the row's last three among them: the lowest index, in
    one CTA to a row and in several, wherever the row begins in a 16-byte word."""
    g = np.random.default_rng(B + first)
    x = np.full((B, V), -9.0) - g.random((B, V))
    for i, r in enumerate(x):
        # (behind what a CTA reads at first, and, with several of them to a row, within the first one's slice)
        inner = g.choice(np.arange(4200, min(V - 3, 6200)), 3 + i % 2, replace=False)
        r[[1, 700, 4199]] = 7.0, 6.5, 6.0
        r[g.choice(np.arange(2000, 4000), 80, replace=False)[:max(0, top - 4)]] = 6.25
        r[inner] = 5.0
        r[V - 3 + i % 3:] = 5.0
    if top == 1:
        x[:, [1, 700, 4199]] = -9.0
    x = x.astype(np.float32)
    wide = torch.full((B + 1, V + 1), float("nan"), device="cuda")
    view = wide.flatten()[first:first + B * (V + 1)].as_strided((B, V), (V + 1, 1))   # (each row begins 4 bytes further in a word)
    view.copy_(torch.from_numpy(x))
    check(torch, x, tokens=np.full((B, 1), V - 1, np.int32), top=top, dev=view)


@pytest.mark.parametrize("B,V", [(1, 151937), (1, 30003), (300, 20002)])
def test_ties_of_coarse_logits(torch, B, V):
    """Logits in steps of 1/4, as from a narrower type: every place of the list is tied; and rising ones, whose list overflows,
    with the row's end as large as the ones before it."""
    x = np.round(rows(B, V, V) * 4) / 4
    x[:, -2:] = np.sort(x, -1)[:, -20:-19]
    check(torch, x, top=20)
    x = np.tile(np.arange(V) // 50 * 0.01, (B, 1)).astype(np.float32)
    x[:, -1] = x[:, -70]
    check(torch, x, tokens=np.full((B, 1), V - 1, np.int32), top=64)


@pytest.mark.parametrize("B", [1, 512])
def test_rows_that_rise_take_a_few_readings(torch, B):
    """A row in which every logit is larger than the ones before overflows the list of alternatives: its slice is read once or
    twice more, not until the list fits by itself. (Half a row rises: the list is full either way.)"""
    from quantized_transformer_decode_gb300 import qw3
    V = 151936
    rising = torch.arange(V, device="cuda") * 1e-3
    half = torch.cat((rising[:V // 2], -rising[V // 2:]))
    g = torch.Generator(device="cuda").manual_seed(1)
    usual = torch.randn(V, generator=g, device="cuda") * 3
    tokens = torch.zeros(B, dtype=torch.int32, device="cuda")
    took = []
    for row in (usual, rising, half):
        x = row.repeat(B, 1)
        for top in (5, 64):
            _, _, ids, _ = qw3.logprobs(x, tokens, top=top)
            want = torch.sort(row, descending=True, stable=True).indices[:top].int()
            assert (ids == want).all()
        best = 1e9
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            qw3.logprobs(x, tokens, top=20)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        took.append(best)
    # (three readings where one is usual, a place in the list asked for by every logit, and what a list of 2048 costs to put in
    # order: 5 to 7 times as long; seventy readings are 300 times)
    assert max(took[1:]) < 20 * took[0], took
